// Host-side state that the library's translation units share: the thread's last
// error, argument helpers, the launch helper and the records of per-kernel timing.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/matopt.h"

namespace mo {

inline thread_local std::string g_err;

inline int fail(int code, const std::string& msg) {
  g_err = msg;
  return code;
}

constexpr size_t ALIGN = 256;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
inline int64_t cdiv(int64_t v, int64_t a) { return (v + a - 1) / a; }
inline size_t dtype_size(int dt) { return dt == MO_F32 ? 4 : 2; }
inline bool valid_dtype(int dt) { return dt == MO_F32 || dt == MO_BF16; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// `rows` rows of `width` bytes, `pitch` bytes apart.
struct ByteRows {
  const void* p;
  int64_t rows, width;
  __int128 pitch;   // any pitch in elements fits
};
// Whether two of them share memory.  Columns of one buffer side by side do not.
inline bool overlap(const ByteRows& a, const ByteRows& b) {
  if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  auto first = [](const ByteRows& r) { return static_cast<__int128>(reinterpret_cast<uintptr_t>(r.p)); };
  auto end = [&](const ByteRows& r) { return first(r) + (r.rows - 1) * r.pitch + r.width; };
  if (end(a) <= first(b) || end(b) <= first(a)) return false;
  if (a.pitch != b.pitch) return true;
  const __int128 apart = ((first(b) - first(a)) % a.pitch + a.pitch) % a.pitch;
  return apart < a.width || apart + b.width > a.pitch;
}

// A call's result and its inputs: kernels read an input while other blocks store.
inline int check_apart(const char* what, const ByteRows& out, std::initializer_list<ByteRows> inputs) {
  for (const ByteRows& in : inputs)
    if (overlap(out, in)) return fail(MO_ERR_INVALID, std::string(what) + " must not overlap an input");
  return MO_OK;
}
inline ByteRows byte_rows(const void* p, int64_t rows, int64_t width, int64_t pitch, int64_t es) {
  return {p, rows, width * es, static_cast<__int128>(pitch) * es};
}

// ---- optional per-kernel timing ------------------------------------------------
struct ProfRec {
  int kind;
  hipEvent_t e0, e1;
};
// Profiling state is shared by every thread that calls the library; g_prof_mu guards
// the record list and the event pool.
inline std::atomic<bool> g_prof{false};
inline std::mutex g_prof_mu;
inline std::vector<ProfRec> g_prof_recs;
inline std::vector<hipEvent_t> g_ev_pool;
enum { PK_MOM = 0, PK_SCALE, PK_PREP, PK_COPY, PK_SYRK, PK_POLY, PK_APPLY, PK_PACK, PK_VOTE, PK_UNPACK,
       PK_SAPPLY, PK_MOMPREP, PK_GROUP, PK_LOOKUP, PK_EGRAD, PK_XMM, PK_XDX, PK_XDW, PK_DISTILL, PK_N };

// (g_prof_mu held)
inline hipEvent_t take_event() {
  if (!g_ev_pool.empty()) {
    hipEvent_t e = g_ev_pool.back();
    g_ev_pool.pop_back();
    return e;
  }
  hipEvent_t e = nullptr;
  (void)hipEventCreate(&e);
  return e;
}

// Launch helper: optional event bracket + launch error check.
// Set for the duration of an allocation-free call: its launches record no profiling
// events (creating one may allocate).
inline thread_local bool g_no_events = false;

template <typename F>
int launch(int pk, hipStream_t stream, F&& f) {
  ProfRec rec{pk, nullptr, nullptr};
  const bool prof = g_prof.load() && !g_no_events;
  if (prof) {
    std::lock_guard<std::mutex> lock(g_prof_mu);
    rec.e0 = take_event();
    rec.e1 = take_event();
  }
  if (rec.e0) (void)hipEventRecord(rec.e0, stream);
  f();
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(MO_ERR_HIP, std::string("kernel launch failed: ") + hipGetErrorString(err));
  if (rec.e0 && rec.e1 && hipEventRecord(rec.e1, stream) == hipSuccess) {
    std::lock_guard<std::mutex> lock(g_prof_mu);
    g_prof_recs.push_back(rec);
  }
  return MO_OK;
}

// Most blocks of 256 threads of one launch (see launch_blocks).
constexpr int64_t MAX_BLOCKS_256 = (int64_t(1) << 24) - 1;

// `blocks` blocks of `threads` threads as launches that the device can hold: a grid of 2^32
// threads or more wraps, without an error.  f(first block, blocks of this launch).
template <typename F>
int launch_blocks(int pk, hipStream_t stream, int64_t blocks, int64_t threads, F&& f) {
  const int64_t most = (int64_t(1) << 31) / threads;
  for (int64_t first = 0; first < blocks; first += most) {
    const int64_t count = blocks - first < most ? blocks - first : most;
    const int rc = launch(pk, stream, [&] { f(first, static_cast<uint32_t>(count)); });
    if (rc != MO_OK) return rc;
  }
  return MO_OK;
}

#define MO_TRY(x)            \
  do {                       \
    int rc_ = (x);           \
    if (rc_ != MO_OK) return rc_; \
  } while (0)

// Runs a C entry's body; a C++ exception (an allocation that failed) becomes a code.
template <typename F>
int32_t entry(F&& body) noexcept {
  try {
    g_err.clear();
    return body();
  } catch (...) {
    return MO_ERR_HIP;
  }
}

// Compute units of the current device (8 if it cannot be asked).
inline int device_cus() {
  static std::atomic<int> cus[64];   // per device, 0 until first asked
  int dev = 0;
  (void)hipGetDevice(&dev);
  int n = (dev >= 0 && dev < 64) ? cus[dev].load() : 0;
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 8;
    if (dev >= 0 && dev < 64) cus[dev].store(n);
  }
  return n;
}

}  // namespace mo
