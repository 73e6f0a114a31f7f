// The loss against a teacher's top logits, with its gradient.
//
// For a row of logits x (V of them), temperature tau, and up to K teacher entries
// (id_j, t_j), entries with an id outside [0, V) left out:
//   q = softmax(x / tau),  p = softmax(t / tau) over the row's entries
//   loss = tau^2 sum_j p_j (log p_j - log q[id_j])
//   dx   = row_grad * tau * (q - p),  p = 0 away from the entries
// With z = (x - max x) / tau, s = sum exp z, u_j = (t_j - max t) / tau, e_j = exp u_j and
// S = sum e_j:
//   loss = tau^2 (sum_j e_j (u_j - z[id_j]) / S + log s - log S),
// differences from the maxima only, so nothing large cancels.  A row without entries
// (or whose entries are all -inf) has loss 0 and gradient 0; lse is given all the same.
// All sums are fp32; the gradient is rounded once, to the logits' type.
//
// One block takes one row (the backward pass: one part of a row).  The forward pass
// and the pass that does both read the row once when it fits the registers of 64 to 512
// threads (up to 64 of each), or, up to 256 KiB, those and LDS; longer rows are read twice.
// Bound by HBM: 4096 rows of 131072 bf16 logits, loss and gradient, 421 us, 5.1 TB/s, more
// than a copy's 4.8 (a kernel that read every row twice: 1154 us).  The forward pass alone,
// 8192 rows of 32768: 95 us, 5.7 TB/s.  2051 such rows, which are two rounds of blocks and
// three rows, take 95 us for the two calls, 4.3 TB/s.  Beyond 256 KiB the loss alone is still
// read once, 2048 rows of 151936 bf16 logits 106 us, 5.9 TB/s; with the gradient 352 us, 3.5
// TB/s of what it cannot do without (1024 rows of 131072 fp32 logits: 293 us, 3.7 TB/s).
#pragma once

#include <type_traits>

#include "common.h"

// fused only where written: the forward pass and the pass that does both then round alike
#pragma clang fp contract(off)

namespace mo {

constexpr int DISTILL_MAX_K = 1024;

struct DistillArgs {
  const void* x;        // n x V logits
  int64_t ldx;
  const void* ids;      // n x k int32 or int64
  const float* t;       // n x k teacher logits
  int64_t V, n;
  int k, ids64;
  float tau;
  const float* row_grad;
  const float* lse_in;  // the backward pass
  float* loss;
  float* lse;
  void* grad;           // n x V, pitch ldg
  int64_t ldg;
  int64_t first_row;    // of this launch
};

__device__ inline float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
constexpr float LOG2E = 1.44269504088896340736f;

template <typename T> struct RowVec;
template <> struct RowVec<bf16_t> { static constexpr int N = 8; };
template <> struct RowVec<float> { static constexpr int N = 4; };

// the sum and the maximum over a block of NT threads of four values each thread
template <int NT, typename OP>
__device__ inline float wave_all(float v, OP op) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = op(v, __shfl_xor(v, d));
  return v;
}
struct OpMax {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct OpSum {
  __device__ float operator()(float a, float b) const { return a + b; }
};
template <int NT, typename OP>
__device__ inline void block_all(float* v, int count, float (*scratch)[16], OP op) {
  for (int i = 0; i < count; ++i) v[i] = wave_all<NT>(v[i], op);
  if (NT == 64) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();   // an earlier use of scratch is over
  if (lane == 0)
    for (int i = 0; i < count; ++i) scratch[i][wave] = v[i];
  __syncthreads();
  for (int i = 0; i < count; ++i) {
    float r = scratch[i][0];
    for (int w = 1; w < NT / 64; ++w) r = op(r, scratch[i][w]);
    v[i] = r;
  }
}

struct __attribute__((packed, aligned(2))) Row16x2 { u32x4_t v; };
struct __attribute__((packed, aligned(4))) Row16x4 { u32x4_t v; };
template <typename T> struct RowLoose { typedef Row16x4 type; };
template <> struct RowLoose<bf16_t> { typedef Row16x2 type; };

// A row of V logits as F whole 16-byte pieces and up to N - 1 single elements behind
// them.  A row may start at any element, so the pieces are loaded and stored with the
// element's alignment only.
template <typename T>
struct Row {
  static constexpr int N = RowVec<T>::N;
  const T* p;
  uint32_t F, rest;
  __device__ Row(const T* row, int64_t V)
      : p(row), F(static_cast<uint32_t>(V / N)), rest(static_cast<uint32_t>(V % N)) {}
  // piece i < F; beyond, the last one (no lane branches), which fix() then makes -inf:
  // that adds nothing to a softmax.  F > 0.
  __device__ inline u32x4_t load(uint32_t i) const {
    const uint32_t at = i < F ? i : F - 1;
    // a uniform base and a 32-bit offset (rows stay below 2^30 bytes)
    typedef __attribute__((address_space(1))) const unsigned char* bytes_t;
    return reinterpret_cast<gptr<const typename RowLoose<T>::type>>((bytes_t)p + at * 16u)->v;
  }
  // `end`: the first piece index that no thread's load of this round reaches (uniform)
  __device__ inline void fix(u32x4_t& v, uint32_t i, uint32_t end) const {
    if (end <= F) return;
    constexpr uint32_t NI = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i < F ? v[k] : NI;
  }
  // the element behind the pieces that thread t holds, -inf if none
  __device__ inline float load_rest(uint32_t t) const {
    return t < rest ? to_f32(global(p)[static_cast<int64_t>(F) * N + t]) : -__builtin_inff();
  }
};

template <typename T>
__device__ inline void unpack(u32x4_t p, float (&f)[RowVec<T>::N]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __builtin_bit_cast(float, p[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, p[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = p[i];   // a value: a bit cast of a vector's element takes element 0
      f[i] = __builtin_bit_cast(float, w);
    }
  }
}
template <typename T>
__device__ inline void store_piece(T* row, uint32_t i, const float (&f)[RowVec<T>::N]) {
  constexpr int N = RowVec<T>::N;
  typedef T vt __attribute__((ext_vector_type(N)));
  vt v;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = from_f32<T>(f[k]);
  typedef __attribute__((address_space(1))) unsigned char* bytes_t;
  reinterpret_cast<gptr<typename RowLoose<T>::type>>((bytes_t)row + i * 16u)->v = __builtin_bit_cast(u32x4_t, v);
}

__device__ inline int64_t teacher_id(const DistillArgs& a, int64_t at) {
  const int64_t id = a.ids64 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
  return (id >= 0 && id < a.V) ? id : -1;
}

// A row's teacher entries in LDS (dynamic, 8 bytes an entry): ids (-1: left out) and
// values, padded to a multiple of four so that they can be read four at a time.
struct Teacher {
  int32_t* id;
  float* e;
  __device__ Teacher(unsigned char* lds, int k)
      : id(reinterpret_cast<int32_t*>(lds)), e(reinterpret_cast<float*>(lds) + ((k + 3) & ~3)) {}
};
__host__ __device__ inline uint32_t teacher_bytes(int k) { return 8u * ((k + 3) & ~3); }
typedef int32_t i32x4v_t __attribute__((ext_vector_type(4)));

template <int NT>
__device__ inline float load_teacher(const DistillArgs& a, int64_t r, const Teacher& s) {
  float tm = -__builtin_inff();
  for (int j = threadIdx.x; j < ((a.k + 3) & ~3); j += NT) {
    const int64_t id = j < a.k ? teacher_id(a, r * a.k + j) : -1;
    const float t = j < a.k ? a.t[r * a.k + j] : 0.f;
    s.id[j] = static_cast<int32_t>(id);
    s.e[j] = t;
    if (id >= 0) tm = fmaxf(tm, t);
  }
  return tm;
}
// For the JS entries with these ids: the values of all entries with the same id, added in
// the entries' order.
template <int JS>
__device__ inline void same_ids(const Teacher& s, int k, const int32_t (&id)[JS], float (&p)[JS]) {
#pragma unroll
  for (int j = 0; j < JS; ++j) p[j] = 0.f;
  for (int i = 0; i < k; i += 4) {
    const i32x4v_t d = *reinterpret_cast<const i32x4v_t*>(&s.id[i]);
    const f32x4_t e = *reinterpret_cast<const f32x4_t*>(&s.e[i]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < JS; ++j) p[j] += d[u] == id[j] ? e[u] : 0.f;
  }
}
// f(id, its entries' sum) for every entry whose id lies in [lo, hi): each thread its own.
// Where a thread has several, four share a pass over the entries (61 rows with 206
// entries, 64 threads: 11 us instead of 17; with one of each thread's four in use the
// other three cost 4% of a call).
template <int NT, typename F>
__device__ inline void each_entry(const Teacher& s, int k, uint32_t lo, uint32_t hi, F&& f) {
  auto pass = [&](auto js) {
    constexpr int JS = decltype(js)::value;
    for (int j0 = threadIdx.x; j0 < k; j0 += JS * NT) {
      int32_t id[JS];
      float p[JS];
      bool any = false;
#pragma unroll
      for (int u = 0; u < JS; ++u) {
        id[u] = j0 + u * NT < k ? s.id[j0 + u * NT] : -1;
        if (id[u] < 0 || static_cast<uint32_t>(id[u]) < lo || static_cast<uint32_t>(id[u]) >= hi) id[u] = -1;
        any |= id[u] >= 0;
      }
      if (!any) continue;
      same_ids<JS>(s, k, id, p);
#pragma unroll
      for (int u = 0; u < JS; ++u)
        if (id[u] >= 0) f(id[u], p[u]);
    }
  };
  if (k <= NT) pass(std::integral_constant<int, 1>{});
  else pass(std::integral_constant<int, 4>{});
}

// exp((x - shift) / tau).  The difference is taken first, so it is exact near the maximum
// whatever the logits' common offset.  (As x * c - shift * c in one instruction, what the two
// products' roundings leave grows with the offset: in a row of -1e9 a factor of 2^18.)
struct Exponent {
  float shift, c;
  __device__ Exponent(float at, float inv_tau) : shift(at), c(LOG2E * inv_tau) {}
  __device__ inline float operator()(float x) const { return fast_exp2((x - shift) * c); }
};

enum DistillMode { D_FWD = 0, D_BOTH = 1 };

// The row stays in NR pieces of registers and NL pieces of LDS per thread; with NR == 0
// it is read twice, 8 pieces of every thread at a time.
template <typename T, int MODE, int NT, int NR, int NL>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(NT == 512 ? 4 : 1)))
void k_distill(DistillArgs a) {
  constexpr int N = RowVec<T>::N;
  constexpr bool HOLD = NR > 0;
  constexpr int NB = HOLD ? NR : 8;
  __shared__ float scratch[4][16];
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn[];
  const Teacher te(dyn, a.k);
  __shared__ __attribute__((aligned(16))) u32x4_t more[NL > 0 ? NL : 1][NL > 0 ? NT : 1];
  const uint32_t tid = threadIdx.x;
  const int64_t r = a.first_row + blockIdx.x;
  const Row<T> row(static_cast<const T*>(a.x) + r * a.ldx, a.V);
  const float inv_tau = 1.f / a.tau;
  constexpr float NINF = -__builtin_inff();

  u32x4_t held[NB];
  float m2[2] = {NINF, NINF};   // maxima of the logits and of the teacher's
  float s_run = 0.f;            // !HOLD: this thread's sum, relative to its own maximum
  const float xr = row.load_rest(tid);
  auto max_of = [&](u32x4_t v) {
    float f[N];
    unpack<T>(v, f);
#pragma unroll
    for (int i = 0; i < N; ++i) m2[0] = fmaxf(m2[0], f[i]);
    if constexpr (HOLD) __builtin_amdgcn_sched_barrier(0);
  };
  if (HOLD && row.F > 0) {
    if constexpr (NL > 0) {
      // through the registers of the pieces that follow
#pragma unroll
      for (int q = 0; q < NL; ++q) held[q] = row.load((NR + q) * NT + tid);
#pragma unroll
      for (int q = 0; q < NL; ++q) {
        row.fix(held[q], (NR + q) * NT + tid, (NR + q + 1) * NT);
        max_of(held[q]);
        more[q][tid] = held[q];
      }
    }
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      held[q] = row.load(q * NT + tid);
      __builtin_amdgcn_sched_barrier(0);   // one offset at a time
    }
  }
  m2[1] = load_teacher<NT>(a, r, te);
  m2[0] = fmaxf(m2[0], xr);
  if (row.F > 0) {
    if constexpr (HOLD) {
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        row.fix(held[q], q * NT + tid, (q + 1) * NT);
        max_of(held[q]);
      }
    } else {
      const float c2 = LOG2E * inv_tau;
      s_run = xr == NINF ? 0.f : 1.f;
      for (uint32_t c0 = 0; c0 < row.F; c0 += NB * NT) {
#pragma unroll
        for (int q = 0; q < NB; ++q) held[q] = row.load(c0 + q * NT + tid);
#pragma unroll
        for (int q = 0; q < NB; ++q) row.fix(held[q], c0 + q * NT + tid, c0 + (q + 1) * NT);
        const float before = m2[0];
#pragma unroll
        for (int q = 0; q < NB; ++q) max_of(held[q]);
        const float ms = m2[0] == NINF ? 0.f : m2[0];
        s_run *= fast_exp2((before - ms) * c2);
#pragma unroll
        for (int q = 0; q < NB; ++q) {
          float f[N];
          unpack<T>(held[q], f);
#pragma unroll
          for (int i = 0; i < N; ++i) s_run += fast_exp2((f[i] - ms) * c2);
        }
      }
    }
  }
  const float own_max = m2[0];
  block_all<NT>(m2, 2, scratch, OpMax());
  const float xm = m2[0] == NINF ? 0.f : m2[0], tmax = m2[1] == NINF ? 0.f : m2[1];
  const Exponent ex(xm, inv_tau);
  // the pieces as they were loaded: without this the compiler keeps the unpacked values
  // of one pass for the next, which do not fit the registers
  auto repack = [&]() {
    if constexpr (HOLD)
#pragma unroll
      for (int q = 0; q < NB; ++q) asm volatile("" : "+v"(held[q]));
  };
  repack();

  // sums: exp z; e_j; tau e_j (u_j - z_j)
  float s3[3] = {0.f, 0.f, 0.f};
  if constexpr (HOLD) {
    s3[0] = ex(xr);
    auto add = [&](u32x4_t v) {
      float f[N];
      unpack<T>(v, f);
#pragma unroll
      for (int i = 0; i < N; ++i) s3[0] += ex(f[i]);
      __builtin_amdgcn_sched_barrier(0);   // one piece after another: few values unpacked at a time
    };
    if (row.F > 0) {
#pragma unroll
      for (int q = 0; q < NR; ++q) add(held[q]);
      if constexpr (NL > 0)
#pragma unroll
        for (int q = 0; q < NL; ++q) add(more[q][tid]);
    }
  } else {
    // own_max - xm may be far below; a thread without logits has the sum 0
    s3[0] = s_run == 0.f ? 0.f : s_run * fast_exp2(((own_max == NINF ? 0.f : own_max) - xm) * (LOG2E * inv_tau));
  }
  for (int j = tid; j < ((a.k + 3) & ~3); j += NT) {
    const int32_t id = te.id[j];
    float e = 0.f;
    if (id >= 0) {
      const float d = te.e[j] - tmax;
      e = fast_exp2(d * (LOG2E * inv_tau));
      // tau e_j (u_j - z_j).  2^-12: up to 1024 terms of the largest size (logits of the
      // type's lowest value and of its highest) stay finite; the power of two is exact
      if (e != 0.f) s3[2] += e * (d * 0x1p-12f - (to_f32(row.p[id]) * 0x1p-12f - xm * 0x1p-12f));
    }
    s3[1] += e;
    te.e[j] = e;
  }
  block_all<NT>(s3, 3, scratch, OpSum());
  const float S = s3[1];
  const bool live = S != 0.f;      // also where it is NaN
  const float log_s = logf(s3[0]);
  if (tid == 0) {
    a.lse[r] = xm * inv_tau + log_s;
    // in an order in which nothing passes fp32's ends that does not in the end
    const float t12 = s3[2] / S, first = a.tau < 1.f ? t12 * (a.tau * 0x1p12f) : t12 * 0x1p12f * a.tau;
    a.loss[r] = live ? first + a.tau * (a.tau * (log_s - logf(S))) : 0.f;
  }
  if constexpr (MODE == D_BOTH) {
    repack();
    const float g = live ? a.tau * a.row_grad[r] : 0.f;
    const float gq = live ? g / s3[0] : 0.f, gp = live ? g / S : 0.f;
    T* out = static_cast<T*>(a.grad) + r * a.ldg;
    auto put = [&](u32x4_t v, uint32_t i) {
      float f[N];
      unpack<T>(v, f);
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = ex(f[k]) * gq;
      if (i < row.F) store_piece(out, i, f);
      __builtin_amdgcn_sched_barrier(0);
    };
    if (!live) {
      const float z[N] = {};
      for (uint32_t i = tid; i < row.F; i += NT) store_piece(out, i, z);
      if (tid < row.rest) out[static_cast<int64_t>(row.F) * N + tid] = from_f32<T>(0.f);
      return;
    }
    if (tid < row.rest) out[static_cast<int64_t>(row.F) * N + tid] = from_f32<T>(ex(xr) * gq);
    if (row.F > 0) {
      if constexpr (HOLD) {
#pragma unroll
        for (int q = 0; q < NR; ++q) put(held[q], q * NT + tid);
        if constexpr (NL > 0)
#pragma unroll
          for (int q = 0; q < NL; ++q) put(more[q][tid], (NR + q) * NT + tid);
      } else {
        for (uint32_t i0 = tid; i0 < row.F; i0 += NB * NT) {
#pragma unroll
          for (int q = 0; q < NB; ++q) held[q] = row.load(i0 + q * NT);
#pragma unroll
          for (int q = 0; q < NB; ++q) put(held[q], i0 + q * NT);
        }
      }
    }
    __syncthreads();   // the row is stored; the teacher's entries overwrite theirs
    each_entry<NT>(te, a.k, 0, static_cast<uint32_t>(a.V), [&](int32_t id, float p) {
      out[id] = from_f32<T>(ex(to_f32(row.p[id])) * gq - p * gp);
    });
  }
}

// A row's maximum (0 for a row of -inf) and sum of exponentials, by a block that holds
// nothing of it.
template <typename T, int NT>
__device__ inline void row_sum(const Row<T>& row, float inv_tau, float (*scratch)[16], float& m, float& sum) {
  constexpr int N = RowVec<T>::N;
  const uint32_t tid = threadIdx.x;
  const float xr = row.load_rest(tid);
  float v[1] = {xr};
  for (uint32_t i = tid; i < row.F; i += NT) {
    float f[N];
    unpack<T>(row.load(i), f);
#pragma unroll
    for (int k = 0; k < N; ++k) v[0] = fmaxf(v[0], f[k]);
  }
  block_all<NT>(v, 1, scratch, OpMax());
  m = v[0] == -__builtin_inff() ? 0.f : v[0];
  const Exponent ex(m, inv_tau);
  v[0] = ex(xr);
  for (uint32_t i = tid; i < row.F; i += NT) {
    float f[N];
    unpack<T>(row.load(i), f);
#pragma unroll
    for (int k = 0; k < N; ++k) v[0] += ex(f[k]);
  }
  block_all<NT>(v, 1, scratch, OpSum());
  sum = v[0];
}

// From this size on the pass from lse sums a row anew: half of fp32's step, the error of the
// exponent, is 2^-15 below, and at 1e7 a factor of 1.6.  Logits that large come from masks
// (-1e9, the type's lowest value) in rows that are masked whole, and from temperatures of
// 0.01.  Every part of such a row reads all of it: rows of 32768 bf16 logits take twice the
// time, rows of 131072 six times.
constexpr float LSE_FINE = 1024.f;

// The backward pass from the forward's lse: block (part, row) stores NT * NV pieces.
template <typename T, int NT, int NV>
__global__ __launch_bounds__(NT) void k_distill_backward(DistillArgs a) {
  constexpr int N = RowVec<T>::N;
  __shared__ float scratch[4][16];
  extern __shared__ __attribute__((aligned(16))) unsigned char dyn[];
  const Teacher te(dyn, a.k);
  const uint32_t tid = threadIdx.x;
  const int64_t r = a.first_row + blockIdx.y;
  const Row<T> row(static_cast<const T*>(a.x) + r * a.ldx, a.V);
  const uint32_t from = blockIdx.x * (NT * NV), to = min(row.F, from + NT * NV);
  const bool last = blockIdx.x + 1 == gridDim.x;   // also holds the elements behind the pieces
  T* out = static_cast<T*>(a.grad) + r * a.ldg;
  const float inv_tau = 1.f / a.tau;
  u32x4_t held[NV];
  if (row.F > 0)
#pragma unroll
    for (int q = 0; q < NV; ++q) held[q] = row.load(from + q * NT + tid);
  const float lse = a.lse_in[r];
  float tm[1] = {load_teacher<NT>(a, r, te)};
  block_all<NT>(tm, 1, scratch, OpMax());
  const float tmax = tm[0] == -__builtin_inff() ? 0.f : tm[0];
  float S[1] = {0.f};
  for (int j = tid; j < ((a.k + 3) & ~3); j += NT) {
    const float e = te.id[j] >= 0 ? fast_exp2((te.e[j] - tmax) * (LOG2E * inv_tau)) : 0.f;
    te.e[j] = e;
    S[0] += e;
  }
  block_all<NT>(S, 1, scratch, OpSum());
  const bool live = S[0] != 0.f;
  const float g = live ? a.tau * a.row_grad[r] : 0.f, gp = live ? g / S[0] : 0.f;
  // exp((x * by - at) * c) * gq: exp(x / tau - lse) * g; or, where fp32 holds lse too
  // coarsely, exp((x - max) / tau) * g / sum, from the row itself.
  float by = inv_tau, at = lse, c = LOG2E, gq = g;
  if (live && !(fabsf(lse) < LSE_FINE)) {
    float m, sum;
    row_sum<T, NT>(row, inv_tau, scratch, m, sum);
    by = 1.f;
    at = m;
    c = LOG2E * inv_tau;
    gq = g / sum;
  }
  auto q_of = [&](float x) { return live ? fast_exp2(__builtin_fmaf(x, by, -at) * c) * gq : 0.f; };
  if (row.F > 0)
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const uint32_t i = from + q * NT + tid;
      float f[N];
      unpack<T>(held[q], f);
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = q_of(f[k]);
      if (i < to) store_piece(out, i, f);
    }
  if (last && tid < row.rest) {
    const int64_t at = static_cast<int64_t>(row.F) * N + tid;
    out[at] = from_f32<T>(q_of(to_f32(row.p[at])));
  }
  if (!live) return;
  __syncthreads();
  const uint32_t lo = from * N, hi = last ? static_cast<uint32_t>(a.V) : to * N;
  each_entry<NT>(te, a.k, lo, hi, [&](int32_t id, float p) {
    out[id] = from_f32<T>(q_of(to_f32(row.p[id])) - p * gp);
  });
}

}  // namespace mo
