// Host side of the distillation loss: mo_distill_forward, mo_distill_backward,
// mo_distill_forward_backward.
#include "distill.h"

#include <algorithm>
#include <cmath>

#include "host.h"

using namespace mo;

namespace {

int check_distill(const void* logits, int64_t ldx, const void* ids, int32_t id_bytes, const float* teacher,
                  int64_t n, int64_t vocab, int64_t k, int32_t dtype, float temperature) {
  if (!valid_dtype(dtype)) return fail(MO_ERR_UNSUPPORTED, "dtype must be MO_F32 or MO_BF16");
  if (id_bytes != 4 && id_bytes != 8) return fail(MO_ERR_UNSUPPORTED, "indices must be 4- or 8-byte integers");
  if (n < 0 || n > 0x7fffffffLL) return fail(MO_ERR_INVALID, "n must be in [0, 2^31)");
  if (vocab < 1 || vocab > (int64_t(1) << 28)) return fail(MO_ERR_INVALID, "vocab must be in [1, 2^28]");
  if (k < 1 || k > DISTILL_MAX_K)
    return fail(MO_ERR_INVALID, "teacher entries per row must be in [1, " + std::to_string(DISTILL_MAX_K) + "]");
  // below, 1 / temperature overflows
  if (!std::isfinite(temperature) || temperature < 0x1p-126f)
    return fail(MO_ERR_INVALID, "temperature must be finite and at least 2^-126");
  if (ldx < vocab) return fail(MO_ERR_INVALID, "logits: the row pitch must be >= vocab");
  if (n > 0 && (!logits || !ids || !teacher)) return fail(MO_ERR_INVALID, "logits, indices or teacher is NULL");
  return MO_OK;
}

int check_grad(const void* logits, int64_t ldx, const void* grad, int64_t ldg, int64_t n, int64_t vocab,
               int32_t dtype) {
  const int64_t es = static_cast<int64_t>(dtype_size(dtype));
  if (overlap(byte_rows(logits, n, vocab, ldx, es), byte_rows(grad, n, vocab, ldg, es)))
    return fail(MO_ERR_INVALID, "grad must not be logits, nor overlap them");
  return MO_OK;
}

template <typename T, int MODE>
int run_rows(const DistillArgs& a, hipStream_t stream) {
  const int64_t pieces = a.V / RowVec<T>::N;
#define MO_ROWS(NT, NR, NL)                                                                                     \
  return launch_blocks(PK_DISTILL, stream, a.n, NT, [&](int64_t first, uint32_t count) {                         \
    DistillArgs b = a;                                                                                          \
    b.first_row = first;                                                                                        \
    hipLaunchKernelGGL((k_distill<T, MODE, NT, NR, NL>), dim3(count), dim3(NT), teacher_bytes(a.k), stream, b); \
  })
  // A row over threads that hold 4 to 16 pieces each: many waves with few registers
  // overlap their loads and exponentials best, idle pieces cost their share.  8192 rows of
  // 32768 bf16 logits, loss and gradient: 215 us with 512 threads, 232 with 256, 263 with
  // 1024; 6000 rows of 50257: 281 us with 13 pieces a thread, 298 with 16, 396 with 8 of
  // 1024 threads.  (With the difference from the maximum folded into one instruction; as it
  // is taken now, the first is 220.)
  if (pieces <= 64 * 4) MO_ROWS(64, 4, 0);
  if (pieces <= 128 * 8) MO_ROWS(128, 8, 0);
  if (pieces <= 256 * 8) MO_ROWS(256, 8, 0);
  if (pieces <= 512 * 6) MO_ROWS(512, 6, 0);
  if (pieces <= 512 * 8) MO_ROWS(512, 8, 0);
  if (pieces <= 512 * 13) MO_ROWS(512, 13, 0);
  if (pieces <= 512 * 16) MO_ROWS(512, 16, 0);
  if (pieces <= 512 * 32) MO_ROWS(512, 23, 9);
  MO_ROWS(512, 0, 0);
#undef MO_ROWS
}

template <typename T>
int run_backward(const DistillArgs& a, hipStream_t stream) {
  const int64_t per = 256 * 8;   // pieces a block
  const int64_t parts = cdiv(std::max<int64_t>(a.V / RowVec<T>::N, 1), per);
  constexpr int64_t MOST = 65535;   // rows of a grid
  for (int64_t first = 0; first < a.n; first += MOST) {
    DistillArgs b = a;
    b.first_row = first;
    MO_TRY(launch(PK_DISTILL, stream, [&] {
      hipLaunchKernelGGL((k_distill_backward<T, 256, 8>), dim3(parts, std::min(MOST, a.n - first)), dim3(256),
                         teacher_bytes(a.k), stream, b);
    }));
  }
  return MO_OK;
}

}  // namespace

extern "C" {

int32_t mo_distill_forward(const void* logits, int64_t ldx, const void* indices, int32_t index_bytes,
                           const float* teacher, int64_t n, int64_t vocab, int64_t k, int32_t dtype,
                           float temperature, float* loss, float* lse, void* stream) {
  return entry([&]() -> int32_t {
    MO_TRY(check_distill(logits, ldx, indices, index_bytes, teacher, n, vocab, k, dtype, temperature));
    if (n == 0) return MO_OK;
    if (!loss || !lse) return fail(MO_ERR_INVALID, "loss or lse is NULL");
    DistillArgs a = {logits, ldx, indices, teacher, vocab, n, static_cast<int>(k), index_bytes == 8, temperature,
                     nullptr, nullptr, loss, lse, nullptr, 0, 0};
    if (dtype == MO_F32) return run_rows<float, D_FWD>(a, static_cast<hipStream_t>(stream));
    return run_rows<bf16_t, D_FWD>(a, static_cast<hipStream_t>(stream));
  });
}

int32_t mo_distill_backward(const void* logits, int64_t ldx, const float* lse, const void* indices,
                            int32_t index_bytes, const float* teacher, const float* row_grad, int64_t n,
                            int64_t vocab, int64_t k, int32_t dtype, float temperature, void* grad, int64_t ldg,
                            void* stream) {
  return entry([&]() -> int32_t {
    MO_TRY(check_distill(logits, ldx, indices, index_bytes, teacher, n, vocab, k, dtype, temperature));
    if (ldg < vocab) return fail(MO_ERR_INVALID, "grad: the row pitch must be >= vocab");
    if (n == 0) return MO_OK;
    if (!lse || !row_grad || !grad) return fail(MO_ERR_INVALID, "lse, row_grad or grad is NULL");
    MO_TRY(check_grad(logits, ldx, grad, ldg, n, vocab, dtype));
    DistillArgs a = {logits, ldx, indices, teacher, vocab, n, static_cast<int>(k), index_bytes == 8, temperature,
                     row_grad, lse, nullptr, nullptr, grad, ldg, 0};
    if (dtype == MO_F32) return run_backward<float>(a, static_cast<hipStream_t>(stream));
    return run_backward<bf16_t>(a, static_cast<hipStream_t>(stream));
  });
}

int32_t mo_distill_forward_backward(const void* logits, int64_t ldx, const void* indices, int32_t index_bytes,
                                    const float* teacher, const float* row_grad, int64_t n, int64_t vocab,
                                    int64_t k, int32_t dtype, float temperature, float* loss, float* lse, void* grad,
                                    int64_t ldg, void* stream) {
  return entry([&]() -> int32_t {
    MO_TRY(check_distill(logits, ldx, indices, index_bytes, teacher, n, vocab, k, dtype, temperature));
    if (ldg < vocab) return fail(MO_ERR_INVALID, "grad: the row pitch must be >= vocab");
    if (n == 0) return MO_OK;
    if (!loss || !lse || !row_grad || !grad) return fail(MO_ERR_INVALID, "loss, lse, row_grad or grad is NULL");
    MO_TRY(check_grad(logits, ldx, grad, ldg, n, vocab, dtype));
    DistillArgs a = {logits, ldx, indices, teacher, vocab, n, static_cast<int>(k), index_bytes == 8, temperature,
                     row_grad, nullptr, loss, lse, grad, ldg, 0};
    if (dtype == MO_F32) return run_rows<float, D_BOTH>(a, static_cast<hipStream_t>(stream));
    return run_rows<bf16_t, D_BOTH>(a, static_cast<hipStream_t>(stream));
  });
}

}  // extern "C"
