// mo_expert_matmul: y[r] = x[r] w[e]^T over the rows of every expert.
#include "experts_host.h"

using namespace mo;

extern "C" int32_t mo_expert_matmul(const void* x, int64_t ldx, const void* w, const int32_t* offsets,
                                    int32_t experts, int64_t n, int64_t k, int64_t m, int32_t dtype,
                                    int32_t out_dtype, void* y, void* stream) {
  return entry([&]() -> int32_t {
    MO_TRY(check_expert("x", x, ldx, k, "w", w, k, k, offsets, experts, n, k, m, dtype, out_dtype, y));
    if (n == 0) return MO_OK;
    const int64_t es = static_cast<int64_t>(dtype_size(dtype)), eo = static_cast<int64_t>(dtype_size(out_dtype));
    MO_TRY(check_result(y, n, m, out_dtype, byte_rows(x, n, k, ldx, es), byte_rows(w, experts * m, k, k, es),
                        offsets, experts));
    XCall c;
    c.a = {x, w, y, offsets, ldx, k, m, n, experts, static_cast<int32_t>(k), static_cast<int32_t>(m),
           aligned16(y) && m * eo % 16 == 0};
    c.dtype = dtype;
    c.out = out_dtype;
    c.p_direct = direct_rows(x, ldx, k, es);
    c.q_direct = direct_rows(w, k, k, es);
    return launch_expert<X_FWD>(PK_XMM, c, static_cast<hipStream_t>(stream));
  });
}
