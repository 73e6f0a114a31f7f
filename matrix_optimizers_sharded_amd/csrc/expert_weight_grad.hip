// mo_expert_weight_grad: dw[e] = dy^T x over the rows of every expert.
#include "experts_host.h"

using namespace mo;

extern "C" int32_t mo_expert_weight_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                         const int32_t* offsets, int32_t experts, int64_t n, int64_t k, int64_t m,
                                         int32_t dtype, int32_t out_dtype, void* dw, void* stream) {
  return entry([&]() -> int32_t {
    MO_TRY(check_expert("dy", dy, lddy, m, "x", x, ldx, k, offsets, experts, n, k, m, dtype, out_dtype, dw));
    if (!dw) return fail(MO_ERR_INVALID, "the result is NULL");   // written whole, without rows too
    const int64_t es = static_cast<int64_t>(dtype_size(dtype)), eo = static_cast<int64_t>(dtype_size(out_dtype));
    MO_TRY(check_result(dw, experts * m, k, out_dtype, byte_rows(dy, n, m, lddy, es), byte_rows(x, n, k, ldx, es),
                        offsets, experts));
    XCall c;
    c.a = {dy, x, dw, offsets, lddy, ldx, k, n, experts, static_cast<int32_t>(k), static_cast<int32_t>(m),
           aligned16(dw) && k * eo % 16 == 0};
    c.dtype = dtype;
    c.out = out_dtype;
    c.p_direct = direct_rows(dy, lddy, m, es);
    c.q_direct = direct_rows(x, ldx, k, es);
    return launch_expert<X_DW>(PK_XDW, c, static_cast<hipStream_t>(stream));
  });
}
