// mo_expert_input_grad: dx[r] = dy[r] w[e] over the rows of every expert.
#include "experts_host.h"

using namespace mo;

extern "C" int32_t mo_expert_input_grad(const void* dy, int64_t lddy, const void* w, const int32_t* offsets,
                                        int32_t experts, int64_t n, int64_t k, int64_t m, int32_t dtype,
                                        int32_t out_dtype, void* dx, void* stream) {
  return entry([&]() -> int32_t {
    MO_TRY(check_expert("dy", dy, lddy, m, "w", w, k, k, offsets, experts, n, k, m, dtype, out_dtype, dx));
    if (n == 0) return MO_OK;
    const int64_t es = static_cast<int64_t>(dtype_size(dtype)), eo = static_cast<int64_t>(dtype_size(out_dtype));
    MO_TRY(check_result(dx, n, k, out_dtype, byte_rows(dy, n, m, lddy, es), byte_rows(w, experts * m, k, k, es),
                        offsets, experts));
    XCall c;
    c.a = {dy, w, dx, offsets, lddy, k, k, n, experts, static_cast<int32_t>(k), static_cast<int32_t>(m),
           aligned16(dx) && k * eo % 16 == 0};
    c.dtype = dtype;
    c.out = out_dtype;
    c.p_direct = direct_rows(dy, lddy, m, es);
    c.q_direct = direct_rows(w, k, k, es);
    return launch_expert<X_DX>(PK_XDX, c, static_cast<hipStream_t>(stream));
  });
}
