// Dense product of e4m3 operands with block scales and a 16-bit y (fp8_dev.h).
#include "fp8_dev.h"

namespace pw {

hipError_t launch_linear_fp8(const ProductArgs& a, hipStream_t s) {
    if (a.out_dtype == PW_F32) return launch_linear_fp8_full(a, s);
    return a.act == PW_ACT_SWIGLU ? launch_fp8_t<E4M3, true>(a, s) : launch_fp8_t<E4M3, false>(a, s);
}

}  // namespace pw
