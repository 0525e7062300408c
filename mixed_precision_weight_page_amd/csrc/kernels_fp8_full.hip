// Dense product of e4m3 operands with block scales and an fp32 y (fp8_dev.h).
#include "fp8_dev.h"

namespace pw {

hipError_t launch_linear_fp8_full(const ProductArgs& a, hipStream_t s) {
    return a.act == PW_ACT_SWIGLU ? launch_fp8_t<E4M3Full, true>(a, s) : launch_fp8_t<E4M3Full, false>(a, s);
}

}  // namespace pw
