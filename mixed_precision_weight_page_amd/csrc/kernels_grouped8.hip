// Products of e4m3 operands grouped by expert, with a 16-bit y (product_dev.h).
#include "product_dev.h"

namespace pw {

hipError_t launch_grouped_fp8(const ProductArgs& a, hipStream_t s) {
    if (a.out_dtype == PW_F32) return launch_grouped_fp8_full(a, s);
    return a.act == PW_ACT_SWIGLU ? launch_grouped_any_size<E4M3, true>(a, s) : launch_grouped_any_size<E4M3, false>(a, s);
}

}  // namespace pw
