// Products of e4m3 operands grouped by expert, with an fp32 y (product_dev.h).
#include "product_dev.h"

namespace pw {

hipError_t launch_grouped_fp8_full(const ProductArgs& a, hipStream_t s) {
    return a.act == PW_ACT_SWIGLU ? launch_grouped_any_size<E4M3Full, true>(a, s) : launch_grouped_any_size<E4M3Full, false>(a, s);
}

}  // namespace pw
