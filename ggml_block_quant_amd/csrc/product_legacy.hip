// product_legacy.hip -- instances of product.h for Q4_0, Q4_1, Q5_0 and Q5_1.
#include "product.h"

namespace ql {

hipError_t launch_product_legacy(int fmt, int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s)
{
    switch (fmt) {
    case FMT_Q4_0: return launch_fmt<FMT_Q4_0>(mode, tile, a, grid, s);
    case FMT_Q4_1: return launch_fmt<FMT_Q4_1>(mode, tile, a, grid, s);
    case FMT_Q5_0: return launch_fmt<FMT_Q5_0>(mode, tile, a, grid, s);
    default: return launch_fmt<FMT_Q5_1>(mode, tile, a, grid, s);
    }
}

hipError_t launch_one_legacy(int fmt, bool bf16, const OneArgs &a, unsigned grid, hipStream_t s)
{
    switch (fmt) {
    case FMT_Q4_0: return launch_one_fmt<FMT_Q4_0>(bf16, a, grid, s);
    case FMT_Q4_1: return launch_one_fmt<FMT_Q4_1>(bf16, a, grid, s);
    case FMT_Q5_0: return launch_one_fmt<FMT_Q5_0>(bf16, a, grid, s);
    default: return launch_one_fmt<FMT_Q5_1>(bf16, a, grid, s);
    }
}

}  // namespace ql
