// product_q8_0.hip -- instances of product.h for Q8_0.
#include "product.h"

namespace ql {

hipError_t launch_product_q8_0(int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s)
{
    return launch_fmt<FMT_Q8_0>(mode, tile, a, grid, s);
}

hipError_t launch_one_q8_0(bool bf16, const OneArgs &a, unsigned grid, hipStream_t s)
{
    return launch_one_fmt<FMT_Q8_0>(bf16, a, grid, s);
}

}  // namespace ql
