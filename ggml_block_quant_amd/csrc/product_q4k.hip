// product_q4k.hip -- instances of product.h for Q4K.
#include "product.h"

namespace ql {

hipError_t launch_product_q4k(int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s)
{
    return launch_fmt<FMT_Q4K>(mode, tile, a, grid, s);
}

hipError_t launch_one_q4k(bool bf16, const OneArgs &a, unsigned grid, hipStream_t s)
{
    return launch_one_fmt<FMT_Q4K>(bf16, a, grid, s);
}

}  // namespace ql
