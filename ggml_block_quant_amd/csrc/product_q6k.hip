// product_q6k.hip -- instances of product.h for Q6K.
#include "product.h"

namespace ql {

hipError_t launch_product_q6k(int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s)
{
    return launch_fmt<FMT_Q6K>(mode, tile, a, grid, s);
}

hipError_t launch_one_q6k(bool bf16, const OneArgs &a, unsigned grid, hipStream_t s)
{
    return launch_one_fmt<FMT_Q6K>(bf16, a, grid, s);
}

}  // namespace ql
