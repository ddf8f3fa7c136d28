// product_q4k.hip -- instances of product.h for Q4K.
#include "product.h"

namespace ql {

hipError_t launch_product_q4k(int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s)
{
    return launch_fmt<FMT_Q4K>(mode, tile, a, grid, s);
}

}  // namespace ql
