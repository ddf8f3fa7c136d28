// product_q6k.hip -- instances of product.h for Q6K.
#include "product.h"

namespace ql {

hipError_t launch_product_q6k(int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s)
{
    return launch_fmt<FMT_Q6K>(mode, tile, a, grid, s);
}

}  // namespace ql
