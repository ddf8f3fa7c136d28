// product_kquants.hip -- instances of product.h for Q5K, Q3K, Q2K and FP8.
#include "product.h"

namespace ql {

hipError_t launch_product_kquants(int fmt, int mode, int tile, const ProductArgs &a, dim3 grid, hipStream_t s)
{
    switch (fmt) {
    case FMT_Q5K: return launch_fmt<FMT_Q5K>(mode, tile, a, grid, s);
    case FMT_Q3K: return launch_fmt<FMT_Q3K>(mode, tile, a, grid, s);
    case FMT_Q2K: return launch_fmt<FMT_Q2K>(mode, tile, a, grid, s);
    default: return launch_fmt<FMT_FP8>(mode, tile, a, grid, s);
    }
}

}  // namespace ql
