// product_kquants.hip -- instances of product.h for Q5K, Q3K, Q2K and FP8.
#include "product.h"

namespace ql {

hipError_t launch_product_kquants(int fmt, int mode, int tile, const ProductArgs &a, unsigned grid, hipStream_t s)
{
    switch (fmt) {
    case FMT_Q5K: return launch_fmt<FMT_Q5K>(mode, tile, a, grid, s);
    case FMT_Q3K: return launch_fmt<FMT_Q3K>(mode, tile, a, grid, s);
    case FMT_Q2K: return launch_fmt<FMT_Q2K>(mode, tile, a, grid, s);
    default: return launch_fmt<FMT_FP8>(mode, tile, a, grid, s);
    }
}

hipError_t launch_one_kquants(int fmt, bool bf16, const OneArgs &a, unsigned grid, hipStream_t s)
{
    switch (fmt) {
    case FMT_Q5K: return launch_one_fmt<FMT_Q5K>(bf16, a, grid, s);
    case FMT_Q3K: return launch_one_fmt<FMT_Q3K>(bf16, a, grid, s);
    case FMT_Q2K: return launch_one_fmt<FMT_Q2K>(bf16, a, grid, s);
    default: return launch_one_fmt<FMT_FP8>(bf16, a, grid, s);
    }
}

}  // namespace ql
