// Compiled tile kernels of the paged attention.
#include "attn_tile.h"

namespace gdp {

template <class T, int DIM>
static AttnKernel pick(int waves)
{
    return waves == 2 ? attn_tile<T, DIM, 2> : waves == 4 ? attn_tile<T, DIM, 4> : nullptr;
}

template <class T>
static AttnKernel pick(int dim, int waves)
{
    return dim == 64 ? pick<T, 64>(waves) : dim == 128 ? pick<T, 128>(waves) : dim == 256 ? pick<T, 256>(waves) : nullptr;
}

AttnKernel attn_tile_kernel(int dtype, int dim, int waves)
{
    return dtype == BLK_BF16 ? pick<BF16>(dim, waves) : dtype == BLK_F16 ? pick<F16>(dim, waves) : nullptr;
}

}  // namespace gdp
