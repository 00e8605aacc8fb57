// Compiled tile kernels of the paged attention.
#include "attn_tile.h"

namespace gdp {

template <class T, int DIM>
static AttnKernel pick(int rows)
{
    return rows == 64 ? attn_tile<T, DIM, 2> : rows == 128 ? attn_tile<T, DIM, 4> : nullptr;
}

template <class T>
static AttnKernel pick(int dim, int rows)
{
    return dim == 64 ? pick<T, 64>(rows) : dim == 128 ? pick<T, 128>(rows) : dim == 256 ? pick<T, 256>(rows) : nullptr;
}

AttnKernel attn_tile_kernel(int dtype, int dim, int rows)
{
    return dtype == BLK_BF16 ? pick<BF16>(dim, rows) : dtype == BLK_F16 ? pick<F16>(dim, rows) : nullptr;
}

}  // namespace gdp
