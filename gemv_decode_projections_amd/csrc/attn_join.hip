// Compiled join kernels of the paged attention.
#include "attn_join.h"

namespace gdp {

template <class T, int DIM>
static AttnKernel pick(int rows)
{
    switch (rows) {
    case 32: return attn_join<T, DIM, 32>;
    case 64: return attn_join<T, DIM, 64>;
    case 128: return attn_join<T, DIM, 128>;
    default: return nullptr;
    }
}

template <class T>
static AttnKernel pick(int dim, int rows)
{
    return dim == 64 ? pick<T, 64>(rows) : dim == 128 ? pick<T, 128>(rows) : dim == 256 ? pick<T, 256>(rows) : nullptr;
}

AttnKernel attn_join_kernel(int dtype, int dim, int rows)
{
    return dtype == BLK_BF16 ? pick<BF16>(dim, rows) : dtype == BLK_F16 ? pick<F16>(dim, rows) : nullptr;
}

}  // namespace gdp
