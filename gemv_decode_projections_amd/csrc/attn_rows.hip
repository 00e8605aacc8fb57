// Compiled row kernels of the paged attention.
#include "attn_rows.h"

namespace gdp {

template <class T, int DIM>
static AttnKernel pick(int nb)
{
    return nb == 1 ? attn_rows<T, DIM, 1> : nb == 2 ? attn_rows<T, DIM, 2> : nullptr;
}

template <class T>
static AttnKernel pick(int dim, int nb)
{
    return dim == 64 ? pick<T, 64>(nb) : dim == 128 ? pick<T, 128>(nb) : dim == 256 ? pick<T, 256>(nb) : nullptr;
}

AttnKernel attn_rows_kernel(int dtype, int dim, int nb)
{
    return dtype == BLK_BF16 ? pick<BF16>(dim, nb) : dtype == BLK_F16 ? pick<F16>(dim, nb) : nullptr;
}

}  // namespace gdp
