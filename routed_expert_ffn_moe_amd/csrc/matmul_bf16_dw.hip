// Gradient of the weights: dw = dy^T x.  (matmul_bf16_tile.h)
#include "matmul_bf16_tile.h"

namespace moe {

void launch_mm16_dw(const Mm16Args &a, int shape, hipStream_t st)
{
    a.out_f32 ? launch_shape<MM_DW, true>(a, shape, st) : launch_shape<MM_DW, false>(a, shape, st);
}

}  // namespace moe
