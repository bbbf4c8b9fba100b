// Forward: y = x w^T.  (matmul_bf16_tile.h)
#include "matmul_bf16_tile.h"

namespace moe {

void launch_mm16_y(const Mm16Args &a, int shape, hipStream_t st)
{
    a.out_f32 ? launch_shape<MM_Y, true>(a, shape, st) : launch_shape<MM_Y, false>(a, shape, st);
}

}  // namespace moe
