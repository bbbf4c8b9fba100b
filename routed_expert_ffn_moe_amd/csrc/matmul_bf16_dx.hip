// Gradient of the rows: dx = dy w.  (matmul_bf16_tile.h)
#include "matmul_bf16_tile.h"

namespace moe {

void launch_mm16_dx(const Mm16Args &a, int shape, hipStream_t st)
{
    a.out_f32 ? launch_shape<MM_DX, true>(a, shape, st) : launch_shape<MM_DX, false>(a, shape, st);
}

}  // namespace moe
