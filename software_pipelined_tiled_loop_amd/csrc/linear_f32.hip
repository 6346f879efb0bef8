// linear_f32.hip -- feed-forward operators on fp32 operands (fp32 accumulation).
#include "linear_variants.hpp"

namespace pgemm {

static const LinVariant k_table[] = {
    LIN_CLASS(DT_F32, 256, 256, 32, 2, 2, 4),  // 8 waves of 128 x 64
    LIN_CLASS(DT_F32, 128, 128, 32, 2, 2, 2),  // 4 waves of 64 x 64
    LIN_FEW_CLASSES(DT_F32),
};

LinKernels linear_kernels_f32() { return LIN_KERNELS(DT_F32, k_table); }

}  // namespace pgemm
