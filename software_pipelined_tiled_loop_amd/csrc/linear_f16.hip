// linear_f16.hip -- feed-forward operators on fp16 operands (fp32 accumulation).
#include "linear_variants.hpp"

namespace pgemm {

static const LinVariant k_table[] = {
    LIN_CLASS(DT_F16, 256, 256, 64, 2, 2, 2),  // 4 waves of 128 x 128
    LIN_CLASS(DT_F16, 128, 128, 64, 2, 2, 2),  // 4 waves of 64 x 64, two workgroups a CU
    LIN_CLASS(DT_F16, 128, 128, 64, 4, 2, 2),  // the same, one a CU, its ring as deep as the loads take
    LIN_FEW_CLASSES(DT_F16),
};

LinKernels linear_kernels_f16() { return LIN_KERNELS(DT_F16, k_table); }

}  // namespace pgemm
