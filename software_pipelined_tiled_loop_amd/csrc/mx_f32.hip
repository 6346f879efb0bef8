// mx_f32.hip -- the norm and the microscaled operators on fp32 values.
#include "mx_variants.hpp"

namespace pgemm {

static const NormVariant<NormArgs> k_norms[] = {NORM_VARIANTS(DT_F32)};
static const NormVariant<NormGradArgs> k_grads[] = {NORM_GRAD_VARIANTS(DT_F32)};
static const MxVariant k_table[] = {MX_VARIANTS_F32};

MxKernels mx_kernels_f32() { return MX_KERNELS(DT_F32, k_norms, k_grads, k_table); }

}  // namespace pgemm
