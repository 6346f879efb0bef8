// mx_bf16.hip -- the norm and the microscaled operators on bf16 values.
#include "mx_variants.hpp"

namespace pgemm {

static const NormVariant<NormArgs> k_norms[] = {NORM_VARIANTS(DT_BF16)};
static const NormVariant<NormGradArgs> k_grads[] = {NORM_GRAD_VARIANTS(DT_BF16)};
static const MxVariant k_table[] = {MX_VARIANTS(DT_BF16)};

MxKernels mx_kernels_bf16() { return MX_KERNELS(DT_BF16, k_norms, k_grads, k_table); }

}  // namespace pgemm
