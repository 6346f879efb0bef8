// mx_bf16.hip -- the norm and the microscaled operators on bf16 values.
#include "mx_variants.hpp"

namespace pgemm {

static const NormVariant k_norms[] = {NORM_VARIANTS(DT_BF16)};
static const MxVariant k_table[] = {MX_VARIANTS(DT_BF16)};

MxKernels mx_kernels_bf16() { return MX_KERNELS(DT_BF16, k_norms, k_table); }

}  // namespace pgemm
