// The bf16 kernels of moe_linear (linear_dev.h).
#include "linear_dev.h"

namespace moe {

void launch_linear_bf16(const LinearParams &p, const LinearPlan &c, hipStream_t st) { launch_typed<false>(p, c, st); }

}  // namespace moe
