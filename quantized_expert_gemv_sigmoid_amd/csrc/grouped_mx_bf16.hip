// The bf16 outputs of moe_grouped_linear on MXFP4 operands (linear_dev.h).
#include "linear_dev.h"

namespace moe {

void launch_grouped_mx_bf16(const GroupedMxParams &p, const LinearPlan &c, hipStream_t st) { launch_typed<false>(p, c, st); }

}  // namespace moe
