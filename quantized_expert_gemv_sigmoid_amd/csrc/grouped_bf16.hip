// The bf16 outputs of moe_grouped_linear on 16-bit operands (linear_dev.h).
#include "linear_dev.h"

namespace moe {

void launch_grouped_bf16(const GroupedParams &p, const LinearPlan &c, hipStream_t st) { launch_typed<false>(p, c, st); }

}  // namespace moe
