// The f16 outputs of moe_mx_linear (linear_dev.h).
#include "linear_dev.h"

namespace moe {

void launch_mx_f16(const MxParams &p, const LinearPlan &c, hipStream_t st) { launch_typed<true>(p, c, st); }

}  // namespace moe
