// The f16 kernels of moe_linear (linear_dev.h).
#include "linear_dev.h"

namespace moe {

void launch_linear_f16(const LinearParams &p, const LinearPlan &c, hipStream_t st) { launch_typed<true>(p, c, st); }

}  // namespace moe
