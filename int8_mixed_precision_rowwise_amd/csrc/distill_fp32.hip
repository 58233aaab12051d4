// Distillation loss over fp32 logits (kernels: distill.h).
#include "distill.h"

namespace i8mp {
hipError_t launch_distill_fp32(const DistillArgs& a, hipStream_t stream) { return distill::launch_typed<float>(a, stream); }
}  // namespace i8mp
