// Distillation loss over bf16 logits (kernels: distill.h).
#include "distill.h"

namespace i8mp {
hipError_t launch_distill_bf16(const DistillArgs& a, hipStream_t stream) { return distill::launch_typed<__bf16>(a, stream); }
}  // namespace i8mp
