// Distillation loss over fp16 logits (kernels: distill.h).
#include "distill.h"

namespace i8mp {
hipError_t launch_distill_fp16(const DistillArgs& a, hipStream_t stream) { return distill::launch_typed<_Float16>(a, stream); }
}  // namespace i8mp
