#include "block.h"
namespace i8mp {
hipError_t launch_block_few(const BlockFew&, hipStream_t) { return hipErrorInvalidValue; }
bool block_few_takes(int64_t, int64_t, int64_t, int64_t) { return false; }
}  // namespace i8mp
