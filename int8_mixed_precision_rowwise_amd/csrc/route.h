// Launchers of the experts' routing (route.hip).
#pragma once

#include "internal.h"

namespace i8mp {

struct RouteArgs {
  const void* logits;
  int64_t T, E, ld;
  int dtype, k, score, normalize;
  float* weights;
  int32_t *experts, *places, *rows, *offsets;
  int32_t* hist;  // [blocks][E], for more than one block of tokens
};
constexpr int kRouteMaxExperts = 1024, kRouteMaxK = 32;
int64_t route_block_tokens(int64_t T, int64_t E, int64_t k);  // tokens a workgroup counts
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);
hipError_t launch_route_bwd(const RouteArgs& a, const int32_t* experts, const float* dweights, void* d, int64_t ldd,
                            hipStream_t stream);

struct CombineArgs {
  int64_t T, R, N;
  int k, dtype;
  const void* Y;
  int64_t ldy;
  const int32_t* places;
  const float* weights;
  const void *residual, *dout;
  int64_t ldr, ldd;
  void *out, *dY;
  int64_t ldo, ldg;
  const int32_t* rows;
  float* dweights;
  bool vec;  // every row starts at 16 bytes, in whole chunks
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream);
hipError_t launch_combine_bwd(const CombineArgs& a, hipStream_t stream);

}  // namespace i8mp
