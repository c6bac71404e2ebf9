// Launchers of a router's balance loss and z loss, and of their gradient
// (balance.hip).
#pragma once

#include "common.h"

namespace moe {

size_t balance_workspace_bytes(int T, int k, int E);
hipError_t launch_balance(const void* logits, int dtype, long long ld, int T, int E, int k, const int32_t* idx,
                          const uint8_t* keep, float* losses, int32_t* counts, int32_t* kept, void* ws,
                          hipStream_t s);
hipError_t launch_balance_gradient(const void* logits, int dtype, long long ld, int T, int E, int k,
                                   const uint8_t* keep, const int32_t* counts, const int32_t* kept, const float* d,
                                   void* dx, hipStream_t s);

}  // namespace moe
