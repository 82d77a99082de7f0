// Launch helpers of the operators around the layer.
#pragma once

namespace redmoe {

// Allow `kern` (a __global__ function) `bytes` of dynamic shared memory on the current device. What
// has been allowed is remembered, so a call that asks again costs a lookup; false on a CUDA error.
bool allow_smem(const void* kern, int bytes);

}  // namespace redmoe
