// ckpt_sizes.hpp -- sizes of rows kept in 8 bits, for host and device code.
#pragma once

#include <hip/hip_runtime.h>

namespace moe {

constexpr int kCkptBlock = 32;  // columns that share a scale byte

__host__ __device__ inline int ckpt_blocks(int width) { return (width + kCkptBlock - 1) / kCkptBlock; }

}  // namespace moe
