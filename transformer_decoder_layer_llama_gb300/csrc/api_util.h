// Argument checks shared by the C-ABI layer files (api.cu, api_cache.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/llama_layer.h"

namespace ll {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The decode attention loads K/V in boxes of min(block_size, 64) rows that must
// tile a 64-key span exactly and keep the 1024-byte swizzle alignment.
inline bool block_size_ok(int bs) { return bs >= 16 && bs <= 256 && (bs & (bs - 1)) == 0; }

inline int cuda_rc(cudaError_t e) { return e == cudaSuccess ? LL_OK : LL_ERR_CUDA; }

}  // namespace ll
