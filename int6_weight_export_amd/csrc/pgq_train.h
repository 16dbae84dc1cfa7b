// pgq_train.h -- host helpers shared by the entry points outside pgq_api.hip (the linear layer and
// the optimizer step).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pgq {

// PGQ_ERR_HIP, after keeping e as the calling thread's latest HIP error (pgq_last_error).
int32_t note_hip_error(hipError_t e);
// 64-bit hash of n bytes, chained through h (descriptor table checksums).
uint64_t hash_bytes(const void* data, size_t n, uint64_t h);

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace pgq
