// api_common.h -- host helpers shared by the C entry points (api.cu,
// api_block.cu).
#pragma once

#include "moe_w8a8.h"
#include "internal.h"

namespace moe {

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline moe_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

inline bool moe_shape_ok(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
    if (T < 0 || T > (int64_t(1) << 20)) return false;
    if (H < 128 || H > 16384 || H % 128) return false;
    if (I < 128 || I > 16384 || I % 128) return false;
    if (E < 1 || E > kMaxExperts) return false;
    if (k < 1 || k > kMaxTopK || k > E) return false;
    return true;
}

template <typename T>
T* at(void* base, size_t off) {
    return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}

// Whether a test forces an INT8 GEMM kernel (moe_w8a8_set_gemm_path).
bool gemm_path_forced();

}  // namespace moe
