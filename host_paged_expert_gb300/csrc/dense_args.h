// Checks of arguments that the C calls of the dense operators share.
#pragma once

#include "dense.cuh"
#include "pe_internal.h"

namespace pe {
namespace dense {

constexpr int kMaxFeatures = 1 << 24;

// Device address of the operators' error word on the current device.
cudaError_t error_word(uint32_t** out);

inline pe_status bad(const char* msg, pe_status st = PE_ERR_INVALID) {
    set_thread_error(msg);
    return st;
}
inline pe_status done(cudaError_t e) {
    if (!e) return PE_OK;
    return bad(cudaGetErrorString(e), PE_ERR_CUDA);
}

inline bool aligned(const void* p, int to = 16) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
// what is read and written one element at a time
inline bool whole(const float* p) { return aligned(p, sizeof(float)); }
inline bool whole(const int32_t* p) { return aligned(p, sizeof(int32_t)); }
inline bool is_elem(int e) { return e == PE_ELEM_BF16 || e == PE_ELEM_F16; }
inline bool is_act(int a) { return a >= PE_ACT_NONE && a <= PE_ACT_RELU; }
inline bool pitch_ok(int64_t ld, int64_t row, int bytes) { return ld >= row && ld * bytes % 16 == 0 && ld < (int64_t(1) << 36); }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace dense
}  // namespace pe
