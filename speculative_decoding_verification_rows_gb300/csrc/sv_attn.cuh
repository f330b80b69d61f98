// sv_attn.cuh -- what the kernels of the attention operators share: element
// types, and the place of a token in a ragged batch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_internal.cuh"

namespace sv {

constexpr int kRotaryMaxDim = 256;   // head elements sv_rotary and sv_kv_append take
constexpr int kAttnMaxDim = 256;     // head elements sv_paged_attention takes

template <typename T>
__device__ __forceinline__ float to_f32(T x)
{
    return (float)x;
}
template <typename T>
__device__ __forceinline__ T from_f32(float x)
{
    return (T)x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x)
{
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x)
{
    return __float2half_rn(x);
}

// Request r's window, on the token axis and of up to `longest` tokens, holds token t.
__device__ __forceinline__ bool window_holds(const int32_t* qo_indptr, int r, int t, int tokens, int longest)
{
    const int q0 = qo_indptr[r], q1 = qo_indptr[r + 1];
    return q0 >= 0 && q0 <= t && t < q1 && q1 <= tokens && q1 - q0 <= longest;
}

// The number of windows that end at or before token t, which is the request that
// holds it, if one does and the bounds only grow.  Called by every thread of the
// block (it holds block barriers), so that the bounds are read side by side
// instead of one after the other.
__device__ __forceinline__ int windows_before(const int32_t* qo_indptr, int n_req, int t)
{
    int r = 0;
    for (int i0 = 0; i0 < n_req; i0 += (int)blockDim.x) {
        const int i = i0 + (int)threadIdx.x;
        r += __syncthreads_count(i < n_req && qo_indptr[i + 1] <= t);
    }
    return r;
}

inline bool aligned_to(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0u; }

// The strides of a heads tensor are multiples of `n` elements and its base of
// n * size bytes.
inline bool heads_aligned(const sv_heads_t& h, int n, int size)
{
    return aligned_to(h.data, (size_t)n * size) && h.stride_token % n == 0 && h.stride_head % n == 0;
}

struct AttnArgs {
    sv_heads_t q, out;
    sv_paged_kv_t cache;
    const int32_t* qo_indptr;
    const int32_t* kv_len;
    float* lse;
    int32_t* status;
    int tokens, head_dim, n_req, max_window, window_keys, full;
    int group;          // query heads per key head
    float scale;
};

// The kernel that takes every layout.
cudaError_t launch_attn_rows(const AttnArgs& a, sv_dtype_t dt, cudaStream_t s);

// The tensor-core kernels: which calls they take (four times as fast on single
// tokens, over a hundred times on prompt chunks), and their workspace.
bool attn_tc_takes(const AttnArgs& a, sv_dtype_t dt);
size_t attn_tc_workspace(int max_window, int group, int head_dim);
cudaError_t launch_attn_tc(const AttnArgs& a, sv_dtype_t dt, void* ws, int num_sms, cudaStream_t s);

int sm_count();   // of the current device

}  // namespace sv
