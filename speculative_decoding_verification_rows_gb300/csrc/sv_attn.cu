// sv_attn.cu -- attention of ragged windows over a paged cache: the entry
// point, and the kernel that takes every layout (sv_attn_tc.cu has the one
// for the usual ones).
#include <math.h>

#include "sv_attn.cuh"

namespace sv {
namespace {

constexpr int kRowThreads = 128;   // threads of a row's CTA
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowElems = kAttnMaxDim / 32;   // head elements a lane can hold

// One CTA per (token, query head).  Its warps take the row's keys in turn; a
// warp holds the head across its lanes (lane l: elements l, l + 32, ...), so a
// score is a warp sum, and keeps a running maximum, sum and weighted sum of
// values.  The warps' results are joined in warp order.  Every access is one
// element wide, so that any stride, page size and head size is served; each
// row reads its request's whole cache from L2, and the warp sum of every key
// bounds it (64 single tokens x 32 heads over 256 to 8,192 keys: 2.8 ms, 25 times
// the tensor-core kernel's 0.108).  fp32, heads other than 64 and 128, pages that
// neither divide nor fill tiles of 128 keys, unaligned tensors and negative scales
// come here.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) attn_rows_kernel(const AttnArgs a)
{
    __shared__ float sm_m[kRowWarps], sm_l[kRowWarps], sm_o[kRowWarps][kAttnMaxDim];
    pdl_enter();
    const int t = (int)(blockIdx.x / (unsigned)a.q.heads), h = (int)(blockIdx.x % (unsigned)a.q.heads);
    const int r = request_of_token(a.qo_indptr, a.n_req, t);
    if (r >= a.n_req) return;                             // padding
    const int q0 = a.qo_indptr[r], q1 = a.qo_indptr[r + 1], n = a.kv_len[r];
    const bool bad = q0 < 0 || q0 > t || q1 > a.tokens || q1 - q0 > a.max_window || n < 0 ||
                     (long long)n > (long long)a.cache.max_pages * a.cache.page_size;
    if (bad) {
        if (a.status && threadIdx.x == 0) atomicOr(&a.status[r], kBadLayout);
        return;
    }
    const long long pos = (long long)n - q1 + t;
    const int end = a.full ? n : (int)max(0ll, min((long long)n, pos + 1));
    const int begin = a.window_keys > 0 ? (int)max(0ll, min((long long)end, pos - a.window_keys + 1)) : 0;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const T* q = (const T*)a.q.data + t * a.q.stride_token + h * a.q.stride_head;
    const int g = h / a.group;
    const T* kc = (const T*)a.cache.k.data + g * a.cache.k.stride_head;
    const T* vc = (const T*)a.cache.v.data + g * a.cache.v.stride_head;
    const int32_t* table = a.cache.page_table + (int64_t)r * a.cache.ld_table;
    float qr[kRowElems], o[kRowElems];
#pragma unroll
    for (int i = 0; i < kRowElems; ++i) {
        const int e = lane + 32 * i;
        qr[i] = e < a.head_dim ? to_f32(q[e]) * a.scale : 0.f;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = begin + warp; j < end; j += kRowWarps) {
        const int page = table[j / a.cache.page_size], slot = j % a.cache.page_size;
        if (page < 0 || page >= a.cache.n_pages) {
            if (a.status && lane == 0) atomicOr(&a.status[r], kBadLayout);
            continue;
        }
        const T* k = kc + page * a.cache.stride_page_k + slot * a.cache.k.stride_token;
        const T* v = vc + page * a.cache.stride_page_v + slot * a.cache.v.stride_token;
        float s = 0.f, vr[kRowElems];
#pragma unroll
        for (int i = 0; i < kRowElems; ++i) {
            const int e = lane + 32 * i;
            vr[i] = e < a.head_dim ? to_f32(v[e]) : 0.f;
            if (e < a.head_dim) s = fmaf(qr[i], to_f32(k[e]), s);
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        if (s == -INFINITY) continue;                     // weight 0
        const float m_new = s > m ? s : m;                // NaN stays out of the maximum, not out of the weight
        const float keep = m == -INFINITY ? 0.f : expf(m - m_new);
        const float p = expf(s - m_new);
        m = m_new;
        l = l * keep + p;
#pragma unroll
        for (int i = 0; i < kRowElems; ++i) o[i] = fmaf(p, vr[i], o[i] * keep);
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < kRowElems; ++i) sm_o[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float mt = -INFINITY, lt = 0.f;
    for (int w = 0; w < kRowWarps; ++w) mt = fmaxf(mt, sm_m[w]);
    float f[kRowWarps];
    for (int w = 0; w < kRowWarps; ++w) {
        f[w] = sm_l[w] == 0.f ? 0.f : sm_m[w] == -INFINITY ? NAN : expf(sm_m[w] - mt);   // NaN: only NaN scores
        if (f[w] != 0.f) lt += sm_l[w] * f[w];
    }
    T* out = (T*)a.out.data + t * a.out.stride_token + h * a.out.stride_head;
    for (int e = (int)threadIdx.x; e < a.head_dim; e += kRowThreads) {
        float x = 0.f;
        for (int w = 0; w < kRowWarps; ++w)
            if (f[w] != 0.f) x += sm_o[w][e] * f[w];
        out[e] = from_f32<T>(lt == 0.f ? 0.f : x / lt);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)t * a.q.heads + h] = lt == 0.f ? -INFINITY : mt + logf(lt);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& a, sv_dtype_t dt, cudaStream_t s)
{
    const dim3 grid((unsigned)a.tokens * (unsigned)a.q.heads);
    if (dt == SV_DTYPE_BF16) return launch_pdl(attn_rows_kernel<__nv_bfloat16>, grid, dim3(kRowThreads), 0, s, a);
    if (dt == SV_DTYPE_F16) return launch_pdl(attn_rows_kernel<__half>, grid, dim3(kRowThreads), 0, s, a);
    return launch_pdl(attn_rows_kernel<float>, grid, dim3(kRowThreads), 0, s, a);
}

}  // namespace sv

using namespace sv;

extern "C" size_t sv_attention_workspace_size(int max_window, int q_heads, int kv_heads, int head_dim)
{
    if (max_window < 0 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || head_dim < 1 ||
        head_dim > kAttnMaxDim)
        return 0;
    return head_dim == 64 || head_dim == 128 ? attn_tc_workspace(max_window, q_heads / kv_heads, head_dim) : 256;
}

extern "C" sv_status_t sv_paged_attention(sv_heads_t q, sv_paged_kv_t cache, sv_dtype_t dt, int tokens, int head_dim,
                                          int n_req, const int32_t* qo_indptr, const int32_t* kv_len, int max_window,
                                          float scale, int window_keys, int flags, sv_heads_t out, float* lse,
                                          int32_t* status, void* ws, size_t ws_bytes, sv_stream_t stream)
{
    if (tokens < 0 || head_dim < 1 || n_req < 1 || max_window < 0 || window_keys < 0 || !isfinite(scale) ||
        (dt != SV_DTYPE_BF16 && dt != SV_DTYPE_F16 && dt != SV_DTYPE_F32) || cache.k.heads < 1 ||
        cache.v.heads != cache.k.heads || q.heads < 1 || q.heads % cache.k.heads || out.heads != q.heads ||
        cache.page_size < 1 || cache.n_pages < 0 || cache.max_pages < 0 || cache.ld_table < cache.max_pages)
        return SV_ERR_INVALID_ARG;
    if (head_dim > kAttnMaxDim || (long long)tokens * q.heads > (1ll << 30)) return SV_ERR_UNSUPPORTED;
    if (tokens == 0) return SV_OK;
    if (!q.data || !out.data || !cache.k.data || !cache.v.data || !cache.page_table || !qo_indptr || !kv_len)
        return SV_ERR_INVALID_ARG;
    const size_t need = sv_attention_workspace_size(max_window, q.heads, cache.k.heads, head_dim);
    if (!ws || !aligned_to(ws, 256) || ws_bytes < need) return SV_ERR_WORKSPACE;
    AttnArgs a{};
    a.q = q;
    a.out = out;
    a.cache = cache;
    a.qo_indptr = qo_indptr;
    a.kv_len = kv_len;
    a.lse = lse;
    a.status = status;
    a.tokens = tokens;
    a.head_dim = head_dim;
    a.n_req = n_req;
    a.max_window = max_window;
    a.window_keys = window_keys;
    a.full = flags & SV_ATTN_FULL ? 1 : 0;
    a.group = q.heads / cache.k.heads;
    a.scale = scale;
    const cudaError_t e = attn_tc_takes(a, dt) ? launch_attn_tc(a, dt, ws, sm_count(), stream)
                                               : launch_attn_rows(a, dt, stream);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
