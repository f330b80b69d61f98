// sv_attn.cu -- attention of ragged windows over a paged cache: the entry
// point, and the kernel that takes every layout (sv_attn_tc.cu has the one
// for the usual ones).
#include <cooperative_groups.h>
#include <math.h>

#include "sv_attn.cuh"

namespace cg = cooperative_groups;

namespace sv {
namespace {

// One CTA per (token, key head, kRows of the head's query heads).  Its warps take
// the cached keys in turn, kKeys at a time; a warp holds the rows and a key
// across its lanes (lane l: elements l, l + 32, ...).  The kRows x kKeys partial
// scores of a lane are summed over the warp all at once: at every step a lane
// keeps half of its sums and hands the others to its partner, so that 32 sums
// take 31 exchanges instead of 160, and lane i ends up with score i.  Each lane
// then has one weight to compute, and its row's maximum and part of the sum.
// The warps' results are joined in warp order.  Where there are few CTAs and the
// cache can be long, a cluster of up to 8 shares the keys and joins its CTAs'
// results through their shared memory, in the order of the CTAs.
//
// Every access is one element wide, so that any stride, page size and head size
// is served; instructions bound it.  64 single tokens over 4,224 keys, 32 heads
// (4 a key head): fp32 heads of 128 0.48 ms (4.6 TB/s; 2.22 with a CTA a row and
// a warp sum a key), bf16 heads of 96 0.48 (2.54), of 256 1.17 (5.1).  One token
// over 131,072 keys, 8 heads of 256: 1.1 ms, 80 without the cluster and the
// shared sums.  1,024 tokens over 2,048 keys, 16 fp32 heads of 64: 1.2 ms (4.9),
// 6 TFLOP/s: prompts are the tensor-core kernel's business.
// fp32, heads other than 64 and 128, pages that neither divide nor fill tiles of
// 128 keys, unaligned tensors and negative scales come here.
constexpr int log2_of(int n) { return n > 1 ? 1 + log2_of(n / 2) : 0; }

template <typename T, int kElems, int kRows>
struct RowShape {
    static constexpr int kKeys = kElems == 8 ? 4 : 8;
    static constexpr int kWarps = kElems == 8 && kRows > 1 ? 8 : 16;   // at most; of 16, a thread has 128 registers
    static constexpr int kScores = kRows * kKeys, kShift = 5 - log2_of(kScores);
    struct Result {
        float m[kRows], l[kRows], o[kRows][32 * kElems];
    };
};

// Where the count of windows that end before a token does not lead to the one
// that holds it (tokens before the first window, broken windows): the first
// request that is in order and holds token t, or n_req.  Says which are not.
__device__ __noinline__ int look_through(const AttnArgs& a, int t)
{
    const long long room = (long long)a.cache.max_pages * a.cache.page_size;
    int r = a.n_req;
    for (int i = a.n_req - 1; i >= 0; --i) {
        const int q0 = a.qo_indptr[i], q1 = a.qo_indptr[i + 1], n = a.kv_len[i];
        if (q0 < 0 || q1 < q0 || q1 > a.tokens || q1 - q0 > a.max_window || n < 0 || n > room) {
            if (a.status && threadIdx.x == 0) atomicOr(&a.status[i], kBadLayout);
        } else if (q0 <= t && t < q1) {
            r = i;
        }
    }
    return r;
}

template <typename T, int kElems, int kRows>
__global__ void __launch_bounds__(RowShape<T, kElems, kRows>::kWarps * 32, 1)
    attn_rows_kernel(const AttnArgs a)
{
    using S = RowShape<T, kElems, kRows>;
    constexpr int kKeys = S::kKeys, kScores = S::kScores, kShift = S::kShift;
    __shared__ float sm_m[S::kWarps][kRows], sm_l[S::kWarps][kRows], sm_o[S::kWarps][kRows][32 * kElems];
    using Result = typename S::Result;
    __shared__ Result of_cta;
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
    const unsigned chunks = (unsigned)(a.group + kRows - 1) / kRows, per_token = chunks * (unsigned)a.cache.k.heads;
    const unsigned unit = blockIdx.x / (unsigned)parts;
    const int t = (int)(unit / per_token), g = (int)(unit % per_token / chunks);
    const int in_group = (int)(unit % chunks) * kRows, h0 = g * a.group + in_group;
    const int rows = min(kRows, a.group - in_group);
    const long long room = (long long)a.cache.max_pages * a.cache.page_size;
    const int before = windows_before(a.qo_indptr, a.n_req, t);
    if (before >= a.n_req) return;                        // padding
    int r = before, n = a.kv_len[r], q1 = a.qo_indptr[r + 1];
    if (!window_holds(a.qo_indptr, r, t, a.tokens, a.max_window) || n < 0 || n > room) {
        r = look_through(a, t);
        if (r >= a.n_req) return;                         // nobody's, or refused
        n = a.kv_len[r];
        q1 = a.qo_indptr[r + 1];
    }
    const long long pos = (long long)n - q1 + t;
    const int end = a.full ? n : (int)max(0ll, min((long long)n, pos + 1));
    const int begin = a.window_keys > 0 ? (int)max(0ll, min((long long)end, pos - a.window_keys + 1)) : 0;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
    const T* kc = (const T*)a.cache.k.data + g * a.cache.k.stride_head;
    const T* vc = (const T*)a.cache.v.data + g * a.cache.v.stride_head;
    const int32_t* table = a.cache.page_table + (int64_t)r * a.cache.ld_table;
    float q[kRows][kElems], o[kRows][kElems];
#pragma unroll
    for (int y = 0; y < kRows; ++y)
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
            const int e = lane + 32 * i;
            const T* x = (const T*)a.q.data + t * a.q.stride_token + (h0 + y) * a.q.stride_head;
            q[y][i] = y < rows && e < a.head_dim ? to_f32(x[e]) * a.scale : 0.f;
            o[y][i] = 0.f;
        }
    float m = -INFINITY, l = 0.f;                         // of the lane's row; l of the lane's keys alone
    const int mine = lane >> kShift;                      // the lane's score: of row mine / kKeys, key mine % kKeys
    for (int64_t i0 = begin + (int64_t)(part * warps + warp) * kKeys; i0 < end; i0 += parts * warps * kKeys) {
        float s[kScores], v[kKeys][kElems];
        // Lane x looks up key x's page.
        const int64_t jx = i0 + lane;
        int page = -1, slot = 0;
        if (lane < kKeys && jx < end) {
            page = table[(int)jx / a.cache.page_size];
            slot = (int)jx % a.cache.page_size;
            if (page < 0 || page >= a.cache.n_pages) {
                page = -1;
                if (a.status) atomicOr(&a.status[r], kBadLayout);
            }
        }
        const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
        if (!there) continue;
#pragma unroll
        for (int x = 0; x < kKeys; ++x) {
            // Loads without branches: in a missing key's place another one's, in an element's past the head the last.
            const int from = there >> x & 1u ? x : __ffs((int)there) - 1;
            const int64_t px = __shfl_sync(0xffffffffu, page, from), sx = __shfl_sync(0xffffffffu, slot, from);
            const T* kx = kc + px * a.cache.stride_page_k + sx * a.cache.k.stride_token;
            float k[kElems];
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                const int e = min(lane + 32 * i, a.head_dim - 1);
                k[i] = to_f32(kx[e]);
                if (lane + 32 * i >= a.head_dim) k[i] = 0.f;
            }
#pragma unroll
            for (int y = 0; y < kRows; ++y) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kElems; ++i) sum = fmaf(q[y][i], k[i], sum);
                s[y * kKeys + x] = sum;
            }
        }
#pragma unroll
        for (int step = 1; step <= 5; ++step) {
            const int half = kScores >> step, off = 32 >> step;
            if (half == 0) s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);   // fewer scores than lanes
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float give = lane & off ? s[i] : s[i + half], keep = lane & off ? s[i + half] : s[i];
                s[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        }
        asm volatile("" ::: "memory");                    // the values' registers are not held beside the scores'
#pragma unroll
        for (int x = 0; x < kKeys; ++x) {
            const int from = there >> x & 1u ? x : __ffs((int)there) - 1;
            const int64_t px = __shfl_sync(0xffffffffu, page, from), sx = __shfl_sync(0xffffffffu, slot, from);
            const T* vx = vc + px * a.cache.stride_page_v + sx * a.cache.v.stride_token;
#pragma unroll
            for (int i = 0; i < kElems; ++i) v[x][i] = to_f32(vx[min(lane + 32 * i, a.head_dim - 1)]);
        }
        const float score = there >> (mine % kKeys) & 1u ? s[0] : -INFINITY;
        float top = score;                                // NaN stays out of the maximum, not out of the weights
#pragma unroll
        for (int x = 1; x < kKeys; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x << kShift));
        top = fmaxf(top, m);
        const float keep = m == -INFINITY ? 0.f : expf(m - top);
        const float w = score == -INFINITY ? 0.f : expf(score - top);
        m = top;
        l = l * keep + w;
        if (__any_sync(0xffffffffu, keep != 1.f)) {
#pragma unroll
            for (int y = 0; y < kRows; ++y) {
                const float ky = __shfl_sync(0xffffffffu, keep, (y * kKeys) << kShift);
#pragma unroll
                for (int i = 0; i < kElems; ++i) o[y][i] *= ky;
            }
        }
#pragma unroll
        for (int x = 0; x < kKeys; ++x)
#pragma unroll
            for (int y = 0; y < kRows; ++y) {
                const float wx = __shfl_sync(0xffffffffu, w, (y * kKeys + x) << kShift);
                if (wx == 0.f) continue;                  // whatever the value is
#pragma unroll
                for (int i = 0; i < kElems; ++i) o[y][i] = fmaf(wx, v[x][i], o[y][i]);
            }
    }
#pragma unroll
    for (int x = 1; x < kKeys; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x << kShift);
    if (mine % kKeys == 0) {
        sm_m[warp][mine / kKeys] = m;
        sm_l[warp][mine / kKeys] = l;
    }
#pragma unroll
    for (int y = 0; y < kRows; ++y)
#pragma unroll
        for (int i = 0; i < kElems; ++i) sm_o[warp][y][lane + 32 * i] = o[y][i];
    __syncthreads();
    // Of results with sums: their largest maximum, and what each counts for.  NaN: only NaN scores.
    auto factor = [](float m, float l, float top) { return l == 0.f ? 0.f : m == -INFINITY ? NAN : expf(m - top); };
    for (int y = 0; y < rows; ++y) {
        float mt = -INFINITY, lt = 0.f;
        for (int w = 0; w < warps; ++w) mt = fmaxf(mt, sm_m[w][y]);
        for (int w = 0; w < warps; ++w) {
            const float f = factor(sm_m[w][y], sm_l[w][y], mt);
            if (f != 0.f) lt += sm_l[w][y] * f;
        }
        for (int e = (int)threadIdx.x; e < 32 * kElems; e += (int)blockDim.x) {
            float x = 0.f;
            for (int w = 0; w < warps; ++w) {
                const float f = factor(sm_m[w][y], sm_l[w][y], mt);
                if (f != 0.f) x += sm_o[w][y][e] * f;
            }
            of_cta.o[y][e] = x;
        }
        if (threadIdx.x == 0) {
            of_cta.m[y] = mt;
            of_cta.l[y] = lt;
        }
    }
    if (parts > 1) cluster.sync(); else __syncthreads();
    for (int y = part; y < rows; y += parts) {            // a row a CTA
        float mt = -INFINITY, lt = 0.f;
        for (int c = 0; c < parts; ++c) mt = fmaxf(mt, cluster.map_shared_rank(&of_cta, c)->m[y]);
        for (int c = 0; c < parts; ++c) {
            const Result& x = *cluster.map_shared_rank(&of_cta, c);
            const float f = factor(x.m[y], x.l[y], mt);
            if (f != 0.f) lt += x.l[y] * f;
        }
        T* out = (T*)a.out.data + t * a.out.stride_token + (h0 + y) * a.out.stride_head;
        for (int e = (int)threadIdx.x; e < a.head_dim; e += (int)blockDim.x) {
            float sum = 0.f;
            for (int c = 0; c < parts; ++c) {
                const Result& x = *cluster.map_shared_rank(&of_cta, c);
                const float f = factor(x.m[y], x.l[y], mt);
                if (f != 0.f) sum += x.o[y][e] * f;
            }
            out[e] = from_f32<T>(lt == 0.f ? 0.f : sum / lt);
        }
        if (a.lse && threadIdx.x == 0)
            a.lse[(int64_t)t * a.q.heads + h0 + y] = lt == 0.f ? -INFINITY : mt + logf(lt);
    }
    if (parts > 1) cluster.sync();                        // nobody reads a CTA that has ended
}

template <typename T, int kElems, int kRows>
cudaError_t launch_rows_as(const AttnArgs& a, cudaStream_t s)
{
    using S = RowShape<T, kElems, kRows>;
    const unsigned units = (unsigned)a.tokens * (unsigned)a.cache.k.heads * (unsigned)((a.group + kRows - 1) / kRows);
    const unsigned wave = 2u * (unsigned)sm_count();
    const unsigned warps = units <= wave ? S::kWarps : 4;
    // Four turns of every warp at least, and no more CTAs than run at once.
    const long long cached = (long long)a.cache.max_pages * a.cache.page_size;
    unsigned parts = 1;
    while (parts < 8 && units * parts * 2 <= wave && cached >= (long long)(parts * 2 * warps * S::kKeys * 4)) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * parts);
    cfg.blockDim = dim3(warps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    pdl_attr(at[0]);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = parts;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_rows_kernel<T, kElems, kRows>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s)
{
    if (a.head_dim <= 128) return a.group > 1 ? launch_rows_as<T, 4, 4>(a, s) : launch_rows_as<T, 4, 1>(a, s);
    return a.group > 1 ? launch_rows_as<T, 8, 4>(a, s) : launch_rows_as<T, 8, 1>(a, s);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& a, sv_dtype_t dt, cudaStream_t s)
{
    return dt == SV_DTYPE_BF16 ? launch_rows<__nv_bfloat16>(a, s)
           : dt == SV_DTYPE_F16 ? launch_rows<__half>(a, s)
                                : launch_rows<float>(a, s);
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
