// sv_rope.cu -- rotary positions, and the append of rotated keys to a paged
// cache.
//
// Both are copies with a little arithmetic: two reads and two writes of a
// vector a rotation of its pairs apart, so HBM bounds them (and launch latency
// when the tokens are few).  The sines are what could cost more than the copy:
// a token has rot_dim / 2 angles but heads * rot_dim / 2 pairs, so a CTA takes
// whole tokens, computes each angle of its tokens once into shared memory and
// uses it for every head.  Measured on a GB300: 16,384 tokens x 40 heads x 128
// bf16 rotated in 56 us (6.0 TB/s, 88% of the copy bandwidth); 12,200 tokens'
// keys, values and queries (48 heads x 128, half of each rotated) placed in 53 us
// (5.7 TB/s, 84%); a window of 8 tokens 2.8 us of GPU time.  Many small
// CTAs hide their lookups and sines behind one another: reading ahead of them
// within a thread cost registers, so occupancy, and was slower (65 us for 55 of
// an earlier state), and so were 2 or 8 tokens a CTA.
//
// The angle: position p times a frequency f in turns.  p f in fp32 would be
// off by p f 2^-24 turns (at p = 131,072 and f = 0.16: 1e-3).  With f = hi +
// lo, p hi is split into its rounded product and the exact rest of it by an
// fma, the whole turns of the product are taken off exactly, and the rest
// terms are added to the fraction.  Past 2^24 the rest terms reach tens of turns
// and are split in the same way: four sums of numbers below 2, rounded to 2^-24
// or less, are off by 2.4e-7 turns.
#include <limits.h>

#include "sv_attn.cuh"

namespace sv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTok = 4;   // tokens of one CTA
constexpr int64_t kNoSlot = INT64_MIN, kPadding = INT64_MIN + 1;   // in place of a token's offset into the cache

// cos and sin (times mscale) of a position's angle on one pair.
__device__ __forceinline__ float2 rotary_cs(int p, const float* freq, int m, float mscale, bool inverse)
{
    const float hi = freq[2 * m], lo = freq[2 * m + 1];
    const float pf = (float)p;
    const float prod = __fmul_rn(pf, hi);   // rounded, here and where it is used: not to be fused with what follows
    const float err = __fmaf_rn(pf, hi, -prod);
    float rest = __fmaf_rn(pf, lo, err);
    if (fabsf(pf) >= 16777216.f) {          // what was small is not: every part of the rest has whole turns of its own
        const float lost = (float)(int)((long long)p - (long long)pf);   // by the conversion of p
        const float a = __fmul_rn(lost, hi), b = __fmul_rn(pf, lo);
        rest = __fsub_rn(err, rintf(err)) + __fsub_rn(a, rintf(a)) + __fsub_rn(b, rintf(b)) +
               (__fmaf_rn(lost, hi, -a) + __fmaf_rn(pf, lo, -b) + lost * lo);
    }
    float turns = __fsub_rn(prod, rintf(prod)) + rest;
    if (inverse) turns = -turns;
    float s, c;
    sincospif(2.f * turns, &s, &c);
    return make_float2(c * mscale, s * mscale);
}

template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

template <typename T, int VEC>
union Part {
    typename Raw<(int)sizeof(T) * VEC>::type raw;
    T e[VEC];
    __device__ Part() {}
};

struct RopeArgs {
    sv_heads_t q, q_out, k, v;    // sv_rotary: q only
    sv_paged_kv_t cache;
    const int32_t* positions;     // sv_rotary; NULL: positions from the windows
    const int32_t* qo_indptr;
    const int32_t* kv_len;
    int32_t* status;
    sv_rotary_t rope;
    int tokens, head_dim, n_req;
    int per_cta;                  // tokens of a CTA
    int in_place;                 // q_out is q: what is not rotated stays where it is
};

// A head is a set of units: each rotated unit is two parts of VEC elements
// whose pairs it turns (rot_dim / 2 apart, or adjacent in the interleaved
// layout), then two parts a unit (one where they are odd) for what is only
// copied.  A thread keeps one unit of the head and walks over the heads of the
// CTA's tokens.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a)
{
    extern __shared__ float2 cs[];                       // [per_cta][rot_dim / 2]
    __shared__ int64_t base_k[kRopeMaxTok], base_v[kRopeMaxTok];   // the tokens' slots
    __shared__ int pos_sh[kRopeMaxTok];
    pdl_enter();
    const int tid = (int)threadIdx.x;
    const int t0 = (int)blockIdx.x * a.per_cta;
    const int nt = min(a.per_cta, a.tokens - t0);
    const int half = a.rope.rot_dim >> 1;
    if (a.positions) {
        if (tid < nt) pos_sh[tid] = a.positions[t0 + tid];
    } else {
        if (a.status && blockIdx.x == 0)                            // windows that are refused
            for (int i = tid; i < a.n_req; i += kRopeThreads) {
                const int q0 = a.qo_indptr[i], q1 = a.qo_indptr[i + 1];
                if (q0 < 0 || q1 < q0 || q1 > a.tokens) atomicOr(&a.status[i], kBadLayout);
            }
        int r = windows_before(a.qo_indptr, a.n_req, t0);
        if (tid < nt) {
            const int t = t0 + tid;
            while (tid > 0 && r < a.n_req && a.qo_indptr[r + 1] <= t) ++r;
            int end = 0, len = 0;
            if (r < a.n_req) {
                end = a.qo_indptr[r + 1];
                len = a.kv_len[r];
                if (!window_holds(a.qo_indptr, r, t, a.tokens, INT_MAX)) {   // before the first window, or a broken one
                    for (r = 0; r < a.n_req && !window_holds(a.qo_indptr, r, t, a.tokens, INT_MAX); ++r) {}
                    if (r < a.n_req) {
                        end = a.qo_indptr[r + 1];
                        len = a.kv_len[r];
                    }
                }
            }
            int64_t bk = kPadding, bv = kPadding;
            long long p = 0;
            if (r < a.n_req) {
                p = (long long)len - end + t;
                bk = bv = kNoSlot;
                if (p >= 0 && p < (long long)a.cache.max_pages * a.cache.page_size) {
                    const int col = (int)(p / a.cache.page_size), slot = (int)(p % a.cache.page_size);
                    const int page = a.cache.page_table[(int64_t)r * a.cache.ld_table + col];
                    if (page >= 0 && page < a.cache.n_pages) {
                        bk = page * a.cache.stride_page_k + slot * a.cache.k.stride_token;
                        bv = page * a.cache.stride_page_v + slot * a.cache.v.stride_token;
                    }
                }
                if (bk == kNoSlot && a.status) atomicOr(&a.status[r], kBadLayout);
            }
            pos_sh[tid] = (int)p;
            base_k[tid] = bk;
            base_v[tid] = bv;
        }
    }
    __syncthreads();
    for (int i = tid; i < nt * half; i += kRopeThreads) {
        const int t = i / half, m = i - t * half;
        cs[i] = rotary_cs(pos_sh[t], a.rope.freq, m, a.rope.mscale, (a.rope.flags & SV_ROTARY_INVERSE) != 0);
    }
    __syncthreads();
    const int turned = half / VEC;                                  // rotated units of a head
    const int copied = (a.head_dim - 2 * half) / VEC;
    const bool by_two = copied % 2 == 0;
    const int units = turned + (by_two ? copied / 2 : copied);
    const int step = kRopeThreads / units;                          // heads a pass of the CTA covers
    const int unit = tid % units;
    int h = tid / units;
    if (h >= step) return;
    const bool is_turned = unit < turned;
    const bool two = is_turned || by_two;
    const int e0 = is_turned ? (INTER ? 2 * unit * VEC : unit * VEC) : 2 * half + (unit - turned) * VEC * (by_two ? 2 : 1);
    const int e1 = INTER || !is_turned ? e0 + VEC : e0 + half;
    const int nq = a.q.data ? a.q.heads : 0, nk = a.k.data ? a.k.heads : 0;
    const int heads = nq + 2 * nk;
    int t = 0;
    for (;; h += step) {
        while (h >= heads) { h -= heads; ++t; }
        if (t >= nt) return;
        const bool append = nk != 0;
        if (append && base_k[t] == kPadding) continue;
        const T* src;
        T* dst;
        bool turn = is_turned;
        const int64_t tok = t0 + t;
        if (h < nq) {
            if (a.in_place && !is_turned) continue;
            src = (const T*)a.q.data + tok * a.q.stride_token + h * a.q.stride_head;
            dst = (T*)a.q_out.data + tok * a.q_out.stride_token + h * a.q_out.stride_head;
        } else {
            if (base_k[t] == kNoSlot) continue;
            const bool is_k = h < nq + nk;
            const int g = is_k ? h - nq : h - nq - nk;
            src = is_k ? (const T*)a.k.data + tok * a.k.stride_token + g * a.k.stride_head
                       : (const T*)a.v.data + tok * a.v.stride_token + g * a.v.stride_head;
            dst = is_k ? (T*)a.cache.k.data + base_k[t] + g * a.cache.k.stride_head
                       : (T*)a.cache.v.data + base_v[t] + g * a.cache.v.stride_head;
            turn = turn && is_k;
        }
        using R = typename Raw<(int)sizeof(T) * VEC>::type;
        Part<T, VEC> x0, x1;
        // Side by side, with no branch between them: 56 us for 16,384 tokens, 62 when the second waits for one.
        x0.raw = *reinterpret_cast<const R*>(src + e0);
        x1.raw = *reinterpret_cast<const R*>(src + (two ? e1 : e0));
        if (turn) {
            const float2* c = cs + t * half + unit * VEC;
            if (INTER && VEC > 1) {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const float2 w0 = c[i / 2], w1 = c[VEC / 2 + i / 2];
                    const float p0 = to_f32(x0.e[i]), q0 = to_f32(x0.e[i + 1]);
                    const float p1 = to_f32(x1.e[i]), q1 = to_f32(x1.e[i + 1]);
                    x0.e[i] = from_f32<T>(p0 * w0.x - q0 * w0.y);
                    x0.e[i + 1] = from_f32<T>(q0 * w0.x + p0 * w0.y);
                    x1.e[i] = from_f32<T>(p1 * w1.x - q1 * w1.y);
                    x1.e[i + 1] = from_f32<T>(q1 * w1.x + p1 * w1.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float2 w = c[i];
                    const float p = to_f32(x0.e[i]), q = to_f32(x1.e[i]);
                    x0.e[i] = from_f32<T>(p * w.x - q * w.y);
                    x1.e[i] = from_f32<T>(q * w.x + p * w.y);
                }
            }
        }
        *reinterpret_cast<R*>(dst + e0) = x0.raw;
        if (two) *reinterpret_cast<R*>(dst + e1) = x1.raw;
    }
}

template <typename T, int VEC>
cudaError_t launch_rope_vec(RopeArgs a, cudaStream_t s)
{
    a.per_cta = a.tokens >= 2048 ? kRopeMaxTok : 1;
    const dim3 grid((a.tokens + a.per_cta - 1) / a.per_cta);
    const size_t smem = sizeof(float2) * (size_t)a.per_cta * (size_t)(a.rope.rot_dim / 2);
    return a.rope.flags & SV_ROTARY_INTERLEAVED
               ? launch_pdl(rope_kernel<T, VEC, true>, grid, dim3(kRopeThreads), smem, s, a)
               : launch_pdl(rope_kernel<T, VEC, false>, grid, dim3(kRopeThreads), smem, s, a);
}

// The widest access every row of every tensor allows.
template <typename T>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s)
{
    constexpr int kWide = 16 / (int)sizeof(T);
    auto fits = [&](int n) {
        auto ok = [&](const sv_heads_t& h) { return !h.data || heads_aligned(h, n, (int)sizeof(T)); };
        return a.head_dim % n == 0 && (a.rope.rot_dim / 2) % n == 0 && ok(a.q) && ok(a.q_out) && ok(a.k) && ok(a.v) &&
               ok(a.cache.k) && ok(a.cache.v) && a.cache.stride_page_k % n == 0 && a.cache.stride_page_v % n == 0 &&
               a.head_dim / n <= kRopeThreads;
    };
    if (fits(kWide)) return launch_rope_vec<T, kWide>(a, s);
    if (fits(kWide / 2)) return launch_rope_vec<T, kWide / 2>(a, s);
    return launch_rope_vec<T, 1>(a, s);
}

sv_status_t run_rope(const RopeArgs& a, sv_dtype_t dt, cudaStream_t s)
{
    const cudaError_t e = dt == SV_DTYPE_BF16  ? launch_rope<__nv_bfloat16>(a, s)
                          : dt == SV_DTYPE_F16 ? launch_rope<__half>(a, s)
                                               : launch_rope<float>(a, s);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

bool rotary_ok(const sv_rotary_t& r, int head_dim)
{
    return r.rot_dim >= 0 && r.rot_dim <= head_dim && r.rot_dim % 2 == 0 && (r.rot_dim == 0 || r.freq);
}

bool type_ok(sv_dtype_t dt) { return dt == SV_DTYPE_BF16 || dt == SV_DTYPE_F32 || dt == SV_DTYPE_F16; }

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status_t sv_rotary(sv_heads_t x, sv_heads_t y, sv_dtype_t dt, int tokens, int head_dim,
                                 const int32_t* positions, sv_rotary_t rope, sv_stream_t stream)
{
    if (tokens < 0 || head_dim < 1 || x.heads < 1 || y.heads != x.heads || !type_ok(dt) || !rotary_ok(rope, head_dim))
        return SV_ERR_INVALID_ARG;
    if (head_dim > kRotaryMaxDim) return SV_ERR_UNSUPPORTED;
    if (tokens == 0) return SV_OK;
    if (!x.data || !y.data || !positions) return SV_ERR_INVALID_ARG;
    const bool same = x.data == y.data;
    if (same && (x.stride_token != y.stride_token || x.stride_head != y.stride_head)) return SV_ERR_INVALID_ARG;
    RopeArgs a{};
    a.q = x;
    a.q_out = y;
    a.positions = positions;
    a.rope = rope;
    a.tokens = tokens;
    a.head_dim = head_dim;
    a.in_place = same;
    return run_rope(a, dt, stream);
}

extern "C" sv_status_t sv_kv_append(sv_heads_t k, sv_heads_t v, sv_paged_kv_t cache, sv_dtype_t dt, int tokens,
                                    int head_dim, int n_req, const int32_t* qo_indptr, const int32_t* kv_len,
                                    sv_rotary_t rope, sv_heads_t q, sv_heads_t q_out, int32_t* status,
                                    sv_stream_t stream)
{
    if (tokens < 0 || head_dim < 1 || n_req < 1 || !type_ok(dt) || !rotary_ok(rope, head_dim) ||
        (rope.flags & SV_ROTARY_INVERSE) || k.heads < 1 || v.heads != k.heads || cache.k.heads != k.heads ||
        cache.v.heads != k.heads || cache.page_size < 1 || cache.n_pages < 0 || cache.max_pages < 0 ||
        cache.ld_table < cache.max_pages || (q.data && (q.heads < 1 || q_out.heads != q.heads || !q_out.data)))
        return SV_ERR_INVALID_ARG;
    if (head_dim > kRotaryMaxDim) return SV_ERR_UNSUPPORTED;
    if (tokens == 0) return SV_OK;
    if (!k.data || !v.data || !cache.k.data || !cache.v.data || !cache.page_table || !qo_indptr || !kv_len)
        return SV_ERR_INVALID_ARG;
    const bool same = q.data && q.data == q_out.data;
    if (same && (q.stride_token != q_out.stride_token || q.stride_head != q_out.stride_head))
        return SV_ERR_INVALID_ARG;
    RopeArgs a{};
    a.q = q;
    a.q_out = q_out;
    a.k = k;
    a.v = v;
    a.cache = cache;
    a.qo_indptr = qo_indptr;
    a.kv_len = kv_len;
    a.status = status;
    a.rope = rope;
    a.tokens = tokens;
    a.head_dim = head_dim;
    a.n_req = n_req;
    a.in_place = same;
    return run_rope(a, dt, stream);
}
