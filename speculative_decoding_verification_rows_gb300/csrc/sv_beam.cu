// sv_beam.cu -- beam search: the best continuations over beams and vocabulary,
// and state rows that follow their beams' parents.
//
// Selection.  score(b, v) = base_b + (l_{b,v} - m_b), m_b the row's maximum,
// base_b = c_b - ln sum exp(l - m_b).  What a call has to read is every live row
// once; the rest is small.  So one kernel streams the rows (scan_kernel): a warp takes 4 KB
// chunks, sums exp(l - ref) in fp32 against a running reference and leaves the
// chunk's maximum.  The n_out best candidates lie in the n_out best chunks: a
// chunk that n_out others stand before (by maximum, then by place) has n_out
// elements before each of its own.  A second kernel (pick_kernel, a CTA an item)
// bounds the n_out-th best chunk's score from below, reads again the few chunks
// that reach the bound and sorts the elements that do.
//
// Order.  Within a beam it is the logits' and exact.  Between beams it hangs on
// the difference of two normalisers, and fp32 sums are off by up to kNearEps
// (derived below), while candidates of a batch come nearer than that now and
// then.  Where neighbours of different beams do, up to the last selected place or
// as near behind it, their beams' rows are summed again (refine_kernel), terms in
// double-float arithmetic, the sum in whole numbers, and the item's saved
// candidates are sorted once more: the order is then that of scores in 64 bits,
// rows of the same values have the same sum in whatever order, and ties go to
// the lowest place.
//
// Measured on a GB300: 64 items x 16 beams x 248,320 bf16 in 87 us, of which the
// scan is 78.5 (6.48 TB/s, 95% of the copy bandwidth; 334 warp instructions a
// chunk of 2,048 elements, 47% of the issue slots); what follows it is a chain of
// latencies, 12,000 clocks: normalisers 2,900, bound 1,100, chunks read again
// 2,500, order 1,800 and the steps between them.  64 x 16 x 124,160 fp32 in 84 us
// (89% of the copy bandwidth), 32 x 8 x 151,936 bf16 in 19, one item of 4 x 32,000
// in 11 (15 to 20 with the host's part).  An item whose order is checked again costs
// 8 to 12 us more.
//
// Tried and dropped: chunks set out by cp.async to a stage a warp (32 x 8 x
// 151,936 32 us instead of 22 at the time: more instructions, and those are what
// a mid-sized call is bound by), eight vectors a lane in a ring of registers (33
// us: more loads in flight than a warp has scoreboards to wait on one by one),
// candidates' 64-bit scores formed as they are found (fp64 in divergent code).
#include <float.h>
#include <math.h>

#include <atomic>

#include "sv_attn.cuh"
#include "sv_internal.cuh"

namespace sv {
namespace {

constexpr int kMaxBeams = 128;
constexpr int kMaxOut = 256;
constexpr int kBeamMaxVocab = 1 << 19;
constexpr int kScanThreads = 256;
constexpr int kVecs = 8;                     // 16-byte vectors a lane takes of a chunk
constexpr int kMaxSegChunks = 8;             // chunks a warp sums up before it leaves a partial sum
constexpr int kPickThreads = 1024;
constexpr int kSmallPick = 256;              // threads of an item's CTA where items are many; kMaxOut at least
constexpr int kListCap = 2048;               // elements that an item may have at its bound
constexpr int kChunkCap = 1024;              // and chunks
constexpr int kPickHeld = 4;                 // chunk maxima a thread keeps in registers
constexpr int kRefineElems = 4096;           // elements of a row a CTA of refine_kernel sums
constexpr int kRefineTurns = 32;             // elements a thread sums at most: 32 2^58 < 2^64

// |ln sum exp(l - m) - computed| of one row, V <= 2^19.  With p the row's probabilities,
// sum p |l - m| = H - ln Z <= ln V <= 13.2, so an argument's relative error r costs 13.2 r.
// Near zero (references of whole powers of two, see Ref): the argument's rounding and
// log2 e, 13.2 (2^-24 + 2^-26) -> 1.0e-6; ex2.approx 2^-22 -> 2.4e-7; sums by trees of 8
// levels in a chunk, 5 shuffles, 5 of the segments', 2 joins of parts: 20 2^-24 -> 1.2e-6;
// logf, an ulp of 13.2 -> 9.6e-7; the reference's part 5e-8: 3.5e-6 in all.
// Elsewhere: difference and product 2^-24 each, up to kMaxSegChunks moves of the
// reference and the segments' join, 9 (2^-22 + 2^-24) -> 2.7e-6: 6.9e-6.
constexpr double kSumEps = 8e-6, kNearEps = 4e-6;
constexpr float kNear = 0x1p20f;

enum { kDead = 0, kLive = 1, kFinished = 2 };

// What an item's CTA knows of a beam, read in one piece.
struct __align__(16) BeamRec {
    float base, top;    // base in fp32; the row's maximum (0 of a finished beam)
    float score;        // as it was before the call: the outputs may lie where the scores do
    int kind;
};

struct BeamArgs {
    const void* logits;
    int64_t stride_item, stride_beam;
    int n, beams, vocab, n_out, end_token;
    const float* scores;
    const uint8_t* finished;
    int32_t* out_tokens;
    int32_t* out_parents;
    float* out_scores;
    int32_t* status;
    // workspace
    int32_t* n_flagged;      // rows to be summed again
    int32_t* item_units;     // refine units of an item
    int32_t* item_done;
    int32_t* item_list;      // candidates saved, or -1: more than a list holds
    uint32_t* item_mask;     // [n][4] beams that are summed again
    int32_t* flagged;        // [rows]
    BeamRec* rec;            // [rows], of items that are sorted again
    double* base;            // [rows]
    float2* sums;            // [rows][segs] reference, sum
    float* chunk_max;        // [rows][chunks]
    float* list_logit;       // [n][kListCap]
    int32_t* list_flat;
    ulonglong2* refined;     // [rows][refine segments] sums in units of 2^-26 and of 2^-58
    int chunks, seg_chunks, segs, refine_elems, refine_segs;
};

// What the rows' element type says about their layout in 16-byte vectors.
template <int DT>
struct Elem {
    static constexpr int kSize = DT == 0 ? 2 : 4;
    static constexpr int kPerVec = 16 / kSize;
    static constexpr int kChunk = kVecs * 32 * kPerVec;
};

// A row as vectors that start on 16-byte boundaries: element e is slot e + off.
template <int DT>
struct Row {
    const char* base;
    int off;
    int vocab;
    __device__ Row(const BeamArgs& a, int item, int beam)
    {
        const uintptr_t p = reinterpret_cast<uintptr_t>(a.logits) +
                            (uintptr_t)((item * a.stride_item + beam * a.stride_beam) * Elem<DT>::kSize);
        off = (int)(p & 15u) / Elem<DT>::kSize;
        base = reinterpret_cast<const char*>(p & ~(uintptr_t)15u);
        vocab = a.vocab;
    }
    __device__ __forceinline__ uint4 whole(int vec) const
    {
        uint4 r;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "l"(base + (size_t)vec * 16));
        return r;
    }
    // Element e as raw bits, -inf outside the row.
    __device__ __forceinline__ uint32_t bits(int e) const
    {
        if (e < 0 || e >= vocab) return DT == 0 ? 0xFF80u : 0xFF800000u;
        if (DT == 0) return reinterpret_cast<const uint16_t*>(base)[e + off];
        return reinterpret_cast<const uint32_t*>(base)[e + off];
    }
    __device__ __forceinline__ uint4 vec(int v) const
    {
        const int e0 = v * Elem<DT>::kPerVec - off;
        if (e0 >= 0 && e0 + Elem<DT>::kPerVec <= vocab) return whole(v);
        if (DT == 0)
            return make_uint4(bits(e0) | bits(e0 + 1) << 16, bits(e0 + 2) | bits(e0 + 3) << 16,
                              bits(e0 + 4) | bits(e0 + 5) << 16, bits(e0 + 6) | bits(e0 + 7) << 16);
        return make_uint4(bits(e0), bits(e0 + 1), bits(e0 + 2), bits(e0 + 3));
    }
    // A lane's vectors of chunk c; vector i holds elements from vec_first(c, i) on.
    __device__ __forceinline__ void chunk(int c, uint4 (&v)[kVecs]) const
    {
        const int v0 = c * (kVecs * 32) + (int)(threadIdx.x & 31);
        if (c * Elem<DT>::kChunk - off >= 0 && (c + 1) * Elem<DT>::kChunk - off <= vocab) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = whole(v0 + i * 32);
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = vec(v0 + i * 32);
        }
    }
    __device__ __forceinline__ int vec_first(int c, int i) const
    {
        return ((c * kVecs + i) * 32 + (int)(threadIdx.x & 31)) * Elem<DT>::kPerVec - off;
    }
    __device__ __forceinline__ float elem(int e) const
    {
        return __uint_as_float(DT == 0 ? bits(e) << 16 : bits(e));
    }
};

// Element q of a vector, q known at compile time.
template <int DT>
__device__ __forceinline__ float vec_at(const uint4& v, int q)
{
    const int j = DT == 0 ? q >> 1 : q;
    const uint32_t w = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
    if (DT == 0) return __uint_as_float((q & 1) ? (w & 0xFFFF0000u) : (w << 16));
    return __uint_as_float(w);
}

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float warp_max_nan(float x)
{
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
template <int DT>
__device__ __forceinline__ float vec_max(const uint4& v)
{
    if (DT == 0) {
        const uint32_t w = max2_nan(max2_nan(v.x, v.y), max2_nan(v.z, v.w));
        return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
}

using pair_t = unsigned long long;   // two fp32 numbers, for the packed instructions
__device__ __forceinline__ pair_t pack(float lo, float hi)
{
    pair_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack(pair_t p, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b)
{
    pair_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c)
{
    pair_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b)
{
    pair_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.44269504088896340736f;

// What a segment's reference, its maximum so far, is to its sum.  Near zero: terms are
// 2^(x L - c), one packed fma each, L = log2 e in fp32 and c the whole number next to
// ref L, so that moves of the reference and joins of segments are exact, and what the
// sum is off by, 2^(c - m L), is known.  Elsewhere 2^((x - ref) L).
struct Ref {
    float at = -FLT_MAX, c = 0.f;
    bool near = false;

    __device__ __forceinline__ void move(float top)
    {
        at = top;
        near = fabsf(top) < kNear;
        c = near ? rintf(top * kLog2e) : 0.f;
    }
};
__device__ __forceinline__ float whole_exp2(float e)               // of a whole number up to 0
{
    return e < -126.f ? 0.f : __int_as_float(((int)e + 127) << 23);
}
// By what a sum over reference `from` counts in one over `to`, from.at <= to.at.
__device__ __forceinline__ float ref_weight(const Ref& from, const Ref& to)
{
    if (from.near && to.near) return whole_exp2(from.c - to.c);
    if (from.near == to.near) return exp2_approx((from.at - to.at) * kLog2e);
    return from.near ? exp2_approx(fmaf(-to.at, kLog2e, from.c)) : exp2_approx(fmaf(from.at, kLog2e, -to.c));
}
template <bool NEAR>
__device__ __forceinline__ pair_t exp_pair(float x0, float x1, pair_t k)
{
    const pair_t x = pack(x0, x1), l = pack(kLog2e, kLog2e);
    const pair_t y = NEAR ? fma2(x, l, k) : mul2(add2(x, k), l);
    float y0, y1;
    unpack(y, y0, y1);
    return pack(exp2_approx(y0), exp2_approx(y1));
}
template <int DT, bool NEAR>
__device__ __forceinline__ pair_t vec_exp_sum(const uint4& v, pair_t k)
{
    const pair_t s = add2(exp_pair<NEAR>(vec_at<DT>(v, 0), vec_at<DT>(v, 1), k),
                          exp_pair<NEAR>(vec_at<DT>(v, 2), vec_at<DT>(v, 3), k));
    if (DT != 0) return s;
    constexpr int kLast = Elem<DT>::kPerVec - 1;
    return add2(s, add2(exp_pair<NEAR>(vec_at<DT>(v, 4 & kLast), vec_at<DT>(v, 5 & kLast), k),
                        exp_pair<NEAR>(vec_at<DT>(v, 6 & kLast), vec_at<DT>(v, 7 & kLast), k)));
}
template <int DT, bool NEAR>
__device__ __forceinline__ float chunk_exp_sum(const uint4 (&v)[kVecs], float minus)
{
    const pair_t k = pack(minus, minus);
    pair_t t0 = vec_exp_sum<DT, NEAR>(v[0], k), t1 = vec_exp_sum<DT, NEAR>(v[1], k);
#pragma unroll
    for (int i = 2; i < kVecs; i += 2) {
        t0 = add2(t0, vec_exp_sum<DT, NEAR>(v[i], k));
        t1 = add2(t1, vec_exp_sum<DT, NEAR>(v[i + 1], k));
    }
    float x0, x1;
    unpack(add2(t0, t1), x0, x1);
    return x0 + x1;
}

__device__ __forceinline__ int beam_kind(const BeamArgs& a, int row, float* score)
{
    const uint8_t finished = a.finished ? a.finished[row] : 0;
    *score = a.scores[row];
    return *score == -INFINITY ? kDead : finished ? kFinished : kLive;
}
__device__ __forceinline__ bool is_live(const BeamArgs& a, int row)
{
    float score;
    return beam_kind(a, row, &score) == kLive;
}

// A warp's share of rows row0 .. row0 + rows - 1: the unit is a segment of a row.
template <int DT>
__device__ __forceinline__ void scan_rows(const BeamArgs& a, int row0, int rows, int warp, int warps)
{
    const int lane = threadIdx.x & 31;
    // units in turns of `warps`, their rows and segments without a division each
    const int more_rows = warps / a.segs, more_segs = warps - more_rows * a.segs;
    int at = warp / a.segs, seg = warp - at * a.segs;
    if (at >= rows) return;
    bool live = is_live(a, row0 + at), next_live;
    for (int next, next_seg; at < rows; at = next, seg = next_seg, live = next_live) {
        next = at + more_rows;
        next_seg = seg + more_segs;
        if (next_seg >= a.segs) {
            next_seg -= a.segs;
            ++next;
        }
        next_live = next < rows && is_live(a, row0 + next);       // while this one's data is on its way
        if (!live) continue;
        const int row_no = row0 + at;
        const Row<DT> row(a, row_no / a.beams, row_no % a.beams);
        const int c1 = min((seg + 1) * a.seg_chunks, a.chunks);
        float s_hi = 0.f, s_lo = 0.f;
        Ref ref;
        for (int c = seg * a.seg_chunks; c < c1; ++c) {
            uint4 v[kVecs];
            row.chunk(c, v);
            float top = vec_max<DT>(v[0]);
#pragma unroll
            for (int i = 1; i < kVecs; ++i) top = max_nan(top, vec_max<DT>(v[i]));
            top = warp_max_nan(top);
            if (lane == 0) a.chunk_max[(size_t)row_no * a.chunks + c] = top;
            if (top > ref.at) {
                Ref to;
                to.move(top);
                const float f = ref_weight(ref, to);
                s_hi *= f;
                s_lo *= f;
                ref = to;
            }
            const float x = ref.near ? chunk_exp_sum<DT, true>(v, -ref.c) : chunk_exp_sum<DT, false>(v, -ref.at);
            const dfloat s = df_two_sum(s_hi, x);
            s_hi = s.hi;
            s_lo += s.lo;
        }
        float s = s_hi + s_lo;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) a.sums[(size_t)row_no * a.segs + seg] = make_float2(ref.at, s);
    }
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int DT>
__global__ void __launch_bounds__(kScanThreads, 4) scan_kernel(const __grid_constant__ BeamArgs a)
{
    pdl_enter();
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *a.n_flagged = 0;
        for (int i = threadIdx.x; i < a.n; i += kScanThreads) a.item_done[i] = 0;
    }
    scan_rows<DT>(a, 0, a.n * a.beams, blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5),
                  gridDim.x * (kScanThreads / 32));
}

// The order of scores in 64 bits as that of unsigned numbers; -0 and +0 are one.
__device__ __forceinline__ unsigned long long key_of_f64(double x)
{
    const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ double f64_of_key(unsigned long long k)
{
    return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}

// Candidates of an item in shared memory.
struct Entries {
    unsigned long long* key;
    uint32_t* flat;     // beam * vocab + token
    float* logit;
    uint8_t* beam;
};

// order[i] becomes the i-th candidate: descending by score, ascending by place
// among equals (the places are distinct).  Up to T / 2 candidates find their places
// by counting those before them, a few threads each: two barriers, where the
// sorting network has one a stage.  More are sorted (bitonic).
template <int T>
__device__ void sort_entries(const Entries& e, int n, uint16_t* order)
{
    const int bits = n > 1 ? 32 - __clz(n - 1) : 0, p = 1 << bits;
    if (p <= T / 2) {
        __syncthreads();
        const int most = 31 - __clz(T), share_bits = min(5, most - bits), share = 1 << share_bits;
        const int i = threadIdx.x >> share_bits, j0 = threadIdx.x & (share - 1);
        if ((int)(threadIdx.x & ~31u) >> share_bits < n) {        // (for whole warps)
            int before = 0;
            if (i < n) {
                const unsigned long long k = e.key[i];
                const uint32_t f = e.flat[i];
                for (int j = j0; j < n; j += share) {
                    const unsigned long long other = e.key[j];
                    before += other > k;
                    if (other == k && e.flat[j] < f) ++before;
                }
            }
            for (int o = share >> 1; o; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
            if (i < n && j0 == 0) order[before] = (uint16_t)i;
        }
        __syncthreads();
        return;
    }
    for (int i = threadIdx.x; i < n; i += T) order[i] = (uint16_t)i;
    for (int i = n + threadIdx.x; i < p; i += T) {
        e.key[i] = 0ull;
        e.flat[i] = 0xFFFFFFFFu;
        e.logit[i] = -INFINITY;
        e.beam[i] = 0;
    }
    __syncthreads();
    for (int size = 2; size <= p; size <<= 1) {
        for (int stride = size >> 1; stride; stride >>= 1) {
            for (int t = threadIdx.x; t < (p >> 1); t += T) {
                const int i = 2 * t - (t & (stride - 1)), j = i + stride;
                const bool down = (i & size) == 0;
                const unsigned long long ki = e.key[i], kj = e.key[j];
                const uint32_t fi = e.flat[i], fj = e.flat[j];
                const bool before = ki > kj || (ki == kj && fi < fj);   // i stands before j
                if (before != down) {
                    const float li = e.logit[i];
                    const uint8_t bi = e.beam[i];
                    e.key[i] = kj;
                    e.key[j] = ki;
                    e.flat[i] = fj;
                    e.flat[j] = fi;
                    e.logit[i] = e.logit[j];
                    e.logit[j] = li;
                    e.beam[i] = e.beam[j];
                    e.beam[j] = bi;
                }
            }
            __syncthreads();
        }
    }
}

struct PickShared {
    unsigned long long key[kListCap];
    uint32_t flat[kListCap];
    float logit[kListCap];
    BeamRec rec[kMaxBeams];
    double base[kMaxBeams];
    int chunk[kChunkCap];
    union {
        uint16_t order[kListCap];
        int bins[kPickThreads];
    };
    union {
        int scratch[kMaxOut];
        float least[kMaxBeams];    // l - top of a logit that may reach the bound
    };
    uint8_t beam[kListCap];
    uint32_t mask[4];
    float warp_best[32];
    int warp_count[32];
    float bound;
    int bound_found;
    int n_chunks, n_elems, bad, far, flag_at;

    __device__ Entries entries() { return Entries{key, flat, logit, beam}; }
};

// A score in fp32 (a finite one stays finite), and how far it may be from the
// one in 64 bits with the row's true sum.
__device__ __forceinline__ float score32(const BeamRec& b, float l)
{
    return l == -INFINITY ? l : fmaxf(b.base + (l - b.top), -FLT_MAX);
}
__device__ __forceinline__ float slack32(const BeamRec& b, float l)
{
    return (float)kSumEps + 0x1p-22f * (fabsf(b.base) + fabsf(l - b.top));
}
__device__ __forceinline__ unsigned long long score_key(const PickShared& sh, int b, float l)
{
    return key_of_f64(sh.base[b] + ((double)l - (double)sh.rec[b].top));
}

// The item's outputs from its sorted finite candidates.  Where they are fewer
// than n_out, the places of score -inf follow from the lowest on; they are
// among the first n_out places, since fewer than n_out are not -inf.
template <int DT>
__device__ void write_item(const BeamArgs& a, int item, const Entries& e, int n, PickShared& sh)
{
    const int tid = threadIdx.x;
    if (tid < a.n_out && tid < n) {
        const size_t o = (size_t)item * a.n_out + tid;
        const int i = sh.order[tid], b = e.beam[i];
        a.out_tokens[o] = (int)(e.flat[i] - (uint32_t)b * (uint32_t)a.vocab);
        a.out_parents[o] = b;
        a.out_scores[o] = (float)f64_of_key(e.key[i]);
    }
    if (n >= a.n_out) return;
    int empty = 0, b = 0, t = 0;
    if (tid < a.n_out) {
        b = tid / a.vocab;
        t = tid - b * a.vocab;
        if (sh.rec[b].kind == kDead) empty = 1;
        else if (sh.rec[b].kind == kFinished) empty = t != a.end_token;
        else empty = Row<DT>(a, item, b).elem(t) == -INFINITY;
        sh.scratch[tid] = empty;
    }
    __syncthreads();
    if (empty) {
        int at = n;
        for (int i = 0; i < tid; ++i) at += sh.scratch[i];
        if (at < a.n_out) {
            const size_t o = (size_t)item * a.n_out + at;
            a.out_tokens[o] = t;
            a.out_parents[o] = b;
            a.out_scores[o] = -INFINITY;
        }
    }
}

// A lower bound on the n_out-th largest of the threads' values: counted in bins
// of 32 / T below the largest (four barriers), or, where they lie further apart
// than the T bins reach, by bisection (20 barriers).  -FLT_MAX at least: -inf is what
// is not a value (rows that are not read, what lies past the last chunk), and none
// of it may reach the bound.
template <int T>
__device__ float nth_bound(float best, int n_out, PickShared& sh)
{
    constexpr float kPerUnit = (float)(T / 32);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    sh.bins[tid] = 0;
    if (tid == 0) sh.bound_found = 0;
    const float w = warp_max(best);
    if (lane == 0) sh.warp_best[warp] = w;
    __syncthreads();
    const float most = warp_max(lane < T / 32 ? sh.warp_best[lane] : -INFINITY);
    const float down = (most - best) * kPerUnit;
    if (best > -INFINITY && down < (float)T) atomicAdd(&sh.bins[(int)down], 1);
    __syncthreads();
    const int here = sh.bins[tid];
    int upto = here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) sh.warp_count[warp] = upto;
    __syncthreads();
    int before = lane < warp ? sh.warp_count[lane] : 0;
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    upto += before;
    if (upto >= n_out && upto - here < n_out) {                   // (the bin's edge, and what rounding may have moved across it)
        sh.bound = most - ((float)tid + 1.01f) / kPerUnit - 0x1p-22f * fabsf(most);
        sh.bound_found = 1;
    }
    __syncthreads();
    if (sh.bound_found) return fmaxf(sh.bound, -FLT_MAX);         // (a step below the lowest finite number is -inf)
    const uint32_t mine = key_of_f32_bits(__float_as_uint(best));
    uint32_t bound_key = 0u;
    for (int bit = 31; bit >= 12; --bit) {
        const uint32_t tv = bound_key | (1u << bit);
        if (__syncthreads_count(mine >= tv) >= n_out) bound_key = tv;
    }
    return bound_key <= key_of_f32_bits(0xFF800000u) ? -FLT_MAX : f32_of_key(bound_key);
}

// An item's outputs from its rows' sums and chunk maxima, by one CTA.  Returns 0,
// or the number of rows (sh.mask) to be summed again first: the candidates stay
// in shared memory, sh.n_elems of them, or -1 for more than a list holds.
template <int DT, int T>
__device__ int pick_item(const BeamArgs& a, int item, PickShared& sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = item * a.beams;
    const float* chunk_max = a.chunk_max + (size_t)row0 * a.chunks;
    const int total = a.beams * a.chunks;
    // The chunks' maxima set out at once, rows that were not read among them (what lies there is not looked at).
    float held[kPickHeld];
#pragma unroll
    for (int k = 0; k < kPickHeld; ++k) {
        const int i = tid + k * T;
        held[k] = i < total ? __ldcg(&chunk_max[i]) : 0.f;
    }
    if (tid == 0) sh.n_chunks = sh.n_elems = sh.bad = sh.far = 0;
    if (tid < 4) sh.mask[tid] = 0u;
    __syncthreads();
    // normalisers, a warp a beam
    for (int b = warp; b < a.beams; b += T / 32) {
        const float2* sums = a.sums + (size_t)(row0 + b) * a.segs;
        const float2 part = lane < a.segs ? __ldcg(&sums[lane]) : make_float2(-FLT_MAX, 0.f);
        float score;
        int kind = beam_kind(a, row0 + b, &score);
        double base = (double)score;
        float top = 0.f;
        if (!(score < INFINITY)) {
            if (lane == 0) atomicOr(&sh.bad, kBadParam);
            kind = kDead;
        }
        if (kind == kLive) {
            float m = part.x;
            for (int i = lane + 32; i < a.segs; i += 32) m = fmaxf(m, __ldcg(&sums[i]).x);
            m = warp_max(m);
            Ref all, one;
            all.move(m);
            one.move(lane < a.segs ? part.x : m);                 // (no lane of another kind without need)
            dfloat sum{part.y * ref_weight(one, all), 0.f};
            for (int i = lane + 32; i < a.segs; i += 32) {
                const float2 x = __ldcg(&sums[i]);
                one.move(x.x);
                sum = df_add_f(sum, x.y * ref_weight(one, all));
            }
            float s = sum.hi + sum.lo;
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            if (s == 0.f) kind = kDead;                           // nothing but -inf: every score is -inf
            base = (double)score - (double)logf(s);
            if (all.near) base -= (double)(fmaf(-m, kLog2e, all.c) * (float)kLn2);   // up to 0.35: good to 5e-8
            top = m;
            if (lane == 0 && !(fabsf(m) < 0.5f * kNear)) sh.far = 1;   // (nearer ones: segments that are not near count nothing)
        }
        if (lane == 0) {
            sh.rec[b] = BeamRec{(float)base, top, score, kind};
            sh.base[b] = base;
        }
    }
    __syncthreads();
    // A lower bound on the n_out-th best chunk's score: on the n_out-th largest of the threads' best.
    const float per_beam = 1.f / (float)a.chunks;
    auto beam_of = [&](int i) { return (int)(((float)i + 0.5f) * per_beam); };   // i / chunks: off by 128 3 2^-24 < 0.5 / 513 at most
    float best = -INFINITY;
    auto rate = [&](int i, float m) {                             // the most a chunk's best may have, -inf for nothing
        if (i >= total) return -INFINITY;
        const BeamRec b = sh.rec[beam_of(i)];
        if (b.kind != kLive) return -INFINITY;
        if (!(m < INFINITY)) atomicOr(&sh.bad, kNonfinite);
        const float s = score32(b, m), slack = slack32(b, m);
        if (s == -INFINITY) return s;
        best = fmaxf(best, s - slack);
        return s + slack;
    };
    const int mine = total - warp * 32;                           // of the chunks a warp's turns begin at
#pragma unroll
    for (int k = 0; k < kPickHeld; ++k)
        if (k * T < mine) held[k] = rate(tid + k * T, held[k]);
    for (int i = tid + kPickHeld * T; i < total; i += T) rate(i, __ldcg(&chunk_max[i]));
    if (tid < a.beams && sh.rec[tid].kind == kFinished) best = fmaxf(best, sh.rec[tid].base);
    float bound = nth_bound<T>(best, a.n_out, sh);
    if (sh.bad) {                                                 // (its last write is before the barriers above)
        if (tid < a.n_out) {
            const size_t o = (size_t)item * a.n_out + tid;
            a.out_tokens[o] = a.out_parents[o] = -1;
            a.out_scores[o] = __int_as_float(0x7FC00000);
        }
        if (tid == 0 && a.status) atomicOr(&a.status[item], sh.bad);
        return 0;
    }
    // the chunks that may reach it
    auto keep = [&](int i, float most) {
        if (!(most >= bound)) return;
        const int at = atomicAdd(&sh.n_chunks, 1);
        if (at < kChunkCap) sh.chunk[at] = i;
    };
#pragma unroll
    for (int k = 0; k < kPickHeld; ++k)
        if (k * T < mine) keep(tid + k * T, held[k]);
    for (int i = tid + kPickHeld * T; i < total; i += T) keep(i, rate(i, __ldcg(&chunk_max[i])));
    __syncthreads();
    constexpr int kPer = Elem<DT>::kPerVec;
    bool hard = sh.n_chunks > kChunkCap;
    // Few chunks for n_out (one live beam, a small vocabulary, beams far apart) bound it loosely or not at all; then the
    // lanes' best of the listed chunks give another bound.  32,003 tokens of one beam for n_out = 64 took 190 us without
    // it (more elements than a list holds), 14 with it.
    const int enough = a.n_out + 32;
    for (bool fine = bound == -FLT_MAX || total < 4 * a.n_out; !hard; fine = true) {
        if (fine) {
            best = tid < a.beams && sh.rec[tid].kind == kFinished ? sh.rec[tid].base : -INFINITY;
            for (int k = warp; k < sh.n_chunks; k += T / 32) {
                const int i = sh.chunk[k], b = beam_of(i);
                uint4 v[kVecs];
                Row<DT>(a, item, b).chunk(i - b * a.chunks, v);
                float l = vec_max<DT>(v[0]);
#pragma unroll
                for (int g = 1; g < kVecs; ++g) l = fmaxf(l, vec_max<DT>(v[g]));
                const float s = score32(sh.rec[b], l);
                if (s > -INFINITY) best = fmaxf(best, s - slack32(sh.rec[b], l));
            }
            bound = fmaxf(bound, nth_bound<T>(best, a.n_out, sh));
        }
        // Where l - m is near bound - base, score and slack are off by 2^-22 (|base| + |bound - base|).  A bound of -FLT_MAX
        // is none: scores in 64 bits go below it (the lowest score with a token at the lowest value), and every token counts.
        if (tid < a.beams && sh.rec[tid].kind == kLive) {
            const float base = sh.rec[tid].base, at = bound - base;
            const float least = at - (2.f * (float)kSumEps + 0x1p-20f * (fabsf(base) + fabsf(at)));
            sh.least[tid] = bound == -FLT_MAX ? -FLT_MAX : fmaxf(least, -FLT_MAX);
        }
        __syncthreads();
        if (tid < a.beams && sh.rec[tid].kind == kFinished && sh.rec[tid].base >= bound) {   // one candidate: base alone
            const int at = atomicAdd(&sh.n_elems, 1);
            sh.flat[at] = (uint32_t)tid * (uint32_t)a.vocab + (uint32_t)a.end_token;
            sh.logit[at] = 0.f;
            sh.beam[at] = (uint8_t)tid;
        }
        __syncthreads();                                          // (they find room)
        for (int k = warp; k < sh.n_chunks; k += T / 32) {   // a warp a chunk
            const int i = sh.chunk[k], b = beam_of(i), c = i - b * a.chunks;
            const Row<DT> row(a, item, b);
            uint4 v[kVecs];
            row.chunk(c, v);
            const float top = sh.rec[b].top, least = sh.least[b];
            auto reaches = [&](float l) { return fmaxf(l - top, -FLT_MAX) >= least; };   // (-inf too, where the bound is none)
            // a lane's elements that reach the bound, then room for the warp's at once
            unsigned long long in = 0ull;
#pragma unroll
            for (int g = 0; g < kVecs; ++g) {
                if (!reaches(vec_max<DT>(v[g]))) continue;
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    const float l = vec_at<DT>(v[g], q);
                    if (reaches(l) && l > -INFINITY) in |= 1ull << (g * kPer + q);
                }
            }
            const int own = __popcll(in);
            if (!__any_sync(0xFFFFFFFFu, own != 0)) continue;
            int upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += y;
            }
            int at = 0;
            if (lane == 31) at = atomicAdd(&sh.n_elems, upto);
            at = __shfl_sync(0xFFFFFFFFu, at, 31) + upto - own;
            if (!fine && at > enough) continue;                   // to be done again, with another bound
#pragma unroll
            for (int g = 0; g < kVecs; ++g) {
                if (!(in >> (g * kPer) & ((1u << kPer) - 1u))) continue;
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    if (!(in >> (g * kPer + q) & 1u) || at >= kListCap) continue;
                    sh.flat[at] = (uint32_t)b * (uint32_t)a.vocab + (uint32_t)(row.vec_first(c, g) + q);
                    sh.logit[at] = vec_at<DT>(v[g], q);
                    sh.beam[at] = (uint8_t)b;
                    ++at;
                }
            }
        }
        __syncthreads();
        if (sh.n_elems <= enough || fine) break;
        __syncthreads();
        if (tid == 0) sh.n_elems = 0;
    }
    const int n = sh.n_elems;
    hard = hard || n > kListCap;
    const Entries e = sh.entries();
    if (!hard) {
        for (int i = tid; i < n; i += T) sh.key[i] = score_key(sh, sh.beam[i], sh.logit[i]);
        sort_entries<T>(e, n, sh.order);
        write_item<DT>(a, item, e, n, sh);                        // to be written again where the order may be another
        // What the normalisers' errors, eps at most, may have put the wrong way round: neighbours of two beams within 2 eps,
        // and behind the last place those within 2 eps of it.  (Candidates without such neighbours between them keep
        // their order; those further behind have n_out before them in any case.)  One eps for all beams, finished
        // ones too: between two of larger eps a third must not part them.
        const double eps = sh.far ? kSumEps : kNearEps;
        for (int k = tid; k + 1 < n; k += T) {
            const int i1 = sh.order[k + 1], b0 = sh.beam[sh.order[k]], b1 = sh.beam[i1];
            if (b0 == b1) continue;
            const double s0 = f64_of_key(sh.key[sh.order[min(k, a.n_out - 1)]]), s1 = f64_of_key(sh.key[i1]);
            if (s0 - s1 > 2.0 * eps + 0x1p-50 * (fabs(s1) + fabs(sh.base[b0]) + fabs(sh.base[b1]))) continue;
            if (sh.rec[b0].kind == kLive) atomicOr(&sh.mask[b0 >> 5], 1u << (b0 & 31));
            if (sh.rec[b1].kind == kLive) atomicOr(&sh.mask[b1 >> 5], 1u << (b1 & 31));
        }
    } else if (tid < a.beams && sh.rec[tid].kind == kLive) {
        atomicOr(&sh.mask[tid >> 5], 1u << (tid & 31));
    }
    __syncthreads();
    const int again = __popc(sh.mask[0]) + __popc(sh.mask[1]) + __popc(sh.mask[2]) + __popc(sh.mask[3]);
    if (tid == 0 && hard) sh.n_elems = -1;
    return again;
}

template <int DT, int T>
__global__ void __launch_bounds__(T) pick_kernel(const __grid_constant__ BeamArgs a)
{
    __shared__ PickShared sh;
    pdl_enter();
    const int tid = threadIdx.x, item = blockIdx.x, row0 = item * a.beams;
    const int again = pick_item<DT, T>(a, item, sh);
    if (again == 0) return;
    // refine_kernel finishes the item
    __syncthreads();
    const int n = sh.n_elems;
    for (int i = tid; i < n; i += T) {
        a.list_flat[(size_t)item * kListCap + i] = (int32_t)sh.flat[i];
        a.list_logit[(size_t)item * kListCap + i] = sh.logit[i];
    }
    if (tid < a.beams) {
        a.rec[row0 + tid] = sh.rec[tid];
        a.base[row0 + tid] = sh.base[tid];
    }
    if (tid < 4) a.item_mask[item * 4 + tid] = sh.mask[tid];
    if (tid == 0) {
        a.item_list[item] = n;
        a.item_units[item] = again * a.refine_segs;
        sh.flag_at = atomicAdd(a.n_flagged, again);
    }
    __syncthreads();
    if (tid < a.beams && (sh.mask[tid >> 5] >> (tid & 31) & 1u)) {
        int at = sh.flag_at;
        for (int w = 0; w < tid >> 5; ++w) at += __popc(sh.mask[w]);
        at += __popc(sh.mask[tid >> 5] & ((1u << (tid & 31)) - 1u));
        a.flagged[at] = row0 + tid;
    }
}

// The best candidate below `key`, `place` (the previous one's) over the block: every thread brings its own best.
__device__ void block_best(unsigned long long& key, uint32_t& place, unsigned long long* s_key, uint32_t* s_place)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto take = [&](unsigned long long k, uint32_t p) {
        if (k > key || (k == key && p < place)) {
            key = k;
            place = p;
        }
    };
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xFFFFFFFFu, key, o);
        const uint32_t p = __shfl_xor_sync(0xFFFFFFFFu, place, o);
        take(k, p);
    }
    __syncthreads();
    if (lane == 0) {
        s_key[warp] = key;
        s_place[warp] = place;
    }
    __syncthreads();
    for (int w = 0; w < kPickThreads / 32; ++w) take(s_key[w], s_place[w]);
}

// An item with more candidates at its bound than a list holds (rows of few
// distinct values): its n_out best chunks one after the other, then the n_out
// best of their elements.  Returns how many there are.  Right, not fast: a pass
// over the chunks and one over the listed ones' elements for every continuation,
// by one CTA (32 items of 8 x 151,936 of one value: 1.4 ms for 16 continuations, 15
// for 64; 64 of 16 x 248,320, 32: 246, for in three launches items wait for the CTAs
// that finish others).
template <int DT>
__device__ int pick_by_turns(const BeamArgs& a, int item, PickShared& sh)
{
    __shared__ unsigned long long s_key[kPickThreads / 32];
    __shared__ uint32_t s_place[kPickThreads / 32];
    const int tid = threadIdx.x, row0 = item * a.beams;
    unsigned long long last_key = ~0ull;
    uint32_t last = 0u;
    int n_chunks = 0;
    const int total = a.beams * a.chunks;
    for (; n_chunks < a.n_out; ++n_chunks) {
        unsigned long long key = 0ull;
        uint32_t place = 0xFFFFFFFFu;
        for (int i = tid; i < total; i += kPickThreads) {
            const int b = i / a.chunks;
            float m;
            if (sh.rec[b].kind == kLive) m = a.chunk_max[(size_t)row0 * a.chunks + i];
            else if (sh.rec[b].kind == kFinished && i == b * a.chunks) m = 0.f;
            else continue;
            if (m == -INFINITY) continue;
            const unsigned long long k = score_key(sh, b, m);
            if (!(k < last_key || (k == last_key && (uint32_t)i > last))) continue;
            if (k > key || (k == key && (uint32_t)i < place)) {
                key = k;
                place = (uint32_t)i;
            }
        }
        block_best(key, place, s_key, s_place);
        if (place == 0xFFFFFFFFu) break;
        if (tid == 0) sh.chunk[n_chunks] = (int)place;
        last_key = key;
        last = place;
    }
    __syncthreads();
    last_key = ~0ull;
    last = 0u;
    int n = 0;
    for (; n < a.n_out; ++n) {
        unsigned long long key = 0ull;
        uint32_t place = 0xFFFFFFFFu;
        for (int k = tid >> 5; k < n_chunks; k += kPickThreads / 32) {
            const int b = sh.chunk[k] / a.chunks, c = sh.chunk[k] - b * a.chunks;
            auto look = [&](float l, int token) {
                if (l == -INFINITY) return;
                const unsigned long long x = score_key(sh, b, l);
                const uint32_t p = (uint32_t)b * (uint32_t)a.vocab + (uint32_t)token;
                if (!(x < last_key || (x == last_key && p > last))) return;
                if (x > key || (x == key && p < place)) {
                    key = x;
                    place = p;
                }
            };
            if (sh.rec[b].kind == kFinished) {
                look(0.f, a.end_token);
                continue;
            }
            const Row<DT> row(a, item, b);
            uint4 v[kVecs];
            row.chunk(c, v);
#pragma unroll
            for (int g = 0; g < kVecs; ++g)
#pragma unroll
                for (int q = 0; q < Elem<DT>::kPerVec; ++q) look(vec_at<DT>(v[g], q), row.vec_first(c, g) + q);
        }
        block_best(key, place, s_key, s_place);
        if (place == 0xFFFFFFFFu) break;
        if (tid == 0) {
            sh.key[n] = key;
            sh.flat[n] = place;
            sh.beam[n] = (uint8_t)(place / (uint32_t)a.vocab);
            sh.order[n] = (uint16_t)n;
        }
        last_key = key;
        last = place;
    }
    __syncthreads();
    return n;
}

// The sum of a segment of a row again, by one CTA: a term is a double-float
// (2^-46 of itself) cut to units of 2^-58, so the sum of 2^19 is good to 2^-39
// of itself, and scores to 2e-12.
template <int DT>
__device__ void refine_segment(const BeamArgs& a, int row_no, int seg, float top, const dfloat* tab, ulonglong2* part)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Row<DT> row(a, row_no / a.beams, row_no % a.beams);
    const int e1 = min((seg + 1) * a.refine_elems, a.vocab);
    unsigned long long sum = 0ull;                    // of up to kRefineTurns terms
    for (int e0 = seg * a.refine_elems; e0 < e1; e0 += 4 * kPickThreads) {
        float l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = e0 + k * kPickThreads + tid;
            l[k] = row.elem(min(e, a.vocab - 1));
            if (e >= e1) l[k] = -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (l[k] > -INFINITY) sum += fix_df(exp_df(df_two_sum(l[k], -top), tab), 0x1p58f);
    }
    ulonglong2 all = make_ulonglong2(warp_sum_u64(sum >> 32), warp_sum_u64(sum & 0xFFFFFFFFull));
    __syncthreads();
    if (lane == 0) part[warp] = all;
    __syncthreads();
    if (warp == 0) {
        all = part[lane];
        all.x = warp_sum_u64(all.x);
        all.y = warp_sum_u64(all.y);
        if (lane == 0) a.refined[(size_t)row_no * a.refine_segs + seg] = all;
    }
}

// An item's outputs once its rows are summed again; its records and candidates (n, or -1) are in shared memory.
template <int DT>
__device__ void finish_item(const BeamArgs& a, int item, int n, PickShared& sh)
{
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid < a.beams && (sh.mask[tid >> 5] >> (tid & 31) & 1u)) {
        const int r = item * a.beams + tid;
        unsigned long long high = 0ull, low = 0ull;
        for (int i = 0; i < a.refine_segs; ++i) {
            const ulonglong2 x = __ldcg(&a.refined[(size_t)r * a.refine_segs + i]);
            high += x.x;
            low += x.y;
        }
        sh.base[tid] = (double)sh.rec[tid].score - log((double)high * 0x1p-26 + (double)low * 0x1p-58);
    }
    __syncthreads();
    const Entries e = sh.entries();
    if (n >= 0) {
        for (int i = tid; i < n; i += kPickThreads) sh.key[i] = score_key(sh, sh.beam[i], sh.logit[i]);
        sort_entries<kPickThreads>(e, n, sh.order);
    } else {
        n = pick_by_turns<DT>(a, item, sh);
    }
    write_item<DT>(a, item, e, n, sh);
    __syncthreads();
}

// The flagged rows of all items; the CTA that sums an item's last segment finishes the item.
template <int DT>
__global__ void __launch_bounds__(kPickThreads) refine_kernel(const __grid_constant__ BeamArgs a)
{
    __shared__ PickShared sh;
    __shared__ dfloat tab[64];
    __shared__ ulonglong2 part[kPickThreads / 32];
    __shared__ int last;
    pdl_enter();
    const int tid = threadIdx.x;
    const long long units = (long long)*a.n_flagged * a.refine_segs;
    if (blockIdx.x >= units) return;
    fill_exp_table(tab);
    __syncthreads();
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int f = (int)(u / a.refine_segs), seg = (int)(u - (long long)f * a.refine_segs);
        const int row_no = a.flagged[f], item = row_no / a.beams, row0 = item * a.beams;
        refine_segment<DT>(a, row_no, seg, a.rec[row_no].top, tab, part);
        if (tid == 0) {
            __threadfence();
            last = atomicAdd(&a.item_done[item], 1) == a.item_units[item] - 1;
            __threadfence();
        }
        __syncthreads();
        if (!last) continue;
        const int n = a.item_list[item];
        for (int i = tid; i < n; i += kPickThreads) {
            const uint32_t p = (uint32_t)a.list_flat[(size_t)item * kListCap + i];
            sh.flat[i] = p;
            sh.logit[i] = a.list_logit[(size_t)item * kListCap + i];
            sh.beam[i] = (uint8_t)(p / (uint32_t)a.vocab);
        }
        if (tid < a.beams) {
            sh.rec[tid] = a.rec[row0 + tid];
            sh.base[tid] = a.base[row0 + tid];
        }
        if (tid < 4) sh.mask[tid] = a.item_mask[item * 4 + tid];
        finish_item<DT>(a, item, n, sh);
    }
}

// All of it in one launch, a cluster an item: its CTAs scan the item's rows, the
// first of them picks, and all sum rows again where that is needed.
template <int DT>
__global__ void __launch_bounds__(kPickThreads) select_kernel(const __grid_constant__ BeamArgs a)
{
    __shared__ PickShared sh;
    __shared__ dfloat tab[64];
    __shared__ ulonglong2 part[kPickThreads / 32];
    __shared__ int s_again;
    __shared__ uint32_t s_mask[4];
    pdl_enter();
    const int tid = threadIdx.x;
    uint32_t rank, size;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    const int item = blockIdx.x / size, row0 = item * a.beams;
    scan_rows<DT>(a, row0, a.beams, (int)rank * (kPickThreads / 32) + (tid >> 5), (int)size * (kPickThreads / 32));
    cluster_sync();
    int again = 0;
    if (rank == 0) {
        again = pick_item<DT, kPickThreads>(a, item, sh);
        if (again) {
            if (tid < 4) a.item_mask[item * 4 + tid] = sh.mask[tid];
            if (tid < a.beams) a.rec[row0 + tid] = sh.rec[tid];
        }
        if (tid < (int)size) {                         // into every CTA's own memory
            uint32_t there;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_u32(&s_again)), "r"(tid));
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(again) : "memory");
        }
    }
    cluster_sync();
    again = s_again;
    if (again == 0) return;
    if (tid < 4) s_mask[tid] = __ldcg(&a.item_mask[item * 4 + tid]);
    fill_exp_table(tab);
    __syncthreads();
    const int units = again * a.refine_segs;
    for (int u = (int)rank; u < units; u += (int)size) {
        int f = u / a.refine_segs, b = 0;
        const int seg = u - f * a.refine_segs;
        for (;; ++b)                                   // the f-th flagged beam
            if ((s_mask[b >> 5] >> (b & 31) & 1u) && f-- == 0) break;
        refine_segment<DT>(a, row0 + b, seg, __ldcg(&a.rec[row0 + b].top), tab, part);
    }
    cluster_sync();
    if (rank == 0) finish_item<DT>(a, item, sh.n_elems, sh);
}

struct BeamLayout {
    size_t head, item_units, item_done, item_list, item_mask, flagged, rec, base, sums, chunk_max, list_logit,
        list_flat, refined, total;
};

// Sizes for either element type (fp32 rows have the more chunks).
BeamLayout beam_layout(int n, int beams, int vocab)
{
    const size_t rows = (size_t)n * beams, chunks = ((size_t)vocab + 7 + Elem<1>::kChunk - 1) / Elem<1>::kChunk;
    BeamLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    L.head = take(256);
    L.item_units = take(4 * (size_t)n);
    L.item_done = take(4 * (size_t)n);
    L.item_list = take(4 * (size_t)n);
    L.item_mask = take(16 * (size_t)n);
    L.flagged = take(4 * rows);
    L.rec = take(sizeof(BeamRec) * rows);
    L.base = take(8 * rows);
    L.sums = take(8 * rows * chunks);
    L.chunk_max = take(4 * rows * chunks);
    L.list_logit = take(4 * (size_t)n * kListCap);
    L.list_flat = take(4 * (size_t)n * kListCap);
    L.refined = take(16 * rows * (((size_t)vocab + kRefineElems - 1) / kRefineElems));
    L.total = off;
    return L;
}

cudaLaunchConfig_t cluster_config(int clusters, int size, cudaLaunchAttribute (&at)[2], cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * size);
    cfg.blockDim = dim3(kPickThreads);
    cfg.stream = s;
    pdl_attr(at[0]);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = size;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cfg;
}

// The largest cluster of which n run at once, 0 for none.  (On a GB300 15 of eight CTAs do, 36 of four, 76 of two, 152
// of one; a second wave costs as much as the first.)
template <int DT>
cudaError_t cluster_for(int n, int* size)
{
    constexpr int kSizes[4] = {8, 4, 2, 1};
    static std::atomic<int> active[128][4];            // + 1, once a device (callers may be several threads)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < 4; ++i) {
        int many = dev >= 0 && dev < 128 ? active[dev][i] - 1 : -1;
        if (many < 0) {
            cudaLaunchAttribute at[2];
            cudaLaunchConfig_t cfg = cluster_config(1, kSizes[i], at, nullptr);
            cfg.attrs = at + 1;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&many, select_kernel<DT>, &cfg);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 128) active[dev][i] = many + 1;
        }
        if (n <= many) {
            *size = kSizes[i];
            return cudaSuccess;
        }
    }
    *size = 0;
    return cudaSuccess;
}

template <int DT>
cudaError_t launch_select(BeamArgs a, cudaStream_t s)
{
    using E = Elem<DT>;
    const int sms = sm_count();
    const long long rows = (long long)a.n * a.beams;
    a.chunks = (a.vocab + E::kPerVec - 1 + E::kChunk - 1) / E::kChunk;
    // Segments such that the warp with the most of them has the least to do: its chunks, and a third of a chunk's
    // time for every segment (32 x 8 x 151,936: segments of 4 chunks, two for some warps, took 26,000 clocks, 1 chunk 16,000).
    auto segments = [&](long long of_rows, long long warps) {
        double least = 0.0;
        for (int n = 1; n <= kMaxSegChunks; ++n) {
            const long long segs = (a.chunks + n - 1) / n, turns = (of_rows * segs + warps - 1) / warps;
            const double cost = (double)turns * (n + 0.33);
            if (n > 1 && cost >= least) continue;
            least = cost;
            a.seg_chunks = n;
            a.segs = (int)segs;
        }
    };
    auto refined_by = [&](int elems) {
        const int turns = (elems + kPickThreads - 1) / kPickThreads;
        a.refine_elems = kPickThreads * (turns < 4 ? 4 : turns > kRefineTurns ? kRefineTurns : turns);
        a.refine_segs = (a.vocab + a.refine_elems - 1) / a.refine_elems;
    };
    // One launch of clusters saves two launches (5 us of the host, 2 of the GPU), but an item has its cluster's warps
    // alone: taken where they get no more than two chunks beyond what the whole GPU's would (us on the GPU in one launch
    // and in three: 32 x 8 x 32,000 12.6 and 17.3, 32 x 8 x 151,936 18.6 and 19.0, 1 x 16 x 151,936 19.1 and 14.6).
    int cluster = 0;
    cudaError_t e = cluster_for<DT>(a.n, &cluster);
    if (e != cudaSuccess) return e;
    const double item_chunks = (double)a.beams * a.chunks;
    const int item_warps = cluster * (kPickThreads / 32);
    if (cluster && item_chunks / item_warps <= a.n * item_chunks / (32.0 * sms) + 2.0) {
        segments(a.beams, item_warps);
        refined_by((a.vocab + cluster - 1) / cluster);            // a CTA sums its part of every row
        cudaLaunchAttribute at[2];
        const cudaLaunchConfig_t cfg = cluster_config(a.n, cluster, at, s);
        e = cudaLaunchKernelEx(&cfg, select_kernel<DT>, a);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const long long warps = (long long)sms * 4 * (kScanThreads / 32);
    segments(rows, warps);
    refined_by(kRefineElems);
    const long long units = rows * a.segs;                        // below 2^31
    long long grid = (units + kScanThreads / 32 - 1) / (kScanThreads / 32);
    if (grid > 4LL * sms) grid = 4LL * sms;
    e = launch_pdl(scan_kernel<DT>, dim3((unsigned)grid), dim3(kScanThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    // More items than SMs: four small CTAs an SM, where an item has few chunks to read again or there are many waves
    // (n x beams x vocabulary, n_out; us with large and small CTAs: 1,024 x 4 x 1,000, 8: 76 and 26; 160 x 4 x 32,000, 8:
    // 22.9 and 18.1; 700 x 8 x 9,000, 16: 67 and 45; 300 x 16 x 32,000, 32: 78 and 82; 200 x 8 x 151,936, 16: 86 and 92).
    e = a.n > sms && (a.n_out <= 8 || a.n > 4 * sms) ? launch_pdl(pick_kernel<DT, kSmallPick>, dim3(a.n), dim3(kSmallPick), 0, s, a)
            : launch_pdl(pick_kernel<DT, kPickThreads>, dim3(a.n), dim3(kPickThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(refine_kernel<DT>, dim3(sms), dim3(kPickThreads), 0, s, a);
}

bool beam_sizes_ok(int n, int beams, int vocab, int n_out)
{
    return n >= 1 && n <= (1 << 20) && beams >= 1 && beams <= kMaxBeams && vocab >= 1 && vocab <= kBeamMaxVocab &&
           n_out >= 1 && n_out <= kMaxOut && n_out <= (long long)beams * vocab &&
           (long long)n * beams <= (1 << 22) && (long long)n * beams * ((long long)vocab / Elem<1>::kChunk + 2) < (1LL << 31);
}

// ---------------------------------------------------------------------------
// State rows follow their parents.
// ---------------------------------------------------------------------------
constexpr int kReorderThreads = 256;

struct ReorderArgs {
    const char* src;
    char* dst;
    int64_t src_item, src_beam, dst_item, dst_beam;   // bytes
    int64_t units;                                    // of a row
    int beams_in, beams_out, in_place;
    const int32_t* parents;
    int32_t* status;
};

// A CTA has some units of every row of its item, so what it reads of the old rows
// is read before it writes any of them and nobody else does either: in place needs
// no second copy of the state.  A thread has a unit of up to ROWS rows in registers
// (with more rows SHARE threads share a unit's, and a barrier stands between their
// reads and writes).  HBM bounds it: 16 x 8 rows of 1 MB, half of them moving,
// in 20.8 to 22.1 us over several boxes (5.7 to 6.1 TB/s of rows moved, 85 to 90% of
// the copy bandwidth); 32 x 8 histories of 4 KB in 2.3 us of the GPU, 7.9 with the host.
template <typename R, int ROWS, int SHARE>
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const __grid_constant__ ReorderArgs a)
{
    constexpr int kWide = kReorderThreads / SHARE;
    __shared__ int32_t parent[kMaxBeams];
    pdl_enter();
    const int64_t item = blockIdx.y;
    for (int i = threadIdx.x; i < a.beams_out; i += kReorderThreads) {
        int p = a.parents[item * a.beams_out + i];
        if (p < 0 || p >= a.beams_in) {
            if (a.status && blockIdx.x == 0) atomicOr(&a.status[item], kBadLayout);
            p = -1;
        } else if (a.in_place && p == i) {
            p = -1;
        }
        parent[i] = p;
    }
    __syncthreads();
    const int64_t u = (int64_t)blockIdx.x * kWide + threadIdx.x % kWide;
    if (SHARE == 1 && u >= a.units) return;
    const char* src = a.src + item * a.src_item + u * (int64_t)sizeof(R);
    char* dst = a.dst + item * a.dst_item + u * (int64_t)sizeof(R);
    const int rows = u < a.units ? a.beams_out : 0;
    for (int i0 = (int)threadIdx.x / kWide * ROWS; i0 < a.beams_out || SHARE > 1; i0 += ROWS) {   // in place one turn does
        R x[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (i0 + i < rows && parent[i0 + i] >= 0) x[i] = *reinterpret_cast<const R*>(src + parent[i0 + i] * a.src_beam);
        if (SHARE > 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (i0 + i < rows && parent[i0 + i] >= 0) *reinterpret_cast<R*>(dst + (i0 + i) * a.dst_beam) = x[i];
        if (SHARE > 1) return;
    }
}

template <typename R, int ROWS, int SHARE>
cudaError_t launch_reorder(ReorderArgs a, int n, int64_t row_bytes, cudaStream_t s)
{
    a.units = row_bytes / (int64_t)sizeof(R);
    constexpr int kWide = kReorderThreads / SHARE;
    return launch_pdl(reorder_kernel<R, ROWS, SHARE>, dim3((unsigned)((a.units + kWide - 1) / kWide), n), dim3(kReorderThreads),
                      0, s, a);
}
template <typename R>
cudaError_t launch_reorder_rows(const ReorderArgs& a, int n, int64_t row_bytes, cudaStream_t s)
{
    const int rows = a.in_place ? a.beams_out : 1;
    if (rows <= 8) return launch_reorder<R, 8, 1>(a, n, row_bytes, s);
    if (rows <= 16) return launch_reorder<R, 16, 1>(a, n, row_bytes, s);
    if (rows <= 32) return launch_reorder<R, 16, 2>(a, n, row_bytes, s);
    if (rows <= 64) return launch_reorder<R, 16, 4>(a, n, row_bytes, s);
    return launch_reorder<R, 16, 8>(a, n, row_bytes, s);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t sv_beam_workspace_size(int n, int beams, int vocab, int n_out)
{
    return beam_sizes_ok(n, beams, vocab, n_out) ? beam_layout(n, beams, vocab).total : 0;
}

extern "C" sv_status_t sv_beam_select(const void* logits, sv_dtype_t dt, int64_t stride_item, int64_t stride_beam, int n,
                                      int beams, int vocab, const float* scores, const uint8_t* finished, int end_token,
                                      int n_out, int32_t* out_tokens, int32_t* out_parents, float* out_scores,
                                      int32_t* status, void* ws, size_t ws_bytes, sv_stream_t stream)
{
    if (n < 0 || beams < 1 || vocab < 1 || n_out < 1 || (long long)n_out > (long long)beams * vocab ||
        (dt != SV_DTYPE_BF16 && dt != SV_DTYPE_F32) || (finished && (end_token < 0 || end_token >= vocab)))
        return SV_ERR_INVALID_ARG;
    if (n == 0) return SV_OK;
    if (!logits || !scores || !out_tokens || !out_parents || !out_scores ||
        !aligned_to(logits, dt == SV_DTYPE_BF16 ? 2 : 4))
        return SV_ERR_INVALID_ARG;
    if (!beam_sizes_ok(n, beams, vocab, n_out)) return SV_ERR_UNSUPPORTED;
    const BeamLayout L = beam_layout(n, beams, vocab);
    if (!ws || !aligned_to(ws, 256) || ws_bytes < L.total) return SV_ERR_WORKSPACE;
    char* w = static_cast<char*>(ws);
    BeamArgs a{};
    a.logits = logits;
    a.stride_item = stride_item;
    a.stride_beam = stride_beam;
    a.n = n;
    a.beams = beams;
    a.vocab = vocab;
    a.n_out = n_out;
    a.end_token = end_token;
    a.scores = scores;
    a.finished = finished;
    a.out_tokens = out_tokens;
    a.out_parents = out_parents;
    a.out_scores = out_scores;
    a.status = status;
    a.n_flagged = reinterpret_cast<int32_t*>(w + L.head);
    a.item_units = reinterpret_cast<int32_t*>(w + L.item_units);
    a.item_done = reinterpret_cast<int32_t*>(w + L.item_done);
    a.item_list = reinterpret_cast<int32_t*>(w + L.item_list);
    a.item_mask = reinterpret_cast<uint32_t*>(w + L.item_mask);
    a.flagged = reinterpret_cast<int32_t*>(w + L.flagged);
    a.rec = reinterpret_cast<BeamRec*>(w + L.rec);
    a.base = reinterpret_cast<double*>(w + L.base);
    a.sums = reinterpret_cast<float2*>(w + L.sums);
    a.chunk_max = reinterpret_cast<float*>(w + L.chunk_max);
    a.list_logit = reinterpret_cast<float*>(w + L.list_logit);
    a.list_flat = reinterpret_cast<int32_t*>(w + L.list_flat);
    a.refined = reinterpret_cast<ulonglong2*>(w + L.refined);
    const cudaError_t e = dt == SV_DTYPE_BF16 ? launch_select<0>(a, stream) : launch_select<1>(a, stream);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status_t sv_beam_reorder(const void* src, int64_t src_stride_item, int64_t src_stride_beam, void* dst,
                                       int64_t dst_stride_item, int64_t dst_stride_beam, int64_t row_bytes, int n,
                                       int beams_in, int beams_out, const int32_t* parents, int32_t* status,
                                       sv_stream_t stream)
{
    const bool in_place = src == dst;
    if (n < 0 || beams_in < 1 || beams_out < 1 || row_bytes < 0 ||
        (in_place && (beams_in != beams_out || src_stride_item != dst_stride_item || src_stride_beam != dst_stride_beam)))
        return SV_ERR_INVALID_ARG;
    if (n == 0 || row_bytes == 0) return SV_OK;
    if (!src || !dst || !parents) return SV_ERR_INVALID_ARG;
    if (n > 65535 || beams_in > kMaxBeams || beams_out > kMaxBeams || row_bytes > (1LL << 36)) return SV_ERR_UNSUPPORTED;
    ReorderArgs a{};
    a.src = static_cast<const char*>(src);
    a.dst = static_cast<char*>(dst);
    a.src_item = src_stride_item;
    a.src_beam = src_stride_beam;
    a.dst_item = dst_stride_item;
    a.dst_beam = dst_stride_beam;
    a.beams_in = beams_in;
    a.beams_out = beams_out;
    a.in_place = in_place;
    a.parents = parents;
    a.status = status;
    // the widest access that every row allows
    const uint64_t all = (uint64_t)(uintptr_t)src | (uint64_t)(uintptr_t)dst | (uint64_t)src_stride_item |
                         (uint64_t)src_stride_beam | (uint64_t)dst_stride_item | (uint64_t)dst_stride_beam |
                         (uint64_t)row_bytes;
    cudaError_t e;
    if (all % 16 == 0) e = launch_reorder_rows<uint4>(a, n, row_bytes, stream);
    else if (all % 8 == 0) e = launch_reorder_rows<uint2>(a, n, row_bytes, stream);
    else if (all % 4 == 0) e = launch_reorder_rows<uint32_t>(a, n, row_bytes, stream);
    else if (all % 2 == 0) e = launch_reorder_rows<uint16_t>(a, n, row_bytes, stream);
    else e = launch_reorder_rows<uint8_t>(a, n, row_bytes, stream);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
