// sv_attn_tc.cu -- paged attention of bf16 and fp16 heads of 64 or 128 on the
// 5th-generation tensor cores.
//
// Rows.  The query heads of a key head share its keys, so a request's window
// of n tokens and a group of G heads is one matrix of n G rows (row = token G
// + head) per key head.  An item is up to 256 rows of it against the keys they
// see (128 rows where few keys are seen, kNarrowWindow), in tiles of 128 keys.
// An item's tiles are its cost.
//
// Split.  The items of a call, one after the other, are a line of tiles; CTA b
// of B takes tiles [b T / B, (b + 1) T / B) of it, wherever items begin and
// end.  Every CTA so does the same work, for one request of a million keys as
// for hundreds of short ones, with no host knowledge of the lengths.  An item
// that lies in one CTA is written at once; the pieces of the others go to the
// workspace in fp32 with their maximum and sum, and a second kernel joins them
// in the order of the line.
//
// Inside a CTA (one per SM, 16 warps).  Warp 0 walks over the CTA's part of the
// line and loads Q; warp 2 loads key and value tiles by TMA, a box a page, into
// a ring; warps 1 and 3 issue the matrix products of a slot each; two groups of
// four warps are the slots, which turn scores into weights, a thread a row; the
// last four warps write outputs.  A slot has its own scores S and output O in
// TMEM.  An item of more than 128 rows gives each slot half of the rows and both
// read every tile, taking turns at the tensor core, so that one slot makes its
// weights during the other's products; an item of up to 128 rows gives both
// slots all of its rows and every other tile, and the slots' results are joined
// at its end.  The weights P are the left operand of P V from TMEM, so neither
// S nor P ever passes through shared memory: heads of 128 leave room for P only
// in the place of S, heads of 64 have it apart, and their next scores are made
// while the weights are.
//
// What bounds it (one GB300).  Few rows: HBM.  4 requests x 8 tokens x 64 heads
// over 65,536 to 131,072 keys read 1.64 GB in 242 us, 6.78 TB/s, the measured copy
// bandwidth; 64 single tokens over 256 to 8,192 keys take 108 us for 0.61 GB (83%
// of it: some 7 us of the call are its start and the join), 256 ragged windows
// over 128 to 4,096 keys 219 us for 1.23 GB (83%).  Many rows: the chain scores,
// weights, P V, scores of a slot.  Chunks of 2,048 tokens over 8,192 and 16,384
// keys take 0.53 ms (1,430 TFLOP/s, 75% of cuBLAS' burst rate) in a burst and
// 0.56 ms at the card's power limit.  Short items (ragged prompts under a sliding
// window of 512, 52 us) are bound by latencies: start, the first instruction
// fetches, a turn of the chain a tile.
//
// Statistics.  m and l are fp32, one row a thread.  O is rescaled only when a
// row's maximum grows by more than 2^8: weights are then below 2^8 instead of
// 1, which fp32 sums and bf16 weights take without loss; fp16 weights are kept
// 2^7 times larger, away from fp16's subnormals.  Weights are rounded to the
// type of the values because that is what the tensor core multiplies; l sums
// them before the rounding.
//
// What is not seen.  Scores of hidden keys are replaced by -inf, whatever they
// are.  A hidden key's value would still meet weight 0, and 0 times NaN is NaN:
// in tiles with hidden keys the slots write zeros over the values that no row
// of the item sees, and if a value that only some rows see is not finite they
// do that tile's P V themselves, in fp32, leaving out weights of 0.
#include <cuda.h>
#include <float.h>
#include <limits.h>

#include <atomic>
#include <type_traits>

#include "sv_attn.cuh"

namespace sv {
namespace {

constexpr int kTile = 128;              // keys of a tile, rows of a slot
constexpr int kTcThreads = 512;
constexpr int kTcWarps = kTcThreads / 32;
constexpr uint32_t kTmemCols = 512;
// Caches of up to so many tiles (by the width of the page table) are not split:
// a second kernel costs 3 us of the host and as much of the GPU, a tile 1.5.
constexpr int kWholeTiles = 4;

// Without shared heads an item's rows are as many tokens, each with keys of its
// own: where few tiles are seen, items of 128 rows (slots take tiles by turns)
// spare a good part of them against 256 (a slot's rows its own, every tile both
// slots').  So it is up to these windows or, without one, caches of more than
// one item.  us with 128 and 256 rows, 16 heads of 64: 64 prompts of 200-600
// tokens, window 64 133 and 170, window 512 174 and 198; one of 8,000, window
// 640 77 and 83, window 1,024 94 and 95; 32 whole prompts of 640 108 and 133,
// 8 of 1,000 62 and 71; but 64 of 200 67 and 58.  With two query heads a key
// head the same long prompts were slower with 128 rows (60 to 50, window 128).
constexpr int kNarrowWindow = 640;
constexpr int kNarrowCache = 1024;

// ---- PTX ---------------------------------------------------------------------
__device__ __forceinline__ void tc_alloc(uint32_t* where)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_free(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTmemCols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The barrier's phase completes when every product issued so far has.
__device__ __forceinline__ void tc_commit(unsigned long long* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// D (TMEM) (+)= A B^T, A and B in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// The same with A in TMEM.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

#define SV_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), \
                    "=r"(r[o + 6]), "=r"(r[o + 7])
#define SV_W8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), \
                    "r"(r[o + 6]), "r"(r[o + 7])
// 32 columns of the warp's 32 lanes, a lane's columns to a thread.
__device__ __forceinline__ void tc_ld32(uint32_t* r, uint32_t addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24)
        : "r"(addr)
        : "memory");
}
#define SV_P8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), \
                    "+r"(r[o + 6]), "+r"(r[o + 7])
// Waits for the thread's loads; the N registers are not to be read before.
template <int N>
__device__ __forceinline__ void tc_loaded(uint32_t* r)
{
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < N; i += 8) asm volatile("" : SV_P8((r + i), 0));
}
__device__ __forceinline__ void tc_ld16(uint32_t* r, uint32_t addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : SV_R8(r, 0), SV_R8(r, 8)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_st32(const uint32_t* r, uint32_t addr)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::SV_W8(r, 0),
        SV_W8(r, 8), SV_W8(r, 16), SV_W8(r, 24), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_st16(const uint32_t* r, uint32_t addr)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::SV_W8(r, 0),
        SV_W8(r, 8), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_ld8(uint32_t* r, uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : SV_R8(r, 0)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tc_st8(const uint32_t* r, uint32_t addr)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::SV_W8(r, 0), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t tc_ld1(uint32_t addr)
{
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr) : "memory");
    return r;
}
// Some tokens' rows of 64 elements of a group's heads.
__device__ __forceinline__ void tma_q(uint32_t dst, const CUtensorMap* map, int e, int head, int token,
                                      unsigned long long* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(map), "r"(e), "r"(head), "r"(token), "r"(smem_u32(bar))
        : "memory");
}
// A page's rows of one head, or 128 of them, in one box (see make_map).
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int e, int group, int page,
                                         unsigned long long* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(e), "r"(0), "r"(group), "r"(page), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Shared-memory descriptor of 128-byte swizzled rows of 64 16-bit elements in
// groups of 8 rows, `group` bytes apart; `next64` is the distance from one block
// of 64 to the next where the operand's row axis is the contiguous one.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t group, uint32_t next64 = 16)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(next64 >> 4) << 16 | (uint64_t)(group >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp32 accumulators, both operands of one 16-bit type.
__device__ __forceinline__ constexpr uint32_t instr_desc(bool bf16, bool b_rows_contiguous, int n)
{
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_rows_contiguous ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(kTile >> 4) << 24;
}

template <typename T>
struct Kind;
template <>
struct Kind<__nv_bfloat16> {
    static constexpr bool kBf16 = true;
    static constexpr float kBias = 0.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t x)
    {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    static constexpr uint32_t kExpMask = 0x7f80u;   // all ones: infinite or NaN
};
template <>
struct Kind<__half> {
    static constexpr bool kBf16 = false;
    static constexpr float kBias = 7.f;             // log2 of what weights are multiplied by
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t x)
    {
        return __half22float2(*reinterpret_cast<const __half2*>(&x));
    }
    static constexpr uint32_t kExpMask = 0x7c00u;
};

// ---- the line of tiles -----------------------------------------------------------
// x / d for 0 <= x < 2^31 by a multiplication: m = ceil(2^(31 + L) / d) with
// 2^L >= d is off by less than d in 2^(31 + L), so x m / 2^(31 + L) by less than
// 1 / d, which does not reach the next whole number.
struct Divisor {
    uint32_t m, shift;
    __device__ __forceinline__ int operator()(int x) const { return (int)((uint64_t)(uint32_t)x * m >> shift); }
};

struct TcArgs {
    AttnArgs a;
    Divisor by_group, by_page;
    float* part;            // [2 grid][part_rows][D] pieces of items
    float2* part_ml;        // [2 grid][part_rows] their maximum (log2) and sum
    int4* rec;              // [grid][2] what each CTA left there; y of the first: a wait of it gave up
    int part_rows;
    int lanes_shift;        // log2 of the lanes that count a request's tiles
    int item_shift;         // log2 of an item's rows: 8, or 7 where few keys are seen (kNarrowWindow)
    int grid;
    int whole;              // items are not split: each counts as one tile of the line
    unsigned long long inv_grid;   // ceil(2^64 / grid)
    int q_tokens;           // tokens of a box of Q's map, 0: the output warps load Q
    float scale_log2;       // scale log2 e
};

// A request's window as rows and items.
struct Window {
    int n, len, t0, rows, items, shift;
    __device__ __forceinline__ int row0(int item) const { return item << shift; }
    __device__ __forceinline__ int item_rows(int item) const { return min(rows - row0(item), 1 << shift); }
};
__device__ __forceinline__ Window window_of(const TcArgs& t, int r, bool report)
{
    const AttnArgs& a = t.a;
    Window w;
    w.t0 = a.qo_indptr[r];
    const int t1 = a.qo_indptr[r + 1];
    w.len = a.kv_len[r];
    const bool on_axis = w.t0 >= 0 && t1 >= w.t0 && t1 <= a.tokens;
    w.n = on_axis ? t1 - w.t0 : 0;
    const bool bad = !on_axis || w.n > a.max_window || w.len < 0 ||
                     (long long)w.len > (long long)a.cache.max_pages * a.cache.page_size;
    if (bad) {
        if (report && a.status) atomicOr(&a.status[r], kBadLayout);
        w.n = 0;
    }
    w.rows = w.n * a.group;
    w.shift = t.item_shift;
    w.items = (w.rows + (1 << w.shift) - 1) >> w.shift;
    return w;
}
// Keys [lo, hi) that the row of token i of a window sees.  A position may be
// negative and a limit as large as an int: their difference is formed only where
// the limit hides something.
template <typename W>
__device__ __forceinline__ int2 seen(const AttnArgs& a, const W& w, int i)
{
    const int pos = w.len - w.n + i;
    const int hi = a.full ? w.len : max(0, pos + 1);
    const int lo = a.window_keys > 0 && pos >= a.window_keys ? pos - a.window_keys + 1 : 0;
    return make_int2(min(lo, hi), hi);
}
// Key tiles [x, y) of an item; at least one, so that an item without keys is
// still somebody's to write.
__device__ __forceinline__ int2 item_tiles(const TcArgs& t, const Window& w, int item)
{
    const int first = t.by_group(w.row0(item)), last = t.by_group(w.row0(item) + w.item_rows(item) - 1);
    const int lo = seen(t.a, w, first).x, hi = seen(t.a, w, last).y;
    const int x = lo / kTile;
    return make_int2(x, max((hi + kTile - 1) / kTile, x + 1));
}
__device__ __forceinline__ int item_cost(const TcArgs& t, const Window& w, int item)
{
    const int2 x = item_tiles(t, w, item);
    return t.whole ? 1 : x.y - x.x;
}

// A piece of an item: the part of the line one CTA has of it.
struct Piece {
    int r, head, item;
    int row0, rows;         // the item's rows among the window's
    int kt0, nt;            // first key tile and their number; 0: no row sees a key, -1: no more pieces
    int first, last;        // the item's first and last tile are in it
    int t0, n, len;         // the window's first token, its length, the request's cached tokens
    int key_lo, key_hi;     // keys that some row of the item sees
    int all_lo, all_hi;     // keys that every row of it sees
    int lead;               // the slot that has the first tile where tiles alternate

    // An item of more than 128 rows: each slot has rows of its own and every
    // tile; otherwise both have all the rows and every other tile.  A unit is
    // one slot's work on one tile; unit u is slot u & 1's.
    __device__ __forceinline__ bool pair() const { return rows > kTile; }
    __device__ __forceinline__ int steps(int slot) const { return pair() ? nt : (nt + 1 - (slot ^ lead)) >> 1; }
};

// Walks over a CTA's part of the line.
struct Walk {
    long long left;            // tiles still to come
    int r, head, item, done;   // done: tiles of the item behind
    Window w;
    int2 tiles;

    __device__ __forceinline__ void next(const TcArgs& t, Piece& p)
    {
        if (left <= 0) {
            p.nt = -1;
            return;
        }
        const int have = t.whole ? 1 : tiles.y - tiles.x;
        p.r = r;
        p.head = head;
        p.item = item;
        p.row0 = w.row0(item);
        p.rows = w.item_rows(item);
        p.kt0 = tiles.x + done;
        const int nt = (int)min((long long)(have - done), left);
        p.first = done == 0;
        const bool last = done + nt == have;
        p.last = last;
        p.t0 = w.t0;
        p.n = w.n;
        p.len = w.len;
        const int2 top = seen(t.a, w, t.by_group(p.row0)), bottom = seen(t.a, w, t.by_group(p.row0 + p.rows - 1));
        p.key_lo = top.x;
        p.key_hi = bottom.y;
        p.all_lo = bottom.x;
        p.all_hi = top.y;
        p.nt = bottom.y <= top.x ? 0 : t.whole ? tiles.y - tiles.x : nt;
        left -= nt;
        done += nt;
        if (last && left > 0) {
            done = 0;
            if (++item == w.items) {
                item = 0;
                if (++head == t.a.cache.k.heads) {
                    head = 0;
#pragma unroll 1
                    do {
                        if (++r >= t.a.n_req) {                 // not reached: tiles are left
                            left = 0;
                            return;
                        }
                        w = window_of(t, r, false);
                    } while (w.items == 0);
                }
            }
            tiles = item_tiles(t, w, item);
        }
    }
};

// ---- shared memory ----------------------------------------------------------------
constexpr int kPieces = 4;
constexpr int kPieceReaders = 15;   // warps: loads, two slots' products, two slots, output

template <int D>
struct TcSmem {
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kTileBytes = kTile * D * 2;
    // Q: blocks of 64 elements one after the other, 128 rows each.  Keys and values: groups of 8 keys one after the
    // other, each with its blocks of 64 elements (1 KB a block), so that one box of a map fills a page's place.
    static constexpr int kGroup = 1024 * (D / 64);
    static constexpr bool kApart = D == 64;   // TMEM has room for weights beside the scores, after the slot's output
    static constexpr int kWeightsAt = kApart ? 256 + 64 : 0;   // their column, for slot 0
    alignas(1024) unsigned char q[2][kTileBytes];
    alignas(1024) unsigned char kv[kStages][kTileBytes];
    static __device__ __forceinline__ int kv_at(int key, int vec)   // of 8 elements
    {
        return (key >> 3) * kGroup + (vec >> 3) * 1024 + (key & 7) * 128 + ((vec ^ key) & 7) * 16;
    }
    unsigned long long full[kStages], empty[kStages];
    unsigned long long q_full[2], q_empty[2], s_full[2], s_free[2], p_full[2], pv_done[2], o_free[2], ml_full[2], vote[2], drain[2];
    unsigned long long piece_full[kPieces], piece_empty[kPieces];
    Piece pieces[kPieces];          // warp 0 walks ahead of the other roles
    float2 ml[2][kTile];            // the slots' statistics of a finished piece
    long long scan[kTcWarps];
    Walk start;
    uint32_t tmem;
    uint32_t turns[2];              // units of shared tiles whose products each slot has issued
    uint32_t issued;                // ring entries whose loads have begun
    uint32_t q_issued[2];           // loads of each buffer of Q begun (TMA)
    uint32_t q_loads[2];            // warps that have filled each buffer of Q, over all its loads (output warps)
    int odd[2][3];                  // a slot's votes, three by turns: some value is not finite
    int aborted;                    // a wait gave up: every later wait gives up at once
    int by_hand[2];                 // the slot has done this tile's P V itself
};

// Polls of a wait before it gives up.  A build that sets it low, for tests, does
// not sleep between them.
#ifdef SV_ATTN_WAIT_POLLS
constexpr int kPolls = SV_ATTN_WAIT_POLLS;
#define SV_POLL "mbarrier.test_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
#else
constexpr int kPolls = (int)kWaitPolls;
#define SV_POLL "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
#endif

// A bounded wait.  After one that gave up the CTA runs to its end without
// waiting; every row of the call is then written with NaN by it (other CTAs may
// write theirs over that), items that it has a piece of are NaN after the join,
// and every request's status gets SV_ROW_TIMEOUT.  From then on nothing that is
// in use may change hands: no piece is written and no load begun (a stage or a
// piece that seems free may not be).
__device__ __forceinline__ void wait_or_abort(unsigned long long* bar, uint32_t parity, int* aborted)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .u32 n, a;\n\tmov.u32 n, %3;\n"
        "again_%=:\n\t"
        SV_POLL
        "@p bra done_%=;\n\t"
        "ld.volatile.shared.u32 a, [%2];\n\t"
        "setp.ne.u32 p, a, 0;\n\t"
        "@p bra done_%=;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 p, n, 0;\n\t"
        "@p bra again_%=;\n\t"
        "mov.u32 a, 1;\n\t"
        "st.volatile.shared.u32 [%2], a;\n"
        "done_%=:\n\t}" ::"r"(smem_u32(bar)),
        "r"(parity), "r"(smem_u32(aborted)), "n"(kPolls)
        : "memory");
}

// A count in shared memory that is given with what was done before it, and read
// before what relies on that.
__device__ __forceinline__ void give_count(uint32_t* count, uint32_t n)
{
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(count)), "r"(n) : "memory");
}
__device__ __forceinline__ uint32_t take_count(const uint32_t* count)
{
    uint32_t n;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(n) : "r"(smem_u32(count)) : "memory");
    return n;
}

__device__ __forceinline__ uint32_t mbar_test(unsigned long long* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok;
}

// Where the ring holds a piece's tiles: the keys of the first `ahead` tiles,
// then values of tile j and keys of tile j + ahead, j = 0, 1, ...
__device__ __forceinline__ uint32_t entry_v(int j, int nt, int ahead)
{
    return (uint32_t)(min(ahead, nt) + j + max(0, min(j, nt - ahead)));
}
__device__ __forceinline__ uint32_t entry_k(int j, int ahead) { return (uint32_t)(j < ahead ? j : 2 * j - ahead + 1); }

// Bits lo .. hi - 1 of 32.
__device__ __forceinline__ uint32_t columns_seen(int lo, int hi)
{
    const uint32_t below_hi = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u;
    return lo >= 32 ? 0u : lo <= 0 ? below_hi : below_hi & (0xffffffffu << lo);
}
__device__ __forceinline__ bool one_lane()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0u;
}
// threadIdx.x read anew, where keeping it would cost a register all along.
__device__ __forceinline__ int thread_now()
{
    int x;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(x));
    return x;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c)
{
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b)
{
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ unsigned long long pair_of(float lo, float hi)
{
    unsigned long long d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 halves(unsigned long long x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}

// The code is kept small on purpose (one copy of every step, loops that are not
// unrolled): the roles run different parts of it at the same time, and at
// 195 KB, with the steps inlined wherever they occur, instruction misses took
// most of the time of short items (256 ragged windows: 523 us, 272 at 68 KB).
// PAIRS: items of more than 128 rows may come; without their code the same took
// 223 us instead of 242.  Each variant has one way through the scores: with them
// a row is held in registers whole (prompt chunks 582 us for 633), without them
// 64 columns at a time in less code.  A kernel with both, whole rows for pieces of
// 16 tiles or more, took 75 us of a prompt of 3,000 tokens x 16 heads of 64 (4 a
// key head), now 66; 102 of four of 300-2,000 under a window of 2,048, now 88;
// prompt chunks the same.
template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ TcArgs t, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q)
{
    using S = TcSmem<D>;
    constexpr uint32_t kStages = S::kStages;
    extern __shared__ __align__(1024) unsigned char raw[];
    S& sm = *reinterpret_cast<S*>(raw);
    const AttnArgs& a = t.a;
    const int tid = (int)threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (warp == 3) {                               // a lane a barrier of every kind
        if (lane < (int)kStages) {
            mbar_init(&sm.full[lane], 1);
            mbar_init(&sm.empty[lane], 2);         // 2: each slot's products, or twice the one slot's
        }
        if (lane < kPieces) {
            mbar_init(&sm.piece_full[lane], 1);
            mbar_init(&sm.piece_empty[lane], kPieceReaders);
        }
        if (lane < 2) {
            mbar_init(&sm.q_full[lane], 1);
            mbar_init(&sm.q_empty[lane], 2);
            mbar_init(&sm.s_full[lane], 1);
            mbar_init(&sm.s_free[lane], 4);
            mbar_init(&sm.p_full[lane], 4);        // 4: a warp at a time
            mbar_init(&sm.pv_done[lane], 1);
            mbar_init(&sm.o_free[lane], 4);
            mbar_init(&sm.ml_full[lane], 4);
            mbar_init(&sm.vote[lane], 4);
            mbar_init(&sm.drain[lane], 1);
            sm.q_loads[lane] = sm.q_issued[lane] = sm.turns[lane] = 0;
            sm.by_hand[lane] = 0;
            sm.odd[lane][0] = sm.odd[lane][1] = sm.odd[lane][2] = 0;
        }
        if (lane == 0) {
            sm.aborted = 0;
            sm.issued = 0;
            sm.start.left = 0;
        }
        mbar_fence_init();
    }
    if (warp == 2 && lane < 3) {
        const CUtensorMap* map = lane == 0 ? &map_k : lane == 1 ? &map_v : &map_q;
        if (lane < 2 || t.q_tokens) asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    if (warp == 1) tc_alloc(&sm.tmem);
    pdl_enter();

    // The CTA's part of the line: the tiles of every request summed, a few
    // lanes a request where there are few, then the request its part begins in.
    long long total = 0, per_head = 0, incl = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        long long begin = 0, end = 0;
        if (pass == 1) {
            // Two tiles (or one item) a CTA at least; else total / grid by the high word of a product, no division.
            const int least = t.whole ? 1 : 2;
            const bool few = total < (long long)least * t.grid;
            const int b = few ? max(1, (int)total / least) : t.grid, x = (int)blockIdx.x;
            if (x >= b) break;
            const long long each = few ? min(total, (long long)least)
                                       : (long long)__umul64hi((unsigned long long)total, t.inv_grid);
            const int more = (int)(total - each * b);          // the first CTAs have one tile more
            begin = each * x + min(x, more);
            end = begin + each + (x < more);
            if (end <= begin) break;
        }
        long long before = 0;
#pragma unroll 1
        for (int r0 = 0; r0 < a.n_req; r0 += kTcThreads >> t.lanes_shift) {
            const int r = r0 + (tid >> t.lanes_shift), lanes = 1 << t.lanes_shift, sub = tid & (lanes - 1);
            if (pass == 0 || a.n_req > kTcThreads) {
                per_head = 0;
                if (r < a.n_req) {
                    const Window w = window_of(t, r, pass == 0 && blockIdx.x == 0);
#pragma unroll 1
                    for (int i = sub; i < w.items; i += lanes) per_head += item_cost(t, w, i);
                }
#pragma unroll 1
                for (int x = 1; x < lanes; x <<= 1) per_head += __shfl_xor_sync(0xffffffffu, per_head, x);
                if (sub != 0) per_head = 0;              // counted once
                incl = per_head * a.cache.k.heads;
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, incl, x);
                    if (lane >= x) incl += y;
                }
                __syncthreads();
                if (lane == 31) sm.scan[warp] = incl;
                __syncthreads();
                long long upto = lane < kTcWarps ? sm.scan[lane] : 0;      // the warps' sums, every warp for itself
#pragma unroll
                for (int x = 1; x < kTcWarps; x <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, upto, x);
                    if (lane >= x) upto += y;
                }
                const long long chunk = __shfl_sync(0xffffffffu, upto, kTcWarps - 1);
                const long long below = __shfl_sync(0xffffffffu, upto, (warp - 1) & 31);
                if (warp > 0) incl += below;
                if (pass == 0) total += chunk;
                if (pass == 1) incl += before;
                before += chunk;
            }
            const long long mine = per_head * a.cache.k.heads;
            const uint32_t hit = __ballot_sync(0xffffffffu, pass == 1 && incl > begin && incl - mine <= begin);
            if (hit) {                                   // one lane of the CTA; its warp looks for the item
                const int src = __ffs((int)hit) - 1;
                const long long of_head = __shfl_sync(0xffffffffu, per_head, src);
                long long off = __shfl_sync(0xffffffffu, begin - (incl - mine), src);
                Walk k;
                k.left = end - begin;
                k.r = __shfl_sync(0xffffffffu, r, src);
                k.w = window_of(t, k.r, false);
                k.head = 0;
#pragma unroll 1
                for (; off >= of_head; ++k.head) off -= of_head;
#pragma unroll 1
                for (int i0 = 0; i0 < k.w.items; i0 += 32) {
                    k.item = i0 + lane;
                    const int cost = k.item < k.w.items ? item_cost(t, k.w, k.item) : 0;
                    int upto = cost;
#pragma unroll
                    for (int x = 1; x < 32; x <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, upto, x);
                        if (lane >= x) upto += y;
                    }
                    const uint32_t past = __ballot_sync(0xffffffffu, off < upto);
                    if (past) {
                        if (lane == __ffs((int)past) - 1) {
                            k.tiles = item_tiles(t, k.w, k.item);
                            k.done = (int)off - (upto - cost);
                            sm.start = k;
                        }
                        break;
                    }
                    off -= __shfl_sync(0xffffffffu, upto, 31);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    // Piece k of the CTA, for every lane of a reading warp; false after the last.
    auto piece_ready = [&](uint32_t k) {
        wait_or_abort(&sm.piece_full[k % kPieces], k / kPieces & 1u, &sm.aborted);
        return sm.pieces[k % kPieces].nt >= 0 && !*(volatile int*)&sm.aborted;
    };
    // A count in shared memory has reached n: the count.
    auto reached = [&](const uint32_t* count, uint32_t n) {
        uint32_t x = take_count(count);
#pragma unroll 1
        for (int i = 0; (int)(x - n) < 0; ++i) {
            if (i == kPolls) *(volatile int*)&sm.aborted = 1;
            if (*(volatile int*)&sm.aborted) break;
            x = take_count(count);
        }
        return x;
    };
    // The other slot has had so many turns: an order of the products, which hand nothing over.
    auto my_turn = [&](const uint32_t* turns, uint32_t n) {
#pragma unroll 1
        for (int i = 0; (int)(*(const volatile uint32_t*)turns - n) < 0; ++i) {
            if (i == kPolls) *(volatile int*)&sm.aborted = 1;
            if (*(volatile int*)&sm.aborted) break;
        }
    };
    // Entry e of the ring has landed.  A reader that skips entries cannot go by the stage's phase alone: with the
    // entry before e on that stage still to come, the phase of the one before that would pass for e's.
    uint32_t begun = 0;                             // entries known to have begun
    auto landed = [&](uint32_t e) {
        if ((int)(begun - e) <= 0) begun = reached(&sm.issued, e + 1);
        wait_or_abort(&sm.full[e % kStages], e / kStages & 1u, &sm.aborted);
    };
    auto landed_by_now = [&](uint32_t e) {
        begun = take_count(&sm.issued);             // first: before e has begun its stage's phase says nothing
        return __all_sync(0xffffffffu, (int)(begun - e) > 0 && mbar_test(&sm.full[e % kStages], e / kStages & 1u)) != 0;
    };
    auto warp_arrive = [&](unsigned long long* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    auto piece_release = [&](uint32_t k) { warp_arrive(&sm.piece_empty[k % kPieces]); };
    // The slots hold a row of 128 scores a thread, the other warps little: of
    // the 512 x 128 registers of the launch, 128 x 64 + 256 x 176 + 128 x 96.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 2) {
            // ---- loads: lane i has page i of a tile --------------------------------------
            const int page_size = a.cache.page_size;
            const int box_rows = min(page_size, kTile), per_tile = kTile / box_rows;   // pages of a tile, up to 16
            const int head_k = (int)a.cache.k.stride_head, head_v = (int)a.cache.v.stride_head;   // of heads, in elements
            const uint32_t lane_at = (uint32_t)(lane * box_rows / 8 * S::kGroup);                // of the lane's page
            const uint32_t box_bytes = (uint32_t)(box_rows * D * 2);
            uint32_t entry = 0, stage = 0, free_phase = 1;       // the ring; its first round finds it empty
#pragma unroll 1
            for (uint32_t pk = 0; piece_ready(pk); piece_release(pk++)) {
                const Piece& p = sm.pieces[pk % kPieces];
                const int nt = p.nt, key_lane = p.kt0 * kTile + lane * box_rows, key_lo = p.key_lo, key_hi = p.key_hi;
                const int x_k = p.head * head_k, x_v = p.head * head_v;
                const int32_t* table = a.cache.page_table + (int64_t)p.r * a.cache.ld_table;
                const int ahead = PAIRS && p.pair() ? 1 : 2;
                // Page numbers, a lane a page: 32 of them from tile `first` on, the 32 after those, and the 32 after
                // those on their way.  A lane's page of a tile is another lane's number.
                const int span = 32 / per_tile;               // tiles that 32 pages hold
                auto fetch = [&](int tile) -> int {
                    const int key = key_lane + tile * kTile;
                    if (tile + lane / per_tile >= nt || key >= key_hi || key + box_rows <= key_lo) return -1;
                    return table[t.by_page(key)];             // pages that nobody sees are not looked at
                };
                int first = 0, now = fetch(0), next = fetch(span), later = fetch(2 * span);
                // A tile's boxes.  `known`: its stage was seen to be free.  The barrier is told of the bytes by one lane
                // while the others issue: it waits for that lane's arrival whichever comes first.
                auto load = [&](const CUtensorMap* map, int j, int x, bool known) {
                    const int key = key_lane + j * kTile;
                    const bool mine = lane < per_tile && key < key_hi && key + box_rows > key_lo;
                    int page = __shfl_sync(0xffffffffu, j - first < span ? now : next, ((j - first) * per_tile + lane) & 31);
                    const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * box_bytes;
                    if (mine && (unsigned)page >= (unsigned)a.cache.n_pages) {
                        if (a.status) atomicOr(&a.status[p.r], kBadLayout);
                        page = a.cache.n_pages;                // past the end: reads as zeros
                    }
                    const int group = page_size > kTile ? (key - t.by_page(key) * page_size) >> 3 : 0;
                    if (!known) wait_or_abort(&sm.empty[stage], free_phase, &sm.aborted);
                    if (__any_sync(0xffffffffu, *(volatile int*)&sm.aborted)) return;
                    ++entry;
                    if (mine) tma_page(smem_u32(sm.kv[stage]) + lane_at, map, x, group, page, &sm.full[stage]);
                    if (lane == 0) {
                        mbar_expect_tx(&sm.full[stage], bytes);
                        give_count(&sm.issued, entry);
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        free_phase ^= 1u;
                    }
                };
#pragma unroll 1
                for (int u = -ahead; u < nt; ++u) {            // values of tile u, keys of tile u + ahead
                    const bool has_v = u >= 0;
                    const uint32_t other = stage + 1 == kStages ? 0 : stage + 1;
                    const uint32_t free0 = mbar_test(&sm.empty[stage], free_phase),
                                   free1 = mbar_test(&sm.empty[other], other ? free_phase : free_phase ^ 1u);
                    if (u == first + span) {
                        first += span;
                        now = next;
                        next = later;
                        later = fetch(first + 2 * span);
                    }
                    if (has_v) load(&map_v, u, x_v, free0);
                    if (u + ahead < nt) load(&map_k, u + ahead, x_k, has_v ? free1 : free0);
                }
            }
        } else if (warp != 0) {
            // ---- matrix products: warp 1 slot 0's, warp 3 slot 1's, one lane issues them -----
            const int s = warp >> 1;
            constexpr uint32_t kQk = instr_desc(Kind<T>::kBf16, false, kTile);
            constexpr uint32_t kPv = instr_desc(Kind<T>::kBf16, true, D);
            const uint64_t q_desc = smem_desc(smem_u32(sm.q[0]), 1024), k_desc = smem_desc(smem_u32(sm.kv[0]), S::kGroup),
                           v_desc = smem_desc(smem_u32(sm.kv[0]), S::kGroup, 1024);
            constexpr uint32_t kBytes = S::kTileBytes >> 4;    // a tile in a descriptor's units
            const uint32_t o_at = tmem + 256 + s * 128, s_at = tmem + s * kTile, p_at = s_at + S::kWeightsAt;
            uint32_t scores = 0, base = 0, q_uses[2] = {0, 0}, done = 0, o_uses = 0, q_next = 0, turns = 0;
#pragma unroll 1
            for (uint32_t pk = 0; piece_ready(pk); piece_release(pk++)) {
                const Piece& p = sm.pieces[pk % kPieces];
                const bool pair = PAIRS && p.pair();
                const int nt = p.nt, ahead = pair ? 1 : 2, each = pair ? 1 : 2, steps = p.steps(s);
                const uint32_t qb = pair ? (uint32_t)s : q_next;
                if (!pair && nt > 0) q_next ^= 1u;
                if (nt > 0) {
                    if (pair || qb == 0) ++q_uses[0];
                    if (pair || qb == 1) ++q_uses[1];
                    // A slot without steps does not wait: it would not hold the buffer, which may be two loads on.
                    const uint32_t use = qb ? q_uses[1] : q_uses[0];
                    if (steps > 0 && t.q_tokens) {
                        reached(&sm.q_issued[qb], use);
                        wait_or_abort(&sm.q_full[qb], (use - 1) & 1u, &sm.aborted);
                    } else if (steps > 0) {
                        reached(&sm.q_loads[qb], 4u * use);
                        __threadfence_block();
                    }
                }
                const uint64_t qd = q_desc + qb * kBytes;
                int j = pair ? 0 : s ^ p.lead;                   // tile of the next scores
                uint32_t e = base + entry_k(j, ahead), k_stage = e % kStages, v_stage = 0;
                bool edge = false;                               // the values' tile has hidden keys
#pragma unroll 1
                for (int st = 0; st <= steps; ++st) {
                    const uint64_t vd = v_desc + v_stage * kBytes, kd = k_desc + k_stage * kBytes;
                    auto score = [&]() {
                        if (S::kApart) wait_or_abort(&sm.s_free[s], ~scores++ & 1u, &sm.aborted);   // at first they are
                        tc_fence_after();
                        if (one_lane()) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t in = (uint32_t)(k % 4) * 32, block = (uint32_t)(k / 4);
                                tc_mma_ss(s_at, qd + ((block * kTile * 128 + in) >> 4), kd + ((block * 1024 + in) >> 4), kQk, k > 0);
                            }
                            tc_commit(&sm.s_full[s]);
                            tc_commit(&sm.empty[k_stage]);
                            if (!pair) tc_commit(&sm.empty[k_stage]);
                            if (st + 1 == steps) {               // Q's last use
                                tc_commit(&sm.q_empty[qb]);
                                if (pair || nt == 1) tc_commit(&sm.q_empty[qb]);
                            }
                        }
                        __syncwarp();
                    };
                    // Where the slots share the tiles, arithmetic bounds the piece: what can be waited for is, before
                    // the weights, so that nothing stands between the products.  Elsewhere the keys may be far off.
                    bool keys = st < steps && (pair || st == 0 || (S::kApart && landed_by_now(e)));
                    if (keys) landed(e);
                    const bool scored = keys && S::kApart;       // weights apart: the next scores need not wait for them
                    if (scored) score();
                    if (st > 0) {                                // P V of step st - 1
                        if (st == 1) wait_or_abort(&sm.o_free[s], ~o_uses++ & 1u, &sm.aborted);   // at first it is
                        wait_or_abort(&sm.p_full[s], done & 1u, &sm.aborted);
                        ++done;
                        const bool by_hand = edge && *(volatile int*)&sm.by_hand[s];
                        if (pair && !S::kApart) my_turn(&sm.turns[s ^ 1], turns++ + (uint32_t)s);
                        tc_fence_after();
                        if (one_lane()) {
                            if (by_hand) {
                                *(volatile int*)&sm.by_hand[s] = 0;   // before the commit that lets the slot set it again
                                __threadfence_block();
                            } else {
#pragma unroll
                                for (int k = 0; k < kTile / 16; ++k)
                                    tc_mma_ts(o_at, p_at + k * 8, vd + k * (2 * S::kGroup >> 4), kPv, st > 1 || k > 0);
                            }
                            tc_commit(&sm.pv_done[s]);
                            tc_commit(&sm.empty[v_stage]);
                            if (!pair) tc_commit(&sm.empty[v_stage]);
                        }
                        __syncwarp();
                    }
                    if (st < steps && !scored) {                 // scores of step st, in the place of the last weights
                        if (!keys) landed(e);
                        score();
                    }
                    if (pair && !S::kApart && st > 0 && lane == 0) *(volatile uint32_t*)&sm.turns[s] = turns;
                    if (st < steps) {                            // the values that go with these scores, the next keys
                        edge = (p.kt0 + j) * kTile < p.all_lo || (p.kt0 + j + 1) * kTile > p.all_hi;
                        const uint32_t ev = base + entry_v(j, nt, ahead);
                        v_stage = ev % kStages;
                        j += each;
                        e = base + entry_k(j, ahead);
                        k_stage = e % kStages;
                        landed(ev);
                    }
                }
                base += 2u * (uint32_t)nt;
            }
        } else {
            // ---- the walk over the CTA's pieces: one thread ----------------------------------
            if (lane == 0) {
                Walk walk = sm.start;
                uint32_t q_uses[2] = {0, 0}, q_next = 0;
                int lead = 0;
#pragma unroll 1
                for (uint32_t pk = 0;; ++pk) {
                    wait_or_abort(&sm.piece_empty[pk % kPieces], ~(pk / kPieces) & 1u, &sm.aborted);
                    if (*(volatile int*)&sm.aborted) break;            // its readers may not be through with it
                    Piece& p = sm.pieces[pk % kPieces];
                    walk.next(t, p);
                    p.lead = lead;                       // an odd tile is the one slot's, then the other's
                    if (!(PAIRS && p.pair()) && (p.nt & 1)) lead ^= 1;
                    const bool end = p.nt < 0;
                    const bool pair = PAIRS && p.pair();
                    const int bufs = p.nt <= 0 || !t.q_tokens ? 0 : pair ? 2 : 1;
                    const int q_head = p.head * a.group, q_token = p.t0 + t.by_group(p.row0);
                    mbar_arrive(&sm.piece_full[pk % kPieces]);
                    if (end) break;
                    // Its rows of Q; where slots share them, into the buffer the piece before does not use.  Rows past
                    // the box or the window are whatever lies there: rows of the products are independent.
#pragma unroll 1
                    for (int i = 0; i < bufs; ++i) {
                        const uint32_t qb = pair ? (uint32_t)i : q_next;
                        wait_or_abort(&sm.q_empty[qb], ~(qb ? q_uses[1] : q_uses[0]) & 1u, &sm.aborted);
                        if (*(volatile int*)&sm.aborted) break;
                        if (qb) ++q_uses[1]; else ++q_uses[0];
                        mbar_expect_tx(&sm.q_full[qb], (uint32_t)(t.q_tokens * a.group * D * 2));
                        give_count(&sm.q_issued[qb], qb ? q_uses[1] : q_uses[0]);
#pragma unroll
                        for (int x = 0; x < D; x += 64)
                            tma_q(smem_u32(sm.q[qb]) + (uint32_t)(x / 64 * kTile * 128), &map_q, x, q_head,
                                  q_token + i * t.q_tokens, &sm.q_full[qb]);
                    }
                    if (!pair && bufs) q_next ^= 1u;
                }
            }
            __syncwarp();
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        // ---- the slots: a thread a row ---------------------------------------------------
        const int slot = (warp - 4) >> 2, sw = warp & 3, row = sw * 32 + lane;
        const uint32_t lanes = (uint32_t)(sw * 32) << 16;
        const uint32_t s_at = tmem + lanes + slot * kTile, o_at = tmem + lanes + 256 + slot * 128, p_at = s_at + S::kWeightsAt;
        uint32_t steps_done = 0, o_uses = 0, votes = 0, base = 0;
#pragma unroll 1
        for (uint32_t pk = 0; piece_ready(pk); piece_release(pk++)) {
            const Piece& p = sm.pieces[pk % kPieces];
            float m = -INFINITY, l = 0.f;
            {
                const bool pair = PAIRS && p.pair();
                const int my_steps = p.steps(slot);
                const int local = (pair ? slot * kTile : 0) + row;     // row of the item
                const bool warp_valid = local - lane < p.rows;
                int2 see = make_int2(0, INT_MAX);                      // rows of nobody: no masking
                const bool valid = local < p.rows;
                if (valid) see = seen(a, p, t.by_group(p.row0 + local));
                int k0 = (p.kt0 + (pair ? 0 : slot ^ p.lead)) * kTile;
#pragma unroll 1
                for (int st = 0; st < my_steps; ++st, k0 += pair ? kTile : 2 * kTile) {
                    const bool edge = k0 < p.all_lo || k0 + kTile > p.all_hi;      // a tile with hidden keys
                    bool by_hand = false;
                    if (edge) {
                        // Its values as the products may read them, while the scores are on their way.
                        const uint32_t e = base + entry_v(k0 / kTile - p.kt0, p.nt, pair ? 1 : 2), stage = e % kStages;
                        landed(e);
                        unsigned char* vt = sm.kv[stage];
                        const int key = k0 + row;
                        if (key < p.key_lo || key >= p.key_hi) {
#pragma unroll 2
                            for (int c = 0; c < D / 8; ++c)        // in the swizzle's order: no two lanes in one bank
                                *reinterpret_cast<uint4*>(vt + S::kv_at(row, c)) =
                                    make_uint4(0, 0, 0, 0);
                        }
                        fence_async_smem();
                        // Keys that only some rows see: [key_lo, all_lo) and [all_hi, key_hi).
                        if (k0 < min(p.all_lo, p.key_hi) || (k0 < p.key_hi && k0 + kTile > p.all_hi && p.all_hi < p.key_hi)) {
                            uint32_t top = 0;                      // the largest magnitudes, as bits
                            if (key >= p.key_lo && key < p.key_hi && (key < p.all_lo || key >= p.all_hi)) {
#pragma unroll 2
                                for (int c = 0; c < D / 8; ++c) {
                                    const uint4 y = *reinterpret_cast<const uint4*>(vt + S::kv_at(row, c));
                                    top = __vmaxu2(__vmaxu2(top, y.x & 0x7fff7fffu), y.y & 0x7fff7fffu);
                                    top = __vmaxu2(__vmaxu2(top, y.z & 0x7fff7fffu), y.w & 0x7fff7fffu);
                                }
                            }
                            const bool bad = max(top & 0xffffu, top >> 16) >= Kind<T>::kExpMask;
                            // The slot's warps vote and wait for one another (bounded, as every wait: no hardware barrier).
                            const bool any_bad = __any_sync(0xffffffffu, bad);
                            if (any_bad && lane == 0) *(volatile int*)&sm.odd[slot][votes % 3u] = 1;
                            // The next vote's: all have read it two votes ago, nobody writes it before this vote is over.
                            if (row == 0) *(volatile int*)&sm.odd[slot][(votes + 1u) % 3u] = 0;
                            __threadfence_block();
                            warp_arrive(&sm.vote[slot]);
                            wait_or_abort(&sm.vote[slot], votes & 1u, &sm.aborted);
                            by_hand = *(volatile int*)&sm.odd[slot][votes % 3u] != 0;
                            ++votes;
                        }
                    }
                    wait_or_abort(&sm.s_full[slot], steps_done & 1u, &sm.aborted);
                    tc_fence_after();
                    const int lo = see.x - k0, hi = see.y - k0;                    // the row's columns
                    const bool nothing = __all_sync(0xffffffffu, see.x >= k0 + kTile || see.y <= k0);
                    const bool masked = __any_sync(0xffffffffu, see.x > k0 || see.y < k0 + kTile);
                    // A larger maximum: the sums so far under it.
                    auto grow = [&](float mx) {
                        const bool grows = valid && (mx - m) * t.scale_log2 > 8.f;   // from -inf: always, unless mx is -inf
                        if (!__any_sync(0xffffffffu, grows)) return false;
                        const float f = grows ? exp2_approx((m - mx) * t.scale_log2) : 1.f;
                        const bool some = __any_sync(0xffffffffu, grows && l != 0.f);   // a row without weights so far has O = 0
                        if (grows) {
                            m = mx;
                            l *= f;
                        }
                        if (st > 0 && some) {
                            wait_or_abort(&sm.pv_done[slot], (steps_done - 1) & 1u, &sm.aborted);
                            __syncwarp();                    // tensor memory is a whole warp's business
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 8) {
                                uint32_t o[8];
                                tc_ld8(o, o_at + c);
                                tc_loaded<8>(o);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tc_st8(o, o_at + c);
                            }
                        }
                        return true;
                    };
                    // Weights of 32 scores under the maximum m; their sums are added to l0 and l1.
                    unsigned long long l0 = 0, l1 = 0;
                    uint32_t w[16];
                    auto weigh = [&](const uint32_t* s) {
                        const float shift = Kind<T>::kBias - (m == -INFINITY ? 0.f : m * t.scale_log2);
                        const unsigned long long scale2 = pair_of(t.scale_log2, t.scale_log2), shift2 = pair_of(shift, shift);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const uint32_t* q = s + 2 * i;
                            const float2 x = halves(fma2(pair_of(__uint_as_float(q[0]), __uint_as_float(q[1])), scale2, shift2));
                            const float2 y = halves(fma2(pair_of(__uint_as_float(q[2]), __uint_as_float(q[3])), scale2, shift2));
                            const float e0 = exp2_approx(x.x), e1 = exp2_approx(x.y);
                            const float e2 = exp2_approx(y.x), e3 = exp2_approx(y.y);
                            l0 = add2(l0, pair_of(e0, e1));
                            l1 = add2(l1, pair_of(e2, e3));
                            w[i] = Kind<T>::pack(e0, e1);
                            w[i + 1] = Kind<T>::pack(e2, e3);
                        }
                    };
                    // Weights apart from the scores: the next scores may come once these are read, and the last
                    // weights have to be used before the next are written.  (In one place the order is given.)
                    auto scores_read = [&]() {
                        if (S::kApart) {
                            tc_fence_before();
                            warp_arrive(&sm.s_free[slot]);
                        }
                    };
                    auto weights_used = [&]() {
                        if (S::kApart && steps_done > 0) {
                            wait_or_abort(&sm.pv_done[slot], (steps_done - 1) & 1u, &sm.aborted);
                            __syncwarp();
                            tc_fence_after();
                        }
                    };
                    if (nothing) {                                     // no row of the warp sees the tile
                        scores_read();
                        weights_used();
                        if (warp_valid) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = 0u;
#pragma unroll
                            for (int c = 0; c < kTile / 2; c += 16) tc_st16(w, p_at + c);
                        }
                    } else if (PAIRS && warp_valid) {
                        uint32_t s[kTile];                             // fp32 scores
#pragma unroll
                        for (int c = 0; c < kTile; c += 32) tc_ld32(s + c, s_at + c);
                        tc_loaded<kTile>(s);
                        scores_read();
                        if (masked) {
#pragma unroll
                            for (int c = 0; c < kTile; c += 32) {
                                const uint32_t in = columns_seen(lo - c, hi - c);
#pragma unroll
                                for (int i = 0; i < 32; ++i) s[c + i] = in >> i & 1u ? s[c + i] : 0xff800000u;   // -inf
                            }
                        }
                        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                        for (int c = 0; c < kTile; c += 8) {
                            mx0 = fmaxf(fmaxf(mx0, __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
                            mx1 = fmaxf(fmaxf(mx1, __uint_as_float(s[c + 2])), __uint_as_float(s[c + 3]));
                            mx2 = fmaxf(fmaxf(mx2, __uint_as_float(s[c + 4])), __uint_as_float(s[c + 5]));
                            mx3 = fmaxf(fmaxf(mx3, __uint_as_float(s[c + 6])), __uint_as_float(s[c + 7]));
                        }
                        grow(fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)));
                        weigh(s);
                        weights_used();
                        tc_st16(w, p_at);
                        weigh(s + 32);
                        tc_st16(w, p_at + 16);
                        weigh(s + 64);
                        tc_st16(w, p_at + 32);
                        weigh(s + 96);
                        tc_st16(w, p_at + 48);
                    } else if (!PAIRS && warp_valid) {
                        // The same in less code, where memory bounds the items: twice over 64 columns at a time, the
                        // maximum first.
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 2 * kTile; c += 64) {
                            uint32_t s[64];
                            tc_ld32(s, s_at + c % kTile);
                            tc_ld32(s + 32, s_at + c % kTile + 32);
                            tc_loaded<64>(s);
                            if (c == 2 * kTile - 64) scores_read();
                            if (masked) {
                                const int at = c % kTile;
                                const uint32_t in0 = columns_seen(lo - at, hi - at), in1 = columns_seen(lo - at - 32, hi - at - 32);
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    s[i] = in0 >> i & 1u ? s[i] : 0xff800000u;
                                    s[i + 32] = in1 >> i & 1u ? s[i + 32] : 0xff800000u;
                                }
                            }
                            if (c < kTile) {
                                float mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                                for (int i = 0; i < 64; i += 8) {
                                    mx = fmaxf(fmaxf(mx, __uint_as_float(s[i])), __uint_as_float(s[i + 1]));
                                    mx1 = fmaxf(fmaxf(mx1, __uint_as_float(s[i + 2])), __uint_as_float(s[i + 3]));
                                    mx2 = fmaxf(fmaxf(mx2, __uint_as_float(s[i + 4])), __uint_as_float(s[i + 5]));
                                    mx3 = fmaxf(fmaxf(mx3, __uint_as_float(s[i + 6])), __uint_as_float(s[i + 7]));
                                }
                                mx = fmaxf(fmaxf(mx, mx1), fmaxf(mx2, mx3));
                                if (c == kTile - 64) grow(mx);
                            } else {
                                weigh(s);
                                if (c == kTile) weights_used();
                                tc_st16(w, p_at + (c - kTile) / 2);
                                weigh(s + 32);
                                tc_st16(w, p_at + (c - kTile) / 2 + 16);
                            }
                        }
                    }
                    if (!warp_valid && !nothing) {                     // every step is waited for, or a later wait's phase
                        scores_read();                                 // could be taken for an earlier one's
                        weights_used();
                    }
                    if (warp_valid) {
                        const float2 ls = halves(add2(l0, l1));
                        l += ls.x + ls.y;
                        tc_wait_st();
                    }
                    if (by_hand) {
                        const uint32_t e = base + entry_v(k0 / kTile - p.kt0, p.nt, pair ? 1 : 2);
                        const unsigned char* vt = sm.kv[e % kStages];
                        if (warp_valid) {
                            // O is free: the step before has been added to it, or, at a piece's first step, the
                            // output warps have read the last piece's.
                            if (st > 0)
                                wait_or_abort(&sm.pv_done[slot], (steps_done - 1) & 1u, &sm.aborted);
                            else
                                wait_or_abort(&sm.o_free[slot], ~o_uses & 1u, &sm.aborted);
                            __syncwarp();
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = 0u;
                                if (st > 0) {
                                    tc_ld32(o, o_at + c);
                                    tc_loaded<32>(o);
                                }
#pragma unroll 1
                                for (int kk = 0; kk < kTile; ++kk) {
                                    uint32_t w2 = tc_ld1(p_at + kk / 2);
                                    tc_wait_ld();
                                    asm volatile("" : "+r"(w2));
                                    const float2 wf = Kind<T>::unpack(w2);
                                    const float wt = kk & 1 ? wf.y : wf.x;
                                    if (wt != 0.f) {
#pragma unroll
                                        for (int i = 0; i < 32; i += 8) {
                                            const int v = (c + i) / 8;
                                            const uint4 x = *reinterpret_cast<const uint4*>(vt + S::kv_at(kk, v));
                                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                            for (int y = 0; y < 4; ++y) {
                                                const float2 f = Kind<T>::unpack(xs[y]);
                                                uint32_t* q = o + i + 2 * y;
                                                q[0] = __float_as_uint(fmaf(wt, f.x, __uint_as_float(q[0])));
                                                q[1] = __float_as_uint(fmaf(wt, f.y, __uint_as_float(q[1])));
                                            }
                                        }
                                    }
                                    __syncwarp();
                                }
                                tc_st32(o, o_at + c);
                            }
                            tc_wait_st();
                        }
                        if (row == 0) *(volatile int*)&sm.by_hand[slot] = 1;
                    }
                    ++steps_done;
                    tc_fence_before();
                    warp_arrive(&sm.p_full[slot]);
                }
                base += 2u * (uint32_t)p.nt;
                if (my_steps > 0) {
                    wait_or_abort(&sm.o_free[slot], ~o_uses & 1u, &sm.aborted);   // the last piece's have been read
                    ++o_uses;
                    sm.ml[slot][row] = make_float2(m == -INFINITY ? 0.f : m * t.scale_log2, l);
                    warp_arrive(&sm.ml_full[slot]);
                }
            }
        }

    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        // ---- rows of Q in, rows of the output out ------------------------------------------
        const int sw = warp & 3, row = sw * 32 + lane;
        const uint32_t o_at = tmem + ((uint32_t)(sw * 32) << 16) + 256;
        uint32_t q_uses[2] = {0, 0}, steps[2] = {0, 0}, uses[2] = {0, 0}, q_next = 0;
        if (row == 0) t.rec[2 * blockIdx.x] = t.rec[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
        uint32_t pk = 0;
        bool have = false;          // piece pk's output is to come
#pragma unroll 1
        for (;;) {
            // Q of the next piece, where TMA cannot take it: its boxes need groups that divide a tile's rows.
            const uint32_t nk = have ? pk + 1 : 0;
            const bool more = piece_ready(nk);
            if (more) {
                const Piece& n = sm.pieces[nk % kPieces];
                const bool pair = PAIRS && n.pair();
                const int bufs = n.nt == 0 || t.q_tokens ? 0 : pair ? 2 : 1;
#pragma unroll 1
                for (int i = 0; i < bufs; ++i) {
                    const uint32_t qb = pair ? (uint32_t)i : q_next;
                    wait_or_abort(&sm.q_empty[qb], ~(qb ? q_uses[1] : q_uses[0]) & 1u, &sm.aborted);
                    if (qb) ++q_uses[1]; else ++q_uses[0];
                    constexpr int kVecs = D / 8, kStep = kTile / kVecs;      // vectors of a row, rows of a pass
                    const int v = tid % kVecs, top = n.row0 + i * kTile, end = n.row0 + n.rows;
                    const T* src = (const T*)a.q.data + (int64_t)n.head * a.group * a.q.stride_head + v * 8;
                    unsigned char* dst = sm.q[qb] + (v / 8) * (kTile * 128);
#pragma unroll 1
                    for (int x0 = 0; x0 < kVecs; x0 += 8) {
                        uint4 x[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const int r = top + (tid & 127) / kVecs + (x0 + y) * kStep;
                            x[y] = make_uint4(0, 0, 0, 0);
                            if (r < end) {
                                const int tok = t.by_group(r), g = r - tok * a.group;
                                x[y] = *reinterpret_cast<const uint4*>(src + (int64_t)(n.t0 + tok) * a.q.stride_token +
                                                                       (int64_t)g * a.q.stride_head);
                            }
                        }
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const int qr = (tid & 127) / kVecs + (x0 + y) * kStep;
                            *reinterpret_cast<uint4*>(dst + qr * 128 + ((v ^ qr) & 7) * 16) = x[y];
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        __threadfence_block();
                        atomicAdd(&sm.q_loads[qb], 1u);
                    }
                }
                if (!pair && bufs) q_next ^= 1u;
            }

            if (have) {
                const Piece& p = sm.pieces[pk % kPieces];
                const bool pair = PAIRS && p.pair(), both = !pair && p.nt > 1, whole = p.first && p.last;
                const int lead = p.lead;
#pragma unroll 1
                for (int i = 0; i < (pair ? 2 : 1); ++i) {          // rows of one slot, or of both
                    const int s = pair ? i : lead;
                    float f0 = 1.f, f1 = 0.f, mt = 0.f, lt = 0.f;
                    if (p.nt > 0) {
                        wait_or_abort(&sm.ml_full[s], (s ? uses[1] : uses[0]) & 1u, &sm.aborted);
                        wait_or_abort(&sm.pv_done[s], ((s ? steps[1] : steps[0]) + p.steps(s) - 1) & 1u, &sm.aborted);
                        mt = sm.ml[s][row].x;
                        lt = sm.ml[s][row].y;
                    }
                    if (both) {
                        const int z = s ^ 1;
                        wait_or_abort(&sm.ml_full[z], (z ? uses[1] : uses[0]) & 1u, &sm.aborted);
                        wait_or_abort(&sm.pv_done[z], ((z ? steps[1] : steps[0]) + p.steps(z) - 1) & 1u, &sm.aborted);
                        const float2 o = sm.ml[z][row];
                        const float m0 = mt, l0 = lt;
                        if (l0 == 0.f) {
                            mt = o.x;
                        } else if (o.y != 0.f) {
                            mt = fmaxf(m0, o.x);
                        }
                        f0 = l0 == 0.f ? 0.f : exp2_approx(m0 - mt);
                        f1 = o.y == 0.f ? 0.f : exp2_approx(o.x - mt);
                        lt = l0 * f0 + o.y * f1;
                    }
                    tc_fence_after();
                    const int local = i * kTile + row;
                    const bool valid = local < p.rows;
                    if (whole) {
                        const float inv = lt == 0.f ? 0.f : 1.f / lt;
                        f0 *= inv;
                        f1 *= inv;
                    }
                    const int64_t part = (int64_t)(2 * (int)blockIdx.x + (p.first ? 1 : 0)) * t.part_rows + local;
                    const int tok = t.by_group(p.row0 + local), head = p.head * a.group + p.row0 + local - tok * a.group;
                    const int64_t token = p.t0 + tok;
                    if (local - lane < p.rows) {
                        T* out = (T*)a.out.data + token * a.out.stride_token + (int64_t)head * a.out.stride_head;
                        // A slot of weight 0 has no say, whatever it holds: not even 0 times it.
                        const bool drop0 = f0 == 0.f, drop1 = f1 == 0.f, some = __any_sync(0xffffffffu, drop0 || (both && drop1));
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16], o1[16];
                            if (p.nt > 0) tc_ld16(o, o_at + s * 128 + c);
                            if (both) tc_ld16(o1, o_at + (s ^ 1) * 128 + c);
                            tc_loaded<16>(o);
                            tc_loaded<16>(o1);
                            if (some) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    o[i] = drop0 ? 0u : o[i];
                                    o1[i] = drop1 ? 0u : o1[i];
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
                            if (both) {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), f1, __uint_as_float(o[i])));
                            }
                            if (valid && whole) {
                                uint32_t x[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    x[i] = Kind<T>::pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                                *reinterpret_cast<uint4*>(out + c) = make_uint4(x[0], x[1], x[2], x[3]);
                                *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                            } else if (valid) {
#pragma unroll
                                for (int i = 0; i < 16; i += 4)
                                    *reinterpret_cast<uint4*>(t.part + part * D + c + i) =
                                        make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                            }
                        }
                        if (valid && whole) {
                            if (a.lse)
                                a.lse[token * a.q.heads + head] =
                                    lt == 0.f ? -INFINITY : (mt - Kind<T>::kBias) * 0.69314718055994531f + logf(lt);
                        } else if (valid) {
                            t.part_ml[part] = make_float2(mt - Kind<T>::kBias, lt);
                        }
                    }
                    tc_fence_before();
                    if (p.nt > 0) warp_arrive(&sm.o_free[s]);
                    if (both) warp_arrive(&sm.o_free[s ^ 1]);
                }
                steps[0] += p.steps(0);
                steps[1] += p.steps(1);
                if (p.steps(0) > 0) ++uses[0];
                if (p.steps(1) > 0) ++uses[1];
                if (row == 0) {
                    if (!p.first) t.rec[2 * blockIdx.x].x = p.last ? 1 : 2;
                    if (p.first && !p.last) t.rec[2 * blockIdx.x + 1] = make_int4(1, p.r, p.head, p.item);
                }
                piece_release(pk);
            }
            if (!more) break;
            pk = nk;
            have = true;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (sm.aborted) {
        // What is in flight ends before the kernel does: either issuing warp's products, and every buffer's last load.
        const int at = thread_now(), w = at >> 5, i = at & 31;
        unsigned long long* bar = nullptr;
        uint32_t phases = 0;
        if (w == 1 || w == 3) {
            bar = &sm.drain[w >> 1];
            phases = 1;
            if (one_lane()) tc_commit(bar);
            __syncwarp();
        } else if (w == 2 && i < (int)kStages) {
            bar = &sm.full[i];
            phases = (sm.issued + kStages - 1 - (uint32_t)i) / kStages;
        } else if (w == 2 && i < (int)kStages + 2) {
            bar = &sm.q_full[i - (int)kStages];
            phases = sm.q_issued[i - (int)kStages];
        }
#pragma unroll 1
        for (int x = 0; phases > 0 && x < (int)kWaitPolls && !mbar_try_wait(bar, (phases - 1) & 1u); ++x) {}
        __syncwarp();
        if (a.status)
            for (int r = at; r < a.n_req; r += kTcThreads) atomicOr(&a.status[r], kTimeout);
        __syncthreads();                                  // what the CTA has written is written
        if (at == 0) t.rec[2 * blockIdx.x].y = 1;
#pragma unroll 1
        for (int r = 0; r < a.n_req; ++r) {
            const Window w = window_of(t, r, false);
#pragma unroll 1
            for (int i = at; i < w.rows * a.cache.k.heads; i += kTcThreads) {
                const int64_t token = w.t0 + i / a.q.heads, head = i % a.q.heads;
                T* out = (T*)a.out.data + token * a.out.stride_token + head * a.out.stride_head;
#pragma unroll 1
                for (int e = 0; e < D; ++e) out[e] = from_f32<T>(NAN);
                if (a.lse) a.lse[token * a.q.heads + head] = NAN;
            }
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tc_free(tmem);
    }
}

// Joins the pieces of an item: CTA x of the first kernel began it, the ones
// after it have the rest.  A warp a row while pieces are few; the block's four
// warps share a row's pieces when they are many, a quarter each, and join them
// in the order of the line.
constexpr int kFewPieces = 8;
template <typename T, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ TcArgs t)
{
    constexpr int kE = D / 32;
    __shared__ float sum_sh[4][D];
    __shared__ float2 ml_sh[4];
    pdl_enter();
    const AttnArgs& a = t.a;
    const int c0 = (int)blockIdx.x, warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const int4 rec = t.rec[2 * c0 + 1];
    if (!rec.x) return;
    int last = c0 + 1;                                       // the CTA with the item's last piece
    bool lost = t.rec[2 * c0].y != 0;                        // a CTA with a piece gave up
#pragma unroll 1
    for (;; last += 32) {
        const int c = last + lane;
        const int4 left = t.rec[2 * min(c, t.grid - 1)];
        const uint32_t ends = __ballot_sync(0xffffffffu, c >= t.grid - 1 || left.x != 2);
        const uint32_t gone = __ballot_sync(0xffffffffu, left.y != 0);
        lost = lost || (gone & (ends ? ends ^ (ends - 1) : 0xffffffffu)) != 0;   // up to the first end
        if (ends) {
            last += __ffs((int)ends) - 1;
            break;
        }
    }
    const Window w = window_of(t, rec.y, false);
    const int rows = w.item_rows(rec.w), row0 = w.row0(rec.w), n = last - c0 + 1;
    const bool shared = n > kFewPieces;
    const int each = shared ? (n + 3) / 4 : n;               // pieces of a warp
    const int i0 = shared ? warp * each : 0, i1 = min(n, i0 + each);
    const int stride = (int)gridDim.y * (shared ? 1 : 4);
#pragma unroll 1
    for (int row = (int)blockIdx.y * (shared ? 1 : 4) + (shared ? 0 : warp); row < rows; row += stride) {
        // Piece i of the row: the first one is the second record of its CTA.
        auto at = [&](int i) { return (int64_t)(2 * (c0 + i) + (i == 0)) * t.part_rows + row; };
        float mt = -INFINITY, lt = 0.f, x[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = 0.f;
        auto take = [&](auto width) {                        // so many pieces' loads in flight
            constexpr int kW = decltype(width)::value;
#pragma unroll 1
            for (int i = i0; i < i1; i += kW) {
                float2 ml[kW];
                float y[kW][kE];
#pragma unroll
                for (int z = 0; z < kW; ++z) {
                    const int64_t q = at(min(i + z, i1 - 1));
                    ml[z] = t.part_ml[q];
                    if (i + z >= i1) ml[z].y = 0.f;
#pragma unroll
                    for (int e = 0; e < kE; ++e) y[z][e] = t.part[q * D + lane * kE + e];
                }
                float top = mt;
#pragma unroll
                for (int z = 0; z < kW; ++z)
                    if (ml[z].y != 0.f) top = fmaxf(top, ml[z].x);
                const float keep = lt == 0.f ? 0.f : exp2_approx(mt - top);
                mt = top;
                lt *= keep;
#pragma unroll
                for (int e = 0; e < kE; ++e) x[e] = keep == 0.f ? 0.f : x[e] * keep;
#pragma unroll
                for (int z = 0; z < kW; ++z) {
                    if (ml[z].y == 0.f) continue;
                    const float f = exp2_approx(ml[z].x - mt);
                    lt = fmaf(ml[z].y, f, lt);
#pragma unroll
                    for (int e = 0; e < kE; ++e) x[e] = fmaf(y[z][e], f, x[e]);
                }
            }
        };
        if (shared)
            take(std::integral_constant<int, 8>{});
        else
            take(std::integral_constant<int, 2>{});
        if (shared) {
            __syncthreads();                                 // the row before has been read
            if (lane == 0) ml_sh[warp] = make_float2(mt, lt);
#pragma unroll
            for (int e = 0; e < kE; ++e) sum_sh[warp][lane * kE + e] = x[e];
            __syncthreads();
            if (warp != 0) continue;
            float top = -INFINITY;
#pragma unroll
            for (int z = 0; z < 4; ++z)
                if (ml_sh[z].y != 0.f) top = fmaxf(top, ml_sh[z].x);
            lt = 0.f;
#pragma unroll
            for (int e = 0; e < kE; ++e) x[e] = 0.f;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                if (ml_sh[z].y == 0.f) continue;
                const float f = exp2_approx(ml_sh[z].x - top);
                lt = fmaf(ml_sh[z].y, f, lt);
#pragma unroll
                for (int e = 0; e < kE; ++e) x[e] = fmaf(sum_sh[z][lane * kE + e], f, x[e]);
            }
            mt = top;
        }
        if (lost) lt = NAN;
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        const int tok = t.by_group(row0 + row), g = row0 + row - tok * a.group;
        const int64_t token = w.t0 + tok;
        const int head = rec.z * a.group + g;
        T* dst = (T*)a.out.data + token * a.out.stride_token + (int64_t)head * a.out.stride_head + lane * kE;
#pragma unroll
        for (int e = 0; e < kE; e += 2) reinterpret_cast<uint32_t*>(dst)[e / 2] = Kind<T>::pack(x[e] * inv, x[e + 1] * inv);
        if (a.lse && lane == 0)
            a.lse[token * a.q.heads + head] = lt == 0.f ? -INFINITY : mt * 0.69314718055994531f + logf(lt);
    }
}

// ---- host ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// Keys or values for one box a page: x within a row of the cache (a head's
// elements are at its offset, whatever lies between the heads), row of a group
// of 8, block of 64 elements, group, page.  A box is a head's rows of a page (or
// 128 of them), and lands group by group.
bool make_map(CUtensorMap* m, const sv_heads_t& h, int64_t stride_page, const sv_paged_kv_t& c, int head_dim, bool bf16)
{
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t token = (cuuint64_t)h.stride_token * 2, row = (cuuint64_t)head_dim * 2;
    const cuuint64_t dims[5] = {(cuuint64_t)(h.heads - 1) * (cuuint64_t)(h.heads > 1 ? h.stride_head : 0) + (cuuint64_t)head_dim,
                                8, (cuuint64_t)head_dim / 64, (cuuint64_t)c.page_size / 8, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[4] = {token, 128, 8 * token, c.n_pages > 1 ? (cuuint64_t)stride_page * 2 : row};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)head_dim / 64, (cuuint32_t)(c.page_size < kTile ? c.page_size : kTile) / 8, 1};
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, h.data, dims, strides, box,
              step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, head_dim > 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_q_map(CUtensorMap* m, const sv_heads_t& q, int tokens, int head_dim, int group, int box_tokens, bool bf16)
{
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)q.heads, (cuuint64_t)tokens};
    const cuuint64_t row = (cuuint64_t)head_dim * 2;     // stride of an axis of one
    const cuuint64_t strides[2] = {q.heads > 1 ? (cuuint64_t)q.stride_head * 2 : row,
                                   tokens > 1 ? (cuuint64_t)q.stride_token * 2 : row};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)box_tokens};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, q.data, dims, strides, box,
              step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int part_rows(int max_window, int group)
{
    const long long r = (long long)max_window * group;
    return (int)(r > kTile ? 2 * kTile : r < 1 ? 1 : r);
}

Divisor divisor(int d)
{
    uint32_t l = 0;
    while ((1ull << l) < (uint64_t)d) ++l;
    return Divisor{(uint32_t)(((1ull << (31 + l)) + (uint64_t)d - 1) / (uint64_t)d), 31 + l};
}

template <typename T, int D, bool PAIRS>
cudaError_t launch_tc_as(const TcArgs& t, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq, cudaStream_t s)
{
    const size_t smem = sizeof(TcSmem<D>);
    static_assert(sizeof(TcSmem<D>) <= 232448, "shared memory of one CTA");
    static std::atomic<uint64_t> ready{0};                   // a bit a device: the kernel may use that much there
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(attn_tc_kernel<T, D, PAIRS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    e = launch_pdl(attn_tc_kernel<T, D, PAIRS>, dim3(t.grid), dim3(kTcThreads), smem, s, t, mk, mv, mq);
    if (e != cudaSuccess) return e;
    if (t.whole) return cudaSuccess;
    // A few rows a warp rather than one: 18 blocks an item took 57.5 us of ragged prompts of 256-row items, 64 blocks 60.5.
    const int y = t.part_rows < 72 ? (t.part_rows + 3) / 4 : 18;
    return launch_pdl(attn_join_kernel<T, D>, dim3(t.grid - 1, y), dim3(128), 0, s, t);
}

// Windows that fit a slot's rows take a kernel without the code for items that
// do not: instruction misses are a good part of short items' time.
template <typename T, int D>
cudaError_t launch_tc(const TcArgs& t, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq, cudaStream_t s)
{
    return t.part_rows > kTile ? launch_tc_as<T, D, true>(t, mk, mv, mq, s) : launch_tc_as<T, D, false>(t, mk, mv, mq, s);
}

}  // namespace

constexpr int kTcMaxGrid = 152;   // CTAs the workspace has room for: one per SM

size_t attn_tc_workspace(int max_window, int group, int head_dim)
{
    const size_t rows = 2 * (size_t)kTcMaxGrid * (size_t)part_rows(max_window, group);
    return 256 + sizeof(int4) * 2 * kTcMaxGrid + rows * sizeof(float2) + rows * (size_t)head_dim * sizeof(float);
}

bool attn_tc_takes(const AttnArgs& a, sv_dtype_t dt)
{
    const sv_paged_kv_t& c = a.cache;
    const int p = c.page_size;
    return (dt == SV_DTYPE_BF16 || dt == SV_DTYPE_F16) && a.scale >= 0.f && (a.head_dim == 64 || a.head_dim == 128) &&
           ((p >= 8 && p <= kTile && kTile % p == 0) || p % kTile == 0) && c.n_pages > 0 &&
           (long long)c.max_pages * p <= 1ll << 30 && heads_aligned(a.q, 8, 2) && heads_aligned(a.out, 8, 2) &&
           heads_aligned(c.k, 8, 2) && heads_aligned(c.v, 8, 2) && c.stride_page_k % 8 == 0 && c.stride_page_v % 8 == 0 &&
           (long long)c.k.heads * c.k.stride_head < 1ll << 31 && (long long)c.k.heads * c.v.stride_head < 1ll << 31 &&
           c.k.stride_token > 0 && c.v.stride_token > 0 && c.k.stride_head > 0 && c.v.stride_head > 0 &&
           c.stride_page_k > 0 && c.stride_page_v > 0;
}

cudaError_t launch_attn_tc(const AttnArgs& a, sv_dtype_t dt, void* ws, int num_sms, cudaStream_t s)
{
    TcArgs t{};
    t.a = a;
    t.part_rows = part_rows(a.max_window, a.group);
    t.lanes_shift = 0;
    while (t.lanes_shift < 5 && a.n_req <= kTcThreads >> (t.lanes_shift + 1)) ++t.lanes_shift;
    t.item_shift = 8;
    const long long cached = (long long)a.cache.max_pages * a.cache.page_size;
    const bool narrow = cached <= kNarrowCache || (a.window_keys > 0 && a.window_keys <= kNarrowWindow);
    if (a.group == 1 && !a.full && cached > 2 * kTile && narrow) {
        t.item_shift = 7;
        t.part_rows = t.part_rows < kTile ? t.part_rows : kTile;
    }
    t.grid = num_sms < kTcMaxGrid ? (num_sms < 2 ? 2 : num_sms) : kTcMaxGrid;
    t.inv_grid = ~0ull / (unsigned)t.grid + 1;
    char* w = static_cast<char*>(ws);
    const size_t rows = 2 * (size_t)kTcMaxGrid * (size_t)t.part_rows;
    t.rec = reinterpret_cast<int4*>(w);
    t.part_ml = reinterpret_cast<float2*>(w + sizeof(int4) * 2 * kTcMaxGrid);
    t.part = reinterpret_cast<float*>(w + (sizeof(int4) * 2 * kTcMaxGrid + rows * sizeof(float2) + 255) / 256 * 256);
    t.by_group = divisor(a.group);
    t.by_page = divisor(a.cache.page_size);
    t.scale_log2 = fmaxf(a.scale * 1.4426950408889634f, FLT_MIN);   // above 0: hidden scores stay -inf
    // Short caches: an item of up to kWholeTiles tiles is not worth a second kernel.
    t.whole = cached <= (long long)kWholeTiles * kTile;
    const bool bf16 = dt == SV_DTYPE_BF16;
    CUtensorMap mk, mv, mq{};
    if (!make_map(&mk, a.cache.k, a.cache.stride_page_k, a.cache, a.head_dim, bf16) ||
        !make_map(&mv, a.cache.v, a.cache.stride_page_v, a.cache, a.head_dim, bf16))
        return cudaErrorInvalidValue;
    if (kTile % a.group == 0 && a.q.stride_head > 0 && a.q.stride_token > 0) {
        const int longest = a.max_window > 1 ? a.max_window : 1;         // a box has a token, needed or not
        t.q_tokens = kTile / a.group < longest ? kTile / a.group : longest;
        if (!make_q_map(&mq, a.q, a.tokens, a.head_dim, a.group, t.q_tokens, bf16)) return cudaErrorInvalidValue;
    }
    if (a.head_dim == 64)
        return bf16 ? launch_tc<__nv_bfloat16, 64>(t, mk, mv, mq, s) : launch_tc<__half, 64>(t, mk, mv, mq, s);
    return bf16 ? launch_tc<__nv_bfloat16, 128>(t, mk, mv, mq, s) : launch_tc<__half, 128>(t, mk, mv, mq, s);
}

}  // namespace sv
