// sv_pages.cu -- the pages of a paged cache: who holds them, copies of them,
// and tokens that move together.
//
// sv_kv_fork keeps counts, not lists: a page is free when nobody holds it, and
// new pages are the lowest free numbers, so the only state is the table and the
// counts, and the result does not depend on timing.  Its steps need one another's
// results from the whole batch:
//   1  holders: every request gives back what it does not keep and takes what it
//      does not hold; what changes of a table row is set aside;
//   2  the rows set aside are written, begun pages count their writers, the pool's
//      free pages are counted by tiles;
//   3  each request's new pages get their place in the line of free pages (every
//      CTA works out the whole line), and the free pages go to their places.
// They are three kernels for large batches and pools, and one cluster with its
// barriers between them for others, where latencies and launches are what counts.
// Measured on a GB300: 256 windows resized (28,000 pages) in 10.5 us of the GPU,
// 57 by one CTA, of which the three steps are 4,000, 4,000 and 8,000 clocks: the first
// two chains of four to six reads of L2, the third three scans over the block (tiles,
// requests, a tile's pages), three barriers each, one after another in every CTA; 128
// beams of up to 131,072 tokens forked in 12.3 us by three kernels, 38 by one cluster.
//
// The copies are HBM-bound; see the kernels.
#include <atomic>

#include "sv_attn.cuh"
#include "sv_internal.cuh"

namespace sv {
namespace {

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
cudaLaunchConfig_t cluster_config(dim3 grid, int threads, int size, size_t smem, cudaLaunchAttribute (&at)[2], cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    pdl_attr(at[0]);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = size;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cfg;
}

constexpr int kForkThreads = 1024;
constexpr int kTileCols = 256;        // columns of a table row a warp takes
constexpr int kTileWords = kTileCols / 32;
constexpr int kTilePages = 4 * kForkThreads;   // pages of the pool a CTA takes
constexpr int kForkMaxReq = 1 << 14;  // their places in the line fit shared memory
constexpr int kForkCluster = 16;

// What step 1 and 2 know of a request.
struct __align__(16) Need {
    int begun;      // page that it would write on, -1 for none
    int kept;       // columns kept
    int want;       // columns to hold, -1: its count of pages is not one and stays
    int holders;    // of the begun page
};

struct ForkArgs {
    sv_page_pool_t pool;
    const int32_t* parent;
    int group;
    const int32_t* keep_len;
    const int32_t* new_len;
    int32_t* copies;
    int32_t* status;
    // workspace
    Need* need;            // [n_req]
    int32_t* staged;       // [n_req][max_pages] new entries
    uint32_t* changed;     // [n_req][words] which of them
    int32_t* writers;      // [n_pages], of begun pages only
    unsigned long long* best;   // [n_pages], of begun pages only
    int32_t* tile_free;    // [tiles] free pages of a tile
    int32_t* tile_before;  // [tiles] free pages of the tiles before it
    int col_tiles, words, page_tiles;
};
struct Plan {
    int from, kept, want, held;
    bool bad, lost;
};

__device__ __forceinline__ Plan plan_of(const ForkArgs& a, int r)
{
    const int n = a.pool.n_req;
    const uint32_t page = (uint32_t)a.pool.page_size;
    Plan p;
    p.from = r;
    p.held = a.pool.held[r];
    p.bad = p.lost = p.held < 0 || p.held > a.pool.max_pages;
    if (p.lost) p.held = 0;
    p.kept = p.want = p.held;
    long long from = r;
    if (a.parent) {
        const long long low = a.group > 0 ? (long long)(r / a.group) * a.group : 0;
        const int q = a.parent[r];
        if (q < 0 || (a.group > 0 && q >= a.group)) p.bad = true;
        from = low + q;
        if (from >= n) p.bad = true;
    }
    const int keep = a.keep_len[r], room = a.new_len[r];
    if (p.bad) return p;
    const int avail = a.pool.held[from];
    if (avail < 0 || avail > a.pool.max_pages || keep < 0 || keep > (long long)avail * page || room < keep ||
        room > (long long)a.pool.max_pages * page) {
        p.bad = true;
        return p;
    }
    p.from = (int)from;
    p.kept = (int)(((uint32_t)keep + page - 1u) / page);          // (both below 2^31)
    p.want = (int)(((uint32_t)room + page - 1u) / page);
    return p;
}

__device__ __forceinline__ Need load_need(const ForkArgs& a, int r)
{
    const int4 x = __ldcg(reinterpret_cast<const int4*>(&a.need[r]));
    return Need{x.x, x.y, x.z, x.w};
}

__device__ __forceinline__ bool in_pool(const ForkArgs& a, int page) { return page >= 0 && page < a.pool.n_pages; }

// Step 1, a warp a tile of a request's columns.
__device__ __forceinline__ void fork_holders(const ForkArgs& a, int warp, int warps)
{
    const int lane = threadIdx.x & 31;
    const long long units = (long long)a.pool.n_req * a.col_tiles;
    for (long long u = warp; u < units; u += warps) {
        const int r = (int)(u / a.col_tiles), c0 = (int)(u - (long long)r * a.col_tiles) * kTileCols;
        const Plan p = plan_of(a, r);
        const int32_t* mine = a.pool.page_table + (int64_t)r * a.pool.ld_table;
        const int32_t* theirs = a.pool.page_table + (int64_t)p.from * a.pool.ld_table;
        bool bad = p.bad;
        if (c0 == 0 && lane == 0) {
            int begun = -1;
            if (!p.bad && a.keep_len[r] % a.pool.page_size != 0 && a.new_len[r] > a.keep_len[r]) {
                begun = theirs[p.kept - 1];
                if (!in_pool(a, begun)) begun = -1;
            }
            a.need[r] = Need{begun, p.kept, p.lost ? -1 : p.want, 0};
            if (begun >= 0) {
                a.writers[begun] = 0;
                a.best[begun] = 0ull;
            }
        }
        if (p.bad) {
            // keeps what it holds
        } else if (p.from == r) {
            for (int c = max(c0, p.kept) + lane; c < min(c0 + kTileCols, p.held); c += 32) {
                if (in_pool(a, mine[c])) atomicSub(&a.pool.ref_count[mine[c]], 1);
                else bad = true;
            }
        } else {
            const int end = max(p.kept, p.held);
            int had[kTileWords], now[kTileWords];
#pragma unroll
            for (int w = 0; w < kTileWords; ++w) {
                const int c = c0 + w * 32 + lane;
                had[w] = c < p.held ? mine[c] : -1;
                now[w] = c < p.kept ? theirs[c] : -1;
            }
#pragma unroll
            for (int w = 0; w < kTileWords; ++w) {
                const int c = c0 + w * 32 + lane;
                if (c0 + w * 32 >= end) break;
                const bool has = c < p.held, keeps = c < p.kept, same = has && keeps && had[w] == now[w];
                if (has && !same) {
                    if (in_pool(a, had[w])) atomicSub(&a.pool.ref_count[had[w]], 1);
                    else bad = true;
                }
                const bool differs = keeps && !same;
                if (differs) {
                    if (in_pool(a, now[w])) atomicAdd(&a.pool.ref_count[now[w]], 1);
                    else bad = true;
                    a.staged[(int64_t)r * a.pool.max_pages + c] = now[w];
                }
                const uint32_t bits = __ballot_sync(0xFFFFFFFFu, differs);
                if (lane == 0) a.changed[(int64_t)r * a.words + (c0 >> 5) + w] = bits;
            }
        }
        if (a.status && __any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(&a.status[r], kBadLayout);
    }
}

// Step 2: rows, writers, free pages of every tile of the pool.
__device__ __forceinline__ void fork_rows(const ForkArgs& a, int warp, int warps)
{
    const int lane = threadIdx.x & 31;
    const long long units = (long long)a.pool.n_req * a.col_tiles;
    for (long long u = warp; u < units; u += warps) {
        const int r = (int)(u / a.col_tiles), c0 = (int)(u - (long long)r * a.col_tiles) * kTileCols;
        if (c0 == 0 && lane == 0) {
            const int p = __ldcg(&a.need[r].begun);
            if (p >= 0) {
                a.need[r].holders = __ldcg(&a.pool.ref_count[p]);   // step 3 changes the count itself
                atomicAdd(&a.writers[p], 1);
                atomicMax(&a.best[p], (unsigned long long)(uint32_t)a.keep_len[r] << 32 | (uint32_t)(kForkMaxReq - r));
            }
        }
        if (!a.parent) continue;
        const Plan p = plan_of(a, r);
        if (p.from == r) continue;
        uint32_t bits[kTileWords];
#pragma unroll
        for (int w = 0; w < kTileWords; ++w)
            bits[w] = c0 + w * 32 < p.kept ? __ldcg(&a.changed[(int64_t)r * a.words + (c0 >> 5) + w]) : 0u;
#pragma unroll
        for (int w = 0; w < kTileWords; ++w) {
            const int c = c0 + w * 32 + lane;
            if (bits[w] >> lane & 1u)
                a.pool.page_table[(int64_t)r * a.pool.ld_table + c] = __ldcg(&a.staged[(int64_t)r * a.pool.max_pages + c]);
        }
    }
}

// Which of a thread's four pages of a tile are free.
__device__ __forceinline__ uint32_t free_of(const ForkArgs& a, int tile)
{
    const int p0 = tile * kTilePages + (int)threadIdx.x * 4;
    uint32_t bits = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (p0 + i < a.pool.n_pages && __ldcg(&a.pool.ref_count[p0 + i]) == 0) bits |= 1u << i;
    return bits;
}

// Sum over the block of the values of the threads before this one, and of all.
__device__ __forceinline__ int block_before(int x, int* total, int* s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        int w = lane < (int)(blockDim.x >> 5) ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    *total = s_warp[31];
    return sum - x + (warp ? s_warp[warp - 1] : 0);
}

__device__ __forceinline__ void fork_count(const ForkArgs& a, int block, int blocks, int* s_warp)
{
    for (int tile = block; tile < a.page_tiles; tile += blocks) {
        int total;
        block_before(__popc(free_of(a, tile)), &total, s_warp);
        if (threadIdx.x == 0) a.tile_free[tile] = total;
    }
}

// Step 3: who copies, the line of new pages, who is served; then the j-th free page
// goes to the request whose part of the line holds j.
__device__ void fork_assign(const ForkArgs& a, int block, int blocks, int* s_warp, int* s_list, int* s_first)
{
    const int tid = threadIdx.x, n = a.pool.n_req;
    int n_free = 0, line = 0, total;
    for (int t0 = 0; t0 < a.page_tiles; t0 += kForkThreads) {
        const int t = t0 + tid;
        const int before = block_before(t < a.page_tiles ? __ldcg(&a.tile_free[t]) : 0, &total, s_warp);
        if (t < a.page_tiles) a.tile_before[t] = n_free + before;  // every CTA writes the same and reads its own
        n_free += total;
    }
    for (int r0 = 0; r0 < n; r0 += kForkThreads) {
        const int r = r0 + tid;
        int need = 0, copy = 0, keep = 0;
        Need m{-1, 0, 0, 0};
        if (r < n) {
            m = load_need(a, r);
            keep = a.keep_len[r];
            if (m.begun >= 0) {
                const unsigned long long rank = (unsigned long long)(uint32_t)keep << 32 | (uint32_t)(kForkMaxReq - r);
                copy = __ldcg(&a.writers[m.begun]) != m.holders || __ldcg(&a.best[m.begun]) != rank;
            }
            need = max(m.want, m.kept) - m.kept + copy;
        }
        const int first = line + block_before(need, &total, s_warp);
        line += total;
        if (r < n) {
            // the place, the copy's bit, and the one of a request that the free pages do not reach to
            const bool served = need == 0 || first + need <= n_free;
            s_first[r] = first << 2 | copy << 1 | (served ? 0 : 1);
            if (block == 0) {
                if (m.want >= 0) a.pool.held[r] = served ? m.want : m.kept;
                const bool copies = copy && served;
                a.copies[3 * r] = copies ? m.begun : -1;
                if (!copies) a.copies[3 * r + 1] = -1;
                a.copies[3 * r + 2] = copies ? keep % a.pool.page_size : -1;
                if (!served && a.status) atomicOr(&a.status[r], SV_ROW_NO_PAGES);
            }
        }
    }
    __syncthreads();
    for (int tile = block; tile < a.page_tiles; tile += blocks) {
        const int before = a.tile_before[tile];
        if (before >= line) return;                             // the tiles after it begin further on
        const uint32_t bits = free_of(a, tile);
        int at = block_before(__popc(bits), &total, s_warp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (bits >> i & 1u) s_list[at++] = tile * kTilePages + tid * 4 + i;
        __syncthreads();
        for (int i = tid; i < total && before + i < line; i += kForkThreads) {
            const int j = before + i;
            int lo = 0, hi = n;                                 // the last request whose part begins at or before j
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_first[mid] >> 2 <= j) lo = mid;
                else hi = mid;
            }
            const int f = s_first[lo], copy = f >> 1 & 1;
            if (f & 1) continue;
            const Need m = load_need(a, lo);
            const int page = s_list[i], k = j - (f >> 2) - copy;
            if (k < 0) {
                a.copies[3 * lo + 1] = page;
                atomicSub(&a.pool.ref_count[m.begun], 1);       // it has other holders: never a free page
            }
            a.pool.page_table[(int64_t)lo * a.pool.ld_table + m.kept + k] = page;
            a.pool.ref_count[page] = 1;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kForkThreads) fork_holders_kernel(const __grid_constant__ ForkArgs a)
{
    pdl_enter();
    fork_holders(a, blockIdx.x * (kForkThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kForkThreads / 32));
}
__global__ void __launch_bounds__(kForkThreads) fork_rows_kernel(const __grid_constant__ ForkArgs a)
{
    __shared__ int s_warp[32];
    pdl_enter();
    fork_rows(a, blockIdx.x * (kForkThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kForkThreads / 32));
    fork_count(a, blockIdx.x, gridDim.x, s_warp);
}
__global__ void __launch_bounds__(kForkThreads) fork_assign_kernel(const __grid_constant__ ForkArgs a)
{
    extern __shared__ int s_first[];                             // [n_req]
    __shared__ int s_warp[32], s_list[kTilePages];
    pdl_enter();
    fork_assign(a, blockIdx.x, gridDim.x, s_warp, s_list, s_first);
}

// All steps in one cluster.
__global__ void __launch_bounds__(kForkThreads) fork_cluster_kernel(const __grid_constant__ ForkArgs a)
{
    extern __shared__ int s_first[];
    __shared__ int s_warp[32], s_list[kTilePages];
    pdl_enter();
    const int block = blockIdx.x, blocks = gridDim.x;             // one cluster
    const int warp = (threadIdx.x >> 5) * blocks + block, warps = blocks * (kForkThreads / 32);
    fork_holders(a, warp, warps);
    cluster_sync();
    fork_rows(a, warp, warps);
    fork_count(a, block, blocks, s_warp);
    cluster_sync();
    fork_assign(a, block, blocks, s_warp, s_list, s_first);
}

struct ForkLayout {
    size_t need, staged, changed, writers, best, tile_free, tile_before, total;
    int words, page_tiles;
};

ForkLayout fork_layout(int n_req, int max_pages, int n_pages)
{
    ForkLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    const size_t n = (size_t)n_req;
    L.words = (max_pages + kTileCols - 1) / kTileCols * kTileWords;
    L.page_tiles = (n_pages + kTilePages - 1) / kTilePages;
    L.need = take(sizeof(Need) * n);
    L.staged = take(4 * n * (size_t)max_pages);
    L.changed = take(4 * n * (size_t)L.words);
    L.writers = take(4 * (size_t)n_pages);
    L.best = take(8 * (size_t)n_pages);
    L.tile_free = take(4 * (size_t)L.page_tiles);
    L.tile_before = take(4 * (size_t)L.page_tiles);
    L.total = off;
    return L;
}

bool fork_sizes_ok(int n_req, int max_pages, int n_pages)
{
    return n_req >= 1 && n_req <= kForkMaxReq && max_pages >= 0 && n_pages >= 0 && n_pages <= (1 << 30) &&
           (long long)n_req * max_pages <= (1LL << 28);   // (a place in the line is kept in 29 bits)
}

// What the runtime has to be told of the two kernels, once a device.
cudaError_t prepare_fork()
{
    static std::atomic<bool> done[128];               // (callers may be several threads)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev >= 0 && dev < 128 && done[dev])) return e;
    constexpr int kSmem = 4 * kForkMaxReq;
    e = cudaFuncSetAttribute(fork_cluster_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fork_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fork_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess && dev >= 0 && dev < 128) done[dev] = true;
    return e;
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s)
{
    constexpr int kWarps = kForkThreads / 32;
    const long long units = (long long)a.pool.n_req * a.col_tiles;
    const size_t smem = 4 * (size_t)a.pool.n_req;
    cudaError_t e = prepare_fork();
    if (e != cudaSuccess) return e;
    if (units <= 2LL * kForkCluster * kWarps && a.page_tiles <= 4 * kForkCluster) {
        int blocks = 1;
        while (blocks < kForkCluster && (units > (long long)blocks * kWarps || a.page_tiles > blocks)) blocks *= 2;
        cudaLaunchAttribute at[2];
        const cudaLaunchConfig_t cfg = cluster_config(dim3(blocks), kForkThreads, blocks, smem, at, s);
        e = cudaLaunchKernelEx(&cfg, fork_cluster_kernel, a);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const int sms = sm_count();
    auto grid = [&](long long blocks) { return dim3((unsigned)(blocks < 1 ? 1 : blocks > 2LL * sms ? 2LL * sms : blocks)); };
    const long long by_rows = (units + kWarps - 1) / kWarps;
    e = launch_pdl(fork_holders_kernel, grid(by_rows), dim3(kForkThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(fork_rows_kernel, grid(by_rows > a.page_tiles ? by_rows : a.page_tiles), dim3(kForkThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(fork_assign_kernel, grid(a.page_tiles), dim3(kForkThreads), smem, s, a);
}

// ---------------------------------------------------------------------------
// Copies of pages, and tokens that move together.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kCopyUnits = 8;      // units a thread has in flight
constexpr int kMoveUnits = 4;

struct MoveArgs {
    sv_paged_kv_t cache;           // strides in units of R
    int64_t layer_k, layer_v;
    const int32_t* copies;
    const int32_t* first;
    const int32_t* keep;
    const int32_t* n_keep;
    int32_t* status;
    int n, ld_keep, max_keep;
    int per_head;                  // units of a head
    int one;                       // keys and values are one tensor
    int tensors;                   // keys and values of all layers
    int strip;                     // sv_kv_compact: units of a token a CTA takes
    int strips;
};

template <typename R>
__device__ __forceinline__ R* layer_of(const MoveArgs& a, int y, int64_t* page, int64_t* token, int64_t* head)
{
    const bool is_v = !a.one && (y & 1);
    const sv_heads_t& h = is_v ? a.cache.v : a.cache.k;
    *page = is_v ? a.cache.stride_page_v : a.cache.stride_page_k;
    *token = h.stride_token;
    *head = h.stride_head;
    return static_cast<R*>(h.data) + (a.one ? y : y >> 1) * (is_v ? a.layer_v : a.layer_k);
}

// A CTA copies a part of one page of one layer's keys or values; units go in
// the order they lie in memory, heads inside tokens or tokens inside heads.
// 1,021 pages of 16 tokens in 2 layers, heads first, in 42 us (6.3 TB/s, 93% of the
// copy bandwidth); 160 begun pages in 4 layers in 8.
template <typename R>
__global__ void __launch_bounds__(kMoveThreads) copy_kernel(const __grid_constant__ MoveArgs a)
{
    pdl_enter();
    const int src = a.copies[3 * (int64_t)blockIdx.x], dst = a.copies[3 * (int64_t)blockIdx.x + 1],
              tokens = a.copies[3 * (int64_t)blockIdx.x + 2];
    if (src < 0 || dst < 0) return;
    if (src >= a.cache.n_pages || dst >= a.cache.n_pages || tokens < 0 || tokens > a.cache.page_size) {
        if (a.status && threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) atomicOr(a.status, kBadLayout);
        return;
    }
    int64_t page, token, head;
    R* base = layer_of<R>(a, blockIdx.y, &page, &token, &head);
    const R* from = base + src * page;
    R* to = base + dst * page;
    const int heads = a.cache.k.heads;
    const bool tokens_inside = token < head;
    const uint32_t units = (uint32_t)tokens * (uint32_t)heads * (uint32_t)a.per_head;
    const uint32_t inner = tokens_inside ? (uint32_t)tokens : (uint32_t)heads;
    const uint32_t step = gridDim.z * kMoveThreads * kCopyUnits;
    for (uint32_t u0 = blockIdx.z * kMoveThreads * kCopyUnits + threadIdx.x; u0 < units; u0 += step) {
        R x[kCopyUnits];
        int64_t at[kCopyUnits];
#pragma unroll
        for (int i = 0; i < kCopyUnits; ++i) {
            const uint32_t u = u0 + i * kMoveThreads;
            if (u >= units) continue;
            const uint32_t m = u / (uint32_t)a.per_head, o = m / inner, k = m - o * inner;
            at[i] = (u - m * (uint32_t)a.per_head) + (tokens_inside ? k * token + o * head : o * token + k * head);
            x[i] = from[at[i]];
        }
#pragma unroll
        for (int i = 0; i < kCopyUnits; ++i)
            if (u0 + i * kMoveThreads < units) to[at[i]] = x[i];
    }
}

// A CTA has a strip of every token of a request, in one layer's keys or values,
// and goes over the kept tokens in order, some at a turn.  A kept token never
// moves back and tokens keep their order, so what turn t writes has been read by
// turn t or before, and lies before all that turn t + 1 reads.  So while a turn
// is written, the next one's units are on their way, the places of the one after
// that are looked up (once a token, into a ring of three turns) and the list is
// read another turn ahead; one barrier a turn.  CTAs have different strips.  Half
// of 4 x 16,383 tokens (8 heads of 128, strips of 64 bytes) in 51.6 us (5.1 TB/s, 76%
// of the copy bandwidth); 157 when a turn waited for its own lookups and reads.
// With 16-byte units the launch bounds cost spills: 36 bytes with 128 threads, 8 with 512.
//
// A cluster shares a strip's turns where strips alone are too few CTAs.  A list
// of one turn keeps its places for all the layers that its CTA takes, the next
// layer's units on their way while one is written.
template <typename R, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : 9) compact_kernel(const __grid_constant__ MoveArgs a)
{
    __shared__ int64_t s_from[3][THREADS], s_to[3][THREADS];     // a token's old and new place; from -1: it does not move
    pdl_enter();
    uint32_t rank, size;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    const int tid = threadIdx.x, work = blockIdx.x / size, r = work / a.strips, strip = work - r * a.strips;
    const int n = a.n_keep[r];
    const long long first = a.first ? a.first[r] : 0;
    const bool report = a.status && strip == 0 && blockIdx.y == 0;
    if (n < 0 || n > a.max_keep || first < 0) {
        if (report && rank == 0 && tid == 0) atomicOr(&a.status[r], kBadLayout);
        return;
    }
    const int lane = tid % a.strip, row = tid / a.strip, rows = THREADS / a.strip;
    const int share = rows * kMoveUnits;                          // tokens of a CTA's turn; at most THREADS, as a strip has kMoveUnits units or more
    const int turn = share * (int)size, before = share * (int)rank;
    const int s = strip * a.strip + lane;
    const bool mine = s < a.per_head * a.cache.k.heads;
    const int h = s / a.per_head;
    int64_t page, token, head;
    auto strip_of = [&](int y) {
        R* base = layer_of<R>(a, y, &page, &token, &head);
        return base + h * head + (s - h * a.per_head);
    };
    const int32_t* keep = a.keep + (int64_t)r * a.ld_keep;
    const int32_t* table = a.cache.page_table + (int64_t)r * a.cache.ld_table;
    const long long limit = (long long)a.cache.max_pages * a.cache.page_size;
    const uint32_t page_size = (uint32_t)a.cache.page_size;
    // The thread's token of turn t: entries of the list, then its places.
    int k = 0, k_before = -1;
    auto list = [&](int t) {
        const int j = t * turn + before + tid;
        if (tid >= share || j >= n) return;
        k = keep[j];
        k_before = j ? keep[j - 1] : -1;
    };
    auto look_up = [&](int t) {
        const int j = t * turn + before + tid;
        if (tid >= share) return;
        int64_t from = -1, to = 0;
        if (j < n) {
            bool fine = k >= j && k_before < k && first + k < limit;
            if (fine && k != j) {
                const uint32_t p = (uint32_t)(first + k), q = (uint32_t)(first + j);   // sums of two int32
                const uint32_t c0 = p / page_size, c1 = q / page_size;
                const int p0 = table[c0], p1 = table[c1];
                fine = p0 >= 0 && p0 < a.cache.n_pages && p1 >= 0 && p1 < a.cache.n_pages;
                if (fine) {
                    from = p0 * page + (p - c0 * page_size) * token;
                    to = p1 * page + (q - c1 * page_size) * token;
                }
            }
            if (!fine && report) atomicOr(&a.status[r], kBadLayout);
        }
        s_from[t % 3][tid] = from;
        s_to[t % 3][tid] = to;
    };
    R x[kMoveUnits], next[kMoveUnits];
    auto read = [&](const R* base, int t, R (&v)[kMoveUnits]) {   // which of the units move
        uint32_t m = 0u;
        if (!mine) return m;
#pragma unroll
        for (int i = 0; i < kMoveUnits; ++i) {
            const int64_t from = s_from[t % 3][i * rows + row];
            if (from < 0) continue;
            v[i] = base[from];
            m |= 1u << i;
        }
        return m;
    };
    auto write = [&](R* base, int t, uint32_t moves) {
#pragma unroll
        for (int i = 0; i < kMoveUnits; ++i) {
            if (moves >> i & 1u) base[s_to[t % 3][i * rows + row]] = x[i];
            x[i] = next[i];
        }
    };
    auto barrier = [&]() {
        if (size > 1) cluster_sync();
        else __syncthreads();
    };
    if (n <= turn) {
        R* base = strip_of(blockIdx.y);
        list(0);
        look_up(0);
        __syncthreads();
        uint32_t moves = read(base, 0, x);
        for (int y = blockIdx.y; y < a.tensors; y += gridDim.y) { // all of them keys, or values: the places are the same
            const int y1 = y + gridDim.y;
            R* base1 = y1 < a.tensors ? strip_of(y1) : base;
            const uint32_t next_moves = y1 < a.tensors ? read(base1, 0, next) : 0u;
            barrier();
            write(base, 0, moves);
            base = base1;
            moves = next_moves;
        }
        return;
    }
    for (int y = blockIdx.y; y < a.tensors; y += gridDim.y) {
        R* base = strip_of(y);
        list(0);
        look_up(0);
        list(1);
        look_up(1);
        list(2);
        __syncthreads();
        uint32_t moves = read(base, 0, x);
        barrier();
        for (int t = 0; t * turn < n; ++t) {
            const uint32_t next_moves = (t + 1) * turn < n ? read(base, t + 1, next) : 0u;
            write(base, t, moves);
            if ((t + 2) * turn < n) {
                look_up(t + 2);
                list(t + 3);
            }
            barrier();
            moves = next_moves;
        }
    }
}

// The cache's strides in units of `n` elements, if every head of it is made of such units.
bool in_units(MoveArgs& a, int n, int size, int head_dim)
{
    const sv_paged_kv_t& c = a.cache;
    if (head_dim % n || !heads_aligned(c.k, n, size) || !heads_aligned(c.v, n, size) || c.stride_page_k % n ||
        c.stride_page_v % n || a.layer_k % n || a.layer_v % n)
        return false;
    a.cache.k.stride_token /= n;
    a.cache.k.stride_head /= n;
    a.cache.v.stride_token /= n;
    a.cache.v.stride_head /= n;
    a.cache.stride_page_k /= n;
    a.cache.stride_page_v /= n;
    a.layer_k /= n;
    a.layer_v /= n;
    a.per_head = head_dim / n;
    return true;
}

template <typename R>
cudaError_t launch_move(MoveArgs a, int layers, cudaStream_t s)
{
    const long long token = (long long)a.per_head * a.cache.k.heads;
    const int tensors = a.tensors = a.one ? layers : 2 * layers;
    if (a.copies) {
        long long parts = (token * a.cache.page_size + kMoveThreads * kCopyUnits - 1) / (kMoveThreads * kCopyUnits);
        if (parts > 64) parts = 64;
        return launch_pdl(copy_kernel<R>, dim3(a.n, tensors, (unsigned)parts), dim3(kMoveThreads), 0, s, a);
    }
    // Strips as wide as give three CTAs two SMs, of 64 bytes at least, and of which a token is whole ones if it can be (8 x
    // 16,384 tokens, half kept: 99 us with 64 bytes, 93 with 128; 4 requests of those 51 and 58).
    const int least = 64 / (int)sizeof(R);
    a.strip = 32;
    while (a.strip > least && (token % a.strip || 2LL * a.n * tensors * (token / a.strip) < 3LL * sm_count())) a.strip /= 2;
    a.strips = (int)((token + a.strip - 1) / a.strip);
    const long long strips = (long long)a.n * a.strips, sms = sm_count();
    // Accepted paths: small CTAs, some layers each (64 x 9 tokens 5 us, 18 with 512 threads; 256 x 80 31 and 41; 64 x 256
    // 48.7 and 47.9).
    if (a.max_keep <= 128) {
        const int both = a.one ? 1 : 2;
        const long long groups = (16 * sms + strips * both - 1) / (strips * both);
        const int y = both * (int)(groups < layers ? groups : layers);
        return launch_pdl(compact_kernel<R, 128>, dim3((unsigned)strips, y), dim3(128), 0, s, a);
    }
    int size = 1;                                               // two CTAs an SM
    while (size < 8 && 2 * size * strips * tensors <= 2 * sms) size *= 2;
    if (size == 1) return launch_pdl(compact_kernel<R, 512>, dim3((unsigned)strips, tensors), dim3(512), 0, s, a);
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)strips * size, tensors), 512, size, 0, at, s);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, compact_kernel<R, 512>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

sv_status_t run_move(MoveArgs a, sv_dtype_t dt, int head_dim, int layers, cudaStream_t s)
{
    const int size = dt == SV_DTYPE_F32 ? 4 : 2;
    const sv_heads_t &k = a.cache.k, &v = a.cache.v;
    a.one = k.data == v.data && k.stride_token == v.stride_token && k.stride_head == v.stride_head &&
            a.cache.stride_page_k == a.cache.stride_page_v && a.layer_k == a.layer_v;   // moved twice it would be lost
    cudaError_t e;
    if (in_units(a, 16 / size, size, head_dim)) e = launch_move<uint4>(a, layers, s);
    else if (in_units(a, 8 / size, size, head_dim)) e = launch_move<uint2>(a, layers, s);
    else if (in_units(a, 4 / size, size, head_dim)) e = launch_move<uint32_t>(a, layers, s);
    else {
        in_units(a, 1, size, head_dim);
        e = launch_move<uint16_t>(a, layers, s);
    }
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

sv_status_t check_cache(const sv_paged_kv_t& c, sv_dtype_t dt, int head_dim, int layers)
{
    if (head_dim < 1 || layers < 0 || c.k.heads < 1 || c.v.heads != c.k.heads || c.page_size < 1 || c.n_pages < 0 ||
        (dt != SV_DTYPE_BF16 && dt != SV_DTYPE_F16 && dt != SV_DTYPE_F32))
        return SV_ERR_INVALID_ARG;
    const int size = dt == SV_DTYPE_F32 ? 4 : 2;
    if (layers > 32767 || (long long)c.k.heads * head_dim > (1LL << 19) ||
        (long long)c.page_size * c.k.heads * head_dim > (1LL << 30))
        return SV_ERR_UNSUPPORTED;
    if (layers > 0 && (!c.k.data || !c.v.data || !aligned_to(c.k.data, size) || !aligned_to(c.v.data, size)))
        return SV_ERR_INVALID_ARG;
    return SV_OK;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t sv_kv_fork_workspace_size(int n_req, int max_pages, int n_pages)
{
    return fork_sizes_ok(n_req, max_pages, n_pages) ? fork_layout(n_req, max_pages, n_pages).total : 0;
}

extern "C" sv_status_t sv_kv_fork(sv_page_pool_t pool, const int32_t* parent, int group, const int32_t* keep_len,
                                  const int32_t* new_len, int32_t* copies, int32_t* status, void* ws, size_t ws_bytes,
                                  sv_stream_t stream)
{
    if (pool.n_req < 0 || pool.max_pages < 0 || pool.ld_table < pool.max_pages || pool.n_pages < 0 ||
        pool.page_size < 1 || group < 0)
        return SV_ERR_INVALID_ARG;
    if (pool.n_req == 0) return SV_OK;
    if (!pool.page_table || !pool.held || !pool.ref_count || !keep_len || !new_len || !copies) return SV_ERR_INVALID_ARG;
    if (!fork_sizes_ok(pool.n_req, pool.max_pages, pool.n_pages)) return SV_ERR_UNSUPPORTED;
    const ForkLayout L = fork_layout(pool.n_req, pool.max_pages, pool.n_pages);
    if (!ws || !aligned_to(ws, 256) || ws_bytes < L.total) return SV_ERR_WORKSPACE;
    char* w = static_cast<char*>(ws);
    ForkArgs a{};
    a.pool = pool;
    a.parent = parent;
    a.group = group;
    a.keep_len = keep_len;
    a.new_len = new_len;
    a.copies = copies;
    a.status = status;
    a.need = reinterpret_cast<Need*>(w + L.need);
    a.staged = reinterpret_cast<int32_t*>(w + L.staged);
    a.changed = reinterpret_cast<uint32_t*>(w + L.changed);
    a.writers = reinterpret_cast<int32_t*>(w + L.writers);
    a.best = reinterpret_cast<unsigned long long*>(w + L.best);
    a.tile_free = reinterpret_cast<int32_t*>(w + L.tile_free);
    a.tile_before = reinterpret_cast<int32_t*>(w + L.tile_before);
    a.words = L.words;
    a.page_tiles = L.page_tiles;
    a.col_tiles = pool.max_pages > 0 ? L.words / kTileWords : 1;
    return launch_fork(a, stream) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

extern "C" sv_status_t sv_kv_copy(sv_paged_kv_t cache, sv_dtype_t dt, int head_dim, int layers, int64_t stride_layer_k,
                                  int64_t stride_layer_v, const int32_t* copies, int n_copies, int32_t* status,
                                  sv_stream_t stream)
{
    const sv_status_t st = check_cache(cache, dt, head_dim, layers);
    if (st != SV_OK) return st;
    if (n_copies < 0) return SV_ERR_INVALID_ARG;
    if (n_copies == 0 || layers == 0) return SV_OK;
    if (!copies) return SV_ERR_INVALID_ARG;
    MoveArgs a{};
    a.cache = cache;
    a.layer_k = stride_layer_k;
    a.layer_v = stride_layer_v;
    a.copies = copies;
    a.n = n_copies;
    a.status = status;
    return run_move(a, dt, head_dim, layers, stream);
}

extern "C" sv_status_t sv_kv_compact(sv_paged_kv_t cache, sv_dtype_t dt, int head_dim, int layers, int64_t stride_layer_k,
                                     int64_t stride_layer_v, int n_req, const int32_t* first, const int32_t* keep,
                                     int ld_keep, int max_keep, const int32_t* n_keep, int32_t* status,
                                     sv_stream_t stream)
{
    const sv_status_t st = check_cache(cache, dt, head_dim, layers);
    if (st != SV_OK) return st;
    if (n_req < 0 || max_keep < 0 || ld_keep < max_keep || cache.max_pages < 0 || cache.ld_table < cache.max_pages)
        return SV_ERR_INVALID_ARG;
    if (n_req == 0 || layers == 0) return SV_OK;
    if (!n_keep || (max_keep > 0 && !keep) || (cache.max_pages > 0 && !cache.page_table)) return SV_ERR_INVALID_ARG;
    if (n_req > (1 << 16) || max_keep > (1 << 30)) return SV_ERR_UNSUPPORTED;
    MoveArgs a{};
    a.cache = cache;
    a.layer_k = stride_layer_k;
    a.layer_v = stride_layer_v;
    a.first = first;
    a.keep = keep;
    a.n_keep = n_keep;
    a.n = n_req;
    a.ld_keep = ld_keep;
    a.max_keep = max_keep;
    a.status = status;
    return run_move(a, dt, head_dim, layers, stream);
}
