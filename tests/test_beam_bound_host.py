"""The bound that a beam selection's chunks and candidates are held to, run on the host.

`nth_bound` of sv_beam.cu returns a lower bound on the n-th largest of its block's values.  Here its own text is compiled as
host code: a thread of the host for each of the block's, warps' and block's exchanges over arrays with barriers, and the
block's shared memory filled with something else before every call, as another kernel may leave it.  What has to hold of a
result: it is finite, at least n values reach it unless it is the lowest number of all, and what lay in shared memory
before has no part in it.
"""
import os
import struct
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_rows_gb300", "csrc")
LOWEST = float(np.finfo(np.float32).min)
INF = float("inf")

HARNESS = r"""
#include <atomic>
#include <barrier>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <memory>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline
struct Dim { int x; };
static thread_local Dim threadIdx;
static std::unique_ptr<std::barrier<>> g_block, g_warp[32];
static uint32_t g_slot[1024];
static std::atomic<int> g_count;

static uint32_t __float_as_uint(float x) { uint32_t b; memcpy(&b, &x, 4); return b; }
static float __uint_as_float(uint32_t b) { float x; memcpy(&x, &b, 4); return x; }
static void __syncthreads() { g_block->arrive_and_wait(); }
static int __syncthreads_count(int p)
{
    if (threadIdx.x == 0) g_count = 0;
    __syncthreads();
    if (p) ++g_count;
    __syncthreads();
    const int n = g_count;
    __syncthreads();
    return n;
}
// every lane's word, read by all lanes of the warp
template <typename F>
static auto over_warp(uint32_t mine, F f)
{
    const int w0 = threadIdx.x & ~31;
    g_slot[threadIdx.x] = mine;
    g_warp[w0 >> 5]->arrive_and_wait();
    const auto r = f(&g_slot[w0]);
    g_warp[w0 >> 5]->arrive_and_wait();
    return r;
}
static float warp_max(float x)                   // of the numbers among the lanes', as the instruction
{
    return over_warp(__float_as_uint(x), [](const uint32_t* s) {
        float m = NAN;
        for (int i = 0; i < 32; ++i) m = fmaxf(m, __uint_as_float(s[i]));
        return m;
    });
}
static int __shfl_up_sync(unsigned, int x, int o)
{
    const int lane = threadIdx.x & 31;
    return over_warp((uint32_t)x, [&](const uint32_t* s) { return (int)s[lane >= o ? lane - o : lane]; });
}
static int __reduce_add_sync(unsigned, int x)
{
    return over_warp((uint32_t)x, [](const uint32_t* s) {
        int sum = 0;
        for (int i = 0; i < 32; ++i) sum += (int)s[i];
        return sum;
    });
}
static int atomicAdd(int* p, int x) { return __atomic_fetch_add(p, x, __ATOMIC_SEQ_CST); }

struct PickShared {
    int bins[1024];
    float warp_best[32];
    int warp_count[32];
    float bound;
    int bound_found;
};
static PickShared g_shared;

%s

template <int T>
static void block(int cases)
{
    g_block = std::make_unique<std::barrier<>>(T);
    for (int w = 0; w < T / 32; ++w) g_warp[w] = std::make_unique<std::barrier<>>(32);
    std::vector<float> best(T);
    std::vector<std::thread> threads;
    for (int t = 0; t < T; ++t)
        threads.emplace_back([&, t] {
            threadIdx.x = t;
            static int n_out;
            for (int c = 0; c < cases; ++c) {
                if (t == 0) {
                    uint32_t head[2];
                    if (fread(head, 4, 2, stdin) != 2 || fread(best.data(), 4, T, stdin) != (size_t)T) exit(2);
                    n_out = (int)head[0];
                    for (size_t i = 0; i < sizeof g_shared / 4; ++i) memcpy((char*)&g_shared + 4 * i, &head[1], 4);
                }
                __syncthreads();
                const float r = nth_bound<T>(best[t], n_out, g_shared);
                __syncthreads();
                if (t == 0) fwrite(&r, 4, 1, stdout);
            }
        });
    for (auto& t : threads) t.join();
}

int main()
{
    int head[2];
    if (fread(head, 4, 2, stdin) != 2) return 2;
    if (head[0] == 256) block<256>(head[1]);
    else if (head[0] == 1024) block<1024>(head[1]);
    else return 2;
    return 0;
}
"""


def _function(fname, head):
    """The text of a function from `head` to its closing brace in the first column."""
    text = open(os.path.join(CSRC, fname)).read()
    at = text.index(head)
    return text[at:text.index("\n}\n", at) + 3]


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    """Function: (threads, [(n, what shared memory holds, values)]) -> the bounds."""
    where = tmp_path_factory.mktemp("bound")
    parts = [_function("sv_internal.cuh", "__device__ __forceinline__ uint32_t key_of_f32_bits"),
             _function("sv_internal.cuh", "__device__ __forceinline__ float f32_of_key(uint32_t"),
             _function("sv_beam.cu", "template <int T>\n__device__ float nth_bound")]
    (where / "bound.cpp").write_text(HARNESS.replace("%s", "\n".join(parts)))
    subprocess.run(["g++", "-std=c++20", "-O1", "-ffp-contract=off", "-pthread", str(where / "bound.cpp"), "-o",
                    str(where / "bound")], check=True)

    def run(threads, cases):
        data = struct.pack("2i", threads, len(cases))
        for n, stale, values in cases:
            assert len(values) == threads
            data += struct.pack("If", n, stale) + np.asarray(values, np.float32).tobytes()
        r = subprocess.run([str(where / "bound")], input=data, capture_output=True, check=True, timeout=120)
        return np.frombuffer(r.stdout, np.float32)

    return run


def check(threads, cases, got):
    assert len(got) == len(cases)
    for (n, stale, values), bound in zip(cases, got):
        values = np.asarray(values, np.float32)
        assert np.isfinite(bound), (n, stale, bound)
        if bound > LOWEST:
            assert (values >= bound).sum() >= n, (n, stale, bound)


def padded(threads, values):
    return np.concatenate([np.asarray(values, np.float32), np.full(threads - len(values), -INF, np.float32)])


@pytest.mark.parametrize("threads", [256, 1024])
def test_a_bound_is_finite(bounds, threads):
    """Values at fp32's lowest (finished beams with the lowest score): a step below them is not a number to compare with,
    for what is not a value at all, -inf, would reach it."""
    step = 2.0 ** 104                               # of numbers of that size
    near = [LOWEST, LOWEST + step, LOWEST + 3 * step, LOWEST * (1 - 2.0 ** -22), LOWEST * (1 - 2.0 ** -20), LOWEST / 2]
    cases = [(n, -INF, padded(threads, [v] * m)) for v in near for n, m in ((1, 1), (4, 128), (16, 16))]
    check(threads, cases, bounds(threads, cases))


@pytest.mark.parametrize("threads", [256, 1024])
def test_a_bound_is_reached_by_as_many_as_asked(bounds, threads):
    rng = np.random.default_rng(threads)
    cases = []
    for n, m in ((1, 1), (5, 3), (8, threads), (64, 100), (256, 256)):
        for scale, shift in ((1.0, 0.0), (5.0, -100.0), (1e30, 0.0), (0.0, -2.5), (3.0, 1e8)):
            values = padded(threads, rng.standard_normal(m) * scale + shift)
            cases.append((n, -INF, rng.permutation(values)))
    got = bounds(threads, cases)
    check(threads, cases, got)
    for (n, _, values), bound in zip(cases, got):
        finite = np.sort(values[np.isfinite(values)])[::-1]
        if len(finite) < n:
            assert bound == LOWEST
        else:                                       # a bin of 32 / threads, or what a bisection of 20 bits leaves
            nth, most = float(finite[n - 1]), float(finite[0])
            assert float(bound) >= nth - max(33.0 / threads + 2.0 ** -22 * abs(most), 2.0 ** -10 * abs(nth))


@pytest.mark.parametrize("threads", [256, 1024])
def test_what_lay_in_shared_memory_has_no_part_in_a_bound(bounds, threads):
    rng = np.random.default_rng(threads + 1)
    rows = [(4, padded(threads, rng.standard_normal(100) * 3 - 100)), (8, padded(threads, rng.standard_normal(200) * 3)),
            (3, np.full(threads, LOWEST)), (5, padded(threads, [-7.0] * 4))]
    stale = [-INF, 0.0, INF, float("nan"), 1e30, -104.0, -2.0]
    cases = [(n, s, values) for n, values in rows for s in stale]
    got = bounds(threads, cases)
    check(threads, cases, got)
    got = got.reshape(len(rows), len(stale))
    assert (got == got[:, :1]).all()
