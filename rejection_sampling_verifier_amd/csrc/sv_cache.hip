// gfx950 kernels of the paged cache's commit and fork.
//
// Which pages are free is read off the block tables at every call: a page is
// in use if a live entry of the new tables names it.  No reference counts or
// free lists are kept, so nothing can drift, a call can be repeated or replayed
// from a graph, and freeing a sequence is dropping its table row.
//
//   k_cache_plan   one workgroup: the lengths and needs of all sequences, the
//                  set of pages in use as a bitmap in LDS, the lowest free
//                  pages in order, and the call's status.  Page i is bit
//                  i / W of word i % W (W words), so that the consecutive
//                  pages of a sequence fall into different words and the LDS
//                  atomics do not queue up.
//   k_cache_copy   the rest of the device: table rows, lengths and the moved
//                  K/V rows of every layer, 16 bytes per thread and step.
//
// All or nothing: with too few free pages, or an index out of range, the
// tables and lengths go out as they came in and no row moves.

#include <hip/hip_ext.h>

#include "sv_tree.h"

namespace sv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

// Sum of `v` over the threads before this one, and over all of them.
__device__ __forceinline__ int block_scan(int v, int* s_wave, int& all) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(s, o);
        if (lane >= o) s += up;
    }
    __syncthreads();
    if (lane == 63) s_wave[w] = s;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int i = 0; i < kPlanWaves; ++i) {
        if (i < w) before += s_wave[i];
        all += s_wave[i];
    }
    return before + s - v;
}

__device__ __forceinline__ int blocks_of(int rows, int ps_shift) {
    return static_cast<int>((static_cast<int64_t>(rows) + (1 << ps_shift) - 1) >> ps_shift);
}

// The lowest slot that continues `a` (written by atomics, so read past the L1).
__device__ __forceinline__ int first_of(const int32_t* first, int a) {
    return __hip_atomic_load(first + a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(kPlanThreads) void k_cache_plan(CacheParams p) {
    extern __shared__ uint32_t used[];  // W words
    __shared__ int s_wave[kPlanWaves];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int W = (p.pages + 31) / 32;
    const int64_t cap = static_cast<int64_t>(p.width) << p.ps_shift;
    int32_t* const plan = p.plan;
    int32_t* const first = plan + static_cast<int64_t>(p.B) * kPlanWords;  // fork: lowest slot of each ancestor
    int32_t* const fresh = first + p.B;                                    // the new pages, in order
    for (int i = tid; i < W; i += kPlanThreads) used[i] = 0;
    if (tid == 0) s_bad = 0;
    if (p.fork)
        for (int b = tid; b < p.B; b += kPlanThreads) first[b] = 0x7FFFFFFF;
    __syncthreads();
    bool bad = false;
    if (p.fork) {
        for (int b = tid; b < p.B; b += kPlanThreads) {
            const int a = p.ancestor[b];
            if (a >= p.B || a < -1)
                bad = true;
            else if (a >= 0)
                atomicMin(first + a, b);
        }
        __syncthreads();
    }
    // lengths, live pages kept, new pages
    for (int b = tid; b < p.B; b += kPlanThreads) {
        const int old = p.len[b];
        int len = old, want = 0, have = 0;
        if (p.fork) {
            const int a = p.ancestor[b];
            const bool in = a >= 0 && a < p.B;
            len = in ? p.len[a] : 0;
            if (old < 0 || old > cap || len < 0 || len > cap) {
                bad = true;
                len = 0;
            }
            want = blocks_of(len, p.ps_shift);
            have = len >> p.ps_shift;
            // a partly filled last page stays with the lowest slot
            if (have < want && first_of(first, in ? a : 0) == b) have = want;
        } else {
            int rows = p.n_accepted[b] + 1;
            if (rows < 0) rows = 0;
            if (len < 0 || len > cap || rows > p.N || len + static_cast<int64_t>(rows) > cap) {
                bad = true;
                len = rows = 0;
            }
            for (int j = 0; j < rows; ++j) {
                const int node = p.nodes ? p.nodes[static_cast<int64_t>(b) * p.N + j] : j;
                if (node < 0 || node >= p.N) bad = true;
            }
            have = blocks_of(len, p.ps_shift);
            len += rows;
            want = blocks_of(len, p.ps_shift);
        }
        int32_t* const e = plan + static_cast<int64_t>(b) * kPlanWords;
        e[0] = old;
        e[1] = len;
        e[2] = have;
        e[3] = want - have;
    }
    __syncthreads();
    // the pages in use: one wave per sequence, of each ancestor once
    for (int b = w; b < p.B; b += kPlanWaves) {
        int have = plan[static_cast<int64_t>(b) * kPlanWords + 2], row = b;
        if (p.fork) {
            row = p.ancestor[b];
            if (row < 0 || row >= p.B) continue;
            if (first_of(first, row) != b) continue;
        }
        const int32_t* const tab = p.table + row * p.table_stride;
        for (int j = lane; j < have; j += 64) {
            const int pg = tab[j];
            if (pg < 0 || pg >= p.pages)
                bad = true;
            else
                atomicOr(&used[pg % W], 1u << (pg / W));
        }
    }
    if (bad) s_bad = 1;
    __syncthreads();
    // free pages: each thread a run of consecutive ones
    const int run = (p.pages + kPlanThreads - 1) / kPlanThreads;
    const int lo = min(tid * run, p.pages), hi = min(lo + run, p.pages);
    int mine = 0;
    for (int i = lo; i < hi; ++i) mine += !(used[i % W] >> (i / W) & 1);
    int n_free;
    int rank = block_scan(mine, s_wave, n_free);
    // the sequences' places in the list of new pages
    int need = 0;
    for (int base = 0; base < p.B; base += kPlanThreads) {
        const int b = base + tid;
        int32_t* const e = plan + static_cast<int64_t>(b) * kPlanWords;
        int all;
        const int at = block_scan(b < p.B ? e[3] : 0, s_wave, all);
        if (b < p.B) e[3] = need + at;
        need += all;
    }
    const bool fail = s_bad != 0;
    if (tid == 0) *p.status = fail ? -1 : need > n_free ? need - n_free : 0;
    if (fail || need > n_free) return;
    for (int i = lo; i < hi && rank < need; ++i)
        if (!(used[i % W] >> (i / W) & 1)) fresh[rank++] = i;
}

// blockIdx.x: sequence; blockIdx.y: layer, or past the layers the table row.
__global__ __launch_bounds__(kThreads) void k_cache_copy(CacheParams p) {
    const int b = blockIdx.x, tid = threadIdx.x;
    const int32_t* const e = p.plan + static_cast<int64_t>(b) * kPlanWords;
    const int32_t* const fresh = p.plan + static_cast<int64_t>(p.B) * (kPlanWords + 1);
    const int old = e[0], len = e[1], have = e[2];
    const bool done = *p.status == 0;
    const int a = p.fork ? p.ancestor[b] : b;
    if (static_cast<int>(blockIdx.y) == p.layers) {
        const int64_t cap = static_cast<int64_t>(p.width) << p.ps_shift;
        const int live = old < 0 ? 0 : blocks_of(old > cap ? static_cast<int>(cap) : old, p.ps_shift);
        const int want = blocks_of(len, p.ps_shift);
        const int32_t* const src = p.table + (done && a >= 0 ? a : b) * p.table_stride;
        int32_t* const dst = p.out_table + b * p.out_stride;
        for (int j = tid; j < p.width; j += kThreads) {
            int v = -1;
            if (done) {
                if (j < have)
                    v = src[j];
                else if (j < want)
                    v = fresh[e[3] + j - have];
            } else if (j < live) {
                v = src[j];
            }
            dst[j] = v;
        }
        if (tid == 0) p.out_len[b] = done ? len : old;
        return;
    }
    if (!done) return;
    const int64_t layer = blockIdx.y;
    const int psm = (1 << p.ps_shift) - 1;
    uint8_t* const kl = p.k + 16 * (layer * p.ks[0]);
    uint8_t* const vl = p.v + 16 * (layer * p.vs[0]);
    if (p.fork) {
        const int want = blocks_of(len, p.ps_shift);
        if (have == want) return;  // nothing to copy: empty, full pages only, or the page's keeper
        const int64_t from = p.table[a * p.table_stride + have], to = fresh[e[3]];
        const int rows = len & psm;
        const int total = rows * p.heads * p.vec;
        for (int i = tid; i < total; i += kThreads) {
            const int v = i % p.vec, rh = i / p.vec;
            const int h = rh % p.heads, r = rh / p.heads;
            const uint4 x = *reinterpret_cast<const uint4*>(kl + 16 * (from * p.ks[1] + r * p.ks[2] + h * p.ks[3] + v));
            const uint4 y = *reinterpret_cast<const uint4*>(vl + 16 * (from * p.vs[1] + r * p.vs[2] + h * p.vs[3] + v));
            *reinterpret_cast<uint4*>(kl + 16 * (to * p.ks[1] + r * p.ks[2] + h * p.ks[3] + v)) = x;
            *reinterpret_cast<uint4*>(vl + 16 * (to * p.vs[1] + r * p.vs[2] + h * p.vs[3] + v)) = y;
        }
        return;
    }
    const int rows = len - old;
    const int total = rows * p.heads * p.vec;
    const uint8_t* const kt = p.kt + 16 * (layer * p.kts[0] + b * p.kts[1]);
    const uint8_t* const vt = p.vt + 16 * (layer * p.vts[0] + b * p.vts[1]);
    const int32_t* const tab = p.table + b * p.table_stride;
    for (int i = tid; i < total; i += kThreads) {
        const int v = i % p.vec, rh = i / p.vec;
        const int h = rh % p.heads, r = rh / p.heads;
        const int node = p.nodes ? p.nodes[static_cast<int64_t>(b) * p.N + r] : r;
        const int at = old + r, blk = at >> p.ps_shift, slot = at & psm;
        const int64_t page = blk < have ? tab[blk] : fresh[e[3] + blk - have];
        const uint4 x = *reinterpret_cast<const uint4*>(kt + 16 * (node * p.kts[2] + h * p.kts[3] + v));
        const uint4 y = *reinterpret_cast<const uint4*>(vt + 16 * (node * p.vts[2] + h * p.vts[3] + v));
        *reinterpret_cast<uint4*>(kl + 16 * (page * p.ks[1] + slot * p.ks[2] + h * p.ks[3] + v)) = x;
        *reinterpret_cast<uint4*>(vl + 16 * (page * p.vs[1] + slot * p.vs[2] + h * p.vs[3] + v)) = y;
    }
}

}  // namespace

hipError_t launch_cache_plan(const CacheParams& p, hipStream_t st, const LaunchEvents& ev) {
    const unsigned lds = static_cast<unsigned>((p.pages + 31) / 32) * 4;
    if (lds > (32u << 10)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_cache_plan),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return e;
    }
    hipExtLaunchKernelGGL(k_cache_plan, dim3(1), dim3(kPlanThreads), lds, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

hipError_t launch_cache_copy(const CacheParams& p, hipStream_t st, const LaunchEvents& ev) {
    hipExtLaunchKernelGGL(k_cache_copy, dim3(p.B, p.layers + 1), dim3(kThreads), 0, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

}  // namespace sv
