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
    return a < 0 ? -1 : __hip_atomic_load(first + a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Per-sequence values of the plan: in LDS for up to as many sequences as the
// workgroup has threads, else in the workspace (one word each per sequence):
// fork of 64 sequences 5.4 and 6.3 us, commit 6.0 and 6.8.
struct PlanArrays {
    int32_t *len, *have, *row, *first;
};

constexpr int kOwn = -2;  // such a page is there, not read yet (-1: there is none)

// SMALL: one thread per sequence.  Loads are issued for many sequences or
// entries at a time; what the kernel costs for a pool of a few thousand pages is
// a chain of three memory latencies (lengths, tables, writes), the barriers and
// the launch: 4 to 7 us.  Looking for free pages, each thread at its run of the
// bitmap page by page, outgrows that in larger pools: commit 41 us at 65536
// pages and 0.56 ms at 2^20 (fork 32 us and 0.44 ms).
template <bool SMALL>
__global__ __launch_bounds__(kPlanThreads) void k_cache_plan(CacheParams p) {
    extern __shared__ uint32_t used[];  // W words
    __shared__ int s_wave[kPlanWaves];
    __shared__ int s_bad;
    __shared__ int32_t s_arr[SMALL ? 4 * kPlanThreads : 1];
    const int tid = threadIdx.x;
    const int W = (p.pages + 31) / 32;
    const int64_t cap = static_cast<int64_t>(p.width) << p.ps_shift;
    int32_t* const plan = p.plan;
    int32_t* const spare = plan + static_cast<int64_t>(p.B) * kPlanWords;
    int32_t* const fresh = spare + static_cast<int64_t>(p.B) * kPlanSpare;  // the new pages, in order
    // rows of the tables that count (have entries of row `row`), old lengths, and `first`: for a fork
    // the lowest slot of each ancestor, for a commit the partly filled page that is appended to
    const PlanArrays s = SMALL ? PlanArrays{s_arr, s_arr + kPlanThreads, s_arr + 2 * kPlanThreads,
                                            s_arr + 3 * kPlanThreads}
                               : PlanArrays{spare, spare + p.B, spare + 2 * static_cast<int64_t>(p.B),
                                            spare + 3 * static_cast<int64_t>(p.B)};
    bool bad = false;
    // the tables' first entries are on their way while the lengths are looked at
    constexpr int kAhead = 4;
    const int64_t entries = static_cast<int64_t>(p.B) * p.width;
    int32_t ahead[kAhead];
    uint32_t seq[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int64_t i = tid + static_cast<int64_t>(k) * kPlanThreads;
        ahead[k] = 0;
        seq[k] = i < entries ? static_cast<uint32_t>(i) / static_cast<uint32_t>(p.width) : 0;
        if (i < entries) ahead[k] = p.table[seq[k] * p.table_stride + (i - static_cast<int64_t>(seq[k]) * p.width)];
    }
    for (int b = tid; b < p.B; b += kPlanThreads) {
        s.len[b] = p.len[b];
        if (p.fork) s.first[b] = 0x7FFFFFFF;
    }
    for (int i = tid; i < W; i += kPlanThreads) used[i] = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    if (p.fork) {
        for (int b = tid; b < p.B; b += kPlanThreads) {
            const int a = p.ancestor[b];
            if (a >= p.B || a < -1)
                bad = true;
            else if (a >= 0)
                atomicMin(s.first + a, b);
            s.row[b] = a >= 0 && a < p.B ? a : -1;
        }
        __syncthreads();
    }
    // lengths, pages kept, new pages; of row b of the tables `have[b]` entries are in use
    for (int b = tid; b < p.B; b += kPlanThreads) {
        const int old = s.len[b];
        int len = old, want = 0, have = 0;
        if (p.fork) {
            const int a = s.row[b];
            len = a >= 0 ? s.len[a] : 0;
            if (old < 0 || old > cap || len < 0 || len > cap) {
                bad = true;
                len = 0;
            }
            want = blocks_of(len, p.ps_shift);
            have = len >> p.ps_shift;
            // a partly filled last page stays with the lowest slot
            if (have < want && first_of(s.first, a) == b) have = want;
            // the whole ancestor counts, if someone continues it
            const bool go_on = first_of(s.first, b) != 0x7FFFFFFF && old >= 0 && old <= cap;
            s.have[b] = go_on ? blocks_of(old, p.ps_shift) : 0;
        } else {
            const int n = p.n_accepted[b];
            int rows = n < 0 ? 0 : n >= p.N ? p.N + 1 : n + 1;
            if (len < 0 || len > cap || rows > p.N || len + static_cast<int64_t>(rows) > cap) {
                bad = true;
                len = rows = 0;
            }
            have = blocks_of(len, p.ps_shift);
            s.have[b] = have;
            s.row[b] = rows;
            s.first[b] = rows > 0 && (len & ((1 << p.ps_shift) - 1)) ? kOwn : -1;
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
    // the pages in use
    auto mark = [&](uint32_t b, int64_t j, int pg) {
        if (j >= s.have[b]) return;
        if (pg < 0 || pg >= p.pages)
            bad = true;
        else if (!p.fork && j == s.have[b] - 1 && s.first[b] == kOwn)
            s.first[b] = pg;  // marked after all others
        else
            atomicOr(&used[pg % W], 1u << (pg / W));
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int64_t i = tid + static_cast<int64_t>(k) * kPlanThreads;
        if (i < entries) mark(seq[k], i - static_cast<int64_t>(seq[k]) * p.width, ahead[k]);
    }
    for (int64_t at = tid + static_cast<int64_t>(kAhead) * kPlanThreads; at < entries;
         at += static_cast<int64_t>(kAhead) * kPlanThreads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t i = at + static_cast<int64_t>(k) * kPlanThreads;
            seq[k] = i >> 32 ? static_cast<uint32_t>(i / p.width)
                             : static_cast<uint32_t>(i) / static_cast<uint32_t>(p.width);
            const int64_t j = i - static_cast<int64_t>(seq[k]) * p.width;
            ahead[k] = i < entries && j < s.have[seq[k]] ? p.table[seq[k] * p.table_stride + j] : 0;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t i = at + static_cast<int64_t>(k) * kPlanThreads;
            if (i < entries) mark(seq[k], i - static_cast<int64_t>(seq[k]) * p.width, ahead[k]);
        }
    }
    if (!p.fork && p.nodes) {
        for (int i = tid; i < p.B * p.N; i += kPlanThreads) {
            const int b = i / p.N, j = i - b * p.N;
            if (j < s.row[b]) {
                const int node = p.nodes[i];
                if (node < 0 || node >= p.N) bad = true;
            }
        }
    }
    if (!p.fork) {
        // the pages that are appended to: nobody else may name them
        __syncthreads();
        for (int b = tid; b < p.B; b += kPlanThreads) {
            const int pg = s.first[b];
            if (pg < 0) continue;
            const uint32_t bit = 1u << (pg / W);
            if (atomicOr(&used[pg % W], bit) & bit) bad = true;
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
    const int32_t* const fresh = p.plan + static_cast<int64_t>(p.B) * (kPlanWords + kPlanSpare);
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
    const int per_row = p.heads * p.vec;
    const int64_t ksr = p.fork ? p.ks[2] : p.kts[2], ksh = p.fork ? p.ks[3] : p.kts[3];
    const int64_t vsr = p.fork ? p.vs[2] : p.vts[2], vsh = p.fork ? p.vs[3] : p.vts[3];
    const uint8_t *ksrc, *vsrc;
    int64_t page_new = 0;
    int total;
    if (p.fork) {
        const int want = blocks_of(len, p.ps_shift);
        if (have == want) return;  // nothing to copy: empty, full pages only, or the page's keeper
        const int64_t page_old = p.table[a * p.table_stride + have];
        page_new = fresh[e[3]];
        total = (len & psm) * per_row;
        ksrc = kl + 16 * (page_old * p.ks[1]);
        vsrc = vl + 16 * (page_old * p.vs[1]);
    } else {
        total = (len - old) * per_row;
        ksrc = p.kt + 16 * (layer * p.kts[0] + b * p.kts[1]);
        vsrc = p.vt + 16 * (layer * p.vts[0] + b * p.vts[1]);
    }
    const int32_t* const tab = p.table + b * p.table_stride;
    // element i of the rows to move: source row, destination page and slot, head, vector
    struct Place {
        int node, slot, h, v;
        int64_t page;
    };
    auto place = [&](int i) __attribute__((always_inline)) {
        Place q;
        const int r = i / per_row, hv = i - r * per_row;
        q.h = hv / p.vec;
        q.v = hv - q.h * p.vec;
        if (p.fork) {
            q.node = q.slot = r;
            q.page = page_new;
        } else {
            q.node = p.nodes ? p.nodes[static_cast<int64_t>(b) * p.N + r] : r;
            const int at = old + r, blk = at >> p.ps_shift;
            q.page = blk < have ? tab[blk] : fresh[e[3] + blk - have];
            q.slot = at & psm;
        }
        return q;
    };
    auto from = [&](const uint8_t* s, int64_t sr, int64_t sh, const Place& q) __attribute__((always_inline)) {
        return *reinterpret_cast<const uint4*>(s + 16 * (q.node * sr + q.h * sh + q.v));
    };
    auto put = [&](uint8_t* d, const int64_t* s, const Place& q, const uint4& x) __attribute__((always_inline)) {
        *reinterpret_cast<uint4*>(d + 16 * (q.page * s[1] + q.slot * s[2] + q.h * s[3] + q.v)) = x;
    };
    // four loads under way per thread before the first store
    int i = tid;
    for (; i + kThreads < total; i += 2 * kThreads) {
        const Place q0 = place(i), q1 = place(i + kThreads);
        const uint4 k0 = from(ksrc, ksr, ksh, q0), v0 = from(vsrc, vsr, vsh, q0);
        const uint4 k1 = from(ksrc, ksr, ksh, q1), v1 = from(vsrc, vsr, vsh, q1);
        put(kl, p.ks, q0, k0);
        put(vl, p.vs, q0, v0);
        put(kl, p.ks, q1, k1);
        put(vl, p.vs, q1, v1);
    }
    if (i < total) {
        const Place q = place(i);
        const uint4 k0 = from(ksrc, ksr, ksh, q), v0 = from(vsrc, vsr, vsh, q);
        put(kl, p.ks, q, k0);
        put(vl, p.vs, q, v0);
    }
}

}  // namespace

namespace {
template <bool SMALL>
hipError_t plan_launch(const CacheParams& p, hipStream_t st, const LaunchEvents& ev) {
    const unsigned lds = static_cast<unsigned>((p.pages + 31) / 32) * 4;
    if (lds > (32u << 10)) {
        // always the largest amount: calls of other sizes may run at the same time
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_cache_plan<SMALL>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, kMaxPages / 8);
        if (e != hipSuccess) return e;
    }
    hipExtLaunchKernelGGL((k_cache_plan<SMALL>), dim3(1), dim3(kPlanThreads), lds, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_cache_plan(const CacheParams& p, hipStream_t st, const LaunchEvents& ev) {
    return p.B <= kPlanThreads ? plan_launch<true>(p, st, ev) : plan_launch<false>(p, st, ev);
}

hipError_t launch_cache_copy(const CacheParams& p, hipStream_t st, const LaunchEvents& ev) {
    hipExtLaunchKernelGGL(k_cache_copy, dim3(p.B, p.layers + 1), dim3(kThreads), 0, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

}  // namespace sv
