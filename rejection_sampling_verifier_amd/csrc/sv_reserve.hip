// gfx950 kernels of the reservation of cache rows, and of their writing.
//
// As everywhere, the block tables are the whole state: a page is in use if a
// live entry names it.  A reservation lengthens every sequence by its own number
// of rows, takes the lowest free pages in the order of the sequences, and lists
// where the new rows go.
//
//   k_reserve_plan   one workgroup: the places of all sequences in the list of
//                    rows and in that of new pages, the pages in use as a bitmap
//                    in LDS, the lowest free ones, the status.
//   k_reserve_write  the rest of the device: table rows, lengths, slots, positions.
//   k_cache_write    rows into their slots.
//
// The bitmap holds page i in word 32 (i / 1024) + i % 32, bit (i / 32) % 32: the
// consecutive pages of a sequence fall into different words, so that the LDS
// atomics do not queue up, and a vote over 32 lanes on bit j gives the pages
// 1024 k + 32 j + 0..31 in order.

#include <hip/hip_ext.h>

#include "sv_beam.h"

namespace sv {
namespace {

constexpr int kPlanThreads = 1024, kPlanWaves = 16;
constexpr int kFlight = 16;  // segments of table entries a wave has under way

__device__ __forceinline__ int blocks_of(int64_t rows, int ps_shift) {
    return static_cast<int>((rows + (1 << ps_shift) - 1) >> ps_shift);
}

// Sum of `v` over the threads before this one, and over all of them.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_wave, int64_t& all) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t up = __shfl_up(static_cast<long long>(s), o);
        if (lane >= o) s += up;
    }
    __syncthreads();
    if (lane == 63) s_wave[w] = s;
    __syncthreads();
    int64_t before = 0;
    all = 0;
#pragma unroll
    for (int i = 0; i < kPlanWaves; ++i) {
        if (i < w) before += s_wave[i];
        all += s_wave[i];
    }
    return before + s - v;
}

__device__ __forceinline__ int word_of(int page) { return (page >> 10 << 5) | (page & 31); }
__device__ __forceinline__ uint32_t bit_of(int page) { return 1u << (page >> 5 & 31); }

// SMALL: at most one sequence per thread, whose values the tables' walk reads from LDS.
template <bool SMALL>
__global__ __launch_bounds__(kPlanThreads) void k_reserve_plan(ReserveParams p) {
    extern __shared__ uint32_t used[];  // 64 words for every 2048 pages
    __shared__ int64_t s_wave[kPlanWaves];
    __shared__ int s_bad, s_segs[SMALL ? kPlanThreads + 1 : 1], s_have[SMALL ? kPlanThreads : 1],
        s_last[SMALL ? kPlanThreads : 1];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int chunks = (p.pages + 2047) >> 11;
    const int64_t cap = static_cast<int64_t>(p.width) << p.ps_shift;
    int32_t* const fresh = p.plan + static_cast<int64_t>(p.B) * kReserveWords;  // the new pages, in order
    // per sequence: 64-entry segments of live entries before it, live entries, and the page it appends
    // to (the last of them; -1 where there is none), which is marked after all others
    bool bad = false;
    for (int i = tid; i < chunks * 64; i += kPlanThreads) used[i] = 0;
    if (tid == 0) s_bad = 0;
    int64_t segs = 0, rows = 0, need = 0;
    for (int base = 0; base < p.B; base += kPlanThreads) {
        const int b = base + tid;
        int old = 0, have = 0, want = 0, n = 0;
        int64_t len = 0;
        if (b < p.B) {
            len = old = p.len[b];
            n = p.n_new[b];
            if (n < 0) n = 0;
            if (len < 0 || len > cap || len + n > cap) {
                bad = true;
                len = n = 0;
            }
            have = blocks_of(len, p.ps_shift);
            want = blocks_of(len + n, p.ps_shift);
        }
        int64_t all;
        const int seg = (have + 63) >> 6;
        const int64_t s = block_scan(seg, s_wave, all) + segs;
        segs += all;
        const int64_t r = block_scan(n, s_wave, all) + rows;
        rows += all;
        const int64_t f = block_scan(want - have, s_wave, all) + need;
        need += all;
        if (b < p.B) {
            int mine = -1;
            if (n > 0 && (len & ((1 << p.ps_shift) - 1))) {
                mine = p.table[b * p.table_stride + have - 1];
                if (mine < 0 || mine >= p.pages) {
                    bad = true;
                    mine = -1;
                }
            }
            int32_t* const e = p.plan + static_cast<int64_t>(b) * kReserveWords;
            e[0] = old;
            e[1] = static_cast<int32_t>(len + n);
            e[2] = have;
            e[3] = static_cast<int32_t>(f > 0x7FFFFFFF ? 0 : f);
            e[4] = static_cast<int32_t>(r > 0x7FFFFFFF ? 0 : r);
            if (SMALL) {
                s_segs[b] = static_cast<int>(s);
                s_have[b] = have;
                s_last[b] = mine;
            } else {
                e[5] = static_cast<int32_t>(s);
                e[6] = mine;
            }
        }
    }
    if (rows > p.rows) bad = true;
    __syncthreads();
    auto segs_before = [&](int b) { return SMALL ? s_segs[b] : p.plan[static_cast<int64_t>(b) * kReserveWords + 5]; };
    auto have_of = [&](int b) { return SMALL ? s_have[b] : p.plan[static_cast<int64_t>(b) * kReserveWords + 2]; };
    auto last_of = [&](int b) { return SMALL ? s_last[b] : p.plan[static_cast<int64_t>(b) * kReserveWords + 6]; };
    // the pages in use: wave w takes segments w, w + 16, ...; each lane finds the sequence of one
    for (int64_t at = w; at < segs; at += 64 * kPlanWaves) {
        const int64_t mine = at + static_cast<int64_t>(lane) * kPlanWaves;
        int seq = 0, from = 0, have = 0;
        if (mine < segs) {
            for (int hi = p.B; hi - seq > 1;) {  // the last sequence with segments before it <= mine
                const int mid = (seq + hi) >> 1;
                if (segs_before(mid) <= mine)
                    seq = mid;
                else
                    hi = mid;
            }
            from = static_cast<int>(mine - segs_before(seq)) * 64;
            have = have_of(seq) - (last_of(seq) >= 0);
        }
        const int count = static_cast<int>(min(static_cast<int64_t>(64), (segs - at + kPlanWaves - 1) / kPlanWaves));
        constexpr int kNone = -2;  // no entry here
        for (int k0 = 0; k0 < count; k0 += kFlight) {
            int page[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const int b = __builtin_amdgcn_readlane(seq, (k0 + k) & 63);
                const int j = __builtin_amdgcn_readlane(from, (k0 + k) & 63) + lane;
                const int h = k0 + k < count ? __builtin_amdgcn_readlane(have, (k0 + k) & 63) : 0;
                page[k] = j < h ? max(p.table[b * p.table_stride + j], -1) : kNone;
            }
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const int pg = page[k];
                if (static_cast<uint32_t>(pg) < static_cast<uint32_t>(p.pages))
                    atomicOr(&used[word_of(pg)], bit_of(pg));
                else
                    bad |= pg != kNone;
            }
        }
    }
    __syncthreads();
    // the pages that are appended to: nobody else may name them
    for (int b = tid; b < p.B; b += kPlanThreads) {
        const int pg = last_of(b);
        if (pg < 0) continue;
        const uint32_t bit = bit_of(pg);
        if (atomicOr(&used[word_of(pg)], bit) & bit) bad = true;
    }
    if (bad) s_bad = 1;
    __syncthreads();
    // free pages: each wave a run of chunks of 2048 (two halves of 32 words, one word a lane)
    const int per = (chunks + kPlanWaves - 1) / kPlanWaves, c0 = min(w * per, chunks), c1 = min(c0 + per, chunks);
    auto free_word = [&](int c) {
        uint32_t x = ~used[c * 64 + lane];
        // pages past the pool: bit j of this lane is page (2 c + lane / 32) 1024 + 32 j + lane % 32
        const int first = (2 * c + (lane >> 5)) * 1024 + (lane & 31), left = (p.pages - first + 31) >> 5;
        if (left < 32) x &= left <= 0 ? 0u : (1u << left) - 1;
        return x;
    };
    int mine = 0;
    for (int c = c0; c < c1; ++c) mine += __popc(free_word(c));
    int64_t n_free;
    int64_t rank = block_scan(mine, s_wave, n_free);
    const bool fail = s_bad != 0;
    if (tid == 0)
        *p.status = fail ? -1 : need > n_free ? static_cast<int32_t>(min(need - n_free, static_cast<int64_t>(1) << 30)) : 0;
    if (fail || need > n_free) return;
    rank = __shfl(static_cast<long long>(rank), 0);  // free pages before the wave's
    for (int c = c0; c < c1 && rank < need; ++c) {
        const uint32_t x = free_word(c);
        int low = __popc(x);  // of both halves of the chunk
        for (int o = 1; o < 32; o <<= 1) low += __shfl_xor(low, o);
        const int first_half = __builtin_amdgcn_readlane(low, 0), all = first_half + __builtin_amdgcn_readlane(low, 32);
        int64_t at = rank + (lane < 32 ? 0 : first_half);
        const int base = (2 * c + (lane >> 5)) * 1024 + (lane & 31);
        for (int j = 0; j < 32; ++j) {
            const uint64_t vote = __ballot(x >> j & 1);
            const uint32_t half = static_cast<uint32_t>(lane < 32 ? vote : vote >> 32);
            const int64_t place = at + __popc(half & ((1u << (lane & 31)) - 1));
            if ((x >> j & 1) && place < need) fresh[place] = base + 32 * j;
            at += __popc(half);
        }
        rank += all;
    }
}

// blockIdx.x: sequence, or past the last the places of the list that are left over; blockIdx.y: a
// share of its rows, the first also the table row.
__global__ __launch_bounds__(kThreads) void k_reserve_write(ReserveParams p) {
    const int b = blockIdx.x, tid = threadIdx.x;
    const bool done = *p.status == 0;
    const int32_t* const fresh = p.plan + static_cast<int64_t>(p.B) * kReserveWords;
    const int step = gridDim.y * kThreads, i0 = blockIdx.y * kThreads + tid;
    if (b == p.B) {
        int from = 0;
        if (done) {
            const int32_t* const e = p.plan + static_cast<int64_t>(p.B - 1) * kReserveWords;
            from = e[4] + e[1] - e[0];
        }
        for (int64_t i = from + i0; i < p.rows; i += step) {
            p.slots[i] = -1;
            p.position[i] = -1;
        }
        if (i0 == 0) p.start[p.B] = from;
        return;
    }
    const int32_t* const e = p.plan + static_cast<int64_t>(b) * kReserveWords;
    const int old = e[0], len = e[1], have = e[2], place = e[3], first = e[4];
    const int32_t* const src = p.table + b * p.table_stride;
    if (done) {
        for (int64_t i = i0; i < len - old; i += step) {
            const int at = static_cast<int>(old + i), blk = at >> p.ps_shift;
            const int page = blk < have ? src[blk] : fresh[place + blk - have];
            p.slots[first + i] = (page << p.ps_shift) + (at & ((1 << p.ps_shift) - 1));
            p.position[first + i] = at;
        }
    }
    if (blockIdx.y) return;
    const int64_t cap = static_cast<int64_t>(p.width) << p.ps_shift;
    const int live = done ? blocks_of(len, p.ps_shift) : old < 0 ? 0 : blocks_of(old > cap ? cap : old, p.ps_shift);
    int32_t* const dst = p.out_table + b * p.out_stride;
    for (int j = tid; j < p.width; j += kThreads) {
        int v = -1;
        if (j < live) v = done && j >= have ? fresh[place + j - have] : src[j];
        dst[j] = v;
    }
    if (tid == 0) {
        p.out_len[b] = done ? len : old;
        p.start[b] = done ? first : 0;
    }
}

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Row t of a, and of b behind it, becomes the cache row in slot slots[t]; a slot
// outside the cache takes nothing.  16 bytes a thread and step, four under way.
// The stores are nontemporal: 41000 rows of 1152 bytes take 16 us (5.9 TB/s read and
// written), with ordinary stores 34.
__global__ __launch_bounds__(kThreads) void k_cache_write(WriteParams p) {
    const int vec = p.va + p.vb;
    const int64_t n = static_cast<int64_t>(p.T) * vec, step = static_cast<int64_t>(gridDim.x) * kThreads;
    const int mask = (1 << p.ps_shift) - 1;
    constexpr int kAtOnce = 4;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i0 < n; i0 += kAtOnce * step) {
        u32x4 y[kAtOnce];
        uint8_t* to[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t i = i0 + k * step;
            to[k] = nullptr;
            if (i >= n) continue;
            const int t = i >> 32 ? static_cast<int>(i / vec)
                                  : static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(vec));
            const int v = static_cast<int>(i - static_cast<int64_t>(t) * vec);
            const int slot = p.slots[t];
            if (slot < 0 || slot >= p.all) continue;
            to[k] = p.cache + 16 * ((slot >> p.ps_shift) * p.cs[0] + (slot & mask) * p.cs[1] + v);
            y[k] = *reinterpret_cast<const u32x4*>(v < p.va ? p.a + 16 * (t * p.as + v) : p.b + 16 * (t * p.bs + v - p.va));
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (to[k]) __builtin_nontemporal_store(y[k], reinterpret_cast<u32x4*>(to[k]));
    }
}

template <bool SMALL>
hipError_t plan_launch(const ReserveParams& p, hipStream_t st, const LaunchEvents& ev) {
    const unsigned lds = static_cast<unsigned>((p.pages + 2047) / 2048) * 256;
    if (lds > (32u << 10)) {
        // always the largest amount: calls of other sizes may run at the same time
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_reserve_plan<SMALL>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, kMaxPages / 8);
        if (e != hipSuccess) return e;
    }
    hipExtLaunchKernelGGL((k_reserve_plan<SMALL>), dim3(1), dim3(kPlanThreads), lds, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_reserve_plan(const ReserveParams& p, hipStream_t st, const LaunchEvents& ev) {
    return p.B <= kPlanThreads ? plan_launch<true>(p, st, ev) : plan_launch<false>(p, st, ev);
}

hipError_t launch_reserve_write(const ReserveParams& p, hipStream_t st, const LaunchEvents& ev) {
    // a thread for every place of the list, if they are spread evenly
    int64_t share = (p.rows / (p.B + 1) + kThreads) / kThreads;
    if (share > 64) share = 64;
    hipExtLaunchKernelGGL(k_reserve_write, dim3(p.B + 1, static_cast<unsigned>(share)), dim3(kThreads), 0, st, ev.start,
                          ev.stop, 0, p);
    return hipGetLastError();
}

hipError_t launch_cache_write(const WriteParams& p, hipStream_t st, const LaunchEvents& ev) {
    int64_t blocks = (static_cast<int64_t>(p.T) * (p.va + p.vb) + 4 * kThreads - 1) / (4 * kThreads);
    if (blocks > 8192) blocks = 8192;
    hipExtLaunchKernelGGL(k_cache_write, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, st, ev.start, ev.stop,
                          0, p);
    return hipGetLastError();
}

}  // namespace sv
