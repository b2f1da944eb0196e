// gfx950 kernels of tree attention: the nodes of a drafted tree attend to the
// paged cache of their sequence and to their own ancestors.
//
// For every sequence b, node i of depth d and query head e of key head h,
//
//   o = sum_j w_j v_j / sum_j w_j,   w_j = 2^(x_j - m),  x_j = scale log2(e) q.k_j,
//
// over the cache rows j < len (all of them, or with a window w those with
// len + d - j < w or j < sinks) and the tree rows that are i or its ancestors
// (with a window the nearest w of them).
//
// One workgroup takes up to 32, 64 or 128 of the N * G query rows that share a
// key head, so that K and V are read once for all of them, and walks over
// tiles of keys with a running maximum and sum in float32:
//
//   S^T = K Q^T by 32x32x16 MFMA: K is the A operand (16-byte reads of the
//   row-major LDS tile), Q^T the B operand, resident in registers.  A lane
//   then holds one query row (column lane & 31) and 16 of 32 keys, in groups
//   of four: the softmax needs one exchange between the half-waves per tile.
//
//   O^T += V^T P^T: the same lane's 16 weights, rounded to the input type,
//   are the B operand as they stand when the contraction's key order is the
//   one the accumulator layout gives (step t, half h: keys 16 t + 4 h + 0..3,
//   then 16 t + 8 + 4 h + 0..3).  V^T is the A operand in that order, read
//   from the row-major tile by the 4 x 16 transposing LDS load.
//
// The rounding of the weights is the only one below float32 before the output's
// own: bf16 2^-8 relative at most; fp16 2^-11 relative, or 2^-32 of the row's
// largest weight where that is more (weights below 2^-21 of it).  The reference
// m is raised to the largest score (fp16: 7 less) only when a row's new scores
// exceed it by more than 8 (15), so weights reach 2^8 (2^15) at most; the sum
// uses the unrounded weights.
//
// The tiles of all sequences and key heads form one line that is cut into
// equal parts (one per workgroup, or per group of workgroups when the rows
// need several tiles): ragged lengths cost no idle workgroups, and one long
// sequence fills the device.  A (sequence, key head) that a cut divides leaves
// partial (O, m, l) records that k_tree_merge joins in part order, so results
// do not depend on timing.
//
// What bounds it: up to 64 rows per key head the cache's bytes (64 sequences of
// 8192 rows, 8 key heads of 128: 2.1 GB at 5.9 TB/s with 4 to 24 rows, 5.5 with
// 64, of the 7.1 a plain read reaches; 13 TB/s where the rows come from the L2),
// then the matrix instructions and the softmax between them (128 rows 620
// TFLOP/s, 256 rows 740).  A workgroup's two stages keep 32 KB (64 KB with 32
// rows) of K and V under way while the tile before is computed.  Separate slots
// for K and V, refilled one by one, made more instructions and ran 4 to 12 %
// slower; one stage and two workgroups per CU (32 rows) ran 10 % slower from
// memory.  Short calls are a chain of latencies (lengths, table, first tile,
// join): one sequence of a thousand rows takes 11 us and 4 for the join.
//
// Rows of the tile that no query sees (past the length, past the tree, on a
// page outside the pool) are staged as zeros.  Where some rows see a key and
// others do not, infinities and NaN among the values are kept out of the MFMA
// and added for the rows that see them only.

#include <hip/hip_ext.h>

#include "sv_attn.h"
#include "sv_tree.h"

namespace sv {
namespace {

// The K operand of one 32-key subtile, and the V operand of 16 keys, from a
// stage.  The loads are assembly so that the compiler does not wait for the
// next stage's loads before them (it cannot tell the stages apart); each block
// waits for its own.
template <int DP>
__device__ __forceinline__ void read_k(const uint32_t* rd, uint32_t stage, int ks, v8s* r) {
    const uint32_t a0 = rd[0] + stage, a1 = rd[1] + stage, a2 = rd[2] + stage, a3 = rd[3] + stage;
    const int off = ks * 64 * DP;
    if constexpr (DP == 128)
        asm volatile(
            "ds_read_b128 %0, %8 offset:%12\n\tds_read_b128 %1, %9 offset:%12\n\t"
            "ds_read_b128 %2, %10 offset:%12\n\tds_read_b128 %3, %11 offset:%12\n\t"
            "ds_read_b128 %4, %8 offset:%13\n\tds_read_b128 %5, %9 offset:%13\n\t"
            "ds_read_b128 %6, %10 offset:%13\n\tds_read_b128 %7, %11 offset:%13\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
            : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "n"(off), "n"(off + 128)
            : "memory");
    else
        asm volatile(
            "ds_read_b128 %0, %4 offset:%8\n\tds_read_b128 %1, %5 offset:%8\n\t"
            "ds_read_b128 %2, %6 offset:%8\n\tds_read_b128 %3, %7 offset:%8\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
            : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "n"(off)
            : "memory");
}

template <int DP>
__device__ __forceinline__ void read_v(const uint32_t* rd, uint32_t stage, int step, v8s* r) {
    const uint32_t a0 = rd[0] + stage, a1 = rd[1] + stage;
    const int lo = step * 32 * DP, hi = lo + 16 * DP;  // rows 16 step and 8 more
    v4s x[2 * (DP / 32)];
    if constexpr (DP == 128) {
        const uint32_t a2 = rd[2] + stage, a3 = rd[3] + stage;
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
            "ds_read_b64_tr_b16 %2, %9 offset:%12\n\tds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
            "ds_read_b64_tr_b16 %4, %10 offset:%12\n\tds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
            "ds_read_b64_tr_b16 %6, %11 offset:%12\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
            : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "n"(lo), "n"(hi)
            : "memory");
    } else {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %4 offset:%6\n\tds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
            "ds_read_b64_tr_b16 %2, %5 offset:%6\n\tds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
            : "v"(a0), "v"(a1), "n"(lo), "n"(hi)
            : "memory");
    }
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
        r[dt] = __builtin_shufflevector(x[2 * dt], x[2 * dt + 1], 0, 1, 2, 3, 4, 5, 6, 7);
}

// The cache rows of one sequence in tiles: tiles [0, head) from the first row,
// then from tile `head + gap` to the last (the gap is what the window hides
// from every node), then one tile for the tree.
struct Tiles {
    int len, head, gap, cache;  // cache: tiles of cache rows
    __device__ __forceinline__ int total() const { return cache + 1; }
    __device__ __forceinline__ int key_tile(int t) const { return t < head ? t : t + gap; }
};

template <int TK>
__device__ __forceinline__ Tiles tiles_of(const TreeAttnParams& p, int len) {
    Tiles r;
    const int cap = p.width << p.ps_shift;
    r.len = len < 0 ? 0 : len > cap ? cap : len;
    const int all = (r.len + TK - 1) / TK;
    r.head = all;
    r.gap = 0;
    if (p.window > 0 && r.len >= p.window) {
        const int first = (r.len - p.window + 1) / TK;  // the root's window reaches back furthest
        const int kept = (min(p.sinks, r.len) + TK - 1) / TK;
        if (first > kept) {
            r.head = kept;
            r.gap = first - kept;
        }
    }
    r.cache = all - r.gap;
    return r;
}

template <int DT, int DP, int WR>
__global__ __launch_bounds__(kThreads, 2) void k_tree_attn(TreeAttnParams p) {
    constexpr int WK = kWaves / WR;           // waves over keys
    constexpr int RB = 32 * WR;               // query rows
    constexpr bool kShared = WR > 1;          // the waves share their tiles
    constexpr int TK = kShared ? 64 : 128;    // keys per tile
    constexpr int GK = kShared ? 64 : 32;     // of them in one staged group: the tile, or a wave's quarter
    constexpr int KS = TK / (32 * WK);        // 32-key subtiles per wave
    constexpr int NC = DP / 8;                // 16-byte chunks per row
    constexpr int NQ = DP / 16, ND = DP / 32;
    constexpr int kRowB = DP * 2;
    constexpr int kRowsPerLoad = 64 / NC;     // rows one wide load of a wave stages
    constexpr int kRowsPerWave = kShared ? GK / kWaves : GK;
    constexpr int kLoads = kRowsPerWave / kRowsPerLoad;
    constexpr int kVAt = GK * kRowB;          // V behind K in a stage
    constexpr int kStageB = 2 * GK * kRowB;
    constexpr int kGroups = kShared ? 1 : kWaves;

    // dynamic: with a size it knew, the compiler would give a kernel of one
    // workgroup per CU accumulation registers, and move the sums in and out of
    // them in every tile
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int kSlowB = kShared && kStageB < 4 * 8192 ? 4 * 8192 : 0;  // where a stage is too small for the slow path
    uint8_t* const slow = smem + kGroups * 2 * kStageB;
    __shared__ int s_nf;
    constexpr int kOut = DP / 8 / WK;         // groups of four dimensions a wave's lane writes
    static_assert(WK == 1 || kWaves * 32 * DP * 4 <= kGroups * 2 * kStageB, "the waves' results fit the stages");
    __shared__ float s_ml[kWaves][2][64];
    __shared__ int64_t s_sum[kWaves];
    __shared__ int32_t s_scan[kWaves];
    __shared__ int s_b;
    __shared__ int64_t s_before;

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = w % WR, wk = w / WR, hh = lane >> 5, col = lane & 31;
    int c, m;
    if (p.MT == 1) {
        c = blockIdx.x;
        m = 0;
    } else {  // the row tiles of a part on one XCD (workgroups go to the eight in turn)
        const int per = 8 * p.MT;
        c = (blockIdx.x / per) * 8 + (blockIdx.x & 7);
        m = (blockIdx.x % per) / 8;
    }
    if (c >= p.clusters) return;

    // this workgroup's tiles [f0, f1) of the line, and the sequence f0 is in
    int64_t f0, f1, before;
    int b;
    if (!p.merge) {
        b = c / p.Hkv;
        before = 0;
        const int T = tiles_of<TK>(p, p.len[b]).total();
        f0 = static_cast<int64_t>(c % p.Hkv) * T;
        f1 = f0 + T;
    } else {
        int64_t sum = 0;
        for (int i = tid; i < p.B; i += kThreads) sum += tiles_of<TK>(p, p.len[i]).total();
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(static_cast<long long>(sum), o);
        if (lane == 0) s_sum[w] = sum;
        __syncthreads();
        const int64_t seqs = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
        const int64_t total = seqs * p.Hkv;
        const Cut cut(p.clusters, total);
        if (c >= cut.parts) return;
        f0 = cut.start(c);
        f1 = cut.start(c + 1);
        const bool tell = c == 0 && m == 0;  // leaves the sequences' places for the merge
        int64_t carry = 0;
        for (int base = 0; base < p.B; base += kThreads) {
            const int i = base + tid;
            const int v = i < p.B ? tiles_of<TK>(p, p.len[i]).total() : 0;
            int s = v;
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(s, o);
                if (lane >= o) s += up;
            }
            if (lane == 63) s_scan[w] = s;
            __syncthreads();
            int64_t excl = carry + s - v;
            int32_t chunk = 0;
            for (int j = 0; j < kWaves; ++j) {
                if (j < w) excl += s_scan[j];
                chunk += s_scan[j];
            }
            if (i < p.B) {
                if (excl * p.Hkv <= f0 && f0 < (excl + v) * p.Hkv) {
                    s_b = i;
                    s_before = excl;
                }
                if (tell) p.start[i] = excl;
            }
            carry += chunk;
            __syncthreads();
            if (!tell && carry * p.Hkv > f0) break;
        }
        if (tell && tid == 0) p.start[p.B] = seqs;
        b = __builtin_amdgcn_readfirstlane(s_b);
        before = s_before;
    }

    uint8_t* const ring = smem + (kShared ? 0 : w * 2 * kStageB);  // two stages
    // Staging: lane l of a load fills chunk position l % NC of row l / NC, with
    // the chunk that the tile's XOR swizzle puts there.  K rows are read 16 bytes
    // per lane, eight rows at a time; V rows by the transposing load, four rows of
    // two chunks at a time; either way the banks differ.
    const int ld_row = (kShared ? w * kRowsPerWave : 0) + lane / NC;  // row of the group in the first load
    auto k_chunk = [&](int r) { return (lane % NC) ^ (r & 7); };
    const int v_chunk = (lane % NC) ^ (DP == 128 ? ((lane / NC) & 3) << 2 : ((lane / NC >> 1) & 1) << 2);
    // reading: byte addresses within a stage (K: four, the next four are 128 bytes on; V: one per 32 dimensions)
    const uint32_t ring_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) uint8_t*)ring));
    const int sub0 = kShared ? wk * KS : 0;  // the wave's first subtile of the group
    uint32_t k_rd[4], v_rd[ND];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        k_rd[s] = ring_at + (sub0 * 32 + (lane & 31)) * kRowB + (((2 * s + hh) ^ (lane & 7)) << 4);
    {
        const int vrow = (lane & 15) >> 2;                             // row of four
        const int low = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);     // chunk of the four of 32 dimensions
        const int vx = DP == 128 ? vrow << 2 : (vrow >> 1) << 2;
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
            v_rd[dt] = ring_at + kVAt + (sub0 * 32 + 4 * hh + vrow) * kRowB + (((4 * dt + low) ^ vx) << 4) +
                       (lane & 1) * 8;
    }
    // byte offsets of the lane's chunk from the first row of a load, where a wave's rows lie
    // on one page and are stored in full (strides of a page's rows below 2^32 / 8 bytes)
    const uint32_t k_lane[2] = {static_cast<uint32_t>(units(lane / NC, p.kcs[1], k_chunk(ld_row), 1)),
                                static_cast<uint32_t>(units(lane / NC, p.kcs[1], k_chunk(ld_row + kRowsPerLoad), 1))};
    const uint32_t v_lane = static_cast<uint32_t>(units(lane / NC, p.vcs[1], v_chunk, 1));
    const bool wave_page = p.D == DP && (1 << p.ps_shift) >= kRowsPerWave && p.kcs[1] < (1u << 25) && p.vcs[1] < (1u << 25);
    const bool win = p.window > 0;
    const float scale2 = p.scale2;
    const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&kZero);

    int64_t f = f0;
    while (f < f1) {
        const Tiles tl = tiles_of<TK>(p, p.len[b]);
        const int T = tl.total();
        const uint32_t in_seq = static_cast<uint32_t>(f - before * p.Hkv);  // the host refuses more than 2^32 tiles
        const int h = static_cast<int>(in_seq / static_cast<uint32_t>(T));
        const int t0 = static_cast<int>(in_seq - static_cast<uint32_t>(h) * T);
        const int t1 = static_cast<int>(min(static_cast<int64_t>(T), t0 + (f1 - f)));
        const bool whole = t0 == 0 && t1 == T;
        int n = p.N;
        if (p.n_nodes) {
            n = p.n_nodes[b];
            n = n < 0 ? 0 : n > p.N ? p.N : n;
        }
        const int rows = n * p.G;
        const int my_row = m * RB + wr * 32 + col;
        const bool active = m * RB + wr * 32 < rows;  // the wave has rows
        float mx = -INFINITY, l = 0.f;
        v16f o[ND];
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;

        float4 fin[kOut];  // what the wave writes
#pragma unroll
        for (int j = 0; j < kOut; ++j) fin[j] = make_float4(0.f, 0.f, 0.f, 0.f);

        if (m * RB < rows) {
            const int32_t* const tab = p.table + b * p.table_stride;
            const uint8_t* const kcb = p.kc + units(h, p.kcs[2]);
            const uint8_t* const vcb = p.vc + units(h, p.vcs[2]);
            const uint8_t* const ktb = p.kt + units(b, p.kts[0], h, p.kts[2]);
            const uint8_t* const vtb = p.vt + units(b, p.vts[0], h, p.vts[2]);
            const int ps_mask = (1 << p.ps_shift) - 1;
            // first row of the group of tile t: a cache row, or a node
            auto first_row = [&](int t) {
                return (t < tl.cache ? tl.key_tile(t) * TK : 0) + (kShared ? 0 : wk * 32);
            };
            // lane j: the page of row j of the group of tile t
            auto page = [&](int t) {
                int pg = -1;
                if (t < tl.cache) {
                    const int key = first_row(t) + (lane & (GK - 1));
                    if (key < tl.len) pg = tab[key >> p.ps_shift];
                }
                return pg;
            };
            // starts staging tile t; returns the rows that exist (the others are staged as zeros)
            auto stage = [&](int t, int pg, int at) {
                const bool tree = t >= tl.cache;
                const int first = first_row(t);
                uint8_t* const dst = ring + at * kStageB + (kShared ? w * kRowsPerWave * kRowB : 0);
                if (tree) {
                    const uint64_t okm = __ballot(first + (lane & (GK - 1)) < n);
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        const int r = ld_row + i * kRowsPerLoad, kc = k_chunk(r);
                        const bool ok = okm >> r & 1;
                        const uint8_t* const ka = ktb + units(first + r, p.kts[1], kc, 1);
                        const uint8_t* const va = vtb + units(first + r, p.vts[1], v_chunk, 1);
                        to_lds(ok && kc * 8 < p.D ? ka : zero, dst + i * 1024);
                        to_lds(ok && v_chunk * 8 < p.D ? va : zero, dst + kVAt + i * 1024);
                    }
                    return okm;
                }
                const uint64_t okm = __ballot(static_cast<uint32_t>(pg) < static_cast<uint32_t>(p.pages));
                if (okm == ~0ull && wave_page) {
                    // whole rows that all exist, the wave's on one page: scalar addresses
                    const uint32_t page_of = __builtin_amdgcn_readlane(pg, kShared ? w * kRowsPerWave : 0);
                    const uint32_t slot = (first + (kShared ? w * kRowsPerWave : 0)) & ps_mask;
                    const uint8_t* ka = kcb + units(page_of, p.kcs[0], slot, p.kcs[1]);
                    const uint8_t* va = vcb + units(page_of, p.vcs[0], slot, p.vcs[1]);
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        to_lds(ka + k_lane[i & 1], dst + i * 1024);
                        to_lds(va + v_lane, dst + kVAt + i * 1024);
                        ka += units(kRowsPerLoad, p.kcs[1]);
                        va += units(kRowsPerLoad, p.vcs[1]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        const int r = ld_row + i * kRowsPerLoad, kc = k_chunk(r);
                        const bool ok = okm >> r & 1;
                        const uint32_t page_of = __shfl(pg, r);
                        const int slot = (first + r) & ps_mask;
                        const uint8_t* const ka = kcb + units(page_of, p.kcs[0], slot, p.kcs[1]) + 16 * kc;
                        const uint8_t* const va = vcb + units(page_of, p.vcs[0], slot, p.vcs[1]) + 16 * v_chunk;
                        to_lds(ok && kc * 8 < p.D ? ka : zero, dst + i * 1024);
                        to_lds(ok && v_chunk * 8 < p.D ? va : zero, dst + kVAt + i * 1024);
                    }
                }
                return okm;
            };

            int pg = page(t0);
            int pg_next = t0 + 1 < t1 ? page(t0 + 1) : -1;
            uint64_t okm = stage(t0, pg, 0);

            // queries: the B operand, resident; a negative scale is moved into their sign
            v8s q[NQ];
            {
                const bool in = my_row < rows;
                const int node = in ? my_row / p.G : 0;
                const uint8_t* const src = p.q + units(b, p.qs[0], node, p.qs[1]) +
                                           units(h * p.G + (in ? my_row - node * p.G : 0), p.qs[2]);
#pragma unroll
                for (int s = 0; s < NQ; ++s) {
                    const int d = s * 16 + hh * 8;
                    v8s z = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (in && d < p.D) z = *reinterpret_cast<const v8s*>(src + 2 * d);
                    q[s] = p.flip ? z ^ static_cast<short>(0x8000) : z;
                }
            }
            uint64_t set = 0;  // the nodes the row sees
            int low = 0;       // first cache row in the row's window
            if (t1 == T || win) {
                const int node = my_row < rows ? my_row / p.G : 0;
                const int32_t* const par_b = p.parent + static_cast<int64_t>(b) * p.N;
                const uint64_t all = ancestors(par_b, n, lane, 0);
                set = __shfl(static_cast<unsigned long long>(all), node);
                if (win) {
                    low = tl.len + __popcll(set) - p.window;  // depth + 1 nodes on the line
                    if (p.window < kMaxNodes)
                        set = __shfl(static_cast<unsigned long long>(ancestors(par_b, n, lane, p.window)), node);
                }
            }

            // bit r: this lane's row sees row r of the subtile that begins at key0
            auto seen_of = [&](int key0, uint32_t bad, bool tree) {
                uint32_t see = ~bad;
                if (tree)
                    see &= key0 < kMaxNodes ? static_cast<uint32_t>(set >> key0) : 0u;
                else if (win)
                    see &= bits_from(low - key0) | ~bits_from(p.sinks - key0);
                return see;
            };

            int at = 0;
            for (int t = t0; t < t1; ++t, at ^= 1) {
                const bool tree = t >= tl.cache;
                const int kb = first_row(t);
                const bool mixed = tree || (win && kb < tl.len + p.N - p.window);
                // this wave's loads of tile t (all that is in flight) have landed; with the
                // barrier everyone's, and everyone has read the other stage
                __builtin_amdgcn_s_waitcnt(kWaitVm0);
                if (kShared) __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                uint64_t okm_next = 0;
                if (t + 1 < t1) {
                    pg = pg_next;
                    if (t + 2 < t1) pg_next = page(t + 2);
                    okm_next = stage(t + 1, pg, at ^ 1);
                }
                bool nf = false;
                if (mixed) {
                    // infinities and NaN among the values: out of the tile, added below
                    bool mine = false;
                    uint8_t* const part = ring + at * kStageB + kVAt + (kShared ? w * kRowsPerWave * kRowB : 0);
#pragma unroll 1
                    for (int i = 0; i < kLoads; ++i) {
                        v8s* const e = reinterpret_cast<v8s*>(part + i * 1024 + lane * 16);
                        v8s y = *e;
                        const uint4 u = __builtin_bit_cast(uint4, y);
                        if (nonfinite2<DT>(u.x) || nonfinite2<DT>(u.y) || nonfinite2<DT>(u.z) || nonfinite2<DT>(u.w)) {
                            mine = true;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (nonfinite2<DT>(static_cast<uint16_t>(y[j]))) y[j] = 0;
                            *e = y;
                        }
                    }
                    if (kShared) {
                        if (tid == 0) s_nf = 0;
                        __syncthreads();
                        if (mine) s_nf = 1;
                        __syncthreads();
                        nf = __builtin_amdgcn_readfirstlane(s_nf) != 0;
                    } else {
                        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
                        nf = __any(mine);
                    }
                }
                const uint32_t stage_at = at * kStageB;
                v16f x[KS];
                uint32_t bad[KS];  // rows that nothing sees
                if (active) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        bad[ks] = ~static_cast<uint32_t>(okm >> (32 * (sub0 + ks)));
                        v8s kf[NQ];
                        read_k<DP>(k_rd, stage_at, ks, kf);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[ks][i] = 0.f;
#pragma unroll
                        for (int s = 0; s < NQ; ++s) x[ks] = mfma<DT>(kf[s], q[s], x[ks]);
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        if (mixed || bad[ks] != 0) {
                            const uint32_t see = seen_of(kb + (sub0 + ks) * 32, bad[ks], tree) >> 4 * hh;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[ks][i] = see & (1u << (8 * (i >> 2) + (i & 3))) ? x[ks][i] : -INFINITY;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) top = fmaxf(top, x[ks][i]);
                    }
                    top = scaled(half_max(top), scale2);
                    if (__any(top - mx > kUp<DT> + 8.f)) {
                        const float mn = fmaxf(mx, top - kUp<DT>);
                        const float a = shift_of(mx, mn);
                        l *= a;
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[dt][i] *= a;
                        mx = mn;
                    }
                    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            x[ks][i] = __builtin_amdgcn_exp2f(less(scaled(x[ks][i], scale2), ref));
                            l += x[ks][i];
                        }
#pragma unroll
                        for (int t2 = 0; t2 < 2; ++t2) {
                            const v4s lo = pack4<DT>(x[ks][8 * t2], x[ks][8 * t2 + 1], x[ks][8 * t2 + 2],
                                                     x[ks][8 * t2 + 3]);
                            const v4s hi = pack4<DT>(x[ks][8 * t2 + 4], x[ks][8 * t2 + 5], x[ks][8 * t2 + 6],
                                                     x[ks][8 * t2 + 7]);
                            const v8s pf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                            v8s vf[ND];
                            read_v<DP>(v_rd, stage_at, 2 * ks + t2, vf);
#pragma unroll
                            for (int dt = 0; dt < ND; ++dt) o[dt] = mfma<DT>(vf[dt], pf, o[dt]);
                        }
                    }
                }
                if (nf) {  // rare: infinities or NaN among the values, for the rows that see them
                    if (kShared) __syncthreads();  // the stage has been read
                    if (active) {
                        // the wave's weights, and 32 dimensions of its sums at a time, in LDS
                        float* const wp = reinterpret_cast<float*>(kSlowB ? slow + w * 8192 : ring + at * kStageB + (kShared ? w * 8192 : 0));
                        float* const op = wp + 1024;
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            // -1: hidden from the row (a weight of 0 may be a visible key's)
                            const uint32_t see = seen_of(kb + (sub0 + ks) * 32, bad[ks], tree) >> 4 * hh;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                wp[(8 * (i >> 2) + 4 * hh + (i & 3)) * 32 + col] =
                                    see & (1u << (8 * (i >> 2) + (i & 3))) ? x[ks][i] : -1.f;
#pragma unroll
                            for (int dt = 0; dt < ND; ++dt) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) op[i * 64 + lane] = o[dt][i];
                                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
#pragma unroll 1
                                for (int r = 0; r < 32; ++r) {
                                    if (bad[ks] >> r & 1) continue;
                                    const int key = kb + (sub0 + ks) * 32 + r;
                                    const uint8_t* const src =
                                        tree ? vtb + units(key, p.vts[1])
                                             : vcb + units(tab[key >> p.ps_shift], p.vcs[0], key & ps_mask, p.vcs[1]);
                                    const float wgt = wp[r * 32 + col];
#pragma unroll 1
                                    for (int i = 0; i < 16; ++i) {
                                        const int d = 32 * dt + 8 * (i >> 2) + 4 * hh + (i & 3);
                                        if (d >= p.D || wgt < 0.f) continue;
                                        const uint16_t e = *reinterpret_cast<const uint16_t*>(src + 2 * d);
                                        if (nonfinite2<DT>(e)) op[i * 64 + lane] += wgt * to_float<DT>(e);
                                    }
                                }
                                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[dt][i] = op[i * 64 + lane];
                            }
                        }
                    }
                    if (kShared) __syncthreads();
                }
                okm = okm_next;
            }
            l = half_sum(l);

            // the waves that share rows join their results through LDS, each for a part of
            // the dimensions: registers j0.. of every lane, four at a time
            __syncthreads();
            float* const buf = reinterpret_cast<float*>(smem);
            if constexpr (WK > 1) {
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4*>(buf + (w * (DP / 8) + dt * 4 + i / 4) * 256 + lane * 4) =
                            make_float4(o[dt][i], o[dt][i + 1], o[dt][i + 2], o[dt][i + 3]);
                s_ml[w][0][lane] = mx;
                s_ml[w][1][lane] = l;
                __syncthreads();
                float mw[WK], lw[WK];
                float mn = -INFINITY;
#pragma unroll
                for (int k = 0; k < WK; ++k) {
                    mw[k] = s_ml[wr + k * WR][0][lane];
                    lw[k] = s_ml[wr + k * WR][1][lane];
                    mn = fmaxf(mn, mw[k]);
                }
                mx = mn;
                l = 0.f;
#pragma unroll
                for (int k = 0; k < WK; ++k) {
                    mw[k] = shift_of(mw[k], mn);
                    l += mw[k] * lw[k];
                }
#pragma unroll
                for (int j = 0; j < kOut; ++j) {
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < WK; ++k) {
                        const float4 y = *reinterpret_cast<const float4*>(
                            buf + ((wr + k * WR) * (DP / 8) + wk * kOut + j) * 256 + lane * 4);
                        s.x += mw[k] * y.x;
                        s.y += mw[k] * y.y;
                        s.z += mw[k] * y.z;
                        s.w += mw[k] * y.w;
                    }
                    fin[j] = s;
                }
                __syncthreads();  // the stages are free again
            } else {
#pragma unroll
                for (int j = 0; j < kOut; ++j)
                    fin[j] = make_float4(o[j / 4][4 * (j % 4)], o[j / 4][4 * (j % 4) + 1], o[j / 4][4 * (j % 4) + 2],
                                         o[j / 4][4 * (j % 4) + 3]);
            }
        }

        // group j of the wave's results: dimensions 8 (wk kOut + j) + 4 hh + 0..3
        if (whole) {
            if (my_row < p.N * p.G) {
                const int node = my_row / p.G;
                const bool present = my_row < rows;  // an absent node's row is zero, not 0 * fin: fin may be NaN
                const float inv = 1.f / l;
                uint8_t* const dst = p.out + units(b, p.os[0], node, p.os[1]) +
                                     units(h * p.G + my_row - node * p.G, p.os[2]);
#pragma unroll
                for (int j = 0; j < kOut; ++j) {
                    const int d = 8 * (wk * kOut + j);
                    if (d < p.D)
                        *reinterpret_cast<v4s*>(dst + 2 * (d + 4 * hh)) =
                            present ? pack4<DT>(fin[j].x * inv, fin[j].y * inv, fin[j].z * inv, fin[j].w * inv)
                                    : v4s{0, 0, 0, 0};
                }
            }
        } else if (my_row < rows) {
            float* const rec =
                p.part + ((static_cast<int64_t>(c) * 2 + (f == f0 ? 0 : 1)) * p.MT + m) * (RB * (DP + 2));
            const int r = wr * 32 + col;
#pragma unroll
            for (int j = 0; j < kOut; ++j)
                if (8 * (wk * kOut + j) < p.D)
                    *reinterpret_cast<float4*>(rec + r * DP + 8 * (wk * kOut + j) + 4 * hh) = fin[j];
            if (hh == 0 && wk == 0) {
                rec[RB * DP + r] = mx;
                rec[RB * DP + RB + r] = l;
            }
        }
        f += t1 - t0;
        if (t1 == T && h == p.Hkv - 1 && f < f1) {
            before += T;
            ++b;
        }
    }
}

// Joins the partial results of the (sequence, key head)s that were divided:
// o = sum_c 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c over the parts in order.
// DP / 4 threads are a team that takes four dimensions each.  With many parts
// per (sequence, key head), a few rows on many CUs, all teams of a workgroup
// share one row's parts; else each team has a row of its own.
template <int DT, int DP, int RB, bool SPLIT>
__global__ __launch_bounds__(kThreads) void k_tree_merge(TreeAttnParams p) {
    constexpr int TEAM = DP / 4, TEAMS = kThreads / TEAM;
    constexpr int kFlight = 8;  // parts a thread loads at a time
    __shared__ float s_m[kWaves], s_l[TEAMS];
    __shared__ float4 s_o[SPLIT ? kThreads : 1];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
    const int64_t s0 = p.start[b], T = p.start[b + 1] - s0;
    const int64_t total = p.start[p.B] * p.Hkv;
    const Cut cut(p.clusters, total);
    const int64_t first = s0 * p.Hkv + h * T;
    const int c0 = cut.of(first), c1 = cut.of(first + T - 1);
    if (c0 == c1) return;
    const int team = tid / TEAM;
    const int row = SPLIT ? blockIdx.y : blockIdx.y * TEAMS + team;
    const int d = (tid % TEAM) * 4;
    if (row >= p.N * p.G) return;
    int n = p.N;
    if (p.n_nodes) {
        n = p.n_nodes[b];
        n = n < 0 ? 0 : n > p.N ? p.N : n;
    }
    const int node = row / p.G, head = row - node * p.G;
    v4s res = {0, 0, 0, 0};
    if (node < n) {
        const int m = row / RB, r = row - m * RB;
        const int64_t rec = RB * (DP + 2);
        // the first part's record is its second one unless the part begins here
        const int slot0 = cut.start(c0) == first ? 0 : 1;
        auto at = [&](int c) { return p.part + ((static_cast<int64_t>(c) * 2 + (c == c0 ? slot0 : 0)) * p.MT + m) * rec; };
        constexpr int kStep = SPLIT ? kThreads : TEAM;
        float mx = -INFINITY;
        for (int c = c0 + tid % kStep; c <= c1; c += kStep) mx = fmaxf(mx, at(c)[RB * DP + r]);
        for (int o = 1; o < (SPLIT ? 64 : TEAM); o <<= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
        if (SPLIT) {
            if ((tid & 63) == 0) s_m[tid >> 6] = mx;
            __syncthreads();
            mx = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
        }
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kStride = SPLIT ? TEAMS : 1;
        for (int c = c0 + (SPLIT ? team : 0); c <= c1; c += kFlight * kStride) {
            float mc[kFlight], lc[kFlight];
            float4 v[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                if (c + k * kStride > c1) break;
                const float* const q = at(c + k * kStride);
                mc[k] = q[RB * DP + r];
                lc[k] = q[RB * DP + RB + r];
                v[k] = d < p.D ? *reinterpret_cast<const float4*>(q + r * DP + d) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kFlight; ++k)
                if (c + k * kStride <= c1) {
                    const float a = shift_of(mc[k], mx);
                    l += a * lc[k];
                    o.x += a * v[k].x;
                    o.y += a * v[k].y;
                    o.z += a * v[k].z;
                    o.w += a * v[k].w;
                }
        }
        if (SPLIT) {
            s_o[tid] = o;
            if (tid % TEAM == 0) s_l[team] = l;
            __syncthreads();
            if (team > 0) return;
            for (int k = 1; k < TEAMS; ++k) {
                const float4 y = s_o[k * TEAM + tid];
                l += s_l[k];
                o.x += y.x;
                o.y += y.y;
                o.z += y.z;
                o.w += y.w;
            }
        }
        const float inv = 1.f / l;
        res = pack4<DT>(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
    if (d >= p.D || (SPLIT && team > 0)) return;
    uint8_t* const dst = p.out + units(b, p.os[0], node, p.os[1]) + units(h * p.G + head, p.os[2]);
    *reinterpret_cast<v4s*>(dst + 2 * d) = res;
}

// LDS of k_tree_attn: two stages of 64 rows of K and V, or of 32 for each wave,
// and the slow path's 32 KB where they are too small for it.
constexpr int attn_lds(int dp, int wr) {
    return wr == 1 ? 4 * 2 * 2 * 32 * dp * 2 : 2 * 2 * 64 * dp * 2 + (2 * 64 * dp * 2 < 32768 ? 32768 : 0);
}

template <int DT, int DP, int WR>
hipError_t launch_one(const TreeAttnParams& p, hipStream_t st, const LaunchEvents& ev) {
    constexpr int lds = attn_lds(DP, WR);
    if (lds > 65536) {
        const hipError_t e = allow_lds(reinterpret_cast<const void*>(k_tree_attn<DT, DP, WR>), lds);
        if (e != hipSuccess) return e;
    }
    const int64_t grid = p.MT == 1 ? p.clusters : static_cast<int64_t>((p.clusters + 7) / 8) * 8 * p.MT;
    hipExtLaunchKernelGGL((k_tree_attn<DT, DP, WR>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), lds, st,
                          ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

template <int DT, int DP, int RB>
hipError_t merge_one(const TreeAttnParams& p, hipStream_t st, const LaunchEvents& ev) {
    constexpr int TEAMS = kThreads / (DP / 4);
    const int tasks = p.B * p.Hkv, rows = p.N * p.G;
    // many parts per (sequence, key head): a context of 20001 rows over the whole device 4 us
    // shared and 23 alone; with 12 parts of 115 rows each 12 us shared and 7 alone
    if (p.clusters > 16 * tasks)
        hipExtLaunchKernelGGL((k_tree_merge<DT, DP, RB, true>), dim3(tasks, rows), dim3(kThreads), 0, st, ev.start,
                              ev.stop, 0, p);
    else
        hipExtLaunchKernelGGL((k_tree_merge<DT, DP, RB, false>), dim3(tasks, (rows + TEAMS - 1) / TEAMS), dim3(kThreads),
                              0, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t launch_rows_of(const TreeAttnParams& p, int rows, bool merge, hipStream_t st, const LaunchEvents& ev) {
    if (rows == 32) return merge ? merge_one<DT, DP, 32>(p, st, ev) : launch_one<DT, DP, 1>(p, st, ev);
    if (rows == 64) return merge ? merge_one<DT, DP, 64>(p, st, ev) : launch_one<DT, DP, 2>(p, st, ev);
    return merge ? merge_one<DT, DP, 128>(p, st, ev) : launch_one<DT, DP, 4>(p, st, ev);
}

hipError_t launch_any(const TreeAttnParams& p, const TreeAttnShape& s, int dtype, bool merge, hipStream_t st,
                      const LaunchEvents& ev) {
    if (dtype == DT_BF16)
        return s.dp == 128 ? launch_rows_of<DT_BF16, 128>(p, s.rows, merge, st, ev)
                           : launch_rows_of<DT_BF16, 64>(p, s.rows, merge, st, ev);
    return s.dp == 128 ? launch_rows_of<kDTypeF16, 128>(p, s.rows, merge, st, ev)
                       : launch_rows_of<kDTypeF16, 64>(p, s.rows, merge, st, ev);
}

}  // namespace

hipError_t launch_tree_attn(const TreeAttnParams& p, const TreeAttnShape& s, int dtype, hipStream_t st,
                            const LaunchEvents& ev) {
    return launch_any(p, s, dtype, false, st, ev);
}

hipError_t launch_tree_merge(const TreeAttnParams& p, const TreeAttnShape& s, int dtype, hipStream_t st,
                             const LaunchEvents& ev) {
    return launch_any(p, s, dtype, true, st, ev);
}

}  // namespace sv
