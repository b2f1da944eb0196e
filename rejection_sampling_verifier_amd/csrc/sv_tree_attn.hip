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
// The rounding of the weights (bf16: 2^-9 relative each, fp16: 2^-12) is the
// only one below float32 before the output's own.  The maximum is raised only
// when a row's new scores exceed it by more than 2^8, so weights reach 256 at
// most; the sum uses the unrounded weights.
//
// The tiles of all sequences and key heads form one line that is cut into
// equal parts (one per workgroup, or per group of workgroups when the rows
// need several tiles): ragged lengths cost no idle workgroups, and one long
// sequence fills the device.  A (sequence, key head) that a cut divides leaves
// partial (O, m, l) records that k_tree_merge joins in part order, so results
// do not depend on timing.
//
// Rows of the tile that no query sees (past the length, past the tree, on a
// page outside the pool) are staged as zeros.  Where some rows see a key and
// others do not, infinities and NaN among the values are kept out of the MFMA
// and added for the rows that see them only.

#include <hip/hip_ext.h>

#include "sv_tree.h"

namespace sv {
namespace {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

template <int DT>
__device__ __forceinline__ v16f mfma(v8s a, v8s b, v16f c) {
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0,
                                                       0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0,
                                                      0);
}

template <int DT>
__device__ __forceinline__ v4s pack4(float a, float b, float c, float d) {
    if constexpr (DT == DT_BF16) {
        v4b r = {static_cast<__bf16>(a), static_cast<__bf16>(b), static_cast<__bf16>(c), static_cast<__bf16>(d)};
        return __builtin_bit_cast(v4s, r);
    } else {
        v4h r = {static_cast<_Float16>(a), static_cast<_Float16>(b), static_cast<_Float16>(c),
                 static_cast<_Float16>(d)};
        return __builtin_bit_cast(v4s, r);
    }
}

// Whether one of the two 16-bit floats of w is infinite or NaN.
template <int DT>
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
    constexpr uint32_t e = DT == DT_BF16 ? 0x7F80u : 0x7C00u;
    return (w & e) == e || ((w >> 16) & e) == e;
}

template <int DT>
__device__ __forceinline__ float to_float(uint16_t u) {
    if constexpr (DT == DT_BF16)
        return __uint_as_float(static_cast<uint32_t>(u) << 16);
    else
        return static_cast<float>(__builtin_bit_cast(_Float16, u));
}

template <int DT>
__device__ __forceinline__ float nonfinite_term(float wgt, uint32_t e) {
    return nonfinite2<DT>(e) ? wgt * to_float<DT>(static_cast<uint16_t>(e)) : 0.f;
}

// The value in both half-waves: (of lane & 31, of (lane & 31) + 32).
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Bits [n, 32), n clamped to [0, 32].
__device__ __forceinline__ uint32_t bits_from(int n) { return n <= 0 ? ~0u : n >= 32 ? 0u : ~0u << n; }

// 2^(a - b) for a <= b, 1 where they are equal (both may be -inf).
__device__ __forceinline__ float shift_of(float a, float b) {
    return a == b ? 1.f : __builtin_amdgcn_exp2f(a - b);
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

// Parts the line of `total` tiles is cut into, and the part that tile f is in.
__device__ __forceinline__ int parts_of(const TreeAttnParams& p, int64_t total) {
    const int64_t most = (total + p.min_tiles - 1) / p.min_tiles;
    return most < p.clusters ? static_cast<int>(most) : p.clusters;
}
__device__ __forceinline__ int64_t part_start(int64_t total, int parts, int c) { return total * c / parts; }
__device__ __forceinline__ int part_of(int64_t total, int parts, int64_t f) {
    return static_cast<int>(((f + 1) * parts - 1) / total);
}

// Ancestor-or-self sets of the nodes: lane i of a wave holds node i's.
// `near` > 0 keeps the nearest `near` of them only.  A parent outside [0, i)
// ends the line.
__device__ __forceinline__ uint64_t ancestors(const int32_t* parent, int n, int lane, int near) {
    int up = -1;
    if (lane > 0 && lane < n) up = parent[lane];
    if (up >= lane || up < 0) up = -1;
    uint64_t set = 1ull << lane;
    if (near > 0 && near < kMaxNodes) {
        int at = up;
        for (int s = 1; s < near; ++s) {
            if (at >= 0) set |= 1ull << at;
            const int next = __shfl(up, at < 0 ? 0 : at);
            at = at < 0 ? -1 : next;
        }
        return set;
    }
#pragma unroll
    for (int s = 0; s < 6; ++s) {  // paths double in length: 64 nodes need 6 steps
        const int at = up < 0 ? lane : up;
        const uint64_t theirs = __shfl(static_cast<unsigned long long>(set), at);
        const int next = __shfl(up, at);
        if (up >= 0) {
            set |= theirs;
            up = next;
        }
    }
    return set;
}

template <int DT, int DP, int WR, int TK>
__global__ __launch_bounds__(kThreads, 2) void k_tree_attn(TreeAttnParams p) {
    constexpr int WK = kWaves / WR;           // waves over keys
    constexpr int RB = 32 * WR;               // query rows
    constexpr int KS = TK / (32 * WK);        // 32-key subtiles per wave
    constexpr int NC = DP / 8;                // 16-byte chunks per row
    constexpr int RPT = TK * NC / kThreads;   // rows of K (and of V) a thread stages
    constexpr int NQ = DP / 16, ND = DP / 32;
    constexpr int kRowB = DP * 2;
    static_assert(TK * kRowB >= kWaves * 4096, "the slow path keeps a wave's weights in the K tile");
    static_assert(2 * TK * kRowB >= (WK > 1 ? 2 * 64 * (DP / 2) * 4 : 0), "the waves' results are joined in the tiles");

    __shared__ __align__(16) uint8_t smem[2 * TK * kRowB];
    __shared__ uint32_t s_bad[2][TK / 32];  // rows of the tile that nothing sees
    __shared__ uint32_t s_nf[2];            // some row of a mixed tile holds an infinity or NaN
    __shared__ float s_ml[2][2][64];
    __shared__ int64_t s_sum[kWaves];
    __shared__ int32_t s_scan[kWaves];
    __shared__ int s_b;
    __shared__ int64_t s_before;

    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int wr = w % WR, wk = w / WR, hh = lane >> 5;
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
        const int parts = parts_of(p, total);
        if (c >= parts) return;
        f0 = part_start(total, parts, c);
        f1 = part_start(total, parts, c + 1);
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
        b = s_b;
        before = s_before;
    }
    if (tid < 2) s_nf[tid] = 0;
    if (tid < 2 * (TK / 32)) s_bad[tid / (TK / 32)][tid % (TK / 32)] = 0;
    __syncthreads();

    uint8_t* const sk = smem;
    uint8_t* const sv = smem + TK * kRowB;
    // this thread's 16-byte chunk of the rows it stages
    const int ch = tid % NC, row0 = tid / NC;
    constexpr int kRowStep = kThreads / NC;
    const bool ch_in = ch * 8 < p.D;
    const int cin = ch_in ? ch : 0;
    // the rows a thread stages are multiples of 16 (of 32 for 8 chunks) apart: one swizzle for all
    const uint32_t k_at = row0 * kRowB + ((ch ^ (DP == 128 ? (row0 & 15) : ((row0 >> 1) & 7))) << 4);
    const uint32_t v_at = row0 * kRowB + ((ch ^ (DP == 128 ? ((row0 & 3) << 2) : (((row0 >> 1) & 1) << 2))) << 4);
    // lane parts of the LDS addresses; both tiles are XOR-swizzled by 16-byte
    // chunk so that eight lanes of a read touch eight different bank groups
    const int kx = DP == 128 ? (lane & 15) : ((lane >> 1) & 7);
    const int vrow = (lane & 15) >> 2;
    const int vx = DP == 128 ? vrow : (vrow >> 1);
    const int vlow = (((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)) * 16 + (lane & 1) * 8;
    const int my_row = m * RB + wr * 32 + (lane & 31);
    const int my_node = my_row / p.G;
    const int my_head = my_row - my_node * p.G;
    const bool win = p.window > 0;

    int par = 0;
    int64_t f = f0;
    while (f < f1) {
        const Tiles tl = tiles_of<TK>(p, p.len[b]);
        const int T = tl.total();
        const int64_t in_seq = f - before * p.Hkv;
        const int h = static_cast<int>(in_seq / T);
        const int t0 = static_cast<int>(in_seq - static_cast<int64_t>(h) * T);
        const int t1 = static_cast<int>(min(static_cast<int64_t>(T), t0 + (f1 - f)));
        const bool whole = t0 == 0 && t1 == T;
        int n = p.N;
        if (p.n_nodes) {
            n = p.n_nodes[b];
            n = n < 0 ? 0 : n > p.N ? p.N : n;
        }
        const int rows = n * p.G;
        const bool active = m * RB + wr * 32 < rows;  // wave-uniform
        float mx = -INFINITY, l = 0.f;
        v16f o[ND];
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;

        if (m * RB < rows) {
            // queries: the B operand, resident
            v8s q[NQ];
            {
                const bool in = my_row < rows;
                const int64_t off = b * p.qs[0] + my_node * p.qs[1] + static_cast<int64_t>(h * p.G + my_head) * p.qs[2];
                const uint8_t* const src = p.q + 2 * (in ? off : 0);
#pragma unroll
                for (int s = 0; s < NQ; ++s) {
                    const int d = s * 16 + hh * 8;
                    v8s z = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (in && d < p.D) z = *reinterpret_cast<const v8s*>(src + 2 * d);
                    q[s] = z;
                }
            }
            uint64_t set = 0;
            int low = 0;  // first cache row in this row's window
            if (t1 == T || win) {
                const int32_t* const par_b = p.parent + static_cast<int64_t>(b) * p.N;
                const uint64_t all = ancestors(par_b, n, lane, 0);
                const int src = my_node < kMaxNodes ? my_node : 0;
                set = __shfl(static_cast<unsigned long long>(all), src);
                if (win) {
                    low = tl.len + __popcll(set) - p.window;  // depth + 1 nodes on the line
                    if (p.window < kMaxNodes)
                        set = __shfl(static_cast<unsigned long long>(ancestors(par_b, n, lane, p.window)), src);
                }
            }

            int pid[RPT];
            uint4 rk[RPT], rv[RPT];
            uint32_t okm = 0;
            const int32_t* const tab = p.table + b * p.table_stride;
            // this (sequence, key head)'s first cache and tree rows, at this thread's chunk
            const uint8_t* const kcb = p.kc + 2 * (h * p.kcs[2] + cin * 8);
            const uint8_t* const vcb = p.vc + 2 * (h * p.vcs[2] + cin * 8);
            const uint8_t* const ktb = p.kt + 2 * (b * p.kts[0] + h * p.kts[2] + cin * 8);
            const uint8_t* const vtb = p.vt + 2 * (b * p.vts[0] + h * p.vts[2] + cin * 8);
            auto pages = [&](int t) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    pid[i] = -1;
                    if (t < tl.cache) {
                        const int key = tl.key_tile(t) * TK + row0 + i * kRowStep;
                        if (key < tl.len) pid[i] = tab[key >> p.ps_shift];
                    }
                }
            };
            auto load = [&](int t) {
                // rows that nothing sees read a row that exists instead, and become zeros when staged
                okm = 0;
                if (t >= tl.cache) {
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const int r = row0 + i * kRowStep;
                        const bool ok = r < n;
                        okm |= ok ? 1u << i : 0u;
                        const int64_t at = ok ? r : 0;
                        rk[i] = *reinterpret_cast<const uint4*>(ktb + 2 * (at * p.kts[1]));
                        rv[i] = *reinterpret_cast<const uint4*>(vtb + 2 * (at * p.vts[1]));
                    }
                } else {
                    const int first = tl.key_tile(t) * TK + row0;
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const int slot = (first + i * kRowStep) & ((1 << p.ps_shift) - 1);
                        const bool ok = static_cast<uint32_t>(pid[i]) < static_cast<uint32_t>(p.pages);
                        okm |= ok ? 1u << i : 0u;
                        const int64_t at = ok ? pid[i] : 0;
                        rk[i] = *reinterpret_cast<const uint4*>(kcb + 2 * (at * p.kcs[0] + slot * p.kcs[1]));
                        rv[i] = *reinterpret_cast<const uint4*>(vcb + 2 * (at * p.vcs[0] + slot * p.vcs[1]));
                    }
                }
            };

            pages(t0);
            load(t0);
            if (t0 + 1 < t1) pages(t0 + 1);
            for (int t = t0; t < t1; ++t, par ^= 1) {
                const bool tree = t >= tl.cache;
                const int kb = tree ? 0 : tl.key_tile(t) * TK;
                const bool mixed = tree || (win && kb < tl.len + p.N - p.window);
                const uint32_t keep = ch_in ? okm : 0u;
                if (keep != (1u << RPT) - 1u) {
#pragma unroll
                    for (int i = 0; i < RPT; ++i)
                        if (!(keep >> i & 1)) {
                            rk[i] = make_uint4(0, 0, 0, 0);
                            rv[i] = make_uint4(0, 0, 0, 0);
                        }
                }
                __syncthreads();  // the previous tile has been read
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    if (mixed && (nonfinite2<DT>(rv[i].x) || nonfinite2<DT>(rv[i].y) || nonfinite2<DT>(rv[i].z) ||
                                  nonfinite2<DT>(rv[i].w))) {
                        s_nf[par] = 1;
                        uint16_t e[8];
                        __builtin_memcpy(e, &rv[i], 16);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (nonfinite2<DT>(e[j])) e[j] = 0;
                        __builtin_memcpy(&rv[i], e, 16);
                    }
                    *reinterpret_cast<uint4*>(sk + k_at + i * kRowStep * kRowB) = rk[i];
                    *reinterpret_cast<uint4*>(sv + v_at + i * kRowStep * kRowB) = rv[i];
                }
                if (ch == 0 && okm != (1u << RPT) - 1u) {
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const int r = row0 + i * kRowStep;
                        if (!(okm >> i & 1)) atomicOr(&s_bad[par][r >> 5], 1u << (r & 31));
                    }
                }
                __syncthreads();
                // the other parity's marks have been read; its next writers wait at the next barrier
                if (tid < TK / 32) s_bad[par ^ 1][tid] = 0;
                if (tid == kThreads - 1) s_nf[par ^ 1] = 0;
                if (t + 1 < t1) {
                    load(t + 1);
                    if (t + 2 < t1) pages(t + 2);
                }

                const bool nf = mixed && s_nf[par] != 0;
                v16f x[KS];
                if (active) {
                    uint32_t bad[KS];
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int sub = wk * KS + ks;
                        bad[ks] = __builtin_amdgcn_readfirstlane(s_bad[par][sub]);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[ks][i] = 0.f;
                        const uint8_t* const rowp = sk + (sub * 32 + (lane & 31)) * kRowB;
#pragma unroll
                        for (int s = 0; s < NQ; ++s) {
                            const v8s a = *reinterpret_cast<const v8s*>(rowp + (((2 * s + hh) ^ kx) << 4));
                            x[ks] = mfma<DT>(a, q[s], x[ks]);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);  // the phases stay apart: their operands would not fit together
                    float top = -INFINITY;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int sub = wk * KS + ks;
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[ks][i] *= p.scale2;
                        if (mixed || bad[ks]) {
                            // bit r: this lane's row sees row r of the subtile
                            uint32_t see = ~bad[ks];
                            if (tree)
                                see &= sub < 2 ? static_cast<uint32_t>(set >> (32 * (sub & 1))) : 0u;
                            else if (win)
                                see &= bits_from(low - (kb + sub * 32)) | ~bits_from(p.sinks - (kb + sub * 32));
                            see >>= 4 * hh;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[ks][i] = see & (1u << (8 * (i >> 2) + (i & 3))) ? x[ks][i] : -INFINITY;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) top = fmaxf(top, x[ks][i]);
                    }
                    top = half_max(top);
                    if (__any(top > mx + 8.f)) {
                        const float mn = fmaxf(mx, top);
                        const float a = shift_of(mx, mn);
                        l *= a;
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[dt][i] *= a;
                        mx = mn;
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            x[ks][i] = __builtin_amdgcn_exp2f(x[ks][i] - ref);
                            l += x[ks][i];
                        }
#pragma unroll
                        for (int t2 = 0; t2 < 2; ++t2) {
                            const v4s lo = pack4<DT>(x[ks][8 * t2], x[ks][8 * t2 + 1], x[ks][8 * t2 + 2],
                                                     x[ks][8 * t2 + 3]);
                            const v4s hi = pack4<DT>(x[ks][8 * t2 + 4], x[ks][8 * t2 + 5], x[ks][8 * t2 + 6],
                                                     x[ks][8 * t2 + 7]);
                            const v8s pf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                            const uint8_t* const rowp =
                                sv + ((wk * KS + ks) * 32 + 16 * t2 + 4 * hh + vrow) * kRowB + vlow;
#pragma unroll
                            for (int dt = 0; dt < ND; ++dt) {
                                const int cx = DP == 128 ? ((dt ^ vx) << 6) : ((dt ^ vx) << 6);
                                const v4s a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(rowp + cx));
                                const v4s a1 =
                                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(rowp + 8 * kRowB + cx));
                                o[dt] = mfma<DT>(__builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7), pf, o[dt]);
                            }
                        }
                    }
                }
                if (nf) {  // rare: infinities or NaN among the values, for the rows that see them
                    __syncthreads();
                    float* const wp = reinterpret_cast<float*>(sk) + w * 1024;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int sub = wk * KS + ks;
                        if (active) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                wp[(8 * (i >> 2) + 4 * hh + (i & 3)) * 32 + (lane & 31)] = x[ks][i];
                        }
                        __syncthreads();
                        if (active) {
                            for (int r = 0; r < 32; ++r) {
                                const int key = kb + sub * 32 + r;
                                const uint8_t* src;
                                if (tree) {
                                    if (key >= n) break;
                                    src = p.vt + 2 * (b * p.vts[0] + key * p.vts[1] + h * p.vts[2]);
                                } else {
                                    if (key >= tl.len) break;
                                    const int pg = tab[key >> p.ps_shift];
                                    if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(p.pages)) continue;
                                    src = p.vc + 2 * (pg * p.vcs[0] + (key & ((1 << p.ps_shift) - 1)) * p.vcs[1] +
                                                      h * p.vcs[2]);
                                }
                                const float wgt = wp[r * 32 + (lane & 31)];
#pragma unroll
                                for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                                    for (int g = 0; g < 4; ++g) {
                                        const int d = 32 * dt + 8 * g + 4 * hh;
                                        if (32 * dt + 8 * g < p.D) {
                                            const uint2 e = *reinterpret_cast<const uint2*>(src + 2 * d);
                                            if (wgt != 0.f && (nonfinite2<DT>(e.x) || nonfinite2<DT>(e.y))) {
                                                o[dt][4 * g] += nonfinite_term<DT>(wgt, e.x & 0xFFFFu);
                                                o[dt][4 * g + 1] += nonfinite_term<DT>(wgt, e.x >> 16);
                                                o[dt][4 * g + 2] += nonfinite_term<DT>(wgt, e.y & 0xFFFFu);
                                                o[dt][4 * g + 3] += nonfinite_term<DT>(wgt, e.y >> 16);
                                            }
                                        }
                                        asm volatile("" ::: "memory");  // one load at a time: registers stay with the main path
                                    }
                            }
                        }
                        __syncthreads();
                    }
                }
            }
            l = half_sum(l);

            // waves that took other keys of the same rows hand their results over
            if constexpr (WK > 1) {
                float* const buf = reinterpret_cast<float*>(smem);
#pragma unroll
                for (int half = WK / 2; half >= 1; half >>= 1) {
                    const int slot = WR == 2 ? wr : wk % half;
                    __syncthreads();
                    if (wk >= half && wk < 2 * half) {
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                buf[slot * 64 * (DP / 2) + (dt * 16 + i) * 64 + lane] = o[dt][i];
                        s_ml[slot][0][lane] = mx;
                        s_ml[slot][1][lane] = l;
                    }
                    __syncthreads();
                    if (wk < half) {
                        const float m2 = s_ml[slot][0][lane], l2 = s_ml[slot][1][lane];
                        const float mn = fmaxf(mx, m2);
                        const float a1 = shift_of(mx, mn), a2 = shift_of(m2, mn);
                        l = l * a1 + l2 * a2;
                        mx = mn;
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[dt][i] = o[dt][i] * a1 + buf[slot * 64 * (DP / 2) + (dt * 16 + i) * 64 + lane] * a2;
                    }
                }
            }
        }

        if (wk == 0 && my_row < p.N * p.G) {
            if (whole) {
                const bool in = my_row < rows;
                const float inv = in ? 1.f / l : 0.f;
                uint8_t* const dst = p.out + 2 * (b * p.os[0] + my_node * p.os[1] +
                                                  static_cast<int64_t>(h * p.G + my_head) * p.os[2]);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int d = 32 * dt + 8 * g + 4 * hh;
                        if (32 * dt + 8 * g < p.D) {
                            const v4s r = pack4<DT>(o[dt][4 * g] * inv, o[dt][4 * g + 1] * inv, o[dt][4 * g + 2] * inv,
                                              o[dt][4 * g + 3] * inv);  // zeros for an absent node
                            *reinterpret_cast<v4s*>(dst + 2 * d) = r;
                        }
                    }
            } else if (my_row < rows) {
                float* const rec = p.part + ((static_cast<int64_t>(c) * 2 + (f == f0 ? 0 : 1)) * p.MT + m) *
                                                (RB * (DP + 2));
                const int r = wr * 32 + (lane & 31);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *reinterpret_cast<float4*>(rec + r * DP + 32 * dt + 8 * g + 4 * hh) =
                            make_float4(o[dt][4 * g], o[dt][4 * g + 1], o[dt][4 * g + 2], o[dt][4 * g + 3]);
                if (hh == 0) {
                    rec[RB * DP + r] = mx;
                    rec[RB * DP + RB + r] = l;
                }
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
// DP / 4 threads per row, four dimensions each.
template <int DT, int DP, int WR>
__global__ __launch_bounds__(kThreads) void k_tree_merge(TreeAttnParams p) {
    constexpr int TPR = DP / 4, RPB = kThreads / TPR, RB = 32 * WR;
    const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
    const int64_t s0 = p.start[b], T = p.start[b + 1] - s0;
    const int64_t total = p.start[p.B] * p.Hkv;
    const int parts = parts_of(p, total);
    const int64_t first = s0 * p.Hkv + h * T;
    const int c0 = part_of(total, parts, first), c1 = part_of(total, parts, first + T - 1);
    if (c0 == c1) return;
    const int row = blockIdx.y * RPB + threadIdx.x / TPR;
    const int d = (threadIdx.x % TPR) * 4;
    if (row >= p.N * p.G || d >= p.D) return;
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
        const int slot0 = part_start(total, parts, c0) == first ? 0 : 1;
        auto at = [&](int c) { return p.part + ((static_cast<int64_t>(c) * 2 + (c == c0 ? slot0 : 0)) * p.MT + m) * rec; };
        float mx = -INFINITY;
        for (int c = c0; c <= c1; ++c) mx = fmaxf(mx, at(c)[RB * DP + r]);
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0; c <= c1; ++c) {
            const float* const q = at(c);
            const float a = shift_of(q[RB * DP + r], mx);
            const float4 v = *reinterpret_cast<const float4*>(q + r * DP + d);
            l += a * q[RB * DP + RB + r];
            o.x += a * v.x;
            o.y += a * v.y;
            o.z += a * v.z;
            o.w += a * v.w;
        }
        const float inv = 1.f / l;
        res = pack4<DT>(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
    uint8_t* const dst =
        p.out + 2 * (b * p.os[0] + node * p.os[1] + static_cast<int64_t>(h * p.G + head) * p.os[2]);
    *reinterpret_cast<v4s*>(dst + 2 * d) = res;
}

template <int DT, int DP, int WR, int TK>
hipError_t launch_one(const TreeAttnParams& p, hipStream_t st, const LaunchEvents& ev) {
    const int64_t grid =
        p.MT == 1 ? p.clusters : static_cast<int64_t>((p.clusters + 7) / 8) * 8 * p.MT;
    hipExtLaunchKernelGGL((k_tree_attn<DT, DP, WR, TK>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, st,
                          ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

template <int DT, int DP, int WR>
hipError_t merge_one(const TreeAttnParams& p, hipStream_t st, const LaunchEvents& ev) {
    constexpr int RPB = kThreads / (DP / 4);
    hipExtLaunchKernelGGL((k_tree_merge<DT, DP, WR>), dim3(p.B * p.Hkv, (p.N * p.G + RPB - 1) / RPB), dim3(kThreads), 0,
                          st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tree_attn(const TreeAttnParams& p, const TreeAttnShape& s, int dtype, hipStream_t st,
                            const LaunchEvents& ev) {
    const bool bf = dtype == DT_BF16;
    if (s.dp == 128) {
        if (s.wr == 1) return bf ? launch_one<DT_BF16, 128, 1, 128>(p, st, ev) : launch_one<kDTypeF16, 128, 1, 128>(p, st, ev);
        if (s.wr == 2) return bf ? launch_one<DT_BF16, 128, 2, 64>(p, st, ev) : launch_one<kDTypeF16, 128, 2, 64>(p, st, ev);
        return bf ? launch_one<DT_BF16, 128, 4, 64>(p, st, ev) : launch_one<kDTypeF16, 128, 4, 64>(p, st, ev);
    }
    if (s.wr == 1) return bf ? launch_one<DT_BF16, 64, 1, 128>(p, st, ev) : launch_one<kDTypeF16, 64, 1, 128>(p, st, ev);
    if (s.wr == 2) return bf ? launch_one<DT_BF16, 64, 2, 128>(p, st, ev) : launch_one<kDTypeF16, 64, 2, 128>(p, st, ev);
    return bf ? launch_one<DT_BF16, 64, 4, 128>(p, st, ev) : launch_one<kDTypeF16, 64, 4, 128>(p, st, ev);
}

hipError_t launch_tree_merge(const TreeAttnParams& p, const TreeAttnShape& s, int dtype, hipStream_t st,
                             const LaunchEvents& ev) {
    const bool bf = dtype == DT_BF16;
    if (s.dp == 128) {
        if (s.wr == 1) return bf ? merge_one<DT_BF16, 128, 1>(p, st, ev) : merge_one<kDTypeF16, 128, 1>(p, st, ev);
        if (s.wr == 2) return bf ? merge_one<DT_BF16, 128, 2>(p, st, ev) : merge_one<kDTypeF16, 128, 2>(p, st, ev);
        return bf ? merge_one<DT_BF16, 128, 4>(p, st, ev) : merge_one<kDTypeF16, 128, 4>(p, st, ev);
    }
    if (s.wr == 1) return bf ? merge_one<DT_BF16, 64, 1>(p, st, ev) : merge_one<kDTypeF16, 64, 1>(p, st, ev);
    if (s.wr == 2) return bf ? merge_one<DT_BF16, 64, 2>(p, st, ev) : merge_one<kDTypeF16, 64, 2>(p, st, ev);
    return bf ? merge_one<DT_BF16, 64, 4>(p, st, ev) : merge_one<kDTypeF16, 64, 4>(p, st, ev);
}

}  // namespace sv
