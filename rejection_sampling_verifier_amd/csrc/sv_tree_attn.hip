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

// The 16-byte chunks of row r of a V tile are XORed with this.
template <int DP>
__device__ __forceinline__ uint32_t swizzle(int r) {
    return DP == 128 ? ((r & 3) << 2) ^ ((r >> 2) & 3) : (((r >> 1) & 1) << 2) ^ ((r >> 2) & 3);
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

template <int DT, int DP, int NT, int WR>
__global__ __launch_bounds__(kThreads, NT == 1 ? 2 : 1) void k_tree_attn(TreeAttnParams p) {
    constexpr int WK = kWaves / WR;      // waves over keys
    constexpr int WROWS = 32 * NT;       // query rows of a wave
    constexpr int RB = WROWS * WR;       // query rows of the workgroup
    constexpr int TK = 32 * WK;          // keys per tile, 32 per wave
    constexpr int NQ = DP / 16, ND = DP / 32;
    constexpr int kRowB = DP * 2;
    constexpr int kTileB = 32 * kRowB;   // a wave's V tile

    __shared__ __align__(16) uint8_t smem[kWaves * kTileB];
    __shared__ float s_ml[2][2][64];
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
        b = __builtin_amdgcn_readfirstlane(s_b);
        before = s_before;
    }

    uint8_t* const sv = smem + w * kTileB;
    // a lane stages the chunks 2 s + hh of row `col`; the tile is XOR-swizzled by
    // 16-byte chunk: eight lanes of a write, and the sixteen of a transposing
    // read (four rows, two chunks), touch different banks
    const uint32_t v_at = col * kRowB;
    const uint32_t v_x = swizzle<DP>(col);
    const int vrow = (lane & 15) >> 2;                                // row of four in a transposing read
    const int vchunk = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);     // its chunk of the four of 32 dimensions
    const uint32_t vr_at = (4 * hh + vrow) * kRowB + (lane & 1) * 8;
    const bool win = p.window > 0;
    const float scale2 = p.scale2;
    const bool odd_end = p.D % 16 != 0;   // the last 32 bytes of a row are half a row's

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
        const int row0 = m * RB + wr * WROWS;  // the wave's first row
        float mx[NT], l[NT];
        v16f o[NT][ND];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt] = -INFINITY;
            l[nt] = 0.f;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[nt][dt][i] = 0.f;
        }

        if (row0 < rows) {  // the wave has rows; no barrier inside
            // queries: the B operand, resident; a negative scale is moved into their sign
            v8s q[NT][NQ];
            uint64_t set[NT];
            int low[NT];  // first cache row in the row's window
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = row0 + nt * 32 + col;
                const bool in = row < rows;
                const int node = in ? row / p.G : 0;
                const int64_t off = b * p.qs[0] + node * p.qs[1] +
                                    static_cast<int64_t>(h * p.G + (in ? row - node * p.G : 0)) * p.qs[2];
#pragma unroll
                for (int s = 0; s < NQ; ++s) {
                    const int d = s * 16 + hh * 8;
                    v8s z = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (in && d < p.D) z = *reinterpret_cast<const v8s*>(p.q + 2 * (off + d));
                    q[nt][s] = p.flip ? z ^ static_cast<short>(0x8000) : z;
                }
                set[nt] = 0;
                low[nt] = 0;
                if (t1 == T || win) {
                    const int32_t* const par_b = p.parent + static_cast<int64_t>(b) * p.N;
                    const uint64_t all = ancestors(par_b, n, lane, 0);
                    set[nt] = __shfl(static_cast<unsigned long long>(all), node);
                    if (win) {
                        low[nt] = tl.len + __popcll(set[nt]) - p.window;  // depth + 1 nodes on the line
                        if (p.window < kMaxNodes)
                            set[nt] = __shfl(static_cast<unsigned long long>(ancestors(par_b, n, lane, p.window)), node);
                    }
                }
            }

            const int32_t* const tab = p.table + b * p.table_stride;
            // this (sequence, key head)'s rows, at this lane's first chunk
            const uint8_t* const kcb = p.kc + 2 * (h * p.kcs[2] + hh * 8);
            const uint8_t* const vcb = p.vc + 2 * (h * p.vcs[2] + hh * 8);
            const uint8_t* const ktb = p.kt + 2 * (b * p.kts[0] + h * p.kts[2] + hh * 8);
            const uint8_t* const vtb = p.vt + 2 * (b * p.vts[0] + h * p.vts[2] + hh * 8);
            auto page = [&](int t) {  // the page of this lane's row of tile t
                if (t >= tl.cache) return -1;
                const int key = tl.key_tile(t) * TK + wk * 32 + col;
                return key < tl.len ? tab[key >> p.ps_shift] : -1;
            };
            // where this lane's row of tile t is; rows that nothing sees stand in for one that exists
            auto place = [&](int t, int pid, const uint8_t*& ka, const uint8_t*& va) {
                if (t >= tl.cache) {
                    const int r = wk * 32 + col;
                    const bool ok = r < n;
                    const int64_t at = ok ? r : 0;
                    ka = ktb + 2 * (at * p.kts[1]);
                    va = vtb + 2 * (at * p.vts[1]);
                    return ok;
                }
                const int slot = (tl.key_tile(t) * TK + wk * 32 + col) & ((1 << p.ps_shift) - 1);
                const bool ok = static_cast<uint32_t>(pid) < static_cast<uint32_t>(p.pages);
                const int64_t at = ok ? pid : 0;
                ka = kcb + 2 * (at * p.kcs[0] + slot * p.kcs[1]);
                va = vcb + 2 * (at * p.vcs[0] + slot * p.vcs[1]);
                return ok;
            };
            auto fetch = [&](const uint8_t* a, v8s* r) {
                if (p.D == DP) {
#pragma unroll
                    for (int s = 0; s < NQ; ++s) r[s] = *reinterpret_cast<const v8s*>(a + 32 * s);
                } else {
                    const bool half = odd_end && hh;  // chunks past the row's end: read its start, then drop it
#pragma unroll
                    for (int s = 0; s < NQ; ++s) {
                        v8s z = {0, 0, 0, 0, 0, 0, 0, 0};
                        if (16 * s + 16 <= p.D) {
                            z = *reinterpret_cast<const v8s*>(a + 32 * s);
                        } else if (16 * s < p.D) {
                            const v8s y = *reinterpret_cast<const v8s*>(half ? a - 16 : a + 32 * s);
                            z = half ? z : y;
                        }
                        r[s] = z;
                    }
                }
            };

            v8s kr[NQ], vr[NQ];
            const uint8_t *ka, *va;
            bool ok = place(t0, page(t0), ka, va);
            fetch(ka, kr);
            fetch(va, vr);
            int pid = t0 + 1 < t1 ? page(t0 + 1) : -1;
            for (int t = t0; t < t1; ++t) {
                const bool tree = t >= tl.cache;
                const int kb = (tree ? 0 : tl.key_tile(t) * TK) + wk * 32;
                const bool mixed = tree || (win && kb < tl.len + p.N - p.window);
                const uint32_t bad = ~static_cast<uint32_t>(__ballot(ok));  // rows nothing sees
                const bool more = t + 1 < t1;
                bool nf = false;

                v16f x[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[nt][i] = 0.f;
#pragma unroll
                for (int s = 0; s < NQ; ++s)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) x[nt] = mfma<DT>(kr[s], q[nt][s], x[nt]);
                __builtin_amdgcn_sched_barrier(0);
                bool ok_next = false;
                const uint8_t* va_next = va;
                if (more) {
                    ok_next = place(t + 1, pid, ka, va_next);
                    fetch(ka, kr);
                }
                // V rows into the wave's tile, hidden ones as zeros
                if (bad != 0) {
#pragma unroll
                    for (int s = 0; s < NQ; ++s) vr[s] = ok ? vr[s] : static_cast<short>(0);
                }
                if (mixed) {
#pragma unroll
                    for (int s = 0; s < NQ; ++s) {
                        const uint4 u = __builtin_bit_cast(uint4, vr[s]);
                        if (nonfinite2<DT>(u.x) || nonfinite2<DT>(u.y) || nonfinite2<DT>(u.z) || nonfinite2<DT>(u.w)) {
                            nf = true;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (nonfinite2<DT>(static_cast<uint16_t>(vr[s][j]))) vr[s][j] = 0;
                        }
                    }
                    nf = __any(nf);
                }
#pragma unroll
                for (int s = 0; s < NQ; ++s)
                    *reinterpret_cast<v8s*>(sv + v_at + (((2 * s + hh) ^ v_x) << 4)) = vr[s];
                if (more) {
                    fetch(va_next, vr);
                    if (t + 2 < t1) pid = page(t + 2);
                }
                __builtin_amdgcn_sched_barrier(0);

                if (mixed || bad != 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint32_t see = ~bad;  // bit r: this lane's row sees row r of the subtile
                        if (tree)
                            see &= wk < 2 ? static_cast<uint32_t>(set[nt] >> (32 * (wk & 1))) : 0u;
                        else if (win)
                            see &= bits_from(low[nt] - kb) | ~bits_from(p.sinks - kb);
                        see >>= 4 * hh;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[nt][i] = see & (1u << (8 * (i >> 2) + (i & 3))) ? x[nt][i] : -INFINITY;
                    }
                }
                bool grows = false;
                float top[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    top[nt] = x[nt][0];
#pragma unroll
                    for (int i = 1; i < 16; ++i) top[nt] = fmaxf(top[nt], x[nt][i]);
                    top[nt] = half_max(top[nt]) * scale2;
                    grows = grows || top[nt] > mx[nt] + 8.f;
                }
                if (__any(grows)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float mn = fmaxf(mx[nt], top[nt]);
                        const float a = shift_of(mx[nt], mn);
                        l[nt] *= a;
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[nt][dt][i] *= a;
                        mx[nt] = mn;
                    }
                }
                v8s pf[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float ref = mx[nt] == -INFINITY ? 0.f : mx[nt];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[nt][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[nt][i], scale2, -ref));
                        l[nt] += x[nt][i];
                    }
#pragma unroll
                    for (int t2 = 0; t2 < 2; ++t2) {
                        const v4s lo = pack4<DT>(x[nt][8 * t2], x[nt][8 * t2 + 1], x[nt][8 * t2 + 2], x[nt][8 * t2 + 3]);
                        const v4s hi =
                            pack4<DT>(x[nt][8 * t2 + 4], x[nt][8 * t2 + 5], x[nt][8 * t2 + 6], x[nt][8 * t2 + 7]);
                        pf[nt][t2] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                }
#pragma unroll
                for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) {
                        const uint32_t row = vr_at + 16 * t2 * kRowB;
                        const v4s a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (lds_v4s*)(sv + row + (((4 * dt + vchunk) ^ swizzle<DP>(4 * hh + vrow)) << 4)));
                        const v4s a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (lds_v4s*)(sv + row + 8 * kRowB + (((4 * dt + vchunk) ^ swizzle<DP>(8 + 4 * hh + vrow)) << 4)));
                        const v8s a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) o[nt][dt] = mfma<DT>(a, pf[nt][t2], o[nt][dt]);
                    }
                if (nf) {  // rare: infinities or NaN among the values, for the rows that see them
                    float* const wp = reinterpret_cast<float*>(sv);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                        for (int i = 0; i < 16; ++i) wp[(8 * (i >> 2) + 4 * hh + (i & 3)) * 32 + col] = x[nt][i];
                        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                        for (int r = 0; r < 32; ++r) {
                            const int key = kb + r;
                            const uint8_t* src;
                            if (bad >> r & 1) continue;
                            if (tree) {
                                src = p.vt + 2 * (b * p.vts[0] + key * p.vts[1] + h * p.vts[2]);
                            } else {
                                const int pg = tab[key >> p.ps_shift];
                                src = p.vc + 2 * (pg * p.vcs[0] + (key & ((1 << p.ps_shift) - 1)) * p.vcs[1] +
                                                  h * p.vcs[2]);
                            }
                            const float wgt = wp[r * 32 + col];
#pragma unroll
                            for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                                for (int g = 0; g < 4; ++g) {
                                    if (32 * dt + 8 * g < p.D) {
                                        const uint2 e = *reinterpret_cast<const uint2*>(src + 2 * (32 * dt + 8 * g + 4 * hh));
                                        if (wgt != 0.f && (nonfinite2<DT>(e.x) || nonfinite2<DT>(e.y))) {
                                            o[nt][dt][4 * g] += nonfinite_term<DT>(wgt, e.x & 0xFFFFu);
                                            o[nt][dt][4 * g + 1] += nonfinite_term<DT>(wgt, e.x >> 16);
                                            o[nt][dt][4 * g + 2] += nonfinite_term<DT>(wgt, e.y & 0xFFFFu);
                                            o[nt][dt][4 * g + 3] += nonfinite_term<DT>(wgt, e.y >> 16);
                                        }
                                    }
                                    asm volatile("" ::: "memory");  // one load at a time: registers stay with the main path
                                }
                        }
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                }
                ok = ok_next;
                va = va_next;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) l[nt] = half_sum(l[nt]);
        }

        // waves that took other keys of the same rows hand their results over
        if (m * RB < rows) {
            float* const buf = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int half = WK / 2; half >= 1; half >>= 1) {
                const int slot = WR == 2 ? wr : wk % half;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    __syncthreads();
                    if (wk >= half && wk < 2 * half) {
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                buf[slot * 64 * (DP / 2) + (dt * 16 + i) * 64 + lane] = o[nt][dt][i];
                        s_ml[slot][0][lane] = mx[nt];
                        s_ml[slot][1][lane] = l[nt];
                    }
                    __syncthreads();
                    if (wk < half) {
                        const float m2 = s_ml[slot][0][lane], l2 = s_ml[slot][1][lane];
                        const float mn = fmaxf(mx[nt], m2);
                        const float a1 = shift_of(mx[nt], mn), a2 = shift_of(m2, mn);
                        l[nt] = l[nt] * a1 + l2 * a2;
                        mx[nt] = mn;
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[nt][dt][i] =
                                    o[nt][dt][i] * a1 + buf[slot * 64 * (DP / 2) + (dt * 16 + i) * 64 + lane] * a2;
                    }
                }
            }
            __syncthreads();  // the tiles are the waves' own again
        }

        if (wk == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = wr * WROWS + nt * 32 + col, row = m * RB + r;
                if (whole) {
                    if (row < p.N * p.G) {
                        const int node = row / p.G;
                        const float inv = row < rows ? 1.f / l[nt] : 0.f;  // zeros for an absent node
                        uint8_t* const dst = p.out + 2 * (b * p.os[0] + node * p.os[1] +
                                                          static_cast<int64_t>(h * p.G + row - node * p.G) * p.os[2]);
#pragma unroll
                        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                if (32 * dt + 8 * g < p.D)
                                    *reinterpret_cast<v4s*>(dst + 2 * (32 * dt + 8 * g + 4 * hh)) =
                                        pack4<DT>(o[nt][dt][4 * g] * inv, o[nt][dt][4 * g + 1] * inv,
                                                  o[nt][dt][4 * g + 2] * inv, o[nt][dt][4 * g + 3] * inv);
                    }
                } else if (row < rows) {
                    float* const rec =
                        p.part + ((static_cast<int64_t>(c) * 2 + (f == f0 ? 0 : 1)) * p.MT + m) * (RB * (DP + 2));
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            *reinterpret_cast<float4*>(rec + r * DP + 32 * dt + 8 * g + 4 * hh) =
                                make_float4(o[nt][dt][4 * g], o[nt][dt][4 * g + 1], o[nt][dt][4 * g + 2],
                                            o[nt][dt][4 * g + 3]);
                    if (hh == 0) {
                        rec[RB * DP + r] = mx[nt];
                        rec[RB * DP + RB + r] = l[nt];
                    }
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
template <int DT, int DP, int RB>
__global__ __launch_bounds__(kThreads) void k_tree_merge(TreeAttnParams p) {
    constexpr int TPR = DP / 4, RPB = kThreads / TPR;
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

template <int DT, int DP, int NT, int WR>
hipError_t launch_one(const TreeAttnParams& p, hipStream_t st, const LaunchEvents& ev) {
    const int64_t grid = p.MT == 1 ? p.clusters : static_cast<int64_t>((p.clusters + 7) / 8) * 8 * p.MT;
    hipExtLaunchKernelGGL((k_tree_attn<DT, DP, NT, WR>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, st,
                          ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

template <int DT, int DP, int RB>
hipError_t merge_one(const TreeAttnParams& p, hipStream_t st, const LaunchEvents& ev) {
    constexpr int RPB = kThreads / (DP / 4);
    hipExtLaunchKernelGGL((k_tree_merge<DT, DP, RB>), dim3(p.B * p.Hkv, (p.N * p.G + RPB - 1) / RPB), dim3(kThreads), 0,
                          st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t launch_rows_of(const TreeAttnParams& p, int rows, bool merge, hipStream_t st, const LaunchEvents& ev) {
    if (rows == 32) return merge ? merge_one<DT, DP, 32>(p, st, ev) : launch_one<DT, DP, 1, 1>(p, st, ev);
    if (rows == 64) return merge ? merge_one<DT, DP, 64>(p, st, ev) : launch_one<DT, DP, 2, 1>(p, st, ev);
    return merge ? merge_one<DT, DP, 128>(p, st, ev) : launch_one<DT, DP, 2, 2>(p, st, ev);
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
