// gfx950 kernels of attention on latent rows: new tokens and drafted trees
// against a paged cache whose rows are shared by all heads.
//
// For every sequence b, node i and head h,
//
//   o = sum_j w_j c_j[:dv] / sum_j w_j,   w_j = 2^(x_j - m),  x_j = scale log2(e) q.c_j,
//
// over the cache rows j < len and the nodes j that are i or its ancestors.  A row
// c_j is key and value at once: it is read once for all N * H query rows.
//
//   k_latent_attn  all sequences' tiles of 32 keys as one line, cut into equal parts;
//                  a workgroup walks a part for 32 or 64 query rows, and leaves
//                  results of whole sequences, or sums in float32 of pieces;
//   k_latent_join  the pieces of a sequence added up.
//
// 512 values a row are 128 registers of sums for 32 query rows, and each row of the
// cache takes part in two products, so the eight waves have two roles: four make
// the scores and weights of a tile (16 x 16 x 32 products, 16 keys by half the rows
// each), four stage tiles and sum a quarter of the values each (32 x 32 x 16).  A
// ring of four tiles in LDS and two of weights keep them one tile apart, with one
// barrier a tile.  With every wave doing both, the sums spilled (32 trees 281 us,
// 64 tokens 205).
// Rows come by loads that write LDS directly, two tiles ahead; page numbers by
// scalar loads, as the compiler's own vector loads would wait for all of these.
// Weights are rounded once, to the input type.
//
// What bounds it: 64 new tokens of 128 heads over at most 4096 rows (207 MB, 46
// GFLOP) take 90 us and 10 for the join, 32 trees of 16 nodes and 16 heads over at most 8192
// (202 MB, 71 GFLOP) 135 and 10: 480 to 520 TFLOP/s.  A workgroup's start, first tile,
// last tile and results are about 24 us; a tile of 64 rows is 0.9 us, of which the scores'
// chain (products, maximum, exponentials, weights to LDS) is 0.5 and the products
// beside it 0.4.  A part of few tiles is latency: 13 us for one token over 1111 rows.

#include "sv_attn.h"
#include "sv_latent.h"

namespace sv {
namespace {

__device__ __forceinline__ int clamp_len(const LatentParams& p, int len) {
    const int cap = p.width << p.ps_shift;
    return len < 0 ? 0 : len > cap ? cap : len;
}

// The 16-byte chunks of a row are stored at positions XORed with this.  A wide LDS
// read takes 16 lanes at a time (0-3, 12-15, 20-23, 24-27 and so on) over 64
// banks, in which rows of 1152 or 640 bytes alternate between two halves: the key
// operand's 16 lanes (rows 0-3 and 12-15 at one chunk, 4-11 at its neighbour) and
// the transposing read's 32 (four rows at four chunks) then meet no bank twice.
// With row & 7, XORed as usual, the products of scores were as long again.
__device__ __forceinline__ int swizzle(int row) {
    return (row >> 1 & 1) << 2 | ((row >> 2 ^ row >> 3) & 1) << 1 | (row >> 3 & 1);
}

constexpr int kLatThreads = 512, kLatWaves = 8;
constexpr int kLatKeys = 32;  // keys of a tile
constexpr int kLatRing = 4;   // tiles in LDS: one for the values, one for the scores, two under way

// LDS of a kernel of RB rows and DK elements a row: the ring, two tiles' weights.
template <int DK, int RB>
struct LatentLds {
    static constexpr int kStage = kLatKeys * DK * 2;
    static constexpr int kP = RB * kLatKeys * 2;
    static constexpr int kP0 = kLatRing * kStage, kAll = kP0 + 2 * kP;
};

// Tiles of a sequence: its cache rows, then the tree's.
__device__ __forceinline__ int tiles_of(const LatentParams& p, int len) {
    return (clamp_len(p, len) + kLatKeys - 1) / kLatKeys + (p.N + kLatKeys - 1) / kLatKeys;
}

typedef const __attribute__((address_space(4))) int32_t const_i32;

// Everyone's LDS writes are seen, and everyone is here.
__device__ __forceinline__ void meet() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The value in all four quarter-waves: of the lanes with the same lane & 15.
__device__ __forceinline__ float quarter_max(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarter_sum(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

template <int DT>
__device__ __forceinline__ v4f mfma16(v8s a, v8s b, v4f c) {
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0,
                                                       0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0,
                                                      0);
}

template <int DT, int DK, int DV, int RB>
__global__ __launch_bounds__(kLatThreads, 2) void k_latent_attn(LatentParams p) {
    using Lds = LatentLds<DK, RB>;
    constexpr int TK = kLatKeys;
    constexpr int NC = DK / 8;                // 16-byte chunks per row
    constexpr int kLoads = NC / 8;            // wide loads of a value wave and tile
    constexpr int NQ = DK / 32;               // matrix steps of a row
    constexpr int NB = RB / 32;               // blocks of 16 rows a score wave has
    constexpr int RG = RB / 32;               // blocks of 32 rows a value wave has
    constexpr int CB = DV / 32 / 4;           // and of 32 values
    constexpr int kRowB = DK * 2;
    constexpr int kRec = RB * (DV + 2);       // floats of a partial result
    static_assert(NC % 8 == 0 && TK == 32 && CB >= 1, "layout");

    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_a[RB], s_m[RB], s_l[2][RB];
    __shared__ int s_raise[2];
    __shared__ __align__(4) uint8_t s_ok[kLatRing][4];  // rows of the tiles that exist
    __shared__ int64_t s_sum[kLatWaves];
    __shared__ int32_t s_scan[kLatWaves];
    __shared__ int s_b;
    __shared__ int64_t s_before;
    __shared__ unsigned int s_nf;

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool scores = w < 4;                // the others sum values
    const int wv = w & 3;
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
        b = c;
        before = f0 = 0;
        f1 = tiles_of(p, p.len[b]);
    } else {
        int64_t sum = 0;
        for (int i = tid; i < p.B; i += kLatThreads) sum += tiles_of(p, p.len[i]);
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(static_cast<long long>(sum), o);
        if (lane == 0) s_sum[w] = sum;
        __syncthreads();
        int64_t total = 0;
        for (int i = 0; i < kLatWaves; ++i) total += s_sum[i];
        const Cut cut(p.clusters, total);
        if (c >= cut.parts) return;
        f0 = cut.start(c);
        f1 = cut.start(c + 1);
        const bool tell = c == 0 && m == 0;  // leaves the sequences' places for the join
        int64_t carry = 0;
        for (int base = 0; base < p.B; base += kLatThreads) {
            const int i = base + tid;
            const int v = i < p.B ? tiles_of(p, p.len[i]) : 0;
            int s = v;
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(s, o);
                if (lane >= o) s += up;
            }
            if (lane == 63) s_scan[w] = s;
            __syncthreads();
            int64_t excl = carry + s - v, chunk = 0;
            for (int j = 0; j < kLatWaves; ++j) {
                if (j < w) excl += s_scan[j];
                chunk += s_scan[j];
            }
            if (i < p.B) {
                if (excl <= f0 && f0 < excl + v) {
                    s_b = i;
                    s_before = excl;
                }
                if (tell) p.start[i] = excl;
            }
            carry += chunk;
            __syncthreads();
            if (!tell && carry > f0) break;
        }
        if (tell && tid == 0) p.start[p.B] = total;
        b = __builtin_amdgcn_readfirstlane(s_b);
        before = s_before;
    }

    if (tid < 2) s_raise[tid] = 0;
    const uint32_t smem_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) uint8_t*)smem));
    // Staging, by the value waves, eight rows each: wide load k fills 1024 bytes; lane l's 16 are chunk
    // position (64 k + l) % NC of row (64 k + l) / NC.
    meet();
    // eight whole rows on one page: a scalar address and these
    const bool by_eights = p.ps_shift >= 3 && p.kcs[1] < (1u << 25);
    const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&kZero);
    const int ps_mask = (1 << p.ps_shift) - 1;
    const int tree_tiles = (p.N + TK - 1) / TK;
    const uint32_t p_at = smem_at + Lds::kP0;  // weights: 64 bytes a row, its four chunks so that eight rows use all banks
    // score wave wv: 16 keys (kh) against RB / 2 rows (from 16 NB rq on); lane & 15 is a key, then a row
    const int kh = wv & 1, rq = wv >> 1;
    int step = 0;  // of the workgroup, over all its sequences

    int64_t f = f0;
    while (f < f1) {
        // the lane's number, anew for every sequence: what is made of it would otherwise be kept in
        // registers over the whole kernel, and the loops' spilled
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int c16 = lane & 15, g4 = lane >> 4, hh = lane >> 5, col = lane & 31;
        const int len = clamp_len(p, p.len[b]);
        const int cache = (len + TK - 1) / TK, T = cache + tree_tiles;
        const int t0 = static_cast<int>(f - before);
        const int t1 = static_cast<int>(min(static_cast<int64_t>(T), t0 + (f1 - f)));
        const bool whole = t0 == 0 && t1 == T;
        int n = p.N;
        if (p.n_nodes) {
            n = p.n_nodes[b];
            n = n < 0 ? 0 : n > p.N ? p.N : n;
        }
        const int rows = n * p.H;
        const bool any = m * RB < rows;
        const int32_t* const tab = p.table + b * p.table_stride;
        const uint8_t* const nwb = p.nw + units(b, p.nws[0]);
        uint32_t off[kLoads], padded = 0;
        if (!scores) {
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int e = k * 64 + lane, r = e / NC, chunk = (e - r * NC) ^ swizzle(8 * wv + r);
                off[k] = static_cast<uint32_t>(units(r, p.kcs[1], chunk, 1));
                if (chunk * 8 >= p.C) padded |= 1u << k;
            }
        }
        // The page of the wave's eight rows of tile t, where these are whole cache rows on one page: a
        // scalar load, which does not queue behind the rows under way.  -1: not so.
        auto page_of = [&](int t) {
            const int key = t * TK + 8 * wv;
            return by_eights && t < t1 && key + 8 <= len ? *(const_i32*)(tab + (key >> p.ps_shift)) : -1;
        };
        // starts staging the wave's rows of tile t and says which exist (the others are staged as zeros)
        auto stage = [&](int t, int pg) {
            const bool tree = t >= cache;
            const int first = (tree ? t - cache : t) * TK + 8 * wv, slot = (t - t0) % kLatRing;
            const uint32_t to = smem_at + slot * Lds::kStage + wv * (kLoads * 1024);
            const uint32_t most = static_cast<uint32_t>(p.pages);
            if (static_cast<uint32_t>(pg) < most) {
                const uint8_t* const base = p.kc + units(pg, p.kcs[0], first & ps_mask, p.kcs[1]);
                if (p.C == DK) {
#pragma unroll
                    for (int k = 0; k < kLoads; ++k) load_lds(base, off[k], to + k * 1024);
                } else {
                    // chunks past the row's elements are zeros
#pragma unroll
                    for (int k = 0; k < kLoads; ++k)
                        load_lds(padded >> k & 1 ? zero : base + off[k], to + k * 1024);
                }
                if (lane == 0) s_ok[slot][wv] = 0xFF;
                return;
            }
            const int row = first + (lane & 7);  // lane j: whether row j exists, its page
            int pl = -1;
            if (!tree && row < len) pl = tab[row >> p.ps_shift];
            const uint32_t okm =
                static_cast<uint32_t>(tree ? __ballot(row < n) : __ballot(static_cast<uint32_t>(pl) < most)) & 0xFFu;
#pragma unroll 1
            for (int k = 0; k < kLoads; ++k) {
                const int e = k * 64 + lane, r = e / NC, chunk = (e - r * NC) ^ swizzle(8 * wv + r);
                const uint32_t pg_of = __shfl(pl, r);
                const uint8_t* const src =
                    tree ? nwb + units(first + r, p.nws[1], chunk, 1)
                         : p.kc + units(pg_of, p.kcs[0], (first + r) & ps_mask, p.kcs[1]) + 16 * chunk;
                load_lds((okm >> r & 1) && chunk * 8 < p.C ? src : zero, to + k * 1024);
            }
            if (lane == 0) s_ok[slot][wv] = static_cast<uint8_t>(okm);
        };
        // Step t: tile t is there, the weights of tile t - 1 too; tile t + 2 is sent for.  Both kinds of
        // waves go through the same barriers.
        int pg = -1;
        auto begin = [&] {
            const int p0 = page_of(t0), p1 = page_of(t0 + 1);
            pg = page_of(t0 + 2);
            stage(t0, p0);
            if (t0 + 1 < t1) stage(t0 + 1, p1);
        };
        auto arrive = [&](int t) {
            // this wave's loads of tile t have landed, the next tile's stay under way
            if (t + 1 < t1)
                wait_vm<kLoads>();
            else
                wait_vm<0>();
            meet();
            if (t + 2 < t1) stage(t + 2, pg);
            pg = page_of(t + 3);
        };
        // Rows of the tree in tile t that hold infinities or NaN among their values: these values go out
        // of the tile (0 times them would reach the nodes that do not see the row), and whoever sees the
        // row gets a score of NaN instead.
        auto cleaned = [&](int t) {
            uint32_t nf = 0;
            if (!scores) {
                const uint32_t at = ((t - t0) % kLatRing) * Lds::kStage;
#pragma unroll 1
                for (int k = 0; k < kLoads; ++k) {
                    const int e = k * 64 + lane, r = e / NC;
                    if (((e - r * NC) ^ swizzle(8 * wv + r)) * 8 >= p.dv) continue;
                    v8s* const y = reinterpret_cast<v8s*>(smem + at + (wv * kLoads + k) * 1024 + lane * 16);
                    const uint4 u = __builtin_bit_cast(uint4, *y);
                    if (nonfinite2<DT>(u.x) || nonfinite2<DT>(u.y) || nonfinite2<DT>(u.z) || nonfinite2<DT>(u.w)) {
                        nf |= 1u << (8 * wv + r);
                        *y = v8s{0, 0, 0, 0, 0, 0, 0, 0};
                    }
                }
            }
            if (tid == 0) s_nf = 0;
            meet();
            if (nf) atomicOr(&s_nf, nf);
            meet();
            return s_nf;
        };

        if (any && scores) {
            // ---- scores and weights, ahead of the value waves where both want the matrix unit: the sums of
            // the tile before then run under the exponentials
            __builtin_amdgcn_s_setprio(2);
            const bool active = m * RB + 16 * NB * rq < rows;
            int my_row[NB];
            v8s q[NB][NQ];
            uint64_t set[NB];
            uint64_t all = 0;
            if (t1 > cache && p.parent) all = ancestors(p.parent + static_cast<int64_t>(b) * p.N, n, lane, 0);
            const float scale2 = p.scale2;
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                my_row[r] = m * RB + 16 * (NB * rq + r) + c16;
                const bool in = my_row[r] < rows;
                const int node = in ? my_row[r] / p.H : 0;
                set[r] = p.parent ? __shfl(static_cast<unsigned long long>(all), node) : (2ull << node) - 1;
                // queries: the B operand, resident; a negative scale is moved into their sign
                const uint8_t* const src =
                    p.q + units(b, p.qs[0], node, p.qs[1]) + units(in ? my_row[r] - node * p.H : 0, p.qs[2]);
#pragma unroll
                for (int s = 0; s < NQ; ++s) {
                    const int d = s * 32 + g4 * 8;
                    v8s z = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (in && d < p.C) z = *reinterpret_cast<const v8s*>(src + 2 * d);
                    q[r][s] = p.flip ? z ^ static_cast<short>(0x8000) : z;
                }
            }
            const int key = 16 * kh + c16;
            uint32_t k_rd[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) k_rd[s] = smem_at + key * kRowB + (((4 * s + g4) ^ swizzle(key)) << 4);
            // the lane's four weights of a row: keys 16 kh + 4 g4 + 0..3 go where the value waves'
            // operand has them, 16 kh + (0..3, 8..11 | 4..7, 12..15)
            uint32_t p_wr[NB];
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                const int lr = 16 * (NB * rq + r) + c16;
                p_wr[r] = p_at + lr * 64 + (((2 * kh + (g4 & 1)) ^ ((lr >> 2) & 3)) << 4) + (g4 >> 1) * 8;
            }
            float mx[NB], l[NB], l_old[NB];
            v4f x[NB];
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                mx[r] = -INFINITY;
                l[r] = l_old[r] = 0.f;
                x[r] = v4f{0.f, 0.f, 0.f, 0.f};
            }
            // weights of the scores in x relative to the reference, into buffer `at`
            auto weigh = [&](int at) {
#pragma unroll
                for (int r = 0; r < NB; ++r) {
                    const float ref = mx[r] == -INFINITY ? 0.f : mx[r];
                    float y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i] = __builtin_amdgcn_exp2f(less(x[r][i], ref));
                        l[r] += y[i];
                    }
                    *reinterpret_cast<lds_v4s*>(p_wr[r] + at * Lds::kP) = pack4<DT>(y[0], y[1], y[2], y[3]);
                }
            };
#pragma unroll 1
            for (int t = t0; t <= t1; ++t, ++step) {
                meet();
                const int raised = s_raise[(step - 1) & 1];
                const uint32_t ok = *reinterpret_cast<const uint32_t*>(s_ok[(t - t0) % kLatRing]);
                const bool tree = t >= cache;
                const uint32_t at = ((t - t0) % kLatRing) * Lds::kStage;
                // the keys' operands a few steps at a time, those of the next two parts on their way meanwhile
                constexpr int kPart = NQ % 3 ? 2 : 3, kParts = NQ / kPart;
                static_assert(kParts * kPart == NQ && kParts >= 3, "steps");
                v8s kf[3][kPart];
                auto fetch = [&](int part) __attribute__((always_inline)) {
#pragma unroll
                    for (int j = 0; j < kPart; ++j) {
                        const int s = part * kPart + j;
                        kf[part % 3][j] = lds_read(k_rd[s & 1] + at + (s >> 1) * 128);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                };
                if (t > t0 && __builtin_amdgcn_readfirstlane(raised) == step) {
                    // a row of tile t - 1 is too far above its reference: a new one, from both waves that
                    // share the row, and the weights once more
                    float top[NB];
                    if (active) {
#pragma unroll
                        for (int r = 0; r < NB; ++r) {
                            top[r] = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
                            top[r] = quarter_max(top[r]);
                            if (g4 == 0) s_l[kh][16 * (NB * rq + r) + c16] = top[r];
                        }
                    }
                    meet();
                    if (active) {
#pragma unroll
                        for (int r = 0; r < NB; ++r) {
                            const int lr = 16 * (NB * rq + r) + c16;
                            // a row by its own scores alone: what other rows see leaves its bits as they are
                            const float high = fmaxf(top[r], s_l[kh ^ 1][lr]);
                            const float mn = high - mx[r] > kUp<DT> + 8.f ? fmaxf(mx[r], high - kUp<DT>) : mx[r];
                            const float a = shift_of(mx[r], mn);
                            if (g4 == 0 && kh == 0) s_a[lr] = a;
                            mx[r] = mn;
                            l[r] = l_old[r] * a;
                        }
                        weigh((step - 1) & 1);
                    }
                    meet();
                }
                if (t == t1) continue;
                uint32_t nf = 0;
                if (tree) nf = cleaned(t);
                if (active) {
                    v4f x2[NB];  // even and odd steps apart: the chains of sums are half as long
#pragma unroll
                    for (int r = 0; r < NB; ++r) x[r] = x2[r] = v4f{0.f, 0.f, 0.f, 0.f};
                    __builtin_amdgcn_sched_barrier(0);
                    fetch(0);
                    fetch(1);
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
                        if (part + 2 < kParts) fetch(part + 2);
#pragma unroll
                        for (int j = 0; j < kPart; ++j) {
                            const int s = part * kPart + j;
#pragma unroll
                            for (int r = 0; r < NB; ++r) {
                                v4f& sum = s & 1 ? x2[r] : x[r];
                                sum = mfma16<DT>(kf[part % 3][j], q[r][s], sum);
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    bool raise = false;
#pragma unroll
                    for (int r = 0; r < NB; ++r) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[r][i] = scaled(x[r][i] + x2[r][i], scale2);
                    }
                    if (tree || __builtin_amdgcn_readfirstlane(ok) != ~0u) {
                        const int at4 = 16 * kh + 4 * g4;
#pragma unroll
                        for (int r = 0; r < NB; ++r) {
                            uint32_t see = ok;
                            if (tree) see &= static_cast<uint32_t>(set[r] >> (t - cache) * TK);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                x[r][i] = see >> (at4 + i) & 1 ? nf >> (at4 + i) & 1 ? __builtin_nanf("") : x[r][i]
                                                               : -INFINITY;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < NB; ++r) {
                        const float top = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
                        raise |= top - mx[r] > kUp<DT> + 8.f;
                        l_old[r] = l[r];
                    }
                    if (__any(raise) && lane == 0) s_raise[step & 1] = step + 1;
                    weigh(step & 1);
                }
            }
            if (active) {
#pragma unroll
                for (int r = 0; r < NB; ++r) {
                    const int lr = 16 * (NB * rq + r) + c16;
                    const float sum = quarter_sum(l[r]);
                    if (g4 == 0) {
                        s_l[kh][lr] = sum;
                        if (kh == 0) s_m[lr] = mx[r];
                    }
                }
            }
            meet();
        } else {
            // ---- sums of values
            v16f o[RG][CB];
#pragma unroll
            for (int r = 0; r < RG; ++r)
#pragma unroll
                for (int s = 0; s < CB; ++s)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[r][s][i] = 0.f;
            if (any) {
                uint32_t v_rd[2][2];  // odd and even blocks of 32 values; the first rows and eight rows on
                const int vrow = 4 * hh + ((lane & 15) >> 2);
                const int low = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);  // chunk of the four of 32 dimensions
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        v_rd[s][j] = smem_at + (vrow + 8 * j) * kRowB +
                                     (((4 * ((wv * CB + s) & 1) + low) ^ swizzle(vrow + 8 * j)) << 4) + (lane & 1) * 8 +
                                     ((wv * CB + s) >> 1) * 128;
                const uint32_t p_rd = p_at + col * 64;
                const int p_xor = (col >> 2) & 3;
                begin();
#pragma unroll 1
                for (int t = t0; t <= t1; ++t, ++step) {
                    arrive(t);
                    const int raised = s_raise[(step - 1) & 1];
                    if (t > t0 && __builtin_amdgcn_readfirstlane(raised) == step) {
                        meet();
                        meet();
#pragma unroll
                        for (int r = 0; r < RG; ++r) {
                            const float a = s_a[r * 32 + col];
#pragma unroll
                            for (int s = 0; s < CB; ++s)
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[r][s][i] *= a;
                        }
                    }
                    if (t < t1 && t >= cache) cleaned(t);
                    if (t > t0) {
                        const uint32_t at = ((t - 1 - t0) % kLatRing) * Lds::kStage;
                        const uint32_t pa = p_rd + ((step - 1) & 1) * Lds::kP;
                        // operands of 16 keys, then those of the other 16 on their way meanwhile
                        v8s pf[2][RG], vf[2][CB];
                        auto fetch = [&](int t2) __attribute__((always_inline)) {
#pragma unroll
                            for (int r = 0; r < RG; ++r)
                                pf[t2][r] = lds_read(pa + r * 2048 + (((2 * t2 + hh) ^ p_xor) << 4));
#pragma unroll
                            for (int s = 0; s < CB; ++s) {
                                const uint32_t a = at + t2 * 16 * kRowB + (s >> 1) * 128;
                                vf[t2][s] = __builtin_shufflevector(lds_read_tr(v_rd[s & 1][0] + a),
                                                                    lds_read_tr(v_rd[s & 1][1] + a), 0, 1, 2, 3, 4, 5, 6, 7);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        };
                        __builtin_amdgcn_sched_barrier(0);
                        fetch(0);
#pragma unroll
                        for (int t2 = 0; t2 < 2; ++t2) {
                            if (t2 == 0) fetch(1);
#pragma unroll
                            for (int s = 0; s < CB; ++s)
#pragma unroll
                                for (int r = 0; r < RG; ++r) o[r][s] = mfma<DT>(vf[t2][s], pf[t2][r], o[r][s]);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
                meet();  // the sums of the weights are there
            }
            // The results go through the ring, which nobody reads any more, so that rows leave whole:
            // dimensions 32 (wv CB + s) + 8 g + 4 hh + 0..3 of row 32 r + col, four floats in a place
            // XORed with the row (16 rows' writes at a time meet no bank twice)
            if (any && !scores) {
#pragma unroll
                for (int r = 0; r < RG; ++r)
#pragma unroll
                    for (int s = 0; s < CB; ++s)
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const int lr = r * 32 + col, d4 = (32 * (wv * CB + s) + 2 * i + 4 * hh) / 4;
                            const v16f& y = o[r][s];
                            *reinterpret_cast<float4*>(smem + lr * (DV * 4) + ((d4 ^ (lr & 15)) << 4)) =
                                make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                        }
            }
        }
        meet();
        auto sums = [&](int lr, int d4) {
            return *reinterpret_cast<const float4*>(smem + lr * (DV * 4) + ((d4 ^ (lr & 15)) << 4));
        };
        if (whole) {
#pragma unroll 1
            for (int e = tid; e < RB * (DV / 8); e += kLatThreads) {
                const int lr = e / (DV / 8), d = (e - lr * (DV / 8)) * 8, row = m * RB + lr;
                if (row >= p.N * p.H || d >= p.dv) continue;
                const int node = row / p.H;
                uint8_t* const dst = p.out + units(b, p.os[0], node, p.os[1]) + units(row - node * p.H, p.os[2]) + 2 * d;
                v8s y = {0, 0, 0, 0, 0, 0, 0, 0};  // an absent node's row
                if (row < rows) {
                    const float inv = 1.f / (s_l[0][lr] + s_l[1][lr]);
                    const float4 lo = sums(lr, d / 4), hi = sums(lr, d / 4 + 1);
                    y = __builtin_shufflevector(pack4<DT>(lo.x * inv, lo.y * inv, lo.z * inv, lo.w * inv),
                                                pack4<DT>(hi.x * inv, hi.y * inv, hi.z * inv, hi.w * inv), 0, 1, 2, 3,
                                                4, 5, 6, 7);
                }
                *reinterpret_cast<v8s*>(dst) = y;
            }
        } else if (any) {
            float* const rec = p.part + ((static_cast<int64_t>(c) * 2 + (f == f0 ? 0 : 1)) * p.MT + m) * kRec;
            const int last = min(RB, rows - m * RB);
#pragma unroll 4
            for (int e = tid; e < last * (DV / 4); e += kLatThreads) {
                const int lr = e / (DV / 4), d4 = e - lr * (DV / 4);
                if (4 * d4 < p.dv) *reinterpret_cast<float4*>(rec + lr * DV + 4 * d4) = sums(lr, d4);
            }
            if (tid < last) {
                rec[RB * DV + tid] = s_m[tid];
                rec[RB * DV + RB + tid] = s_l[0][tid] + s_l[1][tid];
            }
        }
        meet();  // the stages and sums are free again
        f += t1 - t0;
        if (t1 == T && f < f1) {
            before += T;
            ++b;
        }
    }
}

// Joins the partial results of the sequences that were divided: o = sum_c
// 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c over the parts in order.  A workgroup
// takes one query row; DV / 4 threads are a team that takes four dimensions
// each, and the teams share the row's parts.  Where sequences have few parts a
// wave takes a row instead: no barriers, half the time (sequences of two to
// three parts 19 us with a workgroup each).
template <int DT, int DV, int THREADS>
__global__ __launch_bounds__(THREADS) void k_latent_join(LatentParams p, int RB) {
    constexpr int TEAM = DV / 4, TEAMS = THREADS / TEAM;
    constexpr int kFlight = 8;  // parts a thread loads at a time
    __shared__ float s_m[THREADS / 64], s_l[TEAMS];
    __shared__ float4 s_o[THREADS];
    const int tid = threadIdx.x, b = blockIdx.x;
    const int64_t first = p.start[b], T = p.start[b + 1] - first;
    const Cut cut(p.clusters, p.start[p.B]);
    const int c0 = cut.of(first), c1 = cut.of(first + T - 1);
    if (c0 == c1) return;
    const int team = tid / TEAM, d = (tid % TEAM) * 4;
    const int row = blockIdx.y;
    int n = p.N;
    if (p.n_nodes) {
        n = p.n_nodes[b];
        n = n < 0 ? 0 : n > p.N ? p.N : n;
    }
    const int node = row / p.H, head = row - node * p.H;
    v4s res = {0, 0, 0, 0};
    if (node < n) {
        const int m = row / RB, r = row - m * RB;
        const int64_t rec = RB * (DV + 2);
        // the first part's record is its second one unless the part begins here
        const int slot0 = cut.start(c0) == first ? 0 : 1;
        auto at = [&](int c) { return p.part + ((static_cast<int64_t>(c) * 2 + (c == c0 ? slot0 : 0)) * p.MT + m) * rec; };
        float mx = -INFINITY;
        for (int c = c0 + tid; c <= c1; c += THREADS) mx = fmaxf(mx, at(c)[RB * DV + r]);
        for (int o = 1; o < 64; o <<= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
        if ((tid & 63) == 0) s_m[tid >> 6] = mx;
        __syncthreads();
        for (int i = 0; i < THREADS / 64; ++i) mx = fmaxf(mx, s_m[i]);
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0 + team; c <= c1; c += kFlight * TEAMS) {
            float mc[kFlight], lc[kFlight];
            float4 v[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                if (c + k * TEAMS > c1) break;
                const float* const q = at(c + k * TEAMS);
                mc[k] = q[RB * DV + r];
                lc[k] = q[RB * DV + RB + r];
                v[k] = d < p.dv ? *reinterpret_cast<const float4*>(q + r * DV + d) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kFlight; ++k)
                if (c + k * TEAMS <= c1) {
                    const float a = shift_of(mc[k], mx);
                    l += a * lc[k];
                    o.x += a * v[k].x;
                    o.y += a * v[k].y;
                    o.z += a * v[k].z;
                    o.w += a * v[k].w;
                }
        }
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
        const float inv = 1.f / l;
        res = pack4<DT>(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
    if (team > 0 || d >= p.dv) return;
    *reinterpret_cast<v4s*>(p.out + units(b, p.os[0], node, p.os[1]) + units(head, p.os[2]) + 2 * d) = res;
}

template <int DT, int DV>
__global__ __launch_bounds__(256) void k_latent_join_few(LatentParams p, int RB) {
    constexpr int kD = DV / 256;  // groups of four dimensions a lane has
    const int b = blockIdx.x, lane = threadIdx.x & 63;
    const int row = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first = p.start[b], T = p.start[b + 1] - first;
    const Cut cut(p.clusters, p.start[p.B]);
    const int c0 = cut.of(first), c1 = cut.of(first + T - 1);
    if (c0 == c1 || row >= p.N * p.H) return;
    int n = p.N;
    if (p.n_nodes) {
        n = p.n_nodes[b];
        n = n < 0 ? 0 : n > p.N ? p.N : n;
    }
    const int node = row / p.H, head = row - node * p.H;
    v4s res[kD];
#pragma unroll
    for (int k = 0; k < kD; ++k) res[k] = v4s{0, 0, 0, 0};
    if (node < n) {
        const int m = row / RB, r = row - m * RB;
        const int64_t rec = RB * (DV + 2);
        // the first part's record is its second one unless the part begins here
        const int slot0 = cut.start(c0) == first ? 0 : 1;
        auto at = [&](int c) { return p.part + ((static_cast<int64_t>(c) * 2 + (c == c0 ? slot0 : 0)) * p.MT + m) * rec; };
        float mx = -INFINITY, l = 0.f;
        float4 o[kD];
#pragma unroll
        for (int k = 0; k < kD; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kFlight = 4;
        for (int c = c0; c <= c1; c += kFlight) {
            float mc[kFlight], lc[kFlight];
            float4 v[kFlight][kD];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const float* const q = at(min(c + i, c1));
                mc[i] = c + i <= c1 ? q[RB * DV + r] : -INFINITY;
                lc[i] = q[RB * DV + RB + r];
#pragma unroll
                for (int k = 0; k < kD; ++k) {
                    const int d = k * 256 + lane * 4;
                    v[i][k] = d < p.dv && c + i <= c1 ? *reinterpret_cast<const float4*>(q + r * DV + d)
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            float mn = mx;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) mn = fmaxf(mn, mc[i]);
            const float a = shift_of(mx, mn);
            l *= a;
#pragma unroll
            for (int k = 0; k < kD; ++k) {
                o[k].x *= a;
                o[k].y *= a;
                o[k].z *= a;
                o[k].w *= a;
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                if (c + i > c1) break;
                const float e = shift_of(mc[i], mn);
                l += e * lc[i];
#pragma unroll
                for (int k = 0; k < kD; ++k) {
                    o[k].x += e * v[i][k].x;
                    o[k].y += e * v[i][k].y;
                    o[k].z += e * v[i][k].z;
                    o[k].w += e * v[i][k].w;
                }
            }
            mx = mn;
        }
        const float inv = 1.f / l;
#pragma unroll
        for (int k = 0; k < kD; ++k) res[k] = pack4<DT>(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv);
    }
    uint8_t* const dst = p.out + units(b, p.os[0], node, p.os[1]) + units(head, p.os[2]);
#pragma unroll
    for (int k = 0; k < kD; ++k)
        if (k * 256 + lane * 4 < p.dv) *reinterpret_cast<v4s*>(dst + 2 * (k * 256 + lane * 4)) = res[k];
}

template <int DT, int DK, int DV, int RB>
hipError_t attn_one(const LatentParams& p, hipStream_t st, const LaunchEvents& ev) {
    constexpr int lds = LatentLds<DK, RB>::kAll;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(k_latent_attn<DT, DK, DV, RB>), lds);
    if (e != hipSuccess) return e;
    const int64_t grid = p.MT == 1 ? p.clusters : static_cast<int64_t>((p.clusters + 7) / 8) * 8 * p.MT;
    hipExtLaunchKernelGGL((k_latent_attn<DT, DK, DV, RB>), dim3(static_cast<unsigned>(grid)), dim3(kLatThreads), lds,
                          st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

template <int DT, int DK, int DV>
hipError_t attn_rows(const LatentParams& p, int rows, hipStream_t st, const LaunchEvents& ev) {
    return rows == 32 ? attn_one<DT, DK, DV, 32>(p, st, ev) : attn_one<DT, DK, DV, 64>(p, st, ev);
}

template <int DT, int DV>
hipError_t join_one(const LatentParams& p, const LatentShape& s, hipStream_t st, const LaunchEvents& ev) {
    // a wave a row where a sequence has few parts (2 and 8: 10.6 us for 20.2 with a workgroup a row,
    // 9.7 for 18.8), else a workgroup (36 parts: 6.4 for 15.5)
    if (p.clusters <= 8 * p.B) {
        hipExtLaunchKernelGGL((k_latent_join_few<DT, DV>), dim3(p.B, (p.N * p.H + 3) / 4), dim3(256), 0, st, ev.start,
                              ev.stop, 0, p, s.rows);
        return hipGetLastError();
    }
    const dim3 grid(p.B, p.N * p.H);
    hipExtLaunchKernelGGL((k_latent_join<DT, DV, 256>), grid, dim3(256), 0, st, ev.start, ev.stop, 0, p, s.rows);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_latent_attn(const LatentParams& p, const LatentShape& s, int dtype, hipStream_t st,
                              const LaunchEvents& ev) {
    if (dtype == DT_BF16)
        return s.wide ? attn_rows<DT_BF16, 576, 512>(p, s.rows, st, ev) : attn_rows<DT_BF16, 320, 256>(p, s.rows, st, ev);
    return s.wide ? attn_rows<kDTypeF16, 576, 512>(p, s.rows, st, ev) : attn_rows<kDTypeF16, 320, 256>(p, s.rows, st, ev);
}

hipError_t launch_latent_join(const LatentParams& p, const LatentShape& s, int dtype, hipStream_t st,
                              const LaunchEvents& ev) {
    if (dtype == DT_BF16)
        return s.wide ? join_one<DT_BF16, 512>(p, s, st, ev) : join_one<DT_BF16, 256>(p, s, st, ev);
    return s.wide ? join_one<kDTypeF16, 512>(p, s, st, ev) : join_one<kDTypeF16, 256>(p, s, st, ev);
}

}  // namespace sv
