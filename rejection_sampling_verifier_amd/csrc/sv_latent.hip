// gfx950 kernels of attention on latent rows: new tokens and drafted trees
// against a paged cache whose rows are shared by all heads.
//
// For every sequence b, node i and head h,
//
//   o = sum_j w_j c_j[:dv] / sum_j w_j,   w_j = 2^(x_j - m),  x_j = scale log2(e) q.c_j,
//
// over the cache rows j < len and the nodes j that are i or its ancestors.  A row
// c_j is key and value at once: it is read once for all N * H query rows.

#include "sv_attn.h"
#include "sv_latent.h"

namespace sv {
namespace {

__device__ __forceinline__ int clamp_len(const LatentParams& p, int len) {
    const int cap = p.width << p.ps_shift;
    return len < 0 ? 0 : len > cap ? cap : len;
}

constexpr int kLatThreads = 512, kLatWaves = 8;
constexpr int kLatKeys = 32;  // keys of a tile

// What a kernel of RB rows and DK elements a row keeps in LDS: a ring of tiles,
// the partial scores that two waves exchange, the weights.
template <int DK, int RB>
struct LatentLds {
    static constexpr int kStage = kLatKeys * DK * 2;
    static constexpr int kX = RB / 32 * 2 * 4096;  // two waves per 32 rows
    static constexpr int kP = RB * kLatKeys * 2;
    static constexpr int kFit = ((160 << 10) - 4096 - kX - kP) / kStage;
    static constexpr int kRing = kFit > 4 ? 4 : kFit;
    static constexpr int kX0 = kRing * kStage, kP0 = kX0 + kX, kAll = kP0 + kP;
    static_assert(kRing >= 3, "tiles under way");
};

// Tiles of a sequence: its cache rows, then the tree's.
__device__ __forceinline__ int tiles_of(const LatentParams& p, int len) {
    return (clamp_len(p, len) + kLatKeys - 1) / kLatKeys + (p.N + kLatKeys - 1) / kLatKeys;
}

template <int DT, int DK, int DV, int RB>
__global__ __launch_bounds__(kLatThreads, 2) void k_latent_attn(LatentParams p) {
    using Lds = LatentLds<DK, RB>;
    constexpr int TK = kLatKeys;
    constexpr int NC = DK / 8;                // 16-byte chunks per row
    constexpr int NL = TK * NC / 64;          // wide loads of a tile
    constexpr int kMost = (NL + kLatWaves - 1) / kLatWaves, kLeast = NL / kLatWaves;  // of a wave
    constexpr int NQ = DK / 32;               // matrix steps of half a row
    constexpr int RG = RB / 32;               // groups of 32 rows
    constexpr int CB = DV / 32 / kLatWaves;   // blocks of 32 values a wave sums
    constexpr int kRowB = DK * 2;
    constexpr int kRec = RB * (DV + 2);       // floats of a partial result
    static_assert(NC % 8 == 0 && NL * 64 == TK * NC && CB >= 1, "layout");

    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_a[RB], s_m[RB], s_l[2][RB];
    __shared__ int s_move[2];
    __shared__ int64_t s_sum[kLatWaves];
    __shared__ int32_t s_scan[kLatWaves];
    __shared__ int s_b;
    __shared__ int64_t s_before;
    __shared__ unsigned long long s_nf;

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hh = lane >> 5, col = lane & 31;
    const int rg = w >> 1, kh = w & 1;        // scores: the wave's rows and half of their elements
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

    const uint32_t smem_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) uint8_t*)smem));
    // Staging: wide load i = w + 8 k of a tile fills 1024 bytes; lane l's 16 are chunk position
    // (64 i + l) % NC of row (64 i + l) / NC.  Eight rows are NC / 8 loads.
    uint32_t off[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int e = (w + 8 * k) * 64 + lane, r = e / NC;
        off[k] = static_cast<uint32_t>(units(r & 7, p.kcs[1], (e - r * NC) ^ swizzle(r), 1));
    }
    const int mine = w < NL - kLeast * kLatWaves ? kLeast + 1 : kLeast;  // loads of this wave
    // eight whole rows on one page: a scalar address and these
    const bool by_eights = p.C == DK && p.ps_shift >= 3 && p.kcs[1] < (1u << 25);
    // reading, within a stage: keys 16 bytes a lane (four chunks, the next are 128 bytes on), values transposed
    uint32_t k_rd[4], v_rd[CB];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        k_rd[s] = smem_at + col * kRowB + (((kh * (NC / 2) + 2 * s + hh) ^ swizzle(col)) << 4);
    {
        const int vrow = 4 * hh + ((lane & 15) >> 2);
        const int low = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);  // chunk of the four of 32 dimensions
#pragma unroll
        for (int s = 0; s < CB; ++s)
            v_rd[s] = smem_at + vrow * kRowB + (((4 * (w * CB + s) + low) ^ swizzle(vrow)) << 4) + (lane & 1) * 8;
    }
    const uint32_t x_at = smem_at + Lds::kX0 + lane * 16;              // + 4096 per wave, 1024 per four sums
    const int p_xor = (col >> 1) & 3;                                  // weights: [row][4 chunks], 8 rows on all banks
    const uint32_t p_at = smem_at + Lds::kP0 + col * 64;
    const float scale2 = p.scale2;
    const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&kZero);
    const int ps_mask = (1 << p.ps_shift) - 1;
    const int tree_tiles = (p.N + TK - 1) / TK;

    int64_t f = f0;
    while (f < f1) {
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
        v16f o[RG][CB];
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int s = 0; s < CB; ++s)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[r][s][i] = 0.f;

        if (m * RB < rows) {
            const int my_row = m * RB + rg * 32 + col;  // of the scores
            const bool active = rg < RG && m * RB + rg * 32 < rows;
            const int32_t* const tab = p.table + b * p.table_stride;
            const uint8_t* const nwb = p.nw + units(b, p.nws[0]);
            float mx = -INFINITY, l = 0.f;
            // lane j: the page of row j of tile t
            auto page = [&](int t) {
                int pg = -1;
                if (t < cache) {
                    const int key = t * TK + col;
                    if (key < len) pg = tab[key >> p.ps_shift];
                }
                return pg;
            };
            // starts staging tile t; returns the rows that exist (the others are staged as zeros)
            auto stage = [&](int t, int pg, uint32_t at) {
                const bool tree = t >= cache;
                const int first = (tree ? t - cache : t) * TK;
                const uint32_t okm = static_cast<uint32_t>(
                    tree ? __ballot(first + col < n)
                         : __ballot(static_cast<uint32_t>(pg) < static_cast<uint32_t>(p.pages)));
                const uint32_t to = smem_at + at + w * 1024;
                if (!tree && okm == ~0u && by_eights) {
#pragma unroll
                    for (int k = 0; k < kMost; ++k) {
                        if (k == kLeast && mine == kLeast) break;
                        const int g = (w + 8 * k) / (NC / 8) * 8;
                        const uint32_t pg8 = __builtin_amdgcn_readlane(pg, g);
                        load_lds(p.kc + units(pg8, p.kcs[0], (first + g) & ps_mask, p.kcs[1]), off[k], to + k * 8192);
                    }
                } else {
#pragma unroll 1
                    for (int k = 0; k < mine; ++k) {
                        const int e = (w + 8 * k) * 64 + lane, r = e / NC, chunk = (e - r * NC) ^ swizzle(r);
                        const uint32_t pg_of = __shfl(pg, r);
                        const uint8_t* const src =
                            tree ? nwb + units(first + r, p.nws[1], chunk, 1)
                                 : p.kc + units(pg_of, p.kcs[0], (first + r) & ps_mask, p.kcs[1]) + 16 * chunk;
                        load_lds((okm >> r & 1) && chunk * 8 < p.C ? src : zero, to + k * 8192);
                    }
                }
                return okm;
            };

            // queries: the B operand, resident; a negative scale is moved into their sign
            v8s q[NQ];
            const int node = my_row < rows ? my_row / p.H : 0;
            {
                const uint8_t* const src = p.q + units(b, p.qs[0], node, p.qs[1]) +
                                           units(my_row < rows ? my_row - node * p.H : 0, p.qs[2]);
#pragma unroll
                for (int s = 0; s < NQ; ++s) {
                    const int d = kh * (DK / 2) + s * 16 + hh * 8;
                    v8s z = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (active && my_row < rows && d < p.C) z = *reinterpret_cast<const v8s*>(src + 2 * d);
                    q[s] = p.flip ? z ^ static_cast<short>(0x8000) : z;
                }
            }
            uint64_t set = 0;  // the nodes the row sees
            if (t1 > cache) {
                if (p.parent)
                    set = __shfl(static_cast<unsigned long long>(
                                     ancestors(p.parent + static_cast<int64_t>(b) * p.N, n, lane, 0)),
                                 node);
                else
                    set = (2ull << node) - 1;
            }

            // the ring: tiles t .. t + kRing - 2 are under way or there
            constexpr int kAhead = Lds::kRing - 1;
            uint32_t okm[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                okm[k] = 0;
                if (t0 + k < t1) okm[k] = stage(t0 + k, page(t0 + k), k * Lds::kStage);
            }
            int pg = t0 + kAhead < t1 ? page(t0 + kAhead) : -1;
            uint32_t at = 0, to = kAhead * Lds::kStage;
#pragma unroll 1
            for (int t = t0; t < t1; ++t) {
                const bool tree = t >= cache;
                // this wave's loads of tile t have landed (later tiles' stay under way); with the
                // barrier everyone's, and everyone is done with the tile before it
                if (t + kAhead - 1 < t1) {
                    if (mine > kLeast)
                        wait_vm<(kAhead - 1) * kMost>();
                    else
                        wait_vm<(kAhead - 1) * kLeast>();
                } else {
                    wait_vm<0>();
                }
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
                const uint32_t ok = okm[0];
#pragma unroll
                for (int k = 0; k + 1 < kAhead; ++k) okm[k] = okm[k + 1];
                if (t + kAhead < t1) {
                    okm[kAhead - 1] = stage(t + kAhead, pg, to);
                    if (t + kAhead + 1 < t1) pg = page(t + kAhead + 1);
                }
                uint32_t nf = 0;  // rows of the tree that hold infinities or NaN among their values
                if (tree) {
                    // these go out of the tile (0 times them would reach the nodes that do not see
                    // the row); whoever sees the row gets a score of NaN instead
#pragma unroll 1
                    for (int k = 0; k < mine; ++k) {
                        const int e = (w + 8 * k) * 64 + lane, r = e / NC;
                        if (((e - r * NC) ^ swizzle(r)) * 8 >= p.dv) continue;
                        v8s* const y = reinterpret_cast<v8s*>(smem + at + (w + 8 * k) * 1024 + lane * 16);
                        const uint4 u = __builtin_bit_cast(uint4, *y);
                        if (nonfinite2<DT>(u.x) || nonfinite2<DT>(u.y) || nonfinite2<DT>(u.z) || nonfinite2<DT>(u.w)) {
                            nf |= 1u << r;
                            *y = v8s{0, 0, 0, 0, 0, 0, 0, 0};
                        }
                    }
                    if (tid == 0) s_nf = 0;
                    __syncthreads();
                    if (nf) atomicOr(&s_nf, static_cast<unsigned long long>(nf));
                    __syncthreads();
                    nf = static_cast<uint32_t>(s_nf);
                }
                v16f x;
                if (active) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = 0.f;
#pragma unroll
                    for (int s = 0; s < NQ; ++s) x = mfma<DT>(lds_read(k_rd[s & 3] + at + (s >> 2) * 128), q[s], x);
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *reinterpret_cast<__attribute__((address_space(3))) v4f*>(x_at + w * 4096 + g * 1024) =
                            v4f{x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
                }
                if (tid == 0) s_move[t & 1] = 0;
                __syncthreads();
                if (active) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const v4f y = *reinterpret_cast<__attribute__((address_space(3))) v4f*>(
                            x_at + (w ^ 1) * 4096 + g * 1024);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[4 * g + i] += y[i];
                    }
                    if (tree || ok != ~0u) {
                        uint32_t see = ok;
                        if (tree) see &= static_cast<uint32_t>(set >> (t - cache) * TK);
                        const uint32_t bad = nf >> 4 * hh;
                        see >>= 4 * hh;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t bit = 1u << (8 * (i >> 2) + (i & 3));
                            x[i] = see & bit ? bad & bit ? __builtin_nanf("") : x[i] : -INFINITY;
                        }
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = fmaxf(top, x[i]);
                    top = scaled(half_max(top), scale2);
                    if (__any(top - mx > kUp<DT> + 8.f)) {
                        const float mn = fmaxf(mx, top - kUp<DT>);
                        const float a = shift_of(mx, mn);
                        l *= a;
                        mx = mn;
                        // the sums of all waves move along; the other groups' rows stay
                        s_a[rg * 32 + col] = a;
                        if (lane == 0) atomicOr(&s_move[t & 1], 1 << rg);
                    }
                    const float ref = mx == -INFINITY ? 0.f : mx;
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[i] = __builtin_amdgcn_exp2f(less(scaled(kh ? x[8 + i] : x[i], scale2), ref));
                        l += y[i];
                    }
                    const v4s lo = pack4<DT>(y[0], y[1], y[2], y[3]), hi = pack4<DT>(y[4], y[5], y[6], y[7]);
                    *reinterpret_cast<__attribute__((address_space(3))) v8s*>(
                        p_at + rg * 2048 + (((2 * kh + hh) ^ p_xor) << 4)) =
                        __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                }
                __syncthreads();
                const int move = s_move[t & 1];
                if (move) {
#pragma unroll
                    for (int r = 0; r < RG; ++r) {
                        if (!(move >> r & 1)) continue;
                        const float a = s_a[r * 32 + col];
#pragma unroll
                        for (int s = 0; s < CB; ++s)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[r][s][i] *= a;
                    }
                }
#pragma unroll
                for (int t2 = 0; t2 < 2; ++t2) {
                    v8s pf[RG];
#pragma unroll
                    for (int r = 0; r < RG; ++r) pf[r] = lds_read(p_at + r * 2048 + (((2 * t2 + hh) ^ p_xor) << 4));
#pragma unroll
                    for (int s = 0; s < CB; ++s) {
                        const uint32_t a = v_rd[s] + at + t2 * 16 * kRowB;
                        const v8s vf =
                            __builtin_shufflevector(lds_read_tr(a), lds_read_tr(a + 8 * kRowB), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                        for (int r = 0; r < RG; ++r) o[r][s] = mfma<DT>(vf, pf[r], o[r][s]);
                    }
                }
                at = at + Lds::kStage == Lds::kX0 ? 0 : at + Lds::kStage;
                to = to + Lds::kStage == Lds::kX0 ? 0 : to + Lds::kStage;
            }
            if (active) {
                l = half_sum(l);
                if (hh == 0) {
                    s_l[kh][rg * 32 + col] = l;
                    if (kh == 0) s_m[rg * 32 + col] = mx;
                }
            }
            __syncthreads();
        }

        // dimensions 32 (w CB + s) + 8 g + 4 hh + 0..3 of row 32 r + col
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            const int lr = r * 32 + col, row = m * RB + lr;
            const bool in = row < rows;
            const float l = in ? s_l[0][lr] + s_l[1][lr] : 1.f;
            if (whole) {
                if (row >= p.N * p.H) continue;
                const int node = row / p.H;
                const float inv = 1.f / l;
                uint8_t* const dst = p.out + units(b, p.os[0], node, p.os[1]) + units(row - node * p.H, p.os[2]);
#pragma unroll
                for (int s = 0; s < CB; ++s)
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const int d = 32 * (w * CB + s) + 2 * i + 4 * hh;
                        const v16f& y = o[r][s];
                        if (d < p.dv)  // an absent node's row is zero
                            *reinterpret_cast<v4s*>(dst + 2 * d) =
                                in ? pack4<DT>(y[i] * inv, y[i + 1] * inv, y[i + 2] * inv, y[i + 3] * inv)
                                   : v4s{0, 0, 0, 0};
                    }
            } else if (in) {
                float* const rec = p.part + ((static_cast<int64_t>(c) * 2 + (f == f0 ? 0 : 1)) * p.MT + m) * kRec;
#pragma unroll
                for (int s = 0; s < CB; ++s)
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const int d = 32 * (w * CB + s) + 2 * i + 4 * hh;
                        const v16f& y = o[r][s];
                        if (d < p.dv)
                            *reinterpret_cast<float4*>(rec + lr * DV + d) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                    }
                if (hh == 0 && w == 0) {
                    rec[RB * DV + lr] = s_m[lr];
                    rec[RB * DV + RB + lr] = l;
                }
            }
        }
        __syncthreads();  // the stages and sums are free again
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
// each, and the teams share the row's parts.
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
    if (rows == 32) return attn_one<DT, DK, DV, 32>(p, st, ev);
    if (rows == 64) return attn_one<DT, DK, DV, 64>(p, st, ev);
    return attn_one<DT, DK, DV, 128>(p, st, ev);
}

template <int DT, int DV>
hipError_t join_one(const LatentParams& p, const LatentShape& s, hipStream_t st, const LaunchEvents& ev) {
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
