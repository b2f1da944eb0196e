// gfx950 kernels of products per head and of attention for prompts on latent
// rows, with keys and values expanded per head.
//
// For head h, row s of a sequence and query token i at position p_i,
//
//   k_s = (w_k c_s, e_s),  v_s = w_v c_s,  c_s the row's first R elements, e_s the rest,
//   o_i = sum_{s <= p_i} 2^(x_s - m) v_s / sum_{s <= p_i} 2^(x_s - m),  x_s = scale log2(e) q_i.k_s.
//
//   k_prompt_plan    the sequences' places in one line of rows, and in one of query tiles;
//   k_prompt_expand  keys and values of every head for every row of the line, and again
//                    the values of rows whose largest one float16 does not hold well;
//   k_prompt_attn    128 queries of one head against 64 keys at a time.
//
// Expanding costs latent / (dim_k + dim_p + dim_v) as much again per query and key as
// attending, once per row; attending on the rows themselves would cost 3.4 times the
// products per query (latent 512, dim_k 128, dim_p 64, dim_v 128).  Four prompts of at
// most 4096 tokens, 32 heads: 140 us expanding (92 GFLOP and 180 MB of results), 420 us
// attending (316 GFLOP, 750 TFLOP/s); the softmax between the two products (37 % of a
// SIMD's cycles) does not overlap with them (40 %) as much as two workgroups a CU
// would allow.
//
// Keys are rounded to the input type, as their queries are in it.  Values and
// weights meet in float16 whatever the input type: with both in bfloat16 the outputs'
// error was 1.65 times that of the output's own rounding, with float16 1.18 times.
// float16 ends at 2^16 and its full precision at 2^-14, so a row whose values are very
// large or very small has a power of two of its own (per head): v = u 2^(e - 4), with
// e = 0 where the largest lies in [2^-14, 2^11).  Its weight is multiplied by 2^e,
//
//   o = sum_s 2^(x_s + e_s - r) u_s,   l = sum_s 2^(x_s - m),
//
// with a reference r of the products' own: what a token sees decides its r, and no row
// that it does not see can push its values out of float16's range.

#include "sv_attn.h"
#include "sv_latent.h"

namespace sv {
namespace {

// ---- products: out[t, m] = sum_k x[t, k] w[m, k], 128 outputs m by TT tokens a
// workgroup, 64 of k at a time.
//
// W rows are the matrix instruction's A operand and token rows its B operand,
// both read 16 bytes a lane from LDS, where the eight chunks of a row's 64
// elements are XORed with half the row number: a read takes 16 lanes at a time
// (0-3, 12-15, 20-23, 24-27 and so on) over 64 banks, rows alternate between two
// halves of them, and these lanes' even rows have the eight halves 0-7.  A null token
// row counts as zeros.
template <int TM, int TT>
struct Tile {
    static constexpr int kWaves = TM == 256 ? 8 : 4, kThreads = 64 * kWaves;
    static constexpr int kXAt = TM * 128, kStage = (TM + TT) * 128;
    static constexpr int WM = TT == 32 ? 4 : 2;                                   // waves over outputs
    static constexpr int BM = TM / WM / 32, BT = TT / (kWaves / WM) / 32;         // 32 x 32 blocks of a wave
    static constexpr int kW = TM / 8 / kWaves, kX = TT / 8 / kWaves;              // wide loads of a wave and stage
};

// The chunk that lane `lane` of wide load `idx` of eight rows stages.
__device__ __forceinline__ int product_chunk(int lane, int idx) { return (lane & 7) ^ ((idx & 1) << 2 | lane >> 4); }

template <int DT, class L>
__device__ __forceinline__ void product_tile(uint32_t smem_at, const uint8_t* const* wp, const uint8_t* const* xp,
                                             int K, v16f (*acc)[L::BT]) {
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hh = lane >> 5, col = lane & 31;
    const int wm = w % L::WM, wt = w / L::WM;
    const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&kZero);
    auto stage = [&](int s, uint32_t at) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < L::kW; ++i)
            load_lds(s * 64 + product_chunk(lane, w * L::kW + i) * 8 < K ? wp[i] + s * 128 : zero,
                     smem_at + at + (w * L::kW + i) * 1024);
#pragma unroll
        for (int i = 0; i < L::kX; ++i)
            load_lds(s * 64 + product_chunk(lane, w * L::kX + i) * 8 < K && xp[i] ? xp[i] + s * 128 : zero,
                     smem_at + at + L::kXAt + (w * L::kX + i) * 1024);
    };
    uint32_t a_rd[4], b_rd[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t c = ((2 * k + hh) ^ (col >> 1 & 7)) << 4;
        a_rd[k] = smem_at + (wm * L::BM * 32 + col) * 128 + c;
        b_rd[k] = smem_at + L::kXAt + (wt * L::BT * 32 + col) * 128 + c;
    }
#pragma unroll
    for (int a = 0; a < L::BM; ++a)
#pragma unroll
        for (int b = 0; b < L::BT; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
    const int S = (K + 63) / 64;
    stage(0, 0);
    uint32_t at = 0;
#pragma unroll 1
    for (int s = 0; s < S; ++s) {
        wait_vm<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (s + 1 < S) stage(s + 1, L::kStage - at);
        // the next step's operands are on their way while a step's are multiplied
        v8s a[2][L::BM], b[2][L::BT];
        auto fetch = [&](int k) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < L::BM; ++i) a[k & 1][i] = lds_read(a_rd[k] + at + i * 4096);
#pragma unroll
            for (int i = 0; i < L::BT; ++i) b[k & 1][i] = lds_read(b_rd[k] + at + i * 4096);
            __builtin_amdgcn_sched_barrier(0);
        };
        __builtin_amdgcn_sched_barrier(0);
        fetch(0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k < 3) fetch(k + 1);
#pragma unroll
            for (int i = 0; i < L::BM; ++i)
#pragma unroll
                for (int j = 0; j < L::BT; ++j) acc[i][j] = mfma<DT>(a[k & 1][i], b[k & 1][j], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        at = L::kStage - at;
    }
}

// Results leave through LDS, so that a row's are stored together (16 bytes of a row at a time,
// straight from the registers: 46 us for 42 where 1024 tokens of 128 heads leave the latent
// space).  Where outputs m .. m + 3 of row r lie there: a row's 16 chunks XORed with its number, and a chunk's
// halves with its fifth bit, so that 32 rows' writes meet no bank twice.
template <int TM>
__device__ __forceinline__ int out_at(int r, int m) {
    return r * (2 * TM) + ((m >> 3 ^ (r & 15)) << 4) + ((m >> 2 ^ r >> 4) & 1) * 8;
}

// store(r, m, x): eight outputs from m on, a multiple of 8, of row r.
template <int TM, int TT, class F>
__device__ __forceinline__ void store_rows(const uint8_t* smem, F&& store) {
    constexpr int kRow = TM / 8, kThreads = Tile<TM, TT>::kThreads;  // chunks of a row
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TT * kRow / kThreads; ++i) {
        const int e = i * kThreads + threadIdx.x, r = e / kRow, m = e % kRow * 8;
        const uint4 x = *reinterpret_cast<const uint4*>(smem + (out_at<TM>(r, m) & ~15));
        store(r, m, r & 16 ? make_uint4(x.z, x.w, x.x, x.y) : x);
    }
}

// Neighbouring tasks on one XCD (workgroups go to the eight in turn); -1: none.
__device__ __forceinline__ int64_t task_of(int64_t tasks) {
    const int64_t per = (tasks + 7) / 8, t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    return (blockIdx.x >> 3) < per && t < tasks ? t : -1;
}
inline int64_t grid_of(int64_t tasks) { return (tasks + 7) / 8 * 8; }

template <int DT, int TT>
__global__ __launch_bounds__(kThreads, 2) void k_product(ProductParams p) {
    using L = Tile<128, TT>;
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t smem_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) uint8_t*)smem));
    const int mt = (p.M + 127) / 128, tt = (p.T + TT - 1) / TT;
    const int64_t task = task_of(static_cast<int64_t>(mt) * tt * p.H);
    if (task < 0) return;
    const int h = static_cast<int>(task / (mt * static_cast<int64_t>(tt)));
    const int in_head = static_cast<int>(task - h * (mt * static_cast<int64_t>(tt)));
    const int t0 = in_head / mt * TT, m0 = in_head % mt * 128;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hh = lane >> 5, col = lane & 31, r8 = lane >> 3;
    const uint8_t *wp[L::kW], *xp[L::kX];
#pragma unroll
    for (int i = 0; i < L::kW; ++i)
        wp[i] = p.w + 16 * (h * p.ws[0] + min(m0 + (w * L::kW + i) * 8 + r8, p.M - 1) * p.ws[1] +
                            product_chunk(lane, w * L::kW + i));
#pragma unroll
    for (int i = 0; i < L::kX; ++i)
        xp[i] = p.x + 16 * (min(t0 + (w * L::kX + i) * 8 + r8, p.T - 1) * p.xs[0] + h * p.xs[1] +
                            product_chunk(lane, w * L::kX + i));
    v16f acc[L::BM][L::BT];
    product_tile<DT, L>(smem_at, wp, xp, p.K, acc);
    const int wm = w % L::WM, wt = w / L::WM;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < L::BT; ++b)
#pragma unroll
        for (int a = 0; a < L::BM; ++a)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<v4s*>(smem + out_at<128>((wt * L::BT + b) * 32 + col, (wm * L::BM + a) * 32 + 2 * i + 4 * hh)) =
                    pack4<DT>(acc[a][b][i], acc[a][b][i + 1], acc[a][b][i + 2], acc[a][b][i + 3]);
    store_rows<128, TT>(smem, [&](int r, int m, uint4 x) {
        if (t0 + r < p.T && m0 + m < p.M)
            *reinterpret_cast<uint4*>(p.out + 16 * ((t0 + r) * p.os[0] + h * p.os[1]) + 2 * (m0 + m)) = x;
    });
}

// ---- prompts

__device__ __forceinline__ int clamp_len(const PromptParams& p, int len) {
    const int64_t cap = static_cast<int64_t>(p.width) << p.ps_shift;
    return len < 0 ? 0 : len > cap ? static_cast<int>(cap) : len;
}

// Values are stored times 2^kLift 2^-e: in the middle of float16's range, the size of a
// row's largest one in [2^kLow, 2^kHigh) with e = 0, else brought to 2^14..2^15.
constexpr int kLift = 4, kLow = -14, kHigh = 11;
constexpr int kNone = -32768;  // the exponent of rows without any value but zeros: their weights count for nothing

// e of row r of the line, from the parts of head h's values.
__device__ __forceinline__ int power_of(const PromptParams& p, int h, int r) {
    const int parts = (h * p.dv + p.dv - 1) / p.part - h * p.dv / p.part + 1;
    int top = kNone;
    for (int i = 0; i < parts; ++i)
        top = max(top, static_cast<int>(p.sizes[(static_cast<int64_t>(h) * kSizeParts + i) * p.rows + r]));
    if (top == kNone) return p.there[r] ? kNone : 0;  // nobody sees a row whose page does not exist
    return top >= kLow && top < kHigh ? 0 : top - (kHigh - 1);
}

// The last i in [0, n) with at[i] <= x, for rising at.
__device__ __forceinline__ int last_at(const int64_t* at, int n, int64_t x) {
    int lo = 0;
    for (int hi = n; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// A sequence's queries: rows [first, first + n) of q; n is 0 where the bounds do not rise within [0, T].
struct Queries {
    int first, n;
};
__device__ __forceinline__ Queries queries_of(const PromptParams& p, int b) {
    const int s = p.q_start[b], e = p.q_start[b + 1];
    return s >= 0 && e > s && e <= p.T ? Queries{s, e - s} : Queries{0, 0};
}

__global__ __launch_bounds__(1024) void k_prompt_plan(PromptParams p) {
    __shared__ int64_t s_row[16], s_tile[16];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    int64_t row0 = 0, tile0 = 0;
    for (int base = 0; base < p.B; base += 1024) {
        const int b = base + tid;
        int64_t rows = 0, tiles = 0;
        if (b < p.B) {
            rows = clamp_len(p, p.len[b]);
            tiles = (queries_of(p, b).n + kPromptRows - 1) / kPromptRows;
        }
        int64_t r = rows, t = tiles;
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t ru = __shfl_up(static_cast<long long>(r), o), tu = __shfl_up(static_cast<long long>(t), o);
            if (lane >= o) {
                r += ru;
                t += tu;
            }
        }
        if (lane == 63) {
            s_row[w] = r;
            s_tile[w] = t;
        }
        __syncthreads();
        int64_t ra = 0, ta = 0;
        for (int i = 0; i < 16; ++i) {
            if (i < w) {
                r += s_row[i];
                t += s_tile[i];
            }
            ra += s_row[i];
            ta += s_tile[i];
        }
        if (b < p.B) {
            p.plan[b] = row0 + r - rows;
            p.plan[p.B + 1 + b] = tile0 + t - tiles;
        }
        row0 += ra;
        tile0 += ta;
        __syncthreads();
    }
    if (tid == 0) {
        p.plan[p.B] = row0;
        p.plan[2 * p.B + 1] = tile0;
        *p.odd = 0;
    }
}

// Keys and values of TT rows of the line: a product with the rows gathered from
// their pages.  The first output tile's workgroups also bring the rows' second
// parts into the line.  AGAIN: the rows' powers of two are found from the sizes that the
// first launch left, and values of tiles where one is not 1 are made and stored again.
template <int DT, int TT, bool AGAIN>
__global__ __launch_bounds__(TT == 256 ? 512 : 256, 2) void k_prompt_expand(PromptParams p) {
    using L = Tile<TT, TT>;
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t smem_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) uint8_t*)smem));
    const int mk = p.H * p.dn, mv = p.H * p.dv;
    const int tk = AGAIN ? 0 : (mk + TT - 1) / TT, tv = (mv + TT - 1) / TT, tr = (p.rows + TT - 1) / TT;
    const int64_t task = task_of(static_cast<int64_t>(tk + tv) * tr);
    if (task < 0) return;
    // 1024 rows against all outputs, then the next: the workgroups that an XCD has at a time share
    // about that many rows and 1024 outputs' weights, which its L2 holds
    constexpr int kGroup = 1024 / TT;
    const int rg = static_cast<int>(task / (kGroup * (tk + tv)));
    const int in_rg = static_cast<int>(task - rg * static_cast<int64_t>(kGroup) * (tk + tv));
    const int wide = min(kGroup, tr - kGroup * rg), mt = in_rg / wide, r0 = (kGroup * rg + in_rg - mt * wide) * TT;
    const int64_t total = p.plan[p.B];
    if (r0 >= total) return;
    if (AGAIN) {
        const int h0 = mt * TT / p.dv, heads = min(mt * TT + TT - 1, mv - 1) / p.dv - h0 + 1;
        int found = 0;  // bit 0: a power that is not 1; 1: one that changes values
        for (int i = threadIdx.x; i < heads * TT; i += L::kThreads) {
            const int h = h0 + i / TT, r = r0 + i % TT;
            if (r >= total || r >= p.rows) continue;
            const int e = power_of(p, h, r);
            if (h * p.dv >= mt * TT) p.power[static_cast<int64_t>(h) * p.rows + r] = static_cast<int16_t>(e);
            found |= e == 0 ? 0 : e == kNone ? 1 : 3;
        }
        if (__any(found) && (threadIdx.x & 63) == 0 &&
            !(__hip_atomic_load(p.odd, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) & 4))
            atomicOr(p.odd, 4);
        if (!__syncthreads_or(found & 2)) return;
    }
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hh = lane >> 5, col = lane & 31, r8 = lane >> 3;
    const bool values = AGAIN || mt >= tk;
    const int m0 = (values ? mt - tk : mt) * TT, M = values ? mv : mk, per = values ? p.dv : p.dn;
    const uint8_t* const wt0 = values ? p.wv : p.wk;
    const int64_t* const wst = values ? p.wvs : p.wks;
    // the row of the line, null where its page does not exist
    auto row_of = [&](int r) -> const uint8_t* {
        if (r >= total) return nullptr;
        const int b = last_at(p.plan, p.B, r);
        const int j = r - static_cast<int>(p.plan[b]);
        const int pg = p.table[b * p.table_stride + (j >> p.ps_shift)];
        if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(p.pages)) return nullptr;
        return p.kc + 16 * (pg * p.kcs[0] + (j & ((1 << p.ps_shift) - 1)) * p.kcs[1]);
    };
    const uint8_t *wp[L::kW], *xp[L::kX];
#pragma unroll
    for (int i = 0; i < L::kX; ++i) {
        const uint8_t* const x = row_of(r0 + (w * L::kX + i) * 8 + r8);
        xp[i] = x ? x + 16 * product_chunk(lane, w * L::kX + i) : nullptr;
    }
#pragma unroll
    for (int i = 0; i < L::kW; ++i) {
        const int m = min(m0 + (w * L::kW + i) * 8 + r8, M - 1), h = m / per;
        wp[i] = wt0 + 16 * (h * wst[0] + (m - h * per) * wst[1] + product_chunk(lane, w * L::kW + i));
    }
    if (!AGAIN && mt == 0) {
        for (int r = threadIdx.x >> 3; r < TT && r0 + r < total && r0 + r < p.rows; r += L::kThreads / 8) {
            const uint8_t* const x = row_of(r0 + r);
            for (int c = lane & 7; c < p.dr / 8; c += 8)
                *reinterpret_cast<uint4*>(p.pe + (static_cast<int64_t>(r0 + r) * p.dr + 8 * c) * 2) =
                    x ? *reinterpret_cast<const uint4*>(x + 2 * p.R + 16 * c) : make_uint4(0, 0, 0, 0);
            if ((lane & 7) == 0) {
                p.there[r0 + r] = x != nullptr;
                if (!x) atomicOr(p.odd, 2);
            }
        }
    }
    v16f acc[L::BM][L::BT];
    product_tile<DT, L>(smem_at, wp, xp, p.R, acc);
    const int wm = w % L::WM, wt = w / L::WM;
    auto store = [&](uint8_t* to) {
        store_rows<TT, TT>(smem, [&](int r, int m, uint4 x) {
            const int h = (m0 + m) / per;
            if (r0 + r < total && r0 + r < p.rows && m0 + m < M)
                *reinterpret_cast<uint4*>(to + 2 * ((static_cast<int64_t>(h) * p.rows + r0 + r) * per + m0 + m - h * per)) = x;
        });
    };
    __syncthreads();
    if (!values) {
#pragma unroll
        for (int b = 0; b < L::BT; ++b)
#pragma unroll
            for (int a = 0; a < L::BM; ++a)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<v4s*>(smem + out_at<TT>((wt * L::BT + b) * 32 + col,
                                                          (wm * L::BM + a) * 32 + 2 * i + 4 * hh)) =
                        pack4<DT>(acc[a][b][i], acc[a][b][i + 1], acc[a][b][i + 2], acc[a][b][i + 3]);
        store(p.k);
        return;
    }
    // a wave's eight neighbouring outputs are of one head
    uint32_t most[L::BT] = {};
    int of = -1;
    bool odd = false;
    const int part = (m0 + wm * L::BM * 32) / (L::BM * 32);  // the wave's, of all heads' values
    auto tell = [&] {
#pragma unroll
        for (int b = 0; b < L::BT; ++b) {
            const auto both = __builtin_amdgcn_permlane32_swap(most[b], most[b], false, false);
            const uint32_t top = max(both[0], both[1]);
            const int r = r0 + (wt * L::BT + b) * 32 + col;
            if (hh == 0 && r < total && r < p.rows)
                p.sizes[(static_cast<int64_t>(of) * kSizeParts + part - of * p.dv / (L::BM * 32)) * p.rows + r] =
                    static_cast<int16_t>(top == 0 ? kNone : static_cast<int>(top >> 23) - 127);  // denormal: -127
            most[b] = 0;
        }
    };
#pragma unroll
    for (int a = 0; a < L::BM; ++a)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int m8 = m0 + (wm * L::BM + a) * 32 + 2 * i, h = m8 / per;
            if (m8 >= M) continue;
            if (!AGAIN && h != of) {
                if (of >= 0) tell();
                of = h;
            }
#pragma unroll
            for (int b = 0; b < L::BT; ++b) {
                const int r = r0 + (wt * L::BT + b) * 32 + col;
                if (r >= total || r >= p.rows) continue;
                const int up = AGAIN ? kLift - power_of(p, h, r) : kLift;
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[j] = AGAIN ? ldexpf(acc[a][b][i + j], up) : acc[a][b][i + j] * (1 << kLift);
                    const uint32_t size = __float_as_uint(acc[a][b][i + j]) & 0x7FFFFFFFu;
                    if (size >= 0x7F800000u)
                        odd = true;
                    else
                        most[b] = max(most[b], size);
                }
                *reinterpret_cast<v4s*>(smem + out_at<TT>(r - r0, m8 - m0 + 4 * hh)) = pack4<kDTypeF16>(y[0], y[1], y[2], y[3]);
            }
        }
    if (!AGAIN) {
        if (of >= 0) tell();
        if (odd) atomicOr(p.odd, 1);
    }
    store(p.v);
}

// Where chunk c of row r of a tile lies in LDS, rows of PITCH bytes: c XORed with this, so
// that the 16 lanes of a wide read (rows 0-3, 12-15, 20-23, 24-27 and so on) meet no bank twice.
template <int PITCH>
__device__ __forceinline__ int row_swizzle(int r) {
    return PITCH == 256 ? r & 15 : PITCH == 128 ? r >> 1 & 7 : r >> 2 & 3;
}

// A part of a tile's rows, W elements each: staging and the operands' addresses.
template <int W>
struct Rows {
    static constexpr int kPitch = 2 * W, kChunks = W / 8;
    static constexpr int kLoads = 64 * kChunks / 64 / kWaves;                      // wide loads of a wave
    static constexpr int kAddr = kPitch == 256 ? 8 : kPitch == 128 ? 4 : 2;         // addresses of the operands
    static_assert(kPitch == 256 || kPitch == 192 || kPitch == 128 || kPitch == 64, "layout");
};

// 128 queries of one head (32 a wave) against 64 keys at a time, in a ring of RING
// tiles: with two, two workgroups fill a CU's LDS and take turns at its matrix
// units.  Where there are not that many, a workgroup has two GROUPS of four waves
// that take the tiles in turn, each with a ring of its own, and add up at the end.
// A tile's operands are read from LDS some steps before they are needed.
//
// POWERS: some rows of the line have a power of two of their own.  The products'
// reference is then mx + ko, with ko = 0 until a query sees such a row; ko is kept
// apart, as scores may be so large that float32 holds no power of two beside them.
// The same arithmetic as without for queries that see none, and a loop of its own: with
// one for both, the registers of the usual case would be spilled.
template <int DT, int DN, int DR, int DV, int RING, int GROUPS, bool POWERS>
__device__ __forceinline__ void prompt_attend(const PromptParams& p) {
    using KN = Rows<DN>;
    using KR = Rows<DR>;
    using VR = Rows<DV>;
    constexpr int TK = 64;
    constexpr int kRAt = TK * KN::kPitch, kVAt = kRAt + TK * KR::kPitch, kStage = kVAt + TK * VR::kPitch;
    constexpr int SN = DN / 16, SR = DR / 16, NQ = SN + SR, ND = DV / 32;
    // the transposing read takes four rows at four chunks
    auto v_swizzle = [](int r) { return VR::kPitch == 256 ? (r & 3) << 2 : (r >> 1 & 1) << 2; };
    static_assert(VR::kPitch == 256 || VR::kPitch == 128, "layout");
    extern __shared__ __align__(16) uint8_t smem[];  // nothing beside it: two workgroups fill a CU
    const uint32_t smem_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) uint8_t*)smem));
    const int tid = threadIdx.x, lane = tid & 63, w8 = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w = w8 & 3, group = GROUPS > 1 ? w8 >> 2 : 0;
    const int hh = lane >> 5, col = lane & 31;
    const int64_t tiles = p.plan[2 * p.B + 1], task = task_of(tiles * p.H);
    if (task < 0) return;
    const int h = static_cast<int>(task / tiles);
    const int64_t tile = tiles - 1 - (task - h * tiles);  // long ones first
    const int b = last_at(p.plan + p.B + 1, p.B, tile);
    const int i0 = static_cast<int>(tile - p.plan[p.B + 1 + b]) * kPromptRows;
    const Queries qs = queries_of(p, b);
    const int64_t row0 = p.plan[b];
    const int len = clamp_len(p, p.len[b]);
    const int mine = i0 + w * 32 + col;  // the lane's query
    const bool in = mine < qs.n;
    uint8_t* const dst = p.out + 16 * ((qs.first + mine) * p.os[0] + h * p.os[1]);
    if (len > 0 && row0 + len > p.rows) {  // the line is too short for this sequence
        if (in && !group)
            for (int d = 4 * hh; d < p.dv; d += 8)
                *reinterpret_cast<v4s*>(dst + 2 * d) = pack4<DT>(NAN, NAN, NAN, NAN);
        return;
    }
    const int shift = len - qs.n;  // position of query 0
    const int pos = mine + shift;
    const int low = i0 + w * 32 + shift;  // first and last position of the wave
    const int high = i0 + w * 32 < qs.n ? min(i0 + w * 32 + 31, qs.n - 1) + shift : -1;
    const int last = min(i0 + kPromptRows, qs.n) - 1 + shift;  // of the workgroup
    const int all = last < 0 ? 0 : last / TK + 1, steps = (all + GROUPS - 1) / GROUPS;
    const int T = (all + GROUPS - 1 - group) / GROUPS;  // this group's tiles: group, group + GROUPS, ...
    const uint32_t ring = group * RING * kStage;

    // Staging: chunk e = 64 i + lane of a part of the tile is chunk e % kChunks of row e / kChunks; `off` is
    // where it comes from, relative to the tile's first row.  Dimensions past the head's are zeros.
    uint32_t off_n[KN::kLoads], off_r[KR::kLoads], off_v[VR::kLoads], pad = 0;
    constexpr int kPer = KN::kLoads + KR::kLoads + VR::kLoads;
    const bool padded = p.dn < DN || p.dr < DR || p.dv < DV;
    auto row_n = [&](int i) { return ((w * KN::kLoads + i) * 64 + lane) / KN::kChunks; };
    auto row_r = [&](int i) { return ((w * KR::kLoads + i) * 64 + lane) / KR::kChunks; };
    auto row_v = [&](int i) { return ((w * VR::kLoads + i) * 64 + lane) / VR::kChunks; };
#pragma unroll
    for (int i = 0; i < KN::kLoads; ++i) {
        const int r = row_n(i), c = ((w * KN::kLoads + i) * 64 + lane) % KN::kChunks ^ row_swizzle<KN::kPitch>(r);
        off_n[i] = 2 * (r * p.dn + 8 * c);
        if (8 * c >= p.dn) pad |= 1u << i;
    }
#pragma unroll
    for (int i = 0; i < KR::kLoads; ++i) {
        const int r = row_r(i), c = ((w * KR::kLoads + i) * 64 + lane) % KR::kChunks ^ row_swizzle<KR::kPitch>(r);
        off_r[i] = 2 * (r * p.dr + 8 * c);
        if (8 * c >= p.dr) pad |= 1u << (8 + i);
    }
#pragma unroll
    for (int i = 0; i < VR::kLoads; ++i) {
        const int r = row_v(i), c = ((w * VR::kLoads + i) * 64 + lane) % VR::kChunks ^ v_swizzle(r);
        off_v[i] = 2 * (r * p.dv + 8 * c);
        if (8 * c >= p.dv) pad |= 1u << (16 + i);
    }
    const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&kZero);
    const uint8_t* kb_n = p.k + 2 * (static_cast<int64_t>(h) * p.rows + row0 + group * TK) * p.dn;
    const uint8_t* kb_r = p.pe + 2 * (row0 + group * TK) * p.dr;
    const uint8_t* kb_v = p.v + 2 * (static_cast<int64_t>(h) * p.rows + row0 + group * TK) * p.dv;
    auto stage = [&](int s, uint32_t at) __attribute__((always_inline)) {
        const int t = s * GROUPS + group;
        const uint32_t to = smem_at + ring + at;
        const uint32_t to_n = to + w * KN::kLoads * 1024, to_r = to + kRAt + w * KR::kLoads * 1024,
                       to_v = to + kVAt + w * VR::kLoads * 1024;
        if ((t + 1) * TK <= len && !padded) {
#pragma unroll
            for (int i = 0; i < KN::kLoads; ++i) load_lds(kb_n, off_n[i], to_n + i * 1024);
#pragma unroll
            for (int i = 0; i < KR::kLoads; ++i) load_lds(kb_r, off_r[i], to_r + i * 1024);
#pragma unroll
            for (int i = 0; i < VR::kLoads; ++i) load_lds(kb_v, off_v[i], to_v + i * 1024);
        } else {  // rows past the sequence are zeros, too
            const int left = len - t * TK;
#pragma unroll
            for (int i = 0; i < KN::kLoads; ++i)
                load_lds(!(pad >> i & 1) && row_n(i) < left ? kb_n + off_n[i] : zero, to_n + i * 1024);
#pragma unroll
            for (int i = 0; i < KR::kLoads; ++i)
                load_lds(!(pad >> (8 + i) & 1) && row_r(i) < left ? kb_r + off_r[i] : zero, to_r + i * 1024);
#pragma unroll
            for (int i = 0; i < VR::kLoads; ++i)
                load_lds(!(pad >> (16 + i) & 1) && row_v(i) < left ? kb_v + off_v[i] : zero, to_v + i * 1024);
        }
        kb_n += GROUPS * 2 * TK * p.dn;
        kb_r += GROUPS * 2 * TK * p.dr;
        kb_v += GROUPS * 2 * TK * p.dv;
    };
    // lane j: whether row kb + j exists
    auto there = [&](int kb) {
        const int r = kb + lane;
        return r < len ? p.there[row0 + r] : 0;
    };
    // operands: step s of a key's first part is at rd[s % kAddr], s / kAddr times 32 kAddr bytes on
    uint32_t n_rd[KN::kAddr], r_rd[KR::kAddr], v_rd[ND];
#pragma unroll
    for (int s = 0; s < KN::kAddr; ++s)
        n_rd[s] = smem_at + ring + col * KN::kPitch + (((2 * s + hh) ^ row_swizzle<KN::kPitch>(col)) << 4);
#pragma unroll
    for (int s = 0; s < KR::kAddr; ++s)
        r_rd[s] = smem_at + ring + kRAt + col * KR::kPitch + (((2 * s + hh) ^ row_swizzle<KR::kPitch>(col)) << 4);
    {
        const int vrow = 4 * hh + ((lane & 15) >> 2);
        const int c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
            v_rd[dt] = smem_at + ring + kVAt + vrow * VR::kPitch + (((4 * dt + c) ^ v_swizzle(vrow)) << 4) + (lane & 1) * 8;
    }
    v8s q[NQ];
    {
        const uint8_t* const src = p.q + 16 * ((qs.first + (in ? mine : 0)) * p.qs[0] + h * p.qs[1]);
#pragma unroll
        for (int s = 0; s < NQ; ++s) {
            const int d = s * 16 + hh * 8;
            const int from = d < DN ? (d < p.dn ? d : -1) : (d - DN < p.dr ? d - DN + p.dn : -1);
            v8s z = {0, 0, 0, 0, 0, 0, 0, 0};
            if (in && from >= 0) z = *reinterpret_cast<const v8s*>(src + 2 * from);
            q[s] = p.flip ? z ^ static_cast<short>(0x8000) : z;
        }
    }
    float mx = -INFINITY, l = 0.f, ko = 0.f;
    bool apart = false;  // the query has seen a row with a power of its own
    v16f o[ND];
#pragma unroll
    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;
    const float scale2 = p.scale2;
    constexpr float kRaise = kUp<kDTypeF16> + 8.f;
    const bool odd = *p.odd & 1, gaps = *p.odd & 2;
    constexpr int kAhead = RING - 1;
#pragma unroll
    for (int t = 0; t < kAhead; ++t)
        if (t < T) stage(t, t * kStage);
    uint32_t at = 0, to = kAhead * kStage;
#pragma unroll 1
    for (int t = 0; t < steps; ++t) {
        // this wave's loads of tile t have landed (later tiles' stay under way); with the barrier
        // everyone's, and everyone is done with the tile before it
        if (t + kAhead <= T)
            wait_vm<(kAhead - 1) * kPer>();
        else
            wait_vm<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const int kb = (t * GROUPS + group) * TK;
        const uint64_t okm = gaps ? __ballot(there(kb) != 0) : ~0ull;
        const int power = POWERS && kb + lane < len
                              ? p.power[static_cast<int64_t>(h) * p.rows + row0 + kb + lane] : 0;  // of row kb + lane
        if (t + kAhead < T) stage(t + kAhead, to);
        uint64_t nf = 0;
        if (odd && ((t + 1) * GROUPS) * TK - 1 > i0 + shift) {
            // infinities or NaN are about, and some of the queries do not see all of the tile: these
            // values go out of it (0 times them would reach those queries), and who sees the row gets a
            // score of NaN.  Every wave looks at all rows; then each clears a part.
            unsigned long long rows = 0;
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
                for (int i = pass ? w : 0; i < VR::kLoads * kWaves; i += pass ? kWaves : 1) {
                    v8s* const e = reinterpret_cast<v8s*>(smem + ring + at + kVAt + i * 1024 + lane * 16);
                    const uint4 u = __builtin_bit_cast(uint4, *e);
                    if (nonfinite2<kDTypeF16>(u.x) || nonfinite2<kDTypeF16>(u.y) || nonfinite2<kDTypeF16>(u.z) ||
                        nonfinite2<kDTypeF16>(u.w)) {
                        if (pass)
                            *e = v8s{0, 0, 0, 0, 0, 0, 0, 0};
                        else
                            rows |= 1ull << ((i * 64 + lane) / VR::kChunks);
                    }
                }
                __syncthreads();
            }
            for (int s = 32; s; s >>= 1) rows |= __shfl_xor(rows, s);
            nf = rows;
        }
        if (kb <= high) {
            v16f x[2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int i = 0; i < 16; ++i) x[ks][i] = 0.f;
            // four steps' operands at a time, those of the next two parts on their way meanwhile
            constexpr int kPart = 4, kParts = 2 * NQ / kPart;
            static_assert(kPart * kParts == 2 * NQ, "steps");
            v8s kf[3][kPart];
            auto fetch = [&](int part) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < kPart; ++j) {
                    const int ks = (part * kPart + j) / NQ, s = (part * kPart + j) % NQ;
                    kf[part % 3][j] =
                        s < SN ? lds_read(n_rd[s % KN::kAddr] + at + ks * 32 * KN::kPitch + s / KN::kAddr * (32 * KN::kAddr))
                               : lds_read(r_rd[(s - SN) % KR::kAddr] + at + ks * 32 * KR::kPitch +
                                          (s - SN) / KR::kAddr * (32 * KR::kAddr));
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            __builtin_amdgcn_sched_barrier(0);
            fetch(0);
            fetch(1);
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                if (part + 2 < kParts) fetch(part + 2);
#pragma unroll
                for (int j = 0; j < kPart; ++j) {
                    const int ks = (part * kPart + j) / NQ, s = (part * kPart + j) % NQ;
                    x[ks] = mfma<DT>(kf[part % 3][j], q[s], x[ks]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            // values of 16 keys, those of the next 16 on their way meanwhile
            v8s vf[2][ND];
            auto values = [&](int step) __attribute__((always_inline)) {
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) {
                    const uint32_t a = v_rd[dt] + at + step * 16 * VR::kPitch;
                    vf[step & 1][dt] =
                        __builtin_shufflevector(lds_read_tr(a), lds_read_tr(a + 8 * VR::kPitch), 0, 1, 2, 3, 4, 5, 6, 7);
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            values(0);
            float top = -INFINITY;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if (kb + TK - 1 > low || okm != ~0ull || nf) {
                    const int key0 = kb + 32 * ks;
                    const uint32_t see = (static_cast<uint32_t>(okm >> (32 * ks)) & ~bits_from(pos - key0 + 1)) >> 4 * hh;
                    const uint32_t bad = static_cast<uint32_t>(nf >> (32 * ks)) >> 4 * hh;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t bit = 1u << (8 * (i >> 2) + (i & 3));
                        x[ks][i] = see & bit ? bad & bit ? __builtin_nanf("") : x[ks][i] : -INFINITY;
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, x[ks][i]);
            }
            top = scaled(half_max(top), scale2);
            float by = scale2, ref = 0.f, sum = l;  // the exponents of the weights are x by - ref
            bool whole = true;                      // the weights are those of the sum, too
            if (POWERS) {
                const uint64_t own = __ballot(power != 0);
                if (own) {
                    const uint32_t lo = static_cast<uint32_t>(own & okm) & ~bits_from(pos - kb + 1);
                    const uint32_t hi = static_cast<uint32_t>((own & okm) >> 32) & ~bits_from(pos - kb - 31);
                    apart |= (lo | hi) != 0;
                }
                if (__any(apart)) {
                    whole = false;
                    by = 1.f;
                    const float was = mx;
                    if (top - mx > kRaise) mx = fmaxf(mx, top - kUp<kDTypeF16>);
                    const float m = mx == -INFINITY ? 0.f : mx, a = shift_of(was, mx);
                    sum *= a;
                    float high = -INFINITY;
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float y = less(scaled(x[ks][i], scale2), m);
                            sum += __builtin_amdgcn_exp2f(y);
                            x[ks][i] = y + static_cast<float>(__shfl(power, 32 * ks + 8 * (i >> 2) + (i & 3) + 4 * hh));
                            high = fmaxf(high, x[ks][i]);
                        }
                    high = half_max(high);
                    float f = a;  // what the products so far are multiplied by
                    if (apart) {
                        const float k = was == -INFINITY ? -INFINITY : was == mx ? ko : ko + (was - mx);
                        ko = high - k > kRaise ? fmaxf(k, high - kUp<kDTypeF16>) : k;
                        f = shift_of(k, ko);
                        ref = ko == -INFINITY ? 0.f : ko;
                    }
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[dt][i] *= f;
                }
            }
            if (whole) {
                if (__any(top - mx > kRaise)) {
                    const float was = mx;
                    if (top - mx > kRaise) mx = fmaxf(mx, top - kUp<kDTypeF16>);
                    const float a = shift_of(was, mx);
                    sum *= a;
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[dt][i] *= a;
                }
                ref = mx == -INFINITY ? 0.f : mx;
            }
#pragma unroll
            for (int step = 0; step < 4; ++step) {
                const int ks = step >> 1, t2 = step & 1;
                if (step + 1 < 4) values(step + 1);
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = __builtin_amdgcn_exp2f(less(scaled(x[ks][8 * t2 + i], by), ref));
                    if (!POWERS || whole) sum += y[i];
                }
                const v4s lo = pack4<kDTypeF16>(y[0], y[1], y[2], y[3]), hi = pack4<kDTypeF16>(y[4], y[5], y[6], y[7]);
                const v8s pf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) o[dt] = mfma<kDTypeF16>(vf[step & 1][dt], pf, o[dt]);
            }
            l = sum;
        }
        at = at == kAhead * kStage ? 0 : at + kStage;
        to = to == kAhead * kStage ? 0 : to + kStage;
    }
    if (GROUPS > 1) {
        // the second group's sums through LDS, taken over by the first: 32 queries of each wave by
        // DV values, the reference and the weights' sum, the products' reference
        __syncthreads();
        float* const part = reinterpret_cast<float*>(smem) + w * (16 * ND + 3) * 64 + lane;
        if (group) {
#pragma unroll
            for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(dt * 16 + i) * 64] = o[dt][i];
            part[16 * ND * 64] = mx;
            part[(16 * ND + 1) * 64] = l;
            if (POWERS) part[(16 * ND + 2) * 64] = ko;
        }
        __syncthreads();
        if (group) return;
        const float other = part[16 * ND * 64], top = fmaxf(mx, other);
        float a = shift_of(mx, top), c = shift_of(other, top);
        l = l * a + part[(16 * ND + 1) * 64] * c;
        if (POWERS) {
            const float theirs = part[(16 * ND + 2) * 64];
            const float k = mx == -INFINITY ? -INFINITY : mx == top ? ko : ko + (mx - top);
            const float j = other == -INFINITY ? -INFINITY : other == top ? theirs : theirs + (other - top);
            ko = fmaxf(k, j);
            a = shift_of(k, ko);
            c = shift_of(j, ko);
        }
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[dt][i] = o[dt][i] * a + part[(dt * 16 + i) * 64] * c;
    }
    l = half_sum(l);
    const float inv = l == 0.f ? 0.f : 1.f / l / (1 << kLift);  // a query that sees nothing: zero
    if (!in) return;
    // 2^ko in two steps: the first may leave float32's range where the product does not
    ko = fminf(fmaxf(ko, -1000.f), 1000.f);
    const int up = static_cast<int>(__builtin_rintf(ko));
    const float rest = POWERS ? __builtin_amdgcn_exp2f(ko - up) : 1.f;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int d = 32 * dt + 2 * i + 4 * hh;
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = o[dt][i + j] * inv;
                if (POWERS) y[j] = ldexpf(y[j] * rest, up);
            }
            if (d < p.dv) *reinterpret_cast<v4s*>(dst + 2 * d) = pack4<DT>(y[0], y[1], y[2], y[3]);
        }
}

template <int DT, int DN, int DR, int DV, int RING, int GROUPS>
__global__ __launch_bounds__(GROUPS * kThreads, 2) void k_prompt_attn(PromptParams p) {
    if (*p.odd & 4)
        prompt_attend<DT, DN, DR, DV, RING, GROUPS, true>(p);
    else
        prompt_attend<DT, DN, DR, DV, RING, GROUPS, false>(p);
}

template <int DT, int TT>
hipError_t product_one(const ProductParams& p, hipStream_t st, const LaunchEvents& ev) {
    const int64_t tasks = static_cast<int64_t>((p.M + 127) / 128) * ((p.T + TT - 1) / TT) * p.H;
    hipExtLaunchKernelGGL((k_product<DT, TT>), dim3(static_cast<unsigned>(grid_of(tasks))), dim3(kThreads),
                          2 * Tile<128, TT>::kStage, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

// Tiles of tt outputs by tt rows (again: of the values alone).
int64_t expand_tasks(const PromptParams& p, int tt, bool again) {
    return static_cast<int64_t>((again ? 0 : (p.H * p.dn + tt - 1) / tt) + (p.H * p.dv + tt - 1) / tt) *
           ((p.rows + tt - 1) / tt);
}

template <int DT, int TT, bool AGAIN>
hipError_t expand_one(const PromptParams& p, hipStream_t st, const LaunchEvents& ev) {
    using L = Tile<TT, TT>;
    const int64_t tasks = expand_tasks(p, TT, AGAIN);
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(k_prompt_expand<DT, TT, AGAIN>), 2 * L::kStage);
    if (e != hipSuccess) return e;
    hipExtLaunchKernelGGL((k_prompt_expand<DT, TT, AGAIN>), dim3(static_cast<unsigned>(grid_of(tasks))),
                          dim3(L::kThreads), 2 * L::kStage, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

// The large tile (one workgroup of eight waves a CU) reads and stages half as much per product:
// 1376 of them 140 us for 163 with four times as many small ones, 128 heads on 4096 rows 215 to 235
// for 308; but 294, one round and a bit, 35 us for 32.
template <int DT>
hipError_t expand_tile(const PromptParams& p, bool again, hipStream_t st, const LaunchEvents& ev) {
    const bool large = expand_tasks(p, 256, false) > 2 * p.cus;
    if (again) {
        PromptParams q = p;
        q.part = large ? 128 : 64;
        return expand_one<DT, 128, true>(q, st, ev);
    }
    return large ? expand_one<DT, 256, false>(p, st, ev) : expand_one<DT, 128, false>(p, st, ev);
}

template <int DT, int DN, int DR, int DV, int RING, int GROUPS>
hipError_t prompt_ring(const PromptParams& p, int64_t tasks, hipStream_t st, const LaunchEvents& ev) {
    constexpr int lds = GROUPS * RING * 64 * (DN + DR + DV) * 2;
    static_assert(lds <= 160 << 10 && (GROUPS == 1 || lds >= kWaves * (DV / 2 + 3) * 64 * 4), "LDS");
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(k_prompt_attn<DT, DN, DR, DV, RING, GROUPS>), lds);
    if (e != hipSuccess) return e;
    hipExtLaunchKernelGGL((k_prompt_attn<DT, DN, DR, DV, RING, GROUPS>), dim3(static_cast<unsigned>(grid_of(tasks))),
                          dim3(GROUPS * kThreads), lds, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

template <int DT, int DN, int DR, int DV>
hipError_t prompt_one(const PromptParams& p, hipStream_t st, const LaunchEvents& ev) {
    const int64_t tasks = (p.T / kPromptRows + static_cast<int64_t>(p.B < p.T ? p.B : p.T)) * p.H;  // at most
    // Two groups where there are no more workgroups than CUs: 150 of them 63 us for 83.  With 2600
    // the join at the end and the common barrier cost more than they give (469 us for 430).
    constexpr int kDeep = 2 * 3 * 64 * (DN + DR + DV) * 2 <= (160 << 10) ? 3 : 2;
    return tasks <= p.cus ? prompt_ring<DT, DN, DR, DV, kDeep, 2>(p, tasks, st, ev)
                          : prompt_ring<DT, DN, DR, DV, 2, 1>(p, tasks, st, ev);
}

template <int DT>
hipError_t prompt_dims(const PromptParams& p, hipStream_t st, const LaunchEvents& ev) {
    if (p.dn <= 64 && p.dr <= 64 && p.dv <= 64) return prompt_one<DT, 64, 64, 64>(p, st, ev);
    if (p.dn <= 96 && p.dr <= 32) return prompt_one<DT, 96, 32, 128>(p, st, ev);
    return prompt_one<DT, 128, 64, 128>(p, st, ev);
}

}  // namespace

hipError_t launch_product(const ProductParams& p, int dtype, hipStream_t st, const LaunchEvents& ev) {
    if (dtype == DT_BF16) return p.tt == 32 ? product_one<DT_BF16, 32>(p, st, ev) : product_one<DT_BF16, 128>(p, st, ev);
    return p.tt == 32 ? product_one<kDTypeF16, 32>(p, st, ev) : product_one<kDTypeF16, 128>(p, st, ev);
}

hipError_t launch_prompt_plan(const PromptParams& p, hipStream_t st, const LaunchEvents& ev) {
    hipExtLaunchKernelGGL(k_prompt_plan, dim3(1), dim3(1024), 0, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

hipError_t launch_prompt_expand(const PromptParams& p, int dtype, bool again, hipStream_t st, const LaunchEvents& ev) {
    return dtype == DT_BF16 ? expand_tile<DT_BF16>(p, again, st, ev) : expand_tile<kDTypeF16>(p, again, st, ev);
}

hipError_t launch_prompt_attn(const PromptParams& p, int dtype, hipStream_t st, const LaunchEvents& ev) {
    return dtype == DT_BF16 ? prompt_dims<DT_BF16>(p, st, ev) : prompt_dims<kDTypeF16>(p, st, ev);
}

}  // namespace sv
