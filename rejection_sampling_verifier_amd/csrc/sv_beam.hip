// gfx950 kernels of one step of beam search.
//
// Of sequence b's candidates (beam w, id v) with score
//
//   s(w, v) = score_w + x_wv - log sum_u e^(x_wu)
//
// the W largest, equal ones in the order of the beams, then of logits and ids; a
// finished beam has one candidate, the end token at its own score.
//
//   k_beam_stats   a chunk of a row: its maximum, the sum of its exponentials and
//                  its W largest logits;
//   k_beam_select  a sequence: the rows' logarithms of sums, then the W best.
//
// Within a row the order is that of the logits, exact in any arithmetic.  Between
// rows it depends on the logarithms, which come from float32 exponentials (kBand);
// where two rows' candidates are closer than kBand and that decides, the sequence's
// sums are taken again in float64.  So they are where more than kSelThreads candidates
// reach the selection's bound, with ties or without: see there.
//
// Chunks are cut by id, never by alignment, and sums have a fixed order: equal
// rows give equal sums wherever they lie.
//
// What bounds it: 32 sequences of 8 beams over 128256 float32 ids (131 MB) take 35 us of
// statistics (the reads alone 27, 4.9 TB/s) and 15.5 of selection; one sequence of 4
// beams 4.7 and 9.6, a chain of dependent steps in one workgroup.  Made for few beams:
// one sequence of 12, 16, 24, 32 and 64 takes 29, 81, 1350, 2700 and 8750 us of
// selection, eight of them over 32000 ids 20, 23, 29, 740 and 2300.

#include <hip/hip_ext.h>

#include "sv_beam.h"
#include "sv_device.h"

namespace sv {
namespace {

constexpr uint32_t kLowest = 0x007FFFFFu;  // order key of -inf: such ids are no candidates
constexpr int kListed = 1024;              // candidates a chunk's workgroup ranks at most in one go

// Relative error of an exponential below the row's largest: the argument is taken
// exactly (between bfloat16 numbers with an error of 2^-21 up to 16 below the largest,
// 2^-20 up to 32) and split into its integer and a fraction of two roundings of 2^-25,
// and 2^f has an error of 2^-23: below 2^-20, but for terms further than 32 below,
// which make 2^-39 at most of any sum's error.  The largest is exactly 1, and sums are
// float64 (in float32, eight terms at a time, what the other ids have beside one with
// 1 - 1e-7 of the probability was lost in part or whole).  So a row's logarithm is off
// by 2^-20 of the share that its other ids have; the distance of two rows' candidates
// by twice that at most, and the band is twice as wide again.
constexpr double kBand = 0x1p-18;

// 16 bytes at any element's address.
template <int DT> struct Vec;
template <> struct Vec<DT_F32> { typedef unsigned int T __attribute__((ext_vector_type(4), aligned(4))); };
template <> struct Vec<DT_BF16> { typedef unsigned int T __attribute__((ext_vector_type(4), aligned(2))); };

// Eight logits from id `id0` on, -inf past the end.
template <int DT>
__device__ __forceinline__ void eight(const uint8_t* row, int id0, int V, float* f) {
    constexpr int E = Fmt<DT>::E, VE = Fmt<DT>::VE;
    typedef typename Vec<DT>::T v4u;
    if (id0 + 8 <= V) {
#pragma unroll
        for (int k = 0; k < 8 / VE; ++k) {
            const v4u y = __builtin_nontemporal_load(
                (__attribute__((address_space(1))) const v4u*)(row + static_cast<int64_t>(id0 + k * VE) * E));
            unpack<DT>(make_uint4(y.x, y.y, y.z, y.w), f + k * VE);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = id0 + i < V ? load_elem<DT>(row, id0 + i) : -SV_INF;
    }
}

// e^(x - top) for x <= top (0 below e^-150).
template <int DT>
__device__ __forceinline__ float exp_of(float x, float top) {
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f;  // log2(e)
    const float d = x - top;
    const float n = __builtin_rintf(d * kHi);
    float f = fmaf(d, kLo, fmaf(d, kHi, -n));
    if (DT == DT_F32) {  // what the difference's rounding left (bfloat16: 8 to 13 % of the kernel's time for it)
        const float y = x - d;
        f = fmaf((x - (d + y)) + (y - top), kHi, f);
    }
    return d < -150.f ? 0.f : ldexpf(hw_exp2(f), static_cast<int>(n));
}

// The k-th largest (k from 0) of a wave's values.
__device__ __forceinline__ uint32_t kth_largest(uint32_t x, int k) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int size = 2; size <= 64; size <<= 1)
#pragma unroll
        for (int step = size >> 1; step; step >>= 1) {
            const uint32_t y = __shfl_xor(x, step);
            const bool larger = ((lane & step) == 0) == ((lane & size) == 0);  // this lane keeps the larger one
            x = larger ? max(x, y) : min(x, y);
        }
    return __shfl(x, k);
}

template <int DT, int RUNS>
__global__ __launch_bounds__(kThreads) void k_beam_stats(BeamParams p) {
    __shared__ float s_top[kWaves];
    __shared__ double s_sum[kWaves];
    __shared__ uint32_t s_tau[kWaves];
    __shared__ int s_bad, s_n;
    __shared__ uint64_t s_list[kListed];
    __shared__ unsigned long long s_best[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int r = blockIdx.y, b = r / p.W, chunk = blockIdx.x;
    if (p.scores[r] == -SV_INF || (p.finished && p.finished[r])) return;  // nobody asks
    const uint8_t* const row = p.logits + (b * p.sb + (r - b * p.W) * p.sw) * Fmt<DT>::E;
    const int id0 = chunk * (RUNS * kThreads * 8) + tid * 8;
    if (tid == 0) s_bad = s_n = 0;
    float x[RUNS][8];
#pragma unroll
    for (int k = 0; k < RUNS; ++k) eight<DT>(row, id0 + k * kThreads * 8, p.V, x[k]);
    float top = -SV_INF;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < RUNS; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top = fmaxf(top, x[k][i]);
            bad |= !(x[k][i] < SV_INF);  // NaN or +inf
        }
    const uint32_t most = order_key(top);
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const uint32_t kth = kth_largest(most, p.W - 1);
    if (lane == 0) {
        s_top[w] = top;
        s_tau[w] = kth;
    }
    __syncthreads();
    if (bad) s_bad = 1;
    top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
    // at least W logits of the chunk are no smaller than this (those of one wave)
    const uint32_t tau = max(max(max(s_tau[0], s_tau[1]), max(s_tau[2], s_tau[3])), kLowest + 1);
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum += exp_of<DT>(x[k][i], top);
            const uint32_t key = order_key(x[k][i]);
            if (key >= tau) {
                const int at = atomicAdd(&s_n, 1);
                if (at < kListed)
                    s_list[at] = static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(id0 + k * kThreads * 8 + i);
            }
        }
    }
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) s_sum[w] = sum;
    __syncthreads();
    const int n = s_n;
    uint64_t* const out = p.list + (static_cast<int64_t>(r) * p.chunks + chunk) * p.W;
    int listed = min(n, p.W);
    if (s_bad || top == -SV_INF) {
        listed = 0;
    } else if (n <= kListed) {
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t me = s_list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += s_list[j] > me;
            if (rank < p.W) out[rank] = me;
        }
    } else {  // a long run of equal logits: one after the other
        unsigned long long last = ~0ull;
        for (int i = 0; i < p.W; ++i) {
            unsigned long long best = 0;
#pragma unroll
            for (int k = 0; k < RUNS; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const unsigned long long y = static_cast<uint64_t>(order_key(x[k][j])) << 32 |
                                                 ~static_cast<uint32_t>(id0 + k * kThreads * 8 + j);
                    if (y < last && y > best) best = y;
                }
            for (int o = 32; o; o >>= 1) best = max(best, __shfl_xor(best, o));
            if (lane == 0) s_best[w] = best;
            __syncthreads();
            last = max(max(s_best[0], s_best[1]), max(s_best[2], s_best[3]));
            if (tid == 0) out[i] = last;
            __syncthreads();
        }
    }
    if (tid >= listed && tid < p.W) out[tid] = 0;  // no candidate
    if (tid == 0) {
        const double all = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
        p.rec[static_cast<int64_t>(r) * p.chunks + chunk] =
            BeamChunk{top == -SV_INF ? 0.0 : all, top, s_bad ? -1 : listed};
    }
}

constexpr int kSelThreads = 512, kSelWaves = kSelThreads / 64;

__device__ __forceinline__ uint64_t score_key(double s) {
    const uint64_t u = __double_as_longlong(s + 0.0);
    return u >> 63 ? ~u : u | 1ull << 63;
}

// A candidate: its score (NaN: none), its beam, its logit's order key and its id.
// Of equal scores the lower beam's is first; within a beam the larger logit (also
// where float64 cannot tell the scores apart), then the lower id.
struct Cand {
    double s;
    uint32_t beam, key, id;
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
    if (a.s != b.s) return a.s > b.s;
    if (a.beam != b.beam) return a.beam < b.beam;
    return a.key > b.key || (a.key == b.key && a.id < b.id);
}

template <int DT>
__global__ __launch_bounds__(kSelThreads) void k_beam_select(BeamParams p) {
    __shared__ double s_log[kMaxBeams];   // logarithm of the sum relative to the largest; NaN: the beam gives nothing
    __shared__ float s_top[kMaxBeams];
    __shared__ double s_tau[kSelWaves], s_part[kSelWaves];
    __shared__ Cand s_list[kSelThreads], s_best[kSelWaves];
    __shared__ int s_n, s_near;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, b = blockIdx.x;
    const int W = p.W, per_row = p.chunks * W;
    const float* const scores = p.scores + b * W;
    const int32_t* const done = p.finished ? p.finished + b * W : nullptr;
    const double nan = __builtin_nan("");
    // up to kKept of the lists' entries a thread, on their way while the sums are joined
    constexpr int kKept = 8;
    const int lists = W * per_row, total = lists + (done ? W : 0);
    const uint64_t* const list = p.list + static_cast<int64_t>(b) * W * per_row;
    uint64_t entry[kKept];
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int c = tid + k * kSelThreads;
        entry[k] = c < lists ? list[c] : 0;
    }
    for (int i = w; i < W; i += kSelWaves) {
        double log_sum = nan;
        float top = -SV_INF;
        if (scores[i] != -SV_INF && !(done && done[i])) {
            const BeamChunk* const rec = p.rec + static_cast<int64_t>(b * W + i) * p.chunks;
            bool bad = !(scores[i] < SV_INF);
            for (int c = lane; c < p.chunks; c += 64) {
                top = fmaxf(top, rec[c].top);
                bad |= rec[c].n < 0;
            }
            for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
            double sum = 0.0;
            for (int c = lane; c < p.chunks; c += 64)
                if (rec[c].top != -SV_INF) sum += rec[c].sum * exp(static_cast<double>(rec[c].top) - top);
            for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
            if (!__any(bad) && top != -SV_INF) log_sum = log(sum);
        }
        if (lane == 0) {
            s_log[i] = log_sum;
            s_top[i] = top;
        }
    }
    __syncthreads();

    // candidate c of the lists, and behind them one for every finished beam.  (What a row that is not
    // asked for has in its lists is not looked at: it may be left from another call.)
    auto candidate = [&](int c, uint64_t e) {
        Cand y{nan, 0u, 0u, 0u};
        if (c >= lists) {
            const int i = c - lists;
            if (c < total && done[i] && scores[i] > -SV_INF && scores[i] < SV_INF)
                y = Cand{static_cast<double>(scores[i]), static_cast<uint32_t>(i), 0u, static_cast<uint32_t>(p.end)};
            return y;
        }
        const int i = c / per_row;
        if (s_log[i] != s_log[i] || e == 0) return y;
        y.beam = i;
        y.key = static_cast<uint32_t>(e >> 32);
        y.id = ~static_cast<uint32_t>(e);
        // the logarithm last: what is before it is exact for numbers of ordinary sizes, and beams of equal
        // rows tie wherever their sums of score and logit do
        y.s = (scores[i] + (static_cast<double>(key_value(y.key)) - s_top[i])) - s_log[i];
        return y;
    };
    // all of the thread's candidates: those at hand, then the others
    auto each = [&](auto&& use) {
#pragma unroll
        for (int k = 0; k < kKept; ++k) use(candidate(tid + k * kSelThreads, entry[k]));
        for (int c = tid + kKept * kSelThreads; c < total; c += kSelThreads) use(candidate(c, c < lists ? list[c] : 0));
    };

    for (int round = 0;; ++round) {  // the second with float64 sums
        if (tid == 0) s_n = s_near = 0;
        // A bound that W candidates of one wave's lanes reach: close for few beams.  Lists are sorted and
        // W long, so for 32 and 64 beams a lane has the same rank of every list, and the bound is the
        // largest candidate of about rank W / 2 or W - 1: thousands reach it, and then the sums are
        // taken again and the winners found one after the other.
        double best = -__builtin_huge_val();
        each([&](const Cand& y) {
            if (y.s > best) best = y.s;
        });
        {
            uint64_t x = score_key(best);
#pragma unroll
            for (int size = 2; size <= 64; size <<= 1)
#pragma unroll
                for (int step = size >> 1; step; step >>= 1) {
                    const uint64_t y = __shfl_xor(static_cast<unsigned long long>(x), step);
                    const bool larger = ((lane & step) == 0) == ((lane & size) == 0);
                    x = larger == (x > y) ? x : y;
                }
            x = __shfl(static_cast<unsigned long long>(x), W - 1);
            if (lane == 0) s_tau[w] = __longlong_as_double(x >> 63 ? x & ~(1ull << 63) : ~x);
        }
        __syncthreads();
        double tau = s_tau[0];
        for (int i = 1; i < kSelWaves; ++i) tau = fmax(tau, s_tau[i]);
        if (round == 0) tau -= kBand;
        each([&](const Cand& y) {
            if (y.s >= tau) {
                const int at = atomicAdd(&s_n, 1);
                if (at < kSelThreads) s_list[at] = y;
            }
        });
        __syncthreads();
        const int n = s_n;
        auto put = [&](int rank, const Cand& y) {
            const int i = y.beam, v = y.id, at = b * W + rank;
            p.out_tokens[at] = v;
            p.out_ancestor[at] = b * W + i;
            p.out_scores[at] = static_cast<float>(y.s);
            p.out_finished[at] = (done && done[i]) || v == p.end;
        };
        bool again = round == 0;
        if (n <= kSelThreads) {
            Cand me{};
            int rank = W;
            if (tid < n) {
                me = s_list[tid];
                rank = 0;
                bool near = false;
                for (int j = 0; j < n; ++j) {
                    const Cand y = s_list[j];
                    rank += before(y, me);
                    near |= fabs(y.s - me.s) <= kBand && y.beam != me.beam;
                }
                if (rank < W && near) s_near = 1;
            }
            __syncthreads();
            again = again && s_near != 0;
            if (!again) {
                if (rank < W) put(rank, me);
                if (tid >= n && tid < W) {  // fewer candidates than beams
                    const int at = b * W + tid;
                    p.out_tokens[at] = p.out_ancestor[at] = -1;
                    p.out_scores[at] = -SV_INF;
                    p.out_finished[at] = 0;
                }
            }
        } else if (!again) {  // many equal scores: one after the other
            Cand last{};
            for (int i = 0; i < W; ++i) {
                Cand top{nan, 0u, 0u, 0u};
                each([&](const Cand& y) {
                    if (y.s == y.s && (i == 0 || before(last, y)) && (top.s != top.s || before(y, top))) top = y;
                });
                for (int o = 32; o; o >>= 1) {
                    const Cand y{__shfl_xor(top.s, o), __shfl_xor(top.beam, o), __shfl_xor(top.key, o),
                                 __shfl_xor(top.id, o)};
                    if (y.s == y.s && (top.s != top.s || before(y, top))) top = y;
                }
                if (lane == 0) s_best[w] = top;
                __syncthreads();
                last = s_best[0];
                for (int k = 1; k < kSelWaves; ++k)
                    if (s_best[k].s == s_best[k].s && (last.s != last.s || before(s_best[k], last))) last = s_best[k];
                if (tid == 0) put(i, last);
                __syncthreads();
            }
        }
        if (!again) return;
        __syncthreads();  // everyone has read s_near, also where no row is left to be summed (all beams finished)
        // float64 sums of the rows that take part
        for (int i = 0; i < W; ++i) {
            if (s_log[i] != s_log[i]) continue;
            const uint8_t* const row = p.logits + (b * p.sb + i * p.sw) * Fmt<DT>::E;
            const double top = s_top[i];
            double sum = 0.0;
            for (int64_t v = tid * 8; v < p.V; v += kSelThreads * 8) {
                float x[8];
                eight<DT>(row, static_cast<int>(v), p.V, x);
#pragma unroll 1
                for (int k = 0; k < 8; ++k) sum += exp(x[k] - top);
            }
            for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
            if (lane == 0) s_part[w] = sum;
            __syncthreads();
            if (tid == 0) {
                sum = 0.0;
                for (int k = 0; k < kSelWaves; ++k) sum += s_part[k];
                s_log[i] = log(sum);
            }
            __syncthreads();
        }
    }
}

// Row k of the output is row ancestor[k] of the input, zeros where there is none, by the
// widest vectors that rows and strides allow.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_reorder(ReorderParams p) {
    const int k = blockIdx.y, a = p.ancestor[k];
    T* const dst = reinterpret_cast<T*>(p.dst + k * p.dst_stride);
    const int64_t n = p.bytes / static_cast<int64_t>(sizeof(T)), step = static_cast<int64_t>(gridDim.x) * kThreads;
    int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (a < 0 || a >= p.rows) {
        for (; i < n; i += step) dst[i] = T{};
        return;
    }
    const T* const src = reinterpret_cast<const T*>(p.src + a * p.src_stride);
    for (; i + 3 * step < n; i += 4 * step) {  // four under way
        const T y0 = src[i], y1 = src[i + step], y2 = src[i + 2 * step], y3 = src[i + 3 * step];
        dst[i] = y0;
        dst[i + step] = y1;
        dst[i + 2 * step] = y2;
        dst[i + 3 * step] = y3;
    }
    for (; i < n; i += step) dst[i] = src[i];
}

template <typename T>
hipError_t reorder_one(const ReorderParams& p, hipStream_t st, const LaunchEvents& ev) {
    const int64_t n = p.bytes / static_cast<int64_t>(sizeof(T));
    int64_t blocks = (n + 4 * kThreads - 1) / (4 * kThreads);
    if (blocks > 1024) blocks = 1024;
    hipExtLaunchKernelGGL((k_reorder<T>), dim3(static_cast<unsigned>(blocks), p.rows), dim3(kThreads), 0, st, ev.start,
                          ev.stop, 0, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_beam_stats(const BeamParams& p, int dtype, hipStream_t st, const LaunchEvents& ev) {
    const dim3 grid(p.chunks, p.B * p.W);
#define SV_BEAM(DT, RUNS) \
    hipExtLaunchKernelGGL((k_beam_stats<DT, RUNS>), grid, dim3(kThreads), 0, st, ev.start, ev.stop, 0, p)
    if (dtype == DT_BF16)
        p.runs == 1 ? SV_BEAM(DT_BF16, 1) : SV_BEAM(DT_BF16, 4);
    else
        p.runs == 1 ? SV_BEAM(DT_F32, 1) : SV_BEAM(DT_F32, 4);
#undef SV_BEAM
    return hipGetLastError();
}

hipError_t launch_beam_select(const BeamParams& p, int dtype, hipStream_t st, const LaunchEvents& ev) {
    if (dtype == DT_BF16)
        hipExtLaunchKernelGGL((k_beam_select<DT_BF16>), dim3(p.B), dim3(kSelThreads), 0, st, ev.start, ev.stop, 0, p);
    else
        hipExtLaunchKernelGGL((k_beam_select<DT_F32>), dim3(p.B), dim3(kSelThreads), 0, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

hipError_t launch_reorder(const ReorderParams& p, hipStream_t st, const LaunchEvents& ev) {
    const uint64_t all = reinterpret_cast<uintptr_t>(p.src) | reinterpret_cast<uintptr_t>(p.dst) |
                         static_cast<uint64_t>(p.src_stride) | static_cast<uint64_t>(p.dst_stride) |
                         static_cast<uint64_t>(p.bytes);
    if (all % 16 == 0) return reorder_one<uint4>(p, st, ev);
    if (all % 4 == 0) return reorder_one<uint32_t>(p, st, ev);
    return reorder_one<uint8_t>(p, st, ev);
}

}  // namespace sv
