// gfx950 kernel of the tree verification from given random numbers.
//
// The walk starts at node 0 and tests the current node's children in order.
// With the target's row p and the draft's row q at the current node, the
// distribution left after s refusals is max(0, p - a_s q) / S_s:
//
//   p_0 = p,  p_{s+1} = max(0, p_s - q) / Z_s
//   =>  p_s ~ max(0, p - a_s q),  a_0 = 0, S_0 = 1,
//       a_{s+1} = a_s + S_s,  S_s = sum_v max(0, p_v - a_s q_v),
//
// so a child x is accepted iff u S_s q_x < p_x - a_s q_x and a refusal costs
// one sum over the row, needed only if another sibling follows.  Without q
// (children that were chosen, not drawn) the refused ids are taken out of p
// one by one: x is accepted iff u S < p_x, and S loses p_x.  The last token is
// drawn from what is left at the last node by inverse CDF in id order.
//
// Everything is held in float64: the token is the exact inverse-CDF token
// unless u Z lies within the rounding of the sums (about 1e-15 Z) of a
// boundary.
//
// A sequence's passes depend on each other, and one CU reads a row of 128256
// float32 p and q in about 8 us (64 bytes per clock), so small batches give a
// sequence a team of workgroups.  All of a team walk alike.  A pass over a row
// is cut into 16 ranges per workgroup, one per wave; each workgroup sums its
// ranges, leaves the sums in the workspace, one 64-bit word each, and looks for
// the others'.  It looks a fixed number of times; what it has not found by then
// it computes itself, so no workgroup depends on another one running.  Sums of
// a range are the same whoever computes them, so every workgroup decides alike.
// The first one draws: it re-reads the range that holds the token, then a
// sixteenth of it, then blocks of ids.

#include <hip/hip_ext.h>

#include "sv_tree.h"

namespace sv {
namespace {

#pragma clang fp contract(off)

constexpr int kVThreads = 1024;
constexpr int kVWaves = kVThreads / 64;
static_assert(kVWaves == kVerifyWaves, "ranges per workgroup");

typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));

template <int DT>
struct Prob;
template <>
struct Prob<DT_F32> {
    static constexpr int E = 4;
    static __device__ __forceinline__ float at(const uint8_t* p, int64_t i) {
        return *reinterpret_cast<const float*>(p + 4 * i);
    }
    static __device__ __forceinline__ float get(const uint4& v, int j) {
        return __uint_as_float(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w);
    }
    // the largest bit pattern: above `kLargest` something is negative (or -0), infinite or NaN
    static constexpr uint32_t kLargest = 0x7F7FFFFFu;
    static __device__ __forceinline__ uint32_t top(uint32_t m, uint32_t x) { return m > x ? m : x; }
    static __device__ __forceinline__ bool over(uint32_t m) { return m > kLargest; }
};
template <>
struct Prob<DT_BF16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ float at(const uint8_t* p, int64_t i) {
        return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + 2 * i)) << 16);
    }
    static __device__ __forceinline__ float get(const uint4& v, int j) {
        const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
        return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
    }
    static __device__ __forceinline__ uint32_t top(uint32_t m, uint32_t x) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u16, m),
                                                                      __builtin_bit_cast(v2u16, x)));
    }
    static __device__ __forceinline__ bool over(uint32_t m) { return (m & 0xFFFFu) > 0x7F7Fu || (m >> 16) > 0x7F7Fu; }
};

__device__ __forceinline__ bool is_prob(float p) { return p >= 0.f && p <= 3.402823466e38f; }

// A lane's value, the lane the same for the whole wave.
__device__ __forceinline__ double of_lane(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u), lane));
    const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane));
    return __builtin_bit_cast(double, hi << 32 | lo);
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

// What is left of a row: p (a = 0), max(0, p - a q), or p without the ids in
// the lanes' `gone` (-1: none).
template <int DT>
struct Residual {
    static constexpr int E = Prob<DT>::E;
    static constexpr int kBlock = 64 * E;  // ids a wave takes at a time
    const uint8_t *p, *q;
    int V;
    double a;
    bool use_q;
    int gone;  // per lane
    bool any_gone;

    // the weights of this lane's ids [id, id + E) of the block at `base`
    template <bool Q>
    __device__ __forceinline__ void weights(int id, int base, const uint4& pv, const uint4& qv, double* w) const {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            w[j] = static_cast<double>(Prob<DT>::get(pv, j));
            if (Q) w[j] = fmax(__builtin_fma(-a, static_cast<double>(Prob<DT>::get(qv, j)), w[j]), 0.0);
        }
        if (!Q && any_gone) {
            uint64_t hit = __ballot(gone >= base && gone < base + kBlock);
            while (hit) {
                const int at = __builtin_amdgcn_readlane(gone, __ffsll(static_cast<unsigned long long>(hit)) - 1) - id;
                hit &= hit - 1;
#pragma unroll
                for (int j = 0; j < E; ++j) w[j] = at == j ? 0.0 : w[j];
            }
        }
    }
    // a whole vector; rows need not start on 16-byte boundaries
    __device__ __forceinline__ uint4 vec(const uint8_t* r, int id) const {
        uint4 v;
        __builtin_memcpy(&v, r + static_cast<int64_t>(id) * (16 / E), 16);
        return v;
    }
    // the same near the row's end, zeros behind it
    __device__ __forceinline__ uint4 vec_end(const uint8_t* r, int id) const {
        if (id + E <= V) return vec(r, id);
        uint64_t lo = 0, hi = 0;
#pragma unroll 1
        for (int j = 0; j < E && id + j < V; ++j) {
            const uint32_t f = __float_as_uint(Prob<DT>::at(r, id + j)) >> (E == 8 ? 16 : 0);
            const int at = j * (128 / E);
            if (at < 64)
                lo |= static_cast<uint64_t>(f) << at;
            else
                hi |= static_cast<uint64_t>(f) << (at - 64);
        }
        return make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                          static_cast<uint32_t>(hi >> 32));
    }
    __device__ __forceinline__ uint32_t top_of(uint32_t m, const uint4& v) const {
        return Prob<DT>::top(Prob<DT>::top(Prob<DT>::top(Prob<DT>::top(m, v.x), v.y), v.z), v.w);
    }
    // The sum over ids [lo, hi), lo and hi - lo multiples of kBlock: per wave, the
    // same in every lane.  ok: all entries are probabilities.
    template <bool Q>
    __device__ __forceinline__ double sum_of(int lo, int hi, int lane, bool& ok) const {
        // blocks in flight per wave; the float64 values of more would not fit the registers
        constexpr int kVUnroll = E == 8 ? 2 : 4;
        double acc[2] = {0.0, 0.0};
        uint32_t m = 0;
        if (hi > V) hi = V;
        int base = lo;
        for (; base + kBlock * kVUnroll <= hi; base += kBlock * kVUnroll) {
            uint4 pv[kVUnroll], qv[kVUnroll];
#pragma unroll
            for (int k = 0; k < kVUnroll; ++k) {
                pv[k] = vec(p, base + k * kBlock + lane * E);
                if (Q) qv[k] = vec(q, base + k * kBlock + lane * E);
            }
#pragma unroll
            for (int k = 0; k < kVUnroll; ++k) {
                double w[E];
                m = top_of(m, pv[k]);
                if (Q) m = top_of(m, qv[k]);
                weights<Q>(base + k * kBlock + lane * E, base + k * kBlock, pv[k], qv[k], w);
#pragma unroll
                for (int j = 0; j < E; ++j) acc[j & 1] += w[j];
                __builtin_amdgcn_sched_barrier(0);  // one block's float64 values in registers at a time
            }
        }
        for (; base < hi; base += kBlock) {
            const int id = base + lane * E;
            const uint4 pv = vec_end(p, id), qv = Q ? vec_end(q, id) : make_uint4(0, 0, 0, 0);
            double w[E];
            m = top_of(m, pv);
            if (Q) m = top_of(m, qv);
            weights<Q>(id, base, pv, qv, w);
#pragma unroll
            for (int j = 0; j < E; ++j) acc[j & 1] += w[j];
        }
        if (__any(Prob<DT>::over(m))) {  // a bad entry, or -0
            for (int id = lo + lane; id < hi; id += 64) {
                if (!is_prob(Prob<DT>::at(p, id))) ok = false;
                if (Q && !is_prob(Prob<DT>::at(q, id))) ok = false;
            }
        }
        return wave_sum(acc[0] + acc[1]);
    }
    __device__ __forceinline__ double sum(int lo, int hi, int lane, bool& ok) const {
        return use_q ? sum_of<true>(lo, hi, lane, ok) : sum_of<false>(lo, hi, lane, ok);
    }
};

// What a wave leaves of a range's sum: the sum, or -1 where an entry of the range
// is no probability.  All bits set: not there yet.
constexpr uint64_t kNone = ~0ull;
__global__ __launch_bounds__(kThreads) void k_verify_clear(uint64_t* p, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i < n) p[i] = kNone;
}

// TEAM: several workgroups per sequence.
template <int DT, bool TEAM>
__global__ __launch_bounds__(kVThreads) void k_tree_verify(TreeVerifyParams p) {
    using R = Residual<DT>;
    constexpr int E = R::E;
    __shared__ double s_sum[(TEAM ? kMaxTeam : 1) * kVWaves];
    __shared__ int s_token, s_missing;
    // the team of a sequence on one XCD (workgroups go to the eight in turn)
    const int team = TEAM ? p.team : 1;
    const int b = TEAM ? (blockIdx.x / (8 * team)) * 8 + (blockIdx.x & 7) : blockIdx.x;
    const int me = TEAM ? (blockIdx.x % (8 * team)) / 8 : 0;
    if (b >= p.B) return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int64_t bn = static_cast<int64_t>(b) * p.N;
    const int n = p.n_nodes ? p.n_nodes[b] : p.N;
    const uint8_t* const tgt = p.tgt + b * p.tsb * (16 / E);
    const uint8_t* const dft = p.dft ? p.dft + b * p.dsb * (16 / E) : nullptr;

    // every wave: lane i holds node i
    bool good = n >= 1 && n <= p.N;
    int par = -1, tok = -1;
    double px = 0.0, qx = 0.0, u = 0.0;
    if (good && lane >= 1 && lane < n) {
        par = p.parent[bn + lane];
        tok = p.tokens[bn + lane];
        const float uf = p.u_accept[bn + lane];
        bool in = par >= 0 && par < lane && tok >= 0 && tok < p.V && uf >= 0.f && uf < 1.f;
        if (dft && par >= p.P) in = false;
        if (in) {
            const float x = Prob<DT>::at(tgt, par * p.tsp + tok);
            in = is_prob(x);
            px = x;
            if (dft) {
                const float y = Prob<DT>::at(dft, par * p.dsp + tok);
                in = in && is_prob(y);
                qx = y;
            }
        }
        u = uf;
        good = in;
    }
    const float ul = p.u_final[b];
    good = !__any(!good) && ul >= 0.f && ul < 1.f;  // the same in every wave

    R left;
    left.V = p.V;
    left.any_gone = false;
    left.gone = -1;
    // the row in kVWaves ranges per workgroup of the team, one per wave
    const int ranges = team * kVWaves;
    const int range = (((p.V + ranges - 1) / ranges + R::kBlock - 1) / R::kBlock) * R::kBlock;
    const int per_lane = TEAM ? (ranges + 63) / 64 : 1;
    int pass = 0;
    // the sum of what the row has left; the ranges' sums stay in s_sum
    auto total = [&]() __attribute__((always_inline)) {
        uint64_t* const rec = p.rec + (static_cast<int64_t>(b) * p.passes + pass) * ranges;
        ++pass;
        __syncthreads();  // s_sum's last readers are done
        if (TEAM && tid == 0) s_missing = 0;
        int todo = 1 << me;  // whose ranges this workgroup sums: its own, then those it does not find
        for (bool looked = !TEAM;; looked = true) {
            while (todo) {
                const int r = (__ffs(todo) - 1) * kVWaves + w;
                todo &= todo - 1;
                bool ok = true;
                const double x = left.sum(r * range, (r + 1) * range, lane, ok);
                const double mine = __any(!ok) ? -1.0 : x;
                if (lane == 0) {
                    s_sum[r] = mine;
                    if (!looked)
                        __hip_atomic_store(rec + r, __builtin_bit_cast(uint64_t, mine), __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
                }
            }
            __syncthreads();
            if (looked) break;
            // the others' sums, each a whole word that is there or not
            if (tid < ranges && tid / kVWaves != me) {
                uint64_t x = kNone;
                for (int k = 0; k < p.looks && x == kNone; ++k)
                    x = __hip_atomic_load(rec + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                s_sum[tid] = __builtin_bit_cast(double, x);
                if (x == kNone) atomicOr(&s_missing, 1 << (tid / kVWaves));
            }
            __syncthreads();
            todo = s_missing;
        }
        double z = 0.0;
        bool all = true;
        if (!TEAM) {
#pragma unroll
            for (int i = 0; i < kVWaves; ++i) {
                z += s_sum[i];
                all = all && s_sum[i] >= 0.0;
            }
            good = good && all;
            return z;
        }
        for (int j = 0; j < per_lane; ++j) {
            const int i = lane * per_lane + j;
            const double x = i < ranges ? s_sum[i] : 0.0;
            all = all && x >= 0.0;
            z += x;
        }
        good = good && !__any(!all);
        return wave_sum(z);
    };

    int out_tok = -1, out_node = lane == 0 ? 0 : -1;
    int count = 0;
    if (good) {
        int cur = 0, tested = 0;
        double a = 0.0, S = 1.0;
        uint64_t gone = 0;  // without q: the current node's refused children
        bool last = false;
        double z = 0.0;
        while (good) {
            const uint64_t kids = last ? 0 : __ballot(lane > tested && par == cur);
            bool sum = !kids;
            if (kids) {
                const int i = __ffsll(static_cast<unsigned long long>(kids)) - 1;
                const int x = __builtin_amdgcn_readlane(tok, i);
                const double ui = of_lane(u, i), pi = of_lane(px, i), qi = of_lane(qx, i);
                const bool again = !dft && __any((gone >> lane & 1) && tok == x);
                const bool take = dft ? ui * S * qi < pi - a * qi : !again && ui * S < pi;
                tested = i;
                if (take) {
                    if (lane == count) out_tok = x;
                    ++count;
                    if (lane == count) out_node = i;
                    cur = i;
                    a = 0.0;
                    S = 1.0;
                    gone = 0;
                } else if (dft) {
                    a = a + S;
                    sum = (kids & (kids - 1)) != 0;  // a sibling follows
                } else {
                    gone |= 1ull << i;
                    if (!again) S = S - pi;
                }
            }
            if (!sum) continue;
            // what is left at cur: for the next sibling, or for the last token; where nothing is
            // left for that (rounding of the rows), the target's row itself
            left.p = tgt + cur * p.tsp * (16 / E);
            left.q = dft ? dft + cur * p.dsp * (16 / E) : nullptr;
            left.a = a;
            left.use_q = dft && a > 0.0 && !last;
            left.any_gone = !dft && !last && gone != 0;
            left.gone = left.any_gone && (gone >> lane & 1) ? tok : -1;
            const double s = total();
            if (kids) {
                S = s;
            } else {
                z = s;
                if (z > 0.0 || last) break;
                last = true;
            }
        }
        if (me != 0) return;  // one of the team draws
        good = good && z > 0.0;
        if (good) {
            double t = static_cast<double>(ul) * z;
            // the range that holds t, of sixteen sums; where rounding leaves none, the last one
            // with weight.  t becomes what is left of it there.
            auto find16 = [&](const double* sums) {
                int at = -1, last_one = 0;
                double cum = 0.0, before = 0.0, before_last = 0.0;
#pragma unroll
                for (int i = 0; i < kVWaves; ++i) {
                    const double x = sums[i];
                    if (at < 0 && x > 0.0) {
                        last_one = i;
                        before_last = cum;
                        if (cum + x > t) {
                            at = i;
                            before = cum;
                        }
                    }
                    cum += x;
                }
                t -= at < 0 ? before_last : before;
                return at < 0 ? last_one : at;
            };
            // the same of `number` sums, per lane `each` of them
            auto find = [&](const double* sums, int number, int each) {
                double mine = 0.0;
                for (int j = 0; j < each; ++j) {
                    const int i = lane * each + j;
                    mine += i < number ? sums[i] : 0.0;
                }
                double incl = mine;
                for (int o = 1; o < 64; o <<= 1) {
                    const double up = __shfl_up(incl, o);
                    if (lane >= o) incl += up;
                }
                const uint64_t over = __ballot(incl > t && mine > 0.0), some = __ballot(mine > 0.0);
                const int at = over ? __ffsll(static_cast<unsigned long long>(over)) - 1
                                    : 63 - __clzll(static_cast<long long>(some));
                double cum = of_lane(incl - mine, at), before = cum;
                int found = -1, last_one = -1;
                for (int j = 0; j < each; ++j) {
                    const int i = at * each + j;
                    const double x = i < number ? sums[i] : 0.0;
                    if (found < 0 && x > 0.0) {
                        last_one = i;
                        before = cum;
                    }
                    if (found < 0 && x > 0.0 && cum + x > t) found = i;
                    cum += x;
                }
                t -= before;
                return found >= 0 ? found : last_one;
            };
            const int r1 = TEAM ? find(s_sum, ranges, per_lane) : find16(s_sum);
            __syncthreads();
            const int part = (((range + kVWaves - 1) / kVWaves + R::kBlock - 1) / R::kBlock) * R::kBlock;
            const int lo1 = r1 * range;
            bool ok = true;
            const double mine = left.sum(min(lo1 + w * part, lo1 + range), min(lo1 + (w + 1) * part, lo1 + range), lane,
                                         ok);
            if (lane == 0) s_sum[w] = mine;
            __syncthreads();
            const int r2 = find16(s_sum);
            if (w == 0) {
                const int lo = lo1 + r2 * part, hi = min(min(lo + part, lo1 + range), p.V);
                int found = -1, last_id = -1;
                double cum = 0.0;
                for (int base = lo; base < hi && found < 0; base += R::kBlock) {
                    const int id = base + lane * E;
                    const uint4 pv = left.vec_end(left.p, id);
                    double wt[E];
                    if (left.use_q)
                        left.template weights<true>(id, base, pv, left.vec_end(left.q, id), wt);
                    else
                        left.template weights<false>(id, base, pv, pv, wt);
                    double mass = 0.0;
                    int pos = -1;
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        mass += wt[j];
                        if (wt[j] > 0.0) pos = id + j;
                    }
                    double incl = mass;
                    for (int o = 1; o < 64; o <<= 1) {
                        const double up = __shfl_up(incl, o);
                        if (lane >= o) incl += up;
                    }
                    // the first id whose running sum passes t
                    double run = cum + (incl - mass);
                    int mine_at = -1;
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        run += wt[j];
                        if (mine_at < 0 && wt[j] > 0.0 && run > t) mine_at = id + j;
                    }
                    const uint64_t have = __ballot(mine_at >= 0);
                    if (have) found = __shfl(mine_at, __ffsll(static_cast<unsigned long long>(have)) - 1);
                    const uint64_t some = __ballot(pos >= 0);
                    if (some) last_id = __shfl(pos, 63 - __clzll(static_cast<long long>(some)));
                    cum += __shfl(incl, 63);
                }
                if (lane == 0) s_token = found >= 0 ? found : last_id;
            }
            __syncthreads();
            if (lane == count) out_tok = s_token;
        }
    }
    if (me == 0 && w == 0 && lane < p.N) {
        p.out_tokens[bn + lane] = good ? out_tok : -1;
        p.out_nodes[bn + lane] = good ? out_node : -1;
        if (lane == 0) p.out_n[b] = good ? count : -1;
    }
}

}  // namespace

hipError_t launch_verify_clear(const TreeVerifyParams& p, hipStream_t st, const LaunchEvents& ev) {
    const int64_t n = static_cast<int64_t>(p.B) * p.passes * p.team * kVWaves;
    hipExtLaunchKernelGGL(k_verify_clear, dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                          st, ev.start, ev.stop, 0, p.rec, n);
    return hipGetLastError();
}

namespace {
template <bool TEAM>
hipError_t verify_launch(const TreeVerifyParams& p, int dtype, hipStream_t st, const LaunchEvents& ev) {
    const unsigned grid = static_cast<unsigned>(TEAM ? (p.B + 7) / 8 * 8 * p.team : p.B);
    if (dtype == DT_BF16)
        hipExtLaunchKernelGGL((k_tree_verify<DT_BF16, TEAM>), dim3(grid), dim3(kVThreads), 0, st, ev.start, ev.stop, 0,
                              p);
    else
        hipExtLaunchKernelGGL((k_tree_verify<DT_F32, TEAM>), dim3(grid), dim3(kVThreads), 0, st, ev.start, ev.stop, 0,
                              p);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_tree_verify(const TreeVerifyParams& p, int dtype, hipStream_t st, const LaunchEvents& ev) {
    return p.team > 1 ? verify_launch<true>(p, dtype, st, ev) : verify_launch<false>(p, dtype, st, ev);
}

}  // namespace sv
