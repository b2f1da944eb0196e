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
// One workgroup of 16 waves per sequence.  A sequence's passes depend on each
// other, so a row is not split over workgroups; 64 sequences read about as
// fast as the whole device can (each CU up to 64 bytes per clock).  Each wave
// sums a contiguous range of ids, so the pick re-reads 1/16 of the row, then
// 1/256 of it, then one block of ids.

#include <hip/hip_ext.h>

#include "sv_tree.h"

namespace sv {
namespace {

#pragma clang fp contract(off)

constexpr int kVThreads = 1024;
constexpr int kVWaves = kVThreads / 64;
constexpr int kVUnroll = 4;  // blocks of ids a wave has in flight

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
        uint32_t wv[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (id + j < V) {
                const uint32_t f = __float_as_uint(Prob<DT>::at(r, id + j));
                if (E == 4)
                    wv[j & 3] = f;
                else
                    wv[j >> 1] |= j & 1 ? f : f >> 16;
            }
        return make_uint4(wv[0], wv[1], wv[2], wv[3]);
    }
    __device__ __forceinline__ uint32_t top_of(uint32_t m, const uint4& v) const {
        return Prob<DT>::top(Prob<DT>::top(Prob<DT>::top(Prob<DT>::top(m, v.x), v.y), v.z), v.w);
    }
    // The sum over ids [lo, hi), lo and hi - lo multiples of kBlock: per wave, the
    // same in every lane.  ok: all entries are probabilities.
    template <bool Q>
    __device__ __forceinline__ double sum_of(int lo, int hi, int lane, bool& ok) const {
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

template <int DT>
__global__ __launch_bounds__(kVThreads) void k_tree_verify(TreeVerifyParams p) {
    using R = Residual<DT>;
    constexpr int E = R::E;
    __shared__ double s_sum[2][kVWaves];
    __shared__ int s_ok[2][kVWaves];
    __shared__ int s_token;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
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

    int flip = 0;
    R left;
    left.V = p.V;
    left.any_gone = false;
    left.gone = -1;
    const int range = (((p.V + kVWaves - 1) / kVWaves + R::kBlock - 1) / R::kBlock) * R::kBlock;
    // the row's sum; per-wave sums stay in s_sum[flip ^ 1]
    auto total = [&]() {
        bool ok = true;
        const double mine = left.sum(w * range, (w + 1) * range, lane, ok);
        ok = !__any(!ok);
        if (lane == 0) {
            s_sum[flip][w] = mine;
            s_ok[flip][w] = ok;
        }
        __syncthreads();
        double z = 0.0;
        bool all = true;
#pragma unroll
        for (int i = 0; i < kVWaves; ++i) {
            z += s_sum[flip][i];
            all = all && s_ok[flip][i];
        }
        good = good && all;
        flip ^= 1;
        return z;
    };

    int out_tok = -1, out_node = lane == 0 ? 0 : -1;
    int count = 0;
    if (good) {
        int cur = 0, tested = 0;
        double a = 0.0, S = 1.0;
        auto rows = [&]() {
            left.p = tgt + cur * p.tsp * (16 / E);
            left.q = dft ? dft + cur * p.dsp * (16 / E) : nullptr;
            left.a = a;
            left.use_q = dft && a > 0.0;
        };
        uint64_t gone = 0;  // without q: the current node's refused children
        while (good) {
            const uint64_t kids = __ballot(lane > tested && par == cur);
            if (!kids) break;
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
                if (kids & (kids - 1)) {  // a sibling follows
                    rows();
                    S = total();
                }
            } else {
                gone |= 1ull << i;
                if (!again) S = S - pi;
            }
        }
        // the last token, from what is left at cur
        double z = 0.0;
        if (good) {
            rows();
            if (!dft) {
                left.gone = gone >> lane & 1 ? tok : -1;
                left.any_gone = gone != 0;
            }
            z = total();
            if (good && !(z > 0.0)) {  // nothing left (rounding of the rows): the target's row itself
                left.use_q = false;
                left.any_gone = false;
                left.gone = -1;
                z = total();
            }
            good = good && z > 0.0;
        }
        if (good) {
            double t = static_cast<double>(ul) * z;
            // the wave's range that holds t, then the sixteenth of it; where rounding leaves
            // none, the last one with weight
            auto find = [&](const double* sums) {
                int at = -1, last = 0;
                double cum = 0.0, before = 0.0, before_last = 0.0;
                for (int i = 0; i < kVWaves; ++i) {
                    if (at < 0 && sums[i] > 0.0) {
                        last = i;
                        before_last = cum;
                    }
                    if (at < 0 && cum + sums[i] > t) {
                        at = i;
                        before = cum;
                    }
                    cum += sums[i];
                }
                if (at < 0) {
                    at = last;
                    before = before_last;
                }
                t -= before;
                return at;
            };
            const int w1 = find(s_sum[flip ^ 1]);
            const int part = (((range + kVWaves - 1) / kVWaves + R::kBlock - 1) / R::kBlock) * R::kBlock;
            const int lo1 = w1 * range;
            bool ok = true;
            const double mine = left.sum(min(lo1 + w * part, lo1 + range), min(lo1 + (w + 1) * part, lo1 + range), lane,
                                         ok);
            if (lane == 0) s_sum[flip][w] = mine;
            __syncthreads();
            const int w2 = find(s_sum[flip]);
            if (w == 0) {
                const int lo = lo1 + w2 * part, hi = min(min(lo + part, lo1 + range), p.V);
                int found = -1, last = -1;
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
                    if (some) last = __shfl(pos, 63 - __clzll(static_cast<long long>(some)));
                    cum += __shfl(incl, 63);
                }
                if (lane == 0) s_token = found >= 0 ? found : last;
            }
            __syncthreads();
            if (lane == count) out_tok = s_token;
        }
    }
    if (w == 0 && lane < p.N) {
        p.out_tokens[bn + lane] = good ? out_tok : -1;
        p.out_nodes[bn + lane] = good ? out_node : -1;
        if (lane == 0) p.out_n[b] = good ? count : -1;
    }
}

}  // namespace

hipError_t launch_tree_verify(const TreeVerifyParams& p, int dtype, hipStream_t st, const LaunchEvents& ev) {
    if (dtype == DT_BF16)
        hipExtLaunchKernelGGL(k_tree_verify<DT_BF16>, dim3(p.B), dim3(kVThreads), 0, st, ev.start, ev.stop, 0, p);
    else
        hipExtLaunchKernelGGL(k_tree_verify<DT_F32>, dim3(p.B), dim3(kVThreads), 0, st, ev.start, ev.stop, 0, p);
    return hipGetLastError();
}

}  // namespace sv
