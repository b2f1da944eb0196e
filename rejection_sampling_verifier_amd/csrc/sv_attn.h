// What the attention kernels share: matrix instructions and their operands,
// softmax pieces, direct loads to LDS, the cut of a line of tiles into parts,
// ancestor sets.  Included by device sources only.
#pragma once

#include <hip/hip_ext.h>

#include <mutex>
#include <set>
#include <utility>

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

// The reference m is the running maximum less kUp.  float16's normal numbers end
// at 2^-14: with weights around 2^7 (8 of slack in m: 2^15 at most, of 65504) a
// long tail behind a dominant key keeps its share of the output, with 2^-25 of
// 2^m, 2^-32 of the largest weight, lost per key at most.
template <int DT>
constexpr float kUp = DT == DT_BF16 ? 0.f : 7.f;

// A score and what is left of it above the reference, rounded each: fused, the
// row's largest score would come out as its rounding (not small beside 1 from
// 2^24 on, 2^128 and an infinite weight from 2^31 on) instead of 0.  Time with
// the two: wide trees 557 us, 554 fused; the other shapes alike.
__device__ __forceinline__ float scaled(float x, float scale2) {
#pragma clang fp contract(off)
    return x * scale2;
}
__device__ __forceinline__ float less(float x, float ref) {
#pragma clang fp contract(off)
    return x - ref;
}

// What rows that do not exist, and dimensions past D, are staged from.
__device__ const uint4 kZero = {0, 0, 0, 0};

typedef __attribute__((address_space(1))) const uint32_t global_u32;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

// 16 bytes per lane from `src` to the 1024 at `dst`, without registers.
__device__ __forceinline__ void to_lds(const uint8_t* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds((global_u32*)src, (lds_u32*)dst, 16, 0, 0);
}

// s_waitcnt vmcnt(0) with the other counters left alone (gfx9 encoding: vmcnt
// in bits 0-3 and 14-15, expcnt 4-6, lgkmcnt 8-11).
constexpr int kWaitVm0 = 0x0F70;

// 16 bytes per lane from base + off to the 1024 at LDS address `dst`.  Assembly,
// so that the compiler does not wait for these loads at every read of another
// stage; the kernel waits for them itself (vmcnt).
// (base and dst are the same for all lanes, whether the compiler sees it or not.)
__device__ __forceinline__ void load_lds(const uint8_t* base, uint32_t off, uint32_t dst) {
    const uint64_t b = reinterpret_cast<uintptr_t>(base);
    const uint64_t at = static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32))) << 32 |
                        static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b)));
    dst = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(at), "s"(dst) : "memory");
}
__device__ __forceinline__ void load_lds(const uint8_t* from, uint32_t dst) {
    dst = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(dst) : "memory");
}

typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v8s lds_read(uint32_t at) {
    return *reinterpret_cast<__attribute__((address_space(3))) v8s*>(at);
}
__device__ __forceinline__ v4s lds_read_tr(uint32_t at) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_v4s*>(at));
}

// Until at most N of the wave's global loads are under way.
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Byte offsets of row numbers times strides in 16-byte units.
__device__ __forceinline__ uint64_t units(uint32_t i, uint32_t s) { return (static_cast<uint64_t>(i) * s) << 4; }
__device__ __forceinline__ uint64_t units(uint32_t i, uint32_t s, uint32_t j, uint32_t r) {
    return (static_cast<uint64_t>(i) * s + static_cast<uint64_t>(j) * r) << 4;
}

// Parts the line of `total` tiles is cut into, and the part that tile f is in:
// `extra` parts of `per` + 1 tiles, then parts of `per`.
struct Cut {
    int64_t per, extra;
    int parts;
    __device__ __forceinline__ Cut(int clusters, int64_t total) {
        parts = total < clusters ? static_cast<int>(total) : clusters;
        if (total >> 32 == 0) {  // a 64-bit division costs about half a microsecond
            per = static_cast<uint32_t>(total) / static_cast<uint32_t>(parts);
        } else {
            per = total / parts;
        }
        extra = total - per * parts;
    }
    __device__ __forceinline__ int64_t start(int c) const { return c * per + (c < extra ? c : extra); }
    __device__ __forceinline__ int of(int64_t f) const {
        const int64_t wide = extra * (per + 1);
        const int64_t g = f < wide ? f : f - wide, by = f < wide ? per + 1 : per;
        const int64_t q = (g | by) >> 32 == 0 ? static_cast<uint32_t>(g) / static_cast<uint32_t>(by) : g / by;
        return static_cast<int>(f < wide ? q : extra + q);
    }
};

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
    for (int s = 1; s < n; s *= 2) {  // paths double in length
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

// Lets a kernel use more than 64 KB of LDS, once per kernel and device.
hipError_t allow_lds(const void* kernel, int bytes) {
    static std::mutex mu;
    static std::set<std::pair<const void*, int>> done;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (done.count({kernel, dev})) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done.insert({kernel, dev});
    return e;
}

}  // namespace
}  // namespace sv
