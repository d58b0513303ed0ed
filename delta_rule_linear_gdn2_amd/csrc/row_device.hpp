// Row-wise device helpers of the training operators: sums over lane groups,
// eight-element accesses at any alignment, sigmoid and the counter-based
// random bits of dropout.
#pragma once

#include "gdn2_device.hpp"
#include "launch.hpp"

namespace gdn2 {

template <int CTRL>
__device__ __forceinline__ float dpp_lanes(float x)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}

// Sum over aligned groups of G lanes (4, 8, 16, 32 or 64), in every lane of the
// group: register-to-register exchanges only.  Pairs and quads by lane
// permutation, then the other half of eight and of sixteen lanes by mirroring
// (every lane of a half already holds the half's sum), then lane swaps.
template <int G>
__device__ __forceinline__ float group_sum(float x)
{
    x += dpp_lanes<0xB1>(x);                  // lane ^ 1
    x += dpp_lanes<0x4E>(x);                  // lane ^ 2
    if (G >= 8) x += dpp_lanes<0x141>(x);     // 7 - lane within eight
    if (G >= 16) x += dpp_lanes<0x140>(x);    // 15 - lane within sixteen
    if (G >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if (G >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return x;
}

// Sigmoid with the hardware exponential and reciprocal (about one ulp each).
// It keeps its limits: 0 and 1 at minus and plus infinity, NaN for NaN.
__device__ __forceinline__ float fast_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// STREAM in a store: past the caches, for outputs that no cache will hold until
// they are read.
//
// Eight consecutive elements of a row as loaded (bf16 stays packed until used).
// FULL: the eight exist and sit at a 16-byte boundary.  Otherwise n of them
// exist (n <= 0: none) and the address is aligned to the element only: gfx950
// takes 16-byte accesses at any element boundary, and the last group of a row
// goes element by element.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t u32x4_any __attribute__((aligned(2)));
typedef f32x4_t f32x4_any __attribute__((aligned(4)));

template <bool STREAM, typename V, typename P>
__device__ __forceinline__ void put16(P* p, const V& v)
{
    if (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
    else *reinterpret_cast<V*>(p) = v;
}

template <typename T>
struct Eight;

template <>
struct Eight<bf16raw> {
    u32x4_t u;
    template <bool FULL>
    __device__ __forceinline__ void load(const bf16raw* p, int n)
    {
        if (FULL) {
            if (n > 0) u = *reinterpret_cast<const u32x4_t*>(p);
            else u = u32x4_t{0, 0, 0, 0};
            return;
        }
        if (n >= 8) {
            u = *reinterpret_cast<const u32x4_any*>(p);
        } else {
            uint32_t e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = j < n ? p[j] : 0u;
            u = u32x4_t{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
        }
    }
    __device__ __forceinline__ void get(float* v) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void put(const float* v)
    {
        u = u32x4_t{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                    f32x2_to_bf16x2(v[6], v[7])};
    }
    template <bool FULL, bool STREAM = false>
    __device__ __forceinline__ void store(bf16raw* p, int n) const
    {
        if (FULL) {
            if (n > 0) put16<STREAM>(p, u);
            return;
        }
        if (n >= 8) {
            *reinterpret_cast<u32x4_any*>(p) = u;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[j] = bf16raw(j & 1 ? u[j / 2] >> 16 : u[j / 2] & 0xffffu);
        }
    }
};

template <>
struct Eight<float> {
    f32x4_t a, b;
    template <bool FULL>
    __device__ __forceinline__ void load(const float* p, int n)
    {
        if (FULL) {
            if (n > 0) {
                a = *reinterpret_cast<const f32x4_t*>(p);
                b = *reinterpret_cast<const f32x4_t*>(p + 4);
            } else {
                a = b = f32x4_t{0, 0, 0, 0};
            }
            return;
        }
        if (n >= 8) {
            a = *reinterpret_cast<const f32x4_any*>(p);
            b = *reinterpret_cast<const f32x4_any*>(p + 4);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = j < n ? p[j] : 0.f;
                b[j] = j + 4 < n ? p[j + 4] : 0.f;
            }
        }
    }
    __device__ __forceinline__ void get(float* v) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    }
    __device__ __forceinline__ void put(const float* v)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = v[j];
            b[j] = v[4 + j];
        }
    }
    template <bool FULL, bool STREAM = false>
    __device__ __forceinline__ void store(float* p, int n) const
    {
        if (FULL) {
            if (n > 0) {
                put16<STREAM>(p, a);
                put16<STREAM>(p + 4, b);
            }
            return;
        }
        if (n >= 8) {
            *reinterpret_cast<f32x4_any*>(p) = a;
            *reinterpret_cast<f32x4_any*>(p + 4) = b;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) p[j] = j < 4 ? a[j & 3] : b[j & 3];
        }
    }
};

// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel Random
// Numbers: As Easy as 1, 2, 3", 2011): 128 bits from a 128-bit counter (the
// block in the low half, the call's offset in the high half) and a 64-bit key
// (the seed).  Nothing is carried from one block to the next, so the mask of
// any element is remade from its position alone.
__device__ __forceinline__ u32x4_t philox4x32(uint64_t block, uint64_t offset, uint64_t seed)
{
    uint32_t a = uint32_t(block), b = uint32_t(block >> 32), c = uint32_t(offset), d = uint32_t(offset >> 32);
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = uint64_t(a) * 0xD2511F53u, q = uint64_t(c) * 0xCD9E8D57u;
        const uint32_t na = uint32_t(q >> 32) ^ b ^ k0, nc = uint32_t(p >> 32) ^ d ^ k1;
        b = uint32_t(q);
        d = uint32_t(p);
        a = na;
        c = nc;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4_t{a, b, c, d};
}

// Whether element j (0..7) of a block is kept: its 16 bits, the low half of a
// word first, against the threshold.
__device__ __forceinline__ bool philox_keep(const u32x4_t& bits, int j, uint32_t threshold)
{
    const uint32_t w = bits[j / 2];
    return ((j & 1) ? w >> 16 : w & 0xffffu) >= threshold;
}

}  // namespace gdn2
