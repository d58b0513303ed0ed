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

// Eight consecutive elements of a row as loaded (bf16 stays packed until used).
//
// Where the row length is a multiple of eight, each group is whole and at a
// 16-byte boundary and loaded as it is.  In ragged rows a
// group sits at any element boundary, which gfx950 takes for 16-byte accesses,
// and the last one is short.  That one is loaded whole all the same, with what
// follows it, which is cleared when it is used (in the last row, from the row's
// last eight elements, and shifted into place): taken in pieces, it would be
// waited for where it is loaded, and with it everything loaded before.  It is
// stored in pieces of four, two and one.  Rows of under eight elements are
// loaded in such pieces too.
//
// STREAM in a store: past the caches, for outputs that no cache will hold until
// they are read.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef u32x4_t u32x4_any __attribute__((aligned(2)));
typedef u32x2_t u32x2_any __attribute__((aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef f32x4_t f32x4_any __attribute__((aligned(4)));
typedef f32x2_t f32x2_any __attribute__((aligned(4)));

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
    // A whole group at a 16-byte boundary.
    __device__ __forceinline__ void load(const bf16raw* p) { u = *reinterpret_cast<const u32x4_t*>(p); }
    // A whole group at any boundary.
    __device__ __forceinline__ void load_any(const bf16raw* p) { u = *reinterpret_cast<const u32x4_any*>(p); }
    // The first n < 8 elements, zeros behind them.
    __device__ __forceinline__ void load_pieces(const bf16raw* p, int n)
    {
        u = u32x4_t{0, 0, 0, 0};
        if (n <= 0) return;
        if (n & 4) {
            const u32x2_any v = *reinterpret_cast<const u32x2_any*>(p);
            u[0] = v[0];
            u[1] = v[1];
        }
        if (n & 2) {
            const uint32_t v = *reinterpret_cast<const u32_any*>(p + (n & 4));
            if (n & 4) u[2] = v;
            else u[0] = v;
        }
        if (n & 1) {
            const uint32_t v = p[n & 6];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = (n & 6) == 2 * j ? v : u[j];
        }
    }
    // Keeps the first n elements.
    __device__ __forceinline__ void first(int n)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] &= n > 2 * j + 1 ? 0xffffffffu : n > 2 * j ? 0xffffu : 0u;
    }
    __device__ __forceinline__ void clear() { u = u32x4_t{0, 0, 0, 0}; }
    // by < 8 elements down, zeros behind them.
    __device__ __forceinline__ void shift(int by)
    {
        if (by & 4) u = u32x4_t{u[2], u[3], 0, 0};
        if (by & 2) u = u32x4_t{u[1], u[2], u[3], 0};
        if (by & 1)
            u = u32x4_t{u[0] >> 16 | u[1] << 16, u[1] >> 16 | u[2] << 16, u[2] >> 16 | u[3] << 16, u[3] >> 16};
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
    template <bool STREAM = false>
    __device__ __forceinline__ void store(bf16raw* p) const
    {
        put16<STREAM>(p, u);
    }
    __device__ __forceinline__ void store_any(bf16raw* p) const { *reinterpret_cast<u32x4_any*>(p) = u; }
    // The first n < 8 elements.
    __device__ __forceinline__ void store_pieces(bf16raw* p, int n) const
    {
        if (n & 4) *reinterpret_cast<u32x2_any*>(p) = u32x2_t{u[0], u[1]};
        if (n & 2) *reinterpret_cast<u32_any*>(p + (n & 4)) = n & 4 ? u[2] : u[0];
        if (n & 1) p[n & 6] = bf16raw((n & 4 ? (n & 2 ? u[3] : u[2]) : (n & 2 ? u[1] : u[0])) & 0xffffu);
    }
};

template <>
struct Eight<float> {
    f32x4_t a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = *reinterpret_cast<const f32x4_t*>(p);
        b = *reinterpret_cast<const f32x4_t*>(p + 4);
    }
    __device__ __forceinline__ void load_any(const float* p)
    {
        a = *reinterpret_cast<const f32x4_any*>(p);
        b = *reinterpret_cast<const f32x4_any*>(p + 4);
    }
    __device__ __forceinline__ void load_pieces(const float* p, int n)
    {
        a = b = f32x4_t{0, 0, 0, 0};
        if (n <= 0) return;
        if (n & 4) a = *reinterpret_cast<const f32x4_any*>(p);
        if (n & 2) {
            const f32x2_any v = *reinterpret_cast<const f32x2_any*>(p + (n & 4));
            if (n & 4) {
                b[0] = v[0];
                b[1] = v[1];
            } else {
                a[0] = v[0];
                a[1] = v[1];
            }
        }
        if (n & 1) {
            const float v = p[n & 6];
            a[0] = (n & 6) == 0 ? v : a[0];
            a[2] = (n & 6) == 2 ? v : a[2];
            b[0] = (n & 6) == 4 ? v : b[0];
            b[2] = (n & 6) == 6 ? v : b[2];
        }
    }
    __device__ __forceinline__ void first(int n)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j >= n) a[j] = 0.f;
            if (j + 4 >= n) b[j] = 0.f;
        }
    }
    __device__ __forceinline__ void clear() { a = b = f32x4_t{0, 0, 0, 0}; }
    __device__ __forceinline__ void shift(int by)
    {
        if (by & 4) {
            a = b;
            b = f32x4_t{0, 0, 0, 0};
        }
        if (by & 2) {
            a = f32x4_t{a[2], a[3], b[0], b[1]};
            b = f32x4_t{b[2], b[3], 0, 0};
        }
        if (by & 1) {
            a = f32x4_t{a[1], a[2], a[3], b[0]};
            b = f32x4_t{b[1], b[2], b[3], 0};
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
    template <bool STREAM = false>
    __device__ __forceinline__ void store(float* p) const
    {
        put16<STREAM>(p, a);
        put16<STREAM>(p + 4, b);
    }
    __device__ __forceinline__ void store_any(float* p) const
    {
        *reinterpret_cast<f32x4_any*>(p) = a;
        *reinterpret_cast<f32x4_any*>(p + 4) = b;
    }
    __device__ __forceinline__ void store_pieces(float* p, int n) const
    {
        if (n & 4) *reinterpret_cast<f32x4_any*>(p) = a;
        if (n & 2) *reinterpret_cast<f32x2_any*>(p + (n & 4)) = n & 4 ? f32x2_t{b[0], b[1]} : f32x2_t{a[0], a[1]};
        if (n & 1) p[n & 6] = n & 4 ? (n & 2 ? b[2] : b[0]) : (n & 2 ? a[2] : a[0]);
    }
};

// How the rows of a call lie, a template argument (MODE) of the kernels: whole
// groups at 16-byte boundaries (D a multiple of eight), ragged rows, or rows of
// under eight elements.  The last are apart because their loads in pieces, in
// the same loop, would make the compiler wait before every other load.
constexpr int kWhole = 0, kRagged = 1, kTiny = 2;
inline int row_mode(int64_t D) { return D % 8 == 0 ? kWhole : D > 8 ? kRagged : kTiny; }

// A lane's group of eight of a row of D elements.  In a ragged row it is whole,
// short (the row's last D % 8 elements) or behind the row.  How short, and so
// what is cleared and which pieces are stored, is the same for every row and
// lane, which makes those branches scalar.
template <int MODE>
struct Group {
    uint32_t col, from;  // its first column, and where it is loaded in the last row
    int kind;            // 0 whole, 1 short, 2 behind the row
    __device__ __forceinline__ void init(uint32_t first, uint32_t D)
    {
        col = from = first;
        kind = first >= D ? 2 : MODE == kWhole || first + 8 <= D ? 0 : 1;
        if (MODE == kRagged && kind != 0) from = D - 8;
    }
    // The elements from row[0 .. D) into e, which was cleared once before its first
    // load: groups behind the row are never loaded and stay zero.  `on`: the row
    // exists.  `last`: nothing may be read behind it.  A ragged row's short group
    // is in place after settle().
    template <typename T>
    __device__ __forceinline__ void load(Eight<T>& e, const T* row, uint32_t D, bool on, bool last) const
    {
        if (!on) {
            e.clear();
        } else if (kind != 2) {
            if (MODE == kWhole) e.load(row + col);
            else if (MODE == kRagged) e.load_any(row + (last ? from : col));
            else e.load_pieces(row + col, int(D) - int(col));
        }
    }
    template <typename T>
    __device__ __forceinline__ void settle(Eight<T>& e, uint32_t D, bool last) const
    {
        if (MODE != kRagged || kind != 1) return;
        if (last) e.shift(8 - int(D % 8));
        else e.first(int(D % 8));
    }
    template <typename T>
    __device__ __forceinline__ void store(const Eight<T>& e, T* row, uint32_t D, bool on) const
    {
        if (!on) return;
        if (kind == 0) {
            if (MODE == kWhole) e.store(row + col);
            else e.store_any(row + col);
        } else if (MODE != kWhole && kind == 1) {
            e.store_pieces(row + col, int(D % 8));
        }
    }
    // Whether element j of the group exists.
    __device__ __forceinline__ bool has(int j, uint32_t D, bool on) const
    {
        return on && (MODE == kWhole ? kind == 0 : col + j < D);
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
    // The round keys are two scalar additions a round.  Without this the compiler
    // computes all twenty before a kernel's row loop, and has to park them in
    // vector lanes.
    asm volatile("" : "+s"(k0), "+s"(k1));
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = uint64_t(a) * 0xD2511F53u, q = uint64_t(c) * 0xCD9E8D57u;
        a = __builtin_amdgcn_bitop3_b32(uint32_t(q >> 32), b, k0, 0x96);  // exclusive or of the three
        c = __builtin_amdgcn_bitop3_b32(uint32_t(p >> 32), d, k1, 0x96);
        b = uint32_t(q);
        d = uint32_t(p);
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
