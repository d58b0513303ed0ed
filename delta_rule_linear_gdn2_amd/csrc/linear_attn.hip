// Linear attention with a fixed decay for each head: whole sequences, their
// gradients, and the carries of sequence segments.
//
// The recurrence of a head with decay a (the state S is dk x dv):
//     S_t = a S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t.
// It and the three gradients are one sum, here called a walk, over rows x
// (length DA), y (DA) and z (width):
//     out_i = sum_{j <= i} a^(i-j) (x_i . y_j) z_j + a^(i+1-late) X^T x_i
// with a carry X (DA x width) from before the walk, which becomes
//     X <- a^n X + sum_j a^(n-1+late-j) y_j z_j^T          (n tokens walked).
//     o :  forwards,  x, y, z = q, k, v     X = S     late 0
//     dq:  forwards,  x, y, z = do, v, k    X = S^T   late 0
//     dk:  backwards, x, y, z = v, do, q    X = R^T   late 1
//     dv:  backwards, x, y, z = k, q, do    X = R     late 1
// where R_t = q_t do_t^T + a R_{t+1} is the gradient of S_t.  Backwards, i
// counts from the sequence's last token and X is a R of the token behind it
// (at the end the final state's gradient; what remains is the initial state's).
//
// Chunks of 64 tokens: the products inside a chunk are masked, decayed 64 x 64
// tiles; X passes from chunk to chunk in FP32.
//
// Work split.  One workgroup walks one (sequence segment, head, slice of up to
// 64 columns of z).  X's slice stays in the matrix accumulators of its state
// wavefronts, 16 columns each; four output wavefronts, 16 tokens of a chunk each, form
//     P^T = Y X^T (tokens j x i), masked and decayed in registers, then
//     O^T = Xs^T X^T + Z^T P^T  (columns x tokens i),
// where an accumulator tile is directly the next product's operand, because a
// matrix product does not care for the order of its inner index as long as both
// operands take the same (see Frag).  The decays of a tile are constants of the
// head: each lane keeps its own in registers for the whole walk.
//
// Precision.  bf16 inputs feed bf16 matrix products with FP32 sums.  What is a factor
// again goes in as two bf16 terms (2^-16): P, the copy of X that the outputs read, and
// the factor a^n z of X's update where the caller does not get X.  So an output is
// rounded once, to its own type: 1.66e-3 against 64 bits in relative L2.  With one term
// of the copy it was 2.08e-3, at 125 us instead of 141 (forward) and 346 instead of 396
// (backward) of the shape below; the state's wavefronts forming X^T x from their
// registers instead of the outputs' from LDS took 141.  X itself is FP32.  Where the
// caller gets it, the factor of its update goes in as three bf16 terms that hold all
// 24 bits, so that it is the state of FP32 arithmetic.  FP32 inputs are three bf16
// terms throughout.
//
// What bounds it (8 sequences x 4096 tokens x 16 heads of 128, bf16; 64 chunks a
// workgroup, one workgroup a compute unit): 141 us, where its 537 MB take 106 at a
// large copy's rate.  Without products the same loads, staging and stores take 112,
// without loads and stores the products 98.  A chunk's turn takes about 1500 cycles of
// matrix instructions and 1600 of vector ones on each SIMD; on the two wavefronts that
// it has they overlap in part.  With one term of the copy, at 122 us: two workgroups a
// compute unit (128 registers a lane) spilled loads in flight, 177 to 296 us; twelve
// wavefronts, with the state's rows halved here too, 127; tiles of 32 x 32 with each
// tile of P formed twice 143; loads two chunks ahead instead of one the same.
#include "gdn2_device.hpp"
#include "launch.hpp"

namespace gdn2 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kC = kLinearChunk;
constexpr int kMayCross = 0x6;  // of a scheduling barrier: vector and scalar arithmetic
constexpr int kAuxOut = 2;  // buffer cache policy of the outputs' stores: nt

// Waits for the wavefront's own LDS accesses and meets the others; its global
// loads stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // vmcnt 63, expcnt 7, lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// A window of memory, the same in all lanes: loads past it give zero, stores
// past it are dropped.
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes)
{
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(p)), hi = __builtin_amdgcn_readfirstlane(uint32_t(p >> 32));
    void* pu = reinterpret_cast<void*>((uint64_t(hi) << 32) | lo);
    return __builtin_amdgcn_make_buffer_rsrc(pu, (short)0, int(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) { return f32x2_to_bf16x2(a, b); }

// LDS tiles of rows of D elements, in granules of 16 bytes whose place is XORed
// with a linear map of the row's low four bits.  The maps keep free of bank
// conflicts the 16-byte reads of 16 rows at four granules (the lanes of one access
// cycle hold rows 0-3 and 12-15 at one granule and 4-11 at the next: the images of
// rows 4 and 8 differ in bit 0 alone), the transposing reads of 16 columns of 16
// rows (the images of rows 1, 2 and 4 differ in more than bit 0), and the stores
// of four columns a lane.
template <typename T, int D>
struct Tile {
    static constexpr int kRow = D * int(sizeof(T));
    static constexpr int kGranules = kRow / 16;
    static constexpr __host__ __device__ int swz(int row)
    {
        return kRow >= 256   ? ((row & 7) << 1) ^ (row & 8 ? 9 : 0)
               : kRow == 128 ? (row & 6) ^ (row & 8 ? 5 : 0)
                             : ((row & 4) >> 1) ^ (row & 8 ? 3 : 0);
    }
    static __device__ __forceinline__ int off(int row, int granule) { return row * kRow + ((granule ^ swz(row)) << 4); }
};

// FP32 values as the sum of N bf16 ones, each of what the ones before leave.  Three
// hold all 24 bits; their leading terms are rounded to nearest, so that what they
// leave is at most 2^-8 and 2^-17 of the value and of either sign (cut off, it is
// twice that with the value's own sign, which shrinks every product of two values by
// up to 2^-21; rounding costs 2% of the FP32 calls).  Of two, the first is cut off and
// the second rounded: off by 2^-16, of either sign.  (An infinity leaves a NaN
// behind it, and three terms take what rounds to one, from 2^128 (1 - 2^-9), for one.)
template <int N>
__device__ __forceinline__ void split_pair(float lo, float hi, uint32_t (&t)[N])
{
#pragma unroll
    for (int k = 0; k < N - 1; ++k) {
        if constexpr (N == 3) {
            t[k] = pack2(lo, hi);
            lo -= __uint_as_float(t[k] << 16);
            hi -= __uint_as_float(t[k] & 0xffff0000u);
        } else {
            const uint32_t ul = __float_as_uint(lo), uh = __float_as_uint(hi);
            t[k] = __builtin_amdgcn_perm(uh, ul, 0x07060302);  // the upper halves
            lo -= __uint_as_float(ul & 0xffff0000u);
            hi -= __uint_as_float(uh & 0xffff0000u);
        }
    }
    t[N - 1] = pack2(lo, hi);
}

// Planes of bf16 that hold the elements of type T.
template <typename T>
constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;

// An operand of a 16 x 16 matrix product over 32 inner indices: 16 rows (or
// columns), one per lane & 15, and of the inner indices eight a quarter-wavefront
// g = lane >> 4.
//   rows:     inner index along a tile's rows (the natural order)
//   cols:     inner index down a tile's rows, 16 columns; order "accumulator": of
//             every 16 rows the four 4 g .. + 3 that a lane holds in a 16 x 16
//             accumulator, so that
//   from_acc: two accumulator tiles are the other operand as they are.
// FP32 operands are three bf16 planes, and a product six: what is left out, the
// second plane times the third and below, is at most 2^-24 of it.  (The FP32 matrix instructions take 2.7 times as long.)
template <typename T>
struct Frag {
    static constexpr int PL = kPlanes<T>;
    bf16x8 x[PL];
    static __device__ __forceinline__ int inner(int e, int g) { return 16 * (e >> 2) + 4 * g + (e & 3); }
    template <int D, int ROWS>
    static __device__ __forceinline__ Frag rows(const unsigned char* tile, int row0, int s, int lane)
    {
        using TL = Tile<bf16raw, D>;
        Frag f;
#pragma unroll
        for (int k = 0; k < PL; ++k)
            f.x[k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(tile + k * ROWS * TL::kRow +
                                                                               TL::off(row0 + (lane & 15), 4 * s + (lane >> 4))));
        return f;
    }
    // In each group of 16 lanes the transposing load takes four rows of 16
    // columns: lane 4 r + c reads columns 4 c .. + 3 of row r, and lane l
    // receives column l of the four rows.
    template <int D>
    static __device__ __forceinline__ Frag cols(const unsigned char* tile, int col0, int s, int lane)
    {
        using TL = Tile<bf16raw, D>;
        const int c = col0 + 4 * (lane & 3), r = 4 * (lane >> 4) + ((lane & 15) >> 2);
        const int lo = TL::off(32 * s + r, c >> 3) + ((c & 4) << 1), hi = TL::off(32 * s + 16 + r, c >> 3) + ((c & 4) << 1);
        Frag f;
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            const unsigned char* const t = tile + k * kC * TL::kRow;
            const v4i16 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(t + lo));
            const v4i16 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(t + hi));
            f.x[k] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return f;
    }
    __device__ __forceinline__ void put(int pair, const uint32_t (&t)[PL])
    {
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            u32x4 u = __builtin_bit_cast(u32x4, x[k]);
            u[pair] = t[k];
            x[k] = __builtin_bit_cast(bf16x8, u);
        }
    }
    static __device__ __forceinline__ Frag from_acc(const f32x4* p)
    {
        Frag f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[PL];
            split_pair<PL>(p[i >> 1][2 * (i & 1)], p[i >> 1][2 * (i & 1) + 1], t);
            f.put(i, t);
        }
        return f;
    }
    // Of an operand in accumulator order: inner indices from n on as zeros.
    __device__ __forceinline__ Frag first_rows(int n, int g) const
    {
        Frag f;
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            u32x4 u = __builtin_bit_cast(u32x4, x[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] &= (inner(2 * i, g) < n ? 0xffffu : 0u) | (inner(2 * i + 1, g) < n ? 0xffff0000u : 0u);
            f.x[k] = __builtin_bit_cast(bf16x8, u);
        }
        return f;
    }
    // The elements as FP32.
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = v[2 * i + 1] = 0.f;
#pragma unroll
            for (int k = PL - 1; k >= 0; --k) {
                const uint32_t u = __builtin_bit_cast(u32x4, x[k])[i];
                v[2 * i] = k == PL - 1 ? __uint_as_float(u << 16) : v[2 * i] + __uint_as_float(u << 16);
                v[2 * i + 1] = k == PL - 1 ? __uint_as_float(u & 0xffff0000u) : v[2 * i + 1] + __uint_as_float(u & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ f32x4 times(const Frag& b, f32x4 c) const
    {
        if constexpr (PL == 3) {
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[2], b.x[0], c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[0], b.x[2], c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[1], b.x[1], c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[1], b.x[0], c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[0], b.x[1], c, 0, 0, 0);
        }
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[0], b.x[0], c, 0, 0, 0);
    }
};

// The factor of the carry's update, z times its decays.  FP32: three planes like
// any operand.  bf16: N terms, of which the other operand (one plane) takes each.
template <typename T, bool EXACT>
struct Scaled;

template <bool EXACT>
struct Scaled<float, EXACT> {
    Frag<float> f;
    __device__ __forceinline__ Scaled(const Frag<float>& z, const float* scale)
    {
        float v[8];
        z.get(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[3];
            split_pair<3>(v[2 * i] * scale[2 * i], v[2 * i + 1] * scale[2 * i + 1], t);
            f.put(i, t);
        }
    }
    __device__ __forceinline__ f32x4 times(const Frag<float>& y, f32x4 c) const { return y.times(f, c); }
};

template <bool EXACT>
struct Scaled<bf16raw, EXACT> {
    static constexpr int N = EXACT ? 3 : 2;
    Frag<bf16raw> f[N];
    __device__ __forceinline__ Scaled(const Frag<bf16raw>& z, const float* scale)
    {
        float v[8];
        z.get(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[N];
            split_pair<N>(v[2 * i] * scale[2 * i], v[2 * i + 1] * scale[2 * i + 1], t);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const uint32_t one[1] = {t[k]};
                f[k].put(i, one);
            }
        }
    }
    __device__ __forceinline__ f32x4 times(const Frag<bf16raw>& y, f32x4 c) const
    {
#pragma unroll
        for (int k = N - 1; k >= 0; --k) c = y.times(f[k], c);
        return c;
    }
};

// Four consecutive elements into LDS: as they are, and as operand planes `stride`
// bytes apart.
__device__ __forceinline__ void put4(unsigned char* p, const f32x4& v, bf16raw*)
{
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void put4(unsigned char* p, const f32x4& v, float*) { *reinterpret_cast<f32x4*>(p) = v; }
template <int PL>
__device__ __forceinline__ void put4_planes(unsigned char* p, int stride, const f32x4& v)
{
    uint32_t a[PL], b[PL];
    split_pair<PL>(v[0], v[1], a);
    split_pair<PL>(v[2], v[3], b);
#pragma unroll
    for (int k = 0; k < PL; ++k) *reinterpret_cast<uint2*>(p + k * stride) = make_uint2(a[k], b[k]);
}

// alpha^n for a whole n >= 0, by squaring in 64 bits: off by n 2^-53, far below FP32.
// alpha as the other kernels take it: in [2^-15, 1], NaN as 2^-15.
__device__ __forceinline__ float power(float alpha, uint32_t n)
{
    double a = double(fminf(fmaxf(alpha, 0x1p-15f), 1.0f)), p = 1.0;
    for (; n; n >>= 1, a *= a)
        if (n & 1) p *= a;
    return float(p);
}
// The same for n <= 64.
__device__ __forceinline__ float small_power(float alpha, int n)
{
    double a = double(fminf(fmaxf(alpha, 0x1p-15f), 1.0f)), p = 1.0;
#pragma unroll
    for (int b = 0; b < 7; ++b, a *= a) p = n >> b & 1 ? p * a : p;
    return float(p);
}

// Packed sequences.  Segment m of sequence n has
//   the slot start / seg_len + n + m, distinct for distinct segments of offsets that
//   do not decrease, and below T / seg_len + N for any;
//   the window start / seg_len + m, distinct for distinct segments but the last ones
//   of their sequences, and for those below T / seg_len: a sequence of s > 1 segments
//   ends at or behind window start / seg_len + s - 1, where the next one's begin.
// So a workgroup for every slot finds every segment, and a workgroup and a place for
// every window every segment whose carry is read.  The first window of a sequence of
// several segments is also its own alone.
// Finds n: the last sequence whose first slot (each = 1) or window (each = 0) is not
// above `at`, 64 sequences or borders of 64 ranges at a time.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int N, int T, int seg_len, int each, int at, int lane)
{
    int lo = 0, count = N;
    while (true) {
        const int step = (count + 63) / 64, i = lo + lane * step;
        bool below = false;
        if (lane * step < count) {
            int b = cu[i];
            b = b < 0 ? 0 : b > T ? T : b;
            below = b / seg_len + each * i <= at;
        }
        const int n = __popcll(__ballot(below));
        if (n > 0) {
            lo += (n - 1) * step;
            count -= (n - 1) * step;
        }
        if (step == 1) return lo;
        count = count < step ? count : step;
    }
}

// A workgroup's wavefronts and LDS.  bf16 keeps two chunks in LDS, so that one is
// staged while the other is used (one barrier a chunk); FP32, with three planes,
// has room for one.
template <typename T, int DA, int CW, bool OUT>
struct Shape {
    static constexpr int kOutWaves = OUT ? 4 : 0;  // 16 tokens of a chunk each
    // State wavefronts: 16 columns of X each, in tiles of 16 x 16; half of the rows
    // where there are no output wavefronts beside them.
    static constexpr int kStateRows = !OUT && DA >= 64 ? DA / 2 : DA;
    static constexpr int kStateWaves = CW / 16 * (DA / kStateRows);
    static constexpr int kTiles = kStateRows / 16;
    static constexpr int kThreads = 64 * (kOutWaves + kStateWaves);
    static constexpr int kBufs = sizeof(T) == 2 ? 2 : 1;
    static constexpr int PL = kPlanes<T>;
    static constexpr int kBytesXY = PL * kC * DA * 2, kBytesZ = PL * kC * CW * 2;
    static constexpr int kTermsS = sizeof(T) == 2 ? 2 : 1;  // of the copy of X that outputs read, each of PL planes
    static constexpr int kBytesS = OUT ? kTermsS * PL * CW * DA * 2 : 0;
    static constexpr int kOffY = 0, kOffZ = kBytesXY, kOffX = kOffZ + kBytesZ;
    static constexpr int kBuf = kOffX + (OUT ? kBytesXY : 0);  // one chunk's tiles
    static constexpr int kOffS = kBufs * kBuf;
    static constexpr int kOffO = kOffS + kBufs * kBytesS;      // outputs on their way to memory
    static constexpr int kBytesO = OUT ? kC * CW * int(sizeof(T)) : 0;
    static constexpr bool kTable = sizeof(T) == 4;             // powers of the decay in LDS
    static constexpr int kOffPow = kOffO + kBufs * kBytesO;
    static constexpr int kLds = kOffPow + (kTable ? 80 * 4 : 0);
    static_assert(kLds <= 160 * 1024, "the LDS of a compute unit");
};

// One thread's share of a chunk's tile of kC rows of D elements, in groups of eight.
template <typename T, int D, int THREADS>
struct Stage {
    static constexpr int kG = D / 8, kTotal = kC * kG, kN = (kTotal + THREADS - 1) / THREADS, kWide = int(sizeof(T)) / 2;
    u32x4 v[kN][kWide];
    __device__ __forceinline__ void load(rsrc_t r, uint32_t stride, int L, bool back, int tid)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = tid + i * THREADS;
            if (kTotal % THREADS && at >= kTotal) break;
            const int row = at / kG;
            const uint32_t off = uint32_t(back ? L - 1 - row : row) * stride + uint32_t(at % kG) * (16 * kWide);
            // a row behind the last one (before the first one, walking back) is past the window
#pragma unroll
            for (int j = 0; j < kWide; ++j)
                v[i][j] = __builtin_amdgcn_raw_buffer_load_b128(r, int(row < L ? off + 16 * j : 0x80000000u), 0, 0);
        }
    }
    __device__ __forceinline__ void store(unsigned char* tile, int tid) const
    {
        using TL = Tile<bf16raw, D>;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = tid + i * THREADS;
            if (kTotal % THREADS && at >= kTotal) break;
            unsigned char* const p = tile + TL::off(at / kG, at % kG);
            if constexpr (kWide == 1) {
                *reinterpret_cast<u32x4*>(p) = v[i][0];
            } else {
                u32x4 out[3];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t t[3];
                    split_pair<3>(__uint_as_float(v[i][j >> 1][2 * (j & 1)]), __uint_as_float(v[i][j >> 1][2 * (j & 1) + 1]), t);
                    out[0][j] = t[0], out[1][j] = t[1], out[2][j] = t[2];
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x4*>(p + k * kC * TL::kRow) = out[k];
            }
        }
    }
};

// Zeros for the output rows that no sequence owns, by the blocks behind the walks'.
__device__ __forceinline__ void zero_padding(const LinearLaunch& a, int elem, int threads)
{
    int64_t lo = a.cu_seqlens[0], hi = a.cu_seqlens[a.N];
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    hi = hi < lo ? lo : hi > a.T ? a.T : hi;
    const int64_t step = int64_t(a.pad_blocks) * threads, at = (blockIdx.x - a.walk_blocks) * int64_t(threads) + threadIdx.x;
    const int64_t g = int64_t(a.H) * a.width * elem / 16;  // 16-byte granules a token
    for (int k = 0; k < a.walks; ++k) {
        uint4* const p = static_cast<uint4*>(a.walk[k].out);
        for (int64_t i = at; i < lo * g; i += step) p[i] = make_uint4(0, 0, 0, 0);
        for (int64_t i = hi * g + at; i < a.T * g; i += step) p[i] = make_uint4(0, 0, 0, 0);
    }
}

// Four rows of a column of a carry in memory, `p` at the first: rows `sd` apart.
// Where rows are neighbours (the squares that dq and dk read turned over) they are
// one access.
__device__ __forceinline__ f32x4 load_rows4(const float* p, int64_t sd)
{
    if (sd == 1) return *reinterpret_cast<const f32x4*>(p);
    return f32x4{p[0], p[sd], p[2 * sd], p[3 * sd]};
}
__device__ __forceinline__ void store_rows4(float* p, int64_t sd, const f32x4& v)
{
    if (sd == 1) {
        *reinterpret_cast<f32x4*>(p) = v;
        return;
    }
    p[0] = v[0], p[sd] = v[1], p[2 * sd] = v[2], p[3 * sd] = v[3];
}

// What every wavefront of a workgroup knows of its walk.
struct Place {
    LinearWalk w;
    int n, m, segments, hd, col0;  // segment m of sequence n's `segments`
    int64_t carry, kept;      // where segment 0's carry is, and what comes in while there are several
    int64_t row0, tok;        // tok: forwards the next token, backwards the one behind it
    int left;                 // tokens to walk
    bool last;                // the sequence's last segment
};

// The chunks of a walk as one wavefront sees them: every wavefront stages its
// share of the tiles; output wavefront ROLE forms the outputs of tokens 16 ROLE ..
// + 15 of each chunk, state wavefronts (ROLE kState) keep X.
constexpr int kState = 4;
template <typename T, int DA, int CW, bool OUT, bool EXACT, int ROLE>
__device__ __forceinline__ void walk(const LinearLaunch& a, Place pl, unsigned char* lds, int tid)
{
    using SH = Shape<T, DA, CW, OUT>;
    using F = Frag<T>;
    constexpr bool STATER = ROLE == kState;
    constexpr int NT = SH::kThreads, EB = int(sizeof(T)), TS = SH::kTiles;
    constexpr int kSteps = kC / 32, kPer = 8;   // products over a chunk's tokens, tokens a lane takes in each
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, l = lane & 15;
    const bool back = pl.w.back;
    const int late = back ? 1 : 0;

    const float al = a.alpha[pl.hd];
    const uint32_t strideA = uint32_t(a.H) * DA * EB, strideZ = uint32_t(a.H) * a.width * EB;
    const char* const px = static_cast<const char*>(pl.w.x) + (pl.row0 * a.H + pl.hd) * DA * EB;
    const char* const py = static_cast<const char*>(pl.w.y) + (pl.row0 * a.H + pl.hd) * DA * EB;
    const int64_t zoff = ((pl.row0 * a.H + pl.hd) * a.width + pl.col0) * EB;
    const char* const pz = static_cast<const char*>(pl.w.z) + zoff;

    // Chunk c of the walk, c = 0 .. chunks - 1: its tokens are loaded into registers
    // a chunk before they are staged in LDS.
    struct Staged {
        Stage<T, DA, NT> x, y;
        Stage<T, CW, NT> z;
    };
    Staged st;
    const int chunks = int((uint32_t(pl.left) + kC - 1) / kC);  // left may be 2^31 - 1
    const auto length = [&](int c) { return c + 1 < chunks ? kC : pl.left - c * kC; };
    const auto first = [&](int c) { return back ? pl.tok - int64_t(c) * kC - length(c) : pl.tok + int64_t(c) * kC; };
    const auto fetch = [&](int c, Staged& g) {
        const int n = length(c);
        const int64_t t0 = first(c);
        const rsrc_t ry = make_rsrc(py + t0 * strideA, uint32_t(n - 1) * strideA + DA * EB);
        const rsrc_t rz = make_rsrc(pz + t0 * strideZ, uint32_t(n - 1) * strideZ + CW * EB);
        g.y.load(ry, strideA, n, back, tid);
        g.z.load(rz, strideZ, n, back, tid);
        if (OUT) {
            const rsrc_t rx = make_rsrc(px + t0 * strideA, uint32_t(n - 1) * strideA + DA * EB);
            g.x.load(rx, strideA, n, back, tid);
        }
    };
    const auto stage = [&](const Staged& g, unsigned char* buf) {
        g.y.store(buf + SH::kOffY, tid);
        g.z.store(buf + SH::kOffZ, tid);
        if (OUT) g.x.store(buf + SH::kOffX, tid);
    };
    if (chunks > 0) fetch(0, st);
    // Powers of the decay up to a whole chunk's: a table in LDS, or, as bf16 tiles of 128
    // x 64 leave no room for one, in each lane that of the lane's number, which the others
    // take from it (FP32 calls take 2 to 6% longer that way).
    float* const table = reinterpret_cast<float*>(lds + SH::kOffPow);
    float mine = 0.f, whole = 0.f;
    if constexpr (SH::kTable) {
        for (int i = tid; i <= kC; i += NT) table[i] = small_power(al, i);
        lds_barrier();
    } else {
        mine = small_power(al, lane), whole = small_power(al, kC);
    }
    const auto pw = [&](int n) {
        n = n < 0 ? 0 : n;
        if constexpr (SH::kTable) return table[n];
        const float p = __shfl(mine, n & 63, 64);
        return n == kC ? whole : p;
    };

    // State wavefronts: columns 16 cb .. and rows d0 .., this lane column 16 cb + l
    // and rows d0 + 16 t + 4 g + r of tile t (d0 = 0 where OUT).
    const int cb = STATER ? (wave - SH::kOutWaves) % (CW / 16) : 0;
    const int d0 = STATER ? (wave - SH::kOutWaves) / (CW / 16) * SH::kStateRows : 0;

    // Constants of the head: output wavefronts hold the decays of their tiles of P
    // (by the distance of the tile's tokens) and of the carry's read, state
    // wavefronts those of their z.
    float dec[4][4], read = 0.f, scale[kSteps * kPer];
    const auto scales = [&](int n) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int e = 0; e < kPer; ++e) scale[s * kPer + e] = pw(n - 1 + late - (32 * s + F::inner(e, g)));
    };
    f32x4 X[TS];
    if constexpr (!STATER) {
#pragma unroll
        for (int dt = 0; dt <= ROLE; ++dt)
#pragma unroll
            for (int r = 0; r < 4; ++r) dec[dt][r] = pw(16 * dt + l - (4 * g + r));
        // each lane its own power: taken from another it costs the bf16 backward 1 to 2%
        const int to = 16 * ROLE + l + 1 - late;
        read = SH::kTable ? pw(to) : small_power(al, to);
    } else {
        scales(chunks > 0 ? length(0) : kC);
        // the carry: what comes in, or the segments before this one in order
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) X[t][r] = 0.f;
        const int64_t square = int64_t(DA) * a.width, sd = pl.w.state_d;
        const int64_t c = (pl.col0 + 16 * cb + l) * int64_t(pl.w.state_c);
        if (pl.w.carry_in && pl.m == 0) {
            // Where there are several segments, the launch for carries keeps what comes in:
            // the last segment may write the final carry over it while the first still has
            // to read it.
            float* const keep = pl.w.segment_carry + (pl.kept * a.H + pl.hd) * square + c;
            const float* const in = pl.w.carry_in + (int64_t(pl.n) * a.H + pl.hd) * square + c;
            const bool kept = OUT && pl.segments > 1;
#pragma unroll
            for (int t = 0; t < TS; ++t) {
                const int64_t d = d0 + 16 * t + 4 * g;
                X[t] = load_rows4((kept ? keep : in) + d * sd, sd);
                if (!OUT) store_rows4(keep + d * sd, sd, X[t]);
            }
        }
        if (OUT && pl.m > 0) {
            // two segments' carries on their way at a time; behind the last one it is
            // read again and has no weight
            const float over = power(al, uint32_t(a.seg_len));
            const float* const p = pl.w.segment_carry + (pl.carry * a.H + pl.hd) * square + c;
            for (int j = 0; j < pl.m; j += 2) {
                const bool two = j + 1 < pl.m;
                const float* const p0 = p + j * a.H * square;
                const float* const p1 = two ? p0 + a.H * square : p0;
                f32x4 v[2][TS];
#pragma unroll
                for (int t = 0; t < TS; ++t) {
                    v[0][t] = load_rows4(p0 + (16 * t + 4 * g) * sd, sd);
                    v[1][t] = load_rows4(p1 + (16 * t + 4 * g) * sd, sd);
                }
#pragma unroll
                for (int t = 0; t < TS; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        X[t][r] = over * X[t][r] + v[0][t][r];
                        if (two) X[t][r] = over * X[t][r] + v[1][t][r];
                    }
            }
        }
    }

    // X as the output wavefronts read it: FP32 as three planes, bf16 as two, hi and lo.
    // X - hi is a matrix product added to X, hi as the operand that two of its tiles
    // make times minus the rows of the identity that belong to a tile (`minus`): exact,
    // and eight matrix instructions instead of 64 vector ones (141.5 -> 139 us).
    F minus[2];
    if constexpr (OUT && STATER && SH::PL == 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool mine = l >> 2 == g && i == 2 * h + ((l & 3) >> 1);  // row l is inner index 4 h + (l & 3) of g = l / 4
                const uint32_t pair[1] = {mine ? (l & 1 ? 0xbf800000u : 0xbf80u) : 0u};
                minus[h].put(i, pair);
            }
    }
    const auto publish = [&](unsigned char* lS) {
        if constexpr (OUT && STATER) {
            const auto place = [&](int t) {
                const int d = 16 * t + 4 * g;
                return lS + Tile<bf16raw, DA>::off(16 * cb + l, d >> 3) + ((d & 4) << 1);
            };
            if constexpr (SH::PL == 1) {
                f32x4 rest[TS];
#pragma unroll
                for (int s = 0; s < TS / 2; ++s) {
                    const F hi = F::from_acc(X + 2 * s);
                    const u32x4 u = __builtin_bit_cast(u32x4, hi.x[0]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        *reinterpret_cast<uint2*>(place(2 * s + h)) = make_uint2(u[2 * h], u[2 * h + 1]);
                        rest[2 * s + h] = minus[h].times(hi, X[2 * s + h]);
                    }
                }
#pragma unroll
                for (int t = 0; t < TS; ++t) put4(place(t) + CW * DA * 2, rest[t], static_cast<bf16raw*>(nullptr));
            } else {
#pragma unroll
                for (int t = 0; t < TS; ++t) put4_planes<SH::PL>(place(t), CW * DA * 2, X[t]);
            }
        }
    };
    const auto outputs = [&](const unsigned char* buf, const unsigned char* lS, unsigned char* lO) {
        const unsigned char* const lY = buf + SH::kOffY;
        const unsigned char* const lZ = buf + SH::kOffZ;
        const unsigned char* const lX = buf + SH::kOffX;
        constexpr int ND = DA / 32, NC = CW / 16, NP = ROLE + 1;  // tiles of P: the tokens up to ROLE's
        constexpr int NJ = (NP + 1) / 2;                          // operands that they make
        // The products with x: tiles of Y (16 tokens each) for P, then tiles of the
        // carry (16 columns each).  Operands are read kAhead tiles before their
        // matrix instructions; left to itself the compiler reads each where it is
        // used, and the wavefront waits for LDS forty times a chunk.
        constexpr int kTerms = SH::kTermsS, kTiles = NP + kTerms * NC, kAhead = 8 / (ND * SH::PL), kZ = NC * NJ;
        // z's operands are read with the last of them; for FP32 rows of 128 that takes the
        // registers of loads in flight (packed FP32 backward 67.6 instead of 64.8 us).
        constexpr bool kLate = SH::PL * ND > 8;
        F xf[ND], fr[kAhead + 1][ND], zf[kZ];
        f32x4 p[2 * NJ], o[NC];
        const auto load = [&](int k) {
#pragma unroll
            for (int s = 0; s < ND; ++s)
                fr[k % (kAhead + 1)][s] = k < NP ? F::template rows<DA, kC>(lY, 16 * k, s, lane)
                                                 : F::template rows<DA, CW>(lS + (kTerms - 1 - (k - NP) % kTerms) * (CW * DA * 2),
                                                                            16 * ((k - NP) / kTerms), s, lane);
        };
#pragma unroll
        for (int s = 0; s < ND; ++s) xf[s] = F::template rows<DA, kC>(lX, 16 * ROLE, s, lane);
#pragma unroll
        for (int k = 0; k < kAhead && k < kTiles; ++k) load(k);
        if constexpr (2 * NJ > NP) p[NP] = f32x4{0.f, 0.f, 0.f, 0.f};
        f32x4 acc;
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
            if (k + kAhead < kTiles) load(k + kAhead);
            if (k == kTiles - 1 && !kLate) {
#pragma unroll
                for (int j = 0; j < kZ; ++j) zf[j] = F::template cols<CW>(lZ, 16 * (j / NJ), j % NJ, lane);
            }
            __builtin_amdgcn_sched_barrier(kMayCross);
            if (k < NP || (k - NP) % kTerms == 0) acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < ND; ++s) acc = fr[k % (kAhead + 1)][s].times(xf[s], acc);
            if (k < NP) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc[r] *= dec[k < NP ? ROLE - k : 0][r];
                    if (k == ROLE) acc[r] = 4 * g + r <= l ? acc[r] : 0.f;
                }
                p[k] = acc;
            } else if ((k - NP) % kTerms == kTerms - 1) {
#pragma unroll
                for (int r = 0; r < 4; ++r) o[(k - NP) / kTerms][r] = acc[r] * read;
            }
        }
        // bf16: P goes in as two terms.  Rounded to one, a lone token's outputs would all
        // be off by the rounding of its q . k (3% of the forward at the training shape).
        F pf[NJ][kTerms];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            if constexpr (kTerms == 1) {
                pf[j][0] = F::from_acc(p + 2 * j);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t t[2];
                    split_pair<2>(p[2 * j + (i >> 1)][2 * (i & 1)], p[2 * j + (i >> 1)][2 * (i & 1) + 1], t);
                    const uint32_t hi[1] = {t[0]}, lo[1] = {t[1]};
                    pf[j][0].put(i, hi);
                    pf[j][1].put(i, lo);
                }
            }
        }
        // The last operand of P holds the tokens behind a lane's own as zeros, and zero times
        // what is not finite there is not zero: where an output is not finite, the product
        // is taken again for each token with the rows of z behind it left out.
        const auto last = [&](int c, const F& z, f32x4 acc) {
#pragma unroll
            for (int k = kTerms - 1; k >= 0; --k) acc = z.times(pf[NJ - 1][k], acc);
            return acc;
        };
        f32x4 before[NC];
        float probe = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if constexpr (kLate) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) zf[c * NJ + j] = F::template cols<CW>(lZ, 16 * c, j, lane);
            }
#pragma unroll
            for (int j = 0; j < NJ - 1; ++j)
#pragma unroll
                for (int k = kTerms - 1; k >= 0; --k) o[c] = zf[c * NJ + j].times(pf[j][k], o[c]);
            before[c] = o[c];
            o[c] = last(c, zf[c * NJ + NJ - 1], o[c]);
#pragma unroll
            for (int r = 0; r < 4; ++r) probe = __builtin_fmaf(o[c][r], 0.f, probe);
        }
        if (__builtin_expect(__ballot(probe != 0.f) != 0, 0)) {
#pragma clang loop unroll(disable)
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const f32x4 v = last(c, zf[c * NJ + NJ - 1].first_rows(16 * ROLE + i + 1 - 32 * (NJ - 1), g), before[c]);
                    if (l == i) o[c] = v;
                }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = 16 * c + 4 * g, per = 16 / EB;
            put4(lO + Tile<T, CW>::off(16 * ROLE + l, col / per) + (col % per) * EB, o[c], static_cast<T*>(nullptr));
        }
    };
    // A chunk's outputs from LDS to memory, whole rows of the slice at a time (stored
    // straight from the accumulators, 32 bytes of a row at once, they took 17 us of
    // 132 us without any product).
    const auto flush = [&](int c, const unsigned char* lO) {
        if constexpr (OUT) {
            constexpr int kG = Tile<T, CW>::kGranules, kTotal = kC * kG;
            const int n = length(c);
            const rsrc_t ro = make_rsrc(static_cast<char*>(pl.w.out) + zoff + first(c) * strideZ, uint32_t(n - 1) * strideZ + CW * EB);
#pragma unroll
            for (int i = 0; i < (kTotal + NT - 1) / NT; ++i) {
                const int at = tid + i * NT, row = at / kG;
                if (kTotal % NT && at >= kTotal) break;
                const u32x4 v = *reinterpret_cast<const u32x4*>(lO + Tile<T, CW>::off(row, at % kG));
                const uint32_t off = uint32_t(back ? n - 1 - row : row) * strideZ + uint32_t(at % kG) * 16;
                __builtin_amdgcn_raw_buffer_store_b128(v, ro, int(row < n ? off : 0x80000000u), 0, kAuxOut);
            }
        }
    };
    const auto update = [&](int c, const unsigned char* buf) {
        const int n = length(c);
        if (n < kC) scales(n);
        const float over = SH::kTable || n < kC ? pw(n) : whole;
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) X[t][r] *= over;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const Scaled<T, EXACT> z(F::template cols<CW>(buf + SH::kOffZ, 16 * cb, s, lane), scale + s * kPer);
#pragma unroll
            for (int t = 0; t < TS; ++t) X[t] = z.times(F::template cols<DA>(buf + SH::kOffY, d0 + 16 * t, s, lane), X[t]);
        }
    };

    unsigned char* const lS = lds + SH::kOffS;
    unsigned char* const lO = lds + SH::kOffO;
    if constexpr (SH::kBufs == 1) {
        for (int c = 0; c < chunks; ++c) {
            stage(st, lds);
            publish(lS);
            if (c > 0) flush(c - 1, lO);
            if (c + 1 < chunks) fetch(c + 1, st);
            lds_barrier();
            if constexpr (STATER) update(c, lds);
            else outputs(lds, lS, lO);
            lds_barrier();
        }
        if (chunks > 0) flush(chunks - 1, lO);
    } else if (chunks > 0) {
        // While chunk c is used from buffers c & 1, chunk c + 1 goes from registers to
        // the other ones, c + 2 is on its way into the registers, and the outputs of
        // c - 1 leave.
        stage(st, lds);
        publish(lS);
        if (chunks > 1) fetch(1, st);
        lds_barrier();
        const auto turn = [&](int c, unsigned char* buf, unsigned char* other, unsigned char* s0, unsigned char* s1,
                              unsigned char* o0, unsigned char* o1) {
            if (c > 0) flush(c - 1, o1);
            if constexpr (STATER) {
                update(c, buf);
                if (c + 1 < chunks) publish(s1);
            } else {
                outputs(buf, s0, o0);
            }
            if (c + 1 < chunks) stage(st, other);
            if (c + 2 < chunks) fetch(c + 2, st);
            lds_barrier();
        };
        unsigned char* const b1 = lds + SH::kBuf;
        unsigned char* const lS1 = lS + SH::kBytesS;
        unsigned char* const lO1 = lO + SH::kBytesO;
        for (int c = 0; c < chunks; c += 2) {
            turn(c, lds, b1, lS, lS1, lO, lO1);
            if (c + 1 < chunks) turn(c + 1, b1, lds, lS1, lS, lO1, lO);
        }
        flush(chunks - 1, (chunks & 1) ? lO : lO1);
    }

    if constexpr (STATER) {
        float* const out = OUT ? (pl.last ? pl.w.carry_out : nullptr) : pl.w.segment_carry;
        if (out) {
            const int64_t square = int64_t(DA) * a.width;
            const int64_t sd = pl.w.state_d;
            float* const p = out + ((OUT ? int64_t(pl.n) : pl.carry + pl.m) * a.H + pl.hd) * square +
                             (pl.col0 + 16 * cb + l) * int64_t(pl.w.state_c);
#pragma unroll
            for (int t = 0; t < TS; ++t) store_rows4(p + (d0 + 16 * t + 4 * g) * sd, sd, X[t]);
        }
    }
}

template <typename T, int DA, int CW, bool OUT, bool EXACT>
__global__ __launch_bounds__((Shape<T, DA, CW, OUT>::kThreads)) __attribute__((amdgpu_waves_per_eu(1, 2))) void walk_kernel(LinearLaunch a)
{
    using SH = Shape<T, DA, CW, OUT>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[SH::kLds];
    if (OUT && int64_t(blockIdx.x) >= a.walk_blocks) {
        zero_padding(a, int(sizeof(T)), SH::kThreads);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63;

    // The workgroups of one (segment, head), its column slices and walks, are
    // eight blocks apart: they run at the same time on one XCD, whose L2 serves
    // the rows that they share.
    const int slices = a.width / CW, subs = slices * a.walks;
    const int64_t unit = int64_t(blockIdx.x / (8 * subs)) * 8 + (blockIdx.x & 7);
    const int sub = (blockIdx.x / 8) % subs;
    if (unit >= a.units) return;
    Place pl;
    pl.w = a.walk[sub / slices];
    pl.col0 = (sub % slices) * CW;
    pl.hd = int(unit % a.H);
    const int64_t at = unit / a.H;  // a segment (batched), a slot (packed) or a window (packed, carries)
    pl.n = !a.cu_seqlens       ? int(at / a.segments)
           : a.segments == 1 ? int(at)
                               : __builtin_amdgcn_readfirstlane(find_sequence(a.cu_seqlens, a.N, a.T, a.seg_len, OUT, int(at), lane));
    int64_t bos, eos, brow;
    sequence_bounds(a.cu_seqlens, pl.n, a.T, bos, eos, brow);
    pl.m = a.segments == 1 ? 0 : a.cu_seqlens ? int(at - (bos / a.seg_len + (OUT ? pl.n : 0))) : int(at % a.segments);
    const int64_t len = eos - bos, before = int64_t(pl.m) * a.seg_len;  // tokens walked before this segment
    if (pl.m < 0 || (pl.m > 0 && before >= len)) return;
    pl.segments = len > a.seg_len ? int((len + a.seg_len - 1) / a.seg_len) : 1;
    pl.last = len - before <= a.seg_len;
    if (!OUT && pl.last) return;                                       // no segment needs its carry
    pl.carry = a.cu_seqlens ? bos / a.seg_len : int64_t(pl.n) * a.segments;
    pl.kept = a.cu_seqlens ? a.T / a.seg_len + pl.carry : pl.carry + pl.segments - 1;  // batched: the last one's place
    pl.left = int(pl.last ? len - before : a.seg_len);
    pl.row0 = brow * a.T;
    pl.tok = pl.w.back ? eos - before : bos + before;

    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (wave >= SH::kOutWaves) return walk<T, DA, CW, OUT, EXACT, kState>(a, pl, lds, tid);
    if constexpr (OUT) {
        if (wave == 0) walk<T, DA, CW, OUT, EXACT, 0>(a, pl, lds, tid);
        else if (wave == 1) walk<T, DA, CW, OUT, EXACT, 1>(a, pl, lds, tid);
        else if (wave == 2) walk<T, DA, CW, OUT, EXACT, 2>(a, pl, lds, tid);
        else walk<T, DA, CW, OUT, EXACT, 3>(a, pl, lds, tid);
    }
}

template <typename T, int DA, int CW, bool OUT>
hipError_t launch_shape(LinearLaunch a, bool exact, hipStream_t stream)
{
    if (!OUT) a.units = a.carry_units;
    a.walk_blocks = (a.units + 7) / 8 * 8 * (a.width / CW) * a.walks;
    const int64_t blocks = a.walk_blocks + (OUT ? a.pad_blocks : 0);
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks)), block(Shape<T, DA, CW, OUT>::kThreads);
    if (exact || sizeof(T) == 4)
        hipLaunchKernelGGL((walk_kernel<T, DA, CW, OUT, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((walk_kernel<T, DA, CW, OUT, sizeof(T) == 4>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <typename T, bool OUT>
hipError_t launch_typed(const LinearLaunch& a, int da, bool exact, hipStream_t stream)
{
    const bool wide = linear_slice(a.width, da, sizeof(T) == 2) == 64;
    if (da == 32) return wide ? launch_shape<T, 32, 64, OUT>(a, exact, stream) : launch_shape<T, 32, 32, OUT>(a, exact, stream);
    if (da == 64) return wide ? launch_shape<T, 64, 64, OUT>(a, exact, stream) : launch_shape<T, 64, 32, OUT>(a, exact, stream);
    if constexpr (sizeof(T) == 2)
        if (da == 128 && wide) return launch_shape<T, 128, 64, OUT>(a, exact, stream);
    if (da == 128) return launch_shape<T, 128, 32, OUT>(a, exact, stream);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_linear_walk(const LinearLaunch& a, int da, bool carries_only, bool exact, bool bf16, hipStream_t stream)
{
    if (a.units == 0) return hipSuccess;
    if (carries_only)
        return bf16 ? launch_typed<bf16raw, false>(a, da, exact, stream) : launch_typed<float, false>(a, da, exact, stream);
    return bf16 ? launch_typed<bf16raw, true>(a, da, exact, stream) : launch_typed<float, true>(a, da, exact, stream);
}

}  // namespace gdn2
