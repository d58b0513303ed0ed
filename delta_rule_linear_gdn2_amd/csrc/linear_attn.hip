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
// wavefronts; the output wavefronts (32 tokens x 32 columns each) form
//     P^T = Y X^T (tokens j x i), masked and decayed in registers, then
//     O^T = Xs^T X^T + Z^T P^T  (columns x tokens i),
// where an accumulator tile is directly the next product's operand, because a
// matrix product does not care for the order of its inner index as long as both
// operands take the same (see Frag).  The decays of a tile are constants of the
// head: each lane keeps its own in registers for the whole walk.
//
// Precision.  bf16 inputs feed bf16 matrix products with FP32 sums.  P and the
// copy of X that the outputs read are rounded to bf16, as the outputs are (both
// far below the rounding of sums of such products to bf16 outputs: 2^-9 rms
// each); X itself is not: a^n z is split into three bf16 terms that hold all 24
// bits, so the carry is that of FP32 arithmetic.
#include "gdn2_device.hpp"
#include "launch.hpp"

namespace gdn2 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kC = kLinearChunk;

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

// LDS tiles of rows of D elements, in granules of 16 bytes whose place is
// XORed with a linear map of the row's low four bits: 16-byte reads of
// neighbouring rows at one granule, and the transposed reads below, then fall
// into different banks.
template <typename T, int D>
struct Tile {
    static constexpr int kRow = D * int(sizeof(T));
    static constexpr int kGranules = kRow / 16;
    static constexpr __host__ __device__ int swz(int row)
    {
        return kRow >= 256 ? (row ^ (((row >> 2) ^ (row >> 3)) & 1)) & 15 : kRow == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
    }
    static __device__ __forceinline__ int off(int row, int granule) { return row * kRow + ((granule ^ swz(row)) << 4); }
};

// An operand of a matrix product with 32 rows (or columns), one per lane & 31,
// and an inner index that half-wavefront h = lane >> 5 takes its own part of.
// bf16: 16 inner indices a product; FP32: 8, in four products of two.
//   rows:  inner index along the tile's rows (the natural order)
//   cols:  inner index down the tile's rows, 32 columns; order "accumulator":
//          the rows {8 g + 4 h .. + 3} that a lane holds in a 32 x 32
//          accumulator, so that `from_acc` of another tile is the other operand
template <typename T>
struct Frag;

template <>
struct Frag<bf16raw> {
    static constexpr int kInner = 16;
    bf16x8 x;
    template <int D>
    static __device__ __forceinline__ Frag rows(const unsigned char* tile, int row, int s, int h)
    {
        return {__builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(tile + Tile<bf16raw, D>::off(row, 2 * s + h)))};
    }
    // In each group of 16 lanes the transposing load takes four rows of 16
    // columns: lane 4 r + c reads columns 4 c .. + 3 of row r, and lane l
    // receives column l of the four rows.
    template <int D>
    static __device__ __forceinline__ Frag cols(const unsigned char* tile, int col0, int s, int lane)
    {
        const int h = lane >> 5, c = col0 + (lane & 16) + 4 * (lane & 3), r = 4 * h + ((lane & 15) >> 2);
        using TL = Tile<bf16raw, D>;
        const int lo = TL::off(16 * s + r, c >> 3) + ((c & 4) << 1), hi = TL::off(16 * s + 8 + r, c >> 3) + ((c & 4) << 1);
        const v4i16 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(tile + lo));
        const v4i16 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(tile + hi));
        return {__builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7))};
    }
    static __device__ __forceinline__ Frag from_acc(const f32x16& p, int s)
    {
        const uint4 u = {pack2(p[8 * s], p[8 * s + 1]), pack2(p[8 * s + 2], p[8 * s + 3]), pack2(p[8 * s + 4], p[8 * s + 5]),
                         pack2(p[8 * s + 6], p[8 * s + 7])};
        return {__builtin_bit_cast(bf16x8, u)};
    }
    __device__ __forceinline__ f32x16 times(const Frag& b, f32x16 c) const
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, b.x, c, 0, 0, 0);
    }
    // this^T (b scaled): b's elements times `scale` as three bf16 terms, each the
    // upper 16 bits of what the ones before leave.
    __device__ __forceinline__ static void split(const Frag& b, const float* scale, Frag (&out)[3])
    {
        const uint4 u = __builtin_bit_cast(uint4, b.x);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t t[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo = __uint_as_float(w[i] << 16) * scale[2 * i], hi = __uint_as_float(w[i] & 0xffff0000u) * scale[2 * i + 1];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t ul = __float_as_uint(lo), uh = __float_as_uint(hi);
                t[k][i] = __builtin_amdgcn_perm(uh, ul, 0x07060302);  // the upper halves
                if (k < 2) {
                    lo -= __uint_as_float(ul & 0xffff0000u);
                    hi -= __uint_as_float(uh & 0xffff0000u);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) out[k].x = __builtin_bit_cast(bf16x8, make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]));
    }
    static constexpr int kTerms = 3;
};

template <>
struct Frag<float> {
    static constexpr int kInner = 8;
    f32x4 x;
    template <int D>
    static __device__ __forceinline__ Frag rows(const unsigned char* tile, int row, int s, int h)
    {
        return {*reinterpret_cast<const f32x4*>(tile + Tile<float, D>::off(row, 2 * s + h))};
    }
    template <int D>
    static __device__ __forceinline__ Frag cols(const unsigned char* tile, int col0, int s, int lane)
    {
        const int c = col0 + (lane & 31), r = 8 * s + 4 * (lane >> 5);
        Frag f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f.x[e] = *reinterpret_cast<const float*>(tile + Tile<float, D>::off(r + e, c >> 2) + ((c & 3) << 2));
        return f;
    }
    static __device__ __forceinline__ Frag from_acc(const f32x16& p, int s)
    {
        return {f32x4{p[4 * s], p[4 * s + 1], p[4 * s + 2], p[4 * s + 3]}};
    }
    __device__ __forceinline__ f32x16 times(const Frag& b, f32x16 c) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], b.x[e], c, 0, 0, 0);
        return c;
    }
    __device__ __forceinline__ static void split(const Frag& b, const float* scale, Frag (&out)[1])
    {
        out[0].x = f32x4{b.x[0] * scale[0], b.x[1] * scale[1], b.x[2] * scale[2], b.x[3] * scale[3]};
    }
    static constexpr int kTerms = 1;
};

// The row of a 32 x 32 accumulator that element r of a lane in half h holds.
__device__ __forceinline__ int acc_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// Four consecutive elements into LDS.
__device__ __forceinline__ void put4(unsigned char* p, const float* v, bf16raw*)
{
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void put4(unsigned char* p, const float* v, float*)
{
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
}

// 32 columns (rows of the accumulator) of one token: lane's 16 values to global
// memory.  bf16: the two halves exchange groups of four, so that each lane stores
// 16 contiguous bytes.
__device__ __forceinline__ void store_row(rsrc_t r, uint32_t off, const f32x16& o, int h, bf16raw*)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2(o[2 * i], o[2 * i + 1]);
    // groups g = 0..3 hold columns 8 g + 4 h .. + 3 (two words): lower half ends
    // with columns 16 j .. + 7, upper half with 16 j + 8 .. + 15
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const auto a = __builtin_amdgcn_permlane32_swap(w[4 * j], w[4 * j + 2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[4 * j + 1], w[4 * j + 3], false, false);
        typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
        const u32x4 v = {a[0], b[0], a[1], b[1]};
        __builtin_amdgcn_raw_buffer_store_b128(v, r, int(off + 32 * j + 16 * h), 0, 0);
    }
}
__device__ __forceinline__ void store_row(rsrc_t r, uint32_t off, const f32x16& o, int h, float*)
{
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const u32x4 v = {__float_as_uint(o[4 * g]), __float_as_uint(o[4 * g + 1]), __float_as_uint(o[4 * g + 2]),
                         __float_as_uint(o[4 * g + 3])};
        __builtin_amdgcn_raw_buffer_store_b128(v, r, int(off + 32 * g + 16 * h), 0, 0);
    }
}

// alpha as the other kernels take it: in [2^-15, 1], NaN as 2^-15.
__device__ __forceinline__ double log2_alpha(float alpha)
{
    return log2(double(fminf(fmaxf(alpha, 0x1p-15f), 1.0f)));
}

// Segment m of sequence n in [0, slots): slot = start / seg_len + n + m, which
// is distinct for distinct segments of offsets that do not decrease, and below
// T / seg_len + N for any.  Finds n: the last sequence whose first slot is not
// above `slot`.
__device__ __forceinline__ int slot_sequence(const int32_t* cu, int N, int T, int seg_len, int slot, int lane)
{
    int n = 0;
    for (int base = 0; base < N; base += 64) {
        const int i = base + lane;
        int at = 0x7fffffff;
        if (i < N) {
            int b = cu[i];
            b = b < 0 ? 0 : b > T ? T : b;
            at = b / seg_len + i;
        }
        n += __popcll(__ballot(at <= slot));
    }
    return n > 0 ? n - 1 : 0;
}

template <typename T, int DA, int CW, bool OUT>
struct Shape {
    static constexpr int kOutWaves = OUT ? 2 * (CW / 32) : 0;
    static constexpr int kStateTiles = (DA / 32) * (CW / 32);
    static constexpr int kStateWaves = kStateTiles < 4 ? kStateTiles : 4;
    static constexpr int kTiles = kStateTiles / kStateWaves;  // 32 x 32 tiles of X a state wavefront
    static constexpr int kThreads = 64 * (kOutWaves + kStateWaves);
    static constexpr int kBytesXY = kC * DA * int(sizeof(T)), kBytesZ = kC * CW * int(sizeof(T));
    static constexpr int kOffY = 0, kOffZ = kBytesXY, kOffX = kOffZ + kBytesZ;
    static constexpr int kOffS = kOffX + (OUT ? kBytesXY : 0);
    static constexpr int kOffPow = kOffS + (OUT ? CW * DA * int(sizeof(T)) : 0);
    static constexpr int kLds = kOffPow + 80 * 4;
};

// One thread's granules of a chunk's tile of `rows` of D elements.
template <typename T, int D, int THREADS>
struct Stage {
    static constexpr int kG = Tile<T, D>::kGranules, kTotal = kC * kG, kN = (kTotal + THREADS - 1) / THREADS;
    uint4 v[kN];
    __device__ __forceinline__ void load(rsrc_t r, uint32_t stride, int L, bool back, int tid)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int g = tid + i * THREADS;
            if (kTotal % THREADS && g >= kTotal) break;
            const int row = g / kG;
            const uint32_t off = uint32_t(back ? L - 1 - row : row) * stride + uint32_t(g % kG) * 16;
            // a row behind the last one (before the first one, walking back) is past the window
            const auto x = __builtin_amdgcn_raw_buffer_load_b128(r, int(row < L ? off : 0x80000000u), 0, 0);
            v[i] = make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
    __device__ __forceinline__ void store(unsigned char* tile, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int g = tid + i * THREADS;
            if (kTotal % THREADS && g >= kTotal) break;
            *reinterpret_cast<uint4*>(tile + Tile<T, D>::off(g / kG, g % kG)) = v[i];
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

// What every wavefront of a workgroup knows of its walk.
struct Place {
    LinearWalk w;
    int n, m, segments, hd, col0;  // segment m of sequence n's `segments`
    int64_t slot, row0, tok;  // tok: forwards the next token, backwards the one behind it
    int left;                 // tokens to walk
    bool last;                // the sequence's last segment
};

// The chunks of a walk as one wavefront sees them: every wavefront stages its
// share of the tiles; state wavefronts (STATER) keep X, the others form outputs.
template <typename T, int DA, int CW, bool OUT, bool STATER>
__device__ __forceinline__ void walk(const LinearLaunch& a, Place pl, unsigned char* lds, int tid)
{
    using SH = Shape<T, DA, CW, OUT>;
    using F = Frag<T>;
    constexpr int NT = SH::kThreads, EB = int(sizeof(T)), CB = CW / 32, TS = SH::kTiles;
    constexpr int kSteps = kC / F::kInner, kPer = F::kInner / 2;   // inner indices a lane takes a step
    unsigned char* const lY = lds + SH::kOffY;
    unsigned char* const lZ = lds + SH::kOffZ;
    unsigned char* const lX = lds + SH::kOffX;
    unsigned char* const lS = lds + SH::kOffS;
    float* const pw = reinterpret_cast<float*>(lds + SH::kOffPow);
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const bool back = pl.w.back;
    const int late = back ? 1 : 0;

    const float al = a.alpha[pl.hd];
    for (int i = tid; i <= kC; i += NT) pw[i] = float(exp2(log2_alpha(al) * i));

    const uint32_t strideA = uint32_t(a.H) * DA * EB, strideZ = uint32_t(a.H) * a.width * EB;
    const char* const px = static_cast<const char*>(pl.w.x) + (pl.row0 * a.H + pl.hd) * DA * EB;
    const char* const py = static_cast<const char*>(pl.w.y) + (pl.row0 * a.H + pl.hd) * DA * EB;
    const int64_t zoff = ((pl.row0 * a.H + pl.hd) * a.width + pl.col0) * EB;
    const char* const pz = static_cast<const char*>(pl.w.z) + zoff;

    Stage<T, DA, NT> sx, sy;
    Stage<T, CW, NT> sz;
    const auto fetch = [&](int64_t t0, int n) {
        const rsrc_t ry = make_rsrc(py + t0 * strideA, uint32_t(n - 1) * strideA + DA * EB);
        const rsrc_t rz = make_rsrc(pz + t0 * strideZ, uint32_t(n - 1) * strideZ + CW * EB);
        sy.load(ry, strideA, n, back, tid);
        sz.load(rz, strideZ, n, back, tid);
        if (OUT) {
            const rsrc_t rx = make_rsrc(px + t0 * strideA, uint32_t(n - 1) * strideA + DA * EB);
            sx.load(rx, strideA, n, back, tid);
        }
    };
    int64_t tok = pl.tok;
    int left = pl.left, L = left < kC ? left : kC;
    if (left > 0) fetch(back ? tok - L : tok, L);
    lds_barrier();  // pw

    const int sw = wave - SH::kOutWaves;
    const int ih = wave & 1, cb = STATER ? sw % CB : wave >> 1, db0 = STATER ? sw / CB * TS : 0;

    // Constants of the head: output wavefronts hold the decays of their diagonal
    // and lower tile and of the carry's read, state wavefronts those of their z.
    float dec[2][16], read = 0.f, scale[kSteps * kPer];
    const auto scales = [&](int n) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int j = s * F::kInner + 8 * (e >> 2) + 4 * h + (e & 3), at = n - 1 + late - j;
                scale[s * kPer + e] = pw[at < 0 ? 0 : at];
            }
    };
    f32x16 X[TS];
    if constexpr (!STATER) {
        const int i = lane & 31;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int j = acc_row(r, h);
            dec[0][r] = pw[i >= j ? i - j : 0];
            dec[1][r] = pw[32 + i - j];
        }
        read = pw[32 * ih + i + 1 - late];
    } else {
        scales(L);
        // the carry: what comes in, or the segments before this one in order
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) X[t][r] = 0.f;
        const int64_t sd = pl.w.state_d, square = int64_t(DA) * a.width;
        const int64_t c = (pl.col0 + 32 * cb + (lane & 31)) * int64_t(pl.w.state_c);
        if (pl.w.carry_in && pl.m == 0) {
            // Where there are several segments, the launch for carries leaves what comes in
            // in the slot of the last one, which has no carry to keep: the last segment may
            // write the final carry over it while the first still has to read it.
            const bool kept = OUT && pl.segments > 1;
            const float* p = kept ? pl.w.segment_carry + ((pl.slot + pl.segments - 1) * a.H + pl.hd) * square + c
                                  : pl.w.carry_in + (int64_t(pl.n) * a.H + pl.hd) * square + c;
            float* const keep = OUT ? nullptr : pl.w.segment_carry + ((pl.slot + pl.segments - 1) * a.H + pl.hd) * square + c;
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t at = (32 * (db0 + t) + acc_row(r, h)) * sd;
                    X[t][r] = p[at];
                    if (!OUT) keep[at] = X[t][r];
                }
        }
        if (OUT && pl.m > 0) {
            const float over = float(exp2(log2_alpha(al) * a.seg_len));
            const float* p = pl.w.segment_carry + ((pl.slot - pl.m) * a.H + pl.hd) * square + c;
            for (int j = 0; j < pl.m; ++j, p += a.H * square)
#pragma unroll
                for (int t = 0; t < TS; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) X[t][r] = over * X[t][r] + p[(32 * (db0 + t) + acc_row(r, h)) * sd];
        }
    }

    while (left > 0) {
        sy.store(lY, tid);
        sz.store(lZ, tid);
        if (OUT) sx.store(lX, tid);
        if constexpr (OUT && STATER) {
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int d = 32 * (db0 + t) + 8 * g + 4 * h, per = 16 / EB;
                    const float v[4] = {X[t][4 * g], X[t][4 * g + 1], X[t][4 * g + 2], X[t][4 * g + 3]};
                    put4(lS + Tile<T, DA>::off(32 * cb + (lane & 31), d / per) + (d % per) * EB, v, static_cast<T*>(nullptr));
                }
        }
        const int L1 = left - L < kC ? left - L : kC;
        const int64_t t0 = back ? tok - L : tok, t1 = back ? t0 - L1 : t0 + L;
        if (L1 > 0) fetch(t1, L1);
        lds_barrier();
        if constexpr (!STATER) {
            F xf[DA / F::kInner];
            f32x16 o;
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] = 0.f;
#pragma unroll
            for (int s = 0; s < DA / F::kInner; ++s) {
                xf[s] = F::template rows<DA>(lX, 32 * ih + (lane & 31), s, h);
                o = F::template rows<DA>(lS, 32 * cb + (lane & 31), s, h).times(xf[s], o);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] *= read;
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
                if (jb > ih) break;
                f32x16 p;
#pragma unroll
                for (int r = 0; r < 16; ++r) p[r] = 0.f;
#pragma unroll
                for (int s = 0; s < DA / F::kInner; ++s)
                    p = F::template rows<DA>(lY, 32 * jb + (lane & 31), s, h).times(xf[s], p);
                if (jb == ih) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) p[r] = acc_row(r, h) <= (lane & 31) ? p[r] * dec[0][r] : 0.f;
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) p[r] *= dec[1][r];
                }
#pragma unroll
                for (int s = 0; s < 32 / F::kInner; ++s)
                    o = F::template cols<CW>(lZ, 32 * cb, 32 / F::kInner * jb + s, lane).times(F::from_acc(p, s), o);
            }
            const rsrc_t ro = make_rsrc(static_cast<char*>(pl.w.out) + zoff + t0 * strideZ, uint32_t(L - 1) * strideZ + CW * EB);
            const int i = 32 * ih + (lane & 31);
            const uint32_t off = i < L ? uint32_t(back ? L - 1 - i : i) * strideZ + 32 * cb * EB : 0x80000000u;
            store_row(ro, off, o, h, static_cast<T*>(nullptr));
        } else {
            if (L < kC) scales(L);
            const float over = pw[L];
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) X[t][r] *= over;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                F z[F::kTerms];
                F::split(F::template cols<CW>(lZ, 32 * cb, s, lane), scale + s * kPer, z);
#pragma unroll
                for (int t = 0; t < TS; ++t) {
                    const F y = F::template cols<DA>(lY, 32 * (db0 + t), s, lane);
#pragma unroll
                    for (int k = F::kTerms - 1; k >= 0; --k) X[t] = y.times(z[k], X[t]);
                }
            }
        }
        lds_barrier();
        tok = back ? t0 : t0 + L;
        left -= L;
        L = L1;
    }

    if constexpr (STATER) {
        float* const out = OUT ? (pl.last ? pl.w.carry_out : nullptr) : pl.w.segment_carry;
        if (out) {
            const int64_t square = int64_t(DA) * a.width;
            float* p = out + ((OUT ? int64_t(pl.n) : pl.slot) * a.H + pl.hd) * square +
                       (pl.col0 + 32 * cb + (lane & 31)) * int64_t(pl.w.state_c);
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) p[(32 * (db0 + t) + acc_row(r, h)) * int64_t(pl.w.state_d)] = X[t][r];
        }
    }
}

template <typename T, int DA, int CW, bool OUT>
__global__ __launch_bounds__((Shape<T, DA, CW, OUT>::kThreads)) void walk_kernel(LinearLaunch a)
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
    pl.slot = unit / a.H;
    pl.n = !a.cu_seqlens       ? int(pl.slot / a.segments)
           : a.segments == 1 ? int(pl.slot)
                               : __builtin_amdgcn_readfirstlane(slot_sequence(a.cu_seqlens, a.N, a.T, a.seg_len, int(pl.slot), lane));
    int64_t bos, eos, brow;
    sequence_bounds(a.cu_seqlens, pl.n, a.T, bos, eos, brow);
    pl.m = a.segments == 1 ? 0 : a.cu_seqlens ? int(pl.slot - (bos / a.seg_len + pl.n)) : int(pl.slot % a.segments);
    const int64_t len = eos - bos, before = int64_t(pl.m) * a.seg_len;  // tokens walked before this segment
    if (pl.m < 0 || (pl.m > 0 && before >= len)) return;
    pl.segments = len > a.seg_len ? int((len + a.seg_len - 1) / a.seg_len) : 1;
    pl.last = len - before <= a.seg_len;
    if (!OUT && pl.last) return;                                       // no segment needs its carry
    pl.left = int(pl.last ? len - before : a.seg_len);
    pl.row0 = brow * a.T;
    pl.tok = pl.w.back ? eos - before : bos + before;

    if (__builtin_amdgcn_readfirstlane(tid >> 6) < SH::kOutWaves)
        walk<T, DA, CW, OUT, false>(a, pl, lds, tid);
    else
        walk<T, DA, CW, OUT, true>(a, pl, lds, tid);
}

template <typename T, int DA, int CW, bool OUT>
hipError_t launch_shape(LinearLaunch a, hipStream_t stream)
{
    a.walk_blocks = (a.units + 7) / 8 * 8 * (a.width / CW) * a.walks;
    const int64_t blocks = a.walk_blocks + (OUT ? a.pad_blocks : 0);
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((walk_kernel<T, DA, CW, OUT>), dim3(unsigned(blocks)), dim3(Shape<T, DA, CW, OUT>::kThreads), 0, stream, a);
    return hipGetLastError();
}

template <typename T, bool OUT>
hipError_t launch_typed(const LinearLaunch& a, int da, hipStream_t stream)
{
    const bool wide = a.width % 64 == 0;
    if (da == 32) return wide ? launch_shape<T, 32, 64, OUT>(a, stream) : launch_shape<T, 32, 32, OUT>(a, stream);
    if (da == 64) return wide ? launch_shape<T, 64, 64, OUT>(a, stream) : launch_shape<T, 64, 32, OUT>(a, stream);
    if (da == 128) return wide ? launch_shape<T, 128, 64, OUT>(a, stream) : launch_shape<T, 128, 32, OUT>(a, stream);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_linear_walk(const LinearLaunch& a, int da, bool carries_only, bool bf16, hipStream_t stream)
{
    if (a.units == 0) return hipSuccess;
    if (carries_only) return bf16 ? launch_typed<bf16raw, false>(a, da, stream) : launch_typed<float, false>(a, da, stream);
    return bf16 ? launch_typed<bf16raw, true>(a, da, stream) : launch_typed<float, true>(a, da, stream);
}

}  // namespace gdn2
