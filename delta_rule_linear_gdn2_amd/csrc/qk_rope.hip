// Norms of queries and keys for each head with the position rotation, and the
// gradients.
//
// A head's row x of d channels, with r = 1 / sqrt(mean(x^2) + eps):
//     n = x r weight                                (weight shared by the heads of q, or of k)
//     y = scale * rotate(n, position)               (scale: q_scale for q, 1 for k)
// rotate turns the pair i < rot / 2 of channels, (i, i + rot / 2) or (2 i, 2 i + 1),
// by the angle position * inv_freq[i]; channels from rot on stay.  Backwards,
// with xh = x r and dn = rotate(scale dy, -position):
//     d_weight = sum over tokens and heads of dn xh
//     dx = r (t - xh mean(t xh)),  t = dn weight
// (1 / rms is never raised to a power: see block_bwd.hip).
//
// Angles.  The product of a position and a frequency loses its place within a
// turn in 32 bits (2^20 x 1 has half a radian between neighbours at 2^-4 turns),
// so the turns are formed in 64 bits, position * inv_freq / 2 pi with 1 / 2 pi in
// two parts, and reduced to half a turn before sine and cosine are taken in
// FP32.  They depend on the token alone: a wavefront forms them once and serves
// all heads of the token with them.
//
// Work split.  d / 8 lanes hold a row: two groups of four channels a lane, taken
// so that both members of its four pairs are its own (halves: 4 l .. and
// rot / 2 + 4 l ..; neighbours and channels behind rot: 8 l ..).  A wavefront takes
// 512 / d heads of a token at a time.  Its lane groups share the sines: group g
// forms pair g & 3 of each lane, and four lane exchanges hand them round.
//
// What bounds it: memory.  8 x 4096 tokens of 16 + 16 heads of 128, bf16: 99 us for
// 537 MB (5.4 TB/s; a 1 GiB copy reaches 5.1), vector arithmetic in 46% of the
// cycles; backwards 151 us for 805 MB, of which the sum of the weights' gradients
// takes 5.  Calls of a few tokens take 5 us on the device, less than their host time.
#include "row_device.hpp"

namespace gdn2 {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

template <typename T>
struct Four;
template <>
struct Four<bf16raw> {
    uint2 u;
    __device__ __forceinline__ void load(const bf16raw* p) { u = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(float* v) const
    {
        v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(bf16raw* p, const float* v)
    {
        *reinterpret_cast<uint2*>(p) = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
    }
};
template <>
struct Four<float> {
    float4 u;
    __device__ __forceinline__ void load(const float* p) { u = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(float* v) const { v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w; }
    static __device__ __forceinline__ void store(float* p, const float* v)
    {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};

// Where a lane's channels are and how it turns them.
struct Lane {
    int c0, c1;      // first channels of its two groups of four
    bool turns;      // its pairs are rotated
};
__device__ __forceinline__ Lane lane_place(int l, int rot, bool neighbours)
{
    Lane p;
    p.turns = 8 * l < rot;
    const bool halves = p.turns && !neighbours;
    p.c0 = halves ? 4 * l : 8 * l;
    p.c1 = halves ? rot / 2 + 4 * l : 8 * l + 4;
    return p;
}

// Cosine and sine of the lane's four pairs at a token's position.
template <int D>
__device__ __forceinline__ void token_angles(int pos, float freq, const Lane& p, int lane, float (&c)[4], float (&s)[4])
{
    constexpr int LPH = D / 8;
    constexpr double kTurn = 0.15915494309189535, kTurnLow = -9.839338148398635e-18;  // 1 / 2 pi in two parts
    const double x = double(pos) * double(freq);
    const double whole = rint(x * kTurn);
    const float part = float(fma(x, kTurn, -whole) + x * kTurnLow);
    float mys, myc;
    sincospif(2.f * part, &mys, &myc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int from = i * LPH + (lane & (LPH - 1));
        c[i] = __shfl(myc, from, 64);
        s[i] = __shfl(mys, from, 64);
    }
}

// (v0, v1) as the two channel groups hold the pairs, turned by (c, s).
__device__ __forceinline__ void turn(float (&v)[8], const float (&c)[4], const float (&s)[4], bool neighbours)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = neighbours ? 2 * i : i, b = neighbours ? 2 * i + 1 : i + 4;
        const float x = v[a], y = v[b];
        v[a] = x * c[i] - y * s[i];
        v[b] = y * c[i] + x * s[i];
    }
}

template <typename T, int D, bool NB>
__global__ __launch_bounds__(kThreads) void qk_rope_kernel(QkRopeArgs a)
{
    constexpr int LPH = D / 8, HPW = 64 / LPH;
    const int lane = threadIdx.x & 63, l = lane & (LPH - 1), group = lane / LPH;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Lane p = lane_place(l, a.rot, NB);
    const float freq = p.turns ? a.inv_freq[4 * l + (group & 3)] : 0.f;
    float w[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = i < 4 ? p.c0 + i : p.c1 + i - 4;
        w[0][i] = (a.weight[0] ? a.weight[0][c] : 1.f) * a.q_scale;
        w[1][i] = a.weight[1] ? a.weight[1][c] : 1.f;
    }
    // a task: a token's part-th share of the head blocks of q and k
    const int bq = (a.heads[0] + HPW - 1) / HPW, blocks = bq + (a.heads[1] + HPW - 1) / HPW;
    const int64_t tasks = a.tokens * a.parts;
    for (int64_t task = int64_t(blockIdx.x) * kWaves + wave; task < tasks; task += int64_t(gridDim.x) * kWaves) {
        const int64_t tok = task / a.parts;
        const int part = int(task % a.parts);
        float c[4], s[4];
        token_angles<D>(a.positions ? a.positions[tok] : int(tok % a.T), freq, p, lane, c, s);
        for (int b = part; b < blocks; b += a.parts) {
            const bool isk = b >= bq;
            const int hd = (isk ? b - bq : b) * HPW + group, heads = isk ? a.heads[1] : a.heads[0];
            if (hd >= heads) continue;
            const T* const x = static_cast<const T*>(isk ? a.x[1] : a.x[0]) + (tok * heads + hd) * D;
            T* const y = static_cast<T*>(isk ? a.y[1] : a.y[0]) + (tok * heads + hd) * D;
            Four<T> f0, f1;
            f0.load(x + p.c0);
            f1.load(x + p.c1);
            float v[8];
            f0.get(v);
            f1.get(v + 4);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i] * v[i];
            const float r = rsqrtf(group_sum<LPH>(sum) * (1.f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * r * (isk ? w[1][i] : w[0][i]);
            if (p.turns) turn(v, c, s, NB);
            Four<T>::store(y + p.c0, v);
            Four<T>::store(y + p.c1, v + 4);
        }
    }
}

template <typename T, int D, bool NB>
__global__ __launch_bounds__(kThreads) void qk_rope_bwd_kernel(QkRopeBwdArgs a)
{
    constexpr int LPH = D / 8, HPW = 64 / LPH;
    const int lane = threadIdx.x & 63, l = lane & (LPH - 1), group = lane / LPH;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Lane p = lane_place(l, a.rot, NB);
    const float freq = p.turns ? a.inv_freq[4 * l + (group & 3)] : 0.f;
    float w[2][8], dw[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = i < 4 ? p.c0 + i : p.c1 + i - 4;
        w[0][i] = a.weight[0] ? a.weight[0][c] : 1.f;
        w[1][i] = a.weight[1] ? a.weight[1][c] : 1.f;
        dw[0][i] = dw[1][i] = 0.f;
    }
    const int bq = (a.heads[0] + HPW - 1) / HPW, blocks = bq + (a.heads[1] + HPW - 1) / HPW;
    const int64_t tasks = a.tokens * a.parts;
    for (int64_t task = int64_t(blockIdx.x) * kWaves + wave; task < tasks; task += int64_t(gridDim.x) * kWaves) {
        const int64_t tok = task / a.parts;
        const int part = int(task % a.parts);
        float c[4], s[4];
        token_angles<D>(a.positions ? a.positions[tok] : int(tok % a.T), freq, p, lane, c, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = -s[i];
        const auto row = [&](const void* xs, const void* dys, void* dxs, int heads, int hd, float scale, const float (&wt)[8],
                             float (&dwt)[8]) {
            const int64_t at = (tok * heads + hd) * D;
            const T* const x = static_cast<const T*>(xs) + at;
            const T* const dy = static_cast<const T*>(dys) + at;
            T* const dx = static_cast<T*>(dxs) + at;
            Four<T> f0, f1, g0, g1;
            f0.load(x + p.c0);
            f1.load(x + p.c1);
            g0.load(dy + p.c0);
            g1.load(dy + p.c1);
            float v[8], d[8];
            f0.get(v);
            f1.get(v + 4);
            g0.get(d);
            g1.get(d + 4);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i] * v[i];
            const float r = rsqrtf(group_sum<LPH>(sum) * (1.f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= scale;
            if (p.turns) turn(d, c, s, NB);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] *= r;
                dwt[i] += d[i] * v[i];
                d[i] *= wt[i];
                dot += d[i] * v[i];
            }
            const float mean = group_sum<LPH>(dot) * (1.f / D);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = r * (d[i] - v[i] * mean);
            Four<T>::store(dx + p.c0, d);
            Four<T>::store(dx + p.c1, d + 4);
        };
        for (int b = part; b < blocks; b += a.parts) {
            if (b < bq) {
                const int hd = b * HPW + group;
                if (hd < a.heads[0]) row(a.x[0], a.dy[0], a.dx[0], a.heads[0], hd, a.q_scale, w[0], dw[0]);
            } else {
                const int hd = (b - bq) * HPW + group;
                if (hd < a.heads[1]) row(a.x[1], a.dy[1], a.dx[1], a.heads[1], hd, 1.f, w[1], dw[1]);
            }
        }
    }
    if (!a.partial) return;
    // the workgroup's partial row: lane groups by exchange, wavefronts in turn
    __shared__ float part_row[kWaves][2 * D];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float t = dw[k][i];
#pragma unroll
            for (int off = LPH; off < 64; off *= 2) t += __shfl_xor(t, off, 64);
            if (group == 0) part_row[wave][k * D + (i < 4 ? p.c0 + i : p.c1 + i - 4)] = t;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) t += part_row[k][i];
        a.partial[int64_t(blockIdx.x) * 2 * D + i] = t;
    }
}

// Workgroups: as many as are resident at once (four wavefronts a SIMD), fewer
// for small calls (twice as many: 104 and 161 us instead of 99 and 151); a token's
// heads are shared out where the tokens alone do not fill the device (shares half or
// a quarter of these: the same).
constexpr int64_t kFull = 1024;

int rope_parts(int64_t tokens, int heads_q, int heads_k, int d)
{
    const int per = 512 / d, blocks = (heads_q + per - 1) / per + (heads_k + per - 1) / per;
    const int64_t want = tokens > 0 ? (kFull * kWaves + tokens - 1) / tokens : 1;
    return int(want < blocks ? want : blocks);
}
int64_t rope_blocks(int64_t tokens, int parts)
{
    const int64_t b = (tokens * parts + kWaves - 1) / kWaves;
    return b < kFull ? b : kFull;
}

#define GDN2_ROPE(KERNEL, T_)                                                                                          \
    do {                                                                                                               \
        const dim3 grid(static_cast<unsigned>(blocks));                                                                \
        if (a.d == 32 && a.neighbours) hipLaunchKernelGGL((KERNEL<T_, 32, true>), grid, dim3(kThreads), 0, stream, a); \
        else if (a.d == 32) hipLaunchKernelGGL((KERNEL<T_, 32, false>), grid, dim3(kThreads), 0, stream, a);           \
        else if (a.d == 64 && a.neighbours) hipLaunchKernelGGL((KERNEL<T_, 64, true>), grid, dim3(kThreads), 0, stream, a); \
        else if (a.d == 64) hipLaunchKernelGGL((KERNEL<T_, 64, false>), grid, dim3(kThreads), 0, stream, a);           \
        else if (a.d == 128 && a.neighbours) hipLaunchKernelGGL((KERNEL<T_, 128, true>), grid, dim3(kThreads), 0, stream, a); \
        else if (a.d == 128) hipLaunchKernelGGL((KERNEL<T_, 128, false>), grid, dim3(kThreads), 0, stream, a);         \
        else return hipErrorInvalidValue;                                                                              \
    } while (0)

}  // namespace

int64_t qk_rope_bwd_partials(int64_t tokens, int32_t heads_q, int32_t heads_k, int32_t d)
{
    return rope_blocks(tokens, rope_parts(tokens, heads_q, heads_k, d));
}

hipError_t launch_qk_rope(QkRopeArgs a, bool bf16, hipStream_t stream)
{
    if (a.tokens == 0) return hipSuccess;
    a.parts = rope_parts(a.tokens, a.heads[0], a.heads[1], a.d);
    const int64_t blocks = rope_blocks(a.tokens, a.parts);
    if (bf16) GDN2_ROPE(qk_rope_kernel, bf16raw);
    else GDN2_ROPE(qk_rope_kernel, float);
    return hipGetLastError();
}

hipError_t launch_qk_rope_bwd(QkRopeBwdArgs a, bool bf16, hipStream_t stream)
{
    int64_t blocks = 0;
    if (a.tokens > 0) {
        a.parts = rope_parts(a.tokens, a.heads[0], a.heads[1], a.d);
        blocks = rope_blocks(a.tokens, a.parts);
        if (bf16) GDN2_ROPE(qk_rope_bwd_kernel, bf16raw);
        else GDN2_ROPE(qk_rope_bwd_kernel, float);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.d_weight[0] && !a.d_weight[1]) return hipSuccess;
    ColumnSumArgs c{};
    c.partial = a.partial;
    c.P = blocks;
    c.width = 2 * a.d;
    c.out[0] = a.d_weight[0];
    c.out[1] = a.d_weight[1];
    c.end[0] = a.d;
    c.end[1] = c.end[2] = 2 * a.d;
    return launch_column_sum(c, stream);
}

}  // namespace gdn2
