// The step from one block of a layer to the next, for gfx950, and dropout.
//
// A block's output u joins the residual stream x through a norm, a gate, a
// scale and dropout, and the next block reads the stream through a norm of its
// own (RMS norms over the D channels of a token, rms(z) = sqrt(mean(z^2) + eps)):
//     n  = u / rms(u) * w_post                       (or u)
//     x' = x + scale * m * act(gate) * n             (m: 0, or 1 / (1 - p))
//     h  = x' / rms(x') * w_pre
// x' is rounded to the stream's type before the second norm, so h is the norm
// of what is stored and the backward pass, which reads the stored stream,
// differentiates exactly what ran.  Backward, with t the gradient of x':
//     t  = dx' + (w_pre dh - x' mean(w_pre dh x') / rms(x')^2) / rms(x')      = dx
//     c  = scale * m * t,   dgate = act'(gate) c n (summed over what shares it)
//     du = (w_post a c - u mean(w_post a c u) / rms(u)^2) / rms(u)
//     dw_pre = sum over tokens of dh x' / rms(x'),  dw_post = sum of a c u / rms(u)
// All arithmetic is FP32.  The norms' statistics are remade from u and x',
// which the backward pass reads anyway, so nothing is saved for it, the mask of
// the dropout neither.
//
// HBM-bound, one pass: a token's row is held in registers, eight channels a
// lane, by a group of lanes, a wavefront or several wavefronts (whose sums meet
// in LDS), and a workgroup walks rows with the next row's loads in flight.  The
// weights stay in registers over the rows, and so do the column sums of the
// weight gradients, which a second small kernel adds over the workgroups.
#include "block_device.hpp"

namespace gdn2 {
namespace {

// FULL: D is a multiple of 8, so every group is whole and at a 16-byte boundary.
template <typename T, typename R, int LPR, int WPR, int NI, bool FULL>
__global__ __launch_bounds__((Cover<LPR, WPR, NI>::kThreads)) void block_norm_fwd_kernel(BlockNormArgs a)
{
    using C = Cover<LPR, WPR, NI>;
    __shared__ float lds[2][16][4];
    int turn = 0;
    const int slot = row_slot<LPR, WPR, NI>(), rl = threadIdx.x % C::kRowLanes;
    const int64_t groups = (a.D + 7) / 8;
    const uint64_t offset = a.drop.offset + (a.drop.offset_device ? *a.drop.offset_device : 0);
    const bool has_u = a.u != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
    const float inv_d = 1.0f / float(a.D);
    uint32_t col[NI];
    float wp[NI][8], wr[NI][8], ch[NI][8];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        col[i] = (i * C::kRowLanes + rl) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) wp[i][j] = wr[i][j] = ch[i][j] = 1.f;
        if (post) load_weight(a.w_post, col[i], a.D, wp[i]);
        if (pre) load_weight(a.w_pre, col[i], a.D, wr[i]);
        if (a.gate_layout == kGateChannel) {
            float g[8], da;
            load_weight(static_cast<const float*>(a.gate), col[i], a.D, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) act_value(a.act, g[j], ch[i][j], da);
        }
    }
    Eight<T> nu[NI], ng[NI];
    Eight<R> nx[NI];
    float nt = 0.f;
    auto load_row = [&](int64_t row) {
        const bool live = row < a.rows;
        const int64_t at = row * a.D;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = live ? a.D - int(col[i]) : 0;
            nx[i].template load<FULL>(static_cast<const R*>(a.x) + at + col[i], n);
            if (has_u) nu[i].template load<FULL>(static_cast<const T*>(a.u) + at + col[i], n);
            if (a.gate_layout == kGateFull) ng[i].template load<FULL>(static_cast<const T*>(a.gate) + at + col[i], n);
        }
        if (a.gate_layout == kGateToken) nt = live ? load_as_f32(static_cast<const T*>(a.gate), row) : 0.f;
    };
    const int64_t step = int64_t(gridDim.x) * C::kRows;
    int64_t base = int64_t(blockIdx.x) * C::kRows;
    load_row(base + slot);
    for (; base < a.rows; base += step) {
        const int64_t row = base + slot;
        const bool live = row < a.rows;
        Eight<T> u[NI], g[NI];
        Eight<R> x[NI];
        const float tok = nt;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            u[i] = nu[i];
            g[i] = ng[i];
            x[i] = nx[i];
        }
        if (base + step < a.rows) load_row(row + step);

        float ru = 1.f;
        if (post) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float v[8];
                u[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] = fmaf(v[j], v[j], s[0]);
            }
            row_sums<LPR, WPR, 1>(s, lds, turn);
            ru = __builtin_amdgcn_rsqf(fmaf(s[0], inv_d, a.eps));
        }
        float ta = 1.f, unused;
        if (a.gate_layout == kGateToken) act_value(a.act, tok, ta, unused);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = live ? a.D - int(col[i]) : 0;
            float xv[8];
            x[i].get(xv);
            if (has_u) {
                float uv[8], gv[8];
                u[i].get(uv);
                if (a.gate_layout == kGateFull) g[i].get(gv);
                u32x4_t bits{0, 0, 0, 0};
                if (a.drop.threshold) bits = philox4x32(uint64_t(row * groups + col[i] / 8), offset, a.drop.seed);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float z = uv[j] * ru * wp[i][j] * ch[i][j] * ta;
                    if (a.gate_layout == kGateFull) {
                        float f, df;
                        act_value(a.act, gv[j], f, df);
                        z *= f;
                    }
                    if (a.drop.threshold) z = philox_keep(bits, j, a.drop.threshold) ? z * a.drop.keep : 0.f;
                    xv[j] = fmaf(a.scale, z, xv[j]);
                }
                x[i].put(xv);
                x[i].template store<FULL>(static_cast<R*>(a.x_out) + row * a.D + col[i], n);
                x[i].get(xv);  // what is stored, rounded
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += (FULL ? n > 0 : j < n) ? xv[j] * xv[j] : 0.f;
        }
        if (pre) {
            row_sums<LPR, WPR, 1>(s, lds, turn);
            const float rx = __builtin_amdgcn_rsqf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float v[8];
                x[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * rx * wr[i][j];
                Eight<T> h;
                h.put(v);
                h.template store<FULL>(static_cast<T*>(a.h) + row * a.D + col[i], live ? a.D - int(col[i]) : 0);
            }
        }
    }
}

constexpr int64_t kFwdBlocks = 2048;

template <typename T, typename R>
hipError_t fwd_typed(const BlockNormArgs& a, hipStream_t stream)
{
    const unsigned blocks = unsigned(even_blocks(a.rows, rows_at_once(a.D), kFwdBlocks));
    if (blocks == 0) return hipSuccess;
#define GDN2_FWD(LPR, WPR, NI)                                                                                     \
    do {                                                                                                           \
        if (a.D % 8 == 0)                                                                                          \
            hipLaunchKernelGGL((block_norm_fwd_kernel<T, R, LPR, WPR, NI, true>), dim3(blocks),                    \
                               dim3(Cover<LPR, WPR, NI>::kThreads), 0, stream, a);                                 \
        else                                                                                                       \
            hipLaunchKernelGGL((block_norm_fwd_kernel<T, R, LPR, WPR, NI, false>), dim3(blocks),                   \
                               dim3(Cover<LPR, WPR, NI>::kThreads), 0, stream, a);                                 \
    } while (0)
    GDN2_COVER(a.D, GDN2_FWD);
#undef GDN2_FWD
    return hipGetLastError();
}

// Dropout alone: a lane takes one block of eight elements of a row.
template <typename T, bool FULL>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutCall a, int64_t groups)
{
    const uint64_t offset = a.drop.offset + (a.drop.offset_device ? *a.drop.offset_device : 0);
    const int64_t total = a.rows * groups;
    for (int64_t b = int64_t(blockIdx.x) * 256 + threadIdx.x; b < total; b += int64_t(gridDim.x) * 256) {
        int64_t e = b * 8, n = 8;
        if (!FULL) {
            const int64_t row = b / groups, d = (b - row * groups) * 8;
            e = row * a.D + d;
            n = a.D - d < 8 ? a.D - d : 8;
        }
        Eight<T> r;
        r.template load<FULL>(static_cast<const T*>(a.x) + e, int(n));
        if (a.drop.threshold) {
            float v[8];
            r.get(v);
            const u32x4_t bits = philox4x32(uint64_t(b), offset, a.drop.seed);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = philox_keep(bits, j, a.drop.threshold) ? v[j] * a.drop.keep : 0.f;
            r.put(v);
        }
        r.template store<FULL>(static_cast<T*>(a.y) + e, int(n));
    }
}

template <typename T>
hipError_t dropout_typed(const DropoutCall& a, hipStream_t stream)
{
    const int64_t groups = (a.D + 7) / 8, need = (a.rows * groups + 255) / 256;
    if (need == 0) return hipSuccess;
    const unsigned blocks = unsigned(need < (1 << 20) ? need : (1 << 20));
    if (a.D % 8 == 0)
        hipLaunchKernelGGL((dropout_kernel<T, true>), dim3(blocks), dim3(256), 0, stream, a, groups);
    else
        hipLaunchKernelGGL((dropout_kernel<T, false>), dim3(blocks), dim3(256), 0, stream, a, groups);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm_fwd(const BlockNormArgs& a, bool bf16, bool residual_bf16, hipStream_t stream)
{
    if (!bf16) return fwd_typed<float, float>(a, stream);
    return residual_bf16 ? fwd_typed<bf16raw, bf16raw>(a, stream) : fwd_typed<bf16raw, float>(a, stream);
}

hipError_t launch_dropout(const DropoutCall& a, bool bf16, hipStream_t stream)
{
    return bf16 ? dropout_typed<bf16raw>(a, stream) : dropout_typed<float>(a, stream);
}

}  // namespace gdn2
