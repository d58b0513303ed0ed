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
// Forward: HBM-bound, one pass.  A token's row is held in registers, eight or
// sixteen channels a lane, by a group of lanes, a wavefront or several (whose sums
// meet in LDS); a workgroup walks rows with the next row's loads in flight and the
// weights in registers.  32768 x 2048 bf16 with an FP32 stream, full gate and
// dropout: 176 us, 940 MB at 5.3 TB/s, with no byte beyond inputs and outputs (a
// large copy reaches 5.1).  One decode row: 3 us on the device, 9 us a call.
//
// Dropout alone: 40 us for 32768 x 2048 bf16.
#include "block_device.hpp"

namespace gdn2 {
namespace {

// Wavefronts per SIMD that the register budget is set for; a launch is as many
// workgroups as are resident with it, so that each walks the same number of rows.
// Four where a lane holds eight channels (32768 x 2048 bf16 with an FP32 stream, in
// four such wavefronts a row: 190 us with 2048 workgroups, 178 with the 1024 that are
// resident, and 183, 185 and 186 at five, six and seven a SIMD).  Two wavefronts of
// sixteen a row, the cover of those rows now, take registers for two a SIMD: 512
// workgroups, 176 us.  Sixteen wavefronts are a workgroup of four a SIMD anyway, and
// above 8192 channels their 128 registers spill (36 to 252 bytes a lane, in all but
// whole bf16 rows with a bf16 stream).  FP32 ragged rows of 2049 to 4096 spill 52.
constexpr int fwd_waves_per_simd(int WPR, int NI)
{
    return NI == 1 || WPR == 16 ? 4 : WPR == 4 ? 3 : 2;
}

template <typename T, typename R, int LPR, int WPR, int NI, int MODE>
__global__ __launch_bounds__((Cover<LPR, WPR, NI>::kThreads), (fwd_waves_per_simd(WPR, NI))) void block_norm_fwd_kernel(BlockNormArgs a)
{
    using C = Cover<LPR, WPR, NI>;
    __shared__ float lds[2][16][4];
    int turn = 0;
    const int slot = row_slot<LPR, WPR, NI>(), rl = threadIdx.x % C::kRowLanes;
    const int64_t groups = (a.D + 7) / 8;
    const uint64_t offset = a.drop.offset + (a.drop.offset_device ? *a.drop.offset_device : 0);
    const bool has_u = a.u != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
    const float inv_d = 1.0f / float(a.D);
    const float factor = a.drop.threshold ? a.scale * a.drop.keep : a.scale;
    Group<MODE> grp[NI];
    float wp[NI][8], wr[NI][8];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        grp[i].init((i * C::kRowLanes + rl) * 8, a.D);
        load_weight<MODE>(a.w_post, grp[i], a.D, wp[i]);
        load_weight<MODE>(a.w_pre, grp[i], a.D, wr[i]);
        if (a.gate_layout == kGateChannel) {  // a second weight of the branch
            float g[8], f[8], df[8];
            load_weight<MODE>(static_cast<const float*>(a.gate), grp[i], a.D, g);
            act_values(a.act, g, f, df);
#pragma unroll
            for (int j = 0; j < 8; ++j) wp[i][j] *= f[j];
        }
    }
    // The next row's loads: at the start of a row, into registers of their own,
    // or, for whole rows with four wavefronts a SIMD, when this row's x' is made,
    // into the registers that it frees.
    constexpr bool kEarly = MODE != kWhole || NI > 1;
    Eight<T> nu[NI], ng[NI];
    Eight<R> nx[NI];
    float ntok = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        nu[i].clear();
        ng[i].clear();
        nx[i].clear();
    }
    auto load_row = [&](int64_t row) {
        const bool live = row < a.rows, last = row >= a.rows - 1;
        const int64_t at = row * a.D;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (has_u) grp[i].load(nu[i], static_cast<const T*>(a.u) + at, a.D, live, last);
            if (a.gate_layout == kGateFull) grp[i].load(ng[i], static_cast<const T*>(a.gate) + at, a.D, live, last);
            grp[i].load(nx[i], static_cast<const R*>(a.x) + at, a.D, live, last);
        }
        if (a.gate_layout == kGateToken) ntok = live ? load_as_f32(static_cast<const T*>(a.gate), row) : 0.f;
    };
    const int64_t step = int64_t(gridDim.x) * C::kRows;
    int64_t base = int64_t(blockIdx.x) * C::kRows;
    load_row(base + slot);
    for (; base < a.rows; base += step) {
        const int64_t row = base + slot;
        const bool live = row < a.rows, last = row >= a.rows - 1;
        Eight<T> u[NI], g[NI];
        Eight<R> x[NI];
        const float tok = ntok;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            u[i] = nu[i];
            g[i] = ng[i];
            x[i] = nx[i];
        }
        if (kEarly && base + step < a.rows) load_row(row + step);

        float ru = 1.f;
        if (post) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float v[8];
                grp[i].settle(u[i], a.D, last);
                u[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] = fmaf(v[j], v[j], s[0]);
            }
            row_sums<LPR, WPR, 1>(s, lds, turn);
            ru = __builtin_amdgcn_rsqf(fmaf(s[0], inv_d, a.eps));
        }
        if (a.gate_layout == kGateToken) {
            float f[8], df[8], g8[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) g8[j] = tok;
            act_values(a.act, g8, f, df);
            ru *= f[0];
        }
        float s[1] = {0.f};
        Eight<R> xo[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            float xv[8];
            grp[i].settle(x[i], a.D, last);
            xo[i] = x[i];
            x[i].get(xv);
            if (has_u) {
                float z[8];
                if (!post) grp[i].settle(u[i], a.D, last);
                u[i].get(z);
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] *= ru * wp[i][j];
                if (a.gate_layout == kGateFull) {
                    float gv[8], f[8], df[8];
                    grp[i].settle(g[i], a.D, last);
                    g[i].get(gv);
                    act_values(a.act, gv, f, df);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] *= f[j];
                }
                if (a.drop.threshold) {
                    const u32x4_t bits = philox4x32(uint64_t(row * groups + grp[i].col / 8), offset, a.drop.seed);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] = philox_keep(bits, j, a.drop.threshold) ? z[j] : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) xv[j] = fmaf(factor, z[j], xv[j]);
                xo[i].put(xv);
                grp[i].store(xo[i], static_cast<R*>(a.x_out) + row * a.D, a.D, live);
                xo[i].get(xv);  // what is stored, rounded
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += grp[i].has(j, a.D, live) ? xv[j] * xv[j] : 0.f;
        }
        if (!kEarly && base + step < a.rows) load_row(row + step);
        if (pre) {
            row_sums<LPR, WPR, 1>(s, lds, turn);
            const float rx = __builtin_amdgcn_rsqf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float v[8];
                xo[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * rx * wr[i][j];
                Eight<T> h;
                h.put(v);
                grp[i].store(h, static_cast<T*>(a.h) + row * a.D, a.D, live);
            }
        }
    }
}

template <typename T, typename R>
hipError_t fwd_typed(const BlockNormArgs& a, hipStream_t stream)
{
    int at_once = 1, resident = 1;
#define GDN2_PLAN(LPR, WPR, NI, MODE)          \
    at_once = Cover<LPR, WPR, NI>::kRows,      \
    resident = kSimds * fwd_waves_per_simd(WPR, NI) / Cover<LPR, WPR, NI>::kWaves
    GDN2_COVER(a.D, GDN2_PLAN);
#undef GDN2_PLAN
    const unsigned blocks = unsigned(even_blocks(a.rows, at_once, resident));
    if (blocks == 0) return hipSuccess;
#define GDN2_FWD(LPR, WPR, NI, MODE)                                                          \
    hipLaunchKernelGGL((block_norm_fwd_kernel<T, R, LPR, WPR, NI, MODE>), dim3(blocks),       \
                       dim3(Cover<LPR, WPR, NI>::kThreads), 0, stream, a)
    GDN2_COVER(a.D, GDN2_FWD);
#undef GDN2_FWD
    return hipGetLastError();
}

// Dropout alone: a lane takes one block of eight elements of a row.
template <typename T, int MODE>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutCall a, int64_t groups)
{
    const uint64_t offset = a.drop.offset + (a.drop.offset_device ? *a.drop.offset_device : 0);
    const int64_t total = a.rows * groups;
    const int rest = int(a.D % 8);  // elements of a row's last, short group
    for (int64_t b = int64_t(blockIdx.x) * 256 + threadIdx.x; b < total; b += int64_t(gridDim.x) * 256) {
        const int64_t row = MODE == kWhole ? 0 : b / groups, d = (b - row * groups) * 8;
        const int64_t e = row * a.D + d;
        const bool whole = MODE == kWhole || d + 8 <= a.D;
        const T* x = static_cast<const T*>(a.x) + e;
        T* y = static_cast<T*>(a.y) + e;
        Eight<T> r;
        if (MODE == kWhole) {
            r.load(x);
        } else if (MODE == kRagged) {
            r.load_any(x - (whole ? 0 : 8 - rest));
            if (!whole) r.shift(8 - rest);
        } else {
            r.load_pieces(x, rest);
        }
        if (a.drop.threshold) {
            float v[8];
            r.get(v);
            const u32x4_t bits = philox4x32(uint64_t(b), offset, a.drop.seed);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = philox_keep(bits, j, a.drop.threshold) ? v[j] * a.drop.keep : 0.f;
            r.put(v);
        }
        if (MODE == kWhole) r.store(y);
        else if (whole) r.store_any(y);
        else r.store_pieces(y, rest);
    }
}

template <typename T>
hipError_t dropout_typed(const DropoutCall& a, hipStream_t stream)
{
    const int64_t groups = (a.D + 7) / 8, need = (a.rows * groups + 255) / 256;
    if (need == 0) return hipSuccess;
    const dim3 blocks(unsigned(need < (1 << 20) ? need : (1 << 20))), threads(256);
    switch (row_mode(a.D)) {
        case kWhole: hipLaunchKernelGGL((dropout_kernel<T, kWhole>), blocks, threads, 0, stream, a, groups); break;
        case kRagged: hipLaunchKernelGGL((dropout_kernel<T, kRagged>), blocks, threads, 0, stream, a, groups); break;
        default: hipLaunchKernelGGL((dropout_kernel<T, kTiny>), blocks, threads, 0, stream, a, groups);
    }
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
