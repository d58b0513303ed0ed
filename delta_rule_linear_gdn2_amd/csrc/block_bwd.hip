// Gradients of the step from one block of a layer to the next (formulas:
// block.hip), for gfx950.
//
// 16 bytes of HBM an element (bf16, full gate) and about 61 vector instructions
// (15 of them the dropout, 12 the gate): at 32768 x 2048 HBM bounds it (208 to 214 us
// a call, 1.08 GB, the rate of a large copy), in rows that leave lanes idle the
// instructions do (24424 rows of 1371: 129 us, 82% of that rate).  So a row is read
// once and held in registers: the stream's side (x', dh, dx') makes t, and its
// registers take the next row's loads while the block's side (u, gate) is worked
// on, and the other way round, so the next row is always on its way without a
// second set of registers.  Two sums over the row, one barrier each where it
// spans wavefronts.  The weights' column sums stay in registers over all rows of
// a workgroup.
//
// A norm's gradient is taken as (w dh - x (mean(w dh x) / rms / rms)) / rms, 1 / rms
// going in factor by factor: its cube leaves the FP32 range for rows past 1e12 (and
// below 1e-12, with an eps as small) though the gradient does not.
#include "block_device.hpp"

namespace gdn2 {
namespace {

// Wavefronts per SIMD that the register budget is set for: three (168 registers)
// where a lane holds eight channels, two (256) at sixteen; sixteen wavefronts
// are a workgroup of four a SIMD anyway, and above 8192 channels their 128 registers
// spill 344 to 488 bytes a lane.  Rows under eight elements spill up to 156 without a
// channel gate.
constexpr int bwd_waves_per_simd(int WPR, int NI) { return NI == 1 ? 3 : WPR == 16 ? 4 : 2; }

// The backward pass's covers: three wavefronts for rows of 1025 to 1536 channels,
// whose four would idle a third of their lanes and then bound it by its vector
// instructions (24424 rows of 1371, bf16, gate and dropout: 150 us with four, 131
// with three; 24385 of 1376: 138 and 116).  The forward pass, with fewer of them,
// is faster with four.
#define GDN2_BWD_COVER(D, F)                             \
    do {                                                 \
        if ((D) <= 1024 || (D) > 1536) GDN2_COVER(D, F); \
        else if (row_mode(D) == kWhole) F(64, 3, 1, kWhole); \
        else F(64, 3, 1, kRagged);                       \
    } while (0)

// CHANNEL: the gate is one value per channel, whose gradient is a third column
// sum (without it those registers are free).  MODE: how rows lie.
template <typename T, typename R, int LPR, int WPR, int NI, int MODE, bool CHANNEL>
__global__ __launch_bounds__((Cover<LPR, WPR, NI>::kThreads), (bwd_waves_per_simd(WPR, NI))) void block_norm_bwd_kernel(BlockNormBwdArgs a)
{
    using C = Cover<LPR, WPR, NI>;
    __shared__ float lds[2][16][4];
    __shared__ float cols[C::kRows > 1 ? C::kWaves : 1][C::kRows > 1 ? 64 * 8 : 1];
    int turn = 0;
    const int slot = row_slot<LPR, WPR, NI>(), rl = threadIdx.x % C::kRowLanes;
    const int64_t groups = (a.D + 7) / 8;
    const uint64_t offset = a.drop.offset + (a.drop.offset_device ? *a.drop.offset_device : 0);
    const bool has_u = a.u != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
    const bool has_dx = a.d_x_out != nullptr, full_gate = !CHANNEL && a.gate_layout == kGateFull,
               token_gate = !CHANNEL && a.gate_layout == kGateToken;
    const bool reads_u = has_u && (post || a.gate_layout != kGateNone);
    const float inv_d = 1.0f / float(a.D);
    const float factor = a.drop.threshold ? a.scale * a.drop.keep : a.scale;
    Group<MODE> grp[NI];
    float wp[NI][8], wr[NI][8], ch[NI][8], acc_post[NI][8], acc_pre[NI][8], acc_gate[NI][8];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        grp[i].init((i * C::kRowLanes + rl) * 8, a.D);
        load_weight<MODE>(a.w_post, grp[i], a.D, wp[i]);
        load_weight<MODE>(a.w_pre, grp[i], a.D, wr[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc_post[i][j] = acc_pre[i][j] = acc_gate[i][j] = 0.f;
        if (CHANNEL) {
            float gv[8], df[8];
            load_weight<MODE>(static_cast<const float*>(a.gate), grp[i], a.D, gv);
            act_values(a.act, gv, ch[i], df);
        }
    }
    Eight<T> u[NI], g[NI], dh[NI];
    Eight<R> x[NI], dx[NI];
    float tok = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        u[i].clear();
        g[i].clear();
        dh[i].clear();
        x[i].clear();
        dx[i].clear();
    }
    auto load_stream = [&](int64_t row) {
        const bool live = row < a.rows, last = row >= a.rows - 1;
        const int64_t at = row * a.D;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (pre) {
                grp[i].load(x[i], static_cast<const R*>(a.x) + at, a.D, live, last);
                grp[i].load(dh[i], static_cast<const T*>(a.d_h) + at, a.D, live, last);
            }
            if (has_dx) grp[i].load(dx[i], static_cast<const R*>(a.d_x_out) + at, a.D, live, last);
        }
    };
    auto load_block = [&](int64_t row) {
        const bool live = row < a.rows, last = row >= a.rows - 1;
        const int64_t at = row * a.D;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (reads_u) grp[i].load(u[i], static_cast<const T*>(a.u) + at, a.D, live, last);
            if (full_gate) grp[i].load(g[i], static_cast<const T*>(a.gate) + at, a.D, live, last);
        }
        if (token_gate) tok = live ? load_as_f32(static_cast<const T*>(a.gate), row) : 0.f;
    };
    const int64_t step = int64_t(gridDim.x) * C::kRows;
    int64_t base = int64_t(blockIdx.x) * C::kRows;
    load_stream(base + slot);
    load_block(base + slot);
    for (; base < a.rows; base += step) {
        const int64_t row = base + slot;
        const bool live = row < a.rows, last = row >= a.rows - 1;

        // t, the gradient of x'
        float t[NI][8];
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (pre) {
                float xv[8], hv[8];
                grp[i].settle(x[i], a.D, last);
                grp[i].settle(dh[i], a.D, last);
                x[i].get(xv);
                dh[i].get(hv);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[0] = fmaf(xv[j], xv[j], s[0]);
                    s[1] = fmaf(wr[i][j] * hv[j], xv[j], s[1]);
                }
            }
            if (has_dx) grp[i].settle(dx[i], a.D, last);
            if (reads_u) grp[i].settle(u[i], a.D, last);
            if (full_gate) grp[i].settle(g[i], a.D, last);
            if (post) {
                float v[8];
                u[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[2] = fmaf(v[j], v[j], s[2]);
            }
        }
        if (pre || post) row_sums<LPR, WPR, 3>(s, lds, turn);
        const float rx = __builtin_amdgcn_rsqf(fmaf(s[0], inv_d, a.eps));
        const float back_x = rx * (rx * s[1] * inv_d);
        const float ru = post ? __builtin_amdgcn_rsqf(fmaf(s[2], inv_d, a.eps)) : 1.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (has_dx) {
                dx[i].get(t[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] = 0.f;
            }
            if (pre) {
                float xv[8], hv[8];
                x[i].get(xv);
                dh[i].get(hv);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc_pre[i][j] = fmaf(hv[j] * rx, xv[j], acc_pre[i][j]);
                    t[i][j] = fmaf(rx, fmaf(-back_x, xv[j], wr[i][j] * hv[j]), t[i][j]);
                }
            }
            Eight<R> out;
            out.put(t[i]);
            grp[i].store(out, static_cast<R*>(a.d_x) + row * a.D, a.D, live);
        }
        if (base + step < a.rows) load_stream(row + step);
        if (!has_u) continue;

        float ta = 1.f, dta = 0.f;
        if (token_gate) {
            float g8[8], f[8], df[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) g8[j] = tok;
            act_values(a.act, g8, f, df);
            ta = f[0];
            dta = df[0];
        }
        float q[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            // scale * t, nothing behind the row's end; the gate's part of its gradient, c n
#pragma unroll
            for (int j = 0; j < 8; ++j) t[i][j] = grp[i].has(j, a.D, live) ? factor * t[i][j] : 0.f;
            float uv[8], hat[8], dg[8];
            u[i].get(uv);
#pragma unroll
            for (int j = 0; j < 8; ++j) hat[j] = uv[j] * ru;
            if (full_gate) {
                float gv[8], f[8], df[8];
                g[i].get(gv);
                act_values(a.act, gv, f, df);
#pragma unroll
                for (int j = 0; j < 8; ++j) dg[j] = df[j] * (t[i][j] * (hat[j] * wp[i][j]));
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] *= f[j];
            } else if (CHANNEL || token_gate) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dg[j] = t[i][j] * (hat[j] * wp[i][j]);
                    t[i][j] *= CHANNEL ? ch[i][j] : ta;
                }
            }
            // the mask comes after the products: what a dropped element holds, NaN and
            // infinity too, reaches neither gradient
            if (a.drop.threshold) {
                const u32x4_t bits = philox4x32(uint64_t(row * groups + grp[i].col / 8), offset, a.drop.seed);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool keep = philox_keep(bits, j, a.drop.threshold);
                    t[i][j] = keep ? t[i][j] : 0.f;
                    dg[j] = keep ? dg[j] : 0.f;
                }
            }
            if (full_gate) {
                if (a.d_gate) {
                    Eight<T> out;
                    out.put(dg);
                    grp[i].store(out, static_cast<T*>(a.d_gate) + row * a.D, a.D, live);
                }
            } else if (CHANNEL) {
#pragma unroll
                for (int j = 0; j < 8; ++j) acc_gate[i][j] += dg[j];
            } else if (token_gate) {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[1] += dg[j];
            }
            if (post) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc_post[i][j] = fmaf(t[i][j], hat[j], acc_post[i][j]);
                    t[i][j] *= wp[i][j];
                    q[0] = fmaf(t[i][j], uv[j], q[0]);
                }
            }
        }
        if (post || token_gate) row_sums<LPR, WPR, 2>(q, lds, turn);
        if (token_gate && a.d_gate && rl == 0 && live) store_from_f32(static_cast<T*>(a.d_gate), row, dta * q[1]);
        const float back_u = ru * (ru * q[0] * inv_d);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (post) {
                float uv[8];
                u[i].get(uv);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] = ru * fmaf(-back_u, uv[j], t[i][j]);
            }
            Eight<T> out;
            out.put(t[i]);
            grp[i].store(out, static_cast<T*>(a.d_u) + row * a.D, a.D, live);
        }
        if (base + step < a.rows) load_block(row + step);
    }

    // this workgroup's column sums into its partial row: over the row slots of
    // a wavefront by lane exchanges, then over the wavefronts in LDS
    const int sums = (a.d_w_post != nullptr) + (a.d_w_pre != nullptr) + (CHANNEL && a.d_gate);
    int64_t at = int64_t(blockIdx.x) * sums * a.D;
    auto put_sum = [&](float (&acc)[NI][8]) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (C::kRows > 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = acc[i][j];
#pragma unroll
                    for (int off = LPR; off < 64; off *= 2) v += __shfl_xor(v, off, 64);
                    cols[threadIdx.x / 64][(threadIdx.x % 64) * 8 + j] = v;
                }
                __syncthreads();
                if (slot == 0) {
                    const int lane = threadIdx.x % 64;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float v = 0.f;
                        for (int w = threadIdx.x / 64; w < C::kWaves; w += WPR) v += cols[w][lane * 8 + j];
                        acc[i][j] = v;
                    }
                }
                __syncthreads();
            }
            if (slot == 0) {
                Eight<float> out;
                out.put(acc[i]);
                grp[i].store(out, a.partial + at, a.D, true);
            }
        }
        at += a.D;
    };
    if (a.d_w_post) put_sum(acc_post);
    if (a.d_w_pre) put_sum(acc_pre);
    if (CHANNEL && a.d_gate) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {  // act'(gate) is the column's own
            float gv[8], f[8], df[8];
            load_weight<MODE>(static_cast<const float*>(a.gate), grp[i], a.D, gv);
            act_values(a.act, gv, f, df);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc_gate[i][j] *= df[j];
        }
        put_sum(acc_gate);
    }
}

template <typename T, typename R>
hipError_t bwd_typed(const BlockNormBwdArgs& a, hipStream_t stream)
{
    const unsigned blocks = unsigned(block_bwd_partials(a.rows, a.D));
    if (blocks > 0) {
#define GDN2_BWD(LPR, WPR, NI, MODE)                                                                      \
    do {                                                                                                  \
        if (a.gate_layout == kGateChannel)                                                                \
            hipLaunchKernelGGL((block_norm_bwd_kernel<T, R, LPR, WPR, NI, MODE, true>), dim3(blocks),     \
                               dim3(Cover<LPR, WPR, NI>::kThreads), 0, stream, a);                        \
        else                                                                                              \
            hipLaunchKernelGGL((block_norm_bwd_kernel<T, R, LPR, WPR, NI, MODE, false>), dim3(blocks),    \
                               dim3(Cover<LPR, WPR, NI>::kThreads), 0, stream, a);                        \
    } while (0)
        GDN2_BWD_COVER(a.D, GDN2_BWD);
#undef GDN2_BWD
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    ColumnSumArgs c{};
    c.partial = a.partial;
    c.P = blocks;
    int n = 0;
    for (float* out : {a.d_w_post, a.d_w_pre, a.gate_layout == kGateChannel ? static_cast<float*>(a.d_gate) : nullptr})
        if (out) {
            c.out[n] = out;
            c.width += a.D;
            c.end[n++] = c.width;
        }
    for (; n < 3; ++n) c.end[n] = c.width;
    return launch_column_sum(c, stream);
}

}  // namespace

int64_t block_bwd_partials(int64_t rows, int32_t D)
{
    // as many workgroups as are resident at once
    int at_once = 1, resident = 1;
#define GDN2_PLAN(LPR, WPR, NI, MODE)          \
    at_once = Cover<LPR, WPR, NI>::kRows,      \
    resident = kSimds * bwd_waves_per_simd(WPR, NI) / Cover<LPR, WPR, NI>::kWaves
    GDN2_BWD_COVER(D, GDN2_PLAN);
#undef GDN2_PLAN
    return even_blocks(rows, at_once, resident);
}

hipError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, bool bf16, bool residual_bf16, hipStream_t stream)
{
    if (!bf16) return bwd_typed<float, float>(a, stream);
    return residual_bf16 ? bwd_typed<bf16raw, bf16raw>(a, stream) : bwd_typed<bf16raw, float>(a, stream);
}

}  // namespace gdn2
