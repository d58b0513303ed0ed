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
#include "row_device.hpp"

namespace gdn2 {
namespace {

__device__ __forceinline__ void act_value(int act, float g, float& a, float& da)
{
    if (act == 2) {
        a = g;
        da = 1.f;
        return;
    }
    const float s = fast_sigmoid(g);
    a = act == 0 ? s : g * s;
    da = act == 0 ? s * (1.f - s) : s * (1.f + g * (1.f - s));
}

// How a workgroup covers rows: LPR lanes (LPR < 64) or WPR wavefronts a row, NI
// groups of eight channels a lane.
template <int LPR, int WPR, int NI>
struct Cover {
    static constexpr int kThreads = WPR <= 4 ? 256 : WPR * 64;
    static constexpr int kWaves = kThreads / 64;
    static constexpr int kRowLanes = LPR * WPR;
    static constexpr int kRows = kThreads / kRowLanes;  // rows at a time per workgroup
};

// Sums of M values over a row's lanes.  Over several wavefronts they meet in
// LDS, in two buffers in turn: a wavefront that writes a buffer again has
// passed the barrier that every reader of its last contents reached after
// reading, so one barrier a sum is enough.
template <int LPR, int WPR, int M>
__device__ __forceinline__ void row_sums(float (&v)[M], float (*lds)[16][2], int& turn)
{
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = group_sum<LPR>(v[i]);
    if (WPR == 1) return;
    const int wave = threadIdx.x / 64, first = wave / WPR * WPR;
    if (threadIdx.x % 64 == 0) {
#pragma unroll
        for (int i = 0; i < M; ++i) lds[turn][wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < WPR; ++j) s += lds[turn][first + j][i];
        v[i] = s;
    }
    turn ^= 1;
}

__device__ __forceinline__ void load_weight(const float* w, int col, int D, float* v)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = col + j < D ? w[col + j] : 0.f;
}

// FULL: D is a multiple of 8, so every group is whole and at a 16-byte boundary.
template <typename T, typename R, int LPR, int WPR, int NI, bool FULL>
__global__ __launch_bounds__((Cover<LPR, WPR, NI>::kThreads)) void block_norm_fwd_kernel(BlockNormArgs a)
{
    using C = Cover<LPR, WPR, NI>;
    __shared__ float lds[2][16][2];
    int turn = 0;
    const int slot = threadIdx.x / C::kRowLanes, rl = threadIdx.x % C::kRowLanes;
    const int64_t groups = (a.D + 7) / 8;
    const uint64_t offset = a.drop.offset + (a.drop.offset_device ? *a.drop.offset_device : 0);
    const bool has_u = a.u != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
    const float inv_d = 1.0f / float(a.D);
    int col[NI];
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
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = live ? a.D - col[i] : 0;
            const int64_t e = row * a.D + col[i];
            nx[i].template load<FULL>(static_cast<const R*>(a.x) + e, n);
            if (has_u) nu[i].template load<FULL>(static_cast<const T*>(a.u) + e, n);
            if (a.gate_layout == kGateFull) ng[i].template load<FULL>(static_cast<const T*>(a.gate) + e, n);
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
            const int n = live ? a.D - col[i] : 0;
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
                h.template store<FULL>(static_cast<T*>(a.h) + row * a.D + col[i], live ? a.D - col[i] : 0);
            }
        }
    }
}

template <typename T, typename R, int LPR, int WPR, int NI, bool FULL>
__global__ __launch_bounds__((Cover<LPR, WPR, NI>::kThreads)) void block_norm_bwd_kernel(BlockNormBwdArgs a)
{
    using C = Cover<LPR, WPR, NI>;
    __shared__ float lds[2][16][2];
    __shared__ float cols[C::kRows > 1 ? C::kWaves : 1][C::kRows > 1 ? 64 * 8 : 1];
    int turn = 0;
    const int slot = threadIdx.x / C::kRowLanes, rl = threadIdx.x % C::kRowLanes;
    const int64_t groups = (a.D + 7) / 8;
    const uint64_t offset = a.drop.offset + (a.drop.offset_device ? *a.drop.offset_device : 0);
    const bool has_u = a.u != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
    const bool has_dx = a.d_x_out != nullptr;
    const bool reads_u = has_u && (post || a.gate_layout != kGateNone);
    const float inv_d = 1.0f / float(a.D);
    int col[NI];
    float wp[NI][8], wr[NI][8], ch[NI][8], acc_post[NI][8], acc_pre[NI][8], acc_gate[NI][8];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        col[i] = (i * C::kRowLanes + rl) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            wp[i][j] = wr[i][j] = ch[i][j] = 1.f;
            acc_post[i][j] = acc_pre[i][j] = acc_gate[i][j] = 0.f;
        }
        if (post) load_weight(a.w_post, col[i], a.D, wp[i]);
        if (pre) load_weight(a.w_pre, col[i], a.D, wr[i]);
        if (a.gate_layout == kGateChannel) {
            float g[8], da;
            load_weight(static_cast<const float*>(a.gate), col[i], a.D, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) act_value(a.act, g[j], ch[i][j], da);
        }
    }
    Eight<T> nu[NI], ng[NI], nh[NI];
    Eight<R> nx[NI], nd[NI];
    float nt = 0.f;
    auto load_row = [&](int64_t row) {
        const bool live = row < a.rows;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = live ? a.D - col[i] : 0;
            const int64_t e = row * a.D + col[i];
            if (pre) {
                nx[i].template load<FULL>(static_cast<const R*>(a.x) + e, n);
                nh[i].template load<FULL>(static_cast<const T*>(a.d_h) + e, n);
            }
            if (has_dx) nd[i].template load<FULL>(static_cast<const R*>(a.d_x_out) + e, n);
            if (reads_u) nu[i].template load<FULL>(static_cast<const T*>(a.u) + e, n);
            if (a.gate_layout == kGateFull) ng[i].template load<FULL>(static_cast<const T*>(a.gate) + e, n);
        }
        if (a.gate_layout == kGateToken) nt = live ? load_as_f32(static_cast<const T*>(a.gate), row) : 0.f;
    };
    const int64_t step = int64_t(gridDim.x) * C::kRows;
    int64_t base = int64_t(blockIdx.x) * C::kRows;
    load_row(base + slot);
    for (; base < a.rows; base += step) {
        const int64_t row = base + slot;
        const bool live = row < a.rows;
        Eight<T> u[NI], g[NI], dh[NI];
        Eight<R> x[NI], dx[NI];
        const float tok = nt;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            u[i] = nu[i];
            g[i] = ng[i];
            dh[i] = nh[i];
            x[i] = nx[i];
            dx[i] = nd[i];
        }
        if (base + step < a.rows) load_row(row + step);

        // t, the gradient of x'
        float t[NI][8];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (has_dx) {
                dx[i].get(t[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] = 0.f;
            }
        }
        float ru = 1.f;
        if (pre) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float xv[8], hv[8];
                x[i].get(xv);
                dh[i].get(hv);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[0] = fmaf(xv[j], xv[j], s[0]);
                    s[1] = fmaf(wr[i][j] * hv[j], xv[j], s[1]);
                }
            }
            row_sums<LPR, WPR, 2>(s, lds, turn);
            const float rx = __builtin_amdgcn_rsqf(fmaf(s[0], inv_d, a.eps));
            const float back = rx * rx * rx * s[1] * inv_d;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float xv[8], hv[8];
                x[i].get(xv);
                dh[i].get(hv);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc_pre[i][j] = fmaf(hv[j], xv[j] * rx, acc_pre[i][j]);
                    t[i][j] += rx * wr[i][j] * hv[j] - xv[j] * back;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            Eight<R> out;
            out.put(t[i]);
            out.template store<FULL>(static_cast<R*>(a.d_x) + row * a.D + col[i], live ? a.D - col[i] : 0);
        }
        if (!has_u) continue;

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
        float ta = 1.f, dta = 0.f;
        if (a.gate_layout == kGateToken) act_value(a.act, tok, ta, dta);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = live ? a.D - col[i] : 0;
            float uv[8], gv[8], dg[8];
            if (reads_u) u[i].get(uv);
            if (a.gate_layout == kGateFull) g[i].get(gv);
            u32x4_t bits{0, 0, 0, 0};
            if (a.drop.threshold) bits = philox4x32(uint64_t(row * groups + col[i] / 8), offset, a.drop.seed);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float c = a.scale * t[i][j];
                if (a.drop.threshold) c = philox_keep(bits, j, a.drop.threshold) ? c * a.drop.keep : 0.f;
                if (!(FULL ? n > 0 : j < n)) c = 0.f;  // behind the row's end
                const float hat = reads_u ? uv[j] * ru : 0.f, nn = hat * wp[i][j];
                float f = ch[i][j] * ta;
                if (a.gate_layout == kGateFull) {
                    float df;
                    act_value(a.act, gv[j], f, df);
                    dg[j] = df * c * nn;
                } else if (a.gate_layout == kGateChannel) {
                    acc_gate[i][j] = fmaf(c, nn, acc_gate[i][j]);
                } else if (a.gate_layout == kGateToken) {
                    s[1] = fmaf(c, nn, s[1]);
                }
                const float dn = c * f;
                t[i][j] = dn;
                if (post) {
                    acc_post[i][j] = fmaf(dn, hat, acc_post[i][j]);
                    s[0] = fmaf(wp[i][j] * dn, uv[j], s[0]);
                }
            }
            if (a.gate_layout == kGateFull && a.d_gate) {
                Eight<T> out;
                out.put(dg);
                out.template store<FULL>(static_cast<T*>(a.d_gate) + row * a.D + col[i], n);
            }
        }
        if (post || a.gate_layout == kGateToken) row_sums<LPR, WPR, 2>(s, lds, turn);
        if (a.gate_layout == kGateToken && a.d_gate && rl == 0 && live)
            store_from_f32(static_cast<T*>(a.d_gate), row, dta * s[1]);
        const float back = ru * ru * ru * s[0] * inv_d;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (post) {
                float uv[8];
                u[i].get(uv);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] = ru * wp[i][j] * t[i][j] - uv[j] * back;
            }
            Eight<T> out;
            out.put(t[i]);
            out.template store<FULL>(static_cast<T*>(a.d_u) + row * a.D + col[i], live ? a.D - col[i] : 0);
        }
    }

    // this workgroup's column sums into its partial row: over the row slots of
    // a wavefront by lane exchanges, then over the wavefronts in LDS
    const int sums = (a.d_w_post != nullptr) + (a.d_w_pre != nullptr) + (a.gate_layout == kGateChannel && a.d_gate);
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
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col[i] + j < a.D) a.partial[at + col[i] + j] = acc[i][j];
            }
        }
        at += a.D;
    };
    if (a.d_w_post) put_sum(acc_post);
    if (a.d_w_pre) put_sum(acc_pre);
    if (a.gate_layout == kGateChannel && a.d_gate) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {  // act'(gate) is the column's own
            float g[8], f, df;
            load_weight(static_cast<const float*>(a.gate), col[i], a.D, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                act_value(a.act, g[j], f, df);
                acc_gate[i][j] *= df;
            }
        }
        put_sum(acc_gate);
    }
}

// Workgroups of a launch over `rows` rows, `at_once` of them a workgroup.
int64_t blocks_for(int64_t rows, int at_once, int64_t most)
{
    const int64_t need = (rows + at_once - 1) / at_once;
    return need < most ? need : most;
}

// The cover of a row of D channels: calls f(Cover parameters as template
// arguments).  Narrow rows take a lane group, then one wavefront, then as many
// as leave eight channels a lane; the widest take sixteen.
#define GDN2_COVER(D, F)                     \
    do {                                     \
        if ((D) <= 64) F(8, 1, 1);           \
        else if ((D) <= 256) F(32, 1, 1);    \
        else if ((D) <= 512) F(64, 1, 1);    \
        else if ((D) <= 1024) F(64, 2, 1);   \
        else if ((D) <= 2048) F(64, 4, 1);   \
        else if ((D) <= 4096) F(64, 8, 1);   \
        else if ((D) <= 8192) F(64, 16, 1);  \
        else F(64, 16, 2);                   \
    } while (0)

int rows_at_once(int32_t D)
{
    int n = 1;
#define GDN2_ROWS(LPR, WPR, NI) n = Cover<LPR, WPR, NI>::kRows
    GDN2_COVER(D, GDN2_ROWS);
#undef GDN2_ROWS
    return n;
}

constexpr int64_t kFwdBlocks = 2048, kBwdBlocks = 1024;

template <typename T, typename R>
hipError_t fwd_typed(const BlockNormArgs& a, hipStream_t stream)
{
    const unsigned blocks = unsigned(blocks_for(a.rows, rows_at_once(a.D), kFwdBlocks));
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

template <typename T, typename R>
hipError_t bwd_typed(const BlockNormBwdArgs& a, hipStream_t stream)
{
    const unsigned blocks = unsigned(block_bwd_partials(a.rows, a.D));
    if (blocks > 0) {
#define GDN2_BWD(LPR, WPR, NI)                                                                                     \
    do {                                                                                                           \
        if (a.D % 8 == 0)                                                                                          \
            hipLaunchKernelGGL((block_norm_bwd_kernel<T, R, LPR, WPR, NI, true>), dim3(blocks),                    \
                               dim3(Cover<LPR, WPR, NI>::kThreads), 0, stream, a);                                 \
        else                                                                                                       \
            hipLaunchKernelGGL((block_norm_bwd_kernel<T, R, LPR, WPR, NI, false>), dim3(blocks),                   \
                               dim3(Cover<LPR, WPR, NI>::kThreads), 0, stream, a);                                 \
    } while (0)
        GDN2_COVER(a.D, GDN2_BWD);
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

int64_t block_bwd_partials(int64_t rows, int32_t D) { return blocks_for(rows, rows_at_once(D), kBwdBlocks); }

hipError_t launch_block_norm_fwd(const BlockNormArgs& a, bool bf16, bool residual_bf16, hipStream_t stream)
{
    if (!bf16) return fwd_typed<float, float>(a, stream);
    return residual_bf16 ? fwd_typed<bf16raw, bf16raw>(a, stream) : fwd_typed<bf16raw, float>(a, stream);
}

hipError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, bool bf16, bool residual_bf16, hipStream_t stream)
{
    if (!bf16) return bwd_typed<float, float>(a, stream);
    return residual_bf16 ? bwd_typed<bf16raw, bf16raw>(a, stream) : bwd_typed<bf16raw, float>(a, stream);
}

hipError_t launch_dropout(const DropoutCall& a, bool bf16, hipStream_t stream)
{
    return bf16 ? dropout_typed<bf16raw>(a, stream) : dropout_typed<float>(a, stream);
}

}  // namespace gdn2
