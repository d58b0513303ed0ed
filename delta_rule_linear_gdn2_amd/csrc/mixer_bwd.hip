// Backward of the token mixer around the recurrence (mixer.hip), for gfx950.
//
// Epilogue, y = o / rms(o) * w * act(g) per row of dv values, rms(o) =
// sqrt(mean(o^2) + eps):
//     dn = dy act(g),  do = (w dn - o mean(w dn o) / rms(o)^2) / rms(o)
//     dg = act'(g) dy w o / rms(o),  dw = sum over rows of dn o / rms(o)
// Prologue, per channel of a convolution path, with y_t = sum_i W_i
// x_{t-K+1+i} inside a sequence (inputs before its start come from the carried
// state), v = SiLU(y) and, for q and k, q = s v r with r = (sum over the head's
// v^2 + eps)^(-1/2):
//     dv  = s r (dq - v r^2 sum(v dq)),   dy = dv SiLU'(y)
//     dx_t = sum_i W_i dy_{t+K-1-i} over the sequence's tokens,
//     dW_i = sum_t dy_t x_{t-K+1+i}
// and db_logit = db b (1 - b).  The gradients at the K - 1 positions before a
// sequence are the carried state's; the gradient of the state after a sequence
// belongs to its last K - 1 inputs.  y, the activations and the norms are
// remade from the inputs; all arithmetic is FP32.
//
// HBM-bound, one pass.  Epilogue: dv / 8 lanes a row, eight channels a lane,
// the weight's gradient in registers over many rows.  Prologue: one wavefront
// per (path, batch row, group of heads, run of tokens); a lane holds its
// channels' filters, the window of the last K - 1 inputs, the K - 1 unfinished
// input gradients and the filters' gradients.  An input's gradient needs the
// K - 1 tokens after it, so a run reads that many tokens past its end (and
// before its start).  The filters' gradients of a run go to the workspace and
// are added by the column-sum kernel.
#include "row_device.hpp"

namespace gdn2 {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Epilogue.

template <typename T, int DV>
__global__ __launch_bounds__(kThreads) void epilogue_bwd_kernel(EpilogueBwdArgs a)
{
    constexpr int G = DV / 8, RPW = 64 / G, RPB = RPW * (kThreads / 64);
    __shared__ float cols[kThreads / 64][DV];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int c0 = (lane % G) * 8;
    float w[8], acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        w[j] = a.weight[c0 + j];
        acc[j] = 0.f;
    }
    for (int64_t base = int64_t(blockIdx.x) * RPB; base < a.rows; base += int64_t(gridDim.x) * RPB) {
        const int64_t r = base + wave * RPW + lane / G;
        const int n = r < a.rows ? 8 : 0;
        const int64_t e = r * DV + c0;
        Eight<T> ro, rg, ry;
        ro.template load<true>(static_cast<const T*>(a.o) + e, n);
        rg.template load<true>(static_cast<const T*>(a.gate) + e, n);
        ry.template load<true>(static_cast<const T*>(a.d_y) + e, n);
        float o[8], g[8], y[8], dn[8], dg[8];
        ro.get(o);
        rg.get(g);
        ry.get(y);
        float ss = 0.f, so = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = fast_sigmoid(g[j]);
            const float f = a.act == 0 ? s : g[j] * s;
            const float df = a.act == 0 ? s * (1.f - s) : s * (1.f + g[j] * (1.f - s));
            dn[j] = y[j] * f;
            dg[j] = df * y[j] * w[j] * o[j];
            ss = fmaf(o[j], o[j], ss);
            so = fmaf(w[j] * dn[j], o[j], so);
        }
        ss = group_sum<G>(ss);
        so = group_sum<G>(so);
        const float rr = __builtin_amdgcn_rsqf(ss * (1.0f / DV) + a.eps);
        const float back = rr * rr * rr * so * (1.0f / DV);
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            acc[j] = fmaf(dn[j], o[j] * rr, acc[j]);
            d[j] = rr * w[j] * dn[j] - o[j] * back;
            dg[j] *= rr;
        }
        Eight<T> out;
        out.put(d);
        out.template store<true>(static_cast<T*>(a.d_o) + e, n);
        out.put(dg);
        out.template store<true>(static_cast<T*>(a.d_gate) + e, n);
    }
    if (!a.d_weight) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float v = acc[j];
#pragma unroll
        for (int off = G; off < 64; off *= 2) v += __shfl_xor(v, off, 64);
        if (lane < G) cols[wave][c0 + j] = v;
    }
    __syncthreads();
    if (threadIdx.x < DV) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) v += cols[i][threadIdx.x];
        a.partial[int64_t(blockIdx.x) * DV + threadIdx.x] = v;
    }
}

constexpr int64_t kEpiBlocks = 1024;

template <typename T>
hipError_t epilogue_typed(const EpilogueBwdArgs& a, hipStream_t stream)
{
    const unsigned blocks = unsigned(epilogue_bwd_partials(a.rows, a.dv));
    if (blocks > 0) {
        switch (a.dv) {
            case 32: hipLaunchKernelGGL((epilogue_bwd_kernel<T, 32>), dim3(blocks), dim3(kThreads), 0, stream, a); break;
            case 64: hipLaunchKernelGGL((epilogue_bwd_kernel<T, 64>), dim3(blocks), dim3(kThreads), 0, stream, a); break;
            case 128: hipLaunchKernelGGL((epilogue_bwd_kernel<T, 128>), dim3(blocks), dim3(kThreads), 0, stream, a); break;
            default: return hipErrorInvalidValue;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.d_weight) return hipSuccess;
    return launch_column_sum({a.partial, blocks, a.dv, {a.d_weight, nullptr, nullptr}, {a.dv, a.dv, a.dv}}, stream);
}

// ---------------------------------------------------------------------------
// Prologue.

// Sequence of packed position t: the last n with cu[n] <= t, offsets clamped
// like every other kernel's.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int N, int32_t T, int64_t t)
{
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        int64_t c = cu[mid];
        c = c < 0 ? 0 : (c > T ? T : c);
        if (c <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// CPL consecutive channels: eight as one group, four or two as half and
// quarter of one.
template <int CPL>
__device__ __forceinline__ void load_channels(const bf16raw* p, float* v)
{
#pragma unroll
    for (int j = 0; j < CPL / 2; ++j) {
        const uint32_t u = reinterpret_cast<const uint32_t*>(p)[j];
        v[2 * j] = __uint_as_float(u << 16);
        v[2 * j + 1] = __uint_as_float(u & 0xffff0000u);
    }
}
template <int CPL>
__device__ __forceinline__ void load_channels(const float* p, float* v)
{
#pragma unroll
    for (int j = 0; j < CPL; ++j) v[j] = p[j];
}
template <int CPL>
__device__ __forceinline__ void store_channels(bf16raw* p, const float* v)
{
#pragma unroll
    for (int j = 0; j < CPL / 2; ++j) reinterpret_cast<uint32_t*>(p)[j] = f32x2_to_bf16x2(v[2 * j], v[2 * j + 1]);
}
template <int CPL>
__device__ __forceinline__ void store_channels(float* p, const float* v)
{
#pragma unroll
    for (int j = 0; j < CPL; ++j) p[j] = v[j];
}

// One convolution path (PATH 0 q, 1 k, 2 v; head width D) of one wavefront's
// run.  KM bounds the filter's taps: tap i of K sits at index KM - K + i, and
// everything below index KM - K stays untouched.
template <typename T, int D, int PATH, int KM>
__device__ __forceinline__ void conv_bwd_path(const PrologueBwdArgs& a, int64_t wid, int lane)
{
    constexpr int CPL = KM <= 4 ? 8 : KM <= 8 ? 4 : 2;  // channels per lane
    constexpr int LPH = D / CPL, HPW = 64 / LPH;        // lanes per head, heads per wavefront
    constexpr int W = KM - 1;                           // window entries
    const int ng = (a.H + HPW - 1) / HPW;
    const int64_t nruns = (int64_t(a.T) + a.run - 1) / a.run;
    if (wid >= int64_t(a.B) * nruns * ng) return;
    const int h = int(wid % ng) * HPW + lane / LPH;
    if (h >= a.H) return;  // lanes past the last head share no sum with live ones
    const int64_t run = (wid / ng) % nruns, brow = wid / ng / nruns;
    const int64_t t0 = run * a.run, t1 = t0 + a.run < a.T ? t0 + a.run : a.T;
    const int K = a.K, low = KM - K;
    const int chan = h * D + (lane % LPH) * CPL;        // first channel within the path
    const int64_t stride = int64_t(a.H) * D, row0 = brow * a.T * stride + chan;
    const int64_t nch = int64_t(a.H) * (2 * a.dk + a.dv);
    const int64_t state_chan = int64_t(PATH) * a.H * a.dk + chan;  // q, k, v in turn
    const T* x = static_cast<const T*>(a.x[PATH]);
    const T* dout = static_cast<const T*>(a.d_out[PATH]);
    T* dx = static_cast<T*>(a.d_x[PATH]);

    float w[KM][CPL], dw[KM][CPL];
#pragma unroll
    for (int i = 0; i < KM; ++i)
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            w[i][c] = i >= low ? a.conv[PATH][int64_t(chan + c) * K + (i - low)] : 0.f;
            dw[i][c] = 0.f;
        }

    int n = int(brow);
    int64_t bos = 0, eos = a.T, unused;
    if (a.cu_seqlens) {
        n = sequence_of(a.cu_seqlens, a.N, a.T, t0);
        sequence_bounds(a.cu_seqlens, n, a.T, bos, eos, unused);
    }
    // xw[j]: the input W - j positions before the current token; pend[j]: the
    // gradient gathered so far for that position
    float xw[W > 0 ? W : 1][CPL], pend[W > 0 ? W : 1][CPL];
    auto restart = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int64_t s = t - W + j;
#pragma unroll
            for (int c = 0; c < CPL; ++c) xw[j][c] = pend[j][c] = 0.f;
            if (j < low) continue;
            if (s >= bos) {
                load_channels<CPL>(x + row0 + s * stride, xw[j]);
            } else if (a.conv_state_in) {
                const int64_t js = (K - 1) - (bos - s);
                if (js >= 0) {
#pragma unroll
                    for (int c = 0; c < CPL; ++c)
                        xw[j][c] = a.conv_state_in[(int64_t(n) * nch + state_chan + c) * (K - 1) + js];
                }
            }
        }
    };
    // the finished gradient of position s of the current sequence
    auto finish = [&](int64_t s, const float* v) {
        if (s >= bos) {
            if (s >= t0 && s < t1) store_channels<CPL>(dx + row0 + s * stride, v);
        } else if (a.d_state_in && bos >= t0 && bos < t1) {
            const int64_t js = (K - 1) - (bos - s);
            if (js >= 0) {
#pragma unroll
                for (int c = 0; c < CPL; ++c)
                    a.d_state_in[(int64_t(n) * nch + state_chan + c) * (K - 1) + js] = v[c];
            }
        }
    };
    restart(t0);
    for (int64_t t = t0; t < t1 + K - 1 && t < a.T; ++t) {
        if (t >= eos) {  // the next non-empty sequence starts here (packed input only)
            if (t >= t1) break;
            n = sequence_of(a.cu_seqlens, a.N, a.T, t);
            sequence_bounds(a.cu_seqlens, n, a.T, bos, eos, unused);
            restart(t);
        }
        float xt[CPL], g[CPL], y[CPL], v[CPL], sg[CPL];
        load_channels<CPL>(x + row0 + t * stride, xt);
        load_channels<CPL>(dout + row0 + t * stride, g);
        float ss = 0.f, sv = 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            float acc = w[W][c] * xt[c];
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (i >= low) acc = fmaf(w[i][c], xw[i][c], acc);
            y[c] = acc;
            sg[c] = fast_sigmoid(acc);
            v[c] = acc * sg[c];
            ss = fmaf(v[c], v[c], ss);
            sv = fmaf(v[c], g[c], sv);
        }
        float r = 1.f, back = 0.f;
        if (PATH < 2) {
            ss = group_sum<LPH>(ss);
            sv = group_sum<LPH>(sv);
            r = __builtin_amdgcn_rsqf(ss + a.eps_l2);
            back = r * r * r * sv;
            if (PATH == 0) {
                r *= a.q_scale;
                back *= a.q_scale;
            }
        }
        const bool mine = t < t1;
        float done[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const float dv = PATH < 2 ? r * g[c] - v[c] * back : g[c];
            const float dy = dv * sg[c] * (1.f + y[c] * (1.f - sg[c]));
            if (mine) {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (i >= low) dw[i][c] = fmaf(dy, xw[i][c], dw[i][c]);
                dw[W][c] = fmaf(dy, xt[c], dw[W][c]);
            }
            // position W - j back gets w[j] dy; the oldest one is then finished, the others move one back
            done[c] = w[W][c] * dy;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (j < low) continue;
                const float p = fmaf(w[j][c], dy, pend[j][c]);
                if (j == low) done[c] = p;
                else pend[j - 1][c] = p;
                if (j > low) xw[j - 1][c] = xw[j][c];
            }
            if (W > 0 && low < W) {
                pend[W - 1][c] = w[W][c] * dy;
                xw[W - 1][c] = xt[c];
            }
        }
        finish(t - (K - 1), done);
        if (t == eos - 1) {  // no later token adds to the last K - 1 positions
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (j < low) continue;
                const int64_t s = t + 1 - W + j;
                float p[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c)
                    p[c] = pend[j][c] +
                           (a.d_state_out ? a.d_state_out[(int64_t(n) * nch + state_chan + c) * (K - 1) + (j - low)] : 0.f);
                finish(s, p);
            }
        }
    }
    if (a.partial) {
        float* out = a.partial + ((brow * nruns + run) * nch + state_chan) * K;
#pragma unroll
        for (int c = 0; c < CPL; ++c)
#pragma unroll
            for (int i = 0; i < KM; ++i)
                if (i >= low) out[c * K + (i - low)] = dw[i][c];
    }
}

// Gate logits: eight channels a lane over the wavefront's run.
template <typename T, int D, int WHICH>
__device__ __forceinline__ void gate_bwd_path(const PrologueBwdArgs& a, int64_t wid, int lane)
{
    constexpr int LPH = D / 8, HPW = 64 / LPH;
    const int ng = (a.H + HPW - 1) / HPW;
    const int64_t nruns = (int64_t(a.T) + a.run - 1) / a.run;
    if (wid >= int64_t(a.B) * nruns * ng) return;
    const int h = int(wid % ng) * HPW + lane / LPH;
    if (h >= a.H) return;
    const int64_t run = (wid / ng) % nruns, brow = wid / ng / nruns;
    const int64_t t0 = run * a.run, t1 = t0 + a.run < a.T ? t0 + a.run : a.T;
    const int64_t stride = int64_t(a.H) * D, row0 = brow * a.T * stride + h * D + (lane % LPH) * 8;
    const T* logit = static_cast<const T*>(a.logit[WHICH]) + row0;
    const T* dg = static_cast<const T*>(a.d_gate[WHICH]) + row0;
    T* out = static_cast<T*>(a.d_logit[WHICH]) + row0;
    for (int64_t t = t0; t < t1; ++t) {
        Eight<T> rl, rd;
        rl.template load<true>(logit + t * stride, 8);
        rd.template load<true>(dg + t * stride, 8);
        float l[8], d[8];
        rl.get(l);
        rd.get(d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = fast_sigmoid(l[j]);
            d[j] *= s * (1.f - s);
        }
        rd.put(d);
        rd.template store<true>(out + t * stride, 8);
    }
}

// blockIdx.y + first: 0 q, 1 k, 2 b (head width dk), 3 v, 4 w (dv).  One launch
// takes all five where dk = dv, else one takes the first three and one the rest.
template <typename T, int D, int KM>
__global__ __launch_bounds__(kThreads) void prologue_bwd_kernel(PrologueBwdArgs a, int first)
{
    const int lane = threadIdx.x % 64;
    const int64_t wid = int64_t(blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
    switch (blockIdx.y + first) {
        case 0: conv_bwd_path<T, D, 0, KM>(a, wid, lane); break;
        case 1: conv_bwd_path<T, D, 1, KM>(a, wid, lane); break;
        case 2: gate_bwd_path<T, D, 0>(a, wid, lane); break;
        case 3: conv_bwd_path<T, D, 2, KM>(a, wid, lane); break;
        default: gate_bwd_path<T, D, 1>(a, wid, lane); break;
    }
}

// Sequences without tokens carry their state through, and its gradient back.
__global__ __launch_bounds__(kThreads) void state_grad_passthrough_kernel(PrologueBwdArgs a)
{
    const int64_t per = int64_t(a.H) * (2 * a.dk + a.dv) * (a.K - 1);
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= int64_t(a.N) * per) return;
    int64_t bos, eos, brow;
    sequence_bounds(a.cu_seqlens, int(i / per), a.T, bos, eos, brow);
    if (eos > bos) return;
    a.d_state_in[i] = a.d_state_out ? a.d_state_out[i] : 0.f;
}

template <typename T, int D>
hipError_t prologue_paths(const PrologueBwdArgs& a, int first, int count, hipStream_t stream)
{
    const int cpl = a.K <= 4 ? 8 : a.K <= 8 ? 4 : 2, hpw = 64 / (D / cpl);
    const int64_t waves = int64_t(a.B) * ((int64_t(a.T) + a.run - 1) / a.run) * ((a.H + hpw - 1) / hpw);
    const int64_t blocks = (waves + 3) / 4;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    const dim3 grid{unsigned(blocks), unsigned(count), 1}, block{kThreads, 1, 1};
    if (a.K == 1)
        hipLaunchKernelGGL((prologue_bwd_kernel<T, D, 1>), grid, block, 0, stream, a, first);
    else if (a.K <= 4)
        hipLaunchKernelGGL((prologue_bwd_kernel<T, D, 4>), grid, block, 0, stream, a, first);
    else if (a.K <= 8)
        hipLaunchKernelGGL((prologue_bwd_kernel<T, D, 8>), grid, block, 0, stream, a, first);
    else
        hipLaunchKernelGGL((prologue_bwd_kernel<T, D, 16>), grid, block, 0, stream, a, first);
    return hipGetLastError();
}

template <typename T>
hipError_t prologue_width(const PrologueBwdArgs& a, int d, int first, int count, hipStream_t stream)
{
    switch (d) {
        case 32: return prologue_paths<T, 32>(a, first, count, stream);
        case 64: return prologue_paths<T, 64>(a, first, count, stream);
        case 128: return prologue_paths<T, 128>(a, first, count, stream);
        default: return hipErrorInvalidValue;
    }
}

template <typename T>
hipError_t prologue_typed(const PrologueBwdArgs& a, hipStream_t stream)
{
    if (a.T > 0) {
        hipError_t e = prologue_width<T>(a, a.dk, 0, a.dk == a.dv ? 5 : 3, stream);
        if (e == hipSuccess && a.dk != a.dv) e = prologue_width<T>(a, a.dv, 3, 2, stream);
        if (e != hipSuccess) return e;
    }
    if (a.d_state_in && a.K > 1 && (a.cu_seqlens || a.T == 0)) {
        const int64_t n = int64_t(a.N) * a.H * (2 * a.dk + a.dv) * (a.K - 1);
        const int64_t blocks = (n + kThreads - 1) / kThreads;
        if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL(state_grad_passthrough_kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.d_conv[0] && !a.d_conv[1] && !a.d_conv[2]) return hipSuccess;
    const int64_t k = int64_t(a.H) * a.dk * a.K, v = int64_t(a.H) * a.dv * a.K;
    const int64_t parts = int64_t(a.B) * ((int64_t(a.T) + a.run - 1) / a.run);
    return launch_column_sum({a.partial, parts, 2 * k + v, {a.d_conv[0], a.d_conv[1], a.d_conv[2]}, {k, 2 * k, 2 * k + v}},
                             stream);
}

}  // namespace

int64_t epilogue_bwd_partials(int64_t rows, int32_t dv)
{
    const int64_t at_once = (kThreads / 64) * (64 / (dv / 8));
    const int64_t need = (rows + at_once - 1) / at_once;
    return need < kEpiBlocks ? need : kEpiBlocks;
}

int32_t prologue_bwd_run(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t K)
{
    (void)B, (void)T, (void)H, (void)dk, (void)dv, (void)K;
    return 64;
}

hipError_t launch_mixer_epilogue_bwd(const EpilogueBwdArgs& a, bool bf16, hipStream_t stream)
{
    return bf16 ? epilogue_typed<bf16raw>(a, stream) : epilogue_typed<float>(a, stream);
}

hipError_t launch_mixer_prologue_bwd(const PrologueBwdArgs& a, bool bf16, hipStream_t stream)
{
    return bf16 ? prologue_typed<bf16raw>(a, stream) : prologue_typed<float>(a, stream);
}

}  // namespace gdn2
