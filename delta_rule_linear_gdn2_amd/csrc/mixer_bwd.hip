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
// remade from the inputs; all arithmetic is FP32, with 1 / rms and r going in factor by
// factor (their cubes leave its range before the gradients do).
//
// HBM-bound, one pass.  Epilogue: dv / 8 lanes a row, eight channels a lane, the
// weight's gradient in registers over many rows (524288 rows of 128 bf16: 130 us
// a call, 671 MB at 5.2 TB/s).  Prologue: one wavefront per (path, batch row, group
// of heads, run of tokens); a lane holds its channels' filters, the window of the
// last K - 1 inputs, the K - 1 unfinished input gradients and the filters'
// gradients.  An input's gradient needs the K - 1 tokens after it, so a run reads
// that many tokens past its end (and before its start).  The filters' gradients of
// a run go to the workspace and are added by the column-sum kernel.  B=8, T=4096,
// H=16, d=128, K=4, bf16: 424 us a call; the kernel's 416 us move 2.07 GB, 1.03
// times inputs and outputs, with 61% of the vector issue slots taken beside.
// Outputs are written past the caches (2% less time than through them).
#include <type_traits>

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
        const bool on = r < a.rows;
        const int64_t e = r * DV + c0;
        Eight<T> ro, rg, ry;
        if (on) ro.load(static_cast<const T*>(a.o) + e);
        else ro.clear();
        if (on) rg.load(static_cast<const T*>(a.gate) + e);
        else rg.clear();
        if (on) ry.load(static_cast<const T*>(a.d_y) + e);
        else ry.clear();
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
        const float back = rr * (rr * so * (1.0f / DV));
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            acc[j] = fmaf(dn[j], o[j] * rr, acc[j]);
            d[j] = rr * fmaf(-o[j], back, w[j] * dn[j]);
            dg[j] *= rr;
        }
        Eight<T> out;
        out.put(d);
        if (on) out.template store<true>(static_cast<T*>(a.d_o) + e);
        out.put(dg);
        if (on) out.template store<true>(static_cast<T*>(a.d_gate) + e);
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

// Tokens [t0, t1) of run `run` that some sequence owns (packed input may end in
// padding, which is not read and, but for padding_path, not written); t1 <= t0:
// none.
__device__ __forceinline__ void owned_tokens(const PrologueBwdArgs& a, int64_t run, int& t0, int& t1)
{
    t0 = int(run * a.run);
    t1 = a.T - t0 > a.run ? t0 + a.run : a.T;
    if (!a.cu_seqlens) return;
    const int first = a.cu_seqlens[0], end = a.cu_seqlens[a.N];
    t0 = first > t0 ? first : t0;
    t1 = end < t1 ? end : t1;
}

// CPL consecutive channels of a row, as loaded: eight, four or two (bf16 stays
// packed until used).  They sit at a boundary of their own size.
template <typename T, int CPL>
struct Channels;
template <int CPL>
struct Channels<bf16raw, CPL> {
    typedef uint32_t raw_t __attribute__((ext_vector_type(CPL / 2 > 1 ? CPL / 2 : 2)));
    uint32_t u[CPL / 2];
    __device__ __forceinline__ void load(const bf16raw* p)
    {
        if (CPL == 2) {
            u[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            const raw_t v = *reinterpret_cast<const raw_t*>(p);
#pragma unroll
            for (int j = 0; j < CPL / 2; ++j) u[j] = v[j];
        }
    }
    __device__ __forceinline__ void get(float* v) const
    {
#pragma unroll
        for (int j = 0; j < CPL / 2; ++j) {
            v[2 * j] = __uint_as_float(u[j] << 16);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(bf16raw* p, const float* v)
    {
        if (CPL == 2) {
            *reinterpret_cast<uint32_t*>(p) = f32x2_to_bf16x2(v[0], v[1]);
        } else {
            raw_t r;
#pragma unroll
            for (int j = 0; j < CPL / 2; ++j) r[j] = f32x2_to_bf16x2(v[2 * j], v[2 * j + 1]);
            put16<true>(p, r);
        }
    }
};
template <int CPL>
struct Channels<float, CPL> {
    static constexpr int V = CPL < 4 ? CPL : 4;
    typedef float raw_t __attribute__((ext_vector_type(V)));
    float u[CPL];
    __device__ __forceinline__ void load(const float* p)
    {
#pragma unroll
        for (int i = 0; i < CPL / V; ++i) {
            const raw_t v = reinterpret_cast<const raw_t*>(p)[i];
#pragma unroll
            for (int j = 0; j < V; ++j) u[i * V + j] = v[j];
        }
    }
    __device__ __forceinline__ void get(float* v) const
    {
#pragma unroll
        for (int j = 0; j < CPL; ++j) v[j] = u[j];
    }
    static __device__ __forceinline__ void store(float* p, const float* v)
    {
#pragma unroll
        for (int i = 0; i < CPL / V; ++i) {
            raw_t r;
#pragma unroll
            for (int j = 0; j < V; ++j) r[j] = v[i * V + j];
            put16<true>(p + i * V, r);
        }
    }
};

// Filters, window, unfinished and filter gradients take (4 KM + 8) registers a
// channel: with eight channels a lane, four taps spilled (640 us at the shape above,
// one wavefront a SIMD); four a lane fit 185 (FP32 202).
constexpr int channels_per_lane(int KM) { return KM <= 1 ? 8 : KM <= 4 ? 4 : 2; }
constexpr int kStep = 4;  // tokens per unrolled step

// One convolution path (PATH 0 q, 1 k, 2 v; head width D) of one wavefront's
// run.  KM bounds the filter's taps (KM = K up to four): tap i of K sits at
// index KM - K + i, and everything below index KM - K stays untouched.
//
// Tokens go kStep at a time with the next step's loads in flight; a step that a
// sequence's start or end falls into goes token by token.  The window and the
// unfinished gradients of a step are one array each, indexed by constants, so
// nothing moves between registers inside a step.
template <typename T, int D, int PATH, int KM>
__device__ __forceinline__ void conv_bwd_path(const PrologueBwdArgs& a, int64_t wid, int lane)
{
    constexpr int CPL = channels_per_lane(KM);
    constexpr int LPH = D / CPL, HPW = 64 / LPH;  // lanes per head, heads per wavefront
    constexpr int W = KM - 1;                     // window entries
    using Ch = Channels<T, CPL>;
    const int ng = (a.H + HPW - 1) / HPW;
    const int64_t nruns = (int64_t(a.T) + a.run - 1) / a.run;
    if (wid >= int64_t(a.B) * nruns * ng) return;
    const int h = int(wid % ng) * HPW + lane / LPH;
    if (h >= a.H) return;  // lanes past the last head share no sum with live ones
    const int64_t run = (wid / ng) % nruns, brow = wid / ng / nruns;
    int t0, t1;
    owned_tokens(a, run, t0, t1);
    const int K = KM <= 4 ? KM : a.K, low = KM - K;
    const int chan = h * D + (lane % LPH) * CPL;  // first channel within the path
    const int64_t stride = int64_t(a.H) * D, row0 = brow * a.T * stride;
    const int64_t nch = int64_t(a.H) * (2 * a.dk + a.dv);
    const int64_t state_chan = int64_t(PATH) * a.H * a.dk + chan;  // q, k, v in turn
    // a token's address: a scalar and this lane's channel
    const T* x = static_cast<const T*>(a.x[PATH]) + row0;
    const T* dout = static_cast<const T*>(a.d_out[PATH]) + row0;
    T* dx = static_cast<T*>(a.d_x[PATH]) + row0;

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
    // xw[j]: for j < W the input W - j positions before the step's first token,
    // then the step's inputs; pend[j]: the gradient gathered for that position
    float xw[W + kStep][CPL], pend[W + kStep][CPL];
    auto restart = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int64_t s = t - W + j;
#pragma unroll
            for (int c = 0; c < CPL; ++c) xw[j][c] = pend[j][c] = 0.f;
            if (j < low) continue;
            if (s >= bos) {
                Ch r;
                r.load(x + s * stride + chan);
                r.get(xw[j]);
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
            if (s >= t0 && s < t1) Ch::store(dx + s * stride + chan, v);
        } else if (a.d_state_in && bos >= t0 && bos < t1) {
            const int64_t js = (K - 1) - (bos - s);
            if (js >= 0) {
#pragma unroll
                for (int c = 0; c < CPL; ++c)
                    a.d_state_in[(int64_t(n) * nch + state_chan + c) * (K - 1) + js] = v[c];
            }
        }
    };
    // token with its input at xw[W + i]: its part of the gradients
    auto token = [&](int i, const float* g, bool mine) {
        float v[CPL], dy[CPL];
        float ss = 0.f, sv = 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            float y = w[W][c] * xw[W + i][c];
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (j >= low) y = fmaf(w[j][c], xw[i + j][c], y);
            const float sg = fast_sigmoid(y);
            v[c] = y * sg;
            dy[c] = fmaf(v[c], 1.f - sg, sg);  // SiLU'(y)
            if (PATH < 2) {
                ss = fmaf(v[c], v[c], ss);
                sv = fmaf(v[c], g[c], sv);
            }
        }
        float r = 1.f, back = 0.f;
        if (PATH < 2) {
            ss = group_sum<LPH>(ss);
            sv = group_sum<LPH>(sv);
            r = __builtin_amdgcn_rsqf(ss + a.eps_l2);
            back = r * (r * sv);
            if (PATH == 0) r *= a.q_scale;
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            dy[c] = PATH < 2 ? (dy[c] * r) * fmaf(-v[c], back, g[c]) : dy[c] * g[c];  // products side by side
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (j >= low) pend[i + j][c] = fmaf(w[j][c], dy[c], pend[i + j][c]);
            pend[i + W][c] = w[W][c] * dy[c];
        }
        if (mine) {
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (j >= low) {
#pragma unroll
                    for (int c = 0; c < CPL; ++c) dw[j][c] = fmaf(dy[c], xw[i + j][c], dw[j][c]);
                }
        }
    };
    // the window and the unfinished gradients `by` tokens on
    auto advance = [&](auto by) {
        constexpr int S = decltype(by)::value;
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                xw[j][c] = j >= low ? xw[j + S][c] : 0.f;
                pend[j][c] = pend[j + S][c];
            }
    };

    // tokens past t1 complete this run's gradients
    const int64_t last = t0 >= t1 ? t0 : int64_t(t1) + K - 1 < a.T ? t1 + K - 1 : a.T;
    // a whole step inside one sequence, neither its first K - 1 tokens nor its last one
    auto whole = [&](int64_t t) { return t + kStep <= last && t + kStep < eos && t - (K - 1) >= bos; };
    Ch rx[kStep], rg[kStep];
    auto load_step = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            rx[i].load(x + (t + i) * stride + chan);
            rg[i].load(dout + (t + i) * stride + chan);
        }
    };
    if (t0 < t1) restart(t0);
    int64_t ahead = -1;  // the step whose loads are in flight
    for (int64_t t = t0; t < last;) {
        if (whole(t)) {
            if (ahead != t) load_step(t);
            Ch g[kStep];
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                rx[i].get(xw[W + i]);
                g[i] = rg[i];
            }
            if (whole(t + kStep)) {
                load_step(t + kStep);
                ahead = t + kStep;
            }
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                float gi[CPL];
                g[i].get(gi);
                token(i, gi, t + i < t1);
                __builtin_amdgcn_sched_barrier(0);  // tokens interleaved would hold more registers at once
                // position t + i - (K - 1) is inside the sequence and before t1
                if (t + i - (K - 1) >= t0) {
                    if (KM <= 4) {
                        Ch::store(dx + (t + i - (K - 1)) * stride + chan, pend[i]);
                    } else {
#pragma unroll
                        for (int j = 0; j < KM; ++j)
                            if (j == low) Ch::store(dx + (t + i - (K - 1)) * stride + chan, pend[i + j]);
                    }
                }
            }
            advance(std::integral_constant<int, kStep>{});
            t += kStep;
            continue;
        }
        if (t >= eos) {  // the next non-empty sequence starts here (packed input only)
            if (t >= t1) break;
            n = sequence_of(a.cu_seqlens, a.N, a.T, t);
            sequence_bounds(a.cu_seqlens, n, a.T, bos, eos, unused);
            restart(t);
        }
        Ch one;
        float g[CPL];
        one.load(x + t * stride + chan);
        one.get(xw[W]);
        one.load(dout + t * stride + chan);
        one.get(g);
        token(0, g, t < t1);
#pragma unroll
        for (int j = 0; j < KM; ++j)
            if (j == low) finish(t - (K - 1), pend[j]);
        advance(std::integral_constant<int, 1>{});
        if (t == eos - 1) {  // no later token adds to the last K - 1 positions
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (j < low) continue;
                float p[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c)
                    p[c] = pend[j][c] +
                           (a.d_state_out ? a.d_state_out[(int64_t(n) * nch + state_chan + c) * (K - 1) + (j - low)] : 0.f);
                finish(t + 1 - W + j, p);
            }
        }
        ++t;
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

// Gate logits: eight channels a lane over the wavefront's run, eight tokens'
// loads at a time.
template <typename T, int D, int WHICH>
__device__ __forceinline__ void gate_bwd_path(const PrologueBwdArgs& a, int64_t wid, int lane)
{
    constexpr int LPH = D / 8, HPW = 64 / LPH, M = sizeof(T) == 2 ? 8 : 4;
    const int ng = (a.H + HPW - 1) / HPW;
    const int64_t nruns = (int64_t(a.T) + a.run - 1) / a.run;
    if (wid >= int64_t(a.B) * nruns * ng) return;
    const int h = int(wid % ng) * HPW + lane / LPH;
    if (h >= a.H) return;
    const int64_t run = (wid / ng) % nruns, brow = wid / ng / nruns;
    int t0, t1;
    owned_tokens(a, run, t0, t1);
    const int64_t stride = int64_t(a.H) * D, row0 = brow * a.T * stride;
    const int chan = h * D + (lane % LPH) * 8;
    const T* logit = static_cast<const T*>(a.logit[WHICH]) + row0;
    const T* dg = static_cast<const T*>(a.d_gate[WHICH]) + row0;
    T* out = static_cast<T*>(a.d_logit[WHICH]) + row0;
    for (int64_t t = t0; t < t1; t += M) {
        Eight<T> rl[M], rd[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int64_t at = (t + i < t1 ? t + i : t1 - 1) * stride;
            rl[i].load(logit + at + chan);
            rd[i].load(dg + at + chan);
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            if (t + i >= t1) break;
            float l[8], d[8];
            rl[i].get(l);
            rd[i].get(d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = fast_sigmoid(l[j]);
                d[j] *= s * (1.f - s);
            }
            rd[i].put(d);
            rd[i].template store<true>(out + (t + i) * stride + chan);
        }
    }
}

// Sequences without tokens carry their state through, and its gradient back.
__device__ __forceinline__ void empty_sequences_path(const PrologueBwdArgs& a)
{
    if (!a.d_state_in || a.K == 1) return;
    const int64_t per = int64_t(a.H) * (2 * a.dk + a.dv) * (a.K - 1), total = int64_t(a.N) * per;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total; i += int64_t(gridDim.x) * kThreads) {
        int64_t bos, eos, brow;
        sequence_bounds(a.cu_seqlens, int(i / per), a.T, bos, eos, brow);
        if (eos <= bos) a.d_state_in[i] = a.d_state_out ? a.d_state_out[i] : 0.f;
    }
}

// Zeros to the gradients of the tokens in front of the first sequence and behind the
// last, where the call asks for them: two ranges of each buffer.
template <typename T>
__device__ __forceinline__ void padding_path(const PrologueBwdArgs& a)
{
    if (!a.cu_seqlens || !a.zero_padding) return;
    const int first = a.cu_seqlens[0], end = a.cu_seqlens[a.N];
    const int64_t lead = first < 0 ? 0 : first < a.T ? first : a.T, tail = a.T - (end < 0 ? 0 : end < a.T ? end : a.T);
    if (lead == 0 && tail == 0) return;
    const Eight<T> zero = {};
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        T* out = static_cast<T*>(i < 3 ? a.d_x[i] : a.d_logit[i - 3]);
        const int64_t per = int64_t(a.H) * (i == 2 || i == 4 ? a.dv : a.dk) / 8;  // groups of eight a token
        const int64_t skip = (a.T - tail - lead) * per, total = (lead + tail) * per;
        for (int64_t g = int64_t(blockIdx.x) * kThreads + threadIdx.x; g < total; g += int64_t(gridDim.x) * kThreads)
            zero.store(out + (g < lead * per ? g : g + skip) * 8);
    }
}

// blockIdx.y: 0 q, 1 k, 2 v, 3 b, 4 w, 5 the empty sequences and the padding.  The head width is
// looked up here, so a call is one launch whether or not dk = dv.
template <typename T, int KM>
__global__ __launch_bounds__(kThreads) void prologue_bwd_kernel(PrologueBwdArgs a)
{
    const int lane = threadIdx.x % 64;
    // the same in every lane, so runs, sequences and addresses are scalars
    const int64_t wid = int64_t(blockIdx.x) * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    switch (blockIdx.y * 256 + (blockIdx.y == 2 || blockIdx.y == 4 ? a.dv : a.dk)) {
        case 32: conv_bwd_path<T, 32, 0, KM>(a, wid, lane); break;
        case 64: conv_bwd_path<T, 64, 0, KM>(a, wid, lane); break;
        case 128: conv_bwd_path<T, 128, 0, KM>(a, wid, lane); break;
        case 256 + 32: conv_bwd_path<T, 32, 1, KM>(a, wid, lane); break;
        case 256 + 64: conv_bwd_path<T, 64, 1, KM>(a, wid, lane); break;
        case 256 + 128: conv_bwd_path<T, 128, 1, KM>(a, wid, lane); break;
        case 512 + 32: conv_bwd_path<T, 32, 2, KM>(a, wid, lane); break;
        case 512 + 64: conv_bwd_path<T, 64, 2, KM>(a, wid, lane); break;
        case 512 + 128: conv_bwd_path<T, 128, 2, KM>(a, wid, lane); break;
        case 768 + 32: gate_bwd_path<T, 32, 0>(a, wid, lane); break;
        case 768 + 64: gate_bwd_path<T, 64, 0>(a, wid, lane); break;
        case 768 + 128: gate_bwd_path<T, 128, 0>(a, wid, lane); break;
        case 1024 + 32: gate_bwd_path<T, 32, 1>(a, wid, lane); break;
        case 1024 + 64: gate_bwd_path<T, 64, 1>(a, wid, lane); break;
        case 1024 + 128: gate_bwd_path<T, 128, 1>(a, wid, lane); break;
        default: empty_sequences_path(a); padding_path<T>(a); break;
    }
}

template <typename T>
hipError_t prologue_typed(const PrologueBwdArgs& a, hipStream_t stream)
{
    const bool empties = a.d_state_in && a.K > 1 && (a.cu_seqlens || a.T == 0);
    const bool rest = empties || (a.cu_seqlens && a.zero_padding);
    if (a.T > 0 || empties) {
        const int d = a.dk > a.dv ? a.dk : a.dv, hpw = 64 / (d / channels_per_lane(a.K));
        const int64_t waves = int64_t(a.B) * ((int64_t(a.T) + a.run - 1) / a.run) * ((a.H + hpw - 1) / hpw);
        const int64_t blocks = waves > 0 ? (waves + 3) / 4 : 1;
        if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
        const dim3 grid{unsigned(blocks), rest ? 6u : 5u, 1}, block{kThreads, 1, 1};
#define GDN2_TAPS(KM) hipLaunchKernelGGL((prologue_bwd_kernel<T, KM>), grid, block, 0, stream, a)
        switch (a.K) {
            case 1: GDN2_TAPS(1); break;
            case 2: GDN2_TAPS(2); break;
            case 3: GDN2_TAPS(3); break;
            case 4: GDN2_TAPS(4); break;
            default:
                if (a.K <= 8) GDN2_TAPS(8);
                else GDN2_TAPS(16);
        }
#undef GDN2_TAPS
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

// Long runs repeat few tokens at their ends and leave few partial rows; short ones
// give a small call enough wavefronts, and a large one several rounds of the 2048
// that are resident.  So: the longest of 32, 16, 8 (and, for short filters, 4)
// steps that leaves a thousand convolution wavefronts, 32 only with four thousand
// (four taps; longer filters pay more for a run's end).  5003 packed tokens of 6
// heads: 41 us with four steps, 37 with eight; 4096 tokens of 16 heads: 82 us with
// eight, 75 with sixteen; 4 x 4096 FP32 tokens of 16 heads: 462 us with 32, 428 with
// sixteen.  The length is such that a run and the K - 1 tokens after it are whole
// steps.
int32_t prologue_bwd_run(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t K)
{
    const int cpl = channels_per_lane(K), d = dk < dv ? dk : dv, hpw = 64 / (d / cpl);
    const int64_t per_run = 3 * int64_t(B) * ((H + hpw - 1) / hpw);  // convolution wavefronts
    const auto length = [K](int32_t steps) { return steps * kStep - (K - 1); };
    const auto waves = [&](int32_t steps) { return per_run * ((int64_t(T) + length(steps) - 1) / length(steps)); };
    int32_t steps = 32;
    while (steps > (K <= 4 ? 4 : 8) && waves(steps) < (steps == 32 && K <= 4 ? 4096 : 1024)) steps /= 2;
    return length(steps);
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
