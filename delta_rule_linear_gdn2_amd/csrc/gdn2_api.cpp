// C ABI of the GDN-2 library: argument validation and kernel dispatch.
//
// Every check runs on the host before anything is enqueued, so argument
// errors come back synchronously and never reach the device.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <limits>

#include "gdn2.h"
#include "launch.hpp"

namespace {

constexpr int32_t kVersion = 10000;  // 1.0.0

// Tokens per sequence from which gdn2_recurrent_fwd runs the chunkwise kernel
// (measured crossover on MI355X at N = 256, H = 16, d = 128: about 20).
constexpr int32_t kRecurrentChunkMinT = 24;

bool supported_head(int32_t d) { return d == 32 || d == 64 || d == 128; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};

Span span(const void* p, int64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + uintptr_t(bytes)};
}

bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

int element_bytes(gdn2_dtype dt) { return dt == GDN2_DTYPE_BF16 ? 2 : 4; }

// Compute units of the current device, cached per device id.
int32_t device_cus()
{
    static std::atomic<int32_t> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
    if (dev < 64) {
        const int32_t c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
        cus = 256;
    if (dev < 64) cache[dev].store(cus, std::memory_order_relaxed);
    return cus;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Sequence segments for chunkwise calls with few (sequence, head) chains: the
// plan and its workspace.  The matrix-core kernel runs one workgroup per
// (chain, 64-column value tile), one per CU, walking the sequence chunk by
// chunk, so B x H x dv / 64 workgroups leave most of the GPU idle when that
// is small.  Cutting each row into P segments gives P-fold parallelism for
// the cost of a second pass (see segments.hip):
//   pass 1: segments 0 .. P - 2 of every row, each with dv + dk columns (the
//           real ones from a zero state, segment 0 from the caller's; dk map
//           columns from the identity), final states into the workspace;
//           outputs of segment 0 only;
//   combine: the true incoming state of segments 1 .. P - 1;
//   pass 2: segments 1 .. P - 1 from those states, outputs and the final
//           state.
// P is chosen so that pass 1 fills the GPU once (at most one workgroup per
// CU); segments are whole chunks of at least 256 tokens, at least three are
// needed for a gain, and rows shorter than 1024 tokens keep the single pass.
struct SegPlan {
    int32_t P = 0, len = 0;
    size_t out_bytes = 0, in_bytes = 0, total = 0;
};

SegPlan seg_plan(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, bool packed, bool bf16, int32_t cus)
{
    SegPlan sp;
    if (!bf16 || dk != 128 || dv % 64 != 0 || packed || B <= 0 || H <= 0 || T < 1024) return sp;
    const int64_t per_seg = int64_t(B) * H * ((dv + dk) / 64);  // pass-1 workgroups per segment
    const int64_t fit = cus / per_seg;                          // segments pass 1 can hold at once
    if (fit < 2) return sp;
    int64_t P = fit + 1;
    int64_t len = ((T + P - 1) / P + 63) / 64 * 64;
    if (len < 256) len = 256;
    P = (T + len - 1) / len;
    if (P < 3) return sp;
    sp.P = int32_t(P);
    sp.len = int32_t(len);
    sp.out_bytes = align256(size_t(B) * P * H * dk * (dv + dk) * 4);
    sp.in_bytes = align256(size_t(B) * P * H * dk * dv * 4);
    sp.total = sp.out_bytes + sp.in_bytes;
    return sp;
}

}  // namespace

extern "C" {

const char* gdn2_status_string(gdn2_status s)
{
    switch (s) {
        case GDN2_OK: return "GDN2_OK";
        case GDN2_ERR_NULL_POINTER: return "GDN2_ERR_NULL_POINTER: a required pointer is NULL";
        case GDN2_ERR_BAD_SHAPE: return "GDN2_ERR_BAD_SHAPE: invalid or inconsistent sizes";
        case GDN2_ERR_UNSUPPORTED: return "GDN2_ERR_UNSUPPORTED: head size not supported (dk, dv in {32, 64, 128})";
        case GDN2_ERR_BAD_DTYPE: return "GDN2_ERR_BAD_DTYPE: unknown dtype";
        case GDN2_ERR_MISALIGNED: return "GDN2_ERR_MISALIGNED: tensor pointer not 16-byte aligned";
        case GDN2_ERR_ALIAS: return "GDN2_ERR_ALIAS: an output overlaps an input";
        case GDN2_ERR_WORKSPACE: return "GDN2_ERR_WORKSPACE: workspace too small";
        case GDN2_ERR_HIP: return "GDN2_ERR_HIP: the HIP runtime reported an error";
        default: break;
    }
    return "GDN2: unknown status";
}

int32_t gdn2_version(void) { return kVersion; }

size_t gdn2_chunk_fwd_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs,
                                      gdn2_dtype dtype)
{
    return seg_plan(B, T, H, dk, dv, num_seqs > 0, dtype == GDN2_DTYPE_BF16, device_cus()).total;
}

}  // extern "C"

namespace {

// A gate layout: flags only, and the tie only between a scalar erase gate and
// the (then absent) write gate.
bool valid_gates(int32_t g)
{
    const int32_t all = GDN2_GATES_SCALAR_ERASE | GDN2_GATES_SCALAR_WRITE | GDN2_GATES_TIED | GDN2_GATES_SCALAR_DECAY;
    if (g & ~all) return false;
    if (g & GDN2_GATES_TIED) return (g & GDN2_GATES_SCALAR_ERASE) && !(g & GDN2_GATES_SCALAR_WRITE);
    return true;
}

gdn2_status chunk_fwd(const void* q, const void* k, const void* v, const float* alpha, const void* b, const void* w,
                      const float* initial_state, float* final_state, void* o, const int32_t* cu_seqlens, int32_t B,
                      int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs, gdn2_dtype dtype,
                      int32_t gates, void* workspace, size_t workspace_bytes, void* stream)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (!valid_gates(gates)) return GDN2_ERR_BAD_SHAPE;
    if (B <= 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0) return GDN2_ERR_BAD_SHAPE;
    if (cu_seqlens && (B != 1 || num_seqs <= 0)) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dk) || !supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    const bool tied = gates & GDN2_GATES_TIED;
    if (tied) w = nullptr;  // ignored
    const int32_t N = cu_seqlens ? num_seqs : B;
    if (T > 0 && (!q || !k || !v || !alpha || !b || (!tied && !w) || !o)) return GDN2_ERR_NULL_POINTER;
    const void* ptrs[] = {q, k, v, alpha, b, w, o, initial_state, final_state, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_MISALIGNED;
    if (cu_seqlens && (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return GDN2_ERR_MISALIGNED;
    const bool bf16 = dtype == GDN2_DTYPE_BF16;
    // the segmented path runs when the caller passes the workspace it needs
    const SegPlan sp = workspace ? seg_plan(B, T, H, dk, dv, cu_seqlens != nullptr, bf16, device_cus()) : SegPlan{};
    if (sp.P > 0 && workspace_bytes < sp.total) return GDN2_ERR_WORKSPACE;

    const int64_t tokens = int64_t(B) * T * H;
    const int eb = element_bytes(dtype);
    const Span sq = span(q, tokens * dk * eb), sk = span(k, tokens * dk * eb);
    const Span sb = span(b, gates & GDN2_GATES_SCALAR_ERASE ? tokens * eb : tokens * dk * eb);
    const Span sv = span(v, tokens * dv * eb), so = span(o, tokens * dv * eb);
    const Span sw = span(w, tied ? 0 : gates & GDN2_GATES_SCALAR_WRITE ? tokens * eb : tokens * dv * eb);
    const Span sa = span(alpha, gates & GDN2_GATES_SCALAR_DECAY ? tokens * 4 : tokens * dk * 4);
    const int64_t state_bytes = int64_t(N) * H * dk * dv * 4;
    const Span si = span(initial_state, initial_state ? state_bytes : 0);
    const Span sf = span(final_state, final_state ? state_bytes : 0);
    const Span sc = span(cu_seqlens, cu_seqlens ? int64_t(N + 1) * 4 : 0);
    for (Span in : {sq, sk, sv, sa, sb, sw, si, sc})
        if (overlap(so, in)) return GDN2_ERR_ALIAS;
    for (Span in : {sq, sk, sv, sa, sb, sw, sc, so})
        if (overlap(sf, in)) return GDN2_ERR_ALIAS;
    if (overlap(sf, si) && final_state != initial_state) return GDN2_ERR_ALIAS;
    const Span sws = span(workspace, int64_t(sp.total));
    for (Span x : {sq, sk, sv, sa, sb, sw, si, sc, so, sf})
        if (overlap(sws, x)) return GDN2_ERR_ALIAS;

    gdn2::ChunkArgs a{q, k, v, alpha, b, w, initial_state, final_state, o, cu_seqlens,
                      B, T, H, dk, dv, N, device_cus(), gates};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (sp.P > 0 && T > 0) {
        float* seg_out = static_cast<float*>(workspace);
        float* seg_in = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + sp.out_bytes);
        gdn2::ChunkArgs p1 = a;  // pass 1: segments 0 .. P - 2, real and map columns
        p1.dv = dv + dk;
        p1.dv_io = dv;
        p1.N = B * (sp.P - 1);
        p1.seg_len = sp.len;
        p1.seg_total = sp.P;
        p1.seg_first = 0;
        p1.seg_count = sp.P - 1;
        p1.seg_o_all = 0;
        p1.seg_states_out = seg_out;
        gdn2::ChunkArgs p2 = a;  // pass 2: segments 1 .. P - 1 from their true incoming states
        p2.dv_io = dv;
        p2.N = B * (sp.P - 1);
        p2.seg_len = sp.len;
        p2.seg_total = sp.P;
        p2.seg_first = 1;
        p2.seg_count = sp.P - 1;
        p2.seg_o_all = 1;
        p2.seg_states_in = seg_in;
        hipError_t e = gdn2::launch_chunk_fwd_mfma(p1, st);
        if (e == hipSuccess) e = gdn2::launch_segment_combine(seg_out, seg_in, B, H, dk, dv, sp.P, st);
        if (e == hipSuccess) e = gdn2::launch_chunk_fwd_mfma(p2, st);
        return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
    }
    const hipError_t e = gdn2::chunk_fwd_mfma_supported(a, bf16) ? gdn2::launch_chunk_fwd_mfma(a, st)
                                                                 : gdn2::launch_chunk_fwd_simple(a, bf16, st);
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status recurrent(const void* q, const void* k, const void* v, const float* alpha, const void* b, const void* w,
                      float* state, void* o, int32_t N, int32_t T, int32_t H, int32_t dk, int32_t dv,
                      gdn2_dtype dtype, int32_t gates, void* stream)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (!valid_gates(gates)) return GDN2_ERR_BAD_SHAPE;
    if (N <= 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dk) || !supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    const bool tied = gates & GDN2_GATES_TIED;
    if (tied) w = nullptr;  // ignored
    if (!state || (T > 0 && (!q || !k || !v || !alpha || !b || (!tied && !w) || !o))) return GDN2_ERR_NULL_POINTER;
    const void* ptrs[] = {q, k, v, alpha, b, w, state, o};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_MISALIGNED;
    const int64_t tokens = int64_t(N) * T * H;
    const int eb = element_bytes(dtype);
    const Span sq = span(q, tokens * dk * eb), sk = span(k, tokens * dk * eb);
    const Span sb = span(b, gates & GDN2_GATES_SCALAR_ERASE ? tokens * eb : tokens * dk * eb);
    const Span sv = span(v, tokens * dv * eb), so = span(o, tokens * dv * eb);
    const Span sw = span(w, tied ? 0 : gates & GDN2_GATES_SCALAR_WRITE ? tokens * eb : tokens * dv * eb);
    const Span sa = span(alpha, gates & GDN2_GATES_SCALAR_DECAY ? tokens * 4 : tokens * dk * 4);
    const Span ss = span(state, int64_t(N) * H * dk * dv * 4);
    for (Span in : {sq, sk, sv, sa, sb, sw, ss})
        if (overlap(so, in)) return GDN2_ERR_ALIAS;
    for (Span in : {sq, sk, sv, sa, sb, sw})
        if (overlap(ss, in)) return GDN2_ERR_ALIAS;
    if (T == 0) return GDN2_OK;  // nothing to do: the state is unchanged

    // From about 20 tokens per sequence the chunkwise matrix-core kernel is
    // faster (the same mathematics, the [N, T, H, .] inputs taken as a batch,
    // the state updated in place): hand the call to it where it applies.
    const bool bf16 = dtype == GDN2_DTYPE_BF16;
    if (T >= kRecurrentChunkMinT) {
        gdn2::ChunkArgs c{q, k, v, alpha, b, w, state, state, o, nullptr, N, T, H, dk, dv, N, device_cus(), gates};
        if (gdn2::chunk_fwd_mfma_supported(c, bf16)) {
            const hipError_t e = gdn2::launch_chunk_fwd_mfma(c, static_cast<hipStream_t>(stream));
            return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
        }
    }
    gdn2::StepArgs a{q, k, v, alpha, b, w, state, o, N, H, dk, dv, gates, T};
    const hipError_t e = gdn2::launch_recurrent(a, dtype == GDN2_DTYPE_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status mixer_prologue(const void* xq, const void* xk, const void* xv, const float* conv_q,
                           const float* conv_k, const float* conv_v, const void* b_logit, const void* w_logit,
                           const float* conv_state_in, float* conv_state_out, void* q, void* k, void* v, void* b,
                           void* w, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H, int32_t dk,
                           int32_t dv, int32_t K, int32_t num_seqs, float q_scale, float eps_l2, gdn2_dtype dtype,
                           void* stream)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (B <= 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0 || K < 1 || K > 16) return GDN2_ERR_BAD_SHAPE;
    if (cu_seqlens && (B != 1 || num_seqs <= 0)) return GDN2_ERR_BAD_SHAPE;
    if (!(eps_l2 >= 0.f)) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dk) || !supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    const int32_t N = cu_seqlens ? num_seqs : B;
    if (T > 0 && (!xq || !xk || !xv || !conv_q || !conv_k || !conv_v || !b_logit || !w_logit || !q || !k || !v ||
                  !b || !w))
        return GDN2_ERR_NULL_POINTER;
    const void* ptrs[] = {xq, xk, xv, conv_q, conv_k, conv_v, b_logit, w_logit, conv_state_in, conv_state_out,
                          q, k, v, b, w};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_MISALIGNED;
    if (cu_seqlens && (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return GDN2_ERR_MISALIGNED;
    const int64_t tokens = int64_t(B) * T * H;
    const int eb = element_bytes(dtype);
    const int64_t st_bytes = int64_t(N) * H * (2 * dk + dv) * (K - 1) * 4;
    const Span s_in = span(conv_state_in, conv_state_in ? st_bytes : 0);
    const Span in[] = {span(xq, tokens * dk * eb), span(xk, tokens * dk * eb), span(xv, tokens * dv * eb),
                       span(conv_q, int64_t(H) * dk * K * 4), span(conv_k, int64_t(H) * dk * K * 4),
                       span(conv_v, int64_t(H) * dv * K * 4), span(b_logit, tokens * dk * eb),
                       span(w_logit, tokens * dv * eb), s_in,
                       span(cu_seqlens, cu_seqlens ? int64_t(N + 1) * 4 : 0)};
    const Span out[] = {span(q, tokens * dk * eb), span(k, tokens * dk * eb), span(v, tokens * dv * eb),
                        span(b, tokens * dk * eb), span(w, tokens * dv * eb),
                        span(conv_state_out, conv_state_out ? st_bytes : 0)};
    // The state may be updated in place only when each sequence is one token
    // (a decode step): then one wavefront reads and writes each state row.
    const bool in_place_ok = !cu_seqlens && T == 1 && conv_state_out == conv_state_in;
    for (int i = 0; i < 6; ++i) {
        for (const Span& x : in) {
            if (i == 5 && in_place_ok && x.lo == s_in.lo) continue;
            if (overlap(out[i], x)) return GDN2_ERR_ALIAS;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GDN2_ERR_ALIAS;
    }
    gdn2::MixerArgs a{xq, xk, xv, conv_q, conv_k, conv_v, b_logit, w_logit, conv_state_in, conv_state_out,
                      q, k, v, b, w, cu_seqlens, B, T, H, dk, dv, K, N, q_scale, eps_l2};
    const hipError_t e = gdn2::launch_mixer_prologue(a, dtype == GDN2_DTYPE_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status mixer_epilogue(const void* o, const void* gate, const float* weight, void* y, int64_t rows, int32_t dv,
                           float eps, int32_t act, gdn2_dtype dtype, void* stream)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (rows < 0 || dv <= 0 || (act != 0 && act != 1) || !(eps > 0.f)) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    if (rows > 0 && (!o || !gate || !weight || !y)) return GDN2_ERR_NULL_POINTER;
    const void* ptrs[] = {o, gate, weight, y};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_MISALIGNED;
    const int eb = element_bytes(dtype);
    const Span sy = span(y, rows * dv * eb);
    for (Span x : {span(o, rows * dv * eb), span(gate, rows * dv * eb), span(weight, int64_t(dv) * 4)})
        if (overlap(sy, x)) return GDN2_ERR_ALIAS;
    gdn2::EpilogueArgs a{o, gate, weight, y, rows, dv, eps, act};
    const hipError_t e = gdn2::launch_mixer_epilogue(a, dtype == GDN2_DTYPE_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

// Spans of a call's inputs and outputs: every output must be clear of every
// input and of the other outputs, but that output may_out may be input may_in
// exactly (in place).
gdn2_status check_spans(std::initializer_list<Span> in, std::initializer_list<Span> out, int may_out = -1,
                        int may_in = -1)
{
    int i = 0;
    for (const Span& o : out) {
        int j = 0;
        for (const Span& x : in) {
            const bool in_place = i == may_out && j == may_in && o.lo == x.lo;
            if (!in_place && overlap(o, x)) return GDN2_ERR_ALIAS;
            ++j;
        }
        j = 0;
        for (const Span& p : out)
            if (j++ < i && overlap(o, p)) return GDN2_ERR_ALIAS;
        ++i;
    }
    return GDN2_OK;
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

bool misaligned(std::initializer_list<const void*> ptrs)
{
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return true;
    return false;
}

constexpr int64_t kMaxRows = int64_t(1) << 40;  // byte counts of [rows, D] stay far inside 64 bits

// The norms' eps of the training operators: a normal FP32 number.  A row of zeros takes
// 1 / sqrt(eps), and the hardware's reciprocal square root of a subnormal number is infinity.
bool eps_ok(float eps) { return eps >= std::numeric_limits<float>::min(); }

// The dropout arguments, checked: p is a probability, the device offset aligned.
gdn2_status dropout_args(double p, uint64_t seed, uint64_t offset, const uint64_t* offset_device,
                         gdn2::DropoutArgs& d)
{
    if (!(p >= 0.0 && p <= 1.0)) return GDN2_ERR_BAD_SHAPE;
    if (reinterpret_cast<uintptr_t>(offset_device) & 7u) return GDN2_ERR_MISALIGNED;
    const uint32_t threshold = uint32_t(p * 65536.0 + 0.5);
    d = {threshold, threshold < 65536 ? float(65536.0 / (65536 - threshold)) : 0.f, seed, offset, offset_device};
    return GDN2_OK;
}

// Type, size, gate and dropout checks that the block norm's two directions share.
gdn2_status block_norm_check(bool has_u, const void* gate, const float* weight_post, int64_t rows, int32_t D,
                             float eps, int32_t gate_layout, int32_t gate_act, double p, uint64_t seed,
                             uint64_t offset, const uint64_t* offset_device, gdn2_dtype dtype, gdn2_dtype rdtype,
                             gdn2::DropoutArgs& drop)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (rdtype != GDN2_DTYPE_F32 && rdtype != dtype) return GDN2_ERR_BAD_DTYPE;
    if (rows < 0 || rows > kMaxRows || D <= 0 || !eps_ok(eps)) return GDN2_ERR_BAD_SHAPE;
    if (gate_layout < 0 || gate_layout > 3 || gate_act < 0 || gate_act > 2) return GDN2_ERR_BAD_SHAPE;
    if (D > gdn2::kBlockMaxD) return GDN2_ERR_UNSUPPORTED;
    if (gdn2_status s = dropout_args(p, seed, offset, offset_device, drop)) return s;
    if (gate_layout == gdn2::kGateNone && gate) return GDN2_ERR_BAD_SHAPE;
    if (rows > 0 && !has_u && (gate_layout != gdn2::kGateNone || weight_post || drop.threshold))
        return GDN2_ERR_BAD_SHAPE;
    if (gate_layout != gdn2::kGateNone && rows > 0 && !gate) return GDN2_ERR_NULL_POINTER;
    return GDN2_OK;
}

int64_t gate_bytes(int32_t layout, int64_t rows, int32_t D, int eb)
{
    return layout == gdn2::kGateChannel ? int64_t(D) * 4
           : layout == gdn2::kGateToken ? rows * eb
           : layout == gdn2::kGateFull  ? rows * D * eb
                                        : 0;
}

Span span_or_none(const void* p, int64_t bytes) { return span(p, p ? bytes : 0); }

gdn2_status block_norm_fwd(const void* x, const void* u, const void* gate, const float* weight_post,
                           const float* weight_pre, void* x_out, void* h, int64_t rows, int32_t D, float eps,
                           float scale, int32_t gate_layout, int32_t gate_act, double p, uint64_t seed,
                           uint64_t offset, const uint64_t* offset_device, gdn2_dtype dtype, gdn2_dtype rdtype,
                           void* stream)
{
    gdn2::DropoutArgs drop;
    if (gdn2_status s = block_norm_check(u != nullptr, gate, weight_post, rows, D, eps, gate_layout, gate_act, p, seed,
                                         offset, offset_device, dtype, rdtype, drop))
        return s;
    if (!u && x_out) return GDN2_ERR_BAD_SHAPE;
    if (rows > 0 && (!x || (u && !x_out) || (!u && !h) || !weight_pre != !h)) return GDN2_ERR_NULL_POINTER;
    if (misaligned({x, u, gate, weight_post, weight_pre, x_out, h})) return GDN2_ERR_MISALIGNED;
    const int eb = element_bytes(dtype), rb = element_bytes(rdtype);
    const int64_t n = rows * D, wb = int64_t(D) * 4;
    if (gdn2_status s = check_spans(
            {span_or_none(x, n * rb), span_or_none(u, n * eb), span_or_none(gate, gate_bytes(gate_layout, rows, D, eb)),
             span_or_none(weight_post, wb), span_or_none(weight_pre, wb), span_or_none(offset_device, 8)},
            {span_or_none(x_out, n * rb), span_or_none(h, n * eb)}, 0, 0))
        return s;
    gdn2::BlockNormArgs a{x,    u, gate, weight_post, weight_pre, x_out,    h,   rows,
                          D, eps, scale, gate_layout, gate_act,   drop};
    const hipError_t e = gdn2::launch_block_norm_fwd(a, dtype == GDN2_DTYPE_BF16, rdtype == GDN2_DTYPE_BF16,
                                                     static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

size_t block_norm_bwd_workspace(int64_t rows, int32_t D)
{
    if (rows <= 0 || rows > kMaxRows || D <= 0 || D > gdn2::kBlockMaxD) return 0;
    return align256(size_t(gdn2::block_bwd_partials(rows, D)) * 3 * size_t(D) * 4);
}

gdn2_status block_norm_bwd(const void* x_out, const void* u, const void* gate, const float* weight_post,
                           const float* weight_pre, const void* d_x_out, const void* d_h, void* d_x, void* d_u,
                           void* d_gate, float* d_weight_post, float* d_weight_pre, int64_t rows, int32_t D, float eps,
                           float scale, int32_t gate_layout, int32_t gate_act, double p, uint64_t seed,
                           uint64_t offset, const uint64_t* offset_device, gdn2_dtype dtype, gdn2_dtype rdtype,
                           void* workspace, size_t workspace_bytes, void* stream)
{
    gdn2::DropoutArgs drop;
    if (gdn2_status s = block_norm_check(u != nullptr, gate, weight_post, rows, D, eps, gate_layout, gate_act, p, seed,
                                         offset, offset_device, dtype, rdtype, drop))
        return s;
    if ((!u && d_u) || (gate_layout == gdn2::kGateNone && d_gate) || (!weight_post && d_weight_post) ||
        (!weight_pre && d_weight_pre))
        return GDN2_ERR_BAD_SHAPE;
    if (rows > 0 && (!d_x || (u && !d_u) || (weight_pre && !x_out) || (!d_x_out && !d_h) || !weight_pre != !d_h))
        return GDN2_ERR_NULL_POINTER;
    if (misaligned({x_out, u, gate, weight_post, weight_pre, d_x_out, d_h, d_x, d_u, d_gate, d_weight_post,
                    d_weight_pre, workspace}))
        return GDN2_ERR_MISALIGNED;
    const bool sums = d_weight_post || d_weight_pre || (gate_layout == gdn2::kGateChannel && d_gate);
    const size_t need = sums ? block_norm_bwd_workspace(rows, D) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN2_ERR_WORKSPACE;
    const int eb = element_bytes(dtype), rb = element_bytes(rdtype);
    const int64_t n = rows * D, wb = int64_t(D) * 4, gb = gate_bytes(gate_layout, rows, D, eb);
    if (gdn2_status s = check_spans(
            {span_or_none(d_x_out, n * rb), span_or_none(weight_pre ? x_out : nullptr, n * rb), span_or_none(u, n * eb),
             span_or_none(gate, gb), span_or_none(weight_post, wb), span_or_none(weight_pre, wb),
             span_or_none(d_h, n * eb), span_or_none(offset_device, 8)},
            {span_or_none(d_x, n * rb), span_or_none(d_u, n * eb), span_or_none(d_gate, gb),
             span_or_none(d_weight_post, wb), span_or_none(d_weight_pre, wb),
             span_or_none(need ? workspace : nullptr, int64_t(need))},
            0, 0))
        return s;
    gdn2::BlockNormBwdArgs a{x_out, u,     gate,         weight_post,  weight_pre, d_x_out, d_h,   d_x,         d_u,
                             d_gate, d_weight_post, d_weight_pre, rows, D,       eps,   scale,       gate_layout,
                             gate_act, drop, static_cast<float*>(workspace)};
    const hipError_t e = gdn2::launch_block_norm_bwd(a, dtype == GDN2_DTYPE_BF16, rdtype == GDN2_DTYPE_BF16,
                                                     static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status dropout(const void* x, void* y, int64_t rows, int64_t D, double p, uint64_t seed, uint64_t offset,
                    const uint64_t* offset_device, gdn2_dtype dtype, void* stream)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    constexpr int64_t kMost = int64_t(1) << 56;
    if (rows < 0 || D <= 0 || D > kMost || (rows > 0 && (D - 1) / 8 + 1 > (kMost - 1) / rows)) return GDN2_ERR_BAD_SHAPE;
    gdn2::DropoutArgs drop;
    if (gdn2_status s = dropout_args(p, seed, offset, offset_device, drop)) return s;
    if (rows > 0 && (!x || !y)) return GDN2_ERR_NULL_POINTER;
    if (misaligned({x, y})) return GDN2_ERR_MISALIGNED;
    const int eb = element_bytes(dtype);
    if (gdn2_status s = check_spans({span_or_none(x, rows * D * eb), span_or_none(offset_device, 8)},
                                    {span_or_none(y, rows * D * eb)}, 0, 0))
        return s;
    const hipError_t e = gdn2::launch_dropout({x, y, rows, D, drop}, dtype == GDN2_DTYPE_BF16,
                                              static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

size_t epilogue_bwd_workspace(int64_t rows, int32_t dv)
{
    if (rows <= 0 || rows > kMaxRows || !supported_head(dv)) return 0;
    return align256(size_t(gdn2::epilogue_bwd_partials(rows, dv)) * size_t(dv) * 4);
}

gdn2_status mixer_epilogue_bwd(const void* o, const void* gate, const float* weight, const void* d_y, void* d_o,
                               void* d_gate, float* d_weight, int64_t rows, int32_t dv, float eps, int32_t act,
                               gdn2_dtype dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (rows < 0 || rows > kMaxRows || dv <= 0 || (act != 0 && act != 1) || !eps_ok(eps)) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    if (rows > 0 && (!o || !gate || !weight || !d_y || !d_o || !d_gate)) return GDN2_ERR_NULL_POINTER;
    if (misaligned({o, gate, weight, d_y, d_o, d_gate, d_weight, workspace})) return GDN2_ERR_MISALIGNED;
    const size_t need = d_weight ? epilogue_bwd_workspace(rows, dv) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN2_ERR_WORKSPACE;
    const int64_t n = rows * dv * element_bytes(dtype), wb = int64_t(dv) * 4;
    if (gdn2_status s = check_spans({span_or_none(o, n), span_or_none(gate, n), span_or_none(weight, wb), span_or_none(d_y, n)},
                                    {span_or_none(d_o, n), span_or_none(d_gate, n), span_or_none(d_weight, wb),
                                     span_or_none(need ? workspace : nullptr, int64_t(need))}))
        return s;
    gdn2::EpilogueBwdArgs a{o, gate, weight, d_y, d_o, d_gate, d_weight, rows, dv, eps, act, static_cast<float*>(workspace)};
    const hipError_t e = gdn2::launch_mixer_epilogue_bwd(a, dtype == GDN2_DTYPE_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

constexpr int32_t kMaxHeads = 1 << 20;  // a token's channels and filter taps stay far inside 32 bits

// Byte counts of [rows, T, H, d] tensors stay far inside 64 bits.
bool tokens_ok(int64_t rows, int64_t T, int64_t H) { return H <= kMaxHeads && rows * T <= kMaxRows / H; }

size_t prologue_bwd_workspace(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t K)
{
    if (B <= 0 || T <= 0 || H <= 0 || !supported_head(dk) || !supported_head(dv) || K < 1 || K > 16) return 0;
    if (!tokens_ok(B, T, H)) return 0;
    const int64_t run = gdn2::prologue_bwd_run(B, T, H, dk, dv, K), runs = (int64_t(T) + run - 1) / run;
    return align256(size_t(B) * size_t(runs) * size_t(H) * size_t(2 * dk + dv) * size_t(K) * 4);
}

gdn2_status mixer_prologue_bwd(const void* const (&x)[3], const float* const (&conv)[3], const void* const (&logit)[2],
                               const float* conv_state_in, const void* const (&d_out)[3],
                               const void* const (&d_gate)[2], const float* d_state_out, void* const (&d_x)[3],
                               float* const (&d_conv)[3], void* const (&d_logit)[2], float* d_state_in,
                               const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                               int32_t K, int32_t num_seqs, float q_scale, float eps_l2, bool zero_padding,
                               gdn2_dtype dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (B <= 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0 || K < 1 || K > 16) return GDN2_ERR_BAD_SHAPE;
    if (cu_seqlens && (B != 1 || num_seqs <= 0)) return GDN2_ERR_BAD_SHAPE;
    if (!(eps_l2 >= 0.f)) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dk) || !supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    const int32_t N = cu_seqlens ? num_seqs : B;
    if (!tokens_ok(B, T, H) || !tokens_ok(N, 1, H)) return GDN2_ERR_BAD_SHAPE;
    if (T > 0)
        for (const void* p : {x[0], x[1], x[2], static_cast<const void*>(conv[0]), static_cast<const void*>(conv[1]),
                              static_cast<const void*>(conv[2]), logit[0], logit[1], d_out[0], d_out[1], d_out[2],
                              d_gate[0], d_gate[1], static_cast<const void*>(d_x[0]), static_cast<const void*>(d_x[1]),
                              static_cast<const void*>(d_x[2]), static_cast<const void*>(d_logit[0]),
                              static_cast<const void*>(d_logit[1])})
            if (!p) return GDN2_ERR_NULL_POINTER;
    if (misaligned({x[0], x[1], x[2], conv[0], conv[1], conv[2], logit[0], logit[1], conv_state_in, d_out[0], d_out[1],
                    d_out[2], d_gate[0], d_gate[1], d_state_out, d_x[0], d_x[1], d_x[2], d_conv[0], d_conv[1],
                    d_conv[2], d_logit[0], d_logit[1], d_state_in, workspace}))
        return GDN2_ERR_MISALIGNED;
    if (cu_seqlens && (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return GDN2_ERR_MISALIGNED;
    const size_t need = d_conv[0] || d_conv[1] || d_conv[2] ? prologue_bwd_workspace(B, T, H, dk, dv, K) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN2_ERR_WORKSPACE;
    const int64_t tokens = int64_t(B) * T * H, nk = tokens * dk * element_bytes(dtype),
                  nv = tokens * dv * element_bytes(dtype), ck = int64_t(H) * dk * K * 4, cv = int64_t(H) * dv * K * 4;
    const int64_t st = int64_t(N) * H * (2 * dk + dv) * (K - 1) * 4;
    if (gdn2_status s = check_spans(
            {span_or_none(x[0], nk), span_or_none(x[1], nk), span_or_none(x[2], nv), span_or_none(conv[0], ck),
             span_or_none(conv[1], ck), span_or_none(conv[2], cv), span_or_none(logit[0], nk),
             span_or_none(logit[1], nv), span_or_none(conv_state_in, st), span_or_none(d_out[0], nk),
             span_or_none(d_out[1], nk), span_or_none(d_out[2], nv), span_or_none(d_gate[0], nk),
             span_or_none(d_gate[1], nv), span_or_none(d_state_out, st), span_or_none(cu_seqlens, int64_t(N + 1) * 4)},
            {span_or_none(d_x[0], nk), span_or_none(d_x[1], nk), span_or_none(d_x[2], nv), span_or_none(d_conv[0], ck),
             span_or_none(d_conv[1], ck), span_or_none(d_conv[2], cv), span_or_none(d_logit[0], nk),
             span_or_none(d_logit[1], nv), span_or_none(d_state_in, st),
             span_or_none(need ? workspace : nullptr, int64_t(need))}))
        return s;
    gdn2::PrologueBwdArgs a{};
    for (int i = 0; i < 3; ++i) {
        a.x[i] = x[i];
        a.conv[i] = conv[i];
        a.d_out[i] = d_out[i];
        a.d_x[i] = d_x[i];
        a.d_conv[i] = d_conv[i];
    }
    for (int i = 0; i < 2; ++i) {
        a.logit[i] = logit[i];
        a.d_gate[i] = d_gate[i];
        a.d_logit[i] = d_logit[i];
    }
    a.conv_state_in = conv_state_in;
    a.d_state_out = d_state_out;
    a.d_state_in = d_state_in;
    a.cu_seqlens = cu_seqlens;
    a.B = B, a.T = T, a.H = H, a.dk = dk, a.dv = dv, a.K = K, a.N = N;
    a.q_scale = q_scale, a.eps_l2 = eps_l2;
    a.zero_padding = zero_padding;
    a.run = gdn2::prologue_bwd_run(B, T, H, dk, dv, K);
    a.partial = need ? static_cast<float*>(workspace) : nullptr;
    const hipError_t e = gdn2::launch_mixer_prologue_bwd(a, dtype == GDN2_DTYPE_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

// ---- linear attention with a fixed decay for each head ----------------------

constexpr int32_t kLinearMaxHeads = 1 << 15;  // a chunk's rows stay inside the 32 bits of a buffer offset

// Segments of the walks over sequences, and what their carries take.  A walk is
// one workgroup per (segment, head, column slice, walk), one a compute unit at a
// time; more than one segment a sequence takes a launch more, for their carries.
struct LinearPlan {
    int32_t seg_len = 0, segments = 1;
    int64_t slots = 0;       // that the walks for outputs are started for (see linear_attn.hip)
    int64_t carries = 0;     // that the launch for carries is started for
    size_t carry_bytes = 0;  // one state per carry and head; packed, one more for what comes in
};

int32_t linear_slices(int32_t width, int32_t da, bool bf16) { return width / gdn2::linear_slice(width, da, bf16); }

// What the plan needs to know of a call: its workgroups per (sequence, head), in all
// launches for outputs, in the largest of them (a backward with dk != dv has two, one
// behind the other) and in the one for carries.
struct LinearShape {
    int32_t all_subs, subs, carry_subs, widest;
    bool bf16;
};

// Microseconds that a call over B H groups of `chunks` chunks takes in P segments,
// as measured on MI355X for small calls: a workgroup's start and end 5, a chunk
// 1.0 to 1.6 (bf16) or 2.4 to 4.5 (FP32) with heads up to 64 or of 128, reading a
// segment's carry 0.5, the launch for carries 7 and half a walk's slots.  In one
// piece / by this rule, with a state out: 4096 tokens of 16 heads of 128 forward 121 /
// 45, 1024 tokens 35 / 22, 16384 tokens of 2 heads 459 / 55; 512 tokens stay in one
// piece (20).  Backward, FP32, 4096 tokens of 4 heads of 64 x 128: 501 /
// 71; counting the workgroups of its two launches as one's, 91.
double linear_cost(int64_t groups, int64_t chunks, int64_t P, const LinearShape& sh, int64_t cus)
{
    const double chunk = sh.bf16 ? (sh.widest < 128 ? 1.0 : 1.5) : (sh.widest < 128 ? 2.4 : 4.5);
    const double walk = chunk * double((chunks + P - 1) / P);
    const double rounds = double((groups * sh.subs * P + cus - 1) / cus);
    if (P == 1) return rounds * (5 + walk);
    const double carry_rounds = double((groups * sh.carry_subs * (P - 1) + 2 * cus - 1) / (2 * cus));
    return rounds * (5 + walk) + 0.5 * double(P - 1) + 7 + carry_rounds * walk;
}

LinearPlan linear_plan(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs, const LinearShape& sh,
                       int32_t cus)
{
    constexpr int64_t kMost = 64;  // segments a row
    const int64_t rows = num_seqs > 0 ? num_seqs : B, chunk = gdn2::kLinearChunk, chunks = (int64_t(T) + chunk - 1) / chunk;
    LinearPlan p;
    p.seg_len = T > 0 ? T : 1;
    p.slots = rows;
    int64_t len = T;
    if (num_seqs > 0) {
        // The lengths are on the device.  Segments of 0.8 of a compute unit's share of
        // the whole (sequences end inside segments, and a round of fewer chunks more is
        // better than one more chunk: FP32 backward of 3001 tokens in 7 sequences of 4
        // heads of 64 x 128, the mean of three sets of cuts, 67 us at the whole share, 60
        // here and at 0.6), none under four chunks (FP32: two); but where the sequences
        // alone fill the device only what is eight times their mean is cut, which cuts at
        // random hardly ever leave (5003 tokens in 24 sequences of 6 heads 30.2 -> 29.7
        // us, 20000 in 20 of 16 heads 161 -> 144, bf16 backward of 12000 in 6 of 8 heads
        // 125 -> 121).  A long sequence among many short ones loses by it: 32736 tokens
        // beside 32 of one token, 16 heads of 128, 338 us, the same without the 32 210.
        const int64_t groups = int64_t(H) * sh.all_subs;
        len = int64_t(T) * groups * 4 / (5 * int64_t(cus));
        if (groups * num_seqs >= cus) len = std::max(len, 8 * int64_t(T) / num_seqs);
        len = std::max((len + chunk - 1) / chunk * chunk, (sh.bf16 ? 4 : 2) * chunk);
    } else {
        const int64_t groups = int64_t(B) * H;
        double best = linear_cost(groups, chunks, 1, sh, cus);
        for (int64_t P = 2; P <= std::min(chunks, kMost); ++P) {
            const double cost = linear_cost(groups, chunks, P, sh, cus);
            if (cost < best) best = cost, len = (chunks + P - 1) / P * chunk;
        }
    }
    if (len >= T) return p;
    p.seg_len = int32_t(len);
    p.segments = int32_t((T + len - 1) / len);
    p.carries = num_seqs > 0 ? T / len : rows * p.segments;
    p.slots = num_seqs > 0 ? T / len + num_seqs : p.carries;
    p.carry_bytes = align256(size_t(num_seqs > 0 ? 2 * p.carries : p.carries) * size_t(H) * size_t(dk) * size_t(dv) * 4);
    return p;
}

bool linear_sizes(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs)
{
    return B > 0 && T >= 0 && H > 0 && H <= kLinearMaxHeads && num_seqs >= 0 && tokens_ok(B, T, H) &&
           tokens_ok(num_seqs, 1, H) && tokens_ok(B, 1, H) && supported_head(dk) && supported_head(dv);
}

LinearPlan linear_fwd_plan(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs, gdn2_dtype dtype)
{
    const bool bf16 = dtype == GDN2_DTYPE_BF16;
    const int32_t v = linear_slices(dv, dk, bf16);
    return linear_plan(B, T, H, dk, dv, num_seqs, {v, v, v, std::max(dk, dv), bf16}, device_cus());
}

LinearPlan linear_bwd_plan(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs, gdn2_dtype dtype)
{
    const bool bf16 = dtype == GDN2_DTYPE_BF16;
    const int32_t k = linear_slices(dk, dv, bf16), v = linear_slices(dv, dk, bf16);
    const int32_t all = 2 * k + v, most = dk == dv ? all : std::max(2 * k, v);
    return linear_plan(B, T, H, dk, dv, num_seqs, {all, most, 2 * v, std::max(dk, dv), bf16}, device_cus());
}

gdn2::LinearLaunch linear_launch(const float* alpha, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H, int32_t N,
                                 const LinearPlan& p, bool zero_padding)
{
    gdn2::LinearLaunch a{};
    a.alpha = alpha;
    a.cu_seqlens = cu_seqlens;
    a.B = B, a.T = T, a.H = H, a.N = N;
    a.seg_len = p.seg_len, a.segments = p.segments;
    a.units = p.slots * H, a.carry_units = p.carries * H;
    a.pad_blocks = cu_seqlens && zero_padding && T > 0 ? 64 : 0;
    return a;
}

// The sizes, pointers and type that both directions check alike.
gdn2_status linear_check(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs, const float* alpha,
                         const int32_t* cu_seqlens, gdn2_dtype dtype)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (B <= 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0) return GDN2_ERR_BAD_SHAPE;
    if (cu_seqlens && (B != 1 || num_seqs <= 0)) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dk) || !supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    if (!linear_sizes(B, T, H, dk, dv, cu_seqlens ? num_seqs : 0)) return GDN2_ERR_BAD_SHAPE;
    if (!alpha) return GDN2_ERR_NULL_POINTER;
    if (misaligned4(alpha) || misaligned4(cu_seqlens)) return GDN2_ERR_MISALIGNED;
    return GDN2_OK;
}

gdn2_status linear_attn_fwd(const void* q, const void* k, const void* v, const float* alpha, const float* initial_state,
                            float* final_state, void* o, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H,
                            int32_t dk, int32_t dv, int32_t num_seqs, bool zero_padding, gdn2_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream)
{
    if (gdn2_status s = linear_check(B, T, H, dk, dv, num_seqs, alpha, cu_seqlens, dtype)) return s;
    const int32_t N = cu_seqlens ? num_seqs : B;
    if (T > 0 && (!q || !k || !v || !o)) return GDN2_ERR_NULL_POINTER;
    if (misaligned({q, k, v, o, initial_state, final_state, workspace})) return GDN2_ERR_MISALIGNED;
    LinearPlan p = linear_fwd_plan(B, T, H, dk, dv, cu_seqlens ? num_seqs : 0, dtype);
    if (!workspace && p.carry_bytes) {  // one segment a sequence
        p = LinearPlan{};
        p.seg_len = T;
        p.slots = N;
    }
    if (workspace && workspace_bytes < p.carry_bytes) return GDN2_ERR_WORKSPACE;
    const int64_t rows = int64_t(B) * T * H, nk = rows * dk * element_bytes(dtype), nv = rows * dv * element_bytes(dtype);
    const int64_t st = int64_t(N) * H * dk * dv * 4;
    if (gdn2_status s = check_spans({span_or_none(q, nk), span_or_none(k, nk), span_or_none(v, nv), span_or_none(alpha, H * 4),
                                     span_or_none(initial_state, st), span_or_none(cu_seqlens, int64_t(N + 1) * 4)},
                                    {span_or_none(final_state, st), span_or_none(o, nv),
                                     span_or_none(p.carry_bytes ? workspace : nullptr, int64_t(p.carry_bytes))}, 0, 4))
        return s;
    const bool bf16 = dtype == GDN2_DTYPE_BF16, exact = final_state != nullptr;
    gdn2::LinearLaunch a = linear_launch(alpha, cu_seqlens, B, T, H, N, p, zero_padding);
    a.walks = 1;
    a.width = dv;
    a.walk[0] = {q, k, v, o, initial_state, final_state, static_cast<float*>(p.carry_bytes ? workspace : nullptr), dv, 1, 0};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = p.segments > 1 ? gdn2::launch_linear_walk(a, dk, true, exact, bf16, s) : hipSuccess;
    if (e == hipSuccess) e = gdn2::launch_linear_walk(a, dk, false, exact, bf16, s);
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status linear_attn_bwd(const void* q, const void* k, const void* v, const float* alpha, const float* initial_state,
                            const void* d_o, const float* d_final_state, void* dq, void* dk_, void* dv_,
                            float* d_initial_state, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H, int32_t dk,
                            int32_t dv, int32_t num_seqs, bool zero_padding, gdn2_dtype dtype, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    if (gdn2_status s = linear_check(B, T, H, dk, dv, num_seqs, alpha, cu_seqlens, dtype)) return s;
    const int32_t N = cu_seqlens ? num_seqs : B;
    if (T > 0 && (!q || !k || !v || !d_o || !dq || !dk_ || !dv_)) return GDN2_ERR_NULL_POINTER;
    if (misaligned({q, k, v, d_o, initial_state, d_final_state, dq, dk_, dv_, d_initial_state, workspace}))
        return GDN2_ERR_MISALIGNED;
    LinearPlan p = linear_bwd_plan(B, T, H, dk, dv, cu_seqlens ? num_seqs : 0, dtype);
    if (!workspace && p.carry_bytes) {
        p = LinearPlan{};
        p.seg_len = T;
        p.slots = N;
    }
    const size_t need = 2 * p.carry_bytes;
    if (workspace && workspace_bytes < need) return GDN2_ERR_WORKSPACE;
    const int64_t rows = int64_t(B) * T * H, nk = rows * dk * element_bytes(dtype), nv = rows * dv * element_bytes(dtype);
    const int64_t st = int64_t(N) * H * dk * dv * 4;
    if (gdn2_status s = check_spans({span_or_none(q, nk), span_or_none(k, nk), span_or_none(v, nv), span_or_none(alpha, H * 4),
                                     span_or_none(initial_state, st), span_or_none(d_o, nv), span_or_none(d_final_state, st),
                                     span_or_none(cu_seqlens, int64_t(N + 1) * 4)},
                                    {span_or_none(dq, nk), span_or_none(dk_, nk), span_or_none(dv_, nv),
                                     span_or_none(d_initial_state, st),
                                     span_or_none(need ? workspace : nullptr, int64_t(need))}))
        return s;
    const bool bf16 = dtype == GDN2_DTYPE_BF16, exact = d_initial_state != nullptr;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    float* const carry_s = static_cast<float*>(need ? workspace : nullptr);
    float* const carry_r = need ? reinterpret_cast<float*>(static_cast<char*>(workspace) + p.carry_bytes) : nullptr;
    gdn2::LinearLaunch a = linear_launch(alpha, cu_seqlens, B, T, H, N, p, zero_padding);
    hipError_t e = hipSuccess;
    if (p.segments > 1) {
        // the segments' own states, and gradients of states
        a.walks = 2;
        a.width = dv;
        a.walk[0] = {nullptr, k, v, nullptr, initial_state, nullptr, carry_s, dv, 1, 0};
        a.walk[1] = {nullptr, q, d_o, nullptr, d_final_state, nullptr, carry_r, dv, 1, 1};
        e = gdn2::launch_linear_walk(a, dk, true, exact, bf16, s);
    }
    const gdn2::LinearWalk to_k{v, d_o, q, dk_, d_final_state, nullptr, carry_r, 1, dv, 1};
    const gdn2::LinearWalk to_v{k, q, d_o, dv_, d_final_state, d_initial_state, carry_r, dv, 1, 1};
    const gdn2::LinearWalk to_q{d_o, v, k, dq, initial_state, nullptr, carry_s, 1, dv, 0};
    a.walk[0] = to_k;
    a.width = dk;
    if (dk == dv) {  // the walks that read the same rows in the same order run side by side
        a.walk[1] = to_v;
        a.walk[2] = to_q;
        a.walks = 3;
        if (e == hipSuccess) e = gdn2::launch_linear_walk(a, dk, false, exact, bf16, s);
    } else {
        a.walk[1] = to_q;
        a.walks = 2;
        if (e == hipSuccess) e = gdn2::launch_linear_walk(a, dv, false, false, bf16, s);
        a.walk[0] = to_v;
        a.walks = 1;
        a.width = dv;
        if (e == hipSuccess) e = gdn2::launch_linear_walk(a, dk, false, exact, bf16, s);
    }
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status linear_attn_step(const void* q, const void* k, const void* v, const float* alpha, float* state, void* o,
                             int32_t N, int32_t H, int32_t dk, int32_t dv, gdn2_dtype dtype, void* stream)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (N < 0 || H <= 0 || dk <= 0 || dv <= 0) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dk) || !supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    if (!tokens_ok(N, 1, H)) return GDN2_ERR_BAD_SHAPE;
    if (N == 0) return GDN2_OK;
    if (!q || !k || !v || !alpha || !state || !o) return GDN2_ERR_NULL_POINTER;
    if (misaligned({q, k, v, state, o}) || misaligned4(alpha)) return GDN2_ERR_MISALIGNED;
    const int64_t rows = int64_t(N) * H, nk = rows * dk * element_bytes(dtype), nv = rows * dv * element_bytes(dtype);
    if (gdn2_status s = check_spans({span(q, nk), span(k, nk), span(v, nv), span(alpha, int64_t(H) * 4)},
                                    {span(state, rows * dk * dv * 4), span(o, nv)}))
        return s;
    const hipError_t e = gdn2::launch_linear_step({q, k, v, alpha, state, o, N, H, dk, dv}, dtype == GDN2_DTYPE_BF16,
                                                  static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

// ---- norms of queries and keys with the position rotation --------------------

bool qk_sizes(int32_t B, int32_t T, int32_t Hq, int32_t Hk)
{
    return B > 0 && T >= 0 && Hq > 0 && Hk > 0 && Hq <= kLinearMaxHeads && Hk <= kLinearMaxHeads && tokens_ok(B, T, Hq) &&
           tokens_ok(B, T, Hk);
}

size_t qk_norm_rope_bwd_workspace(int32_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t d)
{
    if (!qk_sizes(B, T, Hq, Hk) || !supported_head(d)) return 0;
    return align256(size_t(gdn2::qk_rope_bwd_partials(int64_t(B) * T, Hq, Hk, d)) * 2 * size_t(d) * 4);
}

gdn2_status qk_check(int32_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t d, int32_t rot, const float* inv_freq,
                     const int32_t* positions, float eps, gdn2_dtype dtype)
{
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (!qk_sizes(B, T, Hq, Hk) || d <= 0 || rot < 0 || rot > d || rot % 8 != 0 || !eps_ok(eps)) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(d)) return GDN2_ERR_UNSUPPORTED;
    if (rot > 0 && !inv_freq) return GDN2_ERR_NULL_POINTER;
    if (rot == 0 && inv_freq) return GDN2_ERR_BAD_SHAPE;
    if (misaligned4(positions)) return GDN2_ERR_MISALIGNED;
    return GDN2_OK;
}

gdn2_status qk_norm_rope(const void* q, const void* k, const float* weight_q, const float* weight_k, const float* inv_freq,
                         const int32_t* positions, void* q_out, void* k_out, int32_t B, int32_t T, int32_t Hq, int32_t Hk,
                         int32_t d, int32_t rot, bool neighbours, float q_scale, float eps, gdn2_dtype dtype, void* stream)
{
    if (gdn2_status s = qk_check(B, T, Hq, Hk, d, rot, inv_freq, positions, eps, dtype)) return s;
    if (T == 0) return GDN2_OK;
    if (!q || !k || !q_out || !k_out) return GDN2_ERR_NULL_POINTER;
    if (misaligned({q, k, weight_q, weight_k, inv_freq, q_out, k_out})) return GDN2_ERR_MISALIGNED;
    const int64_t tokens = int64_t(B) * T, row = int64_t(d) * element_bytes(dtype);
    const Span in_q = span(q, tokens * Hq * row), in_k = span(k, tokens * Hk * row), out_q = span(q_out, tokens * Hq * row),
               out_k = span(k_out, tokens * Hk * row);
    const Span w[] = {span_or_none(weight_q, d * 4), span_or_none(weight_k, d * 4), span_or_none(inv_freq, rot * 2),
                      span_or_none(positions, tokens * 4)};
    if (gdn2_status s = check_spans({in_q, w[0], w[1], w[2], w[3]}, {out_q, out_k}, 0, 0)) return s;  // q_out may be q
    if (gdn2_status s = check_spans({in_k}, {out_k, out_q}, 0, 0)) return s;                          // k_out may be k
    gdn2::QkRopeArgs a{{q, k}, {q_out, k_out}, {weight_q, weight_k}, inv_freq, positions, tokens, T, {Hq, Hk}, d, rot,
                       neighbours, q_scale, eps, 0};
    const hipError_t e = gdn2::launch_qk_rope(a, dtype == GDN2_DTYPE_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status qk_norm_rope_bwd(const void* q, const void* k, const float* weight_q, const float* weight_k,
                             const float* inv_freq, const int32_t* positions, const void* d_q_out, const void* d_k_out,
                             void* d_q, void* d_k, float* d_weight_q, float* d_weight_k, int32_t B, int32_t T, int32_t Hq,
                             int32_t Hk, int32_t d, int32_t rot, bool neighbours, float q_scale, float eps,
                             gdn2_dtype dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (gdn2_status s = qk_check(B, T, Hq, Hk, d, rot, inv_freq, positions, eps, dtype)) return s;
    if ((d_weight_q && !weight_q) || (d_weight_k && !weight_k)) return GDN2_ERR_BAD_SHAPE;
    if (T > 0 && (!q || !k || !d_q_out || !d_k_out || !d_q || !d_k)) return GDN2_ERR_NULL_POINTER;
    if (misaligned({q, k, weight_q, weight_k, inv_freq, d_q_out, d_k_out, d_q, d_k, d_weight_q, d_weight_k, workspace}))
        return GDN2_ERR_MISALIGNED;
    const size_t need = d_weight_q || d_weight_k ? qk_norm_rope_bwd_workspace(B, T, Hq, Hk, d) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN2_ERR_WORKSPACE;
    const int64_t tokens = int64_t(B) * T, nq = tokens * Hq * d * element_bytes(dtype), nk = tokens * Hk * d * element_bytes(dtype),
                  nw = int64_t(d) * 4;
    if (gdn2_status s = check_spans({span_or_none(q, nq), span_or_none(k, nk), span_or_none(weight_q, nw), span_or_none(weight_k, nw),
                                     span_or_none(inv_freq, rot * 2), span_or_none(positions, tokens * 4),
                                     span_or_none(d_q_out, nq), span_or_none(d_k_out, nk)},
                                    {span_or_none(d_q, nq), span_or_none(d_k, nk), span_or_none(d_weight_q, nw),
                                     span_or_none(d_weight_k, nw), span_or_none(need ? workspace : nullptr, int64_t(need))}))
        return s;
    gdn2::QkRopeBwdArgs a{{q, k}, {d_q_out, d_k_out}, {d_q, d_k}, {weight_q, weight_k}, {d_weight_q, d_weight_k}, inv_freq,
                          positions, tokens, T, {Hq, Hk}, d, rot, neighbours, q_scale, eps, 0,
                          need ? static_cast<float*>(workspace) : nullptr};
    const hipError_t e = gdn2::launch_qk_rope_bwd(a, dtype == GDN2_DTYPE_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

// Workspace regions of the backward pass.  FP32 path: chunk-start states,
// chunk-end state gradients (slots x H x dk x dv FP32 each, per batch row), U
// and dX rows (B x T x H x dv FP32 each) and each chunk's prepared triangular
// algebra (slots x H per batch row), each region 256-byte aligned.  The
// matrix-core path (bf16, dk = dv = 128, T > 0) puts its range flag in the
// first 256 bytes; after it, its own regions (bf16 states and state gradients
// per 64-token slot, bf16 U and dX rows per slot) and the FP32 path's, which
// runs instead when the flag is raised, share the same memory.
struct BwdWorkspace {
    int64_t slots, slots64;
    size_t states, rows, prep, states16, rows16, total;
    bool mfma;
};

BwdWorkspace bwd_workspace(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, bool varlen, int32_t N,
                           gdn2_dtype dtype)
{
    BwdWorkspace w;
    w.slots = T == 0 ? 0 : (int64_t(T) + gdn2::kBwdChunk - 1) / gdn2::kBwdChunk + (varlen ? N : 0);
    w.states = align256(size_t(B) * size_t(w.slots) * size_t(H) * size_t(dk) * size_t(dv) * 4);
    w.rows = align256(size_t(B) * size_t(T) * size_t(H) * size_t(dv) * 4);
    w.prep = align256(size_t(B) * size_t(w.slots) * size_t(H) * size_t(gdn2::chunk_bwd_prep_floats(dk)) * 4);
    w.total = 2 * w.states + 2 * w.rows + w.prep;
    w.mfma = T > 0 && gdn2::chunk_bwd_mfma_shape(dtype == GDN2_DTYPE_BF16, dk, dv);
    w.slots64 = T == 0 ? 0 : (int64_t(T) + 63) / 64 + (varlen ? N : 0);
    w.states16 = align256(size_t(B) * size_t(w.slots64) * size_t(H) * size_t(dk) * size_t(dv) * 2);
    w.rows16 = align256(size_t(B) * size_t(w.slots64) * size_t(H) * 64 * size_t(dv) * 2);
    if (w.mfma) w.total = 256 + std::max(w.total, 2 * w.states16 + 2 * w.rows16);
    return w;
}

// Host-side checks of a backward call (no HIP call): sizes, pointers,
// alignment, workspace size and overlaps.  ws receives the workspace layout.
// With own_workspace the library supplies the workspace itself: the caller's
// workspace arguments are ignored and no workspace check is made here.
gdn2_status chunk_bwd_check(const void* q, const void* k, const void* v, const float* alpha, const void* b,
                            const void* w, const float* initial_state, const void* d_o, const float* d_final_state,
                            void* dq, void* dk_, void* dv_, float* dalpha, void* db, void* dw,
                            float* d_initial_state, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H,
                            int32_t dk, int32_t dv, int32_t num_seqs, gdn2_dtype dtype, const void* workspace,
                            size_t workspace_bytes, bool own_workspace, BwdWorkspace& ws)
{
    if (own_workspace) {
        workspace = nullptr;
        workspace_bytes = 0;
    }
    if (dtype != GDN2_DTYPE_F32 && dtype != GDN2_DTYPE_BF16) return GDN2_ERR_BAD_DTYPE;
    if (B <= 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0) return GDN2_ERR_BAD_SHAPE;
    if (cu_seqlens && (B != 1 || num_seqs <= 0)) return GDN2_ERR_BAD_SHAPE;
    if (!supported_head(dk) || !supported_head(dv)) return GDN2_ERR_UNSUPPORTED;
    const int32_t N = cu_seqlens ? num_seqs : B;
    if (T > 0 && (!q || !k || !v || !alpha || !b || !w || !d_o || !dq || !dk_ || !dv_ || !dalpha || !db || !dw))
        return GDN2_ERR_NULL_POINTER;
    const void* ptrs[] = {q, k, v, alpha, b, w, initial_state, d_o, d_final_state,
                          dq, dk_, dv_, dalpha, db, dw, d_initial_state, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_MISALIGNED;
    if (cu_seqlens && (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return GDN2_ERR_MISALIGNED;

    ws = bwd_workspace(B, T, H, dk, dv, cu_seqlens != nullptr, N, dtype);
    if (!own_workspace && ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return GDN2_ERR_WORKSPACE;

    const int64_t tokens = int64_t(B) * T * H;
    const int eb = element_bytes(dtype);
    const int64_t state_bytes = int64_t(N) * H * dk * dv * 4;
    const Span in[] = {span(q, tokens * dk * eb), span(k, tokens * dk * eb), span(v, tokens * dv * eb),
                       span(alpha, tokens * dk * 4), span(b, tokens * dk * eb), span(w, tokens * dv * eb),
                       span(initial_state, initial_state ? state_bytes : 0), span(d_o, tokens * dv * eb),
                       span(d_final_state, d_final_state ? state_bytes : 0),
                       span(cu_seqlens, cu_seqlens ? int64_t(N + 1) * 4 : 0)};
    const Span out[] = {span(dq, tokens * dk * eb), span(dk_, tokens * dk * eb), span(dv_, tokens * dv * eb),
                        span(dalpha, tokens * dk * 4), span(db, tokens * dk * eb), span(dw, tokens * dv * eb),
                        span(d_initial_state, d_initial_state ? state_bytes : 0),
                        span(workspace, ws.total > 0 && !own_workspace ? int64_t(ws.total) : 0)};
    constexpr int kDInit = 6;
    for (int i = 0; i < 8; ++i) {
        for (const Span& x : in) {
            // the initial-state gradient may replace the final-state gradient in place
            if (i == kDInit && d_initial_state == d_final_state && x.lo == in[8].lo) continue;
            if (overlap(out[i], x)) return GDN2_ERR_ALIAS;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GDN2_ERR_ALIAS;
    }
    return GDN2_OK;
}

// Launches a checked backward call on the given workspace.
gdn2_status chunk_bwd_launch(const void* q, const void* k, const void* v, const float* alpha, const void* b,
                             const void* w, const float* initial_state, const void* d_o, const float* d_final_state,
                             void* dq, void* dk_, void* dv_, float* dalpha, void* db, void* dw,
                             float* d_initial_state, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H,
                             int32_t dk, int32_t dv, int32_t num_seqs, gdn2_dtype dtype, void* workspace,
                             const BwdWorkspace& ws, void* stream)
{
    const int32_t N = cu_seqlens ? num_seqs : B;
    gdn2::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.alpha = alpha; a.b = b; a.w = w;
    a.initial_state = initial_state; a.d_o = d_o; a.d_final_state = d_final_state;
    a.dq = dq; a.dk = dk_; a.dv = dv_; a.dalpha = dalpha; a.db = db; a.dw = dw;
    a.d_initial_state = d_initial_state; a.cu_seqlens = cu_seqlens;
    a.B = B; a.T = T; a.H = H; a.dk_ = dk; a.dv_ = dv; a.N = N;
    a.slots = ws.slots;
    unsigned char* base = static_cast<unsigned char*>(workspace);
    if (ws.mfma) {
        a.range_flag = reinterpret_cast<int32_t*>(base);
        base += 256;
        a.slots64 = ws.slots64;
        a.ws_s16 = reinterpret_cast<uint16_t*>(base);
        a.ws_ds16 = reinterpret_cast<uint16_t*>(base + ws.states16);
        a.ws_u16 = reinterpret_cast<uint16_t*>(base + 2 * ws.states16);
        a.ws_dx16 = reinterpret_cast<uint16_t*>(base + 2 * ws.states16 + ws.rows16);
    }
    a.ws_states = ws.total ? reinterpret_cast<float*>(base) : nullptr;
    a.ws_dstates = ws.total ? reinterpret_cast<float*>(base + ws.states) : nullptr;
    a.ws_u = ws.total ? reinterpret_cast<float*>(base + 2 * ws.states) : nullptr;
    a.ws_dx = ws.total ? reinterpret_cast<float*>(base + 2 * ws.states + ws.rows) : nullptr;
    a.ws_prep = ws.total ? reinterpret_cast<float*>(base + 2 * ws.states + 2 * ws.rows) : nullptr;
    const hipError_t e = ws.mfma ? gdn2::launch_chunk_bwd_mfma(a, static_cast<hipStream_t>(stream))
                                 : gdn2::launch_chunk_bwd(a, dtype == GDN2_DTYPE_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP;
}

gdn2_status chunk_bwd(const void* q, const void* k, const void* v, const float* alpha, const void* b, const void* w,
                      const float* initial_state, const void* d_o, const float* d_final_state, void* dq, void* dk_,
                      void* dv_, float* dalpha, void* db, void* dw, float* d_initial_state,
                      const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                      int32_t num_seqs, gdn2_dtype dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    BwdWorkspace ws{};
    const gdn2_status st = chunk_bwd_check(q, k, v, alpha, b, w, initial_state, d_o, d_final_state, dq, dk_, dv_,
                                           dalpha, db, dw, d_initial_state, cu_seqlens, B, T, H, dk, dv, num_seqs,
                                           dtype, workspace, workspace_bytes, false, ws);
    if (st != GDN2_OK) return st;
    return chunk_bwd_launch(q, k, v, alpha, b, w, initial_state, d_o, d_final_state, dq, dk_, dv_, dalpha, db, dw,
                            d_initial_state, cu_seqlens, B, T, H, dk, dv, num_seqs, dtype, workspace, ws, stream);
}

// The same on the library's own scratch array: the host checks run first
// (the array cannot overlap caller memory), then the workspace size against
// the array's capacity (larger: GDN2_ERR_WORKSPACE); then the array's device
// address on the current device is looked up (once per device) and the
// kernels run on it.  Nothing is allocated.
gdn2_status chunk_bwd_noalloc(const void* q, const void* k, const void* v, const float* alpha, const void* b,
                              const void* w, const float* initial_state, const void* d_o,
                              const float* d_final_state, void* dq, void* dk_, void* dv_, float* dalpha, void* db,
                              void* dw, float* d_initial_state, const int32_t* cu_seqlens, int32_t B, int32_t T,
                              int32_t H, int32_t dk, int32_t dv, int32_t num_seqs, gdn2_dtype dtype, void* stream)
{
    BwdWorkspace ws{};
    const gdn2_status st = chunk_bwd_check(q, k, v, alpha, b, w, initial_state, d_o, d_final_state, dq, dk_, dv_,
                                           dalpha, db, dw, d_initial_state, cu_seqlens, B, T, H, dk, dv, num_seqs,
                                           dtype, nullptr, 0, true, ws);
    if (st != GDN2_OK) return st;
    if (ws.total > gdn2::kScratchBytes) return GDN2_ERR_WORKSPACE;
    void* scratch = nullptr;
    if (ws.total > 0 && gdn2::scratch_pointer(&scratch) != hipSuccess) return GDN2_ERR_HIP;
    return chunk_bwd_launch(q, k, v, alpha, b, w, initial_state, d_o, d_final_state, dq, dk_, dv_, dalpha, db, dw,
                            d_initial_state, cu_seqlens, B, T, H, dk, dv, num_seqs, dtype, scratch, ws, stream);
}

}  // namespace

extern "C" {

gdn2_status gdn2_chunk_fwd(const void* q, const void* k, const void* v, const float* alpha,
                           const void* b, const void* w, const float* initial_state,
                           float* final_state, void* o, const int32_t* cu_seqlens, int32_t B,
                           int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs,
                           gdn2_dtype dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    return chunk_fwd(q, k, v, alpha, b, w, initial_state, final_state, o, cu_seqlens, B, T, H, dk, dv, num_seqs,
                     dtype, GDN2_GATES_FULL, workspace, workspace_bytes, stream);
}

gdn2_status gdn2_chunk_fwd_gates(const void* q, const void* k, const void* v, const float* alpha,
                                 const void* b, const void* w, const float* initial_state,
                                 float* final_state, void* o, const int32_t* cu_seqlens, int32_t B,
                                 int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs,
                                 gdn2_dtype dtype, int32_t gates, void* workspace,
                                 size_t workspace_bytes, void* stream)
{
    return chunk_fwd(q, k, v, alpha, b, w, initial_state, final_state, o, cu_seqlens, B, T, H, dk, dv, num_seqs,
                     dtype, gates, workspace, workspace_bytes, stream);
}

gdn2_status gdn2_recurrent_step(const void* q, const void* k, const void* v, const float* alpha,
                                const void* b, const void* w, float* state, void* o, int32_t N,
                                int32_t H, int32_t dk, int32_t dv, gdn2_dtype dtype, void* stream)
{
    return recurrent(q, k, v, alpha, b, w, state, o, N, 1, H, dk, dv, dtype, GDN2_GATES_FULL, stream);
}

gdn2_status gdn2_recurrent_step_gates(const void* q, const void* k, const void* v, const float* alpha,
                                      const void* b, const void* w, float* state, void* o, int32_t N,
                                      int32_t H, int32_t dk, int32_t dv, gdn2_dtype dtype,
                                      int32_t gates, void* stream)
{
    return recurrent(q, k, v, alpha, b, w, state, o, N, 1, H, dk, dv, dtype, gates, stream);
}

gdn2_status gdn2_recurrent_fwd(const void* q, const void* k, const void* v, const float* alpha, const void* b,
                               const void* w, float* state, void* o, int32_t N, int32_t T, int32_t H, int32_t dk,
                               int32_t dv, gdn2_dtype dtype, int32_t gates, void* stream)
{
    return recurrent(q, k, v, alpha, b, w, state, o, N, T, H, dk, dv, dtype, gates, stream);
}

gdn2_status gdn2_chunk_bwd(const void* q, const void* k, const void* v, const float* alpha, const void* b,
                           const void* w, const float* initial_state, const void* d_o, const float* d_final_state,
                           void* dq, void* dk, void* dv, float* dalpha, void* db, void* dw, float* d_initial_state,
                           const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H, int32_t dk_size,
                           int32_t dv_size, int32_t num_seqs, gdn2_dtype dtype, void* workspace,
                           size_t workspace_bytes, void* stream)
{
    return chunk_bwd(q, k, v, alpha, b, w, initial_state, d_o, d_final_state, dq, dk, dv, dalpha, db, dw,
                     d_initial_state, cu_seqlens, B, T, H, dk_size, dv_size, num_seqs, dtype, workspace,
                     workspace_bytes, stream);
}

gdn2_status gdn2_chunk_bwd_noalloc(const void* q, const void* k, const void* v, const float* alpha, const void* b,
                                   const void* w, const float* initial_state, const void* d_o,
                                   const float* d_final_state, void* dq, void* dk, void* dv, float* dalpha, void* db,
                                   void* dw, float* d_initial_state, const int32_t* cu_seqlens, int32_t B, int32_t T,
                                   int32_t H, int32_t dk_size, int32_t dv_size, int32_t num_seqs, gdn2_dtype dtype,
                                   void* stream)
{
    return chunk_bwd_noalloc(q, k, v, alpha, b, w, initial_state, d_o, d_final_state, dq, dk, dv, dalpha, db, dw,
                             d_initial_state, cu_seqlens, B, T, H, dk_size, dv_size, num_seqs, dtype, stream);
}

size_t gdn2_chunk_bwd_noalloc_max_workspace_bytes(void) { return gdn2::kScratchBytes; }

size_t gdn2_chunk_bwd_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs,
                                      gdn2_dtype dtype)
{
    (void)dtype;
    if (B <= 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0) return 0;
    return bwd_workspace(B, T, H, dk, dv, num_seqs > 0, num_seqs, dtype).total;
}

gdn2_status gdn2_mixer_prologue(const void* xq, const void* xk, const void* xv, const float* conv_q,
                                const float* conv_k, const float* conv_v, const void* b_logit, const void* w_logit,
                                const float* conv_state_in, float* conv_state_out, void* q, void* k, void* v,
                                void* b, void* w, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H,
                                int32_t dk, int32_t dv, int32_t kernel_size, int32_t num_seqs, float q_scale,
                                float eps_l2, gdn2_dtype dtype, void* stream)
{
    return mixer_prologue(xq, xk, xv, conv_q, conv_k, conv_v, b_logit, w_logit, conv_state_in, conv_state_out, q, k,
                          v, b, w, cu_seqlens, B, T, H, dk, dv, kernel_size, num_seqs, q_scale, eps_l2, dtype,
                          stream);
}

gdn2_status gdn2_mixer_epilogue(const void* o, const void* gate, const float* weight, void* y, int64_t rows,
                                int32_t dv, float eps, int32_t gate_act, gdn2_dtype dtype, void* stream)
{
    return mixer_epilogue(o, gate, weight, y, rows, dv, eps, gate_act, dtype, stream);
}

gdn2_status gdn2_block_norm_fwd(const void* x, const void* u, const void* gate, const float* weight_post,
                                const float* weight_pre, void* x_out, void* h, int64_t rows, int32_t D, float eps,
                                float residual_scale, int32_t gate_layout, int32_t gate_act, double dropout_p,
                                uint64_t seed, uint64_t offset, const uint64_t* offset_device, gdn2_dtype dtype,
                                gdn2_dtype residual_dtype, void* stream)
{
    return block_norm_fwd(x, u, gate, weight_post, weight_pre, x_out, h, rows, D, eps, residual_scale, gate_layout,
                          gate_act, dropout_p, seed, offset, offset_device, dtype, residual_dtype, stream);
}

gdn2_status gdn2_block_norm_bwd(const void* x_out, const void* u, const void* gate, const float* weight_post,
                                const float* weight_pre, const void* d_x_out, const void* d_h, void* d_x, void* d_u,
                                void* d_gate, float* d_weight_post, float* d_weight_pre, int64_t rows, int32_t D,
                                float eps, float residual_scale, int32_t gate_layout, int32_t gate_act,
                                double dropout_p, uint64_t seed, uint64_t offset, const uint64_t* offset_device,
                                gdn2_dtype dtype, gdn2_dtype residual_dtype, void* workspace, size_t workspace_bytes,
                                void* stream)
{
    return block_norm_bwd(x_out, u, gate, weight_post, weight_pre, d_x_out, d_h, d_x, d_u, d_gate, d_weight_post,
                          d_weight_pre, rows, D, eps, residual_scale, gate_layout, gate_act, dropout_p, seed, offset,
                          offset_device, dtype, residual_dtype, workspace, workspace_bytes, stream);
}

size_t gdn2_block_norm_bwd_workspace_bytes(int64_t rows, int32_t D) { return block_norm_bwd_workspace(rows, D); }

gdn2_status gdn2_dropout(const void* x, void* y, int64_t rows, int64_t D, double dropout_p, uint64_t seed,
                         uint64_t offset, const uint64_t* offset_device, gdn2_dtype dtype, void* stream)
{
    return dropout(x, y, rows, D, dropout_p, seed, offset, offset_device, dtype, stream);
}

gdn2_status gdn2_mixer_epilogue_bwd(const void* o, const void* gate, const float* weight, const void* d_y, void* d_o,
                                    void* d_gate, float* d_weight, int64_t rows, int32_t dv, float eps,
                                    int32_t gate_act, gdn2_dtype dtype, void* workspace, size_t workspace_bytes,
                                    void* stream)
{
    return mixer_epilogue_bwd(o, gate, weight, d_y, d_o, d_gate, d_weight, rows, dv, eps, gate_act, dtype, workspace,
                              workspace_bytes, stream);
}

size_t gdn2_mixer_epilogue_bwd_workspace_bytes(int64_t rows, int32_t dv) { return epilogue_bwd_workspace(rows, dv); }

gdn2_status gdn2_mixer_prologue_bwd(const void* xq, const void* xk, const void* xv, const float* conv_q,
                                    const float* conv_k, const float* conv_v, const void* b_logit,
                                    const void* w_logit, const float* conv_state_in, const void* d_q, const void* d_k,
                                    const void* d_v, const void* d_b, const void* d_w, const float* d_conv_state_out,
                                    void* d_xq, void* d_xk, void* d_xv, float* d_conv_q, float* d_conv_k,
                                    float* d_conv_v, void* d_b_logit, void* d_w_logit, float* d_conv_state_in,
                                    const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H, int32_t dk,
                                    int32_t dv, int32_t kernel_size, int32_t num_seqs, float q_scale, float eps_l2,
                                    gdn2_dtype dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    return mixer_prologue_bwd({xq, xk, xv}, {conv_q, conv_k, conv_v}, {b_logit, w_logit}, conv_state_in,
                              {d_q, d_k, d_v}, {d_b, d_w}, d_conv_state_out, {d_xq, d_xk, d_xv},
                              {d_conv_q, d_conv_k, d_conv_v}, {d_b_logit, d_w_logit}, d_conv_state_in, cu_seqlens, B,
                              T, H, dk, dv, kernel_size, num_seqs, q_scale, eps_l2, false, dtype, workspace,
                              workspace_bytes, stream);
}

gdn2_status gdn2_mixer_prologue_bwd_zeroed(const void* xq, const void* xk, const void* xv, const float* conv_q,
                                           const float* conv_k, const float* conv_v, const void* b_logit,
                                           const void* w_logit, const float* conv_state_in, const void* d_q,
                                           const void* d_k, const void* d_v, const void* d_b, const void* d_w,
                                           const float* d_conv_state_out, void* d_xq, void* d_xk, void* d_xv,
                                           float* d_conv_q, float* d_conv_k, float* d_conv_v, void* d_b_logit,
                                           void* d_w_logit, float* d_conv_state_in, const int32_t* cu_seqlens,
                                           int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                                           int32_t kernel_size, int32_t num_seqs, float q_scale, float eps_l2,
                                           gdn2_dtype dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    return mixer_prologue_bwd({xq, xk, xv}, {conv_q, conv_k, conv_v}, {b_logit, w_logit}, conv_state_in,
                              {d_q, d_k, d_v}, {d_b, d_w}, d_conv_state_out, {d_xq, d_xk, d_xv},
                              {d_conv_q, d_conv_k, d_conv_v}, {d_b_logit, d_w_logit}, d_conv_state_in, cu_seqlens, B,
                              T, H, dk, dv, kernel_size, num_seqs, q_scale, eps_l2, true, dtype, workspace,
                              workspace_bytes, stream);
}

size_t gdn2_mixer_prologue_bwd_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv,
                                               int32_t kernel_size)
{
    return prologue_bwd_workspace(B, T, H, dk, dv, kernel_size);
}

gdn2_status gdn2_linear_attn_fwd(const void* q, const void* k, const void* v, const float* alpha,
                                 const float* initial_state, float* final_state, void* o, const int32_t* cu_seqlens,
                                 int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs,
                                 int32_t zero_padding, gdn2_dtype dtype, void* workspace, size_t workspace_bytes,
                                 void* stream)
{
    return linear_attn_fwd(q, k, v, alpha, initial_state, final_state, o, cu_seqlens, B, T, H, dk, dv, num_seqs,
                           zero_padding != 0, dtype, workspace, workspace_bytes, stream);
}

size_t gdn2_linear_attn_fwd_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t num_seqs,
                                            gdn2_dtype dtype)
{
    return linear_sizes(B, T, H, dk, dv, num_seqs) ? linear_fwd_plan(B, T, H, dk, dv, num_seqs, dtype).carry_bytes : 0;
}

gdn2_status gdn2_linear_attn_bwd(const void* q, const void* k, const void* v, const float* alpha,
                                 const float* initial_state, const void* d_o, const float* d_final_state, void* dq,
                                 void* dk, void* dv, float* d_initial_state, const int32_t* cu_seqlens, int32_t B,
                                 int32_t T, int32_t H, int32_t dk_size, int32_t dv_size, int32_t num_seqs,
                                 int32_t zero_padding, gdn2_dtype dtype, void* workspace, size_t workspace_bytes,
                                 void* stream)
{
    return linear_attn_bwd(q, k, v, alpha, initial_state, d_o, d_final_state, dq, dk, dv, d_initial_state, cu_seqlens, B,
                           T, H, dk_size, dv_size, num_seqs, zero_padding != 0, dtype, workspace, workspace_bytes, stream);
}

size_t gdn2_linear_attn_bwd_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t dk_size, int32_t dv_size,
                                            int32_t num_seqs, gdn2_dtype dtype)
{
    return linear_sizes(B, T, H, dk_size, dv_size, num_seqs)
               ? 2 * linear_bwd_plan(B, T, H, dk_size, dv_size, num_seqs, dtype).carry_bytes
               : 0;
}

gdn2_status gdn2_linear_attn_step(const void* q, const void* k, const void* v, const float* alpha, float* state, void* o,
                                  int32_t N, int32_t H, int32_t dk, int32_t dv, gdn2_dtype dtype, void* stream)
{
    return linear_attn_step(q, k, v, alpha, state, o, N, H, dk, dv, dtype, stream);
}

gdn2_status gdn2_qk_norm_rope(const void* q, const void* k, const float* weight_q, const float* weight_k,
                              const float* inv_freq, const int32_t* positions, void* q_out, void* k_out, int32_t B,
                              int32_t T, int32_t Hq, int32_t Hk, int32_t d, int32_t rot, int32_t interleaved,
                              float q_scale, float eps, gdn2_dtype dtype, void* stream)
{
    return qk_norm_rope(q, k, weight_q, weight_k, inv_freq, positions, q_out, k_out, B, T, Hq, Hk, d, rot,
                        interleaved != 0, q_scale, eps, dtype, stream);
}

gdn2_status gdn2_qk_norm_rope_bwd(const void* q, const void* k, const float* weight_q, const float* weight_k,
                                  const float* inv_freq, const int32_t* positions, const void* d_q_out,
                                  const void* d_k_out, void* d_q, void* d_k, float* d_weight_q, float* d_weight_k,
                                  int32_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t d, int32_t rot,
                                  int32_t interleaved, float q_scale, float eps, gdn2_dtype dtype, void* workspace,
                                  size_t workspace_bytes, void* stream)
{
    return qk_norm_rope_bwd(q, k, weight_q, weight_k, inv_freq, positions, d_q_out, d_k_out, d_q, d_k, d_weight_q,
                            d_weight_k, B, T, Hq, Hk, d, rot, interleaved != 0, q_scale, eps, dtype, workspace,
                            workspace_bytes, stream);
}

size_t gdn2_qk_norm_rope_bwd_workspace_bytes(int32_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t d)
{
    return qk_norm_rope_bwd_workspace(B, T, Hq, Hk, d);
}

}  // extern "C"
