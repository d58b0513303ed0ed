// Host-visible launch interface between the C ABI layer and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn2 {

// Gate layout flags (the values of gdn2_gate_flags).
constexpr int32_t kScalarErase = 1, kScalarWrite = 2, kTied = 4, kScalarDecay = 8;

struct ChunkArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* alpha;
    const void* b;
    const void* w;
    const float* initial_state;
    float* final_state;
    void* o;
    const int32_t* cu_seqlens;
    int32_t B, T, H, dk, dv, N;
    int32_t cus;    // compute units of the device
    int32_t gates;  // gdn2_gate_flags, validated: 1 scalar erase, 2 scalar write, 4 write tied to erase, 8 scalar decay
    // Sequence segments (matrix-core kernel only; seg_len = 0: off).  Each
    // batch row (no cu_seqlens) is cut into seg_total segments of seg_len
    // tokens (the last may be shorter); launch sequence n is segment
    // seg_first + n % seg_count of row n / seg_count, and N = B * seg_count.
    // Value columns j >= dv_io are map columns: they start from the identity
    // (column j holds e_{j - dv_io}), take z = 0 and write no output, so they
    // carry the segment's state map.  Initial state of a segment: from
    // seg_states_in ([B][seg_total][H][dk][dv_io]) if given, else the
    // caller's initial_state for segment 0 and zero otherwise.  Final state:
    // into seg_states_out ([B][seg_total][H][dk][dv], every column) if given,
    // else the caller's final_state for the row's last segment.  o (dv_io
    // columns) is written for every segment when seg_o_all, else for segment
    // 0 only.
    int32_t seg_len, seg_total, seg_first, seg_count, seg_o_all;
    int32_t dv_io;  // columns of v, w, o and the caller's states (0: dv)
    const float* seg_states_in;
    float* seg_states_out;
};

struct StepArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* alpha;
    const void* b;
    const void* w;
    float* state;
    void* o;
    int32_t N, H, dk, dv;
    int32_t gates;  // as in ChunkArgs
    int32_t T;      // tokens per sequence: inputs [N, T, H, .], o [N, T, H, dv]
};

// Chunkwise backward.  Chunk-start states and chunk-end state gradients sit
// in "slots": slot m of batch row n for packed-free input, and for packed
// sequences slot (bos + m * kBwdChunk) / kBwdChunk + n of row 0 (distinct
// for distinct chunks, fewer than ceil(T / kBwdChunk) + N).
constexpr int kBwdChunk = 32;

struct BwdArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* alpha;
    const void* b;
    const void* w;
    const float* initial_state;
    const void* d_o;
    const float* d_final_state;
    void* dq;
    void* dk;
    void* dv;
    float* dalpha;
    void* db;
    void* dw;
    float* d_initial_state;
    const int32_t* cu_seqlens;
    int32_t B, T, H, dk_, dv_, N;
    int64_t slots;       // chunk slots per batch row
    float* ws_states;    // [B][slots][H][dk][dv] state at each chunk start
    float* ws_dstates;   // [B][slots][H][dk][dv] gradient of the state at each chunk end
    float* ws_u;         // [B * T * H][dv] U rows
    float* ws_dx;        // [B * T * H][dv] dX rows
    float* ws_prep;      // [B][slots][H][chunk_bwd_prep_floats(dk)] per-chunk triangular algebra
    // The matrix-core path (bf16, dk = dv = 128, 64-token chunks), whose
    // workspace shares the memory above:
    int64_t slots64;     // 64-token chunk slots per batch row
    uint16_t* ws_s16;     // [B][slots64][H][dk][dv] state at each chunk start
    uint16_t* ws_ds16;    // [B][slots64][H][dk][dv] gradient of the state at each chunk end
    uint16_t* ws_u16;     // [B][slots64][H][64][dv] U rows of each chunk
    uint16_t* ws_dx16;    // [B][slots64][H][64][dv] dX rows of each chunk
    int32_t* range_flag; // set when some chunk decays below the split range: the FP32 path then runs
    const int32_t* gate; // FP32 path kernels do nothing when this is set and *gate == 0
};

// Whether a backward call takes the matrix-core path.
inline bool chunk_bwd_mfma_shape(bool bf16, int dk, int dv) { return bf16 && dk == 128 && dv == 128; }
hipError_t launch_chunk_bwd_mfma(const BwdArgs& a, hipStream_t stream);

// Floats of one chunk's prepared block in ws_prep.
int64_t chunk_bwd_prep_floats(int dk);

// Token-mixer prologue: q, k, v, b, w from projection outputs.
struct MixerArgs {
    const void* xq;
    const void* xk;
    const void* xv;
    const float* conv_q;  // [H * dk][K]
    const float* conv_k;  // [H * dk][K]
    const float* conv_v;  // [H * dv][K]
    const void* b_logit;
    const void* w_logit;
    const float* conv_state_in;  // [N][H * (2 dk + dv)][K - 1] or null (zeros)
    float* conv_state_out;       // same layout, or null
    void* q;
    void* k;
    void* v;
    void* b;
    void* w;
    const int32_t* cu_seqlens;
    int32_t B, T, H, dk, dv, K, N;
    float q_scale, eps_l2;
};

// Token-mixer epilogue: RMS norm times weight times act(gate), per row of dv.
struct EpilogueArgs {
    const void* o;
    const void* gate;
    const float* weight;  // [dv]
    void* y;
    int64_t rows;
    int32_t dv;
    float eps;
    int32_t act;  // 0 sigmoid, 1 SiLU
};

// Dropout: element e of a row is kept when its 16 random bits are at least the
// threshold, and then multiplied by `keep` = 2^16 / (2^16 - threshold) (0 when
// nothing is kept).  threshold 0: no dropout, no bits are made.
struct DropoutArgs {
    uint32_t threshold;
    float keep;
    uint64_t seed, offset;
    const uint64_t* offset_device;  // added to offset; or null
};

struct DropoutCall {
    const void* x;
    void* y;
    int64_t rows, D;
    DropoutArgs drop;
};

// The step from one block to the next: x_out = x + scale * dropout(act(gate) *
// norm(u)), h = norm(x_out).  Null: u (h is the norm of x), w_post (no norm of
// u), w_pre with h (no norm of x_out).
constexpr int32_t kBlockMaxD = 16384;
constexpr int32_t kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3;
struct BlockNormArgs {
    const void* x;
    const void* u;
    const void* gate;
    const float* w_post;
    const float* w_pre;
    void* x_out;
    void* h;
    int64_t rows;
    int32_t D;
    float eps, scale;
    int32_t gate_layout, act;  // act: 0 sigmoid, 1 SiLU, 2 identity
    DropoutArgs drop;
};

// Its gradients.  Null: d_x_out (zero), w_pre with d_h, u with d_u, w_post,
// and any of d_gate, d_w_post, d_w_pre (not wanted).
struct BlockNormBwdArgs {
    const void* x;  // the stored stream, x_out of the forward call
    const void* u;
    const void* gate;
    const float* w_post;
    const float* w_pre;
    const void* d_x_out;
    const void* d_h;
    void* d_x;
    void* d_u;
    void* d_gate;
    float* d_w_post;
    float* d_w_pre;
    int64_t rows;
    int32_t D;
    float eps, scale;
    int32_t gate_layout, act;
    DropoutArgs drop;
    float* partial;  // [block_bwd_partials(rows, D)][sums * D], the wanted sums in the order post, pre, channel gate
};
int64_t block_bwd_partials(int64_t rows, int32_t D);

struct EpilogueBwdArgs {
    const void* o;
    const void* gate;
    const float* weight;
    const void* d_y;
    void* d_o;
    void* d_gate;
    float* d_weight;  // or null
    int64_t rows;
    int32_t dv;
    float eps;
    int32_t act;
    float* partial;  // [epilogue_bwd_partials(rows, dv)][dv]
};
int64_t epilogue_bwd_partials(int64_t rows, int32_t dv);

struct PrologueBwdArgs {
    const void* x[3];         // xq, xk, xv
    const float* conv[3];     // [H * d][K]
    const void* logit[2];     // b, w
    const float* conv_state_in;
    const void* d_out[3];     // dq, dk, dv
    const void* d_gate[2];    // db, dw
    const float* d_state_out;
    void* d_x[3];
    float* d_conv[3];         // or null
    void* d_logit[2];
    float* d_state_in;        // or null
    const int32_t* cu_seqlens;
    int32_t B, T, H, dk, dv, K, N;
    float q_scale, eps_l2;
    bool zero_padding;        // write zeros to the gradients of tokens that no sequence owns
    int32_t run;              // tokens per wavefront
    float* partial;           // [B * ceil(T / run)][H * (2 dk + dv) * K], or null when no filter gradient is wanted
};
// Tokens per wavefront of the prologue's backward for these sizes.
int32_t prologue_bwd_run(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, int32_t K);

// out[i][c - begin] = sum over the P rows of partial[.][c], for the columns
// [begin, end[i]) of segment i (begin: the end of segment i - 1).
struct ColumnSumArgs {
    const float* partial;
    int64_t P, width;
    float* out[3];
    int64_t end[3];
};

// Linear attention with a fixed decay for each head, as walks (see
// linear_attn.hip): x, y [B, T, H, DA], z and out [B, T, H, width].
constexpr int kLinearChunk = 64;
// Columns a workgroup walks: 64 where they divide the width, but 32 for FP32 rows x,
// y of 128, whose tiles fill the LDS.
inline int linear_slice(int width, int da, bool bf16) { return width % 64 == 0 && (bf16 || da < 128) ? 64 : 32; }
struct LinearWalk {
    const void* x;        // null in a launch for carries only
    const void* y;
    const void* z;
    void* out;
    const float* carry_in;   // [N][H] squares, or null (zeros)
    float* carry_out;        // [N][H] squares, or null
    float* segment_carry;    // squares, by place and head: the segments' own carries, or null without segments
    int32_t state_d, state_c;  // strides of a square's row d (of DA) and column c (of width)
    int32_t back;            // walk from the sequence's end
};
struct LinearLaunch {
    LinearWalk walk[3];
    int32_t walks;
    const float* alpha;      // [H]
    const int32_t* cu_seqlens;
    int32_t B, T, H, N, width;
    // Sequences are walked in segments of seg_len tokens: `segments` for each
    // batch row, or, packed, as slots and windows say (find_sequence; segments == 1:
    // one segment a sequence).  Units are H for each segment or slot, and in a launch
    // for carries only for each segment or window.
    int32_t seg_len, segments;
    int64_t units, carry_units;
    int64_t walk_blocks;     // set by the launch
    int32_t pad_blocks;      // blocks that write zeros to rows that no sequence owns
};
// Decode step: q, k [N, H, dk], v, o [N, H, dv], state [N, H, dk, dv] in place.
struct LinearStepArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* alpha;  // [H]
    float* state;
    void* o;
    int32_t N, H, dk, dv;
};

// Norms of q and k for each head, then the position rotation: x, y [tokens,
// heads, d] for q and k.  rot channels are turned (a multiple of 8), paired by
// halves or with their neighbours.
struct QkRopeArgs {
    const void* x[2];
    void* y[2];
    const float* weight[2];    // [d], or null (ones)
    const float* inv_freq;     // [rot / 2]
    const int32_t* positions;  // [tokens], or null: token % T
    int64_t tokens;
    int32_t T, heads[2], d, rot;
    bool neighbours;
    float q_scale, eps;
    int32_t parts;             // set by the launch
};
struct QkRopeBwdArgs {
    const void* x[2];
    const void* dy[2];
    void* dx[2];
    const float* weight[2];
    float* d_weight[2];        // or null
    const float* inv_freq;
    const int32_t* positions;
    int64_t tokens;
    int32_t T, heads[2], d, rot;
    bool neighbours;
    float q_scale, eps;
    int32_t parts;             // set by the launch
    float* partial;            // [qk_rope_bwd_partials(...)][2 d], or null when no d_weight is wanted
};
int64_t qk_rope_bwd_partials(int64_t tokens, int32_t heads_q, int32_t heads_k, int32_t d);

// Each returns hipSuccess or the launch error; bf16 selects the input dtype.
hipError_t launch_qk_rope(QkRopeArgs a, bool bf16, hipStream_t stream);
hipError_t launch_qk_rope_bwd(QkRopeBwdArgs a, bool bf16, hipStream_t stream);
// exact: the carries are those of FP32 arithmetic (the caller gets one of them).
hipError_t launch_linear_walk(const LinearLaunch& a, int da, bool carries_only, bool exact, bool bf16, hipStream_t stream);
hipError_t launch_linear_step(const LinearStepArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_column_sum(const ColumnSumArgs& a, hipStream_t stream);
hipError_t launch_dropout(const DropoutCall& a, bool bf16, hipStream_t stream);
hipError_t launch_block_norm_fwd(const BlockNormArgs& a, bool bf16, bool residual_bf16, hipStream_t stream);
hipError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, bool bf16, bool residual_bf16, hipStream_t stream);
hipError_t launch_mixer_epilogue_bwd(const EpilogueBwdArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_mixer_prologue_bwd(const PrologueBwdArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_mixer_prologue(const MixerArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_mixer_epilogue(const EpilogueArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_chunk_bwd(const BwdArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_recurrent(const StepArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_chunk_fwd_simple(const ChunkArgs& a, bool bf16, hipStream_t stream);

// Library-owned device scratch (scratch.hip): its capacity, and its device
// address on the current device (looked up once per device).
constexpr size_t kScratchBytes = size_t(256) << 20;
hipError_t scratch_pointer(void** out);

// Segment combine (segments.hip): S_in(1) = S_out(0), S_in(p + 1) = M_p
// S_in(p) + N_p for the layouts of ChunkArgs::seg_states_out (dv + dk
// columns) and ::seg_states_in (dv columns).
hipError_t launch_segment_combine(const float* seg_out, float* seg_in, int B, int H, int dk, int dv, int P,
                                  hipStream_t stream);

// Matrix-core chunk kernel: bf16 inputs, dk = 128, dv a multiple of 64.
bool chunk_fwd_mfma_supported(const ChunkArgs& a, bool bf16);
hipError_t launch_chunk_fwd_mfma(const ChunkArgs& a, hipStream_t stream);

}  // namespace gdn2
