// What the two directions of the block step (block.hip, block_bwd.hip) share: how
// rows are laid over lanes and wavefronts, their sums, and the gate.
#pragma once

#include "row_device.hpp"

namespace gdn2 {
namespace {

// Conditions that are the same for a whole launch (norms, gate, dropout) are
// asked once per group of eight channels, with a loop over the eight inside:
// asked per element they cost a scalar branch each and keep the compiler from
// interleaving the eight chains.

// A gate's activation and its derivative over eight channels: 0 sigmoid s, 1
// SiLU g s, 2 the value itself.  Both derivatives are f (1 - s), plus s for SiLU.
__device__ __forceinline__ void act_values(int act, const float* g, float* f, float* df)
{
    if (act == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = g[j];
            df[j] = 1.f;
        }
    } else if (act == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = fast_sigmoid(g[j]);
            f[j] = g[j] * s;
            df[j] = fmaf(f[j], 1.f - s, s);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = fast_sigmoid(g[j]);
            df[j] = f[j] * (1.f - f[j]);
        }
    }
}

// How a workgroup covers rows: LPR lanes (LPR < 64) or WPR wavefronts a row, NI
// groups of eight channels a lane.
template <int LPR, int WPR, int NI>
struct Cover {
    static constexpr int kThreads = WPR == 1 || WPR == 2 ? 256 : WPR * 64;
    static constexpr int kWaves = kThreads / 64;
    static constexpr int kRowLanes = LPR * WPR;
    static constexpr int kRows = kThreads / kRowLanes;  // rows at a time per workgroup
};

// The row of this lane among those that the workgroup takes at a time: where a
// row spans whole wavefronts, the same in every lane, which makes its address a
// scalar.
template <int LPR, int WPR, int NI>
__device__ __forceinline__ int row_slot()
{
    const int slot = threadIdx.x / Cover<LPR, WPR, NI>::kRowLanes;
    return LPR == 64 ? __builtin_amdgcn_readfirstlane(slot) : slot;
}

// Sums of M values over a row's lanes.  Over several wavefronts they meet in
// LDS, in two buffers in turn: a wavefront that writes a buffer again has
// passed the barrier that every reader of its last contents reached after
// reading, so one barrier a sum is enough.
template <int LPR, int WPR, int M>
__device__ __forceinline__ void row_sums(float (&v)[M], float (*lds)[16][4], int& turn)
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

// Eight channels of a weight (zero behind the last), or ones without it.
template <int MODE>
__device__ __forceinline__ void load_weight(const float* w, const Group<MODE>& group, int D, float* v)
{
    if (!w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.f;
        return;
    }
    Eight<float> e;
    e.clear();
    group.load(e, w, D, true, true);
    group.settle(e, D, true);
    e.get(v);
}

// The cover of a row of D channels: calls F(Cover parameters, MODE).  Narrow rows
// take a group of lanes, so that few lanes idle; then one wavefront, then as
// many as leave eight channels a lane.  From 2048 channels on a lane takes
// sixteen: half the wavefronts meet at a row's barriers, and the loads of two
// groups are in flight (2048 whole channels, bf16, 32768 rows, backward: 220 us
// with four wavefronts of eight a lane, 208 with two of sixteen; forward 178 and
// 176).  Ragged rows of up to 2048 keep four wavefronts: their short and absent
// groups then idle in fewer lanes (5003 rows of 1371, FP32, forward: 25 us, 39
// with two).
#define GDN2_COVER(D, F)                                                           \
    do {                                                                           \
        if (row_mode(D) == kTiny) F(4, 1, 1, kTiny);                               \
        else if (row_mode(D) == kWhole) GDN2_WIDTH(D, F, F(64, 2, 2, kWhole), kWhole); \
        else GDN2_WIDTH(D, F, F(64, 4, 1, kRagged), kRagged);                      \
    } while (0)
#define GDN2_WIDTH(D, F, UP_TO_2048, MODE)         \
    do {                                           \
        if ((D) <= 32) F(4, 1, 1, MODE);           \
        else if ((D) <= 64) F(8, 1, 1, MODE);      \
        else if ((D) <= 128) F(16, 1, 1, MODE);    \
        else if ((D) <= 256) F(32, 1, 1, MODE);    \
        else if ((D) <= 512) F(64, 1, 1, MODE);    \
        else if ((D) <= 1024) F(64, 2, 1, MODE);   \
        else if ((D) <= 2048) UP_TO_2048;          \
        else if ((D) <= 4096) F(64, 4, 2, MODE);   \
        else if ((D) <= 8192) F(64, 8, 2, MODE);   \
        else F(64, 16, 2, MODE);                   \
    } while (0)

constexpr int kSimds = 256 * 4;  // compute units of an MI355X, four SIMDs each

// Workgroups of a launch over `rows` rows that walk the same number of rounds of
// `at_once` rows each, at most `most` of them.
inline int64_t even_blocks(int64_t rows, int at_once, int64_t most)
{
    const int64_t need = (rows + at_once - 1) / at_once;
    if (need <= most) return need;
    const int64_t rounds = (need + most - 1) / most;
    return (need + rounds - 1) / rounds;
}

}  // namespace
}  // namespace gdn2
