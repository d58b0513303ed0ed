// Decode step of linear attention with a fixed decay for each head: per
// (sequence, head), S <- a S + k v^T in place and o = S^T q from the new state.
//
// Column j of the state evolves with v_j alone, so one wavefront owns 32
// columns of a head, as in recurrent_step.hip: lane l holds columns
// 4 (l & 7) .. + 3 of the dk / 8 rows g dk / 8 .., g = l >> 3.  A lane needs q and k
// of its own rows only, which it loads for itself (eight lanes the same
// addresses); the sums over the rows are register sums and three lane exchanges.
// No LDS and no barrier.
#include "gdn2_device.hpp"
#include "launch.hpp"

namespace gdn2 {
namespace {

constexpr int kCols = 32;          // value columns per wavefront
constexpr int kAuxLoad = 2;        // buffer cache policy of the state loads: nt
constexpr int kAuxStore = 2 | 16;  // of the state stores: nt, sc1

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, int(bytes), 0x00020000);
}

// N consecutive elements at a boundary of N elements.
template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + i);
        v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
    }
}
template <int N>
__device__ __forceinline__ void load_row(const bf16raw* p, float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p + i);
        v[i] = __uint_as_float(x.x << 16), v[i + 1] = __uint_as_float(x.x & 0xffff0000u);
        v[i + 2] = __uint_as_float(x.y << 16), v[i + 3] = __uint_as_float(x.y & 0xffff0000u);
    }
}
__device__ __forceinline__ void store_o4(float* o, const float (&x)[4]) { *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void store_o4(bf16raw* o, const float (&x)[4])
{
    *reinterpret_cast<uint2*>(o) = make_uint2(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]));
}

// Sum over the eight row groups (lanes 8 apart), in every lane.
__device__ __forceinline__ float rowgroup_sum(float x)
{
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x128, 0xF, 0xF, true));  // lane ^ 8 (rotate by 8 of 16)
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <typename T, int DK, int DV>
__global__ __launch_bounds__(64) void linear_step_kernel(LinearStepArgs a)
{
    constexpr int NQ = DV / kCols, NP = DK / 8;  // column slices of a head, rows of a lane
    const int slice = (blockIdx.x % (8 * NQ)) / 8;
    const int64_t head = int64_t(blockIdx.x / (8 * NQ)) * 8 + (blockIdx.x & 7);
    if (head >= int64_t(a.N) * a.H) return;
    const int lane = threadIdx.x, g = lane >> 3, c0 = slice * kCols + 4 * (lane & 7);

    const rsrc_t rs = make_rsrc(a.state + head * DK * DV, DK * DV * 4);
    float k[NP], q[NP], v[4];
    load_row(static_cast<const T*>(a.k) + head * DK + g * NP, k);
    load_row(static_cast<const T*>(a.v) + head * DV + c0, v);
    load_row(static_cast<const T*>(a.q) + head * DK + g * NP, q);
    const float decay = fminf(fmaxf(a.alpha[head % a.H], 0x1p-15f), 1.0f);
    u32x4 st[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) st[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, ((g * NP + i) * DV + c0) * 4, 0, kAuxLoad);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        u32x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float s = decay * __uint_as_float(st[i][j]) + k[i] * v[j];
            y[j] = __float_as_uint(s);
            o[j] += s * q[i];
        }
        __builtin_amdgcn_raw_buffer_store_b128(y, rs, ((g * NP + i) * DV + c0) * 4, 0, kAuxStore);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = rowgroup_sum(o[j]);
    if (g == 0) store_o4(static_cast<T*>(a.o) + head * DV + c0, o);
}

template <typename T, int DK, int DV>
hipError_t launch_dkdv(const LinearStepArgs& a, hipStream_t stream)
{
    const int64_t heads = int64_t(a.N) * a.H, blocks = (heads + 7) / 8 * 8 * (DV / kCols);
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((linear_step_kernel<T, DK, DV>), dim3(unsigned(blocks)), dim3(64), 0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_typed(const LinearStepArgs& a, hipStream_t stream)
{
#define GDN2_STEP_CASE(DK_, DV_) \
    if (a.dk == DK_ && a.dv == DV_) return launch_dkdv<T, DK_, DV_>(a, stream);
    GDN2_STEP_CASE(32, 32) GDN2_STEP_CASE(32, 64) GDN2_STEP_CASE(32, 128)
    GDN2_STEP_CASE(64, 32) GDN2_STEP_CASE(64, 64) GDN2_STEP_CASE(64, 128)
    GDN2_STEP_CASE(128, 32) GDN2_STEP_CASE(128, 64) GDN2_STEP_CASE(128, 128)
#undef GDN2_STEP_CASE
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_linear_step(const LinearStepArgs& a, bool bf16, hipStream_t stream)
{
    return bf16 ? launch_typed<bf16raw>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace gdn2
