// Decode step of linear attention with a fixed decay for each head: per
// (sequence, head), S <- a S + k v^T in place and o = S^T q from the new state.
//
// Column j of the state evolves with v_j alone, so one wavefront owns 32
// columns of a head: lane l holds columns 4 (l & 7) .. + 3 of the rows 8 i + g,
// g = l >> 3, so that one access takes eight neighbouring rows.  A lane needs q and
// k of its own rows only, which it loads for itself (eight lanes the same address);
// the sums over the rows are register sums and three lane exchanges.  No LDS and no
// barrier.
//
// What bounds it is HBM: 256 sequences x 16 heads of 128 x 128 (541 MB) take 101 us,
// 5.35 TB/s, where a large device copy reaches 5.06.  Rows g dk / 8 .. in each lane
// took 104 us, all stores behind the last load 106, stores without the system-scope
// hint 106, plain accesses 109.
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

__device__ __forceinline__ void load4(const float* p, float (&v)[4])
{
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
__device__ __forceinline__ void load4(const bf16raw* p, float (&v)[4])
{
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
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
#pragma unroll
    for (int i = 0; i < NP; ++i) k[i] = load_as_f32(static_cast<const T*>(a.k), head * DK + 8 * i + g);
    load4(static_cast<const T*>(a.v) + head * DV + c0, v);
#pragma unroll
    for (int i = 0; i < NP; ++i) q[i] = load_as_f32(static_cast<const T*>(a.q), head * DK + 8 * i + g);
    const float decay = fminf(fmaxf(a.alpha[head % a.H], 0x1p-15f), 1.0f);
    u32x4 st[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) st[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, ((8 * i + g) * DV + c0) * 4, 0, kAuxLoad);
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
        __builtin_amdgcn_raw_buffer_store_b128(y, rs, ((8 * i + g) * DV + c0) * 4, 0, kAuxStore);
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
