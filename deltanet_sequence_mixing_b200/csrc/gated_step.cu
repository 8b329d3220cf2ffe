// One token of the gated linear recurrence for each of B x H cached states, in
// place:  S <- alpha S + k^T v,  o = q S  (the state after the write).
//
// Bound by HBM: each Dk x Dv float32 state is read once and written once.  No
// reduction stands between the read and the write (the delta rule's step has
// one), so a state may be cut into column slices that never meet: one CTA
// takes NC columns of one head.  256 x 32 states of 128 x 128: 160 us, 6.7 TB/s;
// one sequence of 16 heads: 1.7 us.  Slices of 16 columns take 162 and 1.65 us
// there (5.5 us for 4.2 at 8 x 32 states), slices of 64 158 and 2.1 us.
#include <cuda_bf16.h>

#include "kernels.h"

namespace dn {
namespace {

__device__ __forceinline__ float4 load4(const float* p, size_t i) { return *reinterpret_cast<const float4*>(p + i); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p, size_t i) {
  const uint2 u = *reinterpret_cast<const uint2*>(p + i);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ float load1(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p, size_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void store1(float* p, size_t i, float x) { p[i] = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, size_t i, float x) { p[i] = __float2bfloat16_rn(x); }

constexpr int NC = 32, kThreads = 128, kLanes = NC / 4, kRows = kThreads / kLanes;

template <typename TI, int DK>
__global__ void __launch_bounds__(kThreads) gated_step_kernel(const GatedStepProblem p) {
  constexpr int RPT = DK / kRows;  // rows of a thread
  __shared__ float qs[DK], ks[DK];
  __shared__ __align__(16) float red[kThreads / 32][NC];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid % kLanes, r = tid / kLanes;
  const int nsl = p.Dv / NC;
  const size_t bh = blockIdx.x / nsl;
  const int j0 = (int)(blockIdx.x % nsl) * NC;
  float* S = p.S + bh * DK * p.Dv + j0 + 4 * l;
  float4 s[RPT];  // every state load is issued before anything waits
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)(r + kRows * i) * p.Dv));
  const TI* q = static_cast<const TI*>(p.q) + bh * DK;
  const TI* k = static_cast<const TI*>(p.k) + bh * DK;
  if (tid < DK) {
    qs[tid] = load1(q, tid);
    ks[tid] = load1(k, tid);
  }
  const float4 v = load4(static_cast<const TI*>(p.v), bh * p.Dv + j0 + 4 * l);
  const float a = p.alpha ? p.alpha[bh] : 1.f;
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const float ki = ks[r + kRows * i], qi = qs[r + kRows * i];
    s[i].x = fmaf(ki, v.x, a * s[i].x);
    s[i].y = fmaf(ki, v.y, a * s[i].y);
    s[i].z = fmaf(ki, v.z, a * s[i].z);
    s[i].w = fmaf(ki, v.w, a * s[i].w);
    __stcs(reinterpret_cast<float4*>(S + (size_t)(r + kRows * i) * p.Dv), s[i]);
    o.x = fmaf(qi, s[i].x, o.x);
    o.y = fmaf(qi, s[i].y, o.y);
    o.z = fmaf(qi, s[i].z, o.z);
    o.w = fmaf(qi, s[i].w, o.w);
  }
#pragma unroll
  for (int m = kLanes; m < 32; m <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
  }
  if (lane < kLanes) *reinterpret_cast<float4*>(&red[warp][4 * l]) = o;
  __syncthreads();
  if (tid < NC) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) x += red[w][tid];
    store1(static_cast<TI*>(p.o), bh * p.Dv + j0 + tid, x);
  }
}

template <typename TI>
cudaError_t launch_t(const GatedStepProblem& p, cudaStream_t st) {
  const unsigned grid = (unsigned)((size_t)p.B * p.H * (p.Dv / NC));
  if (p.Dk == 128)
    gated_step_kernel<TI, 128><<<grid, kThreads, 0, st>>>(p);
  else
    gated_step_kernel<TI, 64><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_step(const GatedStepProblem& p, cudaStream_t st) {
  return p.bf16 ? launch_t<__nv_bfloat16>(p, st) : launch_t<float>(p, st);
}

}  // namespace dn
