// Gated linear recurrence on float32 inputs, on CUDA cores: forward and
// gradient.  Per (b, h), with a Dk x Dv state,
//     S_t = alpha_t S_{t-1} + k_t^T v_t,   o_t = q_t S_t.
//
// Chunks of C = 32 tokens entered with S.  With D_ij the product of alpha over
// (j, i], G_i the product over [0, i], c_j the product over (j, C) and gamma
// the product over the chunk (tokens past T count as alpha = 1, q = k = v = 0):
//   forward   O = diag(G) Q S + (tril(Q K^T) * D) V,   S <- gamma S + K^T diag(c) V
//   reverse   R <- gamma R + Q^T diag(G) dO            (R: the loss's derivative by S)
//   gradient  A = tril(Q K^T) * D, B = tril(dO V^T) * D
//             dQ = B K + diag(G) dO S^T
//             dK = B^T Q + diag(c) V R^T,   dV = A^T dO + diag(c) K R
// The decays are running products of alpha, never exponentials of sums of
// logarithms: a hard wipe (alpha = 0) is exact, and D_ij keeps its relative
// accuracy however strongly the chunk as a whole decays.
//
// The gradient of log alpha_t is the sum of all paths from a write before t to
// a read at or after it:
//   sum_{i >= t > j} M_ij + sum_{i >= t} r_i + sum_{j < t} e_j + gamma <S, R>
//   M = (Q K^T) * (dO V^T) * D,  r_i = q_i . (G_i dO_i S^T),  e_j = k_j . (c_j v_j R^T)
// where the first term is the suffix sum of (row sum - column sum) of M below
// its diagonal.  Sums stay inside one chunk, so no error travels along T.
//
// Kernels: every chunk's own increment of the state, side by side (`local`); the
// states between them, one multiply-add per chunk and element (`between`);
// outputs or gradients of every chunk, side by side (`out`, `grad`).  The
// gradient takes the first two forward with (k, v) and from the end with
// (q, dO).  With heads enough to fill the GPU the forward instead walks the
// chunks of each head (`out` without stored states): the same products without
// the states' way through memory.
//
// Bound by the products' operands on their way out of shared memory, short
// sequences by the launches.  (Tensor cores take float32 only as tf32, a product
// as three of split operands; these kernels do not.)  Read along the depth four
// at a time: the gradient of B2 H16 T1024 D128 434 us, of B2 H3 T777 Dk 128 Dv 64
// 53, the forward of the first 210, of B1 H2 T256 D64 14.5; one at a time 791,
// 64, 309 and 18.6.
#include "kernels.h"

namespace dn {
namespace {

constexpr int C = kGatedSimtChunk, kThreads = 256, NV = 32, CP = C + 4;
static_assert(C == 32, "one lane per token of a chunk");

// acc[x][y] += sum_{k < nk} A(r0 + 16 x, k) B(k, c0 + 16 y) for thread (r0, c0) of
// the CTA's 16 x 16 grid.  AK: A(i, k) = A[i * ap + k], else A[k * ap + i]; BK:
// B(k, j) = B[j * bp + k], else B[k * bp + j].  What runs along k is read four at
// a time: the operands' way out of shared memory is what the products wait for.
// Pitches are 4 over a power of two, so that eight rows' pieces meet in no bank.
template <int RX, int RY, bool AK, bool BK>
__device__ __forceinline__ void product(int nk, const float* A, int ap, const float* B, int bp,
                                        float (&acc)[RX][RY]) {
  const int r0 = threadIdx.x >> 4, c0 = threadIdx.x & 15;
#pragma unroll 4
  for (int k = 0; k < nk; k += 4) {
    float a[RX][4], b[RY][4];
#pragma unroll
    for (int x = 0; x < RX; ++x) {
      const int i = r0 + 16 * x;
      if (AK) {
        const float4 v = *reinterpret_cast<const float4*>(A + i * ap + k);
        a[x][0] = v.x; a[x][1] = v.y; a[x][2] = v.z; a[x][3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[x][e] = A[(k + e) * ap + i];
      }
    }
#pragma unroll
    for (int y = 0; y < RY; ++y) {
      const int j = c0 + 16 * y;
      if (BK) {
        const float4 v = *reinterpret_cast<const float4*>(B + j * bp + k);
        b[y][0] = v.x; b[y][1] = v.y; b[y][2] = v.z; b[y][3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) b[y][e] = B[(k + e) * bp + j];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int x = 0; x < RX; ++x)
#pragma unroll
        for (int y = 0; y < RY; ++y) acc[x][y] = fmaf(a[x][e], b[y][e], acc[x][y]);
  }
}

// A tile of R rows of W floats, `stride` apart in global memory, `pitch` in shared
// memory; rows from n on are zero.
template <int R, int W>
__device__ __forceinline__ void load_tile(float* dst, int pitch, const float* src, size_t stride, int n) {
#pragma unroll 8
  for (int i = threadIdx.x; i < R * W / 4; i += kThreads) {
    const int r = i / (W / 4), d = i % (W / 4) * 4;
    const float4 x = r < n ? *reinterpret_cast<const float4*>(src + r * stride + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(dst + r * pitch + d) = x;
  }
}

// One warp: the chunk's decays from alpha (n tokens; 1 behind them).
// into[i] = G_i, out[j] = c_j, D (if not null) the C x C matrix of D_ij, zero
// above the diagonal.  Returns gamma.
__device__ __forceinline__ float chunk_decays(const float* alpha, int n, float* into, float* out, float* D) {
  const int lane = threadIdx.x & 31;
  const float a = alpha && lane < n ? alpha[lane] : 1.f;
  float pre = a;                                             // product over [0, lane]
  float suf = __shfl_down_sync(0xffffffffu, a, 1);           // product over (lane, C)
  if (lane == 31) suf = 1.f;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, pre, o), y = __shfl_down_sync(0xffffffffu, suf, o);
    if (lane >= o) pre *= x;
    if (lane + o < 32) suf *= y;
  }
  into[lane] = pre;
  out[lane] = suf;
  if (D) {
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float ai = __shfl_sync(0xffffffffu, a, i);
      d = i == lane ? 1.f : d * ai;
      D[i * CP + lane] = i < lane ? 0.f : d;
    }
  }
  return __shfl_sync(0xffffffffu, pre, 31);
}

// ----------------------------------------------------------------- states --
// One CTA per (b, h, chunk) and direction (blockIdx.y: 0 forward, 1 from the
// end): the chunk's increment X^T diag(f) Z of the state, and gamma.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) gated_simt_local_kernel(const GatedProblem p, float* S, float* R,
                                                                    float* gammas) {
  constexpr int KP = DK + 4, VP = DV + 4, RK = DK / 16, RV = DV / 16;
  __shared__ float into[C], out[C];
  extern __shared__ __align__(16) float sm[];
  float* Xs = sm;           // C x KP
  float* Zs = Xs + C * KP;  // C x VP
  const int tid = threadIdx.x, r0 = tid >> 4, c0 = tid & 15;
  const int T = p.T, nch = (T + C - 1) / C;
  const size_t bh = blockIdx.x / nch;
  const int c = (int)(blockIdx.x % nch), t0 = c * C, n = min(C, T - t0);
  const bool rev = blockIdx.y;
  const float* x = static_cast<const float*>(rev ? p.q : p.k) + (bh * T + t0) * DK;
  const float* z = static_cast<const float*>(rev ? p.dO : p.v) + (bh * T + t0) * DV;
  load_tile<C, DK>(Xs, KP, x, DK, n);
  load_tile<C, DV>(Zs, VP, z, DV, n);
  if (tid < 32) {
    const float g = chunk_decays(p.alpha ? p.alpha + bh * T + t0 : nullptr, n, into, out, nullptr);
    if (tid == 0 && !rev) gammas[blockIdx.x] = g;
  }
  __syncthreads();
  for (int i = tid; i < C * DK; i += kThreads) Xs[(i / DK) * KP + i % DK] *= rev ? into[i / DK] : out[i / DK];
  __syncthreads();
  float a[RK][RV] = {};
  product<RK, RV, false, false>(C, Xs, KP, Zs, VP, a);
  float* dst = (rev ? R : S) + (size_t)blockIdx.x * DK * DV;
#pragma unroll
  for (int xx = 0; xx < RK; ++xx)
#pragma unroll
    for (int y = 0; y < RV; ++y) dst[(r0 + 16 * xx) * DV + c0 + 16 * y] = a[xx][y];
}

// Four elements of the state per thread, over the chunks of their (b, h): each
// chunk's increment becomes the state that the chunk is entered with, in the
// scan's direction.
__global__ void __launch_bounds__(kThreads) gated_simt_between_kernel(const GatedProblem p, float* S, float* R,
                                                                      const float* gammas) {
  const int nch = (p.T + C - 1) / C, elems = p.Dk * p.Dv, quads = elems / 4;
  const size_t at = (size_t)blockIdx.x * kThreads + threadIdx.x, bh = at / quads;  // quads is a multiple of kThreads
  const bool rev = blockIdx.y;
  const float* S_in = rev ? p.dS_T : p.S0;
  float* S_end = rev ? p.dS0 : p.S_out;
  float4* st = reinterpret_cast<float4*>((rev ? R : S) + bh * nch * elems) + at % quads;
  const float* g = gammas + bh * nch;
  float4 s = S_in ? reinterpret_cast<const float4*>(S_in + bh * elems)[at % quads] : make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int AHEAD = 8;
  for (int c0 = 0; c0 < nch; c0 += AHEAD) {
    float4 d[AHEAD];
    float gam[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int cc = c0 + i, c = rev ? nch - 1 - cc : cc;
      if (cc < nch) {
        d[i] = st[(size_t)c * quads];
        gam[i] = g[c];
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int cc = c0 + i, c = rev ? nch - 1 - cc : cc;
      if (cc < nch) {
        st[(size_t)c * quads] = s;
        s = make_float4(fmaf(gam[i], s.x, d[i].x), fmaf(gam[i], s.y, d[i].y), fmaf(gam[i], s.z, d[i].z),
                        fmaf(gam[i], s.w, d[i].w));
      }
    }
  }
  if (S_end) reinterpret_cast<float4*>(S_end + bh * elems)[at % quads] = s;
}

// ----------------------------------------------------------------- outputs --
// One CTA per (b, h, 32 columns of Dv) over all chunks, or with PAR per chunk
// too, from the stored states.
template <int DK, bool PAR>
__global__ void __launch_bounds__(kThreads) gated_simt_out_kernel(const GatedProblem p, const float* states) {
  constexpr int KP = DK + 4, VP = NV + 4, RK = DK / 16;
  __shared__ float into[C], out[C], gam;
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;               // C x KP
  float* Vs = Ks + C * KP;      // C x VP
  float* Ss = Vs + C * VP;      // DK x VP
  float* Qs = Ss + DK * VP;     // C x KP
  float* Ps = Qs + C * KP;      // C x CP
  float* Ds = Ps + C * CP;      // C x CP
  const int tid = threadIdx.x, r0 = tid >> 4, c0 = tid & 15;
  const int T = p.T, Dv = p.Dv, nch = (T + C - 1) / C, nsl = Dv / NV, per = PAR ? nch : 1;
  const size_t bh = blockIdx.x / nsl / per;
  const int j0 = (int)(blockIdx.x % nsl) * NV, only = (int)(blockIdx.x / nsl % per);
  const size_t sblk = (size_t)DK * Dv;
  const float* k = static_cast<const float*>(p.k) + bh * T * DK;
  const float* q = static_cast<const float*>(p.q) + bh * T * DK;
  const float* v = static_cast<const float*>(p.v) + bh * T * Dv + j0;
  float* o = static_cast<float*>(p.o) + bh * T * Dv + j0;
  const float* alpha = p.alpha ? p.alpha + bh * T : nullptr;
  const float* S_in = PAR ? states + (bh * nch + only) * sblk : p.S0 ? p.S0 + bh * sblk : nullptr;

  float s[RK][2];  // this thread's rows r0 + 16 x, columns c0 + 16 y of the state
#pragma unroll
  for (int xx = 0; xx < RK; ++xx)
#pragma unroll
    for (int y = 0; y < 2; ++y) s[xx][y] = S_in ? S_in[(size_t)(r0 + 16 * xx) * Dv + j0 + c0 + 16 * y] : 0.f;

  for (int c = only; c < (PAR ? only + 1 : nch); ++c) {
    const int t0 = c * C, n = min(C, T - t0);
    __syncthreads();  // the products of the chunk before have read the tiles
    load_tile<C, DK>(Ks, KP, k + (size_t)t0 * DK, DK, n);
    load_tile<C, DK>(Qs, KP, q + (size_t)t0 * DK, DK, n);
    load_tile<C, NV>(Vs, VP, v + (size_t)t0 * Dv, Dv, n);
    if (tid < 32) {
      const float g = chunk_decays(alpha ? alpha + t0 : nullptr, n, into, out, Ds);
      if (tid == 0) gam = g;
    }
#pragma unroll
    for (int xx = 0; xx < RK; ++xx)
#pragma unroll
      for (int y = 0; y < 2; ++y) Ss[(r0 + 16 * xx) * VP + c0 + 16 * y] = s[xx][y];
    __syncthreads();
    float a[2][2] = {};
    product<2, 2, true, true>(DK, Qs, KP, Ks, KP, a);
#pragma unroll
    for (int xx = 0; xx < 2; ++xx)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = r0 + 16 * xx, j = c0 + 16 * y;
        Ps[i * CP + j] = j <= i ? a[xx][y] * Ds[i * CP + j] : 0.f;
      }
    float qs[2][2] = {};
    product<2, 2, true, false>(DK, Qs, KP, Ss, VP, qs);
    __syncthreads();
#pragma unroll
    for (int xx = 0; xx < 2; ++xx)
#pragma unroll
      for (int y = 0; y < 2; ++y) qs[xx][y] *= into[r0 + 16 * xx];
    product<2, 2, true, false>(C, Ps, CP, Vs, VP, qs);
#pragma unroll
    for (int xx = 0; xx < 2; ++xx)
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (r0 + 16 * xx < n) o[(size_t)(t0 + r0 + 16 * xx) * Dv + c0 + 16 * y] = qs[xx][y];
    if (PAR) break;
    __syncthreads();  // P V has read Vs
    for (int i = tid; i < C * NV; i += kThreads) Vs[(i / NV) * VP + i % NV] *= out[i / NV];
    __syncthreads();
#pragma unroll
    for (int xx = 0; xx < RK; ++xx)
#pragma unroll
      for (int y = 0; y < 2; ++y) s[xx][y] *= gam;
    product<RK, 2, false, false>(C, Ks, KP, Vs, VP, s);
  }
  if (!PAR && p.S_out) {
#pragma unroll
    for (int xx = 0; xx < RK; ++xx)
#pragma unroll
      for (int y = 0; y < 2; ++y)
        p.S_out[bh * sblk + (size_t)(r0 + 16 * xx) * Dv + j0 + c0 + 16 * y] = s[xx][y];
  }
}

// --------------------------------------------------------------- gradient --
// One CTA per (b, h, chunk): S the state entering the chunk, R the derivative
// by the state leaving it.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) gated_simt_grad_kernel(const GatedProblem p, const float* Sst,
                                                                   const float* Rst) {
  constexpr int KP = DK + 4, VP = DV + 4, RK = DK / 16, RV = DV / 16;
  __shared__ float into[C], out[C], gam, row[C], col[C], rr[C], ee[C], through[kThreads / 32];
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + C * KP;
  float* Vs = Ks + C * KP;
  float* Os = Vs + C * VP;
  float* As = Os + C * VP;  // C x CP
  float* Bs = As + C * CP;
  float* Ds = Bs + C * CP;  // D, then M
  float* Hs = Ds + C * CP;  // DK x VP: S, then R
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r0 = tid >> 4, c0 = tid & 15;
  const int T = p.T, nch = (T + C - 1) / C;
  const size_t bh = blockIdx.x / nch;
  const int c = (int)(blockIdx.x % nch), t0 = c * C, n = min(C, T - t0);
  const size_t kbase = (bh * T + t0) * DK, vbase = (bh * T + t0) * DV, sbase = (size_t)blockIdx.x * DK * DV;
  const float* q = static_cast<const float*>(p.q) + kbase;
  const float* k = static_cast<const float*>(p.k) + kbase;
  const float* v = static_cast<const float*>(p.v) + vbase;
  const float* dO = static_cast<const float*>(p.dO) + vbase;
  load_tile<C, DK>(Qs, KP, q, DK, n);
  load_tile<C, DK>(Ks, KP, k, DK, n);
  load_tile<C, DV>(Vs, VP, v, DV, n);
  load_tile<C, DV>(Os, VP, dO, DV, n);
  load_tile<DK, DV>(Hs, VP, Sst + sbase, DV, DK);
  if (tid < 32) {
    const float g = chunk_decays(p.alpha ? p.alpha + bh * T + t0 : nullptr, n, into, out, Ds);
    if (tid == 0) gam = g;
  }
  __syncthreads();
  {
    float a[2][2] = {}, b[2][2] = {};
    product<2, 2, true, true>(DK, Qs, KP, Ks, KP, a);
    product<2, 2, true, true>(DV, Os, VP, Vs, VP, b);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = r0 + 16 * x, j = c0 + 16 * y, at = i * CP + j;
        const float d = Ds[at];
        As[at] = j <= i ? a[x][y] * d : 0.f;
        Bs[at] = j <= i ? b[x][y] * d : 0.f;
        Ds[at] = j < i ? a[x][y] * b[x][y] * d : 0.f;
      }
  }
  __syncthreads();
  if (tid < C) {  // row and column sums of M
    float x = 0.f, y = 0.f;
#pragma unroll 8
    for (int j = 0; j < C; ++j) {
      x += Ds[tid * CP + j];
      y += Ds[j * CP + tid];
    }
    row[tid] = x;
    col[tid] = y;
  }
  // rows r0 + 16 x of a C x (16 RY) result, inter-chunk part `in` scaled by its row's decay
  auto rowdot16 = [&](float x) {  // over the 16 threads of a row
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  {
    float in[2][RK] = {};
    product<2, RK, true, true>(DV, Os, VP, Hs, VP, in);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = r0 + 16 * x;
      float dot = 0.f;
#pragma unroll
      for (int y = 0; y < RK; ++y) {
        in[x][y] *= into[i];
        dot = fmaf(in[x][y], Qs[i * KP + c0 + 16 * y], dot);
      }
      dot = rowdot16(dot);
      if (c0 == 0) rr[i] = dot;
    }
    product<2, RK, true, false>(C, Bs, CP, Ks, KP, in);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < RK; ++y)
        if (r0 + 16 * x < n)
          (static_cast<float*>(p.dq) + kbase)[(size_t)(r0 + 16 * x) * DK + c0 + 16 * y] = in[x][y];
  }
  __syncthreads();
  {
    float sr = 0.f;  // <S, R>, while R takes the place of S
#pragma unroll 8
    for (int i = tid; i < DK * DV / 4; i += kThreads) {
      const float4 x = reinterpret_cast<const float4*>(Rst + sbase)[i];
      float4* h = reinterpret_cast<float4*>(Hs + i / (DV / 4) * VP + i % (DV / 4) * 4);
      const float4 y = *h;
      sr = fmaf(y.x, x.x, fmaf(y.y, x.y, fmaf(y.z, x.z, fmaf(y.w, x.w, sr))));
      *h = x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sr += __shfl_xor_sync(0xffffffffu, sr, o);
    if (lane == 0) through[warp] = sr;
  }
  __syncthreads();
  {
    float in[2][RK] = {};
    product<2, RK, true, true>(DV, Vs, VP, Hs, VP, in);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = r0 + 16 * x;
      float dot = 0.f;
#pragma unroll
      for (int y = 0; y < RK; ++y) {
        in[x][y] *= out[j];
        dot = fmaf(in[x][y], Ks[j * KP + c0 + 16 * y], dot);
      }
      dot = rowdot16(dot);
      if (c0 == 0) ee[j] = dot;
    }
    product<2, RK, false, false>(C, Bs, CP, Qs, KP, in);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < RK; ++y)
        if (r0 + 16 * x < n)
          (static_cast<float*>(p.dk) + kbase)[(size_t)(r0 + 16 * x) * DK + c0 + 16 * y] = in[x][y];
  }
  {
    float in[2][RV] = {};
    product<2, RV, true, false>(DK, Ks, KP, Hs, VP, in);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < RV; ++y) in[x][y] *= out[r0 + 16 * x];
    product<2, RV, false, false>(C, As, CP, Os, VP, in);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < RV; ++y)
        if (r0 + 16 * x < n)
          (static_cast<float*>(p.dv) + vbase)[(size_t)(r0 + 16 * x) * DV + c0 + 16 * y] = in[x][y];
  }
  if (!p.dlog_alpha) return;
  __syncthreads();
  if (warp == 0) {
    float sr = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) sr += through[w];
    float suf = row[lane] - col[lane] + rr[lane], pre = ee[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_down_sync(0xffffffffu, suf, o), y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane + o < 32) suf += x;
      if (lane >= o) pre += y;
    }
    pre = __shfl_up_sync(0xffffffffu, pre, 1);  // writes before this token
    if (lane == 0) pre = 0.f;
    // no path crosses a wipe: its derivative is 0, not the sums' rounding
    if (lane < n)
      p.dlog_alpha[bh * T + t0 + lane] = p.alpha[bh * T + t0 + lane] == 0.f ? 0.f : suf + pre + gam * sr;
  }
}

template <int DK, int DV>
constexpr size_t grad_smem() {
  return sizeof(float) * (2 * C * (DK + 4) + 2 * C * (DV + 4) + 3 * C * CP + DK * (DV + 4));
}

int chunks(const GatedProblem& p) { return (p.T + C - 1) / C; }

template <typename K>
cudaError_t prepare(K kern, size_t smem) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <int DK, bool PAR>
cudaError_t outputs(const GatedProblem& p, const float* states, cudaStream_t stream) {
  auto kern = gated_simt_out_kernel<DK, PAR>;
  constexpr size_t smem = sizeof(float) * (2 * C * (DK + 4) + (C + DK) * (NV + 4) + 2 * C * CP);
  cudaError_t e = prepare(kern, smem);
  if (e != cudaSuccess) return e;
  const size_t grid = (size_t)p.B * p.H * (p.Dv / NV) * (PAR ? chunks(p) : 1);
  kern<<<(unsigned)grid, kThreads, smem, stream>>>(p, states);
  return cudaGetLastError();
}

// The state between all chunks: S, and with both directions R.
template <int DK, int DV>
cudaError_t states(const GatedProblem& p, float* S, float* R, float* gammas, cudaStream_t stream) {
  auto kern = gated_simt_local_kernel<DK, DV>;
  constexpr size_t smem = sizeof(float) * C * (DK + DV + 8);
  cudaError_t e = prepare(kern, smem);
  if (e != cudaSuccess) return e;
  const unsigned dirs = R ? 2 : 1;
  const size_t BH = (size_t)p.B * p.H;
  kern<<<dim3((unsigned)(BH * chunks(p)), dirs), kThreads, smem, stream>>>(p, S, R, gammas);
  gated_simt_between_kernel<<<dim3((unsigned)(BH * (DK * DV / 4 / kThreads)), dirs), kThreads, 0, stream>>>(p, S, R,
                                                                                                          gammas);
  return cudaGetLastError();
}

cudaError_t states_of(const GatedProblem& p, float* S, float* R, float* gammas, cudaStream_t stream) {
  if (p.Dk == 128)
    return p.Dv == 128 ? states<128, 128>(p, S, R, gammas, stream) : states<128, 64>(p, S, R, gammas, stream);
  return p.Dv == 128 ? states<64, 128>(p, S, R, gammas, stream) : states<64, 64>(p, S, R, gammas, stream);
}

template <int DK, int DV>
cudaError_t grad(const GatedProblem& p, const float* S, const float* R, cudaStream_t stream) {
  auto kern = gated_simt_grad_kernel<DK, DV>;
  constexpr size_t smem = grad_smem<DK, DV>();
  cudaError_t e = prepare(kern, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((size_t)p.B * p.H * chunks(p)), kThreads, smem, stream>>>(p, S, R);
  return cudaGetLastError();
}

size_t gamma_floats(size_t BH, int T) { return (BH * ((T + C - 1) / C) + 63) / 64 * 64; }

}  // namespace

// The forward walks the chunks of each head where one chunk is all there is, or
// where 32-column slices of heads fill the GPU four times over and the stored
// states would only be memory.  Measured (T512; walk | chunks side by side, us):
// D128 32 heads 135 | 111, 48 218 | 161, 64 229 | 211, 72 229 | 240, 80 (a third
// wave of CTAs) 310 | 273, 128 444 | 428; D64 296 heads, 592 slices, 244 | 252;
// H4 T100 25 | 14.5.
bool gated_simt_walks(int BH, int T, int Dv, int sms) {
  return T <= C || (long long)BH * (Dv / NV) >= 4LL * sms;
}

size_t gated_simt_bytes(int BH, int T, int Dk, int Dv, int directions) {
  const size_t nch = ((size_t)T + C - 1) / C;
  return sizeof(float) * (gamma_floats(BH, T) + directions * BH * nch * Dk * Dv);
}

cudaError_t launch_gated_simt_fwd(const GatedProblem& p, cudaStream_t stream) {
  if (!p.scratch)
    return p.Dk == 128 ? outputs<128, false>(p, nullptr, stream) : outputs<64, false>(p, nullptr, stream);
  float* gammas = static_cast<float*>(p.scratch);
  float* S = gammas + gamma_floats((size_t)p.B * p.H, p.T);
  const cudaError_t e = states_of(p, S, nullptr, gammas, stream);
  if (e != cudaSuccess) return e;
  return p.Dk == 128 ? outputs<128, true>(p, S, stream) : outputs<64, true>(p, S, stream);
}

cudaError_t launch_gated_simt_bwd(const GatedProblem& p, cudaStream_t stream) {
  const size_t BH = (size_t)p.B * p.H;
  float* gammas = static_cast<float*>(p.scratch);
  float* S = gammas + gamma_floats(BH, p.T);
  float* R = S + BH * chunks(p) * p.Dk * p.Dv;
  GatedProblem b = p;
  b.S_out = nullptr;
  const cudaError_t e = states_of(b, S, R, gammas, stream);
  if (e != cudaSuccess) return e;
  if (p.Dk == 128) return p.Dv == 128 ? grad<128, 128>(p, S, R, stream) : grad<128, 64>(p, S, R, stream);
  return p.Dv == 128 ? grad<64, 128>(p, S, R, stream) : grad<64, 64>(p, S, R, stream);
}

}  // namespace dn
