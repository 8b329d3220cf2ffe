// Per-head norm of query and key rows with the rotation by position, forward
// and gradient, reading strided (B, T, H, D) and writing contiguous
// (B, H, T, D) (the gradient the other way round).  Per row x of D values:
//     z = x or silu(x)
//     y = z r w,   r = 1 / sqrt(mean(z^2) + eps)     (rms)
//                  r = 1 / max(||z||_2, eps)         (l2)
//     out = y turned: the pairs (y_a, y_b) of the first `rot` columns by the
//           angle position * inv_freq[i], a = i, b = i + rot/2 (halves) or
//           a = 2i, b = 2i + 1 (interleaved); the other columns pass.
// Gradient, d the incoming row turned back:
//     dw = sum over rows of d z r
//     dz = r (w d - z r (sum(w d z r) / m)),  m = D (rms), 1 (l2; the second
//          term is absent where ||z|| < eps),   dx = dz silu'(x)
//
// Bound by HBM: one read and one write of every row (two reads in the
// gradient).  A row belongs to D / 16 lanes, and each lane holds two 16-byte
// pieces that form whole pairs (pieces l and l + rot/16 of the rotated half, or
// neighbours), so the turn needs no exchange and the norm three shuffles.
// Angles: position * inv_freq in float64, in turns, its whole part dropped,
// then sine and cosine in float32: exact to float32 at any position.  A CTA
// computes them once for a token and uses them for all of its heads.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace dn {
namespace {

constexpr int kThreads = 256, kMaxTokens = 16;

template <int N>
__device__ __forceinline__ void load_piece(const float* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + i);
    x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
  }
}
__device__ __forceinline__ void load_piece(const __nv_bfloat16* p, float (&x)[8]) {
  unpack_bf16x8(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void store_piece(float* p, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const float (&x)[8]) { st_bf16x8(p, x); }

// Column of a lane's two pieces: pairs of pieces of the rotated halves first,
// then neighbours.
__device__ __forceinline__ void pieces_of(int l, int rot, int interleaved, int& c0, int& c1) {
  const int rp = rot / 16;  // pieces of one rotated half
  if (!interleaved && l < rp) {
    c0 = 8 * l;
    c1 = 8 * (l + rp);
  } else {
    c0 = 16 * l;  // the rotated halves fill columns [0, 16 rp)
    c1 = 16 * l + 8;
  }
}

// The turn by +angle (way = 1) or -angle (way = -1) of a lane's 16 values.
template <bool INTER>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float2* cs, int l, float way) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = cs[8 * l + i], w = cs[8 * l + 4 + i];
      const float x0 = a[2 * i], x1 = a[2 * i + 1], y0 = b[2 * i], y1 = b[2 * i + 1];
      a[2 * i] = x0 * u.x - way * x1 * u.y;
      a[2 * i + 1] = x1 * u.x + way * x0 * u.y;
      b[2 * i] = y0 * w.x - way * y1 * w.y;
      b[2 * i + 1] = y1 * w.x + way * y0 * w.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 u = cs[8 * l + i];
      const float x0 = a[i], x1 = b[i];
      a[i] = x0 * u.x - way * x1 * u.y;
      b[i] = x1 * u.x + way * x0 * u.y;
    }
  }
}

__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + __expf(-x)); }

// cos and sin of the angles of tokens [n0, n0 + nt) (flat over B x T).
__device__ __forceinline__ void fill_turns(const QkProblem& p, long long n0, int nt, float2* cs) {
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const long long n = n0 + i / half;
    const long long b = n / p.T, t = n % p.T;
    const double pos = p.positions ? (double)p.positions[b * p.pos_stride_b + t] : (double)t;
    double turns = pos * (double)p.inv_freq[i % half] * 0.15915494309189533576888;  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    cs[i] = make_float2(c, s);
  }
}

template <int D>
__device__ __forceinline__ float row_sum(float x) {  // over the D / 16 lanes of a row
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
__device__ __forceinline__ float row_scale(const QkProblem& p, float ss, bool& floored) {
  if (p.l2) {
    const float norm = sqrtf(ss);
    floored = norm < p.eps;  // false for a NaN, which stays one
    return 1.f / (floored ? p.eps : norm);
  }
  floored = false;
  return rsqrtf(ss * (1.f / D) + p.eps);
}

struct Row {  // one row's place
  bool live, is_k;
  int h;
  long long b, t;
};

template <int D>
__device__ __forceinline__ Row row_of(const QkProblem& p, long long n0, int nt, int i) {
  const int heads = p.Hq + p.Hk;
  Row r;
  r.live = i < nt * heads;
  const int tok = r.live ? i / heads : 0;
  const int hh = r.live ? i - tok * heads : 0;
  r.is_k = hh >= p.Hq;
  r.h = r.is_k ? hh - p.Hq : hh;
  r.b = (n0 + tok) / p.T;
  r.t = (n0 + tok) - r.b * p.T;
  return r;
}

template <typename TI, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const QkProblem p, int tokens) {
  constexpr int L = D / 16, ROWS = kThreads / L;
  extern __shared__ float2 cs[];
  const long long N = (long long)p.B * p.T, n0 = (long long)blockIdx.x * tokens;
  const int nt = (int)(N - n0 < tokens ? N - n0 : tokens), heads = p.Hq + p.Hk, half = p.rot / 2;
  const int l = threadIdx.x % L;
  int c0, c1;
  pieces_of(l, p.rot, INTER, c0, c1);
  const bool turned = l < p.rot / 16;
  if (half) fill_turns(p, n0, nt, cs);
  __syncthreads();
  for (int i0 = 0; i0 < nt * heads; i0 += ROWS) {
    const int i = i0 + threadIdx.x / L;
    const Row r = row_of<D>(p, n0, nt, i);
    const int tok = r.live ? i / heads : 0;
    float a[8] = {}, b[8] = {};
    if (r.live) {
      const TI* x = r.is_k ? static_cast<const TI*>(p.k) + r.b * p.ks_b + r.t * p.ks_t + r.h * p.ks_h
                           : static_cast<const TI*>(p.q) + r.b * p.qs_b + r.t * p.qs_t + r.h * p.qs_h;
      load_piece(x + c0, a);
      load_piece(x + c1, b);
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (p.silu) {
        a[e] *= sigmoid_f(a[e]);
        b[e] *= sigmoid_f(b[e]);
      }
      ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
    }
    ss = row_sum<D>(ss);
    if (!r.live) continue;
    bool floored;
    const float scale = row_scale<D>(p, ss, floored);
    const float* w = r.is_k ? p.k_weight : p.q_weight;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] *= scale * (w ? w[c0 + e] : 1.f);
      b[e] *= scale * (w ? w[c1 + e] : 1.f);
    }
    if (turned) turn<INTER>(a, b, cs + tok * half, l, 1.f);
    TI* o = static_cast<TI*>(r.is_k ? p.k_out : p.q_out) +
            ((r.b * (r.is_k ? p.Hk : p.Hq) + r.h) * (long long)p.T + r.t) * D;
    store_piece(o + c0, a);
    store_piece(o + c1, b);
  }
}

// Gradient.  CTAs walk the token tiles with a stride, so that the weights'
// gradients stay in registers until the end; every CTA then leaves its two
// rows of partial sums and a second kernel adds them in a fixed order.
template <typename TI, typename TG, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_bwd_kernel(const QkProblem p, int tokens) {
  constexpr int L = D / 16, ROWS = kThreads / L;
  extern __shared__ float2 cs[];
  __shared__ float part[kThreads / 32][D];
  const long long N = (long long)p.B * p.T;
  const int heads = p.Hq + p.Hk, half = p.rot / 2;
  const int l = threadIdx.x % L, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int c0, c1;
  pieces_of(l, p.rot, INTER, c0, c1);
  const bool turned = l < p.rot / 16;
  float dw[2][16] = {};
  for (long long n0 = (long long)blockIdx.x * tokens; n0 < N; n0 += (long long)gridDim.x * tokens) {
    const int nt = (int)(N - n0 < tokens ? N - n0 : tokens);
    __syncthreads();  // the turns of the tile before have been read
    if (half) fill_turns(p, n0, nt, cs);
    __syncthreads();
    for (int i0 = 0; i0 < nt * heads; i0 += ROWS) {
      const int i = i0 + threadIdx.x / L;
      const Row r = row_of<D>(p, n0, nt, i);
      const int tok = r.live ? i / heads : 0;
      const long long in = r.is_k ? r.b * p.ks_b + r.t * p.ks_t + r.h * p.ks_h
                                  : r.b * p.qs_b + r.t * p.qs_t + r.h * p.qs_h;
      float a[8] = {}, b[8] = {}, da[8] = {}, db[8] = {};
      if (r.live) {
        const TI* x = static_cast<const TI*>(r.is_k ? p.k : p.q) + in;
        const TG* g = static_cast<const TG*>(r.is_k ? p.dk_in : p.dq_in) +
                      ((r.b * (r.is_k ? p.Hk : p.Hq) + r.h) * (long long)p.T + r.t) * D;
        load_piece(x + c0, a);
        load_piece(x + c1, b);
        load_piece(g + c0, da);
        load_piece(g + c1, db);
        if (turned) turn<INTER>(da, db, cs + tok * half, l, -1.f);
      }
      float sa[8], sb[8], ss = 0.f;  // silu' where it applies
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sa[e] = sb[e] = 1.f;
        if (p.silu) {
          const float s0 = sigmoid_f(a[e]), s1 = sigmoid_f(b[e]);
          sa[e] = s0 * fmaf(a[e], 1.f - s0, 1.f);
          sb[e] = s1 * fmaf(b[e], 1.f - s1, 1.f);
          a[e] *= s0;
          b[e] *= s1;
        }
        ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
      }
      ss = row_sum<D>(ss);
      bool floored;
      const float scale = row_scale<D>(p, ss, floored);
      const float* w = r.is_k ? p.k_weight : p.q_weight;
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] *= scale;  // the normed row
        b[e] *= scale;
        if (w && r.live) {
          const float ga = da[e] * a[e], gb = db[e] * b[e];
          dw[0][e] += r.is_k ? 0.f : ga;
          dw[0][8 + e] += r.is_k ? 0.f : gb;
          dw[1][e] += r.is_k ? ga : 0.f;
          dw[1][8 + e] += r.is_k ? gb : 0.f;
          da[e] *= w[c0 + e];
          db[e] *= w[c1 + e];
        }
        dot = fmaf(da[e], a[e], fmaf(db[e], b[e], dot));
      }
      dot = row_sum<D>(dot) * (p.l2 ? 1.f : 1.f / D);
      if (floored) dot = 0.f;
      if (!r.live) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        da[e] = scale * (da[e] - a[e] * dot) * sa[e];
        db[e] = scale * (db[e] - b[e] * dot) * sb[e];
      }
      const long long to = r.is_k ? r.b * p.dks_b + r.t * p.dks_t + r.h * p.dks_h
                                  : r.b * p.dqs_b + r.t * p.dqs_t + r.h * p.dqs_h;
      TI* o = static_cast<TI*>(r.is_k ? p.k_out : p.q_out) + to;
      store_piece(o + c0, da);
      store_piece(o + c1, db);
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float x = dw[which][e];
#pragma unroll
      for (int o = L; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane < L) part[warp][(e < 8 ? c0 : c1) + (e & 7)] = x;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
      float x = 0.f;
#pragma unroll
      for (int ww = 0; ww < kThreads / 32; ++ww) x += part[ww][d];
      p.partial[((size_t)blockIdx.x * 2 + which) * D + d] = x;
    }
  }
}

// Sums of the CTAs' partial rows: 8 columns per CTA, 32 threads per column.
__global__ void __launch_bounds__(256) qk_weight_kernel(const float* partial, int n, int D, float* dqw, float* dkw) {
  __shared__ float red[32][8];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int col = blockIdx.x * 8 + c, which = col / D, d = col % D;
  float x = 0.f;
  for (int i = g; i < n; i += 32) x += partial[((size_t)i * 2 + which) * D + d];
  red[g][c] = x;
  __syncthreads();
  if (threadIdx.x < 8) {
    x = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) x += red[i][c];
    float* out = which ? dkw : dqw;
    if (out) out[d] = x;
  }
}

// Tokens of a tile: about 128 rows, at most kMaxTokens tables of turns.
int tile_tokens(const QkProblem& p) {
  const int heads = p.Hq + p.Hk, t = 128 / heads;
  return t < 1 ? 1 : t > kMaxTokens ? kMaxTokens : t;
}

template <typename TI, int D>
cudaError_t fwd(const QkProblem& p, cudaStream_t st) {
  const int tokens = tile_tokens(p);
  const unsigned grid = (unsigned)(((long long)p.B * p.T + tokens - 1) / tokens);
  const size_t smem = (size_t)tokens * (p.rot / 2) * sizeof(float2);
  if (p.interleaved)
    qk_fwd_kernel<TI, D, true><<<grid, kThreads, smem, st>>>(p, tokens);
  else
    qk_fwd_kernel<TI, D, false><<<grid, kThreads, smem, st>>>(p, tokens);
  return cudaGetLastError();
}

template <typename TI, typename TG, int D>
cudaError_t bwd(const QkProblem& p, cudaStream_t st) {
  const int tokens = tile_tokens(p);
  const unsigned grid = (unsigned)qk_bwd_ctas(p.B, p.T, p.Hq, p.Hk);
  const size_t smem = (size_t)tokens * (p.rot / 2) * sizeof(float2);
  if (p.interleaved)
    qk_bwd_kernel<TI, TG, D, true><<<grid, kThreads, smem, st>>>(p, tokens);
  else
    qk_bwd_kernel<TI, TG, D, false><<<grid, kThreads, smem, st>>>(p, tokens);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  qk_weight_kernel<<<2 * D / 8, 256, 0, st>>>(p.partial, (int)grid, D, p.dq_weight, p.dk_weight);
  return cudaGetLastError();
}

template <typename TI, typename TG>
cudaError_t bwd_d(const QkProblem& p, cudaStream_t st) {
  return p.D == 128 ? bwd<TI, TG, 128>(p, st) : bwd<TI, TG, 64>(p, st);
}

}  // namespace

int qk_bwd_ctas(int B, int T, int Hq, int Hk) {
  QkProblem p{};
  p.Hq = Hq;
  p.Hk = Hk;
  const int tokens = tile_tokens(p);
  const long long tiles = ((long long)B * T + tokens - 1) / tokens;
  constexpr long long kCtas = 148 * 3;  // what the register use leaves resident on 148 SMs
  return (int)(tiles < kCtas ? tiles : kCtas);
}

cudaError_t launch_qk_fwd(const QkProblem& p, cudaStream_t st) {
  if (p.bf16) return p.D == 128 ? fwd<__nv_bfloat16, 128>(p, st) : fwd<__nv_bfloat16, 64>(p, st);
  return p.D == 128 ? fwd<float, 128>(p, st) : fwd<float, 64>(p, st);
}

cudaError_t launch_qk_bwd(const QkProblem& p, cudaStream_t st) {
  if (!p.bf16) return bwd_d<float, float>(p, st);
  return p.grad_bf16 ? bwd_d<__nv_bfloat16, __nv_bfloat16>(p, st) : bwd_d<__nv_bfloat16, float>(p, st);
}

}  // namespace dn
