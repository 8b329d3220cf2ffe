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
// neighbours), so the turn needs no exchange and the norm three shuffles.  A
// lane's columns are the same in every row: the weights (and in the gradient
// their sums) stay in registers, one half of the grid taking the queries and the
// other the keys.
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

// The turn by +angle (way = 1) or -angle (way = -1) of a lane's 16 values: the
// cosines and sines of its 8 pairs stand in a row.
template <bool INTER>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float* cs, const float* sn, float way) {
  float c[8], s[8];
  load_piece(cs, c);
  load_piece(sn, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x = INTER ? (i < 4 ? a[2 * (i & 3)] : b[2 * (i & 3)]) : a[i];
    float& y = INTER ? (i < 4 ? a[2 * (i & 3) + 1] : b[2 * (i & 3) + 1]) : b[i];
    const float x0 = x, ws = way * s[i];
    x = x0 * c[i] - y * ws;
    y = y * c[i] + x0 * ws;
  }
}

__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + __expf(-x)); }

// cos and sin of the angles of tokens [n0, n0 + nt) (flat over B x T): `half`
// cosines, then as many sines, for each token.
__device__ __forceinline__ void fill_turns(const QkProblem& p, int n0, int nt, float* turns) {
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tok = i / half, f = i - tok * half, b = (n0 + tok) / p.T, t = (n0 + tok) - b * p.T;
    const double pos = p.positions ? (double)p.positions[b * p.pos_stride_b + t] : (double)t;
    double x = pos * (double)p.inv_freq[f] * 0.15915494309189533576888;  // 1 / (2 pi)
    x -= rint(x);
    float s, c;
    sincospif(2.f * (float)x, &s, &c);
    turns[2 * half * tok + f] = c;
    turns[2 * half * tok + half + f] = s;
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

// One tensor of the two, as a CTA sees it.
struct Side {
  const void* x;
  const void* g;       // gradient: the derivative by the output
  const float* w;
  void* out;
  int H;
  long long xb, xt, xh;  // strides of x
  long long ob, ot, oh;  // gradient: of out
};
__device__ __forceinline__ Side side_of(const QkProblem& p, bool key) {
  if (key) return Side{p.k, p.dk_in, p.k_weight, p.k_out, p.Hk, p.ks_b, p.ks_t, p.ks_h, p.dks_b, p.dks_t, p.dks_h};
  return Side{p.q, p.dq_in, p.q_weight, p.q_out, p.Hq, p.qs_b, p.qs_t, p.qs_h, p.dqs_b, p.dqs_t, p.dqs_h};
}

// The rows of a tile of nt tokens with H heads, ROWS of them at a time: this
// thread's token and head, stepped without a division.
template <int ROWS>
struct Walk {
  int tok, h, dtok, dh, H;
  __device__ Walk(int first, int heads) : H(heads) {
    tok = first / heads;
    h = first - tok * heads;
    dtok = ROWS / heads;
    dh = ROWS - dtok * heads;
  }
  __device__ void step() {
    tok += dtok;
    h += dh;
    if (h >= H) {
      h -= H;
      ++tok;
    }
  }
};

template <typename TI, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const QkProblem p, int tokens) {
  constexpr int L = D / 16, ROWS = kThreads / L;
  extern __shared__ float turns[];
  const Side s = side_of(p, blockIdx.y);
  const int N = p.B * p.T, n0 = (int)blockIdx.x * tokens, nt = min(tokens, N - n0), half = p.rot / 2;
  const int l = threadIdx.x % L;
  if (s.H == 0) return;
  int c0, c1;
  pieces_of(l, p.rot, INTER, c0, c1);
  const bool turned = l < p.rot / 16;
  float wa[8], wb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wa[e] = s.w ? s.w[c0 + e] : 1.f;
    wb[e] = s.w ? s.w[c1 + e] : 1.f;
  }
  if (half) fill_turns(p, n0, nt, turns);
  __syncthreads();
  Walk<ROWS> at(threadIdx.x / L, s.H);
  for (int i0 = 0; i0 < nt * s.H; i0 += ROWS, at.step()) {
    const bool live = at.tok < nt;
    const int n = n0 + at.tok, b = n / p.T, t = n - b * p.T;
    float x[8] = {}, y[8] = {};
    if (live) {
      const TI* in = static_cast<const TI*>(s.x) + b * s.xb + t * s.xt + at.h * s.xh;
      load_piece(in + c0, x);
      load_piece(in + c1, y);
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (p.silu) {
        x[e] *= sigmoid_f(x[e]);
        y[e] *= sigmoid_f(y[e]);
      }
      ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
    }
    ss = row_sum<D>(ss);
    if (!live) continue;
    bool floored;
    const float scale = row_scale<D>(p, ss, floored);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] *= scale * wa[e];
      y[e] *= scale * wb[e];
    }
    if (turned) turn<INTER>(x, y, turns + 2 * half * at.tok + 8 * l, turns + 2 * half * at.tok + half + 8 * l, 1.f);
    TI* o = static_cast<TI*>(s.out) + (((long long)b * s.H + at.h) * p.T + t) * D;
    store_piece(o + c0, x);
    store_piece(o + c1, y);
  }
}

// Gradient.  CTAs walk the token tiles with a stride, so that the weights'
// gradients stay in registers until the end; every CTA then leaves its row of
// partial sums and a second kernel adds them in a fixed order.
template <typename TI, typename TG, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_bwd_kernel(const QkProblem p, int tokens) {
  constexpr int L = D / 16, ROWS = kThreads / L;
  extern __shared__ float turns[];
  __shared__ float part[kThreads / 32][D];
  const Side s = side_of(p, blockIdx.y);
  const int N = p.B * p.T, half = p.rot / 2;
  const int l = threadIdx.x % L, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int c0, c1;
  pieces_of(l, p.rot, INTER, c0, c1);
  const bool turned = l < p.rot / 16;
  float wa[8], wb[8], dwa[8] = {}, dwb[8] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wa[e] = s.w ? s.w[c0 + e] : 1.f;
    wb[e] = s.w ? s.w[c1 + e] : 1.f;
  }
  for (long long first = (long long)blockIdx.x * tokens; s.H > 0 && first < N; first += (long long)gridDim.x * tokens) {
    const int n0 = (int)first, nt = min(tokens, N - n0);
    __syncthreads();  // the turns of the tile before have been read
    if (half) fill_turns(p, n0, nt, turns);
    __syncthreads();
    Walk<ROWS> at(threadIdx.x / L, s.H);
    for (int i0 = 0; i0 < nt * s.H; i0 += ROWS, at.step()) {
      const bool live = at.tok < nt;
      const int n = n0 + at.tok, b = n / p.T, t = n - b * p.T;
      float x[8] = {}, y[8] = {}, dx[8] = {}, dy[8] = {};
      if (live) {
        const TI* in = static_cast<const TI*>(s.x) + b * s.xb + t * s.xt + at.h * s.xh;
        const TG* g = static_cast<const TG*>(s.g) + (((long long)b * s.H + at.h) * p.T + t) * D;
        load_piece(in + c0, x);
        load_piece(in + c1, y);
        load_piece(g + c0, dx);
        load_piece(g + c1, dy);
        if (turned)
          turn<INTER>(dx, dy, turns + 2 * half * at.tok + 8 * l, turns + 2 * half * at.tok + half + 8 * l, -1.f);
      }
      // z over x in place; silu' is formed again from x at the end
      float ss = 0.f, zx[8], zy[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        zx[e] = p.silu ? x[e] * sigmoid_f(x[e]) : x[e];
        zy[e] = p.silu ? y[e] * sigmoid_f(y[e]) : y[e];
        ss = fmaf(zx[e], zx[e], fmaf(zy[e], zy[e], ss));
      }
      ss = row_sum<D>(ss);
      bool floored;
      const float scale = row_scale<D>(p, ss, floored);
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        zx[e] *= scale;  // the normed row
        zy[e] *= scale;
        if (live) {
          dwa[e] = fmaf(dx[e], zx[e], dwa[e]);
          dwb[e] = fmaf(dy[e], zy[e], dwb[e]);
        }
        dx[e] *= wa[e];
        dy[e] *= wb[e];
        dot = fmaf(dx[e], zx[e], fmaf(dy[e], zy[e], dot));
      }
      dot = row_sum<D>(dot) * (p.l2 ? 1.f : 1.f / D);
      if (floored) dot = 0.f;
      if (!live) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dx[e] = scale * (dx[e] - zx[e] * dot);
        dy[e] = scale * (dy[e] - zy[e] * dot);
        if (p.silu) {
          const float g0 = sigmoid_f(x[e]), g1 = sigmoid_f(y[e]);
          dx[e] *= g0 * fmaf(x[e], 1.f - g0, 1.f);
          dy[e] *= g1 * fmaf(y[e], 1.f - g1, 1.f);
        }
      }
      TI* o = static_cast<TI*>(s.out) + b * s.ob + t * s.ot + at.h * s.oh;
      store_piece(o + c0, dx);
      store_piece(o + c1, dy);
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
      dwa[e] += __shfl_xor_sync(0xffffffffu, dwa[e], o);
      dwb[e] += __shfl_xor_sync(0xffffffffu, dwb[e], o);
    }
    if (lane < L) {
      part[warp][c0 + e] = dwa[e];
      part[warp][c1 + e] = dwb[e];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float x = 0.f;
#pragma unroll
    for (int ww = 0; ww < kThreads / 32; ++ww) x += part[ww][d];
    p.partial[((size_t)blockIdx.x * 2 + blockIdx.y) * D + d] = x;
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
  const int heads = p.Hq > p.Hk ? p.Hq : p.Hk, t = 128 / heads;
  return t < 1 ? 1 : t > kMaxTokens ? kMaxTokens : t;
}

template <typename TI, int D>
cudaError_t fwd(const QkProblem& p, cudaStream_t st) {
  const int tokens = tile_tokens(p);
  const dim3 grid((unsigned)(((long long)p.B * p.T + tokens - 1) / tokens), 2);
  const size_t smem = (size_t)tokens * p.rot * sizeof(float);
  if (p.interleaved)
    qk_fwd_kernel<TI, D, true><<<grid, kThreads, smem, st>>>(p, tokens);
  else
    qk_fwd_kernel<TI, D, false><<<grid, kThreads, smem, st>>>(p, tokens);
  return cudaGetLastError();
}

template <typename TI, typename TG, int D>
cudaError_t bwd(const QkProblem& p, cudaStream_t st) {
  const int tokens = tile_tokens(p);
  const unsigned ctas = (unsigned)qk_bwd_ctas(p.B, p.T, p.Hq, p.Hk);
  const size_t smem = (size_t)tokens * p.rot * sizeof(float);
  if (p.interleaved)
    qk_bwd_kernel<TI, TG, D, true><<<dim3(ctas, 2), kThreads, smem, st>>>(p, tokens);
  else
    qk_bwd_kernel<TI, TG, D, false><<<dim3(ctas, 2), kThreads, smem, st>>>(p, tokens);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  qk_weight_kernel<<<2 * D / 8, 256, 0, st>>>(p.partial, (int)ctas, D, p.dq_weight, p.dk_weight);
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
  constexpr long long kCtas = 148 * 2;  // times two tensors: what is resident on 148 SMs
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
