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
// Angles: position * inv_freq in turns, its whole part dropped, in float64 (far
// positions in pairs of doubles), then sine and cosine in float32: as good as
// float32 at any position.
// A CTA computes them once for a token and uses them for all of its heads.
// B4 T4096 H16 D128 in bf16, full rotation: forward 54 us (5 TB/s), gradient 90 us
// (4.5 TB/s).  What is left is the latency of the loads that 32 warps of an SM
// have in flight (32 KB) and half of the issue slots: loads a row ahead took the
// registers of as many warps and gained nothing.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace dn {
namespace {

constexpr int kThreads = 256, kMaxTokens = 16;

// Eight values of a row as four pairs, in two-wide arithmetic: a row's work is
// mostly instructions beside its loads (one value at a time the forward of B4
// T4096 H16 D128 took 64.5 us, the gradient 139 us).
struct V8 {
  float2 v[4];
};
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{ .reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};"
      " fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ void load_piece(const float* p, V8& x) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x.v[0] = make_float2(a.x, a.y);
  x.v[1] = make_float2(a.z, a.w);
  x.v[2] = make_float2(b.x, b.y);
  x.v[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void load_piece(const __nv_bfloat16* p, V8& x) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void store_piece(float* p, const V8& x) {
  *reinterpret_cast<float4*>(p) = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
}
__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const V8& x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2_bf16(x.v[0].x, x.v[0].y), pack2_bf16(x.v[1].x, x.v[1].y),
                                            pack2_bf16(x.v[2].x, x.v[2].y), pack2_bf16(x.v[3].x, x.v[3].y));
}

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

// The turn by +angle, or back by it, of a lane's 16 values: the cosines and
// sines of its 8 pairs stand in a row.
template <bool INTER, bool BACK>
__device__ __forceinline__ void turn(V8& a, V8& b, const float* cs, const float* sn) {
  V8 c, s;
  load_piece(cs, c);
  load_piece(sn, s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {  // pairs 2 i and 2 i + 1: in a (i < 2) or b
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2& x = (i < 2 ? a : b).v[(2 * i + h) & 3];
        const float cc = h ? c.v[i].y : c.v[i].x, sh = h ? s.v[i].y : s.v[i].x, ss = BACK ? -sh : sh;
        x = make_float2(x.x * cc - x.y * ss, x.y * cc + x.x * ss);
      }
    } else {
      const float2 n = make_float2(-s.v[i].x, -s.v[i].y), x = a.v[i], y = b.v[i];
      a.v[i] = fma2(y, BACK ? s.v[i] : n, mul2(x, c.v[i]));
      b.v[i] = fma2(x, BACK ? n : s.v[i], mul2(y, c.v[i]));
    }
  }
}

// The hardware's exponential, for float32 rows too: off by 2 + 1.2 |x| units in
// the last place (4e-7 at 4, 2e-6 at -30, where silu is 3e-12).
__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + __expf(-x)); }
__device__ __forceinline__ float2 silu2(float2 x) { return make_float2(x.x * sigmoid_f(x.x), x.y * sigmoid_f(x.y)); }

// Where the rows of a tile's tokens begin (head 0) in the input and the output.
struct Tile {
  long long in[kMaxTokens], out[kMaxTokens];
};
__device__ __forceinline__ void fill_tile(const QkProblem& p, int n0, int nt, long long xb, long long xt, long long ob,
                                          long long ot, Tile& tile) {
  if (threadIdx.x < nt) {
    const int b = (n0 + (int)threadIdx.x) / p.T, t = n0 + (int)threadIdx.x - b * p.T;
    tile.in[threadIdx.x] = b * xb + t * xt;
    tile.out[threadIdx.x] = b * ob + t * ot;
  }
}

// pos * f / (2 pi) without its whole turns.  Up to 2^24 one double leaves 2^-31
// turns behind for f up to 1; farther out (2^-21 at 2^34) the products that may
// have whole turns are carried as two: a + b = p f exactly (f has 24 bits, so b
// has few), and 1 / (2 pi) = kTurn + kTurnLow to 2^-109; whole turns leave a
// kTurn inside a fused multiply-add.  That is off by less than 2^-40 turns at any
// position; at near ones too it would cost the gradient of B4 T4096 H16 D128
// 96.4 us for 95.0, the forward 57.8 for 57.4.
__device__ __forceinline__ float part_of_turn(long long pos, double f) {
  constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLow = -0x1.6b01ec5417056p-57;
  double x;
  if (pos >= -(1ll << 24) && pos <= (1ll << 24)) {
    x = (double)pos * f * kTurn;
  } else {
    // past 2^53 the low bits, which a double may not hold, go by themselves
    const long long low = pos >= -(1ll << 53) && pos <= (1ll << 53) ? 0 : pos & 2047;
    const double p = (double)(pos - low), a = p * f, b = fma(p, f, -a);
    x = fma(a, kTurn, -rint(a * kTurn)) + fma(a, kTurnLow, b * kTurn);
    if (low) x = fma((double)low * f, kTurn, x);
  }
  return (float)(x - rint(x));
}

// cos and sin of the angles of tokens [n0, n0 + nt) (flat over B x T): `half`
// cosines, then as many sines, for each token.
__device__ __forceinline__ void fill_turns(const QkProblem& p, int n0, int nt, float* turns) {
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tok = i / half, f = i - tok * half, b = (n0 + tok) / p.T, t = (n0 + tok) - b * p.T;
    const long long pos = p.positions ? p.positions[b * p.pos_stride_b + t] : t;
    float s, c;
    sincospif(2.f * part_of_turn(pos, (double)p.inv_freq[f]), &s, &c);
    turns[2 * half * tok + f] = c;
    turns[2 * half * tok + half + f] = s;
  }
}

template <int D>
__device__ __forceinline__ float row_sum(float2 x) {  // over the D / 16 lanes of a row
  float y = x.x + x.y;
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  return y;
}

template <int D, bool L2>
__device__ __forceinline__ float row_scale(float eps, float ss, bool& floored) {
  floored = false;
  if (L2) {
    const float norm = sqrtf(ss);
    floored = norm < eps;  // false for a NaN, which stays one
    return 1.f / (floored ? eps : norm);
  }
  return rsqrtf(ss * (1.f / D) + eps);
}

// One tensor of the two, as a CTA sees it.
struct Side {
  const void* x;
  const void* g;  // gradient: the derivative by the output
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

template <typename TI, int D, bool INTER, bool L2, bool SILU>
__global__ void __launch_bounds__(kThreads, 4) qk_fwd_kernel(const QkProblem p, int tokens) {
  constexpr int L = D / 16, ROWS = kThreads / L;
  extern __shared__ __align__(16) float turns[];
  __shared__ Tile tile[2];
  const int N = p.B * p.T, n0 = (int)blockIdx.x * tokens, nt = min(tokens, N - n0), half = p.rot / 2;
  const int l = threadIdx.x % L;
  int c0, c1;
  pieces_of(l, p.rot, INTER, c0, c1);
  const bool turned = l < p.rot / 16;
  const long long oh = (long long)p.T * D;
  fill_turns(p, n0, nt, turns);
  // both tensors, or by blockIdx.y one of them
  const int first = gridDim.y == 1 ? 0 : blockIdx.y, last = gridDim.y == 1 ? 1 : blockIdx.y;
  for (int key = first; key <= last; ++key) {
    const Side s = side_of(p, key);
    fill_tile(p, n0, nt, s.xb, s.xt, oh * s.H, D, tile[key]);
  }
  __syncthreads();
#pragma unroll 1
  for (int key = first; key <= last; ++key) {
    const Side s = side_of(p, key);
    if (s.H == 0) continue;
    V8 wa, wb;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      wa.v[e] = s.w ? make_float2(s.w[c0 + 2 * e], s.w[c0 + 2 * e + 1]) : both(1.f);
      wb.v[e] = s.w ? make_float2(s.w[c1 + 2 * e], s.w[c1 + 2 * e + 1]) : both(1.f);
    }
    Walk<ROWS> at(threadIdx.x / L, s.H);
    for (int i0 = 0; i0 < nt * s.H; i0 += ROWS, at.step()) {
      const bool live = at.tok < nt;
      V8 x = {}, y = {};
      if (live) {
        const TI* in = static_cast<const TI*>(s.x) + tile[key].in[at.tok] + at.h * s.xh;
        load_piece(in + c0, x);
        load_piece(in + c1, y);
      }
      float2 ss = both(0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (SILU) {
          x.v[e] = silu2(x.v[e]);
          y.v[e] = silu2(y.v[e]);
        }
        ss = fma2(x.v[e], x.v[e], fma2(y.v[e], y.v[e], ss));
      }
      const float sum = row_sum<D>(ss);
      if (!live) continue;
      bool floored;
      const float2 scale = both(row_scale<D, L2>(p.eps, sum, floored));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x.v[e] = mul2(x.v[e], mul2(scale, wa.v[e]));
        y.v[e] = mul2(y.v[e], mul2(scale, wb.v[e]));
      }
      const float* cs = turns + 2 * half * at.tok + 8 * l;
      if (turned) turn<INTER, false>(x, y, cs, cs + half);
      TI* o = static_cast<TI*>(s.out) + tile[key].out[at.tok] + at.h * oh;
      store_piece(o + c0, x);
      store_piece(o + c1, y);
    }
  }
}

// Gradient.  CTAs walk the token tiles with a stride, so that the weights'
// gradients stay in registers until the end; every CTA then leaves its row of
// partial sums and a second kernel adds them in a fixed order.
template <typename TI, typename TG, int D, bool INTER, bool L2, bool SILU>
__global__ void __launch_bounds__(kThreads, SILU ? 2 : 3) qk_bwd_kernel(const QkProblem p, int tokens) {
  constexpr int L = D / 16, ROWS = kThreads / L;
  extern __shared__ __align__(16) float turns[];
  __shared__ Tile tile, place;  // of x and of the derivative by the output; of the derivative by x
  __shared__ float part[kThreads / 32][D];
  const Side s = side_of(p, blockIdx.y);
  const int N = p.B * p.T, half = p.rot / 2;
  const int l = threadIdx.x % L, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int c0, c1;
  pieces_of(l, p.rot, INTER, c0, c1);
  const bool turned = l < p.rot / 16;
  V8 wa, wb, dwa = {}, dwb = {};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    wa.v[e] = s.w ? make_float2(s.w[c0 + 2 * e], s.w[c0 + 2 * e + 1]) : both(1.f);
    wb.v[e] = s.w ? make_float2(s.w[c1 + 2 * e], s.w[c1 + 2 * e + 1]) : both(1.f);
  }
  const long long gh = (long long)p.T * D;
  for (long long first = (long long)blockIdx.x * tokens; s.H > 0 && first < N; first += (long long)gridDim.x * tokens) {
    const int n0 = (int)first, nt = min(tokens, N - n0);
    __syncthreads();  // the tile before has been worked on
    fill_turns(p, n0, nt, turns);
    fill_tile(p, n0, nt, s.xb, s.xt, gh * s.H, D, tile);
    fill_tile(p, n0, nt, s.ob, s.ot, 0, 0, place);
    __syncthreads();
    Walk<ROWS> at(threadIdx.x / L, s.H);
    for (int i0 = 0; i0 < nt * s.H; i0 += ROWS, at.step()) {
      const bool live = at.tok < nt;
      V8 x = {}, y = {}, dx = {}, dy = {};
      if (live) {
        const TI* in = static_cast<const TI*>(s.x) + tile.in[at.tok] + at.h * s.xh;
        const TG* g = static_cast<const TG*>(s.g) + tile.out[at.tok] + at.h * gh;
        load_piece(in + c0, x);
        load_piece(in + c1, y);
        load_piece(g + c0, dx);
        load_piece(g + c1, dy);
      }
      V8 zx, zy;
      float2 ss = both(0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        zx.v[e] = SILU ? silu2(x.v[e]) : x.v[e];
        zy.v[e] = SILU ? silu2(y.v[e]) : y.v[e];
        ss = fma2(zx.v[e], zx.v[e], fma2(zy.v[e], zy.v[e], ss));
      }
      const float* cs = turns + 2 * half * at.tok + 8 * l;
      if (live && turned) turn<INTER, true>(dx, dy, cs, cs + half);
      bool floored;
      const float2 scale = both(row_scale<D, L2>(p.eps, row_sum<D>(ss), floored));
      float2 dots = both(0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        zx.v[e] = mul2(zx.v[e], scale);  // the normed row
        zy.v[e] = mul2(zy.v[e], scale);
        if (live) {
          dwa.v[e] = fma2(dx.v[e], zx.v[e], dwa.v[e]);
          dwb.v[e] = fma2(dy.v[e], zy.v[e], dwb.v[e]);
        }
        dx.v[e] = mul2(dx.v[e], wa.v[e]);
        dy.v[e] = mul2(dy.v[e], wb.v[e]);
        dots = fma2(dx.v[e], zx.v[e], fma2(dy.v[e], zy.v[e], dots));
      }
      float dot = row_sum<D>(dots) * (L2 ? 1.f : 1.f / D);
      if (floored) dot = 0.f;
      if (!live) continue;
      const float2 less = both(-dot);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dx.v[e] = mul2(scale, fma2(zx.v[e], less, dx.v[e]));
        dy.v[e] = mul2(scale, fma2(zy.v[e], less, dy.v[e]));
        if (SILU) {
          auto slope = [](float v) {
            const float g = sigmoid_f(v);
            return g * fmaf(v, 1.f - g, 1.f);
          };
          dx.v[e] = mul2(dx.v[e], make_float2(slope(x.v[e].x), slope(x.v[e].y)));
          dy.v[e] = mul2(dy.v[e], make_float2(slope(y.v[e].x), slope(y.v[e].y)));
        }
      }
      TI* o = static_cast<TI*>(s.out) + place.in[at.tok] + at.h * s.oh;
      store_piece(o + c0, dx);
      store_piece(o + c1, dy);
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a = e & 1 ? dwa.v[e / 2].y : dwa.v[e / 2].x, b = e & 1 ? dwb.v[e / 2].y : dwb.v[e / 2].x;
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane < L) {
      part[warp][c0 + e] = a;
      part[warp][c1 + e] = b;
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

// Tokens of a tile: about 256 rows, at most kMaxTokens tables of turns, and then
// as many fewer as spread the tiles evenly over `ctas` that run at once (B4 T4096
// H16 D128: 16 tokens are 1.73 waves of the forward, 60.4 us, 14 are 1.98, 56.6;
// in the gradient 16 are 4.6 rounds, 91.8 us, 15 are 4.9, 89.9; one token of 64
// sequences H32 takes 2.7 us in 64 tiles, 7.2 in 8).
int tile_tokens(const QkProblem& p, long long ctas) {
  const int heads = p.Hq > p.Hk ? p.Hq : p.Hk;
  int t = 256 / heads;
  t = t < 1 ? 1 : t > kMaxTokens ? kMaxTokens : t;
  const long long N = (long long)p.B * p.T, waves = ((N + t - 1) / t + ctas - 1) / ctas;
  return (int)((N + waves * ctas - 1) / (waves * ctas));
}

// CTAs of the forward that run at once (four to each of B200's 148 SMs; on fewer
// the tiles only spread less evenly) and of the gradient, for each tensor: the silu's derivative takes registers for two CTAs an SM instead
// of three.
constexpr int kFwdCtas = 148 * 4;
int bwd_ctas(bool silu) { return silu ? 148 : 148 * 3 / 2; }

// With tokens enough for one tile of 256 rows on every place, one CTA takes queries
// and keys, so that a token's sines are formed once; with fewer the two run side
// by side.  One CTA | two, H16 D128 in tiles of 16 tokens: 16384 tokens 56.2 | 57.6
// us, 9472 31.9 | 33.6, 4096 19.4 | 15.3, 1024 13.0 | 7.8.
bool one_cta(const QkProblem& p) {
  const int heads = p.Hq > p.Hk ? p.Hq : p.Hk, t = 256 / heads;
  return (long long)p.B * p.T >= (long long)kFwdCtas * (t < 1 ? 1 : t > kMaxTokens ? kMaxTokens : t);
}

// f(INTER, L2, SILU) for the problem's options.
template <typename F>
void by_options(const QkProblem& p, F f) {
  auto silu = [&](auto inter, auto l2) {
    if (p.silu)
      f(inter, l2, std::true_type{});
    else
      f(inter, l2, std::false_type{});
  };
  auto norm = [&](auto inter) {
    if (p.l2)
      silu(inter, std::true_type{});
    else
      silu(inter, std::false_type{});
  };
  if (p.interleaved)
    norm(std::true_type{});
  else
    norm(std::false_type{});
}

template <typename TI, int D>
cudaError_t fwd(const QkProblem& p, cudaStream_t st) {
  const bool both_tensors = one_cta(p);
  const int tokens = tile_tokens(p, both_tensors ? kFwdCtas : kFwdCtas / 2);
  const unsigned tiles = (unsigned)(((long long)p.B * p.T + tokens - 1) / tokens);
  const dim3 grid(tiles, both_tensors ? 1 : 2);
  const size_t smem = (size_t)tokens * p.rot * sizeof(float);
  by_options(p, [&](auto inter, auto l2, auto silu) {
    qk_fwd_kernel<TI, D, inter(), l2(), silu()><<<grid, kThreads, smem, st>>>(p, tokens);
  });
  return cudaGetLastError();
}

template <typename TI, typename TG, int D>
cudaError_t bwd(const QkProblem& p, cudaStream_t st) {
  const int tokens = tile_tokens(p, bwd_ctas(p.silu));
  const unsigned ctas = (unsigned)qk_bwd_ctas(p.B, p.T, p.Hq, p.Hk, p.silu);
  const size_t smem = (size_t)tokens * p.rot * sizeof(float);
  by_options(p, [&](auto inter, auto l2, auto silu) {
    qk_bwd_kernel<TI, TG, D, inter(), l2(), silu()><<<dim3(ctas, 2), kThreads, smem, st>>>(p, tokens);
  });
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

int qk_bwd_ctas(int B, int T, int Hq, int Hk, int silu) {
  QkProblem p{};
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hk = Hk;
  // one wave of what is resident (92 us at B4 T4096 H16 D128; a third more CTAs,
  // and so a second wave, 113 us)
  const long long tokens = tile_tokens(p, bwd_ctas(silu)), tiles = ((long long)B * T + tokens - 1) / tokens;
  return (int)(tiles < bwd_ctas(silu) ? tiles : bwd_ctas(silu));
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
