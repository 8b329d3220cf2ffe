// Gated linear recurrence on tcgen05 tensor cores (bf16 operands, float32
// accumulation and state):  S_t = alpha_t S_{t-1} + k_t^T v_t,  o_t = q_t S_t.
//
// Chunks of C = 128 tokens entered with S.  D_ij is the product of alpha over
// (j, i], G_i over [0, i], c_j over (j, C), gamma over the chunk:
//   O = diag(G) (Q S) + (tril(Q K^T) * D) V,     S <- gamma S + K^T (diag(c) V)
// Every decay is a product of alphas.  With the chunk in four blocks of 32,
// one for each warp's rows: within a block D is a running product along the
// row; between blocks it is pre_i * (products of whole blocks) * suf_j, three
// factors of at most one each that underflow only where D does.  So a score
// costs two multiplications, a wipe (alpha = 0) is exact, and nothing needs an
// exponential.
//
// Roundings to bf16: the decayed scores (one, as the second product's operand)
// and the copy of S that Q reads.  The state itself is held to float32: its
// increment's right operand diag(c) V goes in as two bf16 values (hi + lo, the
// next 8 bits), side by side as N = 128, whose two halves of the accumulator
// are added to the float32 state in registers.
//
// One CTA per (b, h, segment of the sequence, 64 columns of Dv), one CTA per SM:
//   warp 0       TMA of K, Q (two stages) and V
//   warp 1       MMA issue, per chunk c: K^T V~ (c), Q S (c), Q K^T (c+1), P V (c),
//                so that each product's operands have had the other three's time
//   warps 4-7    P (c) = scores * D, TMEM to TMEM (P is the A operand there)
//   warps 8-11   state: S <- gamma S + hi + lo in registers, bf16 tile for Q S
//   warps 12-15  O (c) = G_i QS + PV to a staging tile, stored by TMA
//   warps 16-19  V~ (c) = diag(c) V as hi and lo tiles (gated only)
// C = 128 and full-height MMAs because an SS product of M = 128 reads 4 KB of A
// for every 16 of K whatever N is: larger chunks spread the state's products
// over more tokens, and shared-memory bandwidth is what the kernel spends.
//
// A long sequence over few heads is cut into G segments: a first launch of the
// state part alone (from zero, K and V only) leaves every segment's end state
// and total decay, and each segment's CTA of the main launch starts from
// S0 and the segments before it (S <- Gamma_u S + Send_u), all in float32.
//
// The gradient uses the state part twice: forward with (K, V), and from the end
// with (Q, dO) and the row factors G_i in the place of c_j, storing the state
// at every chunk boundary as bf16 hi and lo.
#include <cuda.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace dn {
namespace {

constexpr int C = kGatedChunk, NV = 64;
static_assert(C == 128, "four warps of 32 rows");
constexpr uint32_t kBlk = 16384;  // 128 rows x 128 bytes (64 bf16 columns)
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpP = 4, kWarpState = 8, kWarpO = 12, kWarpV = 16;
constexpr int kThreads = 20 * 32;
constexpr int kBarP = 1, kBarO = 2, kBarS = 3;
// TMEM columns: scores (and P) [2], increment hi | lo, Q S, P V
constexpr uint32_t TM_SC = 0, TM_DS = 256, TM_QS = 384, TM_PV = 448;

// Shared memory of the main kernel.
template <int DK>
struct OutLayout {
  static constexpr int KB = DK / 64;
  static constexpr uint32_t K_OFF = 0;                  // [2][KB] blocks
  static constexpr uint32_t Q_OFF = K_OFF + 2 * KB * kBlk;
  static constexpr uint32_t V_OFF = Q_OFF + 2 * KB * kBlk;  // [2]
  static constexpr uint32_t VT_OFF = V_OFF + 2 * kBlk;  // hi, lo
  static constexpr uint32_t S_OFF = VT_OFF + 2 * kBlk;  // DK rows x 128 bytes
  static constexpr uint32_t O_OFF = S_OFF + DK * 128;
  static constexpr uint32_t SUF_OFF = O_OFF + kBlk;     // [2][128] floats, then [2][4] block products
  static constexpr uint32_t BAR_OFF = SUF_OFF + 2 * 512 + 32;
  static constexpr uint32_t BYTES = BAR_OFF + 256;
  static constexpr uint32_t ALLOC = BYTES + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
};
// Of the state kernel: NST stages of X and Z, the scaled copy, the stored state.
constexpr int NST = 3;
template <int DK>
struct StateLayout {
  static constexpr int KB = DK / 64;
  static constexpr uint32_t X_OFF = 0;  // [NST][KB] blocks
  static constexpr uint32_t Z_OFF = X_OFF + NST * KB * kBlk;
  static constexpr uint32_t VT_OFF = Z_OFF + NST * kBlk;
  static constexpr uint32_t ST_OFF = VT_OFF + 2 * kBlk;  // hi, lo: DK rows x 128 bytes each
  static constexpr uint32_t BAR_OFF = ST_OFF + 2 * DK * 128;
  static constexpr uint32_t BYTES = BAR_OFF + 256;
  static constexpr uint32_t ALLOC = BYTES + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
};

// mbarriers (8 bytes each), two per name: chunk parity
enum : uint32_t {
  B_FULLQK = 0, B_FULLV = 16, B_SC = 32, B_P = 48, B_VT = 64, B_DS = 80, B_DSFREE = 96, B_S = 112,
  B_QS = 128, B_PV = 144, B_OFREE = 160, B_FIN = 176, B_TMEM = 184, B_ABORT = 188
};
// of the state kernel: B_XFULL and B_XFREE one per stage
enum : uint32_t {
  C_FULL = 0, C_FREE = 24, C_VT = 48, C_DS = 64, C_DSFREE = 80, C_FIN = 96, C_TMEM = 104, C_ABORT = 108
};

// The alphas of chunk c that a lane needs: tokens 32 k + lane of each block k (1 past T).
__device__ __forceinline__ void load_alpha(const float* alpha, int T, int c, float (&a)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = c * C + 32 * k + (int)(threadIdx.x & 31);
    a[k] = t < T ? __ldg(alpha + t) : 1.f;
  }
}
__device__ __forceinline__ float warp_product(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x *= __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Product over [0, lane] of the warp's values.
__device__ __forceinline__ float prefix_product(float a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, a, o);
    if (lane >= o) a *= x;
  }
  return a;
}
// Product over (lane, 32).
__device__ __forceinline__ float suffix_product(float a) {
  const int lane = threadIdx.x & 31;
  float s = __shfl_down_sync(0xffffffffu, a, 1);
  if (lane == 31) s = 1.f;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_down_sync(0xffffffffu, s, o);
    if (lane + o < 32) s *= x;
  }
  return s;
}
// G_i of the warp's row i = 32 w + lane; c_j of row j.
__device__ __forceinline__ float decay_into(const float (&a)[4], int w) {
  float x = prefix_product(w == 0 ? a[0] : w == 1 ? a[1] : w == 2 ? a[2] : a[3]);
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    const float b = warp_product(a[u]);
    if (u < w) x *= b;
  }
  return x;
}
__device__ __forceinline__ float decay_out(const float (&a)[4], int w) {
  float x = suffix_product(w == 0 ? a[0] : w == 1 ? a[1] : w == 2 ? a[2] : a[3]);
#pragma unroll
  for (int u = 1; u < 4; ++u) {
    const float b = warp_product(a[u]);
    if (u > w) x *= b;
  }
  return x;
}
__device__ __forceinline__ float decay_chunk(const float (&a)[4]) {
  return warp_product(a[0] * a[1] * a[2] * a[3]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float lo_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_half(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight values as bf16 hi, and what is left of them as bf16 lo.
__device__ __forceinline__ void split8(const float* x, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack2_bf16(x[2 * i], x[2 * i + 1]);
    l[i] = pack2_bf16(x[2 * i] - lo_half(h[i]), x[2 * i + 1] - hi_half(h[i]));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Row `row` of a 64-column tile scaled by f into the hi and lo tiles.
__device__ __forceinline__ void scale_row(const uint8_t* tile, uint8_t* hi, uint8_t* lo, int row, float f) {
#pragma unroll
  for (int c0 = 0; c0 < 8; c0 += 4) {
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const uint4*>(tile + sw128_off(row, c0 + i));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
      unpack_bf16x8(u[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= f;
      uint4 h, l;
      split8(x, h, l);
      *reinterpret_cast<uint4*>(hi + sw128_off(row, c0 + i)) = h;
      *reinterpret_cast<uint4*>(lo + sw128_off(row, c0 + i)) = l;
    }
  }
}

// The 64 columns of this thread's state row, entering segment g: the caller's
// state and the segments passed before it in the scan's direction.
template <int DK, bool REV>
__device__ __forceinline__ void enter_state(const GatedScan& p, size_t bh, int g, int j0, int row, float (&s)[NV]) {
  const size_t sblk = (size_t)DK * p.Dv, at = (size_t)row * p.Dv + j0;
  const float* src = p.S_in ? p.S_in + bh * p.S_in_stride + at : nullptr;
#pragma unroll
  for (int j = 0; j < NV; j += 4) {
    const float4 v = src ? *reinterpret_cast<const float4*>(src + j) : make_float4(0.f, 0.f, 0.f, 0.f);
    s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
  }
  const int n = REV ? p.G - 1 - g : g;
  for (int i = 0; i < n; ++i) {
    const size_t u = bh * p.G + (REV ? p.G - 1 - i : i);
    const float gam = p.seg_decay[u];
    const float4* e = reinterpret_cast<const float4*>(p.seg_end + u * sblk + at);
#pragma unroll
    for (int j = 0; j < NV; j += 4) {
      const float4 v = __ldg(e + j / 4);
      s[j] = fmaf(gam, s[j], v.x);
      s[j + 1] = fmaf(gam, s[j + 1], v.y);
      s[j + 2] = fmaf(gam, s[j + 2], v.z);
      s[j + 3] = fmaf(gam, s[j + 3], v.w);
    }
  }
}
__device__ __forceinline__ void leave_state(float* dst, const float (&s)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; j += 4)
    *reinterpret_cast<float4*>(dst + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
}

// s <- gamma s + this lane's increment (its hi and lo halves at taddr, + 64)
template <bool GATED>
__device__ __forceinline__ void add_increment(float (&s)[NV], float gamma, uint32_t taddr) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t x[16], y[16];
    tmem_ld16(taddr + 16 * h, x);
    if (GATED) tmem_ld16(taddr + 64 + 16 * h, y);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (GATED)
        s[16 * h + e] = fmaf(gamma, s[16 * h + e], __uint_as_float(x[e]) + __uint_as_float(y[e]));
      else
        s[16 * h + e] += __uint_as_float(x[e]);
    }
  }
}

// ------------------------------------------------------------- main kernel --
template <int DK, bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    gated_out_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                     const GatedScan p) {
  using L = OutLayout<DK>;
  constexpr int KB = L::KB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = warp_uniform(smem_u32(sm));
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)warp_uniform((uint32_t)tid >> 5), w = warp & 3;
  const int nsl = p.Dv / NV, T = p.T;
  const int slice = blockIdx.x % nsl, g = (blockIdx.x / nsl) % p.G, bh = blockIdx.x / nsl / p.G;
  const int j0 = slice * NV, nch = (T + C - 1) / C;
  const int first = g * p.seg_chunks, n = min(p.seg_chunks, nch - first);  // chunks [first, first + n)
  const uint32_t bar = sb + L::BAR_OFF;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::BAR_OFF + B_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::BAR_OFF + B_ABORT);
  const float* alpha = GATED ? p.alpha + (size_t)bh * T : nullptr;

  if (tid == 0) {
    for (uint32_t i = 0; i < 2; ++i) {
      for (uint32_t b : {B_FULLQK, B_FULLV, B_SC, B_DS, B_QS, B_PV}) mbar_init(bar + b + 8 * i, 1);
      for (uint32_t b : {B_P, B_VT, B_DSFREE, B_S, B_OFREE}) mbar_init(bar + b + 8 * i, 4);  // one arrival per warp
    }
    mbar_init(bar + B_FIN, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  const WaitCtl wc{abort_flag, p.status, kWaitLimitNs};
  const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
  auto full = [&](uint32_t b, int c) { return mbar_wait(bar + b + 8 * (c & 1), (c >> 1) & 1, wc); };
  auto wait_all = [&](uint32_t b, int c) { return __all_sync(0xffffffffu, full(b, c)) != 0; };
  auto arrive = [&](uint32_t b, int c) {  // one arrival for the warp, after all its lanes
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + b + 8 * (c & 1));
  };

  if (warp == kWarpTma) {
    // ------------------------------------------------------------------ TMA --
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      int qk = 0, v = 0;  // issued
      for (int c = 0; c < n; ++c) {
        const int s = c & 1, row = (first + c) * C;
        // K (c-2) was last read by its increment, Q by Q S, V by P V
        if (c >= 2 && !(full(B_DS, c - 2) && full(B_QS, c - 2))) break;
        mbar_expect_tx(bar + B_FULLQK + 8 * s, 2 * KB * kBlk);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          tma_load_3d(sb + L::K_OFF + (s * KB + kb) * kBlk, &tmK, bar + B_FULLQK + 8 * s, kb * 64, row, bh);
          tma_load_3d(sb + L::Q_OFF + (s * KB + kb) * kBlk, &tmQ, bar + B_FULLQK + 8 * s, kb * 64, row, bh);
        }
        qk = c + 1;
        if (c >= 2 && !full(B_PV, c - 2)) break;
        mbar_expect_tx(bar + B_FULLV + 8 * s, kBlk);
        tma_load_3d(sb + L::V_OFF + s * kBlk, &tmV, bar + B_FULLV + 8 * s, j0, row, bh);
        v = c + 1;
      }
      int zero = 0;  // never leave with copies in flight
      const WaitCtl drain{&zero, p.status, kWaitLimitNs};
      for (int c = qk > 2 ? qk - 2 : 0; c < qk; ++c) (void)mbar_wait(bar + B_FULLQK + 8 * (c & 1), (c >> 1) & 1, drain);
      for (int c = v > 2 ? v - 2 : 0; c < v; ++c) (void)mbar_wait(bar + B_FULLV + 8 * (c & 1), (c >> 1) & 1, drain);
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ MMA --
    auto scores = [&](int c) {
      constexpr uint32_t id = idesc_bf16(128, 128, false, false);
      const uint32_t s = (c & 1) * KB * kBlk;
      const uint64_t dq = desc_k(sb + L::Q_OFF + s), dk = desc_k(sb + L::K_OFF + s);
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        const uint32_t off = (ks >> 2) * kBlk + (ks & 3) * 32;
        mma_bf16_ss_elect(tmem + TM_SC + 128 * (c & 1), desc_step(dq, off), desc_step(dk, off), id, ks > 0);
      }
      mma_commit_elect(bar + B_SC + 8 * (c & 1));
    };
    // K^T [hi | lo] (gated) or K^T V; with DK = 64 the product's upper 64 rows
    // are computed from the next block and never read
    auto increment = [&](int c) {
      constexpr uint32_t id = idesc_bf16(128, GATED ? 128 : 64, true, true);
      const uint64_t da = desc_mn(sb + L::K_OFF + (c & 1) * KB * kBlk, kBlk);
      const uint64_t db = desc_mn(sb + (GATED ? L::VT_OFF : L::V_OFF + (c & 1) * kBlk), kBlk);
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        mma_bf16_ss_elect(tmem + TM_DS, desc_step(da, ks * 2048), desc_step(db, ks * 2048), id, ks > 0);
      mma_commit_elect(bar + B_DS + 8 * (c & 1));
    };
    auto read_state = [&](int c) {
      constexpr uint32_t id = idesc_bf16(128, 64, false, true);
      const uint64_t dq = desc_k(sb + L::Q_OFF + (c & 1) * KB * kBlk), ds = desc_mn(sb + L::S_OFF, kBlk);
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks)
        mma_bf16_ss_elect(tmem + TM_QS, desc_step(dq, (ks >> 2) * kBlk + (ks & 3) * 32), desc_step(ds, ks * 2048), id,
                          ks > 0);
      mma_commit_elect(bar + B_QS + 8 * (c & 1));
    };
    auto inner = [&](int c) {
      constexpr uint32_t id = idesc_bf16(128, 64, false, true);
      const uint64_t dv = desc_mn(sb + L::V_OFF + (c & 1) * kBlk, kBlk);
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        mma_bf16_ts_elect(tmem + TM_PV, tmem + TM_SC + 128 * (c & 1) + 8 * ks, desc_step(dv, ks * 2048), id, ks > 0);
      mma_commit_elect(bar + B_PV + 8 * (c & 1));
    };
    bool ok = wait_all(B_FULLQK, 0);
    if (ok) {
      tc_fence_after();
      scores(0);
    }
    for (int c = 0; c < n && ok; ++c) {
      ok = wait_all(GATED ? B_VT : B_FULLV, c) && (c < 1 || wait_all(B_DSFREE, c - 1));
      if (!ok) break;
      tc_fence_after();
      increment(c);
      ok = wait_all(B_S, c) && (c < 1 || wait_all(B_OFREE, c - 1));
      if (!ok) break;
      tc_fence_after();
      read_state(c);
      if (c + 1 < n) {
        // scores (c+1) overwrite P (c-1), which P V (c-1) has read
        ok = wait_all(B_FULLQK, c + 1) && (c < 1 || wait_all(B_PV, c - 1));
        if (!ok) break;
        tc_fence_after();
        scores(c + 1);
      }
      ok = wait_all(B_P, c) && (GATED ? true : wait_all(B_FULLV, c));
      if (!ok) break;
      tc_fence_after();
      inner(c);
    }
    tc_fence_after();  // no MMA may outlive TMEM
    mma_commit_elect(bar + B_FIN);
    int zero = 0;
    const WaitCtl fin{&zero, p.status, kWaitLimitNs};
    (void)mbar_wait(bar + B_FIN, 0, fin);
  } else if (warp >= kWarpP && warp < kWarpP + 4) {
    // -------------------------------------------------------------- scores --
    float a = 1.f, next = 1.f;
    auto load = [&](int c) {
      const int t = (first + c) * C + 32 * w + lane;
      return GATED && t < T ? __ldg(alpha + t) : 1.f;
    };
    next = load(0);
    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      a = next;
      if (c + 1 < n) next = load(c + 1);
      float pre = 1.f, mid = 1.f;
      float* suf = reinterpret_cast<float*>(sm + L::SUF_OFF) + (c & 1) * C;
      float* blk = reinterpret_cast<float*>(sm + L::SUF_OFF + 1024) + (c & 1) * 4;
      if (GATED) {
        pre = prefix_product(a);
        suf[32 * w + lane] = suffix_product(a);
        if (lane == 31) blk[w] = pre;
      }
      // every warp's factors are in place (and all have left the buffer of chunk c-2)
      ok = named_bar_and(kBarP, 128, full(B_SC, c));
      if (!ok) break;
      tc_fence_after();
      const uint32_t sc = lanes + TM_SC + 128 * (c & 1);
      // column blocks from the diagonal down, then zeros above it: block cb is
      // read before P overwrites it (P's columns 16 cb .. of the same lanes)
      uint32_t d[16];
#pragma unroll 1
      for (int cb = 0; cb < 4; ++cb) {
        if (cb > w) {
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i] = 0;
        } else {
          uint32_t x[32];
          tmem_ld32(sc + 32 * cb, x);
          if (cb < w) {
            if (GATED) {
              mid = pre;
              for (int u = cb + 1; u < w; ++u) mid *= blk[u];
            }
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
              if (GATED) f = *reinterpret_cast<const float4*>(suf + 32 * cb + j);
              if (GATED) { f.x *= mid; f.y *= mid; f.z *= mid; f.w *= mid; }
              d[j / 2] = pack2_bf16(__uint_as_float(x[j]) * f.x, __uint_as_float(x[j + 1]) * f.y);
              d[j / 2 + 1] = pack2_bf16(__uint_as_float(x[j + 2]) * f.z, __uint_as_float(x[j + 3]) * f.w);
            }
          } else {
            tmem_wait_ld();
            float run = 1.f;
#pragma unroll
            for (int j = 30; j >= 0; j -= 2) {  // columns j + 1, then j
              if (GATED && j < 30) {
                const float t = __shfl_sync(0xffffffffu, a, j + 2 < 32 ? j + 2 : 31);
                run = j + 1 < lane ? run * t : 1.f;
              }
              const float hi = j + 1 <= lane ? __uint_as_float(x[j + 1]) * run : 0.f;
              if (GATED) {
                const float t = __shfl_sync(0xffffffffu, a, j + 1);
                run = j < lane ? run * t : 1.f;
              }
              d[j / 2] = pack2_bf16(j <= lane ? __uint_as_float(x[j]) * run : 0.f, hi);
            }
          }
        }
        tmem_st16(sc + 16 * cb, d);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(B_P, c);
    }
  } else if (warp >= kWarpState && warp < kWarpState + 4) {
    // --------------------------------------------------------------- state --
    const int row = 32 * w + lane;
    const bool live = row < DK;
    float s[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) s[j] = 0.f;
    if (live) enter_state<DK, false>(p, bh, g, j0, row, s);
    auto put = [&]() {
      if (live) {
#pragma unroll
        for (int c16 = 0; c16 < 8; ++c16) st_bf16x8(sm + L::S_OFF + sw128_off(row, c16), s + 8 * c16);
      }
      fence_proxy_async_smem();
    };
    put();
    arrive(B_S, 0);
    float a[4] = {1.f, 1.f, 1.f, 1.f};
    if (GATED) load_alpha(alpha, T, first, a);
    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      const float gamma = GATED ? decay_chunk(a) : 1.f;
      if (GATED && c + 1 < n) load_alpha(alpha, T, first + c + 1, a);
      ok = wait_all(B_DS, c);
      if (!ok) break;
      tc_fence_after();
      add_increment<GATED>(s, gamma, lanes + TM_DS);
      tc_fence_before();
      arrive(B_DSFREE, c);
      if (c + 1 < n) {
        ok = wait_all(B_QS, c);  // Q S (c) has read the tile
        if (!ok) break;
        put();
        arrive(B_S, c + 1);
      }
    }
    if (ok && live && p.S_out && g == p.G - 1)
      leave_state(p.S_out + (size_t)bh * DK * p.Dv + (size_t)row * p.Dv + j0, s);
  } else if (warp >= kWarpO && warp < kWarpO + 4) {
    // -------------------------------------------------------------- output --
    const int row = 32 * w + lane;
    const bool leader = warp == kWarpO && lane == 0;
    float a[4] = {1.f, 1.f, 1.f, 1.f};
    if (GATED) load_alpha(alpha, T, first, a);
    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      const float into = GATED ? decay_into(a, w) : 1.f;
      if (GATED && c + 1 < n) load_alpha(alpha, T, first + c + 1, a);
      if (leader) bulk_wait_group_read<0>();  // the staging tile is free
      ok = named_bar_and(kBarO, 128, full(B_PV, c) && full(B_QS, c));
      if (!ok) break;
      tc_fence_after();
      uint4 out[8];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t x[16], y[16];
        tmem_ld16(lanes + TM_QS + 16 * h, x);
        tmem_ld16(lanes + TM_PV + 16 * h, y);
        tmem_wait_ld();
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          o[e / 2] = pack2_bf16(fmaf(into, __uint_as_float(x[e]), __uint_as_float(y[e])),
                                fmaf(into, __uint_as_float(x[e + 1]), __uint_as_float(y[e + 1])));
        out[2 * h] = make_uint4(o[0], o[1], o[2], o[3]);
        out[2 * h + 1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
      tc_fence_before();
      arrive(B_OFREE, c);
#pragma unroll
      for (int c16 = 0; c16 < 8; ++c16) *reinterpret_cast<uint4*>(sm + L::O_OFF + sw128_off(row, c16)) = out[c16];
      fence_proxy_async_smem();
      named_bar_sync(kBarO, 128);
      if (leader) {
        tma_store_3d(&tmO, sb + L::O_OFF, j0, (first + c) * C, bh);
        bulk_commit_group();
      }
    }
    if (leader) bulk_wait_group_all();
  } else if (GATED && warp >= kWarpV) {
    // --------------------------------------------------------- diag(c) V --
    const int row = 32 * w + lane;
    float a[4];
    load_alpha(alpha, T, first, a);
    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      const float out = decay_out(a, w);
      if (c + 1 < n) load_alpha(alpha, T, first + c + 1, a);
      ok = wait_all(B_FULLV, c) && (c < 1 || wait_all(B_DS, c - 1));
      if (!ok) break;
      scale_row(sm + L::V_OFF + (c & 1) * kBlk, sm + L::VT_OFF, sm + L::VT_OFF + kBlk, row, out);
      fence_proxy_async_smem();
      arrive(B_VT, c);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ state kernel --
// x = k, z = v (forward) or x = q, z = dO from the end (REV); the segments'
// end states from zero (STORE = false), or every chunk's entry state in the
// scan's direction as bf16 hi and lo, from the segment's true entry (STORE).
constexpr int kStateThreads = 12 * 32;  // TMA 0, MMA 1, state 4-7, scaling 8-11
template <int DK, bool GATED, bool REV, bool STORE>
__global__ void __launch_bounds__(kStateThreads, 1)
    gated_state_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmZ,
                       const __grid_constant__ CUtensorMap tmS, const GatedScan p) {
  using L = StateLayout<DK>;
  constexpr int KB = L::KB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = warp_uniform(smem_u32(sm));
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)warp_uniform((uint32_t)tid >> 5), w = warp & 3;
  const int nsl = p.Dv / NV, T = p.T, segs = STORE ? p.G : p.G - 1;
  const int slice = blockIdx.x % nsl, bh = blockIdx.x / nsl / segs;
  // without STORE the scan's last segment is not needed
  const int g = (int)(blockIdx.x / nsl) % segs + (!STORE && REV ? 1 : 0);
  const int j0 = slice * NV, nch = (T + C - 1) / C;
  const int first = g * p.seg_chunks, n = min(p.seg_chunks, nch - first);
  auto chunk = [&](int i) { return REV ? first + n - 1 - i : first + i; };
  const uint32_t bar = sb + L::BAR_OFF;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::BAR_OFF + C_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::BAR_OFF + C_ABORT);
  const float* alpha = GATED ? p.alpha + (size_t)bh * T : nullptr;

  if (tid == 0) {
    for (uint32_t i = 0; i < (uint32_t)NST; ++i) {
      mbar_init(bar + C_FULL + 8 * i, 1);
      mbar_init(bar + C_FREE + 8 * i, 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(bar + C_VT + 8 * i, 4);
      mbar_init(bar + C_DS + 8 * i, 1);
      mbar_init(bar + C_DSFREE + 8 * i, 4);
    }
    mbar_init(bar + C_FIN, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  const WaitCtl wc{abort_flag, p.status, kWaitLimitNs};
  auto wait2 = [&](uint32_t b, int i) {  // a barrier pair by parity
    return __all_sync(0xffffffffu, mbar_wait(bar + b + 8 * (i & 1), (i >> 1) & 1, wc)) != 0;
  };
  auto wait_stage = [&](uint32_t b, int i) { return mbar_wait(bar + b + 8 * (i % NST), (i / NST) & 1, wc); };

  if (warp == kWarpTma) {
    if (lane == 0) {
      prefetch_tmap(&tmX);
      prefetch_tmap(&tmZ);
      int issued = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i % NST, row = chunk(i) * C;
        if (i >= NST && !wait_stage(C_FREE, i - NST)) break;
        const uint32_t f = bar + C_FULL + 8 * s;
        mbar_expect_tx(f, (KB + 1) * kBlk);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) tma_load_3d(sb + L::X_OFF + (s * KB + kb) * kBlk, &tmX, f, kb * 64, row, bh);
        tma_load_3d(sb + L::Z_OFF + s * kBlk, &tmZ, f, j0, row, bh);
        issued = i + 1;
      }
      int zero = 0;  // never leave with copies in flight
      const WaitCtl drain{&zero, p.status, kWaitLimitNs};
      for (int i = issued > NST ? issued - NST : 0; i < issued; ++i)
        (void)mbar_wait(bar + C_FULL + 8 * (i % NST), (i / NST) & 1, drain);
    }
  } else if (warp == kWarpMma) {
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int s = i % NST, b = i & 1;
      ok = (GATED ? wait2(C_VT, i) : __all_sync(0xffffffffu, wait_stage(C_FULL, i)) != 0) &&
           (i < 2 || wait2(C_DSFREE, i - 2));
      if (!ok) break;
      tc_fence_after();
      constexpr uint32_t id = idesc_bf16(128, GATED ? 128 : 64, true, true);
      const uint64_t da = desc_mn(sb + L::X_OFF + s * KB * kBlk, kBlk);
      const uint64_t db = desc_mn(sb + (GATED ? L::VT_OFF : L::Z_OFF + s * kBlk), kBlk);
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        mma_bf16_ss_elect(tmem + 128 * b, desc_step(da, ks * 2048), desc_step(db, ks * 2048), id, ks > 0);
      mma_commit_elect(bar + C_DS + 8 * b);
      mma_commit_elect(bar + C_FREE + 8 * s);
    }
    tc_fence_after();  // no MMA may outlive TMEM
    mma_commit_elect(bar + C_FIN);
    int zero = 0;
    const WaitCtl fin{&zero, p.status, kWaitLimitNs};
    (void)mbar_wait(bar + C_FIN, 0, fin);
  } else if (warp >= 4 && warp < 8) {
    const int row = 32 * w + lane;
    const bool live = row < DK, leader = warp == 4 && lane == 0;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
    float s[NV], total = 1.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) s[j] = 0.f;
    if (STORE && live) enter_state<DK, REV>(p, bh, g, j0, row, s);
    // The main kernel takes the caller's state from the slot that the last
    // segment leaves unused, so that it may write S_out over S0.
    if (!STORE && !REV && live && g == 0 && p.S_in) {
      const size_t at = (size_t)row * p.Dv + j0, sblk = (size_t)DK * p.Dv;
      const float4* src = reinterpret_cast<const float4*>(p.S_in + bh * p.S_in_stride + at);
      float4* dst = reinterpret_cast<float4*>(p.seg_end + ((size_t)bh * p.G + p.G - 1) * sblk + at);
#pragma unroll
      for (int j = 0; j < NV / 4; ++j) dst[j] = src[j];
    }
    float a[4] = {1.f, 1.f, 1.f, 1.f};
    if (GATED) load_alpha(alpha, T, chunk(0), a);
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const float gamma = GATED ? decay_chunk(a) : 1.f;
      total *= gamma;
      if (GATED && i + 1 < n) load_alpha(alpha, T, chunk(i + 1), a);
      if (STORE) {
        if (leader) bulk_wait_group_read<0>();  // the staging tiles are free
        named_bar_sync(kBarS, 128);
        if (live) {
#pragma unroll
          for (int c16 = 0; c16 < 8; ++c16) {
            uint4 h, l;
            split8(s + 8 * c16, h, l);
            *reinterpret_cast<uint4*>(sm + L::ST_OFF + sw128_off(row, c16)) = h;
            *reinterpret_cast<uint4*>(sm + L::ST_OFF + DK * 128 + sw128_off(row, c16)) = l;
          }
        }
        fence_proxy_async_smem();
        named_bar_sync(kBarS, 128);
        if (leader) {
          const int at = (bh * nch + chunk(i)) * 2;
          tma_store_3d(&tmS, sb + L::ST_OFF, j0, 0, at);
          tma_store_3d(&tmS, sb + L::ST_OFF + DK * 128, j0, 0, at + 1);
          bulk_commit_group();
        }
      }
      // with STORE the four warps meet at barriers, so they leave together
      ok = STORE ? named_bar_and(kBarS, 128, mbar_wait(bar + C_DS + 8 * (i & 1), (i >> 1) & 1, wc)) : wait2(C_DS, i);
      if (!ok) break;
      tc_fence_after();
      add_increment<GATED>(s, gamma, lanes + 128 * (i & 1));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + C_DSFREE + 8 * (i & 1));
    }
    if (leader) bulk_wait_group_all();
    if (ok && live) {
      const size_t at = (size_t)row * p.Dv + j0, sblk = (size_t)DK * p.Dv;
      if (STORE) {
        if (p.S_out && g == (REV ? 0 : p.G - 1)) leave_state(p.S_out + (size_t)bh * sblk + at, s);
      } else {
        leave_state(p.seg_end + ((size_t)bh * p.G + g) * sblk + at, s);
        if (leader && slice == 0) p.seg_decay[(size_t)bh * p.G + g] = total;
      }
    }
  } else if (GATED && warp >= 8) {
    const int row = 32 * w + lane;
    float a[4];
    load_alpha(alpha, T, chunk(0), a);
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const float f = REV ? decay_into(a, w) : decay_out(a, w);
      if (i + 1 < n) load_alpha(alpha, T, chunk(i + 1), a);
      ok = __all_sync(0xffffffffu, wait_stage(C_FULL, i)) && (i < 1 || wait2(C_DS, i - 1));
      if (!ok) break;
      scale_row(sm + L::Z_OFF + (i % NST) * kBlk, sm + L::VT_OFF, sm + L::VT_OFF + kBlk, row, f);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + C_VT + 8 * (i & 1));
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 256);
}

template <int DK, bool GATED>
cudaError_t launch_out(const GatedProblem& p, const GatedScan& s, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mo;
  const int BH = p.B * p.H;
  if (!make_tmap_3d_bf16(&mq, p.q, DK, p.T, BH, C) || !make_tmap_3d_bf16(&mk, p.k, DK, p.T, BH, C) ||
      !make_tmap_3d_bf16(&mv, p.v, p.Dv, p.T, BH, C) || !make_tmap_3d_bf16(&mo, p.o, p.Dv, p.T, BH, C))
    return cudaErrorInvalidValue;
  auto kern = gated_out_kernel<DK, GATED>;
  constexpr int smem = (int)OutLayout<DK>::ALLOC;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // without a gate the scaling warps have nothing to do
  kern<<<(unsigned)((size_t)BH * s.G * (p.Dv / NV)), GATED ? kThreads : 32 * kWarpV, smem, st>>>(mq, mk, mv, mo, s);
  return cudaGetLastError();
}

// The state kernel over x (BH,T,DK) and z (BH,T,Dv).
template <int DK, bool GATED, bool REV, bool STORE>
cudaError_t launch_state(const void* x, const void* z, void* states, int BH, const GatedScan& s, cudaStream_t st) {
  CUtensorMap mx, mz, ms;
  const int nch = (s.T + C - 1) / C;
  if (!make_tmap_3d_bf16(&mx, x, DK, s.T, BH, C) || !make_tmap_3d_bf16(&mz, z, s.Dv, s.T, BH, C))
    return cudaErrorInvalidValue;
  ms = mz;
  if (STORE && !make_tmap_3d_bf16(&ms, states, s.Dv, DK, 2 * BH * nch, DK)) return cudaErrorInvalidValue;
  auto kern = gated_state_kernel<DK, GATED, REV, STORE>;
  constexpr int smem = (int)StateLayout<DK>::ALLOC;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const size_t segs = STORE ? s.G : s.G - 1;
  kern<<<(unsigned)(BH * segs * (s.Dv / NV)), GATED ? kStateThreads : 256, smem, st>>>(mx, mz, ms, s);
  return cudaGetLastError();
}

GatedScan gated_scan_of(const GatedProblem& p, void* scratch) {
  GatedScan s{};
  s.alpha = p.alpha;
  s.T = p.T;
  s.Dv = p.Dv;
  s.status = p.status;
  const int BH = p.B * p.H;
  s.G = p.G;
  s.seg_chunks = p.seg_chunks;
  s.seg_decay = static_cast<float*>(scratch);
  s.seg_end = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + ((size_t)BH * s.G * 4 + 255) / 256 * 256);
  return s;
}

template <int DK, bool GATED>
cudaError_t fwd(const GatedProblem& p, cudaStream_t st) {
  const int BH = p.B * p.H;
  GatedScan s = gated_scan_of(p, p.scratch);
  const size_t sblk = (size_t)DK * p.Dv;
  s.S_in = p.S0;
  s.S_in_stride = sblk;
  s.S_out = p.S_out;
  if (s.G > 1) {
    cudaError_t e = launch_state<DK, GATED, false, false>(p.k, p.v, nullptr, BH, s, st);
    if (e != cudaSuccess) return e;
    if (p.S0) {
      s.S_in = s.seg_end + (s.G - 1) * sblk;
      s.S_in_stride = s.G * sblk;
    }
  }
  return launch_out<DK, GATED>(p, s, st);
}

}  // namespace

// Segments: enough for one CTA on every SM, where the state part run twice
// (about half a chunk's cost each time, and some three chunks of launch and
// entry) costs less than the chunks it takes off the longest chain.
void gated_segments(int BH, int T, int Dv, int sms, int* G, int* seg_chunks) {
  const int nch = (T + C - 1) / C;
  const long long ctas = (long long)BH * (Dv / NV);
  *G = 1;
  *seg_chunks = nch;
  if (ctas < 1 || sms < 2 * ctas) return;
  const int g = (int)(sms / ctas);
  const int per = (nch + g - 1) / g;
  if (2 * nch <= 3 * per + 6) return;
  *seg_chunks = per;
  *G = (nch + per - 1) / per;
}

size_t gated_segment_bytes(int BH, int G, int Dk, int Dv) {
  return G > 1 ? ((size_t)BH * G * 4 + 255) / 256 * 256 + (size_t)BH * G * Dk * Dv * 4 : 0;
}

cudaError_t launch_gated_tc_fwd(const GatedProblem& p, cudaStream_t st) {
  if (p.alpha) return p.Dk == 128 ? fwd<128, true>(p, st) : fwd<64, true>(p, st);
  return p.Dk == 128 ? fwd<128, false>(p, st) : fwd<64, false>(p, st);
}

}  // namespace dn
