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
//   warp 0       TMA of K, Q (two stages) and V (three)
//   warps 1, 2   MMA issue: Q K^T (c), P V (c-1) | K^T V~ (c), Q S (c).  Issuing a
//                chunk's MMAs and waiting for their operands takes one warp longer
//                than the tensor core needs to run them, so there are two
//   warp 3       the decays of a chunk's rows, ahead
//   warps 4-11   V~ (c) = diag(c) V as hi and lo tiles, then P (c) = scores * D,
//                TMEM to TMEM (P is the A operand there); two warps to 32 rows,
//                half of the columns each
//   warps 12-15  state: S <- gamma S + hi + lo in registers, bf16 tile for Q S
//   warps 16-19  O (c) = G_i QS + PV
// C = 128 and full-height MMAs because an SS product of M = 128 reads 4 KB of A
// for every 16 of K whatever N is: larger chunks spread the state's products
// over more tokens, and shared-memory bandwidth is what the kernel spends (the
// operands, the tiles in and the scaling are 2700 of a chunk's 3400 cycles).  B4
// H16 T4096 D128: 64 to 68 us for 274 MB (41 us at a copy's rate).  32 warps of
// 64 registers instead of 20 took 83 us where these took 78.
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
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpMma2 = 2, kWarpDecay = 3, kWarpP = 4, kWarpState = 12, kWarpO = 16;
constexpr int kThreads = 20 * 32;
constexpr int kBarS = 1, kBarJoin = 2;
// TMEM columns: scores [2] (P's halves in columns 0-31 and 64-95 of them), increment hi | lo, Q S, P V
constexpr uint32_t TM_SC = 0, TM_DS = 256, TM_QS = 384, TM_PV = 448;

// A chunk's decays: the products of the blocks of 32 tokens, and of every token
// the product over the tokens of its block behind it.
constexpr uint32_t kDecayBytes = 16 + 4 * C;

// Shared memory of the main kernel.
template <int DK>
struct OutLayout {
  static constexpr int KB = DK / 64;
  static constexpr uint32_t K_OFF = 0;                  // [2][KB] blocks
  static constexpr uint32_t Q_OFF = K_OFF + 2 * KB * kBlk;
  static constexpr uint32_t V_OFF = Q_OFF + 2 * KB * kBlk;  // [3]
  static constexpr uint32_t VT_OFF = V_OFF + 3 * kBlk;  // hi, lo
  static constexpr uint32_t S_OFF = VT_OFF + 2 * kBlk;  // DK rows x 128 bytes
  static constexpr uint32_t SUF_OFF = S_OFF + DK * 128;  // [3]: 4 block products, 128 floats
  static constexpr uint32_t BAR_OFF = SUF_OFF + 3 * kDecayBytes;
  static constexpr uint32_t BYTES = BAR_OFF + 272;
  static constexpr uint32_t ALLOC = BYTES + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
};
// Of the state kernel: two stages of X and Z, the scaled copy of Z twice, the
// stored state.
template <int DK>
struct StateLayout {
  static constexpr int KB = DK / 64;
  static constexpr uint32_t X_OFF = 0;  // [2][KB] blocks
  static constexpr uint32_t Z_OFF = X_OFF + 2 * KB * kBlk;
  static constexpr uint32_t VT_OFF = Z_OFF + 2 * kBlk;   // [2]: hi, lo
  static constexpr uint32_t ST_OFF = VT_OFF + 4 * kBlk;  // hi, lo: DK rows x 128 bytes each
  static constexpr uint32_t BAR_OFF = ST_OFF + 2 * DK * 128;
  static constexpr uint32_t BYTES = BAR_OFF + 128;
  static constexpr uint32_t ALLOC = BYTES + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
};

// mbarriers (8 bytes each), two per name (chunk parity; B_FIN: one per issuer),
// three for B_FULLV, B_VFREE and B_DECAY (stage).  A parity can only be told from the one
// before it, so whoever waits for a phase must stand between it and the next but one
enum : uint32_t {
  B_FULLK = 0, B_FULLQ = 16, B_FULLV = 32, B_SC = 56, B_P = 72, B_VT = 88, B_DS = 104, B_DSFREE = 120, B_S = 136,
  B_QS = 152, B_PV = 168, B_OFREE = 184, B_VFREE = 200, B_DECAY = 224, B_FIN = 248, B_TMEM = 264
};
// of the state kernel, two per name (chunk parity)
enum : uint32_t { C_FULL = 0, C_FREE = 16, C_VT = 32, C_DS = 48, C_DSFREE = 64, C_FIN = 80, C_TMEM = 88 };

// mbar_wait made short, its limit in polls instead of nanoseconds.  The roles of
// a kernel run different code at the same time and wait at some thirty places;
// where their loops together outgrow the SM's instruction cache, every warp
// stalls on fetches.  A poll sleeps until the phase completes or the hint of 200
// us runs out, so 2^15 of them are up to 6.5 seconds.  Polls that come back at
// once are still about a millisecond; the longest wait of a running pipeline is
// that for a late segment's state, 0.25 us for each segment before it, 37 us for
// the 148 that a head of 64 columns can be cut into on 148 SMs.  Whoever gives up
// says so and leaves; who waits for it runs out in turn.
constexpr int kWaitPolls = 32768;
// It says so in the workspace and, since a call's workspace may be gone before
// anybody asks (scratch of one call, or of a graph), in a word of the device's own.
__device__ unsigned int device_word;
__device__ __noinline__ void give_up(unsigned int* status) {
  if (status) atomicOr(status, kStatusTimeoutBit);
  atomicOr(&device_word, kStatusTimeoutBit);
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, unsigned int* status,
                                         int polls = kWaitPolls) {
#pragma unroll 1
  while (!mbar_try_wait_suspend(bar, parity)) {
    if (--polls == 0) {
      give_up(status);
      return false;
    }
  }
  return true;
}

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
  const float x = prefix_product(w == 0 ? a[0] : w == 1 ? a[1] : w == 2 ? a[2] : a[3]);
  // blocks before this one, as one product per lane
  return x * warp_product((w > 0 ? a[0] : 1.f) * (w > 1 ? a[1] : 1.f) * (w > 2 ? a[2] : 1.f));
}
__device__ __forceinline__ float decay_out(const float (&a)[4], int w) {
  const float x = suffix_product(w == 0 ? a[0] : w == 1 ? a[1] : w == 2 ? a[2] : a[3]);
  return x * warp_product((w < 1 ? a[1] : 1.f) * (w < 2 ? a[2] : 1.f) * (w < 3 ? a[3] : 1.f));
}
// The same c_j from a chunk's shared decays.
__device__ __forceinline__ float decay_to_end(const float* d, int w, int lane) {
  float x = d[4 + 32 * w + lane];
  if (w < 3) x *= d[3];
  if (w < 2) x *= d[2];
  if (w < 1) x *= d[1];
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

// Two products in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// 32 bytes to global memory, past L1 and in one instruction where they are
// 32-byte aligned (whole sectors).  B4 H16 T4096 D128 forward: 64 to 68 us so, 78
// with room made in L1, 85 in 16-byte stores.
__device__ __forceinline__ void st_global32(void* dst, const uint32_t* r, bool wide) {
  if (!wide) {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    return;
  }
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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

// 16-byte pieces [c0, c1) of row `row` of a 64-column tile, scaled by f into the
// hi and lo tiles, in bf16 arithmetic: with f = f_hi + f_lo (bf16 each, 2^-17 left behind), hi = v f_hi
// rounded, v f_hi - hi fits bf16 exactly (a product of two 8-bit significands
// has 16 bits), and lo = that + v f_lo: three instructions for two values.
__device__ __forceinline__ void scale_row(const uint8_t* tile, uint8_t* hi, uint8_t* lo, int row, float f, int c0,
                                          int c1) {
  const uint32_t fh = pack2_bf16(f, f);
  const float rest = f - lo_half(fh);
  const uint32_t fl = pack2_bf16(rest, rest);
  constexpr uint32_t kNegZero = 0x80008000u;  // v f + (-0) = v f, its sign kept
#pragma unroll 1
  for (; c0 < c1; c0 += 2) {
    uint4 u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] = *reinterpret_cast<const uint4*>(tile + sw128_off(row, c0 + i));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      uint32_t h[4], l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(h[e]) : "r"(v[e]), "r"(fh), "r"(kNegZero));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(l[e]) : "r"(v[e]), "r"(fh), "r"(h[e] ^ 0x80008000u));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(l[e]) : "r"(v[e]), "r"(fl), "r"(l[e]));
      }
      *reinterpret_cast<uint4*>(hi + sw128_off(row, c0 + i)) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(lo + sw128_off(row, c0 + i)) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
}

// Where columns [col, col + 4) of row `row` of segment u's end state lie: four
// columns of all rows together, so that a warp's 32 rows are 512 bytes in a row
// (by rows, every lane a line of its own, a segment took 1 us to enter).
template <int DK>
__device__ __forceinline__ float4* segment_at(const GatedScan& p, size_t u, int col, int row) {
  return reinterpret_cast<float4*>(p.seg_end + u * DK * p.Dv) + (size_t)(col / 4) * DK + row;
}
// NC columns of this thread's state row, entering segment g: the caller's
// state and the segments passed before it in the scan's direction.
template <int DK, int NC>
__device__ __forceinline__ void enter_state(const GatedScan& p, bool rev, size_t bh, int g, int j0, int row,
                                            float (&s)[NC]) {
  const float* src = p.S_in ? p.S_in + bh * p.S_in_stride + (size_t)row * p.Dv + j0 : nullptr;
#pragma unroll
  for (int j = 0; j < NC; j += 4) {
    const float4 v = src ? *reinterpret_cast<const float4*>(src + j) : make_float4(0.f, 0.f, 0.f, 0.f);
    s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
  }
  const int n = rev ? p.G - 1 - g : g;
#pragma unroll 2
  for (int i = 0; i < n; ++i) {
    const size_t u = bh * p.G + (rev ? p.G - 1 - i : i);
    const float gam = __ldg(p.seg_decay + u);
    const float4* e = segment_at<DK>(p, u, j0, row);
#pragma unroll
    for (int j = 0; j < NC; j += 4) {
      const float4 v = __ldg(e + (size_t)(j / 4) * DK);
      s[j] = fmaf(gam, s[j], v.x);
      s[j + 1] = fmaf(gam, s[j + 1], v.y);
      s[j + 2] = fmaf(gam, s[j + 2], v.z);
      s[j + 3] = fmaf(gam, s[j + 3], v.w);
    }
  }
}
template <int NC>
__device__ __forceinline__ void leave_state(float* dst, const float (&s)[NC]) {
#pragma unroll
  for (int j = 0; j < NC; j += 4)
    *reinterpret_cast<float4*>(dst + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
}

// s <- gamma s + this lane's increment (its hi and lo halves at taddr, + 64)
template <bool GATED, int NC>
__device__ __forceinline__ void add_increment(float (&s)[NC], float gamma, uint32_t taddr) {
#pragma unroll
  for (int h = 0; h < NC / 16; ++h) {
    uint32_t x[16], y[16];
    tmem_ld16(taddr + 16 * h, x);
    if (GATED) tmem_ld16(taddr + 64 + 16 * h, y);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      s[16 * h + e] = GATED ? fmaf(gamma, s[16 * h + e], __uint_as_float(x[e]) + __uint_as_float(y[e]))
                            : s[16 * h + e] + __uint_as_float(x[e]);
  }
}

// ------------------------------------------------------------- main kernel --
template <int DK, bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    gated_out_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, __nv_bfloat16* o_all, const GatedScan p) {
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
  const float* alpha = GATED ? p.alpha + (size_t)bh * T : nullptr;

  if (tid == 0) {
    for (uint32_t i = 0; i < 2; ++i) {
      for (uint32_t b : {B_FULLK, B_FULLQ, B_SC, B_DS, B_QS, B_PV}) mbar_init(bar + b + 8 * i, 1);
      for (uint32_t b : {B_DSFREE, B_S, B_OFREE}) mbar_init(bar + b + 8 * i, 4);  // one arrival per warp
      for (uint32_t b : {B_P, B_VT}) mbar_init(bar + b + 8 * i, 8);
    }
    for (uint32_t i = 0; i < 3; ++i) {
      mbar_init(bar + B_FULLV + 8 * i, 1);
      mbar_init(bar + B_VFREE + 8 * i, 1);
      mbar_init(bar + B_DECAY + 8 * i, 1);
    }
    mbar_init(bar + B_FIN, 1);
    mbar_init(bar + B_FIN + 8, 1);
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
  unsigned int* const wc = p.status;
  const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
  auto done = [&](uint32_t b, int c) { return wait_bar(bar + b + 8 * (c & 1), (c >> 1) & 1, wc); };
  auto full_v = [&](int c) { return wait_bar(bar + B_FULLV + 8 * (c % 3), (c / 3) & 1, wc); };
  auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
  // chunk c's decays: block products, then the rows'.  They take the place of
  // chunk c-3's once the increment (c-2) and P (c-2) are there and all who read
  // those are done: the scaling warps before P (c-2); the state's, which added
  // the increment (c-3) before the increment (c-2) could run; the outputs', which
  // read them before they drained O (c-4), which Q S (c-3) waited for and the
  // increment (c-2) follows.  At c = 3 there is no O before: it takes a wait for
  // O (0), which they drain after they have read the decays of chunks 0 and 1.
  // (Waiting for O (c-3) at every c: 67.7 us for 66.6 at B4 H16 T4096 D128.)
  auto decays = [&](int c) { return reinterpret_cast<float*>(sm + L::SUF_OFF + (c % 3) * kDecayBytes); };
  auto have_decays = [&](int c) {
    return !GATED || wait_bar(bar + B_DECAY + 8 * (c % 3), (c / 3) & 1, wc);
  };
  auto arrive = [&](uint32_t b, int c) {  // one arrival for the warp, after all its lanes
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + b + 8 * (c & 1));
  };

  // The state that a later segment is entered with: sixteen warps take as many
  // columns of it each and pass them to the state's warps in V~'s place, which
  // the scaling warps leave alone until then.  (The state's four warps alone
  // took 1.2 us for every segment before theirs.)
  const bool joined = g > 0;
  auto passed = [&](int col, int row) {
    return reinterpret_cast<float4*>(sm + L::VT_OFF) + (size_t)(col / 4) * DK + row;
  };
  if (joined && warp >= kWarpP) {
    const int row = 32 * w + lane, col = 16 * ((warp - kWarpP) >> 2);
    if (row < DK) {
      float s[16];
      enter_state<DK>(p, false, bh, g, j0 + col, row, s);
#pragma unroll
      for (int j = 0; j < 16; j += 4) *passed(col + j, row) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
    }
    named_bar_sync(kBarS, 512);
  }

  if (warp == kWarpTma) {
    // ------------------------------------------------------------------ TMA --
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      int nk = 0, nq = 0, nv = 0;  // issued
      for (int c = 0; c < n; ++c) {
        const int s = c & 1, row = (first + c) * C;
        // P V (c-3) has read the stage (and so has K^T V or V~: K (c-1) waited for the increment)
        if (c >= 3 && !wait_bar(bar + B_VFREE + 8 * (c % 3), (c / 3 - 1) & 1, wc)) break;
        mbar_expect_tx(bar + B_FULLV + 8 * (c % 3), kBlk);
        tma_load_3d(sb + L::V_OFF + (c % 3) * kBlk, &tmV, bar + B_FULLV + 8 * (c % 3), j0, row, bh);
        nv = c + 1;
        if (c >= 2 && !(done(B_DS, c - 2) && done(B_SC, c - 2))) break;
        mbar_expect_tx(bar + B_FULLK + 8 * s, KB * kBlk);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          tma_load_3d(sb + L::K_OFF + (s * KB + kb) * kBlk, &tmK, bar + B_FULLK + 8 * s, kb * 64, row, bh);
        nk = c + 1;
        if (c >= 2 && !done(B_QS, c - 2)) break;
        mbar_expect_tx(bar + B_FULLQ + 8 * s, KB * kBlk);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          tma_load_3d(sb + L::Q_OFF + (s * KB + kb) * kBlk, &tmQ, bar + B_FULLQ + 8 * s, kb * 64, row, bh);
        nq = c + 1;
      }
      // never leave with copies in flight
      for (int c = nk > 2 ? nk - 2 : 0; c < nk; ++c) (void)wait_bar(bar + B_FULLK + 8 * (c & 1), (c >> 1) & 1, wc);
      for (int c = nq > 2 ? nq - 2 : 0; c < nq; ++c) (void)wait_bar(bar + B_FULLQ + 8 * (c & 1), (c >> 1) & 1, wc);
      for (int c = nv > 3 ? nv - 3 : 0; c < nv; ++c) (void)wait_bar(bar + B_FULLV + 8 * (c % 3), (c / 3) & 1, wc);
    }
  } else if (warp == kWarpMma || warp == kWarpMma2) {
    // ------------------------------------------------------------------ MMA --
    auto scores = [&](int c) {
      constexpr uint32_t id = idesc_bf16(128, 128, false, false);
      const uint32_t s = (c & 1) * KB * kBlk;
      const uint64_t dq = desc_k(sb + L::Q_OFF + s), dk = desc_k(sb + L::K_OFF + s);
#pragma unroll 2
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
      const uint64_t db = desc_mn(sb + (GATED ? L::VT_OFF : L::V_OFF + (c % 3) * kBlk), kBlk);
#pragma unroll 2
      for (int ks = 0; ks < C / 16; ++ks)
        mma_bf16_ss_elect(tmem + TM_DS, desc_step(da, ks * 2048), desc_step(db, ks * 2048), id, ks > 0);
      mma_commit_elect(bar + B_DS + 8 * (c & 1));
    };
    auto read_state = [&](int c) {
      constexpr uint32_t id = idesc_bf16(128, 64, false, true);
      const uint64_t dq = desc_k(sb + L::Q_OFF + (c & 1) * KB * kBlk), ds = desc_mn(sb + L::S_OFF, kBlk);
#pragma unroll 2
      for (int ks = 0; ks < DK / 16; ++ks)
        mma_bf16_ss_elect(tmem + TM_QS, desc_step(dq, (ks >> 2) * kBlk + (ks & 3) * 32), desc_step(ds, ks * 2048), id,
                          ks > 0);
      mma_commit_elect(bar + B_QS + 8 * (c & 1));
    };
    auto inner = [&](int c) {
      constexpr uint32_t id = idesc_bf16(128, 64, false, true);
      const uint64_t dv = desc_mn(sb + L::V_OFF + (c % 3) * kBlk, kBlk);
#pragma unroll 2
      for (int ks = 0; ks < C / 16; ++ks)
        mma_bf16_ts_elect(tmem + TM_PV, tmem + TM_SC + 128 * (c & 1) + 64 * (ks >> 2) + 8 * (ks & 3),
                          desc_step(dv, ks * 2048), id, ks > 0);
      mma_commit_elect(bar + B_PV + 8 * (c & 1));
      mma_commit_elect(bar + B_VFREE + 8 * (c % 3));
    };
    bool ok = true;
    if (warp == kWarpMma) {
      for (int c = 0; c <= n && ok; ++c) {
        if (c < n) {
          // P V (c-2) has read the P that these scores overwrite
          ok = all(done(B_FULLK, c) && done(B_FULLQ, c) && (c < 2 || done(B_PV, c - 2)));
          if (!ok) break;
          tc_fence_after();
          scores(c);
        }
        if (c >= 1) {
          ok = all(done(B_P, c - 1) && full_v(c - 1) && (c < 2 || done(B_OFREE, c - 2)));
          if (!ok) break;
          tc_fence_after();
          inner(c - 1);
        }
      }
    } else {
      for (int c = 0; c < n && ok; ++c) {
        ok = all(done(B_FULLK, c) && (GATED ? done(B_VT, c) : full_v(c)) && (c < 1 || done(B_DSFREE, c - 1)));
        if (!ok) break;
        tc_fence_after();
        increment(c);
        ok = all(done(B_FULLQ, c) && done(B_S, c) && (c < 1 || done(B_OFREE, c - 1)));
        if (!ok) break;
        tc_fence_after();
        read_state(c);
      }
    }
    tc_fence_after();  // no MMA may outlive TMEM
    const uint32_t fin_bar = bar + B_FIN + (warp == kWarpMma ? 0 : 8);
    mma_commit_elect(fin_bar);
    (void)wait_bar(fin_bar, 0, wc);
  } else if (warp == kWarpDecay) {
    // -------------------------------------------------------------- decays --
    bool ok = true;
    for (int c = 0; GATED && c < n && ok; ++c) {
      ok = c < 2 || all(done(B_DS, c - 2) && done(B_P, c - 2) && (c != 3 || done(B_OFREE, 0)));
      if (!ok) break;
      float* d = decays(c);
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int t = (first + c) * C + 32 * k + lane;
        const float a = t < T ? __ldg(alpha + t) : 1.f, s = suffix_product(a);
        d[4 + 32 * k + lane] = s;
        if (lane == 0) d[k] = s * a;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + B_DECAY + 8 * (c % 3));
    }
  } else if (warp >= kWarpP && warp < kWarpP + 8) {
    // -------------------------------------------------------------- scores --
    const int half = (warp - kWarpP) >> 2, row = 32 * w + lane;
    float ahead = 1.f;
    auto load = [&](int c) {
      const int t = (first + c) * C + row;
      return GATED && c < n && t < T ? __ldg(alpha + t) : 1.f;
    };
    ahead = load(0);
    if (GATED && joined) named_bar_sync(kBarJoin, 384);
    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      const float a = ahead, pre = GATED ? prefix_product(a) : 1.f;
      ahead = load(c + 1);
      const float* bl = decays(c);
      const float* sf = bl + 4;
      if (GATED) {  // the increment (c-1) has read V~ (c-1)
        ok = all(have_decays(c) && full_v(c) && (c < 1 || done(B_DS, c - 1)));
        if (!ok) break;
        scale_row(sm + L::V_OFF + (c % 3) * kBlk, sm + L::VT_OFF, sm + L::VT_OFF + kBlk, row, decay_to_end(bl, w, lane),
                  4 * half, 4 * half + 4);
        fence_proxy_async_smem();
        arrive(B_VT, c);
      }
      ok = all(done(B_SC, c));
      if (!ok) break;
      tc_fence_after();
      const uint32_t sc = lanes + TM_SC + 128 * (c & 1);
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const int cb = 2 * half + b;
        uint32_t d[16];
        if (cb > w) {
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i] = 0;
        } else {
          uint32_t x[32];
          float2 f[16];
          tmem_ld32(sc + 32 * cb, x);
          if (GATED && cb < w) {
            float mid = pre;
            if (cb + 1 < w) mid *= bl[w - 1];
            if (cb + 2 < w) mid *= bl[w - 2];
            const float2 m2 = make_float2(mid, mid);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float4 u = *reinterpret_cast<const float4*>(sf + 32 * cb + 2 * j);
              f[j] = mul2(make_float2(u.x, u.y), m2);
              f[j + 1] = mul2(make_float2(u.z, u.w), m2);
            }
          } else if (GATED) {  // the products of alpha over (column, row], zero right of the diagonal
            float run = lane == 31 ? 1.f : 0.f;
            f[15].y = run;
#pragma unroll
            for (int j = 30; j >= 0; --j) {
              const float t = __shfl_sync(0xffffffffu, a, j + 1);
              run = j == lane ? 1.f : run * t;
              if (j & 1) f[j / 2].y = run;
              else f[j / 2].x = run;
            }
          }
          tmem_wait_ld();
          if (!GATED && cb == w) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j > lane) x[j] = 0;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 v = make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
            if (GATED) v = mul2(v, f[j]);
            d[j] = pack2_bf16(v.x, v.y);
          }
        }
        tmem_st16(sc + 64 * half + 16 * b, d);  // over what this warp has read
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
    if (joined && live) {
#pragma unroll
      for (int j = 0; j < NV; j += 4) {
        const float4 v = *passed(j, row);
        s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
      }
    } else if (live && p.S_in) {
      const float* src = p.S_in + bh * p.S_in_stride + (size_t)row * p.Dv + j0;
#pragma unroll
      for (int j = 0; j < NV; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(src + j);
        s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
      }
    }
    if (GATED && joined) named_bar_sync(kBarJoin, 384);
    auto put = [&]() {
      if (live) {
#pragma unroll
        for (int c16 = 0; c16 < 8; ++c16) st_bf16x8(sm + L::S_OFF + sw128_off(row, c16), s + 8 * c16);
      }
      fence_proxy_async_smem();
    };
    put();
    arrive(B_S, 0);
    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      ok = all(have_decays(c) && done(B_DS, c));
      if (!ok) break;
      tc_fence_after();
      const float* d = decays(c);
      add_increment<GATED>(s, GATED ? d[0] * d[1] * d[2] * d[3] : 1.f, lanes + TM_DS);
      tc_fence_before();
      arrive(B_DSFREE, c);
      if (c + 1 < n) {
        ok = all(done(B_QS, c));  // Q S (c) has read the tile
        if (!ok) break;
        put();
        arrive(B_S, c + 1);
      }
    }
    if (ok && live && p.S_out && g == p.G - 1)
      leave_state(p.S_out + (size_t)bh * DK * p.Dv + (size_t)row * p.Dv + j0, s);
  } else if (warp >= kWarpO) {
    // ------------------------------------------------------------- outputs --
    const int row = 32 * w + lane;
    __nv_bfloat16* o_row = o_all + (size_t)bh * T * p.Dv + j0;
    const bool wide = (reinterpret_cast<uintptr_t>(o_all) & 31) == 0;  // rows are multiples of 128 bytes
    auto load = [&](int c) {
      const int t = (first + c) * C + row;
      return GATED && c < n && t < T ? __ldg(alpha + t) : 1.f;
    };
    float ahead = load(0), into = 1.f;
    bool ok = true;
    for (int c = 0; c <= n && ok; ++c) {
      const float into_before = into;
      if (GATED && c < n) {
        into = prefix_product(ahead);
        ahead = load(c + 1);
        ok = all(have_decays(c));
        if (!ok) break;
        const float* d = decays(c);
        if (w > 0) into *= d[0];
        if (w > 1) into *= d[1];
        if (w > 2) into *= d[2];
      }
      if (c >= 1) {
        ok = all(done(B_QS, c - 1) && done(B_PV, c - 1));
        if (!ok) break;
        tc_fence_after();
        const int t = (first + c - 1) * C + row;
        __nv_bfloat16* dst = o_row + (size_t)t * p.Dv;
#pragma unroll 1
        for (int h = 0; h < NV; h += 16) {
          uint32_t x[16], y[16], r[8];
          tmem_ld16(lanes + TM_QS + h, x);
          tmem_ld16(lanes + TM_PV + h, y);
          tmem_wait_ld();
          if (h + 16 == NV) {
            tc_fence_before();
            arrive(B_OFREE, c - 1);
          }
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            r[e / 2] = pack2_bf16(fmaf(into_before, __uint_as_float(x[e]), __uint_as_float(y[e])),
                                  fmaf(into_before, __uint_as_float(x[e + 1]), __uint_as_float(y[e + 1])));
          if (t < T) st_global32(dst + h, r, wide);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ state kernel --
// Forward (blockIdx.y = 0: x = k, z = v) and from the end (1: x = q, z = dO):
// the segments' end states from zero (STORE = false), or every chunk's entry
// state in the scan's direction as bf16 hi and lo, from the segment's true entry
// (STORE).  With the scaled Z twice, scaling a chunk runs beside the products of
// the one before; what is left is bound by what a chunk moves through shared
// memory (copies in and out, the scaled Z, the operands).  Both scans of B4 H16
// T4096 D128 with their 537 MB: 105 us (82 at a copy's rate; 2 x 48 as two
// launches of one scaled copy each, 110 as two CTAs of 64-token halves on an SM).
constexpr int kStateThreads = 20 * 32;  // TMA 0, MMA 1, state 4-11, scaling 12-19
template <int DK, bool GATED, bool STORE>
__global__ void __launch_bounds__(kStateThreads, 1)
    gated_state_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmR,
                       const __grid_constant__ GatedScan fwd, const __grid_constant__ GatedScan rvs) {
  using L = StateLayout<DK>;
  constexpr int KB = L::KB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = warp_uniform(smem_u32(sm));
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)warp_uniform((uint32_t)tid >> 5), w = warp & 3;
  const bool rev = blockIdx.y;
  const GatedScan& p = rev ? rvs : fwd;
  const int nsl = p.Dv / NV, T = p.T, segs = STORE ? p.G : p.G - 1;
  const int slice = blockIdx.x % nsl, bh = blockIdx.x / nsl / segs;
  // without STORE the scan's last segment is not needed
  const int g = (int)(blockIdx.x / nsl) % segs + (!STORE && rev ? 1 : 0);
  const int j0 = slice * NV, nch = (T + C - 1) / C;
  const int first = g * p.seg_chunks, n = min(p.seg_chunks, nch - first);
  auto chunk = [&](int i) { return rev ? first + n - 1 - i : first + i; };
  const uint32_t bar = sb + L::BAR_OFF;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::BAR_OFF + C_TMEM);
  const float* alpha = GATED ? p.alpha + (size_t)bh * T : nullptr;

  if (tid == 0) {
    for (uint32_t i = 0; i < 2; ++i) {
      for (uint32_t b : {C_FULL, C_FREE, C_DS}) mbar_init(bar + b + 8 * i, 1);
      mbar_init(bar + C_VT + 8 * i, 8);
      mbar_init(bar + C_DSFREE + 8 * i, 8);
    }
    mbar_init(bar + C_FIN, 1);
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
  auto done = [&](uint32_t b, int i) { return wait_bar(bar + b + 8 * (i & 1), (i >> 1) & 1, p.status); };
  auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };

  if (warp == kWarpTma) {
    if (lane == 0) {
      const CUtensorMap* mx = rev ? &tmQ : &tmK;
      const CUtensorMap* mz = rev ? &tmO : &tmV;
      prefetch_tmap(mx);
      prefetch_tmap(mz);
      int issued = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i & 1, row = chunk(i) * C;
        if (i >= 2 && !done(C_FREE, i - 2)) break;
        const uint32_t f = bar + C_FULL + 8 * s;
        mbar_expect_tx(f, (KB + 1) * kBlk);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          tma_load_3d(sb + L::X_OFF + (s * KB + kb) * kBlk, mx, f, kb * 64, row, bh);
        tma_load_3d(sb + L::Z_OFF + s * kBlk, mz, f, j0, row, bh);
        issued = i + 1;
      }
      // never leave with copies in flight
      for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i) (void)done(C_FULL, i);
    }
  } else if (warp == kWarpMma) {
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int s = i & 1;
      ok = all(done(GATED ? C_VT : C_FULL, i) && (i < 2 || done(C_DSFREE, i - 2)));
      if (!ok) break;
      tc_fence_after();
      constexpr uint32_t id = idesc_bf16(128, GATED ? 128 : 64, true, true);
      const uint64_t da = desc_mn(sb + L::X_OFF + s * KB * kBlk, kBlk);
      const uint64_t db = desc_mn(sb + (GATED ? L::VT_OFF + s * 2 * kBlk : L::Z_OFF + s * kBlk), kBlk);
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        mma_bf16_ss_elect(tmem + 128 * s, desc_step(da, ks * 2048), desc_step(db, ks * 2048), id, ks > 0);
      mma_commit_elect(bar + C_FREE + 8 * s);
      mma_commit_elect(bar + C_DS + 8 * s);
    }
    tc_fence_after();  // no MMA may outlive TMEM
    mma_commit_elect(bar + C_FIN);
    (void)wait_bar(bar + C_FIN, 0, p.status);
  } else if (warp >= 4 && warp < 12) {
    const int row = 32 * w + lane, half = (warp - 4) >> 2, jc = j0 + 32 * half;
    const bool live = row < DK, leader = warp == 4 && lane == 0;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16) + 32 * half;
    const size_t at = (size_t)row * p.Dv + jc, sblk = (size_t)DK * p.Dv;
    float s[NV / 2], total = 1.f;
#pragma unroll
    for (int j = 0; j < NV / 2; ++j) s[j] = 0.f;
    if (STORE && live) enter_state<DK>(p, rev, bh, g, jc, row, s);
    // The main kernel takes the caller's state from the slot that the last
    // segment leaves unused, so that it may write S_out over S0.
    if (!STORE && !rev && live && g == 0 && p.S_in) {
      const float4* src = reinterpret_cast<const float4*>(p.S_in + bh * p.S_in_stride + at);
      float4* dst = reinterpret_cast<float4*>(p.seg_end + ((size_t)bh * p.G + p.G - 1) * sblk + at);
#pragma unroll
      for (int j = 0; j < NV / 8; ++j) dst[j] = src[j];
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
        named_bar_sync(kBarS, 256);
        if (live) {
#pragma unroll
          for (int c16 = 0; c16 < 4; ++c16) {
            uint4 h, l;
            split8(s + 8 * c16, h, l);
            *reinterpret_cast<uint4*>(sm + L::ST_OFF + sw128_off(row, 4 * half + c16)) = h;
            *reinterpret_cast<uint4*>(sm + L::ST_OFF + DK * 128 + sw128_off(row, 4 * half + c16)) = l;
          }
        }
        fence_proxy_async_smem();
        named_bar_sync(kBarS, 256);
        if (leader) {
          const CUtensorMap* ms = rev ? &tmR : &tmS;
          const int to = (bh * nch + chunk(i)) * 2;
          tma_store_3d(ms, sb + L::ST_OFF, j0, 0, to);
          tma_store_3d(ms, sb + L::ST_OFF + DK * 128, j0, 0, to + 1);
          bulk_commit_group();
        }
      }
      // with STORE the eight warps meet at barriers, so they leave together
      ok = STORE ? named_bar_and(kBarS, 256, done(C_DS, i)) : all(done(C_DS, i));
      if (!ok) break;
      tc_fence_after();
      add_increment<GATED>(s, gamma, lanes + 128 * (i & 1));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + C_DSFREE + 8 * (i & 1));
    }
    if (leader) bulk_wait_group_all();
    if (ok && live) {
      if (STORE) {
        if (p.S_out && g == (rev ? 0 : p.G - 1)) leave_state(p.S_out + (size_t)bh * sblk + at, s);
      } else {
        float4* e = segment_at<DK>(p, (size_t)bh * p.G + g, jc, row);
#pragma unroll
        for (int j = 0; j < NV / 2; j += 4) e[(size_t)(j / 4) * DK] = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        if (leader && slice == 0) p.seg_decay[(size_t)bh * p.G + g] = total;
      }
    }
  } else if (GATED && warp >= 12) {
    const int row = 32 * w + lane, c16 = 4 * ((warp - 12) >> 2);
    float a[4];
    load_alpha(alpha, T, chunk(0), a);
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const float f = rev ? decay_into(a, w) : decay_out(a, w);
      if (i + 1 < n) load_alpha(alpha, T, chunk(i + 1), a);
      ok = all(done(C_FULL, i) && (i < 2 || done(C_FREE, i - 2)));  // the products have read the copy's place
      if (!ok) break;
      uint8_t* vt = sm + L::VT_OFF + (i & 1) * 2 * kBlk;
      scale_row(sm + L::Z_OFF + (i & 1) * kBlk, vt, vt + kBlk, row, f, c16, c16 + 4);
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

// --------------------------------------------------------- gradient kernel --
// Every chunk's gradient from its entry state S and the derivative R by the
// state it leaves (both as bf16 hi and lo):
//   A = tril(Q K^T) * D,  B = tril(dO V^T) * D
//   dV = A^T dO + diag(c) K R,  dK = B^T Q + diag(c) V R^T,  dQ = B K + diag(G) dO S^T
// and, where there is a gate, the derivative by log alpha_t: the sum of all
// paths from a write before t to a read at or after it,
//   sum_{i >= t > j} M_ij + sum_{i >= t} r_i + sum_{j < t} e_j + gamma <S, R>
//   M = (Q K^T) * (dO V^T) * D,  r_i = q_i . G_i (dO S^T)_i,  e_j = k_j . c_j (V R^T)_j
// (the first term: the suffix sum of row sums less column sums of M below its
// diagonal, both from the same float32 values).  Its sums do not leave the
// chunk, so no error travels along T; dO S^T and V R^T take hi and lo (16 bits)
// so that r and e hold to float32, the outputs themselves to one rounding of A or
// B.  Without a gate nothing needs more than the outputs, and S and R are read
// rounded once (hi alone), as K R is in either case.
//
// One CTA per SM walks over the (b, h, chunk)s.  Everything of a chunk is in
// shared memory at once except the states: R hi and S hi follow one another in a
// tile of their own, R lo comes to A's place before A is made, S lo to V's when V
// has been read.  dV is staged over A for its TMA store, dK over K, dQ over Q.
// The next chunk's tiles are loaded as their places fall free, while this one's
// last gradients are made and stored.  Every barrier completes once a chunk.
//   warp 0 TMA, warp 1 MMA, warps 4-11 epilogues (two warps to 32 rows, each
//   half of the columns), warps 12-19 <S, R> (R in registers) and the sums
//
// B4 H16 T4096 D128, the scans included: 251 us (floor 72: the inputs and
// gradients once).  A chunk's 352 KB in and out take 60% of it and the epilogues
// of A, B and M most of the rest; the two overlap by the loads ahead.  Gradients
// stored from registers took 275 us, the products with R first 268 to 282, heads
// in batches to keep the states in L2 277.
constexpr int kGradThreads = 20 * 32, kGradPlain = 12 * 32, kBarE = 1, kBarT = 2;
enum : uint32_t {  // mbarriers, 8 bytes each
  G_QK = 0, G_VO = 8, G_RH = 16, G_RL = 24, G_SH = 32, G_SL = 40,               // loaded
  G_SC = 48, G_XR = 56, G_DV = 64, G_DK = 72, G_DQ = 80,                        // products done
  G_P = 88, G_ACCFREE = 96, G_ENDFREE = 104, G_DOTS = 112,                      // epilogues' warps
  G_RHREAD = 120, G_RLREAD = 128, G_SREAD = 136,                                // <S, R>'s warps
  G_PAFREE = 144, G_KFREE = 152, G_QFREE = 160, G_FIN = 168, G_TMEM = 176       // stores have read
};
template <int DK, int DV>
struct GradLayout {
  static constexpr int KB = DK / 64, VB = DV / 64;
  static constexpr uint32_t SBLK = DK * 128, STATE = VB * SBLK;  // one 64-column block, a state tile
  static constexpr uint32_t Q_OFF = 0, K_OFF = Q_OFF + KB * kBlk, V_OFF = K_OFF + KB * kBlk, O_OFF = V_OFF + VB * kBlk;
  static constexpr uint32_t PA_OFF = O_OFF + VB * kBlk, PB_OFF = PA_OFF + 2 * kBlk, X_OFF = PB_OFF + 2 * kBlk;
  static constexpr uint32_t END = X_OFF + STATE;
  static constexpr uint32_t SUF_OFF = END;  // suf[128], block products [4]
  static constexpr uint32_t THR_OFF = SUF_OFF + 132 * 4;  // [2]: <S, R> of 8 warps, gamma
  static constexpr uint32_t BAR_OFF = (THR_OFF + 18 * 4 + 7) / 8 * 8;
  static constexpr uint32_t BYTES = BAR_OFF + 184;
  static constexpr uint32_t ALLOC = BYTES + 1024;
  // the rows' sums at the end, over B: F[2][128], e[2][128], column sums [4][128]
  static constexpr uint32_t FSUM = PB_OFF, ESUM = FSUM + 1024, CSUM = ESUM + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
  static_assert(STATE <= VB * kBlk && STATE <= 2 * kBlk, "the states' places");
  static_assert(END % 1024 == 0, "128-byte swizzle atoms stay aligned");
};
// TMEM: scores, then A^T dO, then B K | dO V^T, then B^T Q | V R^T | K R, then dO S^T
constexpr uint32_t TG_A = 0, TG_B = 128, TG_C = 256, TG_D = 384;

// Sums of 16 columns over the warp's rows: lane l < 16 ends with the sum of
// column fold16_col(l).
__device__ __forceinline__ float fold16(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1, n = 8; o < 16; o <<= 1, n >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float mine = up ? v[i + n] : v[i], theirs = up ? v[i] : v[i + n];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, o);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}
__device__ __forceinline__ int fold16_col(int l) {
  return (l & 1) * 8 + ((l >> 1) & 1) * 4 + ((l >> 2) & 1) * 2 + ((l >> 3) & 1);
}

// out = f * inter + intra for this thread's row and columns [c0, c0 + NC) into
// the staged tile; returns the dot product of f * inter with the same row of
// `with` (which may be the staged tile itself).
template <int NC, bool DOT>
__device__ __forceinline__ float grad_row(uint32_t inter, uint32_t intra, float f, const uint8_t* with, uint8_t* stage,
                                          int row, int c0) {
  float dot = 0.f;
#pragma unroll
  for (int c = 0; c < NC; c += 16) {
    uint32_t x[16], y[16];
    tmem_ld16(inter + c0 + c, x);
    tmem_ld16(intra + c0 + c, y);
    tmem_wait_ld();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = c0 + c + 8 * h;
      const uint32_t at = (uint32_t)(col >> 6) * kBlk + sw128_off(row, (col >> 3) & 7);
      float u[8], o[8];
      if (DOT) unpack_bf16x8(*reinterpret_cast<const uint4*>(with + at), u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = f * __uint_as_float(x[8 * h + e]);
        if (DOT) dot = fmaf(v, u[e], dot);
        o[e] = v + __uint_as_float(y[8 * h + e]);
      }
      st_bf16x8(stage + at, o);
    }
  }
  return dot;
}

template <int DK, int DV, bool GATED>
__global__ void __launch_bounds__(kGradThreads, 1)
    gated_grad_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                      const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmR,
                      const __grid_constant__ CUtensorMap tmDQ, const __grid_constant__ CUtensorMap tmDK,
                      const __grid_constant__ CUtensorMap tmDV, const float* alpha_all, float* dlog_alpha, int T,
                      int tasks, unsigned int* status) {
  using L = GradLayout<DK, DV>;
  constexpr int KB = L::KB, VB = L::VB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = warp_uniform(smem_u32(sm));
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)warp_uniform((uint32_t)tid >> 5), w = warp & 3;
  const int nch = (T + C - 1) / C;
  const uint32_t bar = sb + L::BAR_OFF;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::BAR_OFF + G_TMEM);
  float* suf = reinterpret_cast<float*>(sm + L::SUF_OFF);
  float* blk = suf + C;
  float* thr_all = reinterpret_cast<float*>(sm + L::THR_OFF);

  if (tid == 0) {
    for (uint32_t b = G_QK; b <= G_FIN; b += 8) {
      const bool warps = (b >= G_P && b <= G_SREAD);
      mbar_init(bar + b, warps ? 8 : 1);  // one arrival per warp
    }
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
  unsigned int* const wc = status;
  // a role's own chunk: its number among the CTA's, and its place
  int it = 0, bh = 0, t0 = 0, task = blockIdx.x;
  auto begin = [&]() {
    if (task >= tasks) return false;
    bh = task / nch;
    t0 = (task - bh * nch) * C;
    return true;
  };
  auto next = [&]() {
    task += gridDim.x;
    ++it;
  };
  auto wait = [&](uint32_t b) { return wait_bar(bar + b, it & 1, wc); };
  auto wait_before = [&](uint32_t b) { return it == 0 || wait_bar(bar + b, (it - 1) & 1, wc); };
  auto wait_all = [&](uint32_t b) { return __all_sync(0xffffffffu, wait(b)) != 0; };
  auto arrive = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + b);
  };

  if (warp == kWarpTma) {
    if (lane == 0) {
      uint32_t got[6];
      int n = 0, at = 0;
      auto expect = [&](uint32_t b, uint32_t bytes) {
        mbar_expect_tx(bar + b, bytes);
        got[n++] = b;
      };
      auto state = [&](uint32_t b, const CUtensorMap* m, uint32_t to, int z) {
        expect(b, L::STATE);
#pragma unroll
        for (int i = 0; i < VB; ++i) tma_load_3d(sb + to + i * L::SBLK, m, bar + b, 64 * i, 0, z);
      };
      auto rows = [&](uint32_t b, const CUtensorMap* m, uint32_t to, int blocks) {
        for (int i = 0; i < blocks; ++i) tma_load_3d(sb + to + i * kBlk, m, bar + b, 64 * i, t0, bh);
      };
      bool ok = true;
      for (; ok && begin(); next()) {
        at = 2 * task;
        // the chunk before has come to its end with dO, V, X (its loads have landed, too) ...
        ok = wait_before(G_DQ) && (!GATED || wait_before(G_SREAD));
        if (!ok) break;
        n = 0;
        expect(G_VO, 2 * VB * kBlk);
        rows(G_VO, &tmO, L::O_OFF, VB);
        rows(G_VO, &tmV, L::V_OFF, VB);
        state(G_RH, &tmR, L::X_OFF, at);
        if (GATED) {  // ... with A's place, and its stores with K and Q
          ok = wait_before(G_PAFREE);
          if (!ok) break;
          state(G_RL, &tmR, L::PA_OFF, at + 1);
        }
        ok = wait_before(G_KFREE) && wait_before(G_QFREE);
        if (!ok) break;
        expect(G_QK, 2 * KB * kBlk);
        rows(G_QK, &tmK, L::K_OFF, KB);
        rows(G_QK, &tmQ, L::Q_OFF, KB);
        ok = wait(G_XR);  // the products with R (and V) have run
        if (!ok) break;
        if (GATED) state(G_SL, &tmS, L::V_OFF, at + 1);
        ok = !GATED || wait(G_RHREAD);
        if (!ok) break;
        state(G_SH, &tmS, L::X_OFF, at);
        // The SMs run through their chunks at one pace, so their loads and stores
        // come in bursts with nothing in between: the next chunk's tiles go to L2
        // while the epilogues work on this one.
        const int ahead = task + (int)gridDim.x;
        if (ahead < tasks) {
          const int nbh = ahead / nch, nt0 = (ahead - nbh * nch) * C;
#pragma unroll 1
          for (int i = 0; i < VB; ++i) {
            prefetch_l2_3d(&tmO, 64 * i, nt0, nbh);
            prefetch_l2_3d(&tmV, 64 * i, nt0, nbh);
            for (int lo = 0; lo < (GATED ? 2 : 1); ++lo) {
              prefetch_l2_3d(&tmR, 64 * i, 0, 2 * ahead + lo);
              prefetch_l2_3d(&tmS, 64 * i, 0, 2 * ahead + lo);
            }
          }
#pragma unroll 1
          for (int i = 0; i < KB; ++i) {
            prefetch_l2_3d(&tmK, 64 * i, nt0, nbh);
            prefetch_l2_3d(&tmQ, 64 * i, nt0, nbh);
          }
        }
      }
      // never leave with copies in flight: those of the last chunk
      if (ok && it > 0) --it;
      for (int i = 0; i < n; ++i) (void)wait(got[i]);
    }
  } else if (warp == kWarpMma) {
    // A: K-major tile of 64-column blocks `ab` apart; B: K-major blocks `bb` apart
    auto kk = [&](uint32_t d, uint32_t a, uint32_t ab, uint32_t b, uint32_t bb, int depth, int N, uint32_t acc) {
      const uint32_t id = idesc_bf16(128, N, false, false);
      const uint64_t da = desc_k(sb + a), db = desc_k(sb + b);
#pragma unroll
      for (int ks = 0; ks < depth / 16; ++ks)
        mma_bf16_ss_elect(tmem + d, desc_step(da, (ks >> 2) * ab + (ks & 3) * 32),
                          desc_step(db, (ks >> 2) * bb + (ks & 3) * 32), id, acc | (uint32_t)(ks > 0));
    };
    // A: K-major; B: MN-major tile (rows are the depth), blocks `bb` apart
    auto kn = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t bb, int depth, int N) {
      const uint32_t id = idesc_bf16(128, N, false, true);
      const uint64_t da = desc_k(sb + a), db = desc_mn(sb + b, bb);
#pragma unroll
      for (int ks = 0; ks < depth / 16; ++ks)
        mma_bf16_ss_elect(tmem + d, desc_step(da, (ks >> 2) * kBlk + (ks & 3) * 32), desc_step(db, ks * 2048), id,
                          ks > 0);
    };
    // A: MN-major (the transposed P tile); B: MN-major
    auto nn = [&](uint32_t d, uint32_t a, uint32_t b, int N) {
      const uint32_t id = idesc_bf16(128, N, true, true);
      const uint64_t da = desc_mn(sb + a, kBlk), db = desc_mn(sb + b, kBlk);
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        mma_bf16_ss_elect(tmem + d, desc_step(da, ks * 2048), desc_step(db, ks * 2048), id, ks > 0);
    };
    bool ok = true;
    for (; ok && begin(); next()) {
      // the epilogues of the chunk before have read the accumulators
      ok = __all_sync(0xffffffffu, wait_before(G_ENDFREE)) && wait_all(G_VO) && wait_all(G_RH);
      if (!ok) break;
      tc_fence_after();
      kk(TG_C, L::V_OFF, kBlk, L::X_OFF, L::SBLK, DV, DK, 0);  // V R^T, hi
      if (GATED) {
        ok = wait_all(G_RL);
        if (!ok) break;
        tc_fence_after();
        kk(TG_C, L::V_OFF, kBlk, L::PA_OFF, L::SBLK, DV, DK, 1);  // V R^T, lo
      }
      ok = wait_all(G_QK);
      if (!ok) break;
      tc_fence_after();
      kk(TG_A, L::Q_OFF, kBlk, L::K_OFF, kBlk, DK, 128, 0);  // Q K^T
      kk(TG_B, L::O_OFF, kBlk, L::V_OFF, kBlk, DV, 128, 0);  // dO V^T
      mma_commit_elect(bar + G_SC);
      kn(TG_D, L::K_OFF, L::X_OFF, L::SBLK, DK, DV);  // K R
      mma_commit_elect(bar + G_XR);
      ok = wait_all(G_P);
      if (!ok) break;
      tc_fence_after();
      nn(TG_A, L::PA_OFF, L::O_OFF, DV);  // A^T dO
      mma_commit_elect(bar + G_DV);
      nn(TG_B, L::PB_OFF, L::Q_OFF, DK);  // B^T Q
      ok = wait_all(G_ACCFREE);           // dV's parts have been read
      if (!ok) break;
      tc_fence_after();
      kn(TG_A, L::PB_OFF, L::K_OFF, kBlk, C, DK);  // B K
      mma_commit_elect(bar + G_DK);                // with it, K and Q are free to be staged over
      ok = wait_all(G_SH);
      if (!ok) break;
      tc_fence_after();
      kk(TG_D, L::O_OFF, kBlk, L::X_OFF, L::SBLK, DV, DK, 0);  // dO S^T, hi
      if (GATED) {
        ok = wait_all(G_SL);
        if (!ok) break;
        tc_fence_after();
        kk(TG_D, L::O_OFF, kBlk, L::V_OFF, L::SBLK, DV, DK, 1);  // dO S^T, lo
      }
      mma_commit_elect(bar + G_DQ);
    }
    tc_fence_after();  // no MMA may outlive TMEM
    mma_commit_elect(bar + G_FIN);
    (void)wait_bar(bar + G_FIN, 0, wc);
  } else if (warp >= 4 && warp < 12) {
    // ----------------------------------------------------------- epilogues --
    const int row = 32 * w + lane, half = (warp - 4) >> 2;
    const bool leader = warp == 4 && lane == 0;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
    // the eight warps meet at every staged tile, so they leave together
    auto store = [&](const CUtensorMap* m, uint32_t from, int blocks) {
      fence_proxy_async_smem();
      named_bar_sync(kBarE, 256);
      if (leader) {
        for (int i = 0; i < blocks; ++i) tma_store_3d(m, sb + from + i * kBlk, 64 * i, t0, bh);
        bulk_commit_group();
      }
      __syncwarp();
    };
    bool ok = true;
    for (; ok && begin(); next()) {
      float a = 1.f, pre = 1.f, into = 1.f, out = 1.f;
      if (GATED) {
        float al[4];
        load_alpha(alpha_all + (size_t)bh * T, T, t0 / C, al);
        into = decay_into(al, w);
        out = decay_out(al, w);
        a = w == 0 ? al[0] : w == 1 ? al[1] : w == 2 ? al[2] : al[3];
        pre = prefix_product(a);
        if (half == 0) {
          suf[row] = suffix_product(a);
          if (lane == 31) blk[w] = pre;
          const float gamma = decay_chunk(al);
          if (leader) thr_all[9 * (it & 1) + 8] = gamma;
        }
      }
      // ---- A, B and M's sums ----
      float fsum = 0.f, esum = 0.f, csum[4] = {0.f, 0.f, 0.f, 0.f};
      ok = named_bar_and(kBarE, 256, wait(G_SC));
      if (ok) {
        tc_fence_after();
        float run = 0.f;
        bool room = false;  // A's place is free of R lo
#pragma unroll 1
        for (int pc = 3; pc >= 0; --pc) {  // 16 columns at a time, the right ones first
          const int c0 = 64 * half + 16 * pc, cb = c0 >> 5;
          uint32_t pa[8], pb[8];
          if (cb <= w) {
            uint32_t x[16], y[16];
            float m[16];
            tmem_ld16(lanes + TG_A + c0, x);
            tmem_ld16(lanes + TG_B + c0, y);
            if (GATED && cb < w) {
              float mid = pre;
              if (cb + 1 < w) mid *= blk[w - 1];
              if (cb + 2 < w) mid *= blk[w - 2];
#pragma unroll
              for (int j = 0; j < 16; ++j) m[j] = mid * suf[c0 + j];
            } else {  // the product of alpha over (column, row], zero right of the diagonal
              const int b0 = c0 & 31;
#pragma unroll
              for (int j = 15; j >= 0; --j) {
                if (GATED) {
                  const float t = __shfl_sync(0xffffffffu, a, b0 + j + 1);
                  run = b0 + j == lane ? 1.f : run * t;
                  m[j] = run;
                } else {
                  m[j] = cb < w || b0 + j <= lane ? 1.f : 0.f;
                }
              }
            }
            tmem_wait_ld();
            const int diag = cb == w ? lane - (c0 & 31) : -1;  // the diagonal's column of the piece
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float s0 = __uint_as_float(x[j]), s1 = __uint_as_float(x[j + 1]);
              const float b0 = __uint_as_float(y[j]) * m[j], b1 = __uint_as_float(y[j + 1]) * m[j + 1];
              pa[j / 2] = pack2_bf16(s0 * m[j], s1 * m[j + 1]);
              pb[j / 2] = pack2_bf16(b0, b1);
              m[j] = j == diag ? 0.f : s0 * b0;
              m[j + 1] = j + 1 == diag ? 0.f : s1 * b1;
              if (GATED) fsum += m[j] + m[j + 1];
            }
            if (GATED) {
              const float v = fold16(m);
              csum[0] = pc == 0 ? v : csum[0];
              csum[1] = pc == 1 ? v : csum[1];
              csum[2] = pc == 2 ? v : csum[2];
              csum[3] = pc == 3 ? v : csum[3];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) pa[i] = pb[i] = 0;
          }
          if (GATED && !room) room = wait(G_XR) && wait(G_RLREAD);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = (uint32_t)half * kBlk + sw128_off(row, 2 * pc + h);
            *reinterpret_cast<uint4*>(sm + L::PA_OFF + at) =
                make_uint4(pa[4 * h], pa[4 * h + 1], pa[4 * h + 2], pa[4 * h + 3]);
            *reinterpret_cast<uint4*>(sm + L::PB_OFF + at) =
                make_uint4(pb[4 * h], pb[4 * h + 1], pb[4 * h + 2], pb[4 * h + 3]);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        arrive(G_P);
      }
      ok = named_bar_and(kBarE, 256, ok && wait(G_DV));
      if (ok) {
        tc_fence_after();
        grad_row<DV / 2, false>(lanes + TG_D, lanes + TG_A, out, nullptr, sm + L::PA_OFF, row, half * (DV / 2));
        tc_fence_before();
        arrive(G_ACCFREE);
        store(&tmDV, L::PA_OFF, VB);
        ok = named_bar_and(kBarE, 256, wait(G_DK));
      }
      if (ok) {
        tc_fence_after();
        esum = grad_row<DK / 2, GATED>(lanes + TG_C, lanes + TG_B, out, sm + L::K_OFF, sm + L::K_OFF, row,
                                       half * (DK / 2));
        store(&tmDK, L::K_OFF, KB);
        if (leader) {
          bulk_wait_group_read<1>();
          mbar_arrive(bar + G_PAFREE);
        }
        __syncwarp();
        ok = named_bar_and(kBarE, 256, wait(G_DQ));
      }
      if (ok) {
        tc_fence_after();
        fsum += grad_row<DK / 2, GATED>(lanes + TG_D, lanes + TG_A, into, sm + L::Q_OFF, sm + L::Q_OFF, row,
                                        half * (DK / 2));
        tc_fence_before();
        arrive(G_ENDFREE);
        if (GATED) {  // B has been read: its place takes the sums
          reinterpret_cast<float*>(sm + L::FSUM)[half * C + row] = fsum;
          reinterpret_cast<float*>(sm + L::ESUM)[half * C + row] = esum;
          if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<float*>(sm + L::CSUM)[w * C + 64 * half + 16 * i + fold16_col(lane)] = csum[i];
          }
          arrive(G_DOTS);
        }
        store(&tmDQ, L::Q_OFF, KB);
        if (leader) {
          bulk_wait_group_read<1>();
          mbar_arrive(bar + G_KFREE);
          bulk_wait_group_read<0>();
          mbar_arrive(bar + G_QFREE);
        }
        __syncwarp();
      }
    }
    if (leader) bulk_wait_group_all();
  } else if (GATED && warp >= 12) {
    // ------------------------------------------------- <S, R> and the sums --
    constexpr int NP = (int)(L::STATE / 16 / 256);  // 16-byte pieces of a state tile to a thread
    const int i0 = tid - 12 * 32;
    float r[NP][8];
    auto piece = [&](uint32_t tile, int i, float (&x)[8]) {
      unpack_bf16x8(*reinterpret_cast<const uint4*>(sm + tile + 16 * (i0 + 256 * i)), x);
    };
    bool ok = true;
    for (; ok && begin(); next()) {
      float* thr = thr_all + 9 * (it & 1);
      const float* alpha = alpha_all + (size_t)bh * T;
      float dot = 0.f;
      ok = wait_all(G_RH);
      if (ok) {
#pragma unroll
        for (int i = 0; i < NP; ++i) piece(L::X_OFF, i, r[i]);
        arrive(G_RHREAD);
        ok = wait_all(G_RL);
      }
      if (ok) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          float x[8];
          piece(L::PA_OFF, i, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) r[i][e] += x[e];
        }
        arrive(G_RLREAD);
      }
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        ok = ok && wait_all(part ? G_SL : G_SH);
        if (ok) {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            float x[8];
            piece(part ? L::V_OFF : L::X_OFF, i, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = fmaf(x[e], r[i][e], dot);
          }
        }
      }
      if (ok) arrive(G_SREAD);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (lane == 0) thr[warp - 12] = dot;
      ok = named_bar_and(kBarT, 256, ok && wait(G_DOTS));
      if (ok && dlog_alpha && warp == 12) {  // four tokens to a lane
        float sr = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sr += thr[i];
        sr *= thr[8];
        const float* F = reinterpret_cast<const float*>(sm + L::FSUM);
        const float* E = reinterpret_cast<const float*>(sm + L::ESUM);
        const float* S = reinterpret_cast<const float*>(sm + L::CSUM);
        float f[4], e[4];
#pragma unroll
        for (int k = 3; k >= 0; --k) {  // suffix sums of the lane's own tokens
          const int t = 4 * lane + k;
          f[k] = F[t] + F[C + t] - (S[t] + S[C + t] + S[2 * C + t] + S[3 * C + t]) + (k < 3 ? f[k + 1] : 0.f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = E[4 * lane + k] + E[C + 4 * lane + k] + (k > 0 ? e[k - 1] : 0.f);
        float suff = f[0], pref = e[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x = __shfl_down_sync(0xffffffffu, suff, o), y = __shfl_up_sync(0xffffffffu, pref, o);
          if (lane + o < 32) suff += x;
          if (lane >= o) pref += y;
        }
        suff = __shfl_down_sync(0xffffffffu, suff, 1);  // tokens of later lanes
        pref = __shfl_up_sync(0xffffffffu, pref, 1);    // of earlier ones
        if (lane == 31) suff = 0.f;
        if (lane == 0) pref = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = t0 + 4 * lane + k;
          // no path crosses a wipe: its derivative is 0, not the sums' rounding
          if (t < T)
            dlog_alpha[(size_t)bh * T + t] =
                alpha[t] == 0.f ? 0.f : f[k] + suff + pref + (k > 0 ? e[k - 1] : 0.f) + sr;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// Nothing ever arrives on the barrier: the wait runs out after `polls` polls.
__global__ void wait_polls_selftest_kernel(unsigned int* status, int polls) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    fence_mbar_init();
    (void)wait_bar(smem_u32(&bar), 0, status, polls);
  }
}

template <int DK, bool GATED>
cudaError_t launch_out(const GatedProblem& p, const GatedScan& s, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  const int BH = p.B * p.H;
  if (!make_tmap_3d_bf16(&mq, p.q, DK, p.T, BH, C) || !make_tmap_3d_bf16(&mk, p.k, DK, p.T, BH, C) ||
      !make_tmap_3d_bf16(&mv, p.v, p.Dv, p.T, BH, C))
    return cudaErrorInvalidValue;
  auto kern = gated_out_kernel<DK, GATED>;
  constexpr int smem = (int)OutLayout<DK>::ALLOC;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((size_t)BH * s.G * (p.Dv / NV)), kThreads, smem, st>>>(
      mq, mk, mv, static_cast<__nv_bfloat16*>(p.o), s);
  return cudaGetLastError();
}

// The state kernel: the forward scan, and with `r` the one from the end too.
template <int DK, bool GATED, bool STORE>
cudaError_t launch_state(const GatedProblem& p, const GatedScan& f, const GatedScan* r, void* S, void* R,
                         cudaStream_t st) {
  CUtensorMap mk, mv, ms, mq, mo, mr;
  const int BH = p.B * p.H, nch = (p.T + C - 1) / C;
  if (!make_tmap_3d_bf16(&mk, p.k, DK, p.T, BH, C) || !make_tmap_3d_bf16(&mv, p.v, p.Dv, p.T, BH, C))
    return cudaErrorInvalidValue;
  mq = mk;
  mo = ms = mr = mv;
  if (r && (!make_tmap_3d_bf16(&mq, p.q, DK, p.T, BH, C) || !make_tmap_3d_bf16(&mo, p.dO, p.Dv, p.T, BH, C)))
    return cudaErrorInvalidValue;
  if (STORE && (!make_tmap_3d_bf16(&ms, S, p.Dv, DK, 2 * BH * nch, DK) ||
                !make_tmap_3d_bf16(&mr, R, p.Dv, DK, 2 * BH * nch, DK)))
    return cudaErrorInvalidValue;
  auto kern = gated_state_kernel<DK, GATED, STORE>;
  constexpr int smem = (int)StateLayout<DK>::ALLOC;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const size_t segs = STORE ? f.G : f.G - 1;
  kern<<<dim3((unsigned)(BH * segs * (p.Dv / NV)), r ? 2 : 1), GATED ? kStateThreads : 12 * 32, smem, st>>>(
      mk, mv, ms, mq, mo, mr, f, r ? *r : f);
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
  GatedScan s = gated_scan_of(p, p.scratch);
  const size_t sblk = (size_t)DK * p.Dv;
  s.S_in = p.S0;
  s.S_in_stride = sblk;
  s.S_out = p.S_out;
  if (s.G > 1) {
    cudaError_t e = launch_state<DK, GATED, false>(p, s, nullptr, nullptr, nullptr, st);
    if (e != cudaSuccess) return e;
    if (p.S0) {
      s.S_in = s.seg_end + (s.G - 1) * sblk;
      s.S_in_stride = s.G * sblk;
    }
  }
  return launch_out<DK, GATED>(p, s, st);
}

template <int DK, int DV, bool GATED>
cudaError_t launch_grad(const GatedProblem& p, const void* S, const void* R, cudaStream_t st) {
  const int BH = p.B * p.H, nch = (p.T + C - 1) / C;
  CUtensorMap mq, mk, mv, mo, ms, mr, mdq, mdk, mdv;
  if (!make_tmap_3d_bf16(&mq, p.q, DK, p.T, BH, C) || !make_tmap_3d_bf16(&mk, p.k, DK, p.T, BH, C) ||
      !make_tmap_3d_bf16(&mv, p.v, DV, p.T, BH, C) || !make_tmap_3d_bf16(&mo, p.dO, DV, p.T, BH, C) ||
      !make_tmap_3d_bf16(&ms, S, DV, DK, 2 * BH * nch, DK) || !make_tmap_3d_bf16(&mr, R, DV, DK, 2 * BH * nch, DK) ||
      !make_tmap_3d_bf16(&mdq, p.dq, DK, p.T, BH, C) || !make_tmap_3d_bf16(&mdk, p.dk, DK, p.T, BH, C) ||
      !make_tmap_3d_bf16(&mdv, p.dv, DV, p.T, BH, C))
    return cudaErrorInvalidValue;
  auto kern = gated_grad_kernel<DK, DV, GATED>;
  constexpr int smem = (int)GradLayout<DK, DV>::ALLOC;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int tasks = BH * nch;
  kern<<<p.sms > 0 && p.sms < tasks ? p.sms : tasks, GATED ? kGradThreads : kGradPlain, smem, st>>>(
      mq, mk, mv, mo, ms, mr, mdq, mdk, mdv, p.alpha, p.dlog_alpha, p.T, tasks, p.status);
  return cudaGetLastError();
}

// The workspace of the gradient: the segments' states of both scans, then S
// and R of every chunk as bf16 hi and lo.
template <int DK, bool GATED>
cudaError_t bwd(const GatedProblem& p, cudaStream_t st) {
  const int BH = p.B * p.H, nch = (p.T + C - 1) / C;
  const size_t seg = gated_segment_bytes(BH, p.G, DK, p.Dv), sblk = (size_t)DK * p.Dv;
  uint8_t* ws = static_cast<uint8_t*>(p.scratch);
  uint8_t* S = ws + 2 * seg;
  uint8_t* R = S + (size_t)BH * nch * 2 * sblk * 2;
  GatedScan f = gated_scan_of(p, ws), r = gated_scan_of(p, ws + seg);
  f.S_in = p.S0;
  r.S_in = p.dS_T;
  r.S_out = p.dS0;
  f.S_in_stride = r.S_in_stride = sblk;
  cudaError_t e = cudaSuccess;
  if (p.G > 1) {
    GatedScan ends = f;  // the caller's state stays where it is: nothing writes over it here
    ends.S_in = nullptr;
    e = launch_state<DK, GATED, false>(p, ends, &r, nullptr, nullptr, st);
  }
  if (e == cudaSuccess) e = launch_state<DK, GATED, true>(p, f, &r, S, R, st);
  if (e != cudaSuccess) return e;
  return p.Dv == 128 ? launch_grad<DK, 128, GATED>(p, S, R, st) : launch_grad<DK, 64, GATED>(p, S, R, st);
}

}  // namespace

size_t gated_bwd_bytes(int BH, int T, int G, int Dk, int Dv) {
  return 2 * gated_segment_bytes(BH, G, Dk, Dv) + (size_t)BH * ((T + C - 1) / C) * 2 * 2 * Dk * Dv * 2;
}

cudaError_t launch_gated_tc_bwd(const GatedProblem& p, cudaStream_t st) {
  if (p.alpha) return p.Dk == 128 ? bwd<128, true>(p, st) : bwd<64, true>(p, st);
  return p.Dk == 128 ? bwd<128, false>(p, st) : bwd<64, false>(p, st);
}

// Segments: as many as there are SMs for, no more than 3 sqrt(chunks) (each
// costs the later ones an entry), and none where the pass over their states
// costs more than it takes off the longest chain.  In us, measured with Dk = Dv
// = 128 for one head to 32 over 1024 to 65536 tokens: the forward 1.73 a chunk
// in one chain, or 2.7 a chunk of a segment + 0.25 a segment + 5; the
// gradient's scans 1.04, or 2.1 + 0.4 a segment + 3.  (B1 H1 T8192: forward in
// one chain 114, in 8 | 16 | 32 | 64 segments 35 | 27 | 26 | 31, gradient 84, in
// 8 | 16 | 32 | 64 41 | 36 | 39 | 51.  B1 H32: 2 segments at T8192 108 for 119,
// at T2048 38 for 37; the gradient of H16 T8192 in 2 segments 169 for 165.)
void gated_segments(int BH, int T, int Dv, int sms, int directions, int* G, int* seg_chunks) {
  const int nch = (T + C - 1) / C;
  const long long ctas = (long long)BH * (Dv / NV) * directions;
  *G = 1;
  *seg_chunks = nch;
  if (ctas < 1 || sms < 2 * ctas) return;
  long long g = sms / ctas;
  while (g * g > 9LL * nch) --g;
  if (g < 2) return;
  const long long per = (nch + g - 1) / g, n = (nch + per - 1) / per;
  if (directions == 1 ? 7LL * nch <= 11 * per + n + 24 : 5LL * nch <= 10 * per + 2 * n + 20) return;
  *seg_chunks = (int)per;
  *G = (int)n;
}

size_t gated_segment_bytes(int BH, int G, int Dk, int Dv) {
  return G > 1 ? ((size_t)BH * G * 4 + 255) / 256 * 256 + (size_t)BH * G * Dk * Dv * 4 : 0;
}

cudaError_t launch_wait_polls_selftest(unsigned int* status, int polls, cudaStream_t st) {
  wait_polls_selftest_kernel<<<1, 32, 0, st>>>(status, polls);
  return cudaGetLastError();
}

cudaError_t gated_device_word(void** at) { return cudaGetSymbolAddress(at, device_word); }

cudaError_t launch_gated_tc_fwd(const GatedProblem& p, cudaStream_t st) {
  if (p.alpha) return p.Dk == 128 ? fwd<128, true>(p, st) : fwd<64, true>(p, st);
  return p.Dk == 128 ? fwd<128, false>(p, st) : fwd<64, false>(p, st);
}

}  // namespace dn
