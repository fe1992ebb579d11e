// Decode attention over a 4-bit (E2M1, block-scaled) paged cache.
//
// The mathematics is that of the other decode kernels (online softmax in base
// 2, one pass over the keys, pieces joined by their LSEs); what differs is the
// route from the cache to the tensor cores.  A key and a value of one head
// are D / 2 bytes of codes and D / 16 of scales each, so at head size 128 a
// page of 16 keys is 1 KB of codes a matrix: far below the size at which TMA
// boxes reach the HBM rate (a box costs its SM about 200 cycles).  Here each
// warp copies its own key tiles with 16-byte cp.async into its own two-stage
// ring (no barrier across warps), and its lanes read exactly the codes of
// their own MMA fragments from there, convert them (cvt e2m1x2 -> f16x2,
// times the block scale: both exact in f16) and feed them to mma.sync.
//
//  S^T = K Q^T   The keys are the MMA's 16 rows (A), the packed query rows its
//    8 columns (B).  Lane (g8 = lane / 4, c4 = lane % 4) holds, for its two
//    keys of a 16-key subtile, the c4-th run of the row; the order of the
//    head dimension in the MMA's k steps is free (Q is laid out the same
//    way), so a run is one 16-byte read (D = 128) whose codes feed eight k
//    steps.
//  O^T = V^T P^T  The head dimensions are the rows (A), the query rows the
//    columns (B).  Lane (g8, c4) holds the g8-th run of four keys' rows:
//    its nibbles are interleaved into (key, next key) pairs with two bit
//    selects per eight codes, then converted and scaled with the pair of
//    block scales.  P^T, the accumulator of the first product, becomes the
//    B operand with one 8 x 8 transpose per register (movmatrix).
//
// Key m of a subtile's MMA row order is kappa(m) = 4 (m / 2) + m % 2 for
// m < 8 and two more for m + 8: lane c4's four V keys are then 4 c4 .. + 3.
//
// With 8 query rows or fewer (one n tile) each MMA covers 16 keys and no row
// is padding beyond 8, half of what 16-row query tiles would issue; 9 to 16
// rows take two n tiles over the same converted operands.
//
// Each warp walks its own key tiles of a CTA's range, one tile ahead of its
// reads; the warps meet once, at the end.  The running maximum is raised (and
// O rescaled) only when a logit passes it by 2^6: P stays below 64, which f16
// holds with the same relative error, and the common tile needs no reduction
// across lanes.
//
// Keys outside [lo, hi) of the request are never seen: their logits are
// -inf and their V scales 0 (a code is always finite, only a scale can be
// NaN).  Where the rows of a request see different keys, NaN scales of V are
// set aside and added to the rows that see the key.
#include <math.h>

#include <type_traits>

#include "pkv_common.cuh"

namespace pkv {
namespace dfp4 {

constexpr int kWarps = 4;
constexpr float kRaise = 6.f;      // log2 slack of the running maximum

// One stage of a warp's ring: MT subtiles of 16 keys, K codes, V codes, then
// 16 rows of 16 bytes of K scales and as many of V scales (row r: the scales
// of key r of each subtile, side by side).
//
// Swizzles (of the 16-byte chunks of a subtile's rows), so that the lanes of
// one read phase touch different banks: K is read as rows kappa(g8), chunk
// c4; V as rows 4 c4 + e, eight (D = 64: four) bytes at g8.
template <int D>
struct Geo {
  static constexpr int MT = D == 256 ? 1 : 2;
  static constexpr int RB = D / 2;                 // bytes of a row's codes
  static constexpr int SUB = 16 * RB;              // ... of a subtile
  static constexpr int CPR = RB / 16;              // chunks of a row
  static constexpr int OFF_V = MT * SUB;
  static constexpr int OFF_KF = 2 * MT * SUB;
  static constexpr int OFF_VF = OFF_KF + 256;
  static constexpr int STAGE = OFF_VF + 256;
  static constexpr int STAGES = 2;

  static __device__ __forceinline__ uint32_t k_off(int r, int ch) {
    if (D == 64) return (r ^ (2 * ((r >> 2) & 1))) * RB + ch * 16;
    if (D == 128) return r * RB + ch * 16;
    return r * RB + (ch ^ (4 * (r & 1))) * 16;
  }
  static __device__ __forceinline__ uint32_t v_off(int r, int ch) {
    if (D == 64)
      return ((r & ~3) | ((r & 3) ^ ((r >> 2) & 3))) * RB + ch * 16;
    if (D == 128)
      return (r ^ ((r >> 3) & 1)) * RB + (ch ^ (2 * ((r >> 2) & 1))) * 16;
    return r * RB + (ch ^ (2 * ((r >> 2) & 3))) * 16;
  }
};

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// N-byte global -> shared copy (4, 8: through L1); src_bytes 0 writes zeros.
template <int N>
__device__ __forceinline__ void cp_async_n(uint32_t dst, const void* src,
                                           int src_bytes) {
  if constexpr (N == 16)
    cp_async_16(dst, src, src_bytes);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;\n" ::"r"(dst),
                 "l"(src), "r"(src_bytes), "n"(N));
}

// D(16 x 8) += A(16 x 16) B(16 x 8), f16 in, fp32 accumulate.
__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1,
                                    uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  const uint32_t a[4] = {a0, a1, a2, a3};
  mma_16816<__half>(d, a, b0, b1);
}

// 1 / denominator and the natural LSE of a row whose sum is l relative to m
// (base 2).  NaN sums stay NaN.
__device__ __forceinline__ void finish(float m, float l, const float* sinks,
                                       int h, float* inv, float* lse) {
  const float z = sinks ? sinks[h] * kLog2e : -INFINITY;
  const float M = fmaxf(m, z);
  if (M == -INFINITY) {                 // nothing seen (or all NaN)
    *inv = l != l ? l : 0.f;
    *lse = l != l ? l : -INFINITY;
    return;
  }
  const float em = m == -INFINITY ? (l != l ? 1.f : 0.f) : ex2(m - M);
  const float den = l * em + (sinks ? ex2(z - M) : 0.f);
  *inv = em / den;
  *lse = (M + lg2(den)) * kLn2;
}

// log2(e) softcap tanh(x / softcap) of a logit given in base 2, as t =
// log2(e) softcap and u = 2 / softcap: t (1 - 2 / (1 + 2^(x u))) keeps the
// absolute error near one ulp of the cap (tanh.approx loses 2^-11 of the
// logit).
__device__ __forceinline__ float soft_cap(float x, float t, float u) {
  return t - __fdividef(2.f * t, 1.f + ex2(x * u));
}

template <int D, int NR>
struct Smem {
  // query fragments (one 16-byte load serves two k steps of every subtile)
  // and the warps' states at the end
  static constexpr int ROWS = 8 * NR;
  static constexpr int QBYTES = (D / 32) * NR * 32 * 16;
  static constexpr int OSTRIDE = ROWS * D + 4 * (ROWS / 2);   // floats a warp
  static constexpr int OBYTES = kWarps * OSTRIDE * 4;
  static constexpr int MLBYTES = kWarps * ROWS * 8;
  // (the states take the rings' place)
  static constexpr int RBYTES = kWarps * Geo<D>::STAGES * Geo<D>::STAGE;
  static constexpr int BYTES =
      QBYTES + (RBYTES > OBYTES + MLBYTES ? RBYTES : OBYTES + MLBYTES);
};

template <int D, int NR>
constexpr int min_ctas() {
  return NR == 1 ? (D == 256 ? 3 : 4) : (D == 256 ? 2 : 3);
}

template <typename T, int D, int NR>
__global__ void __launch_bounds__(kWarps * 32, min_ctas<D, NR>())
decode_fp4_kernel(const AttnParams p, int splits) {
  // the fold of the pieces may become resident once every CTA has started
  // (it waits for this grid before reading them)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using SM = Smem<D, NR>;
  using GE = Geo<D>;
  constexpr int MT = GE::MT;
  constexpr int KT = 16 * MT;            // keys of a warp's tile
  constexpr int KS = D / 16;             // k steps of S, and m tiles of O
  constexpr int KW = D / 32;             // words of a lane's K codes per key
  constexpr int VW = D / 64;             // words of a lane's V codes per key
  extern __shared__ __align__(16) unsigned char smem[];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g8 = lane >> 2, c4 = lane & 3;
  const int G = p.G;
  // CTAs in the order (request, piece, KV head): neighbours read the same
  // pages
  const int h = blockIdx.x % p.Hkv;
  const unsigned rest = blockIdx.x / p.Hkv;
  const int sp = rest % splits;
  const int b = rest / splits;

  const int q0 = p.cu_q[b];
  const int q_len = min(p.cu_q[b + 1] - q0, p.total_q - q0);
  if (q0 < 0 || q_len <= 0) return;
  const int rows = q_len * G;
  if (rows < p.min_rows || rows > p.max_rows) return;
  if (rows > 8 * NR) {
    // more query rows than the call's max_seqlen_q allows: not computed
    if (sp == 0 && h == 0 && threadIdx.x == 0) atomicOr(p.err, kErrQueryLen);
    return;
  }
  const int L = p.seqused_k[b];
  const int64_t tab = static_cast<int64_t>(p.max_blocks) * p.BS;
  const int L_tab = L < tab ? L : static_cast<int>(tab);
  if (L_tab < L && sp == 0 && h == 0 && threadIdx.x == 0)
    atomicOr(p.err, kErrBadTable);
  int kmin, kmax;
  key_range(L, q_len, 0, q_len - 1, p.causal, p.wl, p.wr, kmin, kmax);
  int lo = kmin, hi = kmax;
  if (p.chunk > 0) {
    const int ns = split_count(kmin, kmax, p.chunk, splits);
    if (sp >= ns) return;
    split_bounds(kmin, kmax, p.chunk, ns, sp, lo, hi);
  }
  hi = max(lo, min(hi, L_tab));

  // ---- queries: lane (g8, c4) takes row g8 (and g8 + 8), the dimensions of
  // its K run.  A bf16 row is scaled by the power of two that puts its
  // largest magnitude in [2^14, 2^15): exact in f16; the factor joins the
  // row's logit scale.
  float row_scale[NR][2];   // logit scale (base 2) of rows 2 c4, 2 c4 + 1
  {
    const T* Q = static_cast<const T*>(p.q);
    const float base_scale = p.scale * *p.k_scale * kLog2e;
    uint4* qs = reinterpret_cast<uint4*>(smem);
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = g8 + 8 * n;
      uint4 raw[KW];
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < KW; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const T* src = Q + static_cast<int64_t>(q0 + r / G) * p.q_st +
                       static_cast<int64_t>(h * G + r % G) * p.q_sh;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          // word i of the run: 8 dimensions (D = 256: two runs of 4 words)
          const int d = D == 256 ? 128 * (i >> 2) + 32 * c4 + 8 * (i & 3)
                                 : 8 * KW * c4 + 8 * i;
          raw[i] = *reinterpret_cast<const uint4*>(src + d);
        }
      }
      float qmul = 1.f, back = 1.f;
      if constexpr (!std::is_same<T, __half>::value) {
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          float x[8];
          widen8<T>(raw[i], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int shift = 0;
        if (mx > 0.f) {
          shift = static_cast<int>((__float_as_uint(mx) >> 23) & 0xff) - 141;
          shift = max(-100, min(100, shift));
        }
        qmul = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
        back = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        row_scale[n][e] =
            __shfl_sync(0xffffffffu, back, (2 * c4 + e) * 4) * base_scale;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[e] = std::is_same<T, __half>::value
                     ? w[e]
                     : pack2<__half>(elem_f32<T>(w[e], 0) * qmul,
                                     elem_f32<T>(w[e], 1) * qmul);
        // 8 dimensions: the B operands of k steps 2 i and 2 i + 1
        if (KW < kWarps || (i & (kWarps - 1)) == warp)
          qs[(i * NR + n) * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
      }
    }
  }
  __syncthreads();

  const bool plain = p.softcap <= 0.f && p.alibi == nullptr;
  const float cap_t = p.softcap * kLog2e;
  const float cap_u = p.softcap > 0.f ? 2.f / p.softcap : 0.f;
  const int ctx = L - q_len;
  int pos[NR][2];
  float slope[NR][2];
  bool live[NR][2];
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * c4 + e;
      live[n][e] = r < rows;
      pos[n][e] = ctx + r / G;
      slope[n][e] =
          p.alibi && r < rows ? p.alibi[h * G + r % G] * kLog2e : 0.f;
    }
  // keys in [full_lo, full_hi) are seen by every row
  int full_lo = lo, full_hi = hi;
  {
    const int p_lo = ctx, p_hi = ctx + q_len - 1;
    if (p.wl >= 0) full_lo = max(full_lo, p_hi - p.wl);
    if (p.causal) full_hi = min(full_hi, p_lo + 1);
    if (p.wr >= 0) full_hi = min(full_hi, p_lo + p.wr + 1);
  }

  float o[KS][NR][4];
#pragma unroll
  for (int i = 0; i < KS; ++i)
#pragma unroll
    for (int n = 0; n < NR; ++n)
      o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
  float m[NR][2], l[NR][2];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }

  // ---- the warp's tiles: kt0 + (warp + i kWarps) KT
  const int kt0 = lo & ~15;
  const int tiles = hi > lo ? (hi - kt0 + KT - 1) / KT : 0;
  const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
  const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
  const int subs = mine * MT;
  auto sub_key = [&](int s) {            // first key of my subtile s
    return kt0 + (warp + (s / MT) * kWarps) * KT + (s % MT) * 16;
  };
  // page and first row in it of subtile s0 + lane (-1: past the range, or a
  // page outside the cache, whose keys read as zero)
  auto fetch = [&](int s0, int& id, int& row) {
    const int s = s0 + lane;
    const int k0 = s < subs ? sub_key(s) : hi;
    id = -1;
    row = 0;
    if (k0 >= hi) return;
    const int j = p.bs_shift >= 0 ? k0 >> p.bs_shift : k0 / p.BS;
    row = k0 - j * p.BS;
    id = __ldg(bt + j);
    if (id < 0 || id >= p.num_blocks) {
      atomicOr(p.err, kErrBadBlock);
      id = -1;
    }
  };
  int ids, rows0, ids_next, rows0_next;
  fetch(0, ids, rows0);
  fetch(32, ids_next, rows0_next);
  const int kap = 4 * (g8 >> 1) + (g8 & 1);
  const uint32_t c_sb = static_cast<uint32_t>(p.c_sb);
  const uint32_t f_sb = static_cast<uint32_t>(p.f_sb);
  const uint32_t c_sr = static_cast<uint32_t>(p.c_sr);
  const uint32_t f_sr = static_cast<uint32_t>(p.f_sr);
  // this lane's copies: chunk lane + 32 i of a subtile's codes, and the
  // scales of one row (lanes 0 .. 15 of K, 16 .. 31 of V)
  constexpr int NC = GE::SUB / 16 / 32;  // chunks of a lane
  constexpr int RI = 32 / GE::CPR;       // rows from one to the next
  const int cp_r = lane / GE::CPR, cp_c = lane % GE::CPR;
  const uint8_t* const KC = static_cast<const uint8_t*>(p.kc) +
                            static_cast<int64_t>(h) * p.c_sh + cp_r * c_sr +
                            16 * cp_c;
  const int64_t k_to_v = static_cast<const uint8_t*>(p.vc) -
                         static_cast<const uint8_t*>(p.kc);
  const uint8_t* const SF = (lane < 16 ? p.k_sf : p.v_sf) +
                            static_cast<int64_t>(h) * p.f_sh +
                            (lane & 15) * f_sr;
  const uint32_t ring = smem_u32(smem) + SM::QBYTES +
                        warp * (GE::STAGES * GE::STAGE);
  uint32_t k_dst[NC], v_dst[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    k_dst[i] = ring + GE::k_off(cp_r + RI * i, cp_c);
    v_dst[i] = ring + GE::OFF_V + GE::v_off(cp_r + RI * i, cp_c);
  }
  const uint32_t f_dst = ring + GE::OFF_KF + (lane >> 4) * 256 +
                         (lane & 15) * 16;
  auto issue = [&](int s0, uint32_t stage) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int id = __shfl_sync(0xffffffffu, ids, (s0 + i) & 31);
      const uint32_t row = __shfl_sync(0xffffffffu, rows0, (s0 + i) & 31);
      const int n = id < 0 ? 0 : 16;
      const uint32_t page = id < 0 ? 0 : id;
      const uint8_t* src = KC + static_cast<uint64_t>(page) * c_sb +
                           row * c_sr;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const uint8_t* ks = src + j * RI * c_sr;
        cp_async_16(stage + k_dst[j] + i * GE::SUB, ks, n);
        cp_async_16(stage + v_dst[j] + i * GE::SUB, ks + k_to_v, n);
      }
      cp_async_n<D / 16>(stage + f_dst + i * (D / 16),
                         SF + static_cast<uint64_t>(page) * f_sb + row * f_sr,
                         id < 0 ? 0 : D / 16);
    }
  };

  if (mine > 0) issue(0, 0);
  cp_async_commit();
  if (mine > 1) issue(MT, GE::STAGE);
  cp_async_commit();
  for (int it = 0; it < mine; ++it) {
    const int kt = kt0 + (warp + it * kWarps) * KT;
    const uint32_t stage = (it & 1) * GE::STAGE;
    const uint32_t st = ring + stage;
    cp_async_wait<1>();
    __syncwarp();
    // ---- S^T
    float sc[MT][NR][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < NR; ++n)
        sc[i][n][0] = sc[i][n][1] = sc[i][n][2] = sc[i][n][3] = 0.f;
    uint32_t kw[MT][2][KW], kf[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = kap + 2 * e;
        const uint32_t src = st + i * GE::SUB;
        const uint32_t fs = st + GE::OFF_KF + r * 16 + i * (D / 16);
        if constexpr (D == 64) {
          const uint2 v = lds64(src + GE::k_off(r, c4 >> 1) + 8 * (c4 & 1));
          kw[i][e][0] = v.x;
          kw[i][e][1] = v.y;
          kf[i][e] = lds8(fs + c4);
        } else {
          kf[i][e] = 0;
#pragma unroll
          for (int q = 0; q < D / 128; ++q) {
            const uint4 v = lds128(src + GE::k_off(r, 4 * q + c4));
            kw[i][e][4 * q] = v.x;
            kw[i][e][4 * q + 1] = v.y;
            kw[i][e][4 * q + 2] = v.z;
            kw[i][e][4 * q + 3] = v.w;
            kf[i][e] |= lds16(fs + 8 * q + 2 * c4) << (16 * q);
          }
        }
      }
    // block scales of the lane's keys, two groups (D = 64: two keys) a word
    constexpr int FW = D == 256 ? 2 : 1;
    uint32_t fk[MT][2][FW];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if constexpr (D == 64) {
        fk[i][0][0] = e4m3x2_to_f16(__byte_perm(kf[i][0], kf[i][1], 0x40));
        fk[i][1][0] = 0;
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int q = 0; q < FW; ++q)
            fk[i][e][q] = e4m3x2_to_f16(kf[i][e] >> (16 * q));
      }
    }
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      uint4 qb[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n)
        qb[n] = reinterpret_cast<const uint4*>(smem)[(w * NR + n) * 32 + lane];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t a[4], c[4];
        e2m1x8_to_f16(kw[i][0][w], a[0], a[1], a[2], a[3]);
        e2m1x8_to_f16(kw[i][1][w], c[0], c[1], c[2], c[3]);
        uint32_t fa, fc;
        if constexpr (D == 64) {
          fa = __byte_perm(fk[i][0][0], 0, 0x1010);
          fc = __byte_perm(fk[i][0][0], 0, 0x3232);
        } else {
          const uint32_t sel = (w & 2) ? 0x3232u : 0x1010u;
          fa = __byte_perm(fk[i][0][w >> 2], 0, sel);
          fc = __byte_perm(fk[i][1][w >> 2], 0, sel);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] = hmul2_u32(a[e], fa);
          c[e] = hmul2_u32(c[e], fc);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          mma(sc[i][n], a[0], c[0], a[1], c[1], qb[n].x, qb[n].y);
          mma(sc[i][n], a[2], c[2], a[3], c[3], qb[n].z, qb[n].w);
        }
      }
    }
    // ---- logits (base 2) and masks
    const bool interior = kt >= full_lo && kt + KT <= full_hi;
    float mx[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) mx[n][0] = mx[n][1] = -INFINITY;
    if (plain && interior) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (the product is rounded once, here: a fused multiply-add with
            // the maximum would differ from it by half an ulp of the logit,
            // which may be far above 1)
            sc[i][n][e] *= row_scale[n][e & 1];
            mx[n][e & 1] = fmaxf(mx[n][e & 1], sc[i][n][e]);
          }
    } else {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = sc[i][n][e] * row_scale[n][e & 1];   // (base 2)
            if (p.softcap > 0.f) x = soft_cap(x, cap_t, cap_u);
            const int key = kt + 16 * i + kap + (e & 2);
            const int at = pos[n][e & 1];
            if (p.alibi)
              x -= slope[n][e & 1] * fabsf(static_cast<float>(at - key));
            if (!interior) {
              bool ok = live[n][e & 1] && key >= lo && key < hi;
              if (p.causal) ok = ok && key <= at;
              if (p.wl >= 0) ok = ok && key >= at - p.wl;
              if (p.wr >= 0) ok = ok && key <= at + p.wr;
              x = ok ? x : -INFINITY;
            }
            sc[i][n][e] = x;
            mx[n][e & 1] = fmaxf(mx[n][e & 1], x);
          }
      }
    }
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) raise = raise || mx[n][e] > m[n][e] + kRaise;
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = mx[n][e];
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          t = fmaxf(t, m[n][e]);
          const float al = t == m[n][e] ? 1.f : ex2(m[n][e] - t);
          m[n][e] = t;
          l[n][e] *= al;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[i][n][e] *= al;
            o[i][n][e + 2] *= al;
          }
        }
    }
    // P and its sums, and P^T as the B operand of each subtile
    uint32_t pb[MT][NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const float base0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
      const float base1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float* x = sc[i][n];
        x[0] = ex2(x[0] - base0);
        x[1] = ex2(x[1] - base1);
        x[2] = ex2(x[2] - base0);
        x[3] = ex2(x[3] - base1);
        l[n][0] += x[0] + x[2];
        l[n][1] += x[1] + x[3];
        // P rounds to f16 (half a step of 2^-11 relative) for the MMA; the
        // sums keep the float32 values
        pb[i][n][0] = movmatrix(pack2<__half>(x[0], x[1]));
        pb[i][n][1] = movmatrix(pack2<__half>(x[2], x[3]));
      }
    }
    // ---- O^T += V^T P^T
    constexpr int VG = D == 256 ? 2 : 1;     // block scales of a lane
    // scales of the lane's four keys, a byte each, per subtile and group
    uint32_t vf[MT][VG];
    if constexpr (D == 64) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[e] = lds8(st + GE::OFF_VF + (4 * c4 + e) * 16 + i * 4 +
                      (g8 >> 1));
        vf[i][0] = __byte_perm(__byte_perm(f[0], f[1], 0x40),
                               __byte_perm(f[2], f[3], 0x40), 0x5410);
      }
    } else {
      // rows are keys, columns groups (of two subtiles at D = 128)
      uint32_t d0, d1;
      ldmatrix_b8_trans(st + GE::OFF_VF + (lane & 15) * 16, d0, d1);
      vf[0][0] = d0;
      vf[MT - 1][VG - 1] = d1;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (!interior) {
        // keys outside [lo, hi): a scale of 0
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = kt + 16 * i + 4 * c4 + e;
          if (key < lo || key >= hi)
#pragma unroll
            for (int v = 0; v < VG; ++v) vf[i][v] &= ~(0xffu << (8 * e));
        }
        // NaN scales: set aside, and added to the rows that see the key
        uint32_t nan_bits[VG];
        bool any = false;
#pragma unroll
        for (int v = 0; v < VG; ++v) {
          nan_bits[v] = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (((vf[i][v] >> (8 * e)) & 0x7fu) == 0x7fu)
              nan_bits[v] |= 1u << (4 * c4 + e);
          any = any || nan_bits[v] != 0;
        }
        if (__any_sync(0xffffffffu, any)) {
#pragma unroll
          for (int v = 0; v < VG; ++v) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((nan_bits[v] >> (4 * c4 + e)) & 1u)
                vf[i][v] &= ~(0xffu << (8 * e));
            nan_bits[v] |= __shfl_xor_sync(0xffffffffu, nan_bits[v], 1);
            nan_bits[v] |= __shfl_xor_sync(0xffffffffu, nan_bits[v], 2);
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int at = pos[n][e];
                bool hit = false;
                for (int j = 0; j < 16; ++j) {
                  const int key = kt + 16 * i + j;
                  bool ok = (nan_bits[v] >> j) & 1u;
                  if (p.causal) ok = ok && key <= at;
                  if (p.wl >= 0) ok = ok && key >= at - p.wl;
                  if (p.wr >= 0) ok = ok && key <= at + p.wr;
                  hit = hit || ok;
                }
                if (hit) {
#pragma unroll
                  for (int w = 0; w < KS / VG; ++w) {
                    o[v * (KS / VG) + w][n][e] = NAN;
                    o[v * (KS / VG) + w][n][e + 2] = NAN;
                  }
                }
              }
          }
        }
      }
#pragma unroll
      for (int v = 0; v < VG; ++v) {
        const uint32_t s01 = e4m3x2_to_f16(vf[i][v]);
        const uint32_t s23 = e4m3x2_to_f16(vf[i][v] >> 16);
        // the lane's run of the four keys' rows: 16 dimensions (D = 64: 8)
        constexpr int RW = D == 64 ? 1 : 2;
        uint32_t vw[4][RW];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * c4 + e;
          const uint32_t src = st + GE::OFF_V + i * GE::SUB;
          if constexpr (D == 64) {
            vw[e][0] = lds32(src + GE::v_off(r, g8 >> 2) + 4 * (g8 & 3));
          } else {
            const uint2 x = lds64(src + GE::v_off(r, 4 * v + (g8 >> 1)) +
                                  8 * (g8 & 1));
            vw[e][0] = x.x;
            vw[e][1] = x.y;
          }
        }
#pragma unroll
        for (int w = 0; w < RW; ++w) {
          const uint32_t w0 = vw[0][w], w1 = vw[1][w];
          const uint32_t w2 = vw[2][w], w3 = vw[3][w];
          // bytes (key, next key) of the even and of the odd dimensions
          const uint32_t e01 = (w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u);
          const uint32_t o01 = ((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u);
          const uint32_t e23 = (w2 & 0x0f0f0f0fu) | ((w3 << 4) & 0xf0f0f0f0u);
          const uint32_t o23 = ((w2 >> 4) & 0x0f0f0f0fu) | (w3 & 0xf0f0f0f0u);
          uint32_t a0[4], a1[4], a2[4], a3[4];
          e2m1x8_to_f16(e01, a0[0], a0[1], a0[2], a0[3]);
          e2m1x8_to_f16(o01, a1[0], a1[1], a1[2], a1[3]);
          e2m1x8_to_f16(e23, a2[0], a2[1], a2[2], a2[3]);
          e2m1x8_to_f16(o23, a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x0 = hmul2_u32(a0[e], s01);
            const uint32_t x1 = hmul2_u32(a1[e], s01);
            const uint32_t x2 = hmul2_u32(a2[e], s23);
            const uint32_t x3 = hmul2_u32(a3[e], s23);
#pragma unroll
            for (int n = 0; n < NR; ++n)
              mma(o[(v * RW + w) * 4 + e][n], x0, x1, x2, x3, pb[i][n][0],
                  pb[i][n][1]);
          }
        }
      }
    }
    // this stage is read: the tile after the next one into it
    __syncwarp();
    const int s_new = (it + 2) * MT;
    if (it + 2 < mine) {
      if ((s_new & 31) == 0) {
        ids = ids_next;
        rows0 = rows0_next;
        fetch(s_new + 32, ids_next, rows0_next);
      }
      issue(s_new, stage);
    }
    cp_async_commit();
  }
  cp_async_wait<0>();
  __syncthreads();       // (the states take the rings' place)

  // ---- the warps' states meet: row r of warp w at r D + 4 (r / 2) floats
  // (conflict-free float4 stores)
  float* ow = reinterpret_cast<float*>(smem + SM::QBYTES);
  float2* ml = reinterpret_cast<float2*>(smem + SM::QBYTES + SM::OBYTES);
  float* mine_o = ow + warp * SM::OSTRIDE;
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = l[n][e];
      t += __shfl_xor_sync(0xffffffffu, t, 4);
      t += __shfl_xor_sync(0xffffffffu, t, 8);
      t += __shfl_xor_sync(0xffffffffu, t, 16);
      const int r = 8 * n + 2 * c4 + e;
      if (g8 == 0) ml[warp * SM::ROWS + r] = make_float2(m[n][e], t);
      // o[i]: dimensions 2 (i % 8) and the next one of the lane's run
      // i / 8 (16 g8 of each 128; D = 64: 8 g8), two m tiles a store
      float* dst = mine_o + r * D + 4 * (r >> 1) + (D == 64 ? 8 : 16) * g8;
#pragma unroll
      for (int i = 0; i < KS; i += 2)
        *reinterpret_cast<float4*>(dst + 128 * (i >> 3) + 2 * (i & 7)) =
            make_float4(o[i][n][e], o[i][n][e + 2], o[i + 1][n][e],
                        o[i + 1][n][e + 2]);
    }
  __syncthreads();
  const float vscale = *p.v_scale;
  for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
    const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * SM::ROWS + r].x);
    const float base = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 s = ml[w * SM::ROWS + r];
      // a warp that saw nothing but NaN keeps its NaN sum
      const float f = s.x == -INFINITY ? (s.y == 0.f ? 0.f : 1.f)
                                       : ex2(s.x - base);
      if (f == 0.f) continue;
      const float4 v = *reinterpret_cast<const float4*>(
          ow + w * SM::OSTRIDE + r * D + 4 * (r >> 1) + col);
      sum += f * s.y;
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    const int tok = q0 + r / G, hq = h * G + r % G;
    float inv, lse;
    finish(M, sum, p.chunk > 0 ? nullptr : p.sinks, hq, &inv, &lse);
    inv *= vscale;
    if (p.chunk > 0) {
      const int64_t row = part_row(p.part_tpr, b, q0, tok);
      *reinterpret_cast<float4*>(
          p.part_o +
          ((static_cast<int64_t>(sp) * p.part_rows + row) * p.Hq + hq) * D +
          col) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv,
                             acc.w * inv);
      if (col == 0)
        p.part_lse[(static_cast<int64_t>(sp) * p.Hq + hq) * p.part_rows +
                   row] = lse;
    } else {
      T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(tok) * p.o_st +
               static_cast<int64_t>(hq) * p.o_sh + col;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack2<T>(acc.x * inv, acc.y * inv),
                     pack2<T>(acc.z * inv, acc.w * inv));
      if (p.lse && col == 0)
        p.lse[static_cast<int64_t>(hq) * p.total_q + tok] = lse;
    }
  }
}

// Fold the pieces of each (token, head) by their LSEs: one warp each, lanes
// over the columns.  The sink joins here, once.
template <typename T, int D>
__global__ void __launch_bounds__(128) combine_kernel(const CombineParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int b = blockIdx.x;
  if (h >= p.Hq) return;
  const int q0 = p.cu_q[b];
  const int q_len = min(p.cu_q[b + 1] - q0, p.total_q - q0);
  if (q0 < 0 || q_len <= 0) return;
  const int rows = q_len * p.G;
  if (rows < p.min_rows || rows > p.max_rows) return;
  int kmin, kmax;
  key_range(p.seqused_k[b], q_len, 0, q_len - 1, p.causal, p.wl, p.wr, kmin,
            kmax);
  const int ns = split_count(kmin, kmax, p.chunk, p.splits);
  for (int i = 0; i < q_len; ++i) {
    const int tok = q0 + i;
    const int64_t row = part_row(p.part_tpr, b, q0, tok);
    const int64_t l_st = static_cast<int64_t>(p.Hq) * p.part_rows;
    const float* pl = p.part_lse + static_cast<int64_t>(h) * p.part_rows + row;
    const float* po = p.part_o + (row * p.Hq + h) * D;
    const int64_t o_st = static_cast<int64_t>(p.part_rows) * p.Hq * D;
    float M = -INFINITY;
    for (int s = lane; s < ns; s += 32) M = fmaxf(M, pl[s * l_st]);
#pragma unroll
    for (int o = 16; o; o >>= 1)
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.f : M * kLog2e;
    float sum = 0.f;
    constexpr int CPL = D >= 128 ? D / 128 : 1;     // float4s a lane
    float4 acc[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool on = D >= 128 || lane < D / 4;
#pragma unroll 4
    for (int s = 0; s < ns; ++s) {
      const float w = ex2(pl[s * l_st] * kLog2e - base);   // -inf -> 0
      sum += w;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        if (!on) continue;
        const float4 v = *reinterpret_cast<const float4*>(
            po + s * o_st + (lane + 32 * c) * 4);
        if (w == 0.f) continue;
        acc[c].x += w * v.x;
        acc[c].y += w * v.y;
        acc[c].z += w * v.z;
        acc[c].w += w * v.w;
      }
    }
    float inv, lse;
    finish(M * kLog2e, sum, p.sinks, h, &inv, &lse);
    T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(tok) * p.o_st +
             static_cast<int64_t>(h) * p.o_sh;
#pragma unroll
    for (int c = 0; c < CPL; ++c)
      if (on)
        *reinterpret_cast<uint2*>(dst + (lane + 32 * c) * 4) =
            make_uint2(pack2<T>(acc[c].x * inv, acc[c].y * inv),
                       pack2<T>(acc[c].z * inv, acc[c].w * inv));
    if (p.lse && lane == 0)
      p.lse[static_cast<int64_t>(h) * p.total_q + tok] = lse;
  }
}

template <typename T, int D, int NR>
cudaError_t launch(const AttnParams& p, int splits, cudaStream_t stream) {
  using SM = Smem<D, NR>;
  auto kern = decode_fp4_kernel<T, D, NR>;
  cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(kern), SM::BYTES);
  if (e != cudaSuccess) return e;
  const int64_t ctas = static_cast<int64_t>(p.batch) * splits * p.Hkv;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  note_launch();
  kern<<<static_cast<unsigned>(ctas), kWarps * 32, SM::BYTES, stream>>>(
      p, splits);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t dispatch_rows(const AttnParams& p, int splits,
                          cudaStream_t stream) {
  const bool one = p.sk_rows <= 8;       // packed query rows of a request
  return one ? launch<T, D, 1>(p, splits, stream)
             : launch<T, D, 2>(p, splits, stream);
}

template <typename T>
cudaError_t dispatch(const AttnParams& p, int D, int splits,
                     cudaStream_t stream) {
  switch (D) {
    case 64: return dispatch_rows<T, 64>(p, splits, stream);
    case 128: return dispatch_rows<T, 128>(p, splits, stream);
    case 256: return dispatch_rows<T, 256>(p, splits, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dfp4

int decode_fp4_ctas_per_sm(int D, int rows) {
  return rows <= 8 ? (D == 256 ? 3 : 4) : (D == 256 ? 2 : 3);
}

cudaError_t launch_decode_attn_fp4(const AttnParams& p, int D, bool bf16,
                                   int splits, cudaStream_t stream) {
  return bf16 ? dfp4::dispatch<__nv_bfloat16>(p, D, splits, stream)
              : dfp4::dispatch<__half>(p, D, splits, stream);
}

cudaError_t launch_fp4_combine(const CombineParams& p, bool bf16, bool pdl,
                               cudaStream_t stream) {
  note_launch();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch), (p.Hq + 3) / 4);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  auto go = [&](auto kern) { return cudaLaunchKernelEx(&cfg, kern, p); };
  cudaError_t e;
  switch (p.D) {
    case 64:
      e = bf16 ? go(dfp4::combine_kernel<__nv_bfloat16, 64>)
               : go(dfp4::combine_kernel<__half, 64>);
      break;
    case 128:
      e = bf16 ? go(dfp4::combine_kernel<__nv_bfloat16, 128>)
               : go(dfp4::combine_kernel<__half, 128>);
      break;
    default:
      e = bf16 ? go(dfp4::combine_kernel<__nv_bfloat16, 256>)
               : go(dfp4::combine_kernel<__half, 256>);
      break;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pkv
