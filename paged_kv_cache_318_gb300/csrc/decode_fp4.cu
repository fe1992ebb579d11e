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
// Each warp walks its own key tiles of its group's range, one tile ahead of its
// reads; the warps meet once, at the end.  P = 2^(logit - reference), with the
// reference 9 below the running maximum and raised (O rescaled) only when a
// logit passes it by 15: the common tile needs no reduction across lanes.  P
// rounds to f16: by at most 2^-11 of itself down to 2^-14, that is 2^-23 of the
// largest weight, and by at most 2^-25 below, so n keys lose at most n 2^-34 of
// the largest weight; the sums keep the float32 values.  Each row is raised by
// its own logits, whatever the others of its tile do: with a fixed split its
// bits are the same in every call.
//
// What bounds it: 2 Hkv (D / 2 + D / 16) bytes a key from HBM, then the SM's
// own work, about 590 instructions for a warp's 32 keys (128 conversions, 128
// scalings, 32 MMAs at 8 rows).  Measured on a GB300 whose copy reaches 6.79
// TB/s, back to back: 8 requests of 131072 keys, 64/8 heads, D 128, 0.204 ms
// (5.9 TB/s, 87 %); 124 windows of 4096 keys, two tokens each, 16/8 heads, D
// 256, soft-cap, 0.210 ms (5.3 TB/s, 78 %); 64 requests of 512-4096 keys,
// 32/8 heads, 0.048 ms (3.8 TB/s: 3 us go to the launch, 3 to finding the
// share, 3 to the first pages and 6 to the join); 2 requests of 131072 keys,
// 128/8 heads (16 rows), 0.081 ms (3.7 TB/s: 655 instructions a tile from two
// warps a scheduler that wait on their own chains).  The steps, on the first
// of these: codes loaded straight into registers 0.390 ms, each warp's ring
// 0.269, equal shares and 128-byte aligned stages 0.216, warps' states joined
// pairwise so that 4 groups fit an SM 0.211, these as one CTA 0.203; the reference
// below the maximum costs 0.3 to 0.5 % of each of these.  Measured
// and not kept: equal shares for warps (0.222), 3 groups an SM (the same),
// shares cut so that an SM's groups take pieces as they finish (0.253), larger
// shares for an SM's older CTAs (0.217 to 0.229), more stages for 9 to 16 rows
// (the same), subtiles of 16 keys one after the other there (0.098 against
// 0.083).
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
// P is 2^(logit - reference) and the reference 2^kRoom below a row's running
// maximum, raised when a logit passes it by 2^kTop: P stays at or below 2^15,
// where f16 ends, and the smallest P that f16 holds (2^-24, half of it rounds
// away) is 2^-33 of the maximum.
constexpr float kRoom = 9.f;
constexpr float kTop = 15.f;
constexpr float kUnroom = 1.f / 512.f;            // 2^-kRoom
// Tiles of a group's share at least, so that each warp has some.
constexpr int kMinTiles = 2 * kWarps;
// What a unit costs a group beside its tiles, in tiles: its queries, the join
// of the warps' states and the store.  (64 requests of 512-4096 keys, 32/8 heads:
// 0 tiles 55.9 us, 4 51.3, 8 49.8, 12 50.4, 16 51.3; later 4 49.3, 8 47.5, 12
// 47.5.)
constexpr int kUnitCost = 8;
constexpr int kFoldThreads = 256;

inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

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

// 16 bytes that this call reads once: first to leave L2, so that what other
// kernels read stays there (and this one's tables: 64 requests of 512-4096
// keys 47.5 us against 50.0 with plain copies, 8 x 131072 the same).
__device__ __forceinline__ void cp_async_once(uint32_t dst, const void* src,
                                              int src_bytes, uint64_t policy) {
  asm volatile(
      "cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n"
      ::"r"(dst), "l"(src), "r"(src_bytes), "l"(policy));
}

// One half of an f16x2 in both.
__device__ __forceinline__ uint32_t spread(uint32_t v, int high) {
  const __half2 x = *reinterpret_cast<const __half2*>(&v);
  const __half2 r = high ? __high2half2(x) : __low2half2(x);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// D(16 x 8) = A(16 x 16) B(16 x 8), f16 in, fp32 accumulate; mma: D += ...
__device__ __forceinline__ void mma_first(float* d, uint32_t a0, uint32_t a1,
                                          uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
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

// f a + g b, rounded the same way in every instance of the kernel.
__device__ __forceinline__ float fold2(float f, float a, float g, float b) {
  return __fmaf_rn(f, a, __fmul_rn(g, b));
}

template <int D, int NR>
struct Smem {
  // Groups of kWarps warps on an SM: as many as their registers allow without
  // spills in the loop.  (9 to 16 rows of D = 128: 2 read 2 requests of 131072
  // keys, 128/8 heads, in 0.083 ms, 3 with spills in 0.093; of D = 64: 2 take
  // 0.070 ms on 64 x 4096 keys, 3 take 0.064.)
  static constexpr int RESIDENT = NR == 1 ? (D == 256 ? 3 : 4)
                                          : (D == 64 ? 3 : 2);
  // ... and of a CTA, where each takes a share.  CTAs of one SM run at speeds
  // of their own, the oldest fastest (of four equal shares of 8 x 131072 keys
  // the first ended at 153 us and the last at 209); groups of one CTA end
  // together (at 198).  Where the SM's work bounds the call they also wait
  // together: 9 to 16 rows 0.088 against 0.083 ms, D = 256 0.211 against
  // 0.209 on 124 windows of 4096 keys.
  static constexpr int GROUPS = NR == 1 && D <= 128 ? RESIDENT : 1;
  // query fragments (one 16-byte load serves two k steps of every subtile),
  // the warps' rings, and two warps' states (as their lanes hold them) at
  // the end of a unit
  static constexpr int QBYTES = (D / 32) * NR * 32 * 16;
  static constexpr int SREGS = D / 16 * NR * 4;              // O of a lane
  static constexpr int SBYTES = 32 * (SREGS + 4 * NR) * 4;
  static constexpr int OFF_RING = QBYTES;
  static constexpr int OFF_S =
      OFF_RING + kWarps * Geo<D>::STAGES * Geo<D>::STAGE;
  static constexpr int BYTES = OFF_S + kWarps / 2 * SBYTES;
  static_assert(BYTES % 128 == 0, "a group's stages are 128-byte aligned");
};

// What a request's rows see of its keys.
struct Req {
  int q0, q_len, rows, L, lo, hi;      // rows 0: not of this launch
};
// A range without keys is [0, 0): a window that starts past the table's end
// must not lead to a column behind it.
__device__ __forceinline__ void no_keys(Req& r) {
  if (r.hi <= r.lo) r.lo = r.hi = 0;
}
__device__ __forceinline__ Req request(const AttnParams& p, int b,
                                       int max_rows, bool flag) {
  Req r{};
  const int L = p.seqused_k[b];          // (three loads in flight at once)
  r.q0 = p.cu_q[b];
  r.q_len = min(p.cu_q[b + 1] - r.q0, p.total_q - r.q0);
  if (r.q0 < 0 || r.q_len <= 0) return r;
  const int rows = r.q_len * p.G;
  if (rows < p.min_rows || rows > p.max_rows) return r;
  if (rows > max_rows) {
    // more query rows than the call's max_seqlen_q allows: not computed
    if (flag) atomicOr(p.err, kErrQueryLen);
    return r;
  }
  r.rows = rows;
  r.L = L;
  const int64_t tab = static_cast<int64_t>(p.max_blocks) * p.BS;
  const int L_tab = r.L < tab ? r.L : static_cast<int>(tab);
  if (flag && L_tab < r.L) atomicOr(p.err, kErrBadTable);
  int kmin, kmax;
  key_range(r.L, r.q_len, 0, r.q_len - 1, p.causal, p.wl, p.wr, kmin, kmax);
  r.lo = kmin;
  r.hi = min(kmax, L_tab);
  no_keys(r);
  return r;
}

// A run of tiles of one (request, KV head), as a group works through it.
struct Piece {
  int b, h;
  Req r;
  int kt0;              // first key of tile 0 of the unit (or of the split)
  int t0, t1;           // tiles
  int slot;             // partial slot, or -1
};

template <typename T, int D, int NR>
__global__ void __launch_bounds__(kWarps * 32 * Smem<D, NR>::GROUPS,
                                  Smem<D, NR>::RESIDENT /
                                      Smem<D, NR>::GROUPS)
decode_fp4_kernel(const AttnParams p, int splits) {
  // the fold of the pieces may become resident once every CTA has started
  // (it waits for this grid before reading them)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // launched as a programmatic dependent of the kernel before it: nothing is
  // read before that one is complete (a no-op for a plain launch)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  using SM = Smem<D, NR>;
  using GE = Geo<D>;
  constexpr int MT = GE::MT;
  constexpr int KT = 16 * MT;            // keys of a warp's tile
  constexpr int KS = D / 16;             // k steps of S, and m tiles of O
  constexpr int KW = D / 32;             // words of a lane's K codes per key
  constexpr int NT = kWarps * 32;
  // (a cp.async chunk pair that straddles 32 bytes of shared memory costs two
  // L2 sectors: 0.226 against 0.216 ms on 8 x 131072 keys)
  extern __shared__ __align__(128) unsigned char all_smem[];
  constexpr int GR = SM::GROUPS;
  __shared__ long long scans[GR][kWarps];
  // what the inner loop seldom needs: the piece, and by packed row the token
  // of its request and its ALiBi slope (base 2)
  __shared__ Piece pieces[GR];
  __shared__ int row_toks[GR][16];
  __shared__ float row_slopes[GR][16];

  // The CTA's groups share nothing: each is what a CTA of its own would be
  // (one where the call is not a sequence).
  const int grp = threadIdx.x / NT, tid = threadIdx.x % NT;
  const int lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, c4 = lane & 3;
  unsigned char* const smem = all_smem + grp * SM::BYTES;
  long long* const scan = scans[grp];
  Piece& cur = pieces[grp];
  int* const row_tok = row_toks[grp];
  float* const row_slope = row_slopes[grp];
  auto group_sync = [&]() {
    asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "n"(NT) : "memory");
  };
  const int G = p.G;
  const bool sequence = p.sk_chunks > 0;
  // a share that begins inside a unit: the unit, its first token and rows
  int4* const marks = reinterpret_cast<int4*>(p.sk_marks);
  const float base_scale = p.scale * *p.k_scale * kLog2e;
  const float vscale = *p.v_scale;

  // ---- the group's first piece
  Piece pc;
  int left = 0;          // what of its share is past this piece's unit
  auto tiles_of = [&](const Req& r) {
    const int k0 = r.lo & ~15;
    return r.rows == 0 ? 0 : (r.hi - k0 - 1) / KT + 1;   // (1: no keys)
  };
  if (!sequence) {
    // one (request, piece, KV head) each; neighbours read the same pages
    pc.h = blockIdx.x % p.Hkv;
    const unsigned rest = blockIdx.x / p.Hkv;
    const int sp = rest % splits;
    pc.b = rest / splits;
    pc.r = request(p, pc.b, 8 * NR, sp == 0 && pc.h == 0 && tid == 0);
    if (pc.r.rows == 0) return;
    pc.slot = -1;
    if (p.chunk > 0) {
      // (the pieces are cut before the table's end clips the range)
      int kmin, kmax;
      key_range(pc.r.L, pc.r.q_len, 0, pc.r.q_len - 1, p.causal, p.wl, p.wr,
                kmin, kmax);
      const int ns = split_count(kmin, kmax, p.chunk, splits);
      if (sp >= ns) return;
      int lo, hi;
      split_bounds(kmin, kmax, p.chunk, ns, sp, lo, hi);
      pc.r.lo = lo;
      pc.r.hi = min(hi, pc.r.hi);
      no_keys(pc.r);
      pc.slot = sp;
    }
    pc.kt0 = pc.r.lo & ~15;
    pc.t0 = 0;
    pc.t1 = tiles_of(pc.r);
  } else {
    // The units (request, KV head) in order, each kUnitCost and its tiles
    // long, form a sequence of length N, of which every group takes an equal
    // run (the tiles in it).  Thread t adds up a run of requests; the one
    // whose run holds the start of the group's share finds it.
    const int per = (p.batch + NT - 1) / NT;
    const int b_lo = min(p.batch, tid * per);
    const int b_hi = min(p.batch, b_lo + per);
    long long sum = 0;
    Req mine_req{};
    for (int b = b_lo; b < b_hi; ++b) {
      mine_req = request(p, b, p.sk_rows, blockIdx.x == 0 && grp == 0);
      if (mine_req.rows > 0)
        sum += static_cast<long long>(kUnitCost + tiles_of(mine_req)) * p.Hkv;
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    group_sync();
    long long N = 0, excl = incl - sum;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) excl += scan[w];
      N += scan[w];
    }
    // at least kMinTiles tiles a group
    const long long Cs =
        max(1LL, min(static_cast<long long>(p.sk_chunks), N / kMinTiles));
    const int c = blockIdx.x * GR + grp;
    if (c >= Cs || N == 0) {
      if (tid == 0) marks[c] = make_int4(-1, 0, 0, 0);
      return;
    }
    auto bound = [&](long long k) -> long long {     // (32-bit where it can)
      return N < (1 << 16) ? static_cast<unsigned>(k * N) /
                                 static_cast<unsigned>(Cs)
                           : k * N / Cs;
    };
    const long long T0 = bound(c), T1 = bound(c + 1);
    if (sum > 0 && T0 >= excl && T0 < excl + sum) {
      long long at = excl;
      for (int b = b_lo; b < b_hi; ++b) {
        const Req r = per == 1 ? mine_req : request(p, b, p.sk_rows, false);
        const int n = r.rows > 0 ? kUnitCost + tiles_of(r) : 0;
        const long long all = static_cast<long long>(n) * p.Hkv;
        if (T0 < at + all) {
          const long long off = T0 - at;
          cur.b = b;
          cur.h = static_cast<int>(off < (1LL << 32)
                                       ? static_cast<unsigned>(off) /
                                             static_cast<unsigned>(n)
                                       : off / n);
          cur.t0 = static_cast<int>(off - static_cast<long long>(cur.h) * n);
          cur.r = r;
          break;
        }
        at += all;
      }
    }
    group_sync();
    pc = cur;
    pc.kt0 = pc.r.lo & ~15;
    const int n = tiles_of(pc.r);
    const long long end = T1 - T0 + pc.t0 - kUnitCost;   // from tile 0
    pc.t1 = static_cast<int>(min(static_cast<long long>(n), end));
    pc.t0 = max(0, pc.t0 - kUnitCost);
    left = static_cast<int>(end - n);
    if (pc.t1 <= 0) {                    // none of the unit's tiles
      if (tid == 0) marks[c] = make_int4(-1, 0, 0, 0);
      return;
    }
    group_sync();                     // (`cur` is written again)
    // a unit cut by the share's ends leaves its part in slot 2 c (begun
    // before) or 2 c + 1 (ending after)
    pc.slot = pc.t0 > 0 ? 2 * c : pc.t1 < n ? 2 * c + 1 : -1;
    if (tid == 0)
      marks[c] = make_int4(pc.t0 > 0 ? pc.b * p.Hkv + pc.h : -1, pc.r.q0,
                           pc.r.rows, 0);
  }
  // the piece after `a` in the group's share (left > kUnitCost)
  auto next_piece = [&](const Piece& a) {
    Piece x = a;
    if (++x.h == p.Hkv) {
      x.h = 0;
      do {
        ++x.b;
        x.r = request(p, x.b, p.sk_rows, false);
      } while (x.r.rows == 0 && x.b + 1 < p.batch);
      x.kt0 = x.r.lo & ~15;
    }
    const int n = tiles_of(x.r);
    x.t0 = 0;
    x.t1 = min(n, left - kUnitCost);
    left -= kUnitCost + n;
    x.slot = x.t1 < n ? 2 * static_cast<int>(blockIdx.x * GR + grp) + 1 : -1;
    return x;
  };

  // ---- copies: chunk lane + 32 i of a subtile's codes, and the scales of
  // one row (lanes 0 .. 15 of K, 16 .. 31 of V)
  const int kap = 4 * (g8 >> 1) + (g8 & 1);
  const uint32_t c_sb = static_cast<uint32_t>(p.c_sb);
  const uint32_t f_sb = static_cast<uint32_t>(p.f_sb);
  const uint32_t c_sr = static_cast<uint32_t>(p.c_sr);
  const uint32_t f_sr = static_cast<uint32_t>(p.f_sr);
  constexpr int NC = GE::SUB / 16 / 32;  // chunks of a lane
  constexpr int RI = 32 / GE::CPR;       // rows from one to the next
  const int cp_r = lane / GE::CPR, cp_c = lane % GE::CPR;
  const int64_t k_to_v = static_cast<const uint8_t*>(p.vc) -
                         static_cast<const uint8_t*>(p.kc);
  const uint32_t ring = smem_u32(smem) + SM::OFF_RING +
                        warp * (GE::STAGES * GE::STAGE);
  uint32_t k_dst[NC], v_dst[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    k_dst[i] = ring + GE::k_off(cp_r + RI * i, cp_c);
    v_dst[i] = ring + GE::OFF_V + GE::v_off(cp_r + RI * i, cp_c);
  }
  const uint32_t f_dst = ring + GE::OFF_KF + (lane >> 4) * 256 +
                         (lane & 15) * 16;

  // state of the copies: the piece's tiles warp, warp + kWarps, ..., as
  // subtiles s = 0 .. subs - 1; lane i holds subtile i of the current batch
  // of 32: its page and first row in it (-1: past the range, or a page
  // outside the cache, whose keys read as zero)
  int ids, rows0, ids_next, rows0_next;
  const uint8_t* KC;
  const uint8_t* SF;
  int mine, key0;
  auto fetch = [&](int s0, int b, int hi, int& id, int& row) {
    const int s = s0 + lane;
    const int k0 = key0 + (s / MT) * (kWarps * KT) + (s % MT) * 16;
    id = -1;
    row = 0;
    if (s >= mine * MT || k0 >= hi) return;
    const int j = p.bs_shift >= 0 ? k0 >> p.bs_shift : k0 / p.BS;
    row = k0 - j * p.BS;
    id = __ldg(p.block_table + static_cast<int64_t>(b) * p.bt_stride + j);
    if (id < 0 || id >= p.num_blocks) {
      atomicOr(p.err, kErrBadBlock);
      id = -1;
    }
  };
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
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
        cp_async_once(stage + k_dst[j] + i * GE::SUB, ks, n, policy);
        cp_async_once(stage + v_dst[j] + i * GE::SUB, ks + k_to_v, n, policy);
      }
      cp_async_n<D / 16>(stage + f_dst + i * (D / 16),
                         SF + static_cast<uint64_t>(page) * f_sb + row * f_sr,
                         id < 0 ? 0 : D / 16);
    }
  };
  // a piece's pages, then its first two tiles
  auto begin_pages = [&](const Piece& x) {
    const int n = x.t1 - x.t0;
    mine = n > warp ? (n - warp + kWarps - 1) / kWarps : 0;
    key0 = x.kt0 + (x.t0 + warp) * KT;
    KC = static_cast<const uint8_t*>(p.kc) +
         static_cast<int64_t>(x.h) * p.c_sh + cp_r * c_sr + 16 * cp_c;
    SF = (lane < 16 ? p.k_sf : p.v_sf) + static_cast<int64_t>(x.h) * p.f_sh +
         (lane & 15) * f_sr;
    fetch(0, x.b, x.r.hi, ids, rows0);
    fetch(32, x.b, x.r.hi, ids_next, rows0_next);
  };
  auto begin_copies = [&]() {
    if (mine > 0) issue(0, 0);
    cp_async_commit();
    if (mine > 1) issue(MT, GE::STAGE);
    cp_async_commit();
  };

  // the lane's reads of a stage: the swizzles make them constants apart but
  // for one bit (rows kap + 2 e of K, rows 4 c4 + e of V)
  const uint32_t k_rd = ring + GE::k_off(kap, D == 64 ? c4 >> 1 : c4) +
                        (D == 64 ? 8 * (c4 & 1) : 0);
  const uint32_t k_rd1 =
      ring + (D == 64    ? GE::k_off(kap + 2, c4 >> 1) + 8 * (c4 & 1)
              : D == 128 ? GE::k_off(kap + 2, c4)
                         : GE::k_off(kap, 4 + c4));
  const uint32_t v_rd =
      ring + GE::OFF_V +
      (D == 64 ? GE::v_off(4 * c4, g8 >> 2) + 4 * (g8 & 3)
               : GE::v_off(4 * c4, g8 >> 1) + 8 * (g8 & 1));
  const uint32_t v_rd1 =
      ring + GE::OFF_V +
      (D == 64    ? GE::v_off(4 * c4 + 1, g8 >> 2) + 4 * (g8 & 3)
       : D == 128 ? GE::v_off(4 * c4 + 1, g8 >> 1) + 8 * (g8 & 1)
                  : GE::v_off(4 * c4, 4 + (g8 >> 1)) + 8 * (g8 & 1));
  const uint32_t f_rd = ring + GE::OFF_KF + kap * 16 +
                        (D == 64 ? c4 : 2 * c4);
  const uint32_t vf_rd = ring + GE::OFF_VF +
                         (D == 64 ? 64 * c4 + (g8 >> 1) : (lane & 15) * 16);
  auto k_at = [&](uint32_t stage, int e, int q) -> uint32_t {
    if (D == 256) return (q ? k_rd1 : k_rd) + stage + e * (2 * GE::RB);
    return (e ? k_rd1 : k_rd) + stage;
  };
  auto v_at = [&](uint32_t stage, int e, int v) -> uint32_t {
    if (D == 256) return (v ? v_rd1 : v_rd) + stage + e * GE::RB;
    if (D == 128)
      return ((e & 1) ? v_rd1 : v_rd) + stage + (e >> 1) * (2 * GE::RB);
    // (rows e ^ c4 of the four)
    return v_rd + stage + (static_cast<int>((e ^ c4) - c4) * GE::RB);
  };

  if (tid < 16) row_tok[tid] = tid / G;
  const bool plain = p.softcap <= 0.f && p.alibi == nullptr;
  const float cap_t = p.softcap * kLog2e;
  const float cap_u = p.softcap > 0.f ? 2.f / p.softcap : 0.f;

  // ---- queries: lane (g8, c4) takes row g8 (and g8 + 8), the dimensions of
  // its K run.  A bf16 row is scaled by the power of two that puts its
  // largest magnitude in [2^14, 2^15): exact in f16 for the elements above
  // 2^-31 of the largest, and off by at most 2^-39 of it for smaller ones; the
  // factor joins the row's logit scale.
  uint4 raw[NR][KW];
  auto load_queries = [&](const Piece& x, int rows) {
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = g8 + 8 * n;
#pragma unroll
      for (int i = 0; i < KW; ++i) raw[n][i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int t = r / G;
        const T* src = static_cast<const T*>(p.q) +
                       static_cast<int64_t>(x.r.q0 + t) * p.q_st +
                       static_cast<int64_t>(x.h * G + r - t * G) * p.q_sh;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          // word i of the run: 8 dimensions (D = 256: two runs of 4 words)
          const int d = D == 256 ? 128 * (i >> 2) + 32 * c4 + 8 * (i & 3)
                                 : 8 * KW * c4 + 8 * i;
          raw[n][i] = *reinterpret_cast<const uint4*>(src + d);
        }
      }
    }
  };

  begin_pages(pc);
  load_queries(pc, pc.r.rows);
  begin_copies();
  for (;;) {
    if (tid == 0) cur = pc;
    if (p.alibi && tid < 16)
      row_slope[tid] =
          tid < pc.r.rows ? p.alibi[pc.h * G + tid % G] * kLog2e : 0.f;
    uint64_t row_scale[NR];   // logit scales (base 2), rows 2 c4, 2 c4 + 1
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float qmul = 1.f, back = 1.f;
      if constexpr (!std::is_same<T, __half>::value) {
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          float x[8];
          widen8<T>(raw[n][i], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int shift = 0;
        if (mx > 0.f) {
          shift = static_cast<int>((__float_as_uint(mx) >> 23) & 0xff) - 141;
          shift = max(-100, min(113, shift));
        }
        qmul = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
        back = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
      }
      row_scale[n] =
          pair(__shfl_sync(0xffffffffu, back, 8 * c4) * base_scale,
               __shfl_sync(0xffffffffu, back, 8 * c4 + 4) * base_scale);
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint32_t w[4] = {raw[n][i].x, raw[n][i].y, raw[n][i].z,
                               raw[n][i].w};
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[e] = std::is_same<T, __half>::value
                     ? w[e]
                     : pack2<__half>(elem_f32<T>(w[e], 0) * qmul,
                                     elem_f32<T>(w[e], 1) * qmul);
        // 8 dimensions: the B operands of k steps 2 i and 2 i + 1
        if (KW < kWarps || (i & (kWarps - 1)) == warp)
          reinterpret_cast<uint4*>(smem)[(i * NR + n) * 32 + lane] =
              make_uint4(f[0], f[1], f[2], f[3]);
      }
    }
    group_sync();

    // my tiles i0 <= it < i1 are seen whole by every row
    int i0, i1;
    {
      int full_lo = pc.r.lo, full_hi = pc.r.hi;
      const int p_lo = pc.r.L - pc.r.q_len, p_hi = pc.r.L - 1;
      if (p.wl >= 0) full_lo = max(full_lo, p_hi - p.wl);
      if (p.causal) full_hi = min(full_hi, p_lo + 1);
      if (p.wr >= 0) full_hi = min(full_hi, p_lo + p.wr + 1);
      constexpr int STEP = kWarps * KT;
      i0 = max(0, (full_lo - key0 + STEP - 1) / STEP);
      i1 = full_hi - key0 >= KT ? (full_hi - key0 - KT) / STEP + 1 : 0;
    }
    const volatile Piece* cold = &cur;

    float o[KS][NR][4];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int n = 0; n < NR; ++n)
        o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    float m[NR][2];                    // the references
    uint64_t l[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n] = pair(0.f, 0.f);
    }

    for (int it = 0; it < mine; ++it) {
      const uint32_t stage = (it & 1) * GE::STAGE;
      cp_async_wait<1>();
      __syncwarp();
      // ---- S^T
      float sc[MT][NR][4];
      uint32_t kw[MT][2][KW], kf[MT][2];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t fs = f_rd + stage + e * 32 + i * (D / 16);
          if constexpr (D == 64) {
            const uint2 v = lds64(k_at(stage, e, 0) + i * GE::SUB);
            kw[i][e][0] = v.x;
            kw[i][e][1] = v.y;
            kf[i][e] = lds8(fs);
          } else {
            kf[i][e] = 0;
#pragma unroll
            for (int q = 0; q < D / 128; ++q) {
              const uint4 v = lds128(k_at(stage, e, q) + i * GE::SUB);
              kw[i][e][4 * q] = v.x;
              kw[i][e][4 * q + 1] = v.y;
              kw[i][e][4 * q + 2] = v.z;
              kw[i][e][4 * q + 3] = v.w;
              kf[i][e] |= lds16(fs + 8 * q) << (16 * q);
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
          qb[n] =
              reinterpret_cast<const uint4*>(smem)[(w * NR + n) * 32 + lane];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t a[4], c[4];
          e2m1x8_to_f16(kw[i][0][w], a[0], a[1], a[2], a[3]);
          e2m1x8_to_f16(kw[i][1][w], c[0], c[1], c[2], c[3]);
          uint32_t fa, fc;
          if constexpr (D == 64) {
            fa = spread(fk[i][0][0], 0);
            fc = spread(fk[i][0][0], 1);
          } else {
            fa = spread(fk[i][0][w >> 2], w & 2);
            fc = spread(fk[i][1][w >> 2], w & 2);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = hmul2_u32(a[e], fa);
            c[e] = hmul2_u32(c[e], fc);
          }
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            if (w == 0)
              mma_first(sc[i][n], a[0], c[0], a[1], c[1], qb[n].x, qb[n].y);
            else
              mma(sc[i][n], a[0], c[0], a[1], c[1], qb[n].x, qb[n].y);
            mma(sc[i][n], a[2], c[2], a[3], c[3], qb[n].z, qb[n].w);
          }
        }
      }
      // ---- logits (base 2) and masks
      const bool interior = it >= i0 && it < i1;
      float mx[NR][2];
      // (the products are rounded here, once: a fused multiply-add with the
      // maximum would differ from it by half an ulp of the logit, which may
      // be far above 1)
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          float* x = sc[i][n];
          unpair(mul2(pair(x[0], x[1]), row_scale[n]), x[0], x[1]);
          unpair(mul2(pair(x[2], x[3]), row_scale[n]), x[2], x[3]);
        }
      if (!plain) {
        if (p.softcap > 0.f) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                sc[i][n][e] = soft_cap(sc[i][n][e], cap_t, cap_u);
        }
        if (p.alibi) {
          const int at0 = cold->r.L - cold->r.q_len -
                          (key0 + it * (kWarps * KT) + kap);
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = 8 * n + 2 * c4 + e;
              const float sl = row_slope[r];
              const int at = at0 + row_tok[r];
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                sc[i][n][e] -= sl * fabsf(static_cast<float>(at - 16 * i));
                sc[i][n][e + 2] -=
                    sl * fabsf(static_cast<float>(at - 16 * i - 2));
              }
            }
        }
      }
      if (!interior) {
        const int k0 = key0 + it * (kWarps * KT) + kap;
        const int ctx = cold->r.L - cold->r.q_len;
        const int rows = cold->r.rows;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // keys [from, to) that this row sees
            const int r = 8 * n + 2 * c4 + e;
            const int at = ctx + row_tok[r];
            int from = cold->r.lo, to = cold->r.hi;
            if (p.causal) to = min(to, at + 1);
            if (p.wr >= 0) to = min(to, at + p.wr + 1);
            if (p.wl >= 0) from = max(from, at - p.wl);
            if (r >= rows) to = from;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int f = 0; f < 4; f += 2) {
                const int key = k0 + 16 * i + f;
                if (key < from || key >= to) sc[i][n][e + f] = -INFINITY;
              }
          }
      }
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[n][e] = fmaxf(sc[0][n][e], sc[0][n][e + 2]);
#pragma unroll
          for (int i = 1; i < MT; ++i)
            mx[n][e] = fmaxf(mx[n][e], fmaxf(sc[i][n][e], sc[i][n][e + 2]));
        }
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          raise = raise || mx[n][e] - m[n][e] > kTop;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = mx[n][e];
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            // (by the row's own logits alone: its bits must not depend on
            // the rows beside it, which may be padding; at logits of 2^27
            // t - kRoom may round to t - 16, out of f16's range)
            if (t - m[n][e] > kTop) {
              const float low = t - kRoom;
              t = t - low > kTop ? t : low;
            } else {
              t = m[n][e];
            }
            al[e] = t == m[n][e] ? 1.f : ex2(m[n][e] - t);
            m[n][e] = t;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              o[i][n][e] *= al[e];
              o[i][n][e + 2] *= al[e];
            }
          }
          l[n] = mul2(l[n], pair(al[0], al[1]));
        }
      }
      // P and its sums, and P^T as the B operand of each subtile
      uint32_t pb[MT][NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float base[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0],
                               m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          float* x = sc[i][n];
          // (a packed sum could be fused with the product above)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = ex2(__fsub_rn(x[e], base[e & 1]));
          l[n] = add2(l[n], add2(pair(x[0], x[1]), pair(x[2], x[3])));
          // P rounds to f16 for the MMA, the sums keep the float32 values
          // (see the head of this file)
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
            f[e] = lds8(vf_rd + stage + e * 16 + i * 4);
          vf[i][0] = __byte_perm(__byte_perm(f[0], f[1], 0x40),
                                 __byte_perm(f[2], f[3], 0x40), 0x5410);
        }
      } else {
        // rows are keys, columns groups (of two subtiles at D = 128)
        uint32_t d0, d1;
        ldmatrix_b8_trans(vf_rd + stage, d0, d1);
        vf[0][0] = d0;
        vf[MT - 1][VG - 1] = d1;
      }
      if (!interior) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          // keys outside [lo, hi): a scale of 0
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + it * (kWarps * KT) + 16 * i + 4 * c4 + e;
            if (key < cold->r.lo || key >= cold->r.hi)
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
                  const int at = cold->r.L - cold->r.q_len +
                                 row_tok[8 * n + 2 * c4 + e];
                  bool hit = false;
                  for (int j = 0; j < 16; ++j) {
                    const int key = key0 + it * (kWarps * KT) + 16 * i + j;
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
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int v = 0; v < VG; ++v) {
          const uint32_t s01 = e4m3x2_to_f16(vf[i][v]);
          const uint32_t s23 = e4m3x2_to_f16(vf[i][v] >> 16);
          // the lane's run of the four keys' rows: 16 dimensions (D = 64: 8)
          constexpr int RW = D == 64 ? 1 : 2;
          uint32_t vw[4][RW];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (D == 64) {
              vw[e][0] = lds32(v_at(stage, e, 0) + i * GE::SUB);
            } else {
              const uint2 x = lds64(v_at(stage, e, v) + i * GE::SUB);
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
          fetch(s_new + 32, cold->b, cold->r.hi, ids_next, rows0_next);
        }
        issue(s_new, stage);
      }
      cp_async_commit();
    }

    // ---- the next piece's pages and copies begin before the end of this one
    const Piece done = cur;
    const bool more_pieces = left > kUnitCost;
    if (more_pieces) {
      pc = next_piece(done);
      begin_pages(pc);
    }
    float sum[NR][2];                    // of the whole rows
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      unpair(l[n], sum[n][0], sum[n][1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = sum[n][e];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        sum[n][e] = t;
      }
    }
    // the warps' states meet pairwise: the upper half's go through shared
    // memory into the lower half's registers
    float4* state = reinterpret_cast<float4*>(
        smem + SM::OFF_S + (warp & (kWarps / 2 - 1)) * SM::SBYTES) + lane;
    auto put = [&](float4* dst) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int n = 0; n < NR; ++n)
          dst[(i * NR + n) * 32] =
              make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
#pragma unroll
      for (int n = 0; n < NR; ++n)
        dst[(KS * NR + n) * 32] =
            make_float4(m[n][0], m[n][1], sum[n][0], sum[n][1]);
    };
    auto join = [&](const float4* src) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float4 t = src[(KS * NR + n) * 32];
        const float tm[2] = {t.x, t.y}, tl[2] = {t.z, t.w};
        float f[2], g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float M = fmaxf(m[n][e], tm[e]);
          // (a warp that saw nothing but NaN keeps its NaN sum)
          f[e] = m[n][e] == -INFINITY ? (sum[n][e] == 0.f ? 0.f : 1.f)
                                      : ex2(m[n][e] - M);
          g[e] = tm[e] == -INFINITY ? (tl[e] == 0.f ? 0.f : 1.f)
                                    : ex2(tm[e] - M);
          sum[n][e] = fold2(f[e], sum[n][e], g[e], tl[e]);
          m[n][e] = M;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const float4 v = src[(i * NR + n) * 32];
          o[i][n][0] = fold2(f[0], o[i][n][0], g[0], v.x);
          o[i][n][1] = fold2(f[1], o[i][n][1], g[1], v.y);
          o[i][n][2] = fold2(f[0], o[i][n][2], g[0], v.z);
          o[i][n][3] = fold2(f[1], o[i][n][3], g[1], v.w);
        }
      }
    };
    if (warp >= 2) put(state);
    if (more_pieces) begin_copies();
    group_sync();
    if (warp < 2) join(state);
    if (warp == 1) put(state);
    group_sync();
    if (warp == 0) {
      join(state + SM::SBYTES / 16);
      // lane (g8, c4) holds, of rows 2 c4 and 2 c4 + 1, the runs of 16 (D =
      // 64: 8) dimensions at 16 g8 of each 128 (D = 64: 8 g8)
      constexpr int RUN = D == 64 ? 8 : 16;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * c4 + e;
          if (r >= done.r.rows) continue;
          const int tok = done.r.q0 + row_tok[r];
          const int hq = done.h * G + r - row_tok[r] * G;
          float inv, lse;
          // (O and the sum are relative to the reference, kRoom below)
          finish(m[n][e] + kRoom, sum[n][e] * kUnroom,
                 done.slot >= 0 ? nullptr : p.sinks, hq, &inv, &lse);
          inv *= kUnroom * vscale;
          if (done.slot >= 0) {
            // partial rows: [slot][row] of the shares, or of the split
            int64_t row = static_cast<int64_t>(done.slot) * p.sk_rows + r;
            int64_t at = row;
            if (!sequence) {
              const int64_t pr = part_row(p.part_tpr, done.b, done.r.q0, tok);
              row = (static_cast<int64_t>(done.slot) * p.part_rows + pr) *
                        p.Hq + hq;
              at = (static_cast<int64_t>(done.slot) * p.Hq + hq) *
                       p.part_rows + pr;
            }
            float* dst = p.part_o + row * D + RUN * g8;
#pragma unroll
            for (int i = 0; i < KS; i += 2)
              *reinterpret_cast<float4*>(dst + 128 * (i >> 3) + 2 * (i & 7)) =
                  make_float4(o[i][n][e] * inv, o[i][n][e + 2] * inv,
                              o[i + 1][n][e] * inv, o[i + 1][n][e + 2] * inv);
            if (g8 == 0) p.part_lse[at] = lse;
          } else {
            T* dst = static_cast<T*>(p.out) +
                     static_cast<int64_t>(tok) * p.o_st +
                     static_cast<int64_t>(hq) * p.o_sh + RUN * g8;
#pragma unroll
            for (int i = 0; i < KS; i += 4)
              *reinterpret_cast<uint4*>(dst + 128 * (i >> 3) + 2 * (i & 7)) =
                  make_uint4(
                      pack2<T>(o[i][n][e] * inv, o[i][n][e + 2] * inv),
                      pack2<T>(o[i + 1][n][e] * inv, o[i + 1][n][e + 2] * inv),
                      pack2<T>(o[i + 2][n][e] * inv, o[i + 2][n][e + 2] * inv),
                      pack2<T>(o[i + 3][n][e] * inv,
                               o[i + 3][n][e + 2] * inv));
            if (p.lse && g8 == 0)
              p.lse[static_cast<int64_t>(hq) * p.total_q + tok] = lse;
          }
        }
    }
    if (!more_pieces) break;
    load_queries(pc, pc.r.rows);
    // (the queries and the piece are read: two barriers ago)
  }
  cp_async_wait<0>();
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

// Join the parts of the units that the ends of the shares cut.  A unit
// in np parts has its first in slot 2 (s - 1) + 1 of share s - 1 (where it
// begins) and the others in slots 2 s, 2 (s + 1), ... of the shares that mark
// it as begun before.  Block c stands at the start of share c: the np - 1
// blocks inside a unit divide its (row, 4 columns) items, and where a block
// has threads over, groups of them take every kg-th part.
template <typename T, int D>
__global__ void __launch_bounds__(kFoldThreads)
fold_kernel(const AttnParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int HALF = kFoldThreads / 2;
  __shared__ unsigned others[kFoldThreads / 32];
  __shared__ float row_base[16], row_inv[16], row_lse[16];
  __shared__ float4 part[kFoldThreads];
  const int4* const marks = reinterpret_cast<const int4*>(p.sk_marks);
  const int c = blockIdx.x + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the run of shares around c that mark its unit: the lower half of the
  // threads looks back, the upper half on (the first step's marks load beside
  // c's own)
  const int dir = tid < HALF ? -1 : 1, i_th = tid < HALF ? tid : tid - HALF;
  auto unit_at = [&](int at) {
    return at < 0 || at >= p.sk_chunks ? -1 : marks[at].x;
  };
  const int4 mark = marks[c];
  int near = unit_at(c + dir * (1 + i_th));
  const int u = mark.x;
  if (u < 0) return;
  int first = c, last = c;
  {
    bool open[2] = {true, true};
    for (int step = 1;; step += HALF) {
      if (step > 1) near = unit_at(c + dir * (step + i_th));
      const unsigned o = __ballot_sync(0xffffffffu, near != u);
      if (lane == 0) others[warp] = o;
      __syncthreads();
      int reach[2] = {HALF, HALF};
#pragma unroll
      for (int w = HALF / 32 - 1; w >= 0; --w)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const unsigned m = others[d * (HALF / 32) + w];
          if (m) reach[d] = 32 * w + __ffs(m) - 1;
        }
      if (open[0]) first -= reach[0];
      if (open[1]) last += reach[1];
      open[0] = open[0] && reach[0] == HALF;
      open[1] = open[1] && reach[1] == HALF;
      if (!open[0] && !open[1]) break;
      __syncthreads();
    }
  }
  const int np = last - first + 2;       // parts, shares first - 1 .. last
  const int h = u % p.Hkv, q0 = mark.y, rows = mark.z;
  // The first part is worked on by itself, so that the slots of the others are
  // evenly spaced.
  const int begun = 2 * (first - 1) + 1;
  auto later = [&](int k) { return 2 * (first - 1 + k); };
  auto row_of = [&](int slot, int r) -> int64_t {
    return static_cast<int64_t>(slot) * p.sk_rows + r;
  };
  // this block's items
  const int all = rows * (D / 4);
  const int per = (all + np - 2) / (np - 1);
  const int i0 = (c - first) * per, i1 = min(all, i0 + per);
  if (i0 >= i1) return;
  const int width = min(i1 - i0, kFoldThreads);
  const int kg = kFoldThreads / width;
  const int grp = tid / width, in = tid - grp * width;
  // the thread's first values are on their way while the rows' sums are taken
  const int mine_at = grp == 0 ? begun : later(grp);
  float4 ahead = make_float4(0.f, 0.f, 0.f, 0.f);
  float ahead_lse = -INFINITY;
  if (grp < kg && grp < np) {
    const int i = i0 + in, r = i / (D / 4);
    const int64_t at = row_of(mine_at, r);
    ahead = *reinterpret_cast<const float4*>(p.part_o + at * D +
                                             (i - r * (D / 4)) * 4);
    ahead_lse = p.part_lse[at];
  }
  const int r0 = i0 / (D / 4), r1 = (i1 - 1) / (D / 4);
  for (int r = r0 + warp; r <= r1; r += kFoldThreads / 32) {
    const float lse0 = p.part_lse[row_of(begun, r)];
    const float mine =
        lane + 1 < np ? p.part_lse[row_of(later(lane + 1), r)] : -INFINITY;
    float M = fmaxf(lse0, mine);
    for (int k = lane + 33; k < np; k += 32)
      M = fmaxf(M, p.part_lse[row_of(later(k), r)]);
#pragma unroll
    for (int o = 16; o; o >>= 1)
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.f : M * kLog2e;
    float sum = ex2(mine * kLog2e - base);
    for (int k = lane + 33; k < np; k += 32)
      sum += ex2(p.part_lse[row_of(later(k), r)] * kLog2e - base);
    if (lane == 0) sum += ex2(lse0 * kLog2e - base);
#pragma unroll
    for (int o = 16; o; o >>= 1)
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      row_base[r] = base;
      finish(M == -INFINITY ? M : base, sum, p.sinks, h * p.G + r % p.G,
             &row_inv[r], &row_lse[r]);
    }
  }
  __syncthreads();
  for (int ib = i0; ib < i1; ib += width) {
    const int i = ib + in;
    const bool on = i < i1 && grp < kg;
    const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      const float base = row_base[r];
      auto add = [&](float lse, const float4& v) {
        const float w = ex2(lse * kLog2e - base);
        if (w == 0.f) return;                               // (-inf)
        acc.x += w * v.x;
        acc.y += w * v.y;
        acc.z += w * v.z;
        acc.w += w * v.w;
      };
      auto load = [&](int slot) {
        const int64_t at = row_of(slot, r);
        const float4 v =
            *reinterpret_cast<const float4*>(p.part_o + at * D + col);
        add(p.part_lse[at], v);
      };
      if (ib == i0)
        add(ahead_lse, ahead);
      else if (grp < np)
        load(mine_at);
#pragma unroll 4
      for (int k = grp + kg; k < np; k += kg) load(later(k));
    }
    if (kg > 1) {
      __syncthreads();
      part[tid] = acc;
      __syncthreads();
      if (grp == 0)
        for (int g = 1; g < kg; ++g) {
          const float4 v = part[g * width + in];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
    }
    if (on && grp == 0) {
      const float inv = row_inv[r];
      const int t = q0 + r / p.G, hq = h * p.G + r % p.G;
      T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(t) * p.o_st +
               static_cast<int64_t>(hq) * p.o_sh + col;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack2<T>(acc.x * inv, acc.y * inv),
                     pack2<T>(acc.z * inv, acc.w * inv));
      if (p.lse && col == 0)
        p.lse[static_cast<int64_t>(hq) * p.total_q + t] = row_lse[r];
    }
  }
}

template <typename T, int D, int NR>
cudaError_t launch(const AttnParams& p, int splits, bool pdl,
                   cudaStream_t stream) {
  using SM = Smem<D, NR>;
  auto kern = decode_fp4_kernel<T, D, NR>;
  cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(kern),
                              SM::GROUPS * SM::BYTES);
  if (e != cudaSuccess) return e;
  // a share a group; else one group a unit
  const int groups = p.sk_chunks > 0 ? SM::GROUPS : 1;
  const int64_t ctas =
      p.sk_chunks > 0 ? p.sk_chunks / groups
                      : static_cast<int64_t>(p.batch) * splits * p.Hkv;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  note_launch();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kWarps * 32 * groups);
  cfg.dynamicSmemBytes = SM::BYTES * groups;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, p, splits);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D>
cudaError_t dispatch_rows(const AttnParams& p, int splits, bool pdl,
                          cudaStream_t stream) {
  const bool one = decode_fp4_rows(p.sk_rows) == 8;
  return one ? launch<T, D, 1>(p, splits, pdl, stream)
             : launch<T, D, 2>(p, splits, pdl, stream);
}

template <typename T>
cudaError_t dispatch(const AttnParams& p, int D, int splits, bool pdl,
                     cudaStream_t stream) {
  switch (D) {
    case 64: return dispatch_rows<T, 64>(p, splits, pdl, stream);
    case 128: return dispatch_rows<T, 128>(p, splits, pdl, stream);
    case 256: return dispatch_rows<T, 256>(p, splits, pdl, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dfp4

int decode_fp4_rows(int rows) { return rows <= 8 ? 8 : 16; }

int decode_fp4_resident(int D, int rows) {
  const bool one = decode_fp4_rows(rows) == 8;
  switch (D) {
    case 64:
      return one ? dfp4::Smem<64, 1>::RESIDENT : dfp4::Smem<64, 2>::RESIDENT;
    case 128:
      return one ? dfp4::Smem<128, 1>::RESIDENT : dfp4::Smem<128, 2>::RESIDENT;
    default:
      return one ? dfp4::Smem<256, 1>::RESIDENT : dfp4::Smem<256, 2>::RESIDENT;
  }
}

cudaError_t launch_decode_attn_fp4(const AttnParams& p, int D, bool bf16,
                                   int splits, bool pdl,
                                   cudaStream_t stream) {
  AttnParams a = p;
  a.sk_chunks = 0;
  return bf16 ? dfp4::dispatch<__nv_bfloat16>(a, D, splits, pdl, stream)
              : dfp4::dispatch<__half>(a, D, splits, pdl, stream);
}

cudaError_t launch_decode_attn_fp4_shares(const AttnParams& p, int D,
                                          bool bf16, int shares, bool pdl,
                                          void* scratch,
                                          cudaStream_t stream) {
  AttnParams a = p;
  char* ws = static_cast<char*>(scratch);
  const size_t slots = static_cast<size_t>(2) * shares;
  a.chunk = 0;
  a.sk_chunks = shares;
  a.part_o = reinterpret_cast<float*>(ws);
  ws += dfp4::up256(slots * p.sk_rows * D * 4);
  a.part_lse = reinterpret_cast<float*>(ws);
  ws += dfp4::up256(slots * p.sk_rows * 4);
  a.sk_marks = reinterpret_cast<int2*>(ws);
  cudaError_t e = bf16 ? dfp4::dispatch<__nv_bfloat16>(a, D, 1, pdl, stream)
                       : dfp4::dispatch<__half>(a, D, 1, pdl, stream);
  if (e != cudaSuccess || shares < 2) return e;
  note_launch();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(shares - 1));
  cfg.blockDim = dim3(dfp4::kFoldThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  auto go = [&](auto kern) { return cudaLaunchKernelEx(&cfg, kern, a); };
  switch (D) {
    case 64:
      e = bf16 ? go(dfp4::fold_kernel<__nv_bfloat16, 64>)
               : go(dfp4::fold_kernel<__half, 64>);
      break;
    case 128:
      e = bf16 ? go(dfp4::fold_kernel<__nv_bfloat16, 128>)
               : go(dfp4::fold_kernel<__half, 128>);
      break;
    default:
      e = bf16 ? go(dfp4::fold_kernel<__nv_bfloat16, 256>)
               : go(dfp4::fold_kernel<__half, 256>);
      break;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t decode_fp4_shares_bytes(int D, int shares, int rows) {
  const size_t slots = static_cast<size_t>(2) * shares;
  return dfp4::up256(slots * rows * D * 4) + dfp4::up256(slots * rows * 4) +
         dfp4::up256(static_cast<size_t>(shares) * 16);
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
