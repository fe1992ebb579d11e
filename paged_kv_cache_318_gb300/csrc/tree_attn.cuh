// Attention of a tree of drafted tokens over a paged cache (tcgen05 + TMEM +
// TMA): the kernel, for 16-bit caches (tree_attn.cu) and for caches of codes
// (tree_codes.cu).
//
// Request b has n rows (row 0: the last certain token; the others drafted,
// each with an earlier row as its parent) and L keys, the rows' own keys last:
// row a's key is ctx + a, ctx = L - n.  Row i, depth(i) steps below row 0, sits
// at position ctx + depth(i) and sees key j < ctx unless the window hides it
// (j < position - window), its own key and those of its ancestors at most
// `window` steps away.  Everything else is the attention of the other kernels:
// s = scale q k, soft-cap, softmax with an optional sink, natural LSE.
//
// A unit is one (request, KV head, block of packed rows): packed row R is row
// R / G, query head g G + R % G, so the G heads of a KV head share every K/V
// tile; a block holds 256 packed rows (128 at head size 256).  Almost all keys
// lie before the draft and need no mask, and what bounds the usual tree (up to
// 128 packed rows) is reading them once.  So the units' key tiles form one
// sequence and every CTA (one per SM) takes an equal share of it, whatever the
// lengths; a unit that a share's end cuts leaves one fp32 partial per piece,
// and fold_kernel joins the pieces by their LSEs.
//
// Inside a CTA two streams x = 0, 1 (softmax warps 4 x .. 4 x + 3, a score
// buffer S_x and an accumulator O_x in tensor memory) keep the tensor core
// busy: while one stream's softmax works, the other's products run.
//   up to 128 rows   both streams hold the same rows; stream x takes every
//                    other key tile, and the two states meet at the piece's
//                    end (each thread reads both accumulators)
//   more             stream x holds rows 128 x .. and both take every tile
// The probabilities overwrite the scores as packed 16-bit pairs and feed P V
// from tensor memory.  Head size 256 has room for one accumulator: one stream
// of 64-key tiles with two score buffers, S of the next tile running under the
// softmax.
//
// K and V tiles share one ring in the order in which the products take them
// (place_k, place_v), so that the stages not in use are all prefetch.  Each
// stream has an MMA warp of its own: one warp for both, which also kept the
// order across the pieces' borders, ran 3000 clocks of its own instructions a
// tile, more than the tile's share of HBM (64 KB: 2800).
//
// Measured (32/8 heads of 128 unless said; time on the device, launches in a
// graph): 64 requests of 16 rows over 512 to 4096 keys 122 us, 5.5 TB/s while
// the kernel runs; one of 61 rows over 16384 keys 30 us; 4 of 64 rows over 65536
// keys, 64/8 heads, 410 to 450 us, 1220 to 1340 TFLOP/s; 124 of 2 to 8 rows,
// windows of 4095 keys, 16/8 heads of 256, 565 us, 6.7 TB/s; 48 of 12 rows over
// 4364 keys: 16 bits 158 us, E4M3 158, 4 bits 187.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <atomic>
#include <type_traits>

#include "pkv_common.cuh"
#include "tcgen05_util.cuh"
#include "tma_util.cuh"

namespace pkv {
namespace tree {

using namespace tc;

constexpr int kNoParent = 255;         // in the byte list of parents
static_assert(PKV_TREE_MAX_ROWS <= 256, "parents are bytes");

// Probabilities are held relative to 2^-OFF of the row's reference maximum,
// and the reference moves when the maximum grows by more than THR (log2
// units), so a probability stays below 2^(THR + OFF).  bf16 has float32's
// range.  f16 ends at 2^16 above and 2^-24 below: with OFF = 11 weights keep
// all their bits down to 2^-25 of the largest and vanish below 2^-35 (with
// OFF = 0, keys 16.6 nats below an attention sink would vanish).
// They round to T because the tensor cores take V's type on both sides: half a
// step of each, which moves an output by at most eps / 2 sum p |v| (measured:
// the output is 1.35 times as far from float64 as one that only rounds itself).
// Their sum is of the unrounded ones, in float32.
template <typename T>
struct Range {
  static constexpr float THR = 8.f, OFF = 0.f;
};
template <>
struct Range<__half> {
  static constexpr float THR = 4.f, OFF = 11.f;
};

// What the cache holds: 16-bit values, E4M3 codes, or E2M1 codes with E4M3
// block scales.
enum Kv { kValues = 0, kE4m3 = 1, kE2m1 = 2 };

template <int D, int KV>
struct Cfg {
  static constexpr int NX = D == 256 ? 1 : 2;          // streams
  static constexpr int BN = D == 256 ? 64 : 128;       // keys of a tile
  static constexpr int NCB = D / 64;                   // 64-column blocks
  static constexpr int ROWS = NX * BM;                 // rows of a block
  static constexpr int STAGE = BN * D * 2;             // one K or V tile
  static constexpr int STAGES =
      KV == kE2m1 ? (D == 64 ? 6 : 4) : KV ? (D == 64 ? 6 : 3) : D == 64 ? 8 : 5;
  static constexpr int Q_TILE = BM * D * 2;
  // tensor memory: (S_x, O_x) per stream, or (S_0, S_1, O)
  static constexpr int S_STEP = NX == 2 ? BN + D : BN;
  static constexpr int O_COL = NX == 2 ? BN : 2 * BN;  // of stream 0
  static_assert(NX * (BN + D) + (NX == 1 ? BN : 0) <= 512, "TMEM columns");
  static constexpr int SM_WARPS = 4 * NX;
  // the MMA warps (one per stream) on the schedulers that have the least to do
  // for a small tree, whose rows are those of softmax warps 0, 1, 4 and 5
  static constexpr int DEAL_WARP = SM_WARPS, LOAD_WARP = SM_WARPS + 1,
                       MMA_WARP = SM_WARPS + 2;
  // codes: the warps that copy and widen them, in place of the loader
  static constexpr int CODE_WARP = SM_WARPS + 4,
                       CODE_WARPS = KV ? 8 : 0,
                       GROUP = CODE_WARPS / 2;   // warps that share a tile
  static constexpr int THREADS = (SM_WARPS + 4 + CODE_WARPS) * 32;
  // warps that take every piece and are done with it at once
  static constexpr int TAKERS = 1 + NX + CODE_WARPS;
  // tiles of codes on their way
  static constexpr int CODE_ROW = KV == kE4m3 ? D : D / 2;   // bytes
  static constexpr int CODE_TILE = BN * CODE_ROW;
  static constexpr int AHEAD = KV == 0 ? 0 : 4;
  // The two groups that widen codes take the ring's places in turn.  A waiter
  // sees one parity, so each phase of a barrier has to be waited for by one
  // group: with an odd number of stages there are two `empty` barriers a stage,
  // each for one group's turns.
  static constexpr int EMPTIES = KV && STAGES % 2 ? 2 : 1;
  static_assert(AHEAD % 2 == 0, "a group keeps to its places of codes");
  static constexpr int SLOTS = 2;                      // pieces in flight
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = OFF_Q + NX * Q_TILE;
  static constexpr int OFF_CODES = OFF_RING + STAGES * STAGE;
  static constexpr int OFF_BAR = OFF_CODES + AHEAD * CODE_TILE;
  static constexpr int BAR_BYTES =
      (8 * (((NX == 2 ? 3 : 1) + EMPTIES) * STAGES + (KV ? 24 : 26) +
            2 * AHEAD) + 15) /
      16 * 16;
  static constexpr int OFF_PIECE = OFF_BAR + BAR_BYTES;
  static constexpr int PIECE_BYTES = 64;
  static_assert(OFF_PIECE % 16 == 0, "pieces are copied as vectors");
  static constexpr int OFF_PAR = OFF_PIECE + SLOTS * PIECE_BYTES;
  static constexpr int OFF_XCH = OFF_PAR + SLOTS * PKV_TREE_MAX_ROWS;
  static constexpr int SMEM_USED = OFF_XCH + (NX == 2 ? 2 * BM * 8 : 0);
  // one CTA per SM (it takes all of tensor memory)
  static constexpr int SMEM = SMEM_USED < 120 * 1024 ? 120 * 1024 : SMEM_USED;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  // Codes: 640 or 512 threads, launched with 96 or 128 registers each; the
  // softmax warps take 144 or 200, the others keep 64 or 104.  (A kernel that
  // uses setmaxnreg is compiled for as many registers as its launch bounds
  // leave; _build.py refuses any other count.)
  static constexpr bool SPLIT_REGS = KV != 0;
  static constexpr int LAUNCH_REGS = NX == 2 ? 96 : 128,
                       SOFTMAX_REGS = NX == 2 ? 144 : 200,
                       OTHER_REGS = NX == 2 ? 64 : 104;
  static_assert(!SPLIT_REGS ||
                    NX * 128 * SOFTMAX_REGS +
                            (THREADS - NX * 128) * OTHER_REGS <=
                        THREADS * LAUNCH_REGS,
                "register split");
};

struct Params {
  const void* q;
  int64_t q_st, q_sh;
  void* out;
  int64_t o_st, o_sh;
  float* lse;
  int total_q, batch, max_n;
  const int32_t* cu_q;
  const int32_t* seqused_k;
  const int32_t* parents;
  const int32_t* block_table;
  int64_t bt_stride;
  int max_blocks;
  int64_t num_blocks;
  int Hq, Hkv, G, BS, RB;
  int bs_shift;             // log2(BS) of a power of two, else -1
  float inv_g;              // 1 / G
  float scale, softcap;
  const float* sinks;
  // caches of codes: value = code (* block scale, strides in bytes) * scale
  const uint8_t *k_sf, *v_sf;
  int64_t f_sb, f_sr, f_sh;
  const float* k_scale;
  const float* v_scale;
  int wl;
  int kv_order_hnd, kv_rg, q_tma, out_v8, once;
  // shares may cut units: partials [slot][rows_cap] (O rows, LSEs) of CTA c in
  // slots 2 c (of the unit it starts inside, or all of its share) and 2 c + 1
  // (of the unit it starts and does not end); marks[c]: the latter's geometry
  int split, rows_cap;
  float* part_o;
  float* part_lse;
  int4* marks;              // two per CTA: (pieces, q0, rows, row0), (g, gave
                            // up, ...)
  unsigned* err;
  uint64_t wait_ns;         // limit of the bounded waits
};

// A run of consecutive key tiles of one unit.
struct Piece {
  int live;                 // 0: no more pieces
  int b, g, q0, n, rows, row0, ctx;
  int kt0, nt;              // first key of the first tile, tiles
  int klo, khi;             // keys any row sees; khi also bounds the reads
  int pair;                 // more than 128 rows
  int whole, slot;          // the whole unit; else its partial's slot
  int pad;
};
static_assert(sizeof(Piece) == 64, "copied as 4 x 16 bytes");

// What a request asks for; rows <= 0: nothing.
struct Req {
  int q0, n, ctx, klo, khi, kstart, tiles, units;
};

__device__ __forceinline__ Req request(const Params& p, int b, int BN,
                                       int ROWS, unsigned* flag) {
  Req r{};
  if (b >= p.batch) return r;
  r.q0 = p.cu_q[b];
  const int end = p.cu_q[b + 1];
  int L = p.seqused_k[b];
  r.n = min(end, p.total_q) - r.q0;
  if (r.q0 < 0 || r.n <= 0) return r;
  if (r.n > p.max_n) {
    *flag |= kErrQueryLen;
    return r;
  }
  if (L < 0) L = 0;
  r.ctx = L - r.n;
  // keys past the table row are not read
  const int64_t tab = static_cast<int64_t>(p.max_blocks) * p.BS;
  r.khi = L > tab ? static_cast<int>(tab) : L;
  if (r.khi < L) *flag |= kErrBadTable;
  // (the shallowest row may be row 0, at position ctx)
  r.klo = p.wl >= 0 ? min(max(r.ctx - p.wl, 0), r.khi) : 0;
  r.kstart = r.klo / p.RB * p.RB;
  // a request without keys still has one (empty) tile: its rows are written
  r.tiles = max((r.khi - r.kstart + BN - 1) / BN, 1);
  r.units = (r.n * p.G + ROWS - 1) / ROWS * p.Hkv;
  return r;
}

// R / G for a packed row (R < 2^20; exact: the product is off by far less than
// the half).
__device__ __forceinline__ int row_of(int R, float inv_g) {
  return static_cast<int>((static_cast<float>(R) + 0.5f) * inv_g);
}

// Places in the ring of a piece's K and V tiles, counted from its first: the
// order in which the products take them.
//   pair            S(0) | P V(0) S(1) | P V(1) S(2) | ...   of both streams
//   else, two lines of tiles (or of score buffers):
//                   S(0) | S(1) | P V(0) S(2) | P V(1) S(3) | ...
__device__ __forceinline__ int place_k(int j, bool pair) {
  return pair ? 2 * j : j < 2 ? j : 2 * j - 1;
}
__device__ __forceinline__ int place_v(int j, int nt, bool pair) {
  return pair ? 2 * j + 1 : min(2 * j + 2, 2 * nt - 1);
}

// Eight values, f16 pairs h, as T to 16 bytes of shared memory.
template <typename T>
__device__ __forceinline__ void store_wide(uint32_t at, const uint32_t* h) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      w[i] = h[i];
    } else {
      const __half2 v = *reinterpret_cast<const __half2*>(&h[i]);
      w[i] = pack2<T>(__low2float(v), __high2float(v));
    }
  }
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
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

// Bits [lo, hi) of 32-bit word w of a tile's mask.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int w) {
  const int a = max(lo - 32 * w, 0), b = min(hi - 32 * w, 32);
  if (b <= a) return 0u;
  return (b == 32 ? 0xffffffffu : (1u << b) - 1u) & (0xffffffffu << a);
}

template <typename T, int D, int KV>
__global__ void __launch_bounds__(Cfg<D, KV>::THREADS, 1)
tree_attn_kernel(const Params p, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CUtensorMap tm_q) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using C = Cfg<D, KV>;
  constexpr int BN = C::BN, NX = C::NX, ST = C::STAGES;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = smem_raw;
  const uint32_t base_u = smem_u32(smem_raw);
  if (base_u & 1023u) {            // 128-byte swizzle atoms need 1 KB
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) {
      atomicOr(p.err, kErrSmemAlign);
      if (p.split) {
        p.marks[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
        p.marks[2 * blockIdx.x + 1] = make_int4(0, 1, 0, 0);
      }
    }
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.G, RB = p.RB;
  const uint32_t sQ = base_u + C::OFF_Q;
  const uint32_t sR = base_u + C::OFF_RING;
  const uint32_t bar0 = base_u + C::OFF_BAR;
  // A stage's loads of stream 0, of stream 1 and of both complete on barriers
  // of their own: a waiter sees one parity, so it has to wait for every load of
  // a barrier, and the streams run ahead of one another.
  constexpr int SETS = NX == 2 ? 3 : 1;
  auto full = [&](int set, int s) { return bar0 + 8 * (set * ST + s); };
  auto empty = [&](int s, int group = 0) {
    return bar0 + 8 * ((SETS + (C::EMPTIES == 2 ? group : 0)) * ST + s);
  };
  constexpr int B0 = (SETS + C::EMPTIES) * ST;
  static_assert(SETS * ST <= 32, "parities in a word");
  auto s_full = [&](int x) { return bar0 + 8 * (B0 + x); };
  auto p_full = [&](int x) { return bar0 + 8 * (B0 + 2 + x); };
  auto o_ready = [&](int x) { return bar0 + 8 * (B0 + 4 + x); };
  auto o_free = [&](int x) { return bar0 + 8 * (B0 + 6 + x); };
  auto q_full = [&](int s) { return bar0 + 8 * (B0 + 8 + s); };
  auto q_empty = [&](int s) { return bar0 + 8 * (B0 + 10 + s); };
  auto it_full = [&](int s) { return bar0 + 8 * (B0 + 12 + s); };
  auto it_empty = [&](int s) { return bar0 + 8 * (B0 + 14 + s); };
  const uint32_t xbar = bar0 + 8 * (B0 + 16);       // the streams' states
  const uint32_t pv_done = bar0 + 8 * (B0 + 17);    // (one stream)
  const uint32_t drain_bar = bar0 + 8 * (B0 + 18);
  auto par_full = [&](int s) { return bar0 + 8 * (B0 + 19 + s); };
  // codes of a tile have arrived / are widened
  auto raw_full = [&](int s) { return bar0 + 8 * (B0 + 21 + s); };
  auto raw_empty = [&](int s) { return bar0 + 8 * (B0 + 21 + C::AHEAD + s); };
  // the streams' turns at the tensor core
  auto turn = [&](int x) { return bar0 + 8 * (B0 + 21 + 2 * C::AHEAD + x); };
  // the probabilities of a tile's first half (16-bit caches, two streams)
  constexpr bool HALVES = NX == 2 && KV == 0;
  auto p_half = [&](int x) { return bar0 + 8 * (B0 + 23 + 2 * C::AHEAD + x); };
  constexpr int OFF_WORDS =
      C::OFF_BAR + 8 * (B0 + (KV ? 23 : 25) + 2 * C::AHEAD);
  static_assert(OFF_WORDS + 8 <= C::OFF_PIECE, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + OFF_WORDS);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(base + OFF_WORDS + 4);

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      for (int k = 0; k < SETS; ++k)
        mbar_init(full(k, s), KV ? C::GROUP : 1);
      for (int g = 0; g < C::EMPTIES; ++g) mbar_init(empty(s, g), NX);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 128);
      mbar_init(o_ready(s), 1);
      mbar_init(o_free(s), NX * 128);
      mbar_init(q_full(s), p.q_tma ? 1 : 32);
      mbar_init(q_empty(s), NX);
      mbar_init(it_full(s), 1);
      mbar_init(it_empty(s), C::SM_WARPS + C::TAKERS);
      mbar_init(par_full(s), 1);
      mbar_init(turn(s), 1);
      if (KV == 0) mbar_init(p_half(s), 128);
    }
    for (int s = 0; s < C::AHEAD; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), C::GROUP);
    }
    mbar_init(xbar, 256);
    mbar_init(pv_done, 1);
    mbar_init(drain_bar, NX);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::MMA_WARP) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::
            "r"(smem_u32(tmem_slot))
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;"
                 ::: "memory");
  }
  if (tid == 0) {
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
    if (p.q_tma) prefetch_map(&tm_q);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // everything that this kernel reads or writes comes after the kernel
  // queued before it (a no-op unless launched as its programmatic dependent)
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // (A poll is one instruction of a converged warp on one address, so its lanes
  // get one answer and what is collective behind it stays whole.  Votes on it
  // measured 1 to 3 % slower, in the slow path alone too.)
  auto wait_for = [&](uint32_t bar, uint32_t parity) -> bool {
    return mbar_wait_lim(bar, parity, abort_flag, p.err, p.wait_ns);
  };
  // The CTA's n-th piece (all lanes of a reader warp call it in order).  The
  // slot is given back by release(n).
  auto take = [&](int n, Piece& pc) -> int {
    const int s = n & 1;
    if (!wait_for(it_full(s), (n >> 1) & 1)) return -1;
    const int4* src = reinterpret_cast<const int4*>(
        base + C::OFF_PIECE + s * C::PIECE_BYTES);
    int4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = src[k];
    memcpy(&pc, w, sizeof(Piece));
    return pc.live ? 1 : 0;
  };
  auto release = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(it_empty(n & 1));
  };
  // K / V tile layout: a 128-byte swizzle atom is 8 keys x 64 columns; cbs is
  // the stride between column blocks, gs between 8-key groups (the 5-D boxes
  // land as [8-key group][column block], the 4-D ones as [column block][key])
  // (widened codes take the former)
  const uint32_t cbs =
      KV || p.kv_rg ? 1024u : static_cast<uint32_t>(BN * 128);
  const uint32_t gs =
      KV || p.kv_rg ? static_cast<uint32_t>(C::NCB * 1024) : 1024u;

  if (warp >= C::SM_WARPS) {
    if constexpr (C::SPLIT_REGS)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == C::LOAD_WARP) {
      // ------------------------------------------------- K / V loader
      // Step i of a piece loads K tile i (lanes 0 .. 15, a page's box each) and
      // V tile i - lag (lanes 16 .. 31), which are next to one another in the
      // ring.  A lane's page id is fetched a step ahead.  Boxes behind the last
      // key, and those of a page outside the cache, start outside the tensor:
      // they arrive as zeros.  Codes go to the places that the code warps read.
      // (With pages of 16 keys the copies set the pace of small tiles: a row of
      // 128 bytes takes about 7 clocks.  A second loader warp changed nothing;
      // one elected lane in a loop, fed by shuffles, was slower: 228 us against
      // 158 on 48 requests of 12 rows over 4364 16-bit keys.)
      constexpr int RING = KV ? C::AHEAD : ST;
      const int half = lane >> 4, box = lane & 15;
      const void* tm = half ? static_cast<const void*>(&tm_v)
                            : static_cast<const void*>(&tm_k);
      const uint64_t pol = l2_evict_first_policy();
      const int boxes = BN / RB;
      const int per_page = p.BS / RB;  // boxes of a page
      // pages of a tile, and boxes beyond them
      const int tile_cols = boxes / per_page;
      const int tile_subs = boxes - tile_cols * per_page;
      int at = 0;                      // loads of the pieces before
      uint32_t sent = 0, ever = 0;     // lane 0: loads of each barrier, mod 2
      bool ok = true;
      for (int n = 0; ok; ++n) {
        Piece pc;
        if (take(n, pc) <= 0) break;
        release(n);
        const int lag = NX == 2 && !pc.pair ? 2 : 1;
        const bool pair = pc.pair;
        const int32_t* bt =
            p.block_table + static_cast<int64_t>(pc.b) * p.bt_stride;
        // this lane's entry of its next tile
        int k0 = pc.kt0 + box * RB;
        int col = k0 / p.BS, sub = (k0 - col * p.BS) / RB;
        int nxt = box < boxes && k0 < pc.khi ? __ldg(bt + col) : 0;
#pragma unroll 1
        for (int i = 0; i < pc.nt + lag; ++i) {
          const int j = half ? i - lag : i;
          const bool mine = j >= 0 && j < pc.nt;
          int id = nxt;
          const int row = sub * RB;
          bool dead = k0 >= pc.khi;              // (no key in this lane's box)
          if (mine) {
            k0 += BN;
            col += tile_cols;
            sub += tile_subs;
            if (sub >= per_page) {
              sub -= per_page;
              ++col;
            }
            nxt = box < boxes && k0 < pc.khi ? __ldg(bt + col) : 0;
          }
          const int pos = at + (half ? place_v(j, pc.nt, pair)
                                     : place_k(j, pair));
          const int st = pos % RING;
          const int set = NX == 1 || KV ? 0 : pair ? 2 : j & 1;
          const uint32_t bar = KV ? raw_full(st) : full(set, st);
          int stop = 0;
          if (box == 0 && mine) {
            if (pos >= RING &&
                !mbar_wait_lim(KV ? raw_empty(st) : empty(st),
                               (pos / RING - 1) & 1, abort_flag, p.err,
                               p.wait_ns))
              stop = 1;
            else
              mbar_expect_tx(bar, KV ? C::CODE_TILE : C::STAGE);
          }
          if (__any_sync(0xffffffffu, stop)) {
            ok = false;
            break;
          }
          if (box < boxes && mine) {
            if (!dead && (id < 0 || id >= p.num_blocks)) {
              atomicOr(p.err, kErrBadBlock);
              dead = true;
            }
            if (KV) {
              const int c1 = p.kv_order_hnd ? row : pc.g;
              const int c2 = p.kv_order_hnd ? pc.g : row;
              const uint32_t to = base_u + C::OFF_CODES + st * C::CODE_TILE +
                                  box * RB * C::CODE_ROW;
              tma_load_4d_hint(to, tm, 0, c1, c2, dead ? -1 : id, bar, pol);
            } else if (p.kv_rg) {
              const uint32_t to =
                  sR + st * C::STAGE + box * (RB / 8) * gs;
              // (a box has RB / 8 groups)
              const int c3 = p.kv_order_hnd ? row >> 3
                             : dead         ? -(RB >> 3)
                                    : id * (p.BS >> 3) + (row >> 3);
              const int c4 = !p.kv_order_hnd ? pc.g
                             : dead          ? -1
                                             : id * p.Hkv + pc.g;
              if (p.once)
                tma_load_5d_hint(to, tm, 0, 0, 0, c3, c4, bar, pol);
              else
                tma_load_5d(to, tm, 0, 0, 0, c3, c4, bar);
            } else {
              const uint32_t to = sR + st * C::STAGE + box * RB * 128;
              const int c1 = p.kv_order_hnd ? row : pc.g;
              const int c2 = p.kv_order_hnd ? pc.g : row;
#pragma unroll 1
              for (int cb = 0; cb < C::NCB; ++cb)
                if (p.once)
                  tma_load_4d_hint(to + cb * cbs, tm, cb * 64, c1, c2,
                                   dead ? -1 : id, bar, pol);
                else
                  tma_load_4d(to + cb * cbs, tm, cb * 64, c1, c2,
                              dead ? -1 : id, bar);
            }
          }
          // (for the end: which barrier each load went to)
          const uint32_t bit = box == 0 && mine ? 1u << (set * RING + st) : 0u;
          const uint32_t bits =
              bit | __shfl_xor_sync(0xffffffffu, bit, 16);
          if (lane == 0) sent ^= bits;
          if (lane == 0) ever |= bits;
        }
        at += 2 * pc.nt;
      }
      // no copy may be in flight when the CTA exits
      if (lane == 0)
        for (int k = 0; k < (KV ? RING : SETS * ST); ++k)
          if (ever >> k & 1)
            mbar_drain(KV ? raw_full(k) : full(0, k), (sent >> k & 1) ^ 1);
    } else if (KV != 0 && warp >= C::CODE_WARP) {
      // ------------------------------------------------- codes widened
      // From the loader's rows of codes to the 16-bit layout that the products
      // read: exactly, the tensor scales joining the logits and the output.
      // Two groups of warps take the places of the ring in turn, so that one
      // converts while the other waits, fences and signs off (head size 256,
      // 48 requests of 4364 keys: 375 us with one group of 8, 320 with two of
      // 4 for 4 bits, 258 and 226 for E4M3; 199 and 187 at 128 for 4 bits).  A
      // warp widens 16 rows at a time: they lie in one page, whose block scales
      // it fetches.
      if constexpr (KV != 0) {
        constexpr int RW = BN / C::GROUP;                // rows of a warp
        constexpr int H = RW / 16;
        static_assert(H * 16 == RW, "whole sixteens");
        constexpr int VALS = KV == kE4m3 ? 16 : 32;      // values of 16 bytes
        constexpr int ROW = D / VALS;                    // 16 bytes of a row
        constexpr int RI = 32 / ROW;                     // rows at a time
        constexpr int PER = 16 / RI;
        const int cw = warp - C::CODE_WARP, ln = lane / ROW, cp = lane % ROW;
        const int group = cw / C::GROUP, sub = cw % C::GROUP;
        // row and eight of step i's row
        auto row_in_8 = [&](int i) {
          return RI >= 8 ? ln & 7 : i % (8 / (RI < 8 ? RI : 8)) * RI + ln;
        };
        auto eights = [&](int i) {
          return RI >= 8 ? i * (RI / 8) + (ln >> 3) : i / (8 / (RI < 8 ? RI : 8));
        };
        int pos = group;               // place in the ring
        bool ok = true;
        for (int n = 0; ok; ++n) {
          Piece pc;
          if (take(n, pc) <= 0) break;
          release(n);
          const int total = 2 * pc.nt, steps = pc.nt * H;
          const bool low = pc.kt0 < pc.klo;
          const bool high = pc.kt0 + pc.nt * BN > pc.khi;
          // step s: rows 16 (s % H) .. of place 2 (s / H) + group of the piece:
          // its tile, and K (0) or V
          auto tile = [&](int s, int& v) -> int {
            const int q = s / H * 2 + group;
            if (pc.pair) {
              v = q & 1;
              return q >> 1;
            }
            v = q == total - 1 || (q > 1 && !(q & 1));
            return q == total - 1 ? pc.nt - 1 : v ? (q - 2) >> 1 : (q + 1) >> 1;
          };
          // block scales: the table's entry two steps ahead, the scales of
          // this lane's bytes one ahead
          const int32_t* bt =
              p.block_table + static_cast<int64_t>(pc.b) * p.bt_stride;
          int blk = 0;
          uint16_t sf[PER] = {}, sf_next[PER] = {};
          auto first_key = [&](int s, int& v) -> int {
            return pc.kt0 + tile(s, v) * BN + sub * RW + s % H * 16;
          };
          auto entry = [&](int s) {
            int v;
            const int key = first_key(s, v);
            if (KV == kE2m1 && s < steps && key < pc.khi)
              blk = __ldg(bt + (p.bs_shift >= 0 ? key >> p.bs_shift
                                                : key / p.BS));
          };
          auto scales = [&](int s) {
            int v;
            const int key = first_key(s, v);
            if (KV == kE2m1 && s < steps && key < pc.khi && blk >= 0 &&
                blk < p.num_blocks) {
              const int row = p.bs_shift >= 0 ? key & (p.BS - 1) : key % p.BS;
              const uint8_t* from = (v ? p.v_sf : p.k_sf) + blk * p.f_sb +
                                    (row + ln) * p.f_sr + pc.g * p.f_sh +
                                    cp * 2;
#pragma unroll
              for (int i = 0; i < PER; ++i)
                sf_next[i] = __ldg(reinterpret_cast<const uint16_t*>(
                    from + i * RI * p.f_sr));
            } else {
#pragma unroll
              for (int i = 0; i < PER; ++i) sf_next[i] = 0;
            }
          };
          entry(0);
          scales(0);
          entry(1);
#pragma unroll 1
          for (int s = 0; s < steps; ++s) {
            int v;
            const int i_tile = tile(s, v), part = s % H;
            if (KV == kE2m1) {
#pragma unroll
              for (int i = 0; i < PER; ++i) sf[i] = sf_next[i];
              scales(s + 1);
              entry(s + 2);
            }
            const int st = pos % ST, slot = pos % C::AHEAD;
            if (part == 0 &&
                !wait_for(raw_full(slot), (pos / C::AHEAD) & 1)) {
              ok = false;
              break;
            }
            const int row0 = sub * RW + part * 16;
            const uint32_t to = sR + st * C::STAGE + row0 / 8 * gs;
            const unsigned char* src = base + C::OFF_CODES +
                                       slot * C::CODE_TILE +
                                       row0 * C::CODE_ROW + lane * 16;
            // (all codes at once: the stores below let no load past them)
            uint4 ws[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i)
              ws[i] = *reinterpret_cast<const uint4*>(src + i * 512);
            if (part == 0 && pos >= ST &&
                !wait_for(empty(st, group),
                           (pos - ST) / (ST * C::EMPTIES) & 1)) {
              ok = false;
              break;
            }
            // (V rows that no row of the block sees are zeros: they may hold
            // another request's NaN)
            const int key0 = pc.kt0 + i_tile * BN + row0 + ln;
            const bool edge = v && ((low && i_tile == 0) ||
                                    (high && i_tile == pc.nt - 1));
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              uint4 w = ws[i];
              if (edge && (key0 + i * RI < pc.klo || key0 + i * RI >= pc.khi)) {
                w = make_uint4(0, 0, 0, 0);
                sf[i] = 0;
              }
              const int r8 = row_in_8(i);
              const uint32_t line = to + eights(i) * gs + r8 * 128;
              if constexpr (KV == kE4m3) {
                const uint32_t dst = line + (cp >> 2) * 1024;
                // (the two halves in an order that keeps the lanes of a row
                // in different banks)
                const bool odd = (cp >> 2) & 1;
                const uint32_t c0 = (cp & 3) * 2 + (odd ? 1 : 0);
                uint32_t x[4], y[4];
                e4m3x4_to_f16(odd ? w.z : w.x, x[0], x[1]);
                e4m3x4_to_f16(odd ? w.w : w.y, x[2], x[3]);
                e4m3x4_to_f16(odd ? w.x : w.z, y[0], y[1]);
                e4m3x4_to_f16(odd ? w.y : w.w, y[2], y[3]);
                store_wide<T>(dst + ((c0 ^ r8) << 4), x);
                store_wide<T>(dst + ((c0 ^ 1 ^ r8) << 4), y);
              } else {
                const uint32_t dst = line + (cp >> 1) * 1024;
                const uint32_t f = e4m3x2_to_f16(sf[i]);
                const uint32_t f0 = __byte_perm(f, f, 0x1010),
                               f1 = __byte_perm(f, f, 0x3232);
                const uint32_t part[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  uint32_t h[4];
                  e2m1x8_to_f16(part[k], h[0], h[1], h[2], h[3]);
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    h[e] = hmul2_u32(h[e], k < 2 ? f0 : f1);
                  store_wide<T>(dst + ((((cp & 1) * 4 + k) ^ r8) << 4), h);
                }
              }
            }
            if (part != H - 1) continue;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              const int set = NX == 1 ? 0 : pc.pair ? 2 : i_tile & 1;
              mbar_arrive(full(set, st));
              mbar_arrive(raw_empty(slot));
            }
            pos += 2;
          }
        }
      }
    } else if (warp >= C::MMA_WARP && warp < C::MMA_WARP + NX) {
      // -------------------------------------- MMA issuer of stream x
      const int x = NX == 2 ? warp - C::MMA_WARP : 0;
      constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
      constexpr uint32_t ID_S = idesc(128, BN, kBF16, false);
      constexpr uint32_t ID_PV = idesc(128, D, kBF16, true);
      const uint32_t acc = tmem + x * C::S_STEP + C::O_COL;
      uint32_t s_cnt = 0, pv_cnt = 0;  // products issued
      uint32_t turns = 0;
      int at = 0;                      // loads of the pieces before
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool r = wait_for(bar, parity & 1);
        tc_fence_after();
        return r;
      };
      // The load in stage st has landed.
      uint32_t f_turn = 0;             // parities of full: ST bits a set
      auto loaded = [&](int st, int set) -> bool {
        const int bit = set * ST + st;
        const bool r = wait(full(set, st), f_turn >> bit);
        f_turn ^= 1u << bit;
        return r;
      };
      for (int n = 0; ok; ++n) {
        Piece pc;
        if (take(n, pc) <= 0) break;
        release(n);
        const bool pair = pc.pair;
        const bool alt = NX == 2 && !pair;
        // tiles of this stream: j0, j0 + step, ...
        const int j0 = alt ? x : 0, step = alt ? 2 : 1;
        const int tiles = (pc.nt - j0 + step - 1) / step;
        const int set = NX == 1 ? 0 : pair ? 2 : x;
        const int qt = NX == 1 ? 0 : pair ? x : n & 1;
        const uint64_t qd = sdesc(sQ + qt * C::Q_TILE, 16, 1024);
        if (tiles == 0) {
          // (no phase of q_empty, o_free or o_ready is left out)
          mma_commit_warp(q_empty(n & 1));
          if (n > 0 && !wait(o_free(x), n - 1)) break;
        }
        // Step k: P V of this stream's tile k - 1, S of its tile k (one stream:
        // the other way round, S has a buffer of its own).  Whatever can be
        // waited for and worked out before the probabilities come, is.
        auto score = [&](int st) {
          const int buf = NX == 1 ? s_cnt & 1 : x;
          const uint64_t kd = sdesc(sR + st * C::STAGE, 16, gs);
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            mma_f16_warp(tmem + buf * C::S_STEP,
                         qd + (((c >> 2) * (BM * 128) + (c & 3) * 32) >> 4),
                         kd + (((c >> 2) * cbs + (c & 3) * 32) >> 4), ID_S,
                         c > 0 ? 1 : 0);
          mma_commit_warp(s_full(buf));
          ++s_cnt;
        };
        // (place pos; its stage's next turn is the other group's, if any)
        auto consumed = [&](int pos) {
          const uint32_t bar = empty(pos % ST, (pos + ST) & 1);
          mma_commit_warp(bar);
          if (alt) mma_commit_warp(bar);             // (for the other stream)
        };
        if (tiles > 0 && !wait(q_full(n & 1), n >> 1)) break;
#pragma unroll 1
        for (int k = 0; k <= tiles && tiles > 0; ++k) {
          const int jk = j0 + k * step, jv = jk - step;
          const int pk = at + place_k(jk, pair);
          const int pv = at + place_v(jv, pc.nt, pair);
          const int sk = pk % ST, sv = pv % ST;
          if (k < tiles && NX == 1) {
            if (!loaded(sk, set)) {
              ok = false;
              break;
            }
            score(sk);
            consumed(pk);
          }
          if (k > 0) {
            if (!loaded(sv, set)) {
              ok = false;
              break;
            }
            // rows of V that no row of the block sees become zero (they may
            // hold another request's NaN): those before the window in the
            // first box, those behind the last key in the last one
            const int kt = pc.kt0 + jv * BN;
            if (KV == 0 && (kt < pc.klo || kt + BN > pc.khi)) {
              const int lo = min(max(pc.klo - kt, 0), BN);
              const int hi = max(min(pc.khi - kt, BN), lo);
              const int top = min((hi + RB - 1) / RB * RB, BN);
              const uint32_t v0 = sR + sv * C::STAGE;
#pragma unroll 1
              for (int e = lane; e < (lo + top - hi) * 8; e += 32) {
                int r = e >> 3;
                if (r >= lo) r += hi - lo;
                const uint32_t to =
                    v0 + (r >> 3) * gs + (r & 7) * 128 + ((e & 7) << 4);
#pragma unroll
                for (int cb = 0; cb < C::NCB; ++cb)
                  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::
                                   "r"(to + cb * cbs),
                               "r"(0)
                               : "memory");
              }
              fence_proxy_async();
              __syncwarp();
            }
            // the epilogue of the piece before has read the accumulator
            if (k == 1 && n > 0 && !wait(o_free(x), n - 1)) {
              ok = false;
              break;
            }
          }
          if (k < tiles && NX == 2 && KV == 0 && !loaded(sk, set)) {
            ok = false;
            break;
          }
          if (k > 0) {
            const int buf = NX == 1 ? pv_cnt & 1 : x;
            const uint64_t vd = sdesc(sR + sv * C::STAGE, cbs, gs);
            const uint32_t keep = k > 1 ? 1u : 0u;
            if (!wait(HALVES ? p_half(x) : p_full(buf),
                      NX == 1 ? pv_cnt >> 1 : pv_cnt) ||
                (NX == 2 && pair && !wait(turn(x), turns + 1 - x))) {
              ok = false;
              break;
            }
            auto products = [&](int c) {
              mma_f16_tmem_a_warp(acc, tmem + buf * C::S_STEP + 8 * c,
                                  vd + ((c * 2 * gs) >> 4), ID_PV,
                                  c > 0 ? 1u : keep);
            };
            constexpr int FIRST = HALVES ? BN / 32 : BN / 16;
#pragma unroll
            for (int c = 0; c < FIRST; ++c) products(c);
            if constexpr (HALVES) {
              // (the first half runs under the second half of the softmax:
              // 190 -> 185 us on 64 requests of 64 rows over 2368 keys)
              if (!wait(p_full(x), pv_cnt)) {
                ok = false;
                break;
              }
#pragma unroll
              for (int c = FIRST; c < BN / 16; ++c) products(c);
            }
            ++pv_cnt;
            if constexpr (NX == 1) mma_commit_warp(pv_done);
            if (NX == 1 || KV != 0) consumed(pv);
          }
          if (NX == 2) {
            // (codes: the widening of the next K waits for V's stage, so V is
            // given back before K is waited for: 173 -> 165 us on 48 requests
            // of 4364 E4M3 keys)
            if (k < tiles && KV != 0 && !loaded(sk, set)) {
              ok = false;
              break;
            }
            if (k < tiles) score(sk);
            if (k > 0 && KV == 0) consumed(pv);
            if (k < tiles) consumed(pk);
            // Of two streams that take every tile, one's P V and next S run as
            // a whole while the other is at its softmax.  (Left to themselves
            // the two interleave, end together, and then the tensor core waits
            // for two softmaxes at once, 2000 clocks of 4500 a tile: 483 us
            // against 430 on 4 requests of 64 rows, 64 heads, 65600 keys.)
            if (pair && k > 0) {
              ++turns;
              if (lane == 0) mbar_arrive(turn(1 - x));
            }
          }
          if (k == tiles - 1) mma_commit_warp(q_empty(n & 1));
        }
        if (!ok) break;
        mma_commit_warp(o_ready(x));
        at += 2 * pc.nt;
      }
      // every MMA of this CTA is complete before TMEM is freed
      mma_commit_warp(drain_bar);
      mbar_drain(drain_bar, 0);
    } else if (warp == C::DEAL_WARP) {
      // -------------------------- the pieces, their queries and parents
      // This CTA's share [beg, end) of the sequence of all units' tiles (of
      // units, when they are not to be cut).  A lane sums the weights of a run
      // of requests; one warp does it, as the other warps have nothing to wait
      // for but the first piece (a scan by the whole block took 2900 clocks).
      unsigned flag = 0;
      auto weight = [&](const Req& r) -> unsigned {
        return static_cast<unsigned>(p.split ? r.tiles * r.units : r.units);
      };
      auto scan = [&](unsigned v) -> unsigned {     // inclusive, over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += y;
        }
        return v;
      };
      const int run = (p.batch + 31) / 32;
      unsigned sum = 0;
#pragma unroll 4
      for (int i = 0; i < run; ++i)
        sum += weight(request(p, lane * run + i, BN, C::ROWS, &flag));
      const unsigned incl = scan(sum);
      const unsigned n_all = __shfl_sync(0xffffffffu, incl, 31);
      // (as many CTAs as tiles at most: no share between two others is empty)
      const unsigned ctas = min(gridDim.x, n_all);
      unsigned beg = 0, end = 0;
      if (blockIdx.x < ctas) {
        const unsigned each = n_all / ctas, more = n_all - each * ctas;
        beg = blockIdx.x * each + blockIdx.x * more / ctas;
        end = (blockIdx.x + 1) * each + (blockIdx.x + 1) * more / ctas;
      }
      int b = 0;
      unsigned off = 0, rem = end - beg;
      int wb = -1;                     // request of lane 0 below
      Req mine{};                      // request wb + lane
      if (rem > 0) {
        const unsigned hit =
            __ballot_sync(0xffffffffu, beg >= incl - sum && beg < incl);
        const int src = __ffs(hit) - 1;
        off = beg - __shfl_sync(0xffffffffu, incl - sum, src);
        // ... and within the run
        for (wb = src * run;; wb += 32) {
          unsigned f = 0;
          mine = request(p, wb + lane, BN, C::ROWS, &f);
          const unsigned w = weight(mine), in = scan(w);
          const unsigned m =
              __ballot_sync(0xffffffffu, off >= in - w && off < in);
          if (m) {
            const int at = __ffs(m) - 1;
            off -= __shfl_sync(0xffffffffu, in - w, at);
            b = wb + at;
            break;
          }
          off -= __shfl_sync(0xffffffffu, in, 31);
          if (wb + 32 >= p.batch) {    // (the lengths changed under the call)
            rem = 0;
            break;
          }
        }
      }
      if (flag && blockIdx.x == 0) atomicOr(p.err, flag);
      int prev_pair = 1;
      bool marked = false;
      int q_issued = 0;                // query loads as TMA boxes
      for (int n = 0;; ++n) {
        Piece pc{};
        unsigned unit_end = 0;         // of a unit that goes on after the share
        if (rem > 0) {
          // the request that the next tile belongs to
          for (;;) {
            if (wb < 0 || b >= wb + 32) {
              unsigned f = 0;
              wb = b;
              mine = request(p, wb + lane, BN, C::ROWS, &f);
            }
            const unsigned m = __ballot_sync(
                0xffffffffu, mine.units > 0 && wb + lane >= b);
            if (m) {
              const int at = wb + __ffs(m) - 1;
              if (at != b) off = 0;
              b = at;
              break;
            }
            b = wb + 32;
            off = 0;
            if (b >= p.batch) break;
          }
          if (b >= p.batch) rem = 0;   // (the lengths changed under the call)
        }
        if (rem > 0) {
          const int src = b - wb;
          auto get = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
          const int tiles = get(mine.tiles), units = get(mine.units);
          const int wt = p.split ? tiles : 1;
          const int u = static_cast<int>(off / static_cast<unsigned>(wt));
          const int t = p.split ? static_cast<int>(off) - u * wt : 0;
          const int nblk = units / p.Hkv;
          const int g = u / nblk, rb = u - g * nblk;
          const int nt =
              p.split ? min(static_cast<int>(rem), tiles - t) : tiles;
          pc.live = 1;
          pc.b = b;
          pc.g = g;
          pc.q0 = get(mine.q0);
          pc.n = get(mine.n);
          pc.row0 = rb * C::ROWS;
          pc.rows = min(pc.n * G - pc.row0, C::ROWS);
          pc.ctx = get(mine.ctx);
          pc.kt0 = get(mine.kstart) + t * BN;
          pc.nt = nt;
          pc.klo = get(mine.klo);
          pc.khi = get(mine.khi);
          pc.pair = NX == 2 && pc.rows > BM;
          pc.whole = t == 0 && nt == tiles;
          pc.slot = 2 * blockIdx.x + (t == 0 ? 1 : 0);
          unit_end = !pc.whole && t == 0 ? end - rem + tiles : 0;
          off += p.split ? nt : 1;
          rem -= p.split ? nt : 1;
          if (off == static_cast<unsigned>(units * wt)) {
            ++b;
            off = 0;
          }
        }
        const int s = n & 1;
        if (n >= 2 && !wait_for(it_empty(s), (n / 2 - 1) & 1))
          break;
        if (lane == 0) {
          int4 w[4];
          memcpy(w, &pc, sizeof(Piece));
          int4* dst = reinterpret_cast<int4*>(base + C::OFF_PIECE +
                                              s * C::PIECE_BYTES);
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[k] = w[k];
          mbar_arrive(it_full(s));
        }
        if (!pc.live) break;
        if (unit_end) {
          // its tiles run on to those of CTA `last`
          const int last = static_cast<int>(
              (static_cast<uint64_t>(unit_end) * ctas - 1) / n_all);
          if (lane == 0) {
            p.marks[2 * blockIdx.x] =
                make_int4(last - static_cast<int>(blockIdx.x) + 1, pc.q0,
                          pc.rows, pc.row0);
            p.marks[2 * blockIdx.x + 1] = make_int4(pc.g, 0, 0, 0);
          }
          marked = true;
        }
        // parents: loads first, bytes in shared memory after the queries
        constexpr int PER = PKV_TREE_MAX_ROWS / 32;
        int par[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int i = k * 32 + lane;
          par[k] = i < pc.n ? __ldg(p.parents + pc.q0 + i) : -1;
        }
        // the row tile(s) that this piece's queries go to are free: two pieces
        // of one row tile take them in turn
        const bool alt = NX == 2 && !pc.pair;
        const int before = alt && !prev_pair ? n - 2 : n - 1;
        if (before >= 0 && !wait_for(q_empty(before & 1), (before >> 1) & 1))
          break;
        prev_pair = pc.pair || NX == 1;
        const uint32_t dq = sQ + (alt ? (n & 1) * C::Q_TILE : 0);
        const int qt = pc.rows > BM ? 2 : 1;
        if (p.q_tma) {
          // one box per (row tile, 64 columns): 128 / G rows x the G heads.
          // Rows past the request are the next tokens' (or zeros): they only
          // feed scores that no output is taken from.
          if (lane == 0) {
            mbar_expect_tx(q_full(s), qt * C::Q_TILE);
            for (int t = 0; t < qt; ++t)
#pragma unroll
              for (int cb = 0; cb < C::NCB; ++cb)
                tma_load_3d(dq + t * C::Q_TILE + cb * (BM * 128), &tm_q,
                            cb * 64, pc.g * G,
                            pc.q0 + (pc.row0 + t * BM) / G, q_full(s));
          }
          ++q_issued;
        } else {
          const T* Q = static_cast<const T*>(p.q);
          for (int rr = lane; rr < qt * BM; rr += 32) {
            const int R = pc.row0 + rr;
            const bool okq = rr < pc.rows;
            const T* src = Q;
            if (okq)
              src = Q + static_cast<int64_t>(pc.q0 + R / G) * p.q_st +
                    static_cast<int64_t>(pc.g * G + R % G) * p.q_sh;
            const uint32_t dst = dq + (rr / BM) * C::Q_TILE;
            const int rq = rr % BM;
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch)
              cp_async_16(dst + (ch >> 3) * (BM * 128) + sw128(rq, ch & 7),
                          okq ? src + ch * 8 : src, okq ? 16 : 0);
          }
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async();
          mbar_arrive(q_full(s));
        }
        unsigned char* pb = base + C::OFF_PAR + s * PKV_TREE_MAX_ROWS;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int i = k * 32 + lane;
          const bool no = par[k] < -1 || par[k] >= i;
          if (i < pc.n) {
            bad |= no;
            pb[i] = static_cast<unsigned char>(
                no || par[k] < 0 ? kNoParent : par[k]);
          }
        }
        if (bad) atomicOr(p.err, kErrBadTree);
        __syncwarp();
        if (lane == 0) mbar_arrive(par_full(s));
      }
      if (p.split && lane == 0 && !marked)
        p.marks[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
      // no query box may be in flight when the CTA exits
      if (lane == 0)
        for (int n = max(0, q_issued - 2); n < q_issued; ++n)
          mbar_drain(q_full(n & 1), (n >> 1) & 1);
    }
  } else {
    // ------------------------------------------------- softmax warps
    if constexpr (C::SPLIT_REGS)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(
          C::SOFTMAX_REGS));
    constexpr float THR = Range<T>::THR, OFF = Range<T>::OFF;
    const int x = NX == 2 ? warp >> 2 : 0;
    const int r = tid & 127;                   // row of its tile == TMEM lane
    const float scale_log2 =
        p.scale * (p.k_scale ? *p.k_scale : 1.f) * kLog2e;
    const float vscale = p.v_scale ? *p.v_scale : 1.f;
    const bool capped = p.softcap > 0.f;
    const float cap_t = p.softcap * kLog2e;
    const float cap_u = capped ? 2.f / p.softcap : 0.f;
    // raw: the scale joins the exponent (max(scale s) = scale max(s))
    const bool raw = !capped && scale_log2 > 0.f;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float2* xch = reinterpret_cast<float2*>(base + C::OFF_XCH);
    int cnt = 0;                               // tiles seen by this stream
    int n_x = 0;                               // states exchanged
    for (int n = 0;; ++n) {
      Piece pc;
      if (take(n, pc) <= 0) break;
      const bool alt = NX == 2 && !pc.pair;
      const int row = (pc.pair ? x * BM : 0) + r;       // of the block
      const bool valid = row < pc.rows;
      const bool live = (row & ~31) < pc.rows;          // any row of the warp
      const int R = pc.row0 + (valid ? row : 0);
      const int node = row_of(R, p.inv_g);
      const int h = pc.g * G + R - node * G;
      const int tok = pc.q0 + node;
      const unsigned char* par =
          base + C::OFF_PAR + (n & 1) * PKV_TREE_MAX_ROWS;
      bool ok = true;
      // first key before the draft that this row sees
      int k_first = 0;
      if (p.wl >= 0 && live) {
        ok = wait_for(par_full(n & 1), (n >> 1) & 1);
        int depth = 0;
        for (int a = par[node]; ok && a != kNoParent; a = par[a]) ++depth;
        k_first = max(pc.ctx + depth - p.wl, 0);
      }
      // tiles inside [full_lo, full_hi) need no mask
      const int full_lo =
          p.wl >= 0 ? max(pc.ctx + pc.n - 1 - p.wl, 0) : 0;
      const int full_hi = min(pc.ctx, pc.khi);
      float m_ref = -INFINITY, l = 0.f;
      const int j0 = alt ? x : 0, jd = alt ? 2 : 1;
      for (int j = j0; ok && j < pc.nt; j += jd, ++cnt) {
        const int buf = NX == 2 ? x : cnt & 1;
        const int turn = NX == 2 ? cnt : cnt >> 1;
        if (!wait_for(s_full(buf), turn & 1)) {
          ok = false;
          break;
        }
        if (!live) {
          if (HALVES) mbar_arrive(p_half(x));
          mbar_arrive(p_full(buf));
          continue;
        }
        tc_fence_after();
        const int kt = pc.kt0 + j * BN;
        const bool masked = kt < full_lo || kt + BN > full_hi;
        const uint32_t s_addr = tmem + lane_base + buf * C::S_STEP;
        uint32_t w[BN / 32];
        if (masked) {
          // one bit a key: those before the draft in the window, and the
          // chain of rows from this one upwards
#pragma unroll
          for (int i = 0; i < BN / 32; ++i)
            w[i] = range_bits(k_first - kt, full_hi - kt, i);
          const int rel0 = pc.ctx - kt;        // row 0's key in the tile
          if (rel0 < BN) {
            if (!wait_for(par_full(n & 1), (n >> 1) & 1)) {
              ok = false;
              break;
            }
            const int in_tile = min(BN, pc.khi - kt);
            int a = node;
#pragma unroll 1
            for (int far = 0;; ++far) {
              if (p.wl >= 0 && far > p.wl) break;
              const int rel = rel0 + a;
              if (rel >= 0 && rel < in_tile) {
#pragma unroll
                for (int i = 0; i < BN / 32; ++i)
                  w[i] |= (rel >> 5) == i ? 1u << (rel & 31) : 0u;
              }
              a = par[a];
              if (a == kNoParent) break;
            }
          }
        }
        if (!raw || masked) {
          // the final logits, 32 keys at a time, back to where they came from
          // (a short loop: in line with the code below, for every key of the
          // tile, it pushed that out of the instruction cache)
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            float v[32];
            tmem_ld32(s_addr + c, v);
            tmem_wait_ld();
            if (!raw) {
              // log2 units; soft-cap t (1 - 2 / (1 + 2^(u x))), within about
              // an ulp of the cap (the hardware tanh loses 2^-11 of it), so
              // that large caps are refused: a series for small logits beside
              // it measured 1 to 4 % of every call
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                v[e] *= scale_log2;
                if (capped)
                  v[e] = cap_t -
                         __fdividef(2.f * cap_t, 1.f + ex2(v[e] * cap_u));
              }
            }
            if (masked) {
              // (a select: whatever stands in a hidden place is dropped)
              uint32_t bits = w[0];
#pragma unroll
              for (int i = 1; i < BN / 32; ++i)
                if (c == 32 * i) bits = w[i];
#pragma unroll
              for (int e = 0; e < 32; ++e)
                v[e] = (bits >> e) & 1u ? v[e] : -INFINITY;
            }
            tmem_st32(s_addr + c, v);
          }
          tmem_wait_st();
        }
        // The tile 64 keys at a time, read from tensor memory twice (for the
        // maximum, then for the exponentials): half the registers of a row, and
        // code that stays in the instruction cache.
        float mx8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < BN; c += 64) {
          float v[64];
          tmem_ld32(s_addr + c, v);
          tmem_ld32(s_addr + c + 32, v + 32);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 64; e += 2)
            mx8[(e >> 1) & 7] = max3f(mx8[(e >> 1) & 7], v[e], v[e + 1]);
        }
        float mx =
            max3f(max3f(mx8[0], mx8[1], mx8[2]), max3f(mx8[3], mx8[4], mx8[5]),
                  fmaxf(mx8[6], mx8[7]));
        if (raw) mx *= scale_log2;
        const bool grow = mx > m_ref + THR;
        float alpha = 1.f;
        if (grow) {
          alpha = ex2(m_ref - mx);
          m_ref = mx;
          l *= alpha;
        }
        const float base_m = (m_ref == -INFINITY ? 0.f : m_ref) - OFF;
        if (j >= jd && __any_sync(0xffffffffu, grow)) {
          // the products so far are complete: with two streams the commit
          // behind s_full covered them
          if constexpr (NX == 1) {
            if (!wait_for(pv_done, (cnt - 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          const uint32_t o_addr =
              tmem + lane_base + x * C::S_STEP + C::O_COL;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float ov[32];
            tmem_ld32(o_addr + c, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] *= alpha;
            tmem_st32(o_addr + c, ov);
          }
        }
        float sum8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sum8[e] = 0.f;
        const float sc = raw ? scale_log2 : 1.f;
        // P over the first BN / 2 columns of S (read by then): column c holds
        // the keys 2c (low half) and 2c + 1 (high half)
#pragma unroll 1
        for (int c = 0; c < BN; c += 64) {
          float v[64];
          tmem_ld32(s_addr + c, v);
          tmem_ld32(s_addr + c + 32, v + 32);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float x0 = v[e], x1 = v[e + 1];
            fma2(x0, x1, sc, -base_m);
            x0 = ex2(x0);
            x1 = ex2(x1);
            add2(sum8[2 * ((e >> 1) & 3)], sum8[2 * ((e >> 1) & 3) + 1], x0,
                 x1);
            v[e >> 1] = __uint_as_float(pack2<T>(x0, x1));
          }
          tmem_st32(s_addr + (c >> 1), v);
          if constexpr (HALVES) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(c == 0 ? p_half(x) : p_full(x));
          }
        }
        l += ((sum8[0] + sum8[1]) + (sum8[2] + sum8[3])) +
             ((sum8[4] + sum8[5]) + (sum8[6] + sum8[7]));
        if constexpr (!HALVES) {
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_full(buf));
        }
      }
      if (!ok) break;
      release(n);

      // ---- epilogue: O of each stream relative to m (log2 units)
      float m = m_ref == -INFINITY ? m_ref : m_ref - OFF;
      float f0 = 1.f, f1 = 0.f;                // weights of O_0 and O_1
      if (alt) {
        // (the other stream has read the state of the piece before)
        if (n > 0 && !wait_for(o_free(0), (n - 1) & 1))
          break;
        xch[x * BM + r] = make_float2(m, l);
        mbar_arrive(xbar);
        if (!wait_for(xbar, n_x & 1)) break;
        ++n_x;
        const float2 o = xch[(x ^ 1) * BM + r];
        const float M = fmaxf(m, o.x);
        const float a = m == -INFINITY ? (l != l ? 1.f : 0.f) : ex2(m - M);
        const float c = o.x == -INFINITY ? (o.y != o.y ? 1.f : 0.f)
                                         : ex2(o.x - M);
        // (the same order of the sum in both streams)
        f0 = x == 0 ? a : c;
        f1 = x == 0 ? c : a;
        const float l0 = x == 0 ? l : o.y, l1 = x == 0 ? o.y : l;
        l = l0 * f0 + l1 * f1;
        m = M;
      }
      if (!wait_for(o_ready(x), n & 1)) break;
      if (alt && !wait_for(o_ready(x ^ 1), n & 1)) break;
      tc_fence_after();
      float inv, lse_v;
      finish(m, l, pc.whole ? p.sinks : nullptr, h, &inv, &lse_v);
      inv *= vscale;
      f0 *= inv;
      f1 *= inv;
      const bool has1 = alt && pc.nt > 1;
      if (live) {
        T* dst = static_cast<T*>(p.out) + static_cast<int64_t>(tok) * p.o_st +
                 static_cast<int64_t>(h) * p.o_sh;
        float* part = p.part_o +
                      (static_cast<int64_t>(pc.slot) * p.rows_cap + row) * D;
        // alternating streams share the columns of a row (16 at a time: a
        // loop that stays in the instruction cache; unrolled over 32 columns
        // of both accumulators an epilogue took 4500 clocks)
        const int c1 = alt ? (x + 1) * (D / 2) : D;
#pragma unroll 1
        for (int c = alt ? x * (D / 2) : 0; c < c1; c += 16) {
          float ov[16], o1[16];
          const uint32_t at = tmem + lane_base + C::O_COL + c;
          tmem_ld16(at + (alt ? 0 : x * C::S_STEP), ov);
          if (NX == 2 && has1) tmem_ld16(at + C::S_STEP, o1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            ov[e] *= f0;
            if (NX == 2 && has1) ov[e] += o1[e] * f1;
          }
          if (!valid) continue;
          uint32_t w[8];
          if (!pc.whole) {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(ov[k]);
            st_global_v8(part + c, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(ov[8 + k]);
            st_global_v8(part + c + 8, w);
            continue;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = pack2<T>(ov[2 * k], ov[2 * k + 1]);
          if (p.out_v8) {
            st_global_v8(dst + c, w);
          } else {
            *reinterpret_cast<uint4*>(dst + c) =
                make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + c + 8) =
                make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        if (valid && !(alt && x == 1)) {
          if (!pc.whole)
            p.part_lse[static_cast<int64_t>(pc.slot) * p.rows_cap + row] =
                lse_v;
          else if (p.lse)
            p.lse[static_cast<int64_t>(h) * p.total_q + tok] = lse_v;
        }
      }
      tc_fence_before();
      if (alt) {
        mbar_arrive(o_free(0));
        mbar_arrive(o_free(1));
      } else {
        // (counted for both streams' threads)
        for (int k = 0; k < NX; ++k) mbar_arrive(o_free(x));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // (the join leaves a unit alone that has a piece in a CTA that gave up)
  if (p.split && tid == 0) p.marks[2 * blockIdx.x + 1].y = *abort_flag;
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    asm volatile(
        "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem)
        : "memory");
  }
}

// Launches the kernel for one head size and kind of cache.
template <typename T, int D, int KV>
cudaError_t launch(const Params& p, const CUtensorMap& mk,
                   const CUtensorMap& mv, const CUtensorMap& mq, int grid,
                   const cudaLaunchAttribute* attr, cudaStream_t stream) {
  using C = Cfg<D, KV>;
  auto kern = tree_attn_kernel<T, D, KV>;
  cudaError_t e;
  if (C::SPLIT_REGS) {
    // the split inside the kernel adds up to the launch's registers (with fewer
    // it would wait for ever).  The build has made sure of the count, which is
    // the same on every device; it is asked for once.
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kern);
      if (e != cudaSuccess) return e;
      regs.store(fa.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) != C::LAUNCH_REGS)
      return cudaErrorInvalidConfiguration;
  }
  e = smem_opt_in(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = const_cast<cudaLaunchAttribute*>(attr);
  cfg.numAttrs = attr ? 1 : 0;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, p, mk, mv, mq);
}
template <typename T, int KV>
cudaError_t launch_d(const Params& p, int D, const CUtensorMap& mk,
                     const CUtensorMap& mv, const CUtensorMap& mq, int grid,
                     const cudaLaunchAttribute* attr, cudaStream_t stream) {
  switch (D) {
    case 64: return launch<T, 64, KV>(p, mk, mv, mq, grid, attr, stream);
    case 128: return launch<T, 128, KV>(p, mk, mv, mq, grid, attr, stream);
    case 256: return launch<T, 256, KV>(p, mk, mv, mq, grid, attr, stream);
  }
  return cudaErrorInvalidValue;
}
// Caches of codes (tree_codes.cu).
cudaError_t launch_codes(const Params& p, int D, bool bf16, int kv,
                         const CUtensorMap& mk, const CUtensorMap& mv,
                         const CUtensorMap& mq, int grid,
                         const cudaLaunchAttribute* attr, cudaStream_t stream);

}  // namespace tree
}  // namespace pkv
