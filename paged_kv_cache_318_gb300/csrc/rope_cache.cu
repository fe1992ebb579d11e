// Head norms and rotary positions of q and k in one pass, with the rotated
// keys and the values appended to a paged cache on the way.
//
// For a row x of D values (one head of one token), with the head norm
//   n = x * (1 / sqrt(mean(x^2) + eps)) * (w + offset)       (or n = x)
// and, for pair i < rot / 2 with c, s the table's entries at the position of
// the pair's axis,
//   y_a = n_a c - n_b s,   y_b = n_b c + n_a s
// where (a, b) = (i, i + rot / 2) ("neox") or (2 i, 2 i + 1); dimensions from
// rot on pass through.  All of it is float32 with one rounding at the end.
// The sum of squares is taken pairwise (neighbours first, error at most
// log2(D) half ulps), and the products of a rotation are rounded one by one,
// so a row's bits depend neither on the kernel that takes it nor on the rows
// beside it: a row that is quantized next has the same codes everywhere.
//
// A row is read once and written once (2 D + 2 D bytes for 16 bits), and the
// table row of a token once per warp that works on the token: HBM would bound
// it, and the instructions (about 17 a value) nearly do too.  Measured on a
// GB300 whose copy reaches 6.79 TB/s, back to back: 11207 tokens of 32/8
// heads, D 128, with norms into the 4-bit cache 48.5 us (5.1 TB/s, issue
// slots 65 % busy, 11 % of the SM time in the last wave of blocks), 8103
// tokens of 16/8 heads, D 256, into E4M3 47.3 us (5.1 TB/s), 8192 of them
// with 3 axes and no cache 45.3 us (4.6 TB/s); 64 tokens 5.4 us, all latency.
// What it took from 97, 85 and 60 us: packed float32 pairs, weights and
// table entries kept in registers over a token's rows, rows copied two
// passes ahead, quotients by a rounded reciprocal, pointers that walk.
// Measured and not kept: the token cut in two (3 axes 51 us against 45),
// three or more passes ahead (the same), six blocks an SM (spills).
//
// rope_kernel: a lane owns the 8-value chunks A and B of a row, rot / 2 apart,
// so that a rotation never leaves the lane and every load and store of a row
// is a run of whole 16-byte chunks; D / 16 lanes share a row and 512 / D rows
// make one pass of a warp.  A warp works through the passes of one token (all
// of them when there are many tokens, one when there are few) and keeps the
// token's cos and sin in registers.  It takes D = 64, 128, 256, rows on
// 16-byte boundaries, and rot = D / 2^n >= 32 (neox) or any multiple of 8
// (adjacent pairs).  rope_any_kernel takes everything else: one warp a row,
// through shared memory.
#include <type_traits>

#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxD = 512;
constexpr int kDepth = 2;        // passes on their way to a warp

// Axis whose position rotates pair i.
__device__ __forceinline__ int pair_axis(const RopeLaunch& p, int i) {
  if (p.axes == 1) return 0;
  if (p.woven) {
    const int a = i % p.axes;
    return i < p.axes * p.sections[a] ? a : 0;
  }
  int a = 0, end = p.sections[0];
  while (a + 1 < p.axes && i >= end) end += p.sections[++a];
  return a;
}

// The token's positions; false if the token is to be skipped: a negative
// position is padding, one past the table is flagged.
__device__ __forceinline__ bool read_positions(const RopeLaunch& p, int64_t t,
                                               bool flag, int64_t* pos) {
  bool ok = true, bad = false;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    if (a >= p.axes) break;
    pos[a] = __ldg(p.positions + a * p.pos_st + t);
    ok = ok && pos[a] >= 0;
    bad = bad || pos[a] >= p.max_position;
  }
  if (ok && bad && flag) atomicOr(p.err, kErrBadPosition);
  return ok && !bad;
}

// The token's cache row: -1 = none (padding, or flagged as outside).
__device__ __forceinline__ int64_t read_slot(const RopeLaunch& p, int64_t t,
                                             bool flag) {
  const int64_t s = __ldg(p.slots + t);
  if (s < 0) return -1;
  if (s >= p.num_slots) {
    if (flag) atomicOr(p.err, kErrBadSlot);
    return -1;
  }
  return s;
}

template <typename T>
__device__ __forceinline__ float table_at(const RopeLaunch& p, int64_t pos,
                                          int i) {
  const int64_t at = pos * p.table_st + i;
  return p.table_f32 ? __ldg(static_cast<const float*>(p.table) + at)
                     : to_f32<T>(static_cast<const T*>(p.table)[at]);
}

// N consecutive table entries of one row (16-byte aligned).
template <typename T, int N>
__device__ __forceinline__ void table_run(const RopeLaunch& p, int64_t pos,
                                          int i, float* out) {
  const int64_t at = pos * p.table_st + i;
  if (p.table_f32) {
    const float* src = static_cast<const float*>(p.table) + at;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src + j));
      out[j] = v.x;
      out[j + 1] = v.y;
      out[j + 2] = v.z;
      out[j + 3] = v.w;
    }
  } else {
    const T* src = static_cast<const T*>(p.table) + at;
    if constexpr (N == 8) {
      widen8<T>(__ldg(reinterpret_cast<const uint4*>(src)), out);
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
      out[0] = elem_f32<T>(v.x, 0);
      out[1] = elem_f32<T>(v.x, 1);
      out[2] = elem_f32<T>(v.y, 0);
      out[3] = elem_f32<T>(v.y, 1);
    }
  }
}

// Sums of squares of the four pairs of A and of B, neighbours first.
__device__ __forceinline__ uint64_t squares(const uint64_t* x) {
  uint64_t s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0, a1, b0, b1;
    unpair(mul2(x[i], x[i]), a0, a1);
    unpair(mul2(x[4 + i], x[4 + i]), b0, b1);
    s[i] = pair(__fadd_rn(a0, a1), __fadd_rn(b0, b1));
  }
  return add2(add2(s[0], s[1]), add2(s[2], s[3]));
}
__device__ __forceinline__ uint64_t shfl_xor2(uint64_t v, int o) {
  float a, b;
  unpair(v, a, b);
  return pair(__shfl_xor_sync(0xffffffffu, a, o),
              __shfl_xor_sync(0xffffffffu, b, o));
}

__device__ __forceinline__ float inv_rms(float sum, int D, float eps) {
  return __frcp_rn(__fsqrt_rn(
      __fadd_rn(__fdiv_rn(sum, static_cast<float>(D)), eps)));
}

// y_a, y_b of one pair.
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float ya = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float yb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = ya;
  b = yb;
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const uint64_t* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpair(x[i], a, b);
    w[i] = pack2<T>(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void widen8(const uint4& raw, uint64_t* x) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = pair(elem_f32<T>(w[i], 0), elem_f32<T>(w[i], 1));
}

__device__ __forceinline__ uint32_t e4m3_codes4(const float* x, float scale) {
  uint16_t lo, hi;
  // cvt puts its first operand in the upper byte
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo)
      : "f"(__fdiv_rn(x[1], scale)), "f"(__fdiv_rn(x[0], scale)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi)
      : "f"(__fdiv_rn(x[3], scale)), "f"(__fdiv_rn(x[2], scale)));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The E4M3 codes of four values, x / scale rounded to float32 first.  With
// y = fl(1 / scale) and q = fl(x y), q + fl(x - q scale) y is the correctly
// rounded quotient (Markstein 1990) where nothing over- or underflows: the
// scale is in [2^-60, 2^60] and x is cut to where every quotient saturates.
struct Fp8Scale {
  float scale, inv, limit;     // limit < 0: an ordinary division
};
__device__ __forceinline__ Fp8Scale fp8_scale(float scale) {
  Fp8Scale s;
  s.scale = scale;
  s.inv = __frcp_rn(scale);
  s.limit = scale >= 0x1p-60f && scale <= 0x1p60f ? 480.f * scale : -1.f;
  return s;
}
__device__ __forceinline__ uint64_t quotients(float x0, float x1,
                                              const Fp8Scale& s) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x0) : "f"(s.limit));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x0) : "f"(-s.limit));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x1) : "f"(s.limit));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x1) : "f"(-s.limit));
  const uint64_t x = pair(x0, x1), y = pair(s.inv, s.inv);
  const uint64_t q = mul2(x, y);
  return fma2(fma2(q, pair(-s.scale, -s.scale), x), y, q);
}
__device__ __forceinline__ uint32_t e4m3_codes4(const float* x,
                                                const Fp8Scale& s) {
  if (s.limit < 0.f) return e4m3_codes4(x, s.scale);
  float q[4];
  unpair(quotients(x[0], x[1], s), q[0], q[1]);
  unpair(quotients(x[2], x[3], s), q[2], q[3]);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo)
      : "f"(q[1]), "f"(q[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi)
      : "f"(q[3]), "f"(q[2]));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// How the pairs lie: (i, i + D / 2) over the whole row, (i, i + rot / 2) over
// a part of it, or neighbours.
enum { kWhole = 0, kPart = 1, kNeighbours = 2 };

template <typename T, int D, int STORE, int PAIRS>
__global__ void __launch_bounds__(kThreads, 5)
rope_kernel(const RopeLaunch p, int parts) {
  // an attention kernel queued next as a programmatic dependent may become
  // resident now (it waits for this grid before reading what this writes)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr bool NEOX = PAIRS != kNeighbours;
  constexpr int LPR = D / 16;             // lanes of a row
  constexpr int RPW = 32 / LPR;           // rows of a pass
  const int lane = threadIdx.x & 31;
  const int j = lane % LPR, sub = lane / LPR;
  // chunk numbers: inside each block of `span` values, A is in the first
  // half and B at the same place of the second
  const int span = PAIRS == kPart ? p.rot : D;
  const int nb = span / 16;               // lanes of a span
  const int blk0 = j / nb;
  const int ca = blk0 * (span / 8) + (j - blk0 * nb), cb = ca + nb;
  const bool rot_a = PAIRS == kWhole || 8 * ca < p.rot;
  const bool rot_b = PAIRS == kWhole || 8 * cb < p.rot;
  const int half = PAIRS == kWhole ? D / 2 : p.rot / 2;
  const uint64_t one2 = pair(p.one, p.one), minus2 = pair(-p.one, -p.one);
  // the lane's first pair of each four (adjacent pairs) or of the eight
  const int ia = NEOX ? 8 * ca : 4 * ca, ib = NEOX ? ia + 4 : 4 * cb;
  const int pq = (p.Hq + RPW - 1) / RPW, pk = (p.Hkv + RPW - 1) / RPW;
  // is this lane's row there in the last pass of q, of k and v?
  const bool q_last = (pq - 1) * RPW + sub < p.Hq;
  const bool k_last = (pk - 1) * RPW + sub < p.Hkv;
  __shared__ uint4 places[kDepth * 2 * kThreads];
  const uint32_t mine = smem_u32(places + threadIdx.x);
  const int64_t work = p.num_tokens * parts;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) +
                   (threadIdx.x >> 5);
       w < work; w += step) {
    const int64_t t = parts == 1 ? w : w / parts;
    const int part = parts == 1 ? 0 : static_cast<int>(w - t * parts);
    // The token's passes part, part + parts, ... in the order q, k, v; every
    // thread copies its own chunks of the next kDepth ones to its own places
    // in shared memory (nothing of them waits for the position or the slot).
    // `src` walks down the heads of one kind.
    int kind = 0, left = pq - part;       // of the pass that is next
    const T* src = static_cast<const T*>(p.q) + t * p.q_st +
                   (part * RPW + sub) * p.q_sh + 8 * ca;
    int64_t down = parts * RPW * p.q_sh;
    auto issue = [&](int i) {
      while (left <= 0 && kind < (STORE == kRopeRows ? 1 : 2)) {
        const int h = -left * RPW + sub;
        ++kind;
        left += pk;
        const int64_t sh = kind == 1 ? p.k_sh : p.v_sh;
        src = (kind == 1 ? static_cast<const T*>(p.k) + t * p.k_st
                         : static_cast<const T*>(p.v) + t * p.v_st) +
              h * sh + 8 * ca;
        down = parts * RPW * sh;
      }
      if (left > 0) {
        // (the last pass of a kind may have fewer rows)
        const int bytes = left > 1 || (kind == 0 ? q_last : k_last) ? 16 : 0;
        const T* at = bytes ? src : static_cast<const T*>(p.k);
        const uint32_t dst = mine + (i % kDepth) * (kThreads * 32);
        cp_async_16(dst, at, bytes);
        cp_async_16(dst + kThreads * 16, at + 8 * (cb - ca), bytes);
        left -= parts;
        src += down;
      }
      cp_async_commit();
    };
    for (int i = 0; i < kDepth; ++i) issue(i);
    int done = 0;                         // passes worked on
    int64_t slot = -1, blk = 0, off = 0;
    if constexpr (STORE != kRopeRows)
      slot = read_slot(p, t, part == 0 && lane == 0);
    int64_t pos[4] = {0, 0, 0, 0};
    if (!read_positions(p, t, part == 0 && lane == 0, pos)) {
      cp_async_wait<0>();                 // (nothing reads these rows)
      continue;
    }
    if (STORE != kRopeRows && slot >= 0)
      split_slot(slot, p.BS, p.bs_shift, &blk, &off);
    // cos and sin of the lane's eight pairs, two to an operand
    uint64_t c[4], s[4];
    {
      float cf[8], sf[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) cf[e] = sf[e] = 0.f;
      if (p.axes == 1) {
        if constexpr (NEOX) {
          if (rot_a) {
            table_run<T, 8>(p, pos[0], ia, cf);
            table_run<T, 8>(p, pos[0], half + ia, sf);
          }
        } else {
          if (rot_a) {
            table_run<T, 4>(p, pos[0], ia, cf);
            table_run<T, 4>(p, pos[0], half + ia, sf);
          }
          if (rot_b) {
            table_run<T, 4>(p, pos[0], ib, cf + 4);
            table_run<T, 4>(p, pos[0], half + ib, sf + 4);
          }
        }
      } else {
        int woven = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = e < 4 ? ia + e : ib + e - 4;
          if (i >= half) continue;
          int a;
          if (p.woven) {               // i mod axes, counted on
            woven = e == 0 || e == 4 ? i % p.axes
                                     : woven + 1 == p.axes ? 0 : woven + 1;
            a = i < p.axes * p.sections[woven] ? woven : 0;
          } else {
            a = pair_axis(p, i);
          }
          const int64_t at = a == 0 ? pos[0]
                             : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
          cf[e] = table_at<T>(p, at, i);
          sf[e] = table_at<T>(p, at, half + i);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[e] = pair(cf[2 * e], cf[2 * e + 1]);
        s[e] = pair(sf[2 * e], sf[2 * e + 1]);
      }
    }

    // The passes of one kind of row (q, k or v).
    int before = 0;                       // passes of the kinds before
    auto rows = [&](auto kind_tag, int H, const T* weight, auto&& store) {
      constexpr int kind = decltype(kind_tag)::value;
      const int n = (H + RPW - 1) / RPW;
      int i = part + done * parts - before;
      before += n;
      if (i >= n) return;
      uint64_t wv[8];
      if (kind < 2 && p.norm) {
        widen8<T>(__ldg(reinterpret_cast<const uint4*>(weight + 8 * ca)), wv);
        widen8<T>(__ldg(reinterpret_cast<const uint4*>(weight + 8 * cb)),
                  wv + 4);
        const uint64_t o = pair(p.weight_offset, p.weight_offset);
#pragma unroll
        for (int e = 0; e < 8; ++e) wv[e] = add2(wv[e], o);
      }
      for (; i < n; i += parts) {
        const int h = i * RPW + sub;
        cp_async_wait<kDepth - 1>();
        const uint32_t place = mine + (done % kDepth) * (kThreads * 32);
        const uint4 now[2] = {lds128(place), lds128(place + kThreads * 16)};
        issue(done + kDepth);
        ++done;
        uint64_t x[8];
        widen8<T>(now[0], x);
        widen8<T>(now[1], x + 4);
        if (kind < 2) {
          if (p.norm) {
            uint64_t ab = squares(x);
            float sa, sb;
            // neighbours first: lanes of the span, then A with B, then spans
            if (PAIRS != kPart) {
#pragma unroll
              for (int o = 1; o < LPR; o *= 2) ab = add2(ab, shfl_xor2(ab, o));
              unpair(ab, sa, sb);
              sa = __fadd_rn(sa, sb);
            } else {
              for (int o = 1; o < nb; o *= 2) ab = add2(ab, shfl_xor2(ab, o));
              unpair(ab, sa, sb);
              sa = __fadd_rn(sa, sb);
              for (int o = nb; o < LPR; o *= 2)
                sa = __fadd_rn(sa, __shfl_xor_sync(0xffffffffu, sa, o));
            }
            // (D is a power of two: the product is the quotient)
            const float r = __frcp_rn(__fsqrt_rn(
                __fadd_rn(__fmul_rn(sa, 1.f / D), p.eps)));
            const uint64_t r2 = pair(r, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = mul2(mul2(x[e], r2), wv[e]);
          }
          if constexpr (NEOX) {
            if (rot_a) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // (the sums as x 1 + y, with a 1 that is not known here: a
                // packed sum of products would come out as one fused
                // multiply-add)
                const uint64_t a = x[e], b = x[4 + e];
                x[e] = fma2(mul2(b, s[e]), minus2, mul2(a, c[e]));
                x[4 + e] = fma2(mul2(b, c[e]), one2, mul2(a, s[e]));
              }
            }
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (!(q ? rot_b : rot_a)) continue;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float a, b, cc[2], ss[2];
                unpair(x[4 * q + e], a, b);
                unpair(c[2 * q + (e >> 1)], cc[0], cc[1]);
                unpair(s[2 * q + (e >> 1)], ss[0], ss[1]);
                rotate(a, b, cc[e & 1], ss[e & 1]);
                x[4 * q + e] = pair(a, b);
              }
            }
          }
        }
        store(h, h < H, x, now);
      }
    };
    auto row_store = [&](T* base, int64_t sh) {
      return [=](int h, bool on, const uint64_t* x, const uint4*) {
        if (!on) return;
        T* dst = base + h * sh;
        *reinterpret_cast<uint4*>(dst + 8 * ca) = pack8<T>(x);
        *reinterpret_cast<uint4*>(dst + 8 * cb) = pack8<T>(x + 4);
      };
    };
    // For the 4-bit cache, chunks 2 m and 2 m + 1 share a block scale: they
    // are a lane's and its neighbour's (lane ^ 1) chunks.
    auto cache_store = [&](auto value_tag) {
      constexpr bool value = decltype(value_tag)::value != 0;
      const int64_t row = blk * p.c_sb + off * p.c_sr;
      [[maybe_unused]] const int64_t frow = blk * p.f_sb + off * p.f_sr;
      const float scale =
          STORE < kRopeCacheFp8 ? 1.f : value ? *p.v_scale : *p.k_scale;
      [[maybe_unused]] const float sixth =
          STORE == kRopeCacheFp4 ? fp4_sixth(scale) : 0.f;
      const Fp8Scale s8 = STORE == kRopeCacheFp8 ? fp8_scale(scale)
                                                 : Fp8Scale{};
      return [=, &p](int h, bool on, const uint64_t* x, const uint4* raw) {
        void* base = value ? p.vc : p.kc;
        if constexpr (STORE == kRopeCache16) {
          if (!on) return;
          T* dst = static_cast<T*>(base) + row + h * p.c_sh;
          *reinterpret_cast<uint4*>(dst + 8 * ca) =
              value ? raw[0] : pack8<T>(x);
          *reinterpret_cast<uint4*>(dst + 8 * cb) =
              value ? raw[1] : pack8<T>(x + 4);
        } else {
          float f[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) unpair(x[e], f[2 * e], f[2 * e + 1]);
          uint8_t* dst = static_cast<uint8_t*>(base) + row + h * p.c_sh;
          if constexpr (STORE == kRopeCacheFp8) {
            if (!on) return;
            *reinterpret_cast<uint2*>(dst + 8 * ca) =
                make_uint2(e4m3_codes4(f, s8), e4m3_codes4(f + 4, s8));
            *reinterpret_cast<uint2*>(dst + 8 * cb) =
                make_uint2(e4m3_codes4(f + 8, s8), e4m3_codes4(f + 12, s8));
          } else {
            // (the even lane takes the scale of both lanes' A, the odd lane
            // of both lanes' B)
            const bool odd = lane & 1;
            float m[2] = {0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                m[q] = max_nan(m[q], fabsf(f[8 * q + e]));
            const float top = max_nan(
                odd ? m[1] : m[0],
                __shfl_xor_sync(0xffffffffu, odd ? m[0] : m[1], 1));
            const Fp4Scale sc = fp4_scale(top, scale, sixth);
            const float other = __shfl_xor_sync(0xffffffffu, sc.inv, 1);
            if (!on) return;
            uint8_t* sf = (value ? p.v_sf : p.k_sf) + frow + h * p.f_sh;
            *reinterpret_cast<uint32_t*>(dst + 4 * ca) =
                fp4_codes8(f, odd ? other : sc.inv);
            *reinterpret_cast<uint32_t*>(dst + 4 * cb) =
                fp4_codes8(f + 8, odd ? sc.inv : other);
            sf[(odd ? cb : ca) >> 1] = static_cast<uint8_t>(sc.code);
          }
        }
      };
    };
    using Q = std::integral_constant<int, 0>;
    using K = std::integral_constant<int, 1>;
    using V = std::integral_constant<int, 2>;
    rows(Q{}, p.Hq, static_cast<const T*>(p.q_weight),
         row_store(static_cast<T*>(p.q_out) + t * p.qo_st, p.qo_sh));
    if constexpr (STORE == kRopeRows) {
      rows(K{}, p.Hkv, static_cast<const T*>(p.k_weight),
           row_store(static_cast<T*>(p.k_out) + t * p.ko_st, p.ko_sh));
    } else if (slot >= 0) {
      rows(K{}, p.Hkv, static_cast<const T*>(p.k_weight),
           cache_store(Q{}));
      rows(V{}, p.Hkv, static_cast<const T*>(nullptr), cache_store(K{}));
    } else {
      cp_async_wait<0>();                 // (nothing reads rows of k and v)
    }
  }
}

// Any head size (a multiple of 8 up to 512), rotation width, stride and
// alignment: one warp a row.
template <typename T, int STORE>
__global__ void __launch_bounds__(kThreads)
rope_any_kernel(const RopeLaunch p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float rows[kThreads / 32][2][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* xs = rows[warp][0];
  float* ys = rows[warp][1];
  const int D = p.D, half = p.rot / 2;
  int dp = 32;                            // D up to a power of two
  while (dp < D) dp *= 2;
  const int per = dp / 32;
  const int heads = p.Hq + (STORE == kRopeRows ? p.Hkv : 2 * p.Hkv);
  const int64_t work = p.num_tokens * heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp;
       w < work; w += step) {
    const int64_t t = w / heads;
    const int r = static_cast<int>(w - t * heads);
    const int kind = r < p.Hq ? 0 : r < p.Hq + p.Hkv ? 1 : 2;
    const int h = kind == 0 ? r : kind == 1 ? r - p.Hq : r - p.Hq - p.Hkv;
    int64_t pos[4] = {0, 0, 0, 0};
    if (!read_positions(p, t, r == 0 && lane == 0, pos)) continue;
    int64_t slot = -1, blk = 0, off = 0;
    if constexpr (STORE != kRopeRows) {
      slot = read_slot(p, t, r == 0 && lane == 0);
      if (kind > 0 && slot < 0) continue;
      if (slot >= 0) split_slot(slot, p.BS, p.bs_shift, &blk, &off);
    }
    const T* src = static_cast<const T*>(kind == 0   ? p.q
                                         : kind == 1 ? p.k
                                                     : p.v) +
                   t * (kind == 0 ? p.q_st : kind == 1 ? p.k_st : p.v_st) +
                   h * (kind == 0 ? p.q_sh : kind == 1 ? p.k_sh : p.v_sh);
    __syncwarp();                         // the row before is done
    for (int d = lane; d < D; d += 32) xs[d] = to_f32<T>(src[d]);
    __syncwarp();
    float* ready = xs;
    if (kind < 2) {
      if (p.norm) {
        float sq[kMaxD / 32];
#pragma unroll
        for (int e = 0; e < kMaxD / 32; ++e) {
          const int d = lane * per + e;
          sq[e] = e < per && d < D ? __fmul_rn(xs[d], xs[d]) : 0.f;
        }
#pragma unroll
        for (int n = 1; n < kMaxD / 32; n *= 2)
#pragma unroll
          for (int e = 0; e + n < kMaxD / 32; e += 2 * n)
            if (n < per) sq[e] = __fadd_rn(sq[e], sq[e + n]);
        float sum = sq[0];
#pragma unroll
        for (int o = 1; o < 32; o *= 2)
          sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
        const float rms = inv_rms(sum, D, p.eps);
        const T* wt = static_cast<const T*>(kind == 0 ? p.q_weight
                                                      : p.k_weight);
        __syncwarp();
        for (int d = lane; d < D; d += 32)
          xs[d] = __fmul_rn(__fmul_rn(xs[d], rms),
                            __fadd_rn(to_f32<T>(wt[d]), p.weight_offset));
        __syncwarp();
      }
      for (int d = lane; d < D; d += 32) {
        float v = xs[d];
        if (d < p.rot) {
          const int i = p.neox ? (d < half ? d : d - half) : d >> 1;
          const bool second = p.neox ? d >= half : (d & 1);
          const int other = p.neox ? (second ? d - half : d + half) : d ^ 1;
          const int a = pair_axis(p, i);
          const int64_t at = a == 0 ? pos[0]
                             : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
          float lo = second ? xs[other] : v, hi = second ? v : xs[other];
          rotate(lo, hi, table_at<T>(p, at, i), table_at<T>(p, at, half + i));
          v = second ? hi : lo;
        }
        ys[d] = v;
      }
      ready = ys;
      __syncwarp();
    }
    if (kind == 0 || STORE == kRopeRows) {
      T* dst = static_cast<T*>(kind == 0 ? p.q_out : p.k_out) +
               t * (kind == 0 ? p.qo_st : p.ko_st) +
               h * (kind == 0 ? p.qo_sh : p.ko_sh);
      for (int d = lane; d < D; d += 32) dst[d] = from_f32<T>(ready[d]);
      continue;
    }
    const int64_t row = blk * p.c_sb + off * p.c_sr + h * p.c_sh;
    void* base = kind == 2 ? p.vc : p.kc;
    const float scale = STORE < kRopeCacheFp8 ? 1.f
                        : kind == 2           ? *p.v_scale
                                              : *p.k_scale;
    if constexpr (STORE == kRopeCache16) {
      T* dst = static_cast<T*>(base) + row;
      // a value row is copied bit for bit, NaN payloads included
      for (int d = lane; d < D; d += 32)
        dst[d] = kind == 2 ? src[d] : from_f32<T>(ready[d]);
    } else if constexpr (STORE == kRopeCacheFp8) {
      uint8_t* dst = static_cast<uint8_t*>(base) + row;
      for (int d = lane * 4; d < D; d += 128) {
        const uint32_t codes = e4m3_codes4(ready + d, scale);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dst[d + e] = static_cast<uint8_t>(codes >> (8 * e));
      }
    } else if constexpr (STORE == kRopeCacheFp4) {
      uint8_t* dst = static_cast<uint8_t*>(base) + row;
      uint8_t* sf = (kind == 2 ? p.v_sf : p.k_sf) + blk * p.f_sb +
                    off * p.f_sr + h * p.f_sh;
      for (int g = lane; g < D / 16; g += 32) {
        float top = 0.f;
        for (int e = 0; e < 16; ++e)
          top = max_nan(top, fabsf(ready[16 * g + e]));
        const Fp4Scale s = fp4_scale(top, scale, fp4_sixth(scale));
        for (int e = 0; e < 2; ++e) {
          const uint32_t codes = fp4_codes8(ready + 16 * g + 8 * e, s.inv);
          for (int b = 0; b < 4; ++b)
            dst[8 * g + 4 * e + b] = static_cast<uint8_t>(codes >> (8 * b));
        }
        sf[g] = static_cast<uint8_t>(s.code);
      }
    }
  }
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// rope_kernel's conditions (see the head of this file).
bool whole_chunks(const RopeLaunch& p, RopeStore store) {
  if (p.D != 64 && p.D != 128 && p.D != 256) return false;
  if (p.neox) {
    if (p.rot < 32 || p.D % p.rot || (p.rot & (p.rot - 1))) return false;
  } else if (p.rot % 8) {
    return false;
  }
  const int tb = p.table_f32 ? 4 : 2;
  // a lane reads 8 (neox) or 4 (adjacent pairs) entries from each half row
  const int run = (p.neox ? 8 : 4) * tb < 16 ? (p.neox ? 8 : 4) * tb : 16;
  if (p.axes == 1 &&
      (reinterpret_cast<uintptr_t>(p.table) % run || p.table_st * tb % run ||
       p.rot / 2 * tb % run))
    return false;
  auto rows16 = [](const void* b, int64_t st, int64_t sh) {
    return on16(b) && st % 8 == 0 && sh % 8 == 0;
  };
  if (p.Hq && (!rows16(p.q, p.q_st, p.q_sh) ||
               !rows16(p.q_out, p.qo_st, p.qo_sh)))
    return false;
  if (!rows16(p.k, p.k_st, p.k_sh)) return false;
  if (!on16(p.q_weight) || !on16(p.k_weight)) return false;
  if (store == kRopeRows) return rows16(p.k_out, p.ko_st, p.ko_sh);
  if (!rows16(p.v, p.v_st, p.v_sh)) return false;
  // a lane's store: 16 bytes (16-bit), 8 (E4M3) or 4 (4-bit)
  const int unit = store == kRopeCache16 ? 8 : store == kRopeCacheFp8 ? 8 : 4;
  const int bytes = store == kRopeCache16 ? 16 : unit;
  return reinterpret_cast<uintptr_t>(p.kc) % bytes == 0 &&
         reinterpret_cast<uintptr_t>(p.vc) % bytes == 0 &&
         p.c_sb % unit == 0 && p.c_sr % unit == 0 && p.c_sh % unit == 0;
}

template <typename T, int D, int STORE>
cudaError_t launch_chunks(const RopeLaunch& p, cudaStream_t stream) {
  constexpr int rpw = 512 / D;
  const int pk = (p.Hkv + rpw - 1) / rpw;
  const int passes = (p.Hq + rpw - 1) / rpw + (STORE ? 2 : 1) * pk;
  // one warp works through a token, or through a part of one while the
  // warps would not fill the GPU
  const int64_t fill = static_cast<int64_t>(current_sm_count()) * 32;
  int64_t parts = (fill + p.num_tokens - 1) / p.num_tokens;
  if (parts > passes) parts = passes;
  const int64_t blocks = (p.num_tokens * parts + kThreads / 32 - 1) /
                         (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(current_sm_count()) * 64;
  const unsigned grid = static_cast<unsigned>(blocks < cap ? blocks : cap);
  note_launch();
  auto go = [&](auto kern) {
    kern<<<grid, kThreads, 0, stream>>>(p, static_cast<int>(parts));
  };
  if (!p.neox)
    go(rope_kernel<T, D, STORE, kNeighbours>);
  else if (p.rot == D)
    go(rope_kernel<T, D, STORE, kWhole>);
  else
    go(rope_kernel<T, D, STORE, kPart>);
  return cudaGetLastError();
}

template <typename T, int STORE>
cudaError_t launch_store(const RopeLaunch& p, cudaStream_t stream) {
  if (whole_chunks(p, static_cast<RopeStore>(STORE))) {
    switch (p.D) {
      case 64: return launch_chunks<T, 64, STORE>(p, stream);
      case 128: return launch_chunks<T, 128, STORE>(p, stream);
      default: return launch_chunks<T, 256, STORE>(p, stream);
    }
  }
  const int64_t rows = p.num_tokens *
                       (p.Hq + (STORE == kRopeRows ? 1 : 2) * p.Hkv);
  const int64_t blocks = (rows + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(current_sm_count()) * 16;
  note_launch();
  rope_any_kernel<T, STORE>
      <<<static_cast<unsigned>(blocks < cap ? blocks : cap), kThreads, 0,
         stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RopeLaunch& p, RopeStore store,
                        cudaStream_t stream) {
  switch (store) {
    case kRopeRows: return launch_store<T, kRopeRows>(p, stream);
    case kRopeCache16: return launch_store<T, kRopeCache16>(p, stream);
    case kRopeCacheFp8: return launch_store<T, kRopeCacheFp8>(p, stream);
    default: return launch_store<T, kRopeCacheFp4>(p, stream);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& launch, RopeStore store, bool bf16,
                        cudaStream_t stream) {
  if (launch.num_tokens == 0) return cudaSuccess;
  RopeLaunch p = launch;
  p.one = 1.f;
  p.bs_shift = shift_of(p.BS);
  return bf16 ? launch_type<__nv_bfloat16>(p, store, stream)
              : launch_type<__half>(p, store, stream);
}

}  // namespace pkv
