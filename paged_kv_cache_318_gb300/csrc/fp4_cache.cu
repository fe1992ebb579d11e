// 4-bit KV cache: the quantizing write and the read-back.
//
// A cache row of D values is D / 2 bytes of E2M1 codes (two to a byte, the
// lower index in the lower four bits) and D / 16 E4M3 scales, one for each 16
// values; one float32 scale covers the whole tensor.  A value reads back as
// code * block scale * tensor scale.  The code (2 significant bits) times the
// block scale (4) has at most 6, and its exponent fits both 16-bit types, so
// that product is exact in bf16 and f16: the prefill kernels run on exact
// 16-bit copies of the pages and fold the tensor scales into the logit scale
// and the output, as they do for E4M3 caches.
//
// All three kernels stream: HBM bounds them (the write reads 2 D and writes
// D / 2 + D / 16 bytes a row, the read-back the reverse).
//
// The write: a thread owns one group of 16 values, so a group's maximum, its
// scale and its codes never leave the thread; the next group loads while one
// is quantized (its row does not wait for its slot), three blocks of 256
// threads an SM.  Measured on a GB300 whose copy reaches 6.79 TB/s: 11207
// tokens of 8 heads, D 128, 14.9 us back to back (3.95 TB/s; 18.4 us without
// the loads ahead), of which a launch is about 3; 124 tokens 4.8 us, all
// latency.
//
// The read-back: a thread turns 8 codes into 16 bytes and has four rows of
// each matrix loading at once; the page copy of 8 prompts (20 MB of codes
// into 83 MB) costs 24 us before the prefill kernel, 31 with 16 values a
// thread and one row at a time.
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// 16 consecutive 16-bit values -> 8 bytes of codes and the group's scale.
template <typename T>
__device__ __forceinline__ void quantize16(uint4 r0, uint4 r1, float scale,
                                           float sixth, uint8_t* codes,
                                           uint8_t* sf) {
  float x[16];
  widen8<T>(r0, x);
  widen8<T>(r1, x + 8);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max_nan(top, fabsf(x[i]));
  const Fp4Scale s = fp4_scale(top, scale, sixth);
  *reinterpret_cast<uint2*>(codes) =
      make_uint2(fp4_codes8(x, s.inv), fp4_codes8(x + 8, s.inv));
  *sf = static_cast<uint8_t>(s.code);
}

// 8 codes and their group's scale -> 8 values; with `scaled`, times `scale`
// before the rounding to T (else the exact product alone).
template <typename T>
__device__ __forceinline__ uint4 dequantize8(uint32_t codes, uint32_t sf,
                                             bool scaled, float scale) {
  const uint32_t s2 = e4m3x2_to_f16(sf * 0x0101u);
  uint32_t o[4], f[4];
  e2m1x8_to_f16(codes, f[0], f[1], f[2], f[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = hmul2_u32(f[i], s2);
    const __half2 hv = *reinterpret_cast<const __half2*>(&v);
    float a = __low2float(hv), b = __high2float(hv);
    if (scaled) {
      a = __fmul_rn(a, scale);
      b = __fmul_rn(b, scale);
    }
    o[i] = pack2<T>(a, b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The block's threads cover whole tokens: thread i takes group i % per_token
// of token i / per_token (a token with more groups than threads is looped
// over), so the index math runs once per thread.
template <typename T>
__global__ void __launch_bounds__(kThreads)
cache_write_fp4_kernel(const T* __restrict__ key, const T* __restrict__ value,
                       int64_t k_st, int64_t k_sh, int64_t v_st, int64_t v_sh,
                       uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                       int64_t c_sb, int64_t c_sr, int64_t c_sh,
                       uint8_t* __restrict__ k_sf, uint8_t* __restrict__ v_sf,
                       int64_t f_sb, int64_t f_sr, int64_t f_sh,
                       const int64_t* __restrict__ slots, int64_t num_tokens,
                       int groups, int group_shift, int per_token,
                       int tokens_per_block, int BS, int bs_shift,
                       int64_t num_slots,
                       const float* __restrict__ k_scale,
                       const float* __restrict__ v_scale, unsigned* err) {
  // an attention kernel queued next as a programmatic dependent may become
  // resident now (it waits for this grid before reading the cache)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tl = threadIdx.x / per_token;
  if (tl >= tokens_per_block) return;
  const int r0 = threadIdx.x - tl * per_token;
  const float ks = *k_scale, vs = *v_scale;
  const float ks6 = fp4_sixth(ks), vs6 = fp4_sixth(vs);
  const int64_t step = static_cast<int64_t>(gridDim.x) * tokens_per_block;
  int64_t t = static_cast<int64_t>(blockIdx.x) * tokens_per_block + tl;
  // the next item's rows and slot load while this one's are worked on (and
  // the rows do not wait for the slot)
  struct Item {
    uint4 k0, k1, v0, v1;
    int64_t slot;
  };
  auto load = [&](int64_t tok, int r, Item& x) {
    const int h = group_shift >= 0 ? r >> group_shift : r / groups;
    const int g = r - h * groups;
    const uint4* kp =
        reinterpret_cast<const uint4*>(key + tok * k_st + h * k_sh + g * 16);
    const uint4* vp =
        reinterpret_cast<const uint4*>(value + tok * v_st + h * v_sh + g * 16);
    x.slot = __ldg(slots + tok);
    x.k0 = kp[0];
    x.k1 = kp[1];
    x.v0 = vp[0];
    x.v1 = vp[1];
  };
  int r = r0;
  Item x;
  if (t < num_tokens) load(t, r, x);
  while (t < num_tokens) {
    const Item now = x;
    const int r_now = r;
    r += kThreads;                                // (a large token's rest)
    if (r >= per_token) {
      r = r0;
      t += step;
    }
    if (t < num_tokens) load(t, r, x);
    if (now.slot < 0) continue;                   // padding slot
    if (now.slot >= num_slots) {                  // outside the cache: skip
      if (r_now == 0) atomicOr(err, kErrBadSlot);
      continue;
    }
    int64_t blk, off;
    split_slot(now.slot, BS, bs_shift, &blk, &off);
    const int h = group_shift >= 0 ? r_now >> group_shift : r_now / groups;
    const int g = r_now - h * groups;
    const int64_t c = blk * c_sb + off * c_sr + h * c_sh + g * 8;
    const int64_t f = blk * f_sb + off * f_sr + h * f_sh + g;
    quantize16<T>(now.k0, now.k1, ks, ks6, kc + c, k_sf + f);
    quantize16<T>(now.v0, now.v1, vs, vs6, vc + c, v_sf + f);
  }
}

// One block of rows, [BS, Hkv, D] values from the codes of MATS matrices
// (whose caches share their strides).  A thread turns 8 codes into 16 bytes,
// so a warp stores 512 bytes in a row; it keeps its place in the row and
// walks down the rows, kRows of each matrix loading at once.
constexpr int kRows = 4;
template <typename T, int MATS>
__device__ __forceinline__ void dequantize_block(
    const uint8_t* const (&codes)[MATS], const uint8_t* const (&sf)[MATS],
    int64_t c_sr, int64_t c_sh, int64_t f_sr, int64_t f_sh, int BS, int Hkv,
    int groups, bool bad, bool scaled, float scale, T* const (&out)[MATS]) {
  const int eighths = 2 * groups, per_row = Hkv * eighths;
  // whole rows at a time (a row of more eighths than threads is looped over)
  const int rows = per_row >= kThreads ? 1 : kThreads / per_row;
  const int row0 = per_row >= kThreads ? 0 : threadIdx.x / per_row;
  if (row0 >= rows) return;
  for (int r = threadIdx.x - row0 * per_row; r < per_row; r += kThreads) {
    const int h = r / eighths, g = r - h * eighths;
    const int64_t c = h * c_sh + g * 4, f = h * f_sh + (g >> 1);
    for (int row = row0; row < BS; row += rows * kRows) {
      uint32_t code[kRows][MATS], s[kRows][MATS];
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          const int64_t at = row + i * rows;
          code[i][m] = s[i][m] = 0;               // (zeros)
          if (at < BS && !bad) {
            code[i][m] = __ldg(reinterpret_cast<const uint32_t*>(
                codes[m] + at * c_sr + c));
            s[i][m] = __ldg(sf[m] + at * f_sr + f);
          }
        }
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          const int64_t at = row + i * rows;
          if (at < BS)
            *reinterpret_cast<uint4*>(out[m] + (at * per_row + r) * 8) =
                dequantize8<T>(code[i][m], s[i][m], scaled, scale);
        }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
fp4_dequant_blocks_kernel(const uint8_t* __restrict__ codes, int64_t c_sb,
                          int64_t c_sr, int64_t c_sh,
                          const uint8_t* __restrict__ sf, int64_t f_sb,
                          int64_t f_sr, int64_t f_sh,
                          const float* __restrict__ scale,
                          const int64_t* __restrict__ ids, int64_t n,
                          int64_t num_blocks, int Hkv, int groups, int BS,
                          T* __restrict__ out, unsigned* err) {
  const float sc = *scale;
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int64_t blk = ids ? __ldg(ids + i) : i;
    const bool bad = blk < 0 || blk >= num_blocks;
    if (bad && threadIdx.x == 0) atomicOr(err, kErrBadBlock);
    const uint8_t* c[1] = {codes + (bad ? 0 : blk * c_sb)};
    const uint8_t* f[1] = {sf + (bad ? 0 : blk * f_sb)};
    T* const o[1] = {out + i * BS * Hkv * groups * 16};
    dequantize_block<T, 1>(c, f, c_sr, c_sh, f_sr, f_sh, BS, Hkv, groups, bad,
                           true, sc, o);
  }
}

// The pages of prefill-class requests as exact 16-bit copies: page j of
// request b is block b * max_blocks + j of the copies (the contract of
// launch_fp8_dequant_pages).
template <typename T>
__global__ void __launch_bounds__(kThreads)
fp4_dequant_pages_kernel(const AttnParams p, T* __restrict__ mock_k,
                         T* __restrict__ mock_v, int32_t* __restrict__ table,
                         int groups) {
  const int64_t pages = static_cast<int64_t>(p.batch) * p.max_blocks;
  const int64_t elems = static_cast<int64_t>(p.BS) * p.Hkv * groups * 16;
  // (the item counter of the prefill kernel that follows)
  if (p.sched && blockIdx.x == 0 && threadIdx.x == 0) *p.sched = 0;
  for (int64_t m = blockIdx.x; m < pages; m += gridDim.x) {
    const int b = static_cast<int>(
        pages <= 0xffffffffLL ? static_cast<unsigned>(m) /
                                    static_cast<unsigned>(p.max_blocks)
                              : m / p.max_blocks);
    const int j = static_cast<int>(m - static_cast<int64_t>(b) *
                                           p.max_blocks);
    if (threadIdx.x == 0) table[m] = static_cast<int32_t>(m);
    // (four loads in flight at once)
    const int q0 = p.cu_q[b];
    const int L = p.seqused_k[b];
    const int blk = p.block_table[static_cast<int64_t>(b) * p.bt_stride + j];
    const int q_len = min(p.cu_q[b + 1] - q0, p.total_q - q0);
    if (q0 < 0 || q_len <= 0 || q_len * p.G < p.min_rows) continue;
    const int64_t L_tab = min(static_cast<int64_t>(L),
                              static_cast<int64_t>(p.max_blocks) * p.BS);
    if (static_cast<int64_t>(j) * p.BS >= L_tab) continue;
    const bool bad = blk < 0 || blk >= p.num_blocks;
    if (bad && threadIdx.x == 0) atomicOr(p.err, kErrBadBlock);
    const int64_t co = bad ? 0 : blk * p.c_sb, fo = bad ? 0 : blk * p.f_sb;
    const uint8_t* c[2] = {static_cast<const uint8_t*>(p.kc) + co,
                           static_cast<const uint8_t*>(p.vc) + co};
    const uint8_t* f[2] = {p.k_sf + fo, p.v_sf + fo};
    T* const o[2] = {mock_k + m * elems, mock_v + m * elems};
    dequantize_block<T, 2>(c, f, p.c_sr, p.c_sh, p.f_sr, p.f_sh, p.BS, p.Hkv,
                           groups, bad, false, 1.f, o);
  }
}

unsigned capped_grid(int64_t blocks, int per_sm) {
  const int64_t cap = static_cast<int64_t>(current_sm_count()) * per_sm;
  return static_cast<unsigned>(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_cache_write_fp4(
    const void* key, const void* value, int64_t k_st, int64_t k_sh,
    int64_t v_st, int64_t v_sh, void* kc, void* vc, const int64_t* cs,
    uint8_t* k_sf, uint8_t* v_sf, const int64_t* fs, const int64_t* slots,
    int64_t num_tokens, int Hkv, int D, int BS, int64_t num_blocks, bool bf16,
    const float* k_scale, const float* v_scale, unsigned* err,
    cudaStream_t stream) {
  const int groups = D / 16, per_token = Hkv * groups;
  const int tpb = per_token >= kThreads ? 1 : kThreads / per_token;
  const unsigned grid = capped_grid((num_tokens + tpb - 1) / tpb, 3);
  note_launch();
  auto go = [&](auto kern, const auto* k, const auto* v) {
    kern<<<grid, kThreads, 0, stream>>>(
        k, v, k_st, k_sh, v_st, v_sh, static_cast<uint8_t*>(kc),
        static_cast<uint8_t*>(vc), cs[0], cs[1], cs[2], k_sf, v_sf, fs[0],
        fs[1], fs[2], slots, num_tokens, groups, shift_of(groups), per_token,
        tpb, BS, shift_of(BS), num_blocks * BS, k_scale, v_scale, err);
  };
  if (bf16)
    go(cache_write_fp4_kernel<__nv_bfloat16>,
       static_cast<const __nv_bfloat16*>(key),
       static_cast<const __nv_bfloat16*>(value));
  else
    go(cache_write_fp4_kernel<__half>, static_cast<const __half*>(key),
       static_cast<const __half*>(value));
  return cudaGetLastError();
}

cudaError_t launch_fp4_dequant_blocks(const void* codes, const int64_t* cs,
                                      const uint8_t* sf, const int64_t* fs,
                                      const float* scale, const int64_t* ids,
                                      int64_t n, int64_t num_blocks, int Hkv,
                                      int D, int BS, void* out, bool bf16,
                                      unsigned* err, cudaStream_t stream) {
  const unsigned grid = capped_grid(n, 16);
  note_launch();
  if (bf16)
    fp4_dequant_blocks_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(
        static_cast<const uint8_t*>(codes), cs[0], cs[1], cs[2], sf, fs[0],
        fs[1], fs[2], scale, ids, n, num_blocks, Hkv, D / 16, BS,
        static_cast<__nv_bfloat16*>(out), err);
  else
    fp4_dequant_blocks_kernel<__half><<<grid, kThreads, 0, stream>>>(
        static_cast<const uint8_t*>(codes), cs[0], cs[1], cs[2], sf, fs[0],
        fs[1], fs[2], scale, ids, n, num_blocks, Hkv, D / 16, BS,
        static_cast<__half*>(out), err);
  return cudaGetLastError();
}

cudaError_t launch_fp4_dequant_pages(const AttnParams& p, int D, bool bf16,
                                     void* mock_k, void* mock_v,
                                     int32_t* mock_table,
                                     cudaStream_t stream) {
  const unsigned grid =
      capped_grid(static_cast<int64_t>(p.batch) * p.max_blocks, 16);
  note_launch();
  if (bf16)
    fp4_dequant_pages_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(
        p, static_cast<__nv_bfloat16*>(mock_k),
        static_cast<__nv_bfloat16*>(mock_v), mock_table, D / 16);
  else
    fp4_dequant_pages_kernel<__half><<<grid, kThreads, 0, stream>>>(
        p, static_cast<__half*>(mock_k), static_cast<__half*>(mock_v),
        mock_table, D / 16);
  return cudaGetLastError();
}

}  // namespace pkv
