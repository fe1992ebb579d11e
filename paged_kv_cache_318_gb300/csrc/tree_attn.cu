// Attention of a tree of drafted tokens: the join of the pieces, and the launch
// (the kernel and its design: tree_attn.cuh).
#include <limits.h>

#include "tree_attn.cuh"

namespace pkv {
namespace tree {

// Joins the pieces of the units that the shares' ends cut.  Blocks (x, .) look
// through the marks of CTAs x, x + gridDim.x, ..; a unit's rows go round the
// warps of the blocks (., y): M = the largest partial LSE (and the sink), w_k =
// e^(lse_k - M), out = sum w_k o_k / sum w_k, lse = M + ln sum w_k.  Where a
// wait ran out in one of a unit's CTAs, its rows stay as they are.
constexpr int kFoldThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kFoldThreads, 2)
fold_kernel(const Params p, int ctas) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int WARPS = kFoldThreads / 32, V = D / 32, N = V > 4 ? 4 : 8;
  const int lane = threadIdx.x & 31;
  for (int c0 = blockIdx.x; c0 < ctas; c0 += 32 * gridDim.x) {
    const int mine = c0 + lane * gridDim.x;
    const unsigned cut = __ballot_sync(
        0xffffffffu, mine < ctas && p.marks[2 * mine].x > 0);
    for (unsigned left = cut; left; left &= left - 1) {
      const int c = c0 + (__ffs(left) - 1) * gridDim.x;
      const int4 m0 = p.marks[2 * c];
      const int g = p.marks[2 * c + 1].x;
      const int np = min(m0.x, ctas - c);
      const int rows = min(m0.z, p.rows_cap);
      for (int row = blockIdx.y * WARPS + (threadIdx.x >> 5); row < rows;
           row += gridDim.y * WARPS) {
        const int R = m0.w + row;
        const int node = row_of(R, p.inv_g);
        const int tok = m0.y + node, h = g * p.G + R - node * p.G;
        // piece k: the tail of CTA c's share, then the heads of the next ones'
        auto at = [&](int k) -> int64_t {
          const int slot = k == 0 ? 2 * c + 1 : 2 * (c + k);
          return static_cast<int64_t>(slot) * p.rows_cap + row;
        };
        const float z = p.sinks ? p.sinks[h] : -INFINITY;
        float M = z;
        int gone = 0;
        for (int k0 = 0; k0 < np; k0 += 32) {
          const bool in = k0 + lane < np;
          const float s = in ? p.part_lse[at(k0 + lane)] : -INFINITY;
          gone |= in ? p.marks[2 * (c + k0 + lane) + 1].y : 0;
          M = fmaxf(M, s);
        }
        if (__any_sync(0xffffffffu, gone)) break;
#pragma unroll
        for (int o = 16; o; o >>= 1)
          M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float ref = M == -INFINITY ? 0.f : M;
        float sum = p.sinks ? ex2((z - ref) * kLog2e) : 0.f;
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
        // (N pieces' rows are under way at once)
#pragma unroll 1
        for (int k0 = 0; k0 < np; k0 += N) {
          float s[N], o[N][V];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int k = min(k0 + i, np - 1);
            s[i] = p.part_lse[at(k)];
            const float* src = p.part_o + at(k) * D + lane * V;
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const float2 t = *reinterpret_cast<const float2*>(src + e);
              o[i][e] = t.x;
              o[i][e + 1] = t.y;
            }
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            // (a NaN sum stays NaN)
            const float w = k0 + i < np ? ex2((s[i] - ref) * kLog2e) : 0.f;
            sum += w;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(w, o[i][e], acc[e]);
          }
        }
        const float inv = sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f;
        T* dst = static_cast<T*>(p.out) +
                 static_cast<int64_t>(tok) * p.o_st +
                 static_cast<int64_t>(h) * p.o_sh + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 2)
          *reinterpret_cast<uint32_t*>(dst + e) =
              pack2<T>(acc[e] * inv, acc[e + 1] * inv);
        if (p.lse && lane == 0)
          p.lse[static_cast<int64_t>(h) * p.total_q + tok] =
              sum > 0.f ? ref + lg2(sum) * kLn2
                        : sum != sum ? sum : -INFINITY;
      }
    }
  }
}

int block_rows(int D) {
  return D == 256 ? Cfg<256, 0>::ROWS : Cfg<128, 0>::ROWS;
}
// Rows of a partial: the most packed rows of a block.
int rows_cap(int D, int G, int max_n) {
  const int64_t r = static_cast<int64_t>(max_n) * G;
  return static_cast<int>(r < block_rows(D) ? r : block_rows(D));
}
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace tree

size_t tree_scratch_bytes(int D, int G, int max_n, int sms) {
  const size_t rows = static_cast<size_t>(tree::rows_cap(D, G, max_n));
  return tree::align256(2 * sizeof(int4) * sms) +
         tree::align256(2 * rows * sms * sizeof(float)) +
         2 * rows * sms * D * sizeof(float);
}

cudaError_t launch_tree_attn(const AttnParams& a, const int32_t* parents,
                             int max_n, int64_t max_k, int D, bool bf16,
                             int sms, void* scratch, bool pdl,
                             cudaStream_t stream) {
  using namespace tree;
  Params p{};
  p.q = a.q;
  p.q_st = a.q_st;
  p.q_sh = a.q_sh;
  p.out = a.out;
  p.o_st = a.o_st;
  p.o_sh = a.o_sh;
  p.lse = a.lse;
  p.total_q = a.total_q;
  p.batch = a.batch;
  p.max_n = max_n;
  p.cu_q = a.cu_q;
  p.seqused_k = a.seqused_k;
  p.parents = parents;
  p.block_table = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.G;
  p.inv_g = 1.f / static_cast<float>(a.G);
  p.BS = a.BS;
  p.bs_shift = a.bs_shift;
  p.scale = a.scale;
  p.softcap = a.softcap;
  p.sinks = a.sinks;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.wl = a.wl;
  p.err = a.err;
  p.wait_ns = a.wait_ns;
  int RB = 16;
  while (RB * 2 <= 64 && a.BS % (RB * 2) == 0) RB *= 2;
  p.RB = RB;
  p.kv_order_hnd = a.c_sh > a.c_sr ? 1 : 0;
  p.out_v8 = (reinterpret_cast<uintptr_t>(a.out) % 32 == 0 &&
              (a.o_st * 2) % 32 == 0 && (a.o_sh * 2) % 32 == 0)
                 ? 1
                 : 0;
  const int64_t packed = static_cast<int64_t>(max_n) * a.G;
  const int64_t blocks = (packed + block_rows(D) - 1) / block_rows(D);
  // (every tile is read by one CTA only: evict first; 48 requests of 12 rows over
  // 4364 keys 156 us against 168, over a cache whose pages hold keys and values
  // in turn 171 against 176.  Tiles that another CTA reads too stay: 4 requests
  // of 64 rows, 64 heads, 65600 keys 405 us against 422.  Codes go first either
  // way: with 512 packed rows E4M3 505 us against 508 on those 4 requests, 253
  // against 257 on 16 of 40 rows over 8232 keys, 288 against 295 at head size
  // 256; 4 bits 523 against 521.)
  p.once = blocks <= 1;
  // an upper bound of the tiles (a window adds up to a tile at either end)
  const int bn = tree_tile_keys(D);
  int64_t keys = max_k;
  if (a.wl >= 0 && static_cast<int64_t>(a.wl) + max_n + RB < keys)
    keys = static_cast<int64_t>(a.wl) + max_n + RB;
  const int64_t units = static_cast<int64_t>(a.batch) * a.Hkv * blocks;
  const int64_t tiles = units * ((keys + bn - 1) / bn + 1);
  // (units of one tile are not cut, and need no join behind the kernel; where
  // the tables could name more tiles than 32 bits count, whole units go round)
  const int64_t cols = static_cast<int64_t>(a.max_blocks) * a.BS / bn + 2;
  p.split = scratch != nullptr && keys > bn && cols <= INT_MAX / units;
  p.rows_cap = rows_cap(D, a.G, max_n);
  const int64_t most = p.split ? tiles : units;
  const int grid = static_cast<int>(most < sms ? most : sms);
  if (p.split) {
    char* s = static_cast<char*>(scratch);
    p.marks = reinterpret_cast<int4*>(s);
    s += align256(2 * sizeof(int4) * sms);
    p.part_lse = reinterpret_cast<float*>(s);
    s += align256(2 * static_cast<size_t>(p.rows_cap) * sms * sizeof(float));
    p.part_o = reinterpret_cast<float*>(s);
  }
  CUtensorMap mk, mv, mq;
  memset(&mq, 0, sizeof(mq));
  const int kv = a.k_sf ? kE2m1 : a.kv_fp8 ? kE4m3 : kValues;
  if (kv != kValues) {
    p.k_sf = a.k_sf;
    p.v_sf = a.v_sf;
    p.f_sb = a.f_sb;
    p.f_sr = a.f_sr;
    p.f_sh = a.f_sh;
    const int row = kv == kE4m3 ? D : D / 2;
    if (!make_code_map(&mk, a.kc, row, a.BS, a.Hkv, a.num_blocks, a.c_sb,
                       a.c_sr, a.c_sh, RB, p.kv_order_hnd) ||
        !make_code_map(&mv, a.vc, row, a.BS, a.Hkv, a.num_blocks, a.c_sb,
                       a.c_sr, a.c_sh, RB, p.kv_order_hnd))
      return cudaErrorInvalidValue;
  } else {
    // one box per page and matrix where the view allows it
    p.kv_rg = make_kv_rg_map(&mk, a.kc, bf16, D, a.BS, a.Hkv, a.num_blocks,
                             a.c_sb, a.c_sr, a.c_sh, RB, p.kv_order_hnd) &&
              make_kv_rg_map(&mv, a.vc, bf16, D, a.BS, a.Hkv, a.num_blocks,
                             a.c_sb, a.c_sr, a.c_sh, RB, p.kv_order_hnd);
    if (!p.kv_rg &&
        (!make_kv_map(&mk, a.kc, bf16, D, a.BS, a.Hkv, a.num_blocks, a.c_sb,
                      a.c_sr, a.c_sh, RB, p.kv_order_hnd) ||
         !make_kv_map(&mv, a.vc, bf16, D, a.BS, a.Hkv, a.num_blocks, a.c_sb,
                      a.c_sr, a.c_sh, RB, p.kv_order_hnd)))
      return cudaErrorInvalidValue;
  }
  p.q_tma = make_rows_map(&mq, a.q, bf16, D, a.Hq, a.total_q, a.q_st, a.q_sh,
                          a.G);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const cudaLaunchAttribute* at = pdl ? attr : nullptr;
  cudaError_t e =
      kv != kValues ? launch_codes(p, D, bf16, kv, mk, mv, mq, grid, at,
                                   stream)
      : bf16 ? launch_d<__nv_bfloat16, kValues>(p, D, mk, mv, mq, grid, at,
                                                stream)
             : launch_d<__half, kValues>(p, D, mk, mv, mq, grid, at, stream);
  if (e != cudaSuccess || !p.split) return e;
  cudaLaunchConfig_t cfg = {};
  // (a block per share, or two per unit where there are few units: one request
  // of 8 units over 16384 keys 30 us, 38 with a block per share)
  cfg.gridDim = dim3(static_cast<unsigned>(2 * units < grid ? 2 * units : grid),
                     (p.rows_cap + 7) / 8);
  cfg.blockDim = dim3(kFoldThreads);
  cfg.stream = stream;
  cfg.attrs = const_cast<cudaLaunchAttribute*>(at);
  cfg.numAttrs = at ? 1 : 0;
  auto join = [&](auto fold) {
    note_launch();
    return cudaLaunchKernelEx(&cfg, fold, p, grid);
  };
  switch (D) {
    case 64:
      return bf16 ? join(fold_kernel<__nv_bfloat16, 64>)
                  : join(fold_kernel<__half, 64>);
    case 128:
      return bf16 ? join(fold_kernel<__nv_bfloat16, 128>)
                  : join(fold_kernel<__half, 128>);
    default:
      return bf16 ? join(fold_kernel<__nv_bfloat16, 256>)
                  : join(fold_kernel<__half, 256>);
  }
}

}  // namespace pkv
