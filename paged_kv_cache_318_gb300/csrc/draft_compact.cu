// Compaction of paged caches after verification: the rows of a draft that
// stand move together behind the context, in every cache given (keys and
// values of every layer, codes or block scales of a quantized cache: rows are
// moved as bytes).
//
//   cache[slot(ctx + i)] = cache[slot(ctx + rows[i])],  i < count
//
// Rows grow (rows[i] >= i), so a place that is written has been read, or is
// read by an earlier i: a thread that owns the same bytes of every row may load
// a few rows, then store them, and go on, without a copy in between.  Reads and
// writes of the moved rows are all there is to do: HBM bounds large calls, one
// launch and the chain count -> table -> rows small ones.
// Measured on the device, launches in a graph: 64 drafts of 24 to 32 rows in 32
// caches of 8 x 128 bf16, 17 MB both ways, 5.8 us; 7 rows in 4 caches 2.7 us.
#include "pkv_common.cuh"

namespace pkv {
namespace compact {

constexpr int kThreads = 256;
constexpr int kAhead = 8;               // rows in flight per thread

struct Params {
  CompactCaches caches;
  int64_t c_sb, c_sr, c_sh;             // bytes
  int heads, per_head, per_token, bs;   // per_*: vectors of a row
  const int32_t* table;
  int64_t bt_stride;
  int max_blocks;
  int64_t num_blocks;
  const int32_t* cu_q;
  const int32_t* seqused_k;
  const int32_t* rows;
  int64_t rows_st;
  int max_rows;
  const int32_t* count;
  int total_q;
  unsigned* err;
};

template <typename V>
__global__ void __launch_bounds__(kThreads) compact_kernel(const Params p) {
  __shared__ int64_t src[PKV_TREE_MAX_ROWS], dst[PKV_TREE_MAX_ROWS];
  const int b = blockIdx.x;
  const int k = min(p.count[b], p.max_rows);
  const int start = p.cu_q[b];
  const int n = min(p.cu_q[b + 1], p.total_q) - start;
  if (k <= 0 || start < 0 || n <= 0) return;
  const int ctx = p.seqused_k[b] - n;
  // ---- byte offsets of the rows that move (-1: stays, or left out)
  const int32_t* rows = p.rows + b * p.rows_st;
  unsigned bad = p.count[b] > p.max_rows ? kErrBadTree : 0u;
  int moves = 0;
  for (int i = threadIdx.x; i < k; i += kThreads) {
    const int r = rows[i];
    int64_t from = -1, to = -1;
    if (r < i || r >= n || (i > 0 && rows[i - 1] >= r) || ctx < 0) {
      bad |= kErrBadTree;
    } else if (r != i) {
      const int at[2] = {ctx + r, ctx + i};
      int64_t off[2];
      bool ok = true;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = at[e] / p.bs;
        const int blk = col < p.max_blocks
                            ? p.table[b * p.bt_stride + col]
                            : -1;
        if (blk < 0 || blk >= p.num_blocks) {
          bad |= col < p.max_blocks ? kErrBadBlock : kErrBadTable;
          ok = false;
        }
        off[e] = blk * p.c_sb + (at[e] - col * p.bs) * p.c_sr;
      }
      if (ok) {
        from = off[0];
        to = off[1];
        moves = 1;
      }
    }
    src[i] = from;
    dst[i] = to;
  }
  if (bad && blockIdx.y == 0) atomicOr(p.err, bad);
  if (!__syncthreads_or(moves)) return;
  // ---- this thread's vector of every row of one cache
  // (a cache's rows may have more vectors than the grid has threads)
  for (int64_t id = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
       id < static_cast<int64_t>(p.per_token) * p.caches.n;
       id += static_cast<int64_t>(gridDim.y) * kThreads) {
    const int c = static_cast<int>(id / p.per_token);
    const int v = static_cast<int>(id - static_cast<int64_t>(c) * p.per_token);
    const int h = v / p.per_head;
    char* base = static_cast<char*>(p.caches.ptr[c]) + h * p.c_sh +
                 static_cast<int64_t>(v - h * p.per_head) * sizeof(V);
    for (int i0 = 0; i0 < k; i0 += kAhead) {
      V t[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (i0 + e < k && src[i0 + e] >= 0)
          t[e] = *reinterpret_cast<const V*>(base + src[i0 + e]);
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (i0 + e < k && src[i0 + e] >= 0)
          *reinterpret_cast<V*>(base + dst[i0 + e]) = t[e];
    }
  }
}

}  // namespace compact

cudaError_t launch_compact(const CompactLaunch& a, cudaStream_t stream) {
  using namespace compact;
  Params p{};
  p.caches = a.caches;
  p.c_sb = a.c_sb;
  p.c_sr = a.c_sr;
  p.c_sh = a.c_sh;
  p.heads = a.heads;
  p.bs = a.bs;
  p.table = a.table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.cu_q = a.cu_q;
  p.seqused_k = a.seqused_k;
  p.rows = a.rows;
  p.rows_st = a.rows_st;
  p.max_rows = a.max_rows;
  p.count = a.count;
  p.total_q = a.total_q;
  p.err = a.err;
  // the widest vector that divides a row and every address
  uint64_t bits = static_cast<uint64_t>(a.row_bytes) | a.c_sb | a.c_sr |
                  a.c_sh;
  for (int i = 0; i < a.caches.n; ++i)
    bits |= reinterpret_cast<uintptr_t>(a.caches.ptr[i]);
  int w = 16;
  while (w > 1 && bits % w) w /= 2;
  p.per_head = a.row_bytes / w;
  p.per_token = p.per_head * a.heads;
  const int64_t y =
      (static_cast<int64_t>(p.per_token) * a.caches.n + kThreads - 1) /
      kThreads;
  const dim3 grid(a.batch, static_cast<unsigned>(y < 65535 ? y : 65535));
  note_launch();
  switch (w) {
    case 16: compact_kernel<uint4><<<grid, kThreads, 0, stream>>>(p); break;
    case 8: compact_kernel<uint2><<<grid, kThreads, 0, stream>>>(p); break;
    case 4: compact_kernel<uint32_t><<<grid, kThreads, 0, stream>>>(p); break;
    case 2: compact_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p); break;
    default: compact_kernel<uint8_t><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace pkv
