// Verification of drafted tokens against the target model's probabilities.
//
// A request's rows form a tree (see tree_attn.cu): row i holds token x_i,
// drafted from the distribution q of its parent's row (or, without draft
// probabilities, proposed outright), and the target's distribution p behind
// it.  With given numbers u in [0, 1) the walk from row 0 keeps, at each row,
// what is left of its distribution, R = p, and its mass Z = 1, and tries the
// row's children c in order:
//   u_c q(x_c) Z < R(x_c)   c stands: the walk goes on there
//   else, with draft        R <- max(R - Z q, 0), Z <- sum R
//   without (q = 1)         Z <- max(Z - R(x_c), 0), R(x_c) <- 0
// Where no child stands, the token that follows is the first whose running sum
// of R exceeds u_0 sum R.  So the tokens said are distributed as if the target
// had drawn each of them.
//
// What has to be read is a few single elements and, per request, the last
// row's p (and q) once: HBM bounds a batch, the chain of dependent reads a
// single request.  The elements p(x_i), q(x_i) of all rows are fetched side by
// side at the start, so the walk itself runs in shared memory.  A cluster of 1
// to 8 CTAs shares the vocabulary of a request; every CTA walks the same way,
// and only the sums cross between them.
//
// Measured on the device, launches in a graph: one chain of 5 over 32001 tokens
// 11 us; 64 chains of 5 over 131072, both distributions, 22 us (3.1 TB/s); 48
// trees of 16 without the draft's 19 us; 24 trees of 9 to 24 over 100003 in bf16
// 34 us, about 3 us for each rejection on a request's way.
//
// The answers are whole numbers that turn on sums over the vocabulary: with
// 100000 near-equal probabilities, a sum that is off by 1e-8 of itself moves
// the sampled token once in a thousand draws.  Sums of 32 values are therefore
// carried as two floats (a value and its rounding error, about 2^-48), sums
// across lanes and chunks and all comparisons in float64.
#include <math.h>

#include <mutex>
#include <type_traits>

#include "pkv_common.cuh"

namespace pkv {
namespace verify {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxRows = PKV_TREE_MAX_ROWS;
constexpr int kChunk = 1024;            // vocabulary entries of a partial sum
constexpr int kMaxRanks = 8;            // CTAs of a request
constexpr int kMaxChunks = PKV_VERIFY_MAX_VOCAB / kChunk + 1;

struct Params {
  const void* target;
  int64_t t_st;
  const void* draft;
  int64_t d_st;
  const int32_t* tokens;
  const float* uniform;
  const int32_t* cu_q;
  const int32_t* parents;               // null: each row's parent is the one before
  int total_q, max_n, vocab;
  int32_t* out_tokens;                  // [batch, max_n]
  int32_t* out_rows;
  int32_t* out_count;
  unsigned* err;
};

struct Shared {
  int par[kMaxRows], tok[kMaxRows];
  float u[kMaxRows], pt[kMaxRows], qt[kMaxRows];
  int said[kMaxRows], rows[kMaxRows];
  // of the row the walk is at: with draft, the masses that q was taken off
  // with (as a double and as two floats); without, the tokens taken out
  double z[kMaxRows];
  float zh[kMaxRows], zl[kMaxRows];
  int gone[kMaxRows];
  double chunk[kMaxChunks];
  double total[2][kMaxRanks];           // the CTAs' sums, of even and odd passes
  double all;                           // ... and theirs
  float left[33 * 32];                  // a chunk, 32 entries and a gap
  double mass;
  int node, next, m, count, known, ask; // known: the mass is; ask: a sum is
                                        // wanted (else: the end)
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// v to *p of the CTA with this rank in the cluster.
__device__ __forceinline__ void put(double* p, int rank, double v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(a)
      : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}

// A sum and the rounding errors made on the way (Knuth's two-sum).
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x);
    const float b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)),
                                 __fsub_rn(x, b)));
    hi = s;
  }
};

// Two such sums side by side.
struct Sum4 {
  uint64_t hi, lo;
  __device__ __forceinline__ void add(uint64_t x) {
    const uint64_t neg = pair(-1.f, -1.f);
    const uint64_t s = add2(hi, x);
    const uint64_t b = fma2(hi, neg, s);             // s - hi
    const uint64_t t = fma2(b, neg, s);              // s - b
    lo = add2(lo, add2(fma2(t, neg, hi), fma2(b, neg, x)));
    hi = s;
  }
};

// Entries x .. x + VEC - 1 of a row, as 16 bytes; zero outside [0, vocab).
template <typename T>
__device__ __noinline__ uint4 edge(const T* row, int x, int vocab) {
  constexpr int VEC = 16 / static_cast<int>(sizeof(T));
  union {
    uint4 v;
    T e[VEC];
  } r;
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    r.e[e] = x + e >= 0 && x + e < vocab ? row[x + e] : from_f32<T>(0.f);
  return r.v;
}

// Places of a row: entry x lies at place x + pad, and places divide into
// 16-byte vectors of memory.
template <typename T>
__device__ __forceinline__ int pad_of(const T* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

// What is left, R, of the entries at places c kChunk .. of a row of `target`
// after q (the same entries of `draft`) has been taken off m times, or m tokens
// have been taken out (no `draft`): this lane's share of their sum, and with
// `keep` the values to s.left.  (One piece of code
// for both: a launch runs it a few times only, so what it costs is to be
// fetched.  Unrolled twice over, the kernel spent most of its time on that.)
template <typename T>
__device__ __noinline__ Sum2 chunk_rest(Shared& s, const T* target,
                                        const T* draft, int c, int m,
                                        int vocab, bool keep) {
  constexpr int VEC = 16 / static_cast<int>(sizeof(T));
  constexpr int PER = kChunk / (32 * VEC), W = VEC / 2;
  const int lane = threadIdx.x & 31;
  // vector k of a lane is number 32 k + lane of the chunk; all loads are under
  // way together
  const int x0 = c * kChunk - pad_of(target) + lane * VEC;
  uint4 a[PER], b[PER];
  const int first = c * kChunk - pad_of(target);
  if (first >= 0 && first + kChunk <= vocab &&
      (m == 0 || !draft || pad_of(draft) == pad_of(target))) {
    const uint4* from = reinterpret_cast<const uint4*>(target + x0);
#pragma unroll
    for (int k = 0; k < PER; ++k) a[k] = __ldg(from + k * 32);
    if (m > 0 && draft) {
      from = reinterpret_cast<const uint4*>(draft + x0);
#pragma unroll
      for (int k = 0; k < PER; ++k) b[k] = __ldg(from + k * 32);
    }
  } else {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      a[k] = edge(target, x0 + k * 32 * VEC, vocab);
      if (m > 0 && draft) b[k] = edge(draft, x0 + k * 32 * VEC, vocab);
    }
  }
  auto two = [](const uint4& v, int w) -> uint64_t {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    if constexpr (std::is_same<T, float>::value)
      return pair(__uint_as_float(u[2 * w]), __uint_as_float(u[2 * w + 1]));
    else
      return pair(elem_f32<T>(u[w], 0), elem_f32<T>(u[w], 1));
  };
  auto positive = [](uint64_t v) -> uint64_t {
    float x, y;
    unpair(v, x, y);
    return pair(fmaxf(x, 0.f), fmaxf(y, 0.f));
  };
  uint64_t r[PER * W];
#pragma unroll
  for (int k = 0; k < PER; ++k)
#pragma unroll
    for (int w = 0; w < W; ++w) r[k * W + w] = positive(two(a[k], w));
#pragma unroll 1
  for (int i = 0; i < m; ++i) {
    if (!draft) {
      // (zero itself, not a difference of sums: nothing may be left of a row
      // whose every token was taken out)
      const int at = s.gone[i] - first;
      if (at >= 0 && at < kChunk && (at / VEC & 31) == lane) {
#pragma unroll
        for (int k = 0; k < PER * W; ++k) {
          const bool hit = k == at / (32 * VEC) * W + at % VEC / 2;
          float x, y;
          unpair(r[k], x, y);
          r[k] = pair(hit && !(at & 1) ? 0.f : x, hit && (at & 1) ? 0.f : y);
        }
      }
      continue;
    }
    // (the mass as two floats; the first is 1)
    const uint64_t zh = pair(-s.zh[i], -s.zh[i]),
                   zl = pair(-s.zl[i], -s.zl[i]);
#pragma unroll
    for (int k = 0; k < PER; ++k)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        // (below 0 or NaN: none, as in the target)
        const uint64_t q = positive(two(b[k], w));
        uint64_t& v = r[k * W + w];
        v = positive(fma2(zl, q, fma2(zh, q, v)));
      }
  }
  Sum4 t{0, 0};
#pragma unroll
  for (int k = 0; k < PER * W; ++k) t.add(r[k]);
  if (keep) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = (k * 32 + lane) * VEC;
      float* to = s.left + i + (i >> 5);
#pragma unroll
      for (int w = 0; w < W; ++w) unpair(r[k * W + w], to[2 * w], to[2 * w + 1]);
    }
  }
  float h0, h1, l0, l1;
  unpair(t.hi, h0, h1);
  unpair(t.lo, l0, l1);
  Sum2 sum{h0, __fadd_rn(l0, l1)};
  sum.add(h1);
  return sum;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
verify_kernel(const Params p) {
  __shared__ Shared s;
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int b = blockIdx.x / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int start = p.cu_q[b];
  int n = min(p.cu_q[b + 1], p.total_q) - start;
  if (start < 0 || n < 0) n = 0;
  if (n > p.max_n) {
    if (tid == 0 && rank == 0) atomicOr(p.err, kErrQueryLen);
    n = 0;
  }
  int32_t* out_t = p.out_tokens + static_cast<int64_t>(b) * p.max_n;
  int32_t* out_r = p.out_rows + static_cast<int64_t>(b) * p.max_n;
  if (n == 0) {                          // (the same in the whole cluster)
    if (rank == 0) {
      for (int i = tid; i < p.max_n; i += kThreads) out_t[i] = out_r[i] = -1;
      if (tid == 0) p.out_count[b] = 0;
    }
    return;
  }
  const bool draft = p.draft != nullptr;
  cluster_arrive();                      // (this CTA runs: others may write to it)

  // ---- every row's numbers, and what its parent's row gives its token
  for (int i = tid; i < n; i += kThreads) {
    const int row = start + i;
    int par = p.parents ? p.parents[row] : i - 1;
    const int tok = i > 0 ? p.tokens[row] : 0;
    s.u[i] = p.uniform[row];
    float pt = 0.f, qt = 0.f;
    const bool bad = par < -1 || par >= i || tok < 0 || tok >= p.vocab;
    if (bad) {
      if (rank == 0) atomicOr(p.err, kErrBadTree);
      par = -1;                          // (never reached)
    } else if (i > 0 && par >= 0) {
      pt = to_f32(static_cast<const T*>(p.target)[(start + par) * p.t_st +
                                                  tok]);
      if (draft)
        qt = to_f32(static_cast<const T*>(p.draft)[(start + par) * p.d_st +
                                                   tok]);
    }
    s.par[i] = i > 0 ? par : -1;
    s.tok[i] = tok;
    s.pt[i] = fmaxf(pt, 0.f);
    s.qt[i] = fmaxf(qt, 0.f);
  }
  if (tid == 0) {
    s.node = 0;
    s.next = 1;
    s.m = 0;
    s.count = 1;
    s.rows[0] = 0;
    s.mass = 1.0;
    s.known = 1;
    s.ask = 0;
  }
  __syncthreads();
  cluster_wait();

  const int chunks = (p.vocab + 15 + kChunk - 1) / kChunk;
  const int c_lo = static_cast<int>(int64_t{chunks} * rank / ranks);
  const int c_hi = static_cast<int>(int64_t{chunks} * (rank + 1) / ranks);
  const T* tr = nullptr;                 // the rows at hand, and their pad
  const T* dr = nullptr;
  int pad = 0, pass = 0;
  // Sum of what is left of the node's row after m times, over the whole
  // vocabulary; the chunks' sums stay in s.chunk.  (float64 is done by one warp
  // only: an SM adds two values a clock.)
  auto sum = [&](int node, int m) -> double {
    tr = static_cast<const T*>(p.target) + (start + node) * p.t_st;
    dr = draft ? static_cast<const T*>(p.draft) + (start + node) * p.d_st
               : nullptr;
    pad = pad_of(tr);
    for (int c = c_lo + warp; c < c_hi; c += kWarps) {
      Sum2 a = chunk_rest(s, tr, dr, c, m, p.vocab, false);
#pragma unroll 1
      for (int o = 16; o; o >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, a.hi, o);
        const float l = __shfl_xor_sync(0xffffffffu, a.lo, o);
        a.add(h);
        a.lo = __fadd_rn(a.lo, l);
      }
      if (lane == 0)
        s.chunk[c - c_lo] = static_cast<double>(a.hi) + a.lo;
    }
    __syncthreads();
    if (warp == 0) {
      double t = 0.0;
      for (int c = lane; c < c_hi - c_lo; c += 32) t += s.chunk[c];
#pragma unroll
      for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane < ranks) put(&s.total[pass & 1][rank], lane, t);
    }
    cluster_arrive();
    cluster_wait();
    if (tid == 0) {
      double all = 0.0;
      for (uint32_t r = 0; r < ranks; ++r) all += s.total[pass & 1][r];
      s.all = all;
    }
    __syncthreads();
    ++pass;
    return s.all;
  };

  // ---- the walk: warp 0 goes on until it needs a sum, or to the end
  for (;;) {
    if (warp == 0) {
      int node = s.node, i = s.next, m = s.m, count = s.count, ask = 0;
      // (after a rejection with draft probabilities the mass is not known yet)
      double mass = s.mass;
      bool known = s.known;
      while (i < n) {
        const int r = i + lane;
        const unsigned kids =
            __ballot_sync(0xffffffffu, r < n && s.par[r] == node);
        if (!kids) {
          i += 32;
          continue;
        }
        i += __ffs(kids) - 1;
        if (!known) {
          ask = 1;
          break;
        }
        const int x = s.tok[i];
        double have = s.pt[i];
        double likely = 1.0;
        if (draft) {
          likely = s.qt[i];
          for (int k = 0; k < m; ++k) have = fmax(have - s.z[k] * likely, 0.0);
        } else {
          for (int k = lane; k - lane < m; k += 32)
            if (__any_sync(0xffffffffu, k < m && s.gone[k] == x)) have = 0.0;
        }
        if (static_cast<double>(s.u[i]) * likely * mass < have) {
          if (lane == 0) {
            s.said[count - 1] = x;
            s.rows[count] = i;
          }
          ++count;
          node = i;
          m = 0;
          mass = 1.0;
        } else if (draft) {
          if (lane == 0) {
            s.z[m] = mass;
            s.zh[m] = static_cast<float>(mass);
            s.zl[m] = static_cast<float>(mass - static_cast<float>(mass));
          }
          ++m;
          known = false;
        } else if (have > 0.0) {
          if (lane == 0) s.gone[m] = x;
          ++m;
          mass = fmax(mass - have, 0.0);
        }
        __syncwarp();
        ++i;
      }
      if (lane == 0) {
        s.node = node;
        s.next = i;
        s.m = m;
        s.count = count;
        s.mass = mass;
        s.known = known;
        s.ask = ask;
      }
    }
    __syncthreads();
    if (!s.ask) break;
    const double z = sum(s.node, s.m);
    if (tid == 0) {
      s.mass = z;
      s.known = 1;
    }
    __syncthreads();
  }

  // ---- the token that follows
  const int node = s.node, count = s.count;
  int m = s.m;
  double all = sum(node, m);
  if (!(all > 0.0) && m > 0) {           // nothing is left: the row as it is
    m = 0;
    all = sum(node, 0);
  }
  if (rank == 0) {
    for (int i = tid; i < p.max_n; i += kThreads) {
      if (i != count - 1) out_t[i] = i < count - 1 ? s.said[i] : -1;
      out_r[i] = i < count ? s.rows[i] : -1;
    }
    if (tid == 0) {
      p.out_count[b] = count;
      if (!(all > 0.0)) out_t[count - 1] = -1;
    }
  }
  if (warp == 0 && all > 0.0) {
    const double want = fmax(static_cast<double>(s.u[0]), 0.0) * all;
    // the first CTA whose running sum exceeds it; none (u_0 >= 1): the last
    // with any mass
    double before = 0.0, run = 0.0, mine_before = 0.0;
    int owner = -1, last = -1;
    const int par = (pass - 1) & 1;
    for (uint32_t r = 0; r < ranks; ++r) {
      const double t = s.total[par][r];
      if (r == rank) mine_before = run;
      if (t > 0.0) last = r;
      run += t;
      if (owner < 0 && t > 0.0 && run > want) owner = r;
    }
    const bool past = owner < 0;
    if (past) owner = last;
    before = mine_before;
    if (owner == static_cast<int>(rank)) {
      // ... then its chunk (32 at a time; rounding must not pick one without
      // mass) ...
      int found = -1, some = -1;
      double at = before;
      for (int c0 = 0; c0 < c_hi - c_lo && found < 0; c0 += 32) {
        const double own = c0 + lane < c_hi - c_lo ? s.chunk[c0 + lane] : 0.0;
        double in = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, in, o);
          if (lane >= o) in += y;
        }
        const unsigned hit =
            __ballot_sync(0xffffffffu, !past && own > 0.0 && at + in > want);
        const unsigned any = __ballot_sync(0xffffffffu, own > 0.0);
        if (any) some = c0 + 31 - __clz(any);
        if (hit) {
          const int src = __ffs(hit) - 1;
          found = c0 + src;
          at += __shfl_sync(0xffffffffu, in - own, src);
        } else {
          at += __shfl_sync(0xffffffffu, in, 31);
        }
      }
      // (rounding may leave a sum's last bit short: the last chunk with mass)
      const bool end = found < 0;
      if (end) found = some;
      // ... then the 32 entries (a lane's) that hold it ...
      const int x0 = (c_lo + found) * kChunk - pad;
      chunk_rest(s, tr, dr, c_lo + found, m, p.vocab, true);
      __syncwarp();
      Sum2 a{0.f, 0.f};
#pragma unroll 4
      for (int e = 0; e < 32; ++e) a.add(s.left[lane * 33 + e]);
      const double own = static_cast<double>(a.hi) + a.lo;
      auto scan = [&](double x) -> double {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        return x;
      };
      const double in = scan(own);
      const unsigned hit =
          __ballot_sync(0xffffffffu, !end && own > 0.0 && at + in > want);
      const unsigned any = __ballot_sync(0xffffffffu, own > 0.0);
      // (none: the last one with mass)
      const int src = hit ? __ffs(hit) - 1 : any ? 31 - __clz(any) : 0;
      at += __shfl_sync(0xffffffffu, in - own, src);
      // ... then the entry
      const float r = s.left[src * 33 + lane];
      const double inr = scan(static_cast<double>(r));
      const unsigned hit1 =
          __ballot_sync(0xffffffffu, hit != 0 && r > 0.f && at + inr > want);
      const unsigned any1 = __ballot_sync(0xffffffffu, r > 0.f);
      const int e1 = hit1 ? __ffs(hit1) - 1 : any1 ? 31 - __clz(any1) : 0;
      const int token = x0 + src * 32 + e1;
      if (lane == 0) out_t[count - 1] = token;
    }
  }
}

}  // namespace verify

cudaError_t launch_verify(const VerifyLaunch& a, int elem, cudaStream_t stream) {
  using namespace verify;
  Params p{};
  p.target = a.target;
  p.t_st = a.t_st;
  p.draft = a.draft;
  p.d_st = a.d_st;
  p.tokens = a.tokens;
  p.uniform = a.uniform;
  p.cu_q = a.cu_q;
  p.parents = a.parents;
  p.total_q = a.total_q;
  p.max_n = a.max_n;
  p.vocab = a.vocab;
  p.out_tokens = a.out_tokens;
  p.out_rows = a.out_rows;
  p.out_count = a.out_count;
  p.err = a.err;
  auto kern = elem == PKV_F32    ? verify_kernel<float>
              : elem == PKV_BF16 ? verify_kernel<__nv_bfloat16>
                                 : verify_kernel<__half>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // CTAs of a request: as many as one wave holds, with 4 chunks each at least.
  // (Clusters do not cross the GPU's SM groups, so the driver says how many
  // fit: 76 of 2 CTAs, but 46 of 3 and 15 of 8 on 152 SMs.)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::mutex mu;
  static int fits[64][kMaxRanks + 1] = {};     // clusters, per device and size
  const int chunks = (a.vocab + 15 + kChunk - 1) / kChunk;
  int c = chunks / 4 < kMaxRanks ? chunks / 4 : kMaxRanks;
  for (; c > 1; --c) {
    if (static_cast<int64_t>(a.batch) * c > current_sm_count()) continue;
    std::lock_guard<std::mutex> lk(mu);
    int& n = fits[dev & 63][c];
    if (n == 0) {
      attr[0].val.clusterDim.x = c;
      cfg.gridDim = dim3(c);
      e = cudaOccupancyMaxActiveClusters(&n, verify_kernel<float>, &cfg);
      if (e != cudaSuccess) return e;
      if (n == 0) n = -1;
    }
    if (a.batch <= n) break;
  }
  if (c < 1) c = 1;
  attr[0].val.clusterDim.x = c;
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * c);
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace pkv
