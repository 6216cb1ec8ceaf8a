// Embedding of the packed stream and its gradient by sorted tokens.
//
//     out[t] = scale * table[ids[t]]                      (a negative id: a zero row)
//     dtable[v] = scale * sum_{t : ids[t] = v} dout[t]    (negative ids add nothing)
//
// The gradient is deterministic: every row of dtable is a sum in token order, in fp32, rounded
// once.  Tokens are sorted by id (stable), equal ids form runs of the sorted order, and the runs
// are summed.  Kernels (one stream, programmatic dependent launches):
//   embed_fwd_kernel     one 16-byte vector per thread and step, several rows per block when rows
//                        are short; HBM-bound
//   embed_sort_kernel    cluster 0: least-significant-digit radix sort of (id, token) in one launch,
//                        eight CTAs that exchange digit counts through distributed shared memory
//                        (the sorted pairs stay in L2); the other clusters meanwhile write the zero
//                        rows of the ids that no token has, so the sort costs no time of its own
//                        when a whole table is written
//   embed_reduce_kernel  chunks of P sorted tokens x columns: rows of dout are read once, sixteen
//                        (fp32: eight) rows in flight per thread, sums of runs that lie inside a chunk are final, the
//                        others go to two fp32 rows per chunk
//   embed_join_kernel    runs over several chunks: the chunks' sums, a block per run
// What bounds the gradient: HBM, mostly its writes (a fill alone runs at 3.8-4.0 TB/s here, a copy at
// 6.8).
#include <algorithm>

#include "common.cuh"

namespace va {

namespace {

constexpr int kFwdThreads = 256, kFwdUnroll = 4;
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;               // one cluster
constexpr int kMaxBins = 512;
constexpr int kSortBatch = 4;              // keys a lane loads together
constexpr int kPresentWords = 8192;        // ids a filling CTA looks at together: 32 per word
constexpr int kZeroBytes = 8192;           // of one bulk store of zeros
constexpr int kReduceThreads = 256;
constexpr int kW = 8;                      // columns per thread: one vector of bf16, two of fp32
constexpr int kMaxP = 128;                 // sorted tokens per chunk, at most

struct EmbedParams {
  const int32_t* ids;
  int T, V, D;
  float scale;
  const void* src;  // table (forward), dout (gradient)
  int64_t s_rs;
  void* dst;  // out, dtable
  int64_t d_rs;
  int32_t* status;
  // gradient
  int accumulate;
  int2 *pair0, *pair1;                 // [T] (id, token), ping-pong
  int bits, passes, width;             // radix: `passes` digits of `width` bits
  float* part;                         // [chunks][2][D]
  int P;                               // sorted tokens per chunk
};


// kW consecutive values of a row as loaded (n of them without VEC: 16-byte accesses); values() gives
// them in fp32.
template <class T> struct Raw;
template <> struct Raw<float> {
  float4 a, b;
  template <bool VEC>
  __device__ __forceinline__ void load(const float* p, int n) {
    if constexpr (VEC) {
      a = __ldcs(reinterpret_cast<const float4*>(p));
      b = __ldcs(reinterpret_cast<const float4*>(p + 4));
    } else {
      float x[kW];
#pragma unroll
      for (int i = 0; i < kW; ++i) x[i] = i < n ? p[i] : 0.f;
      a = make_float4(x[0], x[1], x[2], x[3]);
      b = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
  __device__ __forceinline__ void values(float (&x)[kW]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <> struct Raw<__nv_bfloat16> {
  uint4 u;
  template <bool VEC>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n) {
    if constexpr (VEC) {
      u = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
      uint32_t h[kW];
#pragma unroll
      for (int i = 0; i < kW; ++i) h[i] = i < n ? reinterpret_cast<const uint16_t*>(p)[i] : 0u;
      u = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
  }
  __device__ __forceinline__ void values(float (&x)[kW]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <bool VEC, int W>
__device__ __forceinline__ void store_row(float* p, int n, const float (&x)[W]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < W; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < n) p[i] = x[i];
  }
}
template <bool VEC, int W>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, int n, const float (&x)[W]) {
  if constexpr (VEC) {
    static_assert(W == 8, "one vector");
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                              pack_bf16(x[6], x[7]));
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(x[i]);
  }
}

// Threads that share a row: enough for its columns at `vecs` vectors each, at most a block.
int lanes_per_row(int D, int threads, int vecs) {
  int n = 1;
  while (n < threads && n * kW * vecs < D) n *= 2;
  return n;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int load_remote(const int* p, int rank) {
  int v;
  asm volatile("{\n .reg .b32 ra;\n mapa.shared::cluster.u32 ra, %1, %2;\n ld.shared::cluster.u32 %0, [ra];\n}\n"
               : "=r"(v)
               : "r"(smem_u32(p)), "r"(rank)
               : "memory");
  return v;
}

}  // namespace

// Row group g of block b handles token b * groups + g; its lanes take the columns in vectors.
template <class T, bool VEC>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const EmbedParams p, int lpr) {
  griddep_begin();
  const int groups = kFwdThreads / lpr, g = threadIdx.x / lpr, lane = threadIdx.x % lpr;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * groups + g;
  if (t >= p.T) return;
  const int id = __ldg(p.ids + t);
  T* dst = static_cast<T*>(p.dst) + t * p.d_rs;
  const bool in = id >= 0 && id < p.V;
  const T* src = static_cast<const T*>(p.src) + (in ? id : 0) * p.s_rs;
  // an id past the table: a row of NaN (the error shows without a synchronisation) and the status
  const float fill = id < 0 ? 0.f : NAN;
  if (id >= p.V && lane == 0 && p.status) atomicCAS(p.status, 0, VA_ERR_BAD_IDS);
  for (int c0 = lane * kW; c0 < p.D; c0 += kFwdUnroll * lpr * kW) {
    Raw<T> raw[kFwdUnroll];
#pragma unroll
    for (int u = 0; u < kFwdUnroll; ++u) {
      const int c = c0 + u * lpr * kW;
      if (in && c < p.D) raw[u].template load<VEC>(src + c, p.D - c);
    }
#pragma unroll
    for (int u = 0; u < kFwdUnroll; ++u) {
      const int c = c0 + u * lpr * kW;
      if (c >= p.D) break;
      float x[kW];
      raw[u].values(x);
#pragma unroll
      for (int i = 0; i < kW; ++i) x[i] = in ? x[i] * p.scale : fill;
      store_row<VEC>(dst + c, p.D - c, x);
    }
  }
}

// The zero rows of [v0, v1) that no token has (clusters after the first).  VEC: whole rows by bulk
// stores out of zeroed shared memory, one instruction per kZeroBytes; else thread by thread.
template <class T, bool VEC>
__device__ void fill_absent(const EmbedParams& p, uint32_t* present, int v0, int v1) {
  T* dst = static_cast<T*>(p.dst);
  uint4* zeros = reinterpret_cast<uint4*>(present + kPresentWords);
  for (int i = threadIdx.x; VEC && i < kZeroBytes / 16; i += kSortThreads) zeros[i] = make_uint4(0, 0, 0, 0);
  if (VEC) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  for (int a = v0; a < v1; a += kPresentWords * 32) {
    const int n = min(v1 - a, kPresentWords * 32);
    __syncthreads();
    for (int i = threadIdx.x; i < (n + 31) / 32; i += kSortThreads) present[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int t = threadIdx.x; t < p.T; t += kSortThreads) {
      const unsigned r = static_cast<unsigned>(__ldg(p.ids + t)) - static_cast<unsigned>(a);
      if (r < static_cast<unsigned>(n)) atomicOr(&present[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    if constexpr (VEC) {  // a row per thread
      const int bytes = p.D * static_cast<int>(sizeof(T));
      for (int r = threadIdx.x; r < n; r += kSortThreads) {
        if ((present[r >> 5] >> (r & 31)) & 1u) continue;
        uint8_t* row = reinterpret_cast<uint8_t*>(dst + static_cast<int64_t>(a + r) * p.d_rs);
        for (int at = 0; at < bytes; at += kZeroBytes)
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(row + at),
                       "r"(smem_u32(zeros)), "r"(min(kZeroBytes, bytes - at))
                       : "memory");
      }
    } else {
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      const float zero[kW] = {};
      for (int r = warp; r < n; r += kSortWarps) {
        if ((present[r >> 5] >> (r & 31)) & 1u) continue;
        T* row = dst + static_cast<int64_t>(a + r) * p.d_rs;
        for (int c = lane * kW; c < p.D; c += 32 * kW) store_row<VEC>(row + c, p.D - c, zero);
      }
    }
  }
  if (VEC) {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

// Cluster 0 sorts, the others fill.  Stable: warp g of the cluster owns the g-th contiguous share
// of the input, and equal digits keep the order (warp, round, lane).
template <class T, bool VEC>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedParams p) {
  extern __shared__ __align__(16) int sm[];
  griddep_begin();
  if (blockIdx.x >= kSortCtas) {
    const int n = gridDim.x - kSortCtas, i = blockIdx.x - kSortCtas;
    const int per = (p.V + n - 1) / n;
    const int64_t v0 = static_cast<int64_t>(per) * i;
    if (v0 < p.V)
      fill_absent<T, VEC>(p, reinterpret_cast<uint32_t*>(sm), static_cast<int>(v0),
                          static_cast<int>(std::min<int64_t>(p.V, v0 + per)));
    return;
  }
  int* cnt = sm;                              // [warps][bins]: counts, then next ranks
  uint32_t* lanes = reinterpret_cast<uint32_t*>(sm + kSortWarps * kMaxBins);  // [warps][bins]: who has it
  int* hist = sm + 2 * kSortWarps * kMaxBins; // [bins] of this CTA, read by the others
  int* scan = hist + kMaxBins;                // [warps]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int share = ((p.T + kSortCtas * kSortWarps * 32 - 1) / (kSortCtas * kSortWarps * 32)) * 32;  // tokens per warp
  const int64_t b0 = static_cast<int64_t>(rank * kSortWarps + warp) * share;
  const int beg = static_cast<int>(std::min<int64_t>(p.T, b0)), end = static_cast<int>(std::min<int64_t>(p.T, b0 + share));
  if (rank == 0 && tid == 0) *p.status = VA_OK;
  bool bad = false;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.width, bins = 1 << p.width;
    const int2* in = (pass & 1) ? p.pair1 : p.pair0;
    int2* out = (pass & 1) ? p.pair0 : p.pair1;
    // ids outside [0, V) take the key V: they follow every other and are left out
    auto pair_of = [&](int i) -> int2 {
      if (pass > 0) return __ldcg(in + i);
      const int id = __ldg(p.ids + i);
      if (id >= p.V) bad = true;
      return make_int2(id < 0 || id >= p.V ? p.V : id, i);
    };
    for (int i = tid; i < kSortWarps * bins; i += kSortThreads) cnt[i] = lanes[i] = 0;
    __syncthreads();
    int* mine = cnt + warp * bins;
    uint32_t* who = lanes + warp * bins;
    for (int i0 = beg; i0 < end; i0 += 32 * kSortBatch) {
      int k[kSortBatch];
#pragma unroll
      for (int u = 0; u < kSortBatch; ++u) {
        const int i = i0 + 32 * u + lane;
        k[u] = i < end ? pair_of(i).x : -1;
      }
#pragma unroll
      for (int u = 0; u < kSortBatch; ++u) {
        if (k[u] >= 0) atomicAdd(&mine[(k[u] >> shift) & (bins - 1)], 1);
      }
    }
    __syncthreads();
    int total = 0;  // of this CTA, bin tid
    if (tid < bins) {
      for (int w = 0; w < kSortWarps; ++w) {
        const int x = cnt[w * bins + tid];
        cnt[w * bins + tid] = total;
        total += x;
      }
      hist[tid] = total;
    }
    cluster_barrier();
    int all = 0, before = 0;
    if (tid < bins) {
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        const int x = load_remote(hist + tid, r);
        if (r < rank) before += x;
        all += x;
      }
    }
    // exclusive scan of `all` over the bins
    int incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int base = before + incl - all;
    for (int w = 0; w < warp; ++w) base += scan[w];
    if (tid < bins)
      for (int w = 0; w < kSortWarps; ++w) cnt[w * bins + tid] += base;
    __syncthreads();
    for (int i0 = beg; i0 < end; i0 += 32 * kSortBatch) {
      int2 k[kSortBatch];
#pragma unroll
      for (int u = 0; u < kSortBatch; ++u) {
        const int i = i0 + 32 * u + lane;
        k[u] = i < end ? pair_of(i) : make_int2(-1, 0);
      }
#pragma unroll
      for (int u = 0; u < kSortBatch; ++u) {
        if (i0 + 32 * u >= end) break;
        // the lanes with the same digit meet in shared memory (the warp match instruction takes 64
        // cycles of the SM each: T = 131072 sorted in 67 us with it, 44 without)
        const bool have = k[u].x >= 0;
        const int d = (k[u].x >> shift) & (bins - 1);
        if (have) atomicOr(&who[d], 1u << lane);
        __syncwarp();
        const unsigned peers = have ? who[d] : 0u;
        const int at = have ? mine[d] + __popc(peers & ((1u << lane) - 1)) : 0;
        __syncwarp();
        if (have) {
          if (lane == __ffs(peers) - 1) {
            mine[d] += __popc(peers);
            who[d] = 0;
          }
          out[at] = k[u];
        }
        __syncwarp();
      }
    }
    cluster_barrier();  // the sorted pairs are visible, and no CTA's counts are read any more
  }
  if (bad) atomicExch(p.status, VA_ERR_BAD_IDS);
}

// One group of lpr threads per chunk of P sorted tokens (grid.y: further columns).  (The pairs are read
// coherently: a block may be resident while the sort still writes them, see griddep_begin().)
template <class TI, class TO, bool VI, bool VO>
__global__ void __launch_bounds__(kReduceThreads) embed_reduce_kernel(const EmbedParams p, const int2* pair,
                                                                      int lpr) {
  constexpr int kRows = sizeof(TI) == 2 ? 16 : 8;  // rows of dout in flight per thread
  extern __shared__ int sm[];
  griddep_begin();
  const int groups = kReduceThreads / lpr, g = threadIdx.x / lpr, lane = threadIdx.x % lpr;
  const int64_t chunk = static_cast<int64_t>(blockIdx.x) * groups + g, b0 = chunk * p.P;
  // the chunk's keys and tokens, with a key from before it and one from after it (V: none)
  int* keys = sm + g * (2 * p.P + 2) + 1;
  int* toks = keys + p.P + 1;
  for (int i = lane - 1; i < p.P + 1; i += lpr) {
    const int64_t at = b0 + i;
    const bool in = at >= 0 && at < p.T;
    const int2 kt = in ? __ldcg(pair + at) : make_int2(p.V, 0);
    keys[i] = kt.x;
    if (i >= 0 && i < p.P) toks[i] = kt.y;
  }
  __syncthreads();
  const int c = (blockIdx.y * lpr + lane) * kW, n = p.D - c;
  if (b0 >= p.T || n <= 0) return;
  const TI* src = static_cast<const TI*>(p.src) + c;
  TO* dst = static_cast<TO*>(p.dst) + c;
  float* part = p.part + chunk * 2 * p.D + c;
  int cur = keys[0];
  if (cur >= p.V) return;
  const bool joined = keys[-1] == cur;  // the first run began before the chunk
  bool first = true;
  float acc[kW] = {};
  const auto put = [&]() {  // the run that ends here
    if (first && joined) {
#pragma unroll
      for (int i = 0; i < kW; ++i)
        if (i < n) part[i] = acc[i];
    } else {
      TO* row = dst + cur * p.d_rs;
      float x[kW] = {};
      if (p.accumulate) {
        Raw<TO> old;
        old.template load<VO>(row, n);
        old.values(x);
      }
#pragma unroll
      for (int i = 0; i < kW; ++i) x[i] = fmaf(acc[i], p.scale, x[i]);
      store_row<VO>(row, n, x);
    }
    first = false;
  };
  for (int i0 = 0; i0 < p.P && keys[i0] < p.V; i0 += kRows) {
    Raw<TI> raw[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (keys[i0 + u] < p.V) raw[u].template load<VI>(src + toks[i0 + u] * p.s_rs, n);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int k = keys[i0 + u];
      if (k >= p.V) break;
      if (k != cur) {
        put();
        cur = k;
#pragma unroll
        for (int i = 0; i < kW; ++i) acc[i] = 0.f;
      }
      float x[kW];
      raw[u].values(x);
#pragma unroll
      for (int i = 0; i < kW; ++i) acc[i] += x[i];
    }
  }
  if (keys[p.P] == cur) {  // goes on in the next chunk
    float* q = first && joined ? part : part + p.D;
#pragma unroll
    for (int i = 0; i < kW; ++i)
      if (i < n) q[i] = acc[i];
  } else {
    put();
  }
}

// Runs over several chunks: the chunks' sums are added, in order, by the row group whose chunk the run
// starts in, or for a long run (a frequent token) by the whole block, whose groups take equal shares
// of the chunks and whose shares are added in order.
template <class TO, bool VO>
__global__ void __launch_bounds__(kReduceThreads) embed_join_kernel(const EmbedParams p, const int2* pair, int lpr) {
  constexpr int kAhead = 8;  // chunks' sums in flight per thread
  constexpr int kAlone = 16; // chunks of a run that one row group adds by itself
  __shared__ int found[kReduceThreads], found_last[kReduceThreads], nfound;
  __shared__ float share[kReduceThreads][kW];
  griddep_begin();
  const auto key = [&](int64_t i) { return __ldcg(&pair[i].x); };
  const int groups = kReduceThreads / lpr, g = threadIdx.x / lpr, lane = threadIdx.x % lpr;
  if (threadIdx.x == 0) nfound = 0;
  __syncthreads();
  const int c = (blockIdx.y * lpr + lane) * kW, n = p.D - c;
  const float* part = p.part + c;
  const auto load = [&](Raw<float>& x, const float* q) {
    if (p.D % kW == 0) x.load<true>(q, n);
    else x.load<false>(q, n);
  };
  // acc += the sums of chunks [q0, q1) of the run that starts in `chunk`: there it is the chunk's second
  // row, else the first
  const auto add = [&](float (&acc)[kW], int64_t chunk, int64_t q0, int64_t q1) {
    for (int64_t q = q0; n > 0 && q < q1; q += kAhead) {
      Raw<float> raw[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (q + u < q1) load(raw[u], part + ((q + u) * 2 + (q + u == chunk ? 1 : 0)) * p.D);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (q + u >= q1) break;
        float x[kW];
        raw[u].values(x);
#pragma unroll
        for (int i = 0; i < kW; ++i) acc[i] += x[i];
      }
    }
  };
  const auto finish = [&](const float (&acc)[kW], int cur) {
    if (n <= 0) return;
    TO* row = static_cast<TO*>(p.dst) + cur * p.d_rs + c;
    float x[kW] = {};
    if (p.accumulate) {
      Raw<TO> old;
      old.template load<VO>(row, n);
      old.values(x);
    }
#pragma unroll
    for (int i = 0; i < kW; ++i) x[i] = fmaf(acc[i], p.scale, x[i]);
    store_row<VO>(row, n, x);
  };
  {  // the run that starts in this group's chunk and goes on in the next one
    const int64_t chunk = static_cast<int64_t>(blockIdx.x) * groups + g, b0 = chunk * p.P;
    if (b0 + p.P < p.T) {
      const int beg = static_cast<int>(b0), end = beg + p.P, cur = key(end - 1);
      if (cur < p.V && key(end) == cur &&
          !(key(beg) == cur && beg > 0 && key(beg - 1) == cur)) {
        // its end: the first sorted token with a larger key, looked for at doubling distances first
        int lo = end, hi = p.T;
        for (int64_t d = p.P; lo + d < p.T; d *= 2) {
          if (key(lo + d) > cur) {
            hi = static_cast<int>(lo + d);
            break;
          }
          lo += static_cast<int>(d);
        }
        while (lo < hi) {
          const int mid = lo + ((hi - lo) >> 1);
          if (key(mid) > cur) hi = mid;
          else lo = mid + 1;
        }
        const int last = (lo - 1) / p.P;
        if (last - chunk < kAlone || groups == 1) {
          float acc[kW] = {};
          add(acc, chunk, chunk, static_cast<int64_t>(last) + 1);
          finish(acc, cur);
        } else if (lane == 0) {
          const int f = atomicAdd(&nfound, 1);  // (any order: rows of their own)
          found[f] = g;
          found_last[f] = last;
        }
      }
    }
  }
  __syncthreads();
  for (int f = 0; f < nfound; ++f) {  // the whole block on one run
    const int64_t chunk = static_cast<int64_t>(blockIdx.x) * groups + found[f];
    const int64_t stop = static_cast<int64_t>(found_last[f]) + 1, per = (stop - chunk + groups - 1) / groups;
    const int64_t q0 = chunk + g * per;
    float acc[kW] = {};
    add(acc, chunk, q0, q0 + per < stop ? q0 + per : stop);
    __syncthreads();  // the previous run's shares have been read
#pragma unroll
    for (int i = 0; i < kW; ++i) share[threadIdx.x][i] = acc[i];
    __syncthreads();
    if (g != 0) continue;
    for (int h = 1; h < groups; ++h)
#pragma unroll
      for (int i = 0; i < kW; ++i) acc[i] += share[h * lpr + lane][i];
    finish(acc, key((chunk + 1) * p.P));
  }
}

// ---------------------------------------------------------------- host side

namespace {

bool rows_vec(const void* p, int64_t rs, int D, int elem) {
  return D % kW == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && rs * elem % 16 == 0;
}

// Shared memory of the reduce kernel: keys and tokens of every chunk of a block.
size_t chunk_smem(int P, int lpr) { return static_cast<size_t>(kReduceThreads / lpr) * (2 * P + 2) * sizeof(int); }

// Sorted tokens per chunk: enough chunks to fill the GPU (a thousand threads an SM), few enough that
// most runs lie inside one (T = 8192, D = 4096: reduce and join 41 us with 16, 35 with 32, 36 with 64).
int chunk_tokens(int T, int D) {
  const int lpr = lanes_per_row(D, kReduceThreads, 1);
  const int64_t vecs = static_cast<int64_t>(T) * ((D + kW - 1) / kW);
  int P = 16;
  while (P < kMaxP && vecs / P > 152 * 1024 && chunk_smem(2 * P, lpr) <= 48 << 10) P *= 2;
  return P;
}

template <class T, bool VEC>
cudaError_t launch_sort(const EmbedParams& p, int ctas, cudaStream_t st) {
  const auto kernel = embed_sort_kernel<T, VEC>;
  const size_t smem = std::max<size_t>((2 * kSortWarps * kMaxBins + kMaxBins + kSortWarps) * sizeof(int),
                                       kPresentWords * sizeof(uint32_t) + kZeroBytes);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSortCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class TI, class TO, bool VI>
cudaError_t launch_reduce(const EmbedParams& p, bool vo, dim3 grid, const int2* pair, int lpr,
                          cudaStream_t st) {
  const size_t smem = chunk_smem(p.P, lpr);
  return vo ? launch_pdl(embed_reduce_kernel<TI, TO, VI, true>, grid, dim3(kReduceThreads), smem, st, p, pair, lpr)
            : launch_pdl(embed_reduce_kernel<TI, TO, VI, false>, grid, dim3(kReduceThreads), smem, st, p, pair, lpr);
}
template <class TI, class TO>
cudaError_t launch_reduce(const EmbedParams& p, bool vi, bool vo, dim3 grid, const int2* pair, int lpr, cudaStream_t st) {
  return vi ? launch_reduce<TI, TO, true>(p, vo, grid, pair, lpr, st)
            : launch_reduce<TI, TO, false>(p, vo, grid, pair, lpr, st);
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t embed_bwd_workspace(int T, int D) {
  const int P = chunk_tokens(T, D);
  const size_t chunks = (static_cast<size_t>(T) + P - 1) / P;
  return sizeof(WsHeader) + 2 * align256(static_cast<size_t>(T) * sizeof(int2)) +
         align256(chunks * 2 * D * sizeof(float));
}

cudaError_t launch_embed_fwd(const void* table, int bf16, int64_t t_rs, const int32_t* ids, int T, int V, int D,
                             float scale, void* out, int64_t o_rs, int32_t* status, cudaStream_t st) {
  EmbedParams p{};
  p.ids = ids;
  p.T = T;
  p.V = V;
  p.D = D;
  p.scale = scale;
  p.src = table;
  p.s_rs = t_rs;
  p.dst = out;
  p.d_rs = o_rs;
  p.status = status;
  const int elem = bf16 ? 2 : 4;
  const bool vec = rows_vec(table, t_rs, D, elem) && rows_vec(out, o_rs, D, elem);
  const int lpr = lanes_per_row(D, kFwdThreads, kFwdUnroll), groups = kFwdThreads / lpr;
  const dim3 grid((T + groups - 1) / groups), block(kFwdThreads);
  if (bf16)
    return vec ? launch_pdl(embed_fwd_kernel<__nv_bfloat16, true>, grid, block, 0, st, p, lpr)
               : launch_pdl(embed_fwd_kernel<__nv_bfloat16, false>, grid, block, 0, st, p, lpr);
  return vec ? launch_pdl(embed_fwd_kernel<float, true>, grid, block, 0, st, p, lpr)
             : launch_pdl(embed_fwd_kernel<float, false>, grid, block, 0, st, p, lpr);
}

// The three launches of varlen_embed_bwd, in this order on one stream (without tokens the first one
// alone: it writes every row's zeros).
cudaError_t launch_embed_bwd(int stage, const void* dout, int in_bf16, int64_t i_rs, const int32_t* ids, int T, int V,
                             int D, float scale, void* dtable, int out_bf16, int64_t o_rs, int accumulate, void* ws,
                             cudaStream_t st) {
  EmbedParams p{};
  p.ids = ids;
  p.T = T;
  p.V = V;
  p.D = D;
  p.scale = scale;
  p.src = dout;
  p.s_rs = i_rs;
  p.dst = dtable;
  p.d_rs = o_rs;
  p.accumulate = accumulate;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.status = &reinterpret_cast<WsHeader*>(w)->status;
  const size_t one = align256(static_cast<size_t>(T) * sizeof(int2));
  p.pair0 = reinterpret_cast<int2*>(w + sizeof(WsHeader));
  p.pair1 = reinterpret_cast<int2*>(w + sizeof(WsHeader) + one);
  p.part = reinterpret_cast<float*>(w + sizeof(WsHeader) + 2 * one);
  p.P = chunk_tokens(T, D);
  p.bits = 1;
  while (p.bits < 31 && (V >> p.bits) > 0) ++p.bits;  // keys 0 .. V
  p.passes = (p.bits + 8) / 9;
  p.width = (p.bits + p.passes - 1) / p.passes;
  const bool vi = rows_vec(dout, i_rs, D, in_bf16 ? 2 : 4), vo = rows_vec(dtable, o_rs, D, out_bf16 ? 2 : 4);
  if (stage == 0) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // Clusters.  Two CTAs fit an SM, but a cluster stays within one of the GPU's SM groups: three quarters
    // of the slots, so that none is left for a second wave.
    const int fill = accumulate ? 0 : std::max(1, 3 * sms / (2 * kSortCtas) - 1);
    const int ctas = kSortCtas * (1 + fill);
    if (out_bf16) return vo ? launch_sort<__nv_bfloat16, true>(p, ctas, st) : launch_sort<__nv_bfloat16, false>(p, ctas, st);
    return vo ? launch_sort<float, true>(p, ctas, st) : launch_sort<float, false>(p, ctas, st);
  }
  const int2* pair = (p.passes & 1) ? p.pair1 : p.pair0;
  const int lpr = lanes_per_row(D, kReduceThreads, 1), groups = kReduceThreads / lpr;
  const int64_t chunks = (static_cast<int64_t>(T) + p.P - 1) / p.P;
  const dim3 grid(static_cast<unsigned>((chunks + groups - 1) / groups), (D + lpr * kW - 1) / (lpr * kW));
  if (stage == 1) {
    if (in_bf16)
      return out_bf16 ? launch_reduce<__nv_bfloat16, __nv_bfloat16>(p, vi, vo, grid, pair, lpr, st)
                      : launch_reduce<__nv_bfloat16, float>(p, vi, vo, grid, pair, lpr, st);
    return out_bf16 ? launch_reduce<float, __nv_bfloat16>(p, vi, vo, grid, pair, lpr, st)
                    : launch_reduce<float, float>(p, vi, vo, grid, pair, lpr, st);
  }
  const dim3 block(kReduceThreads);
  if (out_bf16)
    return vo ? launch_pdl(embed_join_kernel<__nv_bfloat16, true>, grid, block, 0, st, p, pair, lpr)
              : launch_pdl(embed_join_kernel<__nv_bfloat16, false>, grid, block, 0, st, p, pair, lpr);
  return vo ? launch_pdl(embed_join_kernel<float, true>, grid, block, 0, st, p, pair, lpr)
            : launch_pdl(embed_join_kernel<float, false>, grid, block, 0, st, p, pair, lpr);
}

}  // namespace va
