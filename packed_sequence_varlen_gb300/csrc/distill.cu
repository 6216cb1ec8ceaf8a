// Distillation of the packed stream from a teacher's top logits, with its logit gradient.
//
// Row t has K teacher entries (id, logit a) and the student logits z over V classes.  With the
// temperature tau, over the row's present entries (id >= 0, a > -inf)
//     p_k = softmax(a / tau)_k,   q = softmax(z / tau) over all V classes,
//     L_t = tau^2 sum_k p_k (ln p_k - ln q_{id_k}),
//     dL_t / dz_c = tau (q_c - sum_{k : id_k = c} p_k)          (sum_k p_k = 1),
// and the objective is the packed loss's: the sum over eligible rows divided once by their
// count N.  A row is eligible when its target is not ignore_index and it has a present entry;
// the others are skipped before any arithmetic (logits never read, gradient rows zero).
//
// Kernels (one stream, programmatic dependent launches):
//   distill_count_kernel   one warp per row: eligibility, entry ids in [0, V) -> per-row flags and
//                          one count per block
//   distill_rows_kernel    one cluster of C CTAs per row at a time: see below
//   distill_reduce_kernel  one CTA: N, the sum of the per-row losses in float64 in a fixed
//                          order, the mean; status
//
// Rows.  What bounds it: HBM, z read once and the gradient written once.  So a row stays in
// shared memory between its log-sum-exp and its gradient: CTA rank c of the cluster holds the
// c-th slice, and each of its warps a piece of the slice that it loads with one bulk copy, scans
// for its maximum, sums, overwrites with the gradient and hands to one bulk store, on its own;
// the only barriers of a row are the ones of the (max, sum) exchange.  Rows may start anywhere:
// the elements before the first and after the last 16-byte boundary (at most 7 each) go through
// registers.  The log-sum-exp, p and the row losses are fp32, a gradient value is rounded once.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "sm100_ptx.cuh"

namespace va {
using namespace sm100;

namespace {

constexpr int kDistWarps = 8;
constexpr int kDistThreads = 32 * kDistWarps;
constexpr int kMaxCluster = 8;
constexpr int kMaxParts = 512;       // blocks of the count kernel
constexpr int kMaxSlice = 200 << 10; // bytes of a row's slice that one CTA can hold
constexpr int kReduceThreads = 1024;

struct DistillParams {
  const void* z;
  int64_t z_rs;  // row strides in elements
  const int32_t* ids;
  int64_t ids_rs;
  const void* a;
  int64_t a_rs;
  int a_bf16;
  const int32_t* targets;  // null: every row has a target
  int T, V, K, ignore;
  float temperature;
  void* grad;  // may be null
  int64_t g_rs;
  WsHeader* hdr;
  int32_t* parts;  // [nparts] eligible rows per count block, bit 30: an id outside [0, V)
  int nparts;
  uint8_t* flags;  // [T] eligible
  float* kl;       // [T] row losses
  float* loss;     // {sum, mean}
  int32_t* count;
  int pv;  // 16-byte vectors of a warp's piece (capacity)
  int C;   // CTAs per row
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// The 16-byte vector's W values as fp32 (bf16 is the upper half of an fp32).
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Merges running (max, sum of exp2((x - max) sl2)) pairs; a NaN sum stays NaN.  The maximum is
// kept in the logits' own units and subtracted before the scale: the difference is exact where it
// matters whatever the logits' common offset, and rows filled with the type's lowest value stay
// finite.
__device__ __forceinline__ void ms_merge(float& m, float& s, float m2, float s2, float sl2) {
  const float mx = fmaxf(m, m2);
  if (mx == -INFINITY) {
    s += s2;
    return;
  }
  s = s * fast_exp2((m - mx) * sl2) + s2 * fast_exp2((m2 - mx) * sl2);
  m = mx;
}

// x[e] = exp2((x[e] - m) sl2 + b), in place.
template <int W>
__device__ __forceinline__ void exp_row(float (&x)[W], float m, float sl2, float b) {
#pragma unroll
  for (int e = 0; e < W; e += 2) {
    float d0, d1;
    fadd2(d0, d1, x[e], x[e + 1], -m, -m);
    ffma2(d0, d1, d0, d1, sl2, sl2, b, b);
    x[e] = fast_exp2(d0);
    x[e + 1] = fast_exp2(d1);
  }
}

// Untiled bulk copies: both addresses 16-byte aligned, a positive multiple of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Writes a float pair at the same shared-memory offset of the cluster's CTA `rank`.
__device__ __forceinline__ void store_remote2(uint32_t addr, uint32_t rank, float x, float y) {
  asm volatile("{\n .reg .b32 ra;\n mapa.shared::cluster.u32 ra, %0, %1;\n st.shared::cluster.v2.f32 [ra], {%2, %3};\n}\n" ::"r"(
                   addr),
               "r"(rank), "f"(x), "f"(y)
               : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float teacher(const DistillParams& p, int64_t row, int k) {
  return p.a_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.a)[row * p.a_rs + k])
                  : static_cast<const float*>(p.a)[row * p.a_rs + k];
}

// Shared memory behind the pieces.
struct DistillSmem {
  uint64_t full[kDistWarps];  // one mbarrier per warp: its piece has landed
  float2 red[2][kDistWarps];        // (max, sum) of each warp, by row parity
  float2 cred[2][kMaxCluster];      // (max, sum) of each CTA of the cluster
  float entropy[2];                 // sum_k p_k log2 p_k
  int pad_, abort_flag;
  uint64_t wait_limit;  // right behind the abort flag (wait_limit_slot), 8-byte aligned
  int total[kDistWarps], bad[kDistWarps];
};
static_assert(offsetof(DistillSmem, wait_limit) == offsetof(DistillSmem, abort_flag) + 4 &&
                  offsetof(DistillSmem, wait_limit) % 8 == 0,
              "see wait_limit_slot");

}  // namespace

__global__ void __launch_bounds__(kDistThreads) distill_count_kernel(DistillParams p) {
  griddep_begin();
  __shared__ int tot[kDistWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 0, bad = 0;
  for (int row = blockIdx.x * kDistWarps + warp; row < p.T; row += gridDim.x * kDistWarps) {
    bool any = false;
    if (!p.targets || __ldg(p.targets + row) != p.ignore) {
      for (int k = lane; k < p.K; k += 32) {
        const int id = __ldg(p.ids + row * p.ids_rs + k);
        if (id < 0 || !(teacher(p, row, k) > -INFINITY)) continue;
        any = true;
        bad |= id >= p.V;
      }
    }
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) {
      p.flags[row] = any;
      p.kl[row] = 0.f;
    }
    n += any;
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) tot[warp] = n | (bad << 30);
  __syncthreads();
  if (threadIdx.x == 0) {
    int N = 0, b = 0;
    for (int w = 0; w < kDistWarps; ++w) {
      N += tot[w] & ((1 << 30) - 1);
      b |= tot[w] >> 30;
    }
    p.parts[blockIdx.x] = N | (b << 30);
    if (blockIdx.x == 0) p.hdr->status = VA_OK;
  }
}

// GRAD: write the gradient.  CL: more than one CTA per row.
template <class T, bool GRAD, bool CL>
__global__ void __launch_bounds__(kDistThreads, 3) distill_rows_kernel(const DistillParams p) {
  constexpr int W = 16 / sizeof(T);
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_begin();
  uint4* pieces = reinterpret_cast<uint4*>(smem);
  DistillSmem& sh = *reinterpret_cast<DistillSmem*>(smem + static_cast<size_t>(kDistWarps) * p.pv * 16);
  int* id_s = reinterpret_cast<int*>(&sh + 1);             // [2][K] ids (-1: no entry), by row parity
  float* p_s = reinterpret_cast<float*>(id_s + 2 * p.K);   // [2][K] p_k
  float* z_s = p_s + 2 * p.K;                              // [2][K] z_{id_k}
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CL ? static_cast<int>(cluster_rank()) : 0;
  const int C = CL ? p.C : 1;
  const int first = blockIdx.x / C, step = gridDim.x / C;
  volatile int* abort_flag = &sh.abort_flag;

  // N and the id check
  int n = 0, bad = 0;
  for (int i = tid; i < p.nparts; i += kDistThreads) {
    const int x = p.parts[i];
    n += x & ((1 << 30) - 1);
    bad |= x >> 30;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    sh.total[warp] = n;
    sh.bad[warp] = bad;
    mbar_init(smem_u32(&sh.full[warp]), 1);
    fence_barrier_init();
  }
  if (tid == 0) {
    sh.abort_flag = 0;
    sh.wait_limit = kTimeoutNs;
  }
  __syncthreads();
  n = bad = 0;
  for (int w = 0; w < kDistWarps; ++w) {
    n += sh.total[w];
    bad |= sh.bad[w];
  }
  if (bad || n == 0) {  // the same in every CTA
    if (blockIdx.x == 0 && tid == 0) set_status(p.hdr, VA_ERR_BAD_TARGETS);
    return;
  }
  if (CL) cluster_barrier();  // every CTA of the cluster runs before one writes into another

  const float sl2 = kLog2e / p.temperature;
  const float gmul = p.temperature / static_cast<float>(n), lgm = __log2f(gmul);
  const T* z = static_cast<const T*>(p.z);
  T* grad = static_cast<T*>(p.grad);
  uint4* piece = pieces + static_cast<size_t>(warp) * p.pv;
  const uint32_t piece_a = smem_u32(piece), bar = smem_u32(&sh.full[warp]);

  // A row's cut: `head` elements up to its first 16-byte boundary, vectors, the tail; this
  // warp's piece is the vectors [v0, v0 + nv).
  struct Cut {
    int head, body, v0, nv;
  };
  auto cut = [&](const T* zr) {
    Cut c;
    const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(zr) & 15u);
    c.head = min(p.V, static_cast<int>(((16u - mis) & 15u) / sizeof(T)));
    c.body = (p.V - c.head) / W;  // vectors
    const int per = (c.body + C * kDistWarps - 1) / (C * kDistWarps);  // <= p.pv
    c.v0 = min(c.body, (rank * kDistWarps + warp) * per);
    c.nv = min(c.body, c.v0 + per) - c.v0;
    return c;
  };
  uint32_t phase = 0;
  auto load = [&](int row) {  // whole warp; the piece has been handed out
    const T* zr = z + row * p.z_rs;
    const Cut c = cut(zr);
    if (lane == 0 && c.nv > 0) {
      mbar_expect_tx(bar, c.nv * 16);
      bulk_load(piece_a, zr + c.head + static_cast<int64_t>(c.v0) * W, c.nv * 16, bar);
    }
  };

  int row = first;
  bool have = row < p.T && p.flags[row];
  if (have) load(row);
  int par = 0;
  bool ok = true;
  for (; row < p.T; row += step) {
    const int next = row + step;
    const bool next_have = next < p.T && p.flags[next];
    const T* zr = z + row * p.z_rs;
    T* gr = GRAD ? grad + row * p.g_rs : nullptr;
    const Cut c = cut(zr);
    const int tail0 = c.head + c.body * W;  // first element of the tail
    T* gp = GRAD ? gr + c.head + static_cast<int64_t>(c.v0) * W : nullptr;
    const bool vec = GRAD && (reinterpret_cast<uintptr_t>(gp) & 15u) == 0;
    // the elements outside the vectors: rank 0's first threads take the head, the next the tail
    int edge = -1;
    if (rank == 0 && tid < 2 * W) edge = tid < W ? (tid < c.head ? tid : -1) : (tail0 + tid - W < p.V ? tail0 + tid - W : -1);
    if (!have) {  // not eligible: no arithmetic on its logits, a zero gradient row
      if (GRAD) {
        if (vec) {
          for (int i = lane; i < c.nv; i += 32) __stcs(reinterpret_cast<uint4*>(gp) + i, make_uint4(0, 0, 0, 0));
        } else {
          for (int i = lane; i < c.nv * W; i += 32) gp[i] = from_f<T>(0.f);
        }
        if (edge >= 0) gr[edge] = from_f<T>(0.f);
      }
      if (next_have) load(next);
      have = next_have;
      continue;
    }
    int* ids = id_s + par * p.K;
    float* pk = p_s + par * p.K;
    float* zk = z_s + par * p.K;
    if (warp == kDistWarps - 1) {  // the teacher's entries, while the pieces arrive
      float mx = -INFINITY;
      for (int k = lane; k < p.K; k += 32) {
        const int id = __ldg(p.ids + row * p.ids_rs + k);
        const float a = teacher(p, row, k);
        const bool in = id >= 0 && a > -INFINITY;
        ids[k] = in ? id : -1;
        pk[k] = in ? a : -INFINITY;
        zk[k] = in ? to_f(zr[id]) : 0.f;
        mx = fmaxf(mx, in ? a : -INFINITY);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float s = 0.f;
      for (int k = lane; k < p.K; k += 32) s += ids[k] >= 0 ? fast_exp2((pk[k] - mx) * sl2) : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float ls = __log2f(s), inv = 1.f / s;
      float ent = 0.f;
      for (int k = lane; k < p.K; k += 32) {
        const float x = (pk[k] - mx) * sl2, pr = ids[k] >= 0 ? fast_exp2(x) * inv : 0.f;
        pk[k] = pr;
        if (pr != 0.f) ent += pr * (x - ls);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ent += __shfl_xor_sync(0xffffffffu, ent, o);
      if (lane == 0) sh.entropy[par] = ent;
    }
    // (max, sum of exp2) of this warp's piece and of the row's edge elements
    const float ze = edge >= 0 ? to_f(zr[edge]) : -INFINITY;
    if (c.nv > 0) {
      if (ok) ok = wwait(bar, phase, abort_flag, p.hdr, 60);
      phase ^= 1;
    }
    float m = ze == ze ? ze : -INFINITY;  // (a NaN reaches the sum)
    for (int i = lane; i < c.nv; i += 32) {
      float x[W];
      unpack(piece[i], x);
#pragma unroll
      for (int e = 0; e < W; ++e) m = fmaxf(m, x[e]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = 0.f;
    const float m0 = m == -INFINITY ? 0.f : m;
    for (int i = lane; i < c.nv; i += 32) {
      float x[W];
      unpack(piece[i], x);
      exp_row(x, m0, sl2, 0.f);
#pragma unroll
      for (int e = 0; e < W; ++e) s += x[e];
    }
    if (edge >= 0) s += fast_exp2((ze - m0) * sl2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sh.red[par][warp] = make_float2(m, s);
    __syncthreads();
    m = sh.red[par][0].x;
    s = sh.red[par][0].y;
#pragma unroll
    for (int w = 1; w < kDistWarps; ++w) ms_merge(m, s, sh.red[par][w].x, sh.red[par][w].y, sl2);
    if (CL) {
      if (tid < C) store_remote2(smem_u32(&sh.cred[par][rank]), tid, m, s);
      cluster_barrier();
      m = sh.cred[par][0].x;
      s = sh.cred[par][0].y;
      for (int r = 1; r < C; ++r) ms_merge(m, s, sh.cred[par][r].x, sh.cred[par][r].y, sl2);
    }
    const float ls2 = __log2f(s);
    if (rank == 0 && warp == 0) {  // the row loss: sum_k p_k (ln p_k - (z_k - max) / tau + ln s)
      float cross = 0.f;
      for (int k = lane; k < p.K; k += 32)
        if (pk[k] != 0.f) cross += pk[k] * ((zk[k] - m) / p.temperature);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) cross += __shfl_xor_sync(0xffffffffu, cross, o);
      if (lane == 0) p.kl[row] = p.temperature * p.temperature * ((sh.entropy[par] + ls2) * kLn2 - cross);
    }
    if (GRAD) {
      // gradient tau / N (q_c - P_c), P_c the teacher's weight on class c; the piece first gets
      // the q part, then its teacher entries are written over
      const float b = lgm - ls2;
      for (int i = lane; i < c.nv; i += 32) {
        float x[W];
        unpack(piece[i], x);
        exp_row(x, m, sl2, b);
        piece[i] = pack(x);
      }
      if (edge >= 0) {
        float P = 0.f;
        for (int k = 0; k < p.K; ++k) P += ids[k] == edge ? pk[k] : 0.f;
        gr[edge] = from_f<T>(fast_exp2(fmaf(ze - m, sl2, b)) - P * gmul);
      }
      // A class may be listed twice: each entry first leaves its number in its cell; one that finds
      // another number there shares the class, and then every entry sums over its equals.
      T* cell = reinterpret_cast<T*>(piece);
      const int c0 = c.head + c.v0 * W, c1 = c0 + c.nv * W;
      using Raw = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
      __syncwarp();
      for (int k = lane; k < p.K; k += 32) {
        const int id = ids[k];
        if (id >= c0 && id < c1) reinterpret_cast<Raw*>(cell)[id - c0] = static_cast<Raw>(k);
      }
      __syncwarp();
      bool twice = false;
      for (int k = lane; k < p.K; k += 32) {
        const int id = ids[k];
        if (id >= c0 && id < c1) twice |= reinterpret_cast<Raw*>(cell)[id - c0] != static_cast<Raw>(k);
      }
      twice = __any_sync(0xffffffffu, twice);
      for (int k = lane; k < p.K; k += 32) {
        const int id = ids[k];
        if (id < c0 || id >= c1) continue;
        float P = pk[k];
        if (twice) {
          P = 0.f;
          for (int k2 = 0; k2 < p.K; ++k2) P += ids[k2] == id ? pk[k2] : 0.f;
        }
        cell[id - c0] = from_f<T>(fast_exp2(fmaf(zk[k] - m, sl2, b)) - P * gmul);
      }
      if (vec) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && c.nv > 0 && ok) {
          bulk_store(gp, piece_a, c.nv * 16);
          tma_store_commit();
          tma_store_wait_read();
        }
      } else {
        __syncwarp();
        for (int i = lane; i < c.nv * W; i += 32) gp[i] = cell[i];
        fence_proxy_async_smem();  // the reads above come before the next bulk load's writes
      }
    } else {
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (next_have && ok) load(next);
    have = next_have;
    par ^= 1;
  }
  tma_store_wait_all();
  if (!ok && lane == 0) {  // a wait gave up: let this warp's own copy land (bounded again)
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, phase ^ 1) && globaltimer() - t0 < 50000000ull) {
    }
  }
}

__global__ void __launch_bounds__(kReduceThreads) distill_reduce_kernel(DistillParams p) {
  griddep_begin();
  __shared__ double part[kReduceThreads / 32];
  __shared__ int tot[kReduceThreads / 32];
  double acc = 0.0;  // fixed assignment of rows to threads and a fixed reduction order
  for (int t = threadIdx.x; t < p.T; t += kReduceThreads) acc += static_cast<double>(p.kl[t]);
  int n = 0;
  for (int i = threadIdx.x; i < p.nparts; i += kReduceThreads) n += p.parts[i] & ((1 << 30) - 1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) {
    part[threadIdx.x >> 5] = acc;
    tot[threadIdx.x >> 5] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
    int N = 0;
    for (int w = 0; w < kReduceThreads / 32; ++w) {
      sum += part[w];
      N += tot[w];
    }
    const bool good = p.hdr->status == VA_OK;
    p.loss[0] = good ? static_cast<float>(sum) : NAN;
    p.loss[1] = good ? static_cast<float>(sum / N) : NAN;
    *p.count = N;
  }
}

// ---------------------------------------------------------------- host side

namespace {

int count_blocks(int T) { return std::min(kMaxParts, (T + kDistWarps - 1) / kDistWarps); }

template <class T, bool GRAD, bool CL>
cudaError_t launch_rows_t(const DistillParams& p, int grid, size_t smem, cudaStream_t st) {
  const auto kernel = distill_rows_kernel<T, GRAD, CL>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kDistThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL ? p.C : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class T>
cudaError_t launch_rows(const DistillParams& p, int grid, size_t smem, cudaStream_t st) {
  if (p.C > 1) return p.grad ? launch_rows_t<T, true, true>(p, grid, smem, st) : launch_rows_t<T, false, true>(p, grid, smem, st);
  return p.grad ? launch_rows_t<T, true, false>(p, grid, smem, st) : launch_rows_t<T, false, false>(p, grid, smem, st);
}

}  // namespace

// Whether a row of V classes fits the cluster's shared memory.
bool distill_row_fits(int V, int elem) {
  return static_cast<int64_t>(V) * elem <= static_cast<int64_t>(kMaxSlice) * kMaxCluster;
}

size_t distill_parts_bytes() { return kMaxParts * sizeof(int32_t); }

// The three launches of varlen_token_distill, in this order on one stream.
cudaError_t launch_token_distill(int stage, const void* z, int bf16, int64_t z_rs, const int32_t* ids, int64_t ids_rs,
                                 const void* a, int a_bf16, int64_t a_rs, const int32_t* targets, int T, int V, int K,
                                 int ignore, float temperature, void* grad, int64_t g_rs, void* hdr, int32_t* parts,
                                 uint8_t* flags, float* kl, float* loss, int32_t* count, cudaStream_t st) {
  DistillParams p{z, z_rs, ids, ids_rs, a, a_rs, a_bf16, targets, T, V, K, ignore, temperature, grad, g_rs,
                  static_cast<WsHeader*>(hdr), parts, count_blocks(T), flags, kl, loss, count, 0, 1};
  if (stage == 0) return launch_pdl(distill_count_kernel, dim3(p.nparts), dim3(kDistThreads), 0, st, p);
  if (stage == 2) return launch_pdl(distill_reduce_kernel, dim3(1), dim3(kReduceThreads), 0, st, p);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int elem = bf16 ? 2 : 4;
  // CTAs per row: the fewest whose slices leave room for three CTAs on an SM (loads, arithmetic
  // and stores of different rows overlap), more while the rows alone leave SMs idle.
  const int64_t bytes = static_cast<int64_t>(V) * elem;
  const auto slice = [&](int C) { return (bytes + C - 1) / C; };
  while (p.C < kMaxCluster && slice(p.C) > (68 << 10)) p.C *= 2;
  while (p.C < kMaxCluster && static_cast<int64_t>(T) * p.C < 2 * sms && slice(p.C) > (8 << 10)) p.C *= 2;
  const int64_t body = bytes / 16;
  p.pv = static_cast<int>((body + p.C * kDistWarps - 1) / (p.C * kDistWarps));
  const size_t smem = static_cast<size_t>(kDistWarps) * p.pv * 16 + sizeof(DistillSmem) + static_cast<size_t>(K) * 24;
  const int per_sm = std::max<int>(1, std::min<int>(3, (227 << 10) / static_cast<int>(smem + 1024)));
  const int clusters = std::max(1, std::min(T, sms * per_sm / p.C));
  return bf16 ? launch_rows<__nv_bfloat16>(p, clusters * p.C, smem, st) : launch_rows<float>(p, clusters * p.C, smem, st);
}

}  // namespace va
