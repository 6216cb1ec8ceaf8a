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
// c-th slice (one bulk copy in, one out), and its NW working warps each scan a piece of it for the
// maximum, sum it and overwrite it with the gradient.  A CTA takes its rows one after the other; three
// CTAs share an SM, so one's copies run under the others' arithmetic.  (Deeper pipelines inside one
// CTA of 16 warps measured no faster: what a row costs there is the latency of its reductions.)
// One more warp per CTA prepares the teacher's entries a row ahead (loaded two rows ahead), and handles
// the elements before the row's first and after its last 16-byte boundary (at most 7 each), so rows may
// start anywhere.  The (max, sum) pairs cross the cluster by asynchronous stores that count on the
// receiver's barrier: a release at cluster scope instead cost 2000 cycles a row.  The log-sum-exp, p
// and the row losses are fp32, a gradient value is rounded once; every CTA adds its rows' losses in
// fp64.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "sm100_ptx.cuh"

namespace va {
using namespace sm100;

namespace {

constexpr int kCountWarps = 8;
constexpr int kMaxWarps = 8;         // working warps of a CTA of the rows kernel
constexpr int kMaxCluster = 8;
constexpr int kEdge = 16;            // elements outside the 16-byte vectors: < 8 on each side
constexpr int kMaxParts = 512;       // blocks of the count kernel
constexpr int kMaxCtas = 4096;       // of the rows kernel
constexpr int kSeenBits = 15;
constexpr int kMaxSlice = 160 << 10; // bytes of a row's slice that one CTA can hold
constexpr int kSmemBytes = 227 << 10;
constexpr int kReduceThreads = 1024;
constexpr int kSmGroups = 16;        // at most, of the GPU

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
  double* sums;    // [CTAs of the rows kernel] row losses
  int32_t* ctas;   // their number, from the rows kernel to the reduce kernel
  float* loss;     // {sum, mean}
  int32_t* count;
  int pv;  // 16-byte vectors of a warp's piece (capacity)
  int C;   // CTAs per row
  int NW;  // working warps per CTA
  uint64_t wait_ns;  // test hook: a wait limit in ns, and rank 0 of a cluster loads nothing; 0 = none
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

// Exponents are formed as (x - max) * (log2(e) / tau): the difference comes first, so it is exact
// where it matters whatever the logits' common offset, and rows filled with the type's lowest value
// stay finite.
//
// x[e] = exp2((x[e] - m) sl2 + b), in place.  ONE: as x[e] sl2 + b with b = (its b) - m sl2, a third
// fewer instructions before the exponential; b's rounding costs 2^-24 |m sl2| then, which kOneLimit
// keeps at 2^-16 of the result, against bf16's half step of 2^-8 (fp32 rows do not use it).
constexpr float kOneLimit = 256.f;
template <bool ONE, int W>
__device__ __forceinline__ void exp_row(float (&x)[W], float m, float sl2, float b) {
#pragma unroll
  for (int e = 0; e < W; e += 2) {
    float d0 = x[e], d1 = x[e + 1];
    if (!ONE) fadd2(d0, d1, d0, d1, -m, -m);
    ffma2(d0, d1, d0, d1, sl2, sl2, b, b);
    x[e] = fast_exp2(d0);
    x[e + 1] = fast_exp2(d1);
  }
}

// Calls f(vectors) on `n` 16-byte vectors of shared memory, a warp's lanes in turn; four per lane
// are loaded together.
template <class F>
__device__ __forceinline__ void each_vec(uint4* v, int n, F&& f) {
  int i = threadIdx.x & 31;
  for (; i + 96 < n; i += 128) {
    uint4 u[4] = {v[i], v[i + 32], v[i + 64], v[i + 96]};
#pragma unroll
    for (int j = 0; j < 4; ++j) f(u[j], i + 32 * j);
  }
  for (; i < n; i += 32) f(v[i], i);
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
// Writes a float pair at this CTA's address `addr`, taken in the cluster's CTA `rank`, and counts its 8
// bytes on that CTA's barrier at `bar`: no fence, the data travels with its completion.
__device__ __forceinline__ void send_pair(uint32_t addr, uint32_t bar, uint32_t rank, float x, float y) {
  asm volatile(
      "{\n .reg .b32 ra, rb;\n mapa.shared::cluster.u32 ra, %0, %2;\n mapa.shared::cluster.u32 rb, %1, %2;\n"
      " st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [ra], {%3, %4}, [rb];\n}\n" ::"r"(addr),
      "r"(bar), "r"(rank), "f"(x), "f"(y)
      : "memory");
}
// Barrier of the cluster's threads (a CTA launched alone is a cluster of its own), in two halves:
// what was written before the arrival is visible after the wait.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float teacher(const DistillParams& p, int64_t row, int k) {
  return p.a_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.a)[row * p.a_rs + k])
                  : static_cast<const float*>(p.a)[row * p.a_rs + k];
}

// Elementwise maximum of a vector's values, kept packed for bf16.
struct VecMaxF {
  float m = -INFINITY;
  __device__ __forceinline__ void add(const uint4& u) {
    m = fmax3(m, __uint_as_float(u.x), __uint_as_float(u.y));
    m = fmax3(m, __uint_as_float(u.z), __uint_as_float(u.w));
  }
  __device__ __forceinline__ float get() const { return m; }
};
struct VecMaxB {
  uint32_t m = 0xff80ff80u;  // (-inf, -inf)
  __device__ __forceinline__ void one(uint32_t x) { asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x)); }
  __device__ __forceinline__ void add(const uint4& u) {
    one(u.x);
    one(u.y);
    one(u.z);
    one(u.w);
  }
  __device__ __forceinline__ float get() const {
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};
template <class T> struct VecMax;
template <> struct VecMax<float> : VecMaxF {};
template <> struct VecMax<__nv_bfloat16> : VecMaxB {};

__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Shared memory behind the slice.
struct DistillSmem {
  uint64_t full, done;                            // the slice has landed / holds the gradient
  uint64_t swapped[2];                            // every warp's pair of a row is here, by row parity
  float2 pair[2][kMaxCluster * (kMaxWarps + 1)];  // (max, sum) of every warp of the cluster
  float edge[2][kEdge];                           // logits outside the vectors
  float entropy[2];                               // sum_k p_k log2 p_k
  int twice[2];                                   // the row may list a class more than once
  uint32_t seen[1 << (kSeenBits - 5)];            // hashes of the classes of the row being prepared
  int total[kMaxWarps + 1], bad[kMaxWarps + 1];
  int abort_flag_pad, abort_flag;
  uint64_t wait_limit;  // right behind the abort flag (wait_limit_slot), 8-byte aligned
};
static_assert(offsetof(DistillSmem, wait_limit) == offsetof(DistillSmem, abort_flag) + 4 &&
                  offsetof(DistillSmem, wait_limit) % 8 == 0,
              "see wait_limit_slot");

}  // namespace

__global__ void __launch_bounds__(32 * kCountWarps) distill_count_kernel(DistillParams p) {
  constexpr int kBatch = 4;  // entries a lane loads together
  griddep_begin();
  __shared__ int tot[kCountWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 0, bad = 0;
  for (int row = blockIdx.x * kCountWarps + warp; row < p.T; row += gridDim.x * kCountWarps) {
    // (target, ids and logits are loaded side by side: one latency, not three; the target by a coherent
    // load, since the kernel that writes the targets may still run when this one becomes resident)
    const bool has = !p.targets || p.targets[row] != p.ignore;
    bool any = false;
    for (int k0 = lane; k0 < p.K; k0 += 32 * kBatch) {
      int id[kBatch];
      float a[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = k0 + 32 * u;
        id[u] = k < p.K ? __ldg(p.ids + row * p.ids_rs + k) : -1;
        a[u] = k < p.K ? teacher(p, row, k) : -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (!has || id[u] < 0 || !(a[u] > -INFINITY)) continue;
        any = true;
        bad |= id[u] >= p.V;
      }
    }
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) p.flags[row] = any;
    n += any;
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) tot[warp] = n | (bad << 30);
  __syncthreads();
  if (threadIdx.x == 0) {
    int N = 0, b = 0;
    for (int w = 0; w < kCountWarps; ++w) {
      N += tot[w] & ((1 << 30) - 1);
      b |= tot[w] >> 30;
    }
    p.parts[blockIdx.x] = N | (b << 30);
    if (blockIdx.x == 0) p.hdr->status = VA_OK;
  }
}

// The rows of one cluster in order, r = first, first + step, ...: next() gives the next eligible
// one (-1: none left) and calls skip(r) for every other.  Whole warp; flags are read 32 at a time.
struct RowList {
  const uint8_t* flags;
  int64_t at;  // next row to look at
  int T, step, i = 32;
  unsigned mask = 0;
  template <class Skip>
  __device__ __forceinline__ int next(Skip&& skip) {
    for (; at < T; at += step, ++i) {
      if (i == 32) {
        const int64_t r = at + static_cast<int64_t>(threadIdx.x & 31) * step;
        mask = __ballot_sync(0xffffffffu, r < T && flags[r]);
        i = 0;
      }
      if ((mask >> i) & 1u) {
        const int r = static_cast<int>(at);
        at += step;
        ++i;
        return r;
      }
      skip(static_cast<int>(at));
    }
    return -1;
  }
};

// GRAD: write the gradient.
template <class T, bool GRAD>
__global__ void __launch_bounds__((kMaxWarps + 1) * 32, 3) distill_rows_kernel(const DistillParams p) {
  constexpr int W = 16 / sizeof(T);
  constexpr bool kBf = sizeof(T) == 2;
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_begin();
  const int NW = p.NW, C = p.C, nthreads = (NW + 1) * 32;
  uint4* slice = reinterpret_cast<uint4*>(smem);
  DistillSmem& sh = *reinterpret_cast<DistillSmem*>(smem + static_cast<size_t>(NW) * p.pv * 16);
  int* id_s = reinterpret_cast<int*>(&sh + 1);             // [2][K] ids (-1: no entry), by row parity
  float* p_s = reinterpret_cast<float*>(id_s + 2 * p.K);   // [2][K] p_k
  float* z_s = p_s + 2 * p.K;                              // [2][K] z_{id_k}
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int first = blockIdx.x / C, step = gridDim.x / C;
  volatile int* abort_flag = &sh.abort_flag;

  // N and the id check
  int n = 0, bad = 0;
  for (int i = tid; i < p.nparts; i += nthreads) {
    const int x = p.parts[i];
    n += x & ((1 << 30) - 1);
    bad |= x >> 30;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    sh.total[warp] = n;
    sh.bad[warp] = bad;
  }
  if (blockIdx.x == 0 && tid == 0) *p.ctas = gridDim.x;
  if (tid == 0) {
    mbar_init(smem_u32(&sh.full), 1);
    mbar_init(smem_u32(&sh.done), NW);
    for (int x = 0; x < 2; ++x) mbar_init(smem_u32(&sh.swapped[x]), NW + 1);
    fence_barrier_init();
    sh.abort_flag = 0;
    sh.wait_limit = p.wait_ns ? p.wait_ns : kTimeoutNs;
  }
  cluster_arrive();  // (also: every CTA of the cluster runs before one writes into another)
  cluster_wait();
  n = bad = 0;
  for (int w = 0; w <= NW; ++w) {
    n += sh.total[w];
    bad |= sh.bad[w];
  }
  if (bad || n == 0) {  // the same in every CTA
    if (blockIdx.x == 0 && tid == 0) set_status(p.hdr, VA_ERR_BAD_TARGETS);
    return;
  }

  const float sl2 = kLog2e / p.temperature;
  const float gmul = p.temperature / static_cast<float>(n), lgm = __log2f(gmul);
  const T* z = static_cast<const T*>(p.z);
  T* grad = static_cast<T*>(p.grad);

  // A row's cut: `head` elements up to its first 16-byte boundary, `body` vectors, the tail; warp w
  // of rank r holds the vectors [r NW + w, r NW + w + 1) pv.
  const auto head_of = [&](const T* zr) {
    const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(zr) & 15u);
    return min(p.V, static_cast<int>(((16u - mis) & 15u) / sizeof(T)));
  };
  // A warp whose wait gives up ends that row, reading no table that it has not waited for, and takes no
  // other: whoever counts on it gives up in turn, and nobody goes on with tables or barriers a row ahead.
  bool ok = true;
  // (max, sum of exp2) of this warp's part of the it-th row, to every CTA of the cluster.  A pair of
  // row it + 2 may overwrite one of row it: its warp has seen every pair of row it + 1, and a warp
  // gives that one after it has read those of row it.
  const auto publish = [&](int it, float m, float s) {
    __syncwarp();
    float2* at = &sh.pair[it & 1][rank * (NW + 1) + warp];
    const uint32_t bar = smem_u32(&sh.swapped[it & 1]);
    if (lane < C && lane != rank) send_pair(smem_u32(at), bar, lane, m, s);
    if (lane == rank) {
      *at = make_float2(m, s);
      if (warp == NW && C > 1) mbar_expect_tx(bar, (C - 1) * (NW + 1) * 8);  // the other CTAs' pairs
      else mbar_arrive(bar);
    }
    __syncwarp();
  };
  // the row's (max, log2 of the sum) from every warp's pair
  const int npairs = C * (NW + 1);
  const auto merge = [&](int it, float& m, float& ls) {
    if (ok) ok = wwait(smem_u32(&sh.swapped[it & 1]), (it >> 1) & 1, abort_flag, p.hdr, 62);
    const float2* pair = sh.pair[it & 1];
    float mx = -INFINITY;
    for (int i = lane; i < npairs; i += 32) mx = fmaxf(mx, pair[i].x);
    m = warp_max(mx);
    const float m0 = m == -INFINITY ? 0.f : m;
    float s = 0.f;
    for (int i = lane; i < npairs; i += 32) {
      const float2 q = pair[i];
      s += q.x == -INFINITY ? q.y : q.y * fast_exp2((q.x - m0) * sl2);  // (a NaN sum stays NaN)
    }
    ls = __log2f(warp_sum(s));
  };

  RowList rows{p.flags, first, p.T, step};
  if (warp < NW) {
    // ------------------------------------------------------------ a piece of every row
    struct Cut {
      int c0, nv;  // first element, vectors
    };
    const int at_vec = (rank * NW + warp) * p.pv;  // C NW pv >= body
    const auto cut = [&](const T* zr) {
      const int head = head_of(zr), body = (p.V - head) / W, v0 = min(body, at_vec);
      return Cut{head + v0 * W, min(body - v0, p.pv)};
    };
    const auto zero = [&](int row) {  // not eligible: no arithmetic on its logits, a zero gradient row
      if (!GRAD) return;
      const Cut c = cut(z + row * p.z_rs);
      T* g = grad + row * p.g_rs + c.c0;
      if ((reinterpret_cast<uintptr_t>(g) & 15u) == 0) {
        for (int i = lane; i < c.nv; i += 32) __stcs(reinterpret_cast<uint4*>(g) + i, make_uint4(0, 0, 0, 0));
      } else {
        for (int i = lane; i < c.nv * W; i += 32) g[i] = from_f<T>(0.f);
      }
    };
    // warp 0 moves the slice (its own piece is the slice's first one)
    const auto slice_bytes = [&](const T* zr, const Cut& c) {
      const int body = (p.V - head_of(zr)) / W;
      return min(body - min(body, at_vec), NW * p.pv) * 16;
    };
    const auto load = [&](int row) {
      const T* zr = z + row * p.z_rs;
      const Cut c = cut(zr);
      const int bytes = slice_bytes(zr, c);
      if (lane != 0) return;
      if (bytes > 0) {
        mbar_expect_tx(smem_u32(&sh.full), bytes);
        bulk_load(smem_u32(smem), zr + c.c0, bytes, smem_u32(&sh.full));
      } else {
        mbar_arrive(smem_u32(&sh.full));
      }
    };
    uint4* piece = slice + static_cast<size_t>(warp) * p.pv;
    T* cell = reinterpret_cast<T*>(piece);
    int r0 = rows.next(zero);
    bool loading = r0 >= 0;
    if (warp == 0 && r0 >= 0 && !(p.wait_ns && rank == 0)) load(r0);
    int it = 0;
    for (; r0 >= 0; ++it) {
      const int slot = it & 1;
      const Cut c = cut(z + r0 * p.z_rs);
      const int c0 = c.c0, c1 = c0 + c.nv * W;
      if (ok) ok = wwait(smem_u32(&sh.full), it & 1, abort_flag, p.hdr, 60);
      loading = loading && !ok;
      VecMax<T> vm;
      each_vec(piece, c.nv, [&](const uint4& u, int) { vm.add(u); });
      float m = warp_max(vm.get());
      {
        const float m0 = m == -INFINITY ? 0.f : m;
        float s0 = 0.f, s1 = 0.f;
        const auto sum = [&](auto one, float b) {
          each_vec(piece, c.nv, [&](const uint4& u, int) {
            float x[W];
            unpack(u, x);
            exp_row<decltype(one)::value>(x, m0, sl2, b);
#pragma unroll
            for (int e = 0; e < W; e += 2) fadd2(s0, s1, s0, s1, x[e], x[e + 1]);
          });
        };
        if (kBf && fabsf(m0 * sl2) < kOneLimit) sum(std::true_type{}, -m0 * sl2);
        else sum(std::false_type{}, 0.f);
        publish(it, m, warp_sum(s0 + s1));
      }
      int r1 = rows.next(zero);
      float ls;
      merge(it, m, ls);
      if (!ok) r1 = -1;  // the last row
      // the logits of the listed classes of this piece
      const int* ids = id_s + slot * p.K;
      const float* pk = p_s + slot * p.K;
      float* zk = z_s + slot * p.K;
      unsigned hits = 0;  // this lane's entries (lane + 32 u) whose class is in the piece
      for (int k = lane, u = 0; ok && k < p.K; k += 32, ++u) {
        const int id = ids[k];
        if (id < c0 || id >= c1) continue;
        hits |= 1u << u;
        zk[k] = to_f(cell[id - c0]);
      }
      if (GRAD) {
        // tau / N (q_c - P_c), P_c the teacher's weight on class c: the piece first gets the q part,
        // then its teacher entries are written over
        __syncwarp();
        const float off = lgm - ls;
        const auto fill = [&](auto one, float b) {
          each_vec(piece, c.nv, [&](const uint4& u, int i) {
            float x[W];
            unpack(u, x);
            exp_row<decltype(one)::value>(x, m, sl2, b);
            piece[i] = pack(x);
          });
        };
        if (kBf && fabsf(m * sl2) < kOneLimit) fill(std::true_type{}, off - m * sl2);
        else fill(std::false_type{}, off);
        // A class may be listed twice: where the row's hashes say so, each entry first leaves its
        // number in its cell; one that finds another number there shares the class, and then every
        // entry sums over its equals.
        using Raw = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
        const auto each_hit = [&](auto&& f) {
          for (unsigned h = hits; h; h &= h - 1) f(lane + 32 * (__ffs(h) - 1));
        };
        __syncwarp();
        bool twice = sh.twice[slot] != 0;
        if (twice) {
          each_hit([&](int k) { reinterpret_cast<Raw*>(cell)[ids[k] - c0] = static_cast<Raw>(k); });
          __syncwarp();
          twice = false;
          each_hit([&](int k) { twice |= reinterpret_cast<Raw*>(cell)[ids[k] - c0] != static_cast<Raw>(k); });
          twice = __any_sync(0xffffffffu, twice);
        }
        each_hit([&](int k) {
          const int id = ids[k];
          float P = pk[k];
          if (twice) {
            P = 0.f;
            for (int k2 = 0; k2 < p.K; ++k2) P += ids[k2] == id ? pk[k2] : 0.f;
          }
          cell[id - c0] = from_f<T>(fast_exp2(fmaf(zk[k] - m, sl2, off)) - P * gmul);
        });
        T* g = grad + r0 * p.g_rs + c0;
        if ((reinterpret_cast<uintptr_t>(g) & 15u) != 0) {  // on another 16-byte phase than the logits
          __syncwarp();
          for (int i = lane; i < c.nv * W; i += 32) g[i] = cell[i];
        }
      }
      fence_proxy_async_smem();  // the accesses above come before the copies below
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.done));
      if (warp == 0) {
        if (ok) ok = wwait(smem_u32(&sh.done), it & 1, abort_flag, p.hdr, 61);
        if (!ok) break;
        const T* zr = z + r0 * p.z_rs;
        T* g = GRAD ? grad + r0 * p.g_rs + c0 : nullptr;
        if (GRAD && (reinterpret_cast<uintptr_t>(g) & 15u) == 0) {
          const int bytes = slice_bytes(zr, c);
          if (lane == 0 && bytes > 0) {
            bulk_store(g, smem_u32(smem), bytes);
            tma_store_commit();
            tma_store_wait_read();
          }
          __syncwarp();
        }
        if (r1 >= 0) {
          load(r1);
          loading = true;
        }
      }
      r0 = r1;
    }
    if (warp == 0 && lane == 0) {
      tma_store_wait_all();
      const uint64_t t0 = globaltimer();  // row it's wait gave up: let its copy land (bounded again)
      while (!ok && loading && !mbar_try_wait(smem_u32(&sh.full), it & 1) && globaltimer() - t0 < 50000000ull) {
      }
    }
  } else {
    // ------------------------------------------------------------ the teacher's entries, the edges
    const auto edge_of = [&](const T* zr) {  // this lane's element (rank 0), or -1
      const int head = head_of(zr), tail = head + (p.V - head) / W * W;
      if (rank != 0 || lane >= 2 * W) return -1;
      const int e = lane < W ? lane : tail + lane - W;
      return lane < W ? (e < head ? e : -1) : (e < p.V ? e : -1);
    };
    const auto zero = [&](int row) {
      const int e = GRAD ? edge_of(z + row * p.z_rs) : -1;
      if (e >= 0) grad[row * p.g_rs + e] = from_f<T>(0.f);
    };
    // A row's first entries and its edge element, loaded a row before teach() takes them.
    constexpr int kAhead = 4;
    int fid[kAhead];
    float fa[kAhead], fe = -INFINITY;
    const auto fetch = [&](int row) {
      const T* zr = z + row * p.z_rs;
      const int e = edge_of(zr);
      fe = e >= 0 ? to_f(zr[e]) : -INFINITY;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = lane + 32 * u;
        fid[u] = k < p.K ? __ldg(p.ids + row * p.ids_rs + k) : -1;
        fa[u] = k < p.K ? teacher(p, row, k) : -INFINITY;
      }
    };
    const auto teach = [&](int row, int slot) {
      int* ids = id_s + slot * p.K;
      float* pk = p_s + slot * p.K;
      if (lane < kEdge) sh.edge[slot][lane] = fe;
      const auto hash = [](int id) { return (static_cast<uint32_t>(id) * 2654435761u) >> (32 - kSeenBits); };
      float mx = -INFINITY;
      bool twice = false;  // one hash seen twice: perhaps a class listed twice
      const auto take = [&](int k, int id, float a) {
        const bool in = id >= 0 && a > -INFINITY;
        ids[k] = in ? id : -1;
        pk[k] = in ? a : -INFINITY;
        mx = fmaxf(mx, in ? a : -INFINITY);
        const uint32_t h = hash(id), bit = 1u << (h & 31);
        if (in) twice |= (atomicOr(&sh.seen[h >> 5], bit) & bit) != 0;
      };
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (lane + 32 * u < p.K) take(lane + 32 * u, fid[u], fa[u]);
#pragma unroll 4
      for (int k = lane + 32 * kAhead; k < p.K; k += 32) take(k, __ldg(p.ids + row * p.ids_rs + k), teacher(p, row, k));
      mx = warp_max(mx);
      twice = __any_sync(0xffffffffu, twice);
      float s = 0.f;
      for (int k = lane; k < p.K; k += 32) {
        if (ids[k] < 0) continue;
        s += fast_exp2((pk[k] - mx) * sl2);
        sh.seen[hash(ids[k]) >> 5] = 0;
      }
      s = warp_sum(s);
      const float ls = __log2f(s), inv = 1.f / s;
      float ent = 0.f;
      for (int k = lane; k < p.K; k += 32) {
        const float x = (pk[k] - mx) * sl2, pr = ids[k] >= 0 ? fast_exp2(x) * inv : 0.f;
        pk[k] = pr;
        if (pr != 0.f) ent += pr * (x - ls);
      }
      ent = warp_sum(ent);
      if (lane == 0) {
        sh.twice[slot] = twice;
        sh.entropy[slot] = ent;
      }
      __syncwarp();
    };
    for (int i = lane; i < (1 << (kSeenBits - 5)); i += 32) sh.seen[i] = 0;
    __syncwarp();
    const float t2 = p.temperature * p.temperature, tau = p.temperature;
    double loss = 0.0;  // lane 0: this CTA's part of its rows' losses, in row order
    int r0 = rows.next(zero), r1 = -1;
    if (r0 >= 0) {
      fetch(r0);
      teach(r0, 0);
      r1 = rows.next(zero);
      if (r1 >= 0) fetch(r1);
    }
    for (int it = 0; r0 >= 0 && ok; ++it) {
      const int slot = it & 1;
      const int* ids = id_s + slot * p.K;
      const float *pk = p_s + slot * p.K, *zk = z_s + slot * p.K;
      const float x = lane < kEdge ? sh.edge[slot][lane] : -INFINITY;
      float m = warp_max(x), ls;
      const float m0 = m == -INFINITY ? 0.f : m;
      publish(it, m, warp_sum(lane < kEdge ? fast_exp2((x - m0) * sl2) : 0.f));
      int r2 = -1;
      if (r1 >= 0) {
        teach(r1, slot ^ 1);
        r2 = rows.next(zero);
        if (r2 >= 0) fetch(r2);
      }
      merge(it, m, ls);
      // The row loss tau^2 sum_k p_k (ln p_k - (z_k - max) / tau + ln s): rank 0 has the first and last
      // term and the edges' classes, every CTA adds the classes of its slice
      const T* zr = z + r0 * p.z_rs;
      const int e = edge_of(zr);
      float cross = 0.f;
      if (e >= 0) {
        float P = 0.f;
        for (int k = 0; k < p.K; ++k) P += ids[k] == e ? pk[k] : 0.f;
        if (P != 0.f) cross = P * (x - m);
        if (GRAD) grad[r0 * p.g_rs + e] = from_f<T>(fast_exp2(fmaf(x - m, sl2, lgm - ls)) - P * gmul);
      }
      const int head = head_of(zr), body = (p.V - head) / W;
      const int s0 = head + min(body, rank * NW * p.pv) * W, s1 = head + min(body, (rank + 1) * NW * p.pv) * W;
      if (ok) ok = wwait(smem_u32(&sh.done), it & 1, abort_flag, p.hdr, 61);  // zk is there
      for (int k = lane; k < p.K; k += 32)
        if (ids[k] >= s0 && ids[k] < s1 && pk[k] != 0.f) cross += pk[k] * (zk[k] - m);
      cross = warp_sum(cross);
      if (lane == 0) loss += t2 * ((rank == 0 ? (sh.entropy[slot] + ls) * kLn2 : 0.f) - cross / tau);
      r0 = r1;
      r1 = r2;
    }
    if (lane == 0) p.sums[blockIdx.x] = loss;
  }
  cluster_arrive();  // no CTA leaves while another one may still write into it
  cluster_wait();
  if (*abort_flag) {  // pairs that nobody waited for may be on their way here: nothing is sent any more, let them land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
}

__global__ void __launch_bounds__(kReduceThreads) distill_reduce_kernel(DistillParams p) {
  griddep_begin();
  __shared__ double part[kReduceThreads / 32];
  __shared__ int tot[kReduceThreads / 32];
  double acc = 0.0;  // fixed assignment of rows to CTAs, of those to threads, and a fixed order
  if (p.hdr->status == VA_OK)
    for (int t = threadIdx.x, n = *p.ctas; t < n; t += kReduceThreads) acc += p.sums[t];
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

int count_blocks(int T) { return std::min(kMaxParts, (T + kCountWarps - 1) / kCountWarps); }

template <class T, bool GRAD>
cudaError_t launch_rows_t(const DistillParams& p, int grid, int slots, size_t smem, cudaStream_t st) {
  const auto kernel = distill_rows_kernel<T, GRAD>;
  // The limit is the kernel's, shared by every host thread: always the same, so that no call lowers it
  // between another's setting and launch.  (A call's own size is the launch's.)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((p.NW + 1) * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // Rows are dealt to the clusters beforehand, so all of them have to run at once.  A cluster stays within
  // one of the GPU's SM groups, which leaves fewer than C slots of each unused: a grid near the limit is cut
  // to what fits, and starts on an empty GPU rather than in the gaps that the count kernel leaves
  // (T = 16384, V = 131072 bf16: 110 clusters of four fit, not 114; a second wave made 2010 us out of 1340,
  // by either cause).
  if (p.C > 1 && grid + kSmGroups * p.C > slots) {
    cfg.numAttrs = 1;
    int most = 0;
    e = cudaOccupancyMaxActiveClusters(&most, kernel, &cfg);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(std::min(grid, std::max(1, most) * p.C));
  }
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class T>
cudaError_t launch_rows(const DistillParams& p, int grid, int slots, size_t smem, cudaStream_t st) {
  return p.grad ? launch_rows_t<T, true>(p, grid, slots, smem, st) : launch_rows_t<T, false>(p, grid, slots, smem, st);
}

}  // namespace

// Whether a row of V classes fits the cluster's shared memory.
bool distill_row_fits(int V, int elem) {
  return static_cast<int64_t>(V) * elem <= static_cast<int64_t>(kMaxSlice) * kMaxCluster;
}

size_t distill_parts_bytes() { return (kMaxParts + 2) * sizeof(int32_t) + kMaxCtas * sizeof(double); }

// The three launches of varlen_token_distill, in this order on one stream.
cudaError_t launch_token_distill(int stage, const void* z, int bf16, int64_t z_rs, const int32_t* ids, int64_t ids_rs,
                                 const void* a, int a_bf16, int64_t a_rs, const int32_t* targets, int T, int V, int K,
                                 int ignore, float temperature, void* grad, int64_t g_rs, void* hdr, int32_t* parts,
                                 uint8_t* flags, float* loss, int32_t* count, uint64_t wait_ns, cudaStream_t st) {
  DistillParams p{z, z_rs, ids, ids_rs, a, a_rs, a_bf16, targets, T, V, K, ignore, temperature, grad, g_rs,
                  static_cast<WsHeader*>(hdr), parts, count_blocks(T), flags,
                  reinterpret_cast<double*>(parts + kMaxParts + 2), parts + kMaxParts, loss, count, 0, 1, kMaxWarps,
                  wait_ns};
  if (stage == 0) return launch_pdl(distill_count_kernel, dim3(p.nparts), dim3(32 * kCountWarps), 0, st, p);
  if (stage == 2) return launch_pdl(distill_reduce_kernel, dim3(1), dim3(kReduceThreads), 0, st, p);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t bytes = static_cast<int64_t>(V) * (bf16 ? 2 : 4);
  const auto slice = [&](int C) { return (bytes + C - 1) / C; };
  const size_t fixed = sizeof(DistillSmem) + static_cast<size_t>(K) * 24 + 1024;
  // CTAs per row: the fewest whose slice fits an SM three times, when that is at most five, else twice, else
  // once (us a call, bf16 V = 151936, T = 4096: 456 with five CTAs, 522 with four of 76 KB that fit twice,
  // 596 with eight; fp32 V = 128256, T = 2048: 391 with five that fit twice, 416 with eight that fit three
  // times; fp32 V = 50257, T = 4096: 293 with three, 296 with two that fit twice).  More while the rows alone
  // leave SMs idle.  Working warps: 2 KB of the slice each and more, the more entries the teacher's one warp
  // has to prepare meanwhile (T = 15738, V = 5127, K = 252 bf16 without gradient: 206 us a call, 224 with 2 KB).
  const auto fewest = [&](int per_sm) {
    int C = 1;
    while (C <= kMaxCluster && slice(C) + 16 * kMaxWarps + fixed > kSmemBytes / per_sm) ++C;
    return C;
  };
  p.C = fewest(3);
  if (p.C > 5) p.C = fewest(2);
  if (p.C > kMaxCluster) p.C = fewest(1);  // (distill_row_fits)
  while (2 * p.C <= kMaxCluster && static_cast<int64_t>(T) * p.C * 2 <= sms && slice(p.C) > (8 << 10)) p.C *= 2;
  while (p.NW > 1 && slice(p.C) <= static_cast<int64_t>(p.NW) * (2048 + 16 * K)) p.NW /= 2;
  const int64_t body = bytes / 16;
  p.pv = static_cast<int>((body + p.C * p.NW - 1) / (p.C * p.NW));
  const size_t smem = static_cast<size_t>(p.NW) * p.pv * 16 + fixed - 1024;
  const int per_sm = std::max<int>(1, std::min<int>(27 / (p.NW + 1), kSmemBytes / static_cast<int>(smem + 1024)));
  const int clusters = std::max(1, std::min(std::min(T, kMaxCtas / p.C), sms * per_sm / p.C));
  const int grid = clusters * p.C, slots = sms * per_sm;
  return bf16 ? launch_rows<__nv_bfloat16>(p, grid, slots, smem, st) : launch_rows<float>(p, grid, slots, smem, st);
}

}  // namespace va
