// Log probabilities of given tokens with the distribution's entropy and its top alternatives, and their gradient
// with respect to the logits.  Row t, p = softmax(z / tau):
//
//   lse = ln sum exp(z / tau),  logprob = z_y / tau - lse,  H = -sum p ln p = ln s - w / s
// with s = sum e, w = sum e u, e = exp(u), u = (z - m) / tau for a reference m near the row's maximum.
//   dz_c = (dl ([c == y] - p_c) - dH p_c (ln p_c + H)) / tau
//
// Forward: one read of the row.  A thread's part gives (m, s, w), its reference moved only when a value passes it by
// 2^8, so the sums are hardly ever rescaled; differences are formed before the scale, so a row of the type's
// lowest value stays finite.  With alternatives a thread also keeps the largest logit of its part: the k-th largest of
// these is a lower bound of the row's k-th largest logit, and only the few parts that reach it are looked at again
// (in L2).  Candidates are ordered as whole numbers, value first, then the lower id, and ranked by counting.  A row
// with too many candidates (equal logits, mostly) has its k-th value found bit by bit instead.
//
// Backward: p from the saved lse, one read, one write.  What an lse has lost by its rounding to fp32 is p's relative
// error, half its last bit: 2^-20 below 32, which is what fp32 gradients keep, 2^-17 below 256, which bf16 ones do not
// see; the sums of a row whose lse is larger are formed again.
#include <algorithm>

#include "elem.cuh"
#include "logprobs.cuh"

namespace va {

namespace {

constexpr float kLog2eLo = static_cast<float>(1.4426950408889634 - static_cast<double>(kLog2e));

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kU = 4;          // 16-byte pieces a thread has in flight
constexpr int kCtasPerSm = 4;  // resident at once (launch bounds)
constexpr int kCand = 1024;    // candidates a row may have before it takes the slow way

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Whole numbers in the order of the values (-0 as 0, NaN above all).
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); }

// Sums relative to m, in powers of two: s = sum 2^t, w = sum 2^t t, t = (z - m) scale.
struct Sums {
  float m, s, w;
};

// u = (z - m) scale no smaller than -200, where 2^u is 0 anyway (0 times -inf would be NaN).
__device__ __forceinline__ float shifted(float z, float m, float scale) { return max_nan((z - m) * scale, -200.f); }

__device__ __forceinline__ void rescale(Sums& a, float m, float scale) {  // m >= a.m
  if (a.m == -INFINITY) {
    a.m = m;
    return;
  }
  const float d = shifted(a.m, m, scale), f = fast_exp2(d);
  a.w = f * fmaf(a.s, d, a.w);
  a.s *= f;
  a.m = m;
}

__device__ __forceinline__ void merge(Sums& a, Sums b, float scale) {
  const float m = fmaxf(a.m, b.m);
  if (m > a.m) rescale(a, m, scale);
  if (m > b.m) rescale(b, m, scale);
  a.s += b.s;
  a.w += b.w;
}

// Adds N values whose largest (NaN left out) is cm.
template <int N>
__device__ __forceinline__ void add(Sums& a, const float (&x)[N], float cm, float scale, float slack) {
  if (cm > a.m + slack) rescale(a, cm, scale);
  const float m = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = shifted(x[i], m, scale), e = fast_exp2(t);
    a.s += e;
    a.w = fmaf(e, t, a.w);
  }
}

template <class T> struct Row { static constexpr int W = 16 / sizeof(T); };

template <class T, class F>
__device__ __forceinline__ void each_piece(const T* z, int Vv, F&& f) {
  constexpr int W = Row<T>::W, step = kThreads * W;
  for (int c0 = threadIdx.x * W; c0 < Vv; c0 += kU * step) {
    Pack<T, W> raw[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (c0 + u * step < Vv) raw[u] = load_pack<T, W>(z + c0 + u * step);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (c0 + u * step >= Vv) continue;
      float x[W];
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = raw[u][i];
      f(c0 + u * step, x);
    }
  }
}

struct RowSmem {
  Sums warp[kWarps];
  uint32_t part_max[kThreads];       // largest logit of every thread's part
  unsigned long long cand[kCand];    // value, then ~id
  int count;
  int total[kWarps];
};

// A row's sums, the same in every thread; gm: the largest logit of this thread's part.
template <class T>
__device__ __forceinline__ Sums row_sums(const T* z, int V, int Vv, float scale, RowSmem& sh, float& gm) {
  constexpr int W = Row<T>::W;
  Sums a{-INFINITY, 0.f, 0.f};
  const float slack = 8.f / scale;
  gm = -INFINITY;
  each_piece(z, Vv, [&](int, const float (&x)[W]) {
    float cm = x[0];
#pragma unroll
    for (int i = 1; i < W; ++i) cm = fmaxf(cm, x[i]);
    gm = fmaxf(gm, cm);
    add(a, x, cm, scale, slack);
  });
  for (int c = Vv + threadIdx.x; c < V; c += kThreads) {
    const float x[1] = {elem_f(z[c])};
    gm = fmaxf(gm, x[0]);
    add(a, x, x[0], scale, slack);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.w = __shfl_xor_sync(0xffffffffu, a.w, o);
    merge(a, b, scale);
  }
  if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = a;
  __syncthreads();
  a = sh.warp[0];
  for (int w = 1; w < kWarps; ++w) merge(a, sh.warp[w], scale);
  return a;
}

__device__ __forceinline__ int block_sum(int n, RowSmem& sh) {
  n = __reduce_add_sync(0xffffffffu, n);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.total[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < kWarps; ++w) n += sh.total[w];
  return n;
}

__device__ __forceinline__ void put(RowSmem& sh, uint32_t o, int id) {
  const int at = atomicAdd(&sh.count, 1);
  if (at < kCand) sh.cand[at] = static_cast<unsigned long long>(o) << 32 | ~static_cast<uint32_t>(id);
}

// The slow way: the k-th largest value bit by bit, then all above it and the first ids that have it.
template <class T>
__device__ void exact_candidates(const T* z, int V, int k, RowSmem& sh) {
  uint32_t kth = 0;  // the largest value that at least k logits reach
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t t = kth | 1u << bit;
    int n = 0;
    for (int c = threadIdx.x; c < V; c += kThreads) n += order_of(elem_f(z[c])) >= t;
    if (block_sum(n, sh) >= k) kth = t;
  }
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  for (int c = threadIdx.x; c < V; c += kThreads) {
    const uint32_t o = order_of(elem_f(z[c]));
    if (o > kth) put(sh, o, c);  // fewer than k
  }
  __syncthreads();
  int left = k - sh.count;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int c0 = 0; c0 < V && left > 0; c0 += kThreads) {  // in the order of ids
    const int c = c0 + threadIdx.x;
    const bool is = c < V && order_of(elem_f(z[c])) == kth;
    const uint32_t who = __ballot_sync(0xffffffffu, is);
    if (lane == 0) sh.total[warp] = __popc(who);
    __syncthreads();
    int before = __popc(who & ((1u << lane) - 1)), all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.total[w];
      all += sh.total[w];
    }
    if (is && before < left) put(sh, kth, c);
    left -= all;
    __syncthreads();
  }
}

// The k largest logits with their ids, ranked, as (value, ~id) in sh.cand; returns how many candidates there are.
template <class T>
__device__ __forceinline__ int top_candidates(const T* z, int V, int Vv, int k, float gm, RowSmem& sh) {
  constexpr int W = Row<T>::W;
  const uint32_t mine = order_of(gm);
  sh.part_max[threadIdx.x] = mine;
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  // the k-th largest of the parts' maxima: whoever has fewer than k above it and reaches k with its equals
  int above = 0, equal = 0;
  for (int i = 0; i < kThreads; ++i) {
    above += sh.part_max[i] > mine;
    equal += sh.part_max[i] == mine;
  }
  if (above < k && above + equal >= k) sh.total[0] = static_cast<int>(mine);  // (all that do write the same)
  __syncthreads();
  const uint32_t bound = static_cast<uint32_t>(sh.total[0]);
  if (mine >= bound) {
    for (int c0 = threadIdx.x * W; c0 < Vv; c0 += kThreads * W) {
      const Pack<T, W> raw = load_pack<T, W>(z + c0);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t o = order_of(raw[i]);
        if (o >= bound) put(sh, o, c0 + i);
      }
    }
    for (int c = Vv + threadIdx.x; c < V; c += kThreads) {
      const uint32_t o = order_of(elem_f(z[c]));
      if (o >= bound) put(sh, o, c);
    }
  }
  __syncthreads();
  if (sh.count > kCand) {
    __syncthreads();
    exact_candidates(z, V, k, sh);
    __syncthreads();
  }
  return min(sh.count, kCand);
}

}  // namespace

template <class T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logprobs_fwd_kernel(const LogprobParams p) {
  griddep_begin();
  __shared__ RowSmem sh;
  constexpr int W = Row<T>::W;
  const int Vv = p.vec ? p.V / W * W : 0;
  for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int y = p.tok[row];
    if (y == p.ignore) {  // no arithmetic on its logits
      if (threadIdx.x == 0) p.logprob[row] = p.entropy[row] = p.lse[row] = 0.f;
      for (int i = threadIdx.x; i < p.k; i += kThreads) {
        p.top_ids[static_cast<int64_t>(row) * p.k + i] = -1;
        p.top_logprobs[static_cast<int64_t>(row) * p.k + i] = 0.f;
      }
      continue;
    }
    const T* z = static_cast<const T*>(p.z) + row * p.z_rs;
    float gm;
    const Sums a = row_sums(z, p.V, Vv, p.scale, sh, gm);
    const float m = a.m == -INFINITY ? 0.f : a.m, l2 = __log2f(a.s);
    if (threadIdx.x == 0) {
      const bool ok = y >= 0 && y < p.V;
      if (!ok && p.status) *p.status = VA_ERR_BAD_TARGETS;
      p.logprob[row] = ok ? fmaf(elem_f(z[y]) - m, p.inv_t, -l2 * kLn2) : NAN;
      p.entropy[row] = (l2 - a.w / a.s) * kLn2;
      p.lse[row] = static_cast<float>(static_cast<double>(m) / p.temperature + static_cast<double>(l2) * 0.69314718055994531);
    }
    if (p.k > 0) {
      const int n = top_candidates(z, p.V, Vv, p.k, gm, sh);
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long c = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > c;
        if (rank < p.k) {
          p.top_ids[static_cast<int64_t>(row) * p.k + rank] = static_cast<int32_t>(~static_cast<uint32_t>(c));
          p.top_logprobs[static_cast<int64_t>(row) * p.k + rank] =
              fmaf(value_of(static_cast<uint32_t>(c >> 32)) - m, p.inv_t, -l2 * kLn2);
        }
      }
    }
    __syncthreads();
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logprobs_bwd_kernel(const LogprobParams p) {
  griddep_begin();
  __shared__ RowSmem sh;
  constexpr int W = Row<T>::W;
  const int Vv = p.vec ? p.V / W * W : 0;
  for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int y = p.tok[row];
    T* gr = static_cast<T*>(p.grad) + row * p.g_rs;
    if (y == p.ignore) {
      Pack<T, W> zero;
#pragma unroll
      for (int i = 0; i < W; ++i) zero.set(i, 0.f);
      for (int c = threadIdx.x * W; c < Vv; c += kThreads * W) store_pack_cs(gr + c, zero);
      for (int c = Vv + threadIdx.x; c < p.V; c += kThreads) gr[c] = elem_of<T>(0.f);
      continue;
    }
    const T* z = static_cast<const T*>(p.z) + row * p.z_rs;
    // log2 p = (z - m) scale - l2, with m = 0 where lse is precise enough; then the products' low halves count in fp32
    const float lse = p.lse[row];
    float m = 0.f, l2 = lse * kLog2e, l2_lo = fmaf(lse, kLog2e, -l2) + lse * kLog2eLo, scale_lo = p.scale_lo;
    if (!(fabsf(lse) <= (sizeof(T) == 2 ? 256.f : 32.f))) {
      float gm;
      const Sums a = row_sums(z, p.V, Vv, p.scale, sh, gm);
      m = a.m == -INFINITY ? 0.f : a.m;
      l2 = __log2f(a.s);
      l2_lo = scale_lo = 0.f;
      __syncthreads();  // the whole row is read before any of it is written: grad may be the logits
    }
    const bool ok = y >= 0 && y < p.V;
    const float dl = ok ? p.dlogprob[row] * p.inv_t : NAN, dh = p.dentropy ? p.dentropy[row] * p.inv_t : 0.f;
    // dz = p (c1 + c2 log2 p) + [c == y] dl
    const float c1 = -fmaf(dh, p.dentropy ? p.entropy[row] : 0.f, dl), c2 = -dh * kLn2;
    const auto one = [&](float x, int c) {
      const float u = sizeof(T) == 4 ? max_nan(x - m, -1e30f) : x - m;  // (-inf times the low half would be NaN)
      float t = fmaf(u, p.scale, -l2);
      if (sizeof(T) == 4) t += fmaf(u, scale_lo, -l2_lo);
      t = max_nan(t, -200.f);
      const float v = fast_exp2(t) * fmaf(c2, t, c1);
      return c == y ? v + dl : v;
    };
    each_piece(z, Vv, [&](int c0, const float (&x)[W]) {
      Pack<T, W> o;
#pragma unroll
      for (int i = 0; i < W; ++i) o.set(i, one(x[i], c0 + i));
      store_pack_cs(gr + c0, o);
    });
    for (int c = Vv + threadIdx.x; c < p.V; c += kThreads) gr[c] = elem_of<T>(one(elem_f(z[c]), c));
  }
}

// ---------------------------------------------------------------- host side

namespace {

int row_ctas(int T) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return static_cast<int>(std::min<int64_t>(T, static_cast<int64_t>(std::max(sms, 1)) * kCtasPerSm));
}

bool rows16(const void* p, int64_t rs, int es) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && rs * es % 16 == 0; }

}  // namespace

cudaError_t launch_logprobs_fwd(LogprobParams p, int bf16, cudaStream_t st) {
  p.vec = rows16(p.z, p.z_rs, bf16 ? 2 : 4);
  const dim3 grid(row_ctas(p.T));
  return bf16 ? launch_pdl(logprobs_fwd_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, p)
              : launch_pdl(logprobs_fwd_kernel<float>, grid, dim3(kThreads), 0, st, p);
}

cudaError_t launch_logprobs_bwd(LogprobParams p, int bf16, cudaStream_t st) {
  p.vec = rows16(p.z, p.z_rs, bf16 ? 2 : 4) && rows16(p.grad, p.g_rs, bf16 ? 2 : 4);
  const dim3 grid(row_ctas(p.T));
  return bf16 ? launch_pdl(logprobs_bwd_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, p)
              : launch_pdl(logprobs_bwd_kernel<float>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace va
