// Log probabilities of given tokens with the distribution's entropy and its top alternatives, and their gradient
// with respect to the logits.  Row t, p = softmax(z / tau):
//
//   lse = ln sum exp(z / tau),  logprob = z_y / tau - lse,  H = -sum p ln p
//   dz_c = (dl ([c == y] - p_c) - dH p_c (ln p_c + H)) / tau
//
// Forward: one read of the row, in powers of two: with c = log2(e) / tau and a reference r,
//   s = sum 2^t, w = sum 2^t t, t = c z - r;   log2 p = t - log2 s,  H = ln 2 (log2 s - w / s).
// A thread moves its reference only when a value passes it by 2^8, so its sums are hardly ever rescaled.  t is one
// multiply-add: r's rounding drops out of p, as every t has it; c's does not (p is that of a temperature off by it, 2^-25
// relative at most: the error of ln p is that share of the distance to r).  r's rounding, half a step of c z, has to stay
// small for 2^t, though: references begin at -2^24, and rows whose reference ends at +-2^24 or beyond (or is no number) have
// their sums formed again from differences to the maximum; so rows of one large value, or of the type's lowest, come out
// right, and so do ordinary rows with such values in masked places.  Logits far below the reference are raised to
// where 2^t is 0 anyway (0 times -inf would be NaN), NaN is kept.
//
// A block reads its rows through a ring of kDepth groups of kU 16-byte pieces a thread, copied asynchronously: a
// thread's pieces are its own, so nothing waits for the block, and the next row is on its way while this one's
// sums are joined and its alternatives are looked for.
//
// Alternatives: each thread keeps the largest logit of its part; the k-th largest of the parts' maxima (cut to 16 bits)
// is a lower bound of the row's k-th largest logit, and only threads whose part reaches it look at it again (in L2).
// Candidates are ordered as whole numbers, value first, then the lower id, and ranked by counting.  A row
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

constexpr int kU = 4;          // 16-byte pieces of a group
constexpr int kDepth = 3;      // groups a thread has on their way
constexpr int kCand = 256;     // candidates a row may have before it takes the slow way
constexpr float kFar = 16777216.f;  // references beyond this (c z, where half a step is 1): differences before products

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of two bf16 pairs, NaN left out
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float low_f(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float high_f(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// Whole numbers in the order of the values (-0 as 0, NaN above all).
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); }

// s = sum 2^t and w = sum 2^t t, t = c z - r, in two halves.
struct Sums {
  float r, s[2], w[2];
};

__device__ __forceinline__ void move_to(Sums& a, float r) {  // r >= a.r
  const float d = fmaxf(a.r - r, -200.f), f = fast_exp2(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a.w[i] = f * fmaf(a.s[i], d, a.w[i]);
    a.s[i] *= f;
  }
  a.r = r;
}

__device__ __forceinline__ void add2(Sums& a, float x0, float x1, float c) {
  float t0, t1;
  ffma2(t0, t1, x0, x1, c, c, -a.r, -a.r);
  const float e0 = fast_exp2(t0), e1 = fast_exp2(t1);
  fadd2(a.s[0], a.s[1], a.s[0], a.s[1], e0, e1);
  ffma2(a.w[0], a.w[1], e0, e1, t0, t1, a.w[0], a.w[1]);
}

// The largest logit of a piece (NaN left out).
template <class T>
__device__ __forceinline__ float largest(const uint4& raw) {
  if (sizeof(T) == 2) {
    const uint32_t m = max2(max2(raw.x, raw.y), max2(raw.z, raw.w));
    return fmaxf(low_f(m), high_f(m));
  }
  return fmaxf(fmaxf(__uint_as_float(raw.x), __uint_as_float(raw.y)), fmaxf(__uint_as_float(raw.z), __uint_as_float(raw.w)));
}

template <class T>
__device__ __forceinline__ uint4 larger(const uint4& a, const uint4& b) {
  const auto one = [](uint32_t x, uint32_t y) {
    return sizeof(T) == 2 ? max2(x, y) : __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
  };
  return make_uint4(one(a.x, b.x), one(a.y, b.y), one(a.z, b.z), one(a.w, b.w));
}

// What a thread has seen of a row.
template <class T>
struct Part {
  static constexpr int W = 16 / sizeof(T);
  Sums a;
  float top;       // the largest logit (NaN left out)
  uint32_t floor;  // logits are raised to this: bf16 a pair, fp32 its bits

  __device__ __forceinline__ void start(float c) {
    a.r = -kFar;
    a.s[0] = a.s[1] = a.w[0] = a.w[1] = 0.f;
    top = -INFINITY;
    set_floor(-(1.015625f * kFar + 200.f) / c);
  }
  __device__ __forceinline__ void set_floor(float x) {
    if (sizeof(T) == 2) floor = pack_bf16(x, x);
    else floor = __float_as_uint(x);
  }
  __device__ __forceinline__ void see(float m, float c) {  // m: the largest of what comes next
    top = fmaxf(top, m);
    if (m * c > a.r + 8.f) {
      move_to(a, m * c);
      set_floor(m - 200.f / c - fabsf(m) * 0.015625f);
    }
  }
  __device__ __forceinline__ void add(const uint4 (&raw)[kU], float c) {
    uint4 m = raw[0];
#pragma unroll
    for (int u = 1; u < kU; ++u) m = larger<T>(m, raw[u]);
    see(largest<T>(m), c);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      if (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = max2_nan(w[i], floor);
          add2(a, low_f(x), high_f(x), c);
        }
      } else {
        const float lo = __uint_as_float(floor);
#pragma unroll
        for (int i = 0; i < 4; i += 2)
          add2(a, max_nan(__uint_as_float(w[i]), lo), max_nan(__uint_as_float(w[i + 1]), lo), c);
      }
    }
  }
  __device__ __forceinline__ void add(T z, float c) {  // one logit
    const float x = elem_f(z);
    see(x, c);
    const float lo = sizeof(T) == 2 ? low_f(floor) : __uint_as_float(floor);
    const float t = fmaf(max_nan(x, lo), c, -a.r), e = fast_exp2(t);
    a.s[0] += e;
    a.w[0] = fmaf(e, t, a.w[0]);
  }
};

// How a row lies in memory: `head` elements up to its first 16-byte boundary, `body` pieces, `tail` elements.
template <class T>
struct Cut {
  static constexpr int W = 16 / sizeof(T);
  int head, body, tail;
  __device__ __forceinline__ Cut(const T* z, int V) {
    const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z) & 15u);
    head = min(V, static_cast<int>(((16u - mis) & 15u) / sizeof(T)));
    body = (V - head) / W;
    tail = V - head - body * W;
  }
  __device__ __forceinline__ int edge(int i) const { return i < head ? i : i + body * W; }  // i < head + tail
};

// What a block's warps share of a row.  A block has two of them and takes them in turn: the first barrier of a row
// comes after every warp is done with the row before the last.
template <int NT>
struct RowSmem {
  unsigned long long cand[kCand];  // value, then ~id
  float sums[3][NT / 32];          // the warps' (r, s, w)
  uint32_t part[256];              // the parts' largest logits
  int total[NT / 32];
  uint8_t list[NT / 32][32];       // a warp's threads whose part is looked at again
  int count;
};

template <int NT>
__device__ __forceinline__ void block_sync() {
  if (NT == 32) __syncwarp();
  else __syncthreads();
}

__device__ __forceinline__ float warp_max(float x) {  // one instruction on whole numbers; no NaN comes here
  return value_of(__reduce_max_sync(0xffffffffu, order_of(x)));
}
template <int N>
__device__ __forceinline__ float warp_sum(float x) {  // over N lanes that follow one another
#pragma unroll
  for (int o = N >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A row's sums: log2 p = t - l, t = c z - r; mean_t = sum p t.
struct RowSums {
  float r, l, mean_t;
};

// The block's sums, the same in every thread.
template <int NT>
__device__ __forceinline__ RowSums join(Sums a, RowSmem<NT>& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float r = warp_max(a.r);
  move_to(a, r);
  float s = warp_sum<32>(a.s[0] + a.s[1]), w = warp_sum<32>(a.w[0] + a.w[1]);
  if (NT > 32) {
    if (lane == 0) {
      sh.sums[0][warp] = r;
      sh.sums[1][warp] = s;
      sh.sums[2][warp] = w;
    }
    __syncthreads();
    constexpr int N = NT / 32;
    Sums b;
    b.r = sh.sums[0][lane % N];
    b.s[0] = sh.sums[1][lane % N];
    b.w[0] = sh.sums[2][lane % N];
    b.s[1] = b.w[1] = 0.f;
    r = warp_max(b.r);
    move_to(b, r);
    s = warp_sum<N>(b.s[0]);
    w = warp_sum<N>(b.w[0]);
  }
  return RowSums{r, __log2f(s), w / s};
}

// A row's sums again, from differences to its maximum: r = c m, t = (z - m) c.
template <class T, int NT>
__device__ RowSums far_sums(const T* z, int V, float c, RowSmem<NT>& sh, float& m) {
  float top = -INFINITY;
  for (int i = threadIdx.x; i < V; i += NT) top = fmaxf(top, elem_f(z[i]));
  block_sync<NT>();
  const float r0 = join(Sums{top, {0.f, 0.f}, {0.f, 0.f}}, sh).r;
  m = r0 == -INFINITY ? 0.f : r0;
  Sums a{0.f, {0.f, 0.f}, {0.f, 0.f}};
  for (int i = threadIdx.x; i < V; i += NT) {
    const float t = max_nan((elem_f(z[i]) - m) * c, -200.f), e = fast_exp2(t);
    a.s[0] += e;
    a.w[0] = fmaf(e, t, a.w[0]);
  }
  block_sync<NT>();
  RowSums q = join(a, sh);
  q.r = 0.f;
  return q;
}

template <int NT>
__device__ __forceinline__ int block_sum(int n, RowSmem<NT>& sh) {
  n = __reduce_add_sync(0xffffffffu, n);
  if (NT == 32) return n;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.total[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < NT / 32; ++w) n += sh.total[w];
  return n;
}

template <int NT>
__device__ __forceinline__ void put(RowSmem<NT>& sh, uint32_t o, int id) {
  const int at = atomicAdd(&sh.count, 1);
  if (at < kCand) sh.cand[at] = static_cast<unsigned long long>(o) << 32 | ~static_cast<uint32_t>(id);
}

// The slow way: the k-th largest value bit by bit, then all above it and the first ids that have it.
template <class T, int NT>
__device__ __noinline__ void exact_candidates(const T* z, int V, int k, RowSmem<NT>& sh) {
  constexpr int kShift = sizeof(T) == 2 ? 16 : 0;  // (a bf16's order is in the upper half)
  const auto key = [&](int c) { return order_of(elem_f(z[c])) >> kShift; };
  uint32_t kth = 0;  // the largest value that at least k logits reach
  for (int bit = 31 - kShift; bit >= 0; --bit) {
    const uint32_t t = kth | 1u << bit;
    int n = 0;
    for (int c = threadIdx.x; c < V; c += NT) n += key(c) >= t;
    if (block_sum(n, sh) >= k) kth = t;
  }
  if (threadIdx.x == 0) sh.count = 0;
  block_sync<NT>();
  for (int c = threadIdx.x; c < V; c += NT)
    if (key(c) > kth) put(sh, order_of(elem_f(z[c])), c);  // fewer than k
  block_sync<NT>();
  int left = k - sh.count;
  block_sync<NT>();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int c0 = 0; c0 < V && left > 0; c0 += NT) {  // in the order of ids
    const int c = c0 + threadIdx.x;
    const bool is = c < V && key(c) == kth;
    const uint32_t who = __ballot_sync(0xffffffffu, is);
    if (lane == 0) sh.total[warp] = __popc(who);
    block_sync<NT>();
    int before = __popc(who & ((1u << lane) - 1)), all = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += sh.total[w];
      all += sh.total[w];
    }
    if (is && before < left) put(sh, order_of(elem_f(z[c])), c);
    left -= all;
    block_sync<NT>();
  }
}

// The k-th largest of 32 N numbers, N a lane, by its upper 16 bits, two at a time: what is returned is at most it.
template <int N>
__device__ __forceinline__ uint32_t kth_of(const uint32_t (&v)[N], int k) {
  uint32_t kth = 0;
#pragma unroll
  for (int bit = 30; bit >= 16; bit -= 2) {
    int n[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 3; ++j) n[j] += __popc(__ballot_sync(0xffffffffu, v[i] >= (kth | (j + 1u) << bit)));
    kth |= static_cast<uint32_t>((n[0] >= k) + (n[1] >= k) + (n[2] >= k)) << bit;
  }
  return kth;
}

// The parts of a row: up to 16 alternatives are bounded by the maxima of 32 parts, more by those of 128 or 256 (the
// more, the closer, but the search for the k-th takes a vote for each 32 of them and bit); a short row's pieces lie
// with as many threads.
template <int NT>
__device__ __forceinline__ int part_words(int k, int body) {
  return NT == 32 || (k <= 16 && body >= NT) ? 1 : NT >= 128 && k <= 64 && body >= NT ? 4 : NT < 256 ? NT / 32 : 8;
}

// Written before the barrier of the row's sums.
template <int NT>
__device__ __forceinline__ void put_part(uint32_t mine, int words, RowSmem<NT>& sh) {
  const int per = NT / (32 * words);
  for (int o = per >> 1; o > 0; o >>= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, o));
  if (threadIdx.x % per == 0) sh.part[threadIdx.x / per] = mine;
}
template <int NT, int N>
__device__ __forceinline__ uint32_t part_bound(int k, const RowSmem<NT>& sh) {
  uint32_t v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = sh.part[32 * i + (threadIdx.x & 31)];
  return kth_of(v, k);
}

// The k largest logits with their ids, and maybe others, as (value, ~id) in sh.cand; returns how many.
template <class T, int NT>
__device__ __forceinline__ int top_candidates(const T* z, int V, const Cut<T>& cut, int k, uint32_t mine, int words,
                                              RowSmem<NT>& sh) {
  constexpr int W = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  uint32_t bound;
  if (NT == 32) {
    const uint32_t v[1] = {mine};
    bound = kth_of(v, k);  // (k <= 32: see pick_fwd)
  } else {
    bound = words == 1 ? part_bound<NT, 1>(k, sh) : words == 4 ? part_bound<NT, 4>(k, sh) : part_bound<NT, 8>(k, sh);
  }
  // a warp's lanes share the pieces of those of its threads whose part reaches the bound
  const float least = bound < order_of(-INFINITY) ? -INFINITY : value_of(bound);
  const auto look = [&](float x, int c) {
    const uint32_t o = order_of(x);
    if (o >= bound) put(sh, o, c);
  };
  const uint32_t who = __ballot_sync(0xffffffffu, mine >= bound);
  uint8_t* list = sh.list[threadIdx.x >> 5];
  if (mine >= bound) list[__popc(who & ((1u << lane) - 1))] = static_cast<uint8_t>(lane);
  __syncwarp();
  const int per = (cut.body + NT - 1) / NT, n = __popc(who) * per;
#pragma unroll 2
  for (int w = lane; w < n; w += 32) {
    const int j = w / per, i = (threadIdx.x & ~31) + list[j] + (w - j * per) * NT;
    if (i >= cut.body) continue;
    const Pack<T, W> raw = load_pack<T, W>(z + cut.head + i * W);
    if (largest<T>(*reinterpret_cast<const uint4*>(&raw)) < least) continue;  // (all NaN: looked at)
#pragma unroll
    for (int e = 0; e < W; ++e) look(raw[e], cut.head + i * W + e);
  }
  if (mine >= bound && threadIdx.x < cut.head + cut.tail) look(elem_f(z[cut.edge(threadIdx.x)]), cut.edge(threadIdx.x));
  block_sync<NT>();
  if (sh.count > kCand) {
    block_sync<NT>();
    exact_candidates(z, V, k, sh);
    block_sync<NT>();
  }
  return min(sh.count, kCand);
}

// The next row at or after `row` (of this block's) that has a token.
__device__ __forceinline__ int next_row(const LogprobParams& p, int row) {
  while (row < p.T && p.tok[row] == p.ignore) row += gridDim.x;
  return min(row, p.T);
}

template <int NT> constexpr int ctas_per_sm() { return NT == 32 ? 20 : NT == 128 ? 7 : NT == 256 ? 4 : 2; }

}  // namespace

// NT: threads of a block (see pick_fwd).
template <class T, int NT>
__global__ void __launch_bounds__(NT, ctas_per_sm<NT>()) logprobs_fwd_kernel(const LogprobParams p) {
  griddep_begin();
  extern __shared__ __align__(16) uint8_t smem[];
  uint4 (*ring)[kU][NT] = reinterpret_cast<uint4 (*)[kU][NT]>(smem);
  RowSmem<NT>* const shared = reinterpret_cast<RowSmem<NT>*>(smem + sizeof(uint4) * kDepth * kU * NT);
  const int tid = threadIdx.x;
  const float c = p.scale;
  const T* z0 = static_cast<const T*>(p.z);
  // the groups on their way: group ig of row irow comes next
  const int groups = max(1, (p.V / Part<T>::W + kU * NT - 1) / (kU * NT));
  int irow = next_row(p, blockIdx.x), ig = 0, ileft = 0;
  const uint4* from = nullptr;
  const auto issue = [&](int slot) {
    if (irow < p.T) {
      if (ig == 0) {
        const T* z = z0 + irow * p.z_rs;
        const Cut<T> cut(z, p.V);
        ileft = cut.body - tid;
        from = reinterpret_cast<const uint4*>(z + cut.head) + tid;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (u * NT < ileft) copy16(&ring[slot][u][tid], from + u * NT);
      ileft -= kU * NT;
      from += kU * NT;
      if (++ig == groups) {
        ig = 0;
        irow = next_row(p, irow + gridDim.x);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) issue(d);
  int slot = 0, fill = kDepth - 1;  // read next, written next
  int turn = 0;
  if (tid == 0) shared[0].count = 0;
  for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int y = p.tok[row];
    if (y == p.ignore) {  // no arithmetic on its logits
      if (tid == 0) p.logprob[row] = p.entropy[row] = p.lse[row] = 0.f;
      for (int i = tid; i < p.k; i += NT) {
        p.top_ids[static_cast<int64_t>(row) * p.k + i] = -1;
        p.top_logprobs[static_cast<int64_t>(row) * p.k + i] = 0.f;
      }
      continue;
    }
    const T* z = z0 + row * p.z_rs;
    const Cut<T> cut(z, p.V);
    const bool ok = y >= 0 && y < p.V;
    const float zy = tid == 0 && ok ? elem_f(z[y]) : 0.f;
    Part<T> part;
    part.start(c);
    if (tid < cut.head + cut.tail) part.add(z[cut.edge(tid)], c);
    for (int g = 0; g < groups; ++g) {
      issue(fill);
      copy_wait<kDepth - 1>();
      uint4 raw[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) raw[u] = ring[slot][u][tid];
      if ((g + 1) * kU * NT > cut.body) {  // a group that is not whole
        constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if ((g * kU + u) * NT + tid >= cut.body) raw[u] = make_uint4(none, none, none, none);
      }
      part.add(raw, c);
      slot = slot + 1 == kDepth ? 0 : slot + 1;
      fill = fill + 1 == kDepth ? 0 : fill + 1;
    }
    RowSmem<NT>& sh = shared[turn];
    turn ^= 1;
    const uint32_t mine = order_of(part.top);
    const int words = part_words<NT>(p.k, p.V / Part<T>::W - 1);
    if (NT > 32 && p.k > 0) put_part(mine, words, sh);
    RowSums q = join(part.a, sh);
    if (tid == 0) shared[turn].count = 0;  // (behind the barrier: nobody is at the row before any more)
    // ln p = (z - m) / tau - l, m near the largest logit
    float m = q.r * p.inv_c, l2 = q.l - fmaf(m, c, -q.r);
    if (!(fabsf(q.r) < kFar)) {
      q = far_sums(z, p.V, c, sh, m);
      l2 = q.l;
    }
    const float l = l2 * kLn2;
    if (tid == 0) {
      if (!ok && p.status) *p.status = VA_ERR_BAD_TARGETS;
      p.logprob[row] = ok ? fmaf(zy - m, p.inv_t, -l) : NAN;
      p.entropy[row] = (q.l - q.mean_t) * kLn2;
      p.lse[row] = static_cast<float>(static_cast<double>(m) / p.temperature + static_cast<double>(l2) * 0.69314718055994531);
    }
    if (p.k > 0) {
      const int n = top_candidates(z, p.V, cut, p.k, mine, words, sh);
      for (int i = tid; i < n; i += NT) {
        const unsigned long long v = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > v;
        if (rank < p.k) {
          p.top_ids[static_cast<int64_t>(row) * p.k + rank] = static_cast<int32_t>(~static_cast<uint32_t>(v));
          p.top_logprobs[static_cast<int64_t>(row) * p.k + rank] =
              fmaf(value_of(static_cast<uint32_t>(v >> 32)) - m, p.inv_t, -l);
        }
      }
      if (NT == 32) __syncwarp();
    }
  }
}

// Blocks share a row's `slices` (one where the gradient lies on the logits: a row's sums may be formed again).
template <class T, int NT>
__global__ void __launch_bounds__(NT, NT == 32 ? 24 : 4) logprobs_bwd_kernel(const LogprobParams p) {
  griddep_begin();
  __shared__ RowSmem<NT> sh;
  constexpr int W = 16 / sizeof(T);
  const int tid = threadIdx.x;
  const int64_t items = static_cast<int64_t>(p.T) * p.slices;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int row = static_cast<int>(item / p.slices), slice = static_cast<int>(item % p.slices);
    const int y = p.tok[row];
    const T* z = static_cast<const T*>(p.z) + row * p.z_rs;
    T* gr = static_cast<T*>(p.grad) + row * p.g_rs;
    Cut<T> cut(gr, p.V);
    const bool same = ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(gr)) & 15u) == 0;
    const int i0 = static_cast<int>(static_cast<int64_t>(cut.body) * slice / p.slices);
    const int i1 = static_cast<int>(static_cast<int64_t>(cut.body) * (slice + 1) / p.slices);
    const bool edges = slice == 0 && tid < cut.head + cut.tail;
    if (y == p.ignore) {
      Pack<T, W> zero;
#pragma unroll
      for (int i = 0; i < W; ++i) zero.set(i, 0.f);
      for (int i = i0 + tid; i < i1; i += NT) store_pack_cs(gr + cut.head + i * W, zero);
      if (edges) gr[cut.edge(tid)] = elem_of<T>(0.f);
      continue;
    }
    // log2 p = (z - m) c - l2, with m = 0 where lse is precise enough; then the products' low halves count in fp32
    const float lse = p.lse[row];
    float m = 0.f, l2 = lse * kLog2e, l2_lo = fmaf(lse, kLog2e, -l2) + lse * kLog2eLo, c_lo = p.scale_lo;
    if (!(fabsf(lse) <= (sizeof(T) == 2 ? 256.f : 32.f))) {
      l2 = far_sums(z, p.V, p.scale, sh, m).l;
      l2_lo = c_lo = 0.f;
      block_sync<NT>();  // the whole row is read before any of it is written
    }
    const bool ok = y >= 0 && y < p.V;
    const float dl = ok ? p.dlogprob[row] * p.inv_t : NAN, dh = p.dentropy ? p.dentropy[row] * p.inv_t : 0.f;
    // dz = p (c1 + c2 log2 p) + [c == y] dl
    const float c1 = -fmaf(dh, p.dentropy ? p.entropy[row] : 0.f, dl), c2 = -dh * kLn2;
    const auto one = [&](float x) {
      const float u = sizeof(T) == 4 ? max_nan(x - m, -1e30f) : x - m;  // (-inf times the low half would be NaN)
      float t = fmaf(u, p.scale, -l2);
      if (sizeof(T) == 4) t += fmaf(u, c_lo, -l2_lo);
      t = max_nan(t, -200.f);
      return fast_exp2(t) * fmaf(c2, t, c1);
    };
    const auto write = [&](int i, const Pack<T, W>& raw) {
      Pack<T, W> o;
      float v[W];
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = one(raw[j]);
      const int at = y - (cut.head + i * W);
      if (static_cast<unsigned>(at) < static_cast<unsigned>(W)) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] += j == at ? dl : 0.f;
      }
#pragma unroll
      for (int j = 0; j < W; ++j) o.set(j, v[j]);
      store_pack_cs(gr + cut.head + i * W, o);
    };
    if (same) {
      for (int b = i0 + tid; b < i1; b += kU * NT) {
        Pack<T, W> raw[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (b + u * NT < i1) raw[u] = load_pack<T, W>(z + cut.head + (b + u * NT) * W);
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (b + u * NT < i1) write(b + u * NT, raw[u]);
      }
    } else {  // the logits' rows lie otherwise than the gradient's: element by element
      for (int i = i0 + tid; i < i1; i += NT) {
        Pack<T, W> raw;
#pragma unroll
        for (int j = 0; j < W; ++j) raw.e[j] = z[cut.head + i * W + j];
        write(i, raw);
      }
    }
    if (edges) {
      const int e = cut.edge(tid);
      gr[e] = elem_of<T>(one(elem_f(z[e])) + (e == y ? dl : 0.f));
    }
  }
}

// ---------------------------------------------------------------- host side

namespace {

template <class T, int NT>
cudaError_t run_fwd(const LogprobParams& p, int sms, cudaStream_t st) {
  const auto kernel = logprobs_fwd_kernel<T, NT>;
  constexpr size_t smem = sizeof(uint4) * kDepth * kU * NT + 2 * sizeof(RowSmem<NT>);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(std::min<int64_t>(p.T, static_cast<int64_t>(sms) * ctas_per_sm<NT>()));
  return launch_pdl(kernel, dim3(grid), dim3(NT), smem, st, p);
}

// us a call: a warp a row for rows up to 16 KB (T = 16384, V = 3000 bf16, k = 0: 40, with 256 threads 78); 128 threads for few
// alternatives of rows up to 64 KB (T = 8192, V = 32768 bf16, k = 5: 113, with 256 threads 128; k = 20: 163 and 171, but V = 131072, k = 20: 175
// and 132, as each part that is looked at again is twice as long) and for up to 64 of rows up to 16 KB (T = 16384, V = 1000, k = 64: 130, with
// 256 277; V = 8000 212 and 280; k = 128 has more candidates than 128 parts can tell apart: V = 8000 1473 and 425); 512 while every row has a block at once (T = 64, V = 32000, k = 20:
// 8.4, with 256 9.4, with 1024 8.9).
template <class T>
cudaError_t pick_fwd(const LogprobParams& p, cudaStream_t st) {
  const int sms = device_sms();
  const int64_t bytes = static_cast<int64_t>(p.V) * sizeof(T);
  if (bytes <= 16384 && p.k <= 32) return run_fwd<T, 32>(p, sms, st);
  if (p.T <= 2 * sms) return run_fwd<T, 512>(p, sms, st);
  return bytes <= 65536 && (p.k <= 8 || (p.k <= 64 && bytes <= 16384)) ? run_fwd<T, 128>(p, sms, st) : run_fwd<T, 256>(p, sms, st);
}

// us a call: a warp a row for rows up to 4 KB, up to 16 KB where there are rows enough to fill the GPU that way (T = 16384, bf16, V = 3000:
// 42, with 256 threads 66; V = 8000 91 and 93; fp32, V = 1500 42 and 60).
template <class T>
cudaError_t pick_bwd(LogprobParams p, cudaStream_t st) {
  const int sms = device_sms();
  const int64_t bytes = static_cast<int64_t>(p.V) * sizeof(T);
  if (bytes <= (p.T >= 8 * sms ? 16384 : 4096)) {
    p.slices = 1;
    return launch_pdl(logprobs_bwd_kernel<T, 32>, dim3(static_cast<unsigned>(std::min<int64_t>(p.T, sms * 24))), dim3(32), 0,
                      st, p);
  }
  // few rows: pieces of at least a group a thread, until there is one for every block that fits
  const int64_t fit = static_cast<int64_t>(sms) * 4, group = kU * 256 * 16;
  const uintptr_t z = reinterpret_cast<uintptr_t>(p.z), g = reinterpret_cast<uintptr_t>(p.grad);
  const uintptr_t zn = (static_cast<uintptr_t>(p.T - 1) * p.z_rs + p.V) * sizeof(T);
  const uintptr_t gn = (static_cast<uintptr_t>(p.T - 1) * p.g_rs + p.V) * sizeof(T);
  const bool apart = z + zn <= g || g + gn <= z;
  p.slices = apart ? static_cast<int>(std::max<int64_t>(1, std::min(fit / p.T, bytes / group))) : 1;
  const int grid = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(p.T) * p.slices, fit));
  return launch_pdl(logprobs_bwd_kernel<T, 256>, dim3(grid), dim3(256), 0, st, p);
}

}  // namespace

cudaError_t launch_logprobs_fwd(LogprobParams p, int bf16, cudaStream_t st) {
  return bf16 ? pick_fwd<__nv_bfloat16>(p, st) : pick_fwd<float>(p, st);
}

cudaError_t launch_logprobs_bwd(LogprobParams p, int bf16, cudaStream_t st) {
  return bf16 ? pick_bwd<__nv_bfloat16>(p, st) : pick_bwd<float>(p, st);
}

}  // namespace va
