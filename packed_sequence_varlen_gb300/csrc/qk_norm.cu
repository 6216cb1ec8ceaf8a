// Norm of every query and key head with the position rotation, in one pass, and its gradient.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  u = n w,
//   y = u with its first `rot` dims turned pair by pair by pos * inv_freq[i]:
//       (a, b) -> (a cos - b sin, b cos + a sin)
// pairs (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved.  Backward: g = dy turned back,
//   dw = sum over tokens and heads of g n,   dx = r (g w - n mean(g w n)).
//
// Layout: a head of d elements is held by G lanes of a warp (G the power of two at or above d / 8), a
// lane holding four pairs: dims 4 u .. 4 u + 3 and rot / 2 + 4 u .. of unit u < rot / 8 (8 u .. 8 u + 7 when interleaved, and
// for the dims that are not turned, as pairs with an angle of 0).  So nothing but the sums crosses lanes.  A group is the
// 32 / G heads that a warp takes at a time.
//
// Work: the groups of all tokens, token by token, are one sequence, of which every warp takes an equal stretch; so
// whatever the sizes the warps end together, and results do not change from call to call.  A warp's groups are copied
// to a ring of its own in shared memory, kRing bytes ahead, 16 bytes a lane: nothing waits for another warp.
//
// Angles: inv_freq / 2 pi as a fraction of a turn in 64 bits (whole numbers: fp64 is slow here), times the position modulo
// 2^64: whole turns drop out exactly, so a position of a million is turned as accurately as the first.
//
// Weight gradients: a warp's sums stay in registers over all its groups, are added in the block in warp order and
// written as one row per block; qk_norm_join_kernel adds the rows in order.
#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "qk_norm.cuh"
#include "vec.cuh"

namespace va {

namespace {

constexpr int kQkThreads = 256, kQkWarps = kQkThreads / 32;
constexpr int kRing = 8192;  // bytes a warp has on their way
constexpr int kBlocks = 2;   // blocks an SM (three with 80 registers: forward 66 us instead of 62)

using V4 = Vec<4>;

// The dims of a lane's two pieces, and whether it has any and whether they are turned.
struct Unit {
  int a, b;
  bool on, turned;
};
__device__ __forceinline__ Unit unit_of(int u, int d, int rot, int interleaved) {
  Unit r;
  r.on = 8 * u < d;
  r.turned = 8 * u < rot;
  r.a = r.turned && !interleaved ? 4 * u : 8 * u;
  r.b = r.turned && !interleaved ? rot / 2 + 4 * u : 8 * u + 4;
  return r;
}

// inv_freq as a fraction of a turn per position, times 2^64: its 24 bits times 1 / 2 pi to 96 bits, shifted.
__device__ __forceinline__ uint64_t turn_of(float inv_freq) {
  const uint32_t b = __float_as_uint(inv_freq), field = (b >> 23) & 255u;
  const uint64_t m = (b & 0x7fffffu) | (field ? 0x800000u : 0u);
  const int shift = 32 - (static_cast<int>(field ? field : 1u) - 150);  // the value is m 2^(field - 150)
  const unsigned __int128 c = static_cast<unsigned __int128>(0x28be60dbu) << 64 | 0x9391054a7f09d5f4ull;
  const unsigned __int128 x = c * m;
  const uint64_t t = shift >= 128 ? 0 : shift >= 0 ? static_cast<uint64_t>(x >> shift)
                     : shift > -64 ? static_cast<uint64_t>(x) << -shift : 0;
  return b >> 31 ? 0 - t : t;
}

__device__ __forceinline__ void angle(int pos, uint64_t turn, float& c, float& s) {
  const uint64_t f = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turn;  // mod a turn
  sincospif(static_cast<float>(static_cast<int32_t>(f >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
}

__device__ __forceinline__ float load_w(const void* w, int bf16, int i) {
  if (!w) return 1.f;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}

// A lane's eight numbers as the first and the second of its four pairs.
template <bool IL>
__device__ __forceinline__ void to_pairs(const V4& p, const V4& q, V4& a, V4& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    a[j] = !IL ? p[j] : j < 2 ? p[2 * j] : q[2 * j - 4];
    b[j] = !IL ? q[j] : j < 2 ? p[2 * j + 1] : q[2 * j - 3];
  }
}
template <bool IL>
__device__ __forceinline__ void to_pieces(const V4& a, const V4& b, V4& p, V4& q) {
  if constexpr (IL) {
    p = V4{{a[0], b[0], a[1], b[1]}};
    q = V4{{a[2], b[2], a[3], b[3]}};
  } else {
    p = a;
    q = b;
  }
}

__device__ __forceinline__ float across(const V4& v) { return (v[0] + v[1]) + (v[2] + v[3]); }
// The sums of N numbers over the G lanes of a head.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int G) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < G)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// A place in the sequence of groups (a token's queries, then its keys), and a lane's element of it in N tensors:
// moving on is an addition, the strides are multiplied only where a token's queries or keys begin.
struct Rows {
  const void* base[2];
  int64_t rs[2], hs[2];
};
template <class T, int N>
struct Cursor {
  int token, q, head;  // head: the group's first
  const T* at[N];
  int64_t step[N];
  template <class R>
  __device__ __forceinline__ void begin(const R& rows, int sub, int per, int off) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Rows r = rows(n);
      const int64_t rs = q ? r.rs[1] : r.rs[0], hs = q ? r.hs[1] : r.hs[0];
      at[n] = static_cast<const T*>(q ? r.base[1] : r.base[0]) + token * rs + (head + sub) * hs + off;
      step[n] = per * hs;
    }
  }
  template <class R>
  __device__ __forceinline__ void next(const R& rows, int H0, int H1, int sub, int per, int off) {
    head += per;
    if (head >= (q ? H1 : H0)) {
      head = 0;
      token += q;
      q ^= 1;
      begin(rows, sub, per, off);
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) at[n] += step[n];
    }
  }
};

// What a lane keeps of the call: its dims, the queries' and keys' weights (as pairs), its four frequencies.
template <bool IL>
struct LaneState {
  Unit un;
  int sub, per, Sq, groups;
  V4 wa[2], wb[2];
  uint64_t turn[4];
  __device__ __forceinline__ LaneState(const QkParams& p, int G) {
    const int lane = threadIdx.x & 31, u = lane & (G - 1);
    sub = lane / G;
    per = 32 / G;
    un = unit_of(u, p.d, p.rot, IL);
    Sq = (p.H[0] + per - 1) / per;
    groups = Sq + (p.H[1] + per - 1) / per;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      V4 first, second;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        first[j] = un.on ? load_w(p.w[q], p.w_bf16, un.a + j) : 0.f;
        second[j] = un.on ? load_w(p.w[q], p.w_bf16, un.b + j) : 0.f;
      }
      to_pairs<IL>(first, second, wa[q], wb[q]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) turn[j] = un.on && un.turned ? turn_of(p.inv_freq[4 * u + j]) : 0;
  }
  __device__ __forceinline__ void angles(int pos, V4& c, V4& s) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) angle(pos, turn[j], c[j], s[j]);
  }
  template <class T, int N>
  __device__ __forceinline__ Cursor<T, N> place(int64_t i) const {
    Cursor<T, N> c;
    c.token = static_cast<int>(i / groups);
    const int g = static_cast<int>(i % groups);
    c.q = g >= Sq;
    c.head = (g - (c.q ? Sq : 0)) * per;
    return c;
  }
};

}  // namespace

// GT: lanes per head, so that the sums have no loop (16384 tokens, 12 + 1 heads of 256 bf16 57 us, with a loop 62); 0: as the call
// says.
template <class T, bool IL, int GT>
__global__ void __launch_bounds__(kQkThreads, kBlocks) qk_norm_fwd_kernel(QkParams p) {
  griddep_begin();
  constexpr int kPiece = 8 * sizeof(T), kStage = 32 * kPiece, D = kRing / kStage;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* const ring = smem + warp * kRing;
  const int G = GT ? GT : p.G;
  const LaneState<IL> l(p, G);
  const int64_t all = static_cast<int64_t>(p.T) * l.groups, warps = static_cast<int64_t>(gridDim.x) * kQkWarps;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kQkWarps + warp;
  const int64_t first = all * me / warps;
  const int mine = static_cast<int>(all * (me + 1) / warps - first);
  const int u = lane & (G - 1);
  const auto in = [&](int) { return Rows{{p.x[0], p.x[1]}, {p.x_rs[0], p.x_rs[1]}, {p.x_hs[0], p.x_hs[1]}}; };
  const auto out = [&](int) { return Rows{{p.y[0], p.y[1]}, {p.y_rs[0], p.y_rs[1]}, {p.y_hs[0], p.y_hs[1]}}; };
  Cursor<T, 1> ask = l.template place<T, 1>(first), at = ask;
  ask.begin(in, l.sub, l.per, 8 * u);
  at.begin(out, l.sub, l.per, 0);
  uint8_t* const mine_ring = ring + (l.sub * G + u) * kPiece;
  const auto issue = [&](int i, int to) {
    if (i < mine) {
      if (l.un.on && ask.head + l.sub < (ask.q ? p.H[1] : p.H[0])) {
#pragma unroll
        for (int k = 0; k < kPiece / 16; ++k) copy16(mine_ring + to + 16 * k, ask.at[0] + 16 / sizeof(T) * k);
      }
      ask.next(in, p.H[0], p.H[1], l.sub, l.per, 8 * u);
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) issue(i, i * kStage);
  const float inv_d = 1.f / static_cast<float>(p.d);
  V4 c, s, ca, sb, cb, sa;  // the token's, and with the weights: y_a = r (x_a ca - x_b sb), y_b = r (x_b cb + x_a sa)
  int here = 0, pos = p.pos[min(at.token, p.T - 1)];
  for (int i = 0; i < mine; ++i) {
    issue(i + D - 1, (here - kStage) & (kRing - 1));
    if (i == 0 || at.head == 0) {
      if (i == 0 || at.q == 0) {
        l.angles(pos, c, s);
        pos = p.pos[min(at.token + 1, p.T - 1)];  // the next token's
      }
      const bool k = at.q != 0;
      const V4 wa = k ? l.wa[1] : l.wa[0], wb = k ? l.wb[1] : l.wb[0];
      ca = mul(c, wa);
      sa = mul(s, wa);
      cb = mul(c, wb);
      sb = mul(s, wb);
#pragma unroll
      for (int j = 0; j < 4; ++j) sb[j] = -sb[j];
    }
    copy_wait<D - 1>();
    __syncwarp();
    const bool on = l.un.on && at.head + l.sub < (at.q ? p.H[1] : p.H[0]);
    const T* row = reinterpret_cast<const T*>(ring + here) + l.sub * G * 8;
    V4 xa = fill<4>(0.f), xb = xa;
    if (on) to_pairs<IL>(wide_of(load_pack<T, 4>(row + l.un.a)), wide_of(load_pack<T, 4>(row + l.un.b)), xa, xb);
    float ss[1] = {across(fma(xb, xb, mul(xa, xa)))};
    group_sum(ss, G);
    const float r = rsqrtf(fmaf(ss[0], inv_d, p.eps));
    __syncwarp();  // the stage is written again
    if (on) {
      const V4 rr = fill<4>(r);
      const V4 ya = mul(fma(xb, sb, mul(xa, ca)), rr), yb = mul(fma(xa, sa, mul(xb, cb)), rr);
      V4 first4, second4;
      to_pieces<IL>(ya, yb, first4, second4);
      T* y = const_cast<T*>(at.at[0]);
      store_pack(y + l.un.a, narrow<T, 4>(first4));
      store_pack(y + l.un.b, narrow<T, 4>(second4));
    }
    at.next(out, p.H[0], p.H[1], l.sub, l.per, 0);
    here = (here + kStage) & (kRing - 1);
  }
}

template <class T, bool IL, int GT>
__global__ void __launch_bounds__(kQkThreads, kBlocks) qk_norm_bwd_kernel(QkParams p) {
  griddep_begin();
  constexpr int kPiece = 8 * sizeof(T), kHalf = 32 * kPiece, kStage = 2 * kHalf, D = kRing / kStage;  // x, then dy
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* const ring = smem + warp * kRing;
  const int G = GT ? GT : p.G;
  const LaneState<IL> l(p, G);
  const int64_t all = static_cast<int64_t>(p.T) * l.groups, warps = static_cast<int64_t>(gridDim.x) * kQkWarps;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kQkWarps + warp;
  const int64_t first = all * me / warps;
  const int mine = static_cast<int>(all * (me + 1) / warps - first);
  const int u = lane & (G - 1);
  const auto in = [&](int n) {
    return n == 0 ? Rows{{p.x[0], p.x[1]}, {p.x_rs[0], p.x_rs[1]}, {p.x_hs[0], p.x_hs[1]}}
                  : Rows{{p.dy[0], p.dy[1]}, {p.dy_rs[0], p.dy_rs[1]}, {p.dy_hs[0], p.dy_hs[1]}};
  };
  const auto out = [&](int) { return Rows{{p.y[0], p.y[1]}, {p.y_rs[0], p.y_rs[1]}, {p.y_hs[0], p.y_hs[1]}}; };
  Cursor<T, 2> ask = l.template place<T, 2>(first);
  Cursor<T, 1> at = l.template place<T, 1>(first);
  ask.begin(in, l.sub, l.per, 8 * u);
  at.begin(out, l.sub, l.per, 0);
  uint8_t* const mine_ring = ring + (l.sub * G + u) * kPiece;
  const auto issue = [&](int i, int to) {
    if (i < mine) {
      if (l.un.on && ask.head + l.sub < (ask.q ? p.H[1] : p.H[0])) {
#pragma unroll
        for (int k = 0; k < kPiece / 16; ++k) {
          copy16(mine_ring + to + 16 * k, ask.at[0] + 16 / sizeof(T) * k);
          copy16(mine_ring + to + kHalf + 16 * k, ask.at[1] + 16 / sizeof(T) * k);
        }
      }
      ask.next(in, p.H[0], p.H[1], l.sub, l.per, 8 * u);
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) issue(i, i * kStage);
  const float inv_d = 1.f / static_cast<float>(p.d);
  V4 c, s, dwa[2], dwb[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) dwa[q] = dwb[q] = fill<4>(0.f);
  int here = 0, pos = p.pos[min(at.token, p.T - 1)];
  // one group of the queries (Q 0) or keys
  const auto group = [&](auto which) {
    constexpr int q = decltype(which)::value;
    const bool on = l.un.on && at.head + l.sub < p.H[q];
    const T* row = reinterpret_cast<const T*>(ring + here) + l.sub * G * 8;
    const T* grow = reinterpret_cast<const T*>(ring + here + kHalf) + l.sub * G * 8;
    V4 xa = fill<4>(0.f), xb = xa, ya = xa, yb = xa;
    if (on) {
      to_pairs<IL>(wide_of(load_pack<T, 4>(row + l.un.a)), wide_of(load_pack<T, 4>(row + l.un.b)), xa, xb);
      to_pairs<IL>(wide_of(load_pack<T, 4>(grow + l.un.a)), wide_of(load_pack<T, 4>(grow + l.un.b)), ya, yb);
    }
    V4 ms;
#pragma unroll
    for (int j = 0; j < 4; ++j) ms[j] = -s[j];
    const V4 ga = fma(yb, s, mul(ya, c)), gb = fma(ya, ms, mul(yb, c));  // turned back
    const V4 ua = mul(ga, l.wa[q]), ub = mul(gb, l.wb[q]);
    float sum[2] = {across(fma(xb, xb, mul(xa, xa))), across(fma(ub, xb, mul(ua, xa)))};  // of x^2 and of g w x
    group_sum(sum, G);
    __syncwarp();  // the stage is written again
    const float r = on ? rsqrtf(fmaf(sum[0], inv_d, p.eps)) : 0.f;  // (a lane without a head: zeros, whatever eps is)
    const V4 rr = fill<4>(r), m = fill<4>(-sum[1] * inv_d * r * r);  // x m = -n mean(g w n) / r
    dwa[q] = fma(ga, mul(xa, rr), dwa[q]);
    dwb[q] = fma(gb, mul(xb, rr), dwb[q]);
    if (on) {
      V4 first4, second4;
      to_pieces<IL>(mul(fma(xa, m, ua), rr), mul(fma(xb, m, ub), rr), first4, second4);
      T* dx = const_cast<T*>(at.at[0]);
      store_pack(dx + l.un.a, narrow<T, 4>(first4));
      store_pack(dx + l.un.b, narrow<T, 4>(second4));
    }
  };
  for (int i = 0; i < mine; ++i) {
    issue(i + D - 1, (here - kStage) & (kRing - 1));
    if (i == 0 || (at.head == 0 && at.q == 0)) {
      l.angles(pos, c, s);
      pos = p.pos[min(at.token + 1, p.T - 1)];  // the next token's
    }
    copy_wait<D - 1>();
    __syncwarp();
    if (at.q == 0) group(std::integral_constant<int, 0>{});
    else group(std::integral_constant<int, 1>{});
    at.next(out, p.H[0], p.H[1], l.sub, l.per, 0);
    here = (here + kStage) & (kRing - 1);
  }
  if (!p.part) return;
  copy_wait<0>();
  __syncthreads();  // the rings become the warps' sums
  float* const sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    V4 first4, second4;
    to_pieces<IL>(dwa[q], dwb[q], first4, second4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      for (int o = G; o < 32; o <<= 1) {
        first4[j] += __shfl_xor_sync(0xffffffffu, first4[j], o);
        second4[j] += __shfl_xor_sync(0xffffffffu, second4[j], o);
      }
      if (l.sub == 0 && l.un.on) {
        sums[(warp * 2 + q) * kQkMaxDim + l.un.a + j] = first4[j];
        sums[(warp * 2 + q) * kQkMaxDim + l.un.b + j] = second4[j];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.d; i += kQkThreads) {
    const int q = i >= p.d;
    float a = 0.f;
    for (int v = 0; v < kQkWarps; ++v) a += sums[(v * 2 + q) * kQkMaxDim + i - q * p.d];
    p.part[static_cast<int64_t>(blockIdx.x) * 2 * p.d + i] = a;
  }
}

// Adds the blocks' rows of weight gradients: 32 columns a block, a warp every 32nd row, then warp by warp.
__global__ void __launch_bounds__(1024) qk_norm_join_kernel(const QkParams p, int rows) {
  griddep_begin();
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (col < 2 * p.d)
    for (int r = warp; r < rows; r += 32) a += p.part[static_cast<int64_t>(r) * 2 * p.d + col];
  sh[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || col >= 2 * p.d) return;
  a = 0.f;
  for (int v = 0; v < 32; ++v) a += sh[v][lane];
  const int q = col >= p.d, i = col - q * p.d;
  void* out = p.dw[q];
  if (!out) return;
  if (p.w_bf16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(a);
  else static_cast<float*>(out)[i] = a;
}

// ---------------------------------------------------------------- host side

namespace {

// Sets the lanes a head takes; returns the blocks: every one that fits, or as many as have a group for each warp.
int qk_shape(QkParams& p, int per_sm) {
  p.G = 1;
  while (8 * p.G < p.d) p.G *= 2;
  const int per = 32 / p.G;
  const int64_t groups = static_cast<int64_t>(p.T) * ((p.H[0] + per - 1) / per + (p.H[1] + per - 1) / per);
  const int64_t fit = static_cast<int64_t>(device_sms()) * per_sm;
  return static_cast<int>(std::min<int64_t>({(groups + kQkWarps - 1) / kQkWarps, fit, kQkMaxBlocks}));
}

cudaError_t launch_rings(void (*kernel)(QkParams), const QkParams& p, int blocks, cudaStream_t st) {
  constexpr int smem = kQkWarps * kRing;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e != cudaSuccess ? e : launch_pdl(kernel, dim3(blocks), dim3(kQkThreads), smem, st, p);
}

template <class T, bool IL>
cudaError_t run_fwd(const QkParams& p, int blocks, cudaStream_t st) {
  switch (p.G) {
    case 8: return launch_rings(qk_norm_fwd_kernel<T, IL, 8>, p, blocks, st);
    case 16: return launch_rings(qk_norm_fwd_kernel<T, IL, 16>, p, blocks, st);
    case 32: return launch_rings(qk_norm_fwd_kernel<T, IL, 32>, p, blocks, st);
    default: return launch_rings(qk_norm_fwd_kernel<T, IL, 0>, p, blocks, st);
  }
}

template <class T, bool IL>
cudaError_t run_bwd(const QkParams& p, int blocks, cudaStream_t st) {
  static_assert(kRing >= 2 * kQkMaxDim * sizeof(float), "a warp's ring holds its sums");
  switch (p.G) {
    case 8: return launch_rings(qk_norm_bwd_kernel<T, IL, 8>, p, blocks, st);
    case 16: return launch_rings(qk_norm_bwd_kernel<T, IL, 16>, p, blocks, st);
    case 32: return launch_rings(qk_norm_bwd_kernel<T, IL, 32>, p, blocks, st);
    default: return launch_rings(qk_norm_bwd_kernel<T, IL, 0>, p, blocks, st);
  }
}

}  // namespace

size_t qk_norm_bwd_workspace(int d) { return static_cast<size_t>(kQkMaxBlocks) * 2 * d * sizeof(float); }

cudaError_t launch_qk_norm_fwd(QkParams p, int bf16, cudaStream_t st) {
  const int blocks = qk_shape(p, kBlocks);
  if (bf16) return p.interleaved ? run_fwd<__nv_bfloat16, true>(p, blocks, st) : run_fwd<__nv_bfloat16, false>(p, blocks, st);
  return p.interleaved ? run_fwd<float, true>(p, blocks, st) : run_fwd<float, false>(p, blocks, st);
}

// stage 0: the rows' gradients and the blocks' weight gradients, 1: their sum.
cudaError_t launch_qk_norm_bwd(int stage, QkParams p, int bf16, cudaStream_t st) {
  const int blocks = qk_shape(p, kBlocks);
  if (stage == 1) return launch_pdl(qk_norm_join_kernel, dim3((2 * p.d + 31) / 32), dim3(1024), 0, st, p, blocks);
  if (bf16) return p.interleaved ? run_bwd<__nv_bfloat16, true>(p, blocks, st) : run_bwd<__nv_bfloat16, false>(p, blocks, st);
  return p.interleaved ? run_bwd<float, true>(p, blocks, st) : run_bwd<float, false>(p, blocks, st);
}

}  // namespace va
