// Norm of every query and key head with the position rotation, in one pass, and its gradient.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  u = n w,
//   y = u with its first `rot` dims turned pair by pair by pos * inv_freq[i]:
//       (a, b) -> (a cos - b sin, b cos + a sin)
// pairs (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved.  Backward: g = dy turned back,
//   dw = sum over tokens and heads of g n,   dx = r (g w - n mean(g w n)).
//
// Layout: a head of d elements is held by G lanes of a warp (G the power of two at or above d / 8), a
// lane holding two pieces of four elements such that every pair lies in one lane: dims 4 u and rot / 2 + 4 u
// of unit u < rot / 8 (8 u and 8 u + 4 when interleaved, and for the dims that are not turned).  So
// nothing but the sums crosses lanes.  A warp takes a token's heads, or some of them, in turn, and keeps the
// token's cosines and sines in registers.
//
// Angles: inv_freq / 2 pi as a fraction of a turn in 64 bits, times the position modulo 2^64: whole turns
// drop out exactly, so a position of a million is turned as accurately as the first.
//
// Weight gradients: a warp's sums stay in registers over all its heads and tokens, are added in the block in
// warp order and written as one row per block; qk_norm_join_kernel adds the rows in order.  Tokens are
// dealt to the warps by a fixed rule, so results do not change from call to call.
#include <algorithm>

#include "elem.cuh"
#include "qk_norm.cuh"

namespace va {

namespace {

constexpr int kQkThreads = 256, kQkWarps = kQkThreads / 32;
constexpr int kSteps = 4;  // head groups a warp has in flight

// The dims of a lane's two pieces, or first >= d for a lane without a head's part.
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

// inv_freq as a fraction of a turn per position, times 2^64.
__device__ __forceinline__ uint64_t turn_of(float inv_freq) {
  double t = static_cast<double>(inv_freq) * 0.15915494309189533577;
  t -= floor(t);
  return static_cast<uint64_t>(t * 18446744073709551616.0);
}

__device__ __forceinline__ void angle(int pos, uint64_t turn, float& c, float& s) {
  const uint64_t f = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turn;  // mod a turn
  sincospif(static_cast<float>(static_cast<int32_t>(f >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
}

__device__ __forceinline__ float load_w(const void* w, int bf16, int i) {
  if (!w) return 1.f;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}

struct Lane {
  float c[4], s[4];       // the token's cosines and sines for this lane's four pairs (1, 0 when not turned)
  uint64_t turn[4];
};

__device__ __forceinline__ void lane_turns(Lane& l, const QkParams& p, const Unit& un, int u) {
#pragma unroll
  for (int j = 0; j < 4; ++j) l.turn[j] = un.on && un.turned ? turn_of(p.inv_freq[4 * u + j]) : 0;
}

__device__ __forceinline__ void lane_angles(Lane& l, int pos) {
#pragma unroll
  for (int j = 0; j < 4; ++j) angle(pos, l.turn[j], l.c[j], l.s[j]);
}

// x[0..3] the first piece, x[4..7] the second; back: by the negative angle.
template <bool IL, bool BACK>
__device__ __forceinline__ void rotate(float (&x)[8], const Lane& l) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = IL ? 2 * j : j, k = IL ? 2 * j + 1 : j + 4;
    const float s = BACK ? -l.s[j] : l.s[j];
    const float a = x[i], b = x[k];
    x[i] = a * l.c[j] - b * s;
    x[k] = b * l.c[j] + a * s;
  }
}

template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int G) {
  for (int o = G >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// A warp's share of a token: head groups [s0, s1) of the Sq + Sk that the token's queries and keys make.
struct Share {
  int token, s0, s1;
};
__device__ __forceinline__ Share share_of(const QkParams& p, int64_t item, int steps) {
  Share r;
  r.token = static_cast<int>(item / p.chunks);
  const int c = static_cast<int>(item % p.chunks);
  r.s0 = static_cast<int>(static_cast<int64_t>(steps) * c / p.chunks);
  r.s1 = static_cast<int>(static_cast<int64_t>(steps) * (c + 1) / p.chunks);
  return r;
}

}  // namespace

template <class T, bool IL>
__global__ void __launch_bounds__(kQkThreads) qk_norm_fwd_kernel(const QkParams p) {
  griddep_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane & (p.G - 1), sub = lane / p.G, per = 32 / p.G;
  const Unit un = unit_of(u, p.d, p.rot, IL);
  const int Sq = (p.H[0] + per - 1) / per, Sk = (p.H[1] + per - 1) / per;
  float w[2][8];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) w[q][j] = un.on ? load_w(p.w[q], p.w_bf16, (j < 4 ? un.a : un.b - 4) + j) : 0.f;
  Lane l;
  lane_turns(l, p, un, u);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int64_t items = static_cast<int64_t>(p.T) * p.chunks;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kQkWarps + warp; item < items;
       item += static_cast<int64_t>(gridDim.x) * kQkWarps) {
    const Share sh = share_of(p, item, Sq + Sk);
    lane_angles(l, p.pos[sh.token]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int lo = q == 0 ? sh.s0 : max(sh.s0, Sq) - Sq, hi = q == 0 ? min(sh.s1, Sq) : sh.s1 - Sq;
      const T* x = static_cast<const T*>(p.x[q]) + sh.token * p.x_rs[q];
      T* y = static_cast<T*>(p.y[q]) + sh.token * p.y_rs[q];
      for (int s = lo; s < hi; s += kSteps) {
        Pack<T, 4> in[kSteps][2];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int h = (s + i) * per + sub;
          if (s + i < hi && un.on && h < p.H[q]) {
            in[i][0] = load_pack<T, 4>(x + h * p.x_hs[q] + un.a);
            in[i][1] = load_pack<T, 4>(x + h * p.x_hs[q] + un.b);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) in[i][0].set(j, 0.f), in[i][1].set(j, 0.f);
          }
        }
        float ss[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          ss[i] = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss[i] = fmaf(in[i][j >> 2][j & 3], in[i][j >> 2][j & 3], ss[i]);
        }
        group_sum(ss, p.G);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int h = (s + i) * per + sub;
          if (!(s + i < hi && un.on && h < p.H[q])) continue;
          const float r = rsqrtf(fmaf(ss[i], inv_d, p.eps));
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = in[i][j >> 2][j & 3] * r * w[q][j];
          rotate<IL, false>(v, l);
          Pack<T, 4> out[2];
#pragma unroll
          for (int j = 0; j < 8; ++j) out[j >> 2].set(j & 3, v[j]);
          store_pack(y + h * p.y_hs[q] + un.a, out[0]);
          store_pack(y + h * p.y_hs[q] + un.b, out[1]);
        }
      }
    }
  }
}

template <class T, bool IL>
__global__ void __launch_bounds__(kQkThreads) qk_norm_bwd_kernel(const QkParams p) {
  griddep_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane & (p.G - 1), sub = lane / p.G, per = 32 / p.G;
  const Unit un = unit_of(u, p.d, p.rot, IL);
  const int Sq = (p.H[0] + per - 1) / per, Sk = (p.H[1] + per - 1) / per;
  float w[2][8], dw[2][8];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[q][j] = un.on ? load_w(p.w[q], p.w_bf16, (j < 4 ? un.a : un.b - 4) + j) : 0.f;
      dw[q][j] = 0.f;
    }
  Lane l;
  lane_turns(l, p, un, u);
  const float inv_d = 1.f / static_cast<float>(p.d);
  constexpr int kS = kSteps / 2;
  const int64_t items = static_cast<int64_t>(p.T) * p.chunks;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kQkWarps + warp; item < items;
       item += static_cast<int64_t>(gridDim.x) * kQkWarps) {
    const Share sh = share_of(p, item, Sq + Sk);
    lane_angles(l, p.pos[sh.token]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int lo = q == 0 ? sh.s0 : max(sh.s0, Sq) - Sq, hi = q == 0 ? min(sh.s1, Sq) : sh.s1 - Sq;
      const T* x = static_cast<const T*>(p.x[q]) + sh.token * p.x_rs[q];
      const T* dy = static_cast<const T*>(p.dy[q]) + sh.token * p.dy_rs[q];
      T* dx = static_cast<T*>(p.y[q]) + sh.token * p.y_rs[q];
      for (int s = lo; s < hi; s += kS) {
        Pack<T, 4> in[kS][2], gi[kS][2];
#pragma unroll
        for (int i = 0; i < kS; ++i) {
          const int h = (s + i) * per + sub;
          if (s + i < hi && un.on && h < p.H[q]) {
            in[i][0] = load_pack<T, 4>(x + h * p.x_hs[q] + un.a);
            in[i][1] = load_pack<T, 4>(x + h * p.x_hs[q] + un.b);
            gi[i][0] = load_pack<T, 4>(dy + h * p.dy_hs[q] + un.a);
            gi[i][1] = load_pack<T, 4>(dy + h * p.dy_hs[q] + un.b);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              in[i][0].set(j, 0.f), in[i][1].set(j, 0.f), gi[i][0].set(j, 0.f), gi[i][1].set(j, 0.f);
          }
        }
        float sum[2 * kS], g[kS][8];  // sums of x^2 and of g w x
#pragma unroll
        for (int i = 0; i < kS; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) g[i][j] = gi[i][j >> 2][j & 3];
          rotate<IL, true>(g[i], l);
          sum[2 * i] = sum[2 * i + 1] = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = in[i][j >> 2][j & 3];
            sum[2 * i] = fmaf(v, v, sum[2 * i]);
            sum[2 * i + 1] = fmaf(g[i][j] * w[q][j], v, sum[2 * i + 1]);
          }
        }
        group_sum(sum, p.G);
#pragma unroll
        for (int i = 0; i < kS; ++i) {
          const int h = (s + i) * per + sub;
          if (!(s + i < hi && un.on && h < p.H[q])) continue;
          const float r = rsqrtf(fmaf(sum[2 * i], inv_d, p.eps));
          const float m = sum[2 * i + 1] * inv_d * r * r;  // mean(g w n) / |x| of a unit r: x m = n mean(g w n)
          Pack<T, 4> out[2];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = in[i][j >> 2][j & 3];
            dw[q][j] = fmaf(g[i][j], v * r, dw[q][j]);
            out[j >> 2].set(j & 3, r * (g[i][j] * w[q][j] - v * m));
          }
          store_pack(dx + h * p.y_hs[q] + un.a, out[0]);
          store_pack(dx + h * p.y_hs[q] + un.b, out[1]);
        }
      }
    }
  }
  if (!p.part) return;
  __shared__ float sh_dw[kQkWarps][2 * kQkMaxDim];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      for (int o = p.G; o < 32; o <<= 1) dw[q][j] += __shfl_xor_sync(0xffffffffu, dw[q][j], o);
      if (sub == 0 && un.on) sh_dw[warp][q * p.d + (j < 4 ? un.a : un.b - 4) + j] = dw[q][j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.d; i += kQkThreads) {
    float a = 0.f;
    for (int v = 0; v < kQkWarps; ++v) a += sh_dw[v][i];
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

int qk_sms() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return std::max(sms, 1);
}

// Lanes per head, and the pieces a token's heads are cut into: one warp a token unless that leaves most
// of the GPU without work.
void qk_shape(QkParams& p, int sms) {
  p.G = 1;
  while (8 * p.G < p.d) p.G *= 2;
  const int per = 32 / p.G;
  const int steps = (p.H[0] + per - 1) / per + (p.H[1] + per - 1) / per;
  const int64_t want = static_cast<int64_t>(sms) * kQkWarps * 2;
  p.chunks = static_cast<int>(std::min<int64_t>(steps, std::max<int64_t>(1, want / std::max(p.T, 1))));
}

}  // namespace


size_t qk_norm_bwd_workspace(int d) { return static_cast<size_t>(kQkMaxBlocks) * 2 * d * sizeof(float); }

cudaError_t launch_qk_norm_fwd(QkParams p, int bf16, cudaStream_t st) {
  const int sms = qk_sms();
  qk_shape(p, sms);
  const int64_t items = static_cast<int64_t>(p.T) * p.chunks;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((items + kQkWarps - 1) / kQkWarps, sms * 8)));
  if (bf16)
    return p.interleaved ? launch_pdl(qk_norm_fwd_kernel<__nv_bfloat16, true>, grid, dim3(kQkThreads), 0, st, p)
                         : launch_pdl(qk_norm_fwd_kernel<__nv_bfloat16, false>, grid, dim3(kQkThreads), 0, st, p);
  return p.interleaved ? launch_pdl(qk_norm_fwd_kernel<float, true>, grid, dim3(kQkThreads), 0, st, p)
                       : launch_pdl(qk_norm_fwd_kernel<float, false>, grid, dim3(kQkThreads), 0, st, p);
}

// stage 0: the rows' gradients and the blocks' weight gradients, 1: their sum.
cudaError_t launch_qk_norm_bwd(int stage, QkParams p, int bf16, cudaStream_t st) {
  const int sms = qk_sms();
  qk_shape(p, sms);
  const int64_t items = static_cast<int64_t>(p.T) * p.chunks;
  const int blocks = static_cast<int>(
      std::min<int64_t>({(items + kQkWarps - 1) / kQkWarps, static_cast<int64_t>(sms) * 2, kQkMaxBlocks}));
  if (stage == 1) return launch_pdl(qk_norm_join_kernel, dim3((2 * p.d + 31) / 32), dim3(1024), 0, st, p, blocks);
  const dim3 grid(blocks);
  if (bf16)
    return p.interleaved ? launch_pdl(qk_norm_bwd_kernel<__nv_bfloat16, true>, grid, dim3(kQkThreads), 0, st, p)
                         : launch_pdl(qk_norm_bwd_kernel<__nv_bfloat16, false>, grid, dim3(kQkThreads), 0, st, p);
  return p.interleaved ? launch_pdl(qk_norm_bwd_kernel<float, true>, grid, dim3(kQkThreads), 0, st, p)
                       : launch_pdl(qk_norm_bwd_kernel<float, false>, grid, dim3(kQkThreads), 0, st, p);
}

}  // namespace va
