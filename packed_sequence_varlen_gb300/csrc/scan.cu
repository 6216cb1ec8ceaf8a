// Gated linear recurrence over the packed stream, and its gradient.
//
//   h_t = a_t h_{t-1} + x_t,  a_t = exp(g_t),  per channel, restarted at every segment from h0 (or 0)
// Backward, from behind:  e_t = dh_t + f_{t+1},  f_t = a_t e_t,  dx_t = e_t,  dg_t = f_t h_{t-1}, where f_{t+1} is
// the last state's gradient (or 0) at a segment's last row, and f at its first row is h0's gradient.
//
// Both are one scan of affine maps c -> A c + B along the rows (forward: the state; backward: f, rows in
// descending order).  A tile is kWarps runs of R rows by 32 V channels; a warp holds its run in registers:
//   pass 1  the run's map from zero (A = exp(sum of g), B by the recurrence),
//   the runs' maps are combined in the block; the tile's map is published,
//   the state that enters the tile is folded from the maps of the tiles before it in its group of kGroup and
//   the state after the group before that one, which that group's last tile publishes,
//   pass 2  the recurrence again from the state that enters the run, with the outputs.
// So the data is read once and written once.  The fold's order is fixed by the tile's number, whatever is
// finished first, so results do not change from call to call.  A tile takes its number from a counter when it
// starts, so every tile it waits for is already running or done.  A segment's start (backward: its end) inside a
// run replaces the state instead of multiplying it by zero, so nothing of another segment gets in, infinities
// and NaN included, and no tile waits across one.
//
// A = exp(sum of g), rounded once, and not the product of the a: the approximate exponential of an a near 1 has a
// bias, which would add up over thousands of rows (h off by 2e-5 for a decay of 0.9995 a row).
#include <algorithm>

#include "elem.cuh"
#include "scan.cuh"
#include "sm100_ptx.cuh"

namespace va {

namespace {

constexpr int kWarps = 8;
constexpr int kGroup = 32;  // tiles that share a published state
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;   // rows of a run
constexpr int kTileRows = kWarps * kRows;
constexpr int kPrepThreads = 1024;

__device__ __forceinline__ float decay(float g) { return fast_exp2(g * kLog2e); }
// A run's decay, rounded once.
__device__ __forceinline__ float run_decay(float sum) { return 1.f + expm1f(sum); }

__device__ __forceinline__ int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(int32_t* p, int v) {
  asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// The first b in [0, B] with cu[b] >= row (cu[B] = T): a warp looks at 32 places at once.
__device__ __forceinline__ int first_at(const int32_t* cu, int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B + 1;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + (lane + 1) * step - 1;  // the last place of the lane's part
    const bool below = i < lo + n - 1 ? cu[i] < row : false;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    const int end = lo + n;
    lo += k * step;
    n = min(step, end - lo);
  }
  return lo;
}

// Rows row .. row + R - 1 that segments start at (bit i: row + i), cu[b] the first of them or later.
template <int R>
__device__ __forceinline__ uint32_t starts_mask(const int32_t* cu, int B, int b, int row) {
  const int lane = threadIdx.x & 31;
  uint32_t bit = 0;
  if (lane < R && b + lane <= B) {
    const int at = cu[b + lane] - row;
    if (at >= 0 && at < R) bit = 1u << at;
  }
  return __reduce_or_sync(0xffffffffu, bit);
}

// Polls a flag of a tile that has started before; false when the call is to be given up.
__device__ __forceinline__ bool wait_flag(const int32_t* flag, int32_t* status) {
  if (ld_acquire(flag)) return true;
  const uint64_t t0 = sm100::globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (ld_acquire(flag)) return true;
    if ((i & 63u) == 0) {
      if (*reinterpret_cast<volatile int32_t*>(status) != VA_OK) return false;
      if (sm100::globaltimer() - t0 > sm100::kTimeoutNs) {
        atomicCAS(status, 0, VA_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// What the runs of a tile exchange; channel = lane * V + i of the tile's columns.
template <int V>
struct TileSmem {
  float2 run[kWarps][32 * V];   // the runs' maps
  float2 part[kWarps][32 * V];  // the folds of the tiles before
  float carry[32 * V];          // the state after the group before
  int reset[kWarps];            // the run replaces the state
  int number;
  int give_up;
};

// The state that enters this warp's run (`in`), from the runs' maps, the tiles before and the group before.
//   needs     the tile's first row continues a segment that began in tile `from` (both uniform in the block)
// Publishes the tile's map and, in a group's last tile, the state after it.  False: give up.
template <int V>
__device__ __forceinline__ bool enter(const ScanParams& p, TileSmem<V>& sh, int tile, int col, bool needs, int from,
                                      const float (&A)[V], const float (&B)[V], bool reset, float (&in)[V]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wide = p.cols * 32 * V, ch = col * 32 * V + lane * V;
  const int group = tile / kGroup, g0 = group * kGroup;
  const bool last_of_group = tile == g0 + kGroup - 1 && tile + 1 < p.tiles;
#pragma unroll
  for (int i = 0; i < V; ++i) sh.run[warp][lane * V + i] = make_float2(A[i], B[i]);
  if (lane == 0) sh.reset[warp] = reset;
  __syncthreads();
  // the tile's map, and whether it replaces the state
  float tA[V], tB[V];
  bool treset = false;
  for (int w = 0; w < kWarps; ++w) treset |= sh.reset[w] != 0;
  if (warp == 0 && tile + 1 < p.tiles) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      tA[i] = 1.f, tB[i] = 0.f;
      for (int w = 0; w < kWarps; ++w) {
        const float2 m = sh.run[w][lane * V + i];
        tB[i] = sh.reset[w] ? m.y : fmaf(m.x, tB[i], m.y);
        tA[i] = sh.reset[w] ? 0.f : m.x * tA[i];
      }
      __stcg(p.agg + static_cast<int64_t>(tile) * wide + ch + i, make_float2(tA[i], tB[i]));
      if (last_of_group && treset) __stcg(p.carry + static_cast<int64_t>(group) * wide + ch + i, tB[i]);
    }
    __threadfence();
    __syncwarp();
    if (lane == 0) {
      st_release(p.flags + static_cast<int64_t>(tile) * p.cols + col, 1);
      if (last_of_group && treset) st_release(p.flags + static_cast<int64_t>(p.tiles + group) * p.cols + col, 1);
    }
  }
  float state[V] = {};
  if (needs) {
    const int lo = max(g0, from), n = tile - lo, per = (n + kWarps - 1) / kWarps;
    const int t0 = lo + warp * per, t1 = min(t0 + per, tile);
    bool ok = true;
    if (lane < t1 - t0) ok = wait_flag(p.flags + static_cast<int64_t>(t0 + lane) * p.cols + col, p.status);
    if (warp == kWarps - 1 && lane == 31 && from < g0)
      ok = wait_flag(p.flags + static_cast<int64_t>(p.tiles + group - 1) * p.cols + col, p.status);
    if (!__all_sync(0xffffffffu, ok)) sh.give_up = 1;
    __syncwarp();
    float pA[V], pB[V];
#pragma unroll
    for (int i = 0; i < V; ++i) pA[i] = 1.f, pB[i] = 0.f;
    for (int t = t0; t < t1; ++t)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 m = __ldcg(p.agg + static_cast<int64_t>(t) * wide + ch + i);
        pB[i] = fmaf(m.x, pB[i], m.y);
        pA[i] *= m.x;
      }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sh.part[warp][lane * V + i] = make_float2(pA[i], pB[i]);
      if (warp == kWarps - 1)
        sh.carry[lane * V + i] = from < g0 ? __ldcg(p.carry + static_cast<int64_t>(group - 1) * wide + ch + i) : 0.f;
    }
    __syncthreads();
    if (sh.give_up) return false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      state[i] = sh.carry[lane * V + i];
      for (int w = 0; w < kWarps; ++w) {
        const float2 m = sh.part[w][lane * V + i];
        if (w * per < n) state[i] = fmaf(m.x, state[i], m.y);
      }
    }
    if (warp == 0 && last_of_group && !treset) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        __stcg(p.carry + static_cast<int64_t>(group) * wide + ch + i, fmaf(tA[i], state[i], tB[i]));
      __threadfence();
      __syncwarp();
      if (lane == 0) st_release(p.flags + static_cast<int64_t>(p.tiles + group) * p.cols + col, 1);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    in[i] = state[i];
    for (int w = 0; w < warp; ++w) {
      const float2 m = sh.run[w][lane * V + i];
      in[i] = sh.reset[w] ? m.y : fmaf(m.x, in[i], m.y);
    }
  }
  return true;
}

// The tile's number in the scan's order, row tile by row tile.
template <int V>
__device__ __forceinline__ int take_number(const ScanParams& p, TileSmem<V>& sh) {
  if (threadIdx.x == 0) {
    sh.number = atomicAdd(p.ticket, 1);
    sh.give_up = 0;
  }
  __syncthreads();
  return sh.number;
}

}  // namespace

// Checks the boundary contract (block 0) and clears the flags and the tile counter.
__global__ void __launch_bounds__(kPrepThreads) scan_prep_kernel(const ScanParams p, int nflags) {
  griddep_begin();
  for (int i = blockIdx.x * kPrepThreads + threadIdx.x; i < nflags; i += gridDim.x * kPrepThreads) p.flags[i] = 0;
  if (blockIdx.x != 0) return;
  int bad = 0;
  for (int b = threadIdx.x; b < p.B; b += kPrepThreads) bad |= p.cu[b + 1] <= p.cu[b];
  if (threadIdx.x == 0) {
    bad |= p.cu[0] != 0 || p.cu[p.B] != p.T;
    *p.ticket = 0;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *p.status = bad ? VA_ERR_BAD_SEQLENS : VA_OK;
}

template <class TX, class TG, class TH, int V>
__global__ void __launch_bounds__(kThreads, 2) scan_fwd_kernel(const ScanParams p) {
  griddep_begin();
  __shared__ TileSmem<V> sh;
  if (*reinterpret_cast<volatile int32_t*>(p.status) == VA_ERR_BAD_SEQLENS) return;
  const int number = take_number(p, sh);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = number / p.cols, col = number % p.cols;
  const int row0 = tile * kTileRows, row = row0 + warp * kRows, ch = (col * 32 + lane) * V;
  const int n = min(kRows, max(0, p.T - row));  // rows of this run
  const bool on = ch < p.D;
  const TX* x = static_cast<const TX*>(p.x) + row * p.x_rs + ch;
  const TG* g = static_cast<const TG*>(p.g) + row * p.g_rs + ch;
  Pack<TX, V> xs[kRows];
  Pack<TG, V> gs[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (on && r < n) {
      xs[r] = load_pack<TX, V>(x + r * p.x_rs);
      gs[r] = load_pack<TG, V>(g + r * p.g_rs);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) xs[r].set(i, 0.f), gs[r].set(i, 0.f);
    }
  }
  const int b0 = first_at(p.cu, p.B, row);
  const uint32_t starts = n > 0 ? starts_mask<kRows>(p.cu, p.B, b0, row) & bits_below(n) : 0;  // (cu[B] = T is none)
  const auto h0 = [&](int r, float (&v)[V]) {
    const int b = b0 + __popc(starts & bits_below(r));
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p.h0 && on ? p.h0[static_cast<int64_t>(b) * p.D + ch + i] : 0.f;
  };
  float A[V], B[V];
#pragma unroll
  for (int i = 0; i < V; ++i) A[i] = B[i] = 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const bool start = (starts >> r) & 1u;
    if (start) h0(r, B);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float gv = gs[r][i];
      A[i] += gv;
      // (a start without h0: x itself, whatever its decay is)
      B[i] = start && !p.h0 ? xs[r][i] : fmaf(decay(gv), B[i], xs[r][i]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) A[i] = starts ? 0.f : run_decay(A[i]);
  // The segment that the tile's first row continues (uniform in the block).
  const int f = warp == 0 ? b0 : first_at(p.cu, p.B, row0);
  const bool needs = p.cu[f] != row0;
  const int from = needs ? p.cu[f - 1] / kTileRows : tile;
  float h[V];
  if (!enter<V>(p, sh, tile, col, needs, from, A, B, starts != 0, h)) return;
  const uint32_t ends = n > 0 ? starts_mask<kRows>(p.cu, p.B, b0 + (starts & 1u), row + 1) : 0;
  TH* out = static_cast<TH*>(p.out) + row * p.out_rs + ch;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const bool start = (starts >> r) & 1u;
    if (start) h0(r, h);
    Pack<TH, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] = start && !p.h0 ? xs[r][i] : fmaf(decay(gs[r][i]), h[i], xs[r][i]);
      o.set(i, h[i]);
    }
    if (on && r < n) store_pack(out + r * p.out_rs, o);
    if (p.last && on && r < n && ((ends >> r) & 1u)) {
      const int b = b0 + __popc(starts & bits_below(r + 1)) - 1;
#pragma unroll
      for (int i = 0; i < V; ++i) p.last[static_cast<int64_t>(b) * p.D + ch + i] = h[i];
    }
  }
}

// TX: dx, TG: g and dg, TH: dh and h.
template <class TX, class TG, class TH, int V>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(const ScanParams p) {
  griddep_begin();
  __shared__ TileSmem<V> sh;
  if (*reinterpret_cast<volatile int32_t*>(p.status) == VA_ERR_BAD_SEQLENS) return;
  const int number = take_number(p, sh);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = number / p.cols, col = number % p.cols;  // tile 0 holds the last rows
  const int row0 = (p.tiles - 1 - tile) * kTileRows, row = row0 + (kWarps - 1 - warp) * kRows;
  const int ch = (col * 32 + lane) * V;
  const int n = min(kRows, max(0, p.T - row));
  const bool on = ch < p.D;
  const TH* dh = static_cast<const TH*>(p.x) + row * p.x_rs + ch;
  const TG* g = static_cast<const TG*>(p.g) + row * p.g_rs + ch;
  const TH* h = static_cast<const TH*>(p.h) + row * p.h_rs + ch;
  Pack<TH, V> ds[kRows], hs[kRows];
  Pack<TG, V> gs[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (on && r < n) {
      ds[r] = load_pack<TH, V>(dh + r * p.x_rs);
      gs[r] = load_pack<TG, V>(g + r * p.g_rs);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) ds[r].set(i, 0.f), gs[r].set(i, 0.f);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {  // the row before
    if (on && r < n && row + r > 0) hs[r] = load_pack<TH, V>(h + (r - 1) * p.h_rs);
    else
#pragma unroll
      for (int i = 0; i < V; ++i) hs[r].set(i, 0.f);
  }
  const int b0 = first_at(p.cu, p.B, row);
  const uint32_t starts = n > 0 ? starts_mask<kRows>(p.cu, p.B, b0, row) & bits_below(n) : 0;
  const uint32_t ends = n > 0 ? starts_mask<kRows>(p.cu, p.B, b0 + (starts & 1u), row + 1) : 0;
  const auto seg = [&](int r) { return b0 + __popc(starts & bits_below(r + 1)) - 1; };  // row r's segment
  const auto row_of = [&](const float* s, int r, float (&v)[V]) {
    const int64_t at = static_cast<int64_t>(seg(r)) * p.D + ch;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = s && on ? s[at + i] : 0.f;
  };
  float A[V], B[V];
#pragma unroll
  for (int i = 0; i < V; ++i) A[i] = B[i] = 0.f;
#pragma unroll
  for (int r = kRows - 1; r >= 0; --r) {
    if ((ends >> r) & 1u) row_of(p.dlast, r, B);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float gv = gs[r][i];
      A[i] += gv;
      B[i] = decay(gv) * (ds[r][i] + B[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) A[i] = ends ? 0.f : run_decay(A[i]);
  // The segment that goes on behind the tile's last row (uniform in the block).
  const int end = row0 + kTileRows;
  const int f = first_at(p.cu, p.B, min(end, p.T));
  const bool needs = end < p.T && p.cu[f] != end;
  const int from = needs ? p.tiles - 1 - (p.cu[f] - 1) / kTileRows : tile;
  float c[V];
  if (!enter<V>(p, sh, tile, col, needs, from, A, B, ends != 0, c)) return;
  TX* dx = static_cast<TX*>(p.out) + row * p.out_rs + ch;
  TG* dg = static_cast<TG*>(p.dg) + row * p.dg_rs + ch;
#pragma unroll
  for (int r = kRows - 1; r >= 0; --r) {
    const bool start = (starts >> r) & 1u;
    if ((ends >> r) & 1u) row_of(p.dlast, r, c);
    float hp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) hp[i] = hs[r][i];
    if (start) row_of(p.h0, r, hp);
    Pack<TX, V> ox;
    Pack<TG, V> og;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float e = ds[r][i] + c[i];
      c[i] = decay(gs[r][i]) * e;
      ox.set(i, e);
      og.set(i, start && !p.h0 ? 0.f : c[i] * hp[i]);
    }
    if (on && r < n) {
      store_pack(dx + r * p.out_rs, ox);
      store_pack(dg + r * p.dg_rs, og);
      if (p.last && start) {
        const int64_t at = static_cast<int64_t>(seg(r)) * p.D + ch;
#pragma unroll
        for (int i = 0; i < V; ++i) p.last[at + i] = c[i];
      }
    }
  }
}

// Single tokens: h = exp(g) h0 + x, one element vector a thread.  Block (0, 0) checks the boundaries for the
// status word; a row whose own are wrong is left out.
template <class TX, class TG, class TH, int V>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanParams p) {
  griddep_begin();
  const int ch = (blockIdx.y * 64 + (threadIdx.x & 63)) * V;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row < p.T && ch < p.D && p.cu[row] == row && p.cu[row + 1] == row + 1) {
    const Pack<TX, V> x = load_pack<TX, V>(static_cast<const TX*>(p.x) + row * p.x_rs + ch);
    float h[V];
    if (p.h0) {
      const Pack<TG, V> g = load_pack<TG, V>(static_cast<const TG*>(p.g) + row * p.g_rs + ch);
      const float* h0 = p.h0 + static_cast<int64_t>(row) * p.D + ch;
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = fmaf(decay(g[i]), h0[i], x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = x[i];
    }
    Pack<TH, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.set(i, h[i]);
    store_pack(static_cast<TH*>(p.out) + row * p.out_rs + ch, o);
    if (p.last)
#pragma unroll
      for (int i = 0; i < V; ++i) p.last[static_cast<int64_t>(row) * p.D + ch + i] = h[i];
  }
  if (blockIdx.x != 0 || blockIdx.y != 0) return;
  int bad = 0;
  for (int b = threadIdx.x; b <= p.B; b += 256) bad |= p.cu[b] != b;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *p.status = bad ? VA_ERR_BAD_SEQLENS : VA_OK;
}

// ---------------------------------------------------------------- host side

namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Layout {
  int64_t tiles, cols, groups, width;
  size_t flags, agg, carry, total;
};

Layout layout_of(int T, int D, int V) {
  Layout l;
  l.width = 32 * V;
  l.tiles = (static_cast<int64_t>(T) + kTileRows - 1) / kTileRows;
  l.cols = (static_cast<int64_t>(D) + l.width - 1) / l.width;
  l.groups = (l.tiles + kGroup - 1) / kGroup;
  l.flags = sizeof(WsHeader);
  l.agg = align256(l.flags + (l.tiles + l.groups) * l.cols * sizeof(int32_t));
  l.carry = align256(l.agg + l.tiles * l.cols * l.width * sizeof(float2));
  l.total = align256(l.carry + l.groups * l.cols * l.width * sizeof(float));
  return l;
}

// Two channels a lane where every row starts on a boundary of two elements, else one.
template <class T>
bool even(const void* p, int64_t rs) {
  return (reinterpret_cast<uintptr_t>(p) & (2 * sizeof(T) - 1)) == 0 && rs % 2 == 0;
}

void place(ScanParams& p, const Layout& l, void* ws) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  WsHeader* h = reinterpret_cast<WsHeader*>(w);
  p.status = &h->status;
  p.ticket = &h->counter[0];
  p.flags = reinterpret_cast<int32_t*>(w + l.flags);
  p.agg = reinterpret_cast<float2*>(w + l.agg);
  p.carry = reinterpret_cast<float*>(w + l.carry);
  p.tiles = static_cast<int>(l.tiles);
  p.cols = static_cast<int>(l.cols);
}

cudaError_t launch_prep(const ScanParams& p, const Layout& l, cudaStream_t st) {
  const int nflags = static_cast<int>((l.tiles + l.groups) * l.cols);
  const int blocks = 1 + std::min(15, nflags / (4 * kPrepThreads));
  return launch_pdl(scan_prep_kernel, dim3(blocks), dim3(kPrepThreads), 0, st, p, nflags);
}

template <class TX, class TG, class TH>
cudaError_t run_fwd(int stage, ScanParams p, void* ws, cudaStream_t st) {
  const bool two = p.D % 2 == 0 && even<TX>(p.x, p.x_rs) && even<TG>(p.g, p.g_rs) && even<TH>(p.out, p.out_rs);
  const Layout l = layout_of(p.T, p.D, two ? 2 : 1);
  place(p, l, ws);
  if (stage == 0) return launch_prep(p, l, st);
  const dim3 grid(static_cast<unsigned>(l.tiles * l.cols));
  return two ? launch_pdl(scan_fwd_kernel<TX, TG, TH, 2>, grid, dim3(kThreads), 0, st, p)
             : launch_pdl(scan_fwd_kernel<TX, TG, TH, 1>, grid, dim3(kThreads), 0, st, p);
}

template <class TX, class TG, class TH>
cudaError_t run_bwd(int stage, ScanParams p, void* ws, cudaStream_t st) {
  const bool two = p.D % 2 == 0 && even<TH>(p.x, p.x_rs) && even<TG>(p.g, p.g_rs) && even<TH>(p.h, p.h_rs) &&
                   even<TX>(p.out, p.out_rs) && even<TG>(p.dg, p.dg_rs);
  const Layout l = layout_of(p.T, p.D, two ? 2 : 1);
  place(p, l, ws);
  if (stage == 0) return launch_prep(p, l, st);
  const dim3 grid(static_cast<unsigned>(l.tiles * l.cols));
  return two ? launch_pdl(scan_bwd_kernel<TX, TG, TH, 2>, grid, dim3(kThreads), 0, st, p)
             : launch_pdl(scan_bwd_kernel<TX, TG, TH, 1>, grid, dim3(kThreads), 0, st, p);
}

template <class TX, class TG, class TH>
cudaError_t run_step(ScanParams p, void* ws, cudaStream_t st) {
  const bool two = p.D % 2 == 0 && even<TX>(p.x, p.x_rs) && even<TG>(p.g, p.g_rs) && even<TH>(p.out, p.out_rs);
  p.status = &static_cast<WsHeader*>(ws)->status;
  const int V = two ? 2 : 1;
  const dim3 grid((p.T + 3) / 4, (p.D + 64 * V - 1) / (64 * V));
  return two ? launch_pdl(scan_step_kernel<TX, TG, TH, 2>, grid, dim3(256), 0, st, p)
             : launch_pdl(scan_step_kernel<TX, TG, TH, 1>, grid, dim3(256), 0, st, p);
}

using bf16 = __nv_bfloat16;

}  // namespace

// (one channel a lane needs no more than two do: as many maps, twice the flags)
size_t scan_workspace(int T, int D) { return std::max(layout_of(T, D, 1).total, layout_of(T, D, 2).total); }

cudaError_t launch_scan_fwd(int stage, ScanParams p, int xb, int gb, void* ws, cudaStream_t st) {
  if (xb && gb) return run_fwd<bf16, bf16, bf16>(stage, p, ws, st);
  return xb ? run_fwd<bf16, float, float>(stage, p, ws, st) : run_fwd<float, float, float>(stage, p, ws, st);
}

cudaError_t launch_scan_bwd(int stage, ScanParams p, int xb, int gb, void* ws, cudaStream_t st) {
  if (xb && gb) return run_bwd<bf16, bf16, bf16>(stage, p, ws, st);
  return xb ? run_bwd<bf16, float, float>(stage, p, ws, st) : run_bwd<float, float, float>(stage, p, ws, st);
}

cudaError_t launch_scan_step(ScanParams p, int xb, int gb, void* ws, cudaStream_t st) {
  if (xb && gb) return run_step<bf16, bf16, bf16>(p, ws, st);
  return xb ? run_step<bf16, float, float>(p, ws, st) : run_step<float, float, float>(p, ws, st);
}

}  // namespace va
