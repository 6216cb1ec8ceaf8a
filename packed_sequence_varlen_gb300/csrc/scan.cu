// Gated linear recurrence over the packed stream, and its gradient.
//
//   h_t = a_t h_{t-1} + x_t,  a_t = exp(g_t),  per channel, restarted at every segment from h0 (or 0)
// Backward, from behind:  e_t = dh_t + f_{t+1},  f_t = a_t e_t,  dx_t = e_t,  dg_t = f_t h_{t-1}, where f_{t+1} is
// the last state's gradient (or 0) at a segment's last row, and f at its first row is h0's gradient.
//
// Both are one scan of affine maps c -> A c + B along the rows (forward: the state; backward: f, rows in
// descending order).  A tile is W runs of R rows by 32 V channels, a run a warp:
//   pass 1  the run's map from zero (A = exp(sum of g), B by the recurrence),
//   the runs' maps are combined in the block; the tile's map is published,
//   the state that enters the tile is folded from the maps of the tiles before it in its group of kGroup and
//   the state after the group before that one, which that group's last tile publishes,
//   pass 2  the recurrence again from the state that enters the run, with the outputs.
// So the data is read once and written once.  A tile's data is copied to shared memory asynchronously, each thread its own
// part, a few tiles ahead.  The fold's order is fixed by the tile's number, whatever is finished first, so results do
// not change from call to call.  A block takes its tiles' numbers from a counter, so every tile that is waited for is
// a running block's, whatever else the GPU does, and the smallest unfinished one waits for nobody.  What is published is
// its own flag: the places hold a NaN of all ones before, which is never written (no fences, and a single trip to L2
// where it is there).  A segment's start (backward: its end) inside a run replaces the state instead of multiplying
// it by zero, so nothing of another segment gets in, infinities and NaN included, and no tile waits across one.
//
// A = exp(sum of g), rounded once, and not the product of the a: the approximate exponential of an a near 1 has a
// bias, which would add up over thousands of rows (h off by 2e-5 for a decay of 0.9995 a row).
#include <algorithm>

#include "elem.cuh"
#include "scan.cuh"
#include "sm100_ptx.cuh"

namespace va {

namespace {

constexpr int kGroup = 32;  // tiles that share a published state
constexpr int kPrepThreads = 1024;
// Buffers of run maps: a slow warp may still read those of the tile before while a fast one, past a single barrier,
// writes those of the tile after.
constexpr int kRings = 3;

// How a block works: W warps, each with a run of R rows of 32 V channels; S tiles on their way or in work.
// kMost: blocks an SM (shared memory may allow fewer).
template <int V_, int W_, int R_, int S_, int M_>
struct Shape {
  static constexpr int V = V_, W = W_, R = R_, S = S_, kThreads = 32 * W_, kRows = W_ * R_, kWidth = 32 * V_, kMost = M_;
};

template <int BYTES>
__device__ __forceinline__ void copy_piece(void* to, const void* from) {
  if constexpr (BYTES >= 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(BYTES) : "memory");
  } else {
    *static_cast<volatile uint16_t*>(to) = *static_cast<const uint16_t*>(from);
  }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

__device__ __forceinline__ float decay(float g) { return fast_exp2(g * kLog2e); }
// A run's decay, rounded once.
__device__ __forceinline__ float run_decay(float sum) { return 1.f + expm1f(sum); }

constexpr uint32_t kNone = 0xffffffffu;  // a place that nothing has been published in

__device__ __forceinline__ float published(float x) {
  return __float_as_uint(x) == kNone ? __uint_as_float(0x7fffffffu) : x;
}

// N words that another block publishes, N 1, 2, 4 or 8.
template <int N>
__device__ __forceinline__ void peek(const float* p, float (&v)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3])
                   : "l"(p + i)
                   : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p) : "memory");
  } else {
    asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v[0]) : "l"(p) : "memory");
  }
}
template <int N>
__device__ __forceinline__ void show(float* p, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p + i), "f"(published(v[i])) : "memory");
}
template <int N>
__device__ __forceinline__ bool there(const float (&v)[N]) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < N; ++i) ok &= __float_as_uint(v[i]) != kNone;
  return ok;
}

// Waits until the N words of every lane that asks are there (a warp's call); false when the call is to be given up.
template <int N>
__device__ __forceinline__ bool await(const float* p, bool ask, float (&v)[N], int32_t* status) {
  if (ask) peek<N>(p, v);
  if (__all_sync(0xffffffffu, !ask || there<N>(v))) return true;
  const uint64_t t0 = sm100::globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (ask) peek<N>(p, v);
    if (__all_sync(0xffffffffu, !ask || there<N>(v))) return true;
    if ((i & 63u) == 0) {
      bool stop = *reinterpret_cast<volatile int32_t*>(status) != VA_OK;
      if (!stop && sm100::globaltimer() - t0 > sm100::kTimeoutNs) {
        atomicCAS(status, 0, VA_ERR_TIMEOUT);
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}

// What the warps of a block exchange; channel = lane * V + i of the tile's columns.
template <class C>
struct TileSmem {
  alignas(16) float2 run[kRings][C::W][C::kWidth];  // the runs' maps
  alignas(16) float2 part[C::W][C::kWidth];         // the folds of the tiles before
  alignas(16) float carry[C::kWidth];               // the state after the group before
  int reset[kRings][C::W];              // the run replaces the state
  int number[2];
  int give_up;
};

// A tile as a warp sees it: its run's rows and the segments in them.
struct Run {
  int tile, col;      // in the scan's order; tile < 0: none
  int row, n, ch;     // first row, rows, first channel of the lane
  int b0;             // the first segment that starts at `row` or later
  uint32_t starts, ends;
  bool needs, on;     // the tile goes on with a segment that began in tile `from`
  int from;
};

template <class C>
__device__ __forceinline__ Run locate(const ScanParams& p, int number, bool back) {
  Run t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  t.tile = -1;
  if (number >= p.tiles * p.cols) return t;
  t.tile = number / p.cols;
  t.col = number - t.tile * p.cols;
  const int row0 = (back ? p.tiles - 1 - t.tile : t.tile) * C::kRows;
  t.row = row0 + (back ? C::W - 1 - warp : warp) * C::R;
  t.n = min(C::R, max(0, p.T - t.row));
  t.ch = (t.col * 32 + lane) * C::V;
  t.on = t.ch < p.D;
  return t;
}

// Where a tile's segments are looked up: the first segment that starts at a run's first row or later (b0), and at the
// row where the scan enters the tile, from the back behind it (f); then boundaries around them.
struct Hint {
  int b0, f;
};
struct Edges {
  int at, cf, before;  // cu[b0 + lane], cu[f], cu[f - 1]
};
template <class C>
__device__ __forceinline__ Hint hint_of(const ScanParams& p, const Run& t, bool back) {
  Hint h{0, 0};
  if (t.tile < 0) return h;
  const int rt = back ? p.tiles - 1 - t.tile : t.tile, warp = threadIdx.x >> 5;
  h.b0 = p.first[rt * C::W + (back ? C::W - 1 - warp : warp)];
  h.f = p.first[(rt + (back ? 1 : 0)) * C::W];
  return h;
}
__device__ __forceinline__ Edges edges_of(const ScanParams& p, const Hint& h) {
  const int lane = threadIdx.x & 31;
  return Edges{p.cu[min(h.b0 + lane, p.B)], p.cu[h.f], p.cu[max(h.f - 1, 0)]};
}

// The segments of a run.
template <class C>
__device__ __forceinline__ void boundaries(const ScanParams& p, Run& t, const Hint& h, const Edges& e, bool back) {
  static_assert(C::R < 32, "a run's boundaries are looked at by one warp");
  const int lane = threadIdx.x & 31, d = h.b0 + lane <= p.B ? e.at - t.row : -1;
  t.b0 = h.b0;
  t.starts = __reduce_or_sync(0xffffffffu, d >= 0 && d < t.n ? 1u << d : 0u);  // (cu[B] = T is none: d = n)
  t.ends = __reduce_or_sync(0xffffffffu, d >= 1 && d <= t.n ? 1u << (d - 1) : 0u);
  const int enter = back ? (p.tiles - t.tile) * C::kRows : t.tile * C::kRows;  // backward: the row behind the tile
  t.needs = enter < p.T && e.cf != enter;
  t.from = !t.needs ? t.tile : back ? p.tiles - 1 - (e.cf - 1) / C::kRows : e.before / C::kRows;
}

// Row r's segment.
__device__ __forceinline__ int segment_of(const Run& t, int r) { return t.b0 + __popc(t.starts & bits_below(r + 1)) - 1; }

// A row of states for the lane's channels (zeros without them).
template <int V>
__device__ __forceinline__ void state_row(const float* s, int64_t at, bool on, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = s && on ? s[at + i] : 0.f;
}

template <class C>
__device__ __forceinline__ bool last_of_group(const ScanParams& p, const Run& t) {
  return t.tile % kGroup == kGroup - 1 && t.tile + 1 < p.tiles;
}

// Warp 0, behind the barrier of the runs' maps: publishes the tile's map, and the state after a group's last tile
// where a segment's boundary in it makes that known already.
template <class C>
__device__ __forceinline__ void publish(const ScanParams& p, const TileSmem<C>& sh, int ring, const Run& t) {
  constexpr int V = C::V;
  const int lane = threadIdx.x & 31;
  if (t.tile < 0 || t.tile + 1 >= p.tiles) return;
  const int64_t wide = static_cast<int64_t>(p.cols) * C::kWidth, at = t.tile * wide + t.ch;
  bool reset = false;
  float A[V], B[V];
#pragma unroll
  for (int i = 0; i < V; ++i) A[i] = 1.f, B[i] = 0.f;
#pragma unroll
  for (int w = 0; w < C::W; ++w) {
    const bool rw = sh.reset[ring][w] != 0;
    reset |= rw;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 m = sh.run[ring][w][lane * V + i];
      B[i] = rw ? m.y : fmaf(m.x, B[i], m.y);
      A[i] = rw ? 0.f : m.x * A[i];
    }
  }
  float m[2 * V];
#pragma unroll
  for (int i = 0; i < V; ++i) m[2 * i] = A[i], m[2 * i + 1] = B[i];
  show<2 * V>(p.agg + 2 * at, m);
  if (reset && last_of_group<C>(p, t)) show<V>(p.carry + (t.tile / kGroup) * wide + t.ch, B);
}

// The state that enters this warp's run, from the tiles before, the group before and the runs' maps.  False: give up.
template <class C>
__device__ __forceinline__ bool enter(const ScanParams& p, TileSmem<C>& sh, int ring, const Run& t, float (&in)[C::V]) {
  constexpr int V = C::V, W = C::W;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t wide = static_cast<int64_t>(p.cols) * C::kWidth;
#pragma unroll
  for (int i = 0; i < V; ++i) in[i] = 0.f;
  if (t.needs) {
    const int group = t.tile / kGroup, g0 = group * kGroup;
    const int lo = max(g0, t.from), n = t.tile - lo, per = (n + W - 1) / W;
    const int t0 = lo + warp * per, t1 = min(t0 + per, t.tile);
    float A[V], B[V];
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = 1.f, B[i] = 0.f;
    bool ok = true;
    for (int k = t0; k < t1; ++k) {
      float m[2 * V];
      ok &= await<2 * V>(p.agg + 2 * (k * wide + t.ch), true, m, p.status);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        B[i] = fmaf(m[2 * i], B[i], m[2 * i + 1]);
        A[i] *= m[2 * i];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sh.part[warp][lane * V + i] = make_float2(A[i], B[i]);
    if (warp == W - 1) {
      float c[V] = {};
      ok &= await<V>(p.carry + (group - 1) * wide + t.ch, t.from < g0, c, p.status);
#pragma unroll
      for (int i = 0; i < V; ++i) sh.carry[lane * V + i] = c[i];
    }
    if (!ok) sh.give_up = 1;
    __syncthreads();
    if (sh.give_up) return false;
#pragma unroll
    for (int i = 0; i < V; ++i) in[i] = sh.carry[lane * V + i];
    for (int w = 0; w * per < n; ++w)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 m = sh.part[w][lane * V + i];
        in[i] = fmaf(m.x, in[i], m.y);
      }
  }
  // the runs before; warp 0 goes through all of them for the state after the tile
  bool reset = false;
  float after[V];
#pragma unroll
  for (int i = 0; i < V; ++i) after[i] = in[i];
  const bool last = warp == 0 && t.needs && last_of_group<C>(p, t);
  for (int w = 0; w < (last ? W : warp); ++w) {
    const bool rw = sh.reset[ring][w] != 0;
    reset |= rw;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 m = sh.run[ring][w][lane * V + i];
      after[i] = rw ? m.y : fmaf(m.x, after[i], m.y);
    }
  }
  if (last) {
    if (!reset) show<V>(p.carry + (t.tile / kGroup) * wide + t.ch, after);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) in[i] = after[i];
  }
  return true;
}

// A block's tiles: takes their numbers from the counter, keeps S of them on their way, and forms a tile's maps before it
// finishes the tile before, so that whoever waits for them waits little.  One copy of each part of the work: unrolled over
// the stages the code did not stay in the instruction cache (forward of T = 8192, D = 4096 bf16 211 us).
//   fetch(run, stage)          asks for the run's data        first(run, stage, A, B) -> the run's map, true: it replaces the state
//   second(run, stage, in)     the outputs
template <class C, bool BACK, class Fetch, class First, class Second>
__device__ __forceinline__ void run_tiles(const ScanParams& p, TileSmem<C>& sh, Fetch&& fetch, First&& first,
                                          Second&& second) {
  constexpr int V = C::V, S = C::S;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int total = p.tiles * p.cols;
  // numbers: a block takes more than one at once only where there are several for each
  const int ahead = min(S - 1, max(1, total / static_cast<int>(gridDim.x)));
  if (threadIdx.x == 0) {
    sh.give_up = 0;
    sh.number[1] = atomicAdd(p.ticket, ahead);  // (step 0 writes the other)
  }
  __syncthreads();
  const int base = sh.number[1];  // (written again behind the first step's barrier)
  int ask[S - 1];   // the numbers of this step's tile and those after it; total: none
  Hint hint[S - 1];
#pragma unroll
  for (int k = 0; k < S - 1; ++k) {
    ask[k] = k < ahead ? min(base + k, total) : total;
    const Run t = locate<C>(p, ask[k], BACK);
    if (t.tile >= 0) fetch(t, k);
    hint[k] = hint_of<C>(p, t, BACK);
    copy_commit();
  }
  Edges edges = edges_of(p, hint[0]);
  Run old;
  old.tile = -1;
  int stage = 0, ring = 0;
  // step i: data for tile i + S - 1, maps of tile i, outputs of tile i - 1
#pragma unroll 1
  for (int i = 0;; ++i) {
    bool any = old.tile >= 0;
#pragma unroll
    for (int k = 0; k < S - 1; ++k) any |= ask[k] < total;
    if (!any) return;
    int number = 0;
    if (warp == C::W - 1 && lane == 0) number = atomicAdd(p.ticket, 1);
    Run now = locate<C>(p, ask[0], BACK);
    if (now.tile >= 0) boundaries<C>(p, now, hint[0], edges, BACK);
    edges = edges_of(p, hint[1]);  // the next tile's
    copy_wait<S - 2>();
    if (now.tile >= 0) {
      float A[V], B[V];
      const bool reset = first(now, stage, A, B);
#pragma unroll
      for (int k = 0; k < V; ++k) sh.run[ring][warp][lane * V + k] = make_float2(reset ? 0.f : A[k], B[k]);
      if (lane == 0) sh.reset[ring][warp] = reset;
    }
    if (warp == C::W - 1 && lane == 0) sh.number[i & 1] = number;
    __syncthreads();
    const int next = sh.number[i & 1];
    if (warp == 0) publish<C>(p, sh, ring, now);
    const int free = stage == 0 ? S - 1 : stage - 1;  // the stage of the tile before, this one's turn comes last
    if (old.tile >= 0) {
      float in[V];
      if (!enter<C>(p, sh, ring == 0 ? kRings - 1 : ring - 1, old, in)) return;
      second(old, free, in);
    }
#pragma unroll
    for (int k = 0; k + 1 < S - 1; ++k) ask[k] = ask[k + 1], hint[k] = hint[k + 1];
    ask[S - 2] = min(next, total);
    const Run t = locate<C>(p, ask[S - 2], BACK);
    if (t.tile >= 0) fetch(t, free);
    hint[S - 2] = hint_of<C>(p, t, BACK);
    copy_commit();
    old = now;
    stage = stage + 1 == S ? 0 : stage + 1;
    ring = ring + 1 == kRings ? 0 : ring + 1;
  }
}

}  // namespace

// Checks the boundary contract (block 0), empties the published places and looks up the first segment at every run.
__global__ void __launch_bounds__(kPrepThreads) scan_prep_kernel(const ScanParams p, int rows, int64_t words) {
  griddep_begin();
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPrepThreads;
  for (int64_t i = tid; i < words / 4; i += step)
    reinterpret_cast<uint4*>(p.agg)[i] = make_uint4(kNone, kNone, kNone, kNone);
  for (int64_t i = tid; i < p.runs; i += step) {  // the first b in [0, B] with cu[b] >= row (cu[B] = T)
    const int row = static_cast<int>(min(i * rows, static_cast<int64_t>(p.T)));
    int lo = 0, hi = p.B;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] < row) lo = mid + 1;
      else hi = mid;
    }
    p.first[i] = lo;
  }
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

template <class TX, class TG, class TH, class C>
__global__ void __launch_bounds__(C::kThreads, C::kMost) scan_fwd_kernel(const ScanParams p) {
  griddep_begin();
  constexpr int V = C::V, R = C::R;
  extern __shared__ __align__(16) uint8_t smem[];
  TileSmem<C>& sh = *reinterpret_cast<TileSmem<C>*>(smem);
  if (*reinterpret_cast<volatile int32_t*>(p.status) == VA_ERR_BAD_SEQLENS) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a thread's own pieces of the stages: [stage][warp][row][lane]
  Pack<TX, V>* xs = reinterpret_cast<Pack<TX, V>*>(smem + sizeof(TileSmem<C>)) + warp * R * 32 + lane;
  Pack<TG, V>* gs = reinterpret_cast<Pack<TG, V>*>(smem + sizeof(TileSmem<C>) + sizeof(Pack<TX, V>) * 32 * C::kRows * C::S) +
                    warp * R * 32 + lane;
  constexpr int kStage = 32 * C::kRows;
  const auto fetch = [&](const Run& t, int stage) {
    if (!t.on) return;
    const TX* x = static_cast<const TX*>(p.x) + t.row * p.x_rs + t.ch;
    const TG* g = static_cast<const TG*>(p.g) + t.row * p.g_rs + t.ch;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < t.n) {
        copy_piece<sizeof(TX) * V>(xs + stage * kStage + r * 32, x + r * p.x_rs);
        copy_piece<sizeof(TG) * V>(gs + stage * kStage + r * 32, g + r * p.g_rs);
      }
  };
  const auto step = [&](int at, float (&h)[V], float (&A)[V]) {
    const Pack<TX, V> x = xs[at];
    const Pack<TG, V> g = gs[at];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      A[i] += g[i];
      h[i] = fmaf(decay(g[i]), h[i], x[i]);
    }
  };
  const auto start = [&](const Run& t, int r, int at, float (&h)[V]) {  // a segment's first row
    const Pack<TX, V> x = xs[at];
    const Pack<TG, V> g = gs[at];
    state_row<V>(p.h0, static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch, t.on, h);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = p.h0 ? fmaf(decay(g[i]), h[i], x[i]) : x[i];  // (x itself, whatever its decay is)
  };
  const auto first = [&](const Run& t, int stage, float (&A)[V], float (&B)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = B[i] = 0.f;
    const int at = stage * kStage;
    if (t.starts == 0 && t.n == R) {
#pragma unroll
      for (int r = 0; r < R; ++r) step(at + r * 32, B, A);
    } else {
#pragma unroll 1
      for (int r = 0; r < t.n; ++r) {
        if ((t.starts >> r) & 1u) start(t, r, at + r * 32, B);
        else step(at + r * 32, B, A);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = run_decay(A[i]);
    return t.starts != 0;
  };
  const auto second = [&](const Run& t, int stage, float (&h)[V]) {
    TH* out = static_cast<TH*>(p.out) + t.row * p.out_rs + t.ch;
    const int at = stage * kStage;
    float unused[V] = {};
    const auto put = [&](int r) {
      Pack<TH, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i) o.set(i, h[i]);
      if (t.on) store_pack(out + r * p.out_rs, o);
    };
    if (t.starts == 0 && t.n == R && (!p.last || t.ends == 0)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        step(at + r * 32, h, unused);
        put(r);
      }
    } else {
#pragma unroll 1
      for (int r = 0; r < t.n; ++r) {
        if ((t.starts >> r) & 1u) start(t, r, at + r * 32, h);
        else step(at + r * 32, h, unused);
        put(r);
        if (p.last && t.on && ((t.ends >> r) & 1u)) {
          float* last = p.last + static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch;
#pragma unroll
          for (int i = 0; i < V; ++i) last[i] = h[i];
        }
      }
    }
  };
  run_tiles<C, false>(p, sh, fetch, first, second);
}

// TX: dx, TG: g and dg, TH: dh and h.  Tile 0 holds the last rows, warp 0 a tile's last run.
template <class TX, class TG, class TH, class C>
__global__ void __launch_bounds__(C::kThreads, C::kMost) scan_bwd_kernel(const ScanParams p) {
  griddep_begin();
  constexpr int V = C::V, R = C::R;
  extern __shared__ __align__(16) uint8_t smem[];
  TileSmem<C>& sh = *reinterpret_cast<TileSmem<C>*>(smem);
  if (*reinterpret_cast<volatile int32_t*>(p.status) == VA_ERR_BAD_SEQLENS) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kStage = 32 * C::kRows;
  Pack<TH, V>* ds = reinterpret_cast<Pack<TH, V>*>(smem + sizeof(TileSmem<C>)) + warp * R * 32 + lane;
  Pack<TH, V>* hs = ds + kStage * C::S;
  Pack<TG, V>* gs = reinterpret_cast<Pack<TG, V>*>(smem + sizeof(TileSmem<C>) + 2 * sizeof(Pack<TH, V>) * kStage * C::S) +
                    warp * R * 32 + lane;
  const auto fetch = [&](const Run& t, int stage) {
    if (!t.on) return;
    const TH* dh = static_cast<const TH*>(p.x) + t.row * p.x_rs + t.ch;
    const TH* h = static_cast<const TH*>(p.h) + t.row * p.h_rs + t.ch;
    const TG* g = static_cast<const TG*>(p.g) + t.row * p.g_rs + t.ch;
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
      if (r < t.n) {
        copy_piece<sizeof(TH) * V>(ds + stage * kStage + r * 32, dh + r * p.x_rs);
        copy_piece<sizeof(TG) * V>(gs + stage * kStage + r * 32, g + r * p.g_rs);
        if (t.row + r > 0) copy_piece<sizeof(TH) * V>(hs + stage * kStage + r * 32, h + (r - 1) * p.h_rs);  // the row before
      }
  };
  const auto first = [&](const Run& t, int stage, float (&A)[V], float (&B)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = B[i] = 0.f;
    const int at = stage * kStage;
    const auto step = [&](int r) {
      const Pack<TH, V> d = ds[at + r * 32];
      const Pack<TG, V> g = gs[at + r * 32];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        A[i] += g[i];
        B[i] = decay(g[i]) * (d[i] + B[i]);
      }
    };
    if (t.ends == 0 && t.n == R) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r) step(r);
    } else {
#pragma unroll 1
      for (int r = t.n - 1; r >= 0; --r) {
        if ((t.ends >> r) & 1u) state_row<V>(p.dlast, static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch, t.on, B);
        step(r);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = run_decay(A[i]);
    return t.ends != 0;
  };
  const auto second = [&](const Run& t, int stage, float (&f)[V]) {
    TX* dx = static_cast<TX*>(p.out) + t.row * p.out_rs + t.ch;
    TG* dg = static_cast<TG*>(p.dg) + t.row * p.dg_rs + t.ch;
    const int at = stage * kStage;
    // before: the row before's h, at a segment's first row h0 (none: 0, and so is the decay's gradient)
    const auto step = [&](int r, const float (&before)[V], bool none) {
      const Pack<TH, V> d = ds[at + r * 32];
      const Pack<TG, V> g = gs[at + r * 32];
      Pack<TX, V> ox;
      Pack<TG, V> og;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float e = d[i] + f[i];
        f[i] = decay(g[i]) * e;
        ox.set(i, e);
        og.set(i, none ? 0.f : f[i] * before[i]);
      }
      if (t.on) {
        store_pack(dx + r * p.out_rs, ox);
        store_pack(dg + r * p.dg_rs, og);
      }
    };
    const auto stored = [&](int r, float (&before)[V]) {
      const Pack<TH, V> h = hs[at + r * 32];
#pragma unroll
      for (int i = 0; i < V; ++i) before[i] = h[i];
    };
    float before[V];
    if (t.ends == 0 && t.starts == 0 && t.n == R) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        stored(r, before);
        step(r, before, false);
      }
    } else {
#pragma unroll 1
      for (int r = t.n - 1; r >= 0; --r) {
        const int64_t state = static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch;
        const bool start = (t.starts >> r) & 1u;
        if ((t.ends >> r) & 1u) state_row<V>(p.dlast, state, t.on, f);
        if (start) state_row<V>(p.h0, state, t.on, before);
        else stored(r, before);
        step(r, before, start && !p.h0);
        if (p.last && start && t.on) {
#pragma unroll
          for (int i = 0; i < V; ++i) p.last[state + i] = f[i];
        }
      }
    }
  };
  run_tiles<C, true>(p, sh, fetch, first, second);
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
  int64_t tiles, cols, groups, runs, words;
  size_t first, agg, carry, total;
};

Layout layout_of(int T, int D, int rows, int runs, int width) {
  Layout l;
  l.tiles = (static_cast<int64_t>(T) + rows - 1) / rows;
  l.cols = (static_cast<int64_t>(D) + width - 1) / width;
  l.groups = (l.tiles + kGroup - 1) / kGroup;
  l.runs = (l.tiles + 1) * runs;
  l.first = sizeof(WsHeader);
  l.agg = align256(l.first + l.runs * sizeof(int32_t));
  l.carry = l.agg + l.tiles * l.cols * width * 2 * sizeof(float);  // (follows: both are emptied together)
  l.words = (l.tiles * 2 + l.groups) * l.cols * width;
  l.total = align256(l.agg + l.words * sizeof(float));
  return l;
}

// Whether rows can be read N elements at a time.
template <class T>
bool steps_of(const void* p, int64_t rs, int N) {
  return (reinterpret_cast<uintptr_t>(p) & (N * sizeof(T) - 1)) == 0 && rs % N == 0;
}

void place(ScanParams& p, const Layout& l, void* ws) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  WsHeader* h = reinterpret_cast<WsHeader*>(w);
  p.status = &h->status;
  p.ticket = &h->counter[0];
  p.first = reinterpret_cast<int32_t*>(w + l.first);
  p.agg = reinterpret_cast<float*>(w + l.agg);
  p.carry = reinterpret_cast<float*>(w + l.carry);
  p.tiles = static_cast<int>(l.tiles);
  p.cols = static_cast<int>(l.cols);
  p.runs = l.runs;
}

using bf16 = __nv_bfloat16;

int device_sms() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return std::max(sms, 1);
}

// The call's blocks, as many as fit, each with S tiles in shared memory.
template <class C>
cudaError_t run_blocks(int stage, void (*kernel)(ScanParams), size_t piece, ScanParams p, void* ws, cudaStream_t st) {
  const Layout l = layout_of(p.T, p.D, C::kRows, C::W, C::kWidth);
  place(p, l, ws);
  const int sms = device_sms();
  if (stage == 0) {
    const int64_t work = std::max(l.words / 8, l.runs);
    const int blocks = static_cast<int>(std::min<int64_t>(2 * sms, (work + kPrepThreads - 1) / kPrepThreads));
    return launch_pdl(scan_prep_kernel, dim3(blocks), dim3(kPrepThreads), 0, st, p, C::R, l.words);
  }
  const size_t smem = sizeof(TileSmem<C>) + piece * 32 * C::kRows * C::S;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t fit = std::max<int64_t>(1, std::min<int64_t>((227 * 1024) / (smem + 1024), C::kMost));
  const int grid = static_cast<int>(std::min<int64_t>(l.tiles * l.cols, sms * fit));
  return launch_pdl(kernel, dim3(grid), dim3(C::kThreads), smem, st, p);
}

template <class TX, class TG, class TH, class C>
cudaError_t blocks_fwd(int stage, const ScanParams& p, void* ws, cudaStream_t st) {
  return run_blocks<C>(stage, scan_fwd_kernel<TX, TG, TH, C>, (sizeof(TX) + sizeof(TG)) * C::V, p, ws, st);
}
template <class TX, class TG, class TH, class C>
cudaError_t blocks_bwd(int stage, const ScanParams& p, void* ws, cudaStream_t st) {
  return run_blocks<C>(stage, scan_bwd_kernel<TX, TG, TH, C>, (2 * sizeof(TH) + sizeof(TG)) * C::V, p, ws, st);
}

constexpr bool kWide = false;
template <int V> using FwdShape = Shape<V, 8, 16, 3, 2>;
template <int V> using BwdShape = Shape<V, 8, 8, 3, 2>;

// Channels a lane (8 bytes of the widest type where the rows allow it), runs of 16 or 8 rows.
template <class TX, class TG, class TH>
cudaError_t run_fwd(int stage, const ScanParams& p, void* ws, cudaStream_t st) {
  const auto can = [&](int N) {
    return p.D % N == 0 && steps_of<TX>(p.x, p.x_rs, N) && steps_of<TG>(p.g, p.g_rs, N) && steps_of<TH>(p.out, p.out_rs, N);
  };
  if constexpr (sizeof(TH) == 2) {
    if (can(4) && kWide) return blocks_fwd<TX, TG, TH, FwdShape<4>>(stage, p, ws, st);
  }
  return can(2) ? blocks_fwd<TX, TG, TH, FwdShape<2>>(stage, p, ws, st)
                : blocks_fwd<TX, TG, TH, FwdShape<1>>(stage, p, ws, st);
}

template <class TX, class TG, class TH>
cudaError_t run_bwd(int stage, const ScanParams& p, void* ws, cudaStream_t st) {
  const auto can = [&](int N) {
    return p.D % N == 0 && steps_of<TH>(p.x, p.x_rs, N) && steps_of<TG>(p.g, p.g_rs, N) && steps_of<TH>(p.h, p.h_rs, N) &&
           steps_of<TX>(p.out, p.out_rs, N) && steps_of<TG>(p.dg, p.dg_rs, N);
  };
  if constexpr (sizeof(TH) == 2) {
    if (can(4) && kWide) return blocks_bwd<TX, TG, TH, BwdShape<4>>(stage, p, ws, st);
  }
  return can(2) ? blocks_bwd<TX, TG, TH, BwdShape<2>>(stage, p, ws, st)
                : blocks_bwd<TX, TG, TH, BwdShape<1>>(stage, p, ws, st);
}

template <class TX, class TG, class TH>
cudaError_t run_step(ScanParams p, void* ws, cudaStream_t st) {
  const bool two =
      p.D % 2 == 0 && steps_of<TX>(p.x, p.x_rs, 2) && steps_of<TG>(p.g, p.g_rs, 2) && steps_of<TH>(p.out, p.out_rs, 2);
  p.status = &static_cast<WsHeader*>(ws)->status;
  const int V = two ? 2 : 1;
  const dim3 grid((p.T + 3) / 4, (p.D + 64 * V - 1) / (64 * V));
  return two ? launch_pdl(scan_step_kernel<TX, TG, TH, 2>, grid, dim3(256), 0, st, p)
             : launch_pdl(scan_step_kernel<TX, TG, TH, 1>, grid, dim3(256), 0, st, p);
}

}  // namespace

size_t scan_workspace(int T, int D) {
  size_t n = 0;
  for (int rows : {16, 32, 64, 128})
    for (int width : {32, 64, 128}) n = std::max(n, layout_of(T, D, rows, 16, width).total);
  return n;
}

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
