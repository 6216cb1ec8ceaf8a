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
//   the state that enters the tile is folded from the maps of a few tiles before it and a state further back, which
//   every kGroup-th tile publishes,
//   pass 2  the recurrence again from the state that enters the run, with the outputs.
// So the data is read once and written once.  A warp of its own takes the tiles' numbers, looks their segments up and has
// their data copied to shared memory (TMA), a few tiles ahead of the others.  (Rows that are not on 16-byte boundaries are
// read by the others straight from memory, twice.)  The fold's order is fixed by the tile's number, whatever is finished
// first, so results do not change from call to call.  A block takes its tiles' numbers from a counter, so every tile that
// is waited for is a running block's, whatever else the GPU does, and the smallest unfinished one waits for nobody.
// What is published is its own flag: the places hold a NaN of all ones before, which is never written (no fences, and a
// single trip to L2 where it is there).  A segment's start (backward: its end) inside a run replaces the state instead of multiplying
// it by zero, so nothing of another segment gets in, infinities and NaN included, and no tile waits across one.
//
// A = exp(sum of g), rounded once, and not the product of the a: the approximate exponential of an a near 1 has a
// bias, which would add up over thousands of rows (h off by 2e-5 for a decay of 0.9995 a row).
#include <algorithm>

#include "elem.cuh"
#include "scan.cuh"
#include "sm100_ptx.cuh"
#include "tmap.cuh"
#include "vec.cuh"

namespace va {

namespace {

// The last tile of every kGroup publishes the state after it.  A tile folds the maps of the kBack groups before its own
// and of those before it in its own, onto the state before them, which has long been there (its own group's of 32
// tiles, whose start was formed beside it: T = 65536 in one segment, D = 2048 in bf16, backward 363 us; 352 this way).
constexpr int kGroup = 8, kBack = 2;
constexpr int kPrepThreads = 1024;
// Buffers of run maps: a slow warp may still read those of the tile before while a fast one, past a single barrier,
// writes those of the tile after.
constexpr int kRings = 3;

// How a block works: W warps, each with a run of R rows of 32 V channels; S tiles on their way or in work; at most M
// blocks an SM (shared memory may allow fewer).
template <int V_, int W_, int R_, int S_, int M_>
struct Shape {
  static constexpr int V = V_, W = W_, R = R_, S = S_, M = M_;
  static constexpr int kThreads = 32 * (W_ + 1), kRows = W_ * R_, kWidth = 32 * V_, kWords = kRows / 32 + 1;
};

template <int V>
__device__ __forceinline__ Vec<V> decay(const Vec<V>& g) {
  Vec<V> r = mul(g, fill<V>(kLog2e));
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = fast_exp2(r[i]);
  return r;
}
__device__ __forceinline__ float decay(float g) { return fast_exp2(__fmul_rn(g, kLog2e)); }
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
__device__ __forceinline__ bool await(const float* p, bool ask, float (&v)[N], const ScanParams& c) {
  if (ask) peek<N>(p, v);
  if (__all_sync(0xffffffffu, !ask || there<N>(v))) return true;
  const uint64_t t0 = sm100::globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (ask) peek<N>(p, v);
    if (__all_sync(0xffffffffu, !ask || there<N>(v))) return true;
    if ((i & 63u) == 0) {
      bool stop = *reinterpret_cast<volatile int32_t*>(&c.hdr->status) != VA_OK;
      if (!stop && sm100::globaltimer() - t0 > (c.wait_ns ? c.wait_ns : sm100::kTimeoutNs)) {
        set_status(c.hdr, VA_ERR_TIMEOUT);
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}

// A tile as the copying warp leaves it for the others.
template <class C>
struct Slot {
  int tile, col;            // in the scan's order; tile < 0: no more
  int b0;                   // the first segment that starts at the tile's first row or later
  int needs, from;          // the tile goes on with a segment that began in tile `from`
  uint32_t bits[C::kWords]; // bit i: a segment starts at (or the stream ends before) the tile's row i, i <= kRows
};

// What the warps of a block share; channel = lane * V + i of the tile's columns.
template <class C>
struct TileSmem {
  alignas(16) float2 run[kRings][C::W][C::kWidth];  // the runs' maps
  alignas(16) float2 part[C::W][C::kWidth];         // the folds of the tiles before
  alignas(16) float carry[C::kWidth];               // the state after the group before
  uint64_t full[C::S], empty[C::S];
  int reset[kRings][C::W];                          // the run replaces the state
  Slot<C> slot[C::S];
  int stop_first, stop_enter;                       // a wait gave up, before a step's first or second barrier
  alignas(8) int pad;
  int abort_flag;                                   // (followed by its wait limit)
  uint64_t wait_limit;
};

// A tile as a warp sees it: its run's rows and the segments in them.
struct Run {
  int tile, col;
  int row, n, ch;   // first row, rows, first channel of the lane
  int b0;           // the first segment that starts at `row` or later
  uint32_t starts, ends;
  bool needs, on;
  int from;
};

template <class C>
__device__ __forceinline__ Run run_of(const ScanParams& p, const Slot<C>& s, bool back) {
  Run t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  t.tile = s.tile;
  t.col = s.col;
  t.needs = s.needs != 0;
  t.from = s.from;
  const int at = (back ? C::W - 1 - warp : warp) * C::R;  // the run's rows in the tile
  t.row = (back ? p.tiles - 1 - t.tile : t.tile) * C::kRows + at;
  t.n = min(C::R, max(0, p.T - t.row));
  t.ch = (t.col * 32 + lane) * C::V;
  t.on = t.ch < p.D;
  static_assert(32 % C::R == 0 && C::R < 32, "a run's rows lie in one word");
  const uint32_t word = s.bits[at >> 5] >> (at & 31);
  const uint32_t next = ((at + C::R) & 31) ? s.bits[at >> 5] >> ((at & 31) + C::R) : s.bits[(at + C::R) >> 5];
  t.starts = word & bits_below(t.n);                                     // (the stream's end is none)
  t.ends = ((word >> 1) | (next & 1u) << (C::R - 1)) & bits_below(t.n);  // a segment starts behind the row
  t.b0 = s.b0;
  for (int w = 0; w <= at >> 5; ++w) t.b0 += __popc(s.bits[w] & (w < at >> 5 ? ~0u : bits_below(at & 31)));
  return t;
}

// Row r's segment.
__device__ __forceinline__ int segment_of(const Run& t, int r) { return t.b0 + __popc(t.starts & bits_below(r + 1)) - 1; }

// A row of states for the lane's channels (zeros without them).
template <int V>
__device__ __forceinline__ Vec<V> state_row(const float* s, int64_t at, bool on) {
  Vec<V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = s && on ? s[at + i] : 0.f;
  return v;
}

template <class C>
__device__ __forceinline__ bool last_of_group(const ScanParams& p, const Run& t) {
  return t.tile % kGroup == kGroup - 1 && t.tile + 1 < p.tiles;
}

template <class C>
__device__ __forceinline__ void worker_sync() {  // the warps that compute
  asm volatile("bar.sync 1, %0;" ::"n"(32 * C::W) : "memory");
}

// Warp 0, behind the barrier of the runs' maps: publishes the tile's map, and the state after a group's last tile
// where a segment's boundary in it makes that known already.
template <class C>
__device__ __forceinline__ void publish(const ScanParams& p, const TileSmem<C>& sh, int ring, const Run& t) {
  constexpr int V = C::V;
  const int lane = threadIdx.x & 31;
  if (t.tile < 0 || t.tile + 1 >= p.tiles || (p.wait_ns && t.tile == 0)) return;
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

// The maps that a warp folds for a tile, asked for before there is other work to do.
template <class C>
struct Look {
  static constexpr int kMost = ((kBack + 1) * kGroup + C::W - 1) / C::W;
  float m[kMost][2 * C::V], c[C::V];
};
// The tiles before `t` whose maps it folds: [lo, lo + n), `per` a warp; onto the state after group `state`, or onto
// nothing (-1) where its segment began in one of them.
struct Span {
  int lo, n, per, t0, t1, state;
};
template <class C>
__device__ __forceinline__ Span span_of(const Run& t) {
  Span s;
  const int g = t.tile / kGroup - kBack;
  s.state = t.from < g * kGroup ? g - 1 : -1;
  s.lo = max(max(g, 0) * kGroup, t.from);
  s.n = t.tile - s.lo;
  s.per = (s.n + C::W - 1) / C::W;
  s.t0 = s.lo + (threadIdx.x >> 5) * s.per;
  s.t1 = min(s.t0 + s.per, t.tile);
  return s;
}
template <class C>
__device__ __forceinline__ const float* map_place(const ScanParams& p, const Run& t, int tile) {
  return p.agg + 2 * (tile * (static_cast<int64_t>(p.cols) * C::kWidth) + t.ch);
}
template <class C>
__device__ __forceinline__ float* state_place(const ScanParams& p, const Run& t, int group) {
  return p.carry + group * (static_cast<int64_t>(p.cols) * C::kWidth) + t.ch;
}
template <class C>
__device__ __forceinline__ void ask(const ScanParams& p, const Run& t, Look<C>& l) {
  if (t.tile < 0 || !t.needs) return;
  const Span s = span_of<C>(t);
#pragma unroll
  for (int k = 0; k < Look<C>::kMost; ++k)
    if (s.t0 + k < s.t1) peek<2 * C::V>(map_place<C>(p, t, s.t0 + k), l.m[k]);
  if ((threadIdx.x >> 5) == C::W - 1 && s.state >= 0) peek<C::V>(state_place<C>(p, t, s.state), l.c);
}

// The state that enters this warp's run, from the tiles before, the group before and the runs' maps.  False: give up.
template <class C>
__device__ __forceinline__ bool enter(const ScanParams& p, TileSmem<C>& sh, int ring, const Run& t, Look<C>& l,
                                      Vec<C::V>& in) {
  constexpr int V = C::V, W = C::W;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  in = fill<V>(0.f);
  if (t.needs) {
    const Span s = span_of<C>(t);
    Vec<V> A = fill<V>(1.f), B = fill<V>(0.f);
    bool ok = true;
#pragma unroll
    for (int k = 0; k < Look<C>::kMost; ++k)
      if (s.t0 + k < s.t1) {
        if (!__all_sync(0xffffffffu, there<2 * V>(l.m[k])))
          ok &= await<2 * V>(map_place<C>(p, t, s.t0 + k), true, l.m[k], p);
        Vec<V> mA, mB;
#pragma unroll
        for (int i = 0; i < V; ++i) mA[i] = l.m[k][2 * i], mB[i] = l.m[k][2 * i + 1];
        B = fma(mA, B, mB);
        A = mul(A, mA);
      }
#pragma unroll
    for (int i = 0; i < V; ++i) sh.part[warp][lane * V + i] = make_float2(A[i], B[i]);
    if (warp == W - 1) {
      if (s.state >= 0 && !__all_sync(0xffffffffu, there<V>(l.c)))
        ok &= await<V>(state_place<C>(p, t, s.state), true, l.c, p);
#pragma unroll
      for (int i = 0; i < V; ++i) sh.carry[lane * V + i] = s.state >= 0 ? l.c[i] : 0.f;
    }
    if (!ok) sh.stop_enter = 1;
    worker_sync<C>();
    if (sh.stop_enter) return false;
#pragma unroll
    for (int i = 0; i < V; ++i) in[i] = sh.carry[lane * V + i];
    for (int w = 0; w * s.per < s.n; ++w) {
      Vec<V> mA, mB;
#pragma unroll
      for (int i = 0; i < V; ++i) mA[i] = sh.part[w][lane * V + i].x, mB[i] = sh.part[w][lane * V + i].y;
      in = fma(mA, in, mB);
    }
  }
  // the runs before; warp 0 goes through all of them for the state after the tile
  bool reset = false;
  Vec<V> after = in;
  const bool last = warp == 0 && t.needs && last_of_group<C>(p, t);
  for (int w = 0; w < (last ? W : warp); ++w) {
    const bool rw = sh.reset[ring][w] != 0;
    reset |= rw;
    Vec<V> mA, mB;
#pragma unroll
    for (int i = 0; i < V; ++i) mA[i] = sh.run[ring][w][lane * V + i].x, mB[i] = sh.run[ring][w][lane * V + i].y;
    after = rw ? mB : fma(mA, after, mB);
  }
  if (last) {
    if (!reset) show<V>(state_place<C>(p, t, t.tile / kGroup), after.e);
  } else {
    in = after;
  }
  return true;
}

// Tiles for each block (with a single one, or one and a few over, a block finishes it before it takes another).
__device__ __forceinline__ int tiles_each(const ScanParams& p) {
  return max(1, p.tiles * p.cols / static_cast<int>(gridDim.x));
}

// The copying warp: takes the tiles' numbers, looks their segments up, asks for their data.
//   load(tile, col, stage): one lane's, issues the copies that complete on full[stage] (kBytes in all)
template <class C, bool BACK, int kBytes, class Load>
__device__ __forceinline__ void feed(const ScanParams& p, TileSmem<C>& sh, Load&& load) {
  using namespace sm100;
  constexpr int S = C::S;
  const int lane = threadIdx.x & 31, total = p.tiles * p.cols;
  const int most = min(S, tiles_each(p));  // a block's tiles at a time
  volatile int* abort_flag = &sh.abort_flag;
  // a tile's number, and its segments: where the scan enters it (backward: behind it), and the starts in it
  int number = 0, tile = 0, col = 0, row0 = 0, b0 = 0, from = 0, needs = 0;
  uint32_t bits = 0;  // lane i: word i
  const auto take = [&] {
    if (lane == 0) number = atomicAdd(p.ticket, 1);
    number = __shfl_sync(0xffffffffu, number, 0);
    if (number >= total) return;
    tile = number / p.cols;
    col = number - tile * p.cols;
    const int rt = BACK ? p.tiles - 1 - tile : tile;
    row0 = rt * C::kRows;
    b0 = p.first[rt];
    const int f = BACK ? p.first[rt + 1] : b0, enter = BACK ? row0 + C::kRows : row0;
    const int cf = p.cu[f], before = p.cu[max(f - 1, 0)];
    bits = 0;
    for (int b = b0; b <= p.B; b += 32) {
      const int d = b + lane <= p.B ? p.cu[b + lane] - row0 : C::kRows + 1;
#pragma unroll
      for (int w = 0; w < C::kWords; ++w) {
        const uint32_t word = __reduce_or_sync(0xffffffffu, d >> 5 == w && d <= C::kRows ? 1u << (d & 31) : 0u);
        if (lane == w) bits |= word;
      }
      if (__any_sync(0xffffffffu, d > C::kRows)) break;
    }
    needs = enter < p.T && cf != enter;
    from = !needs ? tile : BACK ? p.tiles - 1 - (cf - 1) / C::kRows : before / C::kRows;
  };
  int issued = 0;
  bool ok = true;
  if (most > 1) take();  // a tile ahead of the place for it
  for (int j = 0;; ++j) {
    const int s = j % S;
    if (j >= most) ok = wwait(smem_u32(&sh.empty[(j - most) % S]), ((j - most) / S) & 1, abort_flag, p.hdr, 71);
    if (!ok) break;
    if (most == 1) take();
    Slot<C>& slot = sh.slot[s];
    if (number >= total) {
      if (lane == 0) {
        slot.tile = -1;
        mbar_arrive(smem_u32(&sh.full[s]));
        mbar_arrive(smem_u32(&sh.full[s]));
      }
      return;
    }
    if (lane == 0) {
      if constexpr (kBytes > 0) {
        mbar_expect_tx(smem_u32(&sh.full[s]), kBytes);
        load(row0, col * C::kWidth, s);
      } else {
        mbar_arrive(smem_u32(&sh.full[s]));
      }
      slot.tile = tile;
      slot.col = col;
      slot.b0 = b0;
      slot.needs = needs;
      slot.from = from;
    }
    issued = j + 1;
    if (lane < C::kWords) slot.bits[lane] = bits;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.full[s]));
    if (most > 1) take();
  }
  // given up: the copies on their way land before the block ends (bounded again)
  if constexpr (kBytes > 0) {
    const uint64_t t0 = globaltimer();
    for (int j = max(0, issued - S); j < issued; ++j)
      while (!mbar_try_wait(smem_u32(&sh.full[j % S]), (j / S) & 1) && globaltimer() - t0 < 50000000ull) {
      }
  }
}

// The other warps: form a tile's maps before they finish the tile before, so that whoever waits for them waits little.
//   first(run, stage, A, B)    the run's map, true: it replaces the state        second(run, stage, in)   the outputs
// (One copy of each part of the work: unrolled over the stages the code left the instruction cache; the forward of
// T = 8192, D = 4096 in bf16 took 211 us.)
template <class C, bool BACK, class First, class Second>
__device__ __forceinline__ void work(const ScanParams& p, TileSmem<C>& sh, First&& first, Second&& second) {
  using namespace sm100;
  constexpr int V = C::V, S = C::S;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  volatile int* abort_flag = &sh.abort_flag;
  Run old;
  old.tile = -1;
  int stage = 0, parity = 0, ring = 0, held = 0;
  const bool single = tiles_each(p) == 1;
#pragma unroll 1
  for (;;) {
    const bool ok = wwait(smem_u32(&sh.full[stage]), parity, abort_flag, p.hdr, 72);
    Run now;
    now.tile = -1;
    if (ok) {
      if (sh.slot[stage].tile >= 0) now = run_of<C>(p, sh.slot[stage], BACK);
    } else {
      sh.stop_first = 1;
    }
    Look<C> look;
    ask<C>(p, old, look);
    if (now.tile >= 0) {
      Vec<V> A, B;
      const bool reset = first(now, stage, A, B);
#pragma unroll
      for (int k = 0; k < V; ++k) sh.run[ring][warp][lane * V + k] = make_float2(reset ? 0.f : A[k], B[k]);
      if (lane == 0) sh.reset[ring][warp] = reset;
    }
    worker_sync<C>();
    if (sh.stop_first) break;
    if (warp == 0) publish<C>(p, sh, ring, now);
    if (single) {
      old = now;
      held = stage;
      ask<C>(p, old, look);
    }
    if (old.tile >= 0) {
      Vec<V> in;
      if (!enter<C>(p, sh, single ? ring : ring == 0 ? kRings - 1 : ring - 1, old, look, in)) break;
      second(old, held, in);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[held]));
    }
    if (now.tile < 0) return;
    old = now;
    if (single) old.tile = -1;
    held = stage;
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
    ring = ring + 1 == kRings ? 0 : ring + 1;
  }
  sh.abort_flag = 1;  // given up: the copying warp stops too
}

// Runs a block's warps.
template <class C, bool BACK, int kBytes, class Load, class First, class Second>
__device__ __forceinline__ void run_block(const ScanParams& p, TileSmem<C>& sh, Load&& load, First&& first,
                                          Second&& second) {
  using namespace sm100;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 2);  // the data's bytes, the slot
      mbar_init(smem_u32(&sh.empty[s]), C::W);
    }
    fence_barrier_init();
    sh.stop_first = sh.stop_enter = sh.abort_flag = 0;
    sh.wait_limit = p.wait_ns ? p.wait_ns : kTimeoutNs;
  }
  __syncthreads();
  if (threadIdx.x >= 32 * C::W) feed<C, BACK, kBytes>(p, sh, load);
  else work<C, BACK>(p, sh, first, second);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// Where a run's rows are read: its tile's copy, or memory.
template <class T, class C, bool TMA>
struct Rows {
  static constexpr int kRun = C::R;
  const T* base;       // the thread's first element of stage 0, or of the tensor
  int64_t step;        // between rows
  __device__ __forceinline__ Rows(const uint8_t* smem, const void* global, int64_t rs) {
    const int lane = threadIdx.x & 31;
    base = TMA ? reinterpret_cast<const T*>(smem) + lane * C::V : static_cast<const T*>(global);
    step = TMA ? C::kWidth : rs;
  }
  // the run's first row
  __device__ __forceinline__ const T* at(const Run& t, int stage, bool back) const {
    const int warp = threadIdx.x >> 5;
    if (TMA) return base + (stage * C::kRows + (back ? C::W - 1 - warp : warp) * C::R) * C::kWidth;
    return base + t.row * step + t.ch;
  }
  __device__ __forceinline__ Pack<T, C::V> get(const T* first, int r, const Run& t) const {
    if constexpr (TMA) {
      return load_pack<T, C::V>(first + r * C::kWidth);
    } else {
      Pack<T, C::V> none;
#pragma unroll
      for (int i = 0; i < C::V; ++i) none.set(i, 0.f);
      return t.on ? load_pack<T, C::V>(first + r * step) : none;
    }
  }
};

// Rows of a run that holds a segment's boundary or the stream's end, in order or from the back.  From the copied tile one
// after another; from memory all of them are asked for first.
template <bool TMA, bool BACK = false, class A, class PA, class B, class PB, class F>
__device__ __forceinline__ void rows_of(const A& a, PA pa, const B& b, PB pb, const Run& t, F&& f) {
  constexpr int R = A::kRun;
  if constexpr (TMA) {
#pragma unroll 1
    for (int i = 0; i < t.n; ++i) {
      const int r = BACK ? t.n - 1 - i : i;
      f(r, a.get(pa, r, t), b.get(pb, r, t));
    }
  } else {
    decltype(a.get(pa, 0, t)) va[R];
    decltype(b.get(pb, 0, t)) vb[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < t.n) {
        va[r] = a.get(pa, r, t);
        vb[r] = b.get(pb, r, t);
      }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = BACK ? R - 1 - i : i;
      if (r < t.n) f(r, va[r], vb[r]);
    }
  }
}

// Bytes of a tile of one tensor.
template <class T, class C> constexpr int tile_bytes() { return C::kRows * C::kWidth * static_cast<int>(sizeof(T)); }
template <class C> constexpr int head_bytes() { return (static_cast<int>(sizeof(TileSmem<C>)) + 127) / 128 * 128; }

struct Maps {
  CUtensorMap a, b, c;  // forward: x, g; backward: dh, g, h
};

}  // namespace

// Checks the boundary contract (block 0), empties the published places and looks up the first segment at every tile.
__global__ void __launch_bounds__(kPrepThreads) scan_prep_kernel(const ScanParams p, int rows, int64_t words) {
  griddep_begin();
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPrepThreads;
  for (int64_t i = tid; i < words / 4; i += step)
    reinterpret_cast<uint4*>(p.agg)[i] = make_uint4(kNone, kNone, kNone, kNone);
  for (int64_t i = tid; i <= p.tiles; i += step) {  // the first b in [0, B] with cu[b] >= row (cu[B] = T)
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
  if (threadIdx.x == 0) p.hdr->status = bad ? VA_ERR_BAD_SEQLENS : VA_OK;
}

template <class TX, class TG, class TH, class C, bool TMA>
__global__ void __launch_bounds__(C::kThreads, C::M)
    scan_fwd_kernel(const ScanParams p, const __grid_constant__ Maps maps) {
  griddep_begin();
  constexpr int V = C::V, R = C::R;
  extern __shared__ __align__(128) uint8_t smem[];
  TileSmem<C>& sh = *reinterpret_cast<TileSmem<C>*>(smem);
  if (*reinterpret_cast<volatile int32_t*>(&p.hdr->status) == VA_ERR_BAD_SEQLENS) return;
  constexpr int kX = tile_bytes<TX, C>(), kG = tile_bytes<TG, C>();
  uint8_t* const x_smem = smem + head_bytes<C>();
  uint8_t* const g_smem = x_smem + kX * C::S;
  const Rows<TX, C, TMA> xs(x_smem, p.x, p.x_rs);
  const Rows<TG, C, TMA> gs(g_smem, p.g, p.g_rs);
  const auto load = [&](int row0, int ch0, int stage) {
    const uint32_t bar = smem_u32(&sh.full[stage]);
    tma_load_2d(smem_u32(x_smem + stage * kX), &maps.a, bar, ch0, row0);
    tma_load_2d(smem_u32(g_smem + stage * kG), &maps.b, bar, ch0, row0);
  };
  const auto step = [&](const Pack<TX, V>& x, const Vec<V>& g, Vec<V>& h) { h = fma(decay(g), h, wide_of(x)); };
  const auto start = [&](const Pack<TX, V>& x, const Vec<V>& g, const Run& t, int r, Vec<V>& h) {  // a segment's first row
    h = wide_of(x);  // (x itself without h0, whatever its decay is)
    if (p.h0) h = fma(decay(g), state_row<V>(p.h0, static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch, t.on), h);
  };
  const auto first = [&](const Run& t, int stage, Vec<V>& A, Vec<V>& B) {
    A = B = fill<V>(0.f);
    const TX* const xa = xs.at(t, stage, false);
    const TG* const ga = gs.at(t, stage, false);
    if (t.starts == 0 && t.n == R) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const Vec<V> g = wide_of(gs.get(ga, r, t));
        A = add(A, g);
        step(xs.get(xa, r, t), g, B);
      }
    } else {
      rows_of<TMA>(xs, xa, gs, ga, t, [&](int r, const Pack<TX, V>& x, const Pack<TG, V>& gr) {
        const Vec<V> g = wide_of(gr);
        A = add(A, g);
        if ((t.starts >> r) & 1u) start(x, g, t, r, B);
        else step(x, g, B);
      });
    }
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = run_decay(A[i]);
    return t.starts != 0;
  };
  const auto second = [&](const Run& t, int stage, Vec<V>& h) {
    TH* out = static_cast<TH*>(p.out) + t.row * p.out_rs + t.ch;
    const TX* const xa = xs.at(t, stage, false);
    const TG* const ga = gs.at(t, stage, false);
    if (t.starts == 0 && t.n == R && (!p.last || t.ends == 0)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        step(xs.get(xa, r, t), wide_of(gs.get(ga, r, t)), h);
        if (t.on) store_pack(out + r * p.out_rs, narrow<TH, V>(h));
      }
    } else {
      rows_of<TMA>(xs, xa, gs, ga, t, [&](int r, const Pack<TX, V>& x, const Pack<TG, V>& gr) {
        const Vec<V> g = wide_of(gr);
        if ((t.starts >> r) & 1u) start(x, g, t, r, h);
        else step(x, g, h);
        if (t.on) store_pack(out + r * p.out_rs, narrow<TH, V>(h));
        if (p.last && t.on && ((t.ends >> r) & 1u)) {
          float* last = p.last + static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch;
#pragma unroll
          for (int i = 0; i < V; ++i) last[i] = h[i];
        }
      });
    }
  };
  run_block<C, false, TMA ? kX + kG : 0>(p, sh, load, first, second);
}

// TX: dx, TG: g and dg, TH: dh and h.  Tile 0 holds the last rows, warp 0 a tile's last run.
template <class TX, class TG, class TH, class C, bool TMA>
__global__ void __launch_bounds__(C::kThreads, C::M)
    scan_bwd_kernel(const ScanParams p, const __grid_constant__ Maps maps) {
  griddep_begin();
  constexpr int V = C::V, R = C::R;
  extern __shared__ __align__(128) uint8_t smem[];
  TileSmem<C>& sh = *reinterpret_cast<TileSmem<C>*>(smem);
  if (*reinterpret_cast<volatile int32_t*>(&p.hdr->status) == VA_ERR_BAD_SEQLENS) return;
  constexpr int kH = tile_bytes<TH, C>(), kG = tile_bytes<TG, C>();
  uint8_t* const d_smem = smem + head_bytes<C>();
  uint8_t* const g_smem = d_smem + kH * C::S;
  uint8_t* const h_smem = g_smem + kG * C::S;
  const Rows<TH, C, TMA> ds(d_smem, p.x, p.x_rs), hs(h_smem, p.h, p.h_rs);
  const Rows<TG, C, TMA> gs(g_smem, p.g, p.g_rs);
  const auto load = [&](int row0, int ch0, int stage) {
    const uint32_t bar = smem_u32(&sh.full[stage]);
    tma_load_2d(smem_u32(d_smem + stage * kH), &maps.a, bar, ch0, row0);
    tma_load_2d(smem_u32(g_smem + stage * kG), &maps.b, bar, ch0, row0);
    tma_load_2d(smem_u32(h_smem + stage * kH), &maps.c, bar, ch0, row0 - 1);  // the rows before (zeros before the first)
  };
  const auto first = [&](const Run& t, int stage, Vec<V>& A, Vec<V>& B) {
    A = B = fill<V>(0.f);
    const TH* const da = ds.at(t, stage, true);
    const TG* const ga = gs.at(t, stage, true);
    const auto step = [&](const Pack<TH, V>& d, const Pack<TG, V>& gr) {
      const Vec<V> g = wide_of(gr);
      A = add(A, g);
      B = mul(decay(g), add(wide_of(d), B));
    };
    if (t.ends == 0 && t.n == R) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r) step(ds.get(da, r, t), gs.get(ga, r, t));
    } else {
      rows_of<TMA, true>(ds, da, gs, ga, t, [&](int r, const Pack<TH, V>& d, const Pack<TG, V>& g) {
        if ((t.ends >> r) & 1u) B = state_row<V>(p.dlast, static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch, t.on);
        step(d, g);
      });
    }
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = run_decay(A[i]);
    return t.ends != 0;
  };
  const auto second = [&](const Run& t, int stage, Vec<V>& f) {
    TX* dx = static_cast<TX*>(p.out) + t.row * p.out_rs + t.ch;
    TG* dg = static_cast<TG*>(p.dg) + t.row * p.dg_rs + t.ch;
    const TH* const da = ds.at(t, stage, true);
    const TG* const ga = gs.at(t, stage, true);
    const TH* const ha = hs.at(t, stage, true) - (TMA ? 0 : p.h_rs);
    // before: the row before's h, at a segment's first row h0 (none: 0, and so is the decay's gradient)
    const auto step = [&](int r, const Pack<TH, V>& d, const Pack<TG, V>& g, const Vec<V>& before, bool none) {
      const Vec<V> e = add(wide_of(d), f);
      f = mul(decay(wide_of(g)), e);
      const Vec<V> q = none ? fill<V>(0.f) : mul(f, before);
      if (t.on) {
        store_pack(dx + r * p.out_rs, narrow<TX, V>(e));
        store_pack(dg + r * p.dg_rs, narrow<TG, V>(q));
      }
    };
    if (t.ends == 0 && t.starts == 0 && t.n == R) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r)
        step(r, ds.get(da, r, t), gs.get(ga, r, t), wide_of(hs.get(ha, r, t)), false);
    } else {
      rows_of<TMA, true>(ds, da, gs, ga, t, [&](int r, const Pack<TH, V>& d, const Pack<TG, V>& g) {
        const int64_t state = static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch;
        const bool start = (t.starts >> r) & 1u;
        if ((t.ends >> r) & 1u) f = state_row<V>(p.dlast, state, t.on);
        const Vec<V> before = start ? state_row<V>(p.h0, state, t.on) : wide_of(hs.get(ha, r, t));
        step(r, d, g, before, start && !p.h0);
        if (p.last && start && t.on) {
#pragma unroll
          for (int i = 0; i < V; ++i) p.last[state + i] = f[i];
        }
      });
    }
  };
  run_block<C, true, TMA ? 2 * kH + kG : 0>(p, sh, load, first, second);
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
  if (blockIdx.x != 0 || blockIdx.y != 0 || !p.hdr) return;
  int bad = 0;
  for (int b = threadIdx.x; b <= p.B; b += 256) bad |= p.cu[b] != b;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.hdr->status = bad ? VA_ERR_BAD_SEQLENS : VA_OK;
}

// ---------------------------------------------------------------- host side

namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Layout {
  int64_t tiles, cols, groups, words;
  size_t first, agg, carry, total;
};

Layout layout_of(int T, int D, int rows, int width) {
  Layout l;
  l.tiles = (static_cast<int64_t>(T) + rows - 1) / rows;
  l.cols = (static_cast<int64_t>(D) + width - 1) / width;
  l.groups = (l.tiles + kGroup - 1) / kGroup;
  l.first = sizeof(WsHeader);
  l.agg = align256(l.first + (l.tiles + 1) * sizeof(int32_t));
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
  p.hdr = h;
  p.ticket = &h->counter[0];
  p.first = reinterpret_cast<int32_t*>(w + l.first);
  p.agg = reinterpret_cast<float*>(w + l.agg);
  p.carry = reinterpret_cast<float*>(w + l.carry);
  p.tiles = static_cast<int>(l.tiles);
  p.cols = static_cast<int>(l.cols);
}

using bf16 = __nv_bfloat16;

template <class T>
bool rows16(const void* p, int64_t rs) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && rs * static_cast<int64_t>(sizeof(T)) % 16 == 0;
}

// The call's blocks, as many as fit, each with S tiles of `piece` bytes in shared memory.
template <class C>
cudaError_t run_blocks(int stage, void (*kernel)(ScanParams, Maps), size_t piece, ScanParams p, const Maps& maps, void* ws,
                       cudaStream_t st) {
  const Layout l = layout_of(p.T, p.D, C::kRows, C::kWidth);
  place(p, l, ws);
  const int sms = device_sms();
  if (stage == 0) {
    const int64_t work = std::max(l.words / 8, l.tiles + 1);
    const int blocks = static_cast<int>(std::min<int64_t>(2 * sms, (work + kPrepThreads - 1) / kPrepThreads));
    return launch_pdl(scan_prep_kernel, dim3(blocks), dim3(kPrepThreads), 0, st, p, C::kRows, l.words);
  }
  const size_t smem = head_bytes<C>() + piece * C::S;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t fit = std::max<int64_t>(1, std::min<int64_t>((228 * 1024) / (smem + 1024), C::M));
  const int grid = static_cast<int>(std::min<int64_t>(l.tiles * l.cols, sms * fit));
  return launch_pdl(kernel, dim3(grid), dim3(C::kThreads), smem, st, p, maps);
}

template <int V> using FwdShape = Shape<V, 8, 16, 3, 2>;
// (from memory: short runs, whose rows are all asked for at once)
template <int V> using FwdPlain = Shape<V, 8, 8, 3, 3>;
template <int V> using BwdShape = Shape<V, 8, 8, 3, 2>;
template <int V> using BwdPlain = Shape<V, 8, 8, 3, 3>;

// Two channels a lane where rows lie on boundaries of two elements, else one; copied tiles where they lie on 16 bytes.
template <class TX, class TG, class TH>
cudaError_t run_fwd(int stage, const ScanParams& p, void* ws, cudaStream_t st) {
  using C = FwdShape<2>;
  const bool two =
      p.D % 2 == 0 && steps_of<TX>(p.x, p.x_rs, 2) && steps_of<TG>(p.g, p.g_rs, 2) && steps_of<TH>(p.out, p.out_rs, 2);
  Maps maps{};
  if (!two) return run_blocks<FwdPlain<1>>(stage, scan_fwd_kernel<TX, TG, TH, FwdPlain<1>, false>, 0, p, maps, ws, st);
  if (rows16<TX>(p.x, p.x_rs) && rows16<TG>(p.g, p.g_rs)) {
    if (stage == 1 && !(tmap_matrix(&maps.a, p.x, sizeof(TX) == 2, p.T, p.D, p.x_rs, C::kWidth, C::kRows) &&
                        tmap_matrix(&maps.b, p.g, sizeof(TG) == 2, p.T, p.D, p.g_rs, C::kWidth, C::kRows)))
      return cudaErrorInvalidValue;
    return run_blocks<C>(stage, scan_fwd_kernel<TX, TG, TH, C, true>, tile_bytes<TX, C>() + tile_bytes<TG, C>(), p, maps, ws, st);
  }
  return run_blocks<FwdPlain<2>>(stage, scan_fwd_kernel<TX, TG, TH, FwdPlain<2>, false>, 0, p, maps, ws, st);
}

template <class TX, class TG, class TH>
cudaError_t run_bwd(int stage, const ScanParams& p, void* ws, cudaStream_t st) {
  using C = BwdShape<2>;
  const bool two = p.D % 2 == 0 && steps_of<TH>(p.x, p.x_rs, 2) && steps_of<TG>(p.g, p.g_rs, 2) &&
                   steps_of<TH>(p.h, p.h_rs, 2) && steps_of<TX>(p.out, p.out_rs, 2) && steps_of<TG>(p.dg, p.dg_rs, 2);
  Maps maps{};
  if (!two) return run_blocks<BwdPlain<1>>(stage, scan_bwd_kernel<TX, TG, TH, BwdPlain<1>, false>, 0, p, maps, ws, st);
  if (rows16<TH>(p.x, p.x_rs) && rows16<TG>(p.g, p.g_rs) && rows16<TH>(p.h, p.h_rs)) {
    if (stage == 1 && !(tmap_matrix(&maps.a, p.x, sizeof(TH) == 2, p.T, p.D, p.x_rs, C::kWidth, C::kRows) &&
                        tmap_matrix(&maps.b, p.g, sizeof(TG) == 2, p.T, p.D, p.g_rs, C::kWidth, C::kRows) &&
                        tmap_matrix(&maps.c, p.h, sizeof(TH) == 2, p.T, p.D, p.h_rs, C::kWidth, C::kRows)))
      return cudaErrorInvalidValue;
    return run_blocks<C>(stage, scan_bwd_kernel<TX, TG, TH, C, true>, 2 * tile_bytes<TH, C>() + tile_bytes<TG, C>(), p, maps, ws, st);
  }
  return run_blocks<BwdPlain<2>>(stage, scan_bwd_kernel<TX, TG, TH, BwdPlain<2>, false>, 0, p, maps, ws, st);
}

template <class TX, class TG, class TH>
cudaError_t run_step(ScanParams p, void* ws, cudaStream_t st) {
  const bool two =
      p.D % 2 == 0 && steps_of<TX>(p.x, p.x_rs, 2) && steps_of<TG>(p.g, p.g_rs, 2) && steps_of<TH>(p.out, p.out_rs, 2);
  p.hdr = static_cast<WsHeader*>(ws);
  const int V = two ? 2 : 1;
  const dim3 grid((p.T + 3) / 4, (p.D + 64 * V - 1) / (64 * V));
  return two ? launch_pdl(scan_step_kernel<TX, TG, TH, 2>, grid, dim3(256), 0, st, p)
             : launch_pdl(scan_step_kernel<TX, TG, TH, 1>, grid, dim3(256), 0, st, p);
}

}  // namespace

size_t scan_workspace(int T, int D) {
  size_t n = 0;
  for (int rows : {FwdShape<2>::kRows, FwdPlain<2>::kRows, BwdShape<2>::kRows, BwdPlain<2>::kRows})
    n = std::max({n, layout_of(T, D, rows, 32).total, layout_of(T, D, rows, 64).total});
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
