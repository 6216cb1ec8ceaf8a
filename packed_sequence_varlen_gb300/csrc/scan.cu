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
// So the data is read once and written once.  Four warps of a block serve the ones that work: one takes the tiles'
// numbers, looks their segments up and has their data copied to shared memory, a few tiles ahead (by TMA; rows that do
// not lie on 16-byte boundaries in pieces of 16 bytes, by warps of their own); one folds and publishes the tiles'
// maps; two find the states that enter the tiles while the tiles' own maps are formed.  The fold's order is fixed by
// the tile's number, whatever is finished first, so results do not change from call to call.  A block takes its tiles'
// numbers from a counter, so every tile that is waited for is a running block's, whatever else the GPU does, and the
// smallest unfinished one waits for nobody.  What is published is its own flag: the places hold a NaN of all ones
// before, which is never written (no fences, and a single trip to L2 where it is there).  A segment's start (backward:
// its end) inside a run replaces the state instead of multiplying it by zero, so nothing of another segment gets in,
// infinities and NaN included, and no tile waits across one.
//
// Bound by HBM where there are many rows, else by the trips between tiles: T = 65536, D = 2048, one segment, bf16 158 us
// forward and 276 backward (the bytes at the copy rate: 119, 198), fp32 decays 232 and 417 (198, 357); T = 8192,
// D = 4096, 51 and 75 (30, 50); T = 30000, D = 2047, rows off their boundaries, 151 and 216 (54, 91).
//
// States are fp32 from row to row; h is rounded to the wider type of x and g when stored, which is what the next layer reads
// and half the bytes.  dg takes it as stored: with bf16 h its error is sqrt(2) times its own rounding's (0.0023 of its norm, not
// 0.0017).  A caller may have h and dh in fp32 for that (T = 8192, D = 4096, 57 and 103 us, 40 and 69 by bytes).
//
// A = exp(sum of g) and not the product of the a: the approximate exponential of an a near 1 has a bias, which would
// add up over thousands of rows (h off by 2e-5 for a decay of 0.9995 a row).
#include <algorithm>

#include "elem.cuh"
#include "scan.cuh"
#include "sm100_ptx.cuh"
#include "tmap.cuh"
#include "vec.cuh"

namespace va {

namespace {

// The last tile of every kGroup publishes the state after it.  A tile folds the maps of the kBack groups before its own
// and of those before it in its own, onto the state before them: the further back, the surer it is there, and the
// more there is to fold (T = 65536, D = 2048, one segment, backward, us: with bf16 / fp32 decays kGroup, kBack = 4, 1 295 /
// 423; 4, 2 303 / 425; 8, 1 293 / 416; 8, 2 279 / 413; 8, 3 282 / 433).
constexpr int kGroup = 8, kBack = 2;
constexpr int kPrepThreads = 1024;
// Words of what the first launch looks up for a tile: the first segment that starts at its first row or later, the
// boundary there (backward: behind the tile) or after it and the one before, then a bit for every row that a segment
// starts at, and for the one behind the tile.
constexpr int kRecord = 8;
constexpr int kResolvers = 2;  // warps that find the states that enter a block's tiles, in turn
// Buffers of run maps: a slow warp may still read those of the tile before while a fast one, past a single barrier,
// writes those of the tile after.
constexpr int kRings = 3;

// How a block works: W warps, each with a run of R rows of 32 V channels; S tiles on their way or in work; at most M
// blocks an SM (shared memory may allow fewer); K warps copy where TMA does not.
template <int V_, int W_, int R_, int S_, int M_, int K_ = 0>
struct Shape {
  static constexpr int V = V_, W = W_, R = R_, S = S_, M = M_, K = K_;
  static constexpr int kThreads = 32 * (W_ + 2 + kResolvers + K_), kRows = W_ * R_, kWidth = 32 * V_, kWords = kRows / 32 + 1;
  static_assert(3 + kWords <= kRecord, "a tile's bits fit its record");
};

template <int V>
__device__ __forceinline__ Vec<V> decay(const Vec<V>& g) {
  Vec<V> r = mul(g, fill<V>(kLog2e));
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = fast_exp2(r[i]);
  return r;
}
__device__ __forceinline__ float decay(float g) { return fast_exp2(__fmul_rn(g, kLog2e)); }
// A run's decay exp(sum): sum = k ln 2 + f, |f| <= ln 2 / 2 (Cody and Waite's reduction), 2^k (1 + (f + ... + f^7 / 7!)), the
// Taylor sum's rest below 2^-27 and the addition to 1 its last rounding: within 1.5 half steps over the whole range, so a small
// decay keeps its relative precision, and near 1 without a bias (0.004 half steps), which would add up over a long segment.  (expm1f
// near 1 and expf elsewhere are as exact, but lanes take both paths: T = 8192, D = 4096 bf16 52 and 77 us; so 51 and 75.
// T = 30000, D = 2047 157 and 226; so 151 and 216.)
__device__ __forceinline__ float run_decay(float sum) {
  constexpr float kLn2Lo = static_cast<float>(0.69314718055994531 - static_cast<double>(kLn2)), kWhole = 12582912.f;  // 1.5 2^23
  const float s = sum < -88.f ? -88.f : sum > 89.f ? 89.f : sum;  // (beyond: 0, infinity; NaN is kept)
  const float t = fmaf(s, kLog2e, kWhole), k = t - kWhole;        // t's low bits are k
  const float f = fmaf(-k, kLn2Lo, fmaf(-k, kLn2, s));
  float p = 1.f / 5040.f;
  p = fmaf(p, f, 1.f / 720.f);
  p = fmaf(p, f, 1.f / 120.f);
  p = fmaf(p, f, 1.f / 24.f);
  p = fmaf(p, f, 1.f / 6.f);
  p = fmaf(p, f, 0.5f);
  return (1.f + fmaf(f * f, p, f)) * __uint_as_float((__float_as_uint(t) + 127u) << 23);
}

constexpr uint32_t kNone = 0xffffffffu;  // a place that nothing has been published in

__device__ __forceinline__ float published(float x) {
  return __float_as_uint(x) == kNone ? __uint_as_float(0x7fffffffu) : x;
}

// Words that another block publishes: two channels' maps, or states.
__device__ __forceinline__ void peek(const float* p, float (&v)[4]) {
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void peek(const float* p, float (&v)[2]) {
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p) : "memory");
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

// The waits, bounded; their slow parts in one copy each (the code of a block's warps together has to stay in the
// instruction cache).  Every lane of a warp asks, and gets the same answer.
__device__ __noinline__ bool past_limit(const ScanParams& c, uint64_t since) {
  bool stop = *reinterpret_cast<volatile int32_t*>(&c.hdr->status) != VA_OK;
  if (!stop && sm100::globaltimer() - since > (c.wait_ns ? c.wait_ns : sm100::kTimeoutNs)) {
    set_status(c.hdr, VA_ERR_TIMEOUT);
    stop = true;
  }
  return __any_sync(0xffffffffu, stop);
}
// Asks until what it asks for is there; false when the call is to be given up.
template <class Ask>
__device__ __forceinline__ bool until(const ScanParams& c, Ask&& ask) {
  uint64_t since = 0;
#pragma unroll 1
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xffffffffu, ask())) return true;
    if (i == 0) since = sm100::globaltimer();
    if ((i & 63u) == 63u && past_limit(c, since)) return false;
  }
}
__device__ __noinline__ bool hold_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, WsHeader* hdr, int where) {
  return sm100::wwait(bar, parity, abort_flag, hdr, where);
}
__device__ __forceinline__ bool hold(uint64_t& bar, uint32_t parity, volatile int* abort_flag, WsHeader* hdr, int where) {
  const uint32_t at = smem_u32(&bar);
  if (__all_sync(0xffffffffu, sm100::mbar_try_wait(at, parity))) return true;
  return hold_slow(at, parity, abort_flag, hdr, where);
}

// A tile as the feeding warp leaves it for the others.
template <class C>
struct Slot {
  int tile, col;                       // in the scan's order; tile < 0: no more
  int needs, from;                     // the tile goes on with a segment that began in tile `from`
  int b0[C::W];                        // by run: the first segment that starts at its first row or later,
  uint32_t starts[C::W], ends[C::W];   // bit r: a segment starts at its row r, one ends with it
};

// What the warps of a block share; channel = lane * V + i of the tile's columns.
template <class C>
struct TileSmem {
  alignas(16) float2 run[kRings][C::W][C::kWidth];  // the runs' maps
  alignas(16) float carry[C::S][C::kWidth];         // the state that enters a tile
  uint64_t known[C::S], full[C::S], empty[C::S], carried[C::S];  // the slot, its data too; given back; its state
  int reset[kRings][C::W];                          // the run replaces the state
  Slot<C> slot[C::S];
  int stop[kRings];                                 // a wait gave up before the step's barrier of the runs' maps
  alignas(8) int pad;
  int abort_flag;                                   // (followed by its wait limit)
  uint64_t wait_limit;
};

// A tile as a warp sees it: its run's rows and the segments in them.
struct Run {
  int tile;
  int row, n, ch;   // first row, rows, first channel of the lane
  int b0;           // the first segment that starts at `row` or later
  uint32_t starts, ends;
  int left;         // channels from ch on (none: <= 0)
};

template <class C>
__device__ __forceinline__ Run run_of(const ScanParams& p, const Slot<C>& s, bool back) {
  static_assert(32 % C::R == 0 && C::R < 32 && C::W <= 32, "a run's rows lie in one word, a lane looks a run up");
  Run t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  t.tile = s.tile;
  t.row = (back ? p.tiles - 1 - t.tile : t.tile) * C::kRows + (back ? C::W - 1 - warp : warp) * C::R;
  t.n = min(C::R, max(0, p.T - t.row));
  t.ch = (s.col * 32 + lane) * C::V;
  t.left = p.D - t.ch;
  t.starts = s.starts[warp];
  t.ends = s.ends[warp];
  t.b0 = s.b0[warp];
  return t;
}

// Row r's segment.
__device__ __forceinline__ int segment_of(const Run& t, int r) { return t.b0 + __popc(t.starts & bits_below(r + 1)) - 1; }

// A row of states for the lane's channels (zeros without them).
template <int V>
__device__ __forceinline__ Vec<V> state_row(const float* s, int64_t at, int left) {
  Vec<V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = s && i < left ? s[at + i] : 0.f;
  return v;
}

// The barrier behind the runs' maps: the working warps and the publishing one.
template <class C>
__device__ __forceinline__ void maps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * (C::W + 1)) : "memory");
}

// A lane's places of a tile's map and of a group's state.
template <class C>
__device__ __forceinline__ float* map_place(const ScanParams& p, int tile, int ch) {
  return p.agg + 2 * (tile * (static_cast<int64_t>(p.cols) * C::kWidth) + ch);
}
template <class C>
__device__ __forceinline__ float* state_place(const ScanParams& p, int group, int ch) {
  return p.carry + group * (static_cast<int64_t>(p.cols) * C::kWidth) + ch;
}
__device__ __forceinline__ bool last_of_group(const ScanParams& p, int tile) {
  return tile % kGroup == kGroup - 1 && tile + 1 < p.tiles;
}

// Tiles for each block (with a single one, or one and a few over, a block finishes it before it takes another).
__device__ __forceinline__ int tiles_each(const ScanParams& p) {
  return max(1, p.tiles * p.cols / static_cast<int>(gridDim.x));
}

// The feeding warp: takes the tiles' numbers, lays out their segments, asks for their data.  (One tile's number is taken
// ahead of the place for it, so that the next one's record is there when a place is.)
//   load(row0, ch0, stage, 0): issues the copies of kBytes that complete on full[stage] (one lane)
template <class C, bool BACK, int kBytes, class Load>
__device__ __forceinline__ void feed(const ScanParams& p, TileSmem<C>& sh, Load&& load) {
  using namespace sm100;
  constexpr int S = C::S;
  const int lane = threadIdx.x & 31, total = p.tiles * p.cols;
  const int most = min(S, tiles_each(p));  // a block's tiles at a time
  volatile int* abort_flag = &sh.abort_flag;
  int number = 0, rec = 0;  // a tile's number; lane i: word i of what is known of it
  const auto take = [&] {
    if (lane == 0) number = atomicAdd(p.ticket, 1);
    number = __shfl_sync(0xffffffffu, number, 0);
    if (number < total && lane < kRecord) rec = p.record[static_cast<int64_t>(BACK ? p.tiles - 1 - number / p.cols : number / p.cols) * kRecord + lane];
  };
  int issued = 0;
  bool ok = true;
  if (most > 1) take();  // a tile ahead of the place for it
  for (int j = 0;; ++j) {
    const int s = j % S;
    if (j >= most) ok = hold(sh.empty[(j - most) % S], ((j - most) / S) & 1, abort_flag, p.hdr, 71);
    if (!ok) break;
    if (most == 1) take();
    const bool none = number >= total;
    const int tile = number / p.cols, col = number - tile * p.cols;
    const int row0 = (BACK ? p.tiles - 1 - tile : tile) * C::kRows;
    int from = 0, needs = 0, b0 = 0;  // lane w: b0, starts, ends of the run of warp w
    uint32_t starts = 0, ends = 0;
    if (!none) {
      const int enter = BACK ? row0 + C::kRows : row0;
      const int edge = __shfl_sync(0xffffffffu, rec, 1), before = __shfl_sync(0xffffffffu, rec, 2);
      needs = enter < p.T && edge != enter;
      from = !needs ? tile : BACK ? p.tiles - 1 - (edge - 1) / C::kRows : before / C::kRows;
      // a run's part of the words, and how many starts come before it
      const int at = (BACK ? C::W - 1 - lane : lane) * C::R & (C::kRows - 1), n = p.T - row0 - at;
      const uint32_t bits = static_cast<uint32_t>(rec);
      const uint32_t word = __shfl_sync(0xffffffffu, bits, 3 + (at >> 5)) >> (at & 31);
      const uint32_t next = __shfl_sync(0xffffffffu, bits, 3 + ((at + C::R) >> 5)) >> ((at + C::R) & 31);
      starts = word & bits_below(min(n, C::R));                                     // (the stream's end is none)
      ends = ((word >> 1) | (next & 1u) << (C::R - 1)) & bits_below(min(n, C::R));  // a segment starts behind the row
      b0 = __shfl_sync(0xffffffffu, rec, 0);
#pragma unroll
      for (int w = 0; w < C::kWords; ++w) {
        const uint32_t x = __shfl_sync(0xffffffffu, bits, 3 + w);
        b0 += __popc(w < at >> 5 ? x : w == at >> 5 ? x & bits_below(at & 31) : 0u);
      }
    }
    Slot<C>& slot = sh.slot[s];
    if (none) {
      if (lane == 0) {
        slot.tile = -1;
        mbar_arrive(smem_u32(&sh.known[s]));
        mbar_arrive(smem_u32(&sh.full[s]));
      }
      if (kBytes > 0 && lane == 0) mbar_arrive(smem_u32(&sh.full[s]));
      return;
    }
    if (lane == 0) {
      if constexpr (kBytes > 0) {
        mbar_expect_tx(smem_u32(&sh.full[s]), kBytes);
        load(row0, col * C::kWidth, s, 0);
      }
      slot.tile = tile;
      slot.col = col;
      slot.needs = needs;
      slot.from = from;
    }
    issued = j + 1;
    if (lane < C::W) {
      slot.b0[lane] = b0;
      slot.starts[lane] = starts;
      slot.ends[lane] = ends;
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_u32(&sh.known[s]));
      mbar_arrive(smem_u32(&sh.full[s]));
    }
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

// A warp's way through the block's tiles: stage, the parity of its barriers, the maps' ring.
template <class C>
struct Turn {
  int stage = 0, parity = 0, ring = 0;
  __device__ __forceinline__ void next() {
    if (++stage == C::S) {
      stage = 0;
      parity ^= 1;
    }
    ring = ring + 1 == kRings ? 0 : ring + 1;
  }
};

// A copying warp (without TMA): its part of every tile's rows; a tile is there when every lane's pieces are.
template <class C, bool BACK, class Load>
__device__ __forceinline__ void copy(const ScanParams& p, TileSmem<C>& sh, int part, Load&& load) {
  using namespace sm100;
  volatile int* abort_flag = &sh.abort_flag;
  for (Turn<C> at;; at.next()) {
    if (!hold(sh.known[at.stage], at.parity, abort_flag, p.hdr, 77)) break;
    const int tile = sh.slot[at.stage].tile, col = sh.slot[at.stage].col;
    if (tile < 0) {
      mbar_arrive(smem_u32(&sh.full[at.stage]));
      break;
    }
    load((BACK ? p.tiles - 1 - tile : tile) * C::kRows, col * C::kWidth, at.stage, part);
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.full[at.stage])) : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // (given up: those on their way land before the block ends)
}

// The publishing warp: folds the runs' maps of a tile into the tile's and publishes it, and after a group's last tile the
// state.
template <class C>
__device__ __forceinline__ void publish(const ScanParams& p, TileSmem<C>& sh) {
  using namespace sm100;
  constexpr int V = C::V;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh.abort_flag;
  for (Turn<C> at;; at.next()) {
    if (!hold(sh.full[at.stage], at.parity, abort_flag, p.hdr, 73)) sh.stop[at.ring] = 1;
    const int tile = sh.slot[at.stage].tile, ch = (sh.slot[at.stage].col * 32 + lane) * V;
    maps_sync<C>();
    if (sh.stop[at.ring] || tile < 0) return;
    if (tile + 1 >= p.tiles || (p.wait_ns && tile == 0)) continue;
    Vec<V> A = fill<V>(1.f), B = fill<V>(0.f);
    bool reset = false;
#pragma unroll
    for (int w = 0; w < C::W; ++w) {
      const bool rw = sh.reset[at.ring][w] != 0;
      reset |= rw;
      Vec<V> mA, mB;
#pragma unroll
      for (int i = 0; i < V; ++i) mA[i] = sh.run[at.ring][w][lane * V + i].x, mB[i] = sh.run[at.ring][w][lane * V + i].y;
      B = rw ? mB : fma(mA, B, mB);
      A = rw ? fill<V>(0.f) : mul(A, mA);
    }
    float m[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) m[2 * i] = A[i], m[2 * i + 1] = B[i];
    show<2 * V>(map_place<C>(p, tile, ch), m);
    if (!last_of_group(p, tile)) continue;
    if (!reset) {
      // (the state that enters the tile waits for tiles before it only; the stage is held till this warp comes round)
      if (!hold(sh.carried[at.stage], at.parity, abort_flag, p.hdr, 76)) {
        sh.stop[at.ring + 1 == kRings ? 0 : at.ring + 1] = 1;
        continue;
      }
      Vec<V> in;
#pragma unroll
      for (int i = 0; i < V; ++i) in[i] = sh.carry[at.stage][lane * V + i];
      B = fma(A, in, B);
    }
    show<V>(state_place<C>(p, tile / kGroup, ch), B.e);
  }
}

// A resolving warp: the state that enters a tile, from the maps of the tiles before it and a state further back, from when
// the tile's number is known.  Each of them looks at every tile's slot and takes its share of the tiles.  A slot is given
// back by both of them too: one that has not seen a tile yet would find the slot, and its barrier's parity, two uses on.
template <class C>
__device__ __forceinline__ void resolve(const ScanParams& p, TileSmem<C>& sh, int me) {
  using namespace sm100;
  constexpr int V = C::V, kAhead = 4;  // maps asked for at once
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh.abort_flag;
  int whose = 0;
  for (Turn<C> at;; at.next()) {
    if (!hold(sh.known[at.stage], at.parity, abort_flag, p.hdr, 74)) return;
    const Slot<C>& slot = sh.slot[at.stage];
    const int tile = slot.tile;
    if (tile < 0) return;
    const int ch = (slot.col * 32 + lane) * V, from = slot.from;
    const bool needs = slot.needs != 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.empty[at.stage]));  // (looked at: the slot may be written again)
    const bool mine = whose == me;
    whose = whose + 1 == kResolvers ? 0 : whose + 1;
    if (!mine) continue;
    Vec<V> in = fill<V>(0.f);
    bool ok = true;
    if (needs) {
      // [lo, tile) are folded; then onto the state after the group before them where the segment began further back (the
      // state last: in one long segment each of them waits for the one before)
      const int g = tile / kGroup - kBack, lo = max(max(g, 0) * kGroup, from);
      const bool onto = from < g * kGroup;
      Vec<V> A = fill<V>(1.f), B = fill<V>(0.f);
#pragma unroll 1
      for (int k0 = lo; k0 < tile && ok; k0 += kAhead) {
        float m[kAhead][2 * V];
        ok = until(p, [&] {
          bool all = true;
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (k0 + k < tile) peek(map_place<C>(p, k0 + k, ch), m[k]);
#pragma unroll
          for (int k = 0; k < kAhead; ++k) all &= k0 + k >= tile || there<2 * V>(m[k]);
          return all;
        });
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (k0 + k < tile) {
            Vec<V> mA, mB;
#pragma unroll
            for (int i = 0; i < V; ++i) mA[i] = m[k][2 * i], mB[i] = m[k][2 * i + 1];
            B = fma(mA, B, mB);
            A = mul(A, mA);
          }
      }
      if (onto) {
        ok = ok && until(p, [&] {
               peek(state_place<C>(p, g - 1, ch), in.e);
               return there<V>(in.e);
             });
        in = fma(A, in, B);
      } else {
        in = B;
      }
    }
    if (!ok) {
      sh.abort_flag = 1;
      return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sh.carry[at.stage][lane * V + i] = in[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.carried[at.stage]));
  }
}

// The working warps: form a tile's maps before they finish the tile before, so that whoever waits for them waits little.
//   first(run, stage, A, B)    the run's map, true: it replaces the state        second(run, stage, in)   the outputs
// (One copy of each part of the work: unrolled over the stages the code left the instruction cache; the forward of
// T = 8192, D = 4096 in bf16 took 211 us.)
template <class C, bool BACK, class First, class Second>
__device__ __forceinline__ void work(const ScanParams& p, TileSmem<C>& sh, First&& first, Second&& second) {
  using namespace sm100;
  constexpr int V = C::V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  volatile int* abort_flag = &sh.abort_flag;
  Run old;
  old.tile = -1;
  Turn<C> at, held;
  const bool single = tiles_each(p) == 1;
#pragma unroll 1
  for (;; at.next()) {
    Run now;
    now.tile = -1;
    if (!hold(sh.full[at.stage], at.parity, abort_flag, p.hdr, 72)) sh.stop[at.ring] = 1;
    else if (sh.slot[at.stage].tile >= 0) now = run_of<C>(p, sh.slot[at.stage], BACK);
    if (now.tile >= 0) {
      Vec<V> A, B;
      const bool reset = first(now, at.stage, A, B);
#pragma unroll
      for (int k = 0; k < V; ++k) sh.run[at.ring][warp][lane * V + k] = make_float2(reset ? 0.f : A[k], B[k]);
      if (lane == 0) sh.reset[at.ring][warp] = reset;
    }
    maps_sync<C>();
    if (sh.stop[at.ring]) break;
    const int next = at.ring + 1 == kRings ? 0 : at.ring + 1;
    if (single) {
      old = now;
      held = at;
    }
    if (old.tile >= 0) {
      // (a wait that gives up here leaves its tile, but comes to the next barrier like the others, and stops there)
      if (hold(sh.carried[held.stage], held.parity, abort_flag, p.hdr, 75)) {
        Vec<V> in;
#pragma unroll
        for (int i = 0; i < V; ++i) in[i] = sh.carry[held.stage][lane * V + i];
        for (int w = 0; w < warp; ++w) {
          const bool rw = sh.reset[held.ring][w] != 0;
          Vec<V> mA, mB;
#pragma unroll
          for (int i = 0; i < V; ++i) mA[i] = sh.run[held.ring][w][lane * V + i].x, mB[i] = sh.run[held.ring][w][lane * V + i].y;
          in = rw ? mB : fma(mA, in, mB);
        }
        second(old, held.stage, in);
      } else {
        sh.stop[next] = 1;  // (this step's may still be being read)
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[held.stage]));
    }
    if (now.tile < 0) return;
    old = now;
    held = at;
    if (single) old.tile = -1;
  }
  sh.abort_flag = 1;  // given up: the other warps stop too
}

// Runs a block's warps.
template <class C, bool BACK, int kBytes, class Load, class First, class Second>
__device__ __forceinline__ void run_block(const ScanParams& p, TileSmem<C>& sh, Load&& load, First&& first,
                                          Second&& second) {
  using namespace sm100;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(smem_u32(&sh.known[s]), 1);
      mbar_init(smem_u32(&sh.full[s]), 1 + (kBytes > 0 ? 1 : 32 * C::K));  // the slot, the data
      mbar_init(smem_u32(&sh.empty[s]), C::W + kResolvers);  // the tile is done, and every resolving warp has seen it
      mbar_init(smem_u32(&sh.carried[s]), 1);
      sh.slot[s].tile = -1;
    }
    fence_barrier_init();
    for (int r = 0; r < kRings; ++r) sh.stop[r] = 0;
    sh.abort_flag = 0;
    sh.wait_limit = p.wait_ns ? p.wait_ns : kTimeoutNs;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  if (warp < C::W) work<C, BACK>(p, sh, first, second);
  else if (warp == C::W) feed<C, BACK, kBytes>(p, sh, load);
  else if (warp == C::W + 1) publish<C>(p, sh);
  else if (warp < C::W + 2 + kResolvers) resolve<C>(p, sh, warp - C::W - 2);
  else if constexpr (C::K > 0) copy<C, BACK>(p, sh, warp - C::W - 2 - kResolvers, load);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// A tile's rows as they are copied: by TMA one behind the other, else each with the 16-byte pieces that hold it, at the
// place in its pieces that its address has.
template <class T, class C, bool TMA>
constexpr int pitch() { return C::kWidth * static_cast<int>(sizeof(T)) + (TMA ? 0 : 16); }

// The part `part` of K of the rows [row0, row0 + kRows) of the tensor that has rows [0, T), from channel ch0 on, by a
// warp.  (A piece holds an element of the tensor at least, so none lies outside of its memory, though a piece at its
// edge or a tile's may hold others' elements too, which nobody uses.)
template <class T, class C>
__device__ __forceinline__ void copy_rows(uint8_t* to, const void* from, int64_t rs, int row0, int T_rows, int ch0, int D,
                                          int part) {
  constexpr int kPitch = pitch<T, C, false>(), kPieces = kPitch / 16;
  const uintptr_t base = reinterpret_cast<uintptr_t>(static_cast<const T*>(from) + row0 * rs + ch0);
  const int bytes = min(C::kWidth, D - ch0) * static_cast<int>(sizeof(T)), lo = max(0, -row0), hi = T_rows - row0;
#pragma unroll 3
  for (int i = part * 32 + (threadIdx.x & 31); i < C::kRows * kPieces; i += 32 * C::K) {
    const int r = i / kPieces, at = (i - r * kPieces) * 16;
    const uintptr_t row = base + static_cast<uint64_t>(r * rs) * sizeof(T), piece = (row & ~static_cast<uintptr_t>(15)) + at;
    if (r >= lo && r < hi && piece < row + bytes)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + r * kPitch + at)), "l"(piece) : "memory");
  }
}

// The copied rows of a run.  (Without TMA the lanes behind the last channel read what lies there; it gets nowhere.)
template <class T, class C, bool TMA>
struct Rows {
  const uint8_t* tile;  // stage 0, at the lane's channels
  const T* base;        // the tensor's row that is copied for row 0
  int64_t rs;
  struct Place {
    const uint8_t* at;
    int low;            // of the first row's address
  };
  __device__ __forceinline__ Rows(const uint8_t* smem, const void* global, int64_t rs_, int before)
      : tile(smem + (threadIdx.x & 31) * C::V * sizeof(T)), base(static_cast<const T*>(global) - before * rs_), rs(rs_) {}
  // the run's first row
  __device__ __forceinline__ Place at(const Run& t, int stage, bool back) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kPitch = pitch<T, C, TMA>();
    return {tile + (stage * C::kRows + (back ? C::W - 1 - warp : warp) * C::R) * kPitch,
            TMA ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(base + t.row * rs + t.ch - lane * C::V) & 15)};
  }
  __device__ __forceinline__ Pack<T, C::V> get(const Place& first, int r) const {
    if constexpr (TMA) {
      return load_pack<T, C::V>(reinterpret_cast<const T*>(first.at + r * pitch<T, C, true>()));
    } else {
      const int low = (first.low + r * (static_cast<unsigned>(rs) * static_cast<unsigned>(sizeof(T)))) & 15;
      const T* const row = reinterpret_cast<const T*>(first.at + r * pitch<T, C, false>() + low);
      Pack<T, C::V> v;
#pragma unroll
      for (int i = 0; i < C::V; ++i) v.e[i] = row[i];
      return v;
    }
  }
};

// A row's outputs.  Without TMA rows may begin anywhere: where a lane's pair straddles two words, its second channel is
// stored with the next lane's first.  Every lane of the warp calls it.
template <bool TMA, class T>
__device__ __forceinline__ void put(T* to, const Pack<T, 2>& v, int left) {
  if constexpr (TMA) {
    if (left > 0) store_pack(to, v);
  } else if ((reinterpret_cast<uintptr_t>(to) & (2 * sizeof(T) - 1)) == 0) {  // (the same for every lane)
    if (left > 1) store_pack(to, v);
    else if (left == 1) to[0] = v.e[0];
  } else {
    Pack<T, 2> pair;
    const int lane = threadIdx.x & 31;
    pair.e[0] = v.e[1];
    pair.e[1] = __shfl_down_sync(0xffffffffu, v.e[0], 1);
    if (left > 2 && lane < 31) store_pack(to + 1, pair);
    else if (left > 1) to[1] = v.e[1];
    if (lane == 0 && left > 0) to[0] = v.e[0];
  }
}

// Rows of a run that holds a segment's boundary or the stream's end, in order or from the back.
template <bool BACK = false, class A, class PA, class B, class PB, class F>
__device__ __forceinline__ void rows_of(const A& a, const PA& pa, const B& b, const PB& pb, const Run& t, F&& f) {
#pragma unroll 1
  for (int i = 0; i < t.n; ++i) {
    const int r = BACK ? t.n - 1 - i : i;
    f(r, a.get(pa, r), b.get(pb, r));
  }
}

// Bytes of a tile of one tensor.
template <class T, class C, bool TMA> constexpr int tile_bytes() { return C::kRows * pitch<T, C, TMA>(); }
template <class C> constexpr int head_bytes() { return (static_cast<int>(sizeof(TileSmem<C>)) + 127) / 128 * 128; }

struct Maps {
  CUtensorMap a, b, c;  // forward: x, g; backward: dh, g, h
};

}  // namespace

// Checks the boundary contract (block 0), empties the published places and writes every tile's record.
__global__ void __launch_bounds__(kPrepThreads) scan_prep_kernel(const ScanParams p, int rows, int back, int64_t words) {
  griddep_begin();
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPrepThreads;
  for (int64_t i = tid; i < words / 4; i += step)
    reinterpret_cast<uint4*>(p.agg)[i] = make_uint4(kNone, kNone, kNone, kNone);
  for (int64_t i = tid; i < static_cast<int64_t>(p.tiles) * kRecord; i += step) {
    const int k = static_cast<int>(i % kRecord), row0 = static_cast<int>(i / kRecord) * rows;  // (row0 < T)
    // the first b in [0, B] with cu[b] >= row (cu[B] = T)
    const int row = min(k == 0 ? row0 : k < 3 ? row0 + (back ? rows : 0) : row0 + min(32 * (k - 3), rows), p.T);
    int lo = 0, hi = p.B;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] < row) lo = mid + 1;
      else hi = mid;
    }
    int word = lo;
    if (k == 1) word = p.cu[lo];
    if (k == 2) word = p.cu[max(lo - 1, 0)];
    if (k >= 3) {
      uint32_t bits = 0;
      const int first = row0 + 32 * (k - 3), most = min(first + 31, row0 + rows);
      for (int b = lo; b <= p.B; ++b) {
        const int at = p.cu[b];
        if (at < first || at > most) break;
        bits |= 1u << (at - first);
      }
      word = static_cast<int>(bits);
    }
    p.record[i] = word;
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
  constexpr int kX = tile_bytes<TX, C, TMA>(), kG = tile_bytes<TG, C, TMA>();
  uint8_t* const x_smem = smem + head_bytes<C>();
  uint8_t* const g_smem = x_smem + kX * C::S;
  const Rows<TX, C, TMA> xs(x_smem, p.x, p.x_rs, 0);
  const Rows<TG, C, TMA> gs(g_smem, p.g, p.g_rs, 0);
  const auto load = [&](int row0, int ch0, int stage, int part) {
    if constexpr (TMA) {
      const uint32_t bar = smem_u32(&sh.full[stage]);
      tma_load_2d(smem_u32(x_smem + stage * kX), &maps.a, bar, ch0, row0);
      tma_load_2d(smem_u32(g_smem + stage * kG), &maps.b, bar, ch0, row0);
    } else {
      copy_rows<TX, C>(x_smem + stage * kX, p.x, p.x_rs, row0, p.T, ch0, p.D, part);
      copy_rows<TG, C>(g_smem + stage * kG, p.g, p.g_rs, row0, p.T, ch0, p.D, part);
    }
  };
  const auto step = [&](const Pack<TX, V>& x, const Vec<V>& g, Vec<V>& h) { h = fma(decay(g), h, wide_of(x)); };
  const auto start = [&](const Pack<TX, V>& x, const Vec<V>& g, const Run& t, int r, Vec<V>& h) {  // a segment's first row
    h = wide_of(x);  // (x itself without h0, whatever its decay is)
    if (p.h0) h = fma(decay(g), state_row<V>(p.h0, static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch, t.left), h);
  };
  const auto first = [&](const Run& t, int stage, Vec<V>& A, Vec<V>& B) {
    A = B = fill<V>(0.f);
    const auto xa = xs.at(t, stage, false);
    const auto ga = gs.at(t, stage, false);
    if (t.starts == 0 && t.n == R) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const Vec<V> g = wide_of(gs.get(ga, r));
        A = add(A, g);
        step(xs.get(xa, r), g, B);
      }
    } else {
      rows_of(xs, xa, gs, ga, t, [&](int r, const Pack<TX, V>& x, const Pack<TG, V>& gr) {
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
    const auto xa = xs.at(t, stage, false);
    const auto ga = gs.at(t, stage, false);
    if (t.starts == 0 && t.n == R && (!p.last || t.ends == 0)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        step(xs.get(xa, r), wide_of(gs.get(ga, r)), h);
        put<TMA>(out + r * p.out_rs, narrow<TH, V>(h), t.left);
      }
    } else {
      rows_of(xs, xa, gs, ga, t, [&](int r, const Pack<TX, V>& x, const Pack<TG, V>& gr) {
        const Vec<V> g = wide_of(gr);
        if ((t.starts >> r) & 1u) start(x, g, t, r, h);
        else step(x, g, h);
        put<TMA>(out + r * p.out_rs, narrow<TH, V>(h), t.left);
        if (p.last && ((t.ends >> r) & 1u)) {
          float* last = p.last + static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch;
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i < t.left) last[i] = h[i];
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
  constexpr int kH = tile_bytes<TH, C, TMA>(), kG = tile_bytes<TG, C, TMA>();
  uint8_t* const d_smem = smem + head_bytes<C>();
  uint8_t* const g_smem = d_smem + kH * C::S;
  uint8_t* const h_smem = g_smem + kG * C::S;
  const Rows<TH, C, TMA> ds(d_smem, p.x, p.x_rs, 0), hs(h_smem, p.h, p.h_rs, 1);
  const Rows<TG, C, TMA> gs(g_smem, p.g, p.g_rs, 0);
  const auto load = [&](int row0, int ch0, int stage, int part) {
    // (of h the rows before; there is none before the first, and a segment's first row asks for none)
    if constexpr (TMA) {
      const uint32_t bar = smem_u32(&sh.full[stage]);
      tma_load_2d(smem_u32(d_smem + stage * kH), &maps.a, bar, ch0, row0);
      tma_load_2d(smem_u32(g_smem + stage * kG), &maps.b, bar, ch0, row0);
      tma_load_2d(smem_u32(h_smem + stage * kH), &maps.c, bar, ch0, row0 - 1);
    } else {
      copy_rows<TH, C>(d_smem + stage * kH, p.x, p.x_rs, row0, p.T, ch0, p.D, part);
      copy_rows<TG, C>(g_smem + stage * kG, p.g, p.g_rs, row0, p.T, ch0, p.D, part);
      copy_rows<TH, C>(h_smem + stage * kH, p.h, p.h_rs, row0 - 1, p.T, ch0, p.D, part);
    }
  };
  const auto first = [&](const Run& t, int stage, Vec<V>& A, Vec<V>& B) {
    A = B = fill<V>(0.f);
    const auto da = ds.at(t, stage, true);
    const auto ga = gs.at(t, stage, true);
    const auto step = [&](const Pack<TH, V>& d, const Pack<TG, V>& gr) {
      const Vec<V> g = wide_of(gr);
      A = add(A, g);
      B = mul(decay(g), add(wide_of(d), B));
    };
    if (t.ends == 0 && t.n == R) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r) step(ds.get(da, r), gs.get(ga, r));
    } else {
      rows_of<true>(ds, da, gs, ga, t, [&](int r, const Pack<TH, V>& d, const Pack<TG, V>& g) {
        if ((t.ends >> r) & 1u) B = state_row<V>(p.dlast, static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch, t.left);
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
    const auto da = ds.at(t, stage, true);
    const auto ga = gs.at(t, stage, true);
    const auto ha = hs.at(t, stage, true);
    // before: the row before's h, at a segment's first row h0 (none: 0, and so is the decay's gradient)
    const auto step = [&](int r, const Pack<TH, V>& d, const Pack<TG, V>& g, const Vec<V>& before, bool none) {
      const Vec<V> e = add(wide_of(d), f);
      f = mul(decay(wide_of(g)), e);
      const Vec<V> q = none ? fill<V>(0.f) : mul(f, before);
      put<TMA>(dx + r * p.out_rs, narrow<TX, V>(e), t.left);
      put<TMA>(dg + r * p.dg_rs, narrow<TG, V>(q), t.left);
    };
    if (t.ends == 0 && t.starts == 0 && t.n == R) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r)
        step(r, ds.get(da, r), gs.get(ga, r), wide_of(hs.get(ha, r)), false);
    } else {
      rows_of<true>(ds, da, gs, ga, t, [&](int r, const Pack<TH, V>& d, const Pack<TG, V>& g) {
        const int64_t state = static_cast<int64_t>(segment_of(t, r)) * p.D + t.ch;
        const bool start = (t.starts >> r) & 1u;
        if ((t.ends >> r) & 1u) f = state_row<V>(p.dlast, state, t.left);
        const Vec<V> before = start ? state_row<V>(p.h0, state, t.left) : wide_of(hs.get(ha, r));
        step(r, d, g, before, start && !p.h0);
        if (p.last && start) {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i < t.left) p.last[state + i] = f[i];
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
  size_t record, agg, carry, total;
};

Layout layout_of(int T, int D, int rows, int width) {
  Layout l;
  l.tiles = (static_cast<int64_t>(T) + rows - 1) / rows;
  l.cols = (static_cast<int64_t>(D) + width - 1) / width;
  l.groups = (l.tiles + kGroup - 1) / kGroup;
  l.record = sizeof(WsHeader);
  l.agg = align256(l.record + l.tiles * kRecord * sizeof(int32_t));
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
  p.record = reinterpret_cast<int32_t*>(w + l.record);
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
cudaError_t run_blocks(int stage, int back, void (*kernel)(ScanParams, Maps), size_t piece, ScanParams p, const Maps& maps, void* ws,
                       cudaStream_t st) {
  const Layout l = layout_of(p.T, p.D, C::kRows, C::kWidth);
  place(p, l, ws);
  const int sms = device_sms();
  if (stage == 0) {
    const int64_t work = std::max(l.words / 8, l.tiles * kRecord);
    const int blocks = static_cast<int>(std::min<int64_t>(2 * sms, (work + kPrepThreads - 1) / kPrepThreads));
    return launch_pdl(scan_prep_kernel, dim3(blocks), dim3(kPrepThreads), 0, st, p, C::kRows, back, l.words);
  }
  const size_t smem = head_bytes<C>() + piece * C::S;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t fit = std::max<int64_t>(1, std::min<int64_t>((228 * 1024) / (smem + 1024), C::M));
  const int grid = static_cast<int>(std::min<int64_t>(l.tiles * l.cols, sms * fit));
  return launch_pdl(kernel, dim3(grid), dim3(C::kThreads), smem, st, p, maps);
}

using FwdShape = Shape<2, 8, 16, 3, 2>;
using BwdShape = Shape<2, 8, 8, 3, 2>;
// (fp32 rows are twice the pieces: T = 30000, D = 1022 128 us with two copying warps, 117 with four; bf16 rows, D = 2047,
// 155 and 162; one, 151 and 165)
template <class T> using CopyShape = Shape<2, 8, 8, 3, 2, sizeof(T) == 4 ? 4 : 2>;

// Tiles come by TMA where the inputs' rows lie on 16-byte boundaries and the outputs' on pairs of channels.
template <class TX, class TG, class TH>
cudaError_t run_fwd(int stage, const ScanParams& p, void* ws, cudaStream_t st) {
  using C = FwdShape;
  Maps maps{};
  if (p.D % 2 == 0 && rows16<TX>(p.x, p.x_rs) && rows16<TG>(p.g, p.g_rs) && steps_of<TH>(p.out, p.out_rs, 2)) {
    if (stage == 1 && !(tmap_matrix(&maps.a, p.x, sizeof(TX) == 2, p.T, p.D, p.x_rs, C::kWidth, C::kRows) &&
                        tmap_matrix(&maps.b, p.g, sizeof(TG) == 2, p.T, p.D, p.g_rs, C::kWidth, C::kRows)))
      return cudaErrorInvalidValue;
    return run_blocks<C>(stage, 0, scan_fwd_kernel<TX, TG, TH, C, true>,
                         tile_bytes<TX, C, true>() + tile_bytes<TG, C, true>(), p, maps, ws, st);
  }
  using P = CopyShape<TG>;
  return run_blocks<P>(stage, 0, scan_fwd_kernel<TX, TG, TH, P, false>,
                       tile_bytes<TX, P, false>() + tile_bytes<TG, P, false>(), p, maps, ws, st);
}

template <class TX, class TG, class TH>
cudaError_t run_bwd(int stage, const ScanParams& p, void* ws, cudaStream_t st) {
  using C = BwdShape;
  Maps maps{};
  if (p.D % 2 == 0 && rows16<TH>(p.x, p.x_rs) && rows16<TG>(p.g, p.g_rs) && rows16<TH>(p.h, p.h_rs) &&
      steps_of<TX>(p.out, p.out_rs, 2) && steps_of<TG>(p.dg, p.dg_rs, 2)) {
    if (stage == 1 && !(tmap_matrix(&maps.a, p.x, sizeof(TH) == 2, p.T, p.D, p.x_rs, C::kWidth, C::kRows) &&
                        tmap_matrix(&maps.b, p.g, sizeof(TG) == 2, p.T, p.D, p.g_rs, C::kWidth, C::kRows) &&
                        tmap_matrix(&maps.c, p.h, sizeof(TH) == 2, p.T, p.D, p.h_rs, C::kWidth, C::kRows)))
      return cudaErrorInvalidValue;
    return run_blocks<C>(stage, 1, scan_bwd_kernel<TX, TG, TH, C, true>,
                         2 * tile_bytes<TH, C, true>() + tile_bytes<TG, C, true>(), p, maps, ws, st);
  }
  using P = CopyShape<TG>;
  return run_blocks<P>(stage, 1, scan_bwd_kernel<TX, TG, TH, P, false>,
                       2 * tile_bytes<TH, P, false>() + tile_bytes<TG, P, false>(), p, maps, ws, st);
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
  for (int rows : {FwdShape::kRows, BwdShape::kRows, CopyShape<float>::kRows}) n = std::max(n, layout_of(T, D, rows, FwdShape::kWidth).total);
  return n;
}

cudaError_t launch_scan_fwd(int stage, ScanParams p, int xb, int gb, int hb, void* ws, cudaStream_t st) {
  if (xb && gb) return hb ? run_fwd<bf16, bf16, bf16>(stage, p, ws, st) : run_fwd<bf16, bf16, float>(stage, p, ws, st);
  return xb ? run_fwd<bf16, float, float>(stage, p, ws, st) : run_fwd<float, float, float>(stage, p, ws, st);
}

cudaError_t launch_scan_bwd(int stage, ScanParams p, int xb, int gb, int hb, void* ws, cudaStream_t st) {
  if (xb && gb) return hb ? run_bwd<bf16, bf16, bf16>(stage, p, ws, st) : run_bwd<bf16, bf16, float>(stage, p, ws, st);
  return xb ? run_bwd<bf16, float, float>(stage, p, ws, st) : run_bwd<float, float, float>(stage, p, ws, st);
}

cudaError_t launch_scan_step(ScanParams p, int xb, int gb, int hb, void* ws, cudaStream_t st) {
  if (xb && gb) return hb ? run_step<bf16, bf16, bf16>(p, ws, st) : run_step<bf16, bf16, float>(p, ws, st);
  return xb ? run_step<bf16, float, float>(p, ws, st) : run_step<float, float, float>(p, ws, st);
}

}  // namespace va
