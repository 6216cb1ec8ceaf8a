// Host side of the C ABI: argument checks, workspace layout, launch sequences.
#include <algorithm>
#include <atomic>
#include <cstdio>
#include <initializer_list>
#include <string>
#include <utility>
#include <vector>

#include "attn_params.cuh"
#include "logprobs.cuh"
#include "qk_norm.cuh"
#include "scan.cuh"

namespace va {

// kernels (other translation units)
cudaError_t launch_metadata_scan(const int32_t*, int, int, int, int32_t*, int32_t*, int32_t*, int32_t*,
                                 int32_t*, cudaStream_t);
bool metadata_inline_fill(int n, int T_capacity);
cudaError_t launch_metadata_fill(const int32_t*, int, int, int32_t*, int32_t*, const int32_t*,
                                 cudaStream_t);
cudaError_t launch_validate(const int32_t*, int, int, int, int32_t*, int, cudaStream_t);
cudaError_t launch_cu_from_positions(const int32_t*, int, int, int, int32_t*, int, int32_t*, int32_t*,
                                     int32_t*, cudaStream_t);
cudaError_t launch_plan(const PlanArgs&, cudaStream_t);
cudaError_t launch_validate_plan(const PlanArgs*, int, int, int, int, int, cudaStream_t);
cudaError_t launch_fwd_tc(const FwdParams&, int, int, cudaStream_t);
cudaError_t launch_fwd_tok(const FwdParams&, int, int, cudaStream_t);
void fwd_tc_tiles(int*, int*);
int fwd_tc_token_short();
int bwd_tc_token_short();
cudaError_t launch_bwd_prep(const BwdParams&, const PlanArgs*, int, int, int, int, int, int, cudaStream_t);
cudaError_t launch_unpad_index(int, const int32_t*, int, int, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*,
                               int32_t*, cudaStream_t);
cudaError_t launch_gather_rows(const void*, int64_t, const int32_t*, int, int64_t, void*, int64_t, cudaStream_t);
cudaError_t launch_loss_targets(const int32_t*, const int32_t*, int, int, int, int32_t*, cudaStream_t);
cudaError_t launch_token_ce(int, const void*, int, int64_t, const int32_t*, int, int, int, void*, int64_t, float*,
                            int32_t*, int32_t*, double*, cudaStream_t);
bool distill_row_fits(int, int);
size_t distill_parts_bytes();
cudaError_t launch_token_distill(int, const void*, int, int64_t, const int32_t*, int64_t, const void*, int, int64_t,
                                 const int32_t*, int, int, int, int, float, void*, int64_t, void*, int32_t*, uint8_t*,
                                 float*, int32_t*, uint64_t, cudaStream_t);
size_t embed_bwd_workspace(int, int);
cudaError_t launch_embed_fwd(const void*, int, int64_t, const int32_t*, int, int, int, float, void*, int64_t, int32_t*,
                             cudaStream_t);
cudaError_t launch_embed_bwd(int, const void*, int, int64_t, const int32_t*, int, int, int, float, void*, int, int64_t,
                             int, void*, cudaStream_t);
cudaError_t launch_bwd_dkdv_tc(const BwdParams&, int, int, bool, cudaStream_t);
cudaError_t launch_bwd_dq_tc(const BwdParams&, int, int, bool, cudaStream_t);
cudaError_t launch_sink_join(const BwdParams&, int, cudaStream_t);
void bwd_tc_tiles(int*, int*, int*, int*);

static thread_local std::string g_error;
// Test hooks of the failure paths: a wait limit (ns) armed for the next forward, distillation or recurrence, 0 = none.
static std::atomic<long long> g_stall_next_fwd{0}, g_stall_next_distill{0}, g_stall_next_scan{0};

void set_error(const char* msg) { g_error = msg; }

// ------------------------------------------------------------ launch accounting
enum KernelId {
  K_VALIDATE = 0, K_META_SCAN, K_META_FILL, K_PLAN, K_FWD, K_BWD_PREP, K_BWD_DKDV, K_BWD_DQ,
  K_VALIDATE_PLAN, K_FWD_TOK, K_CU_FROM_POS, K_LOSS_TARGETS, K_CE_COUNT, K_CE_ROWS, K_CE_REDUCE, K_PAD_COUNT,
  K_PAD_SCAN, K_PAD_INDEX, K_GATHER_ROWS, K_DISTILL_COUNT, K_DISTILL_ROWS, K_DISTILL_REDUCE,
  K_EMBED_FWD, K_EMBED_SORT, K_EMBED_REDUCE, K_EMBED_JOIN, K_SINK_JOIN,
  K_QK_NORM_FWD, K_QK_NORM_BWD, K_QK_NORM_JOIN, K_SCAN_PREP, K_SCAN_FWD, K_SCAN_BWD, K_SCAN_STEP, K_LOGPROBS_FWD,
  K_LOGPROBS_BWD, K_COUNT
};
const char* const kKernelNames[K_COUNT] = {
    "validate_cu_seqlens", "metadata_scan", "metadata_fill", "plan",          "fwd",
    "bwd_prep",            "bwd_dkdv",      "bwd_dq",        "validate_plan", "fwd_tok",
    "cu_from_positions",   "loss_targets",  "ce_count",      "ce_rows",       "ce_reduce",
    "pad_count",           "pad_scan",      "pad_index",     "gather_rows", "distill_count", "distill_rows",
    "distill_reduce", "embed_fwd", "embed_sort", "embed_reduce", "embed_join",
    "sink_join", "qk_norm_fwd", "qk_norm_bwd", "qk_norm_join", "scan_prep", "scan_fwd", "scan_bwd", "scan_step",
    "logprobs_fwd", "logprobs_bwd"};

struct Profiler {
  std::vector<cudaEvent_t> start, stop;
  std::vector<int32_t> ids;
  int cap = 0, n = 0;
};
static Profiler g_prof;
static std::atomic<long long> g_launches{0};

// Runs one kernel launch; counts it and, when profiling, brackets it with events.
template <class F>
cudaError_t launch(int id, cudaStream_t st, F&& f) {
  const bool rec = g_prof.cap > 0 && g_prof.n < g_prof.cap;
  if (rec) cudaEventRecord(g_prof.start[g_prof.n], st);
  cudaError_t e = f();
  if (rec) {
    cudaEventRecord(g_prof.stop[g_prof.n], st);
    g_prof.ids[g_prof.n++] = id;
  }
  if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

namespace {

va_status fail(va_status st, const std::string& msg) {
  g_error = msg;
  return st;
}

va_status cuda_fail(cudaError_t e, const char* where) {
  return fail(VA_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Token tiles (runs of short segments planned as tiles of consecutive tokens) pay off when
// short segments are common; they are used for causal calls whose mean segment length T / B
// is below this many tokens.  Results do not depend on the choice: it only selects which
// records cover the short segments and which kernel forms run.
constexpr int64_t kTokenMeanLen = 256;

bool token_tiles(const va_shape& s, int32_t causal, int32_t window) {
  return causal && window < 0 && static_cast<int64_t>(s.T) < kTokenMeanLen * s.B;
}

// Whether a call with a window takes token tiles (its public maps never list them).  They replace a
// masked tile per segment and head; they cost the forward a launch and the backward kernel forms that are
// slower on segment records.  So they need many segments, much of them at most 64 tokens long, which the
// host sees from the mean, and from a longest segment far above it (then the others lie below it).
// Small calls are bound by their launches, and up to 32 segments the planner has a short path.
// Forward + backward in us, device time, without / with token tiles (u: lengths uniform in [m/2, 3m/2], e:
// exponential; the window's kernels have no other form):
//   8/2 heads of 64:   u40 T = 30000 242 / 152, u48 T = 19200 144 / 131, u80 T = 30000 163 / 184, u120 T = 8192 59 / 69,
//                      e40 T = 8192 81 / 71, e80 T = 30000 189 / 185, e120 T = 30000 166 / 184
//   32/8 heads of 128: u40 T = 8192 314 / 228, u56 T = 30000 844 / 783, u80 T = 8192 234 / 270, u240 T = 30000 632 / 650,
//                      e64 T = 30000 837 / 750, e80 T = 8192 266 / 272, e120 T = 8192 230 / 248
//   small calls:       2/1 heads of 64, u40, T = 2400 30 / 40; 8/2 of 64, e48, T = 2880 47 / 53; 8/2 of 64, u24,
//                      T = 2400 53 / 45; 32/8 of 128, u10, T = 340 72 / 47; 27 segments of 10, 8/2 of 64, 26 / 39
// (worst choice among 286 measured calls: 2/1 heads of 64, e56, T = 11200, 45 / 52)
bool window_token_tiles(const va_shape& s) {
  const int64_t T = s.T, B = s.B, tiles = B * s.Hq;
  if (B <= 32 || (tiles < 768 && (T < 4096 || T * s.Hq < 16384))) return false;
  const int64_t mean = 2 * B * s.max_seqlen >= 5 * T ? 96 : 48 + std::min<int64_t>(tiles / 1024, 12);
  return T < mean * B;
}

bool call_token_tiles(const va_shape& s, int32_t causal, int32_t window) {
  return window < 0 ? token_tiles(s, causal, window) : causal && window_token_tiles(s);
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

void tiles(int kind, int* BM, int* BN) {
  if (kind == 0) {
    fwd_tc_tiles(BM, BN);
  } else {
    int a, b, c, d;
    bwd_tc_tiles(&a, &b, &c, &d);
    if (kind == 1) {
      *BM = a;
      *BN = b;
    } else {
      *BM = c;
      *BN = d;
    }
  }
}

// Upper bound on records of a map: blocks per segment <= l/blk + 1.  Tk: rows of K/V
// (cross-attention; -1 = s.T), which the kv-block map is cut from.
int64_t map_capacity(const va_shape& s, int kind, int Tk = -1) {
  int BM, BN;
  tiles(kind, &BM, &BN);
  const int blk = kind == 1 ? BN : BM;
  const int heads = kind == 1 ? s.Hkv : s.Hq;
  const int rows = kind == 1 && Tk >= 0 ? Tk : s.T;
  return (static_cast<int64_t>(rows) / blk + s.B) * heads;
}

// Cross-attention arguments: the K/V stream's rows and longest segment.
va_status check_cross(const va_shape* s, const int32_t* cu_k, int32_t Tk, int32_t max_k, int32_t window) {
  if (!cu_k) return fail(VA_ERR_INVALID_ARG, "cross: cu_seqlens_k is null");
  if (Tk < 1 || max_k < 1 || max_k > Tk) return fail(VA_ERR_INVALID_ARG, "cross: Tk >= 1 and 1 <= max_seqlen_k <= Tk");
  if (static_cast<int64_t>(Tk) * s->Hkv >= (int64_t(1) << 31)) return fail(VA_ERR_UNSUPPORTED, "Tk * Hkv must stay below 2^31");
  if (window != -1) return fail(VA_ERR_UNSUPPORTED, "cross: no local window");
  return VA_OK;
}

va_status check_shape(const va_shape* s) {
  if (!s) return fail(VA_ERR_INVALID_ARG, "shape is null");
  if (s->T < 0 || s->B < 1 || s->Hq < 1 || s->Hkv < 1 || s->max_seqlen < 1)
    return fail(VA_ERR_INVALID_ARG, "shape: T >= 0, B >= 1, heads >= 1, max_seqlen >= 1");
  if (s->d != 64 && s->d != 128) return fail(VA_ERR_UNSUPPORTED, "head dim must be 64 or 128");
  if (s->Hq % s->Hkv) return fail(VA_ERR_UNSUPPORTED, "Hq must be a multiple of Hkv");
  if (s->max_seqlen > std::max(s->T, 1)) return fail(VA_ERR_INVALID_ARG, "max_seqlen > T");
  const int64_t st[8] = {s->q_row_stride, s->q_head_stride, s->k_row_stride, s->k_head_stride,
                         s->v_row_stride, s->v_head_stride, s->o_row_stride, s->o_head_stride};
  for (int64_t x : st)
    if (x <= 0 || x % 8) return fail(VA_ERR_INVALID_ARG, "strides must be positive multiples of 8");
  for (int64_t x : st)
    if (x < s->d) return fail(VA_ERR_INVALID_ARG, "row and head strides must be >= d");
  if (static_cast<int64_t>(s->T) * std::max(s->Hq, s->Hkv) >= (int64_t(1) << 31))
    return fail(VA_ERR_UNSUPPORTED, "T * heads must stay below 2^31");
  return VA_OK;
}

// Window and sink arguments of a valid shape.  No query sees further back than the longest
// segment, so both are cut to it: the kernels' column arithmetic then stays far inside 32 bits.
va_status check_window(const va_shape* s, int32_t causal, int32_t* window, int32_t* sinks, const char* where) {
  if (*window < -1 || (*window >= 0 && !causal))
    return fail(VA_ERR_INVALID_ARG, std::string(where) + ": window needs causal and >= 0 (-1 = none)");
  if (*sinks < 0 || (*sinks > 0 && *window < 0))
    return fail(VA_ERR_INVALID_ARG, std::string(where) + ": sinks >= 0, and sinks need a window");
  *window = std::min(*window, s->max_seqlen);
  *sinks = std::min(*sinks, s->max_seqlen);
  return VA_OK;
}

// A window or sinks over the longest segment hide nothing: such a call is the causal one, whose kernels
// mask less and take runs of short segments as token tiles (T = 29254, segments of 3 to 18 tokens, 8/2
// heads of 64, window 1619, forward and backward: 851 us with the window's kernels, 167 without).
void drop_whole_window(const va_shape* s, int32_t* window, int32_t* sinks) {
  if (*window >= 0 && (*window >= s->max_seqlen - 1 || *sinks >= s->max_seqlen - 1)) {
    *window = -1;
    *sinks = 0;
  }
}

struct FwdLayout {
  size_t map, segoff, total;
  int64_t cap;
};
FwdLayout fwd_layout(const va_shape& s) {
  FwdLayout L;
  L.cap = map_capacity(s, 0);
  L.map = sizeof(WsHeader);
  L.segoff = align256(L.map + static_cast<size_t>(L.cap) * sizeof(TileItem));
  L.total = align256(L.segoff + static_cast<size_t>(s.B) * sizeof(int32_t));
  return L;
}

// q blocks per piece of a kv block that holds sinks, or 0 when its records stay whole.  Such a block is
// seen by its whole segment, max_seqlen / 64 q blocks for each of the g q heads in one serial item, while
// the others see a window.  The map starts with these items, but one longer than an SM's share of all
// steps sets the call's time; then they are cut into pieces of a quarter of the share (with more sink
// blocks, which are more items, longer ones).  The kernel form for pieces costs 3% of dK/dV, hence not
// always.  (d = 128, window 1023, one segment: T = 65536, 12 q heads on one kv head, backward 9.40 ms
// whole, 1.27 in pieces; T = 16384, 32 on 8, 1.18 and 0.81.)
int sink_piece(const va_shape& s, int window, int sinks) {
  if (sinks <= 0) return 0;
  constexpr int kSms = 152;  // a constant: the workspace size must not depend on the device
  const int64_t g = s.Hq / s.Hkv, blocks = (sinks + 127) / 128;
  const int64_t share = static_cast<int64_t>(s.Hq) * (s.T / 128 + 1) * (window / 64 + 2) / kSms;
  const int64_t longest = g * (s.max_seqlen / 64 + 1);
  if (longest <= std::max<int64_t>(share, 64)) return 0;  // (64 steps: 50 us)
  const int64_t P = std::max<int64_t>(8, (share / 4 + g - 1) / g) * ((blocks + 1) / 2);
  return 64 * P < s.max_seqlen ? static_cast<int>(P) : 0;
}

struct BwdLayout {
  size_t dsum, kvmap, qmap, segoff, part, total;
  int64_t cap_kv, cap_q;
  int piece;
};
BwdLayout bwd_layout(const va_shape& s, int Tk = -1, int window = -1, int sinks = 0) {
  BwdLayout L;
  L.cap_kv = map_capacity(s, 1, Tk);
  L.piece = sink_piece(s, window, sinks);
  const int64_t blocks = (sinks + 127) / 128;
  if (L.piece > 0) L.cap_kv += blocks * (s.T / (64 * L.piece) + 1) * s.Hkv;
  L.cap_q = map_capacity(s, 2);
  L.dsum = sizeof(WsHeader);
  L.kvmap = align256(L.dsum + static_cast<size_t>(s.Hq) * s.T * sizeof(float));
  L.qmap = align256(L.kvmap + static_cast<size_t>(L.cap_kv) * sizeof(TileItem));
  L.segoff = align256(L.qmap + static_cast<size_t>(L.cap_q) * sizeof(TileItem));
  L.part = align256(L.segoff + static_cast<size_t>(s.B) * sizeof(int32_t));
  L.total = L.part;
  if (L.piece > 0)
    L.total += static_cast<size_t>(sink_slots(s.T, L.piece)) * blocks * s.Hkv * 2 * 128 * s.d * sizeof(float);
  return L;
}

}  // namespace
}  // namespace va

using namespace va;

static va_status plan_impl(const va_shape* s, const int32_t* cu_dev, const int32_t* cu_k, int32_t Tk, int32_t kind,
                           int32_t causal, int32_t window, int32_t sinks, int32_t* map_dev, int32_t capacity,
                           int32_t* n_items_dev, int32_t* scratch_dev, va_stream_t stream);
static va_status fwd_impl(const void* q, const void* k, const void* v, const int32_t* cu, const int32_t* cu_k,
                          int32_t Tk, int32_t max_k, const va_shape* s, float scale, int32_t causal, int32_t window,
                          int32_t sinks, void* out, float* lse, void* ws, size_t ws_bytes, va_stream_t stream);
static va_status bwd_impl(const void* q, const void* k, const void* v, const void* out, const float* lse,
                          const void* dout, const int32_t* cu, const int32_t* cu_k, int32_t Tk, int32_t max_k,
                          const va_shape* s, float scale, int32_t causal, int32_t window, int32_t sinks, void* dq,
                          void* dk, void* dv, void* ws, size_t ws_bytes, va_stream_t stream);

extern "C" {

const char* varlen_last_error(void) { return g_error.c_str(); }

const char* varlen_version(void) { return "varlen_attn 0.1 (sm_103a)"; }

void varlen_shape_contiguous(va_shape* s, int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                             int32_t max_seqlen) {
  if (!s) return;
  s->T = T;
  s->B = B;
  s->Hq = Hq;
  s->Hkv = Hkv;
  s->d = d;
  s->max_seqlen = max_seqlen;
  s->q_row_stride = static_cast<int64_t>(Hq) * d;
  s->q_head_stride = d;
  s->k_row_stride = static_cast<int64_t>(Hkv) * d;
  s->k_head_stride = d;
  s->v_row_stride = static_cast<int64_t>(Hkv) * d;
  s->v_head_stride = d;
  s->o_row_stride = static_cast<int64_t>(Hq) * d;
  s->o_head_stride = d;
}

va_status varlen_build_metadata(const int32_t* lengths_dev, int32_t n, int32_t pad_to,
                                int32_t T_capacity, int32_t* cu_dev, int32_t* pos_dev,
                                int32_t* seg_dev, int32_t* max_dev, int32_t* status_dev,
                                va_stream_t stream) {
  if (n < 0 || pad_to < 0 || T_capacity < 0 || !cu_dev || !max_dev || !status_dev ||
      (n > 0 && !lengths_dev) || (T_capacity > 0 && (!pos_dev || !seg_dev)))
    return fail(VA_ERR_INVALID_ARG, "build_metadata: null pointer or negative size");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch(K_META_SCAN, cs, [&] {
    return launch_metadata_scan(lengths_dev, n, pad_to, T_capacity, cu_dev, max_dev, status_dev, pos_dev, seg_dev,
                                cs);
  });
  // short streams get their positions and segment ids from the scan's block
  if (e == cudaSuccess && T_capacity > 0 && !metadata_inline_fill(n, T_capacity))
    e = launch(K_META_FILL, cs, [&] {
      return launch_metadata_fill(cu_dev, n, T_capacity, pos_dev, seg_dev, status_dev, cs);
    });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "build_metadata");
}

va_status varlen_validate_cu_seqlens(const int32_t* cu_dev, int32_t B, int32_t T, int32_t max_seqlen,
                                     int32_t* status_dev, va_stream_t stream) {
  if (!cu_dev || !status_dev || B < 1 || T < 0 || max_seqlen < 1)
    return fail(VA_ERR_INVALID_ARG, "validate: null pointer or bad size");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch(K_VALIDATE, cs, [&] {
    return launch_validate(cu_dev, B, T, max_seqlen, status_dev, 0, cs);
  });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "validate");
}

va_status varlen_cu_seqlens_from_positions(const int32_t* position_ids_dev, int32_t T, int32_t reset_at_min,
                                           int32_t strict, int32_t* cu_seqlens_dev, int32_t capacity,
                                           int32_t* B_dev, int32_t* max_seqlen_dev, int32_t* status_dev,
                                           va_stream_t stream) {
  if (!position_ids_dev || !cu_seqlens_dev || !B_dev || !max_seqlen_dev || !status_dev)
    return fail(VA_ERR_INVALID_ARG, "cu_seqlens_from_positions: null pointer");
  if (T < 1 || capacity < 2)
    return fail(VA_ERR_INVALID_ARG, "cu_seqlens_from_positions: T >= 1 and capacity >= 2");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch(K_CU_FROM_POS, cs, [&] {
    return launch_cu_from_positions(position_ids_dev, T, reset_at_min ? 1 : 0, strict ? 1 : 0, cu_seqlens_dev,
                                    capacity, B_dev, max_seqlen_dev, status_dev, cs);
  });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "cu_seqlens_from_positions");
}

va_status varlen_attn_tile_sizes(int32_t kind, int32_t d, int32_t* BM, int32_t* BN) {
  if (kind < 0 || kind > 2 || !BM || !BN) return fail(VA_ERR_INVALID_ARG, "tile_sizes: bad kind");
  if (d != 64 && d != 128) return fail(VA_ERR_UNSUPPORTED, "tile_sizes: d must be 64 or 128");
  int a, b;
  tiles(kind, &a, &b);
  *BM = a;
  *BN = b;
  return VA_OK;
}

size_t varlen_attn_workspace_size(const va_shape* s, int32_t for_bwd) {
  if (check_shape(s) != VA_OK) return 0;
  return for_bwd ? bwd_layout(*s).total : fwd_layout(*s).total;
}

size_t varlen_attn_workspace_size_sinks(const va_shape* s, int32_t window, int32_t sinks, int32_t for_bwd) {
  if (check_shape(s) != VA_OK || check_window(s, 1, &window, &sinks, "workspace_size") != VA_OK) return 0;
  drop_whole_window(s, &window, &sinks);
  return for_bwd ? bwd_layout(*s, -1, window, sinks).total : fwd_layout(*s).total;
}

va_status varlen_attn_plan(const va_shape* s, const int32_t* cu_dev, int32_t kind, int32_t causal,
                           int32_t* map_dev, int32_t capacity, int32_t* n_items_dev,
                           int32_t* scratch_dev, va_stream_t stream) {
  return varlen_attn_plan_window(s, cu_dev, kind, causal, -1, map_dev, capacity, n_items_dev, scratch_dev, stream);
}

va_status varlen_attn_plan_window(const va_shape* s, const int32_t* cu_dev, int32_t kind, int32_t causal,
                                  int32_t window, int32_t* map_dev, int32_t capacity, int32_t* n_items_dev,
                                  int32_t* scratch_dev, va_stream_t stream) {
  return plan_impl(s, cu_dev, nullptr, -1, kind, causal, window, 0, map_dev, capacity, n_items_dev, scratch_dev, stream);
}

va_status varlen_attn_plan_sinks(const va_shape* s, const int32_t* cu_dev, int32_t kind, int32_t causal,
                                 int32_t window, int32_t sinks, int32_t* map_dev, int32_t capacity,
                                 int32_t* n_items_dev, int32_t* scratch_dev, va_stream_t stream) {
  return plan_impl(s, cu_dev, nullptr, -1, kind, causal, window, sinks, map_dev, capacity, n_items_dev, scratch_dev,
                   stream);
}

va_status varlen_attn_plan_cross(const va_shape* s, const int32_t* cu_q, const int32_t* cu_k, int32_t Tk, int32_t kind,
                                 int32_t causal, int32_t* map_dev, int32_t capacity, int32_t* n_items_dev,
                                 int32_t* scratch_dev, va_stream_t stream) {
  return plan_impl(s, cu_q, cu_k, Tk, kind, causal, -1, 0, map_dev, capacity, n_items_dev, scratch_dev, stream);
}

}  // extern "C"

static va_status plan_impl(const va_shape* s, const int32_t* cu_dev, const int32_t* cu_k, int32_t Tk, int32_t kind,
                           int32_t causal, int32_t window, int32_t sinks, int32_t* map_dev, int32_t capacity,
                           int32_t* n_items_dev, int32_t* scratch_dev, va_stream_t stream) {
  va_status st = check_shape(s);
  if (st != VA_OK) return st;
  if (cu_k && (st = check_cross(s, cu_k, Tk, std::max(Tk, 1), window)) != VA_OK) return st;
  if ((st = check_window(s, causal, &window, &sinks, "plan")) != VA_OK) return st;
  if (kind < 0 || kind > 2 || !cu_dev || !map_dev || !n_items_dev || !scratch_dev || capacity < 0)
    return fail(VA_ERR_INVALID_ARG, "plan: bad kind or null pointer");
  if (!aligned16(map_dev)) return fail(VA_ERR_INVALID_ARG, "plan: tile map must be 16-byte aligned");
  if (map_capacity(*s, kind, cu_k ? Tk : -1) > capacity)
    return fail(VA_ERR_WORKSPACE, "plan: capacity below the record bound (T/blk + B) * heads");
  int BM, BN;
  tiles(kind, &BM, &BN);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const PlanArgs pa{cu_dev, s->B, kind == 1 ? s->Hkv : s->Hq, BM, BN, kind, causal ? 1 : 0,
                    reinterpret_cast<TileItem*>(map_dev), capacity, nullptr, n_items_dev,
                    scratch_dev + 4, scratch_dev,
                    (cu_k || !token_tiles(*s, causal, window)) ? 0
                    : kind == 0                                ? fwd_tc_token_short()
                                                               : bwd_tc_token_short(),
                    nullptr, nullptr, window, cu_k, sinks};
  cudaError_t e = launch(K_PLAN, cs, [&] { return launch_plan(pa, cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "plan");
}

extern "C" {

va_status varlen_attn_fwd(const void* q, const void* k, const void* v, const int32_t* cu,
                          const va_shape* s, float scale, int32_t causal, void* out, float* lse,
                          void* ws, size_t ws_bytes, va_stream_t stream) {
  return varlen_attn_fwd_window(q, k, v, cu, s, scale, causal, -1, out, lse, ws, ws_bytes, stream);
}

va_status varlen_attn_fwd_window(const void* q, const void* k, const void* v, const int32_t* cu,
                                 const va_shape* s, float scale, int32_t causal, int32_t window, void* out,
                                 float* lse, void* ws, size_t ws_bytes, va_stream_t stream) {
  return fwd_impl(q, k, v, cu, nullptr, -1, 0, s, scale, causal, window, 0, out, lse, ws, ws_bytes, stream);
}

va_status varlen_attn_fwd_sinks(const void* q, const void* k, const void* v, const int32_t* cu, const va_shape* s,
                                float scale, int32_t causal, int32_t window, int32_t sinks, void* out, float* lse,
                                void* ws, size_t ws_bytes, va_stream_t stream) {
  return fwd_impl(q, k, v, cu, nullptr, -1, 0, s, scale, causal, window, sinks, out, lse, ws, ws_bytes, stream);
}

va_status varlen_attn_fwd_cross(const void* q, const void* k, const void* v, const int32_t* cu_q,
                                const int32_t* cu_k, const va_shape* s, int32_t Tk, int32_t max_seqlen_k, float scale,
                                int32_t causal, void* out, float* lse, void* ws, size_t ws_bytes, va_stream_t stream) {
  return fwd_impl(q, k, v, cu_q, cu_k, Tk, max_seqlen_k, s, scale, causal, -1, 0, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"

static va_status fwd_impl(const void* q, const void* k, const void* v, const int32_t* cu, const int32_t* cu_k,
                          int32_t Tk, int32_t max_k, const va_shape* s, float scale, int32_t causal, int32_t window,
                          int32_t sinks, void* out, float* lse, void* ws, size_t ws_bytes, va_stream_t stream) {
  va_status st = check_shape(s);
  if (st != VA_OK) return st;
  if (cu_k && (st = check_cross(s, cu_k, Tk, max_k, window)) != VA_OK) return st;
  if ((st = check_window(s, causal, &window, &sinks, "fwd")) != VA_OK) return st;
  drop_whole_window(s, &window, &sinks);
  if (!q || !k || !v || !cu || !out || !lse || !ws)
    return fail(VA_ERR_INVALID_ARG, "fwd: null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(ws))
    return fail(VA_ERR_INVALID_ARG, "fwd: pointers must be 16-byte aligned");
  if (!(scale > 0.f) || !(scale < INFINITY)) return fail(VA_ERR_INVALID_ARG, "fwd: scale must be finite and > 0");
  const FwdLayout L = fwd_layout(*s);
  if (ws_bytes < L.total) return fail(VA_ERR_WORKSPACE, "fwd: workspace too small");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(w);
  TileItem* map = reinterpret_cast<TileItem*>(w + L.map);
  if (s->T == 0) {  // nothing to compute; still report a contract violation
    cudaError_t e = launch(K_VALIDATE, cs, [&] {
      return launch_validate(cu, s->B, s->T, s->max_seqlen, &hdr->status, 1, cs);
    });
    return e == cudaSuccess ? VA_OK : cuda_fail(e, "fwd validate");
  }
  int BM, BN;
  tiles(0, &BM, &BN);
  const bool tok = !cu_k && call_token_tiles(*s, causal, window);
  const PlanArgs pa{cu, s->B, s->Hq, BM, BN, 0, causal ? 1 : 0, map, static_cast<int>(L.cap),
                    &hdr->status, &hdr->n_items[0],
                    reinterpret_cast<int32_t*>(w + L.segoff), &hdr->counter[0],
                    tok ? fwd_tc_token_short() : 0, &hdr->n_items[kTokSlot],
                    &hdr->counter[kTokSlot], window, cu_k, sinks};
  cudaError_t e = launch(K_VALIDATE_PLAN, cs, [&] {
    return launch_validate_plan(&pa, 1, s->T, s->max_seqlen, cu_k ? Tk : 0, cu_k ? max_k : 0, cs);
  });
  if (e != cudaSuccess) return cuda_fail(e, "fwd plan");
  FwdParams p{};
  p.q = static_cast<const bf16*>(q);
  p.k = static_cast<const bf16*>(k);
  p.v = static_cast<const bf16*>(v);
  p.o = static_cast<bf16*>(out);
  p.lse = lse;
  p.cu = cu;
  p.items = map;
  p.B = s->B;
  p.hdr = hdr;
  p.slot = 0;
  p.counter = &hdr->counter[0];
  p.T = s->T;
  p.Hq = s->Hq;
  p.Hkv = s->Hkv;
  p.g = s->Hq / s->Hkv;
  p.q_rs = s->q_row_stride;
  p.q_hs = s->q_head_stride;
  p.k_rs = s->k_row_stride;
  p.k_hs = s->k_head_stride;
  p.v_rs = s->v_row_stride;
  p.v_hs = s->v_head_stride;
  p.o_rs = s->o_row_stride;
  p.o_hs = s->o_head_stride;
  p.scale_log2 = scale * kLog2e;
  p.causal = causal ? 1 : 0;
  p.window = window;
  p.sinks = sinks;
  p.cu_k = cu_k;
  p.Tk = cu_k ? Tk : 0;
  const long long stall_ns = g_stall_next_fwd.exchange(0);
  if (stall_ns > 0) {  // test hook: the producers load nothing and the waits give up after stall_ns
    p.wait_ns = static_cast<uint64_t>(stall_ns);
    p.stall = 1;
  }
  // segment records, then (as its programmatic dependent, filling its tail) token records
  e = launch(K_FWD, cs, [&] { return launch_fwd_tc(p, s->d, static_cast<int>(L.cap), cs); });
  if (e != cudaSuccess) return cuda_fail(e, "fwd kernel");
  if (!tok) return VA_OK;
  FwdParams pt = p;
  pt.counter = &hdr->counter[kTokSlot];
  e = launch(K_FWD_TOK, cs, [&] { return launch_fwd_tok(pt, s->d, static_cast<int>(L.cap), cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "fwd token kernel");
}

extern "C" {

va_status varlen_attn_bwd(const void* q, const void* k, const void* v, const void* out,
                          const float* lse, const void* dout, const int32_t* cu, const va_shape* s,
                          float scale, int32_t causal, void* dq, void* dk, void* dv, void* ws,
                          size_t ws_bytes, va_stream_t stream) {
  return varlen_attn_bwd_window(q, k, v, out, lse, dout, cu, s, scale, causal, -1, dq, dk, dv, ws, ws_bytes,
                                stream);
}

va_status varlen_attn_bwd_window(const void* q, const void* k, const void* v, const void* out,
                                 const float* lse, const void* dout, const int32_t* cu, const va_shape* s,
                                 float scale, int32_t causal, int32_t window, void* dq, void* dk, void* dv,
                                 void* ws, size_t ws_bytes, va_stream_t stream) {
  return bwd_impl(q, k, v, out, lse, dout, cu, nullptr, -1, 0, s, scale, causal, window, 0, dq, dk, dv, ws, ws_bytes,
                  stream);
}

va_status varlen_attn_bwd_sinks(const void* q, const void* k, const void* v, const void* out, const float* lse,
                                const void* dout, const int32_t* cu, const va_shape* s, float scale, int32_t causal,
                                int32_t window, int32_t sinks, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                va_stream_t stream) {
  return bwd_impl(q, k, v, out, lse, dout, cu, nullptr, -1, 0, s, scale, causal, window, sinks, dq, dk, dv, ws,
                  ws_bytes, stream);
}

va_status varlen_attn_bwd_cross(const void* q, const void* k, const void* v, const void* out, const float* lse,
                                const void* dout, const int32_t* cu_q, const int32_t* cu_k, const va_shape* s,
                                int32_t Tk, int32_t max_seqlen_k, float scale, int32_t causal, void* dq, void* dk,
                                void* dv, void* ws, size_t ws_bytes, va_stream_t stream) {
  return bwd_impl(q, k, v, out, lse, dout, cu_q, cu_k, Tk, max_seqlen_k, s, scale, causal, -1, 0, dq, dk, dv, ws,
                  ws_bytes, stream);
}

size_t varlen_attn_workspace_size_cross(const va_shape* s, int32_t Tk, int32_t for_bwd) {
  if (check_shape(s) != VA_OK || Tk < 1) return 0;
  return for_bwd ? bwd_layout(*s, Tk).total : fwd_layout(*s).total;
}

}  // extern "C"

static va_status bwd_impl(const void* q, const void* k, const void* v, const void* out, const float* lse,
                          const void* dout, const int32_t* cu, const int32_t* cu_k, int32_t Tk, int32_t max_k,
                          const va_shape* s, float scale, int32_t causal, int32_t window, int32_t sinks, void* dq,
                          void* dk, void* dv, void* ws, size_t ws_bytes, va_stream_t stream) {
  va_status st = check_shape(s);
  if (st != VA_OK) return st;
  if (cu_k && (st = check_cross(s, cu_k, Tk, max_k, window)) != VA_OK) return st;
  if ((st = check_window(s, causal, &window, &sinks, "bwd")) != VA_OK) return st;
  drop_whole_window(s, &window, &sinks);
  if (!q || !k || !v || !out || !lse || !dout || !cu || !dq || !dk || !dv || !ws)
    return fail(VA_ERR_INVALID_ARG, "bwd: null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(dout) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(ws))
    return fail(VA_ERR_INVALID_ARG, "bwd: pointers must be 16-byte aligned");
  if (!(scale > 0.f) || !(scale < INFINITY)) return fail(VA_ERR_INVALID_ARG, "bwd: scale must be finite and > 0");
  const BwdLayout L = bwd_layout(*s, cu_k ? Tk : -1, window, sinks);
  if (ws_bytes < L.total) return fail(VA_ERR_WORKSPACE, "bwd: workspace too small");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(w);
  TileItem* kvmap = reinterpret_cast<TileItem*>(w + L.kvmap);
  TileItem* qmap = reinterpret_cast<TileItem*>(w + L.qmap);
  if (s->T == 0) {
    cudaError_t e = launch(K_VALIDATE, cs, [&] {
      return launch_validate(cu, s->B, s->T, s->max_seqlen, &hdr->status, 1, cs);
    });
    return e == cudaSuccess ? VA_OK : cuda_fail(e, "bwd validate");
  }
  int BM, BN, BM2, BN2;
  tiles(1, &BM, &BN);
  tiles(2, &BM2, &BN2);
  const bool tok = !cu_k && L.piece == 0 && call_token_tiles(*s, causal, window);
  int32_t* segoff = reinterpret_cast<int32_t*>(w + L.segoff);
  const PlanArgs pa[2] = {
      {cu, s->B, s->Hkv, BM, BN, 1, causal ? 1 : 0, kvmap, static_cast<int>(L.cap_kv), &hdr->status,
       &hdr->n_items[1], segoff, &hdr->counter[1], tok ? bwd_tc_token_short() : 0,
       &hdr->n_items[kKvTokSlot], nullptr, window, cu_k, sinks, L.piece},
      {cu, s->B, s->Hq, BM2, BN2, 2, causal ? 1 : 0, qmap, static_cast<int>(L.cap_q), &hdr->status,
       &hdr->n_items[2], segoff, &hdr->counter[2], tok ? bwd_tc_token_short() : 0,
       &hdr->n_items[kQTokSlot], nullptr, window, cu_k, sinks}};
  BwdParams p{};
  p.q = static_cast<const bf16*>(q);
  p.k = static_cast<const bf16*>(k);
  p.v = static_cast<const bf16*>(v);
  p.o = static_cast<const bf16*>(out);
  p.dout = static_cast<const bf16*>(dout);
  p.lse = lse;
  p.dsum = reinterpret_cast<float*>(w + L.dsum);
  p.dq = static_cast<bf16*>(dq);
  p.dk = static_cast<bf16*>(dk);
  p.dv = static_cast<bf16*>(dv);
  p.cu = cu;
  p.B = s->B;
  p.kv_items = kvmap;
  p.q_items = qmap;
  p.hdr = hdr;
  p.kv_slot = 1;
  p.q_slot = 2;
  p.kv_tok_slot = kKvTokSlot;
  p.q_tok_slot = kQTokSlot;
  p.kv_counter = &hdr->counter[1];
  p.q_counter = &hdr->counter[2];
  p.T = s->T;
  p.Hq = s->Hq;
  p.Hkv = s->Hkv;
  p.g = s->Hq / s->Hkv;
  p.q_rs = s->q_row_stride;
  p.q_hs = s->q_head_stride;
  p.k_rs = s->k_row_stride;
  p.k_hs = s->k_head_stride;
  p.v_rs = s->v_row_stride;
  p.v_hs = s->v_head_stride;
  p.o_rs = s->o_row_stride;
  p.o_hs = s->o_head_stride;
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  p.causal = causal ? 1 : 0;
  p.window = window;
  p.sinks = sinks;
  p.piece = L.piece;
  p.sink_blocks = (sinks + 127) / 128;
  p.part = reinterpret_cast<float*>(w + L.part);
  p.cu_k = cu_k;
  p.Tk = cu_k ? Tk : 0;
  // one launch validates, plans both maps and computes D = rowsum(dO * O)
  cudaError_t e = launch(K_BWD_PREP, cs, [&] {
    return launch_bwd_prep(p, pa, 2, s->T, s->max_seqlen, cu_k ? Tk : 0, cu_k ? max_k : 0, s->d, cs);
  });
  if (e == cudaSuccess)
    e = launch(K_BWD_DKDV, cs, [&] { return launch_bwd_dkdv_tc(p, s->d, static_cast<int>(L.cap_kv), tok, cs); });
  if (e == cudaSuccess)
    e = launch(K_BWD_DQ, cs, [&] { return launch_bwd_dq_tc(p, s->d, static_cast<int>(L.cap_q), tok, cs); });
  if (e == cudaSuccess && L.piece > 0) e = launch(K_SINK_JOIN, cs, [&] { return launch_sink_join(p, s->d, cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "bwd kernels");
}

extern "C" {

va_status varlen_unpad_index(const int32_t* mask, int32_t Bp, int32_t S, int32_t* indices, int32_t* inverse,
                             int32_t* cu, int32_t* T_out, int32_t* max_out, int32_t* status, va_stream_t stream) {
  if (!mask || !indices || !inverse || !cu || !T_out || !max_out || !status)
    return fail(VA_ERR_INVALID_ARG, "unpad_index: null pointer");
  if (Bp < 1 || S < 1 || static_cast<int64_t>(Bp) * S >= (int64_t(1) << 31))
    return fail(VA_ERR_INVALID_ARG, "unpad_index: Bp >= 1, S >= 1 and Bp * S < 2^31");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const KernelId ids[3] = {K_PAD_COUNT, K_PAD_SCAN, K_PAD_INDEX};
  cudaError_t e = cudaSuccess;
  for (int stage = 0; stage < 3 && e == cudaSuccess; ++stage)
    e = launch(ids[stage], cs, [&] {
      return launch_unpad_index(stage, mask, Bp, S, indices, inverse, cu, T_out, max_out, status, cs);
    });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "unpad_index");
}

va_status varlen_gather_rows(const void* src, int64_t src_stride, const int32_t* map, int32_t n_rows, int64_t row_bytes,
                             void* dst, int64_t dst_stride, va_stream_t stream) {
  if (!src || !map || !dst || n_rows < 0) return fail(VA_ERR_INVALID_ARG, "gather_rows: null pointer or n_rows < 0");
  if (row_bytes <= 0 || row_bytes % 16 || src_stride % 16 || dst_stride % 16 || src_stride < row_bytes ||
      dst_stride < row_bytes || !aligned16(src) || !aligned16(dst))
    return fail(VA_ERR_INVALID_ARG, "gather_rows: rows, strides and pointers must be 16-byte multiples");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch(K_GATHER_ROWS, cs, [&] {
    return launch_gather_rows(src, src_stride, map, n_rows, row_bytes, dst, dst_stride, cs);
  });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "gather_rows");
}

va_status varlen_loss_targets(const int32_t* ids, const int32_t* cu, int32_t B, int32_t T, int32_t ignore_index,
                              int32_t* targets, va_stream_t stream) {
  if (!ids || !cu || !targets || T < 0 || B < 1) return fail(VA_ERR_INVALID_ARG, "loss_targets: null pointer or bad size");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch(K_LOSS_TARGETS, cs, [&] { return launch_loss_targets(ids, cu, B, T, ignore_index, targets, cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "loss_targets");
}

size_t varlen_token_ce_workspace_size(int32_t T) {
  return T < 0 ? 0 : align256(sizeof(WsHeader) + static_cast<size_t>(T) * sizeof(float));
}

va_status varlen_token_ce(const void* logits, int32_t dtype, int64_t l_rs, const int32_t* targets, int32_t T,
                          int32_t V, int32_t ignore_index, double* loss, int32_t* count, void* grad, int64_t g_rs,
                          void* ws, size_t ws_bytes, va_stream_t stream) {
  if (!logits || !targets || !loss || !count || !ws) return fail(VA_ERR_INVALID_ARG, "token_ce: null pointer");
  if (T < 1 || V < 1 || (dtype != 0 && dtype != 1)) return fail(VA_ERR_INVALID_ARG, "token_ce: T, V >= 1, dtype 0 or 1");
  if (l_rs < V || (grad && g_rs < V)) return fail(VA_ERR_INVALID_ARG, "token_ce: row strides must be >= V");
  if (!aligned16(ws)) return fail(VA_ERR_INVALID_ARG, "token_ce: workspace must be 16-byte aligned");
  if (ws_bytes < varlen_token_ce_workspace_size(T)) return fail(VA_ERR_WORKSPACE, "token_ce: workspace too small");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(w);
  float* nll = reinterpret_cast<float*>(w + sizeof(WsHeader));
  cudaError_t e = cudaSuccess;
  const KernelId ids[3] = {K_CE_COUNT, K_CE_ROWS, K_CE_REDUCE};
  for (int stage = 0; stage < 3 && e == cudaSuccess; ++stage)
    e = launch(ids[stage], cs, [&] {
      return launch_token_ce(stage, logits, dtype, l_rs, targets, T, V, ignore_index, grad, g_rs, nll, count,
                             &hdr->status, loss, cs);
    });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "token_ce");
}

size_t varlen_token_distill_workspace_size(int32_t T) {
  if (T < 0) return 0;
  return align256(sizeof(WsHeader) + distill_parts_bytes() + static_cast<size_t>(T));
}

va_status varlen_token_distill(const void* logits, int32_t dtype, int64_t l_rs, const int32_t* ids, int64_t ids_rs,
                               const void* tl, int32_t t_dtype, int64_t t_rs, const int32_t* targets, int32_t T,
                               int32_t V, int32_t K, int32_t ignore_index, float temperature, float* loss,
                               int32_t* count, void* grad, int64_t g_rs, void* ws, size_t ws_bytes,
                               va_stream_t stream) {
  if (!logits || !ids || !tl || !loss || !count || !ws) return fail(VA_ERR_INVALID_ARG, "token_distill: null pointer");
  if (T < 1 || T >= (1 << 30) || V < 1 || K < 1 || (dtype != 0 && dtype != 1) || (t_dtype != 0 && t_dtype != 1))
    return fail(VA_ERR_INVALID_ARG, "token_distill: 1 <= T < 2^30, V and K >= 1, dtypes 0 or 1");
  if (K > 1024) return fail(VA_ERR_UNSUPPORTED, "token_distill: at most 1024 teacher entries per row");
  if (!distill_row_fits(V, dtype == 1 ? 2 : 4))
    return fail(VA_ERR_UNSUPPORTED, "token_distill: a row of logits must stay within 1,310,720 bytes");
  if (l_rs < V || ids_rs < K || t_rs < K || (grad && g_rs < V))
    return fail(VA_ERR_INVALID_ARG, "token_distill: row strides must be >= the row");
  const uintptr_t ea = dtype == 1 ? 1 : 3;
  if ((reinterpret_cast<uintptr_t>(logits) & ea) || (reinterpret_cast<uintptr_t>(grad) & ea))
    return fail(VA_ERR_INVALID_ARG, "token_distill: logits and grad must be aligned to their type");
  // The row loss is a difference of logarithms of size ln V held in fp32, times the temperature's
  // square: at 64 its error reaches 2^12 2^-24 2 ln V = 0.006 for V = 131072, beyond it the loss drowns.
  if (!(temperature >= 1.f / 64) || !(temperature <= 64.f))
    return fail(VA_ERR_INVALID_ARG, "token_distill: temperature must be in [1/64, 64]");
  if (!aligned16(ws)) return fail(VA_ERR_INVALID_ARG, "token_distill: workspace must be 16-byte aligned");
  if (ws_bytes < varlen_token_distill_workspace_size(T))
    return fail(VA_ERR_WORKSPACE, "token_distill: workspace too small");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  int32_t* parts = reinterpret_cast<int32_t*>(w + sizeof(WsHeader));
  uint8_t* flags = w + sizeof(WsHeader) + distill_parts_bytes();
  cudaError_t e = cudaSuccess;
  const uint64_t stall_ns = static_cast<uint64_t>(g_stall_next_distill.exchange(0));
  const KernelId kid[3] = {K_DISTILL_COUNT, K_DISTILL_ROWS, K_DISTILL_REDUCE};
  for (int stage = 0; stage < 3 && e == cudaSuccess; ++stage)
    e = launch(kid[stage], cs, [&] {
      return launch_token_distill(stage, logits, dtype, l_rs, ids, ids_rs, tl, t_dtype, t_rs, targets, T, V, K,
                                  ignore_index, temperature, grad, g_rs, w, parts, flags, loss, count, stall_ns, cs);
    });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "token_distill");
}

static va_status check_embed(const char* where, const void* a, const void* b, const int32_t* ids, int32_t dtype_a,
                             int32_t dtype_b, int64_t a_rs, int64_t b_rs, int32_t T, int32_t V, int32_t D,
                             float scale) {
  const std::string w(where);
  if (!a || !b || (T > 0 && !ids)) return fail(VA_ERR_INVALID_ARG, w + ": null pointer");
  // (D: the columns of the gradient's grid, 2048 a block, stay within 65535 blocks)
  if (T < 0 || T >= (1 << 30) || V < 1 || V >= (1 << 30) || D < 1 || D > (1 << 26))
    return fail(VA_ERR_INVALID_ARG, w + ": 0 <= T < 2^30, 1 <= V < 2^30, 1 <= D <= 2^26");
  if (dtype_a < 0 || dtype_a > 1 || dtype_b < 0 || dtype_b > 1) return fail(VA_ERR_INVALID_ARG, w + ": dtypes 0 or 1");
  if (a_rs < D || b_rs < D) return fail(VA_ERR_INVALID_ARG, w + ": row strides must be >= D");
  if ((reinterpret_cast<uintptr_t>(a) & (dtype_a == 1 ? 1 : 3)) || (reinterpret_cast<uintptr_t>(b) & (dtype_b == 1 ? 1 : 3)))
    return fail(VA_ERR_INVALID_ARG, w + ": pointers must be aligned to their type");
  if (!(scale > -INFINITY && scale < INFINITY)) return fail(VA_ERR_INVALID_ARG, w + ": scale must be finite");
  return VA_OK;
}

va_status varlen_embed_fwd(const void* table, int32_t dtype, int64_t t_rs, const int32_t* ids, int32_t T, int32_t V,
                           int32_t D, float scale, void* out, int64_t o_rs, int32_t* status, va_stream_t stream) {
  const va_status st = check_embed("embed_fwd", table, out, ids, dtype, dtype, t_rs, o_rs, T, V, D, scale);
  if (st != VA_OK) return st;
  if (T == 0) return VA_OK;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch(K_EMBED_FWD, cs, [&] {
    return launch_embed_fwd(table, dtype, t_rs, ids, T, V, D, scale, out, o_rs, status, cs);
  });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "embed_fwd");
}

size_t varlen_embed_bwd_workspace_size(int32_t T, int32_t D) {
  return T < 0 || D < 1 ? 0 : embed_bwd_workspace(T, D);
}

va_status varlen_embed_bwd(const void* dout, int32_t dtype, int64_t i_rs, const int32_t* ids, int32_t T, int32_t V,
                           int32_t D, float scale, void* dtable, int32_t table_dtype, int64_t o_rs, int32_t accumulate,
                           void* ws, size_t ws_bytes, va_stream_t stream) {
  // without tokens dout is not read and may be null
  const va_status st = check_embed("embed_bwd", T == 0 && !dout ? dtable : dout, dtable, ids, T == 0 ? table_dtype : dtype,
                                   table_dtype, i_rs, o_rs, T, V, D, scale);
  if (st != VA_OK) return st;
  if (!ws || !aligned16(ws)) return fail(VA_ERR_INVALID_ARG, "embed_bwd: workspace must be 16-byte aligned");
  if (ws_bytes < varlen_embed_bwd_workspace_size(T, D)) return fail(VA_ERR_WORKSPACE, "embed_bwd: workspace too small");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const KernelId kid[3] = {K_EMBED_SORT, K_EMBED_REDUCE, K_EMBED_JOIN};
  for (int stage = 0; stage < (T > 0 ? 3 : 1) && e == cudaSuccess; ++stage)
    e = launch(kid[stage], cs, [&] {
      return launch_embed_bwd(stage, dout, dtype, i_rs, ids, T, V, D, scale, dtable, table_dtype, o_rs,
                              accumulate ? 1 : 0, ws, cs);
    });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "embed_bwd");
}

// ------------------------------------------------------------ what may lie on what

static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

// Rows of `row` bytes, `step` apart.
struct RowSpan {
  const void* at;
  int64_t step, row;
};

static RowSpan span_of(const void* p, int64_t stride, int64_t D, int bf16) {
  const int64_t es = bf16 ? 2 : 4;
  return RowSpan{p, stride * es, D * es};
}

// Whether some row of one shares a byte with some row of the other, T rows each.  (Rows side by side in wider ones,
// however they interleave, share none.)
static bool rows_meet(const RowSpan& a, const RowSpan& b, int64_t T) {
  const auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
  if (!overlap(a.at, (T - 1) * a.step + a.row, b.at, (T - 1) * b.step + b.row)) return false;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
  if (T == 1) return true;
  if (a.step == b.step) {  // the first place k rows on at which b ends behind a's beginning
    const int64_t k = std::max(floor_div(-b.row - d, a.step) + 1, -(T - 1));
    return k < T && d + k * a.step < a.row;
  }
  for (int64_t i = 0; i < T; ++i) {  // (different strides over the same memory: rare)
    const int64_t j = std::max<int64_t>(floor_div(i * a.step - b.row - d, b.step) + 1, 0);
    if (j < T && d + j * b.step < i * a.step + a.row) return true;
  }
  return false;
}

// Whether the rows are the same ones, so that each is read before it is written.
static bool rows_same(const RowSpan& a, const RowSpan& b, int64_t T) {
  return a.at == b.at && a.row == b.row && (T == 1 || a.step == b.step);
}

// ------------------------------------------------------------ query / key norm with rotation

static va_status check_qk(const char* where, const va_qk_shape* s, const void* const* rows, int nrows,
                          const int64_t* strides, const void* qw, const void* kw, const float* inv_freq,
                          const int32_t* pos, float eps) {
  const std::string w(where);
  if ((s->T > 0 && !pos) || (s->rot > 0 && !inv_freq)) return fail(VA_ERR_INVALID_ARG, w + ": null pointer");
  if (s->T < 0 || s->T >= (1 << 30) || s->Hq < 1 || s->Hkv < 1 || s->Hq > 65535 || s->Hkv > 65535)
    return fail(VA_ERR_INVALID_ARG, w + ": 0 <= T < 2^30, 1 <= heads <= 65535");
  if (s->dtype < 0 || s->dtype > 1 || s->weight_dtype < 0 || s->weight_dtype > 1)
    return fail(VA_ERR_INVALID_ARG, w + ": dtypes 0 or 1");
  if (s->d < 8 || s->d > kQkMaxDim || s->d % 8 || s->rot < 0 || s->rot > s->d || s->rot % 8)
    return fail(VA_ERR_UNSUPPORTED, w + ": d and rot multiples of 8, rot <= d <= 256");
  if (!(eps >= 0.f && eps < INFINITY)) return fail(VA_ERR_INVALID_ARG, w + ": eps must be >= 0 and finite");
  const uintptr_t wa = s->weight_dtype == 1 ? 1 : 3;
  if ((reinterpret_cast<uintptr_t>(qw) & wa) || (reinterpret_cast<uintptr_t>(kw) & wa))
    return fail(VA_ERR_INVALID_ARG, w + ": weights must be aligned to their type");
  for (int i = 0; i < nrows; ++i) {
    if (s->T > 0 && !rows[i]) return fail(VA_ERR_INVALID_ARG, w + ": null pointer");
    if (!aligned16(rows[i]) || strides[2 * i] % 8 || strides[2 * i + 1] % 8 || strides[2 * i] < 0 ||
        strides[2 * i + 1] < 0)
      return fail(VA_ERR_INVALID_ARG, w + ": pointers must be 16-byte aligned, strides multiples of 8 elements");
  }
  return VA_OK;
}

// Whether two of the heads (T x H, of d elements, their strides at least d) share an element.
static bool heads_meet(int64_t T, int64_t H, int64_t d, int64_t rs, int64_t hs) {
  if (T == 1 || H == 1 || rs >= (H - 1) * hs + d || hs >= (T - 1) * rs + d) return false;  // one inside the other's gaps
  for (int64_t i = 1; i < H; ++i) {  // a token later that starts less than d before or behind head i
    const int64_t t = i * hs / rs;
    if ((t < T && i * hs - t * rs < d) || (t + 1 < T && (t + 1) * rs - i * hs < d)) return true;
  }
  return false;
}

// Written heads lie apart, and on what they may be written over (strides `over`, may be null) only as those lie.
static va_status check_qk_outputs(const char* where, const va_qk_shape* s, void* const* out, const int64_t* strides,
                                  std::initializer_list<std::pair<const void* const*, const int64_t*>> over) {
  const std::string w(where);
  for (int i = 0; i < 2; ++i) {
    const int64_t H = i == 0 ? s->Hq : s->Hkv, rs = strides[2 * i], hs = strides[2 * i + 1];
    if ((s->T > 1 && rs < s->d) || (H > 1 && hs < s->d))
      return fail(VA_ERR_INVALID_ARG, w + ": output strides must be >= d");
    if (heads_meet(s->T, H, s->d, rs, hs)) return fail(VA_ERR_INVALID_ARG, w + ": heads of an output lie on one another");
    for (const auto& in : over)
      if (s->T > 0 && in.first[i] == out[i] && ((s->T > 1 && in.second[2 * i] != rs) || (H > 1 && in.second[2 * i + 1] != hs)))
        return fail(VA_ERR_INVALID_ARG, w + ": an output over its input has its strides");
  }
  return VA_OK;
}

static QkParams qk_params(const va_qk_shape* s, const void* qw, const void* kw, const float* inv_freq,
                          const int32_t* pos, float eps) {
  QkParams p{};
  p.x_rs[0] = s->q_row_stride, p.x_hs[0] = s->q_head_stride, p.x_rs[1] = s->k_row_stride, p.x_hs[1] = s->k_head_stride;
  p.y_rs[0] = s->qo_row_stride, p.y_hs[0] = s->qo_head_stride;
  p.y_rs[1] = s->ko_row_stride, p.y_hs[1] = s->ko_head_stride;
  p.w[0] = qw, p.w[1] = kw;
  p.inv_freq = inv_freq;
  p.pos = pos;
  p.T = s->T, p.H[0] = s->Hq, p.H[1] = s->Hkv, p.d = s->d, p.rot = s->rot;
  p.w_bf16 = s->weight_dtype;
  p.interleaved = s->interleaved != 0;
  p.eps = eps;
  return p;
}

va_status varlen_qk_norm_rope_fwd(const void* q, const void* k, const int32_t* pos, const void* qw, const void* kw,
                                  const float* inv_freq, const va_qk_shape* s, float eps, void* qo, void* ko,
                                  va_stream_t stream) {
  if (!s) return fail(VA_ERR_INVALID_ARG, "qk_norm_rope_fwd: null pointer");
  const void* rows[4] = {q, k, qo, ko};
  const int64_t strides[8] = {s->q_row_stride, s->q_head_stride, s->k_row_stride, s->k_head_stride,
                              s->qo_row_stride, s->qo_head_stride, s->ko_row_stride, s->ko_head_stride};
  va_status st = check_qk("qk_norm_rope_fwd", s, rows, 4, strides, qw, kw, inv_freq, pos, eps);
  void* const out[2] = {qo, ko};
  if (st == VA_OK) st = check_qk_outputs("qk_norm_rope_fwd", s, out, strides + 4, {{rows, strides}});
  if (st != VA_OK || s->T == 0) return st;
  QkParams p = qk_params(s, qw, kw, inv_freq, pos, eps);
  p.x[0] = q, p.x[1] = k, p.y[0] = qo, p.y[1] = ko;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = launch(K_QK_NORM_FWD, cs, [&] { return launch_qk_norm_fwd(p, s->dtype, cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "qk_norm_rope_fwd");
}

size_t varlen_qk_norm_rope_bwd_workspace_size(int32_t d) {
  return d < 8 || d > kQkMaxDim || d % 8 ? 0 : qk_norm_bwd_workspace(d);
}

va_status varlen_qk_norm_rope_bwd(const void* dqo, const void* dko, const void* q, const void* k, const int32_t* pos,
                                  const void* qw, const void* kw, const float* inv_freq, const va_qk_shape* s,
                                  const va_qk_grad_strides* gs, float eps, void* dq, void* dk, void* dqw, void* dkw,
                                  void* ws, size_t ws_bytes, va_stream_t stream) {
  if (!s || !gs) return fail(VA_ERR_INVALID_ARG, "qk_norm_rope_bwd: null pointer");
  const void* rows[6] = {q, k, dqo, dko, dq, dk};
  const int64_t strides[12] = {s->q_row_stride, s->q_head_stride, s->k_row_stride, s->k_head_stride,
                               s->qo_row_stride, s->qo_head_stride, s->ko_row_stride, s->ko_head_stride,
                               gs->dq_row_stride, gs->dq_head_stride, gs->dk_row_stride, gs->dk_head_stride};
  va_status st = check_qk("qk_norm_rope_bwd", s, rows, 6, strides, qw, kw, inv_freq, pos, eps);
  void* const out[2] = {dq, dk};
  if (st == VA_OK) st = check_qk_outputs("qk_norm_rope_bwd", s, out, strides + 8, {{rows, strides}, {rows + 2, strides + 4}});
  if (st != VA_OK) return st;
  if ((dqw && !qw) || (dkw && !kw))
    return fail(VA_ERR_INVALID_ARG, "qk_norm_rope_bwd: a weight's gradient without the weight");
  const uintptr_t wa = s->weight_dtype == 1 ? 1 : 3;
  if ((reinterpret_cast<uintptr_t>(dqw) & wa) || (reinterpret_cast<uintptr_t>(dkw) & wa))
    return fail(VA_ERR_INVALID_ARG, "qk_norm_rope_bwd: weights must be aligned to their type");
  const bool weights = dqw || dkw;
  if (weights && (!ws || !aligned16(ws)))
    return fail(VA_ERR_INVALID_ARG, "qk_norm_rope_bwd: workspace must be 16-byte aligned");
  if (weights && ws_bytes < qk_norm_bwd_workspace(s->d))
    return fail(VA_ERR_WORKSPACE, "qk_norm_rope_bwd: workspace too small");
  QkParams p = qk_params(s, qw, kw, inv_freq, pos, eps);
  p.x[0] = q, p.x[1] = k, p.dy[0] = dqo, p.dy[1] = dko, p.y[0] = dq, p.y[1] = dk;
  for (int i = 0; i < 2; ++i) p.dy_rs[i] = p.y_rs[i], p.dy_hs[i] = p.y_hs[i];  // the outputs' gradients
  p.y_rs[0] = gs->dq_row_stride, p.y_hs[0] = gs->dq_head_stride;
  p.y_rs[1] = gs->dk_row_stride, p.y_hs[1] = gs->dk_head_stride;
  p.dw[0] = dqw, p.dw[1] = dkw;
  p.part = weights ? static_cast<float*>(ws) : nullptr;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (s->T > 0) e = launch(K_QK_NORM_BWD, cs, [&] { return launch_qk_norm_bwd(0, p, s->dtype, cs); });
  if (weights && e == cudaSuccess)
    e = launch(K_QK_NORM_JOIN, cs, [&] { return launch_qk_norm_bwd(1, p, s->dtype, cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "qk_norm_rope_bwd");
}

// ------------------------------------------------------------ gated recurrence


// tokens: a forward of single tokens, which runs without a workspace too.
static va_status check_scan(const char* where, const va_scan_shape* s, const int32_t* cu, const void* ws, size_t ws_bytes,
                            bool tokens) {
  const std::string w(where);
  if (!s || !cu || (!ws && !(tokens && s->B == s->T))) return fail(VA_ERR_INVALID_ARG, w + ": null pointer");
  if (s->T < 1 || s->T >= (1 << 30) || s->B < 1 || s->B > s->T || s->D < 1 || s->D > (1 << 20))
    return fail(VA_ERR_INVALID_ARG, w + ": 1 <= B <= T < 2^30, 1 <= D <= 2^20");
  if (s->x_dtype < 0 || s->x_dtype > 1 || s->gate_dtype < 0 || s->gate_dtype > 1)
    return fail(VA_ERR_INVALID_ARG, w + ": dtypes 0 or 1");
  if (s->x_dtype == 0 && s->gate_dtype == 1)
    return fail(VA_ERR_UNSUPPORTED, w + ": fp32 inputs take fp32 decays");
  if (!aligned16(ws)) return fail(VA_ERR_INVALID_ARG, w + ": workspace must be 16-byte aligned");
  const size_t need = tokens && s->B == s->T ? (ws ? sizeof(WsHeader) : 0) : varlen_scan_workspace_size(s->T, s->B, s->D);
  if (ws_bytes < need) return fail(VA_ERR_WORKSPACE, w + ": workspace too small");
  return VA_OK;
}

static bool scan_h_bf16(const va_scan_shape* s) { return s->x_dtype == 1 && s->gate_dtype == 1 && !s->h_fp32; }

static va_status check_scan_rows(const char* where, const va_scan_shape* s, const void* p, int64_t rs, int bf16) {
  if (!p) return fail(VA_ERR_INVALID_ARG, std::string(where) + ": null pointer");
  if (rs < s->D) return fail(VA_ERR_INVALID_ARG, std::string(where) + ": row strides must be >= D");
  if (reinterpret_cast<uintptr_t>(p) & (bf16 ? 1 : 3))
    return fail(VA_ERR_INVALID_ARG, std::string(where) + ": pointers must be aligned to their type");
  return VA_OK;
}

static va_status check_states(const char* where, std::initializer_list<const float*> states) {
  for (const float* p : states)
    if (reinterpret_cast<uintptr_t>(p) & 3) return fail(VA_ERR_INVALID_ARG, std::string(where) + ": pointers must be aligned to their type");
  return VA_OK;
}

size_t varlen_scan_workspace_size(int32_t T, int32_t B, int32_t D) {
  if (T < 1 || T >= (1 << 30) || B < 1 || B > T || D < 1 || D > (1 << 20)) return 0;
  return scan_workspace(T, D);
}

va_status varlen_scan_fwd(const void* x, const void* g, const int32_t* cu, const va_scan_shape* s, const float* h0,
                          void* h, float* h_last, void* ws, size_t ws_bytes, va_stream_t stream) {
  const char* where = "scan_fwd";
  va_status st = check_scan(where, s, cu, ws, ws_bytes, true);
  const int hb = st == VA_OK && scan_h_bf16(s);
  if (st == VA_OK) st = check_scan_rows(where, s, x, s->x_row_stride, s->x_dtype);
  if (st == VA_OK) st = check_scan_rows(where, s, g, s->gate_row_stride, s->gate_dtype);
  if (st == VA_OK) st = check_scan_rows(where, s, h, s->h_row_stride, hb);
  if (st == VA_OK) st = check_states(where, {h0, h_last});
  if (st != VA_OK) return st;
  const size_t states = static_cast<size_t>(s->B) * s->D * sizeof(float);
  // a segment's first rows read h0 twice, the second time maybe after its last row is done
  if (s->B < s->T && overlap(h0, states, h_last, states))
    return fail(VA_ERR_INVALID_ARG, "scan_fwd: h_last may lie on h0 for single tokens only (T == B)");
  const RowSpan out = span_of(h, s->h_row_stride, s->D, hb);
  for (const RowSpan& in : {span_of(x, s->x_row_stride, s->D, s->x_dtype), span_of(g, s->gate_row_stride, s->D, s->gate_dtype)})
    if (!rows_same(out, in, s->T) && rows_meet(out, in, s->T))
      return fail(VA_ERR_INVALID_ARG, "scan_fwd: h may be an input itself (type and stride), not lie on a part of it");
  ScanParams p{};
  p.x = x, p.g = g, p.out = h;
  p.x_rs = s->x_row_stride, p.g_rs = s->gate_row_stride, p.out_rs = s->h_row_stride;
  p.cu = cu, p.h0 = h0, p.last = h_last;
  p.B = s->B, p.T = s->T, p.D = s->D;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (s->B == s->T) {
    e = launch(K_SCAN_STEP, cs, [&] { return launch_scan_step(p, s->x_dtype, s->gate_dtype, hb, ws, cs); });
  } else {
    p.wait_ns = static_cast<uint64_t>(g_stall_next_scan.exchange(0));
    const KernelId kid[2] = {K_SCAN_PREP, K_SCAN_FWD};
    for (int stage = 0; stage < 2 && e == cudaSuccess; ++stage)
      e = launch(kid[stage], cs, [&] { return launch_scan_fwd(stage, p, s->x_dtype, s->gate_dtype, hb, ws, cs); });
  }
  return e == cudaSuccess ? VA_OK : cuda_fail(e, where);
}

va_status varlen_scan_bwd(const void* dh, const void* h, const void* g, const int32_t* cu, const va_scan_shape* s,
                          const va_scan_grad_strides* gs, const float* h0, const float* dh_last, void* dx, void* dg,
                          float* dh0, void* ws, size_t ws_bytes, va_stream_t stream) {
  const char* where = "scan_bwd";
  if (!gs) return fail(VA_ERR_INVALID_ARG, "scan_bwd: null pointer");
  va_status st = check_scan(where, s, cu, ws, ws_bytes, false);
  const int hb = st == VA_OK && scan_h_bf16(s);
  if (st == VA_OK) st = check_scan_rows(where, s, dh, gs->dh_row_stride, hb);
  if (st == VA_OK) st = check_scan_rows(where, s, h, s->h_row_stride, hb);
  if (st == VA_OK) st = check_scan_rows(where, s, g, s->gate_row_stride, s->gate_dtype);
  if (st == VA_OK) st = check_scan_rows(where, s, dx, gs->dx_row_stride, s->x_dtype);
  if (st == VA_OK) st = check_scan_rows(where, s, dg, gs->dgate_row_stride, s->gate_dtype);
  if (st == VA_OK) st = check_states(where, {h0, dh_last, dh0});
  if (st != VA_OK) return st;
  const size_t states = static_cast<size_t>(s->B) * s->D * sizeof(float);
  if (overlap(dh_last, states, dh0, states) || overlap(h0, states, dh0, states))
    return fail(VA_ERR_INVALID_ARG, "scan_bwd: dh0 must not lie on h0 or dh_last");
  const RowSpan rdh = span_of(dh, gs->dh_row_stride, s->D, hb), rg = span_of(g, s->gate_row_stride, s->D, s->gate_dtype),
                rh = span_of(h, s->h_row_stride, s->D, hb), rdx = span_of(dx, gs->dx_row_stride, s->D, s->x_dtype),
                rdg = span_of(dg, gs->dgate_row_stride, s->D, s->gate_dtype);
  // (a tile reads the row of h before its own, which another tile's gradients would lie on)
  if (rows_meet(rdx, rh, s->T) || rows_meet(rdg, rh, s->T) || rows_meet(rdx, rdg, s->T))
    return fail(VA_ERR_INVALID_ARG, "scan_bwd: dx and dlog_decay must lie neither on h nor on one another");
  for (const RowSpan& to : {rdx, rdg})
    for (const RowSpan& in : {rdh, rg})
      if (!rows_same(to, in, s->T) && rows_meet(to, in, s->T))
        return fail(VA_ERR_INVALID_ARG, "scan_bwd: a gradient may be dh or log_decay itself (type and stride), not lie on a part of it");
  ScanParams p{};
  p.x = dh, p.g = g, p.h = h, p.out = dx, p.dg = dg;
  p.x_rs = gs->dh_row_stride, p.g_rs = s->gate_row_stride, p.h_rs = s->h_row_stride;
  p.out_rs = gs->dx_row_stride, p.dg_rs = gs->dgate_row_stride;
  p.cu = cu, p.h0 = h0, p.dlast = dh_last, p.last = dh0;
  p.B = s->B, p.T = s->T, p.D = s->D;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  p.wait_ns = static_cast<uint64_t>(g_stall_next_scan.exchange(0));
  const KernelId kid[2] = {K_SCAN_PREP, K_SCAN_BWD};
  for (int stage = 0; stage < 2 && e == cudaSuccess; ++stage)
    e = launch(kid[stage], cs, [&] { return launch_scan_bwd(stage, p, s->x_dtype, s->gate_dtype, hb, ws, cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, where);
}

// ------------------------------------------------------------ token log probabilities

static va_status check_logprobs(const char* where, const void* z, int32_t dtype, int64_t z_rs, const int32_t* tok,
                                int32_t T, int32_t V, float temperature) {
  const std::string w(where);
  if (!z || !tok) return fail(VA_ERR_INVALID_ARG, w + ": null pointer");
  if (T < 1 || T >= (1 << 30) || V < 1 || V >= (1 << 30) || (dtype != 0 && dtype != 1))
    return fail(VA_ERR_INVALID_ARG, w + ": 1 <= T and V < 2^30, dtype 0 or 1");
  if (z_rs < V) return fail(VA_ERR_INVALID_ARG, w + ": row strides must be >= the row");
  if (reinterpret_cast<uintptr_t>(z) & (dtype == 1 ? 1 : 3))
    return fail(VA_ERR_INVALID_ARG, w + ": pointers must be aligned to their type");
  if (!(temperature >= 1.f / 64) || !(temperature <= 64.f))
    return fail(VA_ERR_INVALID_ARG, w + ": temperature must be in [1/64, 64]");
  return VA_OK;
}

static void set_temperature(LogprobParams& p, float temperature) {
  const double scale = 1.4426950408889634 / temperature;
  p.temperature = temperature;
  p.inv_t = 1.f / temperature;
  p.scale = static_cast<float>(scale);
  p.scale_lo = static_cast<float>(scale - p.scale);
  p.inv_c = 1.f / p.scale;
}

va_status varlen_token_logprobs_fwd(const void* z, int32_t dtype, int64_t z_rs, const int32_t* tok, int32_t T,
                                    int32_t V, int32_t k, int32_t ignore_index, float temperature, float* logprob,
                                    float* entropy, float* lse, int32_t* top_ids, float* top_logprobs, int32_t* status,
                                    va_stream_t stream) {
  const va_status st = check_logprobs("token_logprobs_fwd", z, dtype, z_rs, tok, T, V, temperature);
  if (st != VA_OK) return st;
  if (!logprob || !entropy || !lse || (k > 0 && (!top_ids || !top_logprobs)))
    return fail(VA_ERR_INVALID_ARG, "token_logprobs_fwd: null pointer");
  if (k < 0 || k > V) return fail(VA_ERR_INVALID_ARG, "token_logprobs_fwd: 0 <= k <= V");
  if (k > kMaxTop) return fail(VA_ERR_UNSUPPORTED, "token_logprobs_fwd: at most 128 alternatives");
  LogprobParams p{};
  p.z = z, p.z_rs = z_rs, p.tok = tok, p.T = T, p.V = V, p.ignore = ignore_index, p.k = k;
  set_temperature(p, temperature);
  p.logprob = logprob, p.entropy = entropy, p.lse = lse, p.top_ids = top_ids, p.top_logprobs = top_logprobs;
  p.status = status;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = launch(K_LOGPROBS_FWD, cs, [&] { return launch_logprobs_fwd(p, dtype, cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "token_logprobs_fwd");
}

va_status varlen_token_logprobs_bwd(const void* z, int32_t dtype, int64_t z_rs, const int32_t* tok, const float* lse,
                                    const float* entropy, const float* dlogprob, const float* dentropy, int32_t T,
                                    int32_t V, int32_t ignore_index, float temperature, void* grad, int64_t g_rs,
                                    va_stream_t stream) {
  const va_status st = check_logprobs("token_logprobs_bwd", z, dtype, z_rs, tok, T, V, temperature);
  if (st != VA_OK) return st;
  if (!lse || !dlogprob || !grad || (dentropy && !entropy))
    return fail(VA_ERR_INVALID_ARG, "token_logprobs_bwd: null pointer");
  if (g_rs < V) return fail(VA_ERR_INVALID_ARG, "token_logprobs_bwd: row strides must be >= the row");
  if (reinterpret_cast<uintptr_t>(grad) & (dtype == 1 ? 1 : 3))
    return fail(VA_ERR_INVALID_ARG, "token_logprobs_bwd: pointers must be aligned to their type");
  const RowSpan from = span_of(z, z_rs, V, dtype), to = span_of(grad, g_rs, V, dtype);
  if (!rows_same(from, to, T) && rows_meet(from, to, T))
    return fail(VA_ERR_INVALID_ARG, "token_logprobs_bwd: grad may be the logits themselves (same stride), not lie on a part of them");
  LogprobParams p{};
  p.z = z, p.z_rs = z_rs, p.tok = tok, p.T = T, p.V = V, p.ignore = ignore_index;
  set_temperature(p, temperature);
  p.lse = const_cast<float*>(lse), p.entropy = const_cast<float*>(entropy);
  p.dlogprob = dlogprob, p.dentropy = dentropy, p.grad = grad, p.g_rs = g_rs;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = launch(K_LOGPROBS_BWD, cs, [&] { return launch_logprobs_bwd(p, dtype, cs); });
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "token_logprobs_bwd");
}

va_status varlen_read_status(const void* ws, int32_t* out, va_stream_t stream) {
  if (!ws || !out) return fail(VA_ERR_INVALID_ARG, "read_status: null pointer");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(out, ws, sizeof(int32_t), cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "read_status");
}

va_status varlen_clear_status(void* ws, va_stream_t stream) {
  if (!ws) return fail(VA_ERR_INVALID_ARG, "clear_status: null pointer");
  cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int32_t), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VA_OK : cuda_fail(e, "clear_status");
}

va_status varlen_profile_enable(int32_t capacity) {
  for (cudaEvent_t e : g_prof.start) cudaEventDestroy(e);
  for (cudaEvent_t e : g_prof.stop) cudaEventDestroy(e);
  g_prof = Profiler{};
  if (capacity < 0) return fail(VA_ERR_INVALID_ARG, "profile_enable: negative capacity");
  if (capacity == 0) return VA_OK;
  g_prof.start.resize(capacity);
  g_prof.stop.resize(capacity);
  g_prof.ids.resize(capacity);
  for (int i = 0; i < capacity; ++i) {
    cudaError_t e = cudaEventCreate(&g_prof.start[i]);
    if (e == cudaSuccess) e = cudaEventCreate(&g_prof.stop[i]);
    if (e != cudaSuccess) {
      g_prof.start.resize(i);
      g_prof.stop.resize(i);
      return cuda_fail(e, "profile_enable");
    }
  }
  g_prof.cap = capacity;
  return VA_OK;
}

va_status varlen_profile_read(int32_t* ids, float* ms, int32_t capacity, int32_t* count) {
  if (!count || (capacity > 0 && (!ids || !ms)))
    return fail(VA_ERR_INVALID_ARG, "profile_read: null pointer");
  const int n = std::min(g_prof.n, capacity);
  for (int i = 0; i < n; ++i) {
    cudaError_t e = cudaEventSynchronize(g_prof.stop[i]);
    if (e == cudaSuccess) e = cudaEventElapsedTime(&ms[i], g_prof.start[i], g_prof.stop[i]);
    if (e != cudaSuccess) return cuda_fail(e, "profile_read");
    ids[i] = g_prof.ids[i];
  }
  *count = n;
  g_prof.n = 0;
  return VA_OK;
}

const char* varlen_kernel_name(int32_t id) {
  return (id >= 0 && id < K_COUNT) ? kKernelNames[id] : "";
}

int64_t varlen_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

va_status varlen_test_stall_next_forward(int64_t wait_limit_ns) {
  if (wait_limit_ns < 1000000 || wait_limit_ns > 2000000000)
    return fail(VA_ERR_INVALID_ARG, "test_stall_next_forward: the limit must be 1 ms .. 2 s");
  g_stall_next_fwd.store(wait_limit_ns);
  return VA_OK;
}

va_status varlen_test_stall_next_distill(int64_t wait_limit_ns) {
  if (wait_limit_ns < 1000000 || wait_limit_ns > 2000000000)
    return fail(VA_ERR_INVALID_ARG, "test_stall_next_distill: the limit must be 1 ms .. 2 s");
  g_stall_next_distill.store(wait_limit_ns);
  return VA_OK;
}

va_status varlen_test_stall_next_scan(int64_t wait_limit_ns) {
  if (wait_limit_ns < 1000000 || wait_limit_ns > 2000000000)
    return fail(VA_ERR_INVALID_ARG, "test_stall_next_scan: the limit must be 1 ms .. 2 s");
  g_stall_next_scan.store(wait_limit_ns);
  return VA_OK;
}

}  // extern "C"
