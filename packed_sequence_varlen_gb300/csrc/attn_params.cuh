// Kernel parameter blocks for the attention kernels.
#pragma once
#include "common.cuh"

namespace va {

using bf16 = __nv_bfloat16;

// Forms of the attention kernels: no local window, a causal local window, a window with sinks, and
// (dK/dV) one whose sink blocks may come in pieces.
enum WinForm : int { kWinNone = 0, kWinLocal = 1, kWinSinks = 2, kWinSplit = 3 };

struct FwdParams {
  const bf16* q;
  const bf16* k;
  const bf16* v;
  bf16* o;
  float* lse;  // [Hq, T]
  const int32_t* cu;
  const TileItem* items;
  int B;  // segments (cu has B + 1 entries)
  WsHeader* hdr;
  int slot;
  int32_t* counter;  // work counter (records are pulled in list order)
  int T, Hq, Hkv, g;
  int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, o_rs, o_hs;
  float scale_log2;  // scale * log2(e)
  int causal;
  int window = -1;   // causal local window: query i sees keys i-w..i; -1 = none
  int sinks = 0;     // with a window: a segment's first keys that every later query still sees
  const int32_t* cu_k = nullptr;  // cross-attention: K/V boundaries (cu is Q's); null = cu
  int Tk = 0;                     // cross-attention: rows of K and V
  // Test hook of the failure path (varlen_test_stall_next_forward): a wait limit in ns
  // (0 = the default) and stall = 1, which makes each CTA's producer publish its first work
  // item and then load nothing, so the consumers' bounded waits run out.
  uint64_t wait_ns = 0;
  int stall = 0;
};

struct BwdParams {
  const bf16* q;
  const bf16* k;
  const bf16* v;
  const bf16* o;
  const bf16* dout;
  const float* lse;  // [Hq, T], natural log
  float* dsum;       // D = rowsum(dO * O), [Hq, T]
  bf16* dq;
  bf16* dk;
  bf16* dv;
  const int32_t* cu;
  int B;  // segments (cu has B + 1 entries)
  const TileItem* kv_items;  // kv-block map
  const TileItem* q_items;   // q-block map (dQ pass)
  WsHeader* hdr;
  int kv_slot, q_slot;          // n_items[slot]: all records of the map
  int kv_tok_slot, q_tok_slot;  // n_items[slot]: the token records at the map's end
  int32_t* kv_counter;
  int32_t* q_counter;
  int T, Hq, Hkv, g;
  int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, o_rs, o_hs;
  float scale;
  float scale_log2;
  int causal;
  int window = -1;   // causal local window: query i sees keys i-w..i; -1 = none
  int sinks = 0;     // with a window: a segment's first keys that every later query still sees
  // Sink kv blocks whose q range is split: q blocks per piece (0 = never), the pieces' fp32 dV and
  // dK [slot][kv block][kv head][2][128][d], the blocks of 128 keys that hold sinks.
  int piece = 0, sink_blocks = 0;
  float* part = nullptr;
  const int32_t* cu_k = nullptr;  // cross-attention: K/V boundaries (cu is Q's); null = cu
  int Tk = 0;                     // cross-attention: rows of K and V
};

// Slot of the partial sums of piece `piece` of the kv block whose keys start at stream row `row`.  A
// split segment of n >= 2 pieces spans more than (n - 1) pieces of rows, which are two slots each, so
// the slots (row / (32 P)) + 1 .. + n of different segments never meet.
__host__ __device__ inline int sink_slot(int row, int P, int piece) { return row / (32 * P) + 1 + piece; }
__host__ __device__ inline int sink_slots(int T, int P) { return T / (32 * P) + 2; }

}  // namespace va
