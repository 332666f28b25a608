// attn_window.cu — windowed extend_attn and varlen_prefill_attn on the tcgen05 tensor cores: new tokens against
// their cached context and causally against themselves, where the row at position i sees the keys
// j <= i with j > i - window (the window) or j < sinks (the first tokens, which stay visible).
//
// Mathematics: with s_j = log2(e) scale (q . k_j) over the keys that a row sees and m any number of their size,
// P_j = 2^(s_j - m):  O = sum P_j v_j,  l = sum P_j,  out = O / l,  lse = (m + log2 l) ln 2. m is the max of the
// scores when the row first meets one, and follows them only when they pass it by more than LAZY: P and O
// keep the precision of their types whatever the power of two in front, and O is rescaled in nearly no tile. P <= 2^20, so
// the keys that a row sees times their largest value may come to 2^108 (over codes P <= 2^15 and values are fp16). In fp16, whose smallest number is 2^-24, m is RAISE below that max: a row's
// largest P is 2^8 at least, and terms down to 2^-33 of it count (with 2^-25, what thousands of keys have in common was
// lost from O, not from l).
//
// Work items. The rows of a request for one KV head are its (token, query head of the group) pairs, tokens
// outermost (a box of Q is G heads x 128 / G tokens), and an item is 256 of them: two tiles of 128, one a
// slot. So an item spans 256 / G tokens, and the keys that some row of it sees are sinks + window + 256 / G - 1.
// (Items of 128 tokens and two heads, as without a window, span up to 128 more: a window of 128 then
// takes twice the products, and every KV head's keys are read G / 2 times.) An item whose rows fit one tile deals
// its key tiles to the slots in turn, both on the one Q tile, and the two states are merged at the end.
//
// Keys come in chunks of 16: a cache block, or 16 new tokens of the request. The chunks that an item walks are
// the first `head` ones, which hold sinks, and those from the first row's window on (WnItem); eight make a key
// tile, whatever they are, so sinks and window share a tile, and the last tile takes products of its chunks
// alone. Tiles that every row sees whole skip the masks; in the others the value rows that no row sees are
// zeroed (P = 0 there must not meet what is not finite).
//
// A slot's chain is S = Q K^T (520 clocks a tile), softmax, O += P V (520), and the tensor core serves the other slot
// meanwhile, so a softmax has some 1000 clocks: a whole row in registers, read once (two threads a row, four warps more: no
// faster, both warps of a row's quarter share a scheduler), and P handed over in two halves. What the products wait for is issued
// by single threads (a barrier that is complete costs a warp 110 clocks, and copies issued by eight lanes 1030 a tile instead
// of 540).
//
// Roles (one CTA per SM, persistent; 12 warps, over codes 20):
//   warps 0-3, 4-7  softmax of slot 0, 1 (thread t owns row t = TMEM lane t) and the epilogue
//   warp 8          claims the items, loads Q and the ring of K tiles
//   warp 9          MMA issuer, one elected thread, waits included: S = Q K^T, O += P V (P from tensor memory)
//   warp 10         loads the ring of V tiles (a K buffer is free before the V buffer of the tile before)
//   warp 11         zeroes value rows of tiles at an edge (over codes it has nothing to do)
//   warps 12-15, 16-19  over codes: Q and the K tiles to fp16, the V tiles to fp16
// Tensor memory (512 columns): S_0 | S_1 | O_0 | O_1, 128 each (D 64: half of the O columns unused); P_s (16-bit pairs)
// overwrites the first half of its S. (Key tiles of 64 with two score buffers a slot: three prompts under 4096 1459 us.)
//
// What bounds it, on a GB300 with 64 query and 8 KV heads of 128 (times of back-to-back calls; the measured peaks are 6776 GB/s and
// 1882 TFLOP/s bf16):
//   three prompts of 4000 to 10,007 tokens under 4096   1305 to 1380 us from GPU to GPU, 1450 to 1530 TFLOP/s (0.77 to 0.81 of
//                                                       measured; 1203 us alone and cool): the two slots' chains, and the
//                                                       power limit
//   8 x 301-512 tokens over 4000-32,000 under 128       49 us for a floor of 18.5: two edge tiles an item, so each item is
//                                                       its chain of Q, S, masks, softmax, P V, epilogue, some 12,000 clocks
//   32 x 4 tokens over 1000-4000 under 1024             37 us, 3.7 TB/s (floor 20.6): 256 items in two rounds of 152
//   2048 tokens over 100,000 under 4096, E4M3 cache     232 us (floor 151; a bf16 cache 214): of it 8 to 16 for the rows
//                                                       converted ahead; with the codes converted by every item 314 to 329,
//                                                       the conversions waiting for shared memory that the products read
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "softmax.cuh"
#include "tc.cuh"

namespace pkv {

namespace {

// What the kernel reads. kWnBf16: a bf16 cache (or none) and the new rows. Over a cache of E4M3 codes the products run
// on fp16 (every E4M3 value is an fp16 number; new values are divided by the value scale). kWnCodes: the codes and
// the new rows land as they are, and converter warps turn them and Q into fp16 in shared memory. kWnPool: fp16 rows that
// the kWnCodes launch before has converted, once for all items that read them (wn_fill); the softmax warps convert Q.
enum { kWnBf16, kWnCodes, kWnPool };

template <int D, int KIND>
struct WnCfg {
  static constexpr bool FP8 = KIND == kWnCodes, F16 = KIND != kWnBf16;
  static constexpr int BN = 128, CHUNKS = BN / 16;        // keys of a tile
  static constexpr int HALVES = D / 64;
  static constexpr int Q_HALF = 128 * 128;                // 128 rows x 128 bytes
  static constexpr int Q_BYTES = HALVES * Q_HALF;         // one 128-row tile of Q
  static constexpr int KV_HALF = BN * 128;
  static constexpr int KV_BYTES = HALVES * KV_HALF;       // one tile of K or V
  static constexpr int NBUF = D == 128 ? 2 : 4;           // tiles of the K ring, and of the V ring
  static constexpr int MAXR = kAttnSetChunk;              // requests of the set one launch holds
  static constexpr int W_K = 8, W_MMA = 9, W_V = 10, W_FIX = 11;
  static constexpr int W_CONV = 12, NCONV = FP8 ? 4 : 0;  // converter warps of Q and K, and as many of V
  static constexpr int THREADS = FP8 ? 640 : 384;
  // launched at 168 registers a thread (kWnCodes: 96); the softmax warps take some of the others'
  static constexpr int REGS_LAUNCH = FP8 ? 96 : 168, REGS_SOFTMAX = FP8 ? 144 : 208, REGS_OTHER = FP8 ? 64 : 80;
  static_assert(256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * REGS_LAUNCH, "register split");
  // How far (in powers of two) scores may pass a row's m before it follows them: far in bf16; in fp16 P stays below 2^16.
  static constexpr float LAZY = F16 ? 15.f : 20.f;
  // and how far below the scores that it follows m is put: fp16 keeps 11 bits of a P from 2^-14 on, and loses one below 2^-25.
  static constexpr float RAISE = F16 ? 8.f : 0.f;
  static constexpr int ITEM_RING = 4;                     // claimed items published to the other roles
  static constexpr int ITEM_READERS = 8 + 2 + (FP8 ? 2 * NCONV : 1);
  static constexpr int RING_OFF = 2 * Q_BYTES;
  static constexpr int REQ_OFF = RING_OFF + 2 * NBUF * KV_BYTES;  // int4 {r, row0, q_len, C}
  static constexpr int START_OFF = REQ_OFF + MAXR * 16;         // prefix of the items, by rank
  static constexpr int PERM_OFF = START_OFF + (MAXR + 4) * 4;   // set positions by cost, heaviest first
  static constexpr int ITEM_OFF = PERM_OFF + MAXR * 4;
  static constexpr int MERGE_OFF = ITEM_OFF + ITEM_RING * 64;   // [slot][128] {m, l} of split items
  // output staging: per softmax warp, 32 rows x 32 bf16 columns (64-byte rows, 64-byte swizzle)
  static constexpr int STAGE_OFF = (MERGE_OFF + 2 * 128 * 8 + 127) / 128 * 128;
  static constexpr int BAR_OFF = STAGE_OFF + 8 * 2048;
};
struct WnBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t k_ready[4], v_ready[4], q_ready;  // converted (K: kWnCodes only, Q: fp16 only); value rows that no row sees zeroed
  uint64_t s_full[2], o_final[2];
  uint64_t p_full[2][2];  // P of the first and of the second 64 columns
  uint64_t o_both;        // both slots' O of a split item
  uint64_t item_full[4], item_empty[4];
  uint64_t rows[4];       // the two warps that share a split item's 32 rows
  uint64_t drained;       // the products in flight when a role gave up
};
template <int D, int KIND>
constexpr int wn_smem() { return 1024 + WnCfg<D, KIND>::BAR_OFF + static_cast<int>(sizeof(WnBars)); }

__device__ __forceinline__ constexpr uint32_t wn_scol(int slot) { return slot * 128u; }
__device__ __forceinline__ constexpr uint32_t wn_ocol(int slot) { return 256u + slot * 128u; }

// A piece of work, published in shared memory by the producer. Chunks are numbered u = 0, 1, ..: the cache blocks
// first (cb of them), then the new tokens sixteen by sixteen; the v-th chunk walked is u = v, or v + gap from
// v = head on.
struct WnItem {
  int r, row0, C, kh;       // request, its first row of q, its cached tokens; KV head
  int tok0, ntok;           // the item's first new token and its tokens
  int split;                // 1: one tile of rows, key tiles dealt to the slots in turn
  int NV;                   // chunks walked (0: no more work)
  int head, gap, cb;
  int low;                  // the first key in the first row's window
  int fs, f0, f1, vt;       // chunks 0 .. fs - 1 and f0 .. f1 - 1 of the walk, but for vt, every row sees whole
  __device__ int tiles() const { return (NV + 7) >> 3; }
  __device__ int last() const { return C + tok0 + ntok - 1; }  // position of the last row
  __device__ int chunk(int v) const { return v < head ? v : v + gap; }
  __device__ int pos(int u) const { return u < cb ? 16 * u : C + 16 * (u - cb); }
  __device__ bool full(int j) const {
    const int a = 8 * j, b = a + 8;
    return b <= fs || (a >= f0 && b <= f1 && (vt < a || vt >= b));
  }
  // chunks of the walk that are cache blocks: the first ones
  __device__ int cached() const { return cb <= head ? cb : max(head, cb - gap); }
};
static_assert(sizeof(WnItem) == 64, "ring entry");

__device__ __forceinline__ int wn_count(const int4& q, int G) { return (q.z * G + 255) >> 8; }
// Keys an item of the request walks, about: the schedule's order.
__device__ __forceinline__ int wn_cost(const AttnParams& p, const int4& q) {
  return static_cast<int>(min(static_cast<int64_t>(q.z) + q.w, static_cast<int64_t>(p.window) + p.sinks));
}

// Item idx of a request {request id, first query row, q_len, cached tokens}, or one half of its tokens (half 0 or 1; -1:
// all). A second half without tokens is the first one again: another CTA, which had nothing else to do, writes the same bits. It
// does because an item's tiles go to the slots in a fixed order (tile j of a split item to slot j % 2), each slot adds them up in
// that order, and the merge takes slot 0 first: were tiles dealt as they arrive, this half's stores would have to be left out.
__device__ __forceinline__ WnItem wn_item(const AttnParams& p, const int4& q, int idx, int half) {
  WnItem it;
  it.r = q.x;
  it.row0 = q.y;
  it.C = q.w;
  const int span = 256 / p.G, tile = idx / p.Hkv;
  it.kh = idx - tile * p.Hkv;
  it.tok0 = span * (wn_count(q, p.G) - 1 - tile);  // later (heavier) rows of a request first
  if (half == 1 && q.z - it.tok0 > span / 2) it.tok0 += span / 2;
  it.ntok = min(half < 0 ? span : span / 2, q.z - it.tok0);
  it.split = it.ntok * p.G <= 128;
  const int P0 = it.C + it.tok0, P1 = it.last();
  it.cb = (it.C + 15) / 16;
  it.low = P0 >= p.window ? P0 - p.window + 1 : 0;
  const int sinks = min(p.sinks, P1 + 1);
  it.head = sinks <= it.C ? (sinks + 15) / 16 : it.cb + (sinks - it.C + 15) / 16;
  const int from = it.low < it.C ? it.low / 16 : it.cb + (it.low - it.C) / 16;
  it.gap = max(from - it.head, 0);
  it.NV = it.cb + (it.tok0 + it.ntok + 15) / 16 - it.gap;
  // chunks that every row sees whole: those of sinks alone (of the cache), and those from the last row's window
  // on up to the first row; the cache's last, partly filled one is none of them
  it.fs = min(it.head, min(sinks, it.C) / 16);
  const int all = P1 >= p.window ? P1 - p.window + 1 : 0;
  it.f0 = (all <= it.C ? min((all + 15) / 16, it.cb) : it.cb + (all - it.C + 15) / 16) - it.gap;
  it.f1 = it.cb + (it.tok0 + 1) / 16 - it.gap;
  it.vt = (it.C & 15) == 0 ? -1 : it.cb - 1 < it.head ? it.cb - 1 : it.cb - 1 - it.gap;
  if (it.vt < it.head && it.cb - 1 >= it.head) it.vt = -1;  // (it lies in the gap)
  return it;
}

// ---- the pool (kWnPool) --------------------------------------------------------------------------------
// The pool holds, request after request, the chunks of 16 keys that some row of the request sees: the `hb` blocks of
// sinks, the cached blocks from the first row's window on, the new tokens. Chunk u of a request lies at its first
// block + u, less `gap` from hb on. A request belongs to it when it has kPoolRows rows a KV head, an item of them, and the pool
// has room: beside long requests, shorter ones left to the codes are a launch of few items before the others' (2048 tokens of
// 64 and 8 heads under 4096 beside 8 requests of 32 tokens: 281 us, 297 from 512 rows on; 1024 under 2048 beside 4 of 32: 102 and
// 121). A call has a pool only with a request of kPoolLong rows (8 x 64 tokens of 64 and 8 heads under 4096, 512 rows each, 101
// us without and 121 with; 8 x 128 193 and 173).
constexpr int kPoolRows = 256, kPoolLong = 1024;
struct WnPooled {
  int cb, hb, gap;
  __device__ WnPooled(const AttnParams& p, int C) {
    const int low = max(C - p.window + 1, 0);
    cb = (C + 15) / 16;
    hb = (min(p.sinks, C) + 15) / 16;
    gap = max((low < C ? low / 16 : cb) - hb, 0);
  }
  __device__ int at(int u) const { return u < hb ? u : u - gap; }
};
// Blocks of the pool for a request {request id, first query row, q_len, cached tokens}; 0: it is too short.
__device__ __forceinline__ int wn_pool_need(const AttnParams& p, const int4& q) {
  if (q.z * p.G < kPoolRows) return 0;
  const WnPooled w(p, q.w);
  return min(w.cb - w.gap + (q.z + 15) / 16, p.pool_blocks + 1);  // (the sum over a launch's requests stays in range)
}
// Where request i of the launch begins in the pool (the requests before it, those without room included), or -1.
__device__ __forceinline__ int wn_pool_base(const AttnParams& p, const int* need, int i) {
  int base = 0;
#pragma unroll 8
  for (int j = 0; j < i; ++j) base += need[j];
  return need[i] > 0 && base + need[i] <= p.pool_blocks ? base : -1;
}

// Request i of this launch's chunk of the set: {request id, first query row, q_len, cached tokens}.
__device__ __forceinline__ int4 wn_request(const AttnParams& p, int begin, int i) {
  const int r = p.order ? p.order[begin + i] : begin + i;
  if (r < 0 || r >= p.batch_reqs) {
    if (blockIdx.x == 0) flag_error(p.err, PKV_DEVERR_REQS);
    return make_int4(0, 0, 0, 0);
  }
  const int row0 = p.cu_q[r], q_len = max(0, p.cu_q[r + 1] - row0);
  if (row0 < 0) {
    if (blockIdx.x == 0) flag_error(p.err, PKV_DEVERR_LEN);
    return make_int4(0, 0, 0, 0);
  }
  int c = 0;
  if (p.seq_lens != nullptr) {
    c = max(0, p.seq_lens[r] - q_len);
    if (c > static_cast<int64_t>(p.max_blocks) * 16) {
      if (blockIdx.x == 0) flag_error(p.err, PKV_DEVERR_LEN);
      c = p.max_blocks * 16;
    }
  }
  // (rows past the last token are never written, and no row before them sees their keys)
  return make_int4(r, row0, static_cast<int>(min(static_cast<int64_t>(q_len), max(p.num_tokens - row0, int64_t(0)))), c);
}
// This launch's chunk of the request set: its first position, and its requests.
__device__ __forceinline__ int wn_set(const AttnParams& p, int& n) {
  int begin = 0;
  n = p.max_reqs;
  if (p.bounds != nullptr) {
    begin = p.bounds[p.cls];
    n = p.bounds[p.cls + 1] - begin;
    if (n > p.max_reqs) {
      if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_REQS);
      n = p.max_reqs;
    }
    n = max(n, 0);
  }
  n = max(0, min(n - p.set_offset, kAttnSetChunk));
  return begin + p.set_offset;
}

// Counters of claimed items and of finished CTAs, in the launch's slot (launch.h); its last CTA to finish sets
// the slot back to zero. Without a slot the items are dealt statically, in snake order.
__device__ unsigned int g_wn_next[kAttnSchedSlots];
__device__ unsigned int g_wn_done[kAttnSchedSlots];

// Bounded wait by one thread that also gives up as soon as another role has given up.
__device__ __forceinline__ bool wn_wait1(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        flag_error(err, PKV_DEVERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}
// The same answer in all lanes, so that warp-collective instructions after it see a whole warp.
__device__ __forceinline__ bool wn_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  return __all_sync(0xffffffffu, wn_wait1(bar, parity, abort_flag, err));
}

// The low n bits (none, or all 32, beyond that range).
__device__ __forceinline__ uint32_t wn_below(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// What a row sees of a walk, in walk columns (column x is key x % 16 of chunk x / 16): those before `sinks` and
// those from `from` on, up to its own, `end` - 1, without the hole behind the last cached token.
struct WnRow {
  int sinks, from, end, hole0, hole1;
  __device__ WnRow(const AttnParams& p, const WnItem& it, int i) {  // the row at position i >= C
    // (a window's start before the first key is the first key: `from` minus a column stays within 32 bits)
    const int C = it.C, cols = 16 * it.cb, gap = 16 * it.gap, low = max(i - p.window + 1, 0);
    sinks = p.sinks <= C ? p.sinks : min(p.sinks, i + 1) - C + cols;
    from = (low < C ? low : low - C + cols) - gap;
    end = i - C + cols - gap + 1;
    hole0 = C - (it.cb - 1 < it.head ? 0 : gap);
    hole1 = it.vt < 0 ? hole0 : hole0 + (cols - C);
  }
  // which of the columns x .. x + 31, a bit each
  __device__ uint32_t seen(int x) const {
    return wn_below(end - x) & (wn_below(sinks - x) | ~wn_below(from - x)) & (wn_below(hole0 - x) | ~wn_below(hole1 - x));
  }
};

// ---- conversions -------------------------------------------------------------------------------
// A K or V tile is [2 halves][128 rows][128 B] (64 16-bit values of a row per half, 128-byte swizzle: 16-byte chunk q of
// row R at R * 128 + ((q ^ (R & 7)) << 4)). A block's codes land, with the same swizzle, where their rows' second half
// goes, so a thread converts its own code row in place: dims 0 .. 63 into the first half, then dims 64 .. 127, read
// before, over the codes. The loops are rolled: the roles' code together does not fit the instruction cache.
__device__ __forceinline__ void wn_conv_codes(uint32_t tile, int R) {
  const uint32_t codes = tile + 16384u + R * 128;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint4 c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) c[q] = ld_shared_v4(codes + (((4 * h + q) ^ (R & 7)) << 4));
    const uint32_t at = tile + h * 16384u + R * 128;
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // 16 codes: two 16-byte chunks of fp16
      st_shared_v4(at + (((2 * q) ^ (R & 7)) << 4),
                   make_uint4(e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].x)), e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].x >> 16)),
                              e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].y)), e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].y >> 16))));
      st_shared_v4(at + (((2 * q + 1) ^ (R & 7)) << 4),
                   make_uint4(e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].z)), e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].z >> 16)),
                              e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].w)), e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].w >> 16))));
    }
  }
}
// bf16 row R of a tile times f -> fp16 in place.
__device__ __forceinline__ void wn_conv_row(uint32_t tile, int R, float f) {
#pragma unroll 1
  for (int h = 0; h < 4; ++h)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // (8 rows: 8 different bank groups)
      const uint32_t a = tile + (h >> 1) * 16384u + R * 128 + (((4 * (h & 1) + q) ^ (R & 7)) << 4);
      const uint4 v = ld_shared_v4(a);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xFFFF0000u) * f);
      st_shared_v4(a, make_uint4(y[0], y[1], y[2], y[3]));
    }
}
template <int HALVES>
__device__ __forceinline__ void wn_zero_row(uint32_t tile, int R) {
#pragma unroll 1
  for (int c = 0; c < HALVES * 8; ++c) st_shared_v4(tile + (c / 8) * 16384u + R * 128 + (c % 8) * 16, make_uint4(0, 0, 0, 0));
}

// One warp: an eighth of pool block b, chunk x of request q: four tokens' rows of K (part 0 .. 3) or of V, a cached block's
// codes or new tokens, 16 bytes a lane at a time.
__device__ __forceinline__ void wn_fill(const AttnParams& p, int b, int x, int part, const int4& q, int lane) {
  const WnPooled w(p, q.w);
  const int cached = w.cb - w.gap, row = p.Hkv * 128, t0 = 4 * (part & 3);  // (row: elements of a token)
  const bool of_v = part >= 4;
  uint4* const out =
      reinterpret_cast<uint4*>(static_cast<__half*>(of_v ? p.pool_v : p.pool_k) + (static_cast<int64_t>(b) * 16 + t0) * row);
  if (x < cached) {
    int src = p.block_tables[static_cast<int64_t>(q.x) * p.max_blocks + (x < w.hb ? x : x + w.gap)];
    if (src < 0 || src >= p.num_blocks) {
      if (lane == 0) flag_error(p.err, PKV_DEVERR_BLOCK);
      src = 0;
    }
    const uint4* const in = reinterpret_cast<const uint4*>((of_v ? p.v_codes : p.k_codes) + src * p.stride_block + t0 * row);
#pragma unroll 4
    for (int e = lane; e < row / 4; e += 32) {
      const uint4 c = in[e];
      out[2 * e] = make_uint4(e4m3x2_to_f16x2(static_cast<uint16_t>(c.x)), e4m3x2_to_f16x2(static_cast<uint16_t>(c.x >> 16)),
                              e4m3x2_to_f16x2(static_cast<uint16_t>(c.y)), e4m3x2_to_f16x2(static_cast<uint16_t>(c.y >> 16)));
      out[2 * e + 1] = make_uint4(e4m3x2_to_f16x2(static_cast<uint16_t>(c.z)), e4m3x2_to_f16x2(static_cast<uint16_t>(c.z >> 16)),
                                  e4m3x2_to_f16x2(static_cast<uint16_t>(c.w)), e4m3x2_to_f16x2(static_cast<uint16_t>(c.w >> 16)));
    }
    return;
  }
  // (rows behind the request's last stay as they were: no row sees them)
  const int tok = 16 * (x - cached) + t0;
  const int64_t first = static_cast<int64_t>(q.y) + tok;
  const int tokens = static_cast<int>(max(min(static_cast<int64_t>(min(4, q.z - tok)), p.num_tokens - first), int64_t(0)));
  const uint4* const in = reinterpret_cast<const uint4*>((of_v ? p.v_new : p.k_new) + first * row);
  const float f = of_v ? 1.f / p.ctx_v_scale : 1.f;
#pragma unroll 4
  for (int e = lane; e < tokens * (row / 8); e += 32) {
    const uint4 v = in[e];
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = pack_f16(__uint_as_float(u[c] << 16) * f, __uint_as_float(u[c] & 0xFFFF0000u) * f);
    out[e] = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

template <int D, int KIND>
__global__ void __launch_bounds__(WnCfg<D, KIND>::THREADS, 1)
    attn_window_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kt,
                       const __grid_constant__ CUtensorMap tm_vt, const __grid_constant__ CUtensorMap tm_ck,
                       const __grid_constant__ CUtensorMap tm_cv) {
  using C = WnCfg<D, KIND>;
  constexpr bool FP8 = C::FP8, F16 = C::F16, POOL = KIND == kWnPool;
  static_assert(!F16 || D == 128, "a code row is one 128-byte box");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                  // [slot][half][128][128 B]
  uint8_t* ring_k = smem + C::RING_OFF;  // [NBUF][half][128][128 B]
  uint8_t* ring_v = ring_k + C::NBUF * C::KV_BYTES;
  int4* s_req = reinterpret_cast<int4*>(smem + C::REQ_OFF);
  int* s_start = reinterpret_cast<int*>(smem + C::START_OFF);
  int* s_perm = reinterpret_cast<int*>(smem + C::PERM_OFF);
  WnItem* s_item = reinterpret_cast<WnItem*>(smem + C::ITEM_OFF);
  WnBars& bar = *reinterpret_cast<WnBars*>(smem + C::BAR_OFF);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_scan[C::MAXR / 32];
  // (kWnCodes: the requests of the pool, in memory that the epilogues use later)
  int4* const fill_req = reinterpret_cast<int4*>(smem + C::STAGE_OFF);
  int2* const fill_at = reinterpret_cast<int2*>(fill_req + C::MAXR);

  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  int n;
  const int begin = wn_set(p, n);

  if (tid == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 1);
    for (int b = 0; b < C::NBUF; ++b) {
      mbar_init(&bar.k_full[b], 1);
      mbar_init(&bar.k_empty[b], 1);
      mbar_init(&bar.v_full[b], 1);
      mbar_init(&bar.v_empty[b], 1);
      mbar_init(&bar.v_ready[b], FP8 ? C::NCONV : 1);
      if (FP8) mbar_init(&bar.k_ready[b], C::NCONV);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&bar.p_full[i][h], 4);
      mbar_init(&bar.o_final[i], 1);
    }
    for (int w = 0; w < 4; ++w) mbar_init(&bar.rows[w], 2);
    for (int i = 0; i < C::ITEM_RING; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_empty[i], C::ITEM_READERS);
    }
    if (F16) mbar_init(&bar.q_ready, POOL ? 8 : C::NCONV);
    mbar_init(&bar.o_both, 1);
    mbar_init(&bar.drained, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == C::W_MMA) tc::tmem_alloc(&s_tmem, 512);

  // the set's requests
  if (F16 && p.pool_blocks > 0) {
    // those of the pool for kWnPool, the others for kWnCodes
    const int4 q = tid < n ? wn_request(p, begin, tid) : make_int4(0, 0, 0, 0);
    if (tid < n) s_perm[tid] = wn_pool_need(p, q);
    __syncthreads();
    if (tid < n) {
      const int base = wn_pool_base(p, s_perm, tid);
      s_req[tid] = make_int4(POOL ? base : q.x, q.y, (base >= 0) == POOL ? q.z : 0, q.w);
      s_start[tid] = wn_cost(p, q);
      if constexpr (FP8) {
        fill_req[tid] = q;
        fill_at[tid] = make_int2(base, base >= 0 ? s_perm[tid] : 0);
      }
    }
    if constexpr (FP8) {
      // the pool's blocks, dealt over the CTAs, before the items that stay with the codes
      __syncthreads();
      for (int i = 0; i < n; ++i) {
        const int2 at = fill_at[i];
        if (at.y == 0) continue;
        // eighths of blocks to warps, the next request's from where this one's end
        const int warps = static_cast<int>(gridDim.x) * (C::THREADS / 32);
        const int me = static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) * warp;
        const int first = static_cast<int>(static_cast<int64_t>(at.x) * 8 % warps);
        for (int e = me >= first ? me - first : me - first + warps; e < 8 * at.y; e += warps)
          wn_fill(p, at.x + (e >> 3), e >> 3, e & 7, fill_req[i], lane);
      }
    }
  } else if (tid < n) {
    const int4 q = wn_request(p, begin, tid);
    s_req[tid] = q;
    s_start[tid] = wn_cost(p, q);
  }
  static_assert(C::MAXR <= C::THREADS, "a thread a request");
  __syncthreads();
  // rank by cost, heaviest first, ties in set order (a stable order every CTA computes alike)
  if (tid < n) {
    const int ki = s_start[tid];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const int kj = s_start[j];
      rank += (kj > ki || (kj == ki && j < tid)) ? 1 : 0;
    }
    s_perm[rank] = tid;
  }
  __syncthreads();
  // exclusive prefix of the requests' items in that order
  {
    const int t = tid < n ? p.Hkv * wn_count(s_req[s_perm[tid]], p.G) : 0;
    int x = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31 && warp < C::MAXR / 32) s_scan[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < C::MAXR / 32; ++w) {
      if (w < warp) before += s_scan[w];
      all += s_scan[w];
    }
    if (tid < n) s_start[tid] = before + x - t;
    if (tid == 0) s_start[C::MAXR] = all;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  // When the last of few rounds of items would leave half the CTAs idle, its items are halved, into those of 128 rows that deal
  // their key tiles to both slots: 256 tokens of 64 and 8 heads under 4096 97 us without, 68 with; 2048 tokens 356 and 315
  // (with the codes converted by every item). Of more rounds it gains nothing: 8 x 301-512 tokens, 5.4 rounds, 50 and 50.
  const int all = s_start[C::MAXR], rest = all % static_cast<int>(gridDim.x);
  const bool few = all <= 4 * static_cast<int>(gridDim.x);
  const int halved = few && 2 * rest <= static_cast<int>(gridDim.x) ? rest : 0, W = all + halved;

  // The k-th item (null: no more, or a wait gave up). A reader frees it when it is through.
  auto take = [&](uint32_t k) -> const WnItem* {
    const uint32_t e = k % C::ITEM_RING;
    if (!wn_wait(&bar.item_full[e], (k / C::ITEM_RING) & 1, &s_abort, p.err)) return nullptr;
    return s_item[e].NV > 0 ? s_item + e : nullptr;
  };
  auto release = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.item_empty[k % C::ITEM_RING]);
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    // ======================= softmax =======================
    const int slot = warp >> 2, quad = warp & 3;
    const int t = tid & 127;  // row of the tile = TMEM lane
    const uint32_t lane_at = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int shift = __ffs(p.G) - 1;  // G is a power of two
    uint32_t sc = 0, oc = 0, bc = 0, rc = 0;  // phases: S of this slot, o_final, o_both, rows
    // kWnPool: the k-th item's Q to fp16, before the epilogue of the item before, so that its first S runs beside that
    auto convert_q = [&](uint32_t k) {
      const WnItem* taken = take(k);
      if (taken == nullptr) return;
      const bool split = taken->split;
      if (!wn_wait(&bar.q_full, k & 1, &s_abort, p.err)) return;
      if (slot == 0 || !split) wn_conv_row(smem_u32(sQ) + slot * C::Q_BYTES, t, 1.f);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_ready);
    };
    if constexpr (POOL) convert_q(0);
    for (uint32_t k = 0;; ++k) {
      const WnItem* taken = take(k);
      if (taken == nullptr) break;
      const WnItem it = *taken;
      release(k);
      float m = -CUDART_INF_F, l = 0.f;
      bool ok = true;
      const int tok = it.tok0 + (((it.split ? 0 : slot * 128) + t) >> shift);
      const bool live = __any_sync(0xffffffffu, tok < it.tok0 + it.ntok);  // the warp has rows of the item
      const int nt = it.tiles(), first = it.split ? slot : 0;
      const WnRow sees(p, it, it.C + tok);
      for (int j = first; j < nt; j += 1 + it.split, ++sc) {
        if (!wn_wait(&bar.s_full[slot], sc & 1, &s_abort, p.err)) { ok = false; break; }
        tc::fence_after_sync();
        if (live) {
          const uint32_t srow = lane_at + wn_scol(slot);
          // Over codes a score of a cached key counts in the key scale's units. A tile of both kinds is brought to those of
          // the new keys.
          const int nc = F16 ? 128 * j < 16 * it.cached() ? 16 * it.cached() - 128 * j : 0 : 0;  // its cached columns
          const bool both = F16 && nc > 0 && nc < min(128, 16 * it.NV - 128 * j);
          const float sl = F16 && nc > 0 && !both ? p.ctx_scale_log2 : p.scale_log2;
          if (both || !it.full(j)) {
            // What is hidden becomes -inf in tensor memory, 32 columns at a time (a warp's rows are few tokens: they see
            // most such groups whole). In registers, with the four groups' code in a row, it is fetched anew
            // for nearly every edge tile: 1340 clocks.
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t seen = sees.seen(128 * j + 32 * c);
              if (!both && __all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
              uint32_t x[32];
              tc::ld32(srow + 32 * c, x);
              tc::wait_ld();
              tc::touch32(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if (F16 && both && 32 * c + e < nc) x[e] = __float_as_uint(__uint_as_float(x[e]) * p.ctx_k_scale);
                x[e] = (seen >> e) & 1u ? x[e] : 0xFF800000u;
              }
              tc::st32(srow + 32 * c, x);
            }
            tc::wait_st();
          }
          // kWnCodes: half a row at a time, the second half read twice, which leaves registers for the converters
          constexpr int G = FP8 ? 2 : 4;  // groups of 32 columns held
          uint32_t v[G][32];
          auto load = [&](int c0) {
#pragma unroll
            for (int c = 0; c < G; ++c) tc::ld32(srow + 32 * (c0 + c), v[c]);
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < G; ++c) tc::touch32(v[c]);  // no use of v may move above the wait
          };
          // row max of the raw scores (the scale is positive, so it commutes with max)
          float mq[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int c0 = 4 - G; c0 >= 0; c0 -= G) {
            load(c0);
#pragma unroll
            for (int e = 0; e < 32; e += 2)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int g = c % G, i = G == 4 ? e : (e & ~3) + 2 * (c / G);  // (four chains whatever G is)
                if (G == 4 || (e & 2) == 0)
                  mq[c] = sm::max3(mq[c], __uint_as_float(v[g][i]), __uint_as_float(v[g][i + 1]));
              }
          }
          const float mx = fmaxf(sm::max3(mq[0], mq[1], mq[2]), mq[3]) * sl;  // -inf stays -inf
          // The decision to follow is per row, but tcgen05.ld/st are warp-collective: the whole warp takes the
          // branch when any of its rows does (alpha is 1 for the others).
          if (__any_sync(0xffffffffu, mx > m + C::LAZY)) {  // (m may be -inf)
            float alpha = 1.f;
            if (mx > m + C::LAZY) {
              const float to = mx - C::RAISE;
              alpha = m == -CUDART_INF_F ? 0.f : ex2_approx(m - to);
              m = to;
            }
            l *= alpha;
            if (j > first) {
              // (O is quiescent: the P V product before was done before S of this tile)
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                const uint32_t a = lane_at + wn_ocol(slot) + c * 32;
                uint32_t o[32];
                tc::ld32(a, o);
                tc::wait_ld();
                tc::touch32(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tc::st32(a, o);
              }
            }
          }
          // P = 2^(s * scale_log2 - m), packed to 16-bit pairs over the first half of S
          const float neg_m = m == -CUDART_INF_F ? 0.f : -m;
          const uint64_t nm2 = sm::f2(neg_m, neg_m), sc2 = sm::f2(sl, sl);
          uint64_t rs2 = sm::f2(0.f, 0.f);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (FP8 && h == 1) load(2);
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const uint64_t x =
                    sm::fma2(sm::f2(__uint_as_float(v[(2 * h + c) % G][e]), __uint_as_float(v[(2 * h + c) % G][e + 1])), sc2, nm2);
                float x0, x1;
                sm::unf2(x, x0, x1);
                const uint64_t pp = sm::f2(ex2_approx(x0), ex2_approx(x1));
                rs2 = sm::add2(rs2, pp);
                pk[16 * c + e / 2] = F16 ? sm::f16x2(pp) : sm::bf16x2(pp);
              }
            tc::st32(srow + 32 * h, pk);
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[slot][h]);
          }
          float r0, r1;
          sm::unf2(rs2, r0, r1);
          l += r0 + r1;
        } else if (lane == 0) {
          mbar_arrive(&bar.p_full[slot][0]);
          mbar_arrive(&bar.p_full[slot][1]);
        }
      }
      if (!ok) break;
      if constexpr (POOL) convert_q(k + 1);
      // ---- epilogue ----
      const int64_t row = static_cast<int64_t>(it.row0) + tok;
      const bool write = tok < it.tok0 + it.ntok && row < p.num_tokens;
      const int64_t flat = row * p.Hq + it.kh * p.G + (t & (p.G - 1));  // (128 is a multiple of G)
      // 32 columns of the warp's rows to `out` from column col on, through the warp's staging tile: a store then
      // writes 64 bytes of each of 8 rows (of 32 rows 16 bytes, four times the cache lines: 3500 clocks an item)
      const uint32_t stage = smem_u32(smem) + C::STAGE_OFF + warp * 2048;
      __nv_bfloat16* dst[4];  // row 8 i + lane / 4 of the warp's (NULL: not there), from 16-byte chunk lane % 4 on
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tr = quad * 32 + 8 * i + (lane >> 2), tk = it.tok0 + (((it.split ? 0 : slot * 128) + tr) >> shift);
        const int64_t rw = static_cast<int64_t>(it.row0) + tk;
        dst[i] = tk < it.tok0 + it.ntok && rw < p.num_tokens
                     ? p.out + (rw * p.Hq + it.kh * p.G + (tr & (p.G - 1))) * D + (lane & 3) * 8
                     : nullptr;
      }
      auto put = [&](const uint32_t (&o)[32], float f, const uint32_t (&o1)[32], float f1, int col) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = __uint_as_float(o[8 * q + e]) * f;
            if (&o != &o1) {
              // (a factor 0 stands for a part without keys: what its O holds is not read as a number)
              x[e] = f == 0.f ? 0.f : x[e];
              x[e] = f1 == 0.f ? x[e] : fmaf(__uint_as_float(o1[8 * q + e]), f1, x[e]);
            }
          }
          // 16-byte chunk q of row `lane`, 64-byte swizzle: conflict-free both ways
          st_shared_v4(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4),
                       make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + (lane >> 2), kk = lane & 3;  // row of the warp's 32, 16-byte chunk
          const uint4 v = ld_shared_v4(stage + rr * 64 + ((kk ^ ((rr >> 1) & 3)) << 4));
          if (dst[i] != nullptr) *reinterpret_cast<uint4*>(dst[i] + col) = v;
        }
        __syncwarp();
      };
      if (!it.split) {
        if (!wn_wait(&bar.o_final[slot], oc & 1, &s_abort, p.err)) break;
        ++oc;
        tc::fence_after_sync();
        if (live) {
          const float inv = l == 0.f ? 0.f : (F16 ? p.ctx_v_scale : 1.f) / l;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {  // (unrolled, its code is fetched anew for every item: 3500 clocks)
            uint32_t o[32];
            tc::ld32(lane_at + wn_ocol(slot) + c * 32, o);
            tc::wait_ld();
            tc::touch32(o);
            put(o, inv, o, 0.f, c * 32);
          }
          if (write && p.lse) p.lse[flat] = l == 0.f ? -CUDART_INF_F : (m + __log2f(l)) * 0.69314718055994531f;
        }
        tc::fence_before_sync();
        continue;
      }
      // a split item: the slots' states of the same rows, merged by both warps of the rows, half of the dims each
      float2* mrg = reinterpret_cast<float2*>(smem + C::MERGE_OFF);
      mrg[slot * 128 + t] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.rows[quad]);
      if (!wn_wait(&bar.rows[quad], rc & 1, &s_abort, p.err)) break;
      ++rc;
      if (!wn_wait(&bar.o_both, bc & 1, &s_abort, p.err)) break;
      ++bc;
      tc::fence_after_sync();
      if (live) {
        const float2 a = mrg[t], b = mrg[128 + t];
        const float mm = fmaxf(a.x, b.x);
        const float w0 = a.y == 0.f ? 0.f : ex2_approx(a.x - mm), w1 = b.y == 0.f ? 0.f : ex2_approx(b.x - mm);
        const float sum = a.y * w0 + b.y * w1, inv = sum == 0.f ? 0.f : (F16 ? p.ctx_v_scale : 1.f) / sum;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          const int col = slot * (D / 2) + c * 32;
          uint32_t o0[32], o1[32];
          tc::ld32(lane_at + wn_ocol(0) + col, o0);
          tc::ld32(lane_at + wn_ocol(1) + col, o1);
          tc::wait_ld();
          tc::touch32(o0);
          tc::touch32(o1);
          put(o0, w0 * inv, o1, w1 * inv, col);
        }
        if (write && slot == 0 && p.lse)
          p.lse[flat] = sum == 0.f ? -CUDART_INF_F : (mm + __log2f(sum)) * 0.69314718055994531f;
      }
      tc::fence_before_sync();
      // both have read O and the states before either lets the next item's products at them
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.rows[quad]);
      if (!wn_wait(&bar.rows[quad], rc & 1, &s_abort, p.err)) break;
      ++rc;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    // ---- loading K or V tiles ----
    // Lane c < 8: where chunk c of tile j lies: its cache block (`paged`; looked at when it is used, so that nothing
    // waits for it here), or ~ its first row of new tokens.
    bool paged = false;
    auto look_up = [&](const WnItem& it, int j) {
      int at = 0;
      paged = false;
      const int v = C::CHUNKS * j + lane;
      if (lane < C::CHUNKS && v < it.NV) {
        const int u = it.chunk(v);
        if (POOL) return ~(16 * (it.r + WnPooled(p, it.C).at(u)));
        paged = u < it.cb;
        at = paged ? p.block_tables[static_cast<int64_t>(it.r) * p.max_blocks + u] : ~(it.row0 + 16 * (u - it.cb));
      }
      return at;
    };
    // Tile i of the ring: the chunks at `where` (one a lane), once the buffer is free; then `peek` for the next tile's,
    // whose round trip to memory passes meanwhile. False: a wait gave up.
    auto load_tile = [&](uint32_t i, int where, int chunks, int kh, uint8_t* ring, uint64_t* full, uint64_t* empty,
                         const CUtensorMap* cache, const CUtensorMap* rows, const CUtensorMap* tile, auto peek) {
      if (paged && (where < 0 || where >= p.num_blocks)) {
        flag_error(p.err, PKV_DEVERR_BLOCK);
        where = 0;
      }
      int at[C::CHUNKS];
#pragma unroll
      for (int c = 0; c < C::CHUNKS; ++c) at[c] = __shfl_sync(0xffffffffu, where, c);
      // a tile of new tokens that follow one another comes in one box a half
      const bool run = at[0] < 0 && __all_sync(0xffffffffu, lane >= chunks || where == at[0] - 16 * lane);
      const int blocks = FP8 ? __popc(__ballot_sync(0xffffffffu, lane < chunks && where >= 0)) : 0;
      peek();
      const uint32_t b = i % C::NBUF;
      bool ok = true;
      if (tc::elect()) {
        if (i >= C::NBUF) ok = wn_wait1(&empty[b], (i / C::NBUF - 1) & 1, &s_abort, p.err);
        if (ok) {
          uint8_t* dst = ring + b * C::KV_BYTES;
          // (a block's codes are half of what its values would be)
          mbar_arrive_expect_tx(&full[b], run ? C::KV_BYTES : chunks * 16 * D * 2 - blocks * 16 * D);
          if (run) {
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf)
              tma_load_3d(dst + hf * C::KV_HALF, tile, &full[b], 0, kh * C::HALVES + hf, ~at[0]);
          } else {
            // (a chunk of new rows is a 4-D box like a block's, the rows' coordinate in place of the block's)
#pragma unroll
            for (int c = 0; c < C::CHUNKS; ++c) {
              if (c >= chunks) break;
              const CUtensorMap* map = at[c] >= 0 ? cache : rows;
              const int row = at[c] >= 0 ? 0 : ~at[c], blk = at[c] >= 0 ? at[c] : 0;
              if (FP8 && at[c] >= 0) {
                tma_load_4d(dst + C::KV_HALF + c * 2048, map, &full[b], 0, kh, 0, blk);
                continue;
              }
#pragma unroll
              for (int hf = 0; hf < C::HALVES; ++hf)
                tma_load_4d(dst + hf * C::KV_HALF + c * 2048, map, &full[b], 0, kh * C::HALVES + hf, row, blk);
            }
          }
        }
      }
      return __all_sync(0xffffffffu, ok) != 0;
    };
    // a wait gave up: the loads in flight are waited for (bounded), so that none lands after the CTA is gone
    auto drain = [&](uint32_t n, uint64_t* full) {
      for (uint32_t i = n > C::NBUF ? n - C::NBUF : 0; i < n; ++i) mbar_wait(&full[i % C::NBUF], (i / C::NBUF) & 1, p.err);
    };

    if (warp == C::W_K) {
      // ======================= items, Q and K =======================
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_kt);
        if (!POOL && p.seq_lens != nullptr) tma_prefetch_desc(&tm_ck);
      }
      uint32_t kc = 0, qn = 0;
      bool ok = true;
      int odd = 0;
      int w = blockIdx.x;
      // item w of the launch (NV 0: there is none)
      WnItem it;
      auto make = [&]() {
        it.NV = 0;
        if (w >= W) return;
        const int x = w < all ? w : w - halved;
        int lo = 0, hi = n - 1;  // the last rank whose prefix is at most x
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_start[mid] <= x) lo = mid; else hi = mid - 1;
        }
        it = wn_item(p, s_req[s_perm[lo]], x - s_start[lo], x < all - halved ? -1 : w >= all);
      };
      // A CTA begins with the item of its own number; the next one is claimed as soon as an item begins and looked
      // up before its last tile, so that neither round trip to memory holds the loads up.
      make();
      int next = look_up(it, 0);
      for (uint32_t k = 0; ok; ++k) {
        const uint32_t e = k % C::ITEM_RING;
        if (k >= C::ITEM_RING && !wn_wait(&bar.item_empty[e], (k / C::ITEM_RING - 1) & 1, &s_abort, p.err)) { ok = false; break; }
        if (lane == 0) {
          s_item[e] = it;
          mbar_arrive(&bar.item_full[e]);
        }
        __syncwarp();
        if (it.NV == 0) break;
        int claimed = 0;
        if (p.sched_slot < 0) {
          claimed = w + (odd ? 2 * blockIdx.x + 1 : 2 * (gridDim.x - blockIdx.x) - 1);
          odd ^= 1;
        } else if (lane == 0) {
          claimed = gridDim.x + min(atomicAdd(&g_wn_next[p.sched_slot], 1u), static_cast<unsigned>(W));
        }
        const int nt = it.tiles(), NV = it.NV, kh = it.kh, q_tiles = it.split ? 1 : 2, q_row = it.row0 + it.tok0;
        for (int j = 0; j < nt && ok; ++j) {
          const int where = next;
          auto peek = [&]() {
            if (j + 1 == nt) {
              w = __shfl_sync(0xffffffffu, claimed, 0);
              make();
              // kWnPool: its Q is on the way to L2 before the buffer is free, since converting it comes before its first S (236
              // and 232 us on 2048 tokens under 4096; over bf16 8 x 301-512 tokens take 49.5 and 50.6)
              if (POOL && it.NV > 0 && tc::elect())
                for (int s = 0; s < (it.split ? 1 : 2); ++s)
#pragma unroll
                  for (int hf = 0; hf < C::HALVES; ++hf)
                    tma_prefetch_l2_4d(&tm_q, 0, hf, it.kh * p.G, it.row0 + it.tok0 + s * (128 / p.G));
              __syncwarp();
            }
            next = look_up(it, j + 1 < nt ? j + 1 : 0);
          };
          if (!(ok = load_tile(kc, where, min(C::CHUNKS, NV - C::CHUNKS * j), kh, ring_k, bar.k_full, bar.k_empty, &tm_ck, &tm_k,
                               &tm_kt, peek)))
            break;
          ++kc;
          if (j == 0) {
            // the Q buffer is free once the previous item's S products are done (the first keys need not wait for that)
            if (k > 0 && !wn_wait(&bar.q_empty, (k - 1) & 1, &s_abort, p.err)) { ok = false; break; }
            if (tc::elect()) {
              mbar_arrive_expect_tx(&bar.q_full, q_tiles * C::Q_BYTES);
              for (int s = 0; s < q_tiles; ++s)
#pragma unroll
                for (int hf = 0; hf < C::HALVES; ++hf)
                  tma_load_4d(sQ + s * C::Q_BYTES + hf * C::Q_HALF, &tm_q, &bar.q_full, 0, hf, kh * p.G, q_row + s * (128 / p.G));
            }
            __syncwarp();
            ++qn;
          }
        }
      }
      if (!ok) {
        drain(kc, bar.k_full);
        if (qn > 0) mbar_wait(&bar.q_full, (qn - 1) & 1, p.err);
      }
    } else if (warp == C::W_V) {
      // ======================= V =======================
      if (lane == 0) {
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_vt);
        if (!POOL && p.seq_lens != nullptr) tma_prefetch_desc(&tm_cv);
      }
      uint32_t vc = 0;
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        const WnItem* taken = take(k);
        if (taken == nullptr) break;
        const WnItem it = *taken;
        release(k);
        const int nt = it.tiles();
        int next = look_up(it, 0);
        for (int j = 0; j < nt; ++j) {
          const int where = next;
          auto peek = [&]() {
            if (j + 1 < nt) next = look_up(it, j + 1);
          };
          if (!(ok = load_tile(vc, where, min(C::CHUNKS, it.NV - C::CHUNKS * j), it.kh, ring_v, bar.v_full, bar.v_empty, &tm_cv,
                               &tm_v, &tm_vt, peek)))
            break;
          ++vc;
        }
      }
      if (*static_cast<volatile int*>(&s_abort)) drain(vc, bar.v_full);
    } else if (warp == C::W_MMA) {
      // ======================= MMA issuer =======================
      if (tc::elect()) {
        constexpr uint32_t kQk = F16 ? tc::idesc_f16(128, 0, 0, 0) : tc::idesc_bf16(128, 0, 0, 0),
                           kPv = F16 ? tc::idesc_f16(128, D, 0, 1) : tc::idesc_bf16(128, D, 0, 1);
        uint64_t* const k_in = FP8 ? bar.k_ready : bar.k_full;  // K that products may read
        // Shared-memory descriptors (tc::smem_desc) as their low words: the address in 16 bytes and the leading
        // offset; the high word is the same for all.
        constexpr uint32_t kLboK = (16u >> 4) << 16, kLboV = (static_cast<uint32_t>(C::KV_HALF) >> 4) << 16;
        auto desc = [](uint32_t lo) { return (static_cast<uint64_t>((1024u >> 4) | 1u << 14 | 2u << 29) << 32) | lo; };
        const uint32_t k_at = smem_u32(ring_k) >> 4, v_at = smem_u32(ring_v) >> 4, q_at = smem_u32(sQ) >> 4;
        uint32_t tc0 = 0;             // key tiles of the items before this one
        uint32_t pn0 = 0, pn1 = 0;    // P V products of each slot
        bool ok = true;
        auto wait = [&](uint64_t* b, uint32_t parity) {
          if (!wn_wait1(b, parity, &s_abort, p.err)) return false;
          tc::fence_after_sync();
          return true;
        };
        auto buf = [&](int j) { return (tc0 + j) % C::NBUF; };
        auto phase = [&](int j) { return ((tc0 + j) / C::NBUF) & 1; };
        auto k_there = [&](int j) { return wait(&k_in[buf(j)], phase(j)); };
        auto v_there = [&](int j) { return wait(&bar.v_ready[buf(j)], phase(j)); };
        // S = Q K^T of tile j (N = 16 chunks)
        auto qk = [&](int slot, int qtile, int j, int chunks) {
          const uint32_t qa = (q_at + qtile * (C::Q_BYTES >> 4)) | kLboK, kb = (k_at + buf(j) * (C::KV_BYTES >> 4)) | kLboK;
          const uint32_t idesc = kQk | static_cast<uint32_t>(2 * chunks) << 17;
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            tc::mma_ss(tmem + wn_scol(slot), desc(qa + (((s / 4) * C::Q_HALF + (s % 4) * 32) >> 4)),
                       desc(kb + (((s / 4) * C::KV_HALF + (s % 4) * 32) >> 4)), idesc, s > 0);
          tc::commit(&bar.s_full[slot]);
        };
        // O += P V of tile j, in two parts as its P comes
        auto pv_part = [&](int slot, int j, int chunks, bool acc, int h) {
          const uint32_t vb = (v_at + buf(j) * (C::KV_BYTES >> 4)) | kLboV;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 4 * h + i;
            if (c < chunks)
              tc::mma_ts(tmem + wn_ocol(slot), tmem + wn_scol(slot) + c * 8, desc(vb + c * 128), kPv, (acc || c > 0) ? 1u : 0u);
          }
        };
        auto pv = [&](int slot, int j, int chunks, bool acc) {
          const uint32_t n = slot ? pn1 : pn0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait(&bar.p_full[slot][h], n & 1)) return false;
            pv_part(slot, j, chunks, acc, h);
          }
          if (slot) ++pn1; else ++pn0;
          return true;
        };
        for (uint32_t k = 0; ok; ++k) {
          const uint32_t e = k % C::ITEM_RING;
          if (!wait(&bar.item_full[e], (k / C::ITEM_RING) & 1)) { ok = false; break; }
          const int NV = *static_cast<volatile int*>(&s_item[e].NV), split = *static_cast<volatile int*>(&s_item[e].split);
          mbar_arrive(&bar.item_empty[e]);
          if (NV == 0) break;
          const int nt = (NV + C::CHUNKS - 1) / C::CHUNKS;
          auto chunks = [&](int j) { return min(C::CHUNKS, NV - C::CHUNKS * j); };
          if (!wait(F16 ? &bar.q_ready : &bar.q_full, k & 1)) { ok = false; break; }
          if (!split) {
            // P V of tile t - 1 and S of tile t, slot by slot (one place in the code for each, so that it stays in
            // the instruction cache beside the other roles'). K and V are looked for while products run that were issued
            // before, and waited for only where they are needed.
            bool k_seen = false;
            for (int t = 0; t <= nt && ok; ++t) {
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                if (t > 0) {
                  if (!(ok = pv(s, t - 1, chunks(t - 1), t > 1))) break;
                  if (t == nt) tc::commit(&bar.o_final[s]);
                  if (s == 1) tc::commit(&bar.v_empty[buf(t - 1)]);
                }
                if (t < nt) {
                  if (s == 0 && !k_seen && !(ok = k_there(t))) break;
                  qk(s, s, t, chunks(t));
                  if (s == 0) {
                    k_seen = t + 1 < nt && mbar_test(&k_in[buf(t + 1)], phase(t + 1));
                  } else {
                    tc::commit(&bar.k_empty[buf(t)]);
                    if (t + 1 == nt) tc::commit(&bar.q_empty);
                    if (!(ok = v_there(t))) break;
                  }
                }
              }
            }
          } else {
            // The tiles go to the slots in turn, and what is issued next is what is there: S of tile jq (its slot's P V
            // is issued then), or a part of P V of tile jp. (In a fixed order P V of one tile waits for K of the
            // next but one, and the ring of V with it.)
            int jq = 0, jp = 0, h = 0;
            uint64_t t0 = 0;
            uint32_t idle = 0;
            while (jp < nt) {
              const int s = jp & 1;
              if (jq < nt && jq < jp + 2 && mbar_test(&k_in[buf(jq)], phase(jq))) {
                tc::fence_after_sync();
                qk(jq & 1, 0, jq, chunks(jq));
                tc::commit(&bar.k_empty[buf(jq)]);
                if (++jq == nt) tc::commit(&bar.q_empty);
                idle = 0;
              } else if (jp < jq && mbar_test(&bar.p_full[s][h], (s ? pn1 : pn0) & 1) &&
                         mbar_test(&bar.v_ready[buf(jp)], phase(jp))) {
                tc::fence_after_sync();
                pv_part(s, jp, chunks(jp), jp > 1, h);
                if (h == 1) {
                  tc::commit(&bar.v_empty[buf(jp)]);
                  if (s) ++pn1; else ++pn0;
                  ++jp;
                }
                h ^= 1;
                idle = 0;
              } else if ((++idle & 255u) == 0) {  // (bounded, as wn_wait1)
                const uint64_t now = globaltimer_ns();
                if (idle == 256u) t0 = now;
                if (now - t0 > kWaitLimitNs) {
                  flag_error(p.err, PKV_DEVERR_TIMEOUT);
                  *static_cast<volatile int*>(&s_abort) = 1;
                }
                if (*static_cast<volatile int*>(&s_abort)) { ok = false; break; }
              }
            }
            if (ok) tc::commit(&bar.o_both);
          }
          tc0 += nt;
        }
        if (!ok) {  // the products in flight are waited for (bounded) before tensor memory is freed
          tc::commit(&bar.drained);
          mbar_wait(&bar.drained, 0, p.err);
        }
      }
      __syncwarp();
    } else if constexpr (FP8) {
      if (warp >= C::W_CONV) {
        // ======================= conversions =======================
        // Four warps convert Q once an item, then each K tile as it lands, four others each V tile, a row a thread. (One
        // group for both: 384 us on 2048 tokens under 4096; two warps each, and the loops unrolled: 423.)
        const bool of_v = warp >= C::W_CONV + C::NCONV;
        const int R = tid & 127;  // (the groups begin at multiples of 128 threads)
        const uint32_t ring_base = smem_u32(of_v ? ring_v : ring_k), q_base = smem_u32(sQ);
        uint64_t *const full = of_v ? bar.v_full : bar.k_full, *const ready = of_v ? bar.v_ready : bar.k_ready;
        const float f = of_v ? 1.f / p.ctx_v_scale : 1.f;
        uint32_t n_tiles = 0;
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
          const WnItem* taken = take(k);
          if (taken == nullptr) break;
          const WnItem it = *taken;
          release(k);
          const int nt = it.tiles(), last = it.last(), sinks = p.sinks;
          if (!of_v) {
            if (!wn_wait(&bar.q_full, k & 1, &s_abort, p.err)) break;
#pragma unroll 1
            for (int s = 0; s < (it.split ? 1 : 2); ++s) wn_conv_row(q_base + s * C::Q_BYTES, R, 1.f);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_ready);
          }
          for (int j = 0; j < nt; ++j, ++n_tiles) {
            const uint32_t b = n_tiles % C::NBUF;
            if (!wn_wait(&full[b], (n_tiles / C::NBUF) & 1, &s_abort, p.err)) { ok = false; break; }
            const int v = C::CHUNKS * j + R / 16;
            if (v < it.NV) {  // (no product takes the rows of other chunks)
              const int u = it.chunk(v), key = it.pos(u) + R % 16;
              const uint32_t tile = ring_base + b * C::KV_BYTES;
              // value rows that no row sees become zeros: P = 0 there must not meet what is not finite
              if (of_v && !((key >= it.low || key < sinks) && key <= last && (u >= it.cb || key < it.C)))
                wn_zero_row<C::HALVES>(tile, R);
              else if (u < it.cb)
                wn_conv_codes(tile, R);
              else
                wn_conv_row(tile, R, f);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[b]);
          }
        }
      }
    } else {
      // ======================= value rows that no row sees =======================
      const uint32_t ring_base = smem_u32(ring_v);
      uint32_t vc = 0;
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        const WnItem* taken = take(k);
        if (taken == nullptr) break;
        const WnItem it = *taken;
        release(k);
        const int nt = it.tiles(), last = it.last(), sinks = p.sinks;
        for (int j = 0; j < nt; ++j, ++vc) {
          const int b = vc % C::NBUF;
          if (!wn_wait(&bar.v_full[b], (vc / C::NBUF) & 1, &s_abort, p.err)) { ok = false; break; }
          if (!it.full(j)) {
            const uint32_t tile = ring_base + b * C::KV_BYTES;
#pragma unroll 1
            for (int R = lane; R < C::BN; R += 32) {
              const int v = C::CHUNKS * j + R / 16;
              if (v >= it.NV) continue;  // (no product takes it)
              const int u = it.chunk(v), key = it.pos(u) + R % 16;
              const bool seen = (key >= it.low || key < sinks) && key <= last && (u >= it.cb || key < it.C);
              if (!seen) wn_zero_row<C::HALVES>(tile, R);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.v_ready[b]);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  // every role of this CTA is done, its producer's claims included: the launch's last CTA to get here sets the
  // slot back to zero for the next launch that uses it
  if (tid == 0 && p.sched_slot >= 0) {
    __threadfence();
    if (atomicAdd(&g_wn_done[p.sched_slot], 1u) == gridDim.x - 1) {
      atomicExch(&g_wn_next[p.sched_slot], 0u);
      atomicExch(&g_wn_done[p.sched_slot], 0u);
    }
  }
}

template <int D, int KIND>
cudaError_t launch(const AttnParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& tkt, const CUtensorMap& tvt, const CUtensorMap& tck, const CUtensorMap& tcv,
                   cudaStream_t stream) {
  constexpr int kSlot = KIND == kWnCodes  ? kAttrWinAttn128Fp8
                        : KIND == kWnPool ? kAttrWinAttn128Pool
                        : D == 64         ? kAttrWinAttn64
                                          : kAttrWinAttn128;
  const cudaError_t e =
      set_smem_attr_once(reinterpret_cast<const void*>(&attn_window_kernel<D, KIND>), wn_smem<D, KIND>(), kSlot);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_window_kernel<D, KIND>, dim3(num_sms()), dim3(WnCfg<D, KIND>::THREADS), wn_smem<D, KIND>(), stream, p, tq,
                    tk, tv, tkt, tvt, tck, tcv);
}

}  // namespace

// Converting ahead saves the items some 1 us a key tile, on the CTA that has most of them, and costs 3 us a round of items (their
// first and last tiles overlap less), 7 us for a launch and 0.15 ns a key and KV head converted. In halves of rounds (the last of few
// rounds may be halved, as in the kernel) and 256ths of a microsecond, fitted to pairs of times; of 69 the rule takes the slower side
// in seven, for 2 to 8 %. Without and with it, us, 64 query and 8 KV heads if no others are named: 2048 tokens under 4096 314 and
// 230, 512 98 and 74, 128 59 and 58; 8 x 512 under 128 84 and 105, 512 135 and 143, 768 165 and 164, 1024 198 and 187; 8 x 256
// under 1024 112 and 116, 2048 185 and 169; 8 x 128 under 1024 66 and 74, 2048 105 and 111, 4096 187 and 174; 1024 under 1024 63
// and 62, 512 37 and 42; 4 x 1024 of 8 and 8 heads under 1024 45 and 64; 8 x 512 of 16 and 1 68 and 62, 8 x 128 27 and 34.
// Converted, and slower: 2 x 2048 of 8 and 8 under 4096 103 and 107; 2048 under 1024 104 and 106, beside 8 x 64 134 and 144,
// beside 8 x 128 152 and 160.
int64_t attn_window_pool_blocks(int64_t num_tokens, int32_t max_reqs, int32_t max_q_len, int32_t max_seq_len, int Hq, int Hkv,
                                int32_t window, int32_t sinks) {
  const int G = Hq / Hkv, sms = num_sms();
  if (static_cast<int64_t>(max_q_len) * G < kPoolLong) return 0;
  const int64_t most = std::min<int64_t>(max_reqs, kAttnSetChunk), reqs = std::min(most, num_tokens * G / kPoolLong);
  const int64_t keys = std::min<int64_t>(max_seq_len, static_cast<int64_t>(window) + sinks);
  const int64_t items = (num_tokens * Hq + 255) / 256, rest = items % sms;
  const int64_t halves = 2 * (items / sms) + (rest == 0 ? 0 : items <= 4 * sms && 2 * rest <= sms ? 1 : 2);
  if (halves * (keys + 256 / G - 384) < 1800 + (reqs * keys + num_tokens) * Hkv / 24) return 0;
  const int64_t all = (static_cast<int64_t>(max_seq_len) + 15) / 16;
  const int64_t seen = (static_cast<int64_t>(sinks) + 15) / 16 + (static_cast<int64_t>(window) + 15) / 16 + 1;
  return std::min(most, num_tokens * G / kPoolRows) * (std::min(all, seen) + 1) + num_tokens / 16;
}

cudaError_t launch_attn_window(const AttnParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const CUtensorMap& tkt, const CUtensorMap& tvt, const CUtensorMap& tck, const CUtensorMap& tcv,
                               const CUtensorMap* pool, int D, bool fp8, cudaStream_t stream, int* launches) {
  *launches += 1;
  if (fp8) {
    if (p.pool_blocks > 0) *launches += 1;
    const cudaError_t e = launch<128, kWnCodes>(p, tq, tk, tv, tkt, tvt, tck, tcv, stream);
    if (e != cudaSuccess || p.pool_blocks == 0) return e;
    return launch<128, kWnPool>(p, tq, pool[0], pool[1], pool[2], pool[3], tck, tcv, stream);
  }
  return D == 64 ? launch<64, kWnBf16>(p, tq, tk, tv, tkt, tvt, tck, tcv, stream)
                 : launch<128, kWnBf16>(p, tq, tk, tv, tkt, tvt, tck, tcv, stream);
}

}  // namespace pkv
