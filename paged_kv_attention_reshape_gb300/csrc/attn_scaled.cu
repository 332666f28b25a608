// attn_scaled.cu — extend_attn over a block-scaled E4M3 cache (an fp32 scale for each 16-token block
// and KV head) on the tcgen05 tensor cores: several new tokens a request against their cached
// context and causally against themselves (vLLM blog "rocm-attention-backend", "Processing
// details: extend path").
//
// Mathematics. For a query row, context positions j of block b with E4M3 values k_j, v_j, and new
// tokens i with bf16 k_i, v_i:
//   u_j = log2(e) scale ks_b (q . k_j) + log2 vs_b,   u_i = log2(e) scale (q . k_i),
//   m the running max of u,  P = 2^(u - m),
//   O = sum_j P_j v_j + sum_i P_i v_i,   l = sum_j P_j / vs_b + sum_i P_i,
//   out = O / l,   lse = (m + log2 l) ln 2.
// The tensor core multiplies the E4M3 values themselves, exact in fp16, and the softmax applies both
// scales in fp32, where nothing is rounded to few bits. Taking the max over u rather than over the
// scores keeps P within [0, 2^15] whatever the scales, and costs nothing per column: the shift of the
// exponent and the factor of the sum are the block's. (Rounding scale * code to bf16 in the
// converter warps, the first form, put 2^-8 of each product into the exponent and of each value into
// the sum, and its conversions, 9 instructions for a pair of codes against 2, took 2.5 times as long:
// 5.7 ms against 2.3 on 8 x 512 tokens over contexts of 4K to 32K, Hq 64 / Hkv 8.)
// Queries and new keys become fp16 and must lie within its range (one that does not makes its scores no numbers);
// new values and their P stay bf16, so values of any size pass. A score that is no number makes l one and so the row's out and lse: the max of u
// passes over it, so a part of the keys (a slot's, a copy's, a piece's) is one without keys for a row where its l
// is 0, whatever its m. A row has a key at least, its own, so that its l is never 0 as a whole.
//
// Work items. The rows of a request for one KV head are its (token, query head of the group) pairs,
// tokens outermost, in tiles of 128 (a box of Q is G heads x 128 / G tokens). An item is two such
// tiles, one a head slot: a KV head's context is read once for 256 rows whatever G is, and a draft
// of 4 tokens at G = 8 is one tile of 32 rows where items of a token tile and a head pair would be
// four, with 4 rows used of 128 (32 x 4 tokens over 1K-4K: 385 us so, 95 packed). An item whose
// rows fit one tile splits its key tiles between the slots instead (even ones to slot 0, odd ones to
// slot 1, both on the one Q tile) and the two states are merged at the end, so both softmax
// warpgroups work on a request of few tokens. Items are claimed from a counter, heaviest first: with
// 256 rows an item they are few and long, and a static deal in snake order lost more to the spread
// of the last round (8 x 512: 2.42 ms against 2.09; 2048 over 100K: 7.45 against 6.35).
//
// Two launches of the one kernel. When the bound on new tokens leaves every request 128 rows at most
// (FEW), all items are split, and a tile's rows are copied to fill it: up to 32 rows four times, up to
// 64 twice, each copy with its own part of every key tile, so that the four warps of a slot share the
// softmax, which one would else do for all (a slot's step 1050 clocks against 2000 to 2700). The
// copies' states are joined with the slots' at the end. There are more converter warps, a fifth buffer in
// place of the second Q tile, and S is read 32 columns at a time, for which no registers need to change
// hands. 32 x 4 tokens over contexts of 1K to 4K, Hq 64 / Hkv 8: 66 us, 93 by the general launch (before
// either had a plan).
//
// Few items. With a workspace, items that are longer than a CTA's part of all, or that would leave CTAs idle
// in a last round, are dealt as equal shares of key tiles; a cut item's pieces leave fp32 partials, which
// a second kernel merges by their maxima and sums. (The plan is the same whoever claims what, so the
// results do not depend on timing.)
//
// What bounds it. Many rows: each slot's chain S, softmax (1900 clocks), P V, S of the next tile, 3650 clocks a
// key tile of 256 rows, in which the tensor core works 2080 (S and P share columns, and two slots fill
// tensor memory): 8 x 512 tokens over 4K to 32K 1.81 ms, 0.71 of the measured bf16 rate, 2048 tokens over
// 100K 4.83 ms, 0.73. FEW: the ring (a tile is loaded in 2400 clocks, converted in 900 to 1500 and held
// through its softmax, and five buffers hold two and a half): 32 x 4 tokens over 1K to 4K 66.5 us, 0.37 of
// the measured HBM rate.
//
// Roles (16 warps, one CTA per SM, persistent):
//   warps 0-3, 4-7  softmax of slot 0, 1 (thread t owns row t = TMEM lane t) and the epilogue; a row of S in
//                   two halves, the second read twice, which leaves registers for four converter warps
//                   (whole rows in 200 registers and two converters: 2.00 ms on the 8 x 512 tokens)
//   warp 8          TMA producer: claims the items, loads Q and the ring of K and V tiles (128 keys). One elected
//                   thread issues a tile's eight copies (eight lanes, one each: 1.83 ms against 1.79)
//   warp 9          MMA issuer, one elected thread, waits included: S = Q K^T, O += P V (P read from tensor
//                   memory). In a branch on lane == 0 every product's operands are moved from per-thread registers,
//                   135 clocks an MMA in this kernel, and the issue bounds it (a slot's softmax then takes 1600 of
//                   4000 clocks); waits by the whole warp and products in elected branches: 1.93 ms
//   warps 12-15     converters: E4M3 code tiles, Q and new keys to fp16 in shared memory, a row a thread (two warps, 1600
//                   clocks a tile of K or V, hold the faster issue back: 2.09 ms; two for K and two for V 1.89).
//                   Rolled loops over the rows and over K and V: unrolled ones cost 8%
//   FEW: warps 10-13 convert K and Q, 14-15 V, 66 us against 71 with two and two
// Tensor memory (512 columns): S_0 | S_1 | O_0 | O_1; P_s overwrites the first half of S_s.
#include <math_constants.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "softmax.cuh"
#include "tc.cuh"

namespace pkv {

namespace {

struct AsBase {
  static constexpr int D = 128, BN = 128, BS = 16, TBLK = BN / BS;
  static constexpr int HALF_BYTES = 128 * 128;       // 128 rows x 128 bytes
  static constexpr int TILE_BYTES = 2 * HALF_BYTES;  // one 128-row tile of Q, K or V in 16 bits
  static constexpr int MAXR = kAttnSetChunk;         // requests of the set one launch holds
  static constexpr int W_LOAD = 8, W_MMA = 9;
  static constexpr int MAXBUF = 5;
  // P = 2^(u - m + RAISE): with the lazy maximum (u <= m + 8) at most 2^15, so that fp16 holds 11 bits of every P down to
  // 2^-21 of the largest possible and rounds smaller ones to 2^-32 of a row's largest term.
  static constexpr float RAISE = 7.f;
  static constexpr int STAGE_WARP_BYTES = 32 * 64;
  static constexpr int ITEM_RING = 4;                // claimed items published to the other roles
  // key tile k of the CTA in slot k % SCALE_RING: the blocks' scales as they land (8 of K, 8 of V), and
  // what the softmax makes of them ({key scale * softmax scale, log2 of the value scale, its inverse,
  // -} a block). Slot k is written again for tile k + 4, whose K is loaded once S of tile k + 2 (with
  // five buffers, P V of tile k + 1) is done, which needs P of tile k + 1 (of tile k, in a split item,
  // where the products P V are issued in order): every reader is past tile k.
  static constexpr int SCALE_RING = 4;
  // Key tiles of a share, at least: 4 tokens over 32,000, Hkv 1: 47 us with 4, 37 with 8, 38 with 12, 41 with 16.
  static constexpr int MIN_TILES = 8;
  static constexpr uint32_t IDESC_QK = tc::idesc_f16(128, 128, 0, 0);
  static constexpr uint32_t IDESC_PV = tc::idesc_f16(128, D, 0, 1), IDESC_PV_NEW = tc::idesc_bf16(128, D, 0, 1);
};
struct AsBars {
  uint64_t q_full, q_empty, q_conv;
  uint64_t kv_full[AsBase::MAXBUF], kv_empty[AsBase::MAXBUF], conv_full[AsBase::MAXBUF];
  uint64_t s_full[2], p_full[2], o_final[2];
  uint64_t item_full[AsBase::ITEM_RING], item_empty[AsBase::ITEM_RING];
  uint64_t drained;                 // the products in flight when a role gave up
  uint64_t rep_full;                // slot 0's copies of the rows are joined (FEW)
  uint64_t merge_full, merge_done;  // slot 1's m and l are in shared memory; slot 0 has read them and O_1
};
// FEW: the launch for sets in which every request's rows for a KV head fit one tile (all items are split).
template <bool FEW>
struct AsCfg : AsBase {
  // converter warps: of K (Q and new keys too) and of V; the general launch's four convert both (its warps 10
  // and 11 are idle: a register split is by groups of four)
  static constexpr int W_CONV = FEW ? 10 : 12, NK = 4, NV = FEW ? 2 : 0, NCONV = NK + NV;
  static constexpr int WARPS = W_CONV + NCONV, THREADS = WARPS * 32;
  // The general launch has 128 registers a thread. (144, 120 and 104 spill nothing: 1.83 ms on 8 x 512 tokens; 144, 128
  // and 96 1.83, 152, 120 and 88 1.84, 152, 104 and 104 1.86, 128 each 1.86.)
  static constexpr int REGS_SOFTMAX = 144, REGS_OTHER = 120, REGS_CONV = 104;
  static_assert(FEW || 256 * REGS_SOFTMAX + 128 * REGS_OTHER + 128 * REGS_CONV == THREADS * 128, "register split");
  static constexpr int NBUF = FEW ? 5 : 4;           // K/V ring: one tile per buffer
  static constexpr int NQ = FEW ? 1 : 2;             // Q tiles of an item
  static constexpr int ROWS = NQ * 128;
  static constexpr int RING_OFF = NQ * TILE_BYTES;
  static constexpr int REQ_OFF = RING_OFF + NBUF * TILE_BYTES;  // int4 {r, row0, q_len, C}
  static constexpr int START_OFF = REQ_OFF + MAXR * 16;
  static constexpr int PERM_OFF = START_OFF + (MAXR + 2) * 4;   // set positions by cost, heaviest first
  static constexpr int WHOLE_OFF = PERM_OFF + MAXR * 4;         // items that are dealt whole
  static constexpr int TAIL_OFF = WHOLE_OFF + MAXR * 4;         // prefix of the key tiles of those in shares
  // output staging: per softmax warp, 32 rows x 32 bf16 columns (64-byte rows, 64-byte swizzle)
  static constexpr int STAGE_OFF = (TAIL_OFF + MAXR * 4 + 127) / 128 * 128;
  static constexpr int ITEM_READERS = 1 + 8 + NCONV;
  static constexpr int ITEM_OFF = STAGE_OFF + 8 * STAGE_WARP_BYTES;
  static constexpr int SCALE_OFF = ITEM_OFF + ITEM_RING * 48;
  static constexpr int FACTOR_OFF = SCALE_OFF + SCALE_RING * 2 * TBLK * 4;
  static constexpr int MERGE_OFF = FACTOR_OFF + SCALE_RING * TBLK * 16;  // slot 1's {m, l} by row (split items)
  static constexpr int REP_OFF = MERGE_OFF + 128 * 8;            // slot 0's {m, l} by row (FEW)
  static constexpr int BAR_OFF = REP_OFF + (FEW ? 128 * 8 : 0);
  static constexpr int SMEM = 1024 + BAR_OFF + static_cast<int>(sizeof(AsBars));
  static_assert(SMEM <= 226 * 1024, "shared memory");
};

__device__ __forceinline__ constexpr uint32_t as_scol(int slot) { return slot * 128u; }
__device__ __forceinline__ constexpr uint32_t as_ocol(int slot) { return 256u + slot * 128u; }

// What a launch leaves in the workspace: {shares} | per share the cut item that begins in it | per slot (two a
// share: of the item that is cut at its start, and of the one at its end) {m, l} of a piece's rows | its O.
struct AsPartials {
  int* head;
  int4* items;  // two a share: {pieces (0: none), the request's first row, the item's, KV head}, {rows, -, -, -}
  float2* ml;   // [slot][ROWS]
  float4* o;    // [slot][32 column quads][ROWS]
};
__host__ __device__ __forceinline__ int64_t as_ml_off(int slots) { return 128 + slots * 32ll; }
__host__ __device__ __forceinline__ int64_t as_o_off(int slots, int rows) { return as_ml_off(slots) + 8ll * slots * rows; }
__host__ __device__ __forceinline__ int64_t as_ws_bytes(int slots, int rows) { return as_o_off(slots, rows) + 512ll * slots * rows; }
__device__ __forceinline__ AsPartials as_partials(char* ws, int slots, int rows) {
  return AsPartials{reinterpret_cast<int*>(ws), reinterpret_cast<int4*>(ws + 128), reinterpret_cast<float2*>(ws + as_ml_off(slots)),
                    reinterpret_cast<float4*>(ws + as_o_off(slots, rows))};
}

// A piece of work, published in shared memory by the producer.
struct AsItem {
  int r, q_len;         // request, new tokens
  int row0;             // the request's first row of q
  int kh;               // KV head
  int base;             // first of the item's rows (rows of the request: token * G + head of the group)
  int split;            // 1: one tile of rows, key tiles dealt to the two slots
  int slot;             // of its partial; -1: the item is whole
  int j0;               // the piece's first key tile; from there on:
  int C, nct, NT;       // cached tokens and their key tiles (none if negative), all key tiles (0: no more work)
  int unused;
};
static_assert(sizeof(AsItem) == 48, "ring entry");
__device__ __forceinline__ int as_pairs(const int4& q, int G) { return (q.z * G + 255) / 256; }
// FEW: rows of a copy. A tile of up to 32 (64) rows holds four (two) copies of them, each of which takes
// its own quarter (half) of every key tile, so that all four warps have the same part of the softmax.
__device__ __forceinline__ int as_span(int rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
// Key tiles an item of the request walks at most: the schedule's order.
__device__ __forceinline__ int as_cost(const int4& q) { return (q.w + 127) / 128 + (q.z + 127) / 128; }

// Item idx of a request {request id, first query row, q_len, cached tokens}, as a whole.
template <bool FEW>
__device__ __forceinline__ AsItem as_item(const AttnParams& p, const int4& q, int idx) {
  AsItem it;
  it.r = q.x;
  it.row0 = q.y;
  it.q_len = q.z;
  it.kh = idx % p.Hkv;
  it.base = 256 * (as_pairs(q, p.G) - 1 - idx / p.Hkv);  // later (heavier) rows of a request first
  const int rows = min(256, q.z * p.G - it.base);
  it.split = FEW || rows <= 128;
  it.slot = -1;
  it.j0 = 0;
  it.C = q.w;
  it.nct = (q.w + 127) / 128;
  it.NT = it.nct + (it.base + rows - 1) / p.G / 128 + 1;
  return it;
}
// The last rank whose prefix is at most x.
__device__ __forceinline__ int as_rank(const int* prefix, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Counters of claimed items and of finished CTAs, in the launch's slot (launch.h); its last CTA to finish sets
// the slot back to zero. Without a slot the pieces are dealt statically, in snake order.
__device__ unsigned int g_as_next[kAttnSchedSlots];
__device__ unsigned int g_as_done[kAttnSchedSlots];

// Bounded wait that also gives up as soon as another role has given up; the same answer in all lanes.
__device__ __forceinline__ bool as_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
      if ((ok = mbar_try_wait(bar, parity))) break;
      if ((i & 63u) == 0) {
        if (*abort_flag) break;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          flag_error(err, PKV_DEVERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The same by one thread.
__device__ __forceinline__ bool as_wait1(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
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

// The k-th piece of work (null: no more, or a wait gave up). A reader frees it when it is through.
template <bool FEW>
__device__ __forceinline__ const AsItem* as_take(const uint8_t* smem, AsBars& bar, uint32_t k, volatile int* abort_flag,
                                                 unsigned int* err) {
  const uint32_t e = k % AsBase::ITEM_RING;
  if (!as_wait(&bar.item_full[e], (k / AsBase::ITEM_RING) & 1, abort_flag, err)) return nullptr;
  const AsItem* it = reinterpret_cast<const AsItem*>(smem + AsCfg<FEW>::ITEM_OFF) + e;
  return it->NT > 0 ? it : nullptr;
}
__device__ __forceinline__ void as_free(AsBars& bar, uint32_t k, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar.item_empty[k % AsBase::ITEM_RING]);
}

// ---- conversions ------------------------------------------------------------------------------------
// A K or V tile buffer is [2 halves][128 rows][128 B] (64 16-bit values of a row per half, 128-byte
// swizzle: 16-byte chunk q of row R at R * 128 + ((q ^ (R & 7)) << 4)). A context tile lands as
// codes, [128 rows][128 B] with the same swizzle, in the buffer's upper half: code row R lies exactly
// where fp16 row R of half 1 goes, and half 0 holds no codes, so a thread converts its own row in
// place: dims 0..63 into half 0, then dims 64..127, all read first, over the codes.
__device__ __forceinline__ void as_conv_codes(uint32_t tile, int R, bool keep) {
  uint4 c[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) c[q] = ld_shared_v4(tile + 16384u + R * 128 + ((q ^ (R & 7)) << 4));
#pragma unroll
  for (int q = 0; q < 8; ++q) {  // 16 codes: two 16-byte chunks of fp16
    uint4 a = make_uint4(0, 0, 0, 0), b = make_uint4(0, 0, 0, 0);
    if (keep) {
      a = make_uint4(e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].x)), e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].x >> 16)),
                     e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].y)), e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].y >> 16)));
      b = make_uint4(e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].z)), e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].z >> 16)),
                     e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].w)), e4m3x2_to_f16x2(static_cast<uint16_t>(c[q].w >> 16)));
    }
    const uint32_t base = tile + (q >> 2) * 16384u + R * 128;
    st_shared_v4(base + (((2 * (q & 3)) ^ (R & 7)) << 4), a);
    st_shared_v4(base + (((2 * (q & 3) + 1) ^ (R & 7)) << 4), b);
  }
}
// A pair of bf16 in fp16. What is beyond fp16 becomes no number, y + 0 y: as an infinity it could make a score -inf and
// its key vanish from the row unseen. (Infinities kept and finite numbers beyond fp16 told from them: 71.7 us against 66.6
// on 32 x 4 tokens.)
__device__ __forceinline__ uint32_t as_f16x2(uint32_t v) {
  uint32_t y = bf16x2_to_f16x2(v);
  asm("{\n\t.reg .b32 z;\n\tmov.b32 z, 0;\n\tfma.rn.f16x2 %0, %0, z, %0;\n\t}" : "+r"(y));
  return y;
}
// bf16 row R of a tile -> fp16 in place.
__device__ __forceinline__ void as_conv_bf16(uint32_t tile, int R) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t a = tile + h * 16384u + R * 128 + ((q ^ (R & 7)) << 4);  // 8 rows: 8 different bank groups
      const uint4 v = ld_shared_v4(a);
      st_shared_v4(a, make_uint4(as_f16x2(v.x), as_f16x2(v.y), as_f16x2(v.z), as_f16x2(v.w)));
    }
}
// The same, and again every `span` rows below.
__device__ __forceinline__ void as_conv_copies(uint32_t tile, int R, int span) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t a = tile + h * 16384u + R * 128 + ((q ^ (R & 7)) << 4);
      const uint4 v = ld_shared_v4(a);
      const uint4 f = make_uint4(as_f16x2(v.x), as_f16x2(v.y), as_f16x2(v.z), as_f16x2(v.w));
      for (int r = 0; r < 128 - R; r += span) st_shared_v4(a + r * 128, f);
    }
}
__device__ __forceinline__ void as_zero_row(uint32_t tile, int R) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 8; ++q) st_shared_v4(tile + h * 16384u + R * 128 + ((q ^ (R & 7)) << 4), make_uint4(0, 0, 0, 0));
}

// Columns n .. 31 of a 32-column chunk of S (raw fp32 bits) become -inf, so that whatever the tensor
// core wrote there never enters the arithmetic.
__device__ __forceinline__ void as_mask(uint32_t (&v)[32], int n) {
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = e < n ? v[e] : 0xFF800000u;
}

template <bool FEW>
__global__ void __launch_bounds__(AsCfg<FEW>::THREADS, 1)
    attn_scaled_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_ck,
                       const __grid_constant__ CUtensorMap tm_cv, char* ws, int ws_slots) {
  using C = AsCfg<FEW>;
  constexpr int D = C::D;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                  // [slot][half][128][128 B]
  uint8_t* ring = smem + C::RING_OFF;  // [NBUF][half][128][128 B]
  int* s_start = reinterpret_cast<int*>(smem + C::START_OFF);
  int* s_perm = reinterpret_cast<int*>(smem + C::PERM_OFF);
  int4* s_req = reinterpret_cast<int4*>(smem + C::REQ_OFF);
  int* s_whole = reinterpret_cast<int*>(smem + C::WHOLE_OFF);
  int* s_tail = reinterpret_cast<int*>(smem + C::TAIL_OFF);
  AsBars& bar = *reinterpret_cast<AsBars*>(smem + C::BAR_OFF);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_plan[3];  // items dealt whole; key tiles dealt in shares; tiles of a share

  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // this launch's chunk of the request set
  int begin = 0, n = p.max_reqs;
  if (p.bounds != nullptr) {
    begin = p.bounds[p.cls];
    n = p.bounds[p.cls + 1] - begin;
    if (n > p.max_reqs) {
      if (blockIdx.x == 0 && tid == 0) flag_error(p.err, PKV_DEVERR_REQS);
      n = p.max_reqs;
    }
    n = max(n, 0);
  }
  begin += p.set_offset;
  n = max(0, min(n - p.set_offset, C::MAXR));

  if (tid == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 1);
    mbar_init(&bar.q_conv, C::NK);
    for (int b = 0; b < C::NBUF; ++b) {
      mbar_init(&bar.kv_full[b], 1 + C::TBLK);  // the producer's bytes, and each block's scales
      mbar_init(&bar.kv_empty[b], 1);
      mbar_init(&bar.conv_full[b], C::NK);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 128);
      mbar_init(&bar.o_final[i], 1);
    }
    for (int i = 0; i < C::ITEM_RING; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_empty[i], C::ITEM_READERS);
    }
    mbar_init(&bar.drained, 1);
    mbar_init(&bar.rep_full, 128);
    mbar_init(&bar.merge_full, 128);
    mbar_init(&bar.merge_done, 128);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == C::W_MMA) tc::tmem_alloc(&s_tmem, 512);

  // the set's requests
  for (int i = tid; i < n; i += C::THREADS) {
    const int r = p.order ? p.order[begin + i] : begin + i;
    int4 q = make_int4(0, 0, 0, 0);
    if (r >= 0 && r < p.batch_reqs) {
      int q_len = max(0, p.cu_q[r + 1] - p.cu_q[r]);
      int c = max(0, p.seq_lens[r] - q_len);
      if (q_len > p.max_q_len) {
        if (blockIdx.x == 0) flag_error(p.err, PKV_DEVERR_LEN);
        q_len = p.max_q_len;
      }
      if (c > static_cast<int64_t>(p.max_blocks) * C::BS) {
        if (blockIdx.x == 0) flag_error(p.err, PKV_DEVERR_LEN);
        c = p.max_blocks * C::BS;
      }
      q = make_int4(r, p.cu_q[r], q_len, c);
    } else if (blockIdx.x == 0) {
      flag_error(p.err, PKV_DEVERR_REQS);
    }
    s_req[i] = q;
  }
  __syncthreads();
  // rank by cost, heaviest first, ties in set order (a stable order every CTA computes alike)
  for (int i = tid; i < n; i += C::THREADS) {
    const int ki = as_cost(s_req[i]);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const int kj = as_cost(s_req[j]);
      rank += (kj > ki || (kj == ki && j < i)) ? 1 : 0;
    }
    s_perm[rank] = i;
  }
  __syncthreads();
  // Plan, by one warp: lane i has the ranks from i * PER on. Items are claimed whole, longest first, unless
  //  - one is longer than 1.2 times a CTA's part of all: then all are dealt as equal shares of key tiles;
  //  - they are nearly alike and the last round would leave a fifth of the CTAs idle: then its items are.
  // (One context of 32,000 tokens for one KV head and 4 new tokens 322 us whole and 37 us in shares; 2048
  // tokens over 100K, 512 items in 3.4 rounds, 6.16 and 5.33 ms. Contexts from 1K to 4K for 256 items
  // balance to 5% whole; a share's two ends cost it some ten tiles.)
  if (warp == 0) {
    constexpr int PER = C::MAXR / 32;
    const int grid = gridDim.x;
    int64_t all = 0;
    int count = 0, longest = 0, shortest = INT_MAX;
#pragma unroll 1
    for (int i = lane * PER; i < min(n, lane * PER + PER); ++i) {
      const int4 q = s_req[s_perm[i]];
      const int items = p.Hkv * as_pairs(q, p.G), cost = as_cost(q);
      if (items > 0) {
        all += static_cast<int64_t>(items) * cost;
        count += items;
        longest = max(longest, cost);
        shortest = min(shortest, cost);
      }
    }
    int before = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
      all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    const int items_all = __shfl_sync(0xffffffffu, before, 31);
    before -= count;
    longest = __reduce_max_sync(0xffffffffu, longest);
    shortest = __reduce_min_sync(0xffffffffu, shortest);
    int whole_all = items_all;
    if (ws != nullptr && longest > C::MIN_TILES) {
      if (5ll * longest * grid > 6 * all)
        whole_all = 0;
      else if (5ll * shortest >= 4ll * longest && items_all % grid <= grid / 5 * 4)
        whole_all = items_all / grid * grid;
    }
    int tail = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      int at = before, sum = tail;
      for (int i = lane * PER; i < min(n, lane * PER + PER); ++i) {
        const int4 q = s_req[s_perm[i]];
        const int items = p.Hkv * as_pairs(q, p.G), whole = min(max(whole_all - at, 0), items);
        if (pass == 1) {
          s_start[i] = min(at, whole_all);
          s_whole[i] = whole;
          s_tail[i] = sum;
        }
        at += items;
        sum += (items - whole) * as_cost(q);
      }
      if (pass == 0) {  // to the exclusive prefix
        const int own = sum;
        tail = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, tail, o);
          if (lane >= o) tail += y;
        }
        const int total = __shfl_sync(0xffffffffu, tail, 31);
        tail -= own;
        if (lane == 0) {
          s_plan[0] = whole_all;
          s_plan[1] = total;
          s_plan[2] = max(C::MIN_TILES, (total + grid - 1) / grid);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  const int shares = (s_plan[1] + s_plan[2] - 1) / s_plan[2], W = s_plan[0] + shares;
  if (ws != nullptr && blockIdx.x == 0 && tid == 0) *as_partials(ws, ws_slots, C::ROWS).head = shares;

  auto convert = [&]() {
      // ======================= converters =======================
      // The first NK warps convert Q once per item, then each K tile as it lands, the others (or, if there are
      // none, the same) each V tile: rows ct, ct + 32 NK, .. a thread.
      const bool of_v = FEW && warp >= C::W_CONV + C::NK;
      const int ct = tid - (C::W_CONV + (of_v ? C::NK : 0)) * 32;
      const uint32_t q_base = smem_u32(sQ), ring_base = smem_u32(ring);
      uint32_t kvc = 0;
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        const AsItem* taken = as_take<FEW>(smem, bar, k, &s_abort, p.err);
        if (taken == nullptr) break;
        const AsItem it = *taken;
        as_free(bar, k, lane);
        if (!of_v) {
          if (!as_wait(&bar.q_full, k & 1, &s_abort, p.err)) break;
          if constexpr (FEW) {
            const int span = as_span(it.q_len * p.G);
            for (int R = ct; R < span; R += C::NK * 32) as_conv_copies(q_base, R, span);
          } else {
            for (int s = 0; s < (it.split ? 1 : 2); ++s) as_conv_bf16(q_base + s * C::TILE_BYTES, ct);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.q_conv);
        }
        for (int j = 0; j < it.NT && ok; ++j) {
#pragma unroll 1
          for (int sel = 0; sel < 2; ++sel, ++kvc) {
            // (every tile is waited for, the other group's too: five buffers hold K and V in turn, and a parity
            // tells a barrier's phase only to one who waited for the phase before)
            const int b = kvc % C::NBUF;
            if (!as_wait(&bar.kv_full[b], (kvc / C::NBUF) & 1, &s_abort, p.err)) { ok = false; break; }
            if (FEW && (sel != 0) != of_v) continue;
            const uint32_t tile = ring_base + b * C::TILE_BYTES;
            if (sel == 0 && ct < 8) {
              // the tile's softmax factors of block ct
              const uint32_t at = kvc / 2 % C::SCALE_RING;
              float4 f = make_float4(p.scale_log2, 0.f, 1.f, 0.f);
              if (j < it.nct) {
                const float* sc = reinterpret_cast<const float*>(smem + C::SCALE_OFF) + at * 16;
                // a zero scale counts as 2^-100: no logarithm of 0, no product of 0 and a masked -inf
                const float ks = fmaxf(sc[ct], 0x1p-100f), vs = fmaxf(sc[8 + ct], 0x1p-100f);
                f = make_float4(ks * p.scale_log2, __log2f(vs), 1.f / vs, 0.f);
              }
              reinterpret_cast<float4*>(smem + C::FACTOR_OFF)[at * 8 + ct] = f;
            }
#pragma unroll 1
            for (int R = ct; R < 128; R += FEW && of_v ? C::NV * 32 : C::NK * 32) {
              if (j < it.nct) {
                // V rows past the context's end become zeros (P = 0 there must not meet a NaN code)
                as_conv_codes(tile, R, sel == 0 || R < it.C - j * 128);
              } else if (sel == 0) {
                as_conv_bf16(tile, R);
              } else if (R >= it.q_len - (j - it.nct) * 128) {
                // new values stay as they come, but for rows past the request's own tokens
                as_zero_row(tile, R);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            // NK arrivals a tile, of K and of V
            if (FEW ? lane < (of_v ? C::NK / C::NV : 1) : lane == 0) mbar_arrive(&bar.conv_full[b]);
          }
        }
      }
  };

  if (warp < 8) {
    if constexpr (!FEW) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    // ======================= softmax warpgroups =======================
    if constexpr (!FEW) {
    const int slot = warp >> 2;
    const int t = tid & 127;  // row of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t sc = 0, oc = 0;  // S tiles of this slot; its O's
    uint32_t tile0 = 0;       // the CTA's key tiles before this item
    uint32_t par = 0;         // parities of the items whose slot 1 has an O (bit 0), of the merges (bit 1)
    for (uint32_t k = 0;; ++k) {
      const AsItem* taken = as_take<FEW>(smem, bar, k, &s_abort, p.err);
      if (taken == nullptr) break;
      float m = -CUDART_INF_F, l = 0.f;
      {
        const AsItem it = *taken;
        if (slot == 1 && it.split && it.NT == 1) {  // its one key tile is slot 0's
          tile0 += it.NT;
          as_free(bar, k, lane);
          continue;
        }
        const int tok = (it.base + (it.split ? 0 : slot * 128) + t) / p.G;  // this row's token
        bool ok = true;
        // a split item's slot walks every other tile, from its own index on
        for (int j = it.split ? slot : 0; j < it.NT; j += 1 + it.split) {
          if (!as_wait(&bar.s_full[slot], sc & 1, &s_abort, p.err)) { ok = false; break; }
          ++sc;
          tc::fence_after_sync();
          // valid keys of this row in tile j: columns [0, kv) (context) or causal (new)
          const bool ctx = j < it.nct;
          const int kv = ctx ? min(128, it.C - j * 128) : min(128, tok - (j - it.nct) * 128 + 1);
          const bool full = __all_sync(0xffffffffu, kv >= 128);
          const uint32_t srow = tmem + lane_off + as_scol(slot);
          // the factors of block g of the tile: {key scale * softmax scale, log2 vs, 1 / vs}
          const float4* fac = reinterpret_cast<const float4*>(smem + C::FACTOR_OFF) + (tile0 + j) % C::SCALE_RING * 8;
          // half a row of S at a time: the second and then the first for the max, and for P the first (whose P lies over
          // its own columns), the second read again
          uint32_t v[2][32];
          auto load = [&](int c0) {
            tc::ld32(srow + c0 * 32, v[0]);
            tc::ld32(srow + (c0 + 1) * 32, v[1]);
            tc::wait_ld();
            tc::touch32(v[0]);  // no use of v may move above the wait
            tc::touch32(v[1]);
            if (!full) {
              as_mask(v[0], kv - c0 * 32);
              as_mask(v[1], kv - (c0 + 1) * 32);
            }
          };
          // the max of a block's raw scores (its factor is positive), then of the blocks' u
          float mx = -CUDART_INF_F;
#pragma unroll
          for (int c0 = 2; c0 >= 0; c0 -= 2) {
            load(c0);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float mg = -CUDART_INF_F;
#pragma unroll
              for (int e = 0; e < 16; e += 2)
                mg = sm::max3(mg, __uint_as_float(v[g / 2][(g & 1) * 16 + e]), __uint_as_float(v[g / 2][(g & 1) * 16 + e + 1]));
              const float4 f = fac[2 * c0 + g];
              mx = fmaxf(mx, fmaf(mg, f.x, f.y));
            }
          }
          float alpha = 1.f;
          if (mx > m + 8.f || m == -CUDART_INF_F) {  // lazy rescale: only when the max really grows
            const float m_new = fmaxf(m, mx);
            if (m_new != -CUDART_INF_F) {
              alpha = (m == -CUDART_INF_F) ? 0.f : ex2_approx(m - m_new);
              m = m_new;
            }
          }
          const float neg_m = m == -CUDART_INF_F ? 0.f : C::RAISE - m;
          // P of the 16 columns of block g, packed over the first half of S: fp16 beside the context's
          // codes, bf16 beside new values; the row sum takes each P over its block's vs
          uint64_t rs2 = sm::f2(0.f, 0.f);
          auto exp_pass = [&](auto f16, int c0) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int gg = 0; gg < 2; ++gg) {
                const float4 f = fac[2 * (c0 + c) + gg];
                const uint64_t sc2 = sm::f2(f.x, f.x), nm2 = sm::f2(neg_m + f.y, neg_m + f.y), iv2 = sm::f2(f.z, f.z);
#pragma unroll
                for (int e = 16 * gg; e < 16 * gg + 16; e += 2) {
                  const uint64_t x = sm::fma2(sm::f2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), sc2, nm2);
                  float x0, x1;
                  sm::unf2(x, x0, x1);
                  const uint64_t pp = sm::f2(ex2_approx(x0), ex2_approx(x1));
                  rs2 = sm::fma2(pp, iv2, rs2);
                  pk[e / 2] = decltype(f16)::value ? sm::f16x2(pp) : sm::bf16x2(pp);
                }
              }
              tc::st16(srow + (c0 + c) * 16, pk);
            }
          };
          if (ctx) {
            exp_pass(std::true_type{}, 0);
            load(2);
            exp_pass(std::true_type{}, 2);
          } else {
            exp_pass(std::false_type{}, 0);
            load(2);
            exp_pass(std::false_type{}, 2);
          }
          float r0, r1;
          sm::unf2(rs2, r0, r1);
          l = l * alpha + (r0 + r1);
          // The rescale decision is per row, but tcgen05.ld/st are warp-collective: the whole
          // warp takes the branch when any of its rows needs it (alpha is 1 for the others).
          if (j > (it.split ? slot : 0) && __any_sync(0xffffffffu, alpha != 1.f)) {
            // O of this row is quiescent: the previous P V product finished before S(j) did
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc::ld32(tmem + lane_off + as_ocol(slot) + c * 32, o);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc::st32(tmem + lane_off + as_ocol(slot) + c * 32, o);
            }
          }
          tc::wait_st();
          tc::fence_before_sync();
          mbar_arrive(&bar.p_full[slot]);
        }
        if (!ok) break;
        tile0 += it.NT;
      }
      // ---- epilogue (the item read again, so that its fields need not stay in registers above) ----
      const AsItem it = reinterpret_cast<const AsItem*>(smem + C::ITEM_OFF)[k % C::ITEM_RING];
      as_free(bar, k, lane);
      const bool both = it.split && it.NT > 1;  // two states of the same rows
      float2* mrg = reinterpret_cast<float2*>(smem + C::MERGE_OFF);
      if (both && slot == 1) {
        // slot 0 merges the two states and writes the rows
        mrg[t] = make_float2(m, l);
        mbar_arrive(&bar.merge_full);
        if (!as_wait(&bar.merge_done, (par >> 1) & 1, &s_abort, p.err)) break;
        par ^= 2;
        ++oc;
        continue;
      }
      if (!as_wait(&bar.o_final[slot], oc & 1, &s_abort, p.err)) break;
      ++oc;
      float w0 = 1.f, w1 = 0.f;  // weights of this slot's O and of slot 1's
      if (both) {
        if (!as_wait(&bar.o_final[1], par & 1, &s_abort, p.err) || !as_wait(&bar.merge_full, (par >> 1) & 1, &s_abort, p.err))
          break;
        par ^= 2;
        const float2 o1 = mrg[t];
        const float mm = fmaxf(m, o1.x);
        w0 = l == 0.f ? 0.f : ex2_approx(m - mm);
        w1 = o1.y == 0.f ? 0.f : ex2_approx(o1.x - mm);
        l = l * w0 + o1.y * w1;
        m = mm;
      }
      if (both || !it.split) par ^= 1;
      tc::fence_after_sync();
      if (it.slot >= 0) {  // a piece: its O over 2^m and {m, l} to the workspace
        const AsPartials part = as_partials(ws, ws_slots, C::ROWS);
        const int row = (it.split ? 0 : slot * 128) + t;
        part.ml[static_cast<int64_t>(it.slot) * C::ROWS + row] = make_float2(m, l);
        float4* dst = part.o + static_cast<int64_t>(it.slot) * 32 * C::ROWS + row;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32], o1[32];
          tc::ld32(tmem + lane_off + as_ocol(slot) + c * 32, o);
          tc::ld32(tmem + lane_off + as_ocol(both ? 1 : slot) + c * 32, o1);
          tc::wait_ld();
          tc::touch32(o);
          tc::touch32(o1);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = __uint_as_float(o[e + i]) * w0;
              if (both) x[i] = fmaf(__uint_as_float(o1[e + i]), w1, x[i]);
            }
            dst[static_cast<int64_t>(c * 8 + e / 4) * C::ROWS] = make_float4(x[0], x[1], x[2], x[3]);
          }
        }
        tc::fence_before_sync();
        if (both) mbar_arrive(&bar.merge_done);
        continue;
      }
      const int base = it.base + (it.split ? 0 : slot * 128);  // the tile's first row of the request
      // flat row of [T * Hq] of tile row tr, or -1 for a row that is not there
      auto flat_row = [&](int tr) -> int64_t {
        const int rr = base + tr, tok = rr / p.G;
        const int64_t tk = static_cast<int64_t>(it.row0) + tok;
        return tok < it.q_len && tk < p.num_tokens ? tk * p.Hq + it.kh * p.G + rr % p.G : -1;
      };
      const float inv = w0 / l, inv1 = w1 / l;
      // O leaves through the warp's staging tile (32 rows x 32 columns at a time): each thread puts
      // its row there, then every store instruction writes 8 rows x 64 contiguous bytes
      uint32_t tid_now;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid_now));
      const uint32_t stg = ((smem_u32(smem_raw) + 1023u) & ~1023u) + C::STAGE_OFF + (tid_now >> 5) * C::STAGE_WARP_BYTES;
      const int wrow0 = static_cast<int>(tid_now & 96u);  // the warp's first row of the tile
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tc::ld32(tmem + lane_off + as_ocol(slot) + c * 32, o);
        tc::wait_ld();
        tc::touch32(o);
        if (both) {
          uint32_t o1[32];
          tc::ld32(tmem + lane_off + as_ocol(1) + c * 32, o1);
          tc::wait_ld();
          tc::touch32(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), inv1, __uint_as_float(o[e]) * inv));
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
        }
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint4 x;
          x.x = pack_bf16(__uint_as_float(o[q4 * 8 + 0]), __uint_as_float(o[q4 * 8 + 1]));
          x.y = pack_bf16(__uint_as_float(o[q4 * 8 + 2]), __uint_as_float(o[q4 * 8 + 3]));
          x.z = pack_bf16(__uint_as_float(o[q4 * 8 + 4]), __uint_as_float(o[q4 * 8 + 5]));
          x.w = pack_bf16(__uint_as_float(o[q4 * 8 + 6]), __uint_as_float(o[q4 * 8 + 7]));
          // 16-byte chunk q4 of row `lane`, 64-byte swizzle: conflict-free both ways
          st_shared_v4(stg + lane * 64 + ((q4 ^ ((lane >> 1) & 3)) << 4), x);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + (lane >> 2), kk = lane & 3;  // row of the warp's 32, 16-byte chunk
          const uint4 x = ld_shared_v4(stg + rr * 64 + ((kk ^ ((rr >> 1) & 3)) << 4));
          const int64_t fr = flat_row(wrow0 + rr);
          if (fr >= 0) *reinterpret_cast<uint4*>(p.out + fr * D + c * 32 + kk * 8) = x;
        }
        __syncwarp();
      }
      tc::fence_before_sync();
      if (both) mbar_arrive(&bar.merge_done);
      if (p.lse) {
        const int64_t fr = flat_row(t);
        if (fr >= 0) p.lse[fr] = (m - AsBase::RAISE + __log2f(l)) * 0.69314718055994531f;
      }
    }
    } else {
    const int slot = warp >> 2;
    const int t = tid & 127;  // row of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t sc = 0, oc = 0;  // S tiles of this slot; its O's
    uint32_t tile0 = 0;       // the CTA's key tiles before this item
    uint32_t par = 0;         // parities of the items whose slot 1 has an O (bit 0), of the merges (bit 1)
    uint32_t rc = 0;          // phases of rep_full
    for (uint32_t k = 0;; ++k) {
      const AsItem* taken = as_take<FEW>(smem, bar, k, &s_abort, p.err);
      if (taken == nullptr) break;
      const AsItem it = *taken;
      as_free(bar, k, lane);
      if (slot == 1 && it.NT == 1) {  // its one key tile is slot 0's
        tile0 += 1;
        continue;
      }
      // thread t: row t % span, keys [t / span * span, + span) of each tile
      const int span = as_span(it.q_len * p.G), row = t & (span - 1), c_lo = (t & ~(span - 1)) / 32, c_hi = c_lo + span / 32;
      const int g_log = __ffs(p.G) - 1;  // G is a power of two
      const int tok = row >> g_log;
      const bool idle = __all_sync(0xffffffffu, tok >= it.q_len);
      const uint32_t srow = tmem + lane_off + as_scol(slot);
      float m = -CUDART_INF_F, l = 0.f;
      bool ok = true;
      for (int j = slot; j < it.NT; j += 2) {
        if (!as_wait(&bar.s_full[slot], sc & 1, &s_abort, p.err)) { ok = false; break; }
        ++sc;
        tc::fence_after_sync();
        if (!idle) {
          const bool ctx = j < it.nct;
          const int kv = ctx ? min(128, it.C - j * 128) : min(128, tok - (j - it.nct) * 128 + 1);
          const float4* fac = reinterpret_cast<const float4*>(smem + C::FACTOR_OFF) + (tile0 + j) % C::SCALE_RING * 8;
          uint32_t v[32];
          auto load = [&](int c) {
            tc::ld32(srow + c * 32, v);
            tc::wait_ld();
            tc::touch32(v);
            as_mask(v, kv - c * 32);
          };
          float mx = -CUDART_INF_F;
#pragma unroll 1
          for (int c = c_hi - 1; c >= c_lo; --c) {
            load(c);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float mg = -CUDART_INF_F;
#pragma unroll
              for (int e = 16 * g; e < 16 * g + 16; e += 2) mg = sm::max3(mg, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              const float4 f = fac[2 * c + g];
              mx = fmaxf(mx, fmaf(mg, f.x, f.y));
            }
          }
          float alpha = 1.f;
          if (mx > m + 8.f || m == -CUDART_INF_F) {  // lazy rescale: only when the max really grows
            const float m_new = fmaxf(m, mx);
            if (m_new != -CUDART_INF_F) {
              alpha = (m == -CUDART_INF_F) ? 0.f : ex2_approx(m - m_new);
              m = m_new;
            }
          }
          const float neg_m = m == -CUDART_INF_F ? 0.f : C::RAISE - m;
          uint64_t rs2 = sm::f2(0.f, 0.f);
          uint32_t pk[16];
#pragma unroll 1
          for (int c = c_lo; c < c_hi; ++c) {
            if (c > c_lo) load(c);  // P so far lies below this chunk of S
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const float4 f = fac[2 * c + g];
              const uint64_t sc2 = sm::f2(f.x, f.x), nm2 = sm::f2(neg_m + f.y, neg_m + f.y), iv2 = sm::f2(f.z, f.z);
#pragma unroll
              for (int e = 16 * g; e < 16 * g + 16; e += 2) {
                const uint64_t x = sm::fma2(sm::f2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, nm2);
                float x0, x1;
                sm::unf2(x, x0, x1);
                const uint64_t pp = sm::f2(ex2_approx(x0), ex2_approx(x1));
                rs2 = sm::fma2(pp, iv2, rs2);
                pk[e / 2] = ctx ? sm::f16x2(pp) : sm::bf16x2(pp);
              }
            }
            tc::st16(srow + c * 16, pk);
          }
          // the other copies' keys
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < c_lo || c >= c_hi) tc::st16(srow + c * 16, pk);
          float r0, r1;
          sm::unf2(rs2, r0, r1);
          l = l * alpha + (r0 + r1);
          if (j > slot && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              tc::ld32(tmem + lane_off + as_ocol(slot) + c * 32, v);
              tc::wait_ld();
              tc::touch32(v);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              tc::st32(tmem + lane_off + as_ocol(slot) + c * 32, v);
            }
          }
          tc::wait_st();
        }
        tc::fence_before_sync();
        mbar_arrive(&bar.p_full[slot]);
      }
      if (!ok) break;
      tile0 += it.NT;
      // ---- epilogue: slot 0 joins the slots' states, then the copies', and writes the rows ----
      const bool both = it.NT > 1;
      float2* mrg = reinterpret_cast<float2*>(smem + C::MERGE_OFF);
      float2* rml = reinterpret_cast<float2*>(smem + C::REP_OFF);
      if (slot == 1) {
        mrg[t] = make_float2(m, l);
        mbar_arrive(&bar.merge_full);
        if (!as_wait(&bar.merge_done, (par >> 1) & 1, &s_abort, p.err)) break;
        par ^= 2;
        ++oc;
        continue;
      }
      if (!as_wait(&bar.o_final[0], oc & 1, &s_abort, p.err)) break;
      ++oc;
      float w0 = 1.f, w1 = 0.f;  // weights of this slot's O and of slot 1's
      bool has0 = l != 0.f, has1 = false;  // whether they had keys
      if (both) {
        if (!as_wait(&bar.o_final[1], par & 1, &s_abort, p.err) || !as_wait(&bar.merge_full, (par >> 1) & 1, &s_abort, p.err))
          break;
        par ^= 3;
        const float2 o1 = mrg[t];
        const float mm = fmaxf(m, o1.x);
        has1 = o1.y != 0.f;
        w0 = has0 ? ex2_approx(m - mm) : 0.f;
        w1 = has1 ? ex2_approx(o1.x - mm) : 0.f;
        l = l * w0 + o1.y * w1;
        m = mm;
      }
      // the copies of a row: their common max and sum
      rml[t] = make_float2(m, l);
      mbar_arrive(&bar.rep_full);
      if (!as_wait(&bar.rep_full, rc & 1, &s_abort, p.err)) break;
      ++rc;
      float mm = -CUDART_INF_F, ll = 0.f;
      for (int i = row; i < 128; i += span) mm = fmaxf(mm, rml[i].x);
      for (int i = row; i < 128; i += span) {
        const float2 o = rml[i];
        ll += o.y == 0.f ? 0.f : o.y * ex2_approx(o.x - mm);
      }
      const bool whole = it.slot < 0;
      const AsPartials part = as_partials(ws, ws_slots, C::ROWS);
      const float wr = ex2_approx(m - mm) / (whole ? ll : 1.f);
      w0 *= wr, w1 *= wr;
      tc::fence_after_sync();
      const int rows = min(it.q_len, static_cast<int>(min(static_cast<int64_t>(it.q_len), p.num_tokens - it.row0))) * p.G;
      const uint32_t stg = smem_u32(smem) + C::STAGE_OFF;  // [128 rows][32 fp32], 128-byte swizzle
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tc::ld32(tmem + as_ocol(0) + lane_off + c * 32, o);
        tc::wait_ld();
        tc::touch32(o);
        // (a state without keys has no part, whatever the tensor core made of its row)
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = has0 ? __float_as_uint(__uint_as_float(o[e]) * w0) : 0u;
        if (both) {
          uint32_t o1[32];
          tc::ld32(tmem + as_ocol(1) + lane_off + c * 32, o1);
          tc::wait_ld();
          tc::touch32(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (has1) o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), w1, __uint_as_float(o[e])));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          st_shared_v4(stg + t * 128 + ((q ^ (t & 7)) << 4), make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]));
        mbar_arrive(&bar.rep_full);
        if (!as_wait(&bar.rep_full, rc & 1, &s_abort, p.err)) { ok = false; break; }
        ++rc;
        // 8 rows x 32 columns a warp at a time, 8 columns a thread
        for (int r0 = (warp & 3) * 8; r0 < min(span, rows); r0 += 32) {
          const int rr = r0 + (lane >> 2), kk = lane & 3;
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0.f;
          for (int i = rr; i < 128; i += span) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 y = ld_shared_v4(stg + i * 128 + (((2 * kk + h) ^ (i & 7)) << 4));
              x[4 * h] += __uint_as_float(y.x);
              x[4 * h + 1] += __uint_as_float(y.y);
              x[4 * h + 2] += __uint_as_float(y.z);
              x[4 * h + 3] += __uint_as_float(y.w);
            }
          }
          if (!whole) {  // a piece: its O over 2^m to the workspace
            float4* dst = part.o + (static_cast<int64_t>(it.slot) * 32 + c * 8 + kk * 2) * C::ROWS + rr;
            dst[0] = make_float4(x[0], x[1], x[2], x[3]);
            dst[C::ROWS] = make_float4(x[4], x[5], x[6], x[7]);
          } else if (rr < rows) {
            const int64_t fr = (static_cast<int64_t>(it.row0) + (rr >> g_log)) * p.Hq + it.kh * p.G + (rr & (p.G - 1));
            *reinterpret_cast<uint4*>(p.out + fr * D + c * 32 + kk * 8) =
                make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
          }
        }
        // the staging tile is free again
        mbar_arrive(&bar.rep_full);
        if (!as_wait(&bar.rep_full, rc & 1, &s_abort, p.err)) { ok = false; break; }
        ++rc;
      }
      if (!ok) break;
      tc::fence_before_sync();
      if (both) mbar_arrive(&bar.merge_done);
      if (!whole) {
        if (t < span) part.ml[static_cast<int64_t>(it.slot) * C::ROWS + t] = make_float2(mm, ll);
      } else if (p.lse && t < min(span, rows))
        p.lse[(static_cast<int64_t>(it.row0) + tok) * p.Hq + it.kh * p.G + (row & (p.G - 1))] =
            (mm - AsBase::RAISE + __log2f(ll)) * 0.69314718055994531f;
    }
    }
  } else if (!FEW && warp >= C::W_CONV) {
    if constexpr (!FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONV));
    convert();
  } else {
    if constexpr (!FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    if (warp == C::W_LOAD) {
      // ======================= TMA producer =======================
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_ck);
        tma_prefetch_desc(&tm_cv);
      }
      uint32_t kvc = 0;
      bool ok = true;
      AsItem* s_item = reinterpret_cast<AsItem*>(smem + C::ITEM_OFF);
      int share = 0, pos = 0, end = 0;  // the share whose pieces are being dealt: tiles [pos, end) of the tail
      int turn = 0;                     // pieces taken of a static deal
      for (uint32_t items = 0; ok; ++items) {
        // take the next piece once the Q buffer is free, and publish it to the other roles
        if (items > 0 && !as_wait(&bar.q_empty, (items - 1) & 1, &s_abort, p.err)) break;
        const int e = static_cast<int>(items % C::ITEM_RING);
        if (items >= C::ITEM_RING && !as_wait(&bar.item_empty[e], (items / C::ITEM_RING - 1) & 1, &s_abort, p.err)) break;
        AsItem it;
        for (;;) {
          if (pos >= end) {
            int w = 0;
            if (p.sched_slot >= 0) {
              if (lane == 0) w = static_cast<int>(atomicAdd(&g_as_next[p.sched_slot], 1u));
              w = __shfl_sync(0xffffffffu, w, 0);
            } else {
              w = turn * gridDim.x + ((turn & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
              ++turn;
            }
            if (w >= W) {
              it.NT = 0;
              break;
            }
            if (w < s_plan[0]) {
              const int lo = as_rank(s_start, n, w);
              it = as_item<FEW>(p, s_req[s_perm[lo]], w - s_start[lo]);
              break;
            }
            share = w - s_plan[0];
            pos = share * s_plan[2];
            end = min(pos + s_plan[2], s_plan[1]);
            if (lane == 0) as_partials(ws, ws_slots, C::ROWS).items[2 * share] = make_int4(0, 0, 0, 0);
          }
          // the item at tile pos of the tail, and the part of it that lies in the share
          const int lo = as_rank(s_tail, n, pos);
          const int4 q = s_req[s_perm[lo]];
          const int cost = as_cost(q), k = (pos - s_tail[lo]) / cost, first = s_tail[lo] + k * cost, from = pos - first;
          pos = min(first + cost, end);
          it = as_item<FEW>(p, q, s_whole[lo] + k);
          if (from >= it.NT) continue;  // (an item of earlier rows has fewer tiles than its request's cost)
          const int pieces = (first + it.NT - 1) / s_plan[2] - first / s_plan[2] + 1;
          if (pieces > 1) {
            if (from == 0 && lane == 0) {
              int4* entry = as_partials(ws, ws_slots, C::ROWS).items + 2 * share;
              entry[0] = make_int4(pieces, it.row0, it.base, it.kh);
              entry[1] = make_int4(min(256, q.z * p.G - it.base), 0, 0, 0);
            }
            it.slot = 2 * share + (from == 0 ? 1 : 0);
            it.j0 = from;
            it.C -= from * 128;
            it.nct -= from;
            it.NT = min(it.NT, pos - first) - from;
          }
          break;
        }
        if (lane == 0) {
          s_item[e] = it;
          mbar_arrive(&bar.item_full[e]);
        }
        if (it.NT == 0) break;
        if (lane == 0) {
          const int nq = it.split ? 1 : 2;
          mbar_arrive_expect_tx(&bar.q_full, nq * C::TILE_BYTES);
          for (int s = 0; s < nq; ++s)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              tma_load_4d(sQ + s * C::TILE_BYTES + hf * C::HALF_BYTES, &tm_q, &bar.q_full, 0, hf, it.kh * p.G,
                          it.row0 + (it.base + s * 128) / p.G);
        }
        const int32_t* table = p.block_tables + static_cast<int64_t>(it.r) * p.max_blocks + it.j0 * 8;
        const int ctx_blocks = (it.C + 15) / 16;
        // a tile's table entries (lanes 0..7, a block each) are read a tile ahead: the loads are on a
        // split item's critical path
        auto entry = [&](int j) {
          const int lb = j * 8 + lane;
          return j < it.nct && lane < 8 ? table[lb < ctx_blocks ? lb : j * 8] : 0;
        };
        const int kh = __shfl_sync(0xffffffffu, it.kh, 0), row0 = __shfl_sync(0xffffffffu, it.row0, 0);
        const int nct = __shfl_sync(0xffffffffu, it.nct, 0);
        int next = entry(0);
        for (int j = 0; j < it.NT && ok; ++j) {
          const bool ctx = j < it.nct;
          int blk = next;
          if (blk < 0 || blk >= p.num_blocks) {
            flag_error(p.err, PKV_DEVERR_BLOCK);
            blk = 0;
          }
          next = entry(j + 1);
          int blks[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) blks[i] = __shfl_sync(0xffffffffu, blk, i);
#pragma unroll 1
          for (int sel = 0; sel < 2; ++sel, ++kvc) {
            const int b = kvc % C::NBUF;
            if (kvc >= C::NBUF && !as_wait(&bar.kv_empty[b], (kvc / C::NBUF - 1) & 1, &s_abort, p.err)) {
              ok = false;
              break;
            }
            uint8_t* dst = ring + b * C::TILE_BYTES;
            if (lane < 8) {
              if (ctx && sel == 0) {  // both scales come with K; kvc / 2 counts the CTA's key tiles
                const int64_t at = static_cast<int64_t>(blk) * p.Hkv + it.kh;
                float* dst_sc = reinterpret_cast<float*>(smem + C::SCALE_OFF) + kvc / 2 % C::SCALE_RING * 16 + lane;
                cp_async4(dst_sc, p.k_scales + at);
                cp_async4(dst_sc + 8, p.v_scales + at);
                cp_async_arrive_noinc(&bar.kv_full[b]);
              } else {
                mbar_arrive(&bar.kv_full[b]);
              }
            }
            __syncwarp();
            if (tc::elect()) {
              mbar_arrive_expect_tx(&bar.kv_full[b], ctx ? C::HALF_BYTES : C::TILE_BYTES);
              if (ctx) {
                // the blocks' 16 rows of codes each into the upper half of the buffer
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  tma_load_4d(dst + C::HALF_BYTES + i * 2048, sel ? &tm_cv : &tm_ck, &bar.kv_full[b], 0, kh, 0, blks[i]);
              } else {
                const int row = row0 + (j - nct) * 128;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                  tma_load_3d(dst + hf * C::HALF_BYTES, sel ? &tm_v : &tm_k, &bar.kv_full[b], 0, kh * 2 + hf, row);
              }
            }
            __syncwarp();
          }
        }
      }
      if (*const_cast<volatile int*>(&s_abort)) {  // a role gave up: wait (bounded) for the copies still in flight
        for (uint32_t i = kvc > C::NBUF ? kvc - C::NBUF : 0; i < kvc; ++i)
          __all_sync(0xffffffffu, mbar_wait(&bar.kv_full[i % C::NBUF], (i / C::NBUF) & 1, p.err));
        cp_async_wait_all();
      }
    } else if (warp == C::W_MMA) {
      // ======================= MMA issuer =======================
      if (tc::elect()) {
        uint32_t kvc = 0, pc0 = 0, pc1 = 0;  // K and V tiles before this item; P tiles consumed per slot
        bool ok = true;
        const uint64_t q_desc = tc::smem_desc(smem_u32(sQ), 16, 1024), k_desc = tc::smem_desc(smem_u32(ring), 16, 1024);
        const uint64_t v_desc = tc::smem_desc(smem_u32(ring), C::HALF_BYTES, 1024);
        auto qk = [&](int slot, int buf, int qtile) {
          const uint64_t qd = q_desc + qtile * (C::TILE_BYTES >> 4), kd = k_desc + buf * (C::TILE_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k / 4) * C::HALF_BYTES + (k % 4) * 32) >> 4;
            tc::mma_ss(tmem + as_scol(slot), qd + off, kd + off, C::IDESC_QK, k > 0);
          }
        };
        auto pv = [&](int slot, int buf, bool acc, bool ctx) {
          const uint64_t vd = v_desc + buf * (C::TILE_BYTES >> 4);
          const uint32_t idesc = ctx ? C::IDESC_PV : C::IDESC_PV_NEW;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc::mma_ts(tmem + as_ocol(slot), tmem + as_scol(slot) + k * 8, vd + ((k * 2048) >> 4), idesc,
                       (acc || k > 0) ? 1u : 0u);
        };
        auto wait_kv = [&](uint32_t h) {
          if (!as_wait1(&bar.conv_full[h % C::NBUF], (h / C::NBUF) & 1, &s_abort, p.err)) return false;
          tc::fence_after_sync();
          return true;
        };
        auto wait_p = [&](int slot) {
          uint32_t& c = slot ? pc1 : pc0;
          if (!as_wait1(&bar.p_full[slot], c & 1, &s_abort, p.err)) return false;
          ++c;
          tc::fence_after_sync();
          return true;
        };
        for (uint32_t items = 0; ok; ++items) {
          const uint32_t e = items % C::ITEM_RING;
          if (!as_wait1(&bar.item_full[e], (items / C::ITEM_RING) & 1, &s_abort, p.err)) break;
          const AsItem it = reinterpret_cast<const AsItem*>(smem + C::ITEM_OFF)[e];
          mbar_arrive(&bar.item_empty[e]);
          if (it.NT == 0) break;
          if (!as_wait1(&bar.q_conv, items & 1, &s_abort, p.err)) break;
          if (it.split) {
            // key tile j goes to slot j % 2: S(j) and the other slot's O += P V of tile j - 1, whichever has
            // its operands first (S(j) overwrites P(j - 2), whose product was issued a step before)
            auto do_s = [&](int j) {
              const uint32_t kh = kvc + 2 * j;
              if (!wait_kv(kh)) return false;
              qk(j & 1, kh % C::NBUF, 0);
              tc::commit(&bar.s_full[j & 1]);
              tc::commit(&bar.kv_empty[kh % C::NBUF]);
              if (j == it.NT - 1) tc::commit(&bar.q_empty);
              return true;
            };
            auto do_pv = [&](int j) {
              const uint32_t vh = kvc + 2 * j + 1;
              if (!as_wait1(&bar.conv_full[vh % C::NBUF], (vh / C::NBUF) & 1, &s_abort, p.err) || !wait_p(j & 1)) return false;
              pv(j & 1, vh % C::NBUF, j >= 2, j < it.nct);
              tc::commit(&bar.kv_empty[vh % C::NBUF]);
              if (j >= it.NT - 2) tc::commit(&bar.o_final[j & 1]);
              return true;
            };
            for (int j = 0; j <= it.NT && ok; ++j) {
              const uint32_t kh = kvc + 2 * j;
              const bool s_first = j == 0 || (j < it.NT && mbar_test(&bar.conv_full[kh % C::NBUF], (kh / C::NBUF) & 1));
              if (s_first) ok = do_s(j);
              if (ok && j > 0) ok = do_pv(j - 1);
              if (ok && !s_first && j < it.NT) ok = do_s(j);
            }
          } else if constexpr (!FEW) {
            // per key tile: S_0(j), O_1 += P_1 V (j - 1), S_1(j), O_0 += P_0 V (j), so that each softmax
            // warpgroup works while the tensor core serves the other
            for (int j = 0; j < it.NT; ++j) {
              const uint32_t kh = kvc + 2 * j, vh = kh + 1;
              if (!(ok = wait_kv(kh))) break;
              qk(0, kh % C::NBUF, 0);
              tc::commit(&bar.s_full[0]);
              if (j > 0) {
                if (!(ok = wait_p(1))) break;
                pv(1, (vh - 2) % C::NBUF, j - 1 > 0, j - 1 < it.nct);
                tc::commit(&bar.kv_empty[(vh - 2) % C::NBUF]);
              }
              qk(1, kh % C::NBUF, 1);
              tc::commit(&bar.s_full[1]);
              tc::commit(&bar.kv_empty[kh % C::NBUF]);
              if (j == it.NT - 1) tc::commit(&bar.q_empty);
              if (!(ok = as_wait1(&bar.conv_full[vh % C::NBUF], (vh / C::NBUF) & 1, &s_abort, p.err) && wait_p(0))) break;
              pv(0, vh % C::NBUF, j > 0, j < it.nct);
              // slot 0's O is final once this product is done: its epilogue may overlap slot 1's last
              // softmax and P V
              if (j == it.NT - 1) tc::commit(&bar.o_final[0]);
            }
            if (!ok || !(ok = wait_p(1))) break;
            const uint32_t vh = kvc + 2 * it.NT - 1;
            pv(1, vh % C::NBUF, it.NT > 1, it.NT - 1 < it.nct);
            tc::commit(&bar.kv_empty[vh % C::NBUF]);
            tc::commit(&bar.o_final[1]);
          }
          kvc += 2 * it.NT;
        }
        if (!ok) {  // a role gave up: wait (bounded) for the products in flight before the tensor memory goes
          tc::commit(&bar.drained);
          mbar_wait(&bar.drained, 0, p.err);
        }
      }
      __syncwarp();
    } else if (FEW) {
      convert();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  // every role of this CTA is done, its producer's claims included: the launch's last CTA to get here
  // sets the scheduler slot back to zero for the next launch that uses it
  if (tid == 0 && p.sched_slot >= 0) {
    __threadfence();
    if (atomicAdd(&g_as_done[p.sched_slot], 1u) == gridDim.x - 1) {
      atomicExch(&g_as_next[p.sched_slot], 0u);
      atomicExch(&g_as_done[p.sched_slot], 0u);
    }
  }
}

// The pieces of the items that were cut, joined by their maxima and sums. A CTA takes 32 rows and 32 columns of
// an item at a time: a warp four of the columns, a thread one of the rows.
constexpr int kMergeShares = 1024;  // CTAs of a launch of the kernel above, at most
__global__ void __launch_bounds__(256) attn_scaled_merge_kernel(const AttnParams p, char* ws, int ws_slots, int ROWS) {
  __shared__ int s_cut[kMergeShares], s_warp[8], s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_count = 0;
  pdl_wait();
  pdl_release();
  const AsPartials part = as_partials(ws, ws_slots, ROWS);
  const int shares = *part.head;
  __syncthreads();
  for (int i0 = 0; i0 < shares; i0 += 256) {  // the shares in which a cut item begins, in order
    const bool cut = i0 + tid < shares && part.items[2 * (i0 + tid)].x > 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, cut);
    if (lane == 0) s_warp[warp] = __popc(mask);
    __syncthreads();
    int at = s_count + __popc(mask & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    if (cut) s_cut[at] = i0 + tid;
    __syncthreads();
    if (tid == 255) s_count = at + (cut ? 1 : 0);
    __syncthreads();
  }
  const int per = ROWS / 32 * 4, units = s_count * per;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int share = s_cut[u / per], part_of = u % per;
    const int4 it = part.items[2 * share];
    const int np = it.x, rows = part.items[2 * share + 1].x;
    const int row = part_of / 4 * 32 + lane, c4 = part_of % 4 * 8 + warp;
    if (part_of / 4 * 32 >= rows) continue;
    // piece 0 is in slot 2 share + 1, piece i in 2 (share + i)
    auto ml = [&](int i) { return part.ml[static_cast<int64_t>(2 * (share + i) + (i == 0)) * ROWS + row]; };
    float m = -CUDART_INF_F, l = 0.f;
#pragma unroll 8
    for (int i = 0; i < np; ++i) m = fmaxf(m, ml(i).x);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < np; ++i) {
      const float2 x = ml(i);
      const float4 y = part.o[(static_cast<int64_t>(2 * (share + i) + (i == 0)) * 32 + c4) * ROWS + row];
      if (x.y != 0.f) {  // (a piece without a key for the row has no part)
        const float w = ex2_approx(x.x - m);
        l = fmaf(x.y, w, l);
        s = make_float4(fmaf(y.x, w, s.x), fmaf(y.y, w, s.y), fmaf(y.z, w, s.z), fmaf(y.w, w, s.w));
      }
    }
    const int rr = it.z + row;
    const int64_t tok = static_cast<int64_t>(it.y) + rr / p.G;
    if (row >= rows || tok >= p.num_tokens) continue;
    const int64_t fr = tok * p.Hq + it.w * p.G + rr % p.G;
    const float inv = 1.f / l;
    *reinterpret_cast<uint2*>(p.out + fr * 128 + c4 * 4) = make_uint2(pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv));
    if (p.lse && c4 == 0) p.lse[fr] = (m - AsBase::RAISE + __log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace

// Whether an item of such a set can be cut, and how many rows a piece has.
static bool scaled_can_cut(int32_t max_seq_len) { return (static_cast<int64_t>(max_seq_len) + 127) / 128 + 1 > AsBase::MIN_TILES; }
static int scaled_rows(int32_t max_q_len, int G) { return static_cast<int64_t>(max_q_len) * G <= 128 ? 128 : 256; }
static int scaled_slots() { return 2 * num_sms(); }  // two for each CTA's share
size_t attn_scaled_workspace(int32_t max_q_len, int32_t max_seq_len, int G) {
  return scaled_can_cut(max_seq_len) ? static_cast<size_t>(as_ws_bytes(scaled_slots(), scaled_rows(max_q_len, G))) : 0;
}

template <bool FEW>
static cudaError_t launch_scaled(const AttnParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const CUtensorMap& tck, const CUtensorMap& tcv, char* ws, cudaStream_t stream, int* launches) {
  using C = AsCfg<FEW>;
  cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(&attn_scaled_kernel<FEW>), C::SMEM,
                                     FEW ? kAttrAttn128BlockFew : kAttrAttn128Block);
  if (e != cudaSuccess) return e;
  const int slots = ws != nullptr ? scaled_slots() : 0;
  e = launch_pdl(attn_scaled_kernel<FEW>, dim3(num_sms()), dim3(C::THREADS), C::SMEM, stream, p, tq, tk, tv, tck, tcv, ws, slots);
  *launches += 1;
  if (e != cudaSuccess || ws == nullptr) return e;
  *launches += 1;
  // (launched early, behind a long kernel, the merge's waiting CTAs cost the next call 3%; behind a short one
  // its early launch saves 3 us)
  if constexpr (FEW) return launch_pdl(attn_scaled_merge_kernel, dim3(4 * num_sms()), dim3(256), 0, stream, p, ws, slots, C::ROWS);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4 * num_sms());
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, attn_scaled_merge_kernel, p, ws, slots, C::ROWS);
}

// ws: attn_scaled_workspace(..) bytes, or null: no item is cut.
cudaError_t launch_attn_scaled(const AttnParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const CUtensorMap& tck, const CUtensorMap& tcv, void* workspace, cudaStream_t stream, int* launches) {
  char* ws = scaled_can_cut(p.max_seq_len) ? static_cast<char*>(workspace) : nullptr;
  return scaled_rows(p.max_q_len, p.G) == 128 ? launch_scaled<true>(p, tq, tk, tv, tck, tcv, ws, stream, launches)
                                              : launch_scaled<false>(p, tq, tk, tv, tck, tcv, ws, stream, launches);
}

}  // namespace pkv
