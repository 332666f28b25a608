// kv_append.cu — kv_append: the new tokens' queries and keys turned by their positions (rotary
// embedding), keys and values appended to the paged cache, in one pass over them (vLLM blog
// "rocm-attention-backend", "Unified attention backends": stage 1 of every forward writes the new
// K/V into the cache).
//
// Work is dealt in items of 16 dims of one head of one token: a rotated item i holds the dims
// whose angles are 8i .. 8i + 7 (both members of every pair, so a row may be rotated in place),
// any other item 16 dims in a row. An item is two 16-byte loads and two stores; a thread keeps one item
// column for all heads of its token, so its 8 cosines and sines are loaded once.
// Rounding: bf16 -> fp32 is exact, each product and sum of the rotation is rounded to fp32 by
// itself (no contraction, so the result does not depend on the compiler), then there is one
// rounding to the type that is stored.
// What bounds it: memory for long batches (each row is read and written once: 5.0 to 6.5 TB/s below),
// the round trips of slot, row and angle for short ones (2 us for one token, 5.5 us for 256 sequences).
// 10,000 tokens of 64 query and 8 KV heads of 128: 66 us into a bf16 cache; 84 us into a block-scaled
// one, where the runs need their rows in registers twice, for the maximum and for the codes; 76 us into a bf16 cache with
// norms of the heads (0.85 of the measured copy), whose additional work a pair of numbers shares an instruction for.
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "softmax.cuh"
#include "tc.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kBlockTokens = 16;  // block size of a block-scaled cache
// Tokens from which rows go through shared memory. The times (64 query and 8 KV heads of 128, a bf16
// cache, us on the GPU) through registers and through shared memory: 256 tokens 4.0 and 3.8, 512 5.8 and
// 4.8, 1024 8.3 and 6.9, 4096 38.8 and 30.2; of 8 and 2 heads of 64: 256 2.3 and 2.8, 512 3.6 and 3.6, 1024
// 4.8 and 4.4. Beside a block-scaled cache it is a launch more, worth it later where a token has many query heads (inputs
// and outputs beyond L2; a prompt's tokens; 64 and 8 heads, 64 and 4, 32 and 8, 8 and 2): 2048 tokens 22.7 and 27.6, 20.6
// and 22.9, 18.8 and 22.0, 12.8 and 12.7; 2800 30.8 and 32.2, 27.7 and 27.3, 25.4 and 25.6, 16.8 and 15.2; 4096 44.6 and
// 40.6, 40.5 and 35.7, 36.6 and 32.6, 23.8 and 19.6. (One token a sequence with 64 and 8 heads: 2800 72.8 and 78.6, 4096
// 106 and 106.) With norms, of a bf16 cache: 64 and 8 heads 256 tokens 6.2 and 6.0, 512 11.1 and 8.5, 1024 19.7 and 13.0; 32 and 8
// 512 8.0 and 6.5, 1024 14.2 and 9.8; 8 and 2 of 64 512 5.0 and 3.7, 1024 10.2 and 6.1; of one with tensor scales 64 and 8 256 6.3 and
// 6.4, 512 11.3 and 9.6, 32 and 8 256 4.6 and 5.1, 512 8.2 and 7.2. Beside a block-scaled cache the norms' registers bring the
// crossing forward: 64 and 8, 32 and 8, 8 and 2 2048 tokens 29.6 and 30.3, 23.2 and 24.2, 17.1 and 15.3; 2800 40.0 and 37.2, 31.2
// and 29.2, 22.7 and 18.9; 8 and 2 1024 11.6 and 13.5.
constexpr int kManyTokens = 512, kManyTokensBlock = 2900, kManyTokensBlockFewHeads = 2048, kFewHeads = 16;
constexpr int kManyTokensBlockNorm = 2300, kManyTokensBlockFewHeadsNorm = 1500;

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
// Eight floats times inv -> eight E4M3 codes (nearest, ties to even, saturating at +-448).
__device__ __forceinline__ uint2 codes8(const float* f, float inv) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(h[i])
        : "f"(__fmul_rn(f[2 * i + 1], inv)), "f"(__fmul_rn(f[2 * i], inv)));
  return make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16));
}

// The dims of item i of a head: two 8-dim chunks starting at a and b.
struct Item {
  int a, b;
  bool turn;
};
__device__ __forceinline__ Item item_of(const AppendParams& p, int i) {
  Item it;
  it.turn = i * 16 < p.rot;
  if (it.turn) {
    it.a = p.rot_off + (p.interleaved ? 16 * i : 8 * i);
    it.b = it.a + (p.interleaved ? 8 : p.rot / 2);
  } else {
    const int d = 16 * i - p.rot;  // the dims that are not rotated, in order
    it.a = d < p.rot_off ? d : d + p.rot;
    it.b = it.a + 8;
  }
  return it;
}
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const AppendParams& p, int64_t pos, int i, Angles& g) {
  const float4* c = reinterpret_cast<const float4*>(p.cos_sin + pos * p.rot + 8 * i);
  const float4* s = reinterpret_cast<const float4*>(p.cos_sin + pos * p.rot + p.rot / 2 + 8 * i);
  const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
  g = Angles{{c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w}, {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w}};
}
// x[0..7] (chunk a), x[8..15] (chunk b) turned in place.
__device__ __forceinline__ void turn(float* x, const Angles& g, bool interleaved) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // the pair of angle j: (x_j, x_{8+j}), or with interleaved pairs (x_{2j}, x_{2j+1})
    const float u = interleaved ? x[2 * j] : x[j], w = interleaved ? x[2 * j + 1] : x[8 + j];
    const float y = __fsub_rn(__fmul_rn(u, g.c[j]), __fmul_rn(w, g.s[j]));
    const float z = __fadd_rn(__fmul_rn(w, g.c[j]), __fmul_rn(u, g.s[j]));
    if (interleaved) {
      x[2 * j] = y;
      x[2 * j + 1] = z;
    } else {
      x[j] = y;
      x[8 + j] = z;
    }
  }
}

// The norm of a head before the rotation: y = R (x w) / sqrt(mean of squares + eps), in fp32. The factor of the row comes last,
// so that the sum of squares (a row's D / 16 items are neighbouring lanes of one warp, as D / 16 is a power of
// two, and add up along a tree of fixed order) is there when it is needed. Two numbers an instruction, and the
// rotation's second product in a fused one: 10,000 tokens of 64 and 8 heads of 128 take 86 us without.
// An item's 16 weights in pairs of fp32.
struct Weights {
  uint64_t a[4], b[4];
};
__device__ __forceinline__ void load_pairs(const void* w, bool f32, int at, uint64_t (&out)[4]) {
  if (f32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 u = __ldg(src), v = __ldg(src + 1);
    out[0] = sm::f2(u.x, u.y), out[1] = sm::f2(u.z, u.w), out[2] = sm::f2(v.x, v.y), out[3] = sm::f2(v.z, v.w);
  } else {
    float x[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + at)), x);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = sm::f2(x[2 * i], x[2 * i + 1]);
  }
}
__device__ __forceinline__ Weights load_weights(const AppendParams& p, const void* w, const Item& it) {
  Weights r = {};
  if (w != nullptr) {
    load_pairs(w, p.norm_f32, it.a, r.a);
    load_pairs(w, p.norm_f32, it.b, r.b);
  }
  return r;
}
// x[0..7] (chunk a), x[8..15] (chunk b) normed and turned in place.
__device__ __forceinline__ void norm_turn(const AppendParams& p, const Weights& w, const Angles& g, bool turns, int items, int lane,
                                          float* x) {
  uint64_t y[8], sq[2] = {sm::f2(0.f, 0.f), sm::f2(0.f, 0.f)};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = sm::f2(x[2 * i], x[2 * i + 1]);
    sq[i & 1] = sm::fma2(y[i], y[i], sq[i & 1]);
    y[i] = sm::mul2(y[i], i < 4 ? w.a[i] : w.b[i - 4]);
  }
  float s0, s1;
  sm::unf2(sm::add2(sq[0], sq[1]), s0, s1);
  float sum = s0 + s1;
  const uint32_t group = items == 32 ? 0xffffffffu : ((1u << items) - 1u) << (lane & ~(items - 1));
  for (int o = items >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(group, sum, o);
  if (turns) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // angles 2j and 2j + 1
      const uint64_t c = sm::f2(g.c[2 * j], g.c[2 * j + 1]), sn = sm::f2(g.s[2 * j], g.s[2 * j + 1]);
      const uint64_t ms = sm::f2(-g.s[2 * j], -g.s[2 * j + 1]);
      if (p.interleaved) {  // the pairs are (x_{2i}, x_{2i+1})
        float u0, w0, u1, w1;
        sm::unf2(y[2 * j], u0, w0);
        sm::unf2(y[2 * j + 1], u1, w1);
        const uint64_t u = sm::f2(u0, u1), v = sm::f2(w0, w1);
        const uint64_t a = sm::fma2(u, c, sm::mul2(v, ms)), b = sm::fma2(v, c, sm::mul2(u, sn));
        sm::unf2(a, u0, u1);
        sm::unf2(b, w0, w1);
        y[2 * j] = sm::f2(u0, w0);
        y[2 * j + 1] = sm::f2(u1, w1);
      } else {
        const uint64_t u = y[j], v = y[4 + j];
        y[j] = sm::fma2(u, c, sm::mul2(v, ms));
        y[4 + j] = sm::fma2(v, c, sm::mul2(u, sn));
      }
    }
  }
  // (D is a power of two: its inverse, and the product, are exact)
  const float inv = rsqrtf(fmaf(sum, p.norm_inv_d, p.norm_eps));
  const uint64_t inv2 = sm::f2(inv, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) sm::unf2(sm::mul2(y[i], inv2), x[2 * i], x[2 * i + 1]);
}

// Whether token t's row is to be written: its slot and position are in range (flagged if not).
__device__ __forceinline__ bool token_ok(const AppendParams& p, int64_t slot, int64_t pos, bool report) {
  if (slot < 0) return false;
  if (slot >= p.num_slots) {
    if (report) flag_error(p.err, PKV_DEVERR_SLOT);
    return false;
  }
  if (p.rot > 0 && (pos < 0 || pos >= p.max_pos)) {
    if (report) flag_error(p.err, PKV_DEVERR_LEN);
    return false;
  }
  return true;
}

// One CTA per group of TW tokens: their query rows and, unless the cache is block-scaled, their key and
// value rows, U rows of each token at a time a thread. The rows' loads, which depend on nothing but
// the token's index, are issued together with those of its slot and position and before those of its
// angles, so that a CTA costs two round trips to memory.
template <int KIND, int TW, int U, bool NORM>
__device__ __forceinline__ void append_rows(const AppendParams& p, int64_t group) {
  const int items = p.D / 16;
  const int i = threadIdx.x % items, h0 = threadIdx.x / items, hstep = blockDim.x / items;
  if (h0 >= hstep) return;  // the threads left over when items does not divide the CTA
  const Item it = item_of(p, i);
  // q heads, then k heads, then v heads
  const int rows = p.Hq + (KIND == PKV_KV_FP8_E4M3_BLOCK ? 0 : p.Hkv * (p.v != nullptr ? 2 : 1));
  const int64_t t0 = group * TW;
  Weights wq, wk;
  if constexpr (NORM) {
    wq = load_weights(p, p.q_norm, it);
    wk = load_weights(p, KIND == PKV_KV_FP8_E4M3_BLOCK ? nullptr : p.k_norm, it);
  }
  int64_t cache_off[TW];
  bool ok[TW];
  Angles g[TW];
  for (int r0 = h0; r0 < rows; r0 += U * hstep) {
    uint4 va[TW][U], vb[TW][U];
#pragma unroll
    for (int w = 0; w < TW; ++w)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * hstep;
        const int64_t t = t0 + w;
        if (r >= rows || t >= p.num_tokens) continue;
        const __nv_bfloat16* src = r < p.Hq           ? p.q + t * p.q_stride + r * p.D
                                   : r < p.Hq + p.Hkv ? p.k + t * p.k_stride + (r - p.Hq) * p.D
                                                      : p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * p.D;
        va[w][u] = *reinterpret_cast<const uint4*>(src + it.a);
        vb[w][u] = *reinterpret_cast<const uint4*>(src + it.b);
      }
    if (r0 == h0) {  // the first rows: the tokens' slots and positions, then their angles
      int64_t slot[TW], pos[TW];
#pragma unroll
      for (int w = 0; w < TW; ++w) {
        slot[w] = t0 + w < p.num_tokens ? p.slots[t0 + w] : -1;
        pos[w] = t0 + w < p.num_tokens && p.rot > 0 ? p.positions[t0 + w] : 0;
      }
#pragma unroll
      for (int w = 0; w < TW; ++w) {
        ok[w] = token_ok(p, slot[w], pos[w], threadIdx.x == 0);
        if (ok[w] && it.turn) load_angles(p, pos[w], i, g[w]);
        cache_off[w] = KIND == PKV_KV_FP8_E4M3_BLOCK || !ok[w]
                           ? 0
                           : (slot[w] / p.block_size) * p.stride_block + (slot[w] % p.block_size) * p.Hkv * p.D;
      }
    }
#pragma unroll
    for (int w = 0; w < TW; ++w)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * hstep;
        const int64_t t = t0 + w;
        if (r >= rows || !ok[w]) continue;
        const bool is_v = r >= p.Hq + p.Hkv;
        float x[16];
        unpack8(va[w][u], x);
        unpack8(vb[w][u], x + 8);
        const bool norms = NORM && (r < p.Hq ? p.q_norm != nullptr : !is_v && p.k_norm != nullptr);
        if (norms) {
          // (the weights' round trip passes beside the row's)
          norm_turn(p, r < p.Hq ? wq : wk, g[w], it.turn, items, threadIdx.x & 31, x);
        } else if (it.turn && !is_v) {
          if (p.interleaved) turn(x, g[w], true); else turn(x, g[w], false);
        }
        const uint4 a = pack8(x), b = pack8(x + 8);
        if (r < p.Hq) {
          __nv_bfloat16* dst = p.q_out + (t * p.Hq + r) * p.D;
          *reinterpret_cast<uint4*>(dst + it.a) = a;
          *reinterpret_cast<uint4*>(dst + it.b) = b;
          continue;
        }
        const int h = is_v ? r - p.Hq - p.Hkv : r - p.Hq;
        if (!is_v && p.k_out != nullptr) {
          __nv_bfloat16* dst = p.k_out + (t * p.Hkv + h) * p.D;
          *reinterpret_cast<uint4*>(dst + it.a) = a;
          *reinterpret_cast<uint4*>(dst + it.b) = b;
        }
        const int64_t off = cache_off[w] + h * p.D;
        if constexpr (KIND == PKV_KV_BF16) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + off;
          *reinterpret_cast<uint4*>(dst + it.a) = a;
          *reinterpret_cast<uint4*>(dst + it.b) = b;
        } else if constexpr (KIND == PKV_KV_FP8_E4M3) {
          uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + off;
          const float inv = is_v ? p.v_inv : p.k_inv;
          *reinterpret_cast<uint2*>(dst + it.a) = codes8(x, inv);
          *reinterpret_cast<uint2*>(dst + it.b) = codes8(x + 8, inv);
        }
      }
  }
}

// 2^ceil(log2(amax / 448)), clamped to [2^-64, 2^120], of a finite amax >= 0: 448 = 1.75 * 2^8, so
// with amax = m 2^e (1 <= m < 2) the exponent is e - 8, or e - 7 when m > 1.75.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = amax > 0.f ? min(max(e, -64), 120) : -64;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// One warp: the run that begins at token t, for one head of K or V of a block-scaled cache (head_dim 128:
// 8 items a row, 4 rows a pass). The run is those of tokens t .. t + 15 that have slots in block blk (rows
// skipped for what is wrong with them, or padding, may lie in between); which they are is read together with
// all the rows that there can be, so a run costs two round trips to memory (the second for the angles).
template <bool NORM>
__device__ __forceinline__ void append_run(const AppendParams& p, int64_t t, int64_t blk, int h, bool is_v, bool report,
                                           int lane) {
  constexpr int DH = 128, PASSES = kBlockTokens / 4;
  const int i = lane & 7, rr = lane >> 3;
  const int most = static_cast<int>(min(static_cast<int64_t>(kBlockTokens), p.num_tokens - t));
  const Item it = item_of(p, i);
  const __nv_bfloat16* src = is_v ? p.v + t * p.v_stride + h * DH : p.k + t * p.k_stride + h * DH;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  uint4 va[PASSES], vb[PASSES];
#pragma unroll
  for (int w = 0; w < PASSES; ++w) {
    const int j = 4 * w + rr;
    va[w] = vb[w] = make_uint4(0, 0, 0, 0);
    if (j < most) {
      va[w] = *reinterpret_cast<const uint4*>(src + j * stride + it.a);
      vb[w] = *reinterpret_cast<const uint4*>(src + j * stride + it.b);
    }
  }
  int64_t my_slot = -1, my_pos = 0;  // lane j: token t + j's
  if (lane < most) {
    my_slot = p.slots[t + lane];
    if (p.rot > 0) my_pos = p.positions[t + lane];
  }
  Weights wk;
  if constexpr (NORM) wk = load_weights(p, is_v ? nullptr : p.k_norm, it);
  float* sc = (is_v ? p.v_scales : p.k_scales) + blk * p.Hkv + h;
  const float s0 = blk * kBlockTokens < p.num_slots ? *sc : 0.f;
  const bool in = my_slot >= 0 && my_slot / kBlockTokens == blk;
  const int my_row = static_cast<int>(my_slot) & (kBlockTokens - 1);
  const int a = __reduce_min_sync(0xffffffffu, in ? my_row : kBlockTokens);  // the block's rows before a were there
  const bool ok = in && token_ok(p, my_slot, my_pos, report);
  const uint32_t mask = __ballot_sync(0xffffffffu, ok);
  if (mask == 0) return;
  float x[PASSES][16];
  uint32_t top = 0;  // the largest finite magnitude, as bits
#pragma unroll
  for (int w = 0; w < PASSES; ++w) {
    const int j = 4 * w + rr;
    const int64_t pos = __shfl_sync(0xffffffffu, my_pos, j);
    const bool live = (mask >> j) & 1u;
    unpack8(va[w], x[w]);
    unpack8(vb[w], x[w] + 8);
    const bool norms = NORM && !is_v && p.k_norm != nullptr;
    if (norms && live) {
      Angles g = {};
      if (it.turn) load_angles(p, pos, i, g);
      norm_turn(p, wk, g, it.turn, DH / 16, lane, x[w]);
    } else if (it.turn && !is_v && live) {
      Angles g;
      load_angles(p, pos, i, g);
      if (p.interleaved) turn(x[w], g, true); else turn(x[w], g, false);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t m = __float_as_uint(x[w][e]) & 0x7FFFFFFFu;
      top = max(top, live && m < 0x7F800000u ? m : 0u);
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const float need = scale_for(__uint_as_float(top));
  const float s1 = a > 0 ? fmaxf(s0, need) : need;
  uint8_t* blk_codes = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + blk * p.stride_block + h * DH;
  if (s1 != s0) {
    if (lane == 0) *sc = s1;
    // the rows that were there, at the new scale: 16 codes a lane
    const float f = __fdiv_rn(s0, s1);
    for (int j = rr; j < a; j += 4) {
      uint4* at = reinterpret_cast<uint4*>(blk_codes + static_cast<int64_t>(j) * p.Hkv * DH + 16 * i);
      const uint4 v = *at;
      const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
      float y[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t hh = e4m3x2_to_f16x2(static_cast<uint16_t>(wv[e >> 1] >> (16 * (e & 1))));
        const float2 ff = __half22float2(*reinterpret_cast<const __half2*>(&hh));
        y[2 * e] = ff.x;
        y[2 * e + 1] = ff.y;
      }
      const uint2 lo = codes8(y, f), hi = codes8(y + 8, f);
      *at = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
  const float inv = __fdiv_rn(1.f, s1);
#pragma unroll
  for (int w = 0; w < PASSES; ++w) {
    const int j = 4 * w + rr;
    const int row = __shfl_sync(0xffffffffu, my_row, j);
    if (!((mask >> j) & 1u)) continue;
    uint8_t* dst = blk_codes + static_cast<int64_t>(row) * p.Hkv * DH;
    *reinterpret_cast<uint2*>(dst + it.a) = codes8(x[w], inv);
    *reinterpret_cast<uint2*>(dst + it.b) = codes8(x[w] + 8, inv);
    if (!is_v && p.k_out != nullptr) {
      __nv_bfloat16* ko = p.k_out + ((t + j) * p.Hkv + h) * DH;
      *reinterpret_cast<uint4*>(ko + it.a) = pack8(x[w]);
      *reinterpret_cast<uint4*>(ko + it.b) = pack8(x[w] + 8);
    }
  }
}

// One CTA: the runs that begin in its group of tokens. A run begins at a token with a slot in a block that
// none of the 15 tokens before it has a slot in.
template <bool NORM>
__device__ __forceinline__ void append_runs(const AppendParams& p, int64_t group) {
  __shared__ int64_t s_block[kBlockTokens];
  __shared__ int s_lead[kBlockTokens];
  __shared__ int s_count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int64_t t0 = group * p.run_tokens;
  if (warp == 0) {
    constexpr int B = kBlockTokens - 1;
    const int64_t t = t0 - B + lane;
    const int64_t s = t >= 0 && t < p.num_tokens ? p.slots[t] : -1;
    const int64_t blk = s >= 0 ? s / kBlockTokens : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, blk), before = ((1u << B) - 1u) << max(lane - B, 0);
    const bool lead = s >= 0 && lane >= B && lane < B + p.run_tokens && (same & before) == 0;
    const uint32_t m = __ballot_sync(0xffffffffu, lead);
    if (lead) {
      const int at = __popc(m & ((1u << lane) - 1u));
      s_lead[at] = lane - B;
      s_block[at] = blk;
    }
    if (lane == 0) s_count = __popc(m);
  }
  __syncthreads();
  const int per = 2 * p.Hkv;  // K and V of each head
  for (int u = warp; u < s_count * per; u += nw) {
    const int l = u / per, v = u % per;
    append_run<NORM>(p, t0 + s_lead[l], s_block[l], v >> 1, v & 1, v == 0, lane);
  }
}

// ---- many tokens: rows through shared memory ---------------------------------------------------------
// One token's rows (q and, unless the cache is block-scaled, k and v) are contiguous, so they come and
// go as bulk copies: a persistent CTA's issuing warp keeps S - 1 tokens' loads in flight whatever the
// other warps do, they turn a token's rows in place, and it sends them on. (kv_append_kernel has as many
// loads in flight as its registers hold: 10,000 tokens of 64 query and 8 KV heads of 128 into a bf16
// cache 90 us, 4.6 TB/s; here 66 us, 6.5 TB/s. 4072 tokens with tensor scales 39.6 and 29 us.)
constexpr int kTurnWarps = kThreads / 32;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most N of this thread's groups of bulk stores have yet to be read out of shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }

// Bytes of one token's rows in a stage; its angles follow.
template <int KIND>
__host__ __device__ __forceinline__ int64_t row_bytes(const AppendParams& p) {
  return 2ll * p.D * (p.Hq + (KIND == PKV_KV_FP8_E4M3_BLOCK ? 0 : p.Hkv * (p.v != nullptr ? 2 : 1)));
}

// CTAs of the kernel an SM holds at most: by their registers, 72 a thread, and 96 with norms.
template <bool NORM>
constexpr int kStreamPerSm = NORM ? 2 : 3;

template <int KIND, uint32_t S, bool NORM>
__global__ void __launch_bounds__(kThreads + 32, kStreamPerSm<NORM>) kv_append_stream_kernel(AppendParams p) {
  extern __shared__ __align__(128) uint8_t sm_rows[];
  __shared__ uint64_t full[S], done[S];
  __shared__ int64_t s_slot[S];  // -1: a token that is skipped
  const int rb = static_cast<int>(row_bytes<KIND>(p)), sb = rb + p.rot * 4;
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&done[s], kTurnWarps);
    }
    fence_mbar_init();
  }
  pdl_wait();
  pdl_release();
  __syncthreads();
  const int64_t step = gridDim.x;
  if (tid >= kThreads) {  // the issuing warp
    // one elected thread (in a branch on the thread index the copies' operands take longer: 69.5 us against 66)
    if (!tc::elect()) return;
    // Token t into stage s; its slot and position were read a token earlier.
    int64_t slot_next = -1, pos_next = 0;
    auto peek = [&](int64_t t) {
      slot_next = t < p.num_tokens ? p.slots[t] : -1;
      pos_next = t < p.num_tokens && p.rot > 0 ? p.positions[t] : 0;
    };
    auto request = [&](int64_t t, uint32_t s) {
      const bool ok = t < p.num_tokens && token_ok(p, slot_next, pos_next, true);
      s_slot[s] = ok ? slot_next : -1;
      uint8_t* dst = sm_rows + s * sb;
      if (ok) {
        mbar_arrive_expect_tx(&full[s], sb);
        if (p.Hq > 0) bulk_load(dst, p.q + t * p.q_stride, 2 * p.Hq * p.D, &full[s]);
        if constexpr (KIND != PKV_KV_FP8_E4M3_BLOCK) {
          bulk_load(dst + 2 * p.Hq * p.D, p.k + t * p.k_stride, 2 * p.Hkv * p.D, &full[s]);
          if (p.v != nullptr) bulk_load(dst + 2 * (p.Hq + p.Hkv) * p.D, p.v + t * p.v_stride, 2 * p.Hkv * p.D, &full[s]);
        }
        if (p.rot > 0) bulk_load(dst + rb, p.cos_sin + pos_next * p.rot, p.rot * 4, &full[s]);
      } else {
        mbar_arrive(&full[s]);
      }
    };
    for (uint32_t s = 0; s < S - 1; ++s) {
      peek(blockIdx.x + s * step);
      request(blockIdx.x + s * step, s);
    }
    peek(blockIdx.x + (S - 1) * step);
    uint32_t k = 0;
    for (int64_t t = blockIdx.x; t < p.num_tokens; t += step, ++k) {
      const uint32_t s = k % S;
      if (!mbar_wait(&done[s], (k / S) & 1, p.err)) {
        // a wait gave up: the loads in flight are waited for (bounded)
        for (uint32_t j = k; j < k + S - 1; ++j) mbar_wait(&full[j % S], (j / S) & 1, p.err);
        break;
      }
      const int64_t slot = s_slot[s];
      if (slot >= 0) {
        const uint8_t* stage = sm_rows + s * sb;
        if (p.Hq > 0) bulk_store(p.q_out + t * p.Hq * p.D, stage, 2 * p.Hq * p.D);
        if constexpr (KIND != PKV_KV_FP8_E4M3_BLOCK) {
          const uint8_t* kr = stage + 2 * p.Hq * p.D;
          if (p.k_out != nullptr) bulk_store(p.k_out + t * p.Hkv * p.D, kr, 2 * p.Hkv * p.D);
          if constexpr (KIND == PKV_KV_BF16) {
            const int64_t off = (slot / p.block_size) * p.stride_block + (slot % p.block_size) * p.Hkv * p.D;
            bulk_store(static_cast<__nv_bfloat16*>(p.k_cache) + off, kr, 2 * p.Hkv * p.D);
            if (p.v != nullptr) bulk_store(static_cast<__nv_bfloat16*>(p.v_cache) + off, kr + 2 * p.Hkv * p.D, 2 * p.Hkv * p.D);
          }
        }
      }
      bulk_commit();
      // the stage of the token before is free once its stores have been read: the next token to request
      bulk_wait_read<1>();
      request(t + (S - 1) * step, (k + S - 1) % S);
      peek(t + S * step);
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    return;
  }
  const int items = p.D / 16, i = tid % items, h0 = tid / items, hstep = kThreads / items;
  const Item it = item_of(p, i);
  const int rows = rb / (2 * p.D);
  Weights wq, wk;
  if constexpr (NORM) {
    wq = load_weights(p, p.q_norm, it);
    wk = load_weights(p, p.k_norm, it);
  }
  uint32_t k = 0;
  for (int64_t t = blockIdx.x; t < p.num_tokens; t += step, ++k) {
    const uint32_t s = k % S;
    if (!mbar_wait(&full[s], (k / S) & 1, p.err)) return;
    uint8_t* stage = sm_rows + s * sb;
    const int64_t slot = s_slot[s];
    if (slot >= 0 && h0 < hstep) {
      Angles g;
      if (it.turn) {
        const float4* cs = reinterpret_cast<const float4*>(stage + rb);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 c = cs[2 * i + j], sn = cs[p.rot / 8 + 2 * i + j];
          g.c[4 * j] = c.x, g.c[4 * j + 1] = c.y, g.c[4 * j + 2] = c.z, g.c[4 * j + 3] = c.w;
          g.s[4 * j] = sn.x, g.s[4 * j + 1] = sn.y, g.s[4 * j + 2] = sn.z, g.s[4 * j + 3] = sn.w;
        }
      }
      const int64_t cache_off =
          KIND == PKV_KV_FP8_E4M3 ? (slot / p.block_size) * p.stride_block + (slot % p.block_size) * p.Hkv * p.D : 0;
      for (int r = h0; r < rows; r += hstep) {
        const bool is_v = r >= p.Hq + p.Hkv;
        uint4* a = reinterpret_cast<uint4*>(stage + 2 * (r * p.D + it.a));
        uint4* b = reinterpret_cast<uint4*>(stage + 2 * (r * p.D + it.b));
        const bool turns = it.turn && !is_v;
        const bool norms = NORM && !is_v && (r < p.Hq ? p.q_norm : p.k_norm) != nullptr;
        if (!turns && !norms && (KIND != PKV_KV_FP8_E4M3 || r < p.Hq)) continue;  // goes out as it came
        float x[16];
        unpack8(*a, x);
        unpack8(*b, x + 8);
        if (turns || norms) {
          if (norms) {
            norm_turn(p, r < p.Hq ? wq : wk, g, turns, items, tid & 31, x);
          } else {
            if (p.interleaved) turn(x, g, true); else turn(x, g, false);
          }
          *a = pack8(x);
          *b = pack8(x + 8);
        }
        if constexpr (KIND == PKV_KV_FP8_E4M3) {
          if (r >= p.Hq) {
            const int h = is_v ? r - p.Hq - p.Hkv : r - p.Hq;
            uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + cache_off + h * p.D;
            const float inv = is_v ? p.v_inv : p.k_inv;
            *reinterpret_cast<uint2*>(dst + it.a) = codes8(x, inv);
            *reinterpret_cast<uint2*>(dst + it.b) = codes8(x + 8, inv);
          }
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&done[s]);
  }
}

// The rows of TW tokens a CTA and, for a block-scaled cache (RUNS), before them the CTAs that append runs.
template <int KIND, int TW, int U, bool RUNS, bool NORM>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendParams p) {
  pdl_wait();
  pdl_release();
  if constexpr (RUNS) {
    if (blockIdx.x < p.run_groups) {
      append_runs<NORM>(p, blockIdx.x);
      return;
    }
    append_rows<KIND, TW, U, NORM>(p, static_cast<int64_t>(blockIdx.x) - p.run_groups);
  } else {
    append_rows<KIND, TW, U, NORM>(p, blockIdx.x);
  }
}
template <bool NORM>
__global__ void __launch_bounds__(kThreads) kv_append_runs_kernel(AppendParams p) {
  pdl_wait();
  pdl_release();
  append_runs<NORM>(p, blockIdx.x);
}

}  // namespace

// Rows through shared memory, if two CTAs of S stages fit an SM. The CTAs divide the tokens among them, so there are no more than
// run at once (kStreamPerSm): 10,000 tokens with norms of 32 and 8 heads of 128 into a bf16 cache 58 us (three CTAs an SM in the
// grid, of which two run: 75), of 64 and 8 into one with tensor scales 96 (123).
// More CTAs with fewer stages where codes are made or little is stored beside q, more stages where the
// copies are all there is: 10,000 tokens of 64 query and 8 KV heads of 128 into a bf16 cache 73.7 us
// with 3 stages and 69.5 with 4 (66 since an elected thread issues); into a block-scaled one 84.5 and 86.
template <int KIND, bool NORM>
static bool launch_stream(const AppendParams& p, cudaStream_t stream, cudaError_t* e) {
  constexpr uint32_t S = KIND == PKV_KV_BF16 ? 4 : 3;
  constexpr int64_t kRoom = 222 * 1024, kPerSm = kStreamPerSm<NORM>;
  const int64_t bytes = (row_bytes<KIND>(p) + p.rot * 4) * S, taken = bytes + 1280;  // with the static and reserved bytes
  if (2 * taken > kRoom) return false;
  *e = set_smem_attr_once(reinterpret_cast<const void*>(&kv_append_stream_kernel<KIND, S, NORM>), static_cast<int>(kRoom / 2),
                          (NORM ? kAttrAppendNorm0 : kAttrAppend0) + KIND);
  if (*e != cudaSuccess) return true;
  const int64_t grid = std::min<int64_t>(p.num_tokens, num_sms() * std::min<int64_t>(kRoom / taken, kPerSm));
  *e = launch_pdl(kv_append_stream_kernel<KIND, S, NORM>, dim3(static_cast<unsigned>(grid)), dim3(kThreads + 32),
                  static_cast<size_t>(bytes), stream, p);
  return true;
}

// Tokens from which launch_rows sends them through shared memory.
template <bool NORM>
static int many_tokens(const AppendParams& p, int kind) {
  if (kind != PKV_KV_FP8_E4M3_BLOCK) return kManyTokens;
  if (NORM) return p.Hq > kFewHeads ? kManyTokensBlockNorm : kManyTokensBlockFewHeadsNorm;
  return p.Hq > kFewHeads ? kManyTokensBlock : kManyTokensBlockFewHeads;
}

template <int KIND, bool NORM>
static cudaError_t launch_rows(const AppendParams& p, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (p.num_tokens >= many_tokens<NORM>(p, KIND) && launch_stream<KIND, NORM>(p, stream, &e)) return e;
  return launch_pdl(kv_append_kernel<KIND, 1, 2, false, NORM>, dim3(static_cast<unsigned>(p.num_tokens)), dim3(kThreads), 0,
                    stream, p);
}

template <bool NORM>
static cudaError_t launch_append(const AppendParams& in, int kind, cudaStream_t stream, int* launches) {
  AppendParams p = in;
  *launches = 1;
  if (kind == PKV_KV_FP8_E4M3) return launch_rows<PKV_KV_FP8_E4M3, NORM>(p, stream);
  if (kind == PKV_KV_BF16) return launch_rows<PKV_KV_BF16, NORM>(p, stream);
  // Tokens of a CTA that appends runs: 1, 4 or 16 of one long sequence (64 query and 8 KV heads, us) 1024
  // 11.1, 9.7, 9.1; 4096 49, 39, 37; of one token a sequence 256 8.1, 18.5, 62; 1024 26, 25, 85; 4096 112, 105, 120.
  p.run_tokens = p.num_tokens <= 1024 ? 1 : (p.num_tokens <= 4096 ? 4 : kBlockTokens);
  p.run_groups = static_cast<uint32_t>((p.num_tokens + p.run_tokens - 1) / p.run_tokens);
  if (p.Hq > 0 && p.num_tokens < many_tokens<NORM>(p, kind))
    return launch_pdl(kv_append_kernel<PKV_KV_FP8_E4M3_BLOCK, 1, 2, true, NORM>,
                      dim3(static_cast<unsigned>(p.run_groups + p.num_tokens)), dim3(kThreads), 0, stream, p);
  cudaError_t e = launch_pdl(kv_append_runs_kernel<NORM>, dim3(p.run_groups), dim3(kThreads), 0, stream, p);
  if (e != cudaSuccess || p.Hq == 0) return e;
  *launches = 2;
  return launch_rows<PKV_KV_FP8_E4M3_BLOCK, NORM>(p, stream);
}

cudaError_t launch_kv_append(const AppendParams& p, int kind, cudaStream_t stream, int* launches) {
  return p.q_norm != nullptr || p.k_norm != nullptr ? launch_append<true>(p, kind, stream, launches)
                                                    : launch_append<false>(p, kind, stream, launches);
}

}  // namespace pkv
