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
#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kBlockTokens = 16;  // block size of a block-scaled cache

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

// One CTA per token: its query rows and, unless the cache is block-scaled, its key and value rows.
template <int KIND>
__device__ __forceinline__ void append_rows(const AppendParams& p, int64_t t) {
  const int items = p.D / 16;
  const int i = threadIdx.x % items, h0 = threadIdx.x / items, hstep = blockDim.x / items;
  if (h0 >= hstep) return;  // the threads left over when items does not divide the CTA
  const int64_t slot = p.slots[t];
  const int64_t pos = p.rot > 0 ? p.positions[t] : 0;
  if (!token_ok(p, slot, pos, threadIdx.x == 0)) return;
  const Item it = item_of(p, i);
  Angles g;
  if (it.turn) load_angles(p, pos, i, g);
  // q heads, then k heads, then v heads
  const int rows = p.Hq + (KIND == PKV_KV_FP8_E4M3_BLOCK ? 0 : p.Hkv * (p.v != nullptr ? 2 : 1));
  const int64_t cache_off = (slot / p.block_size) * p.stride_block + (slot % p.block_size) * p.Hkv * p.D;
  constexpr int U = 4;
  for (int r0 = h0; r0 < rows; r0 += U * hstep) {
    uint4 va[U], vb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * hstep;
      if (r >= rows) continue;
      const __nv_bfloat16* src = r < p.Hq           ? p.q + t * p.q_stride + r * p.D
                                 : r < p.Hq + p.Hkv ? p.k + t * p.k_stride + (r - p.Hq) * p.D
                                                    : p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * p.D;
      va[u] = *reinterpret_cast<const uint4*>(src + it.a);
      vb[u] = *reinterpret_cast<const uint4*>(src + it.b);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * hstep;
      if (r >= rows) continue;
      const bool is_v = r >= p.Hq + p.Hkv;
      float x[16];
      unpack8(va[u], x);
      unpack8(vb[u], x + 8);
      if (it.turn && !is_v) {
        if (p.interleaved) turn(x, g, true); else turn(x, g, false);
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
      const int64_t off = cache_off + h * p.D;
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

// One warp: a run of rows (tokens t + j at block rows a + j, for the bits j of `mask`) of one head
// of K or V of a block-scaled cache (head_dim 128: 8 items a row, 4 rows a pass).
__device__ __forceinline__ void append_run(const AppendParams& p, int64_t t, uint32_t mask, int64_t slot, int h,
                                           bool is_v, int lane) {
  constexpr int DH = 128, PASSES = kBlockTokens / 4;
  const int i = lane & 7, rr = lane >> 3;
  const int64_t blk = slot / kBlockTokens;
  const int a = static_cast<int>(slot % kBlockTokens);
  float* sc = (is_v ? p.v_scales : p.k_scales) + blk * p.Hkv + h;
  const float s0 = a > 0 ? *sc : 0.f;
  const Item it = item_of(p, i);
  const __nv_bfloat16* src = is_v ? p.v + t * p.v_stride + h * DH : p.k + t * p.k_stride + h * DH;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  float x[PASSES][16];
  uint4 va[PASSES], vb[PASSES];
#pragma unroll
  for (int w = 0; w < PASSES; ++w) {
    const int j = 4 * w + rr;
    va[w] = vb[w] = make_uint4(0, 0, 0, 0);
    if ((mask >> j) & 1u) {
      va[w] = *reinterpret_cast<const uint4*>(src + j * stride + it.a);
      vb[w] = *reinterpret_cast<const uint4*>(src + j * stride + it.b);
    }
  }
  uint32_t top = 0;  // the largest finite magnitude, as bits
#pragma unroll
  for (int w = 0; w < PASSES; ++w) {
    unpack8(va[w], x[w]);
    unpack8(vb[w], x[w] + 8);
    const int j = 4 * w + rr;
    if (it.turn && !is_v && ((mask >> j) & 1u)) {
      Angles g;
      load_angles(p, p.positions[t + j], i, g);
      if (p.interleaved) turn(x[w], g, true); else turn(x[w], g, false);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t m = __float_as_uint(x[w][e]) & 0x7FFFFFFFu;
      top = max(top, m < 0x7F800000u ? m : 0u);
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
    if (!((mask >> j) & 1u)) continue;
    uint8_t* dst = blk_codes + static_cast<int64_t>(a + j) * p.Hkv * DH;
    *reinterpret_cast<uint2*>(dst + it.a) = codes8(x[w], inv);
    *reinterpret_cast<uint2*>(dst + it.b) = codes8(x[w] + 8, inv);
    if (!is_v && p.k_out != nullptr) {
      __nv_bfloat16* ko = p.k_out + ((t + j) * p.Hkv + h) * DH;
      *reinterpret_cast<uint4*>(ko + it.a) = pack8(x[w]);
      *reinterpret_cast<uint4*>(ko + it.b) = pack8(x[w] + 8);
    }
  }
}

// One CTA: the runs that begin in its group of tokens. A run begins at a token with a slot whose
// predecessor is not the row before it in the same block.
__device__ __forceinline__ void append_runs(const AppendParams& p, int64_t group) {
  __shared__ int s_lead[kBlockTokens];
  __shared__ int s_count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int64_t t0 = group * p.run_tokens;
  if (warp == 0) {
    const int64_t t = t0 + lane;
    bool lead = false;
    if (lane < p.run_tokens && t < p.num_tokens) {
      const int64_t s = p.slots[t];
      const int64_t before = t > 0 ? p.slots[t - 1] : -1;
      lead = s >= 0 && (s % kBlockTokens == 0 || before != s - 1);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, lead);
    if (lead) s_lead[__popc(m & ((1u << lane) - 1u))] = lane;
    if (lane == 0) s_count = __popc(m);
  }
  __syncthreads();
  const int per = 2 * p.Hkv;  // K and V of each head
  for (int u = warp; u < s_count * per; u += nw) {
    const int64_t t = t0 + s_lead[u / per];
    const int h = (u % per) >> 1;
    const bool is_v = u & 1;
    const int64_t slot = p.slots[t];
    const int a = static_cast<int>(slot % kBlockTokens);
    // the run: tokens t + j at slots slot + j to the end of the block
    bool in = false, ok = false;
    if (lane < kBlockTokens - a && t + lane < p.num_tokens) {
      in = p.slots[t + lane] == slot + lane;
      ok = in && token_ok(p, slot, p.rot > 0 ? p.positions[t + lane] : 0, u % per == 0);
    }
    const int n = __ffs(~__ballot_sync(0xffffffffu, in)) - 1;  // at most 16: the other lanes are never in
    const uint32_t mask = __ballot_sync(0xffffffffu, ok) & ((1u << n) - 1u);
    if (mask == 0) continue;
    append_run(p, t, mask, slot, h, is_v, lane);
  }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendParams p) {
  pdl_wait();
  pdl_release();
  if constexpr (KIND == PKV_KV_FP8_E4M3_BLOCK) {
    if (blockIdx.x < p.run_groups) {
      append_runs(p, blockIdx.x);
      return;
    }
    append_rows<KIND>(p, static_cast<int64_t>(blockIdx.x) - p.run_groups);
  } else {
    append_rows<KIND>(p, blockIdx.x);
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& in, int kind, cudaStream_t stream) {
  AppendParams p = in;
  const dim3 block(kThreads);
  if (kind == PKV_KV_FP8_E4M3_BLOCK) {
    p.run_tokens = p.num_tokens <= 1024 ? 1 : (p.num_tokens <= 4096 ? 4 : kBlockTokens);
    p.run_groups = static_cast<uint32_t>((p.num_tokens + p.run_tokens - 1) / p.run_tokens);
    const int64_t grid = p.run_groups + (p.Hq > 0 ? p.num_tokens : 0);
    return launch_pdl(kv_append_kernel<PKV_KV_FP8_E4M3_BLOCK>, dim3(static_cast<unsigned>(grid)), block, 0, stream, p);
  }
  const dim3 grid(static_cast<unsigned>(p.num_tokens));
  if (kind == PKV_KV_FP8_E4M3) return launch_pdl(kv_append_kernel<PKV_KV_FP8_E4M3>, grid, block, 0, stream, p);
  return launch_pdl(kv_append_kernel<PKV_KV_BF16>, grid, block, 0, stream, p);
}

}  // namespace pkv
