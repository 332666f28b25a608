// decode_scaled.cu — paged_decode_attn over an E4M3 cache with an fp32 scale for each block and
// KV head: one query token per sequence against its paged context.
//
// With scores s_j = scale * ks_b (q . k_j) (b the block of position j, k_j its E4M3 values) and
// running maximum m:  l = sum_j e^(s_j - m),  o = sum_j e^(s_j - m) vs_b v_j,  out = o / l,
// lse = m + ln l. One CTA per (request, KV head) walks the context in tiles of 128 tokens: thread t
// takes token t of the tile for the scores of the group's G query heads, then output dim t for
// the sums.
#include <math_constants.h>

#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kD = 128, kTile = 128, kMaxG = 16, kBS = 16;

__device__ __forceinline__ float2 e4m3x2(uint32_t w) {
  const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__global__ void __launch_bounds__(kTile) decode_scaled_kernel(ScaledDecodeParams p) {
  __shared__ float s_q[kMaxG][kD];
  __shared__ float s_p[kMaxG][kTile];
  __shared__ float s_vs[kTile];
  __shared__ int s_blk[kTile / kBS];
  pdl_wait();
  pdl_release();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int kh = blockIdx.y;
  int begin = 0, n = p.max_reqs;
  if (p.bounds != nullptr) {
    begin = p.bounds[p.cls];
    n = p.bounds[p.cls + 1] - begin;
    if (n > p.max_reqs) {
      if (blockIdx.x == 0 && kh == 0 && t == 0) flag_error(p.err, PKV_DEVERR_REQS);
      n = p.max_reqs;
    }
  }
  if (static_cast<int>(blockIdx.x) >= n) return;
  const int r = p.order ? p.order[begin + blockIdx.x] : begin + static_cast<int>(blockIdx.x);
  if (r < 0 || r >= p.batch_reqs) {
    if (t == 0 && kh == 0) flag_error(p.err, PKV_DEVERR_REQS);
    return;
  }
  const int64_t row = p.cu_q ? p.cu_q[r] : r;
  const int cap = min(static_cast<int64_t>(p.max_seq_len), static_cast<int64_t>(p.max_blocks) * kBS);
  int ctx = p.seq_lens[r];
  if (ctx > cap) {
    if (t == 0 && kh == 0) flag_error(p.err, PKV_DEVERR_LEN);
    ctx = cap;
  }
  const int G = p.G;
  for (int g = 0; g < G; ++g) s_q[g][t] = __bfloat162float(p.q[(row * p.Hq + kh * G + g) * kD + t]);
  float m[kMaxG], l[kMaxG], o[kMaxG];
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    m[g] = -CUDART_INF_F;
    l[g] = o[g] = 0.f;
  }
  for (int t0 = 0; t0 < ctx; t0 += kTile) {
    const int valid = min(kTile, ctx - t0);
    __syncthreads();
    if (t < (valid + kBS - 1) / kBS) {
      int b = p.block_tables[static_cast<int64_t>(r) * p.max_blocks + t0 / kBS + t];
      if (b < 0 || b >= p.num_blocks) {
        flag_error(p.err, PKV_DEVERR_BLOCK);
        b = 0;
      }
      s_blk[t] = b;
    }
    __syncthreads();
    float s[kMaxG];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) s[g] = 0.f;
    if (t < valid) {
      const int64_t b = s_blk[t / kBS];
      const uint4* k = reinterpret_cast<const uint4*>(p.k + b * p.stride_block + ((t % kBS) * static_cast<int64_t>(p.Hkv) + kh) * kD);
      for (int c = 0; c < kD / 16; ++c) {
        const uint4 v = k[c];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int e = 0; e < 8; ++e) {
          const float2 f = e4m3x2(w[e >> 1] >> (16 * (e & 1)));
#pragma unroll
          for (int g = 0; g < kMaxG; ++g)
            if (g < G) s[g] = fmaf(s_q[g][16 * c + 2 * e + 1], f.y, fmaf(s_q[g][16 * c + 2 * e], f.x, s[g]));
        }
      }
      const float f = p.k_scales[b * p.Hkv + kh] * p.scale_log2;
      s_vs[t] = p.v_scales[b * p.Hkv + kh];
#pragma unroll
      for (int g = 0; g < kMaxG; ++g) s_p[g][t] = s[g] * f;
    } else {
#pragma unroll
      for (int g = 0; g < kMaxG; ++g) s_p[g][t] = -CUDART_INF_F;
    }
    __syncthreads();
    float a[kMaxG];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      if (g >= G) continue;
      float mx = m[g];
      for (int j = 0; j < kTile; j += 32) mx = fmaxf(mx, s_p[g][j + lane]);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      a[g] = exp2f(m[g] - mx);
      m[g] = mx;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < kMaxG; ++g)
      if (g < G) s_p[g][t] = exp2f(s_p[g][t] - m[g]);
    __syncthreads();
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      if (g >= G) continue;
      l[g] *= a[g];
      o[g] *= a[g];
    }
    for (int j = 0; j < valid; ++j) {
      const int64_t b = s_blk[j / kBS];
      const uint32_t c = p.v[b * p.stride_block + ((j % kBS) * static_cast<int64_t>(p.Hkv) + kh) * kD + t];
      const float v = e4m3x2(c).x * s_vs[j];
#pragma unroll
      for (int g = 0; g < kMaxG; ++g) {
        if (g >= G) continue;
        l[g] += s_p[g][j];
        o[g] = fmaf(s_p[g][j], v, o[g]);
      }
    }
  }
  (void)warp;
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    if (g >= G) continue;
    const int64_t at = row * p.Hq + kh * G + g;
    p.out[at * kD + t] = __float2bfloat16_rn(ctx > 0 ? o[g] / l[g] : 0.f);
    if (t == 0 && p.lse) p.lse[at] = ctx > 0 ? (m[g] + log2f(l[g])) * 0.69314718055994531f : -CUDART_INF_F;
  }
}

}  // namespace

cudaError_t launch_decode_scaled(const ScaledDecodeParams& p, cudaStream_t stream, int* launches) {
  *launches += 1;
  return launch_pdl(decode_scaled_kernel, dim3(p.max_reqs, p.Hkv), dim3(kTile), 0, stream, p);
}

}  // namespace pkv
