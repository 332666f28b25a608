// decode_scaled.cu — paged_decode_attn over an E4M3 cache with an fp32 scale for each 16-token block
// and KV head: one query token per sequence against its paged context (vLLM blog
// "rocm-attention-backend", "Processing details: decode path"; the cache is the block-scaled kind of
// its FP8 caches).
//
// For the G query heads of a KV head, context positions j (block b), E4M3 values k_j, v_j:
//   u_j = log2(e) scale ks_b (q . k_j) + log2 vs_b,    P_j = 2^(u_j - M),
//   O = sum_j P_j v_j,   l = sum_j P_j / vs_b,   out = O / l,   lse = (M + log2 l) ln 2.
// Taking M over u rather than over the scores folds the value scale into the exponent: the largest
// P of a tile is always the same number, whatever the scales, and v_j is multiplied as it is stored.
//
// Design: the codes go into the tensor cores as they are; nothing is converted but q and P.
//   * A tile is 128 tokens (8 blocks) of one KV head. S^T = K Q^T takes the K codes from shared memory
//     as the M = 128 operand (tcgen05 kind::f8f6f4, E4M3) and the query heads as N columns; O^T = V^T P^T
//     takes the V codes as they lie (M = 128 dims, M-major) and P as N columns.
//   * q and P are split into E4M3 parts, x = hi + lo / 16, which sit side by side on N: NG columns
//     of hi and NG of lo (NG = G padded to 8 or 16). E4M3 has 4 significant bits. A bf16 q (8
//     bits) is exactly hi + lo down to 2^-14 of its head's largest |q|, to 2^-21 of it below (each head
//     has a power of two of its own, so that heads of very different size keep the same bits). P's
//     error is at most 2^-9 of P, to 2^-14 of the tile's largest P, and at most 2^-22 of the largest
//     below: better than bf16's 2^-9 where it counts.
//     The products are exact in fp32.
//   * Every tile has an M of its own (its P spans E4M3's range whatever the rest of the sequence
//     holds) and an O of its own: the 128 threads that read S (thread t is token t) read O as dim
//     t and fold it into registers, o = o 2^(m - m') + O 2^(M - m'). No accumulator is rescaled in
//     tensor memory, and P V of one tile runs while the threads work on the next one's S.
//   * A CTA (one per SM, persistent) runs two such chains, each with its own ring of tiles: per chain
//     four softmax warps, one TMA producer and one MMA issuer. The work split is the other decode
//     kernels': the set's blocks in equal contiguous shares, chain w takes share w / Hkv of KV head
//     w % Hkv, so neighbouring chains stream the heads of the same blocks together.
//   * A sequence cut at share edges is merged by its log-sum-exps along a tree of fan-in 8: fp32
//     partials in the workspace, an arrival counter per tree node (tagged with the call's epoch, set
//     back to zero by the arrival that completes it, so a replayed graph finds none of its own).
//
// What bounds it: with 8 heads a KV head HBM (192 sequences of 1000 to 8000 tokens, Hq 64 / Hkv 8: 290 us, 6.1 TB/s,
// 0.90 of the measured copy); with 16 the softmax warps, 2450 clocks a tile against 1900 for its bytes (256 sequences of
// 2000 to 3000, Hq 64 / Hkv 4: 132 us, 0.74); one sequence of 100,000 tokens its ramp and merge (50 us, 0.61); four of
// at most 200 the set-up and the first tile (8.8 us on the GPU).
#include <math_constants.h>

#include "common.cuh"
#include "decode_shares.cuh"
#include "launch.h"
#include "tc.cuh"

namespace pkv {

namespace {

constexpr int kMaxKvHeads = 256;

template <int NG>
struct SdCfg {
  static constexpr int D = 128, BS = 16, TBLK = 8, BM = 128;
  static constexpr int NN = 2 * NG;                       // columns: hi parts, then lo parts
  static constexpr int HALF = BM * D;                     // K or V of a tile: 128 rows of 128 codes
  static constexpr int NB = 5;                            // ring: K and V tiles alternate
  static constexpr int Q_BYTES = NN * D;                  // [NN rows][128], 128-byte swizzle
  static constexpr int P_BYTES = NN * BM;                 // [NN / 16][128 tokens][16]
  static constexpr int SRING = 8;                         // tiles whose scales are kept
  static constexpr int Q_OFF = NB * HALF;
  static constexpr int P_OFF = Q_OFF + 2 * Q_BYTES;
  static constexpr int SC_OFF = P_OFF + 2 * P_BYTES;      // [SRING][8 ks, 8 vs]
  static constexpr int WMAX_OFF = SC_OFF + SRING * 64;    // [2][4 warps][NG] a warp's max of u
  static constexpr int FAC_OFF = WMAX_OFF + 2 * 4 * NG * 4;  // [4 warps][2][3: M, a, c][NG]
  static constexpr int LSUM_OFF = FAC_OFF + 4 * 2 * 3 * NG * 4;  // [2][4 warps][NG]
  static constexpr int INV_OFF = LSUM_OFF + 2 * 4 * NG * 4;  // [4 warps][NG]
  static constexpr int QINV_OFF = INV_OFF + 4 * NG * 4;   // [2][NG] softmax scale over a head's power of two
  static constexpr int BAR_OFF = QINV_OFF + 2 * NG * 4;
  static constexpr int NBAR = 2 * NB + 13;
  static constexpr int MISC_BYTES = (BAR_OFF + NBAR * 8 - SC_OFF + 127) / 128 * 128;
  static constexpr int CHAIN = (SC_OFF + MISC_BYTES + 1023) / 1024 * 1024;
  static constexpr int MAXR = kSetChunk;
  static constexpr int TAB_BYTES = (4 * MAXR + 4) * 4;
  static constexpr int SMEM = 1024 + 2 * CHAIN + TAB_BYTES;
  static constexpr int THREADS = 384;
  static constexpr int MIN_BLOCKS = TBLK;                 // a share holds at least a tile
  static constexpr uint32_t SCOL = 0, OCOL = 2 * NN, CHAIN_COLS = 4 * NN;  // TMEM: S and O, two buffers each
  static constexpr uint32_t TMEM_COLS = 2 * CHAIN_COLS < 32 ? 32 : 2 * CHAIN_COLS;
  static constexpr uint32_t IDESC_S = tc::idesc_e4m3(128, NN, 0, 0);
  static constexpr uint32_t IDESC_PV = tc::idesc_e4m3(128, NN, 1, 1);
  static_assert(SMEM <= 226 * 1024, "shared memory");
};

// A chain's barriers.
template <int NG>
struct SdBars {
  uint64_t kv_full[SdCfg<NG>::NB], kv_empty[SdCfg<NG>::NB];
  uint64_t s_full[2], s_empty[2], p_full[2], o_full[2], o_empty[2], q_full[2], drained;
};

// Bounded wait that also gives up as soon as another role has given up.
__device__ __forceinline__ bool sd_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
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
__device__ __forceinline__ bool sd_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  return __all_sync(0xffffffffu, sd_wait(bar, parity, abort_flag, err));
}
__device__ __forceinline__ void chain_sync(int chain) { asm volatile("bar.sync %0, 128;" ::"r"(chain + 1) : "memory"); }
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// The tiles of a share in order: its pieces (one per sequence it touches), each cut into tiles of
// up to 8 blocks. Every role of a chain walks the same sequence.
struct SdWalk {
  PieceIter it;
  Piece pc;
  int k, nt;
  bool have;
  __device__ void next_piece() {
    k = 0;
    have = it.next(pc);
    nt = have ? (pc.hi - pc.lo + 7) / 8 : 0;
  }
  __device__ void start(const int* pre, int n, int64_t b0, int64_t b1) {
    it.start(pre, n, 1, b0, b1);
    next_piece();
  }
  __device__ void advance() {
    if (++k == nt) next_piece();
  }
  __device__ int blk0() const { return pc.lo + 8 * k; }
  __device__ int nbl() const { return min(8, pc.hi - blk0()); }
};

// A small batch's pieces: a sequence of b blocks is one piece when b <= whole, else ceil(b / most) pieces
// of nearly equal length; share c takes the c-th of all of them. Not by_sequence when there are more pieces than shares. A whole warp
// computes it (n is at most a few hundred).
struct SdOwn {
  int64_t b0, b1;
  int piece, np;
  bool by_sequence;
};
__device__ __noinline__ SdOwn sd_own(const int* s_pre, int n, int c, int shares, int lane, int whole, int most) {
  SdOwn w{0, 0, 0, 0, false};
  int before = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int lo = i < n ? s_pre[i] : 0, b = i < n ? s_pre[i + 1] - lo : 0, m = b == 0 ? 0 : b <= whole ? 1 : (b + most - 1) / most;
    int x = m;  // pieces up to and with sequence i of this group
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int k = c - before - (x - m);  // share c's piece of sequence i, if it is one
    const uint32_t hit = __ballot_sync(0xffffffffu, k >= 0 && k < m);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int bs = __shfl_sync(0xffffffffu, b, src);
      w.piece = __shfl_sync(0xffffffffu, k, src);
      w.np = __shfl_sync(0xffffffffu, m, src);
      const int at = __shfl_sync(0xffffffffu, lo, src);
      w.b0 = at + static_cast<int64_t>(bs) * w.piece / w.np;
      w.b1 = at + static_cast<int64_t>(bs) * (w.piece + 1) / w.np;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  w.by_sequence = before <= shares;
  return w;
}

// ---- the merge tree of a cut sequence (fan-in 8; see decode_shares.cuh for the places) -----------
constexpr int kSdFanBits = 3, kSdFan = 1 << kSdFanBits;
struct SdCut {
  int c0, np, piece;  // first share, pieces, this chain's piece
  int64_t row;
  __device__ int nodes(int L) const { return (np + (1 << (kSdFanBits * L)) - 1) >> (kSdFanBits * L); }
  __device__ int children(int L, int a) const { return min(kSdFan, nodes(L - 1) - a * kSdFan); }
};
__device__ __forceinline__ float* sd_part(const DecodeParams& p, const SdCut& s, int L, int a, int kh, int g) {
  const int share = s.c0 + (a << (kSdFanBits * L)), slot = a == 0 ? 1 : 0;
  return p.ws_part + (((static_cast<int64_t>(share) * 2 + slot) * p.units + kh) * p.G + g) * (128 + 4);
}
__device__ __forceinline__ unsigned long long* sd_ctr(const DecodeParams& p, const SdCut& s, int L, int a, int kh) {
  const int share = s.c0 + (a << (kSdFanBits * L)), slot = a == 0 ? 1 : 0;
  return p.ws_ctr + ((static_cast<int64_t>(L - 1) * p.launch_shares + share) * 2 + slot) * p.units + kh;
}
__host__ __device__ constexpr int sd_levels(int shares) {
  int L = 1;
  while ((1ll << (kSdFanBits * L)) < shares) ++L;
  return L;
}

// Merge the k children of node (L, a) into out / lse (the root) or into the node's partial: warp w
// of the chain takes heads w, w + 4, .., two at a time; lane l dims 4l .. 4l + 3.
__device__ __forceinline__ void sd_merge(const DecodeParams& p, const SdCut& s, int L, int a, int k, bool root, int kh,
                                         int warp, int lane) {
  // weights: lane 8 j + m holds child m's of head w + 4 j
  const int m8 = lane & 7, hj = warp + 4 * (lane >> 3);
  const bool have = m8 < k && hj < p.G;
  const float l = have ? __ldcg(sd_part(p, s, L - 1, a * kSdFan + m8, kh, hj) + 128) : -CUDART_INF_F;
  for (int g0 = warp, j0 = 0; g0 < p.G; g0 += 8, j0 += 2) {
    float4 v[2][kSdFan];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int m = 0; m < kSdFan; ++m) {
        v[j][m] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (m < k && g0 + 4 * j < p.G)
          v[j][m] = __ldcg(reinterpret_cast<const float4*>(sd_part(p, s, L - 1, a * kSdFan + m, kh, g0 + 4 * j)) + lane);
      }
    float M = l;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float w = have ? __expf(l - M) : 0.f;
    float W = w;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
    const float wn = w / W, lse = M + __logf(W);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = g0 + 4 * j;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int m = 0; m < kSdFan; ++m) {
        const float wm = __shfl_sync(0xffffffffu, wn, 8 * (j0 + j) + m);
        acc.x = fmaf(wm, v[j][m].x, acc.x);
        acc.y = fmaf(wm, v[j][m].y, acc.y);
        acc.z = fmaf(wm, v[j][m].z, acc.z);
        acc.w = fmaf(wm, v[j][m].w, acc.w);
      }
      const float lg = __shfl_sync(0xffffffffu, lse, 8 * (j0 + j));
      if (g >= p.G) continue;
      if (root) {
        const int64_t at = s.row * p.Hq + kh * p.G + g;
        *reinterpret_cast<uint2*>(p.out + at * 128 + 4 * lane) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
        if (p.lse && lane == 0) p.lse[at] = lg;
      } else {
        // child 0 lies where the node goes: every lane has read it by now (the shuffles above)
        float* dst = sd_part(p, s, L, a, kh, g);
        __stcg(reinterpret_cast<float4*>(dst) + lane, acc);
        if (lane == 0) __stcg(dst + 128, lg);
      }
    }
  }
}

// 16 bits of x in E4M3 parts: hi = E4M3(x), lo = E4M3(16 (x - hi)). x in fp16, |x| <= 448.
__device__ __forceinline__ void split_e4m3(uint32_t x2, uint16_t& hi, uint16_t& lo) {
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(x2));
  const uint32_t back = e4m3x2_to_f16x2(hi);
  uint32_t r;
  asm("{\n\t.reg .b32 d, c;\n\tsub.rn.f16x2 d, %1, %2;\n\tmov.b32 c, 0x4C004C00;\n\tmul.rn.f16x2 %0, d, c;\n\t}"
      : "=r"(r)
      : "r"(x2), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(r));
}

template <int NG>
__global__ void __launch_bounds__(SdCfg<NG>::THREADS, 1)
    decode_scaled_kernel(const DecodeParams p, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v) {
  using C = SdCfg<NG>;
  constexpr int NN = C::NN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* s_pre = reinterpret_cast<int*>(smem + 2 * C::CHAIN);
  int* s_ctx = s_pre + C::MAXR + 1;
  int* s_r = s_ctx + C::MAXR;
  int* s_row = s_r + C::MAXR;
  __shared__ int s_scan[C::THREADS / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int2 s_own[2];  // a small batch's share: its piece of a sequence, and that one's pieces
  __shared__ int s_abort, s_quit[2][2], s_go[2][2];

  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // roles: warps 0-3 and 4-7 the softmax of chain 0 and 1, 8-9 their producers, 10-11 their MMA issuers
  const int chain = warp < 8 ? warp >> 2 : (warp & 1);
  uint8_t* base = smem + chain * C::CHAIN;
  SdBars<NG>& bar = *reinterpret_cast<SdBars<NG>*>(base + C::BAR_OFF);
  if (tid < 2) {
    if (tid == 0) s_abort = 0;
    s_quit[tid][0] = s_quit[tid][1] = 0;
    SdBars<NG>& b = *reinterpret_cast<SdBars<NG>*>(smem + tid * C::CHAIN + C::BAR_OFF);
    for (int i = 0; i < C::NB; ++i) {
      mbar_init(&b.kv_full[i], 1 + C::TBLK);  // the producer's bytes, and each block's scales
      mbar_init(&b.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.s_full[i], 1);
      mbar_init(&b.s_empty[i], 4);
      mbar_init(&b.p_full[i], 4);
      mbar_init(&b.o_full[i], 1);
      mbar_init(&b.o_empty[i], 4);
      mbar_init(&b.q_full[i], 4);
    }
    mbar_init(&b.drained, 1);
    fence_mbar_init();
  }
  if (warp == 10) tc::tmem_alloc(&s_tmem, C::TMEM_COLS);
  tc::fence_before_sync();
  int begin, n;
  resolve_set(p, begin, n);
  // (its block-wide barriers also order the set-up above before what follows)
  const int64_t TB = load_set<C::MAXR, C::BS>(p, begin, n, s_pre, s_ctx, s_r, s_row, s_scan);
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem + chain * C::CHAIN_COLS;

  // this chain's share [b0, b1) of the blocks and its KV head
  const int worker = blockIdx.x * 2 + chain, kh = worker % p.Hkv, c = worker / p.Hkv;
  const int nsh = active_shares(TB, p.launch_shares, C::MIN_BLOCKS);
  const Shares sh(TB, nsh);
  const bool busy = TB > 0 && c < nsh;
  int64_t b0 = busy ? sh.start(c) : 0, b1 = busy ? sh.start(c + 1) : 0;
  // A small batch (equal shares of at most four tiles, no more sequences than shares) is cut along its
  // sequences instead (sd_own): short ones are not cut at all, which costs a few more tiles (0.9 us each)
  // and saves the merge (about 4.5 us). 4 sequences of 16 to 200 tokens: 15.9 us in equal shares, 8.8 so.
  if (TB <= static_cast<int64_t>(4 * C::TBLK) * p.launch_shares && n <= p.launch_shares) {
    SdOwn own = sd_own(s_pre, n, c, p.launch_shares, lane, 5 * C::TBLK, 2 * C::TBLK);
    if (!own.by_sequence) own = sd_own(s_pre, n, c, p.launch_shares, lane, 8 * C::TBLK, 8 * C::TBLK);
    if (own.by_sequence) b0 = own.b0, b1 = own.b1;
    if ((warp & 3) == 0 && warp < 8 && lane == 0) s_own[chain] = own.by_sequence ? make_int2(own.piece, own.np) : make_int2(-1, 0);
  } else if ((warp & 3) == 0 && warp < 8 && lane == 0) {
    s_own[chain] = make_int2(-1, 0);
  }

  if (warp < 8) {
    // ======================= softmax: thread t is token t of S, dim t of O =======================
    const int t = tid & 127, w4 = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
    float* wmax = reinterpret_cast<float*>(base + C::WMAX_OFF);
    float* fac = reinterpret_cast<float*>(base + C::FAC_OFF) + w4 * (2 * 3 * NG);
    float* lsum = reinterpret_cast<float*>(base + C::LSUM_OFF);
    float* invs = reinterpret_cast<float*>(base + C::INV_OFF) + w4 * NG;
    float* qinv = reinterpret_cast<float*>(base + C::QINV_OFF);

    // ---- queries: each piece's tile is converted one piece ahead, its rows loaded two ahead ----
    constexpr int QP = 128 / NG;                  // threads per head
    constexpr int QE = 128 / QP;                  // dims per thread (16 or 8)
    const int qh = t / QP, qd = (t % QP) * QE;
    uint4 qraw[QE / 8];
    PieceIter qit;
    Piece qpc;
    bool qhave;
    uint32_t qn = 0;                              // pieces converted
    auto load_q = [&]() {
      qhave = qit.next(qpc);
      if (qhave && qh < p.G) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(s_row[qpc.i]) * p.Hq + kh * p.G + qh) * 128 + qd);
#pragma unroll
        for (int i = 0; i < QE / 8; ++i) qraw[i] = __ldg(src + i);
      } else {
#pragma unroll
        for (int i = 0; i < QE / 8; ++i) qraw[i] = make_uint4(0, 0, 0, 0);
      }
    };
    auto convert_q = [&]() {  // the loaded rows into tile qn % 2, then load the next piece's
      if (!qhave) return;
      float x[QE];
#pragma unroll
      for (int i = 0; i < QE / 8; ++i) {
        const uint32_t wv[4] = {qraw[i].x, qraw[i].y, qraw[i].z, qraw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * i + 2 * j] = __uint_as_float(wv[j] << 16);
          x[8 * i + 2 * j + 1] = __uint_as_float(wv[j] & 0xFFFF0000u);
        }
      }
      uint32_t top = 0;  // the head's largest finite |q|
#pragma unroll
      for (int i = 0; i < QE; ++i) {
        const uint32_t m = __float_as_uint(x[i]) & 0x7FFFFFFFu;
        top = max(top, m < 0x7F800000u ? m : 0u);
      }
#pragma unroll
      for (int bit = QP / 2; bit > 0; bit >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, bit));
      const uint32_t b = qn & 1;
      // 2^e |q| in [128, 256) for the largest
      const int e = min(max(134 - static_cast<int>(top >> 23), -126), 126);
      const float qs = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      // (read a barrier of the chain later: the first piece's after the one below, the next pieces' after the one of a
      // tile of the piece before)
      if (qd == 0) qinv[b * NG + qh] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      uint32_t hi[QE / 4], lo[QE / 4];
#pragma unroll
      for (int i = 0; i < QE; i += 4) {
        uint16_t h[2], l[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float a = x[i + 2 * j] * qs, z = x[i + 2 * j + 1] * qs;
          // hi + lo / 16 from fp32: the residual of hi is exact, and rounds only where it is below 2^-13
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[j]) : "f"(z), "f"(a));
          const uint32_t back = e4m3x2_to_f16x2(h[j]);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
          // an infinite q stays no number
          a = (a - f.x) * 16.f, z = (z - f.y) * 16.f;
          if (fabsf(a) == CUDART_INF_F) a = CUDART_NAN_F;
          if (fabsf(z) == CUDART_INF_F) z = CUDART_NAN_F;
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l[j]) : "f"(z), "f"(a));
        }
        hi[i / 4] = h[0] | (static_cast<uint32_t>(h[1]) << 16);
        lo[i / 4] = l[0] | (static_cast<uint32_t>(l[1]) << 16);
      }
      // rows qh (hi) and NG + qh (lo), 128 bytes each, 16-byte chunks swizzled by the row
      uint8_t* dst = base + C::Q_OFF + b * C::Q_BYTES;
      uint8_t* dh = dst + sw128(qh, qd / 16) + qd % 16;
      uint8_t* dl = dst + sw128(NG + qh, qd / 16) + qd % 16;
      if constexpr (QE == 16) {
        *reinterpret_cast<uint4*>(dh) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dl) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      } else {
        *reinterpret_cast<uint2*>(dh) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(dl) = make_uint2(lo[0], lo[1]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full[b]);
      ++qn;
      load_q();
    };
    qit.start(s_pre, n, 1, b0, b1);
    load_q();
    convert_q();
    chain_sync(chain);

    float o[NG], l[NG], pl[NG];  // the piece's sums; the last tile's P / vs of this token
    float m_run = -CUDART_INF_F, m_fin = 0.f;  // lane h: running max of head h; that of the piece before
#pragma unroll
    for (int h = 0; h < NG; ++h) o[h] = l[h] = 0.f;
    SdCut cuts[2];
    int ncut = 0;
    SdWalk wk;
    wk.start(s_pre, n, b0, b1);
    uint32_t gt = 0, pieces = 0;
    Piece prev = wk.pc;
    uint32_t done = 0;  // pieces finished
    bool bad = false;

    // fold tile g's O (and its P sums) into the registers
    auto fold = [&](uint32_t g) {
      bad |= !sd_wait_warp(&bar.o_full[g & 1], (g >> 1) & 1, &s_abort, p.err);
      tc::fence_after_sync();
      uint32_t v[NN];
      tc::ld_cols(tmem + lane_off + C::OCOL + (g & 1) * NN, v);
      tc::wait_ld();
      tc::touch_cols(v);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.o_empty[g & 1]);
      const float4* fa = reinterpret_cast<const float4*>(fac + (g & 1) * 3 * NG + NG);
      const float4* fc = fa + NG / 4;
#pragma unroll
      for (int q = 0; q < NG / 4; ++q) {
        const float4 a4 = fa[q], c4 = fc[q];
        const float a[4] = {a4.x, a4.y, a4.z, a4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = 4 * q + i;
          o[h] = fmaf(fmaf(__uint_as_float(v[NG + h]), 0.0625f, __uint_as_float(v[h])), cc[i], o[h] * a[i]);
          l[h] = fmaf(pl[h], cc[i], l[h] * a[i]);
        }
      }
    };
    // the piece `pc` is folded: write it out, or leave its partial in the workspace
    auto finish = [&](const Piece& pc) {
      // l over the chain's 128 tokens: halves exchanged until a lane group holds one head
      float r[NG];
#pragma unroll
      for (int h = 0; h < NG; ++h) r[h] = l[h];
#pragma unroll
      for (int cnt = NG / 2, bit = 16; cnt > 0; cnt >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < NG / 2; ++i)
          if (i < cnt) {
            const float send = up ? r[i] : r[i + cnt];
            r[i] = (up ? r[i + cnt] : r[i]) + __shfl_xor_sync(0xffffffffu, send, bit);
          }
      }
#pragma unroll
      for (int bit = 16 / NG; bit > 0; bit >>= 1) r[0] += __shfl_xor_sync(0xffffffffu, r[0], bit);
      // (two buffers: at the end of a share two pieces may finish with no other barrier of the chain in between, and
      // a warp may still read the first one's sums when another writes the second one's)
      constexpr int SH = NG == 16 ? 1 : 2;
      float* ls = lsum + (done++ & 1) * 4 * NG;
      if ((lane & ((1 << SH) - 1)) == 0) ls[w4 * NG + (lane >> SH)] = r[0];
      chain_sync(chain);
      float lse = 0.f;
      if (lane < NG) {
        const float L = ls[lane] + ls[NG + lane] + ls[2 * NG + lane] + ls[3 * NG + lane];
        invs[lane] = 1.f / L;
        lse = (m_fin + __log2f(L)) * 0.69314718055994531f;
      }
      __syncwarp();
      const int64_t row = s_row[pc.i];
      const bool whole = pc.lo == 0 && pc.hi == (s_ctx[pc.i] + C::BS - 1) / C::BS;
      if (whole) {
        __nv_bfloat16* dst = p.out + (row * p.Hq + kh * p.G) * 128 + t;
#pragma unroll
        for (int h = 0; h < NG; ++h)
          if (h < p.G) dst[h * 128] = __float2bfloat16_rn(o[h] * invs[h]);
        if (p.lse && w4 == 0 && lane < p.G) p.lse[row * p.Hq + kh * p.G + lane] = lse;
      } else {
        SdCut s;
        const int2 own = s_own[chain];  // (written before the chain's first barrier)
        s.c0 = own.x >= 0 ? c - own.x : sh.of(s_pre[pc.i]);
        s.np = own.x >= 0 ? own.y : sh.of(s_pre[pc.i + 1] - 1) - s.c0 + 1;
        s.piece = c - s.c0;
        s.row = row;
        float* dst = sd_part(p, s, 0, s.piece, kh, 0);
#pragma unroll
        for (int h = 0; h < NG; ++h)
          if (h < p.G) __stcg(dst + h * 132 + t, o[h] * invs[h]);
        if (w4 == 0 && lane < p.G) __stcg(dst + lane * 132 + 128, lse);
        if (ncut == 0) cuts[0] = s; else cuts[1] = s;
        ++ncut;
      }
#pragma unroll
      for (int h = 0; h < NG; ++h) o[h] = l[h] = 0.f;
    };

    bool quit = false;
    while (wk.have && !quit) {
      const bool first = wk.k == 0;
      if (first) {
        convert_q();  // the next piece's queries
        m_fin = m_run;
        m_run = -CUDART_INF_F;
        ++pieces;
      }
      // ---- S of tile gt ----
      const int ctx = s_ctx[wk.pc.i];
      const int ntok = min(ctx - wk.blk0() * C::BS, wk.nbl() * C::BS);  // the tile's tokens
      const uint32_t buf = gt & 1;
      bad |= !sd_wait_warp(&bar.s_full[buf], (gt >> 1) & 1, &s_abort, p.err);
      tc::fence_after_sync();
      float u[NG];
      {
        uint32_t v[NN];
        tc::ld_cols(tmem + lane_off + C::SCOL + buf * NN, v);
        tc::wait_ld();
        tc::touch_cols(v);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.s_empty[buf]);
        const float* sc = reinterpret_cast<const float*>(base + C::SC_OFF) + gt % C::SRING * 16;
        // a zero scale counts as 2^-100: no logarithm of 0
        const float4* qi4 = reinterpret_cast<const float4*>(qinv + ((pieces & 1) ? 0 : NG));
        const float ks = fmaxf(sc[t >> 4], 0x1p-100f), vs = fmaxf(sc[8 + (t >> 4)], 0x1p-100f);
        const float lvs = __log2f(vs), ivs = 1.f / vs;
        const bool valid = t < ntok;
#pragma unroll
        for (int q = 0; q < NG / 4; ++q) {
          const float4 f4 = qi4[q];
          const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int h = 4 * q + i;
            const float x = fmaf(__uint_as_float(v[NG + h]), 0.0625f, __uint_as_float(v[h]));
            u[h] = valid ? fmaf(x, ks * f[i], lvs) : -CUDART_INF_F;
          }
        }
        float mw[NG];
#pragma unroll
        for (int h = 0; h < NG; ++h) mw[h] = warp_max(u[h]);
        float4* dst = reinterpret_cast<float4*>(wmax + (buf * 4 + w4) * NG);
        if (lane == 0) {
#pragma unroll
          for (int q = 0; q < NG / 4; ++q) dst[q] = make_float4(mw[4 * q], mw[4 * q + 1], mw[4 * q + 2], mw[4 * q + 3]);
          if (bad) s_quit[chain][buf] = 1;
        }
        chain_sync(chain);
        quit = *const_cast<volatile int*>(&s_quit[chain][buf]) != 0;
        float* fw = fac + buf * 3 * NG;
        if (lane < NG) {
          const float* wm = wmax + buf * 4 * NG + lane;
          // P spans [0, 256]: the tile's frame lies 8 binades under its max
          const float M = fmaxf(fmaxf(wm[0], wm[NG]), fmaxf(wm[2 * NG], wm[3 * NG])) - 8.f;
          const float m_new = fmaxf(m_run, M);
          fw[lane] = M;
          fw[NG + lane] = ex2_approx(m_run - m_new);
          fw[2 * NG + lane] = ex2_approx(M - m_new);
          m_run = m_new;
        }
        __syncwarp();
        // ---- P ----
        uint32_t hi[NG / 4], lo[NG / 4];
        float pn[NG];
#pragma unroll
        for (int q = 0; q < NG / 4; ++q) {
          const float4 m4 = reinterpret_cast<const float4*>(fw)[q];
          const float p0 = ex2_approx(u[4 * q] - m4.x), p1 = ex2_approx(u[4 * q + 1] - m4.y);
          const float p2 = ex2_approx(u[4 * q + 2] - m4.z), p3 = ex2_approx(u[4 * q + 3] - m4.w);
          uint16_t h0, h1, l0, l1;
          split_e4m3(pack_f16(p0, p1), h0, l0);
          split_e4m3(pack_f16(p2, p3), h1, l1);
          hi[q] = h0 | (static_cast<uint32_t>(h1) << 16);
          lo[q] = l0 | (static_cast<uint32_t>(l1) << 16);
          pn[4 * q] = p0 * ivs, pn[4 * q + 1] = p1 * ivs, pn[4 * q + 2] = p2 * ivs, pn[4 * q + 3] = p3 * ivs;
        }
        uint8_t* pd = base + C::P_OFF + buf * C::P_BYTES + t * 16;
        if constexpr (NG == 16) {
          *reinterpret_cast<uint4*>(pd) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(pd + 2048) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
          *reinterpret_cast<uint4*>(pd) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
        }
        if (ntok < 128) {
          // V rows past the tile's tokens become zeros: P = 0 there must not meet a NaN code
          const uint32_t hv = 2 * gt + 1;
          bad |= !sd_wait_warp(&bar.kv_full[hv % C::NB], (hv / C::NB) & 1, &s_abort, p.err);
          if (!valid) {
            uint4* vr = reinterpret_cast<uint4*>(base + hv % C::NB * C::HALF + t * 128);
#pragma unroll
            for (int i = 0; i < 8; ++i) vr[i] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[buf]);
        // ---- O of the tile before, while P V of this one runs ----
        if (gt > 0) {
          fold(gt - 1);
          if (first) finish(prev);
        }
#pragma unroll
        for (int h = 0; h < NG; ++h) pl[h] = pn[h];
      }
      prev = wk.pc;
      ++gt;
      wk.advance();
    }
    if (gt > 0 && !quit) {
      fold(gt - 1);
      m_fin = m_run;
      finish(prev);
      // ---- cut pieces enter their trees: the arrivals of both (one thread each), then the merges ----
      if (ncut > 0) {
        SdCut my = cuts[0];
        int L0[2], a0[2];  // the first node with more than one child
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && ncut > 1) my = cuts[1];
          L0[i] = 1, a0[i] = my.piece / kSdFan;
          while (my.children(L0[i], a0[i]) == 1) {
            a0[i] /= kSdFan;
            ++L0[i];
          }
        }
        // the arrival on node (L, a); the one that completes it sets the counter back, so that a replay
        // of this launch starts from no arrivals
        auto arrive = [&](const SdCut& s, int L, int a, unsigned long long cur) {
          unsigned long long* ctr = sd_ctr(p, s, L, a, kh);
          const int k = s.children(L, a);
          const bool all = arrive_counter(ctr, p.epoch, k, cur, p.err) == k;
          if (all) atomicExch(ctr, 0ull);
          return all;
        };
        const bool mine = w4 < ncut && lane == 0;
        const SdCut sm = w4 == 0 ? cuts[0] : cuts[1];
        unsigned long long cur = 0;
        if (mine) cur = *const_cast<volatile unsigned long long*>(sd_ctr(p, sm, w4 == 0 ? L0[0] : L0[1], w4 == 0 ? a0[0] : a0[1], kh));
        __threadfence();
        chain_sync(chain);
        if (mine) s_go[chain][w4] = arrive(sm, w4 == 0 ? L0[0] : L0[1], w4 == 0 ? a0[0] : a0[1], cur);
        chain_sync(chain);
        const bool go[2] = {*const_cast<volatile int*>(&s_go[chain][0]) != 0,
                            ncut > 1 && *const_cast<volatile int*>(&s_go[chain][1]) != 0};
        if (go[0] || go[1]) __threadfence();
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          if (!(i == 0 ? go[0] : go[1])) continue;
          const SdCut s = i == 0 ? cuts[0] : cuts[1];
          int L = i == 0 ? L0[0] : L0[1], a = i == 0 ? a0[0] : a0[1];
          for (;;) {
            const bool root = s.nodes(L) == 1;
            sd_merge(p, s, L, a, s.children(L, a), root, kh, w4, lane);
            if (root) break;
            do {
              a /= kSdFan;
              ++L;
            } while (s.children(L, a) == 1 && s.nodes(L) > 1);
            __threadfence();
            chain_sync(chain);
            if (t == 0) s_go[chain][0] = arrive(s, L, a, 0ull);
            chain_sync(chain);
            if (!*const_cast<volatile int*>(&s_go[chain][0])) break;
            __threadfence();
          }
        }
      }
    }
  } else if (warp < 10) {
    // ======================= TMA producer =======================
    SdWalk wk;
    wk.start(s_pre, n, b0, b1);
    auto entry = [&](const SdWalk& w) {
      return w.have && lane < w.nbl()
                 ? p.block_tables[static_cast<int64_t>(s_r[w.pc.i]) * p.max_blocks + w.blk0() + lane]
                 : 0;
    };
    int next = entry(wk);
    uint32_t h = 0;  // tiles of K or V requested
    bool ok = true;
    while (wk.have && ok) {
      const int nbl = wk.nbl();
      int blk = next;
      if (lane < nbl && (blk < 0 || blk >= p.num_blocks)) {
        flag_error(p.err, PKV_DEVERR_BLOCK);
        blk = 0;
      }
      wk.advance();
      next = entry(wk);
      int blks[C::TBLK];
#pragma unroll
      for (int i = 0; i < C::TBLK; ++i) blks[i] = __shfl_sync(0xffffffffu, blk, i);
#pragma unroll 1
      for (int sel = 0; sel < 2; ++sel, ++h) {
        const uint32_t b = h % C::NB;
        if (h >= C::NB && !sd_wait_warp(&bar.kv_empty[b], (h / C::NB - 1) & 1, &s_abort, p.err)) {
          ok = false;
          break;
        }
        if (lane < C::TBLK) {
          if (lane < nbl) {
            if (sel == 0) {  // both scales come with K
              float* sc = reinterpret_cast<float*>(base + C::SC_OFF) + (h / 2) % C::SRING * 16 + lane;
              const int64_t at = static_cast<int64_t>(blk) * p.Hkv + kh;
              cp_async4(sc, p.k_scales + at);
              cp_async4(sc + 8, p.v_scales + at);
              cp_async_arrive_noinc(&bar.kv_full[b]);
            } else {
              mbar_arrive(&bar.kv_full[b]);
            }
          } else {
            mbar_arrive(&bar.kv_full[b]);
          }
        }
        __syncwarp();
        // one elected thread for all the copies (a lane each: 137 us against 132 on 256 sequences of 2000 to 3000
        // tokens, 297 against 290 on 192 of 1000 to 8000)
        if (tc::elect()) {
          mbar_arrive_expect_tx(&bar.kv_full[b], nbl * 2048);
#pragma unroll
          for (int i = 0; i < C::TBLK; ++i)
            if (i < nbl) tma_load_4d(base + b * C::HALF + i * 2048, sel ? &tm_v : &tm_k, &bar.kv_full[b], 0, kh, 0, blks[i]);
        }
        __syncwarp();
      }
    }
    if (!ok) {  // a role gave up: wait (bounded) for the copies still in flight
      for (uint32_t i = h > C::NB ? h - C::NB : 0; i < h; ++i)
        __all_sync(0xffffffffu, mbar_wait(&bar.kv_full[i % C::NB], (i / C::NB) & 1, p.err));
      cp_async_wait_all();
    }
  } else {
    // ======================= MMA issuer =======================
    // One thread issues S of the next tile as soon as its K and an S buffer are there, and P V of a
    // tile as soon as P, V and an O buffer are: whichever is ready first.
    if (lane == 0) {
      SdWalk wk;
      wk.start(s_pre, n, b0, b1);
      uint32_t ts = 0, tp = 0, pieces = 0;  // tiles whose S, whose P V was issued; pieces begun
      const uint32_t ring = smem_u32(base), qb = smem_u32(base + C::Q_OFF), pb = smem_u32(base + C::P_OFF);
      uint64_t t0 = 0;
      bool gave_up = false;
      for (uint32_t idle = 0; wk.have || tp < ts;) {
        bool did = false;
        // S of tile ts at most one tile ahead of P V: K of tile ts lies where V of tile ts - 3 (NB = 5)
        // lay, and a barrier's parity tells its phase only once the phase before was waited for
        static_assert(C::NB >= 5, "K of tile t must not follow V of tile t - 2 or a later one in its buffer");
        if (wk.have && ts < tp + 2) {
          const uint32_t hk = 2 * ts, kb = hk % C::NB, sb = ts & 1, pi = pieces - (wk.k > 0);
          if (mbar_test(&bar.kv_full[kb], (hk / C::NB) & 1) && (ts < 2 || mbar_test(&bar.s_empty[sb], ((ts >> 1) - 1) & 1)) &&
              (wk.k > 0 || mbar_test(&bar.q_full[pi & 1], (pi >> 1) & 1))) {
            tc::fence_after_sync();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_ss_f8(tmem + C::SCOL + sb * NN, tc::smem_desc(ring + kb * C::HALF + k * 32, 16, 1024),
                            tc::smem_desc(qb + (pi & 1) * C::Q_BYTES + k * 32, 16, 1024), C::IDESC_S, k > 0);
            tc::commit(&bar.s_full[sb]);
            tc::commit(&bar.kv_empty[kb]);
            if (wk.k == 0) ++pieces;
            ++ts;
            wk.advance();
            did = true;
          }
        }
        if (tp < ts) {
          const uint32_t hv = 2 * tp + 1, vb = hv % C::NB, ob = tp & 1;
          if (mbar_test(&bar.p_full[ob], (tp >> 1) & 1) && mbar_test(&bar.kv_full[vb], (hv / C::NB) & 1) &&
              (tp < 2 || mbar_test(&bar.o_empty[ob], ((tp >> 1) - 1) & 1))) {
            tc::fence_after_sync();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              // V: dims along M (one 128-byte row a token), 8-token groups 1024 bytes apart; P: 16
              // columns a token, 8-token groups 128 bytes apart, the lo parts 2048 bytes on
              tc::mma_ss_f8(tmem + C::OCOL + ob * NN, tc::smem_desc(ring + vb * C::HALF + k * 4096, 1024, 1024),
                            tc::smem_desc_plain(pb + ob * C::P_BYTES + k * 512, 128, 2048), C::IDESC_PV, k > 0);
            tc::commit(&bar.o_full[ob]);
            tc::commit(&bar.kv_empty[vb]);
            ++tp;
            did = true;
          }
        }
        if (did) {
          idle = 0;
          continue;
        }
        if ((++idle & 255u) == 0) {
          if (*const_cast<volatile int*>(&s_abort)) gave_up = true;
          if (idle == 256) t0 = globaltimer_ns();
          if (globaltimer_ns() - t0 > kWaitLimitNs) {
            flag_error(p.err, PKV_DEVERR_TIMEOUT);
            *const_cast<volatile int*>(&s_abort) = 1;
            gave_up = true;
          }
          if (gave_up) {  // wait (bounded) for the products in flight before the tensor memory goes
            tc::commit(&bar.drained);
            mbar_wait(&bar.drained, 0, p.err);
            break;
          }
        }
      }
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 10) {
    tc::fence_after_sync();
    tc::tmem_dealloc(s_tmem, C::TMEM_COLS);
  }
}

}  // namespace

// Chains of a launch over its KV heads: two per SM.
static int sd_shares(int Hkv) { return num_sms() * 2 / Hkv; }

bool decode_scaled_supported(int Hkv) { return Hkv <= kMaxKvHeads && sd_shares(Hkv) >= 1; }
size_t decode_scaled_ctr_offset(int Hq, int Hkv) {
  return static_cast<size_t>(sd_shares(Hkv)) * 2 * Hq * 132 * sizeof(float);
}
size_t decode_scaled_workspace_bytes(int Hq, int Hkv) {
  const int shares = sd_shares(Hkv);
  return decode_scaled_ctr_offset(Hq, Hkv) + static_cast<size_t>(sd_levels(shares)) * shares * 2 * Hkv * 8;
}

template <int NG>
static cudaError_t launch_sd(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  using C = SdCfg<NG>;
  cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(&decode_scaled_kernel<NG>), C::SMEM,
                                     NG == 16 ? kAttrDecodeScaled16 : kAttrDecodeScaled8);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_scaled_kernel<NG>, dim3(num_sms()), dim3(C::THREADS), C::SMEM, stream, p, tk, tv);
}

cudaError_t launch_decode_scaled(const DecodeParams& in, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream,
                                 int* launches) {
  DecodeParams p = in;
  p.launch_shares = sd_shares(p.Hkv);
  *launches += 1;
  return p.G > 8 ? launch_sd<16>(p, tk, tv, stream) : launch_sd<8>(p, tk, tv, stream);
}

}  // namespace pkv
