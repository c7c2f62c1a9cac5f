// Selection of cache blocks by a bound on their scores: for query head h and
// block c of KV head g with per-dim bounds lo, hi of the block's keys,
//   q . k <= sum_d max(q_d lo_d, q_d hi_d)   for every key k of the block,
// and a block's score is the largest bound over the group's query heads. The
// first n_first and last n_last blocks of a request are always kept; the
// library's top-k takes the best others, ties to the lower block.
//
// The sums are held in fp64, where a product of two bf16 values is exact and
// the sum is wrong by 2^-46 of its terms at most, and rounded once to fp32: which blocks are
// selected does not depend on the order of the sum. max(q lo, q hi) = max(q, 0) hi +
// min(q, 0) lo, two fused multiply-adds without a select. A bf16 value becomes
// a double by moving its bits: (x >> 3) with the sign kept, as the high word, is
// x * 2^-896 for every finite x, subnormals and zero included; q carries 2^800 and the
// result 2^96 to make up for it.
//
// Split: one warp per 32 blocks of a (request, KV head), a block per lane, so
// that q is uniform over the warp and the sums need no shuffle; the blocks'
// bounds are staged in shared memory with cp.async. Bound by HBM (4 D bytes
// per block and KV head) up to four query heads per KV head, and by the fp64
// pipe above.
#pragma once

#include "kv_store.cuh"
#include "sd_common.cuh"

namespace sd {

constexpr int kBtWarps = 4;
constexpr int kBtThreads = 32 * kBtWarps;
constexpr int kBtBlocks = 32;  // blocks per warp
constexpr int kBtHeads = 4;    // query heads summed at once

struct BlockScoreArgs {
  const __nv_bfloat16 *q, *bounds;
  const int32_t *block_table, *seqlens;
  KvGeom geo;
  int B, H, qpk, max_blocks, cap, n_first, n_last;
  int32_t* keys;    // [B, G, max_blocks] order-preserving
  int32_t* counts;  // [B] blocks of each request
};

template <int D>
struct BlockScoreCfg {
  static constexpr int kRow = 4 * D + 16;  // one block's bounds, padded: 16-byte reads of 8 lanes hit all banks
  static constexpr size_t kSmem = (size_t)kBtWarps * kBtBlocks * kRow;
};

// x * 2^-896 from the bits of the bf16 in the low or high half of w.
__device__ __forceinline__ double bf16_lo_to_scaled(uint32_t w) {
  return __hiloint2double((static_cast<int>(w << 16) >> 3) & 0x8fffe000, 0);
}
__device__ __forceinline__ double bf16_hi_to_scaled(uint32_t w) {
  return __hiloint2double((static_cast<int>(w) >> 3) & 0x8fffe000, 0);
}

template <int D>
__global__ void __launch_bounds__(kBtThreads) block_score_kernel(const __grid_constant__ BlockScoreArgs a) {
  using C = BlockScoreCfg<D>;
  pdl_wait();  // inputs come from earlier work in the stream
  pdl_trigger();
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ double2 s_q[kBtHeads][D];  // (max(q, 0), min(q, 0)) * 2^800
  const KvGeom& geo = a.geo;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y % geo.G, b = blockIdx.y / geo.G;
  const int L = checked_seqlen(a.seqlens, b, a.cap);
  const int count = geo.bs_div.div(L + geo.bs - 1);
  if (blockIdx.x == 0 && g == 0 && tid == 0) a.counts[b] = count;
  if (blockIdx.x * kBtBlocks * kBtWarps >= count) return;
  const int c0 = (blockIdx.x * kBtWarps + warp) * kBtBlocks;
  unsigned char* rows = smem_raw + (size_t)warp * kBtBlocks * C::kRow;

  // ---- stage the bounds of this warp's blocks ----
  const int c = c0 + lane;
  long long at = -1;
  if (c < count) {
    const int tok = c * geo.bs, pi = geo.page_div.div(tok);
    const int page = a.block_table[(size_t)b * geo.max_pages + pi];
    if (page < 0 || page >= geo.num_pages) raise_error(SD_DEVERR_PAGE);
    else at = ((long long)page * geo.blocks_per_page + geo.bs_div.div(tok - pi * geo.page_size)) * geo.G + g;
  }
  constexpr int kPieces = D / 4;  // 16-byte pieces of a row: [lo D][hi D]
  constexpr int kRowsPerStep = 32 / kPieces;
#pragma unroll 8
  for (int i = 0; i < kBtBlocks; i += kRowsPerStep) {
    const int r = i + lane / kPieces;
    const long long src = __shfl_sync(0xffffffffu, at, r);
    cp_async_16(rows + r * C::kRow + (lane % kPieces) * 16, a.bounds + max(src, 0LL) * 2 * D + (lane % kPieces) * 8,
                src >= 0 ? 16 : 0);
  }
  cp_async_commit();

  double best = -INFINITY;
  bool nan = false;
  for (int h0 = 0; h0 < a.qpk; h0 += kBtHeads) {
    __syncthreads();
    for (int i = tid; i < kBtHeads * D; i += kBtThreads) {
      const int h = h0 + i / D;
      const float x = h < a.qpk ? __bfloat162float(a.q[((size_t)b * a.H + g * a.qpk + h) * D + i % D]) : 0.f;
      const double s = __longlong_as_double(0x71f0000000000000ll);  // 2^800
      s_q[i / D][i % D] = x != x ? make_double2(x, x) : make_double2(fmaxf(x, 0.f) * s, fminf(x, 0.f) * s);
    }
    cp_async_wait<0>();
    __syncthreads();
    double acc[kBtHeads];
#pragma unroll
    for (int h = 0; h < kBtHeads; ++h) acc[h] = 0.0;
    const uint4* lo = reinterpret_cast<const uint4*>(rows + lane * C::kRow);
    const uint4* hi = lo + D / 8;
#pragma unroll 2
    for (int d = 0; d < D / 8; ++d) {
      const uint4 x = lo[d], y = hi[d];
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const double kl = e ? bf16_hi_to_scaled(xw[w]) : bf16_lo_to_scaled(xw[w]);
          const double kh = e ? bf16_hi_to_scaled(yw[w]) : bf16_lo_to_scaled(yw[w]);
#pragma unroll
          for (int h = 0; h < kBtHeads; ++h) {
            const double2 qv = s_q[h][8 * d + 2 * w + e];
            acc[h] = fma(qv.x, kh, fma(qv.y, kl, acc[h]));
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kBtHeads; ++h) {
      if (h0 + h >= a.qpk) continue;
      nan |= acc[h] != acc[h];
      best = fmax(best, acc[h]);
    }
  }
  if (c >= count) return;
  int32_t key;
  if (c < a.n_first || c >= count - a.n_last) {
    key = INT32_MAX;  // always kept: above every score
  } else {
    // fp32 bits as an integer of the same order; a NaN or a bad page counts as -inf
    const float f = nan || at < 0 ? -INFINITY : static_cast<float>(best * 7.9228162514264338e28);  // 2^96
    const int u = __float_as_int(f + 0.f);
    key = u >= 0 ? u : (u ^ 0x7fffffff);
  }
  a.keys[((size_t)b * geo.G + g) * a.max_blocks + c] = key;
}

}  // namespace sd
