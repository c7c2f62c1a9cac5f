// Selection of cache blocks by a bound on their scores: for query head h and
// block c of KV head g with per-dim bounds lo, hi of the block's keys,
//   q . k <= sum_d max(q_d lo_d, q_d hi_d)   for every key k of the block
// (as it was before coding), and a block's score is the largest bound over the
// group's query heads. The first n_first and last n_last blocks of a request
// are always kept; the library's top-k takes the best others, ties to the lower
// block.
//
// The sums are held in fp64, where a product of two bf16 values is exact and
// the sum is wrong by 2^-46 of its terms at most, and rounded once to fp32: the
// order of the sum matters only to a score that lies that close to the middle
// of two fp32 numbers, and a row is ranked by scores of one order. max(q lo, q
// hi) is q times one of the two, picked by q's sign. A bf16 value becomes a
// double by moving its bits: (x >> 3) with the sign kept, as the high word, is
// x * 2^-896 for every finite x, subnormals and zero included; q carries 2^800
// and the result 2^96 to make up for it.
//
// Split of the exact scores: D / 4 lanes share a block, four dims each, so that a
// lane keeps its dims of four query heads in registers; the bounds stream
// through a ring of cp.async stages of the warp's own (read straight into
// registers, too few of them were in flight: 39 against 31 us for 131072
// blocks); the sums of four blocks and four heads are reduced over the lanes
// together, halving their number at each step. Bound by issue slots: 80
// instructions a block and warp.
//
// Approximate scores. The indices are those of the exact scores, but few
// blocks lie near enough to the border for the exact score to matter. The
// matrix instructions give 16 blocks x 8 heads at a time to within a bound
// that they sum as well (sum_d |q_d| max(|lo_d|, |hi_d|), times 2^-14): blocks
// further than twice that from the border are settled, and the others, five
// of 1024 for normal values, get their exact scores. The border is found by a
// histogram over the scores' leading bits, refined while a digit holds more
// blocks than are worth scoring (unrefined, rows around a power of two, around
// zero or with one block on a bad page listed hundreds: 128 rows of 1024
// around 2.0 took 72 us, now 19). Where the bound does not hold (values that
// are not finite, or so large or small that a product leaves fp32's range) or
// over 256 blocks lie within it of the border, the row is scored exactly, by
// the one CTA that selects (128 rows of 1024 equal blocks: 72 us a call, of 4096: 262 us).
//
// Split of the selection: rows of up to kBsMaxBlocks blocks are scored and
// selected in one launch by a cluster per (request, KV head), whose CTAs send
// their keys to the first one's shared memory (a second launch cost 3 us at
// small sizes). There a histogram of the 11 bits below the highest differing
// bit gives the digit of the last key to take, whose few keys are ranked
// directly (further digits where they are many). Longer rows are scored by
// block_score_kernel and selected by the library's cluster top-k.
//
// Bound by HBM (4 D bytes per block and KV head) where there are many rows,
// else by the chain of trips to memory. 128 rows of 1024 blocks of 128 dims
// (67 MB, 10.3 us): 21.7 us, of which the scores take 15.8 (exact ones alone 33);
// 8 rows of 256 blocks: 5.7 us.
#pragma once

#include <cooperative_groups.h>

#include <utility>

#include "kv_store.cuh"
#include "sd_common.cuh"

namespace sd {

constexpr int kBtHeads = 4;   // query heads summed at once
constexpr int kBtBatch = 4;   // blocks a lane group has in flight
constexpr int kBtChunk = 32;  // most blocks a warp scores at a time
constexpr int kBtStages = 5;  // batches in the ring
constexpr int kBtRing = kBtStages * 2048;  // bytes of a warp's ring: a batch is 2 KB for either D
constexpr int kBtThreads = 128;            // of block_score_kernel

struct BlockScoreArgs {
  const __nv_bfloat16 *q, *bounds;
  const int32_t *block_table, *seqlens;
  KvGeom geo;
  int B, H, qpk, max_blocks, cap, n_first, n_last;
  int32_t* keys;    // [B, G, max_blocks] order-preserving
  int32_t* counts;  // [B] blocks of each request
};

// High word of x * 2^-896 from the bits of the bf16 in the low or high half of w.
__device__ __forceinline__ uint32_t bf16_lo_scaled_hi(uint32_t w) {
  return static_cast<uint32_t>(static_cast<int>(w << 16) >> 3) & 0x8fffe000u;
}
__device__ __forceinline__ uint32_t bf16_hi_scaled_hi(uint32_t w) {
  return static_cast<uint32_t>(static_cast<int>(w) >> 3) & 0x8fffe000u;
}

// Where lane's block c of request b lies in the pool, in blocks; -1: nowhere.
__device__ __forceinline__ int locate_block(const BlockScoreArgs& a, int b, int c) {
  const KvGeom& geo = a.geo;
  const int tok = c * geo.bs, pi = geo.page_div.div(tok);
  const int page = a.block_table[(size_t)b * geo.max_pages + pi];
  if (page < 0 || page >= geo.num_pages) {
    raise_error(SD_DEVERR_PAGE);
    return -1;
  }
  return page * geo.blocks_per_page + geo.bs_div.div(tok - pi * geo.page_size);
}

// The key of a block: fp32 bits as an integer of the same order; blocks that
// are always kept lie above every score.
__device__ __forceinline__ int32_t block_key(const BlockScoreArgs& a, int c, int count, float score) {
  if (c < a.n_first || c >= count - a.n_last) return INT32_MAX;
  const int u = __float_as_int(score + 0.f);
  return u >= 0 ? u : (u ^ 0x7fffffff);
}

// Scores up to 32 blocks of (b, g) by one warp; lane i < end gets the key of
// its block c. `ring` and `best` (32 floats) are the warp's own.
template <int D>
__device__ __forceinline__ int32_t score_blocks(const BlockScoreArgs& a, int b, int g, int c, int end, int count,
                                                unsigned char* ring, float* best) {
  constexpr int LANES = D / 4, GROUPS = 32 / LANES, STEP = GROUPS * kBtBatch;
  constexpr int kRow = 4 * D;  // bytes of a block's bounds: lo, hi
  static_assert(STEP * kRow * kBtStages == kBtRing, "ring size");
  const KvGeom& geo = a.geo;
  const int lane = threadIdx.x & 31, grp = lane / LANES, l = lane % LANES;

  const int blk = lane < end ? locate_block(a, b, c) : -1;
  best[lane] = -INFINITY;
  __syncwarp();

#pragma unroll 1
  for (int h0 = 0; h0 < a.qpk; h0 += kBtHeads) {
    // ---- four dims of four heads: value times 2^800, and which bound its sign picks ----
    double q[kBtHeads][4];
    uint32_t pick[kBtHeads][4];
#pragma unroll
    for (int h = 0; h < kBtHeads; ++h) {
      uint2 w = make_uint2(0u, 0u);
      if (h0 + h < a.qpk) w = *reinterpret_cast<const uint2*>(a.q + ((size_t)b * a.H + g * a.qpk + h0 + h) * D + 4 * l);
      const float2 x = bf2(w.x), y = bf2(w.y);
      const float e[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        q[h][d] = static_cast<double>(e[d]) * __longlong_as_double(0x71f0000000000000ll);  // 2^800
        pick[h][d] = e[d] < 0.f ? 0x3210u : 0x7654u;
      }
    }
    auto feed = [&](int i0, int stage) {  // blocks i0 .. i0 + STEP - 1
      if (i0 < end) {
        constexpr int kPerCopy = 512 / kRow;  // rows that one copy of the warp covers
#pragma unroll
        for (int i = 0; i < STEP / kPerCopy; ++i) {
          const int r = i * kPerCopy + lane / (32 / kPerCopy), piece = lane % (32 / kPerCopy);
          const int at = __shfl_sync(0xffffffffu, blk, (i0 + r) & 31);
          cp_async_16(ring + stage * (STEP * kRow) + r * kRow + piece * 16,
                      a.bounds + ((long long)max(at, 0) * geo.G + g) * (2 * D) + piece * 8, at >= 0 ? 16 : 0);
        }
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kBtStages - 1; ++i) feed(i * STEP, i);
    int stage = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < end; i0 += STEP) {
      cp_async_wait<kBtStages - 2>();
      __syncwarp();
      feed(i0 + (kBtStages - 1) * STEP, stage == 0 ? kBtStages - 1 : stage - 1);
      const unsigned char* rows = ring + stage * (STEP * kRow) + grp * kBtBatch * kRow + 8 * l;
      stage = stage + 1 == kBtStages ? 0 : stage + 1;
      double v[kBtBatch * kBtHeads];
#pragma unroll
      for (int i = 0; i < kBtBatch; ++i) {
        const uint2 lo = *reinterpret_cast<const uint2*>(rows + i * kRow), hi = *reinterpret_cast<const uint2*>(rows + i * kRow + 2 * D);
        const uint32_t kl[4] = {bf16_lo_scaled_hi(lo.x), bf16_hi_scaled_hi(lo.x), bf16_lo_scaled_hi(lo.y), bf16_hi_scaled_hi(lo.y)};
        const uint32_t kh[4] = {bf16_lo_scaled_hi(hi.x), bf16_hi_scaled_hi(hi.x), bf16_lo_scaled_hi(hi.y), bf16_hi_scaled_hi(hi.y)};
#pragma unroll
        for (int h = 0; h < kBtHeads; ++h) {
          double s = 0.0;
#pragma unroll
          for (int d = 0; d < 4; ++d) s = fma(q[h][d], __hiloint2double(__byte_perm(kl[d], kh[d], pick[h][d]), 0), s);
          v[i * kBtHeads + h] = s;
        }
      }
      // sums over the LANES lanes: at each step a lane hands half of its
      // values to its partner, so 16 values cost 16 exchanges, not 16 x 5
      int n = kBtBatch * kBtHeads;
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) {
        if (n > 1) {
          const bool up = (l & o) != 0;
#pragma unroll
          for (int i = 0; i < kBtBatch * kBtHeads / 2; ++i) {
            if (i < n / 2) {
              const double mine = up ? v[i + n / 2] : v[i], other = up ? v[i] : v[i + n / 2];
              v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
            }
          }
          n /= 2;
        } else {
          v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
      }
      // value of block (bits LANES/2, LANES/4 of l), head (the next two bits)
      float f = static_cast<float>(v[0] * 7.9228162514264338e28);  // 2^96
      const int head = ((l & (LANES / 8)) ? 2 : 0) + ((l & (LANES / 16)) ? 1 : 0);
      if (f != f || h0 + head >= a.qpk) f = -INFINITY;  // a head that is not finite picks nothing
      f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, LANES / 8));
      f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, LANES / 16));
      if ((l & (LANES / 4 - 1)) == 0) {
        const int i = i0 + grp * kBtBatch + ((l & (LANES / 2)) ? 2 : 0) + ((l & (LANES / 4)) ? 1 : 0);
        if (i < end) best[i] = fmaxf(best[i], f);
      }
    }
    cp_async_wait<0>();
    __syncwarp();  // the ring is free for the next heads
  }
  return lane < end ? block_key(a, c, count, blk < 0 ? -INFINITY : best[lane]) : 0;
}

// The score of one block of the pool by one warp, as score_blocks makes it: 8 lanes a
// head, four heads at a time. Little code: it runs cold, on a few blocks.
template <int D>
__device__ __forceinline__ float exact_score(const BlockScoreArgs& a, int b, int g, int blk) {
  constexpr int kDims = D / 8;  // of a lane
  const int lane = threadIdx.x & 31, hq = lane >> 3, d0 = (lane & 7) * kDims;
  if (blk < 0) return -INFINITY;
  const __nv_bfloat16* rows = a.bounds + ((size_t)blk * a.geo.G + g) * (2 * D) + d0;
  float best = -INFINITY;
#pragma unroll 1
  for (int h0 = 0; h0 < a.qpk; h0 += 4) {
    const bool live = h0 + hq < a.qpk;
    const __nv_bfloat16* q = a.q + ((size_t)b * a.H + g * a.qpk + (live ? h0 + hq : 0)) * D + d0;
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kDims; i += 8) {
      const uint2 qa = *reinterpret_cast<const uint2*>(q + i), qb = *reinterpret_cast<const uint2*>(q + i + 4);
      const uint4 lw = *reinterpret_cast<const uint4*>(rows + i), hw = *reinterpret_cast<const uint4*>(rows + D + i);
      const uint32_t qv[4] = {qa.x, qa.y, qb.x, qb.y}, lo[4] = {lw.x, lw.y, lw.z, lw.w}, hi[4] = {hw.x, hw.y, hw.z, hw.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = bf2(qv[j]);
        const uint32_t u = bf16_lo_scaled_hi(x.x < 0.f ? lo[j] : hi[j]), w = bf16_hi_scaled_hi(x.y < 0.f ? lo[j] : hi[j]);
        const double scale = __longlong_as_double(0x71f0000000000000ll);  // 2^800
        s[0] = fma(static_cast<double>(x.x) * scale, __hiloint2double(u, 0), s[0]);
        s[1] = fma(static_cast<double>(x.y) * scale, __hiloint2double(w, 0), s[1]);
      }
    }
    double v = s[0] + s[1];
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    float f = static_cast<float>(v * 7.9228162514264338e28);  // 2^96
    if (f != f || !live) f = -INFINITY;
    f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 8));
    best = fmaxf(best, fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 16)));
  }
  return best;
}

template <bool MAX>
__device__ __forceinline__ uint32_t bf16x2_pick(uint32_t x, uint32_t y) {
  const __nv_bfloat162 p = *reinterpret_cast<const __nv_bfloat162*>(&x), q = *reinterpret_cast<const __nv_bfloat162*>(&y);
  const __nv_bfloat162 r = MAX ? __hmax2(p, q) : __hmin2(p, q);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The scores of blocks c0 .. c0 + len - 1 to within 2^-14 of a bound of their
// terms' sums, by one warp and matrix instructions, as keys[c] (of the
// cluster's first CTA, once `ready` has returned): bound = hi . max(q, 0) + lo
// . min(q, 0), 16 blocks x 8 heads at a time. Returns, as fp32 bits, the largest sum_d
// |q_d| max(|lo_d|, |hi_d|) or score met; infinity (or NaN, above that) where
// the error has no such bound. The error: a product of two bf16 values is exact in fp32, and
// an instruction is taken to align its 17 addends to the largest and to cut
// each, and the sum, at 2^-23 of it at worst; 2 D / 16 = 16 instructions make
// 288 * 2^-23 < 2^-14.8 of the terms' sum. (How it rounds is not documented;
// over 10^8 scores of normal, wide-ranging and cancelling values the
// worst error was 2^-19.2.)
template <int D, class Ready>
__device__ __forceinline__ uint32_t approx_blocks(const BlockScoreArgs& a, int b, int g, int c0, int len, int count,
                                                  unsigned char* ring, int32_t* keys, Ready ready) {
  constexpr int kParts = D / 32;               // a stage: 32 dims of lo and of hi of 16 blocks
  constexpr int kStage = kBtRing / kBtStages;  // 16 rows of 128 bytes
  static_assert(kStage == 16 * 128, "stage size");
  const KvGeom& geo = a.geo;
  const int lane = threadIdx.x & 31, n = lane >> 2, t = lane & 3;
  const int total = ceil_div(max(len, 0), 16) * kParts;
  uint32_t top = 0u;
  const uint32_t ring_at = smem_u32(ring);
  const int crow = lane >> 3, cpiece = lane & 7;
  const __nv_bfloat16* src = a.bounds + (size_t)g * (2 * D) + (cpiece >> 2) * D + (cpiece & 3) * 8;
  // where blocks are, one per lane and 32 blocks ahead: the table's entry is loaded 32 blocks before it is looked at
  int page, in_page, blk, chunk;
  unsigned int ok, ok_before;
  auto look_up = [&](int i) {
    page = INT32_MAX;  // no block
    if (i + lane < len) {
      const int tok = (c0 + i + lane) * geo.bs, pi = geo.page_div.div(tok);
      page = a.block_table[(size_t)b * geo.max_pages + pi];
      if (page == INT32_MAX) page = -1;
      in_page = geo.bs_div.div(tok - pi * geo.page_size);
    }
  };
  auto feed = [&](int s, int slot) {
    if (s < total) {
      const int tile = s / kParts, part = s % kParts;
      if (part == 0 && (tile & 1) == 0) {  // the next 32 blocks
        blk = -1;
        if (page >= 0 && page < geo.num_pages) blk = page * geo.blocks_per_page + in_page;
        else if (page != INT32_MAX) raise_error(SD_DEVERR_PAGE);
        ok_before = ok;
        ok = __ballot_sync(0xffffffffu, blk >= 0);
        chunk = tile >> 1;
        look_up(16 * tile + 32);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + crow, at = __shfl_sync(0xffffffffu, blk, (16 * tile + r) & 31);
        cp_async_16(ring + slot * kStage + r * 128 + ((cpiece ^ (r & 7)) << 4),
                    src + (long long)max(at, 0) * geo.G * (2 * D) + part * 32, at >= 0 ? 16 : 0);
      }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int h0 = 0; h0 < a.qpk; h0 += 8) {
    ok = 0u;
    in_page = 0;
    look_up(0);
#pragma unroll 1
    for (int s = 0; s < kBtStages - 1; ++s) feed(s, s);
    uint32_t qp[D / 16][2], qn[D / 16][2], qa[D / 16][2];
    {
      const bool live = h0 + n < a.qpk;
      const __nv_bfloat16* q = a.q + ((size_t)b * a.H + g * a.qpk + (live ? h0 + n : 0)) * D + 2 * t;
      bool odd = false;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t w = live ? *reinterpret_cast<const uint32_t*>(q + 8 * i) : 0u;
        const uint32_t m = w & 0x7fff7fffu, m0 = m << 16, m1 = m & 0xffff0000u;
        // subnormal, or 2^60 and more (a bound's subnormal part would count)
        odd |= (m0 - 1u) < 0x007fffffu || (m1 - 1u) < 0x007fffffu || max(m0, m1) >= 0x5d800000u;
        qp[i >> 1][i & 1] = bf16x2_pick<true>(w, 0u);
        qn[i >> 1][i & 1] = bf16x2_pick<false>(w, 0u);
        qa[i >> 1][i & 1] = m;
      }
      if (odd) top = 0x7f800000u;
    }
    if (h0 == 0) ready();
    int slot = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < len; i0 += 16) {
      float x[4] = {}, y[4] = {};  // scores; sums of magnitudes
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        cp_async_wait<kBtStages - 2>();
        __syncwarp();
        feed(i0 / 16 * kParts + part + kBtStages - 1, slot == 0 ? kBtStages - 1 : slot - 1);
        const uint32_t row = ring_at + slot * kStage + (lane & 15) * 128;
        slot = slot + 1 == kBtStages ? 0 : slot + 1;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t lo[4], hi[4], m[4];
          ldmatrix_x4_at(lo, row + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
          ldmatrix_x4_at(hi, row + (((4 + 2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
          const int kk = 2 * part + k;
          mma_bf16_16816(x, lo, qn[kk][0], qn[kk][1]);
          mma_bf16_16816(x, hi, qp[kk][0], qp[kk][1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) m[j] = bf16x2_pick<true>(lo[j] & 0x7fff7fffu, hi[j] & 0x7fff7fffu);
          mma_bf16_16816(y, m, qa[kk][0], qa[kk][1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        top = max(top, max(__float_as_uint(x[j]) & 0x7fffffffu, __float_as_uint(y[j]) & 0x7fffffffu));
        if (h0 + 2 * t + (j & 1) >= a.qpk) x[j] = -INFINITY;
      }
      const unsigned int here = (i0 >> 5 == chunk ? ok : ok_before) >> (i0 & 16);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float f = fmaxf(x[2 * r], x[2 * r + 1]);
        f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 1));
        f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 2));
        const int i = i0 + 8 * r + n;
        if (t == 0 && i < len) {
          const int32_t key = block_key(a, c0 + i, count, here >> (8 * r + n) & 1u ? f : -INFINITY);
          if (h0 == 0) keys[c0 + i] = key;
          else atomicMax(keys + c0 + i, key);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();  // the ring is free for the next heads
  }
  return top;
}

// Keys of rows longer than kBsMaxBlocks, for the cluster top-k.
template <int D>
__global__ void __launch_bounds__(kBtThreads, 4) block_score_kernel(const __grid_constant__ BlockScoreArgs a) {
  __shared__ __align__(16) unsigned char s_ring[kBtThreads / 32][kBtRing];
  __shared__ float s_best[kBtThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = blockIdx.y % a.geo.G, b = blockIdx.y / a.geo.G;
  pdl_wait();  // inputs come from earlier work in the stream
  pdl_trigger();
  const int L = checked_seqlen(a.seqlens, b, a.cap);
  const int count = a.geo.bs_div.div(L + a.geo.bs - 1);
  if (blockIdx.x == 0 && g == 0 && threadIdx.x == 0) a.counts[b] = count;
  const int c0 = (blockIdx.x * (kBtThreads / 32) + warp) * kBtChunk;
  if (c0 >= count) return;
  const int end = min(kBtChunk, count - c0);
  const int32_t key = score_blocks<D>(a, b, g, c0 + lane, end, count, s_ring[warp], s_best[warp]);
  if (lane < end) a.keys[((size_t)b * a.geo.G + g) * a.max_blocks + c0 + lane] = key;
}

constexpr int kBsThreads = 256;
constexpr int kBsPer = 16;                            // keys per thread
constexpr int kBsMaxBlocks = kBsThreads * kBsPer;     // longest row
constexpr int kBsBits = 11;
constexpr int kBsBins = 1 << kBsBits;
constexpr int kBsList = 256;                          // keys ranked directly

struct alignas(16) BlockSelectSmem {  // the rings, copied to in 16-byte pieces, follow it
  static constexpr int kWarps = kBsThreads / 32;
  int32_t keys[kBsMaxBlocks];
  uint32_t hist[kBsBins];
  uint32_t mins[kWarps], maxs[kWarps];
  int sums[kWarps], forced[kWarps];
  uint32_t list[kBsList];
  int place[kBsList];  // the blocks of list's keys, and where they are
  int where[kBsList];
  uint32_t mag;
  int sure;
  int n, digit, above, inside, take;
  uint32_t key;
  int cnt[kBsPer * kWarps];
  float best[kWarps][32];
};
static_assert(sizeof(BlockSelectSmem) % 16 == 0, "ring alignment");
constexpr size_t kBsSmem = sizeof(BlockSelectSmem) + (size_t)(kBsThreads / 32) * kBtRing;

// The n largest of sm.keys[0 .. count), count > n, ties to the lower index,
// written ascending, by one CTA; sm.hist is zero, sm.n and sm.sure 0. APPROX:
// the keys are within sm.mag * 2^-14 of the scores. The digit of the last key
// to take then bounds the last score to take to within twice that; blocks above
// are taken, blocks below left, and `rescore` makes exact keys of those between
// for the list to be ranked by. False: too many lie between, or the error has
// no bound (the histogram is zero again). Loops stay rolled here and in the
// scores: these kernels run between others that stream the cache, and fetching
// their code anew cost more than their arithmetic.
template <bool APPROX, class Locate, class Rescore>
__device__ __forceinline__ bool select_blocks(BlockSelectSmem& sm, int count, int n, int32_t* out, Locate locate, Rescore rescore) {
  constexpr int kWarps = kBsThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // keys as unsigned integers of the same order
  auto key_at = [&](int c) { return static_cast<uint32_t>(sm.keys[c]) ^ 0x80000000u; };
  auto each = [&](auto f) {
#pragma unroll 1
    for (int c = tid; c < count; c += kBsThreads) f(c, key_at(c));
  };
  uint32_t mn = ~0u, mx = 0u;
  int forced = 0;
  each([&](int, uint32_t k) {
    forced += k == ~0u;
    if (k != ~0u) mn = min(mn, k), mx = max(mx, k);
  });
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  forced = __reduce_add_sync(0xffffffffu, forced);
  if (lane == 0) sm.mins[warp] = mn, sm.maxs[warp] = mx, sm.forced[warp] = forced;
  __syncthreads();
  forced = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mn = min(mn, sm.mins[w]), mx = max(mx, sm.maxs[w]), forced += sm.forced[w];
  // the keys that are not forced, of which `want` >= 0 are taken: all lie in
  // [mn, mx]. T: the smallest key taken, take: how many equal to it
  int want = n - forced;
  uint32_t T = ~0u;
  int take = 0;
  if (want > 0) {
    int top = 32 - __clz(static_cast<int>(mn ^ mx));  // bits [top, 32) are the same in all
    uint32_t prefix = top == 32 ? 0u : mx >> top;     // of the keys still in question
#pragma unroll 1
    while (true) {
      const int shift = max(0, top - kBsBits);
      const uint32_t mask = (1u << (top - shift)) - 1u;  // top - shift <= 11
      auto in = [&](uint32_t x) { return x != ~0u && x >= mn && (top == 32 ? 0u : x >> top) == prefix; };
      each([&](int, uint32_t k) {
        if (in(k)) atomicAdd(&sm.hist[(k >> shift) & mask], 1u);
      });
      __syncthreads();
      // from the highest digit down: thread t holds bins [t * 8, t * 8 + 8)
      constexpr int kBinsPer = kBsBins / kBsThreads;
      uint32_t h[kBinsPer];
      int own = 0;
#pragma unroll
      for (int j = 0; j < kBinsPer; ++j) h[j] = sm.hist[tid * kBinsPer + j], own += h[j];
      int incl = own;  // this thread's bins and all higher ones of the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_down_sync(0xffffffffu, incl, o);
        if (lane + o < 32) incl += x;
      }
      if (lane == 0) sm.sums[warp] = incl;
      __syncthreads();
      int above = incl - own;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) above += w > warp ? sm.sums[w] : 0;
      if (above < want && above + own >= want) {
#pragma unroll
        for (int j = kBinsPer - 1; j >= 0; --j) {
          if (above < want && above + static_cast<int>(h[j]) >= want) sm.digit = tid * kBinsPer + j, sm.above = above, sm.inside = static_cast<int>(h[j]);
          above += h[j];
        }
      }
#pragma unroll
      for (int j = 0; j < kBinsPer; ++j) sm.hist[tid * kBinsPer + j] = 0u;  // for the next round
      __syncthreads();
      want -= sm.above;  // still to take from this digit
      prefix = (prefix << (top - shift)) | static_cast<uint32_t>(sm.digit);
      top = shift;
      if constexpr (APPROX) {
        auto score_of = [](uint32_t k) {
          const int u = static_cast<int>(k ^ 0x80000000u);
          return __int_as_float(u >= 0 ? u : (u ^ 0x7fffffff));
        };
        const uint32_t d_lo = max(mn, top == 32 ? 0u : prefix << top), d_hi = min(mx, d_lo | ((1u << top) - 1u));
        const float mag = __uint_as_float(sm.mag), gap = mag * 2.5f / 16384.f;
        if (!(mag >= 9.094947e-13f && mag < 1.2676506e30f)) return false;  // 2^-40 (see `odd`), 2^100
        // A digit is as wide as the row's exponents make it: an eighth of the score where the
        // row straddles a power of two. One more round costs as much as two exact scores a warp.
        if (top > 0 && sm.inside > 2 * kWarps && score_of(d_hi) - score_of(d_lo) > gap) continue;
        const float lo = score_of(d_lo) - gap, hi = score_of(d_hi) + gap;
        int above = 0;
        each([&](int c, uint32_t k) {
          if (k == ~0u) return;
          const float f = score_of(k);
          if (f > hi) {
            ++above;
            sm.keys[c] = INT32_MAX;
          } else {
            if (!(f < lo)) {
              const int at = atomicAdd(&sm.n, 1);
              if (at < kBsList) sm.place[at] = c, sm.where[at] = locate(c);
            }
            sm.keys[c] = INT32_MIN;
          }
        });
        above = __reduce_add_sync(0xffffffffu, above);
        if (lane == 0 && above != 0) atomicAdd(&sm.sure, above);
        __syncthreads();
        const int m = sm.n;
        want = n - forced - sm.sure;
        if (m > kBsList) return false;
        rescore(m);  // sm.list[i]: the key of block sm.place[i]
        __syncthreads();
        if (tid < m) {
          const uint32_t x = sm.list[tid];
          const int c = sm.place[tid];
          int more = 0;
#pragma unroll 1
          for (int j = 0; j < m; ++j) more += sm.list[j] > x || (sm.list[j] == x && sm.place[j] < c);
          if (more < want) sm.keys[c] = INT32_MAX;
        }
        __syncthreads();
        break;
      }
      // gather the digit's keys; too many of them overrun the list, not its end
      each([&](int, uint32_t k) {
        if (in(k)) {
          const int at = atomicAdd(&sm.n, 1);
          if (at < kBsList) sm.list[at] = k;
        }
      });
      __syncthreads();
      const int m = sm.n;
      if (m <= kBsList) {
        if (tid < m) {
          const uint32_t x = sm.list[tid];
          int more = 0, same = 0;
#pragma unroll 1
          for (int j = 0; j < m; ++j) more += sm.list[j] > x, same += sm.list[j] == x;
          if (more < want && more + same >= want) sm.key = x, sm.take = want - more;  // equal keys write the same
        }
        __syncthreads();
        T = sm.key, take = sm.take;
        break;
      }
      if (top == 0) {  // all equal
        T = prefix, take = want;
        break;
      }
      __syncthreads();
      if (tid == 0) sm.n = 0;
    }
  }
  // ---- ordered output: key > T, and the first `take` keys equal to T ----
  const int per = ceil_div(count, kBsThreads);
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const int c = i * kBsThreads + tid;
    const uint32_t k = c < count ? key_at(c) : 0u;
    const unsigned int gt = __ballot_sync(0xffffffffu, k > T || k == ~0u), eq = __ballot_sync(0xffffffffu, c < count && k == T && k != ~0u);
    if (lane == 0) sm.cnt[i * kWarps + warp] = __popc(gt) | (__popc(eq) << 16);
  }
  __syncthreads();
  if (warp == 0) {  // exclusive prefix over (i, warp) in index order
    const int m = per * kWarps;
    constexpr int kPer = kBsPer * kWarps / 32;
    int c[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int at = lane * kPer + j;
      c[j] = at < m ? sm.cnt[at] : 0;
      sum += c[j];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    int at = incl - sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      sm.cnt[lane * kPer + j] = at;
      at += c[j];
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const int c = i * kBsThreads + tid;
    const uint32_t k = c < count ? key_at(c) : 0u;
    const bool is_gt = k > T || k == ~0u, is_eq = c < count && k == T && k != ~0u;
    const unsigned int gt = __ballot_sync(0xffffffffu, is_gt), eq = __ballot_sync(0xffffffffu, is_eq);
    const unsigned int lower = (1u << lane) - 1u;
    const int before = sm.cnt[i * kWarps + warp];
    const int g0 = (before & 0xffff) + __popc(gt & lower), e0 = (before >> 16) + __popc(eq & lower);
    if (is_gt || (is_eq && e0 < take)) out[g0 + min(e0, take)] = c;
  }
  return true;
}

// One cluster per (request, KV head) row: every CTA scores its part of the
// row, 8 warps of up to 32 blocks at a time, into the first CTA's keys; that
// one selects. APPROX: by the matrix instructions' scores, and exact ones of
// the blocks near the border.
template <int D, bool APPROX>
__global__ void __launch_bounds__(kBsThreads, 2) block_topk_kernel(const __grid_constant__ BlockScoreArgs a, int n, int32_t* indices) {
  constexpr int kWarps = kBsThreads / 32;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BlockSelectSmem& sm = *reinterpret_cast<BlockSelectSmem*>(smem_raw);
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* ring = smem_raw + sizeof(BlockSelectSmem) + warp * kBtRing;
  const int cs = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.y, b = row / a.geo.G, g = row - b * a.geo.G;
  for (int i = tid; i < kBsBins; i += kBsThreads) sm.hist[i] = 0u;
  if (tid == 0) sm.n = 0, sm.sure = 0, sm.mag = 0u;
  pdl_wait();  // inputs come from earlier work in the stream
  pdl_trigger();
  const int L = checked_seqlen(a.seqlens, b, a.cap);
  const int count = a.geo.bs_div.div(L + a.geo.bs - 1);
  int32_t* out = indices + (size_t)row * n;
  if (count <= n) {  // everything is kept (the whole cluster leaves here)
    for (int i = rank * kBsThreads + tid; i < n; i += cs * kBsThreads) out[i] = i < count ? i : -1;
    return;
  }
  // the first CTA's memory may be written once every CTA has started
  auto started = cluster.barrier_arrive();
  const int per = ceil_div(count, cs), begin = rank * per, stop = min(count, begin + per);
  int32_t* keys = cluster.map_shared_rank(sm.keys, 0);
  if constexpr (APPROX) {
    const int share = (ceil_div(per, kWarps) + 15) & ~15, c0 = begin + warp * share;  // whole tiles
    uint32_t mag = approx_blocks<D>(a, b, g, c0, min(share, stop - c0), count, ring, keys,
                                    [&]() { __syncwarp(); cluster.barrier_wait(std::move(started)); });
    mag = __reduce_max_sync(0xffffffffu, mag);
    if (lane == 0) atomicMax(cluster.map_shared_rank(&sm.mag, 0), mag);
  } else {
    // blocks per warp and pass: a multiple of the batch, the row spread over all warps
    const int chunk = min(kBtChunk, (ceil_div(per, kWarps) + 7) & ~7);
    bool first = true;
#pragma unroll 1
    for (int c0 = begin + warp * chunk; first || c0 < stop; c0 += kWarps * chunk) {
      const int end = min(chunk, stop - c0);
      int32_t key = 0;
      if (end > 0) key = score_blocks<D>(a, b, g, c0 + lane, end, count, ring, sm.best[warp]);
      if (first) {
        __syncwarp();
        cluster.barrier_wait(std::move(started));
        first = false;
      }
      if (lane < end) keys[c0 + lane] = key;
    }
  }
  __syncwarp();
  cluster.sync();  // every key is in place
  if (rank != 0) return;
  if constexpr (APPROX) {
    auto locate = [&](int c) { return locate_block(a, b, c); };
    auto rescore = [&](int m) {
#pragma unroll 1
      for (int i = warp; i < m; i += kWarps) {
        const float f = exact_score<D>(a, b, g, sm.where[i]);
        if (lane == 0) sm.list[i] = static_cast<uint32_t>(block_key(a, sm.place[i], count, f)) ^ 0x80000000u;
      }
    };
    if (select_blocks<true>(sm, count, n, out, locate, rescore)) return;
    __syncthreads();
    if (tid == 0) sm.n = 0;
#pragma unroll 1
    for (int c0 = warp * kBtChunk; c0 < count; c0 += kWarps * kBtChunk) {
      const int end = min(kBtChunk, count - c0);
      const int32_t key = score_blocks<D>(a, b, g, c0 + lane, end, count, ring, sm.best[warp]);
      if (lane < end) sm.keys[c0 + lane] = key;
    }
    __syncthreads();
  }
  select_blocks<false>(sm, count, n, out, [](int) { return 0; }, [](int) {});
}

}  // namespace sd
