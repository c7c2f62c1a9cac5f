// Selection of cache blocks by a bound on their scores: for query head h and
// block c of KV head g with per-dim bounds lo, hi of the block's keys,
//   q . k <= sum_d max(q_d lo_d, q_d hi_d)   for every key k of the block,
// and a block's score is the largest bound over the group's query heads. The
// first n_first and last n_last blocks of a request are always kept; the
// library's top-k takes the best others, ties to the lower block.
//
// The sums are held in fp64, where a product of two bf16 values is exact and
// the sum is wrong by 2^-46 of its terms at most, and rounded once to fp32:
// which blocks are selected does not depend on the order of the sum.
// max(q lo, q hi) is q times one of the two, picked by q's sign. A bf16 value
// becomes a double by moving its bits: (x >> 3) with the sign kept, as the
// high word, is x * 2^-896 for every finite x, subnormals and zero included;
// q carries 2^800 and the result 2^96 to make up for it.
//
// Split of the scores: D / 4 lanes share a block, four dims each, so that a
// lane keeps its dims of four query heads in registers; the bounds stream
// through a ring of cp.async stages of the warp's own (read straight into
// registers, too few of them were in flight: 39 against 31 us for 131072
// blocks); the sums of four blocks and four heads are reduced over the lanes
// together, halving their number at each step. Bound
// by HBM (4 D bytes per block and KV head) up to four query heads per KV
// head, and by issue slots above.
//
// Split of the selection: rows of up to kBsMaxBlocks blocks are scored and
// selected in one launch by a cluster per (request, KV head), whose CTAs send
// their keys to the first one's shared memory (a second launch cost 3 us at
// small sizes). There a histogram of the 11 bits below the highest differing
// bit gives the digit of the last key to take, whose few keys are ranked
// directly (further digits where they are many). Longer rows are scored by
// block_score_kernel and selected by the library's cluster top-k.
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

// Scores blocks c0 .. c0 + end - 1 (end <= 32, end + c0 <= count) of (b, g) by one warp; lane
// i < end gets block c0 + i's key. `ring` and `best` (32 floats) are the warp's own.
template <int D>
__device__ __forceinline__ int32_t score_blocks(const BlockScoreArgs& a, int b, int g, int c0, int end, int count,
                                                unsigned char* ring, float* best) {
  constexpr int LANES = D / 4, GROUPS = 32 / LANES, STEP = GROUPS * kBtBatch;
  constexpr int kRow = 4 * D;  // bytes of a block's bounds: lo, hi
  static_assert(STEP * kRow * kBtStages == kBtRing, "ring size");
  const KvGeom& geo = a.geo;
  const int lane = threadIdx.x & 31, grp = lane / LANES, l = lane % LANES;

  // ---- where the blocks are: one per lane ----
  int blk = -1;
  const int c = c0 + lane;
  if (lane < end) {
    const int tok = c * geo.bs, pi = geo.page_div.div(tok);
    const int page = a.block_table[(size_t)b * geo.max_pages + pi];
    if (page < 0 || page >= geo.num_pages) raise_error(SD_DEVERR_PAGE);
    else blk = page * geo.blocks_per_page + geo.bs_div.div(tok - pi * geo.page_size);
  }
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
  if (lane >= end) return 0;
  if (c < a.n_first || c >= count - a.n_last) return INT32_MAX;  // always kept: above every score
  // fp32 bits as an integer of the same order; a bad page counts as -inf
  const int u = __float_as_int((blk < 0 ? -INFINITY : best[lane]) + 0.f);
  return u >= 0 ? u : (u ^ 0x7fffffff);
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
  const int32_t key = score_blocks<D>(a, b, g, c0, end, count, s_ring[warp], s_best[warp]);
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
  int n, digit, above, take;
  uint32_t key;
  int cnt[kBsPer * kWarps];
  float best[kWarps][32];
};
static_assert(sizeof(BlockSelectSmem) % 16 == 0, "ring alignment");
constexpr size_t kBsSmem = sizeof(BlockSelectSmem) + (size_t)(kBsThreads / 32) * kBtRing;

// The n largest of sm.keys[0 .. count), count > n, ties to the lower index,
// written ascending, by one CTA; sm.hist is zero and sm.n 0. Loops stay rolled here and in the scores: these
// kernels run between others that stream the cache, and fetching their code
// anew cost more than their arithmetic.
__device__ __forceinline__ void select_blocks(BlockSelectSmem& sm, int count, int n, int32_t* out) {
  constexpr int kWarps = kBsThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // keys as unsigned integers of the same order
  auto key_at = [&](int c) { return static_cast<uint32_t>(sm.keys[c]) ^ 0x80000000u; };
  uint32_t mn = ~0u, mx = 0u;
  int forced = 0;
#pragma unroll 1
  for (int c = tid; c < count; c += kBsThreads) {
    const uint32_t k = key_at(c);
    forced += k == ~0u;
    if (k != ~0u) mn = min(mn, k), mx = max(mx, k);
  }
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
#pragma unroll 1
      for (int c = tid; c < count; c += kBsThreads) {
        const uint32_t k = key_at(c);
        if (in(k)) atomicAdd(&sm.hist[(k >> shift) & mask], 1u);
      }
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
          if (above < want && above + static_cast<int>(h[j]) >= want) sm.digit = tid * kBinsPer + j, sm.above = above;
          above += h[j];
        }
      }
#pragma unroll
      for (int j = 0; j < kBinsPer; ++j) sm.hist[tid * kBinsPer + j] = 0u;  // for the next round
      __syncthreads();
      want -= sm.above;  // still to take from this digit
      prefix = (prefix << (top - shift)) | static_cast<uint32_t>(sm.digit);
      top = shift;
      // gather the digit's keys; too many of them overrun the list, not its end
#pragma unroll 1
      for (int c = tid; c < count; c += kBsThreads) {
        const uint32_t k = key_at(c);
        if (in(k)) {
          const int at = atomicAdd(&sm.n, 1);
          if (at < kBsList) sm.list[at] = k;
        }
      }
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
}

// One cluster per (request, KV head) row: every CTA scores its part of the
// row, 8 warps of up to 32 blocks at a time, into the first CTA's keys; that
// one selects.
template <int D>
__global__ void __launch_bounds__(kBsThreads, 2) block_topk_kernel(const __grid_constant__ BlockScoreArgs a, int n, int32_t* indices) {
  constexpr int kWarps = kBsThreads / 32;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BlockSelectSmem& sm = *reinterpret_cast<BlockSelectSmem*>(smem_raw);
  unsigned char* rings = smem_raw + sizeof(BlockSelectSmem);
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.y, b = row / a.geo.G, g = row - b * a.geo.G;
  for (int i = tid; i < kBsBins; i += kBsThreads) sm.hist[i] = 0u;
  if (tid == 0) sm.n = 0;
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
  // blocks per warp and pass: a multiple of the batch, the row spread over all warps
  const int chunk = min(kBtChunk, (ceil_div(per, kWarps) + 7) & ~7);
  int32_t* keys = cluster.map_shared_rank(sm.keys, 0);
  bool first = true;
#pragma unroll 1
  for (int c0 = begin + warp * chunk; first || c0 < stop; c0 += kWarps * chunk) {
    const int end = min(chunk, stop - c0);
    int32_t key = 0;
    if (end > 0) key = score_blocks<D>(a, b, g, c0, end, count, rings + warp * kBtRing, sm.best[warp]);
    if (first) {
      __syncwarp();
      cluster.barrier_wait(std::move(started));
      first = false;
    }
    if (lane < end) keys[c0 + lane] = key;
  }
  __syncwarp();
  cluster.sync();  // every key is in place
  if (rank == 0) select_blocks(sm, count, n, out);
}

}  // namespace sd
