// Decode attention over a paged cache held in 8 bits (int8 or e4m3), with one
// fp32 scale per (block of tokens, KV head) for K and one for V:
//   z_j = scale * sk_j * (q . k8_j)
//   o   = sum_j softmax_j(z) * sv_j * v8_j,   lse = ln sum_j exp(z_j)
// over every cached token of the request, or over listed blocks of
// `index_block` tokens per (request, KV head) (1: the tokens an indexer
// selects).
//
// Mathematics. int8: both products run on the 8-bit matrix instructions with
// the codes as they lie in the cache, and the other operand cut into bytes,
// which fill the columns that a decode group's few heads leave free: q * S
// rounded to a 23-bit integer (S a power of two, so bf16 values down to 2^-14
// of the head's largest are exact) as three signed base-256 digits, the
// weights in fixed point as unsigned bytes: four (32 bits) for up to 4 heads,
// where the fourth lies in a column that is free anyway; three (24 bits) for
// up to 8, with the fourth rounded into them by a sequence that goes evenly
// over its range. (Rounded to the nearest, weights below 2^-24 were lost
// altogether, and 2^18 of them beside a large one are a hundredth of the sum.
// Four bytes for 8 heads: 64 query heads 192 us instead of 170.) (Unpacking
// codes to fp16 instead took 80 to 140 integer instructions per 16 tokens, a
// third of the loop.) e4m3: the 8-bit instruction takes as long as two fp16
// ones after a conversion that it repeats for every part, so codes are
// converted once, exactly, and multiplied in fp16: q * S, exact down to 2^-27
// of the largest, in one part, the weight's rounding (11 bits) and 2^11 times
// the rest (11 more) in two, both times 2^14 so that small weights stay
// normal (16 x 32768 tokens: 8-bit instructions 175 us, fp16 163; codes moved
// to fp16 by shifts and masks 211). Groups of more than 8 query heads would
// need more accumulators than there are registers: for them both products run
// on fp16 in either type, with weights of 11 bits, times 2^14: off by 2^-11
// of the weighted |v| at most, a quarter of the output's own rounding where
// the values do not cancel.
// V's scale joins the exponent: with base-2 logits z and u_j = z_j + log2
// sv_j, the weights a_j = 2^(u_j - M) < 2 multiply V's codes, and the sum of
// 2^(z_j - M), in fp32, divides them at the end. One reference M serves both, and it follows the
// running maximum of u lazily: only a value more than 0.9 above it moves it,
// so the common tile takes no shuffle for the maximum and no rescale. int8
// sums are int32 and join fp32 sums when M moves, and every kKaFoldTiles
// tiles, before they can overflow; the sums of weights are taken over
// kKaSumTiles tiles and then added up. The fp16 instructions cut their fp32
// sums at 2^-23 with every 16 tokens: n tokens in a range lose n * 2^-27 of
// their sum at most, an output's rounding at 2^18 of them.
//
// Layout. Everything is warp-private: a warp owns up to 16 query heads of one
// KV head and streams its tokens through a ring of 32-token cp.async stages
// in shared memory; warps of a CTA take the heads of the same tokens, so that
// a CTA's copies cover whole contiguous pool rows. There is no barrier
// anywhere. Both products take the cache as the matrix instruction's A
// operand (S^T = K Q^T and O^T = V^T P^T: M = 16 tokens or dims, N = 8
// columns of heads and parts). K rows become fragments by a matrix load, V
// rows by a transposing 8-bit matrix load, whose lanes get four consecutive
// tokens of one dim; the tokens' order in the products is free, so row i of S
// is the token for which the weights, transposed once, fall to the lanes that hold its codes.
//
// Split. The tokens of all requests form one list of 32-token tiles, cut into
// equal ranges of one resident wave of CTAs; a range that crosses requests
// writes one partial (O, M, l) for each of them, and a combine merges the
// partials in closed form from the list. Ragged batches need no host
// schedule. Bound by HBM where there is enough to read: 2 D bytes per token
// and KV head. 32 query heads over 8 KV heads of 128: 16 x 32768 tokens (1075
// MB) in 163.4 us, 6.58 TB/s, the rate of a plain copy, in either type (64
// query heads 170 us int8 and 166 e4m3, 128 heads 228 and 186); 16 requests of
// 1040 to 9232 tokens (127 MB, e4m3) 28.5 us; 1000 tokens 7.9 us, launches and
// trips to memory.
#pragma once

#include "kv_store.cuh"
#include "sd_common.cuh"

namespace sd {

constexpr int kKaThreads = 256;
constexpr int kKaWarps = kKaThreads / 32;
constexpr int kKaTile = 32;        // tokens per warp and stage: one row lookup per lane
constexpr int kKaRanges = 148;     // CTAs of a column group in one wave: one per SM
constexpr float kKaSlack = 0.9f;   // log2: how far a weight may pass the running reference
constexpr int kKaFoldTiles = 1024; // int32 sums: 1024 x 32 x 255 x 128 < 2^31
constexpr int kKaSumTiles = 64;    // fp32 sums of weights: small ones beside a large one are lost for so long at most

struct KvAttnArgs {
  const __nv_bfloat16* q;
  const uint8_t *k_pages, *v_pages;
  const float *k_scales, *v_scales;
  const int32_t *block_table, *seqlens, *indices;
  KvGeom geo;
  int B, H, qpk, n_list, index_block;
  FastDiv index_div;
  int cap;
  int cols, col_groups, spw;  // (KV head, head block) columns, groups of 8 of them, warps that share a column
  int ranges;
  float scale_log2;
  float* part_o;
  float2* part_ml;
  __nv_bfloat16* out;
  float* lse;
};

// HPW: query heads per warp (4, 8 or 16). Lane (n, t) of a fragment holds the
// logits of kHL heads for the tokens of rows n and n + 8.
template <int D, int HPW, int TYPE>
struct KvAttnCfg {
  static constexpr bool kHalf = TYPE == SD_KV_E4M3 || HPW == 16;  // both products on fp16 instructions
  static constexpr int kParts = kHalf ? 1 : 3;
  // HPW 4: column 2t + x of S tile j is part 2j + x of head t (fp16: x = 0);
  // else tile (hg, p) is part p of heads 8 hg .. 8 hg + 7
  static constexpr int kSTiles = HPW == 4 ? (kParts + 1) / 2 : HPW / 8 * kParts;
  static constexpr int kQSteps = D / (kHalf ? 16 : 32);  // instructions along D
  // O likewise, with the three parts of the weights; fp16: HPW 4: the weight
  // and its rest, HPW 8: a tile of each, HPW 16: head groups
  static constexpr int kOTiles = kHalf ? (HPW == 4 ? 1 : 2) : HPW == 4 ? 2 : 3;
  static constexpr int kHL = HPW == 4 ? 1 : HPW / 4;
  static constexpr float kUp = kHalf ? 14.f : 0.f;  // fp16 weights are held times 2^14: below 2^15, normal down to 2^-28
  static constexpr int kGroups = HPW == 16 ? 2 : 1;
  static constexpr int kRowBytes = kKaTile * D;                   // K (or V) of a stage
  static constexpr int kStage = 2 * kRowBytes + 2 * kKaTile * 4;  // + the tokens' scales
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr size_t kSmem = (size_t)kKaWarps * kStages * kStage;
};

// Tokens (dense) or list slots of request b that the attention walks.
__device__ __forceinline__ int kv_attn_len(const KvAttnArgs& a, int b) {
  const int L = checked_seqlen(a.seqlens, b, a.cap);
  if (a.indices == nullptr) return L;
  return min(a.n_list, a.index_div.div(L + a.index_block - 1)) * a.index_block;
}
__device__ __forceinline__ int kv_attn_tiles(const KvAttnArgs& a, int b) {
  return ceil_div(kv_attn_len(a, b), kKaTile * a.spw);
}
// The list of `total` tiles cut into n ranges: the first `extra` have q + 1
// tiles, the others q.
struct KvAttnCut {
  int n, q, extra;
  __device__ __forceinline__ KvAttnCut(const KvAttnArgs& a, int total) {
    n = max(1, min(a.ranges, total));
    q = total / n;
    extra = total - q * n;
  }
  __device__ __forceinline__ int start(int i) const { return i * q + min(i, extra); }
  __device__ __forceinline__ int range_of(int t) const {
    const int big = extra * (q + 1);
    return t < big ? t / (q + 1) : extra + (t - big) / q;
  }
};

__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// m16n8k32 over signed bytes; UNSIGNED: b holds unsigned ones.
template <bool UNSIGNED = false>
__device__ __forceinline__ void mma_8bit_16832(uint32_t* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (UNSIGNED) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
// Two 16 x 16 byte matrices, transposed: lane (n, t) gets bytes 4t .. 4t + 3 of
// columns n (r[0], r[2]) and n + 8 (r[1], r[3]).
__device__ __forceinline__ void ldmatrix_bytes_trans_x2(uint32_t* r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 2^x and log2 x by the special-function unit (2^-22 relative, 2^-22 absolute
// near one); results below fp32's normal range are zero.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The same down to fp32's smallest number.
__device__ __forceinline__ float fast_exp2_subnormal(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two codes in the low (HI = 0) or high half of w to fp16x2.
template <int TYPE, int HI>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t w) {
  if constexpr (TYPE == SD_KV_INT8) {
    // w holds code + 128 in each byte: 0x6400 | byte is 1024 + byte in fp16,
    // and subtracting 1152 leaves the code, exactly
    const uint32_t x = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    uint32_t r;
    if constexpr (HI) asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(w));
    else asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(w));
    return r;
  }
}
template <int TYPE>
__device__ __forceinline__ uint32_t bias_codes(uint32_t w) {
  return TYPE == SD_KV_INT8 ? w ^ 0x80808080u : w;
}

// The three digits of four elements of q (already times the head's power of
// two), one word per digit, the most significant first.
__device__ __forceinline__ void q_digits(const float* x, uint32_t* w) {
  // |f| <= 2^22; the bytes of f + 0x808080 are its digits in [-128, 127] plus 128
  uint32_t f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = static_cast<uint32_t>(__float2int_rn(x[j]) + 0x808080) ^ 0x808080u;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t sel = p == 0 ? 0x0062u : p == 1 ? 0x0051u : 0x0040u;
    w[p] = __byte_perm(__byte_perm(f[0], f[1], sel), __byte_perm(f[2], f[3], sel), 0x5410);
  }
}

// Weights in fp16, and 2^11 times what the rounding left.
__device__ __forceinline__ void weight_halves(float w0, float w1, uint32_t* hi, uint32_t* lo) {
  *hi = pack_half2(w0, w1);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(hi));
  *lo = pack_half2((w0 - f.x) * 2048.f, (w1 - f.y) * 2048.f);
}

__device__ __forceinline__ int warp_inclusive_sum(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Tiles of requests [0, end), by one warp.
__device__ __forceinline__ int kv_attn_sum(const KvAttnArgs& a, int end) {
  int n = 0;
#pragma unroll 1
  for (int b = threadIdx.x & 31; b < end; b += 32) n += kv_attn_tiles(a, b);
  return __reduce_add_sync(0xffffffffu, n);
}

// The request that holds tile t of the list, and its first tile, by one
// warp; cnt and incl are the first 32 requests' tiles and their inclusive sums.
__device__ __forceinline__ int kv_attn_find(const KvAttnArgs& a, int t, int cnt, int incl, int* first) {
  const int lane = threadIdx.x & 31;
  int before = 0;
#pragma unroll 1
  for (int base = 0;; base += 32) {
    if (base > 0) {
      cnt = base + lane < a.B ? kv_attn_tiles(a, base + lane) : 0;
      incl = warp_inclusive_sum(cnt);
    }
    const unsigned int past = __ballot_sync(0xffffffffu, before + incl > t);
    if (past != 0 || base + 32 >= a.B) {
      const int w = past != 0 ? __ffs(past) - 1 : 31;
      *first = before + __shfl_sync(0xffffffffu, incl - cnt, w);
      return min(base + w, a.B - 1);
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <int D, int HPW, int TYPE, bool LIST>
__global__ void __launch_bounds__(kKaThreads, 1) kv_attn_kernel(const __grid_constant__ KvAttnArgs a) {
  using C = KvAttnCfg<D, HPW, TYPE>;
  pdl_wait();  // inputs come from earlier work in the stream
  pdl_trigger();

  extern __shared__ __align__(16) unsigned char smem_raw[];
  const KvGeom& geo = a.geo;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, t = lane & 3;  // fragment coordinates
  const int G = geo.G;

  // ---- this CTA's range of the tile list, and the request it starts in
  // (every warp finds them for itself: no barrier) ----
  const int cnt = lane < a.B ? kv_attn_tiles(a, lane) : 0, incl = warp_inclusive_sum(cnt);
  const int total = a.B <= 32 ? __shfl_sync(0xffffffffu, incl, 31) : kv_attn_sum(a, a.B);
  const KvAttnCut cut(a, total);
  const int range = blockIdx.x;
  if (range >= cut.n || total == 0) return;
  const int t_begin = cut.start(range), my = cut.start(range + 1) - t_begin;  // tiles, one stage each
  int first;
  const int b_begin = kv_attn_find(a, t_begin, cnt, incl, &first);
  const int tile_begin = t_begin - first;

  // ---- this warp's column ----
  const int col = a.cols >= kKaWarps ? blockIdx.y * kKaWarps + warp : warp % a.cols;
  const int sub = a.cols >= kKaWarps ? 0 : warp / a.cols;
  if (col >= a.cols || sub >= a.spw) return;
  const int hblocks = a.cols / G;
  const int g = col / hblocks, h0 = g * a.qpk + (col % hblocks) * HPW;
  const int nh = min(HPW, (g + 1) * a.qpk - h0);
  unsigned char* ring = smem_raw + (size_t)warp * C::kStages * C::kStage;

  // ---- the copy side, one row per lane and tile, three steps ahead of each
  // other, so that a list entry, its page and its row are never waited for
  // back to back ----
  int pb = b_begin, ptile = tile_begin, plen = kv_attn_len(a, pb), pL = checked_seqlen(a.seqlens, pb, a.cap);
  int l1_tok = -1, l1_rem = 0, l1_b = 0, l1_L = 0;  // after step 1: list entry (or token)
  int l2_page = -1, l2_slot = 0;                    // after step 2: page and slot
  bool l2_ok = false;
  auto step1 = [&](bool live) {
    l1_tok = -1;
    if (!live) return;
    const int v = (ptile * a.spw + sub) * kKaTile + lane;
    l1_b = pb, l1_L = pL;
    if (v < plen) {
      if constexpr (LIST) {
        const int e = a.index_div.div(v);
        l1_rem = v - e * a.index_block;
        l1_tok = a.indices[((size_t)pb * G + g) * a.n_list + e];
      } else {
        l1_tok = v;
      }
    }
    if ((++ptile) * a.spw * kKaTile >= plen) {  // next request that has tiles
      ptile = 0;
#pragma unroll 1
      do {
        ++pb;
        if (pb >= a.B) {
          plen = 0;
          break;
        }
        plen = kv_attn_len(a, pb);
      } while (plen == 0);
      if (pb < a.B) pL = checked_seqlen(a.seqlens, pb, a.cap);
    }
  };
  auto step2 = [&]() {
    int tok = l1_tok;
    if constexpr (LIST) {
      if (tok >= 0) {
        if (tok >= a.index_div.div(l1_L + a.index_block - 1)) {
          raise_error(SD_DEVERR_INDEX);
          tok = -1;
        } else {
          tok = tok * a.index_block + l1_rem;
          if (tok >= l1_L) tok = -1;
        }
      }
    }
    l2_ok = tok >= 0;
    if (l2_ok) {
      const int pi = geo.page_div.div(tok);
      l2_slot = tok - pi * geo.page_size;
      l2_page = a.block_table[(size_t)l1_b * geo.max_pages + pi];
    }
  };
  constexpr int kPieces = D / 16;             // 16-byte pieces of a row
  constexpr int kRowsPerStep = 32 / kPieces;  // rows one copy instruction of the warp covers
  const int crow = lane / kPieces, cpiece = lane % kPieces;
  // 16-byte piece c of token k's row lies at piece c ^ swizzle(k): the eight
  // rows that one phase of a matrix load touches then fall into distinct banks
  auto k_swizzle = [](int k) { return D == 128 ? (k & 1) | ((k >> 2) & 3) << 1 : (k >> 2) & 3; };
  auto v_swizzle = [](int k) { return D == 128 ? k & 7 : (k >> 1) & 3; };
  const uint32_t ring_at = smem_u32(ring);
  // the cache is streamed past L2's other contents: partials, code
  uint64_t once;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
  const uint8_t* k_src = a.k_pages + cpiece * 16;
  const uint8_t* v_src = a.v_pages + cpiece * 16;
  auto issue = [&](int stage) {
    uint32_t row16 = ~0u;  // this lane's row, in 16-byte units; ~0: no token
    const uint32_t base = ring_at + stage * C::kStage;
    float* sc = reinterpret_cast<float*>(ring + stage * C::kStage + 2 * C::kRowBytes) + lane;
    if (l2_ok && (l2_page < 0 || l2_page >= geo.num_pages)) {
      raise_error(SD_DEVERR_PAGE);
      l2_ok = false;
    }
    if (l2_ok) {
      const int rid = l2_page * geo.page_size + l2_slot;
      row16 = (static_cast<uint32_t>(rid) * G + g) * kPieces;
      const size_t at = (size_t)geo.bs_div.div(rid) * G + g;
      cp_async_4(sc, a.k_scales + at);
      cp_async_4(sc + kKaTile, a.v_scales + at);
    } else {
      sc[0] = -1.f;  // no token here
      sc[kKaTile] = 1.f;
    }
    const bool whole = __all_sync(0xffffffffu, l2_ok);
#pragma unroll
    for (int j = 0; j < kKaTile / kRowsPerStep; ++j) {
      const int k = crow + j * kRowsPerStep;
      const uint32_t row = __shfl_sync(0xffffffffu, row16, k);
      const uint32_t k_at = base + k * D + ((cpiece ^ k_swizzle(k)) << 4);
      const uint32_t v_at = base + C::kRowBytes + k * D + ((cpiece ^ v_swizzle(k)) << 4);
      if (whole) {
        const size_t at = (size_t)row * 16;
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(k_at), "l"(k_src + at), "l"(once) : "memory");
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(v_at), "l"(v_src + at), "l"(once) : "memory");
      } else {  // rows without a token are filled with zeros
        const int bytes = row != ~0u ? 16 : 0;
        const size_t at = row != ~0u ? (size_t)row * 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(k_at), "l"(k_src + at), "r"(bytes) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(v_at), "l"(v_src + at), "r"(bytes) : "memory");
      }
    }
  };

  // ---- the compute side ----
  int cb = b_begin, ctile = tile_begin, clen = kv_attn_len(a, cb);
  uint32_t qf[C::kSTiles][C::kQSteps][2];
  float qs[C::kHL];  // scale of this lane's heads (base-2 logits)
  // Whether the sum of weights takes 2^(z - M) itself, and not w / sv. w may
  // be below fp32's range where w / sv is not; but while every V scale met lies
  // between 2^-43 and 2^15, what that loses is below 2^-97 and the sum above
  // 2^-15. (Groups of up to 8 heads always take it themselves, at no cost; with
  // 16 heads each, 128 query heads 186 us so and 200 always, in e4m3.)
  bool wide = HPW != 16;
  // log2 of what a weight of 1 stands for: M - kUp, rounded up, and weights
  // pass it by slack + kUp, rounded down, so that none leaves its range where logits
  // are so large that their last place is above one
  float m[C::kHL];
  float l[C::kHL], ls[C::kHL];    // sums of weights: the last tiles', and those before
  uint32_t o[C::kOTiles][D / 16][4] = {};  // int32 or fp32 sums; D / 16 tiles of 16 dims
  constexpr bool kFold = !C::kHalf;  // int32 sums
  float of[kFold ? C::kHL : 1][D / 16][2];  // what the int32 sums have been folded into
  int since = 0;                            // tiles since then
  auto lane_head = [&](int i) { return HPW == 4 ? t : (i >> 1) * 8 + 2 * t + (i & 1); };
  constexpr float kDown = 1.f / 16384.f;  // 2^-kUp
  constexpr uint32_t kGolden = 0x9e3779b9u;  // 2^32 over the golden ratio
  // sum of this lane's head i, dim 16 j + n + 8 x, in units of its weights and codes
  auto sum_of = [&](int i, int j, int x) {
    if constexpr (C::kHalf && HPW == 4) {  // the rests are in units of 2^-11
      return fmaf(__uint_as_float(o[0][j][2 * x + 1]), kDown / 2048.f, __uint_as_float(o[0][j][2 * x]) * kDown);
    } else if constexpr (C::kHalf && HPW == 8) {
      return fmaf(__uint_as_float(o[C::kOTiles - 1][j][2 * x + (i & 1)]), kDown / 2048.f, __uint_as_float(o[0][j][2 * x + (i & 1)]) * kDown);
    } else if constexpr (C::kHalf) {
      return __uint_as_float(o[i >> 1][j][2 * x + (i & 1)]) * kDown;
    } else {
      const int k = HPW == 4 ? 2 * x : 2 * x + (i & 1);
      const float p0 = static_cast<float>(static_cast<int>(o[0][j][k]));
      const float p1 = static_cast<float>(static_cast<int>(HPW == 4 ? o[0][j][k + 1] : o[1][j][k]));
      const float p2 = static_cast<float>(static_cast<int>(HPW == 4 ? o[1][j][k] : o[C::kOTiles - 1][j][k]));
      float low = p2;
      if constexpr (HPW == 4) low = fmaf(static_cast<float>(static_cast<int>(o[1][j][k + 1])), 1.f / 256.f, p2);
      // digits of 2^-7, 2^-15, 2^-23 and 2^-31
      return fmaf(p0, 0.0078125f, fmaf(p1, 0.0078125f / 256.f, low * (0.0078125f / 65536.f)));
    }
  };
  uint32_t qraw[C::kGroups][D / 8];  // dims 16 kk + 4t .. + 3 in words 2 kk, 2 kk + 1 of head n (HPW 4: n / 2)
  auto fetch_q = [&](int b) {
#pragma unroll
    for (int hg = 0; hg < C::kGroups; ++hg) {
      const int h = HPW == 4 ? n >> 1 : hg * 8 + n;
      const __nv_bfloat16* src = a.q + ((size_t)b * a.H + h0 + (h < nh ? h : 0)) * D;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint2 x = *reinterpret_cast<const uint2*>(src + kk * 16 + 4 * t);
        qraw[hg][2 * kk] = x.x, qraw[hg][2 * kk + 1] = x.y;
      }
    }
  };
  auto begin_request = [&]() {
    float back_of[C::kGroups];  // scale of qraw's heads
#pragma unroll
    for (int hg = 0; hg < C::kGroups; ++hg) {
      const uint32_t* w = qraw[hg];
      // the largest magnitude, as the bits of the bf16s: that of a value that
      // is not finite is above all others
      uint32_t top = 0u;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) top = max(top, max(w[j] & 0x7fff0000u, (w[j] << 16) & 0x7fff0000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // up = 2^(e - floor(log2 amax)), as two factors since it can pass 2^127
      const int ex = min(max(static_cast<int>(top >> 23), 1), 254);  // biased; 0: zero or subnormal
      const int up = (C::kHalf ? 10 : 21) + 127 - ex;
      const float f0 = __uint_as_float((uint32_t)(up / 2 + 127) << 23), f1 = __uint_as_float((uint32_t)(up - up / 2 + 127) << 23);
      // a query that is not finite makes its head's output NaN
      back_of[hg] = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : a.scale_log2 / f0 / f1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const float2 x = bf2(w[2 * kk]), y = bf2(w[2 * kk + 1]);
        const float e[4] = {x.x * f0 * f1, x.y * f0 * f1, y.x * f0 * f1, y.y * f0 * f1};
        if constexpr (C::kHalf) {  // bf16 values fit fp16 down to 2^-27 of the largest
          const bool live = HPW != 4 || (n & 1) == 0;
          qf[hg][kk][0] = live ? pack_half2(e[0], e[1]) : 0u;
          qf[hg][kk][1] = live ? pack_half2(e[2], e[3]) : 0u;
          continue;
        }
        uint32_t p[3];
        q_digits(e, p);
        if constexpr (HPW == 4) {
          qf[0][kk / 2 % C::kQSteps][kk % 2] = n & 1 ? p[1] : p[0];
          qf[C::kSTiles - 1][kk / 2][kk % 2] = n & 1 ? 0u : p[2];
        } else {
#pragma unroll
          for (int i = 0; i < C::kParts; ++i) qf[hg * C::kParts + i][kk / 2][kk % 2] = p[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < C::kHL; ++i) {
      qs[i] = __shfl_sync(0xffffffffu, back_of[HPW == 4 ? 0 : i >> 1], (HPW == 4 ? 2 * t : 2 * t + (i & 1)) * 4);
      m[i] = -INFINITY;
      l[i] = ls[i] = 0.f;
    }
    wide = HPW != 16;
#pragma unroll
    for (int h = 0; h < C::kOTiles; ++h)
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[h][j][0] = o[h][j][1] = o[h][j][2] = o[h][j][3] = 0u;
    if constexpr (kFold) {
      since = 0;
#pragma unroll
      for (int i = 0; i < C::kHL; ++i)
#pragma unroll
        for (int j = 0; j < D / 16; ++j) of[i][j][0] = of[i][j][1] = 0.f;
    }
  };
  auto flush = [&](int b) {
    const size_t slot = ((size_t)range + b) * a.spw + sub;
#pragma unroll
    for (int i = 0; i < C::kHL; ++i) {
      float s = l[i] + ls[i];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      const int h = lane_head(i);
      if (h >= nh) continue;
      const size_t at = slot * a.H + h0 + h;
      // V scales far from one leave s far from one: what its power of two has
      // beyond 2^32 or below 2^-32 moves into M, by which the combine weighs
      // partials (and no more, so that sums of large values stay in range)
      const int pow = s > 0.f && s < INFINITY ? static_cast<int>(__float_as_uint(s) >> 23) - 127 : 0;
      const int e = pow - max(-32, min(32, pow));
      const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (n == 0) a.part_ml[at] = make_float2(m[i] + static_cast<float>(e), s * f);
      float* dst = a.part_o + at * D + n;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = sum_of(i, j, x);
          if constexpr (kFold) v += of[i][j][x];
          dst[16 * j + 8 * x] = v * f;
        }
      }
    }
  };

  // Row i of an S tile is token pi(i): rows 2j, 2j + 1 are tokens 4j, 4j + 1 and
  // rows 8 + 2j, 9 + 2j tokens 4j + 2, 4j + 3. This lane's logits are tokens tk and
  // tk + 2 (and 16 more for the second tile).
  const int tk = 4 * (n >> 1) + (n & 1);
  // this lane's row address in the matrix loads
  const int k_row = 4 * ((lane >> 1) & 3) + (lane & 1) + 2 * ((lane >> 3) & 1);
  const uint32_t k_read = ring_at + k_row * D, v_read = ring_at + C::kRowBytes + lane * D;
  const int k_sw = k_swizzle(k_row), v_sw = v_swizzle(lane);  // rows 16 apart share a swizzle

  auto feed = [&](int i, int stage) {
    if (i < my) {
      issue(stage);
      step2();
      step1(i + 2 < my);
    }
    cp_async_commit();
  };
  // the first tiles' lookups side by side, one trip for all at each step
  {
    fetch_q(b_begin);
    constexpr int kAhead = C::kStages - 1;
    int tok[kAhead], rem[kAhead], rb[kAhead], rL[kAhead], page[kAhead], slot[kAhead];
    bool ok[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      step1(i < my);
      tok[i] = l1_tok, rem[i] = l1_rem, rb[i] = l1_b, rL[i] = l1_L;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      l1_tok = tok[i], l1_rem = rem[i], l1_b = rb[i], l1_L = rL[i];
      step2();
      page[i] = l2_page, slot[i] = l2_slot, ok[i] = l2_ok;
    }
    step1(kAhead < my);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      l2_page = page[i], l2_slot = slot[i], l2_ok = ok[i];
      if (i < my) issue(i);
      cp_async_commit();
    }
    step2();
    step1(kAhead + 1 < my);
  }
  begin_request();
  int stage = 0;
#pragma unroll 1
  for (int at = 0; at < my; ++at) {
    cp_async_wait<C::kStages - 2>();
    __syncwarp();
    feed(at + C::kStages - 1, stage == 0 ? C::kStages - 1 : stage - 1);
    const uint32_t off = stage * C::kStage;
    const float* sc = reinterpret_cast<const float*>(ring + off + 2 * C::kRowBytes);

    // ---- S^T = K Q^T: 2 x 16 tokens x (heads and parts) ----
    uint32_t s[2][C::kSTiles][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int j = 0; j < C::kSTiles; ++j) s[mt][j][0] = s[mt][j][1] = s[mt][j][2] = s[mt][j][3] = 0u;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint32_t f[4];
        ldmatrix_x4_at(f, k_read + off + mt * 16 * D + (((2 * j + (lane >> 4)) ^ k_sw) << 4));
#pragma unroll
        for (int x = 0; x < (C::kHalf ? 2 : 1); ++x) {
          if constexpr (C::kHalf) {  // codes 0, 1 and 2, 3 of each word are the instruction's column pairs
            const uint32_t w0 = bias_codes<TYPE>(f[2 * x]), w1 = bias_codes<TYPE>(f[2 * x + 1]);
            const uint32_t c[4] = {codes_to_half2<TYPE, 0>(w0), codes_to_half2<TYPE, 0>(w1), codes_to_half2<TYPE, 1>(w0),
                                   codes_to_half2<TYPE, 1>(w1)};
#pragma unroll
            for (int h = 0; h < C::kSTiles; ++h)
              mma_f16_16816(reinterpret_cast<float*>(s[mt][h]), c, qf[h][2 * j + x][0], qf[h][2 * j + x][1]);
          } else {
#pragma unroll
            for (int h = 0; h < C::kSTiles; ++h) mma_8bit_16832(s[mt][h], f, qf[h][j][0], qf[h][j][1]);
          }
        }
      }
    }

    // ---- weights: w[r] is token tk + 2 (r & 1) + 16 (r >> 1) ----
    float w[4][C::kHL], lv[4];
    bool over = kFold && ++since >= kKaFoldTiles;
    if ((at & (kKaSumTiles - 1)) == kKaSumTiles - 1) {
#pragma unroll
      for (int i = 0; i < C::kHL; ++i) ls[i] += l[i], l[i] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int k = tk + 2 * (r & 1) + 16 * (r >> 1), x = 2 * (r & 1);
      const float ks = sc[k], vs = fmaxf(sc[kKaTile + k], kKvMinScale);
      lv[r] = fast_log2(vs) + C::kUp;
#pragma unroll
      for (int i = 0; i < C::kHL; ++i) {
        const uint32_t(*p)[4] = s[r >> 1] + (HPW == 4 ? 0 : (i >> 1) * C::kParts);
        const uint32_t p0 = HPW == 4 ? p[0][x] : p[0][x + (i & 1)];
        float z;
        if constexpr (C::kHalf) {
          z = __uint_as_float(p0);
        } else {
          const uint32_t p1 = HPW == 4 ? p[0][x + 1] : p[1][x + (i & 1)], p2 = HPW == 4 ? p[1][x] : p[C::kParts - 1][x + (i & 1)];
          z = fmaf(static_cast<float>(static_cast<int>(p0) * 256 + static_cast<int>(p1)), 256.f, static_cast<float>(static_cast<int>(p2)));
        }
        w[r][i] = ks >= 0.f ? fmaf(z, qs[i] * ks, lv[r]) : -INFINITY;  // u
        over |= w[r][i] > __fadd_rd(m[i], kKaSlack + C::kUp);
      }
    }
    if (__any_sync(0xffffffffu, over)) {
      since = 0;
#pragma unroll
      for (int i = 0; i < C::kHL; ++i) {
        float mx = fmaxf(fmaxf(w[0][i], w[1][i]), fmaxf(w[2][i], w[3][i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        mx = fmaxf(__fadd_ru(mx, -C::kUp), m[i]);
        // in two halves: sums may be as large as alpha is small
        const float half = mx == -INFINITY ? 1.f : fast_exp2((m[i] - mx) * 0.5f), alpha = half * half;
        m[i] = mx;
        ls[i] = (ls[i] + l[i]) * half * half;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if constexpr (kFold) {
              of[i][j][x] = (of[i][j][x] + sum_of(i, j, x)) * alpha;
            } else {
#pragma unroll
              for (int h = 0; h < C::kOTiles; ++h) {
                if constexpr (HPW == 4) {
                  o[h][j][2 * x] = __float_as_uint(__uint_as_float(o[h][j][2 * x]) * alpha);
                  o[h][j][2 * x + 1] = __float_as_uint(__uint_as_float(o[h][j][2 * x + 1]) * alpha);
                } else if (HPW == 8 || h == i >> 1) {
                  o[h][j][2 * x + (i & 1)] = __float_as_uint(__uint_as_float(o[h][j][2 * x + (i & 1)]) * alpha);
                }
              }
            }
          }
        }
      }
      if constexpr (kFold) {
#pragma unroll
        for (int h = 0; h < C::kOTiles; ++h)
#pragma unroll
          for (int j = 0; j < D / 16; ++j) o[h][j][0] = o[h][j][1] = o[h][j][2] = o[h][j][3] = 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < C::kHL; ++i) {
      const float ref = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
      for (int r = 0; r < 4; ++r) w[r][i] -= ref;
    }
    if constexpr (HPW == 16) {
      bool far = false;
#pragma unroll
      for (int r = 0; r < 4; ++r) far |= fabsf(lv[r]) > 29.f;  // log2 sv + 14
      wide |= __any_sync(0xffffffffu, far) != 0;
    }
    if (wide) {
#pragma unroll
      for (int i = 0; i < C::kHL; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) l[i] += fast_exp2_subnormal(w[r][i] - lv[r]);  // 2^-121 where V is near the largest bf16
    }
#pragma unroll
    for (int i = 0; i < C::kHL; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) w[r][i] = fast_exp2(w[r][i]);
    if (!wide) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float isv = fast_exp2(-lv[r]);
#pragma unroll
        for (int i = 0; i < C::kHL; ++i) l[i] = fmaf(w[r][i], isv, l[i]);
      }
    }

    // ---- P: transposed so that a lane has its column's weights of the tokens
    // 4t .. 4t + 3 (+ 16), whose codes it holds ----
    if constexpr (!C::kHalf) {
      uint32_t pf[C::kOTiles][2];
      const uint32_t weyl = kGolden * (static_cast<uint32_t>(at) * kKaTile + tk);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t p[2][C::kHL];  // parts of rows n and n + 8
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          // three parts of four: the last byte is rounded up as often as its
          // value says, by the multiples of the golden ratio (H. Weyl's
          // sequence), so that weights below 2^-24 are lost singly, not in sum
          const uint32_t up = HPW == 4 ? 0u : (weyl + kGolden * (2 * r + 16 * mt)) >> 24;
#pragma unroll
          for (int i = 0; i < C::kHL; ++i) p[r][i] = __float2uint_rn(w[2 * mt + r][i] * 2147483648.f) + up;  // w < 1.9
        }
        if constexpr (HPW == 4) {
          // 16-bit columns 2t: part 0 | part 2 << 8, 2t + 1: part 1 | part 3 << 8
          const uint32_t x = transpose_8x8(__byte_perm(p[0][0], 0u, 0x0213)), y = transpose_8x8(__byte_perm(p[1][0], 0u, 0x0213));
          pf[0][mt] = __byte_perm(x, y, 0x6420);
          pf[1][mt] = __byte_perm(x, y, 0x7531);
        } else {
          // columns 2t + i: part 0 | part 1 << 8 of head i; then part 2 of both rows
          const uint32_t x = transpose_8x8(__byte_perm(p[0][0], p[0][C::kHL - 1], 0x6723));
          const uint32_t y = transpose_8x8(__byte_perm(p[1][0], p[1][C::kHL - 1], 0x6723));
          const uint32_t z = transpose_8x8(__byte_perm(__byte_perm(p[0][0], p[1][0], 0x0051), __byte_perm(p[0][C::kHL - 1], p[1][C::kHL - 1], 0x0051), 0x5410));
          pf[0][mt] = __byte_perm(x, y, 0x6420);
          pf[1][mt] = __byte_perm(x, y, 0x7531);
          pf[C::kOTiles - 1][mt] = __byte_perm(z, 0u, 0x3120);
        }
      }
      // ---- O^T += V^T P^T: D dims x (heads and parts) ----
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t v[4];  // dims 16 j + n, + 8 of tokens 4t .. 4t + 3, then of 16 more
        ldmatrix_bytes_trans_x2(v, v_read + off + ((j ^ v_sw) << 4));
#pragma unroll
        for (int h = 0; h < C::kOTiles; ++h) mma_8bit_16832<true>(o[h][j], v, pf[h][0], pf[h][1]);
      }
    } else {
      uint32_t pf[C::kOTiles][2][2];
      if constexpr (HPW == 4) {  // columns 2t: weight, 2t + 1: its rest
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t hi, lo;
          weight_halves(w[2 * mt][0], w[2 * mt + 1][0], &hi, &lo);
          pf[0][mt][0] = transpose_8x8(__byte_perm(hi, lo, 0x5410));
          pf[0][mt][1] = transpose_8x8(__byte_perm(hi, lo, 0x7632));
        }
      } else if constexpr (HPW == 8) {  // a tile of weights, one of rests
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint32_t hi, lo;
          weight_halves(w[r][0], w[r][C::kHL - 1], &hi, &lo);
          pf[0][r >> 1][r & 1] = transpose_8x8(hi);
          pf[C::kOTiles - 1][r >> 1][r & 1] = transpose_8x8(lo);
        }
      } else {
#pragma unroll
        for (int h = 0; h < C::kOTiles; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            pf[h][r >> 1][r & 1] = transpose_8x8(pack_half2(w[r][(2 * h) % C::kHL], w[r][(2 * h + 1) % C::kHL]));
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t v[4];
        ldmatrix_bytes_trans_x2(v, v_read + off + ((j ^ v_sw) << 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = bias_codes<TYPE>(v[i]);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint32_t f[4] = {codes_to_half2<TYPE, 0>(v[2 * mt]), codes_to_half2<TYPE, 0>(v[2 * mt + 1]),
                                 codes_to_half2<TYPE, 1>(v[2 * mt]), codes_to_half2<TYPE, 1>(v[2 * mt + 1])};
#pragma unroll
          for (int h = 0; h < C::kOTiles; ++h) mma_f16_16816(reinterpret_cast<float*>(o[h][j]), f, pf[h][mt][0], pf[h][mt][1]);
        }
      }
    }

    if (++stage == C::kStages) stage = 0;
    if ((++ctile) * a.spw * kKaTile >= clen || at + 1 == my) {  // the request or the range ends
      const int done = cb;
      if (at + 1 < my) {
        ctile = 0;
#pragma unroll 1
        do clen = kv_attn_len(a, ++cb);
        while (clen == 0 && cb + 1 < a.B);
        fetch_q(cb);
      }
      flush(done);
      if (at + 1 < my) begin_request();
    }
  }
  cp_async_wait<0>();
}

// Merges the partials of one (request, query head): with M = max M_i,
// o = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i. A CTA takes 4 LANES dims
// of it; a group of LANES lanes takes every GROUPS-th partial, BATCH of them
// in flight together with their (M, l): one trip to L2 for up to BATCH *
// GROUPS partials. Few rows have many partials each and take narrow groups
// (LANES 8, 256 threads), many rows have few and take whole rows (LANES D / 4, 128
// threads). The list is walked before the wait for the attention.
template <int D, int LANES, int THREADS, int BATCH>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv_attn_combine_kernel(const __grid_constant__ KvAttnArgs a) {
  constexpr int GROUPS = THREADS / LANES, SLICES = D / (4 * LANES), WARPS = THREADS / 32;
  __shared__ float2 s_ml[WARPS];
  __shared__ float4 s_o[WARPS][LANES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x / SLICES, slice = blockIdx.x - bh * SLICES;
  const int b = bh / a.H, h = bh - b * a.H;
  // the caller's lengths: no kernel of this call writes them, and this kernel
  // starts only after the attention has passed its own wait
  int total, first, tiles;
  if (a.B <= 32) {
    const int cnt = lane < a.B ? kv_attn_tiles(a, lane) : 0, incl = warp_inclusive_sum(cnt);
    total = __shfl_sync(0xffffffffu, incl, 31);
    first = __shfl_sync(0xffffffffu, incl - cnt, b);
    tiles = __shfl_sync(0xffffffffu, cnt, b);
  } else {
    total = kv_attn_sum(a, a.B);
    first = kv_attn_sum(a, b);
    tiles = kv_attn_tiles(a, b);
  }
  int parts = 0;
  size_t slot0 = 0;
  if (tiles > 0) {
    const KvAttnCut cut(a, total);
    const int r0 = cut.range_of(first), r1 = cut.range_of(first + tiles - 1);
    parts = (r1 - r0 + 1) * a.spw;
    slot0 = (size_t)(r0 + b) * a.spw;
  }
  const int grp = tid / LANES, ln = tid % LANES;
  const float2* ml_at = a.part_ml + (slot0 + grp) * a.H + h;
  const float* o_at = a.part_o + ((slot0 + grp) * a.H + h) * D + slice * (4 * LANES) + 4 * ln;
  const size_t hop = (size_t)GROUPS * a.H;
  pdl_wait();
  pdl_trigger();
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // adds a partial to (M, l, acc); a sum of 0 means that it has no token
  auto add = [&](float m2, float l2, const float4& x) {
    const float m = fmaxf(M, m2);
    const float f1 = l == 0.f ? 0.f : exp2f(M - m), f2 = l2 == 0.f ? 0.f : exp2f(m2 - m);
    M = m;
    l = f1 * l + f2 * l2;
    acc.x = f1 * acc.x + f2 * x.x, acc.y = f1 * acc.y + f2 * x.y;
    acc.z = f1 * acc.z + f2 * x.z, acc.w = f1 * acc.w + f2 * x.w;
  };
#pragma unroll 1
  for (int i0 = grp; i0 < parts; i0 += GROUPS * BATCH) {
    float2 ml[BATCH];
    float4 x[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      ml[j] = make_float2(-INFINITY, 0.f);
      x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + j * GROUPS < parts) {
        ml[j] = *ml_at;
        x[j] = *reinterpret_cast<const float4*>(o_at);
      }
      ml_at += hop;
      o_at += hop * D;
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (i0 + j * GROUPS < parts) add(ml[j].x, ml[j].y, x[j]);
  }
#pragma unroll
  for (int o = LANES; o < 32; o <<= 1) {  // the groups of a warp
    const float m2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const float4 x = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
                                 __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o));
    add(m2, l2, x);
  }
  if (lane < LANES) s_o[warp][lane] = acc;
  if (lane == 0) s_ml[warp] = make_float2(M, l);
  __syncthreads();
  if (tid >= LANES) return;
#pragma unroll 1
  for (int w = 1; w < WARPS; ++w) add(s_ml[w].x, s_ml[w].y, s_o[w][tid]);
  const float inv = l == 0.f ? 0.f : 1.f / l;  // 0: nothing was attended
  *reinterpret_cast<uint2*>(a.out + (size_t)bh * D + slice * (4 * LANES) + 4 * tid) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse != nullptr && slice == 0 && tid == 0) a.lse[bh] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace sd
