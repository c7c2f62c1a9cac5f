// Decode attention over a paged cache held in 8 bits (int8 or e4m3), with one
// fp32 scale per (block of tokens, KV head) for K and one for V:
//   z_j = scale * sk_j * (q . k8_j)
//   o   = sum_j softmax_j(z) * sv_j * v8_j,   lse = ln sum_j exp(z_j)
// over every cached token of the request, or over listed blocks of
// `index_block` tokens per (request, KV head) (1: the tokens an indexer
// selects).
//
// Mathematics. Codes are exact in fp16, so both products run on fp16 matrix
// instructions with fp32 sums; q is scaled per head by a power of two so that
// its largest magnitude lies in [2^14, 2^15), where every bf16 value down to
// 2^-28 of it is exact in fp16. V's scale joins the exponent: with base-2
// logits z and u_j = z_j + log2 sv_j, the weights a_j = 2^(u_j - M) <= 2^8
// multiply the raw codes in fp16 (one rounding, 2^-11) and the sum of
// 2^(z_j - M) in fp32 divides them at the end. One reference M serves both, and
// it follows the running maximum of u lazily: only a value more than 8 above
// it moves it, so the common tile takes no shuffle for the maximum and no
// rescale.
//
// Layout. Everything is warp-private: a warp owns one KV head (8 * NT query
// heads of it) and streams its tokens 16 at a time through a ring of cp.async
// stages in shared memory; warps of a CTA take the heads of the same tokens,
// so that a CTA's copies cover whole contiguous pool rows. No barrier is needed after the work
// list is set up. Both products take the cache as the matrix instruction's A operand (S^T = K Q^T
// and O^T = V^T P^T: M = 16 tokens or dims, N = 8 heads), since a decode
// group has few query heads: m16n8k16 then wastes half of what heads as M = 16
// would. The order of the contracted dims is free as long as q and K agree, as is the
// order of V's dims, so each lane reads 16-byte pieces of rows and unpacks
// them in registers straight into fragments; no transposing load is needed.
//
// Split. The tokens of all requests form one list of 16-token tiles, cut into
// equal ranges of one resident wave of CTAs; a range that crosses requests
// writes one partial (O, M, l) for each of them, and a combine merges the
// partials in closed form from the list. Ragged batches need no host
// schedule. Bound by HBM: 2 D bytes per token and KV head.
#pragma once

#include "kv_store.cuh"
#include "sd_common.cuh"

namespace sd {

constexpr int kKaThreads = 256;
constexpr int kKaWarps = kKaThreads / 32;
constexpr int kKaTile = 16;      // tokens per warp and stage
constexpr int kKaRanges = 296;   // CTAs of a column group in one wave: two per SM
constexpr int kKaMinTiles = 2;   // fewest tiles a range gets (shorter lists use fewer ranges)
constexpr float kKaSlack = 8.f;  // log2: how far a weight may pass the running reference

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

template <int D, int NT>
struct KvAttnCfg {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kRowBytes = kKaTile * D;               // K (or V) of a stage
  static constexpr int kStage = 2 * kRowBytes + 2 * kKaTile * 4;  // + the tokens' scales
  static constexpr int kStages = D == 128 ? 3 : 5;
  static constexpr size_t kSmem = (size_t)kKaWarps * kStages * kStage;
  static constexpr int kCtas = NT == 1 ? 2 : 1;               // resident CTAs per SM
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
// How many ranges the list of `total` tiles is cut into.
__device__ __forceinline__ int kv_attn_ranges(const KvAttnArgs& a, long long total) {
  return static_cast<int>(max(1LL, min((long long)a.ranges, total / kKaMinTiles)));
}

__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
    const __half2_raw r =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(HI ? w >> 16 : w & 0xffffu), __NV_E4M3);
    return static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
  }
}
template <int TYPE>
__device__ __forceinline__ uint32_t bias_codes(uint32_t w) {
  return TYPE == SD_KV_INT8 ? w ^ 0x80808080u : w;
}

// Exclusive position of the CTA's range in the tile list. All threads of the
// CTA call it; `total` and the request that holds tile `first` come back in
// every thread.
__device__ __forceinline__ long long kv_attn_total(const KvAttnArgs& a, long long* s_sum, int threads) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long n = 0;
  for (int b = tid; b < a.B; b += threads) n += kv_attn_tiles(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) s_sum[warp] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < threads / 32; ++w) n += s_sum[w];
  __syncthreads();
  return n;
}

template <int D, int NT, int TYPE, bool LIST>
__global__ void __launch_bounds__(kKaThreads, (KvAttnCfg<D, NT>::kCtas)) kv_attn_kernel(const __grid_constant__ KvAttnArgs a) {
  using C = KvAttnCfg<D, NT>;
  pdl_wait();  // inputs come from earlier work in the stream
  pdl_trigger();

  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ long long s_sum[kKaWarps];
  __shared__ long long s_first;
  __shared__ int s_b;
  const KvGeom& geo = a.geo;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, t = lane & 3;  // fragment coordinates
  const int G = geo.G;

  // ---- this CTA's range of the tile list, and the request it starts in ----
  const long long total = kv_attn_total(a, s_sum, kKaThreads);
  const int nr = kv_attn_ranges(a, total);
  if (blockIdx.x >= nr || total == 0) return;
  const long long t_begin = blockIdx.x * total / nr, t_end = (blockIdx.x + 1) * total / nr;
  {
    long long before = 0;
    for (int base = 0; base < a.B; base += kKaThreads) {
      const int b = base + tid;
      const int cnt = b < a.B ? kv_attn_tiles(a, b) : 0;
      long long incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) s_sum[warp] = incl;
      __syncthreads();
      long long skip = before, all = 0;
      for (int w = 0; w < kKaWarps; ++w) {
        skip += w < warp ? s_sum[w] : 0;
        all += s_sum[w];
      }
      const long long e = skip + incl;
      if (t_begin < e && t_begin >= e - cnt) s_b = b, s_first = e - cnt;
      before += all;
      __syncthreads();
      if (before > t_begin) break;
    }
  }
  const int b_begin = s_b;
  const int tile_begin = static_cast<int>(t_begin - s_first);

  // ---- this warp's column ----
  const int col = a.cols >= kKaWarps ? blockIdx.y * kKaWarps + warp : warp % a.cols;
  const int sub = a.cols >= kKaWarps ? 0 : warp / a.cols;
  if (col >= a.cols || sub >= a.spw) return;  // no barrier below
  const int hblocks = a.cols / G;
  const int g = col / hblocks, h0 = g * a.qpk + (col % hblocks) * C::kHeads;
  const int nh = min(C::kHeads, (g + 1) * a.qpk - h0);
  unsigned char* ring = smem_raw + (size_t)warp * C::kStages * C::kStage;
  const int my = static_cast<int>(t_end - t_begin);  // tiles, one stage each

  // ---- the copy side: three steps ahead of each other, so that a list
  // entry, its page and its row are never waited for back to back ----
  int pb = b_begin, ptile = tile_begin, plen = kv_attn_len(a, pb), pL = checked_seqlen(a.seqlens, pb, a.cap);
  int l1_tok = -1, l1_rem = 0, l1_b = 0, l1_L = 0;  // after step 1: list entry (or token)
  int l2_page = -1, l2_slot = 0;                   // after step 2: page and slot
  bool l2_ok = false;
  const int r = lane & (kKaTile - 1);
  auto step1 = [&](bool live) {
    l1_tok = -1;
    if (!live) return;
    const int v = (ptile * a.spw + sub) * kKaTile + r;
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
  // swizzles: see the reads below
  const int k_at = crow * D + ((D == 128 ? cpiece ^ ((crow & 1) << 2) : cpiece) << 4);
  const int v_at = crow * D + ((D == 128 ? cpiece ^ ((crow & 3) << 1) : cpiece ^ (((crow >> 1) & 1) << 1)) << 4);
  auto issue = [&](int stage) {
    unsigned char* st = ring + stage * C::kStage;
    int rid = -1;
    if (l2_ok) {
      if (l2_page >= 0 && l2_page < geo.num_pages) rid = l2_page * geo.page_size + l2_slot;
      else raise_error(SD_DEVERR_PAGE);
    }
#pragma unroll
    for (int j = 0; j < kKaTile / kRowsPerStep; ++j) {
      const int row = __shfl_sync(0xffffffffu, rid, crow + j * kRowsPerStep);
      const long long off = ((long long)max(row, 0) * G + g) * D + cpiece * 16;
      const int bytes = row >= 0 ? 16 : 0;  // 0: the piece is filled with zeros
      cp_async_16(st + k_at + j * kRowsPerStep * D, a.k_pages + off, bytes);
      cp_async_16(st + C::kRowBytes + v_at + j * kRowsPerStep * D, a.v_pages + off, bytes);
    }
    float* sc = reinterpret_cast<float*>(st + 2 * C::kRowBytes) + lane;  // lanes 0-15: K, 16-31: V
    if (rid >= 0) {
      const float* src = (lane < kKaTile ? a.k_scales : a.v_scales) + (long long)geo.bs_div.div(rid) * G + g;
      cp_async_4(sc, src);
    } else {
      *sc = -1.f;  // no token here
    }
  };

  // ---- the compute side ----
  int cb = b_begin, ctile = tile_begin;
  int cntiles = kv_attn_tiles(a, cb);
  uint32_t qf[NT][D / 16][2];
  float qs[NT][2];                     // scale of heads 2t, 2t + 1 (base-2 logits)
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
  auto load_q = [&]() {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int h = i * 8 + n;
      const __nv_bfloat16* src = a.q + ((size_t)cb * a.H + h0 + (h < nh ? h : 0)) * D;
      uint4 raw[D / 32];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {  // piece t + 4j: 16 dims, 32 bytes
        raw[2 * j] = *reinterpret_cast<const uint4*>(src + (t + 4 * j) * 16);
        raw[2 * j + 1] = *reinterpret_cast<const uint4*>(src + (t + 4 * j) * 16 + 8);
      }
      const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const float2 x = bf2(w[j]);
        amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // up = 2^(14 - floor(log2 amax)), as two factors since it can pass 2^127
      int ex = static_cast<int>(__float_as_uint(amax) >> 23);  // biased; 0: zero or subnormal
      ex = min(max(ex, 1), 254);
      const int up = 14 + 127 - ex;                            // -113 .. 140
      const float f0 = __uint_as_float((uint32_t)(up / 2 + 127) << 23), f1 = __uint_as_float((uint32_t)(up - up / 2 + 127) << 23);
      const float back = a.scale_log2 / f0 / f1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const float2 x = bf2(w[2 * kk]), y = bf2(w[2 * kk + 1]);
        qf[i][kk][0] = pack_half2(x.x * f0 * f1, x.y * f0 * f1);
        qf[i][kk][1] = pack_half2(y.x * f0 * f1, y.y * f0 * f1);
      }
      qs[i][0] = __shfl_sync(0xffffffffu, back, (2 * t) * 4);
      qs[i][1] = __shfl_sync(0xffffffffu, back, (2 * t + 1) * 4);
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
    }
  };
  auto flush = [&]() {
    const size_t slot = ((size_t)blockIdx.x + cb) * a.spw + sub;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float s = l[i][x];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int h = i * 8 + 2 * t + x;
        if (h >= nh) continue;
        const size_t at = slot * a.H + h0 + h;
        if (n == 0) a.part_ml[at] = make_float2(m[i][x], s);
        // this lane's dims of the head: n * D/8 .. + D/8 - 1, dim 2j and 2j + 1 from m-tile j
        float4* dst = reinterpret_cast<float4*>(a.part_o + at * D + n * (D / 8));
#pragma unroll
        for (int j = 0; j < D / 16; j += 2)
          dst[j / 2] = make_float4(o[i][j][x], o[i][j][2 + x], o[i][j + 1][x], o[i][j + 1][2 + x]);
      }
    }
  };

  // A row i (= n, n + 8) of the token tile is token pi(i): pi(2j) = j,
  // pi(2j + 1) = (j + 4) ^ 1, + 8 for the upper half. It makes the rows that one
  // phase of a shared load touches differ in the bits the swizzles use.
  const int tk = (n & 1) ? (((n >> 1) + 4) ^ 1) : (n >> 1);
  const int tv0 = t, tv1 = (t + 4) ^ 1;  // tokens pi(2t), pi(2t + 1)

  step1(my > 0);
  step2();
  step1(my > 1);
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) {
    if (s < my) issue(s);
    cp_async_commit();
    step2();
    step1(s + 2 < my);
  }
  load_q();
  int stage = 0;
  for (int i = 0; i < my; ++i) {
    cp_async_wait<C::kStages - 2>();
    __syncwarp();
    {
      int st = stage + C::kStages - 1;
      if (st >= C::kStages) st -= C::kStages;
      if (i + C::kStages - 1 < my) issue(st);
      cp_async_commit();
      step2();
      step1(i + C::kStages + 1 < my);
    }
    const unsigned char* sk = ring + stage * C::kStage;
    const unsigned char* sv = sk + C::kRowBytes;
    const float* sc = reinterpret_cast<const float*>(sv + C::kRowBytes);

    // ---- S^T = K Q^T: 16 tokens x 8 NT heads ----
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const int piece = D == 128 ? (t + 4 * j) ^ ((tk & 1) << 2) : t;
      const uint4 x = *reinterpret_cast<const uint4*>(sk + tk * D + piece * 16);
      const uint4 y = *reinterpret_cast<const uint4*>(sk + (tk + 8) * D + piece * 16);
      const uint32_t* xw = reinterpret_cast<const uint32_t*>(&x);
      const uint32_t* yw = reinterpret_cast<const uint32_t*>(&y);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t xb = bias_codes<TYPE>(xw[w]), yb = bias_codes<TYPE>(yw[w]);
        const uint32_t af[4] = {codes_to_half2<TYPE, 0>(xb), codes_to_half2<TYPE, 0>(yb), codes_to_half2<TYPE, 1>(xb),
                                codes_to_half2<TYPE, 1>(yb)};
#pragma unroll
        for (int h = 0; h < NT; ++h) mma_f16_16816(s[h], af, qf[h][4 * j + w][0], qf[h][4 * j + w][1]);
      }
    }

    // ---- weights ----
    const float sk0 = sc[tk], sk1 = sc[tk + 8];
    const float lv0 = log2f(fmaxf(sc[kKaTile + tk], FLT_MIN)), lv1 = log2f(fmaxf(sc[kKaTile + tk + 8], FLT_MIN));
    const bool ok0 = sk0 >= 0.f, ok1 = sk1 >= 0.f;
    bool over = false;
#pragma unroll
    for (int h = 0; h < NT; ++h) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        s[h][x] = ok0 ? s[h][x] * (qs[h][x] * sk0) : -INFINITY;
        s[h][2 + x] = ok1 ? s[h][2 + x] * (qs[h][x] * sk1) : -INFINITY;
        over |= s[h][x] + lv0 > m[h][x] + kKaSlack || s[h][2 + x] + lv1 > m[h][x] + kKaSlack;
      }
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int h = 0; h < NT; ++h) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = fmaxf(s[h][x] + lv0, s[h][2 + x] + lv1);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          mx = fmaxf(mx, m[h][x]);
          const float alpha = mx == -INFINITY ? 1.f : exp2f(m[h][x] - mx);
          m[h][x] = mx;
          l[h][x] *= alpha;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) o[h][j][x] *= alpha, o[h][j][2 + x] *= alpha;
        }
      }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      float w[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float ref = m[h][x] == -INFINITY ? 0.f : m[h][x];
        l[h][x] += exp2f(s[h][x] - ref) + exp2f(s[h][2 + x] - ref);
        w[x] = exp2f(s[h][x] + lv0 - ref);
        w[2 + x] = exp2f(s[h][2 + x] + lv1 - ref);
      }
      pf[h][0] = transpose_8x8(pack_half2(w[0], w[1]));
      pf[h][1] = transpose_8x8(pack_half2(w[2], w[3]));
    }

    // ---- O^T += V^T P^T: D dims x 8 NT heads; lane row n holds dims
    // n * D/8 .. n * D/8 + D/8 - 1 of the tokens tv0, tv1 (+ 8) ----
    constexpr int kVW = D / 32;  // 4-byte words of a lane's part of a V row
    uint32_t va[4][kVW];
    const int tok[4] = {tv0, tv1, tv0 + 8, tv1 + 8};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(sv + tok[j] * D + ((n ^ ((tok[j] & 3) << 1)) << 4));
        va[j][0] = x.x, va[j][1] = x.y, va[j][2] = x.z, va[j][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(sv + tok[j] * D + (((n >> 1) ^ (((tok[j] >> 1) & 1) << 1)) << 4) + (n & 1) * 8);
        va[j][0] = x.x, va[j][1] = x.y;
      }
    }
#pragma unroll
    for (int w = 0; w < kVW; ++w) {
      // bytes of two tokens side by side: (tok0 dim d, tok1 dim d), ...
      const uint32_t x0 = bias_codes<TYPE>(__byte_perm(va[0][w], va[1][w], 0x5140));
      const uint32_t x1 = bias_codes<TYPE>(__byte_perm(va[0][w], va[1][w], 0x7362));
      const uint32_t y0 = bias_codes<TYPE>(__byte_perm(va[2][w], va[3][w], 0x5140));
      const uint32_t y1 = bias_codes<TYPE>(__byte_perm(va[2][w], va[3][w], 0x7362));
      const uint32_t f0[4] = {codes_to_half2<TYPE, 0>(x0), codes_to_half2<TYPE, 1>(x0), codes_to_half2<TYPE, 0>(y0),
                              codes_to_half2<TYPE, 1>(y0)};
      const uint32_t f1[4] = {codes_to_half2<TYPE, 0>(x1), codes_to_half2<TYPE, 1>(x1), codes_to_half2<TYPE, 0>(y1),
                              codes_to_half2<TYPE, 1>(y1)};
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        mma_f16_16816(o[h][2 * w], f0, pf[h][0], pf[h][1]);
        mma_f16_16816(o[h][2 * w + 1], f1, pf[h][0], pf[h][1]);
      }
    }

    if (++stage == C::kStages) stage = 0;
    if (++ctile == cntiles || i + 1 == my) {  // the request or the range ends
      flush();
      if (i + 1 < my) {
        ctile = 0;
        do cntiles = kv_attn_tiles(a, ++cb);
        while (cntiles == 0 && cb + 1 < a.B);
        load_q();
      }
    }
  }
  cp_async_wait<0>();
}

// Merges the partials of one (request, query head): with M = max M_i,
// o = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i. One CTA each; a group of
// D / 4 lanes takes every (128 / (D / 4))-th partial.
constexpr int kKaCombineThreads = 128;

template <int D>
__global__ void __launch_bounds__(kKaCombineThreads) kv_attn_combine_kernel(const __grid_constant__ KvAttnArgs a) {
  constexpr int LANES = D / 4, GROUPS = kKaCombineThreads / LANES;
  __shared__ long long s_sum[kKaCombineThreads / 32];
  __shared__ float s_m[kKaCombineThreads / 32];
  __shared__ float s_l[GROUPS];
  __shared__ float4 s_o[GROUPS][LANES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  // the caller's lengths: no kernel of this call writes them, and this kernel
  // starts only after the attention has passed its own wait
  const long long total = kv_attn_total(a, s_sum, kKaCombineThreads);
  long long first = 0;
  for (int i = tid; i < b; i += kKaCombineThreads) first += kv_attn_tiles(a, i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
  if (lane == 0) s_sum[warp] = first;
  __syncthreads();
  first = 0;
  for (int w = 0; w < kKaCombineThreads / 32; ++w) first += s_sum[w];
  const int tiles = kv_attn_tiles(a, b);
  pdl_wait();
  pdl_trigger();
  const size_t bh = (size_t)b * a.H + h;
  if (tiles == 0) {
    if (tid < LANES) *reinterpret_cast<uint2*>(a.out + bh * D + 4 * tid) = make_uint2(0u, 0u);
    if (a.lse != nullptr && tid == 0) a.lse[bh] = -INFINITY;
    return;
  }
  const int nr = kv_attn_ranges(a, total);
  const long long r0 = ((first + 1) * nr - 1) / total, r1 = ((first + tiles) * nr - 1) / total;
  const int parts = static_cast<int>(r1 - r0 + 1) * a.spw;
  const size_t slot0 = (size_t)(r0 + b) * a.spw;
  float M = -INFINITY;
  for (int i = tid; i < parts; i += kKaCombineThreads) M = fmaxf(M, a.part_ml[(slot0 + i) * a.H + h].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
  for (int w = 0; w < kKaCombineThreads / 32; ++w) M = fmaxf(M, s_m[w]);
  const int grp = tid / LANES, ln = tid % LANES;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = grp; i < parts; i += GROUPS) {
    const size_t at = (slot0 + i) * a.H + h;
    const float2 ml = a.part_ml[at];
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + at * D + 4 * ln);
    const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - M);  // sum 0: no token there
    l += f * ml.y;
    acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
  }
  s_o[grp][ln] = acc;
  if (ln == 0) s_l[grp] = l;
  __syncthreads();
  if (tid >= LANES) return;
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < GROUPS; ++i) {
    const float4 x = s_o[i][ln];
    l += s_l[i];
    acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // 0: nothing was attended
  *reinterpret_cast<uint2*>(a.out + bh * D + 4 * ln) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse != nullptr && ln == 0) a.lse[bh] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace sd
