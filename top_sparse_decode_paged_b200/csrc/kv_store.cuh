// Writing tokens into a blocked paged cache: the norm of every query and key
// head, the position rotation, and the store of K and V, in one pass.
//
// For a head row x [D] of the token at position p (fp32 throughout):
//   y = x * rsqrt(mean(x^2) + eps) * w          (skipped where w is null)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = p * inv_freq[i],
//   over the pairs (i, i + R/2), or (2i, 2i + 1), of the first R dims.
// The angle is taken in turns in fp64 and reduced to [-1/2, 1/2] before it is
// rounded to fp32 (a far position times a frequency keeps only a few bits of
// its fraction in fp32). q is rounded once to bf16. K and V go into a bf16,
// int8 or e4m3 pool. An 8-bit pool is cut into blocks of `bs` consecutive
// slots (a page holds whole blocks); a block and KV head have one scale for K
// and one for V:
//   s = max(amax(new rows) / qmax, s of the block's earlier rows, 2^-100)
// with qmax 127 or 448, codes round(y / s), and the earlier rows of a block
// whose scale grew coded anew, round(code * s_old / s_new). A growing scale
// costs an earlier row one more rounding each time it grows, and never
// clips a later token. Entries that are not finite do not enter the scale:
// NaN is coded as 0, infinities as the largest code.
// The block's bounds (smallest and largest bf16(y) of K for every dim) are
// what the block selection reads.
//
// Work split. K and V: one CTA per (touched block, KV head), since the scale
// needs the whole block's rows before any of them is coded; the rows stay in
// registers in between. q: one group of D / 8 lanes per (token, group of
// heads); the token's angles are computed once per group and used for its
// heads. Bound by HBM for prompts and by launch and load latency for a
// decode step.
#pragma once

#include <float.h>

#include "sd_common.cuh"

namespace sd {

constexpr int kKvThreads = 256;
constexpr int kKvMaxBlock = 128;       // largest block_tokens
constexpr float kKvMinScale = 7.888609052210118e-31f;  // 2^-100
constexpr int kKvQHeads = 4;           // q rows a lane group has in flight

// Page geometry of a blocked cache.
struct KvGeom {
  int num_pages, page_size, max_pages, G, bs, blocks_per_page;
  FastDiv page_div, bs_div;
};

struct KvStoreArgs {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const int32_t *tok_start, *positions, *block_table, *seqlens;
  KvGeom geo;
  void *k_pages, *v_pages;
  float *k_scales, *v_scales;
  __nv_bfloat16* bounds;
  int kv_type, B, T, H, cap;
  const __nv_bfloat16 *qw, *kw;
  float eps;
  const float* inv_freq;
  int R;
  bool interleaved;
  __nv_bfloat16* q_out;
  int kv_ctas, heads_per_group, head_groups;
  bool by_row;  // unit u is row u (where every row can start a block), else the u-th touched block
};

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The largest b in [0, B) with tok_start[b] <= r, by the LANES lanes of a
// group together: one load a lane and step. l is the lane in its group.
template <int LANES>
__device__ __forceinline__ int find_request(const int32_t* tok_start, int B, int r, int l) {
  const int base = (threadIdx.x & 31) & ~(LANES - 1);
  int lo = 0;
  for (int span = B; span > 1;) {
    const int step = (span + LANES - 1) / LANES;
    const int i = lo + l * step;
    const bool le = i < B && l * step < span && tok_start[i] <= r;
    const unsigned int ball = __ballot_sync(0xffffffffu, le) >> base;
    const int n = __popc(LANES == 32 ? ball : (ball & ((1u << (LANES & 31)) - 1u)));
    lo += max(n - 1, 0) * step;
    span = step;
  }
  return lo;
}

// A lane's 8 elements of a row: dims 4l .. 4l+3 and D/2 + 4l .. D/2 + 4l+3,
// so that the pairs (i, i + D/2) and (2i, 2i + 1) both lie in one lane.
template <int D>
__device__ __forceinline__ void unpack_row(const uint2& a, const uint2& b, float* e) {
  const float2 x0 = bf2(a.x), x1 = bf2(a.y), x2 = bf2(b.x), x3 = bf2(b.y);
  e[0] = x0.x, e[1] = x0.y, e[2] = x1.x, e[3] = x1.y;
  e[4] = x2.x, e[5] = x2.y, e[6] = x3.x, e[7] = x3.y;
}

template <int D>
__device__ __forceinline__ void load_weight(const __nv_bfloat16* w, int l, float* e) {
  const uint2 a = *reinterpret_cast<const uint2*>(w + 4 * l), b = *reinterpret_cast<const uint2*>(w + D / 2 + 4 * l);
  unpack_row<D>(a, b, e);
}

template <int D>
__device__ __forceinline__ void norm_row(float* e, const float* w, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(e[j], e[j], ss);
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float r = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = e[j] * r * w[j];
}

// Cosine and sine for a lane's elements. FULL: every dim is rotated in pairs
// (i, i + D/2), and elements j and j + 4 share an angle.
template <int D, bool FULL>
struct Rotation {
  static constexpr int N = FULL ? 4 : 8;
  double f[N];  // turns per position (0: not rotated)
  float c[N], s[N];

  __device__ __forceinline__ void init(const float* inv_freq, int R, bool interleaved, int l) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int d = (j < 4 ? 0 : D / 2 - 4) + 4 * l + j;
      int i = interleaved ? d >> 1 : (d < R / 2 ? d : d - R / 2);
      f[j] = d < R || FULL ? static_cast<double>(inv_freq[i]) * 0.15915494309189535 : 0.0;
    }
  }
  __device__ __forceinline__ void at(int pos) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      double t = static_cast<double>(pos) * f[j];
      t -= rint(t);
      sincospif(2.f * static_cast<float>(t), &s[j], &c[j]);
    }
  }
  __device__ __forceinline__ void apply(float* e, int R, bool interleaved, int l) const {
    if constexpr (FULL) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = e[j], b = e[j + 4];
        e[j] = a * c[j] - b * s[j];
        e[j + 4] = b * c[j] + a * s[j];
      }
    } else if (interleaved) {  // unrotated pairs have f = 0: cos 1, sin 0
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float a = e[j], b = e[j + 1];
        e[j] = a * c[j] - b * s[j];
        e[j + 1] = b * c[j] + a * s[j];
      }
    } else {
      // the partner of 4-dim group p is p + R/8 (first half) or p - R/8; it
      // sits in element group (q >= D/8) of lane q mod D/8
      const int np = R / 8;
      float other[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = h * (D / 8) + l;
        const int q = p < np ? p + np : (p < 2 * np ? p - np : p);
        const int src = ((threadIdx.x & 31) & ~(D / 8 - 1)) + (q & (D / 8 - 1));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float o0 = __shfl_sync(0xffffffffu, e[j], src), o1 = __shfl_sync(0xffffffffu, e[4 + j], src);
          other[4 * h + j] = q < D / 8 ? o0 : o1;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = (j < 4 ? 0 : D / 8) + l;
        if (p < 2 * np) e[j] = fmaf(p < np ? -other[j] : other[j], s[j], e[j] * c[j]);
      }
    }
  }
};

__device__ __forceinline__ uint32_t encode4(const float* e, float inv, int kv_type) {
  if (kv_type == SD_KV_INT8) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = max(-127, min(127, __float2int_rn(e[j] * inv)));  // NaN converts to 0
      w |= (static_cast<uint32_t>(c) & 0xffu) << (8 * j);
    }
    return w;
  }
  float z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    z[j] = e[j] * inv;
    z[j] = z[j] == z[j] ? z[j] : 0.f;
  }
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(z[0], z[1]), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z[2], z[3]), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ void decode4(uint32_t w, int kv_type, float* e) {
  if (kv_type == SD_KV_INT8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = static_cast<float>(static_cast<int8_t>((w >> (8 * j)) & 0xffu));
  } else {
    const __half2 lo(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3));
    const __half2 hi(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3));
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    e[0] = a.x, e[1] = a.y, e[2] = b.x, e[3] = b.y;
  }
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.f;
}

// Codes of rows [0, n) at row pitch G * D re-scaled by ratio < 1.
__device__ __forceinline__ void recode_rows(uint8_t* first, long long pitch, int n, int D, float ratio, int kv_type) {
  const int per_row = D / 16;
  for (int i = threadIdx.x; i < n * per_row; i += kKvThreads) {
    uint4* at = reinterpret_cast<uint4*>(first + (i / per_row) * pitch + (i % per_row) * 16);
    uint4 w = *at;
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float e[4];
      decode4(u[j], kv_type, e);
      u[j] = encode4(e, ratio, kv_type);
    }
    *at = w;
  }
}

template <int D>
__device__ __forceinline__ void store_row(void* pages, long long row, int l, const float* e, float inv, int kv_type) {
  if (kv_type == SD_KV_BF16) {
    __nv_bfloat16* at = static_cast<__nv_bfloat16*>(pages) + row * D;
    *reinterpret_cast<uint2*>(at + 4 * l) = make_uint2(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]));
    *reinterpret_cast<uint2*>(at + D / 2 + 4 * l) = make_uint2(pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7]));
  } else {
    uint8_t* at = static_cast<uint8_t*>(pages) + row * D;
    *reinterpret_cast<uint32_t*>(at + 4 * l) = encode4(e, inv, kv_type);
    *reinterpret_cast<uint32_t*>(at + D / 2 + 4 * l) = encode4(e + 4, inv, kv_type);
  }
}

// The new tokens of request b are rows tok_start[b] .. tok_start[b + 1] - 1, at
// positions seqlen - n .. seqlen - 1. Returns the position of row r.
__device__ __forceinline__ int row_position(const KvStoreArgs& a, int b, int r, int* first_row, int* p0, int* p1) {
  const int L = checked_seqlen(a.seqlens, b, a.cap);
  const int r0 = a.tok_start[b], n = a.tok_start[b + 1] - r0;
  if (n > L) raise_error(SD_DEVERR_INDEX);  // more new tokens than the request holds
  *first_row = r0;
  *p0 = L - n;
  *p1 = L;
  return L - n + (r - r0);
}

template <int D, bool FULL>
__device__ void store_queries(const KvStoreArgs& a) {
  constexpr int LANES = D / 8, GROUPS = kKvThreads / LANES;
  const int l = threadIdx.x % LANES;
  const long long item = (long long)(blockIdx.x - a.kv_ctas) * GROUPS + threadIdx.x / LANES;
  const int token = static_cast<int>(item / a.head_groups), hg = static_cast<int>(item % a.head_groups);
  const bool in = token < a.T;
  const int b = find_request<LANES>(a.tok_start, a.B, in ? token : 0, l);
  const bool ok = in && token >= a.tok_start[0] && token < a.tok_start[a.B];
  int pos = 0;
  if (ok) {
    int r0, p0, p1;
    pos = row_position(a, b, token, &r0, &p0, &p1);
    if (a.positions != nullptr) pos = a.positions[token];
  }
  Rotation<D, FULL> rot;
  rot.init(a.inv_freq, a.R, a.interleaved, l);
  rot.at(pos);
  float w[8];
  if (a.qw != nullptr) load_weight<D>(a.qw, l, w);
  const int h0 = hg * a.heads_per_group, h1 = min(a.H, h0 + a.heads_per_group);
  const __nv_bfloat16* src = a.q + token * a.q_stride + 4 * l;
  __nv_bfloat16* dst = a.q_out + (long long)token * a.H * D;
  // the loop bound is the same for every group of a warp (shuffles inside)
  for (int i = 0; i < a.heads_per_group; i += kKvQHeads) {
    uint2 x[kKvQHeads], y[kKvQHeads];
#pragma unroll
    for (int j = 0; j < kKvQHeads; ++j) {
      const int h = h0 + i + j;
      x[j] = y[j] = make_uint2(0u, 0u);
      if (ok && h < h1 && i + j < a.heads_per_group) {
        x[j] = *reinterpret_cast<const uint2*>(src + (long long)h * D);
        y[j] = *reinterpret_cast<const uint2*>(src + (long long)h * D + D / 2);
      }
    }
#pragma unroll
    for (int j = 0; j < kKvQHeads; ++j) {
      const int h = h0 + i + j;
      float e[8];
      unpack_row<D>(x[j], y[j], e);
      if (a.qw != nullptr) norm_row<D>(e, w, a.eps);
      if (a.R > 0) rot.apply(e, a.R, a.interleaved, l);
      if (ok && h < h1 && i + j < a.heads_per_group) store_row<D>(dst, h, l, e, 1.f, SD_KV_BF16);
    }
  }
}

template <int D, bool FULL>
__device__ void store_block(const KvStoreArgs& a) {
  constexpr int LANES = D / 8, RPP = kKvThreads / LANES, PASSES = kKvMaxBlock / RPP;
  __shared__ int s_unit[2];
  __shared__ int s_scan[kKvThreads / 32];
  __shared__ float s_amax[2][kKvThreads / 32];
  __shared__ float s_bounds[2][kKvThreads / 32][D];
  const KvGeom& geo = a.geo;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid % LANES;
  const int unit = blockIdx.x / geo.G, g = blockIdx.x % geo.G, bs = geo.bs;

  // ---- which request and block this unit is ----
  int b, c, r0, p0, p1;  // block c of request b; its first new row and its new positions [p0, p1)
  if (a.by_row) {
    b = find_request<32>(a.tok_start, a.B, unit, lane);
    if (unit < a.tok_start[0] || unit >= a.tok_start[a.B]) return;
    const int p = row_position(a, b, unit, &r0, &p0, &p1);
    if (p < 0) return;
    c = geo.bs_div.div(p);
    if (p != c * bs && unit != r0 && p != 0) return;  // the block belongs to an earlier row
  } else {
    if (tid == 0) s_unit[0] = -1;
    int before = 0;
    for (int base = 0; base < a.B; base += kKvThreads) {
      const int i = base + tid;
      int n = 0;
      if (i < a.B) {
        int fr, q0, q1;
        row_position(a, i, 0, &fr, &q0, &q1);
        q0 = max(q0, 0);
        n = q1 > q0 ? geo.bs_div.div(q1 - 1) - geo.bs_div.div(q0) + 1 : 0;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      int skip = before, all = 0;
      for (int w = 0; w < kKvThreads / 32; ++w) {
        skip += w < warp ? s_scan[w] : 0;
        all += s_scan[w];
      }
      const int e = skip + incl;
      if (unit < e && unit >= e - n) s_unit[0] = i, s_unit[1] = unit - (e - n);
      before += all;
      __syncthreads();
      if (s_unit[0] >= 0) break;
    }
    if (s_unit[0] < 0) return;
    b = s_unit[0];
    row_position(a, b, 0, &r0, &p0, &p1);
    c = geo.bs_div.div(max(p0, 0)) + s_unit[1];
  }
  const int lo = max(max(p0, 0), c * bs), hi = min(p1, c * bs + bs);
  const int row0 = r0 + (lo - p0);
  const int nr = min(hi - lo, a.T - row0);
  if (row0 < 0 || nr <= 0) {
    if (tid == 0) raise_error(SD_DEVERR_INDEX);
    return;
  }
  const int pi = geo.page_div.div(c * bs);
  const int page = a.block_table[(size_t)b * geo.max_pages + pi];
  if (page < 0 || page >= geo.num_pages) {
    if (tid == 0) raise_error(SD_DEVERR_PAGE);
    return;
  }
  const int slot0 = c * bs - pi * geo.page_size;                 // the block's first slot
  const long long blk = ((long long)page * geo.blocks_per_page + geo.bs_div.div(slot0)) * geo.G + g;
  const long long row_base = (long long)page * geo.page_size + slot0;  // its pool row
  const bool earlier = lo > c * bs;

  // ---- load the new rows, norm and rotate K, find both maxima ----
  uint2 vx[PASSES], vy[PASSES];
  float e[PASSES][8];
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    const int i = ps * RPP + tid / LANES;
    uint2 x = make_uint2(0u, 0u), y = x;
    vx[ps] = vy[ps] = x;
    if (ps * RPP < nr && i < nr) {
      const __nv_bfloat16* ks = a.k + (row0 + i) * a.k_stride + (long long)g * D + 4 * l;
      const __nv_bfloat16* vs = a.v + (row0 + i) * a.v_stride + (long long)g * D + 4 * l;
      x = *reinterpret_cast<const uint2*>(ks);
      y = *reinterpret_cast<const uint2*>(ks + D / 2);
      vx[ps] = *reinterpret_cast<const uint2*>(vs);
      vy[ps] = *reinterpret_cast<const uint2*>(vs + D / 2);
    }
    unpack_row<D>(x, y, e[ps]);
  }
  Rotation<D, FULL> rot;
  rot.init(a.inv_freq, a.R, a.interleaved, l);
  float w[8];
  if (a.kw != nullptr) load_weight<D>(a.kw, l, w);
  float mk = 0.f, mv = 0.f, bmin[8], bmax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) bmin[j] = INFINITY, bmax[j] = -INFINITY;
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    if (ps * RPP >= nr) break;
    const int i = ps * RPP + tid / LANES;
    if (a.kw != nullptr) norm_row<D>(e[ps], w, a.eps);
    if (a.R > 0) {
      rot.at(i < nr && a.positions != nullptr ? a.positions[row0 + i] : lo + i);
      rot.apply(e[ps], a.R, a.interleaved, l);
    }
    if (i < nr) {
      float v[8];
      unpack_row<D>(vx[ps], vy[ps], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mk = fmaxf(mk, finite_abs(e[ps][j]));
        mv = fmaxf(mv, finite_abs(v[j]));
        const float kb = __bfloat162float(__float2bfloat16_rn(e[ps][j]));
        bmin[j] = fminf(bmin[j], kb);
        bmax[j] = fmaxf(bmax[j], kb);
      }
    }
  }

  const bool quant = a.kv_type != SD_KV_BF16;
  float sk = 1.f, sv = 1.f;
  if (quant) {
    const float ok = earlier ? a.k_scales[blk] : 0.f, ov = earlier ? a.v_scales[blk] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    if (lane == 0) s_amax[0][warp] = mk, s_amax[1][warp] = mv;
    __syncthreads();  // also: every thread has read the old scales
    for (int i = 0; i < kKvThreads / 32; ++i) mk = fmaxf(mk, s_amax[0][i]), mv = fmaxf(mv, s_amax[1][i]);
    const float qmax = a.kv_type == SD_KV_INT8 ? 127.f : 448.f;
    sk = fmaxf(fmaxf(mk / qmax, kKvMinScale), ok);
    sv = fmaxf(fmaxf(mv / qmax, kKvMinScale), ov);
    if (earlier) {
      const long long at = (row_base * geo.G + g) * D, pitch = (long long)geo.G * D;
      if (sk > ok) recode_rows(static_cast<uint8_t*>(a.k_pages) + at, pitch, lo - c * bs, D, ok / sk, a.kv_type);
      if (sv > ov) recode_rows(static_cast<uint8_t*>(a.v_pages) + at, pitch, lo - c * bs, D, ov / sv, a.kv_type);
    }
    if (tid == 0) a.k_scales[blk] = sk, a.v_scales[blk] = sv;
  }
  const float ik = 1.f / sk, iv = 1.f / sv;
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    const int i = ps * RPP + tid / LANES;
    if (i >= nr) break;
    const long long row = (row_base + (lo - c * bs) + i) * geo.G + g;
    store_row<D>(a.k_pages, row, l, e[ps], ik, a.kv_type);
    float v[8];
    unpack_row<D>(vx[ps], vy[ps], v);
    store_row<D>(a.v_pages, row, l, v, iv, a.kv_type);
  }
  if (a.bounds == nullptr) return;
#pragma unroll
  for (int o = LANES; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bmin[j] = fminf(bmin[j], __shfl_xor_sync(0xffffffffu, bmin[j], o));
      bmax[j] = fmaxf(bmax[j], __shfl_xor_sync(0xffffffffu, bmax[j], o));
    }
  }
  if (lane < LANES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = (j < 4 ? 0 : D / 2 - 4) + 4 * l + j;
      s_bounds[0][warp][d] = bmin[j];
      s_bounds[1][warp][d] = bmax[j];
    }
  }
  __syncthreads();
  if (tid < 2 * D) {
    const int which = tid / D, d = tid % D;
    __nv_bfloat16* at = a.bounds + (blk * 2 + which) * D + d;
    float x = s_bounds[which][0][d];
    for (int i = 1; i < kKvThreads / 32; ++i) x = which ? fmaxf(x, s_bounds[1][i][d]) : fminf(x, s_bounds[0][i][d]);
    if (earlier) {
      const float old = __bfloat162float(*at);
      x = which ? fmaxf(x, old) : fminf(x, old);
    }
    *at = __float2bfloat16_rn(x);
  }
}

template <int D, bool FULL>
__global__ void __launch_bounds__(kKvThreads) kv_store_kernel(const __grid_constant__ KvStoreArgs a) {
  pdl_wait();  // inputs come from earlier work in the stream
  pdl_trigger();
  if (blockIdx.x < a.kv_ctas) store_block<D, FULL>(a);
  else store_queries<D, FULL>(a);
}

// Reads the tokens that a store with the same tok_start and seqlens wrote back
// as bf16 rows [T, G, D]: code * scale, rounded once. One warp per token, a
// 16-element piece per lane and step. Bound by HBM.
struct KvLoadArgs {
  const void *k_pages, *v_pages;
  const float *k_scales, *v_scales;
  const int32_t *tok_start, *block_table, *seqlens;
  KvGeom geo;
  int kv_type, B, T, D, cap;
  __nv_bfloat16 *k_out, *v_out;
};

__global__ void __launch_bounds__(kKvThreads) kv_load_kernel(const __grid_constant__ KvLoadArgs a) {
  pdl_wait();  // inputs come from earlier work in the stream
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int token = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  if (token >= a.T) return;
  const int b = find_request<32>(a.tok_start, a.B, token, lane);
  if (token < a.tok_start[0] || token >= a.tok_start[a.B]) return;
  const int L = checked_seqlen(a.seqlens, b, a.cap);
  const int p = L - (a.tok_start[b + 1] - token);
  const KvGeom& geo = a.geo;
  long long row = -1, blk = 0;
  if (p < 0) {
    raise_error(SD_DEVERR_INDEX);
  } else {
    const int pi = geo.page_div.div(p);
    const int page = a.block_table[(size_t)b * geo.max_pages + pi];
    if (page < 0 || page >= geo.num_pages) {
      raise_error(SD_DEVERR_PAGE);
    } else {
      const int slot = p - pi * geo.page_size;
      row = (long long)page * geo.page_size + slot;
      blk = (long long)page * geo.blocks_per_page + geo.bs_div.div(slot);
    }
  }
  const int per_head = a.D / 16, n = geo.G * per_head;
  for (int i = lane; i < 2 * n; i += 32) {
    const bool is_v = i >= n;
    const int piece = is_v ? i - n : i;
    uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (row >= 0) {
      const long long at = row * geo.G * a.D + piece * 16;
      const void* pages = is_v ? a.v_pages : a.k_pages;
      if (a.kv_type == SD_KV_BF16) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pages) + at);
        o[0] = src[0], o[1] = src[1];
      } else {
        const float s = (is_v ? a.v_scales : a.k_scales)[blk * geo.G + piece / per_head];
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pages) + at);
        const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
        uint32_t* r = reinterpret_cast<uint32_t*>(o);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float e[4];
          decode4(u[j], a.kv_type, e);
          r[2 * j] = pack_bf16x2(e[0] * s, e[1] * s);
          r[2 * j + 1] = pack_bf16x2(e[2] * s, e[3] * s);
        }
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? a.v_out : a.k_out) + (long long)token * geo.G * a.D + piece * 16);
    dst[0] = o[0], dst[1] = o[1];
  }
}

}  // namespace sd
