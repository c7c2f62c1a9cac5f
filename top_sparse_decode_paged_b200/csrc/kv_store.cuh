// Writing tokens into a blocked paged cache: the norm of every query and key
// head, the position rotation, and the store of K and V, in one pass.
//
// For a head row x [D] of the token at position p (fp32 throughout):
//   y = x * rsqrt(mean(x^2) + eps) * w          (skipped where w is null)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = p * inv_freq[i],
//   over the pairs (i, i + R/2), or (2i, 2i + 1), of the first R dims.
// The angle is taken in turns, with the frequency as a 64-bit fixed-point
// fraction of a turn: position times frequency modulo one turn is an integer
// product modulo 2^64. The frequency comes from an fp64 product, off by 2^-54
// turns at a frequency of one radian, so the angle is as exact as one in fp64
// (2^-24 turns at position 2^30), where a far position times a frequency in
// fp32 keeps only a few bits of its fraction. q is rounded once to bf16. K and
// V go into a bf16, int8 or e4m3 pool. An 8-bit pool is cut into blocks of `bs`
// consecutive slots (a page holds whole blocks); a block and KV head have one
// scale for K and one for V:
//   s = max(amax(new rows) / qmax, s of the block's earlier rows, 2^-100)
// with qmax 127 or 448, codes round(y / s), and the earlier rows of a block
// whose scale grew coded anew, round(code * (s_old / s_new)). A growing scale
// costs an earlier row one more rounding each time it grows, and never
// clips a later token. Entries that are not finite do not enter the scale:
// NaN is coded as 0, infinities as the largest code.
// The block's bounds (smallest and largest bf16(y) of K for every dim) are
// what the block selection reads.
//
// Work split, one launch. K and V: the scale needs all of a block's new rows
// before any is coded. A prompt gets one CTA per (touched block, KV head),
// which keeps the rotated rows in shared memory in between; a decode step one
// warp per (token, KV head), K in one part of its lanes and V in the other, and
// units of several rows fall back to the whole CTA. q: one group of D / 8 lanes
// per (token, group of heads); the token's angles are computed once per group
// and used for its heads. 32 query heads over 8 KV heads of 128: four prompts
// into int8 (212 MB of q, 42.5 M instructions) 63.7 us, three prompts into bf16
// 32.8 us, bound by the chains of dependent steps at 24 warps per SM (issue
// slots 66 and 62 % used, HBM 37 % in int8, waits for loads the first stall);
// one token 3.7 us and 64 tokens 4.6 us, bound by launch and load latency.
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
  int kv_ctas, q_ctas, heads_per_group, head_groups;
  bool by_row;  // unit u is row u (where every row can start a block), else the u-th touched block
};

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The largest b in [0, B) with tok_start[b] <= r, by the LANES lanes of a
// group together: one load a lane and step. l is the lane in its group.
template <int LANES>
__device__ __forceinline__ int find_request(const int32_t* tok_start, int B, int r, int l) {
  // in a decode step row r is request r's only one: one load settles that
  const int guess = min(r, B - 1);
  if (__all_sync(0xffffffffu, tok_start[guess] <= r && r < tok_start[guess + 1])) return guess;
  const int base = (threadIdx.x & 31) & ~(LANES - 1);
  int lo = 0;
#pragma unroll 1
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

// Sine and cosine of t * 2^-32 turns: the nearest quarter turn is taken off in
// integers, and on the rest, at most an eighth of a turn, the Taylor sums to
// x^9 and x^8 are off by less than 2^-25.
__device__ __forceinline__ void sin_cos_turns(uint32_t t, float* s, float* c) {
  const uint32_t u = t + 0x20000000u;  // quarter in bits 31, 30; rest + 1/8 below
  const float x = static_cast<float>(static_cast<int>(u & 0x3fffffffu) - 0x20000000) * 1.4629180792671596e-9f;  // 2 pi 2^-32
  const float x2 = x * x;
  const float sn = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float cs = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const bool odd = u & 0x40000000u;
  *s = __uint_as_float(__float_as_uint(odd ? cs : sn) ^ (u & 0x80000000u));
  *c = __uint_as_float(__float_as_uint(odd ? sn : cs) ^ ((u + 0x40000000u) & 0x80000000u));
}

// Cosine and sine for a lane's elements. FULL: every dim is rotated in pairs
// (i, i + D/2), and elements j and j + 4 share an angle.
template <int D, bool FULL>
struct Rotation {
  static constexpr int N = FULL ? 4 : 8;
  unsigned long long f[N];  // turns per position, modulo one turn, in units of 2^-64 (0: not rotated)
  float c[N], s[N];

  __device__ __forceinline__ void init(const float* inv_freq, int R, bool interleaved, int l) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int d = (j < 4 ? 0 : D / 2 - 4) + 4 * l + j;
      const int i = interleaved ? d >> 1 : (d < R / 2 ? d : d - R / 2);
      f[j] = 0;
      if (d < R) {
        const double t = static_cast<double>(inv_freq[i]) * 0.15915494309189535;  // 1 / (2 pi)
        const double u = (t - floor(t)) * 18446744073709551616.0;                 // [0, 2^64]
        f[j] = u < 18446744073709551616.0 ? __double2ull_rn(u) : 0ull;
      }
    }
  }
  __device__ __forceinline__ void at(int pos) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * f[j];
      sin_cos_turns(static_cast<uint32_t>(t >> 32), &s[j], &c[j]);
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

// Codes are round(y / s) of the fp32 quotient: bf16 values divided by a scale
// that came from one of them meet exact ties, and y * (1 / s), one rounding
// more, sends some of them to the wrong neighbour.
//
// Four codes round(e / s), any input: NaN is 0, infinities the largest code.
__device__ __noinline__ uint32_t encode4_any(float e0, float e1, float e2, float e3, float s, int kv_type) {
  const float e[4] = {e0, e1, e2, e3};
  if (kv_type == SD_KV_INT8) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = max(-127, min(127, __float2int_rn(e[j] / s)));  // NaN converts to 0
      w |= (static_cast<uint32_t>(c) & 0xffu) << (8 * j);
    }
    return w;
  }
  float z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    z[j] = e[j] / s;
    z[j] = z[j] == z[j] ? z[j] : 0.f;
  }
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(z[0], z[1]), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z[2], z[3]), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Four codes of z, finite and in int8 at most 127 in magnitude: adding 1.5 *
// 2^23 rounds to a whole number (to even) whose low byte is the code.
__device__ __forceinline__ uint32_t round4(const float* z, int kv_type) {
  if (kv_type == SD_KV_INT8) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(__fadd_rn(z[j], 12582912.f));
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  }
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(z[0], z[1]), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z[2], z[3]), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Whether encode4_finite holds for this scale: its products stay normal.
__device__ __forceinline__ bool plain_scale(float s) { return s >= 8.67361738e-19f && s <= 1.2676506e30f; }  // 2^-60, 2^100

// The codes of encode4_any for finite e and a plain scale, inv = 1 / s. The
// quotient by one residual step (P. Markstein, IBM J. Res. Dev. 34, 1990): q =
// e * inv is off by two units at most, e - q s is exact but for its last bit,
// and what it adds leaves an error of 2^-22 units before the last rounding, so
// that a quotient that is an fp32 number, an exact tie among them, comes out as that
// number. (One that is below 2^-11 loses its residual's low bits, and rounds to
// code 0 all the same.)
__device__ __forceinline__ uint32_t encode4_finite(const float* e, float s, float inv, int kv_type) {
  float z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float q = __fmul_rn(e[j], inv);
    z[j] = __fmaf_rn(__fmaf_rn(-q, s, e[j]), inv, q);
  }
  return round4(z, kv_type);
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

// Codes of rows [0, n), `pitch` bytes apart, scaled by ratio < 1, by `threads`
// threads of which this is number `i0`.
__device__ __noinline__ void recode_rows(uint8_t* first, long long pitch, int n, int D, float ratio, int kv_type, int i0,
                                            int threads) {
  const int per_row = D / 16;
#pragma unroll 2
  for (int i = i0; i < n * per_row; i += threads) {
    uint4* at = reinterpret_cast<uint4*>(first + (i / per_row) * pitch + (i % per_row) * 16);
    uint4 w = *at;
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float e[4];
      decode4(u[j], kv_type, e);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = __fmul_rn(e[i], ratio);
      u[j] = round4(e, kv_type);
    }
    *at = w;
  }
}

template <int D, bool FINITE = false>
__device__ __forceinline__ void store_row(void* pages, long long row, int l, const float* e, float s, float inv, int kv_type) {
  if (kv_type == SD_KV_BF16) {
    __nv_bfloat16* at = static_cast<__nv_bfloat16*>(pages) + row * D;
    *reinterpret_cast<uint2*>(at + 4 * l) = make_uint2(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]));
    *reinterpret_cast<uint2*>(at + D / 2 + 4 * l) = make_uint2(pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7]));
  } else {
    uint8_t* at = static_cast<uint8_t*>(pages) + row * D;
    *reinterpret_cast<uint32_t*>(at + 4 * l) = FINITE ? encode4_finite(e, s, inv, kv_type) : encode4_any(e[0], e[1], e[2], e[3], s, kv_type);
    *reinterpret_cast<uint32_t*>(at + D / 2 + 4 * l) = FINITE ? encode4_finite(e + 4, s, inv, kv_type) : encode4_any(e[4], e[5], e[6], e[7], s, kv_type);
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
__device__ void store_queries(const KvStoreArgs& a, int cta) {
  constexpr int LANES = D / 8, GROUPS = kKvThreads / LANES;
  const int l = threadIdx.x % LANES;
  const int item = cta * GROUPS + threadIdx.x / LANES;
  const int token = item / a.head_groups, hg = item - token * a.head_groups;
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
#pragma unroll 1
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
      if (ok && h < h1 && i + j < a.heads_per_group) store_row<D>(dst, h, l, e, 1.f, 1.f, SD_KV_BF16);
    }
  }
}

// One touched block of a request, under one KV head.
struct KvUnit {
  int b, c;        // request, block
  int row0, nr;    // its first new row and how many
  int lo;          // position of the first
  long long blk;   // index of its scales and bounds
  long long base;  // its first pool row
  bool ok;
};

// Block c of request b with new positions [p0, p1), whose first is row r0.
// `raise`: whether this thread reports bad data. `begin(row0, nr)` is called
// before the page is looked up.
template <class Begin>
__device__ __forceinline__ KvUnit make_unit(const KvStoreArgs& a, int b, int c, int r0, int p0, int p1, int g, bool raise, Begin begin) {
  const KvGeom& geo = a.geo;
  KvUnit u;
  u.b = b, u.c = c, u.ok = false;
  u.lo = max(max(p0, 0), c * geo.bs);
  u.row0 = r0 + (u.lo - p0);
  u.nr = min(min(p1, c * geo.bs + geo.bs) - u.lo, a.T - u.row0);
  u.blk = u.base = 0;
  if (u.row0 < 0 || u.nr <= 0) {
    if (raise) raise_error(SD_DEVERR_INDEX);
    return u;
  }
  begin(u.row0, u.nr);
  const int pi = geo.page_div.div(c * geo.bs);
  const int page = a.block_table[(size_t)b * geo.max_pages + pi];
  if (page < 0 || page >= geo.num_pages) {
    if (raise) raise_error(SD_DEVERR_PAGE);
    return u;
  }
  const int slot0 = c * geo.bs - pi * geo.page_size;
  u.blk = ((long long)page * geo.blocks_per_page + geo.bs_div.div(slot0)) * geo.G + g;
  u.base = (long long)page * geo.page_size + slot0;
  u.ok = true;
  return u;
}

template <int D>
struct KvBlockSmem {
  uint32_t amax[2][kKvThreads / 32];
  __nv_bfloat16 bounds[2][kKvThreads / 32][D];
  int scan[kKvThreads / 32];
  int unit[2];
  KvUnit units[kKvThreads / 32];
};

// The new rows of a unit, K and V, on their way to shared memory. A lane
// copies what it reads later, so its own wait is all that is needed: its K
// elements go to where their fp32 values will stand.
template <int D>
__device__ __forceinline__ void copy_unit_rows(const KvStoreArgs& a, int row0, int nr, int g, float* rows, __nv_bfloat16* vrows) {
  constexpr int LANES = D / 8, RPP = kKvThreads / LANES;
  const int l = threadIdx.x % LANES;
  const __nv_bfloat16* ks = a.k + row0 * a.k_stride + (long long)g * D + 4 * l;
  const __nv_bfloat16* vs = a.v + row0 * a.v_stride + (long long)g * D + 4 * l;
#pragma unroll 1
  for (int i = threadIdx.x / LANES; i < nr; i += RPP) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(rows + i * D + h * (D / 2) + 4 * l)),
                   "l"(ks + i * a.k_stride + h * (D / 2)) : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(vrows + i * D + h * (D / 2) + 4 * l)),
                   "l"(vs + i * a.v_stride + h * (D / 2)) : "memory");
    }
  }
  cp_async_commit();
}

// A unit of any number of rows, by the whole CTA, once its rows are under way
// to `rows` (block_tokens x D floats) and `vrows` (as many bf16).
template <int D, bool FULL>
__device__ void store_unit_cta(const KvStoreArgs& a, const KvUnit u, int g, KvBlockSmem<D>& sm, float* rows, __nv_bfloat16* vrows) {
  constexpr int LANES = D / 8, RPP = kKvThreads / LANES;
  const KvGeom& geo = a.geo;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid % LANES, bs = geo.bs;
  const bool earlier = u.lo > u.c * bs, quant = a.kv_type != SD_KV_BF16;
  const float old_k = earlier && quant ? a.k_scales[u.blk] : 0.f, old_v = earlier && quant ? a.v_scales[u.blk] : 0.f;
  Rotation<D, FULL> rot;
  rot.init(a.inv_freq, a.R, a.interleaved, l);
  float w[8];
  if (a.kw != nullptr) load_weight<D>(a.kw, l, w);
  // largest magnitudes as bits (of fp32 for K, of bf16 pairs for V): those of
  // entries that are not finite are above all others
  uint32_t mk = 0u, mv = 0u;
  __nv_bfloat162 bmin[4], bmax[4];  // of bf16(y); NaN drops out
#pragma unroll
  for (int j = 0; j < 4; ++j) bmin[j] = __float2bfloat162_rn(INFINITY), bmax[j] = __float2bfloat162_rn(-INFINITY);
  cp_async_wait<0>();
#pragma unroll 1
  for (int i0 = 0; i0 < u.nr; i0 += RPP) {
    const int i = i0 + tid / LANES;
    const bool in = i < u.nr;
    float* at = rows + i * D + 4 * l;
    const __nv_bfloat16* vat = vrows + i * D + 4 * l;
    uint2 x = make_uint2(0u, 0u), y = x, vx = x, vy = x;
    if (in) {
      x = *reinterpret_cast<const uint2*>(at);
      y = *reinterpret_cast<const uint2*>(at + D / 2);
      vx = *reinterpret_cast<const uint2*>(vat);
      vy = *reinterpret_cast<const uint2*>(vat + D / 2);
    }
    float e[8];
    unpack_row<D>(x, y, e);
    if (a.kw != nullptr) norm_row<D>(e, w, a.eps);
    if (a.R > 0) {
      rot.at(in && a.positions != nullptr ? a.positions[u.row0 + i] : u.lo + i);
      rot.apply(e, a.R, a.interleaved, l);
    }
    if (in) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mk = max(mk, max(__float_as_uint(e[2 * j]) & 0x7fffffffu, __float_as_uint(e[2 * j + 1]) & 0x7fffffffu));
        const __nv_bfloat162 kb = __floats2bfloat162_rn(e[2 * j], e[2 * j + 1]);
        bmin[j] = __hmin2(bmin[j], kb);
        bmax[j] = __hmax2(bmax[j], kb);
      }
      mv = __vmaxu2(mv, __vmaxu2(__vmaxu2(vx.x & 0x7fff7fffu, vx.y & 0x7fff7fffu), __vmaxu2(vy.x & 0x7fff7fffu, vy.y & 0x7fff7fffu)));
      if (quant) {
        *reinterpret_cast<float4*>(at) = make_float4(e[0], e[1], e[2], e[3]);
        *reinterpret_cast<float4*>(at + D / 2) = make_float4(e[4], e[5], e[6], e[7]);
      } else {
        const long long row = (u.base + (u.lo - u.c * bs) + i) * geo.G + g;
        store_row<D>(a.k_pages, row, l, e, 1.f, 1.f, SD_KV_BF16);
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.v_pages) + row * D + 4 * l;
        *reinterpret_cast<uint2*>(dst) = vx;
        *reinterpret_cast<uint2*>(dst + D / 2) = vy;
      }
    }
  }
  if (quant) {
    mv = max(mv & 0xffffu, mv >> 16) << 16;
    mk = __reduce_max_sync(0xffffffffu, mk);
    mv = __reduce_max_sync(0xffffffffu, mv);
    if (lane == 0) sm.amax[0][warp] = mk, sm.amax[1][warp] = mv;
  }
  if (a.bounds != nullptr) {
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bmin[j] = __hmin2(bmin[j], __shfl_xor_sync(0xffffffffu, bmin[j], o));
        bmax[j] = __hmax2(bmax[j], __shfl_xor_sync(0xffffffffu, bmax[j], o));
      }
    }
    if (lane < LANES) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = (j < 2 ? 0 : D / 2 - 4) + 4 * l + 2 * j;
        *reinterpret_cast<__nv_bfloat162*>(&sm.bounds[0][warp][d]) = bmin[j];
        *reinterpret_cast<__nv_bfloat162*>(&sm.bounds[1][warp][d]) = bmax[j];
      }
    }
  }
  __syncthreads();  // also: every thread has read the old scales
  if (quant) {
    for (int i = 0; i < kKvThreads / 32; ++i) mk = max(mk, sm.amax[0][i]), mv = max(mv, sm.amax[1][i]);
    const bool finite = max(mk, mv) < 0x7f800000u;
    float fk = __uint_as_float(mk), fv = __uint_as_float(mv);
    if (!finite) {  // rare: the maxima of the finite entries alone
      fk = fv = 0.f;
#pragma unroll 1
      for (int i = 0; i < u.nr; ++i) {
#pragma unroll 1
        for (int d = lane; d < D; d += 32) {
          fk = fmaxf(fk, finite_abs(rows[i * D + d]));
          fv = fmaxf(fv, finite_abs(__bfloat162float(vrows[i * D + d])));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        fk = fmaxf(fk, __shfl_xor_sync(0xffffffffu, fk, o));
        fv = fmaxf(fv, __shfl_xor_sync(0xffffffffu, fv, o));
      }
    }
    const float qmax = a.kv_type == SD_KV_INT8 ? 127.f : 448.f;
    const float sk = fmaxf(fmaxf(fk / qmax, kKvMinScale), old_k), sv = fmaxf(fmaxf(fv / qmax, kKvMinScale), old_v);
    if (earlier) {
      const long long at = (u.base * geo.G + g) * D, pitch = (long long)geo.G * D;
      const int n = u.lo - u.c * bs;
      if (sk > old_k) recode_rows(static_cast<uint8_t*>(a.k_pages) + at, pitch, n, D, old_k / sk, a.kv_type, tid, kKvThreads);
      if (sv > old_v) recode_rows(static_cast<uint8_t*>(a.v_pages) + at, pitch, n, D, old_v / sv, a.kv_type, tid, kKvThreads);
    }
    if (tid == 0) a.k_scales[u.blk] = sk, a.v_scales[u.blk] = sv;
    const float ik = 1.f / sk, iv = 1.f / sv;
    const bool plain = finite && plain_scale(sk) && plain_scale(sv);
    const long long first = (u.base + (u.lo - u.c * bs)) * geo.G + g;
#pragma unroll 1
    for (int i = tid / LANES; i < u.nr; i += RPP) {
      const uint2 vx = *reinterpret_cast<const uint2*>(vrows + i * D + 4 * l);
      const uint2 vy = *reinterpret_cast<const uint2*>(vrows + i * D + D / 2 + 4 * l);
      const float4 x = *reinterpret_cast<const float4*>(rows + i * D + 4 * l);
      const float4 y = *reinterpret_cast<const float4*>(rows + i * D + D / 2 + 4 * l);
      const float e[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      const long long row = first + (long long)i * geo.G;
      float v[8];
      unpack_row<D>(vx, vy, v);
      if (plain) {
        store_row<D, true>(a.k_pages, row, l, e, sk, ik, a.kv_type);
        store_row<D, true>(a.v_pages, row, l, v, sv, iv, a.kv_type);
      } else {
        store_row<D>(a.k_pages, row, l, e, sk, ik, a.kv_type);
        store_row<D>(a.v_pages, row, l, v, sv, iv, a.kv_type);
      }
    }
  }
  if (a.bounds != nullptr && tid < D) {  // two dims of one bound each
    const int which = tid / (D / 2), d = 2 * (tid % (D / 2));
    __nv_bfloat162* at = reinterpret_cast<__nv_bfloat162*>(a.bounds + (u.blk * 2 + which) * D + d);
    __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&sm.bounds[which][0][d]);
#pragma unroll 1
    for (int i = 1; i < kKvThreads / 32; ++i) {
      const __nv_bfloat162 o = *reinterpret_cast<const __nv_bfloat162*>(&sm.bounds[which][i][d]);
      x = which ? __hmax2(x, o) : __hmin2(x, o);
    }
    if (earlier) x = which ? __hmax2(x, *at) : __hmin2(x, *at);
    *at = x;
  }
}

// A unit of one row, by one warp: lanes [0, D/8) hold K, [D/8, D/4) hold V.
template <int D, bool FULL>
__device__ void store_unit_warp(const KvStoreArgs& a, const KvUnit& u, int g, uint2 x, uint2 y) {
  constexpr int LANES = D / 8;
  const KvGeom& geo = a.geo;
  const int lane = threadIdx.x & 31, l = lane % LANES, bs = geo.bs;
  const bool is_v = lane / LANES == 1, live = lane < 2 * LANES;
  const bool earlier = u.lo > u.c * bs, quant = a.kv_type != SD_KV_BF16;
  float* scales = is_v ? a.v_scales : a.k_scales;
  void* pages = is_v ? a.v_pages : a.k_pages;
  const float old = earlier && quant ? scales[u.blk] : 0.f;
  uint2 ob[2][2];  // the block's bounds so far
  __nv_bfloat16* at = a.bounds + u.blk * 2 * D + 4 * l;
  if (a.bounds != nullptr && earlier && lane < LANES) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ob[i][0] = *reinterpret_cast<const uint2*>(at + i * D);
      ob[i][1] = *reinterpret_cast<const uint2*>(at + i * D + D / 2);
    }
  }
  float e[8], v[8];
  unpack_row<D>(x, y, e);
  unpack_row<D>(x, y, v);
  if (a.kw != nullptr) {
    float w[8];
    load_weight<D>(a.kw, l, w);
    norm_row<D>(e, w, a.eps);
  }
  if (a.R > 0) {
    Rotation<D, FULL> rot;
    rot.init(a.inv_freq, a.R, a.interleaved, l);
    rot.at(a.positions != nullptr ? a.positions[u.row0] : u.lo);
    rot.apply(e, a.R, a.interleaved, l);
  }
  float m = 0.f;
  bool finite = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    e[j] = is_v ? v[j] : e[j];
    m = fmaxf(m, finite_abs(e[j]));
    finite &= fabsf(e[j]) <= FLT_MAX;
  }
  float s = 1.f;
  if (quant) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float qmax = a.kv_type == SD_KV_INT8 ? 127.f : 448.f;
    s = fmaxf(fmaxf(m / qmax, kKvMinScale), old);
    if (earlier) {
      const float sk = __shfl_sync(0xffffffffu, s, 0), sv = __shfl_sync(0xffffffffu, s, LANES);
      const float ok = __shfl_sync(0xffffffffu, old, 0), ov = __shfl_sync(0xffffffffu, old, LANES);
      const long long first = (u.base * geo.G + g) * D, pitch = (long long)geo.G * D;
      const int n = u.lo - u.c * bs;
      if (sk > ok) recode_rows(static_cast<uint8_t*>(a.k_pages) + first, pitch, n, D, ok / sk, a.kv_type, lane, 32);
      if (sv > ov) recode_rows(static_cast<uint8_t*>(a.v_pages) + first, pitch, n, D, ov / sv, a.kv_type, lane, 32);
    }
    if (live && l == 0) scales[u.blk] = s;
  }
  const long long row = (u.base + (u.lo - u.c * bs)) * geo.G + g;
  if (live) {
    if (finite && plain_scale(s)) store_row<D, true>(pages, row, l, e, s, 1.f / s, a.kv_type);
    else store_row<D>(pages, row, l, e, s, 1.f, a.kv_type);
  }
  if (a.bounds == nullptr || lane >= LANES) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float z[8], o[8];
    unpack_row<D>(ob[i][0], ob[i][1], o);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[j] = __bfloat162float(__float2bfloat16_rn(e[j]));
      if (z[j] != z[j]) z[j] = i ? -INFINITY : INFINITY;  // a NaN key bounds nothing
      if (earlier) z[j] = i ? fmaxf(z[j], o[j]) : fminf(z[j], o[j]);
    }
    *reinterpret_cast<uint2*>(at + i * D) = make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
    *reinterpret_cast<uint2*>(at + i * D + D / 2) = make_uint2(pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
  }
}

// Units by row: warp w of the CTA takes (row, KV head) pair w, if the row is
// the first new one of its block.
template <int D, bool FULL>
__device__ void store_by_row(const KvStoreArgs& a, int cta, KvBlockSmem<D>& sm, float* rows, __nv_bfloat16* vrows) {
  constexpr int LANES = D / 8, kWarps = kKvThreads / 32;
  const KvGeom& geo = a.geo;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LANES;
  const int item = cta * kWarps + warp, row = item / geo.G, g = item - row * geo.G;
  KvUnit u;
  u.ok = false, u.nr = 0;
  uint2 x = make_uint2(0u, 0u), y = x;
  if (row < a.T) {
    const __nv_bfloat16* src = lane / LANES == 1 ? a.v + row * a.v_stride : a.k + row * a.k_stride;
    if (lane < 2 * LANES) {  // needed whether or not the row is the first of its block
      x = *reinterpret_cast<const uint2*>(src + (long long)g * D + 4 * l);
      y = *reinterpret_cast<const uint2*>(src + (long long)g * D + D / 2 + 4 * l);
    }
    const int b = find_request<32>(a.tok_start, a.B, row, lane);
    if (row >= a.tok_start[0] && row < a.tok_start[a.B]) {
      int r0, p0, p1;
      const int p = row_position(a, b, row, &r0, &p0, &p1);
      if (p >= 0 && p < p1) {
        const int c = geo.bs_div.div(p);
        if (p == c * geo.bs || row == r0) u = make_unit(a, b, c, r0, p0, p1, g, lane == 0, [](int, int) {});
      }
    }
  }
  if (u.ok && u.nr == 1) store_unit_warp<D, FULL>(a, u, g, x, y);
  // units of several rows (several tokens of a request among single ones)
  const bool many = u.ok && u.nr > 1;
  if (lane == 0) sm.units[warp] = u;
  if (!__syncthreads_or(many)) return;
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    const KvUnit v = sm.units[w];
    if (!v.ok || v.nr <= 1) continue;
    const int gw = (cta * kWarps + w) % geo.G;
    copy_unit_rows<D>(a, v.row0, v.nr, gw, rows, vrows);
    store_unit_cta<D, FULL>(a, v, gw, sm, rows, vrows);
    __syncthreads();  // its shared memory is free again
  }
}

// Units by touched block: unit u of the list over all requests, one CTA per
// KV head.
template <int D, bool FULL>
__device__ void store_by_block(const KvStoreArgs& a, int cta, KvBlockSmem<D>& sm, float* rows, __nv_bfloat16* vrows) {
  const KvGeom& geo = a.geo;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = cta / geo.G, g = cta % geo.G;
  int r0, p0, p1;
  if (tid == 0) sm.unit[0] = -1;
  int before = 0;
#pragma unroll 1
  for (int base = 0; base < a.B; base += kKvThreads) {
    const int i = base + tid;
    int n = 0;
    if (i < a.B) {
      row_position(a, i, 0, &r0, &p0, &p1);
      p0 = max(p0, 0);
      n = p1 > p0 ? geo.bs_div.div(p1 - 1) - geo.bs_div.div(p0) + 1 : 0;
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int skip = before, all = 0;
#pragma unroll 1
    for (int w = 0; w < kKvThreads / 32; ++w) {
      skip += w < warp ? sm.scan[w] : 0;
      all += sm.scan[w];
    }
    const int e = skip + incl;
    if (unit < e && unit >= e - n) sm.unit[0] = i, sm.unit[1] = unit - (e - n);
    before += all;
    __syncthreads();
    if (sm.unit[0] >= 0) break;
  }
  if (sm.unit[0] < 0) return;
  const int b = sm.unit[0];
  row_position(a, b, 0, &r0, &p0, &p1);
  const KvUnit u = make_unit(a, b, geo.bs_div.div(max(p0, 0)) + sm.unit[1], r0, p0, p1, g, tid == 0,
                             [&](int row0, int nr) { copy_unit_rows<D>(a, row0, nr, g, rows, vrows); });
  if (u.ok) store_unit_cta<D, FULL>(a, u, g, sm, rows, vrows);
  else cp_async_wait<0>();
}

template <int D, bool FULL>
__global__ void __launch_bounds__(kKvThreads, 3) kv_store_kernel(const __grid_constant__ KvStoreArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ KvBlockSmem<D> sm;
  pdl_wait();  // inputs come from earlier work in the stream
  pdl_trigger();
  float* rows = reinterpret_cast<float*>(smem_raw);
  __nv_bfloat16* vrows = reinterpret_cast<__nv_bfloat16*>(rows + a.geo.bs * D);
  // CTAs of both kinds evenly mixed: K and V are bound by issue slots and
  // latency, q by HBM
  const unsigned int all = a.kv_ctas + a.q_ctas;
  const int before = static_cast<int>((unsigned long long)blockIdx.x * a.q_ctas / all);
  const int cta = blockIdx.x - before;
  if (static_cast<int>((blockIdx.x + 1ull) * a.q_ctas / all) > before) store_queries<D, FULL>(a, before);
  else if (a.by_row) store_by_row<D, FULL>(a, cta, sm, rows, vrows);
  else store_by_block<D, FULL>(a, cta, sm, rows, vrows);
}

// Reads the tokens that a store with the same tok_start and seqlens wrote back
// as bf16 rows [T, G, D]: code * scale, rounded once. One warp per token, a
// 16-element piece per lane and step. The four prompts' int8 rows (65.8 MB) in
// 14.5 us after the store, 17.0 with cold caches, bound by each warp's chain
// page, scale, codes.
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
  if (p < 0 || p >= L) {
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
  constexpr int kBatch = 4;  // pieces a lane has in flight
#pragma unroll 1
  for (int i0 = lane; i0 < 2 * n; i0 += 32 * kBatch) {
    uint4 w[kBatch][2];
    float s[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + 32 * j, piece = i >= n ? i - n : i;
      w[j][0] = w[j][1] = make_uint4(0u, 0u, 0u, 0u);
      s[j] = 0.f;
      if (i < 2 * n && row >= 0) {
        const long long at = row * geo.G * a.D + piece * 16;
        const void* pages = i >= n ? a.v_pages : a.k_pages;
        if (a.kv_type == SD_KV_BF16) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pages) + at);
          w[j][0] = src[0], w[j][1] = src[1];
        } else {
          s[j] = (i >= n ? a.v_scales : a.k_scales)[blk * geo.G + piece / per_head];
          w[j][0] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pages) + at);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + 32 * j, piece = i >= n ? i - n : i;
      if (i >= 2 * n) break;
      if (a.kv_type != SD_KV_BF16 && row >= 0) {
        const uint32_t u[4] = {w[j][0].x, w[j][0].y, w[j][0].z, w[j][0].w};
        uint32_t r[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float e[4];
          decode4(u[k], a.kv_type, e);
          r[2 * k] = pack_bf16x2(e[0] * s[j], e[1] * s[j]);
          r[2 * k + 1] = pack_bf16x2(e[2] * s[j], e[3] * s[j]);
        }
        w[j][0] = make_uint4(r[0], r[1], r[2], r[3]);
        w[j][1] = make_uint4(r[4], r[5], r[6], r[7]);
      }
      uint4* dst = reinterpret_cast<uint4*>((i >= n ? a.v_out : a.k_out) + (long long)token * geo.G * a.D + piece * 16);
      dst[0] = w[j][0], dst[1] = w[j][1];
    }
  }
}

}  // namespace sd
