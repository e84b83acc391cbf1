// kv_device.hpp -- device-side pieces that the attention kernels over the
// paged 4-bit cache share: the launch parameters, the lane layout of cached
// rows and their decoding to matrix-core operands.
//
// A wave reads 16 cached rows (keys) at a time: lane l holds row l % 16 and a
// quarter l / 16 of its columns, which is the operand layout of the
// 16x16x32 product: a lane owns 8 consecutive columns of one row per step,
// and which columns a step pairs is free as long as both operands agree.
// Operands of S = K . Q^T:
//   NVFP4  fp16.  E2M1 * E4M3 has at most 6 significant bits and lies in
//          2^-10 .. 2688: exact.  The global scale is applied to the sums.
//   MXFP4  bf16, exact (a power of two times E2M1); the converter applies the
//          scale itself.
//   AFFINE the codes 0..15 themselves, exact in bf16; scale and bias are
//          applied to the fp32 sums per group.
// Operands of O = P . V are fp16 for every format: 11 significant bits for
// the probabilities, and for affine values, which do not fit 8.  NVFP4 values
// are exact; MXFP4 and affine values can leave fp16's range and are taken
// times 2^nb, with nb kept per quarter of the columns and lowered when a
// larger value comes (value_shift).
#pragma once

#include "bsfp_device.hpp"
#include "bsfp_internal.hpp"

namespace bsfp {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

struct KvSide {
  const uint8_t* codes;
  const uint8_t* scales;
  const uint8_t* biases;
  const float* g;
};

struct KvParams {
  const uint16_t* q;
  int64_t q_stride;
  int tokens, heads, kv_heads, group;  // group: query heads per kv head
  KvSide k, v;
  int64_t pages;
  int page_shift;
  const int32_t* table;
  int max_pages;
  const int32_t *kv_lens, *q_starts;
  int requests, max_q;
  float scale;  // times log2 e
  int window;
  uint16_t* out;
  float* lse;
};

__device__ __forceinline__ f32x4_t mma16_f16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}
// The product with keys: fp16 operands for NVFP4, bf16 for the others.
template <int MODE>
__device__ __forceinline__ f32x4_t mma16_keys(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (MODE == BSFP_NVFP4) return mma16_f16(a, b, c);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Two fp32 -> fp16, nearest even.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const f32x2_t f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2_t));
}

// ------------------------------------------------------- rows of the cache

// W words of codes: a lane's quarter of a row has D / 32.
template <int W>
struct Words { uint32_t w[W]; };

// Loads take a wave-uniform base (a run of 16 rows, 64-bit) and the lane's
// place r, qd in it, so the per-lane part of an address is a 32-bit constant.
// The lane's quarter of row r's codes: columns qd * D/4 ...
template <int D>
__device__ __forceinline__ Words<D / 32> load_codes(const uint8_t* base, int r, int qd) {
  Words<D / 32> o;
  const uint32_t at = (uint32_t)(r * (D / 2) + qd * (D / 8));
  if constexpr (D == 64) {
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(base + at);
    o.w[0] = v.x; o.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(base + at + 16 * i);
      o.w[4 * i] = v.x; o.w[4 * i + 1] = v.y; o.w[4 * i + 2] = v.z; o.w[4 * i + 3] = v.w;
    }
  }
  return o;
}

// The same for affine keys, whose products are kept apart by group of 64
// columns: words 2 g and 2 g + 1 are columns 64 g + 16 qd ...
template <int D>
__device__ __forceinline__ Words<D / 32> load_codes_by_group(const uint8_t* base, int r, int qd) {
  Words<D / 32> o;
#pragma unroll
  for (int g = 0; g < D / 64; ++g) {
    const u32x2_t v =
        *reinterpret_cast<const u32x2_t*>(base + (uint32_t)(r * (D / 2) + qd * 8) + g * 32);
    o.w[2 * g] = v.x; o.w[2 * g + 1] = v.y;
  }
  return o;
}

// Column of element 0 of the lane's word j.
template <int MODE, int D>
__device__ __forceinline__ int key_column(int j, int qd) {
  return MODE == BSFP_AFFINE ? (j >> 1) * 64 + qd * 16 + (j & 1) * 8 : qd * (D / 4) + j * 8;
}

// The scales of the lane's quarter of a row: NVFP4 D/64 bytes, MXFP4 one or
// two bytes, AFFINE scale (low half) and bias of the group they lie in.
// scales, biases: of the run's row 0.
template <int MODE, int D>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* scales, const uint8_t* biases, int r,
                                                int qd) {
  if constexpr (MODE == BSFP_NVFP4) {
    const uint8_t* p = scales + (uint32_t)(r * (D / 16) + qd * (D / 64));
    if constexpr (D == 64) return *p;
    else if constexpr (D == 128) return *reinterpret_cast<const uint16_t*>(p);
    else return *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (MODE == BSFP_MXFP4) {
    const uint8_t* p = scales + (uint32_t)(r * (D / 32) + qd * (D / 4) / 32);
    if constexpr (D == 256) return *reinterpret_cast<const uint16_t*>(p);
    else return *p;
  } else {
    const uint32_t at = (uint32_t)(r * (D / 64) + qd * (D / 4) / 64) * 2;
    return *reinterpret_cast<const uint16_t*>(scales + at) |
           (uint32_t)*reinterpret_cast<const uint16_t*>(biases + at) << 16;
  }
}
// Bytes of scales per row.
template <int MODE, int D>
constexpr int scale_bytes() { return MODE == BSFP_NVFP4 ? D / 16 : MODE == BSFP_MXFP4 ? D / 32 : D / 32; }

// NVFP4: word j of the lane's quarter (8 columns) as four fp16 pairs.
template <int D>
__device__ __forceinline__ u32x4_t decode_nvfp4(uint32_t w, uint32_t scales, int j) {
  const f16x2_t s2 = (j & 4) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, false);
  const _Float16 s1 = (j & 2) ? s2.y : s2.x;
  const f16x2_t s = {s1, s1};
  u32x4_t o;
  o.x = __builtin_bit_cast(uint32_t, e2m1x2_to_f16x2<0>(w) * s);
  o.y = __builtin_bit_cast(uint32_t, e2m1x2_to_f16x2<1>(w) * s);
  o.z = __builtin_bit_cast(uint32_t, e2m1x2_to_f16x2<2>(w) * s);
  o.w = __builtin_bit_cast(uint32_t, e2m1x2_to_f16x2<3>(w) * s);
  return o;
}

// The E8M0 byte of word j.
template <int D>
__device__ __forceinline__ int e8m0_byte(uint32_t scales, int j) {
  return (int)((D == 256 && (j & 4)) ? scales >> 8 : scales & 255u);
}

// Keys, NVFP4 and MXFP4: word j as four operand pairs in column order.
template <int MODE, int D>
__device__ __forceinline__ u32x4_t decode_key_word(uint32_t w, uint32_t scales, int j) {
  if constexpr (MODE == BSFP_NVFP4) return decode_nvfp4<D>(w, scales, j);
  const float s = e8m0_decode((uint32_t)e8m0_byte<D>(scales, j));
  u32x4_t o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return o;
}

// Values: word j as four fp16 pairs in column order; MXFP4 and affine ones
// times 2^nb.
template <int MODE, int D>
__device__ __forceinline__ u32x4_t decode_value_word(uint32_t w, uint32_t scales, int j, int nb) {
  u32x4_t o;
  if constexpr (MODE == BSFP_NVFP4) {
    return decode_nvfp4<D>(w, scales, j);
  } else if constexpr (MODE == BSFP_MXFP4) {
    const float s = __uint_as_float((uint32_t)max(e8m0_byte<D>(scales, j) + nb, 1) << 23);
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3));
  } else {
    const float f = __uint_as_float((uint32_t)(127 + nb) << 23);
    // scale and bias in fp16: 8 bits each, exact down to 2^-14, far below the
    // values, which stand around 2^8; the products are rounded once
    const _Float16 sh = (_Float16)(bf16_lo(scales) * f), bh = (_Float16)(bf16_hi(scales) * f);
    const f16x2_t s2 = {sh, sh}, b2 = {bh, bh};
    const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
    // nibbles as E4M3 bytes are code * 2^-9
    auto values = [&](f16x2_t c) {
      return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c, s2, b2));
    };
    const uint32_t v02 = values(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 512.0f, false));
    const uint32_t v46 = values(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 512.0f, true));
    const uint32_t v13 = values(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 512.0f, false));
    const uint32_t v57 = values(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 512.0f, true));
    o.x = __builtin_amdgcn_perm(v13, v02, 0x05040100u);
    o.y = __builtin_amdgcn_perm(v13, v02, 0x07060302u);
    o.z = __builtin_amdgcn_perm(v57, v46, 0x05040100u);
    o.w = __builtin_amdgcn_perm(v57, v46, 0x07060302u);
  }
  return o;
}

// The biased exponent of the lane's largest possible value (0 for a value
// that is not finite, which fp16 shows as such at any scale).
template <int MODE, int D>
__device__ __forceinline__ int value_exponent(uint32_t scales) {
  if constexpr (MODE == BSFP_MXFP4) {
    return D == 256 ? max((int)(scales & 255u), (int)(scales >> 8)) : (int)(scales & 255u);
  } else {
    const float s = bf16_lo(scales), b = bf16_hi(scales);
    const int e = (int)(__float_as_uint(fmaxf(fabsf(b), fabsf(__builtin_fmaf(15.0f, s, b)))) >> 23);
    return e == 255 ? 0 : e;
  }
}

// Values that are not finite: NVFP4 groups whose scale is E4M3's NaN, affine
// ones with a scale or bias that is not finite (kv_append writes such groups
// where the input holds an infinity, and all their values are NaN).  Bit 7 of
// byte j: of group j of the lane's quarter.  MXFP4 has none: every E8M0 byte
// is taken for a power of two.
// A probability of zero does not take such a value out of a sum, so in tiles
// with keys that some rows see and others do not, the values are taken as zero
// and the rows that see them get NaN in those columns.
template <int MODE>
__device__ __forceinline__ uint32_t not_finite(uint32_t scales) {
  if constexpr (MODE == BSFP_NVFP4) {
    return ((scales & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  } else if constexpr (MODE == BSFP_AFFINE) {
    const float s = bf16_lo(scales), b = bf16_hi(scales);
    return fabsf(s) < INFINITY && fabsf(b) < INFINITY && fabsf(__builtin_fmaf(15.0f, s, b)) < INFINITY
               ? 0u : 0x80u;
  } else {
    return 0u;
  }
}
// Groups that it tells apart per quarter of a row.
template <int MODE, int D>
constexpr int kGroupFlags = MODE == BSFP_NVFP4 ? D / 64 : MODE == BSFP_AFFINE ? 1 : 0;
// The scales with those groups' taken as zero.
template <int MODE>
__device__ __forceinline__ uint32_t without(uint32_t scales, uint32_t flags) {
  if constexpr (MODE == BSFP_NVFP4) return scales & ~((flags >> 7) * 0xFFu);
  else return flags ? 0u : scales;
}

// Exponents at which the scaled values stand: the largest is put at 2^8, and
// room is made again when one would pass 2^13 (6 * 2^13 < 65504).
constexpr int kValueExp = 127 + 8, kValueExpMax = 127 + 13;

// The nb for a quarter whose largest biased exponent is e.
__device__ __forceinline__ int value_shift(int e) { return min(kValueExp - e, 120); }

// A key that only some rows see must not cost the others their bits, and would
// where its values are so much larger that a common nb takes the rest of the
// tile out of fp16.  Where the exponents of a tile that some rows do not see
// whole pass the present scale by kValueSpread, the quarters of rows that do not
// fit it are left out at first and then added by themselves: as bf16, which has
// the range (exact for MXFP4, the sum of two for affine), with the probabilities
// as the sum of two.  nb then falls only as far as it must for fp32:
// products of probabilities with values up to 2^115; still larger values are
// finite themselves, so that a probability of zero takes them out.
constexpr int kValueSpread = 12, kValueExpWide = 230, kValueExpTop = 242;
__device__ __forceinline__ int value_shift_wide(int nb, int e) {
  return min(nb, kValueExpWide - min(e, kValueExpTop));
}
// Probabilities (fp16) as bf16, or what that leaves of their 11 bits.
template <bool REST>
__device__ __forceinline__ u32x4_t wide_probabilities(u32x4_t p) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = p[i];  // (a cast of an element in place takes element 0)
    const f16x2_t f = __builtin_bit_cast(f16x2_t, w);
    const float a = (float)f.x, b = (float)f.y;
    o[i] = pack_bf16x2(a, b);
    if constexpr (REST) o[i] = pack_bf16x2(a - bf16_lo(o[i]), b - bf16_hi(o[i]));
  }
  return o;
}
// Values: word j as four bf16 pairs, times 2^nb; REST: what that leaves of
// affine ones (MXFP4 ones are exact).
template <int MODE, int D, bool REST>
__device__ __forceinline__ u32x4_t decode_value_wide(uint32_t w, uint32_t scales, int j, int nb) {
  u32x4_t o;
  if constexpr (MODE == BSFP_MXFP4) {
    const float s = ldexpf(1.0f, e8m0_byte<D>(scales, j) - 127 + nb);
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  } else {
    const float s = ldexpf(bf16_lo(scales), nb), b = ldexpf(bf16_hi(scales), nb);
    auto value = [&](int i) { return __builtin_fmaf((float)(w >> (4 * i) & 15u), s, b); };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = value(2 * i), y = value(2 * i + 1);
      const uint32_t hi = pack_bf16x2(x, y);
      o[i] = REST ? pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi)) : hi;
    }
  }
  return o;
}

// A word of affine codes as bf16 integers, columns in the order
// 0 2 4 6 1 3 5 7 (the nibbles of even and odd columns are split by one mask).
__device__ __forceinline__ u32x4_t decode_codes_split(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  u32x4_t o;
  o.x = nibbles_to_bf16x2<false>(even);
  o.y = nibbles_to_bf16x2<true>(even);
  o.z = nibbles_to_bf16x2<false>(odd);
  o.w = nibbles_to_bf16x2<true>(odd);
  return o;
}

// ------------------------------------------------------- lanes

// Reductions over the four lanes that share a column of a 16x16 product
// (lane, lane ^ 16, lane ^ 32, lane ^ 48), on the lane-swap path.
__device__ __forceinline__ float quad_max(float v) {
  u32x2_t r = __builtin_bit_cast(
      u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  v = fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
  r = __builtin_bit_cast(
      u32x2_t, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
// Maximum and minimum over each group of 16 lanes.
__device__ __forceinline__ int row_max(int v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ int row_min(int v) { return -row_max(-v); }
__device__ __forceinline__ float quad_sum(float v) {
  u32x2_t r = __builtin_bit_cast(
      u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  v = __uint_as_float(r.x) + __uint_as_float(r.y);
  r = __builtin_bit_cast(
      u32x2_t, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// Four 16-bit values of one column from four rows: lane i of a group of 16
// names 4 columns (address of row i / 4, columns 4 (i % 4) ...) and receives
// rows 0..3 of column i.
typedef short s16x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2_t lds_read_transposed(const uint16_t* p) {
  typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// ------------------------------------------------------- requests

// Row numbers are 64-bit: pages * kv_heads * page_size may pass 2^31.
__device__ __forceinline__ int64_t cache_row(const KvParams& p, int page, int head, int offset) {
  return (((int64_t)page * p.kv_heads + head) << p.page_shift) + offset;
}

struct KvRequest {
  int row0, q_len;  // its rows of q
  int kv;           // keys, as given
  int last;         // keys that the table can hold
  int first, end;   // keys that any of its rows sees: [first, end)
};

// From the request's first row, rows and keys.
__device__ __forceinline__ KvRequest kv_request(const KvParams& p, int row0, int q_len, int kv) {
  KvRequest q;
  q.row0 = row0;
  q.q_len = q_len;
  q.kv = kv;
  q.last = p.max_pages << p.page_shift;  // at most kKvMaxKeys
  q.end = q.q_len ? min(q.kv, q.last) : 0;
  q.first = p.window ? (int)max((int64_t)q.kv - q.q_len - p.window + 1, (int64_t)0) : 0;
  q.first = min(q.first, q.end);
  return q;
}

// From the batch's tables, whose values are held within the call's sizes.
__device__ __forceinline__ KvRequest kv_request(const KvParams& p, int r) {
  const int s = min(max(p.q_starts[r], 0), p.tokens), e = min(max(p.q_starts[r + 1], 0), p.tokens);
  return kv_request(p, s, max(e - s, 0), p.pages > 0 ? max(p.kv_lens[r], 0) : 0);
}

// The requests as the kernels look them up: up to 64 stand in the lanes,
// where a second look takes no load.
struct KvRequests {
  const KvParams& p;
  KvRequest mine;  // request `lane`, if there are at most 64
  __device__ __forceinline__ explicit KvRequests(const KvParams& p_) : p(p_), mine() {
    const int lane = threadIdx.x & 63;
    if (p.requests <= 64 && lane < p.requests) mine = kv_request(p, lane);
  }
  // For every lane its own r.
  __device__ __forceinline__ KvRequest of_lane(int r) const {
    return p.requests <= 64 ? mine : kv_request(p, r);
  }
  // r is the same in every lane.
  __device__ __forceinline__ KvRequest at(int r) const {
    if (p.requests <= 64)
      return kv_request(p, __builtin_amdgcn_readlane(mine.row0, r),
                        __builtin_amdgcn_readlane(mine.q_len, r),
                        __builtin_amdgcn_readlane(mine.kv, r));
    return kv_request(p, r);
  }
};

// The keys [lo, hi) that row i of a request sees.
__device__ __forceinline__ void row_keys(const KvParams& p, const KvRequest& q, int i, int& lo,
                                         int& hi) {
  const int pos = q.kv - q.q_len + i;
  hi = pos < 0 ? 0 : min(pos, q.last - 1) + 1;
  lo = p.window && pos >= p.window ? pos - p.window + 1 : 0;
}

// Bit i: key + i lies in [lo, hi), for 16 keys.
__device__ __forceinline__ uint32_t keys_seen(int key, int lo, int hi) {
  const int a = min(max(lo - key, 0), 16), b = min(max(hi - key, 0), 16);
  return ((1u << b) - 1u) & ~((1u << a) - 1u);
}

// ------------------------------------------------------- workgroups

constexpr int kWaves = 4, kThreads = kWaves * 64;

// Operands are read from LDS this many products ahead.  The products, the
// reads and the vector work between them are written in the order of issue,
// with the compiler's scheduler held to it step by step: left alone it puts
// every read right before its product and waits for it.
constexpr int kAhead = 3;
__device__ __forceinline__ void step_end() { __builtin_amdgcn_sched_barrier(0); }

// A key that stands at the maximum has probability 2^kOffset, and the maximum
// is replaced only by one more than a factor of 2^kGrow larger, which spares
// some of the rescaling; 2^(kOffset + kGrow) lies within fp16, with 0.0096 to
// spare in the exponent.
// The exponent is fma(S, c, kOffset - m c): the roundings of m c and of the
// difference, 2^-24 |m c| each, must stay below that, and do up to |m c| = kFar
// (2^-9 in all).  Where a row of the wave is past it, m is taken off S first,
// which is exact for the keys near the maximum, the only ones that can pass the
// bound; for every tile that would be one more instruction per key and row.
// At the end of a segment's part O and l are divided by 2^kOffset, so that sums
// of values near the end of bf16's range do not pass fp32's.
constexpr int kOffsetExp = 15;
constexpr float kOffset = kOffsetExp, kGrow = 0.99f, kFar = 16384.0f;

template <int CTRL>
__device__ __forceinline__ int64_t dpp64(int64_t v) {  // 0 from lanes outside
  const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, 0xF, 0xF, false);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// Lane `from`'s value, as a scalar.
__device__ __forceinline__ int64_t lane64(int64_t v, int from) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)v, from);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(v >> 32), from);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Inclusive sum over the wave.
__device__ __forceinline__ int64_t wave_sum(int64_t v) {
  const int lane = threadIdx.x & 63;
  v += dpp64<0x111>(v);  // from the lanes 1, 2, 4, 8 below in each row of 16 ...
  v += dpp64<0x112>(v);
  v += dpp64<0x114>(v);
  v += dpp64<0x118>(v);
  // ... then over the rows' ends
  const int64_t r0 = lane64(v, 15), r1 = lane64(v, 31), r2 = lane64(v, 47);
  return v + (lane >= 16 ? r0 : 0) + (lane >= 32 ? r1 : 0) + (lane >= 48 ? r2 : 0);
}

// a / b for a >= 0, b > 0, of scalars: 64-bit division is some 150 instructions
// and hardly ever needed.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// A run of the line that the requests' work, laid end to end, makes: tiles
// [start, stop), beginning in request `req` (q), which begins at `base`.  Every
// wave finds it by itself from the lengths: a lane sums a few neighbouring
// requests, a scan over the lanes finds the lane, and a second one over that
// lane's requests the request.  work(q): tiles of a request.
struct Run {
  int64_t start, stop, len, base;
  int req;
  KvRequest q;
};
template <typename F>
__device__ __forceinline__ Run find_run(const KvRequests& reqs, int run, int runs, int min_len,
                                        F work) {
  const int requests = reqs.p.requests;
  const int lane = threadIdx.x & 63, each = (requests + 63) / 64;
  int64_t mine = 0;
  for (int j = 0; j < each; ++j) {
    const int r = lane * each + j;
    if (r < requests) mine += work(reqs.of_lane(r));
  }
  const int64_t incl = wave_sum(mine), total = lane64(incl, 63);
  Run x = {};
  x.len = max(quotient(total + runs - 1, runs), (int64_t)min_len);
  x.start = run * x.len;
  x.stop = min(x.start + x.len, total);
  if (x.start >= x.stop) return x;
  const int at = __builtin_ctzll(__ballot(incl > x.start));
  x.base = lane64(incl - mine, at);
  x.req = at * each;
  if (each <= 1) {
    x.q = reqs.at(x.req);
    return x;
  }
  const int end = min(x.req + each, requests);
  for (int r0 = x.req; r0 < end; r0 += 64) {
    const KvRequest q = kv_request(reqs.p, min(r0 + lane, end - 1));
    const int64_t w = r0 + lane < end ? work(q) : 0, sum = x.base + wave_sum(w);
    const uint64_t past = __ballot(sum > x.start);
    if (past) {
      const int l = __builtin_ctzll(past);
      x.req = r0 + l;
      x.base = lane64(sum - w, l);
      x.q = kv_request(reqs.p, __builtin_amdgcn_readlane(q.row0, l),
                       __builtin_amdgcn_readlane(q.q_len, l), __builtin_amdgcn_readlane(q.kv, l));
      break;
    }
    x.base = lane64(sum, 63);
  }
  return x;
}

// lse from the maximum (times log2 e) and the sum.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

// ------------------------------------------------------- partial states

// A run of the line of key tiles leaves at most two partial states: slot 0 of
// a segment begun by an earlier run, slot 1 of one that goes on in the next.
constexpr int kMaxRuns = 1024;
struct SegmentMeta {  // of the segment that begins in a run and goes on
  int valid, row0, q_len, block, head, parts;
};
struct KvParts {
  float* o;   // [runs][2][rows][D]
  float* ml;  // [runs][2][m, l][rows]
  SegmentMeta* meta;
};
size_t kv_parts_bytes(int runs, int rows, int D);
KvParts kv_parts(void* ws, int runs, int rows, int D);

// The requests of more than kSplitRows query rows per kv head, their partial
// states in ws: the runs of the launch in *runs, *join: whether any segment
// can have been cut.
constexpr int kSplitRows = 16;
constexpr int kPromptRows = 128;  // query rows of a workgroup there
hipError_t launch_kv_prompt(const KvParams& p, int mode, int D, void* ws, int* runs, bool* join,
                            hipStream_t s);
size_t kv_prompt_workspace(int D);

}  // namespace bsfp
