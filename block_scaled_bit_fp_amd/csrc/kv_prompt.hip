// kv_prompt.hip -- attention over the paged 4-bit cache for requests with more
// than kSplitRows query rows per kv head: prompts, prompt chunks, drafts.
//
// A workgroup takes 128 query rows (query * group + head in the group) of one
// kv head, 32 per wave, and walks their keys in tiles of 64: S^T = K . Q^T and
// O^T = V^T . P^T on the 32x32x16 product, so that a query row is a lane
// column.  The 256 threads decode each tile once, a quarter of a row each,
// into LDS as 16-bit operands, with one barrier per tile.  The softmax is that
// of kv_attention.hip.
// While S of tile t is summed, tile t + 1 is decoded into the other buffers
// (in one stretch of code, so that matrix and vector instructions alternate);
// then tile t + 2 is asked for, and the exponentials of tile t alternate with
// the products of O.
//
// Work.  The blocks of a request see more keys the later they stand; block b
// and block n - 1 - b together see about the same number for every b, so the
// pairs of a request all take one length (the largest that a pair can have) on
// the line of key tiles, and a run finds its place by division.  Runs are
// equal, a segment that spans several leaves partial states, and the order on
// the line is by kv head first: the runs of one XCD (every eighth workgroup)
// are neighbours, so an XCD's L2 holds the cache of the one or two kv heads
// that it works on.
//
// Measured (64 query heads over 8 kv heads of 128): two chunks of 1500..2048 rows
// over 4096..8192 keys, 626 GFLOP.  NVFP4: 690..750 us a call by card (836..907
// TFLOP/s; a large bf16 library product: 1230), under a kernel trace, at a lower
// clock, 736..764 for this kernel.  There MXFP4 takes 807 us and affine, with one
// workgroup per CU, 1640.  NVFP4: matrix units 43 % busy, vector issue 62 %, no
// LDS bank conflicts; bound by the vector work beside the products.
// Affine at D = 256 spills: some 150 accesses to scratch a tile (two prompts of
// 700..1000 rows over 2000..3000 keys, 16 heads over 4: 412 us, NVFP4 105).
#include <algorithm>
#include <type_traits>

#include "kv_device.hpp"

namespace bsfp {

namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBlock = kPromptRows;
constexpr int kTile = 64;      // keys
// All in tiles.  Each was measured on both sides (us, this kernel + join; A: two
// prompts of up to 87 rows over 1356 and 2353 keys, affine, 8 heads over 1; B: one
// of 900 over 1300, MXFP4, 8 over 8; C: one of 341 over 2818, MXFP4, 8 over 1; D:
// two of up to 163 over 3697 and 6397, NVFP4, 128 over 8).
// The shortest run.  2: A 21.2 + 10.7, B 26.2 + 10.2, C 24.4 + 13.6; 4: A 25.7 +
// 9.8, B 28.4 + 8.8, C 27.9 + 13.0; D 143.9 + 13.8 and 143.4 + 13.7.
constexpr int kMinRun = 2;
// The longest segment that is never cut.  8: B 26.2 + 10.2; 4: 26.1 + 10.4; 16:
// 45.0 + 8.9; the others alike with all three.
constexpr int kWhole = 8;
// What a segment costs beside its tiles.  3: A 21.2 + 10.7, B 26.2 + 10.2, C 24.4
// + 13.6; 0: A 25.4 + 11.7, B 28.3 + 46.9, C 30.3 + 16.5; 8: A 22.7 + 10.6, B 24.3
// + 24.5, C 26.0 + 15.0.
constexpr int kSegment = 3;

template <int D>
constexpr int k_stride() { return D + 8; }   // halves; rows 4 banks apart
// Rows 16 banks apart (of 64): a transposed read takes 64 bytes of 8 rows.
// Measured over a full CU: 2.8 cycles a read, against 4.3 for D + 16.
template <int D>
constexpr int v_stride() { return D + 32; }

// Where the 16-byte piece of word j of quarter q of a row stands in the
// quarter.  At D = 128 the four quarters of a row, written together, would
// meet in the same banks; measured over a full CU, a write takes 13 cycles
// instead of 16 (K) and 32 (V).
template <int D>
constexpr __device__ int k_piece(int q, int j) { return D == 128 ? j ^ (q & 2) : j; }
template <int D>
constexpr __device__ int v_piece(int q, int j) { return D == 128 ? j ^ q : j; }

__device__ __forceinline__ f32x16_t mma32_f16(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}
// o += v (hi + lo)^T, bf16; by hand as in kv_attention.hip (58 registers spilled
// at MXFP4, D = 128), with 32 steps until the sums are there.
__device__ __forceinline__ void add_wide(f32x16_t& o, u32x4_t v, u32x4_t hi, u32x4_t lo) {
  asm volatile(
      "s_nop 7\n\t"
      "v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0\n\t"
      "s_nop 15\n\t"
      "s_nop 15\n\t"
      "v_mfma_f32_32x32x16_bf16 %0, %1, %3, %0\n\t"
      "s_nop 15\n\t"
      "s_nop 15"
      : "+v"(o) : "v"(v), "v"(hi), "v"(lo));
}
template <int MODE>
__device__ __forceinline__ f32x16_t mma32_keys(u32x4_t a, u32x4_t b, f32x16_t c) {
  if constexpr (MODE == BSFP_NVFP4) return mma32_f16(a, b, c);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ float pair_max(float v) {  // over lane and lane ^ 32
  const u32x2_t r = __builtin_bit_cast(
      u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float pair_sum(float v) {
  const u32x2_t r = __builtin_bit_cast(
      u32x2_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// The keys that rows [a, b) of a request see: all of them in [all_lo, all_hi),
// any in [any_lo, any_hi).
struct Reach { int any_lo, any_hi, all_lo, all_hi; };
__device__ __forceinline__ Reach reach(const KvParams& p, const KvRequest& q, int a, int b) {
  Reach r;
  row_keys(p, q, a / p.group, r.any_lo, r.all_hi);
  row_keys(p, q, (b - 1) / p.group, r.all_lo, r.any_hi);
  return r;
}

struct Work {
  int rows, blocks, pairs;
  int64_t pair_len, head_len, all;  // tiles on the line
};

__device__ __forceinline__ int block_tiles(const KvParams& p, const KvRequest& q, int rows, int b,
                                           int& tile0) {
  const Reach r = reach(p, q, b * kBlock, min(rows, (b + 1) * kBlock));
  tile0 = r.any_lo / kTile;
  return r.any_hi > r.any_lo ? (r.any_hi + kTile - 1) / kTile - tile0 : 0;
}

__device__ __forceinline__ Work prompt_work(const KvParams& p, const KvRequest& q) {
  Work w = {};
  if (q.end <= q.first || (int64_t)q.q_len * p.group <= kSplitRows) return w;
  w.rows = q.q_len * p.group;
  w.blocks = (w.rows + kBlock - 1) / kBlock;
  w.pairs = (w.blocks + 1) / 2;
  if (w.blocks == 1) {
    int t0;
    w.pair_len = block_tiles(p, q, w.rows, 0, t0);
  } else {
    // keys of a pair: both pasts, and kBlock (blocks + 1) rows' queries
    const int64_t past = max(q.kv - q.q_len, 0);
    const int64_t keys = 2 * past + (int64_t)kBlock * (w.blocks + 1) / p.group + 3;
    w.pair_len = max(keys / kTile + 2, (int64_t)q.end / kTile + 1);
    if (p.window) {
      const int64_t one = ((int64_t)p.window + kBlock / p.group + 2) / kTile + 2;
      w.pair_len = min(w.pair_len, 2 * one);
    }
  }
  w.pair_len += w.blocks == 1 ? kSegment : 2 * kSegment;
  w.head_len = w.pairs * w.pair_len;
  w.all = w.head_len * p.kv_heads;
  return w;
}

// Workgroups per CU: what registers and LDS allow.
constexpr int wgs_per_cu(int mode, int D) {
  return D == 256 || (D == 128 && mode == BSFP_AFFINE) ? 1 : 2;
}

template <int D>
struct Buffers {
  uint16_t k[2][kTile * k_stride<D>()];
  uint16_t v[2][kTile * v_stride<D>()];
};

// A thread's quarter of one row, as loaded.
template <int D>
struct Row {
  Words<D / 32> w;
  uint32_t s;
  bool ok;
};

template <int MODE, int D>
__device__ __forceinline__ void load_row(const KvParams& p, const KvSide& side, int head, int key,
                                         int page, int qd, Row<D>& r) {
  r.ok = page >= 0 && page < p.pages;
  const int64_t row = cache_row(p, r.ok ? page : 0, head, key & ((1 << p.page_shift) - 1));
  constexpr int B = scale_bytes<MODE, D>();
  r.w = load_codes<D>(side.codes + row * (D / 2), 0, qd);
  r.s = load_scales<MODE, D>(side.scales + row * B, side.biases + row * B, 0, qd);
}

template <int MODE, int D>
__global__ __launch_bounds__(kThreads, wgs_per_cu(MODE, D)) void kv_prompt_kernel(KvParams p,
                                                                              KvParts parts) {
  constexpr int W = D / 32, KS = D / 16, DT = D / 32, G64 = D / 64;
  constexpr bool kAffine = MODE == BSFP_AFFINE;
  constexpr int kFlags = kGroupFlags<MODE, D>;
  __shared__ __align__(16) Buffers<D> buf;
  __shared__ float s_scale[kAffine ? 2 : 1][kAffine ? G64 : 1][kTile];
  __shared__ float s_bias[kAffine ? 2 : 1][kAffine ? G64 : 1][kTile];
  __shared__ int s_exp[2][4][kWaves], s_least[4][kWaves];
  // a byte for each 16 keys (a wave stages them).  Bit 0: their page is one of
  // the cache's.  Bit 1: some of their values are not finite and taken as zero;
  // s_bad: lane 4 (key % 16) + quarter of the columns, by group of the quarter
  __shared__ uint32_t s_ok[2];
  __shared__ uint64_t s_bad[2][kFlags ? kFlags : 1][kWaves];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int skey = tid >> 2, sq = tid & 3;  // the thread's part of a tile
  const int runs = gridDim.x;
  const int run = runs % 8 ? blockIdx.x : (blockIdx.x % 8) * (runs / 8) + blockIdx.x / 8;

  const KvRequests reqs(p);
  const Run line = find_run(reqs, run, runs, kMinRun,
                            [&](const KvRequest& q) { return prompt_work(p, q).all; });
  if (tid == 0) parts.meta[run].valid = 0;
  if (line.start >= line.stop) return;
  const int64_t start = line.start, stop = line.stop, len = line.len;
  int req = line.req;
  int64_t req_base = line.base;  // where the request begins on the line
  const float gk = (MODE == BSFP_NVFP4 && p.k.g) ? *p.k.g : 1.0f;
  const float gv = (MODE == BSFP_NVFP4 && p.v.g) ? *p.v.g : 1.0f;

  KvRequest q = line.q;
  Work w = prompt_work(p, q);
  // the pair in which the run begins; pairs are numbered head by head
  int64_t pair = quotient(start - req_base, max(w.pair_len, (int64_t)1));
  int second = 0;
  for (;;) {
    if (second > 1) {
      second = 0;
      ++pair;
    }
    if (pair >= (int64_t)w.pairs * p.kv_heads) {  // on to the next request
      req_base += w.all;
      if (req_base >= stop) break;
      do {
        q = reqs.at(++req);
        w = prompt_work(p, q);
      } while (w.all == 0);
      pair = 0;
    }
    const int64_t pair_base = req_base + pair * w.pair_len;
    if (pair_base >= stop) break;
    const int head = (int)quotient(pair, w.pairs), pi = (int)(pair - (int64_t)head * w.pairs);
    const int late = w.blocks - 1 - pi;
    const int block = second ? pi : late;
    int tile0;
    const int tiles = block_tiles(p, q, w.rows, block, tile0);
    int64_t seg = pair_base;
    if (second) {
      int t0;
      seg += block_tiles(p, q, w.rows, late, t0) + kSegment;
      if (pi == late) {
        ++second;
        continue;
      }
    }
    ++second;
    // the segment's part in this run
    int a = 0, b = tiles;
    if (tiles <= kWhole) {
      if (seg < start || seg >= stop) a = b;
    } else {
      a = (int)min(max(start - seg, (int64_t)0), (int64_t)tiles);
      b = (int)min(max(stop - seg, (int64_t)0), (int64_t)tiles);
    }
    const int block_rows = min(w.rows - block * kBlock, kBlock);
    if (tiles == 0) {
      // rows that see no key (more queries than keys); the run that the
      // segment would begin in writes them
      if (seg >= start && seg < stop) {
        for (int i = tid; i < block_rows * (D / 8); i += kThreads) {
          const int row = block * kBlock + i / (D / 8);
          const int64_t orow = (int64_t)(q.row0 + row / p.group) * p.heads + head * p.group +
                               row % p.group;
          reinterpret_cast<u32x4_t*>(p.out)[orow * (D / 8) + i % (D / 8)] = u32x4_t{0, 0, 0, 0};
          if (p.lse && i % (D / 8) == 0) p.lse[orow] = -INFINITY;
        }
      }
      continue;
    }
    if (a >= b) continue;

    // ---- the queries of this lane's row
    const int32_t* table = p.table + (int64_t)req * p.max_pages;
    const int first_row = block * kBlock + wave * 32;
    const int wave_rows = min(max(block_rows - wave * 32, 0), 32);
    const bool live = n < wave_rows;
    const int row = first_row + n;
    const int qi = live ? row / p.group : 0, qh = head * p.group + (live ? row - qi * p.group : 0);
    const uint16_t* qp = p.q + (int64_t)(q.row0 + qi) * p.q_stride + (int64_t)qh * D;
    u32x4_t qf[KS];
    float c = p.scale;
    float qsum[G64];
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      qf[j] = *reinterpret_cast<const u32x4_t*>(qp + j * 16 + half * 8);
      if (!live) qf[j] = u32x4_t{0, 0, 0, 0};
    }
    if constexpr (MODE == BSFP_NVFP4) {
      float x = 0.0f;
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x = fmaxf(x, fmaxf(fabsf(bf16_lo(qf[j][i])), fabsf(bf16_hi(qf[j][i]))));
      x = pair_max(x);
      const int be = min(max((int)(__float_as_uint(x) >> 23), 20), 254);
      const float f = __uint_as_float((uint32_t)(268 - be) << 23);
      c = c * __uint_as_float((uint32_t)(be - 14) << 23) * gk;
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[j][i] = pack_f16x2(bf16_lo(qf[j][i]) * f, bf16_hi(qf[j][i]) * f);
    } else if constexpr (kAffine) {
#pragma unroll
      for (int g = 0; g < G64; ++g) {
        float x = 0.0f;
#pragma unroll
        for (int j = 4 * g; j < 4 * g + 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) x += bf16_lo(qf[j][i]) + bf16_hi(qf[j][i]);
        qsum[g] = pair_sum(x);
      }
#pragma unroll
      for (int j = 0; j < KS; ++j) {  // to the column order of decode_codes_split
        const u32x4_t v = qf[j];
        qf[j].x = __builtin_amdgcn_perm(v.y, v.x, 0x05040100u);
        qf[j].y = __builtin_amdgcn_perm(v.w, v.z, 0x05040100u);
        qf[j].z = __builtin_amdgcn_perm(v.y, v.x, 0x07060302u);
        qf[j].w = __builtin_amdgcn_perm(v.w, v.z, 0x07060302u);
      }
    }
    c = fmaxf(c, 1.1754944e-38f);  // above zero, so that a masked S stays -inf
    int lo, hi;
    row_keys(p, q, qi, lo, hi);
    const Reach all = reach(p, q, block * kBlock, block * kBlock + block_rows);
    // the tiles that every row of the block sees whole
    const int full0 = (all.all_lo + kTile - 1) / kTile, full1 = all.all_hi / kTile;
    const Reach mine = wave_rows ? reach(p, q, first_row, first_row + wave_rows) : Reach{};

    f32x16_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    // bit 4 j + quarter: the row sees a value of that group that is not finite
    uint32_t nans = 0;
    // V of quarter x of the columns is held times 2^nb: in O, in the tile in use
    // and in the tile being staged
    int nb_o[4] = {0, 0, 0, 0}, nb_now[4] = {0, 0, 0, 0}, nb_next[4] = {0, 0, 0, 0};
    bool wide_now = false, wide_next = false;  // some values are left out and added at the end

    const int t_end = tile0 + b;
    auto page_of = [&](int t) {
      const int key = t * kTile + skey;
      return t < t_end && key < q.last ? table[key >> p.page_shift] : -1;
    };
    // Of the quarter that the thread stages.  By value: of an array the compiler
    // would make the choice by address, and keep the array in memory.
    auto own = [&](int x0, int x1, int x2, int x3) {
      return sq < 2 ? (sq ? x1 : x0) : (sq == 2 ? x2 : x3);
    };
    auto largest = [](const int (&x)[kWaves]) {
      return __builtin_amdgcn_readfirstlane(max(max(x[0], x[1]), max(x[2], x[3])));
    };
    // The tile's largest exponents; of the first tile also the least but zero.
    auto publish = [&](const Row<D>& r, int t, bool first) {
      if constexpr (MODE != BSFP_NVFP4) {
        const int key = t * kTile + skey;
        int e = r.ok && key >= all.any_lo && key < all.any_hi ? value_exponent<MODE, D>(r.s) : 0;
        int least = e ? e : 255;
#pragma unroll
        for (int x = 4; x < 64; x <<= 1) e = max(e, __shfl_xor(e, x, 64));
        if (lane < 4) s_exp[t & 1][lane][wave] = e;
        if (first) {
#pragma unroll
          for (int x = 4; x < 64; x <<= 1) least = min(least, __shfl_xor(least, x, 64));
          if (lane < 4) s_least[lane][wave] = least;
        }
      }
    };
    // After the barrier that follows publish: the tile's powers of two.
    auto settle = [&](Row<D>& r, int t, bool first) {
      if constexpr (MODE != BSFP_NVFP4) {
        int e[4], top = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          e[x] = largest(s_exp[t & 1][x]);
          top = max(top, e[x] + nb_next[x]);
        }
        wide_next = false;
        if (__builtin_expect(!first && !wide_now && top <= kValueExpMax, 1)) return;
        int at[4];
        top = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          at[x] = nb_next[x];
          if (first) {
            const int* l4 = s_least[x];
            at[x] = value_shift(min(
                __builtin_amdgcn_readfirstlane(min(min(l4[0], l4[1]), min(l4[2], l4[3]))), e[x]));
          } else if (wide_now) {  // what becomes of it at the end of the tile in use
            at[x] = value_shift_wide(at[x], largest(s_exp[(t + 1) & 1][x]));
          }
          top = max(top, e[x] + at[x]);
        }
        wide_next = top > kValueExp + kValueSpread && !(t >= full0 && t < full1);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          nb_next[x] = !wide_next && (first || e[x] + at[x] > kValueExpMax) ? value_shift(e[x]) : at[x];
        const int nb = own(nb_next[0], nb_next[1], nb_next[2], nb_next[3]);
        if (wide_next && value_exponent<MODE, D>(r.s) + nb > kValueExpMax) r.s = 0;
      }
    };
    bool parted = false;  // bit 1 of s_ok for the wave's rows of the tile being staged
    // Before tile t is staged; tiles that all rows see whole go without.
    auto part_values = [&](Row<D>& r, int t) {
      if constexpr (kFlags > 0) {
        parted = false;
        if (__builtin_expect(t >= full0 && t < full1, 1)) return;
        const int key = t * kTile + skey;
        const uint32_t bad =
            r.ok && key >= all.any_lo && key < all.any_hi ? not_finite<MODE>(r.s) : 0u;
        if (__builtin_expect(!__any(bad), 1)) return;
#pragma unroll
        for (int j = 0; j < kFlags; ++j) {
          const uint64_t lanes = __ballot(bad >> (8 * j + 7) & 1u);
          if (lane == 0) s_bad[t & 1][j][wave] = lanes;
        }
        parted = true;
        r.s = without<MODE>(r.s, bad);
      }
    };
    auto rescale = [&](const int (&to)[4]) {  // of O, to other powers of two
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (nb_o[x] != to[x]) {
          const float f = ldexpf(1.0f, to[x] - nb_o[x]);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            if constexpr (D == 64) {  // a quarter is half of a 32-column tile
              if (d == x / 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[d][(x & 1) * 8 + i] *= f;
              }
            } else {
              if (d / (D / 128) == x) o[d] *= f;
            }
          }
          nb_o[x] = to[x];
        }
    };
    auto stage_k = [&](const Row<D>& r, int t, int j0, int j1) {  // words [j0, j1)
      const int at = t & 1;
      uint16_t* kr = buf.k[at] + skey * k_stride<D>() + sq * (D / 4);
#pragma unroll
      for (int j = j0; j < j1; ++j) {
        if constexpr (kAffine)
          *reinterpret_cast<u32x4_t*>(kr + k_piece<D>(sq, j) * 8) = decode_codes_split(r.w.w[j]);
        else
          *reinterpret_cast<u32x4_t*>(kr + k_piece<D>(sq, j) * 8) =
              decode_key_word<MODE, D>(r.w.w[j], r.s, j);
      }
      if constexpr (kAffine) {
        if (j0 == 0 && sq * (D / 4) % 64 == 0) {
          s_scale[at][sq * (D / 4) / 64][skey] = bf16_lo(r.s);
          s_bias[at][sq * (D / 4) / 64][skey] = bf16_hi(r.s);
        }
      }
    };
    auto stage_v = [&](const Row<D>& r, int t, int j0, int j1) {
      const int at = t & 1, key = t * kTile + skey;
      // a key that no row sees: a value of zero, whatever the page holds
      const bool seen = r.ok && key >= all.any_lo && key < all.any_hi;
      const uint32_t vs = seen ? r.s : 0u;
      const int nb = MODE == BSFP_NVFP4 ? 0 : own(nb_next[0], nb_next[1], nb_next[2], nb_next[3]);
      uint16_t* vr = buf.v[at] + skey * v_stride<D>() + sq * (D / 4);
#pragma unroll
      for (int j = j0; j < j1; ++j)
        *reinterpret_cast<u32x4_t*>(vr + v_piece<D>(sq, j) * 8) =
            decode_value_word<MODE, D>(seen ? r.w.w[j] : 0u, vs, j, nb);
      if (j0 == 0 && lane == 0)
        reinterpret_cast<uint8_t*>(&s_ok[at])[wave] = r.ok | (kFlags > 0 && parted) << 1;
    };
    // The columns 16 j .. of the keys 32 u .. of tile t, as an operand.
    auto key_operand = [&](int at, int i) {
      // piece 2 j + half of the row; k_piece moves pairs of pieces
      const int u = i / KS, j = i % KS, q = j * 64 / D, in = D == 128 ? j ^ (q & 2) / 2 : j;
      return *reinterpret_cast<const u32x4_t*>(buf.k[at] + (u * 32 + n) * k_stride<D>() + in * 16 +
                                               half * 8);
    };
    // The products of S^T, keys 32 u + 8 (i / 4) + 4 half + i % 4 of column n.
    f32x16_t acc;  // affine: the group under way
    auto score = [&](int at, int i, u32x4_t kf, f32x16_t (&sc)[2]) {
      const int u = i / KS, j = i % KS;
      if constexpr (kAffine) {
        acc = mma32_keys<MODE>(kf, qf[j], j % 4 == 0 ? f32x16_t{} : acc);
        if (j % 4 == 3) {  // the group is whole: its scale and bias
          const int g = j / 4;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const int key = u * 32 + 2 * i + half * 4;
            const f32x4_t f = *reinterpret_cast<const f32x4_t*>(&s_scale[at][g][key]);
            const f32x4_t h = *reinterpret_cast<const f32x4_t*>(&s_bias[at][g][key]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = acc[i + e] * f[e] + qsum[g] * h[e];
              sc[u][i + e] = g ? sc[u][i + e] + y : y;
            }
          }
        }
      } else {
        sc[u] = mma32_keys<MODE>(kf, qf[j], j == 0 ? f32x16_t{} : sc[u]);
      }
    };

    // ---- the first tile.  Tiles past the last are staged too, as keys that no
    // row sees, and never used.
    int t = tile0 + a;
    Row<D> rk, rv;
    int page = page_of(t);
    __syncthreads();  // the segment before is done with the buffers
    load_row<MODE, D>(p, p.k, head, t * kTile + skey, page, sq, rk);
    load_row<MODE, D>(p, p.v, head, t * kTile + skey, page, sq, rv);
    page = page_of(t + 1);
    publish(rv, t, true);
    if constexpr (MODE != BSFP_NVFP4) __syncthreads();
    settle(rv, t, true);
    part_values(rv, t);
    stage_k(rk, t, 0, W);
    stage_v(rv, t, 0, W);
    load_row<MODE, D>(p, p.k, head, (t + 1) * kTile + skey, page, sq, rk);
    load_row<MODE, D>(p, p.v, head, (t + 1) * kTile + skey, page, sq, rv);
    page = page_of(t + 2);
    publish(rv, t + 1, false);
    for (; t < t_end; ++t) {
      __syncthreads();
      const int at = t & 1, key0 = t * kTile;
#pragma unroll
      for (int x = 0; x < 4; ++x) nb_now[x] = nb_next[x];
      wide_now = wide_next;
      settle(rv, t + 1, false);
      part_values(rv, t + 1);
      auto load = [&]() {
        load_row<MODE, D>(p, p.k, head, (t + 2) * kTile + skey, page, sq, rk);
        load_row<MODE, D>(p, p.v, head, (t + 2) * kTile + skey, page, sq, rv);
        page = page_of(t + 3);
      };
      // O^T: in steps of 16 keys, 4 half .. + 3 and 8 + 4 half .. + 3 of each in
      // both operands
      const uint16_t* vr = buf.v[at] + (half * 4 + ((lane & 15) >> 2)) * v_stride<D>();
      const int piece = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);  // of 32 columns
      auto value_operand = [&](int i) {
        const uint16_t* r = vr + i / DT * 16 * v_stride<D>() + i % DT * 32 +
                            v_piece<D>(i % DT, piece) * 8 + (lane & 1) * 4;
        const u32x2_t v0 = lds_read_transposed(r);
        const u32x2_t v1 = lds_read_transposed(r + 8 * v_stride<D>());
        return u32x4_t{v0.x, v0.y, v1.x, v1.y};
      };
      // What the exponents are fma(S, c, .) of; past kFar S gets the maximum taken off.
      auto shifted = [&](f32x16_t (&sc)[2]) {
        const float shift = m == -INFINITY ? 0.0f : kOffset - m * c;
        if (__builtin_expect(__any(fabsf(shift) > kFar), 0)) {
          const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
          for (int i = 0; i < 32; ++i) sc[i >> 4][i & 15] -= base;
          return kOffset;
        }
        return shift;
      };
      const bool any_seen = key0 < mine.any_hi && key0 + kTile > mine.any_lo;  // by the wave's rows
      if (any_seen) {
        f32x16_t sc[2];
        u32x4_t kf[2 * KS];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) kf[i] = key_operand(at, i);
        step_end();
        // the wave of the other workgroup on this SIMD fills in its vector work
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) {
          if (i + kAhead < 2 * KS) kf[i + kAhead] = key_operand(at, i + kAhead);
          score(at, i, kf[i], sc);
          // a word of the next tile with every second product (opaque to the
          // compiler, which would decode it before the branch to this path)
          if (i % 4 == 0) {
            asm volatile("" : "+v"(rk.w.w[i / 4]));
            stage_k(rk, t + 1, i / 4, i / 4 + 1);
          }
          if (i % 4 == 2) {
            asm volatile("" : "+v"(rv.w.w[i / 4]));
            stage_v(rv, t + 1, i / 4, i / 4 + 1);
          }
          step_end();
        }
        __builtin_amdgcn_s_setprio(0);
        load();
        const uint32_t ok = __builtin_amdgcn_readfirstlane(s_ok[at]);
        if (key0 < mine.all_lo || key0 + kTile > mine.all_hi || ok != 0x01010101u) {
          if constexpr (kFlags > 0) {
            if (__builtin_expect(ok & 0x02020202u, 0)) {
#pragma unroll
              for (int j = 0; j < kFlags; ++j) {
                uint64_t quarters = 0;  // four bits a key
#pragma unroll
                for (int x = 0; x < kWaves; ++x) {
                  const int z0 = min(max(lo - key0 - x * 16, 0), 16);
                  const int z1 = min(max(hi - key0 - x * 16, z0), 16);
                  const uint64_t seen = z1 > z0 ? ~0ull >> (64 - 4 * (z1 - z0)) << (4 * z0) : 0;
                  if (ok >> (x * 8) & 2u) quarters |= s_bad[at][j][x] & seen;
                }
                uint32_t y = (uint32_t)quarters | (uint32_t)(quarters >> 32);
                y |= y >> 16;
                y |= y >> 8;
                y |= y >> 4;
                nans |= (y & 15u) << (4 * j);
              }
            }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int at16 = u * 32 + (i >> 2) * 8 + half * 4 + (i & 3), key = key0 + at16;
              if (!(ok >> ((u * 2 + (i >> 3)) * 8) & 1) || key < lo || key >= hi)
                sc[u][i] = -INFINITY;
            }
        }
        float mx = sc[0][0];
#pragma unroll
        for (int i = 1; i < 32; ++i) mx = fmaxf(mx, sc[i >> 4][i & 15]);
        mx = fmaxf(pair_max(mx), m);
        // a row without a key so far has m = -inf: any key makes it grow
        if (__any((mx - m) * c > kGrow)) {
          const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - mx) * c);
          l *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d] *= f;
          m = mx;
        }
        if constexpr (MODE != BSFP_NVFP4) rescale(nb_now);
        const float shift = shifted(sc);
        u32x4_t pf[4], vf[4 * DT];
        auto probabilities = [&](int k) {  // pair k of 16
          const int x = k / 4, e = (x & 1) * 8 + 2 * (k % 4);
          const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x >> 1][e], c, shift));
          const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x >> 1][e + 1], c, shift));
          l += e0 + e1;
          pf[x][k % 4] = pack_f16x2(e0, e1);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) vf[i] = value_operand(i);
#pragma unroll
        for (int k = 0; k < 4; ++k) probabilities(k);
        step_end();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < 4 * DT; ++i) {
          if (i + kAhead < 4 * DT) vf[i + kAhead] = value_operand(i + kAhead);
          o[i % DT] = mma32_f16(vf[i], pf[i / DT], o[i % DT]);
#pragma unroll
          for (int k = 4 + i * 4 / DT; k < 4 + (i + 1) * 4 / DT; ++k)
            if (k < 16) probabilities(k);
          step_end();
        }
        __builtin_amdgcn_s_setprio(0);
      } else {
        stage_k(rk, t + 1, 0, W);
        stage_v(rv, t + 1, 0, W);
        load();
      }
      if constexpr (MODE != BSFP_NVFP4) {
        if (__builtin_expect(wide_now, 0)) {  // the values that were left out
          int to[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) to[x] = value_shift_wide(nb_now[x], largest(s_exp[at][x]));
          if (any_seen) rescale(to);
          const int nb = own(nb_now[0], nb_now[1], nb_now[2], nb_now[3]);
          const int nb_wide = own(to[0], to[1], to[2], to[3]);
          auto add = [&](auto rest) {
            __syncthreads();  // all waves are done with the tile as it is
            const int key = key0 + skey;
            Row<D> r;
            load_row<MODE, D>(p, p.v, head, key, page_of(t), sq, r);
            const bool large = r.ok && key >= all.any_lo && key < all.any_hi &&
                               !not_finite<MODE>(r.s) && value_exponent<MODE, D>(r.s) + nb > kValueExpMax;
            uint16_t* row = buf.v[at] + skey * v_stride<D>() + sq * (D / 4);
#pragma unroll
            for (int j = 0; j < W; ++j)
              *reinterpret_cast<u32x4_t*>(row + v_piece<D>(sq, j) * 8) =
                  large ? decode_value_wide<MODE, D, decltype(rest)::value>(r.w.w[j], r.s, j, nb_wide)
                        : u32x4_t{0, 0, 0, 0};
            __syncthreads();
            if (!any_seen) return;
            // the probabilities once more: keeping them would take registers in
            // every tile
            f32x16_t sc[2];
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i) {
              score(at, i, key_operand(at, i), sc);
              step_end();
            }
            const uint32_t ok = __builtin_amdgcn_readfirstlane(s_ok[at]);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int at16 = u * 32 + (i >> 2) * 8 + half * 4 + (i & 3), k = key0 + at16;
                if (!(ok >> ((u * 2 + (i >> 3)) * 8) & 1) || k < lo || k >= hi)
                  sc[u][i] = -INFINITY;
              }
            const float shift = shifted(sc);
#pragma unroll
            for (int x = 0; x < 4; ++x) {  // 16 keys
              u32x4_t pf;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int e = (x & 1) * 8 + 2 * k;
                pf[k] = pack_f16x2(__builtin_amdgcn_exp2f(__builtin_fmaf(sc[x >> 1][e], c, shift)),
                                   __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x >> 1][e + 1], c, shift)));
              }
              const u32x4_t hi = wide_probabilities<false>(pf), lo = wide_probabilities<true>(pf);
#pragma unroll
              for (int d = 0; d < DT; ++d) {
                add_wide(o[d], value_operand(x * DT + d), hi, lo);
                step_end();
              }
            }
          };
          add(std::false_type{});
          if constexpr (kAffine) add(std::true_type{});
        }
      }
      publish(rv, t + 2, false);
    }

    // ---- out, or the partial state
    l = pair_sum(l) * ldexpf(1.0f, -kOffsetExp);
    const float mt = m == -INFINITY ? -INFINITY : m * c;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float f = ldexpf(1.0f, -kOffsetExp - nb_o[x]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        if constexpr (D == 64) {
          if (d == x / 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[d][(x & 1) * 8 + i] *= f;
          }
        } else {
          if (d / (D / 128) == x) o[d] *= f;
        }
      }
    }
    if constexpr (kFlags > 0) {
#pragma unroll
      for (int d = 0; d < 2 * DT; ++d) {  // 16 columns
        const float y = nans >> (d % kFlags * 4 + d * 64 / D) & 1u ? NAN : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[d / 2][(d & 1) * 8 + i] += y;
      }
    }
    const bool whole = b - a == tiles;
    const int slot = run * 2 + (a == 0);
    if (!whole && a == 0 && tid == 0)
      parts.meta[run] = {1, q.row0, q.q_len, block, head,
                         (int)(1 + quotient(seg + tiles - stop + len - 1, len))};
    if (live) {
      const int64_t orow = (int64_t)(q.row0 + qi) * p.heads + qh;
      const int64_t prow = (int64_t)slot * kBlock + wave * 32 + n;
      const float f = l == 0.0f ? 0.0f : gv / l;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4_t v = {o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
          const int d4 = d * 8 + i * 2 + half;  // column / 4
          if (whole)
            reinterpret_cast<u32x2_t*>(p.out)[orow * (D / 4) + d4] =
                u32x2_t{pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f)};
          else
            reinterpret_cast<f32x4_t*>(parts.o)[prow * (D / 4) + d4] = v;
        }
      if (half == 0) {
        if (!whole) {
          parts.ml[(slot * 2) * kBlock + wave * 32 + n] = mt;
          parts.ml[(slot * 2 + 1) * kBlock + wave * 32 + n] = l;
        } else if (p.lse) {
          p.lse[orow] = row_lse(mt, l);
        }
      }
    }
  }
}

int prompt_runs(int mode, int D) {
  return std::min(device_cu_count() * wgs_per_cu(mode, D), kMaxRuns);
}

template <int MODE, int D>
hipError_t run(const KvParams& p, void* ws, int* runs, bool* join, hipStream_t s) {
  *runs = prompt_runs(MODE, D);
  hipLaunchKernelGGL((kv_prompt_kernel<MODE, D>), dim3(*runs), dim3(kThreads), 0, s, p,
                     kv_parts(ws, *runs, kBlock, D));
  // the longest segment there can be; none is cut up to kWhole tiles
  int64_t keys = (int64_t)p.max_pages << p.page_shift;
  if (p.window)
    keys = std::min(keys, (int64_t)p.window + std::min(p.max_q, kBlock / p.group + 2) + kTile - 1);
  *join = (keys + kTile - 1) / kTile > kWhole;
  return hipGetLastError();
}

template <int MODE>
hipError_t run_dim(const KvParams& p, int D, void* ws, int* runs, bool* join, hipStream_t s) {
  return D == 64    ? run<MODE, 64>(p, ws, runs, join, s)
         : D == 128 ? run<MODE, 128>(p, ws, runs, join, s)
                    : run<MODE, 256>(p, ws, runs, join, s);
}

}  // namespace

size_t kv_prompt_workspace(int D) {
  return kv_parts_bytes(prompt_runs(BSFP_NVFP4, D), kBlock, D);  // the most of any format
}

hipError_t launch_kv_prompt(const KvParams& p, int mode, int D, void* ws, int* runs, bool* join,
                            hipStream_t s) {
  switch (mode) {
    case BSFP_NVFP4: return run_dim<BSFP_NVFP4>(p, D, ws, runs, join, s);
    case BSFP_MXFP4: return run_dim<BSFP_MXFP4>(p, D, ws, runs, join, s);
    default: return run_dim<BSFP_AFFINE>(p, D, ws, runs, join, s);
  }
}

}  // namespace bsfp
