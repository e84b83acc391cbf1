// kv_attention.hip -- attention over the paged 4-bit key/value cache
// (bsfp_kv_attention).
//
// Rows.  The query rows of a request that read one kv head, q_len * group of
// them (row = query * group + head in the group), are taken 16 at a time: the
// columns of S^T = K . Q^T and of O^T = V^T . P^T on the 16x16x32 product, so
// a query row is a lane column and its maximum, sum and rescaling factor are
// one register per lane.
//
// Softmax in one pass.  With t = S scale log2 e and m a running bound of t,
// p = 2^(t - m + 15); a new m multiplies the sum l and the accumulators O by
// 2^(m_old - m_new).  out = O / l, lse = (m + log2 (l / 2^15)) ln 2.  m is the
// largest t at its last change and changes only when some t passes it by 0.99,
// so p stays below 2^15.99, within fp16, where the probabilities keep 11 bits
// down to 2^-29 of the largest and vanish only below 2^-40 of it.  For that the
// rounding of t and m must stay small beside 0.01 (kFar in kv_device.hpp).
// NVFP4 queries are bf16 values divided by a power of two per row, which puts
// the row's largest at 2^14..2^15: exact in fp16 down to 2^-28 of it.
//
// Work.  Keys go in tiles of 32.  All (request, 16-row tile, kv head) segments
// laid end to end form one line of key tiles, and every workgroup takes an
// equal run of it, so the load is even whatever the lengths are.  A workgroup
// finds its run from the lengths itself (a scan over the requests).  Segments
// of up to kWhole tiles are not cut: they belong to the run in which they
// begin.  The part of a segment in a run is shared out over the four waves,
// which join their states through LDS; short segments go to one wave each.  A
// segment that spans several runs leaves partial states in the workspace, and a
// second kernel joins them in the order of the line.
//
// Measured (kernel alone, NVFP4, 64 query heads over 8 kv heads of 128): 64
// requests of 512..8192 keys, 211 MB: 43.3 us, 4.9 TB/s; one of 131077 keys,
// 151 MB: 31.3 us, 4.8 TB/s; one of 259 keys: 8.9 us, a chain of loads and cold
// instructions.  256 requests, window 128, MXFP4, 64-wide heads: 15.8 us; most
// runs hold two short segments, one wave each, and the other two waves idle.
// Affine, 32 heads over 32, 134 MB: 41.9 us; vector issue is 59 % busy, mostly
// with decoding, and two waves per SIMD do not cover the rest.
#include <algorithm>
#include <type_traits>

#include "kv_device.hpp"

namespace bsfp {

namespace {

constexpr int kTile = 32;       // keys per step of a wave
constexpr int kRows = kSplitRows;  // query rows of a segment

// All in tiles.  Each was measured on both sides (us, split kernel + join; A: 64
// requests of 512..8192 keys; B: 43 of 143..1097 keys, one 64-wide head; C: one of
// 6826 keys, MXFP4, 16 heads over 4; D: 146 of 21..169 affine keys, 16 heads over
// 2; E: 256 with a window of 128, MXFP4, 64-wide heads).
// The shortest run.  4: C 7.3..8.6 + 5.4, D 12.7; 8: C 8.4 + 4.3, D, whose
// segments then queue in one run, 15.7.
constexpr int kMinRun = 4;
// The longest segment that is never cut.  16: A 43.5, B 9.4..10.2 + 4.0; 8: A
// 43.4, B 8.0 + 4.1; 32: A 44.6, B 12.1 + 3.8; E 16.0 with all three.
constexpr int kWhole = 16;
// The longest segment that one wave takes, where runs are longer than the
// shortest; else each run has about one segment, and the waves share it (D 12.7;
// alone there too, 15.5).  6: E 16.0; 3: E 20.1.
constexpr int kAlone = 6;
static_assert(kAlone <= kWhole, "one wave takes whole segments only");
// What a segment costs beside its tiles, in tiles: it takes that much more of
// the line.  More where the four waves share it.  None: A 51.5, C 10.6 + 5.5, D
// 22.6, E 16.7.
constexpr int kSegmentAlone = 4, kSegmentShared = 12;
constexpr __device__ int segment_length(int tiles) {
  return tiles + (tiles <= kAlone ? kSegmentAlone : kSegmentShared);
}
constexpr int kOperandsAhead = 2;  // V operands read ahead of their products

// Halves per row of the staged V tile: 16 more than D, so that 16 rows apart
// by that stride start 8 banks apart and the transposed reads hit all banks.
template <int D>
constexpr int v_stride() { return D + 16; }
template <int D>
constexpr int o_stride() { return D + 4; }

template <int D>
constexpr int split_lds_bytes() {
  constexpr int v = kWaves * kTile * v_stride<D>() * 2, o = kWaves * kRows * o_stride<D>() * 4;
  return v > o ? v : o;
}

struct Work {
  int tiles, tile0;  // of one segment; tile0: its first key tile
  int64_t all;       // kv_heads * segment_length
};

__device__ __forceinline__ Work request_work(const KvParams& p, const KvRequest& q) {
  Work w;
  w.tile0 = q.first / kTile;
  w.tiles = q.end > q.first && (int64_t)q.q_len * p.group <= kRows
                ? (q.end + kTile - 1) / kTile - w.tile0
                : 0;
  w.all = w.tiles ? (int64_t)p.kv_heads * segment_length(w.tiles) : 0;
  return w;
}

// o += v (hi + lo)^T, bf16.  In place by hand: the builtin on a path of its own
// made the compiler copy the sums (28 registers spilled at MXFP4, D = 128).
// With waits longer than the products take: 16 steps until the sums are there.
__device__ __forceinline__ void add_wide(f32x4_t& o, u32x4_t v, u32x4_t hi, u32x4_t lo) {
  asm volatile(
      "s_nop 7\n\t"
      "v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\t"
      "s_nop 15\n\t"
      "v_mfma_f32_16x16x32_bf16 %0, %1, %3, %0\n\t"
      "s_nop 15"
      : "+v"(o) : "v"(v), "v"(hi), "v"(lo));
}

// A tile's keys or values as loaded: two runs of 16 rows.
template <int MODE, int D>
struct Keys {
  Words<D / 32> c[2];
  uint32_t s[2];
  // affine: scales and biases of the four keys of the lane's sums
  u32x2_t as[MODE == BSFP_AFFINE ? 2 : 1][D / 64], ab[MODE == BSFP_AFFINE ? 2 : 1][D / 64];
};
template <int MODE, int D>
struct Values {
  Words<D / 32> c[2];
  uint32_t s[2];
};

// Row numbers of a tile's two runs of 16 keys; -1 past the keys, past the
// table or where the table names no page of the cache.  Wave-uniform.
struct TileRows { int64_t row[2]; };

__device__ __forceinline__ void load_pages(const KvParams& p, const int32_t* table, int tile,
                                           int end, int (&page)[2]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int key = tile * kTile + u * 16;
    page[u] = key < end ? table[key >> p.page_shift] : -1;
  }
}

__device__ __forceinline__ TileRows tile_rows(const KvParams& p, int head, int tile,
                                              const int (&page)[2]) {
  TileRows t;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int pg = __builtin_amdgcn_readfirstlane(page[u]);
    t.row[u] = pg >= 0 && pg < p.pages
                   ? cache_row(p, pg, head, (tile * kTile + u * 16) & ((1 << p.page_shift) - 1))
                   : -1;
  }
  return t;
}

template <int MODE, int D>
__device__ __forceinline__ void load_keys(const KvParams& p, const TileRows& t, int n, int qd,
                                          Keys<MODE, D>& k) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t row = max(t.row[u], (int64_t)0);
    const uint8_t* codes = p.k.codes + row * (D / 2);
    k.c[u] = MODE == BSFP_AFFINE ? load_codes_by_group<D>(codes, n, qd) : load_codes<D>(codes, n, qd);
    const uint8_t* scales = p.k.scales + row * scale_bytes<MODE, D>();
    if constexpr (MODE == BSFP_AFFINE) {
      const uint8_t* biases = p.k.biases + row * scale_bytes<MODE, D>();
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t at = (uint32_t)(qd * (D / 8)) + 8 * i;
        k.as[u][i] = *reinterpret_cast<const u32x2_t*>(scales + at);
        k.ab[u][i] = *reinterpret_cast<const u32x2_t*>(biases + at);
      }
    } else {
      k.s[u] = load_scales<MODE, D>(scales, nullptr, n, qd);
    }
  }
}

template <int MODE, int D>
__device__ __forceinline__ void load_values(const KvParams& p, const TileRows& t, int n, int qd,
                                            Values<MODE, D>& v) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t row = max(t.row[u], (int64_t)0);
    v.c[u] = load_codes<D>(p.v.codes + row * (D / 2), n, qd);
    v.s[u] = load_scales<MODE, D>(p.v.scales + row * scale_bytes<MODE, D>(),
                                  p.v.biases + row * scale_bytes<MODE, D>(), n, qd);
  }
}

// Element i of the bf16 values that two-word pieces hold.
template <int N>
__device__ __forceinline__ float half_at(const u32x2_t (&v)[N], int i) {
  const uint32_t w = (i >> 1) & 1 ? v[i >> 2].y : v[i >> 2].x;
  return i & 1 ? bf16_hi(w) : bf16_lo(w);
}

// Rows without keys: requests run, run + runs, ..., and the rows past the last
// request (place `requests`).
template <int D>
__device__ __forceinline__ void empty_rows(const KvParams& p, const KvRequests& reqs, int run,
                                           int runs) {
  for (int r = run; r <= p.requests; r += runs) {
    int a, b;
    if (r < p.requests) {
      const KvRequest q = reqs.at(r);
      a = q.row0;
      b = q.end > q.first ? a : a + q.q_len;
    } else {
      a = min(max(p.q_starts[p.requests], 0), p.tokens);
      b = p.tokens;
    }
    const int64_t n8 = (int64_t)(b - a) * p.heads * (D / 8);
    u32x4_t* o = reinterpret_cast<u32x4_t*>(p.out) + (int64_t)a * p.heads * (D / 8);
    for (int64_t i = threadIdx.x; i < n8; i += kThreads) o[i] = u32x4_t{0, 0, 0, 0};
    if (p.lse)
      for (int64_t i = threadIdx.x; i < (int64_t)(b - a) * p.heads; i += kThreads)
        p.lse[(int64_t)a * p.heads + i] = -INFINITY;
  }
}

// Workgroups per CU: what the accumulators leave registers for.
constexpr int wgs_per_cu(int mode, int D) {
  return D == 64 ? (mode == BSFP_AFFINE ? 3 : 4)
         : D == 128 ? (mode == BSFP_AFFINE ? 2 : 3)
                    : (mode == BSFP_AFFINE ? 1 : 2);
}

// ONE: no request has more than one new token (a decode step), so that all rows
// of a segment see the same keys and nothing need be told apart by row.  Us with
// it and with the general one: 64 requests of 512..8192 keys, NVFP4 44.0 and 44.4,
// MXFP4 39.6 and 39.8, affine 58.3 and 59.4; 40 of 551..4029, MXFP4, 22.6 and 24.0.
template <int MODE, int D, bool ONE>
__global__ __launch_bounds__(kThreads, wgs_per_cu(MODE, D)) void kv_split_kernel(KvParams p, KvParts parts) {
  constexpr int W = D / 32, DT = D / 16, G64 = D / 64, kFlags = ONE ? 0 : kGroupFlags<MODE, D>;
  __shared__ __align__(16) uint8_t lds[split_lds_bytes<D>()];
  __shared__ float s_ml[kWaves][2][kRows];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, qd = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int runs = gridDim.x, run = blockIdx.x;

  const float gk = (MODE == BSFP_NVFP4 && p.k.g) ? *p.k.g : 1.0f;
  const float gv = (MODE == BSFP_NVFP4 && p.v.g) ? *p.v.g : 1.0f;
  const KvRequests reqs(p);
  const Run line = find_run(reqs, run, runs, kMinRun,
                            [&](const KvRequest& q) { return request_work(p, q).all; });
  if (tid == 0) parts.meta[run].valid = 0;
  if (line.start >= line.stop) {
    empty_rows<D>(p, reqs, run, runs);
    return;
  }
  const int64_t stop = line.stop;

  int req = line.req;
  KvRequest q = line.q;
  Work w = request_work(p, q);
  // at: place in the request's part of the line
  int64_t at = line.start - line.base, cur = line.start;
  int alone = 0;  // short parts so far
  uint16_t* vt = reinterpret_cast<uint16_t*>(lds) + wave * kTile * v_stride<D>();

  while (cur < stop) {
    // the line up to `stop`, and the rest of a short segment that begins before it
    while (at >= w.all) {  // on to the next request that has keys
      ++req;
      q = reqs.at(req);
      w = request_work(p, q);
      at = 0;
    }
    const int length = segment_length(w.tiles);  // of the segment on the line
    const int head = (int)quotient(at, length), from = (int)(at - (int64_t)head * length);
    // the segment's tiles [skip, skip + count) are this run's
    int skip = 0, count = w.tiles, advance = length - from;
    if (w.tiles > kWhole) {
      advance = (int)min((int64_t)advance, stop - cur);
      skip = min(from, w.tiles);
      count = min(from + advance, w.tiles) - skip;
    } else if (from > 0) {  // begun by the run before
      count = 0;
    }
    cur += advance;
    at += advance;
    const bool single = w.tiles <= kAlone && line.len > kMinRun;
    if (count == 0 || (single && (alone++ & (kWaves - 1)) != wave)) continue;
    const int step = single ? 1 : kWaves;
    const int rows = q.q_len * p.group;
    const int32_t* table = p.table + (int64_t)req * p.max_pages;

    // ---- this wave's tiles.  Two tiles are under way: a tile's keys are decoded
    // and its values staged, and then those of the tile after the next are asked
    // for into the same registers.  Past the last tile the loads go to row 0, so
    // that the count of loads under way, by which the waits go, is the same on
    // every path.
    int tile = w.tile0 + skip + (single ? 0 : wave);
    const int tile_end = w.tile0 + skip + count;
    const int load_end = min(q.end, tile_end * kTile);
    Keys<MODE, D> k0, k1;
    Values<MODE, D> v0, v1;
    TileRows rows0, rows1;
    int page[2], page1[2];
    load_pages(p, table, tile, load_end, page);
    load_pages(p, table, tile + step, load_end, page1);
    // ---- the queries of this lane's row, as operands
    const bool live = n < rows;
    const int qi = live ? n / p.group : 0, qh = head * p.group + (live ? n - qi * p.group : 0);
    const uint16_t* qp = p.q + (int64_t)(q.row0 + qi) * p.q_stride + (int64_t)qh * D;
    u32x4_t qf[W];
    float c = p.scale;  // S -> t
    float qsum[G64];    // affine: the sum of the queries over each group
#pragma unroll
    for (int j = 0; j < W; ++j) {
      qf[j] = *reinterpret_cast<const u32x4_t*>(qp + key_column<MODE, D>(j, qd));
      if (!live) qf[j] = u32x4_t{0, 0, 0, 0};
    }

    rows0 = tile_rows(p, head, tile, page);
    load_keys<MODE, D>(p, rows0, n, qd, k0);
    load_values<MODE, D>(p, rows0, n, qd, v0);
    rows1 = tile_rows(p, head, tile + step, page1);
    load_keys<MODE, D>(p, rows1, n, qd, k1);
    load_values<MODE, D>(p, rows1, n, qd, v1);
    load_pages(p, table, tile + 2 * step, load_end, page);
    if constexpr (MODE == BSFP_NVFP4) {
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a = fmaxf(a, fmaxf(fabsf(bf16_lo(qf[j][i])), fabsf(bf16_hi(qf[j][i]))));
      a = quad_max(a);
      // the largest to 2^14..2^15; a biased exponent held within 20..254
      const int be = min(max((int)(__float_as_uint(a) >> 23), 20), 254);
      const float f = __uint_as_float((uint32_t)(268 - be) << 23);
      c = c * __uint_as_float((uint32_t)(be - 14) << 23) * gk;
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[j][i] = pack_f16x2(bf16_lo(qf[j][i]) * f, bf16_hi(qf[j][i]) * f);
    } else if constexpr (MODE == BSFP_AFFINE) {
#pragma unroll
      for (int g = 0; g < G64; ++g) {
        float s = 0.0f;
#pragma unroll
        for (int j = 2 * g; j < 2 * g + 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s += bf16_lo(qf[j][i]) + bf16_hi(qf[j][i]);
        qsum[g] = quad_sum(s);
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {  // to the column order of decode_codes_split
        const u32x4_t v = qf[j];
        qf[j].x = __builtin_amdgcn_perm(v.y, v.x, 0x05040100u);
        qf[j].y = __builtin_amdgcn_perm(v.w, v.z, 0x05040100u);
        qf[j].z = __builtin_amdgcn_perm(v.y, v.x, 0x07060302u);
        qf[j].w = __builtin_amdgcn_perm(v.w, v.z, 0x07060302u);
      }
    }
    c = fmaxf(c, 1.1754944e-38f);  // above zero, so that a masked S stays -inf
    int lo, hi, any_lo, any_hi, all_lo, all_hi;
    row_keys(p, q, qi, lo, hi);
    row_keys(p, q, 0, any_lo, all_hi);
    row_keys(p, q, q.q_len - 1, all_lo, any_hi);

    f32x4_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x4_t{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;  // m: of S, before the factor c
    int nb = 0;                     // the lane's quarter of V is held times 2^nb
    bool have_nb = MODE == BSFP_NVFP4;

    // One tile; `page` holds the pages of the tile after the next.
    auto use_tile = [&](int tile, Keys<MODE, D>& k, Values<MODE, D>& v, TileRows& rows) {
      const TileRows rows_now = rows;
      const int key0 = tile * kTile;
      const bool edge = key0 < all_lo || key0 + kTile > all_hi || rows_now.row[0] < 0 ||
                        rows_now.row[1] < 0;
      // S^T: keys 4 qd + i (+ 16 u) of column n
      float s[8];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (MODE == BSFP_AFFINE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s[4 * u + i] = 0.0f;
#pragma unroll
          for (int g = 0; g < G64; ++g) {
            f32x4_t acc = {0, 0, 0, 0};
            acc = mma16_keys<MODE>(decode_codes_split(k.c[u].w[2 * g]), qf[2 * g], acc);
            acc = mma16_keys<MODE>(decode_codes_split(k.c[u].w[2 * g + 1]), qf[2 * g + 1], acc);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[4 * u + i] += acc[i] * half_at(k.as[u], i * G64 + g) +
                              qsum[g] * half_at(k.ab[u], i * G64 + g);
          }
        } else {
          f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < W; ++j)
            acc = mma16_keys<MODE>(decode_key_word<MODE, D>(k.c[u].w[j], k.s[u], j), qf[j], acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[4 * u + i] = acc[i];
        }
      }
      rows = tile_rows(p, head, tile + 2 * step, page);
      load_keys<MODE, D>(p, rows, n, qd, k);
      load_pages(p, table, tile + 3 * step, load_end, page);
      if (edge) {
        // keys that no row sees: values of zero, whatever the page holds
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = key0 + u * 16 + n;
          if (rows_now.row[u] < 0 || key < any_lo || key >= any_hi) {
#pragma unroll
            for (int j = 0; j < W; ++j) v.c[u].w[j] = 0;
            v.s[u] = 0;
          }
        }
        if constexpr (kFlags > 0) {
          const uint32_t bad[2] = {not_finite<MODE>(v.s[0]), not_finite<MODE>(v.s[1])};
          if (__builtin_expect(q.q_len > 1 && __any(bad[0] | bad[1]), 0)) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t seen = keys_seen(key0 + u * 16, lo, hi);
#pragma unroll
              for (int j = 0; j < kFlags; ++j) {
                const uint64_t keys = __ballot(bad[u] >> (8 * j + 7) & 1u);
#pragma unroll
                for (int d = 0; d < DT; ++d)
                  if (d % kFlags == j) o[d] += (uint32_t)(keys >> (d * 64 / D * 16)) & seen ? NAN : 0.0f;
              }
              v.s[u] = without<MODE>(v.s[u], bad[u]);
            }
          }
        }
      }
      bool wide = false;  // some values are left out and added at the end of the tile
      if constexpr (MODE != BSFP_NVFP4) {  // room for the tile's values in fp16
        const int x0 = value_exponent<MODE, D>(v.s[0]), x1 = value_exponent<MODE, D>(v.s[1]);
        const int x = max(x0, x1);
        if (__builtin_expect(!have_nb || __any(x + nb > kValueExpMax), 0)) {
          const int mx = row_max(x);
          int to = !have_nb ? value_shift(mx) : mx + nb > kValueExpMax ? value_shift(mx) : nb;
          if (!ONE && edge && q.q_len > 1) {
            // the scale in use, or that of the tile's smallest values but zero
            const int least = row_min(min(x0 ? x0 : 255, x1 ? x1 : 255));
            const int at = have_nb ? nb : value_shift(min(least, mx));
            wide = __any(mx + at > kValueExp + kValueSpread);
            if (wide) {
              to = at;
#pragma unroll
              for (int u = 0; u < 2; ++u)
                if ((u ? x1 : x0) + at > kValueExpMax) v.s[u] = 0;
            }
          }
          if (have_nb) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
              o[d] *= ldexpf(1.0f, __builtin_amdgcn_readlane(to - nb, (d * 64 / D) * 16));
          }
          nb = to;
          have_nb = true;
        }
      }
      // V to LDS, as operands, by rows
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < W; ++j)
          *reinterpret_cast<u32x4_t*>(vt + (u * 16 + n) * v_stride<D>() + qd * (D / 4) + j * 8) =
              decode_value_word<MODE, D>(v.c[u].w[j], v.s[u], j, nb);
      load_values<MODE, D>(p, rows, n, qd, v);
      if (edge) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = key0 + (i >> 2) * 16 + qd * 4 + (i & 3);
          if (rows_now.row[i >> 2] < 0 || key < lo || key >= hi) s[i] = -INFINITY;
        }
      }
      float mx = s[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
      mx = fmaxf(quad_max(mx), m);
      // a row without a key so far has m = -inf: any key makes it grow
      if (__any((mx - m) * c > kGrow)) {
        const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - mx) * c);
        l *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= f;
        m = mx;
      }
      float shift = m == -INFINITY ? 0.0f : kOffset - m * c;
      if (__builtin_expect(__any(fabsf(shift) > kFar), 0)) {
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] -= base;
        shift = kOffset;
      }
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, shift));
        l += e[i];
      }
      u32x4_t pf;
#pragma unroll
      for (int i = 0; i < 4; ++i) pf[i] = pack_f16x2(e[2 * i], e[2 * i + 1]);
      // O^T: the step's keys 4 qd .. + 3 and 16 + 4 qd .. + 3 in both operands
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const uint16_t* vr = vt + (qd * 4 + (n >> 2)) * v_stride<D>() + (n & 3) * 4;
      auto value_operand = [&](int d) {
        const u32x2_t a = lds_read_transposed(vr + d * 16);
        const u32x2_t b = lds_read_transposed(vr + 16 * v_stride<D>() + d * 16);
        return u32x4_t{a.x, a.y, b.x, b.y};
      };
      u32x4_t vf[DT];
#pragma unroll
      for (int d = 0; d < kOperandsAhead; ++d) vf[d] = value_operand(d);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        if (d + kOperandsAhead < DT) vf[d + kOperandsAhead] = value_operand(d + kOperandsAhead);
        o[d] = mma16_f16(vf[d], pf, o[d]);
        step_end();
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if constexpr (MODE != BSFP_NVFP4 && !ONE) {
        if (__builtin_expect(wide, 0)) {  // the values that were left out
          uint32_t scales[2];
          int mx = 0;
          bool large[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int64_t row = max(rows_now.row[u], (int64_t)0) * scale_bytes<MODE, D>();
            scales[u] = load_scales<MODE, D>(p.v.scales + row, p.v.biases + row, n, qd);
            const int key = key0 + u * 16 + n, x = value_exponent<MODE, D>(scales[u]);
            large[u] = rows_now.row[u] >= 0 && key >= any_lo && key < any_hi &&
                       x + nb > kValueExpMax && !not_finite<MODE>(scales[u]);
            if (large[u]) mx = max(mx, x);
          }
          const int to = value_shift_wide(nb, row_max(mx));
#pragma unroll
          for (int d = 0; d < DT; ++d)
            o[d] *= ldexpf(1.0f, __builtin_amdgcn_readlane(to - nb, (d * 64 / D) * 16));
          nb = to;
          const u32x4_t hi = wide_probabilities<false>(pf), lo = wide_probabilities<true>(pf);
          auto add = [&](auto rest) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const Words<W> w =
                  load_codes<D>(p.v.codes + max(rows_now.row[u], (int64_t)0) * (D / 2), n, qd);
#pragma unroll
              for (int j = 0; j < W; ++j) {
                *reinterpret_cast<u32x4_t*>(vt + (u * 16 + n) * v_stride<D>() + qd * (D / 4) + j * 8) =
                    large[u] ? decode_value_wide<MODE, D, decltype(rest)::value>(w.w[j], scales[u], j, nb)
                             : u32x4_t{0, 0, 0, 0};
                step_end();
              }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              add_wide(o[d], value_operand(d), hi, lo);
              step_end();
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          };
          add(std::false_type{});
          if constexpr (MODE == BSFP_AFFINE) add(std::true_type{});
        }
      }
    };
    for (; tile < tile_end; tile += 2 * step) {
      use_tile(tile, k0, v0, rows0);
      if (tile + step >= tile_end) break;
      use_tile(tile + step, k1, v1, rows1);
    }

    // ---- join the waves
#pragma unroll
    for (int d = 0; d < DT; ++d)
      o[d] *= ldexpf(1.0f, -kOffsetExp - __builtin_amdgcn_readlane(nb, (d * 64 / D) * 16));
    l = quad_sum(l) * ldexpf(1.0f, -kOffsetExp);
    const float mt = m == -INFINITY ? -INFINITY : m * c;
    if (single) {
      if (live) {
        const int64_t orow = (int64_t)(q.row0 + qi) * p.heads + qh;
        const float f = l == 0.0f ? 0.0f : gv / l;
#pragma unroll
        for (int d = 0; d < DT; ++d)
          reinterpret_cast<u32x2_t*>(p.out)[orow * (D / 4) + d * 4 + qd] =
              u32x2_t{pack_bf16x2(o[d].x * f, o[d].y * f), pack_bf16x2(o[d].z * f, o[d].w * f)};
        if (p.lse && qd == 0) p.lse[orow] = row_lse(mt, l);
      }
      continue;
    }
    const bool whole = count == w.tiles;
    const int slot = run * 2 + (skip == 0);  // 1: the segment begins in this run
    if (!whole && skip == 0 && tid == 0) {
      const int64_t left = w.tiles - count;
      parts.meta[run] = {1, q.row0, q.q_len, 0, head, (int)(1 + quotient(left + line.len - 1, line.len))};
    }
    __syncthreads();
    float* of = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<f32x4_t*>(of + (wave * kRows + n) * o_stride<D>() + d * 16 + qd * 4) = o[d];
    if (qd == 0) {
      s_ml[wave][0][n] = mt;
      s_ml[wave][1][n] = l;
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int rn = i / (D / 4), d4 = i % (D / 4);
      float M = s_ml[0][0][rn];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) M = fmaxf(M, s_ml[v][0][rn]);
      float L = 0.0f;
      f32x4_t sum = {0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        const float x = s_ml[v][0][rn];
        const float f = x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(x - M);
        // a wave without keys holds zeros
        L += s_ml[v][1][rn] * f;
        sum += *reinterpret_cast<const f32x4_t*>(of + (v * kRows + rn) * o_stride<D>() + d4 * 4) * f;
      }
      if (whole) {
        const int64_t orow =
            (int64_t)(q.row0 + rn / p.group) * p.heads + head * p.group + rn % p.group;
        const float f = L == 0.0f ? 0.0f : gv / L;
        reinterpret_cast<u32x2_t*>(p.out)[orow * (D / 4) + d4] =
            u32x2_t{pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f)};
        if (p.lse && d4 == 0) p.lse[orow] = row_lse(M, L);
      } else {
        reinterpret_cast<f32x4_t*>(parts.o)[((int64_t)slot * kRows + rn) * (D / 4) + d4] = sum;
        if (d4 == 0) {
          parts.ml[(slot * 2) * kRows + rn] = M;
          parts.ml[(slot * 2 + 1) * kRows + rn] = L;
        }
      }
    }
    __syncthreads();
  }
  empty_rows<D>(p, reqs, run, runs);
}

// Joins the partial states of a segment that begins in one run and ends in a
// later one; a workgroup looks at one run of the split kernel (kRows rows) or
// of the prompt kernel (kPromptRows rows).
//   Up to kFewParts parts: each strand of D / 4 threads takes rows of its own
//   and the parts one after the other.
//   More: the largest maximum and the sum first, over the lanes, then the parts
//   shared out over strands, whose sums are added in a fixed order.  For few
//   rows the whole workgroup takes a row, else every wave one of its own.
constexpr int kFewParts = 8;

struct JoinSide {
  KvParts parts;
  int runs, rows;
};

template <int D>
__global__ __launch_bounds__(kThreads) void kv_join_kernel(KvParams p, JoinSide split,
                                                           JoinSide prompt) {
  const bool first = (int)blockIdx.x < split.runs;
  const KvParts parts = first ? split.parts : prompt.parts;
  const int rows = first ? split.rows : prompt.rows, run = blockIdx.x - (first ? 0 : split.runs);
  const SegmentMeta s = parts.meta[run];
  if (!s.valid) return;
  constexpr int Q = D / 4, S = kThreads / Q;
  __shared__ f32x4_t s_o[S][Q];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int live = min(s.q_len * p.group - s.block * rows, rows);
  const float gv = p.v.g ? *p.v.g : 1.0f;
  // part i stands in slot 0 of run + i, part 0 in slot 1
  auto slot = [](int i) { return i * 2 + (i == 0); };
  const f32x4_t* po = reinterpret_cast<const f32x4_t*>(parts.o) + (int64_t)run * 2 * rows * Q;
  const float* pml = parts.ml + (int64_t)run * 4 * rows;
  auto write = [&](int rn, int d4, f32x4_t sum, float M, float L) {
    const float f = L == 0.0f ? 0.0f : gv / L;
    const int row = s.block * rows + rn;
    const int64_t orow =
        (int64_t)(s.row0 + row / p.group) * p.heads + s.head * p.group + row % p.group;
    reinterpret_cast<u32x2_t*>(p.out)[orow * Q + d4] =
        u32x2_t{pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f)};
    if (p.lse && d4 == 0) p.lse[orow] = row_lse(M, L);
  };
  // Maximum and sum of row rn over the parts, from the wave's lanes.
  auto totals = [&](int rn, float& M, float& L) {
    float ml = -INFINITY, ll = 0.0f;
    for (int i = lane; i < s.parts; i += 64) {
      const float m = pml[slot(i) * 2 * rows + rn], l = pml[(slot(i) * 2 + 1) * rows + rn];
      const float mx = fmaxf(ml, m);
      const float f = ml == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml - mx);
      const float g = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - mx);
      ll = ll * f + l * g;
      ml = mx;
    }
    M = team_max<64>(ml);
    L = team_sum<64>(ml == -INFINITY ? ll * 0.0f : ll * __builtin_amdgcn_exp2f(ml - M));
  };
  // Parts from, from + step, ... of row rn.
  auto gather = [&](int rn, int d4, int from, int step, float M) {
    f32x4_t sum = {0, 0, 0, 0};
#pragma unroll 8
    for (int i = from; i < s.parts; i += step) {
      const float m = pml[slot(i) * 2 * rows + rn];
      const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
      sum += po[((int64_t)slot(i) * rows + rn) * Q + d4] * f;
    }
    return sum;
  };
  if (s.parts <= kFewParts) {
    const int d4 = tid % Q, strand = tid / Q;
    for (int rn = blockIdx.y * S + strand; rn < live; rn += gridDim.y * S) {
      float m[kFewParts], l[kFewParts], M = -INFINITY, L = 0.0f;
      f32x4_t o[kFewParts], sum = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) {
        if (i >= s.parts) break;
        m[i] = pml[slot(i) * 2 * rows + rn];
        l[i] = pml[(slot(i) * 2 + 1) * rows + rn];
        o[i] = po[((int64_t)slot(i) * rows + rn) * Q + d4];
        M = fmaxf(M, m[i]);
      }
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) {
        if (i >= s.parts) break;
        const float f = m[i] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[i] - M);
        L += l[i] * f;
        sum += o[i] * f;
      }
      write(rn, d4, sum, M, L);
    }
  } else if (live > kRows) {
    const int d4 = lane % Q, strand = lane / Q;
    for (int rn = blockIdx.y * kWaves + wave; rn < live; rn += gridDim.y * kWaves) {
      float M, L;
      totals(rn, M, L);
      f32x4_t sum = gather(rn, d4, strand, 64 / Q, M);
#pragma unroll
      for (int x = Q; x < 64; x <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], x, 64);
      if (strand == 0) write(rn, d4, sum, M, L);
    }
  } else {
    const int d4 = tid % Q, strand = tid / Q;
    for (int rn = blockIdx.y; rn < live; rn += gridDim.y) {
      float M, L;
      totals(rn, M, L);  // by every wave
      f32x4_t sum = gather(rn, d4, strand, S, M);
      s_o[strand][d4] = sum;
      __syncthreads();
      if (strand == 0) {
#pragma unroll
        for (int j = 1; j < S; ++j) sum += s_o[j][d4];
        write(rn, d4, sum, M, L);
      }
      __syncthreads();
    }
  }
}

template <int MODE, int D>
hipError_t run(const KvParams& p, void* ws, hipStream_t s) {
  JoinSide split = {{}, std::min(device_cu_count() * wgs_per_cu(MODE, D), kMaxRuns), kRows};
  split.parts = kv_parts(ws, split.runs, kRows, D);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(split.runs), dim3(kThreads), 0, s, p, split.parts);
  };
  if (std::min(p.max_q, p.tokens) == 1) go(kv_split_kernel<MODE, D, true>);
  else go(kv_split_kernel<MODE, D, false>);
  hipError_t e = hipGetLastError();
  int live = (int)std::min<int64_t>((int64_t)p.max_q * p.group, kRows);
  // the longest segment there can be; none is cut up to kWhole tiles
  int64_t keys = (int64_t)p.max_pages << p.page_shift;
  if (p.window) keys = std::min(keys, (int64_t)p.window + p.max_q - 1 + kTile - 1);
  if ((keys + kTile - 1) / kTile <= kWhole) split.runs = 0;
  JoinSide prompt = {{}, 0, kPromptRows};
  // no request has more tokens than the call
  if (e == hipSuccess && (int64_t)std::min(p.max_q, p.tokens) * p.group > kRows) {
    void* at = (uint8_t*)ws + kv_parts_bytes(kMaxRuns, kRows, D);
    bool join = false;
    e = launch_kv_prompt(p, MODE, D, at, &prompt.runs, &join, s);
    prompt.parts = kv_parts(at, prompt.runs, kPromptRows, D);
    if (!join) prompt.runs = 0;
    live = 16;
  }
  if (e != hipSuccess || split.runs + prompt.runs == 0) return e;
  hipLaunchKernelGGL(kv_join_kernel<D>, dim3(split.runs + prompt.runs, std::min(live, 16)),
                     dim3(kThreads), 0, s, p, split, prompt);
  return hipGetLastError();
}

template <int MODE>
hipError_t run_dim(const KvParams& p, int D, void* ws, hipStream_t s) {
  return D == 64 ? run<MODE, 64>(p, ws, s) : D == 128 ? run<MODE, 128>(p, ws, s)
                                                      : run<MODE, 256>(p, ws, s);
}

KvSide side(const bsfp_qtensor& t) {
  return {(const uint8_t*)t.codes, (const uint8_t*)t.scales, (const uint8_t*)t.biases,
          t.mode == BSFP_NVFP4 ? t.global_scale : nullptr};
}

}  // namespace

size_t kv_parts_bytes(int runs, int rows, int D) {
  return (size_t)runs * (2 * rows * (size_t)(D + 2) * 4 + sizeof(SegmentMeta));
}

KvParts kv_parts(void* ws, int runs, int rows, int D) {
  float* o = (float*)ws;
  float* ml = o + (size_t)runs * 2 * rows * D;
  return {o, ml, (SegmentMeta*)(ml + (size_t)runs * 4 * rows)};
}

size_t kv_attention_workspace(int64_t tokens, int heads, int kv_heads, int head_dim, int) {
  const size_t split = kv_parts_bytes(kMaxRuns, kRows, head_dim);
  return tokens * (heads / kv_heads) <= kRows ? split : split + kv_prompt_workspace(head_dim);
}

hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t s) {
  const bsfp_kv_cache& c = *a.cache;
  const KvParams p = {a.q, a.q_stride, (int)a.tokens, a.heads, c.kv_heads, a.heads / c.kv_heads,
                      side(*c.k), side(*c.v), c.pages, __builtin_ctz(c.page_size), a.table,
                      a.max_pages, a.kv_lens, a.q_starts, a.requests, a.max_q,
                      a.scale * 1.4426950408889634f, a.window, a.out, a.lse};
  const int D = (int)c.k->cols, mode = c.k->mode;
  switch (mode) {
    case BSFP_NVFP4: return run_dim<BSFP_NVFP4>(p, D, a.ws, s);
    case BSFP_MXFP4: return run_dim<BSFP_MXFP4>(p, D, a.ws, s);
    default: return run_dim<BSFP_AFFINE>(p, D, a.ws, s);
  }
}

}  // namespace bsfp
