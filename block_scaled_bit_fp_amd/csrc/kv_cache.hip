// kv_cache.hip -- the paged 4-bit key/value cache: the step's tables
// (bsfp_kv_plan) and the write of new rows (bsfp_kv_append).
//
// Compiled with -ffp-contract=off like quantize.hip: every fp32 operation is
// one correctly rounded IEEE operation, so appended rows have the codes and
// scales that bsfp_quantize gives them.
#include <algorithm>

#include "bsfp_device.hpp"
#include "bsfp_internal.hpp"

namespace bsfp {

namespace {

// ------------------------------------------------------------------ plan

// Inclusive sums of two values over the THREADS of a workgroup (every thread
// calls; `part` is the workgroup's scratch).
template <int THREADS>
__device__ __forceinline__ void scan2(int64_t& a, int64_t& b, int64_t (*part)[2]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t ua = __shfl_up(a, o, 64), ub = __shfl_up(b, o, 64);
    if (lane >= o) {
      a += ua;
      b += ub;
    }
  }
  if (lane == 63) {
    part[wave][0] = a;
    part[wave][1] = b;
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    a += part[w][0];
    b += part[w][1];
  }
}

// One launch: every workgroup scans the requests (lengths are a few KB and
// come from L2) and then writes its own share of the token outputs; workgroup
// 0 also writes the per-request outputs.  A new page is written to the block
// table by the token that begins it, which is always a token of this step.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void kv_plan_kernel(
    const int32_t* __restrict__ past_lens, const int32_t* __restrict__ q_lens, int requests,
    int page_shift, int32_t* table, int max_pages, const int32_t* __restrict__ free_pages,
    int64_t free_count, const int32_t* __restrict__ free_begin, int64_t tokens,
    int64_t tokens_per_wg, int32_t* __restrict__ kv_lens, int32_t* __restrict__ q_starts,
    int64_t* __restrict__ slots, int32_t* __restrict__ positions, int32_t* __restrict__ state,
    int32_t* __restrict__ next_lens) {
  __shared__ int64_t part[THREADS / 64][2];
  __shared__ int64_t s_tot[2];
  __shared__ int64_t s_end[THREADS];      // running sum of q, inclusive
  __shared__ int32_t s_past[THREADS], s_page0[THREADS], s_old[THREADS];  // page0 < 0: refused
  __shared__ int32_t s_taken[THREADS / 64], s_refused[THREADS / 64];
  const int tid = threadIdx.x;
  const int64_t P = int64_t(1) << page_shift, round = P - 1;
  const int64_t lo = blockIdx.x * tokens_per_wg;
  const int64_t hi = min(lo + tokens_per_wg, tokens);
  const int32_t begin = *free_begin;
  const int64_t avail = begin < 0 ? 0 : max(int64_t(0), free_count - begin);
  int64_t base_q = 0, base_need = 0;  // of the chunks before this one
  int32_t taken = 0, refused = 0;
  for (int r0 = 0; r0 < requests; r0 += THREADS) {
    const int r = r0 + tid;
    const bool in = r < requests;
    const int32_t past = in ? past_lens[r] : 0, q = in ? q_lens[r] : 0;
    const int64_t old = (max(past, 0) + round) >> page_shift;
    // a request that its own lengths rule out asks for no page
    const int64_t len = (int64_t)past + q;
    const bool own_ok = past >= 0 && q >= 0 && len <= min((int64_t)max_pages * P, (int64_t)0x7fffffff);
    const int64_t mine = max(q, 0), own_need = own_ok ? ((len + round) >> page_shift) - old : 0;
    int64_t end = mine, need = own_need;
    scan2<THREADS>(end, need, part);
    end += base_q;
    need += base_need;
    // Tokens beyond `tokens` and pages beyond the free list refuse every later
    // request of the same kind as well (the sums do not fall), so what the
    // refused ones added to the sums moves no admitted request.
    const int64_t off = need - own_need;
    const bool admitted = own_ok && end <= tokens && (own_need == 0 || need <= avail);
    s_end[tid] = end;
    s_past[tid] = past;
    s_old[tid] = (int32_t)old;
    s_page0[tid] = admitted ? (int32_t)min(off, (int64_t)0x7fffffff) : -1;
    if (tid == THREADS - 1) {
      s_tot[0] = end;
      s_tot[1] = need;
    }
    if (blockIdx.x == 0 && in) {
      kv_lens[r] = admitted ? past + q : 0;
      if (next_lens) next_lens[r] = admitted ? past + q : past;
      q_starts[r] = (int32_t)min(end - mine, tokens);
      if (r == requests - 1) q_starts[requests] = (int32_t)min(end, tokens);
      if (admitted && own_need > 0) taken = max(taken, (int32_t)need);
      refused += !admitted;
    }
    __syncthreads();
    // the tokens of this chunk's requests that are this workgroup's
    const int64_t c1 = min(s_tot[0], hi);
    for (int64_t t = max(base_q, lo) + tid; t < c1; t += THREADS) {
      int a = 0, b = THREADS - 1;  // the first request whose end is past t
      while (a < b) {
        const int m = (a + b) >> 1;
        if (s_end[m] > t) b = m; else a = m + 1;
      }
      const int64_t start = a ? s_end[a - 1] : base_q;
      int64_t slot = -1;
      int32_t pos = -1;
      if (s_page0[a] >= 0) {
        pos = s_past[a] + (int32_t)(t - start);
        const int j = pos >> page_shift;
        int32_t* entry = table + (int64_t)(r0 + a) * max_pages + j;
        int32_t page;
        if (j < s_old[a]) {
          page = *entry;
        } else {
          page = free_pages[begin + s_page0[a] + (j - s_old[a])];
          if ((pos & round) == 0) *entry = page;
        }
        if (page >= 0) slot = ((int64_t)page << page_shift) + (pos & round);
      }
      slots[t] = slot;
      positions[t] = pos;
    }
    base_q = s_tot[0];
    base_need = s_tot[1];
    __syncthreads();
  }
  for (int64_t t = max(base_q, lo) + tid; t < hi; t += THREADS) {  // rows of no request
    slots[t] = -1;
    positions[t] = -1;
  }
  if (blockIdx.x == 0) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      taken = max(taken, __shfl_xor(taken, o, 64));
      refused += __shfl_xor(refused, o, 64);
    }
    if ((tid & 63) == 0) {
      s_taken[tid >> 6] = taken;
      s_refused[tid >> 6] = refused;
    }
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < THREADS / 64; ++w) {
        taken = max(taken, s_taken[w]);
        refused += s_refused[w];
      }
      state[0] = begin + taken;
      state[1] = refused;
      if (requests == 0) q_starts[0] = 0;
    }
  }
}

// ------------------------------------------------------------------ append

// Eight values of a group of GROUP (GROUP / 8 adjacent lanes call) -> their
// packed word; sb / bb: the group's scale and bias as stored.  The steps are
// those of the quantizers in quantize.hip.
template <int MODE>
__device__ __forceinline__ uint32_t quantize8(const uint4 xv, float g, uint32_t& sb, uint32_t& bb) {
  float f[8], v[8];
  unpack8(xv, f);
  bb = 0;
  if constexpr (MODE == BSFP_AFFINE) {
    float mn = f[0], mx = f[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) {
      mn = fminf(mn, f[k]);
      mx = fmaxf(mx, f[k]);
    }
    mn = team_min<8>(mn);
    mx = team_max<8>(mx);
    sb = f32_to_bf16((mx - mn) / 15.0f);
    bb = __float_as_uint(mn) >> 16;  // a bf16 value: exact
    const float sc = __uint_as_float(sb << 16);
    const float inv = (sc == 0.0f) ? 0.0f : 1.0f / sc;
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float q = __builtin_rintf((f[k] - mn) * inv);
      w |= (uint32_t)fminf(fmaxf(q, 0.0f), 15.0f) << (4 * k);
    }
    return w;
  } else {
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) a = fmaxf(a, fabsf(f[k]));
    float mul;
    if constexpr (MODE == BSFP_NVFP4) {
      a = team_max<2>(a);
      sb = g != 0.0f ? e4m3_encode(a / (6.0f * g)) : 0u;
      const float d = g != 0.0f ? e4m3_decode(sb) * g : 0.0f;
      if (d == 0.0f) {
        sb = 0;
        return 0;
      }
      mul = 1.0f / d;
    } else {
      a = team_max<4>(a);
      const int e = max((int)(__float_as_uint(a) >> 23) - 129, -127);
      sb = (uint32_t)(e + 127);
      mul = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, exact
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = f[k] * mul;
    return e2m1_pack8(v);
  }
}

struct AppendSide {
  const uint16_t* x;
  int64_t stride;
  uint32_t* codes;
  void* scales;
  uint16_t* biases;
  const float* g;
};

constexpr int kAppendThreads = 256;

// One lane per packed word (one 16-byte load), D / 8 adjacent lanes per row;
// blockIdx.y picks K or V.  The row is asked for together with its slot, so it
// is read whether the slot is good or not.  Row numbers are 32-bit where they
// fit (a 64-bit division is some 150 instructions).
//   8192 rows of 8 x 128 at scattered slots (43 MB): 12.4..13.3 us by card, 3.2 to
// 3.5 TB/s; bound by the scale writes, single bytes of 8 bytes a row.  Two words
// per lane took 1.2 us more, four 1.7.
template <int MODE, int D>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(
    AppendSide k, AppendSide v, const int64_t* __restrict__ slots, int64_t rows, int kv_heads,
    int page_shift, int64_t cache_slots) {
  const AppendSide& s = blockIdx.y ? v : k;
  constexpr int W = D / 8, TEAM = (MODE == BSFP_NVFP4 ? 16 : MODE == BSFP_MXFP4 ? 32 : 64) / 8;
  const float g = (MODE == BSFP_NVFP4 && s.g) ? *s.g : 1.0f;
  const int64_t n = rows * W, step = (int64_t)gridDim.x * kAppendThreads;
  for (int64_t i = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x; i < n; i += step) {
    const int64_t row = i / W;
    const int w = (int)(i % W);
    const int64_t t = rows >> 31 ? row / kv_heads : (uint32_t)row / (uint32_t)kv_heads;
    const int h = (int)(row - t * kv_heads);
    const int64_t slot = slots[t];
    const uint4 xv = *reinterpret_cast<const uint4*>(s.x + t * s.stride + (int64_t)h * D + w * 8);
    if (slot < 0 || slot >= cache_slots) continue;  // a whole row's lanes skip together
    uint32_t sb, bb;
    const uint32_t c = quantize8<MODE>(xv, g, sb, bb);
    const int64_t page = slot >> page_shift, at = slot & ((int64_t(1) << page_shift) - 1);
    const int64_t word = (((page * kv_heads + h) << page_shift) + at) * W + w;
    s.codes[word] = c;
    if (w % TEAM == 0) {
      if constexpr (MODE == BSFP_AFFINE) {
        reinterpret_cast<uint16_t*>(s.scales)[word / TEAM] = (uint16_t)sb;
        s.biases[word / TEAM] = (uint16_t)bb;
      } else {
        reinterpret_cast<uint8_t*>(s.scales)[word / TEAM] = (uint8_t)sb;
      }
    }
  }
}

template <int MODE>
void append_mode(const AppendSide& k, const AppendSide& v, int64_t tokens, const int64_t* slots,
                 const bsfp_kv_cache& c, hipStream_t s) {
  const int D = (int)c.k->cols, shift = __builtin_ctz(c.page_size);
  const int64_t rows = tokens * c.kv_heads;
  const int64_t want = (rows * (D / 8) + kAppendThreads - 1) / kAppendThreads;
  const dim3 grid((uint32_t)std::min<int64_t>(want, (int64_t)device_cu_count() * 16), 2);
  const int64_t cache_slots = c.pages * c.page_size;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kAppendThreads), 0, s, k, v, slots, rows, c.kv_heads,
                       shift, cache_slots);
  };
  if (D == 64) go(kv_append_kernel<MODE, 64>);
  else if (D == 128) go(kv_append_kernel<MODE, 128>);
  else go(kv_append_kernel<MODE, 256>);
}

}  // namespace

hipError_t launch_kv_plan(const int32_t* past, const int32_t* q, int requests, int page_size,
                          int32_t* table, int max_pages, const int32_t* free_pages,
                          int64_t free_count, const int32_t* free_begin, int64_t tokens,
                          int32_t* kv_lens, int32_t* q_starts, int64_t* slots, int32_t* positions,
                          int32_t* state, int32_t* next_lens, hipStream_t s) {
  // one request per thread: with 256 threads 1021 requests take four rounds of
  // the scan, 10.4 us instead of 7.3; up to 256 requests the smaller workgroup
  // starts sooner
  const bool wide = requests > 256;
  const int64_t per = wide ? 2048 : 1024;
  const int64_t wgs = std::max<int64_t>(1, std::min<int64_t>((tokens + per - 1) / per,
                                                             device_cu_count()));
  auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)wgs), dim3(threads), 0, s, past, q, requests,
                       __builtin_ctz(page_size), table, max_pages, free_pages, free_count,
                       free_begin, tokens, (tokens + wgs - 1) / wgs, kv_lens, q_starts, slots,
                       positions, state, next_lens);
  };
  if (wide) go(kv_plan_kernel<1024>, 1024);
  else go(kv_plan_kernel<256>, 256);
  return hipGetLastError();
}

hipError_t launch_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                            int64_t v_stride, int64_t tokens, const int64_t* slots,
                            const bsfp_kv_cache& c, hipStream_t s) {
  const AppendSide ks = {k, k_stride, c.k->codes, c.k->scales, c.k->biases, c.k->global_scale};
  const AppendSide vs = {v, v_stride, c.v->codes, c.v->scales, c.v->biases, c.v->global_scale};
  switch (c.k->mode) {
    case BSFP_NVFP4: append_mode<BSFP_NVFP4>(ks, vs, tokens, slots, c, s); break;
    case BSFP_MXFP4: append_mode<BSFP_MXFP4>(ks, vs, tokens, slots, c, s); break;
    default: append_mode<BSFP_AFFINE>(ks, vs, tokens, slots, c, s); break;
  }
  return hipGetLastError();
}

}  // namespace bsfp
