// api.hip -- the C ABI of libbsfp (declared in include/bsfp.h).
//
// Every entry point validates its arguments on the host before anything is
// enqueued, never throws, and reports failures as a status plus a
// thread-local message (a C++ exception crossing a language bridge
// terminates the process, and an unsupported group size that throws ends a
// whole test binary: "feat(quant): backend quantization capability table and
// load-time convert-or-reject policy", Gate impact).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <iterator>
#include <mutex>

#include "bsfp_device.hpp"
#include "bsfp_internal.hpp"

namespace bsfp {

namespace {

thread_local char g_err[512] = "";

bsfp_status fail(bsfp_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

bsfp_status ok() {
  g_err[0] = '\0';
  return BSFP_OK;
}

bsfp_status device_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(BSFP_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

const char* mode_name(int mode) {
  switch (mode) {
    case BSFP_AFFINE: return "affine";
    case BSFP_MXFP4: return "mxfp4";
    case BSFP_NVFP4: return "nvfp4";
    case BSFP_MXFP8: return "mxfp8";
    default: return "unknown";
  }
}

// A format variant (MXFP8, or affine other than 4-bit group 64).
bool is_variant(const bsfp_qtensor* q) {
  return format_id(q->mode, q->bits, q->group_size) >= FMT_MXFP8;
}

// Checks the descriptor of a quantized tensor; need_data: its code/scale
// buffers must be present (non-empty tensors).
bsfp_status check_qtensor(const bsfp_qtensor* q, const char* fn) {
  if (!q) return fail(BSFP_ERR_ARG, "%s: null tensor descriptor", fn);
  if (format_id(q->mode, q->bits, q->group_size) < 0)
    return fail(BSFP_ERR_UNSUPPORTED,
                "%s: unsupported format (mode %d, bits %d, group %d); supported: "
                "(affine, 4 or 8, 32/64/128), (mxfp4, 4, 32), (nvfp4, 4, 16), (mxfp8, 8, 32)",
                fn, (int)q->mode, (int)q->bits, (int)q->group_size);
  if (q->rows < 0 || q->cols < 0)
    return fail(BSFP_ERR_ARG, "%s: negative shape [%lld, %lld]", fn, (long long)q->rows,
                (long long)q->cols);
  if (q->cols % q->group_size)
    return fail(BSFP_ERR_ARG, "%s: cols %lld is not a multiple of the %s group size %d", fn,
                (long long)q->cols, mode_name(q->mode), (int)q->group_size);
  // element counts (rows * cols) are formed in int64 from here on
  if (q->rows > 0 && q->cols > 0 && q->rows > (int64_t(1) << 40) / q->cols)
    return fail(BSFP_ERR_UNSUPPORTED, "%s: [%lld, %lld] holds more than 2^40 elements", fn,
                (long long)q->rows, (long long)q->cols);
  if (q->rows > 0 && q->cols > 0) {
    if (!q->codes || !q->scales)
      return fail(BSFP_ERR_ARG, "%s: null codes or scales", fn);
    if (!aligned16(q->codes))
      return fail(BSFP_ERR_ARG, "%s: codes pointer is not 16-byte aligned", fn);
    if (q->mode == BSFP_AFFINE && !q->biases)
      return fail(BSFP_ERR_ARG, "%s: affine tensor without biases", fn);
  }
  return ok();
}

std::mutex g_cu_mutex;
int g_cu_count[64] = {0};
int g_max_lds[64] = {0};

}  // namespace

int device_cu_count() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  std::lock_guard<std::mutex> lock(g_cu_mutex);
  if (g_cu_count[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        n <= 0)
      n = 256;
    g_cu_count[dev] = n;
  }
  return g_cu_count[dev];
}

thread_local LaunchEvents g_launch_events = {nullptr, nullptr};

LaunchEvents take_launch_events() {
  const LaunchEvents e = g_launch_events;
  g_launch_events = {nullptr, nullptr};
  return e;
}

int device_max_lds() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 64 * 1024;
  std::lock_guard<std::mutex> lock(g_cu_mutex);
  if (g_max_lds[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMaxSharedMemoryPerBlock, dev) != hipSuccess ||
        n <= 0)
      n = 64 * 1024;
    g_max_lds[dev] = n;
  }
  return g_max_lds[dev];
}

}  // namespace bsfp

// ---------------------------------------------------------------------------
// bsfp_qmm_noalloc: bsfp_qmm with the workspace in the library's own device
// memory, for callers that cannot allocate.  `scratch` is a file-scope device
// array (one copy per GPU, held until the process ends).  In host code its
// name is only a stand-in: its device address on the current GPU comes from
// hipGetSymbolAddress, taken once per device and kept in g_scratch_ptr, and
// only that pointer is ever handed to kernels.
static __device__ __align__(256) uint8_t scratch[BSFP_NOALLOC_WORKSPACE_BYTES];

namespace bsfp {
namespace {
std::mutex g_scratch_mutex;
void* g_scratch_ptr[64] = {nullptr};

// The device address of `scratch` on the current device (nullptr and a
// message on failure).
void* scratch_ptr(const char* fn, bsfp_status* st) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) {
    *st = fail(BSFP_ERR_DEVICE, "%s: hipGetDevice: %s", fn, hipGetErrorString(e));
    return nullptr;
  }
  if (dev < 0 || dev >= 64) {
    *st = fail(BSFP_ERR_UNSUPPORTED, "%s: device %d beyond the 64 the library tracks", fn, dev);
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || !p) {
      *st = fail(BSFP_ERR_DEVICE, "%s: hipGetSymbolAddress(scratch) on device %d: %s", fn, dev,
                 hipGetErrorString(e));
      return nullptr;
    }
    g_scratch_ptr[dev] = p;
  }
  *st = BSFP_OK;
  return g_scratch_ptr[dev];
}
}  // namespace
}  // namespace bsfp

using namespace bsfp;

extern "C" {

const char* bsfp_last_error(void) { return g_err; }

bsfp_status bsfp_time_next_launch(void* start_event, void* stop_event) {
  g_launch_events = {(hipEvent_t)start_event, (hipEvent_t)stop_event};
  return BSFP_OK;
}

const char* bsfp_version(void) { return "bsfp 0.1.0 (gfx950)"; }

bsfp_status bsfp_amax(const uint16_t* x, int64_t n, float* amax_out, bsfp_stream stream) {
  if (n < 0) return fail(BSFP_ERR_ARG, "bsfp_amax: negative n");
  if (!amax_out) return fail(BSFP_ERR_ARG, "bsfp_amax: null output");
  if (n > 0 && (!x || !aligned16(x)))
    return fail(BSFP_ERR_ARG, "bsfp_amax: x is null or not 16-byte aligned");
  return device_status(launch_amax(x, n, amax_out, (hipStream_t)stream), "bsfp_amax");
}

static_assert(BSFP_QUANTIZE_WS_BYTES == kAmaxParts * sizeof(float),
              "the quantize workspace holds one partial maximum per amax workgroup");

// bsfp_quantize, bsfp_quantize_sr (rbits != nullptr: stochastic rounding) and
// bsfp_quantize_ws (parts != nullptr: NVFP4 GS_COMPUTE reduces the amax from
// partial maxima there; checked by the caller).
static bsfp_status quantize_impl(const uint16_t* x, const bsfp_qtensor* q, int32_t gs,
                                 const uint32_t* rbits, bsfp_stream stream, const char* fn,
                                 float* parts = nullptr) {
  bsfp_status st = check_qtensor(q, fn);
  if (st != BSFP_OK) return st;
  const int64_t n = q->rows * q->cols;
  hipStream_t s = (hipStream_t)stream;
  if (q->mode == BSFP_NVFP4) {
    if (gs < BSFP_GS_NONE || gs > BSFP_GS_GIVEN)
      return fail(BSFP_ERR_ARG, "%s: bad global-scale flag %d", fn, (int)gs);
    if (gs != BSFP_GS_NONE && !q->global_scale)
      return fail(BSFP_ERR_ARG, "%s: nvfp4 global scale requested but global_scale is null", fn);
    if (gs == BSFP_GS_COMPUTE && !q->amax)
      return fail(BSFP_ERR_ARG, "%s: BSFP_GS_COMPUTE needs an amax buffer", fn);
  }
  if (n > 0 && (!x || !aligned16(x)))
    return fail(BSFP_ERR_ARG, "%s: x is null or not 16-byte aligned", fn);
  const int64_t n_words = n / 8;
  hipError_t e = hipSuccess;
  switch (q->mode) {
    case BSFP_NVFP4:
      if (gs == BSFP_GS_COMPUTE && parts && n > 0) {
        e = launch_amax_quantize_nvfp4(x, n, q->codes, (uint8_t*)q->scales, parts, q->amax,
                                       q->global_scale, s, rbits);
      } else if (gs == BSFP_GS_COMPUTE) {
        e = launch_amax(x, n, q->amax, s);
        if (e == hipSuccess)
          e = launch_quantize_nvfp4(x, n_words, q->codes, (uint8_t*)q->scales, q->amax, 1,
                                    q->global_scale, s, rbits);
      } else if (n_words > 0) {
        e = launch_quantize_nvfp4(x, n_words, q->codes, (uint8_t*)q->scales,
                                  gs == BSFP_GS_GIVEN ? q->global_scale : nullptr, 0, nullptr, s,
                                  rbits);
      }
      break;
    case BSFP_MXFP4:
      if (n_words > 0)
        e = launch_quantize_mxfp4(x, n_words, q->codes, (uint8_t*)q->scales, s, rbits);
      break;
    default:
      if (is_variant(q))
        e = launch_quantize_variant(x, *q, s);
      else if (n_words > 0)
        e = launch_quantize_affine(x, n_words, q->codes, (uint16_t*)q->scales, q->biases, s);
      break;
  }
  return device_status(e, fn);
}

bsfp_status bsfp_quantize(const uint16_t* x, const bsfp_qtensor* q, int32_t gs,
                          bsfp_stream stream) {
  return quantize_impl(x, q, gs, nullptr, stream, "bsfp_quantize");
}

bsfp_status bsfp_quantize_sr(const uint16_t* x, const bsfp_qtensor* q, int32_t gs,
                             const uint32_t* rbits, bsfp_stream stream) {
  if (q && q->mode != BSFP_NVFP4 && q->mode != BSFP_MXFP4)
    return fail(BSFP_ERR_UNSUPPORTED,
                "bsfp_quantize_sr: stochastic rounding applies to nvfp4 and mxfp4 only");
  if (q && q->rows * q->cols > 0 && (!rbits || !aligned16(rbits)))
    return fail(BSFP_ERR_ARG, "bsfp_quantize_sr: rbits is null or not 16-byte aligned");
  return quantize_impl(x, q, gs, rbits, stream, "bsfp_quantize_sr");
}

bsfp_status bsfp_quantize_ws(const uint16_t* x, const bsfp_qtensor* q, int32_t gs,
                             const uint32_t* rbits, void* workspace, int64_t workspace_bytes,
                             bsfp_stream stream) {
  const char* fn = "bsfp_quantize_ws";
  bsfp_status st = check_qtensor(q, fn);  // also bounds rows * cols
  if (st != BSFP_OK) return st;
  const bool nonempty = q->rows * q->cols > 0;
  if (rbits) {  // the checks of bsfp_quantize_sr
    if (q->mode != BSFP_NVFP4 && q->mode != BSFP_MXFP4)
      return fail(BSFP_ERR_UNSUPPORTED,
                  "%s: stochastic rounding applies to nvfp4 and mxfp4 only", fn);
    if (nonempty && !aligned16(rbits))
      return fail(BSFP_ERR_ARG, "%s: rbits is not 16-byte aligned", fn);
  }
  const bool uses_ws = q->mode == BSFP_NVFP4 && gs == BSFP_GS_COMPUTE;
  if (uses_ws) {
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 4 != 0)
      return fail(BSFP_ERR_ARG, "%s: workspace is null or not 4-byte aligned", fn);
    if (workspace_bytes < BSFP_QUANTIZE_WS_BYTES)
      return fail(BSFP_ERR_ARG, "%s: workspace of %lld bytes, %d needed", fn,
                  (long long)workspace_bytes, (int)BSFP_QUANTIZE_WS_BYTES);
  }
  return quantize_impl(x, q, gs, rbits, stream, fn,
                       uses_ws ? static_cast<float*>(workspace) : nullptr);
}

bsfp_status bsfp_dequantize(const bsfp_qtensor* q, uint16_t* out, bsfp_stream stream) {
  bsfp_status st = check_qtensor(q, "bsfp_dequantize");
  if (st != BSFP_OK) return st;
  if (q->rows * q->cols > 0 && (!out || !aligned16(out)))
    return fail(BSFP_ERR_ARG, "bsfp_dequantize: out is null or not 16-byte aligned");
  return device_status(launch_dequantize(*q, out, (hipStream_t)stream), "bsfp_dequantize");
}

bsfp_status bsfp_qmv(const uint16_t* x, int64_t M, const bsfp_qtensor* w, uint16_t* y,
                     bsfp_stream stream) {
  bsfp_status st = check_qtensor(w, "bsfp_qmv");
  if (st != BSFP_OK) return st;
  if (M < 1 || M > 8) return fail(BSFP_ERR_ARG, "bsfp_qmv: M = %lld outside 1..8", (long long)M);
  if (w->cols == 0) return fail(BSFP_ERR_ARG, "bsfp_qmv: K must be positive");
  if (!x || !aligned16(x)) return fail(BSFP_ERR_ARG, "bsfp_qmv: x is null or not 16-byte aligned");
  if (w->rows > 0 && !y) return fail(BSFP_ERR_ARG, "bsfp_qmv: null y");
  if (is_variant(w) && !qmv_variant_supported((int)M, *w))
    return fail(BSFP_ERR_UNSUPPORTED,
                "bsfp_qmv: %s %d-bit group %d needs x of at most 64 KB and K < 2^28 "
                "(M = %lld, K = %lld)", mode_name(w->mode), (int)w->bits, (int)w->group_size,
                (long long)M, (long long)w->cols);
  return device_status(launch_qmv(x, (int)M, *w, y, (hipStream_t)stream), "bsfp_qmv");
}

bsfp_status bsfp_qmv_batch(const uint16_t* x, int64_t M, const bsfp_qtensor* const* w,
                           int32_t count, uint16_t* const* y, bsfp_stream stream) {
  if (count < 1 || count > BSFP_QMV_BATCH_MAX)
    return fail(BSFP_ERR_ARG, "bsfp_qmv_batch: count = %d outside 1..%d", (int)count,
                BSFP_QMV_BATCH_MAX);
  if (!w || !y) return fail(BSFP_ERR_ARG, "bsfp_qmv_batch: null descriptor or output array");
  for (int i = 0; i < count; ++i)
    if (!w[i]) return fail(BSFP_ERR_ARG, "bsfp_qmv_batch: descriptor %d is null", i);
  for (int i = 0; i < count; ++i) {
    bsfp_status st = check_qtensor(w[i], "bsfp_qmv_batch");
    if (st != BSFP_OK) return st;
    if (w[i]->mode != w[0]->mode || w[i]->bits != w[0]->bits ||
        w[i]->group_size != w[0]->group_size || w[i]->cols != w[0]->cols)
      return fail(BSFP_ERR_ARG,
                  "bsfp_qmv_batch: matrix %d differs from matrix 0 in format or K", i);
    if (w[i]->rows > 0 && (!y[i] || !aligned16(y[i])))
      return fail(BSFP_ERR_ARG, "bsfp_qmv_batch: output %d is null or not 16-byte aligned", i);
  }
  if (M < 1 || M > 8)
    return fail(BSFP_ERR_ARG, "bsfp_qmv_batch: M = %lld outside 1..8", (long long)M);
  if (w[0]->cols == 0) return fail(BSFP_ERR_ARG, "bsfp_qmv_batch: K must be positive");
  if (!x || !aligned16(x))
    return fail(BSFP_ERR_ARG, "bsfp_qmv_batch: x is null or not 16-byte aligned");
  if (is_variant(w[0]) && !qmv_variant_supported((int)M, *w[0]))
    return fail(BSFP_ERR_UNSUPPORTED,
                "bsfp_qmv_batch: %s %d-bit group %d needs x of at most 64 KB and K < 2^28 "
                "(M = %lld, K = %lld)", mode_name(w[0]->mode), (int)w[0]->bits,
                (int)w[0]->group_size, (long long)M, (long long)w[0]->cols);
  return device_status(launch_qmv_batch(x, (int)M, w, y, count, (hipStream_t)stream),
                       "bsfp_qmv_batch");
}

size_t bsfp_qmm_workspace_bytes(int32_t mode, int64_t M, int64_t K, int32_t act) {
  if (mode < BSFP_AFFINE || mode > BSFP_NVFP4 || M < 0 || K < 0) return 0;
  if (act != BSFP_ACT_BF16 && act != BSFP_ACT_SAME) return 0;
  return qmm_workspace_bytes(mode, M, K, act);
}

// Argument checks of bsfp_qmm and bsfp_qmm_noalloc (everything but the
// workspace).  *done is set when the call has nothing to compute.
static bsfp_status check_qmm(const uint16_t* x, int64_t M, const bsfp_qtensor* w, int32_t act,
                             const uint16_t* y, const char* fn, bool* done) {
  *done = false;
  bsfp_status st = check_qtensor(w, fn);
  if (st != BSFP_OK) return st;
  if (is_variant(w))
    return fail(BSFP_ERR_UNSUPPORTED,
                "%s: %s %d-bit group %d runs on the dense path (bsfp_qmm_dense)", fn,
                mode_name(w->mode), (int)w->bits, (int)w->group_size);
  if (M < 0) return fail(BSFP_ERR_ARG, "%s: negative M", fn);
  if (act != BSFP_ACT_BF16 && act != BSFP_ACT_SAME)
    return fail(BSFP_ERR_ARG, "%s: bad activation mode %d", fn, (int)act);
  if (M == 0 || w->rows == 0) {
    *done = true;
    return ok();
  }
  if (w->cols == 0) return fail(BSFP_ERR_ARG, "%s: K must be positive", fn);
  if (!x || !aligned16(x)) return fail(BSFP_ERR_ARG, "%s: x is null or not 16-byte aligned", fn);
  if (!y || !aligned16(y)) return fail(BSFP_ERR_ARG, "%s: y is null or not 16-byte aligned", fn);
  if (w->cols % 64)
    return fail(BSFP_ERR_UNSUPPORTED, "%s: K = %lld is not a multiple of 64", fn,
                (long long)w->cols);
  if ((reinterpret_cast<uintptr_t>(w->scales) & 3) ||
      (w->biases && (reinterpret_cast<uintptr_t>(w->biases) & 3)))
    return fail(BSFP_ERR_ARG, "%s: scales and biases must be 4-byte aligned", fn);
  if (act == BSFP_ACT_SAME && w->mode == BSFP_AFFINE)
    return fail(BSFP_ERR_UNSUPPORTED,
                "%s: BSFP_ACT_SAME is supported for nvfp4 and mxfp4 weights only", fn);
  if (M > (1 << 30) || w->rows > (1 << 30))
    return fail(BSFP_ERR_UNSUPPORTED, "%s: M or N beyond 2^30", fn);
  // every launch shape keeps its grid under 2^32 threads up to 2^33 outputs
  if ((uint64_t)M * (uint64_t)w->rows > (1ULL << 33))
    return fail(BSFP_ERR_UNSUPPORTED, "%s: M * N = %llu beyond 2^33", fn,
                (unsigned long long)M * (unsigned long long)w->rows);
  // the GEMM addresses a 256-row activation tile with 32-bit byte offsets
  if (w->cols > (1 << 22))
    return fail(BSFP_ERR_UNSUPPORTED, "%s: K = %lld beyond 2^22", fn, (long long)w->cols);
  return ok();
}

bsfp_status bsfp_qmm(const uint16_t* x, int64_t M, const bsfp_qtensor* w, int32_t act,
                     void* workspace, size_t workspace_bytes, uint16_t* y, bsfp_stream stream) {
  bool done = false;
  const bsfp_status st = check_qmm(x, M, w, act, y, "bsfp_qmm", &done);
  if (st != BSFP_OK || done) return st;
  const size_t need = qmm_workspace_bytes(w->mode, M, w->cols, act);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(BSFP_ERR_ARG, "bsfp_qmm: workspace needs %zu bytes (16-byte aligned), got %zu",
                need, workspace_bytes);
  return device_status(launch_qmm(x, M, *w, act, workspace, y, (hipStream_t)stream), "bsfp_qmm");
}

bsfp_status bsfp_qmm_noalloc(const uint16_t* x, int64_t M, const bsfp_qtensor* w, int32_t act,
                             uint16_t* y, bsfp_stream stream) {
  bool done = false;
  bsfp_status st = check_qmm(x, M, w, act, y, "bsfp_qmm_noalloc", &done);
  if (st != BSFP_OK || done) return st;
  const size_t need = qmm_workspace_bytes(w->mode, M, w->cols, act);
  if (need > (size_t)BSFP_NOALLOC_WORKSPACE_BYTES)
    return fail(BSFP_ERR_UNSUPPORTED,
                "bsfp_qmm_noalloc: this product needs a %zu-byte workspace, beyond the %zu "
                "bytes of the library's static one (M = %lld, K = %lld); use bsfp_qmm with a "
                "caller workspace", need, (size_t)BSFP_NOALLOC_WORKSPACE_BYTES, (long long)M,
                (long long)w->cols);
  void* ws = nullptr;
  if (need > 0) {
    ws = scratch_ptr("bsfp_qmm_noalloc", &st);
    if (!ws) return st;
  }
  return device_status(launch_qmm(x, M, *w, act, ws, y, (hipStream_t)stream),
                       "bsfp_qmm_noalloc");
}

size_t bsfp_qmm_dense_scratch_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return 0;
  return (size_t)rows * (size_t)cols * 2;
}

bsfp_status bsfp_qmm_dense(const uint16_t* x, int64_t M, const bsfp_qtensor* w, void* scratch,
                           size_t scratch_bytes, uint16_t* y, bsfp_stream stream) {
  bsfp_status st = check_qtensor(w, "bsfp_qmm_dense");
  if (st != BSFP_OK) return st;
  if (M < 0) return fail(BSFP_ERR_ARG, "bsfp_qmm_dense: negative M");
  if (M == 0 || w->rows == 0) return ok();
  if (w->cols == 0) return fail(BSFP_ERR_ARG, "bsfp_qmm_dense: K must be positive");
  if (!x || !aligned16(x))
    return fail(BSFP_ERR_ARG, "bsfp_qmm_dense: x is null or not 16-byte aligned");
  if (!y || !aligned16(y))
    return fail(BSFP_ERR_ARG, "bsfp_qmm_dense: y is null or not 16-byte aligned");
  if (w->cols % 64)
    return fail(BSFP_ERR_UNSUPPORTED, "bsfp_qmm_dense: K = %lld is not a multiple of 64",
                (long long)w->cols);
  if (M > (1 << 30) || w->rows > (1 << 30))
    return fail(BSFP_ERR_UNSUPPORTED, "bsfp_qmm_dense: M or N beyond 2^30");
  if ((uint64_t)M * (uint64_t)w->rows > (1ULL << 33))
    return fail(BSFP_ERR_UNSUPPORTED, "bsfp_qmm_dense: M * N = %llu beyond 2^33",
                (unsigned long long)M * (unsigned long long)w->rows);
  if (w->cols > (1 << 22))
    return fail(BSFP_ERR_UNSUPPORTED, "bsfp_qmm_dense: K = %lld beyond 2^22",
                (long long)w->cols);
  const size_t need = bsfp_qmm_dense_scratch_bytes(w->rows, w->cols);
  if (!scratch || scratch_bytes < need || !aligned16(scratch))
    return fail(BSFP_ERR_ARG,
                "bsfp_qmm_dense: scratch needs %zu bytes (16-byte aligned), got %zu", need,
                scratch_bytes);
  return device_status(launch_qmm_dense(x, M, *w, scratch, y, (hipStream_t)stream),
                       "bsfp_qmm_dense");
}

// ---------------------------------------------------------------------------
// Paged 4-bit key/value cache.

static bool kv_page_size_ok(int p) {
  return p == 16 || p == 32 || p == 64 || p == 128 || p == 256;
}

// Checks a cache: two tensors of one base 4-bit format and of the shape that
// pages, kv_heads and page_size give.
static bsfp_status check_kv_cache(const bsfp_kv_cache* c, const char* fn) {
  if (!c || !c->k || !c->v) return fail(BSFP_ERR_ARG, "%s: null cache or tensor descriptor", fn);
  const bsfp_qtensor* const both[2] = {c->k, c->v};
  for (const bsfp_qtensor* t : both) {
    bsfp_status st = check_qtensor(t, fn);
    if (st != BSFP_OK) return st;
    if (is_variant(t))
      return fail(BSFP_ERR_UNSUPPORTED,
                  "%s: a cache holds nvfp4, mxfp4 or affine 4-bit group 64, not %s %d-bit group %d",
                  fn, mode_name(t->mode), (int)t->bits, (int)t->group_size);
  }
  if (c->k->mode != c->v->mode || c->k->cols != c->v->cols || c->k->rows != c->v->rows)
    return fail(BSFP_ERR_ARG, "%s: K and V differ in format or shape", fn);
  if (!kv_page_size_ok(c->page_size))
    return fail(BSFP_ERR_ARG, "%s: page size %d is not 16, 32, 64, 128 or 256", fn,
                (int)c->page_size);
  if (c->kv_heads < 1 || c->kv_heads > 65535)
    return fail(BSFP_ERR_ARG, "%s: kv_heads = %d outside 1..65535", fn, (int)c->kv_heads);
  if (c->pages < 0 || c->pages > 0x7fffffffLL)
    return fail(BSFP_ERR_ARG, "%s: pages = %lld outside 0..2^31-1", fn, (long long)c->pages);
  if (c->k->cols != 64 && c->k->cols != 128 && c->k->cols != 256)
    return fail(BSFP_ERR_UNSUPPORTED, "%s: head dimension %lld is not 64, 128 or 256", fn,
                (long long)c->k->cols);
  if (c->k->rows != c->pages * c->kv_heads * c->page_size)
    return fail(BSFP_ERR_ARG, "%s: %lld rows, %lld pages x %d heads x %d tokens need %lld", fn,
                (long long)c->k->rows, (long long)c->pages, (int)c->kv_heads, (int)c->page_size,
                (long long)(c->pages * c->kv_heads * c->page_size));
  // scales and biases are read in runs of up to 16 bytes
  for (const bsfp_qtensor* t : both)
    if (c->pages > 0 && (!aligned16(t->scales) || (t->mode == BSFP_AFFINE && !aligned16(t->biases))))
      return fail(BSFP_ERR_ARG, "%s: scales and biases must be 16-byte aligned", fn);
  return ok();
}

struct Range {
  const char* name;
  const void* p;
  int64_t bytes;
};
static bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}

static bsfp_status kv_plan(const char* fn, const int32_t* past_lens, const int32_t* q_lens,
                           int32_t requests, int32_t page_size, int32_t* block_table,
                           int32_t max_pages, const int32_t* free_pages, int64_t free_count,
                           const int32_t* free_begin, int64_t tokens, int32_t* kv_lens,
                           int32_t* q_starts, int64_t* slots, int32_t* positions, int32_t* state,
                           int32_t* next_lens, bsfp_stream stream) {
  if (requests < 0 || max_pages < 0)
    return fail(BSFP_ERR_ARG, "%s: negative requests or max_pages", fn);
  if (tokens < 0 || tokens > 0x7fffffffLL)
    return fail(BSFP_ERR_ARG, "%s: tokens = %lld outside 0..2^31-1", fn, (long long)tokens);
  if (free_count < 0 || free_count > 0x7fffffffLL)
    return fail(BSFP_ERR_ARG, "%s: free_count = %lld outside 0..2^31-1", fn,
                (long long)free_count);
  if (!kv_page_size_ok(page_size))
    return fail(BSFP_ERR_ARG, "%s: page size %d is not 16, 32, 64, 128 or 256", fn,
                (int)page_size);
  if (!q_starts || !state || !free_begin)
    return fail(BSFP_ERR_ARG, "%s: null q_starts, state or free_begin", fn);
  if (requests > 0 && (!past_lens || !q_lens || !kv_lens))
    return fail(BSFP_ERR_ARG, "%s: null lengths", fn);
  if (requests > 0 && max_pages > 0 && !block_table)
    return fail(BSFP_ERR_ARG, "%s: null block_table", fn);
  if (free_count > 0 && !free_pages) return fail(BSFP_ERR_ARG, "%s: null free_pages", fn);
  if (tokens > 0 && (!slots || !positions))
    return fail(BSFP_ERR_ARG, "%s: null slots or positions", fn);
  // every workgroup reads all lengths and the others write meanwhile
  const Range written[] = {
      {"block_table", block_table, (int64_t)requests * max_pages * 4}, {"kv_lens", kv_lens, requests * 4LL},
      {"q_starts", q_starts, (requests + 1LL) * 4}, {"slots", slots, tokens * 8},
      {"positions", positions, tokens * 4}, {"state", state, 8},
      {"next_lens", next_lens, next_lens ? requests * 4LL : 0}};
  const Range read[] = {{"past_lens", past_lens, requests * 4LL}, {"q_lens", q_lens, requests * 4LL},
                        {"free_pages", free_pages, free_count * 4}, {"free_begin", free_begin, 4}};
  for (const Range& w : written) {
    for (const Range& r : read)
      if (overlap(w, r)) return fail(BSFP_ERR_ARG, "%s: %s overlaps %s", fn, w.name, r.name);
    for (const Range* o = &w + 1; o != std::end(written); ++o)
      if (overlap(w, *o)) return fail(BSFP_ERR_ARG, "%s: %s overlaps %s", fn, w.name, o->name);
  }
  return device_status(launch_kv_plan(past_lens, q_lens, requests, page_size, block_table,
                                      max_pages, free_pages, free_count, free_begin, tokens,
                                      kv_lens, q_starts, slots, positions, state, next_lens,
                                      (hipStream_t)stream), fn);
}

bsfp_status bsfp_kv_plan(const int32_t* past_lens, const int32_t* q_lens, int32_t requests,
                         int32_t page_size, int32_t* block_table, int32_t max_pages,
                         const int32_t* free_pages, int64_t free_count,
                         const int32_t* free_begin, int64_t tokens, int32_t* kv_lens,
                         int32_t* q_starts, int64_t* slots, int32_t* positions, int32_t* state,
                         bsfp_stream stream) {
  return kv_plan("bsfp_kv_plan", past_lens, q_lens, requests, page_size, block_table, max_pages,
                 free_pages, free_count, free_begin, tokens, kv_lens, q_starts, slots, positions,
                 state, nullptr, stream);
}

bsfp_status bsfp_kv_plan_carry(const int32_t* past_lens, const int32_t* q_lens, int32_t requests,
                               int32_t page_size, int32_t* block_table, int32_t max_pages,
                               const int32_t* free_pages, int64_t free_count,
                               const int32_t* free_begin, int64_t tokens, int32_t* kv_lens,
                               int32_t* q_starts, int64_t* slots, int32_t* positions,
                               int32_t* state, int32_t* next_lens, bsfp_stream stream) {
  const char* fn = "bsfp_kv_plan_carry";
  if (requests > 0 && !next_lens) return fail(BSFP_ERR_ARG, "%s: null next_lens", fn);
  return kv_plan(fn, past_lens, q_lens, requests, page_size, block_table, max_pages, free_pages,
                 free_count, free_begin, tokens, kv_lens, q_starts, slots, positions, state,
                 next_lens, stream);
}

bsfp_status bsfp_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                           int64_t v_stride, int64_t tokens, const int64_t* slots,
                           const bsfp_kv_cache* cache, bsfp_stream stream) {
  const char* fn = "bsfp_kv_append";
  bsfp_status st = check_kv_cache(cache, fn);
  if (st != BSFP_OK) return st;
  if (tokens < 0) return fail(BSFP_ERR_ARG, "%s: negative tokens", fn);
  if (tokens == 0 || cache->pages == 0) return ok();
  const int64_t row = (int64_t)cache->kv_heads * cache->k->cols;
  if (tokens > (int64_t(1) << 40) / row)
    return fail(BSFP_ERR_UNSUPPORTED, "%s: %lld tokens of %lld values exceed 2^40", fn,
                (long long)tokens, (long long)row);
  if (!k || !v || !aligned16(k) || !aligned16(v))
    return fail(BSFP_ERR_ARG, "%s: k or v is null or not 16-byte aligned", fn);
  if (!slots) return fail(BSFP_ERR_ARG, "%s: null slots", fn);
  if (k_stride % 8 || v_stride % 8 || k_stride < 0 || v_stride < 0)
    return fail(BSFP_ERR_ARG, "%s: token strides %lld and %lld must be multiples of 8", fn,
                (long long)k_stride, (long long)v_stride);
  return device_status(launch_kv_append(k, k_stride, v, v_stride, tokens, slots, *cache,
                                        (hipStream_t)stream), fn);
}

size_t bsfp_kv_attention_workspace_bytes(int64_t tokens, int32_t heads, int32_t kv_heads,
                                         int32_t head_dim, int32_t requests) {
  if (tokens < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || requests < 0) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return kv_attention_workspace(tokens, heads, kv_heads, head_dim, requests);
}

bsfp_status bsfp_kv_attention(const uint16_t* q, int64_t q_stride, int64_t tokens, int32_t heads,
                              const bsfp_kv_cache* cache, const int32_t* block_table,
                              int32_t max_pages, const int32_t* kv_lens, const int32_t* q_starts,
                              int32_t requests, int32_t max_q, float scale, int32_t window,
                              uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                              bsfp_stream stream) {
  const char* fn = "bsfp_kv_attention";
  bsfp_status st = check_kv_cache(cache, fn);
  if (st != BSFP_OK) return st;
  if (tokens < 0 || requests < 0 || max_pages < 0)
    return fail(BSFP_ERR_ARG, "%s: negative tokens, requests or max_pages", fn);
  if ((int64_t)max_pages * cache->page_size > kKvMaxKeys)
    return fail(BSFP_ERR_UNSUPPORTED, "%s: a table of %d pages x %d tokens exceeds %lld keys", fn,
                (int)max_pages, (int)cache->page_size, (long long)kKvMaxKeys);
  if (heads < 1 || heads % cache->kv_heads)
    return fail(BSFP_ERR_UNSUPPORTED, "%s: %d heads are not a multiple of %d kv heads", fn,
                (int)heads, (int)cache->kv_heads);
  if (max_q < 1) return fail(BSFP_ERR_ARG, "%s: max_q = %d below 1", fn, (int)max_q);
  if (window < 0) return fail(BSFP_ERR_ARG, "%s: negative window", fn);
  // the kernels take exponentials to base 2
  if (!(scale > 0.0f) || !(scale * 1.4426950408889634f <= 3.402823466e38f))
    return fail(BSFP_ERR_ARG, "%s: scale must be positive, and finite times log2 e", fn);
  if (tokens == 0) return ok();
  if (tokens > 0x7fffffffLL / heads)
    return fail(BSFP_ERR_UNSUPPORTED, "%s: %lld tokens x %d heads exceed 2^31 - 1 rows", fn,
                (long long)tokens, (int)heads);
  if (!q || !aligned16(q)) return fail(BSFP_ERR_ARG, "%s: q is null or not 16-byte aligned", fn);
  if (!out || !aligned16(out))
    return fail(BSFP_ERR_ARG, "%s: out is null or not 16-byte aligned", fn);
  if (q_stride % 8 || q_stride < 0)
    return fail(BSFP_ERR_ARG, "%s: token stride %lld must be a multiple of 8", fn,
                (long long)q_stride);
  if (!q_starts || (requests > 0 && !kv_lens))
    return fail(BSFP_ERR_ARG, "%s: null q_starts or kv_lens", fn);
  if (requests > 0 && max_pages > 0 && !block_table)
    return fail(BSFP_ERR_ARG, "%s: null block_table", fn);
  const size_t need = kv_attention_workspace(std::min<int64_t>(tokens, max_q), heads, cache->kv_heads,
                                             (int)cache->k->cols, requests);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(BSFP_ERR_ARG, "%s: workspace needs %zu bytes (16-byte aligned), got %zu", fn, need,
                workspace_bytes);
  const KvAttentionArgs a = {q,       q_stride, tokens,   heads, cache,  block_table, max_pages,
                             kv_lens, q_starts, requests, max_q, scale,  window,      out,
                             lse,     workspace};
  return device_status(launch_kv_attention(a, (hipStream_t)stream), fn);
}

}  // extern "C"
