// fa_api.cu -- the C ABI declared in include/fa.h: argument validation, TMA tensor-map
// construction, kernel launches, status reporting.
//
// Everything here runs on the host.  Validation happens before any CUDA call, so a bad
// argument is reported without touching the device.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime_api.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "fa.h"
#include "internal.h"

// Set by kernels when a pipeline wait runs out of time (see sm100.cuh).
__device__ unsigned int g_fa_device_error;

namespace {

thread_local char g_last_error[512] = "";
constexpr int kMaxTrace = 8;
thread_local cudaEvent_t g_trace[kMaxTrace] = {};
thread_local int g_n_trace = 0;

fa_status fail(fa_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

fa_status cuda_fail(cudaError_t e, const char* what) {
  return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// ------------------------------------------------------------------ per-device facts
constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool ready = false;
  int num_sms = 0;
  int cc_major = 0, cc_minor = 0;
  unsigned int* err = nullptr;  // device address of g_fa_device_error
};

std::mutex g_dev_mutex;
DeviceInfo g_dev[kMaxDevices];

fa_status device_info(DeviceInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(FA_ERR_CUDA, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    e = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaGetSymbolAddress(reinterpret_cast<void**>(&d.err), g_fa_device_error);
    if (e != cudaSuccess) return cuda_fail(e, "querying the device");
    d.ready = true;
  }
  *out = d;
  return FA_OK;
}

fa_status require_sm100(const DeviceInfo& d) {
  if (d.cc_major != 10 || d.cc_minor != 0)
    return fail(FA_ERR_UNSUPPORTED,
                "the kernels are built for sm_100a (B200); this device is sm_%d%d",
                d.cc_major, d.cc_minor);
  return FA_OK;
}

// ------------------------------------------------------------------ tensor maps
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// [BH][N][d] bf16 viewed as a 3-D tensor; boxes of 64 elements x `rows` rows x 1 head
// with the 128-byte swizzle that the tensor-core shared-memory descriptors expect (128
// rows for the operand tiles, 32 for the forward's per-warp output stores).  Rows past N
// inside a head read as zeros.
fa_status make_tmap(CUtensorMap* tm, const void* ptr, int BH, int N, int d, int rows = 128) {
  auto fn = encode_fn();
  if (!fn) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                           static_cast<cuuint64_t>(N) * static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return FA_OK;
}

// Packed [tokens][H][d] bf16 viewed as a 3-D tensor {d, H, tokens}; boxes of 64
// elements x 1 head x `rows` tokens, which land in shared memory exactly like the boxes
// above (`rows` rows of 128 bytes, 128-byte swizzle).  Tokens past the end read as zeros.
fa_status make_tmap_packed(CUtensorMap* tm, const void* ptr, int tokens, int H, int d,
                           int rows = 128) {
  auto fn = encode_fn();
  if (!fn) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                           static_cast<cuuint64_t>(H) * static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return FA_OK;
}

// [pages][page][d] bf16 (pages: page number x key head) viewed as a 5-D tensor of (64
// columns, 8 rows, column halves, 8-row groups, pages); boxes of `rows` rows x all columns,
// 128-byte swizzle.
fa_status make_tmap_pages(CUtensorMap* tm, const void* ptr, int pages, int page, int d, int rows) {
  auto fn = encode_fn();
  if (!fn) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(d / 64), static_cast<cuuint64_t>(page / 8),
                        static_cast<cuuint64_t>(pages)};
  cuuint64_t strides[4] = {row, 128, 8 * row, static_cast<cuuint64_t>(page) * row};
  cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(d / 64), static_cast<cuuint32_t>(rows / 8), 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return FA_OK;
}

// [BH][rows] float32 (a per-row statistic padded to whole tiles) viewed as a 3-D tensor
// [1][BH][rows] with boxes of 128 rows, no swizzle.
fa_status make_row_tmap(CUtensorMap* tm, const float* ptr, int BH, int rows) {
  auto fn = encode_fn();
  if (!fn) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(BH), 1};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(rows) * 4,
                           static_cast<cuuint64_t>(rows) * static_cast<cuuint64_t>(BH) * 4};
  cuuint32_t box[3] = {128, 1, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return FA_OK;
}

// ------------------------------------------------------------------ validation
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// [a, a + a_bytes) and [b, b + b_bytes) share a byte
bool overlaps(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// A named argument's bytes (null or empty: absent).
struct Buf {
  const char* name;
  const void* p;
  size_t n;
};

// No output (or workspace) shares a byte with an input or another output.
fa_status check_apart(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
  for (const Buf* o = outs.begin(); o != outs.end(); ++o) {
    if (o->p == nullptr || o->n == 0) continue;
    auto meets = [&](const Buf& x) {
      return x.p != nullptr && x.n > 0 && overlaps(o->p, o->n, x.p, x.n);
    };
    for (const Buf& in : ins)
      if (meets(in)) return fail(FA_ERR_INVALID_ARG, "%s overlaps %s", o->name, in.name);
    for (const Buf* x = outs.begin(); x != o; ++x)
      if (meets(*x)) return fail(FA_ERR_INVALID_ARG, "%s overlaps %s", o->name, x->name);
  }
  return FA_OK;
}

// Longest sequence any call accepts: every length rounded up to whole 256-row units
// still fits a 32-bit int.
constexpr int kMaxRows = 0x7fffffff - 255;

// Checks shared by every call: Nq query rows and Nk key rows per head (Nk == Nq for
// the entry points without the _qk suffix).  Sets *noop when there is nothing to
// compute.
fa_status check_common(int B, int H, int Nq, int Nk, int d, float scale, int causal,
                       bool* noop) {
  if (B < 0 || H < 0 || Nq < 0 || Nk < 0)
    return fail(FA_ERR_INVALID_ARG, "sizes must be non-negative (B=%d H=%d Nq=%d Nk=%d)", B,
                H, Nq, Nk);
  if (d != 64 && d != 128)
    return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (!(std::isfinite(scale) && scale > 0.f))
    return fail(FA_ERR_INVALID_ARG, "scale must be finite and positive");
  if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
  const long long bh = static_cast<long long>(B) * H;
  // work units and row indices are 32-bit on the device, and lengths are rounded up to
  // whole 256-row units in 32-bit arithmetic there
  for (const int n : {Nq, Nk}) {
    if (n > kMaxRows)
      return fail(FA_ERR_INVALID_ARG, "N = %d rows is too large (at most %d)", n, kMaxRows);
    const long long units = (static_cast<long long>(n) + 255) / 256;
    if (bh > 0 && n > 0 && (bh > (1ll << 31) / units || bh * n >= (1ll << 31)))
      return fail(FA_ERR_INVALID_ARG, "B*H*N = %lld rows is too large", bh * n);
  }
  *noop = (bh == 0 || Nq == 0);
  if (*noop) return FA_OK;
  if (Nk == 0) return fail(FA_ERR_INVALID_ARG, "queries need at least one key (Nk=0)");
  if (causal && Nq > Nk)
    return fail(FA_ERR_INVALID_ARG,
                "causal attention needs Nq <= Nk: the queries are the last Nq of the Nk "
                "tokens (Nq=%d Nk=%d)", Nq, Nk);
  return FA_OK;
}

fa_status check_ptr(const void* p, const char* name) {
  if (p == nullptr) return fail(FA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(FA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return FA_OK;
}

#define FA_TRY(x)                      \
  do {                                 \
    fa_status _s = (x);                \
    if (_s != FA_OK) return _s;        \
  } while (0)

// Argument checks of the forward calls (elem = bytes per element of the tensors).
fa_status check_fwd_args(const void* Q, const void* K, const void* V, const void* O,
                         const float* LSE, int B, int H, int Nq, int Nk, int d, float scale,
                         int causal, size_t elem, bool* noop) {
  FA_TRY(check_common(B, H, Nq, Nk, d, scale, causal, noop));
  if (*noop) return FA_OK;
  FA_TRY(check_ptr(Q, "Q"));
  FA_TRY(check_ptr(K, "K"));
  FA_TRY(check_ptr(V, "V"));
  FA_TRY(check_ptr(O, "O"));
  if (LSE != nullptr && (reinterpret_cast<uintptr_t>(LSE) & 3u))
    return fail(FA_ERR_INVALID_ARG, "LSE is not 4-byte aligned");
  const size_t qb = static_cast<size_t>(B) * H * Nq * d * elem;
  const size_t kb = static_cast<size_t>(B) * H * Nk * d * elem;
  if (overlaps(O, qb, Q, qb) || overlaps(O, qb, K, kb) || overlaps(O, qb, V, kb))
    return fail(FA_ERR_INVALID_ARG, "O overlaps an input");
  return FA_OK;
}

// Argument checks of the backward calls (elem = bytes per element of the tensors).
// Q, O, dO, dQ have Nq rows per head; K, V, dK, dV have Nk.
fa_status check_bwd_args(const void* Q, const void* K, const void* V, const void* O,
                         const void* dO, const float* LSE, const void* dQ, const void* dK,
                         const void* dV, int B, int H, int Nq, int Nk, int d, float scale,
                         int causal, const void* workspace, size_t workspace_bytes,
                         size_t elem, bool* noop) {
  FA_TRY(check_common(B, H, Nq, Nk, d, scale, causal, noop));
  if (*noop) return FA_OK;
  FA_TRY(check_ptr(Q, "Q"));
  FA_TRY(check_ptr(K, "K"));
  FA_TRY(check_ptr(V, "V"));
  FA_TRY(check_ptr(O, "O"));
  FA_TRY(check_ptr(dO, "dO"));
  FA_TRY(check_ptr(LSE, "LSE"));
  FA_TRY(check_ptr(dQ, "dQ"));
  FA_TRY(check_ptr(dK, "dK"));
  FA_TRY(check_ptr(dV, "dV"));
  const size_t need = fa_bwd_workspace_bytes(B, H, Nq, d);
  if (need > 0) {
    FA_TRY(check_ptr(workspace, "workspace"));
    if (workspace_bytes < need)
      return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes,
                  need);
  }
  const size_t qb = static_cast<size_t>(B) * H * Nq * d * elem;
  const size_t kb = static_cast<size_t>(B) * H * Nk * d * elem;
  struct Buf {
    const void* p;
    size_t n;
  };
  const Buf ins[5] = {{Q, qb}, {K, kb}, {V, kb}, {O, qb}, {dO, qb}};
  const Buf outs[3] = {{dQ, qb}, {dK, kb}, {dV, kb}};
  for (const Buf& o : outs) {
    for (const Buf& in : ins)
      if (overlaps(o.p, o.n, in.p, in.n))
        return fail(FA_ERR_INVALID_ARG, "a gradient overlaps an input");
    if (need > 0 && overlaps(o.p, o.n, workspace, need))
      return fail(FA_ERR_INVALID_ARG, "a gradient overlaps the workspace");
  }
  if (overlaps(dQ, qb, dK, kb) || overlaps(dQ, qb, dV, kb) || overlaps(dK, kb, dV, kb))
    return fail(FA_ERR_INVALID_ARG, "gradients overlap each other");
  return FA_OK;
}

fa::Problem make_problem(int B, int H, int Nq, int Nk, int d, float scale, int causal,
                         const DeviceInfo& dev, const int* seqlens_q = nullptr,
                         const int* seqlens_k = nullptr, const int* cu_q = nullptr,
                         const int* cu_k = nullptr, int total_q = 0, int total_k = 0) {
  fa::Problem p{};
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.total_q = total_q;
  p.total_k = total_k;
  p.BH = B * H;
  p.N = Nq;
  p.Nk = Nk;
  p.d = d;
  p.scale = scale;
  p.causal = causal;
  p.err = dev.err;
  p.seqlens_q = seqlens_q;
  p.seqlens_k = seqlens_k;
  p.H = H;
  p.trace = g_n_trace ? g_trace : nullptr;
  p.n_trace = g_n_trace;
  return p;
}

// Per-sequence length arrays of the padded-batch calls: both given, 4-byte aligned.
fa_status check_seqlens(const int* seqlens_q, const int* seqlens_k) {
  if (seqlens_q == nullptr || seqlens_k == nullptr)
    return fail(FA_ERR_INVALID_ARG, "seqlens_q and seqlens_k are required");
  if ((reinterpret_cast<uintptr_t>(seqlens_q) | reinterpret_cast<uintptr_t>(seqlens_k)) & 3u)
    return fail(FA_ERR_INVALID_ARG, "seqlens_q and seqlens_k must be 4-byte aligned");
  return FA_OK;
}

// A backward call with keys but no query rows (Nq == 0, or no query tokens in the
// packed layout): no query sees any key, so dK and dV are exactly zero in every key row
// of every sequence; rows past a sequence's key length stay unwritten as elsewhere.
// Its arguments are checked (check_key_grads) before the device is queried.
fa_status check_key_grads(const void* dK, const void* dV, size_t key_bytes) {
  FA_TRY(check_ptr(dK, "dK"));
  FA_TRY(check_ptr(dV, "dV"));
  if (overlaps(dK, key_bytes, dV, key_bytes))
    return fail(FA_ERR_INVALID_ARG, "gradients overlap each other");
  return FA_OK;
}

fa_status zero_key_grads(void* dK, void* dV, const fa::Problem& p, size_t elem,
                         const DeviceInfo& dev, cudaStream_t stream) {
  cudaError_t e = fa::launch_zero_key_rows(dK, dV, p, static_cast<int>(elem), dev.num_sms,
                                           stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the key-gradient zero fill");
  return FA_OK;
}

fa_status fwd_impl(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                   int H, int Nq, int Nk, int d, float scale, int causal, cudaStream_t stream,
                   const int* seqlens_q = nullptr, const int* seqlens_k = nullptr) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_fwd_args(Q, K, V, O, LSE, B, H, Nq, Nk, d, scale, causal, 2, &noop));
  if (noop) return FA_OK;  // empty problem: the pointers are never used (may be NULL)
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  FA_TRY(require_sm100(dev));
  const int BH = B * H;
  CUtensorMap tmQ, tmK, tmV, tmO;
  FA_TRY(make_tmap(&tmQ, Q, BH, Nq, d));
  FA_TRY(make_tmap(&tmK, K, BH, Nk, d));
  FA_TRY(make_tmap(&tmV, V, BH, Nk, d));
  FA_TRY(make_tmap(&tmO, O, BH, Nq, d, 32));
  const fa::Problem p = make_problem(B, H, Nq, Nk, d, scale, causal, dev, seqlens_q, seqlens_k);
  cudaError_t e = fa::launch_fwd_sm100(tmQ, tmK, tmV, tmO, O, LSE, p, dev.num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the forward kernel");
  return FA_OK;
}

fa_status bwd_impl(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                   const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int Nq, int Nk,
                   int d, float scale, int causal, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream, const int* seqlens_q = nullptr,
                   const int* seqlens_k = nullptr) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_bwd_args(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Nq, Nk, d, scale, causal,
                        workspace, workspace_bytes, 2, &noop));
  if (noop) {
    // no work, and then no pointer is used (they may be NULL) -- unless there are keys
    // without queries, whose gradients are zeros to be written
    if (static_cast<long long>(B) * H == 0 || Nk == 0) return FA_OK;
    FA_TRY(check_key_grads(dK, dV, static_cast<size_t>(B) * H * Nk * d * 2));
    DeviceInfo dev;
    FA_TRY(device_info(&dev));
    const fa::Problem p = make_problem(B, H, Nq, Nk, d, scale, causal, dev, seqlens_q,
                                       seqlens_k);
    return zero_key_grads(dK, dV, p, 2, dev, stream);
  }
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  FA_TRY(require_sm100(dev));
  const int BH = B * H;
  CUtensorMap tmQ, tmK, tmV, tmdO, tmL2, tmD, tmdK, tmdV;
  FA_TRY(make_tmap(&tmQ, Q, BH, Nq, d));
  FA_TRY(make_tmap(&tmK, K, BH, Nk, d));
  FA_TRY(make_tmap(&tmV, V, BH, Nk, d));
  FA_TRY(make_tmap(&tmdO, dO, BH, Nq, d));
  FA_TRY(make_tmap(&tmdK, dK, BH, Nk, d, 32));
  FA_TRY(make_tmap(&tmdV, dV, BH, Nk, d, 32));
  const int Npad = static_cast<int>(fa::bwd_padded_rows(Nq));  // Nq <= kMaxRows
  float* ws = static_cast<float*>(workspace);
  FA_TRY(make_row_tmap(&tmD, ws, BH, Npad));
  FA_TRY(make_row_tmap(&tmL2, ws + static_cast<size_t>(BH) * Npad, BH, Npad));
  const fa::Problem p = make_problem(B, H, Nq, Nk, d, scale, causal, dev, seqlens_q, seqlens_k);
  cudaError_t e = fa::launch_bwd_sm100(tmQ, tmK, tmV, tmdO, tmL2, tmD, tmdK, tmdV, O, dO, LSE,
                                       dQ, dK, dV, ws, p, dev.num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the backward kernels");
  return FA_OK;
}

// ------------------------------------------------------------------ modified scores
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The modifications of a _mod call: heads, cap, slopes, prefix lengths, document ranges.
struct ModParams {
  int Hkv;
  float softcap;
  const float* slopes;
  const int* prefix;
  const int* doc_start;
  const int* doc_end;
};

fa_status check_mod(const ModParams& m, int B, int H, int Nq, int Nk, int d, float scale,
                    int causal, bool* noop) {
  FA_TRY(check_common(B, H, Nq, Nk, d, scale, causal, noop));
  if (m.Hkv < 0 || (H > 0 && (m.Hkv == 0 || H % m.Hkv != 0)))
    return fail(FA_ERR_INVALID_ARG, "H=%d query heads cannot share Hkv=%d key heads", H, m.Hkv);
  if (!(std::isfinite(m.softcap) && m.softcap >= 0.f))
    return fail(FA_ERR_INVALID_ARG, "softcap must be finite and non-negative (0: no cap)");
  if (m.softcap > 0.f && !(m.softcap > 1e-9f && m.softcap < 1e9f && scale / m.softcap > 1e-12f &&
                           scale / m.softcap < 1e12f))
    return fail(FA_ERR_INVALID_ARG, "softcap %g is out of range for scale %g",
                static_cast<double>(m.softcap), static_cast<double>(scale));
  if (m.prefix != nullptr && !causal)
    return fail(FA_ERR_INVALID_ARG, "prefix lengths need causal = 1");
  if ((m.doc_start == nullptr) != (m.doc_end == nullptr))
    return fail(FA_ERR_INVALID_ARG, "doc_start and doc_end must be given together");
  if (!aligned4(m.slopes) || !aligned4(m.prefix) || !aligned4(m.doc_start) ||
      !aligned4(m.doc_end))
    return fail(FA_ERR_INVALID_ARG,
                "slopes, prefix, doc_start and doc_end must be 4-byte aligned");
  return FA_OK;
}

fa::Problem make_mod_problem(const ModParams& m, int B, int H, int Nq, int Nk, int d, float scale,
                             int causal, const DeviceInfo& dev) {
  fa::Problem p = make_problem(B, H, Nq, Nk, d, scale, causal, dev);
  p.Hkv = m.Hkv;
  p.softcap = m.softcap;
  p.slopes = m.slopes;
  p.prefix = m.prefix;
  p.doc_start = m.doc_start;
  p.doc_end = m.doc_end;
  return p;
}

fa_status fwd_mod_impl(const void* Q, const void* K, const void* V, void* O, float* LSE,
                       const ModParams& m, int B, int H, int Nq, int Nk, int d, float scale,
                       int causal, cudaStream_t stream) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_mod(m, B, H, Nq, Nk, d, scale, causal, &noop));
  if (noop) return FA_OK;
  FA_TRY(check_ptr(Q, "Q"));
  FA_TRY(check_ptr(K, "K"));
  FA_TRY(check_ptr(V, "V"));
  FA_TRY(check_ptr(O, "O"));
  if (!aligned4(LSE)) return fail(FA_ERR_INVALID_ARG, "LSE is not 4-byte aligned");
  const size_t qb = static_cast<size_t>(B) * H * Nq * d * 2;
  const size_t kb = static_cast<size_t>(B) * m.Hkv * Nk * d * 2;
  const size_t i32 = sizeof(int), keys = static_cast<size_t>(B) * Nk * i32;
  FA_TRY(check_apart({{"O", O, qb}, {"LSE", LSE, static_cast<size_t>(B) * H * Nq * 4}},
                     {{"Q", Q, qb},
                      {"K", K, kb},
                      {"V", V, kb},
                      {"slopes", m.slopes, H * i32},
                      {"prefix", m.prefix, B * i32},
                      {"doc_start", m.doc_start, keys},
                      {"doc_end", m.doc_end, keys}}));
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  FA_TRY(require_sm100(dev));
  CUtensorMap tmQ, tmK, tmV, tmO;
  FA_TRY(make_tmap(&tmQ, Q, B * H, Nq, d));
  FA_TRY(make_tmap(&tmK, K, B * m.Hkv, Nk, d));
  FA_TRY(make_tmap(&tmV, V, B * m.Hkv, Nk, d));
  FA_TRY(make_tmap(&tmO, O, B * H, Nq, d, 32));
  const fa::Problem p = make_mod_problem(m, B, H, Nq, Nk, d, scale, causal, dev);
  cudaError_t e = fa::launch_fwd_sm100(tmQ, tmK, tmV, tmO, O, LSE, p, dev.num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the forward kernel");
  return FA_OK;
}

fa_status bwd_mod_impl(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                       const float* LSE, void* dQ, void* dK, void* dV, const ModParams& m, int B,
                       int H, int Nq, int Nk, int d, float scale, int causal, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_mod(m, B, H, Nq, Nk, d, scale, causal, &noop));
  const size_t qb = static_cast<size_t>(B) * H * Nq * d * 2;
  const size_t kb = static_cast<size_t>(B) * m.Hkv * Nk * d * 2;
  if (noop) {
    // keys without queries have zero gradients (see bwd_impl)
    if (static_cast<long long>(B) * H == 0 || Nk == 0) return FA_OK;
    FA_TRY(check_key_grads(dK, dV, kb));
    FA_TRY(check_apart({{"dK", dK, kb}, {"dV", dV, kb}}, {{"K", K, kb}, {"V", V, kb}}));
    DeviceInfo dev;
    FA_TRY(device_info(&dev));
    const fa::Problem p = make_problem(B, m.Hkv, Nq, Nk, d, scale, causal, dev);
    return zero_key_grads(dK, dV, p, 2, dev, stream);
  }
  FA_TRY(check_ptr(Q, "Q"));
  FA_TRY(check_ptr(K, "K"));
  FA_TRY(check_ptr(V, "V"));
  FA_TRY(check_ptr(O, "O"));
  FA_TRY(check_ptr(dO, "dO"));
  FA_TRY(check_ptr(LSE, "LSE"));
  FA_TRY(check_ptr(dQ, "dQ"));
  FA_TRY(check_ptr(dK, "dK"));
  FA_TRY(check_ptr(dV, "dV"));
  FA_TRY(check_ptr(workspace, "workspace"));
  const size_t need = fa_bwd_workspace_bytes(B, H, Nq, d);
  if (workspace_bytes < need)
    return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes,
                need);
  const size_t i32 = sizeof(int), keys = static_cast<size_t>(B) * Nk * i32;
  FA_TRY(check_apart(
      {{"dQ", dQ, qb}, {"dK", dK, kb}, {"dV", dV, kb}, {"the workspace", workspace, need}},
      {{"Q", Q, qb},
       {"K", K, kb},
       {"V", V, kb},
       {"O", O, qb},
       {"dO", dO, qb},
       {"LSE", LSE, static_cast<size_t>(B) * H * Nq * 4},
       {"slopes", m.slopes, H * i32},
       {"prefix", m.prefix, B * i32},
       {"doc_start", m.doc_start, keys},
       {"doc_end", m.doc_end, keys}}));
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  FA_TRY(require_sm100(dev));
  const int BH = B * H, BHk = B * m.Hkv;
  CUtensorMap tmQ, tmK, tmV, tmdO, tmL2, tmD, tmdK, tmdV;
  FA_TRY(make_tmap(&tmQ, Q, BH, Nq, d));
  FA_TRY(make_tmap(&tmK, K, BHk, Nk, d));
  FA_TRY(make_tmap(&tmV, V, BHk, Nk, d));
  FA_TRY(make_tmap(&tmdO, dO, BH, Nq, d));
  FA_TRY(make_tmap(&tmdK, dK, BHk, Nk, d, 32));
  FA_TRY(make_tmap(&tmdV, dV, BHk, Nk, d, 32));
  const int Npad = static_cast<int>(fa::bwd_padded_rows(Nq));
  float* ws = static_cast<float*>(workspace);
  FA_TRY(make_row_tmap(&tmD, ws, BH, Npad));
  FA_TRY(make_row_tmap(&tmL2, ws + static_cast<size_t>(BH) * Npad, BH, Npad));
  const fa::Problem p = make_mod_problem(m, B, H, Nq, Nk, d, scale, causal, dev);
  cudaError_t e = fa::launch_bwd_sm100(tmQ, tmK, tmV, tmdO, tmL2, tmD, tmdK, tmdV, O, dO, LSE,
                                       dQ, dK, dV, ws, p, dev.num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the backward kernels");
  return FA_OK;
}

// ------------------------------------------------------------------ rotary positions
// A strided view of rows, in bytes: rows of `row` bytes at p + sum of i_k st[k], i_k < n[k].
struct View {
  const void* p;
  long long row, n[3], st[3];
  long long span() const {
    long long last = row;
    for (int k = 0; k < 3; ++k) last += (n[k] - 1) * st[k];
    return last;
  }
  // the same without the dimensions that step by multiples of `period`
  long long span_within(long long period) const {
    long long last = row;
    for (int k = 0; k < 3; ++k)
      if (n[k] > 1 && st[k] % period != 0) last += (n[k] - 1) * st[k];
    return last;
  }
};

View flat_view(const void* p, size_t bytes) {
  return View{p, static_cast<long long>(bytes), {1, 1, 1}, {0, 0, 0}};
}

// Whether two views may share a byte.  They do not if they lie apart, or if their rows,
// taken modulo a stride, do: heads of one fused buffer lie apart modulo its token stride,
// slices of a head-major one modulo its batch stride.
bool may_share(View x, View y) {
  if (!overlaps(x.p, x.span(), y.p, y.span())) return false;
  const long long off = static_cast<const char*>(y.p) - static_cast<const char*>(x.p);
  // a common stride that steps past all that both views cover without it (a pitch between
  // sequences): only equal indices can meet, so one of them stands for all
  for (int pass = 0; pass < 3; ++pass) {
    for (int k = 0; k < 3; ++k) {
      if (x.n[k] <= 1 || y.n[k] <= 1 || x.st[k] != y.st[k]) continue;
      const long long nx = x.n[k], ny = y.n[k];
      x.n[k] = y.n[k] = 1;
      const long long first = off < 0 ? off : 0;
      const long long last = x.span() > off + y.span() ? x.span() : off + y.span();
      if (last - first > x.st[k]) x.n[k] = nx, y.n[k] = ny;
    }
  }
  if (!overlaps(x.p, x.span(), y.p, y.span())) return false;
  for (const View* v : {&x, &y}) {
    for (int k = 0; k < 3; ++k) {
      const long long period = v->st[k];
      if (v->n[k] <= 1 || period <= 0) continue;
      const long long nx = x.span_within(period), ny = y.span_within(period);
      long long at = off % period;
      if (at < 0) at += period;
      if (at >= nx && at + ny <= period) return false;
    }
  }
  return true;
}

// Whether rows of a view may share a byte with one another: each stride has to step past
// all that the smaller ones cover.
bool rows_may_share(const View& x) {
  long long cover = x.row;
  bool done[3] = {x.n[0] <= 1, x.n[1] <= 1, x.n[2] <= 1};
  for (int step = 0; step < 3; ++step) {
    int k = -1;
    for (int i = 0; i < 3; ++i)
      if (!done[i] && (k < 0 || x.st[i] < x.st[k])) k = i;
    if (k < 0) break;
    if (x.st[k] < cover) return true;
    cover += (x.n[k] - 1) * x.st[k];
    done[k] = true;
  }
  return false;
}

// One tensor of heads of a rotary call.  strides: {in b, h, n, out b, h, n} in elements, or
// null for contiguous [B,heads,N,d] on both sides.  view: the input's and the output's.
fa_status rotary_tensor(const char* name, const void* in, void* out, int heads, int B, int N,
                        int d, const long long* strides, int elem, fa::RotaryTensor* x,
                        View view[2]) {
  *x = fa::RotaryTensor{};
  if (heads < 0) return fail(FA_ERR_INVALID_ARG, "%s has %d heads", name, heads);
  if (heads == 0) return FA_OK;
  if (static_cast<long long>(heads) * N > 0x7fffffffll / B)
    return fail(FA_ERR_INVALID_ARG, "%s: heads * tokens is too large", name);
  if (in == nullptr || out == nullptr)
    return fail(FA_ERR_INVALID_ARG, "%s or its output is NULL", name);
  if ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) % elem)
    return fail(FA_ERR_INVALID_ARG, "%s or its output is not aligned to its elements", name);
  const long long dense_n = d, dense_h = dense_n * N, dense_b = dense_h * heads;
  const long long dense[6] = {dense_b, dense_h, dense_n, dense_b, dense_h, dense_n};
  const long long* s = strides != nullptr ? strides : dense;
  for (int o = 0; o < 2; ++o) {
    View& v = view[o];
    v = View{o == 0 ? in : out, static_cast<long long>(d) * elem, {B, heads, N}, {}};
    long long last = d;
    for (int k = 0; k < 3; ++k) {
      const long long st = s[3 * o + k];
      if (st < 0 || st > (1ll << 40))
        return fail(FA_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40]", name);
      if (v.n[k] > 1 && st > ((1ll << 46) - last) / (v.n[k] - 1))
        return fail(FA_ERR_INVALID_ARG, "%s spans too many elements", name);
      last += (v.n[k] - 1) * st;
      v.st[k] = st * elem;
    }
  }
  if (rows_may_share(view[1]))
    return fail(FA_ERR_INVALID_ARG, "%s: rows of the output overlap one another", name);
  bool in_place = in == out;
  for (int k = 0; k < 3; ++k) in_place = in_place && (view[0].n[k] <= 1 || s[k] == s[3 + k]);
  if (!in_place && may_share(view[0], view[1]))
    return fail(FA_ERR_INVALID_ARG, "%s overlaps its output and is not the same tensor", name);
  *x = fa::RotaryTensor{in, out, heads, s[0], s[1], s[2], s[3], s[4], s[5]};
  return FA_OK;
}

fa_status rotary_impl(const void* Q, void* Q_out, const void* K, void* K_out,
                      const float* inv_freq, const int* positions, long long first, int B, int H,
                      int Hkv, int N, int d, int R, int interleaved, int inverse, float mscale,
                      const long long* q_strides, const long long* k_strides, int elem,
                      cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (B < 0 || N < 0)
    return fail(FA_ERR_INVALID_ARG, "sizes must be non-negative (B=%d N=%d)", B, N);
  if (d < 2 || d > 512) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d (2 to 512)", d);
  if (R < 0 || R > d || R % 2)
    return fail(FA_ERR_INVALID_ARG, "R=%d must be even and at most d=%d", R, d);
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return fail(FA_ERR_INVALID_ARG, "interleaved and inverse must be 0 or 1");
  if (!std::isfinite(mscale)) return fail(FA_ERR_INVALID_ARG, "mscale must be finite");
  if (first < -(1ll << 40) || first > (1ll << 40))
    return fail(FA_ERR_INVALID_ARG, "first must be within +-2^40");
  if (static_cast<long long>(B) * N >= (1ll << 31))
    return fail(FA_ERR_INVALID_ARG, "B*N = %lld tokens is too large",
                static_cast<long long>(B) * N);
  if (B == 0 || N == 0) return FA_OK;
  fa::RotaryArgs a{};
  View q[2], k[2];
  FA_TRY(rotary_tensor("Q", Q, Q_out, H, B, N, d, q_strides, elem, &a.x[0], q));
  FA_TRY(rotary_tensor("K", K, K_out, Hkv, B, N, d, k_strides, elem, &a.x[1], k));
  if (H == 0 && Hkv == 0) return FA_OK;
  if (H > 0 && Hkv > 0) {
    if (may_share(q[1], k[1])) return fail(FA_ERR_INVALID_ARG, "the outputs overlap");
    if (may_share(q[1], k[0]) || may_share(k[1], q[0]))
      return fail(FA_ERR_INVALID_ARG, "an output overlaps the other input");
  }
  if (R > 0 && inv_freq == nullptr) return fail(FA_ERR_INVALID_ARG, "inv_freq is NULL");
  if (!aligned4(inv_freq) || !aligned4(positions))
    return fail(FA_ERR_INVALID_ARG, "inv_freq and positions must be 4-byte aligned");
  const View freq = flat_view(inv_freq, static_cast<size_t>(R / 2) * 4);
  const View pos = flat_view(positions, static_cast<size_t>(B) * N * 4);
  for (const View* out : {H > 0 ? &q[1] : nullptr, Hkv > 0 ? &k[1] : nullptr}) {
    if (out == nullptr) continue;
    if ((R > 0 && may_share(*out, freq)) || (positions != nullptr && may_share(*out, pos)))
      return fail(FA_ERR_INVALID_ARG, "an output overlaps inv_freq or positions");
  }
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.first = first;
  a.total = static_cast<long long>(B) * N;
  a.N = N;
  a.d = d;
  a.R = R;
  a.interleaved = interleaved;
  a.copy_rest = (H > 0 && Q != Q_out) || (Hkv > 0 && K != K_out);
  a.mscale = mscale;
  a.sign = inverse ? -1.f : 1.f;
  if (R == 0 && !a.copy_rest) return FA_OK;
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  cudaError_t e = fa::launch_rotary(a, elem, dev.num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the rotary kernel");
  return FA_OK;
}

// ------------------------------------------------------------------ paged cache
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Rows of a key head, its pairs of row tiles, workspace rows of a piece and pieces.
struct TreeSplit {
  long long rows, pairs, piece_rows, pieces;
};

TreeSplit tree_split(int B, int H, int Hkv, int T) {
  TreeSplit s;
  s.rows = static_cast<long long>(H / Hkv) * T;
  s.pairs = (s.rows + 255) / 256;
  s.piece_rows = s.rows <= 128 ? 2 * fa::tree_copies(static_cast<int>(s.rows)) * s.rows : 256;
  s.pieces = fa::kTreeMaxGrid + static_cast<long long>(B) * Hkv * s.pairs;
  return s;
}

fa_status check_tree_sizes(int B, int H, int Hkv, int T, int d) {
  if (B < 0 || H < 0 || T < 0)
    return fail(FA_ERR_INVALID_ARG, "sizes must be non-negative (B=%d H=%d T=%d)", B, H, T);
  if (d != 64 && d != 128)
    return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (T > 64) return fail(FA_ERR_UNSUPPORTED, "T=%d drafted tokens (at most 64)", T);
  if (B > fa::kTreeMaxBatch)
    return fail(FA_ERR_UNSUPPORTED, "B=%d sequences (at most %d)", B, fa::kTreeMaxBatch);
  if (Hkv < 0 || (H > 0 && (Hkv == 0 || H % Hkv != 0)))
    return fail(FA_ERR_INVALID_ARG, "H=%d query heads cannot share Hkv=%d key heads", H, Hkv);
  if (H > 65536) return fail(FA_ERR_INVALID_ARG, "H=%d heads is too large", H);
  if (static_cast<long long>(B) * H * T >= (1ll << 31))
    return fail(FA_ERR_INVALID_ARG, "B*H*T rows is too large");
  return FA_OK;
}

fa_status tree_impl(const void* Q, const void* K_cache, const void* V_cache, void* O, float* LSE,
                    const int* block_table, const int* cache_lens, const int* seqlens_q,
                    const long long* tree_mask, int B, int H, int Hkv, int T, int num_pages,
                    int page, int max_pages, int d, float scale, float softcap, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
  g_last_error[0] = '\0';
  FA_TRY(check_tree_sizes(B, H, Hkv, T, d));
  if (!(std::isfinite(scale) && scale > 0.f))
    return fail(FA_ERR_INVALID_ARG, "scale must be finite and positive");
  ModParams m{Hkv, softcap, nullptr, nullptr, nullptr, nullptr};
  bool noop = false;
  FA_TRY(check_mod(m, 0, H, 0, 0, d, scale, 0, &noop));
  if (num_pages < 0 || max_pages < 0)
    return fail(FA_ERR_INVALID_ARG, "num_pages and max_pages must be non-negative");
  if (page < 8 || page > (1 << 24) || (page < 128 ? 128 % page != 0 : page % 128 != 0))
    return fail(FA_ERR_UNSUPPORTED, "page size %d (8, 16, 32, 64 or a multiple of 128)", page);
  if (B == 0 || H == 0 || T == 0) return FA_OK;
  const TreeSplit sp = tree_split(B, H, Hkv, T);
  const long long max_len = static_cast<long long>(max_pages) * page;
  if (max_len >= (1ll << 30) ||
      static_cast<long long>(B) * Hkv * sp.pairs > (1ll << 30) / (max_len / 128 + 1) ||
      static_cast<long long>(num_pages) * Hkv >= (1ll << 31))
    return fail(FA_ERR_INVALID_ARG, "the cache is too large");
  FA_TRY(check_ptr(Q, "Q"));
  FA_TRY(check_ptr(O, "O"));
  if (num_pages > 0) {
    FA_TRY(check_ptr(K_cache, "K_cache"));
    FA_TRY(check_ptr(V_cache, "V_cache"));
  } else if (max_pages > 0) {
    return fail(FA_ERR_INVALID_ARG, "a block table with max_pages=%d needs pages", max_pages);
  }
  if (cache_lens == nullptr || (max_pages > 0 && block_table == nullptr))
    return fail(FA_ERR_INVALID_ARG, "block_table and cache_lens are required");
  if (!aligned4(block_table) || !aligned4(cache_lens) || !aligned4(seqlens_q) || !aligned4(LSE))
    return fail(FA_ERR_INVALID_ARG,
                "block_table, cache_lens, seqlens_q and LSE must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(tree_mask) & 7u)
    return fail(FA_ERR_INVALID_ARG, "tree_mask is not 8-byte aligned");
  FA_TRY(check_ptr(workspace, "workspace"));
  const size_t need = fa_fwd_tree_workspace_bytes(B, H, Hkv, T, d);
  if (workspace_bytes < need)
    return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes,
                need);
  const size_t qb = static_cast<size_t>(B) * H * T * d * 2;
  const size_t cb = static_cast<size_t>(num_pages) * Hkv * page * d * 2;
  const size_t rows = static_cast<size_t>(B) * T, i32 = sizeof(int);
  FA_TRY(check_apart({{"O", O, qb}, {"LSE", LSE, rows * H * 4}, {"the workspace", workspace, need}},
                     {{"Q", Q, qb},
                      {"K_cache", K_cache, cb},
                      {"V_cache", V_cache, cb},
                      {"block_table", block_table, static_cast<size_t>(B) * max_pages * i32},
                      {"cache_lens", cache_lens, B * i32},
                      {"seqlens_q", seqlens_q, B * i32},
                      {"tree_mask", tree_mask, rows * 8}}));
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  FA_TRY(require_sm100(dev));
  fa::TreeArgs a{};
  a.err = dev.err;
  a.block_table = block_table;
  a.cache_lens = cache_lens;
  a.seqlens_q = seqlens_q;
  a.tree_mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  a.B = B;
  a.Hkv = Hkv;
  a.T = T;
  a.rows = static_cast<int>(sp.rows);
  a.pairs = static_cast<int>(sp.pairs);
  a.piece_rows = static_cast<int>(sp.piece_rows);
  a.page = page;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.max_len = static_cast<int>(max_len);
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.softcap = softcap;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t slots = static_cast<size_t>(sp.pieces) * sp.piece_rows;
  a.parts = reinterpret_cast<float*>(ws);
  a.stats = reinterpret_cast<float2*>(ws + round256(slots * d * 4));
  a.prefix_out = reinterpret_cast<int*>(ws + round256(slots * d * 4) + round256(slots * 8));
  CUtensorMap tmQ, tmK, tmV;
  FA_TRY(make_tmap(&tmQ, Q, B * Hkv, a.rows, d, 128 / fa::tree_copies(a.rows)));
  // (without a page there is no token to load: any valid address does)
  const void* kc = num_pages > 0 ? K_cache : Q;
  const void* vc = num_pages > 0 ? V_cache : Q;
  const int box = page < 128 ? page : 128;
  FA_TRY(make_tmap_pages(&tmK, kc, num_pages > 0 ? num_pages * Hkv : 1, page, d, box));
  FA_TRY(make_tmap_pages(&tmV, vc, num_pages > 0 ? num_pages * Hkv : 1, page, d, box));
  const int grid = dev.num_sms < fa::kTreeMaxGrid ? dev.num_sms : fa::kTreeMaxGrid;
  cudaError_t e = fa::launch_tree_sm100(tmQ, tmK, tmV, O, LSE, a, d, grid, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the tree-attention kernels");
  return FA_OK;
}

// The start-token arrays of the packed-layout calls: both given, 4-byte aligned.
fa_status check_cu(const int* cu_q, const int* cu_k) {
  if (cu_q == nullptr || cu_k == nullptr)
    return fail(FA_ERR_INVALID_ARG, "cu_seqlens_q and cu_seqlens_k are required");
  if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k)) & 3u)
    return fail(FA_ERR_INVALID_ARG, "cu_seqlens_q and cu_seqlens_k must be 4-byte aligned");
  return FA_OK;
}

// Checks of the packed-layout calls: lengths, totals and the start-token arrays.
fa_status check_packed(const int* cu_q, const int* cu_k, int B, int H, int max_q, int max_k,
                       int total_q, int total_k, int d, float scale, int causal, bool* noop) {
  FA_TRY(check_common(B, H, max_q, max_k, d, scale, causal, noop));
  if (total_q < 0 || total_k < 0)
    return fail(FA_ERR_INVALID_ARG, "token totals must be non-negative");
  const long long h = H;
  if (h * total_q >= (1ll << 31) || h * total_k >= (1ll << 31))
    return fail(FA_ERR_INVALID_ARG, "H * tokens is too large");
  if (*noop || total_q == 0) {
    *noop = true;
    return FA_OK;
  }
  return check_cu(cu_q, cu_k);
}

// Pointer and overlap checks of the packed-layout forward calls (elem = bytes per
// element of Q, K, V, O).
fa_status check_packed_fwd_ptrs(const void* Q, const void* K, const void* V, const void* O,
                                const float* LSE, int H, int d, int total_q, int total_k,
                                size_t elem) {
  FA_TRY(check_ptr(Q, "Q"));
  FA_TRY(check_ptr(K, "K"));
  FA_TRY(check_ptr(V, "V"));
  FA_TRY(check_ptr(O, "O"));
  if (LSE != nullptr && (reinterpret_cast<uintptr_t>(LSE) & 3u))
    return fail(FA_ERR_INVALID_ARG, "LSE is not 4-byte aligned");
  const size_t qb = static_cast<size_t>(total_q) * H * d * elem;
  const size_t kb = static_cast<size_t>(total_k) * H * d * elem;
  if (overlaps(O, qb, Q, qb) || overlaps(O, qb, K, kb) || overlaps(O, qb, V, kb))
    return fail(FA_ERR_INVALID_ARG, "O overlaps an input");
  return FA_OK;
}

// Pointer, workspace and overlap checks of the packed-layout backward calls.
fa_status check_packed_bwd_ptrs(const void* Q, const void* K, const void* V, const void* O,
                                const void* dO, const float* LSE, const void* dQ,
                                const void* dK, const void* dV, int H, int d, int total_q,
                                int total_k, const void* workspace, size_t need,
                                size_t workspace_bytes, size_t elem) {
  FA_TRY(check_ptr(Q, "Q"));
  FA_TRY(check_ptr(K, "K"));
  FA_TRY(check_ptr(V, "V"));
  FA_TRY(check_ptr(O, "O"));
  FA_TRY(check_ptr(dO, "dO"));
  FA_TRY(check_ptr(LSE, "LSE"));
  FA_TRY(check_ptr(dQ, "dQ"));
  FA_TRY(check_ptr(dK, "dK"));
  FA_TRY(check_ptr(dV, "dV"));
  FA_TRY(check_ptr(workspace, "workspace"));
  if (workspace_bytes < need)
    return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes,
                need);
  const size_t qb = static_cast<size_t>(total_q) * H * d * elem;
  const size_t kb = static_cast<size_t>(total_k) * H * d * elem;
  struct Buf {
    const void* p;
    size_t n;
  };
  const Buf ins[5] = {{Q, qb}, {K, kb}, {V, kb}, {O, qb}, {dO, qb}};
  const Buf outs[3] = {{dQ, qb}, {dK, kb}, {dV, kb}};
  for (const Buf& o : outs) {
    for (const Buf& in : ins)
      if (overlaps(o.p, o.n, in.p, in.n))
        return fail(FA_ERR_INVALID_ARG, "a gradient overlaps an input");
    if (overlaps(o.p, o.n, workspace, need))
      return fail(FA_ERR_INVALID_ARG, "a gradient overlaps the workspace");
  }
  if (overlaps(dQ, qb, dK, kb) || overlaps(dQ, qb, dV, kb) || overlaps(dK, kb, dV, kb))
    return fail(FA_ERR_INVALID_ARG, "gradients overlap each other");
  return FA_OK;
}

// float32 forward, dense or padded layout (seqlens null: every row of every head).
fa_status fwd_f32_impl(const float* Q, const float* K, const float* V, float* O, float* LSE,
                       int B, int H, int Nq, int Nk, int d, float scale, int causal,
                       cudaStream_t stream, const int* seqlens_q = nullptr,
                       const int* seqlens_k = nullptr) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_fwd_args(Q, K, V, O, LSE, B, H, Nq, Nk, d, scale, causal, 4, &noop));
  if (noop) return FA_OK;  // empty problem: the pointers are never used (may be NULL)
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  const fa::Problem p = make_problem(B, H, Nq, Nk, d, scale, causal, dev, seqlens_q, seqlens_k);
  cudaError_t e = fa::launch_fwd_f32(Q, K, V, O, LSE, p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the float32 forward kernel");
  return FA_OK;
}

// float32 backward, dense or padded layout.
fa_status bwd_f32_impl(const float* Q, const float* K, const float* V, const float* O,
                       const float* dO, const float* LSE, float* dQ, float* dK, float* dV,
                       int B, int H, int Nq, int Nk, int d, float scale, int causal,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream,
                       const int* seqlens_q = nullptr, const int* seqlens_k = nullptr) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_bwd_args(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Nq, Nk, d, scale, causal,
                        workspace, workspace_bytes, 4, &noop));
  if (noop) {
    // as in bwd_impl: keys without queries get zero gradients
    if (static_cast<long long>(B) * H == 0 || Nk == 0) return FA_OK;
    FA_TRY(check_key_grads(dK, dV, static_cast<size_t>(B) * H * Nk * d * 4));
    DeviceInfo dev;
    FA_TRY(device_info(&dev));
    const fa::Problem p = make_problem(B, H, Nq, Nk, d, scale, causal, dev, seqlens_q,
                                       seqlens_k);
    return zero_key_grads(dK, dV, p, 4, dev, stream);
  }
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  const fa::Problem p = make_problem(B, H, Nq, Nk, d, scale, causal, dev, seqlens_q, seqlens_k);
  cudaError_t e = fa::launch_bwd_f32(Q, K, V, O, dO, LSE, dQ, dK, dV,
                                     static_cast<float*>(workspace), p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the float32 backward kernels");
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_abi_version(void) { return 1; }

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT";
  }
  return "FA_ERR_UNKNOWN";
}

const char* fa_last_error_message(void) { return g_last_error; }

fa_status fa_trace_events(cudaEvent_t* events, int n) {
  g_last_error[0] = '\0';
  if (n < 0 || n > kMaxTrace || (n > 0 && events == nullptr))
    return fail(FA_ERR_INVALID_ARG, "fa_trace_events: n=%d (0..%d, events non-NULL)", n,
                kMaxTrace);
  for (int k = 0; k < n; ++k) g_trace[k] = events[k];
  g_n_trace = n;
  return FA_OK;
}

fa_status fa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                 int N, int d, float scale, int causal, cudaStream_t stream) {
  return fwd_impl(Q, K, V, O, LSE, B, H, N, N, d, scale, causal, stream);
}

fa_status fa_fwd_qk(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                    int H, int Nq, int Nk, int d, float scale, int causal,
                    cudaStream_t stream) {
  return fwd_impl(Q, K, V, O, LSE, B, H, Nq, Nk, d, scale, causal, stream);
}

fa_status fa_fwd_varlen(const void* Q, const void* K, const void* V, void* O, float* LSE,
                        const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq,
                        int Nk, int d, float scale, int causal, cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (B > 0 && H > 0 && Nq > 0) FA_TRY(check_seqlens(seqlens_q, seqlens_k));
  return fwd_impl(Q, K, V, O, LSE, B, H, Nq, Nk, d, scale, causal, stream, seqlens_q,
                  seqlens_k);
}

fa_status fa_fwd_packed(const void* Q, const void* K, const void* V, void* O, float* LSE,
                        const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int H,
                        int max_seqlen_q, int max_seqlen_k, int total_q, int total_k, int d,
                        float scale, int causal, cudaStream_t stream) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_packed(cu_seqlens_q, cu_seqlens_k, B, H, max_seqlen_q, max_seqlen_k, total_q,
                      total_k, d, scale, causal, &noop));
  if (noop) return FA_OK;
  FA_TRY(check_packed_fwd_ptrs(Q, K, V, O, LSE, H, d, total_q, total_k, 2));
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  FA_TRY(require_sm100(dev));
  CUtensorMap tmQ, tmK, tmV, tmO;
  FA_TRY(make_tmap_packed(&tmQ, Q, total_q, H, d));
  FA_TRY(make_tmap_packed(&tmK, K, total_k, H, d));
  FA_TRY(make_tmap_packed(&tmV, V, total_k, H, d));
  FA_TRY(make_tmap_packed(&tmO, O, total_q, H, d, 32));
  const fa::Problem p = make_problem(B, H, max_seqlen_q, max_seqlen_k, d, scale, causal, dev,
                                     nullptr, nullptr, cu_seqlens_q, cu_seqlens_k, total_q,
                                     total_k);
  cudaError_t e = fa::launch_fwd_sm100(tmQ, tmK, tmV, tmO, O, LSE, p, dev.num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the forward kernel");
  return FA_OK;
}

fa_status fa_bwd_packed(const void* Q, const void* K, const void* V, const void* O,
                        const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                        const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int H,
                        int max_seqlen_q, int max_seqlen_k, int total_q, int total_k, int d,
                        float scale, int causal, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_packed(cu_seqlens_q, cu_seqlens_k, B, H, max_seqlen_q, max_seqlen_k, total_q,
                      total_k, d, scale, causal, &noop));
  if (noop) {
    // keys without queries get zero gradients (see bwd_impl)
    if (static_cast<long long>(B) * H == 0 || total_k == 0 || max_seqlen_k == 0) return FA_OK;
    FA_TRY(check_cu(cu_seqlens_q, cu_seqlens_k));
    FA_TRY(check_key_grads(dK, dV, static_cast<size_t>(total_k) * H * d * 2));
    DeviceInfo dev;
    FA_TRY(device_info(&dev));
    const fa::Problem p = make_problem(B, H, max_seqlen_q, max_seqlen_k, d, scale, causal, dev,
                                       nullptr, nullptr, cu_seqlens_q, cu_seqlens_k, total_q,
                                       total_k);
    return zero_key_grads(dK, dV, p, 2, dev, stream);
  }
  const size_t need = fa_bwd_workspace_bytes(B, H, max_seqlen_q, d);
  FA_TRY(check_packed_bwd_ptrs(Q, K, V, O, dO, LSE, dQ, dK, dV, H, d, total_q, total_k,
                               workspace, need, workspace_bytes, 2));
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  FA_TRY(require_sm100(dev));
  const int BH = B * H;
  CUtensorMap tmQ, tmK, tmV, tmdO, tmL2, tmD, tmdK, tmdV;
  FA_TRY(make_tmap_packed(&tmQ, Q, total_q, H, d));
  FA_TRY(make_tmap_packed(&tmK, K, total_k, H, d));
  FA_TRY(make_tmap_packed(&tmV, V, total_k, H, d));
  FA_TRY(make_tmap_packed(&tmdO, dO, total_q, H, d));
  FA_TRY(make_tmap_packed(&tmdK, dK, total_k, H, d, 32));
  FA_TRY(make_tmap_packed(&tmdV, dV, total_k, H, d, 32));
  const int Npad = static_cast<int>(fa::bwd_padded_rows(max_seqlen_q));
  float* ws = static_cast<float*>(workspace);
  FA_TRY(make_row_tmap(&tmD, ws, BH, Npad));
  FA_TRY(make_row_tmap(&tmL2, ws + static_cast<size_t>(BH) * Npad, BH, Npad));
  const fa::Problem p = make_problem(B, H, max_seqlen_q, max_seqlen_k, d, scale, causal, dev,
                                     nullptr, nullptr, cu_seqlens_q, cu_seqlens_k, total_q,
                                     total_k);
  cudaError_t e = fa::launch_bwd_sm100(tmQ, tmK, tmV, tmdO, tmL2, tmD, tmdK, tmdV, O, dO, LSE,
                                       dQ, dK, dV, ws, p, dev.num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the backward kernels");
  return FA_OK;
}

fa_status fa_fwd_f32(const float* Q, const float* K, const float* V, float* O, float* LSE,
                     int B, int H, int N, int d, float scale, int causal,
                     cudaStream_t stream) {
  return fwd_f32_impl(Q, K, V, O, LSE, B, H, N, N, d, scale, causal, stream);
}

fa_status fa_fwd_f32_qk(const float* Q, const float* K, const float* V, float* O, float* LSE,
                        int B, int H, int Nq, int Nk, int d, float scale, int causal,
                        cudaStream_t stream) {
  return fwd_f32_impl(Q, K, V, O, LSE, B, H, Nq, Nk, d, scale, causal, stream);
}

fa_status fa_fwd_f32_varlen(const float* Q, const float* K, const float* V, float* O,
                            float* LSE, const int* seqlens_q, const int* seqlens_k, int B,
                            int H, int Nq, int Nk, int d, float scale, int causal,
                            cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (B > 0 && H > 0 && Nq > 0) FA_TRY(check_seqlens(seqlens_q, seqlens_k));
  return fwd_f32_impl(Q, K, V, O, LSE, B, H, Nq, Nk, d, scale, causal, stream, seqlens_q,
                      seqlens_k);
}

fa_status fa_fwd_f32_packed(const float* Q, const float* K, const float* V, float* O,
                            float* LSE, const int* cu_seqlens_q, const int* cu_seqlens_k,
                            int B, int H, int max_seqlen_q, int max_seqlen_k, int total_q,
                            int total_k, int d, float scale, int causal,
                            cudaStream_t stream) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_packed(cu_seqlens_q, cu_seqlens_k, B, H, max_seqlen_q, max_seqlen_k, total_q,
                      total_k, d, scale, causal, &noop));
  if (noop) return FA_OK;
  FA_TRY(check_packed_fwd_ptrs(Q, K, V, O, LSE, H, d, total_q, total_k, 4));
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  const fa::Problem p = make_problem(B, H, max_seqlen_q, max_seqlen_k, d, scale, causal, dev,
                                     nullptr, nullptr, cu_seqlens_q, cu_seqlens_k, total_q,
                                     total_k);
  cudaError_t e = fa::launch_fwd_f32(Q, K, V, O, LSE, p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the float32 forward kernel");
  return FA_OK;
}

size_t fa_bwd_workspace_bytes(int B, int H, int N, int d) {
  (void)d;
  if (B <= 0 || H <= 0 || N <= 0) return 0;
  // D and LSE*log2(e), one float each per query row, rows padded to whole 128-row tiles
  const size_t raw = 2 * static_cast<size_t>(B) * H *
                    static_cast<size_t>(fa::bwd_padded_rows(N)) * sizeof(float);
  return (raw + 255) / 256 * 256;
}

fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                 const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int N, int d,
                 float scale, int causal, void* workspace, size_t workspace_bytes,
                 cudaStream_t stream) {
  return bwd_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, N, d, scale, causal, workspace,
                  workspace_bytes, stream);
}

fa_status fa_bwd_qk(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                    const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int Nq,
                    int Nk, int d, float scale, int causal, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
  return bwd_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Nq, Nk, d, scale, causal, workspace,
                  workspace_bytes, stream);
}

fa_status fa_bwd_varlen(const void* Q, const void* K, const void* V, const void* O,
                        const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                        const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq,
                        int Nk, int d, float scale, int causal, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (B > 0 && H > 0 && (Nq > 0 || Nk > 0)) FA_TRY(check_seqlens(seqlens_q, seqlens_k));
  return bwd_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Nq, Nk, d, scale, causal, workspace,
                  workspace_bytes, stream, seqlens_q, seqlens_k);
}

fa_status fa_bwd_f32(const float* Q, const float* K, const float* V, const float* O,
                     const float* dO, const float* LSE, float* dQ, float* dK, float* dV, int B,
                     int H, int N, int d, float scale, int causal, void* workspace,
                     size_t workspace_bytes, cudaStream_t stream) {
  return bwd_f32_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, N, d, scale, causal,
                      workspace, workspace_bytes, stream);
}

fa_status fa_bwd_f32_qk(const float* Q, const float* K, const float* V, const float* O,
                        const float* dO, const float* LSE, float* dQ, float* dK, float* dV,
                        int B, int H, int Nq, int Nk, int d, float scale, int causal,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return bwd_f32_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Nq, Nk, d, scale, causal,
                      workspace, workspace_bytes, stream);
}

fa_status fa_bwd_f32_varlen(const float* Q, const float* K, const float* V, const float* O,
                            const float* dO, const float* LSE, float* dQ, float* dK,
                            float* dV, const int* seqlens_q, const int* seqlens_k, int B,
                            int H, int Nq, int Nk, int d, float scale, int causal,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (B > 0 && H > 0 && (Nq > 0 || Nk > 0)) FA_TRY(check_seqlens(seqlens_q, seqlens_k));
  return bwd_f32_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Nq, Nk, d, scale, causal,
                      workspace, workspace_bytes, stream, seqlens_q, seqlens_k);
}

fa_status fa_bwd_f32_packed(const float* Q, const float* K, const float* V, const float* O,
                            const float* dO, const float* LSE, float* dQ, float* dK,
                            float* dV, const int* cu_seqlens_q, const int* cu_seqlens_k,
                            int B, int H, int max_seqlen_q, int max_seqlen_k, int total_q,
                            int total_k, int d, float scale, int causal, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_packed(cu_seqlens_q, cu_seqlens_k, B, H, max_seqlen_q, max_seqlen_k, total_q,
                      total_k, d, scale, causal, &noop));
  if (noop) {
    // keys without queries get zero gradients (see bwd_impl)
    if (static_cast<long long>(B) * H == 0 || total_k == 0 || max_seqlen_k == 0) return FA_OK;
    FA_TRY(check_cu(cu_seqlens_q, cu_seqlens_k));
    FA_TRY(check_key_grads(dK, dV, static_cast<size_t>(total_k) * H * d * 4));
    DeviceInfo dev;
    FA_TRY(device_info(&dev));
    const fa::Problem p = make_problem(B, H, max_seqlen_q, max_seqlen_k, d, scale, causal, dev,
                                       nullptr, nullptr, cu_seqlens_q, cu_seqlens_k, total_q,
                                       total_k);
    return zero_key_grads(dK, dV, p, 4, dev, stream);
  }
  const size_t need = fa_bwd_workspace_bytes(B, H, max_seqlen_q, d);
  FA_TRY(check_packed_bwd_ptrs(Q, K, V, O, dO, LSE, dQ, dK, dV, H, d, total_q, total_k,
                               workspace, need, workspace_bytes, 4));
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  const fa::Problem p = make_problem(B, H, max_seqlen_q, max_seqlen_k, d, scale, causal, dev,
                                     nullptr, nullptr, cu_seqlens_q, cu_seqlens_k, total_q,
                                     total_k);
  cudaError_t e = fa::launch_bwd_f32(Q, K, V, O, dO, LSE, dQ, dK, dV,
                                     static_cast<float*>(workspace), p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the float32 backward kernels");
  return FA_OK;
}

fa_status fa_merge(float* O_acc, float* LSE_acc, const void* O_part, const float* LSE_part,
                   void* O_out, int B, int H, int N, int d, cudaStream_t stream) {
  g_last_error[0] = '\0';
  bool noop = false;
  FA_TRY(check_common(B, H, N, N, d, 1.f, 0, &noop));
  if (noop) return FA_OK;  // empty problem: the pointers are never used (may be NULL)
  FA_TRY(check_ptr(O_acc, "O_acc"));
  FA_TRY(check_ptr(O_part, "O_part"));
  if (O_out != nullptr) FA_TRY(check_ptr(O_out, "O_out"));
  if (LSE_acc == nullptr || LSE_part == nullptr)
    return fail(FA_ERR_INVALID_ARG, "LSE_acc and LSE_part are required");
  if ((reinterpret_cast<uintptr_t>(LSE_acc) | reinterpret_cast<uintptr_t>(LSE_part)) & 3u)
    return fail(FA_ERR_INVALID_ARG, "LSE_acc and LSE_part must be 4-byte aligned");
  const size_t rows = static_cast<size_t>(B) * H * N;
  const size_t acc_b = rows * d * 4, part_b = rows * d * 2, lse_b = rows * 4;
  if (overlaps(O_acc, acc_b, O_part, part_b) || overlaps(O_acc, acc_b, LSE_part, lse_b) ||
      overlaps(LSE_acc, lse_b, O_part, part_b) || overlaps(LSE_acc, lse_b, LSE_part, lse_b) ||
      overlaps(O_acc, acc_b, LSE_acc, lse_b))
    return fail(FA_ERR_INVALID_ARG, "the accumulator overlaps the partial result");
  if (O_out != nullptr &&
      (overlaps(O_out, part_b, O_acc, acc_b) || overlaps(O_out, part_b, LSE_acc, lse_b) ||
       overlaps(O_out, part_b, LSE_part, lse_b)))
    return fail(FA_ERR_INVALID_ARG, "O_out overlaps the accumulator");
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  const fa::Problem p = make_problem(B, H, N, N, d, 1.f, 0, dev);
  cudaError_t e = fa::launch_merge(O_acc, LSE_acc, O_part, LSE_part, O_out, p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the merge kernel");
  return FA_OK;
}

fa_status fa_accumulate(float* acc, const void* part, void* out, size_t n,
                        cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (n == 0) return FA_OK;
  if (n % 8 != 0) return fail(FA_ERR_INVALID_ARG, "n=%zu is not a multiple of 8", n);
  if (n >= (size_t(1) << 40)) return fail(FA_ERR_INVALID_ARG, "n=%zu is too large", n);
  FA_TRY(check_ptr(acc, "acc"));
  FA_TRY(check_ptr(part, "part"));
  if (out != nullptr) FA_TRY(check_ptr(out, "out"));
  if (overlaps(acc, n * 4, part, n * 2) ||
      (out != nullptr && (overlaps(out, n * 2, acc, n * 4) || overlaps(out, n * 2, part, n * 2))))
    return fail(FA_ERR_INVALID_ARG, "acc, part and out must not overlap");
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  const fa::Problem p = make_problem(1, 1, 1, 1, 64, 1.f, 0, dev);
  cudaError_t e = fa::launch_accumulate(acc, part, out, static_cast<long long>(n), p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the accumulate kernel");
  return FA_OK;
}

fa_status fa_selftest_timeout(long long limit_cycles, cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (limit_cycles < 0 || limit_cycles > (1ll << 34))
    return fail(FA_ERR_INVALID_ARG, "limit_cycles=%lld out of range (0 .. 2^34)", limit_cycles);
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  const fa::Problem p = make_problem(1, 1, 1, 1, 64, 1.f, 0, dev);
  cudaError_t e = fa::launch_timeout_probe(limit_cycles, p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the timeout probe");
  return FA_OK;
}

fa_status fa_doc_ranges(const int* doc_ids, int* doc_start, int* doc_end, int B, int N,
                        cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (B < 0 || N < 0)
    return fail(FA_ERR_INVALID_ARG, "sizes must be non-negative (B=%d N=%d)", B, N);
  if (N > (1 << 30) || static_cast<long long>(B) * N >= (1ll << 31))
    return fail(FA_ERR_INVALID_ARG, "B*N = %lld tokens is too large", static_cast<long long>(B) * N);
  if (B == 0 || N == 0) return FA_OK;
  if (doc_ids == nullptr || doc_start == nullptr || doc_end == nullptr)
    return fail(FA_ERR_INVALID_ARG, "doc_ids, doc_start and doc_end are required");
  if (!aligned4(doc_ids) || !aligned4(doc_start) || !aligned4(doc_end))
    return fail(FA_ERR_INVALID_ARG, "doc_ids, doc_start and doc_end must be 4-byte aligned");
  const size_t n = static_cast<size_t>(B) * N * 4;
  if (overlaps(doc_start, n, doc_ids, n) || overlaps(doc_end, n, doc_ids, n) ||
      overlaps(doc_start, n, doc_end, n))
    return fail(FA_ERR_INVALID_ARG, "doc_ids, doc_start and doc_end overlap");
  cudaError_t e = fa::launch_doc_ranges(doc_ids, doc_start, doc_end, B, N, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the document-range kernel");
  return FA_OK;
}

fa_status fa_rotary(const void* Q, void* Q_out, const void* K, void* K_out,
                    const float* inv_freq, const int* positions, long long first, int B, int H,
                    int Hkv, int N, int d, int R, int interleaved, int inverse, float mscale,
                    const long long* q_strides, const long long* k_strides,
                    cudaStream_t stream) {
  return rotary_impl(Q, Q_out, K, K_out, inv_freq, positions, first, B, H, Hkv, N, d, R,
                     interleaved, inverse, mscale, q_strides, k_strides, 2, stream);
}

fa_status fa_rotary_f32(const float* Q, float* Q_out, const float* K, float* K_out,
                        const float* inv_freq, const int* positions, long long first, int B,
                        int H, int Hkv, int N, int d, int R, int interleaved, int inverse,
                        float mscale, const long long* q_strides, const long long* k_strides,
                        cudaStream_t stream) {
  return rotary_impl(Q, Q_out, K, K_out, inv_freq, positions, first, B, H, Hkv, N, d, R,
                     interleaved, inverse, mscale, q_strides, k_strides, 4, stream);
}

size_t fa_fwd_tree_workspace_bytes(int B, int H, int Hkv, int T, int d) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0 || T <= 0 || d <= 0) return 0;
  const TreeSplit s = tree_split(B, H, Hkv, T);
  const size_t slots = static_cast<size_t>(s.pieces) * s.piece_rows;
  return round256(slots * d * 4) + round256(slots * 8) + round256((static_cast<size_t>(B) + 1) * 4);
}

fa_status fa_fwd_tree(const void* Q, const void* K_cache, const void* V_cache, void* O, float* LSE,
                      const int* block_table, const int* cache_lens, const int* seqlens_q,
                      const long long* tree_mask, int B, int H, int Hkv, int T, int num_pages,
                      int page, int max_pages, int d, float scale, float softcap, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  return tree_impl(Q, K_cache, V_cache, O, LSE, block_table, cache_lens, seqlens_q, tree_mask, B,
                   H, Hkv, T, num_pages, page, max_pages, d, scale, softcap, workspace,
                   workspace_bytes, stream);
}

fa_status fa_fwd_mod(const void* Q, const void* K, const void* V, void* O, float* LSE,
                     const float* slopes, const int* prefix, const int* doc_start,
                     const int* doc_end, int B, int H, int Hkv, int Nq, int Nk, int d,
                     float scale, int causal, float softcap, cudaStream_t stream) {
  const ModParams m{Hkv, softcap, slopes, prefix, doc_start, doc_end};
  return fwd_mod_impl(Q, K, V, O, LSE, m, B, H, Nq, Nk, d, scale, causal, stream);
}

fa_status fa_bwd_mod(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                     const float* LSE, void* dQ, void* dK, void* dV, const float* slopes,
                     const int* prefix, const int* doc_start, const int* doc_end, int B, int H,
                     int Hkv, int Nq, int Nk, int d, float scale, int causal, float softcap,
                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const ModParams m{Hkv, softcap, slopes, prefix, doc_start, doc_end};
  return bwd_mod_impl(Q, K, V, O, dO, LSE, dQ, dK, dV, m, B, H, Nq, Nk, d, scale, causal,
                      workspace, workspace_bytes, stream);
}

fa_status fa_check_device_error(cudaStream_t stream) {
  g_last_error[0] = '\0';
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  DeviceInfo dev;
  FA_TRY(device_info(&dev));
  unsigned int word = 0;
  e = cudaMemcpy(&word, dev.err, sizeof(word), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
  if (word != 0) {
    const unsigned int zero = 0;
    e = cudaMemcpy(dev.err, &zero, sizeof(zero), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the device error word");
    if (word & 4u)
      return fail(FA_ERR_INVALID_ARG,
                  "a per-sequence length was negative, above the padded length, or (causal) "
                  "had more queries than keys; that sequence was skipped (error word 0x%x)",
                  word);
    if (word & 8u)
      return fail(FA_ERR_INVALID_ARG,
                  "a block table named a page outside the cache; the outputs of its sequence "
                  "are wrong (error word 0x%x)", word);
    if (word & 2u)
      return fail(FA_ERR_CUDA,
                  "a kernel found its dynamic shared memory misaligned and did no work "
                  "(error word 0x%x)", word);
    return fail(FA_ERR_TIMEOUT, "a kernel pipeline wait timed out (error word 0x%x)", word);
  }
  return FA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------------------
// fa_bwd_noalloc: the backward pass for callers that cannot allocate device memory.
//
// Some callers have no way to hand fa_bwd a workspace: a plugin whose host API gives it
// no allocator, code that runs inside a framework step whose memory plan is frozen, or
// a latency-sensitive loop that must not enter cudaMalloc (which can synchronise the
// device).  For them the library keeps its own scratch: the array below, a fixed
// kNoAllocScratchBytes of device memory that every GPU which loads libfa.so holds until
// the process exits.  The caller still provides every input and output.
//
// In host code `g_fa_bwd_scratch` names a host-side stand-in, not device memory, so it
// is never passed to a kernel directly.  The first fa_bwd_noalloc call on a device looks
// up the array's device address with cudaGetSymbolAddress while that device is current
// and caches it; that first call should therefore come before any stream capture.
//
// Every call shares the one array.  fa_bwd fully rewrites the part it uses (D and
// LSE*log2(e) for every padded row) before reading it, so nothing needs clearing between
// calls, but two calls whose kernels overlap on the GPU (different streams, or another
// thread) race on the array and give wrong gradients: serialise them.
// ---------------------------------------------------------------------------------------
namespace {

constexpr size_t kNoAllocScratchBytes = 8u << 20;  // 8 MiB: B*H*ceil(N/128)*128 <= 2^20
static __device__ __align__(256) unsigned char g_fa_bwd_scratch[kNoAllocScratchBytes];

std::mutex g_scratch_mutex;
void* g_scratch_addr[kMaxDevices] = {};

fa_status noalloc_scratch(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(FA_ERR_CUDA, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  if (g_scratch_addr[dev] == nullptr) {
    void* ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_fa_bwd_scratch);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(g_fa_bwd_scratch)");
    g_scratch_addr[dev] = ptr;
  }
  *out = g_scratch_addr[dev];
  return FA_OK;
}

}  // namespace

extern "C" {

size_t fa_bwd_noalloc_max_scratch_bytes(void) { return kNoAllocScratchBytes; }

fa_status fa_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                         const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                         int B, int H, int N, int d, float scale, int causal,
                         cudaStream_t stream) {
  g_last_error[0] = '\0';
  void* scratch = nullptr;
  bool noop = false;
  // sizes first: the scratch arithmetic below assumes validated sizes
  fa_status st = check_common(B, H, N, N, d, scale, causal, &noop);
  if (st != FA_OK || noop) return st;
  const size_t need = fa_bwd_workspace_bytes(B, H, N, d);
  if (need > kNoAllocScratchBytes)
    return fail(FA_ERR_INVALID_ARG,
                "fa_bwd_noalloc: B=%d H=%d N=%d needs %zu bytes of scratch, more than the "
                "library's fixed %zu (B*H*ceil(N/128)*128 must be at most %zu); use fa_bwd "
                "with a workspace",
                B, H, N, need, kNoAllocScratchBytes, kNoAllocScratchBytes / 8);
  st = noalloc_scratch(&scratch);
  if (st != FA_OK) return st;
  return fa_bwd(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, d, scale, causal, scratch,
                kNoAllocScratchBytes, stream);
}

}  // extern "C"
