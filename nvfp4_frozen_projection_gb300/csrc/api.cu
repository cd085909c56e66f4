// C ABI of libpact: argument validation, workspace carving, TMA descriptors and
// kernel launches.  Declarations and the contract of every call are in pact.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/pact.h"
#include "kernels.h"

using namespace pact;

namespace {
std::atomic<uint64_t> g_launches{0};
thread_local cudaEvent_t g_prof_begin = nullptr, g_prof_end = nullptr;
}  // namespace

void pact::note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

namespace {
int fail(int code, const char* fmt, ...);
}

int pact::report_error(int code, const char* msg) { return fail(code, "%s", msg); }

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(PACT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

struct DeviceInfo {
  bool init = false;
  int sms = 0;
  int major = 0, minor = 0;
  unsigned* status = nullptr;
};
DeviceInfo g_dev[64];
std::mutex g_dev_mu;

int device_info(DeviceInfo** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(PACT_ERR_INVALID_ARG, "device index %d", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.init) {
    if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e, "multiprocessor count");
    cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev);
    if ((e = status_word_ptr(&d.status)) != cudaSuccess) return cuda_fail(e, "status word");
    d.init = true;
  }
  if (!(d.major == 10 && d.minor == 3))
    return fail(PACT_ERR_ARCH, "device is sm_%d%d; libpact needs sm_103 (GB300)", d.major,
                d.minor);
  *out = &d;
  return PACT_OK;
}

// ---------------------------------------------------------------- TMA descriptors
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

}  // namespace

// 2-D tiled map over a row-major [rows, inner] matrix of elem-byte elements whose
// rows are ld elements apart (ld = inner when 0).
int pact::make_map(CUtensorMap* m, CUtensorMapDataType dt, int elem_bytes, const void* base,
             uint64_t inner, uint64_t rows, uint32_t box_inner, uint32_t box_rows,
             CUtensorMapSwizzle swz, uint64_t ld) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(PACT_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {(ld ? ld : inner) * (uint64_t)elem_bytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PACT_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return PACT_OK;
}

// 3-D tiled map over BF16 heads [rows, heads, D], value (t, h, d) at t ld + h D + d; boxes of
// 64 columns x box_heads x box_rows, 128-byte swizzle.
static int make_heads_map(CUtensorMap* m, const pact_heads* t, int64_t D, uint32_t box_heads,
                          uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(PACT_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)t->heads, (cuuint64_t)t->rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)t->ld * 2};
  cuuint32_t box[3] = {64, box_heads, box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t->p, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PACT_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return PACT_OK;
}

namespace {

// ---------------------------------------------------------------- validation helpers
int64_t pad_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int check_nvfp4(const pact_nvfp4* t, const char* name, int64_t rows, int64_t cols, uintptr_t al) {
  if (!t) return fail(PACT_ERR_INVALID_ARG, "%s is null", name);
  if (!t->codes || !t->sf || !t->g) return fail(PACT_ERR_INVALID_ARG, "%s has a null field", name);
  if (t->rows != rows || t->cols != cols)
    return fail(PACT_ERR_SHAPE, "%s is [%lld, %lld], expected [%lld, %lld]", name,
                (long long)t->rows, (long long)t->cols, (long long)rows, (long long)cols);
  if (!aligned(t->codes, al) || !aligned(t->sf, al) || !aligned(t->g, 4))
    return fail(PACT_ERR_ALIGN, "%s codes/sf must be %d-byte aligned", name, (int)al);
  return PACT_OK;
}

int check_fp8(const pact_fp8* t, const char* name, int64_t rows, int64_t cols) {
  if (!t) return fail(PACT_ERR_INVALID_ARG, "%s is null", name);
  if (!t->q || !t->s) return fail(PACT_ERR_INVALID_ARG, "%s has a null field", name);
  if (t->rows != rows || t->cols != cols)
    return fail(PACT_ERR_SHAPE, "%s is [%lld, %lld], expected [%lld, %lld]", name,
                (long long)t->rows, (long long)t->cols, (long long)rows, (long long)cols);
  if (!aligned(t->q, 16) || !aligned(t->s, 4))
    return fail(PACT_ERR_ALIGN, "%s q must be 16-byte and s 4-byte aligned", name);
  return PACT_OK;
}

// Row counts up to 2^30 and widths up to 2^24, multiples of 16: row and column indices
// and their sums with a tile's extent fit in 31 bits.
constexpr int64_t kFp8MaxRows = (int64_t)1 << 30, kFp8MaxCols = (int64_t)1 << 24;

int check_fp8_cols(int64_t c, const char* name) {
  if (c < 16 || c % 16 || c > kFp8MaxCols)
    return fail(PACT_ERR_SHAPE, "need %s a multiple of 16, 16 <= %s <= 2^24", name, name);
  return PACT_OK;
}

// Whether two tensors of so many bytes share memory without being the same: an in-place
// call reads each value before its own thread overwrites it, and no other.
bool partly_same(const void* a, const void* b, int64_t bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x != y && (x < y ? y - x : x - y) < (uintptr_t)bytes;
}

int check_heads(const pact_heads* t, const char* name, int64_t rows, int64_t heads, int64_t D) {
  if (!t || !t->p) return fail(PACT_ERR_INVALID_ARG, "%s is required", name);
  if (t->rows < 1 || t->rows > kFp8MaxRows || t->heads < 1 || t->heads > 65536)
    return fail(PACT_ERR_SHAPE, "%s: need 1 <= rows <= 2^30 and 1 <= heads <= 2^16", name);
  if (t->rows != rows || t->heads != heads)
    return fail(PACT_ERR_SHAPE, "%s has %lld rows of %lld heads, expected %lld of %lld", name,
                (long long)t->rows, (long long)t->heads, (long long)rows, (long long)heads);
  if (t->ld % 8 || t->ld < heads * D || t->ld > (int64_t)1 << 30)
    return fail(PACT_ERR_SHAPE, "%s: need ld %% 8 == 0 and heads * D <= ld <= 2^30", name);
  if (!aligned(t->p, 16)) return fail(PACT_ERR_ALIGN, "%s must be 16-byte aligned", name);
  return PACT_OK;
}

// Rows of `width` bytes, `ld` bytes apart.
struct Block {
  uintptr_t at;
  uint64_t rows, width, ld;
};
Block block_of(const pact_heads* t, int64_t D) {
  return Block{(uintptr_t)t->p, (uint64_t)t->rows, 2 * (uint64_t)(t->heads * D), 2 * (uint64_t)t->ld};
}
Block block_of(const float* p, uint64_t values) { return Block{(uintptr_t)p, 1, 4 * values, 4 * values}; }

// Whether two blocks share memory: columns of one matrix that do not meet share none, nor does
// a single row that lies between the rows of the other.  Blocks within each other whose rows
// lie at different distances are taken to meet.
bool share(Block a, Block b) {
  if (a.at > b.at) {
    const Block t = a;
    a = b;
    b = t;
  }
  const uint64_t gap = b.at - a.at;
  if (gap >= (a.rows - 1) * a.ld + a.width) return false;
  if (a.rows == 1 || (b.rows > 1 && a.ld != b.ld)) return true;
  // b begins in a row of a, or behind it, where another one follows
  const uint64_t off = gap % a.ld;
  return off < a.width || off + b.width > a.ld;
}
bool heads_share(const pact_heads* a, const pact_heads* b, int64_t D) {
  return share(block_of(a, D), block_of(b, D));
}

// Whether two tensors of heads of as many rows share memory without being the same one.
bool heads_clash(const pact_heads* a, const pact_heads* b, int64_t D) {
  const bool same = a->p == b->p && a->heads == b->heads && (a->ld == b->ld || a->rows == 1);
  return !same && heads_share(a, b, D);
}

// LoRA rank padded to 16, 32 or 64; the fused GEMM's LoRA operands are twice as
// wide (a hi/lo BF16 pair of the down-projection output).
int rp_for(int r) { return r <= 16 ? 16 : (r <= 32 ? 32 : 64); }

}  // namespace

// ====================================================================== C ABI
extern "C" {

const char* pact_last_error(void) { return g_err; }

#ifdef PACT_DEBUG
const char* pact_version(void) { return "libpact 0.2 (sm_103a, debug: bounds-checked stores, NaN checks)"; }
#else
const char* pact_version(void) { return "libpact 0.2 (sm_103a)"; }
#endif

uint64_t pact_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int pact_profile_next_gemm(void* begin_event, void* end_event) {
  g_prof_begin = (cudaEvent_t)begin_event;
  g_prof_end = (cudaEvent_t)end_event;
  return PACT_OK;
}

int pact_device_supported(void) {
  DeviceInfo* d;
  return device_info(&d);
}

size_t pact_nvfp4_codes_bytes(int64_t rows, int64_t cols) {
  return rows > 0 && cols > 0 ? (size_t)(rows * (cols / 2)) : 0;
}

size_t pact_nvfp4_sf_bytes(int64_t rows, int64_t cols) {
  return rows > 0 && cols > 0 ? (size_t)(pad_to(rows, 128) * pad_to(cols / 16, 4)) : 0;
}

int pact_check_status(pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  unsigned v = 0;
  if ((e = cudaMemcpy(&v, d->status, sizeof(v), cudaMemcpyDeviceToHost)) != cudaSuccess)
    return cuda_fail(e, "read status word");
  if (v) {
    unsigned zero = 0;
    cudaMemcpy(d->status, &zero, sizeof(zero), cudaMemcpyHostToDevice);
    if (v & PACT_DEV_TIMEOUT)
      return fail(PACT_ERR_TIMEOUT, "a kernel wait timed out (status 0x%x)", v);
    if (v & PACT_DEV_BOUNDS)
      return fail(PACT_ERR_DEVICE_STATUS, "a bounds check of the debug build failed (status 0x%x)",
                  v);
    if (v & PACT_DEV_NAN)
      return fail(PACT_ERR_DEVICE_STATUS,
                  "the debug build found a NaN among the input values (status 0x%x)", v);
    return fail(PACT_ERR_DEVICE_STATUS, "device status 0x%x", v);
  }
  return PACT_OK;
}

// ---------------------------------------------------------------- quantisation
size_t pact_quant_nvfp4_workspace_size(int64_t, int64_t) { return 256; }

int pact_quant_nvfp4(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const float* amax_opt,
                     pact_nvfp4* out, void* ws, size_t ws_bytes, pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!x) return fail(PACT_ERR_INVALID_ARG, "x is null");
  if (M < 1 || K < 64 || K % 64) return fail(PACT_ERR_SHAPE, "need M >= 1 and K %% 64 == 0");
  if (pad_to(M, 128) * (K / 16) >= (int64_t)1 << 31)
    return fail(PACT_ERR_SHAPE, "tensor too large: pad128(M) * K / 16 must be < 2^31");
  if (ldx < K || ldx % 8) return fail(PACT_ERR_SHAPE, "need ldx >= K and ldx %% 8 == 0");
  if (!aligned(x, 16)) return fail(PACT_ERR_ALIGN, "x must be 16-byte aligned");
  if ((rc = check_nvfp4(out, "out", M, K, 16))) return rc;
  if (!ws || ws_bytes < pact_quant_nvfp4_workspace_size(M, K) || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  CUtensorMap tmx;
  if ((rc = make_map(&tmx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, K, M, 64, 32,
                     CU_TENSOR_MAP_SWIZZLE_128B, ldx)))
    return rc;
  cudaError_t e = launch_quant_bf16(tmx, x, M, K, ldx, amax_opt, (uint8_t*)out->codes,
                                    (uint8_t*)out->sf, out->g, (unsigned*)ws, d->status, d->sms,
                                    (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "quant launch");
}

// ---------------------------------------------------------------- weight pack
size_t pact_pack_weight_workspace_size(int64_t, int64_t) { return 256; }

static int pack_common(const float* W, int64_t N, int64_t K, pact_nvfp4* out, void* ws,
                       size_t ws_bytes, pact_stream_t stream, int backward, int64_t gu_half) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!W) return fail(PACT_ERR_INVALID_ARG, "W is null");
  if (N < 64 || K < 64 || N % 64 || K % 64)
    return fail(PACT_ERR_SHAPE, "need N %% 64 == 0 and K %% 64 == 0");
  if (!aligned(W, 16)) return fail(PACT_ERR_ALIGN, "W must be 16-byte aligned");
  if ((rc = check_nvfp4(out, backward ? "out_bwd" : "out_fwd", backward ? K : N, backward ? N : K,
                        16)))
    return rc;
  if (!ws || ws_bytes < 256 || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  cudaError_t e = launch_pack_weight(W, N, K, backward, gu_half, (uint8_t*)out->codes,
                                     (uint8_t*)out->sf, out->g, (unsigned*)ws, d->sms,
                                     (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "pack launch");
}

int pact_pack_weight_fwd(const float* W, int64_t N, int64_t K, pact_nvfp4* out_fwd, void* ws,
                         size_t ws_bytes, pact_stream_t stream) {
  return pack_common(W, N, K, out_fwd, ws, ws_bytes, stream, 0, 0);
}

int pact_pack_weight_fwd_gate_up(const float* W, int64_t N, int64_t K, pact_nvfp4* out_fwd,
                                 void* ws, size_t ws_bytes, pact_stream_t stream) {
  if (N % 64) return fail(PACT_ERR_SHAPE, "need N %% 64 == 0 (gate and up each a multiple of 32)");
  return pack_common(W, N, K, out_fwd, ws, ws_bytes, stream, 0, N / 2);
}

int pact_pack_weight_bwd(const float* W, int64_t N, int64_t K, pact_nvfp4* out_bwd, void* ws,
                         size_t ws_bytes, pact_stream_t stream) {
  return pack_common(W, N, K, out_bwd, ws, ws_bytes, stream, 1, 0);
}

// ---------------------------------------------------------------- LoRA linear
// Workspace: the LoRA left operand [M, 2 rp] (hi|lo BF16 pair) and the padded right
// operand [rows, rp], both BF16; the forward also keeps A^T [rp, K] for its
// down-projection.
size_t pact_lora_linear_fwd_workspace_size(int64_t M, int64_t N, int64_t K, int r) {
  if (M < 1 || N < 1 || K < 1 || r < 1 || r > 64) return 0;
  const int rp = rp_for(r);
  return align256((size_t)M * 2 * rp * 2) + align256((size_t)N * rp * 2) +
         align256((size_t)K * rp * 2);
}

size_t pact_lora_linear_dgrad_workspace_size(int64_t M, int64_t, int64_t K, int r) {
  if (M < 1 || K < 1 || r < 1 || r > 64) return 0;
  const int rp = rp_for(r);
  return align256((size_t)M * 2 * rp * 2) + align256((size_t)K * rp * 2);
}

// Shared tail of fwd and dgrad: GEMM OUT[M, Nout] over reduction Kr with the
// NVFP4 operands a [M, Kr], b [Nout, Kr] and the LoRA operands la [M, rpe],
// lb [Nout, rpe] (both BF16, in the workspace).
static int run_gemm(DeviceInfo* d, const pact_nvfp4* a, const pact_nvfp4* b, int64_t M,
                    int64_t Nout, int64_t Kr, const uint16_t* la, const uint16_t* lb, int rpe,
                    const uint16_t* addend, uint16_t* out, float* out_amax, cudaStream_t stream,
                    int64_t gu_half = 0, float* amax3 = nullptr) {
  GemmLaunch L;
  std::memset(&L, 0, sizeof(L));
  const int bn = gemm_block_n(Nout, rpe);
  const int cm = gemm_cluster_m(M, Nout, rpe);  // each CTA of a cluster loads bn / cm rows of B
  int rc;
  const uint32_t rowb = (uint32_t)gemm_stage_row_bytes();
  const CUtensorMapSwizzle absw = rowb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if ((rc = make_map(&L.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a->codes, Kr / 2, M, rowb, 128,
                     absw)))
    return rc;
  if ((rc = make_map(&L.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, b->codes, Kr / 2, Nout, rowb,
                     bn / cm, absw)))
    return rc;
  // LoRA operands: la [M, rpe] (hi|lo pair), lb [Nout, rpe/2]; boxes of at most 64
  // columns (128-byte rows), swizzled by their row width.
  auto lsw = [](uint32_t cols) {
    return cols == 16 ? CU_TENSOR_MAP_SWIZZLE_32B
                      : (cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  };
  const uint32_t rp = (uint32_t)rpe / 2;
  const uint32_t abox = rpe < 64 ? (uint32_t)rpe : 64, bbox = rp < 64 ? rp : 64;
  if ((rc = make_map(&L.tmLA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, la, rpe, M, abox, 128,
                     lsw(abox))))
    return rc;
  const uint32_t lb_rows = gemm_uses_pair(M, Nout, rpe) ? (uint32_t)bn / 2 : (uint32_t)bn;
  if ((rc = make_map(&L.tmLB, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, lb, rp, Nout, bbox, lb_rows,
                     lsw(bbox))))
    return rc;
  // scale factors: each 128-row block is one row of k16p / 4 atoms (512 bytes each),
  // read as 8-byte elements; a stage takes 4 atoms (2 KB) of one A block and of the
  // bn / 128 B blocks of its tile (zero fill past K and past the last block)
  const uint64_t sf_row = (uint64_t)pad_to(Kr / 16, 4) * 16;  // 8-byte elements per block row
  if ((rc = make_map(&L.tmSFA, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8, a->sf, sf_row,
                     (uint64_t)pad_to(M, 128) / 128, 256, 1, CU_TENSOR_MAP_SWIZZLE_NONE)))
    return rc;
  if ((rc = make_map(&L.tmSFB, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8, b->sf, sf_row,
                     (uint64_t)pad_to(Nout, 128) / 128, 256, (uint32_t)bn / 128,
                     CU_TENSOR_MAP_SWIZZLE_NONE)))
    return rc;
  // output: 32 x 32 BF16 blocks written by TMA stores from the epilogue's 64-byte
  // swizzled staging buffers
  if ((rc = make_map(&L.tmOut, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, Nout, M, 32, 32,
                     CU_TENSOR_MAP_SWIZZLE_64B)))
    return rc;
  GemmParams& p = L.p;
  p.sfa = (const uint8_t*)a->sf;
  p.sfb = (const uint8_t*)b->sf;
  p.ga = a->g;
  p.gb = b->g;
  p.addend = addend;
  p.addend32 = addend && aligned(addend, 32);
  p.out = out;
  p.out_amax = (unsigned*)out_amax;
  p.status = d->status;
  p.M = (int)M;
  p.N = (int)Nout;
  p.K = (int)Kr;
  p.k16p = (int)pad_to(Kr / 16, 4);
  p.num_m = (int)((M + 127) / 128);
  p.num_n = (int)((Nout + bn - 1) / bn);
  p.lora_steps = rpe / 16;
  p.gu_half = (int)gu_half;
  p.amax3 = (unsigned*)amax3;
  L.num_sms = d->sms;
  if (out_amax) {
    cudaError_t e = cudaMemsetAsync(out_amax, 0, sizeof(float), stream);
    if (e != cudaSuccess) return cuda_fail(e, "amax reset");
  }
  if (amax3) {
    cudaError_t e = cudaMemsetAsync(amax3, 0, 3 * sizeof(float), stream);
    if (e != cudaSuccess) return cuda_fail(e, "amax reset");
  }
  cudaEvent_t pb = g_prof_begin, pe = g_prof_end;
  g_prof_begin = g_prof_end = nullptr;
  if (pb && cudaEventRecord(pb, stream) != cudaSuccess) return cuda_fail(cudaGetLastError(), "event");
  cudaError_t e = launch_gemm_nvfp4(L, bn, rpe, cm, stream);
  if (e == cudaSuccess && pe && cudaEventRecord(pe, stream) != cudaSuccess)
    return cuda_fail(cudaGetLastError(), "event");
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "gemm launch");
}

static int check_gemm_dims(int64_t M, int64_t N, int64_t K, int r) {
  if (M < 1 || M > (1 << 30)) return fail(PACT_ERR_SHAPE, "need 1 <= M <= 2^30");
  if (N < 64 || N % 64 || K < 64 || K % 64 || N > (1 << 30) || K > (1 << 30))
    return fail(PACT_ERR_SHAPE, "need N %% 64 == 0 and K %% 64 == 0");
  if (r < 1 || r > 64) return fail(PACT_ERR_INVALID_ARG, "need 1 <= r <= 64");
  return PACT_OK;
}

static int lora_fwd_impl(const pact_nvfp4* xq, const pact_nvfp4* w_fwd, const uint16_t* A,
                         const uint16_t* B, int r, float scale, const uint16_t* residual_opt,
                         uint16_t* y, float* out_amax_opt, void* ws, size_t ws_bytes,
                         pact_stream_t stream, int gate_up, float* amax3) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!xq || !w_fwd) return fail(PACT_ERR_INVALID_ARG, "xq and w_fwd are required");
  const int64_t M = xq->rows, K = xq->cols, N = w_fwd->rows;
  if ((rc = check_gemm_dims(M, N, K, r))) return rc;
  if ((rc = check_nvfp4(xq, "xq", M, K, 128)) || (rc = check_nvfp4(w_fwd, "w_fwd", N, K, 128)))
    return rc;
  if (!A || !B || !y) return fail(PACT_ERR_INVALID_ARG, "A, B and y are required");
  if (!aligned(y, 16) || (residual_opt && !aligned(residual_opt, 16)) || !aligned(B, 2) ||
      !aligned(A, 2))
    return fail(PACT_ERR_ALIGN, "y and residual must be 16-byte aligned");
  if (!ws || ws_bytes < pact_lora_linear_fwd_workspace_size(M, N, K, r) || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  const int rp = rp_for(r);
  const int64_t gu_half = gate_up ? N / 2 : 0;
  if (gate_up && (N % 64 || !amax3 || !aligned(amax3, 4)))
    return fail(PACT_ERR_INVALID_ARG, "gate|up forward: need N %% 64 == 0 and a 4-byte aligned amax3");
  uint16_t* t = (uint16_t*)ws;
  uint16_t* bt = (uint16_t*)((char*)ws + align256((size_t)M * 2 * rp * 2));
  uint16_t* at = (uint16_t*)((char*)bt + align256((size_t)N * rp * 2));
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_lora_down_fwd((const uint8_t*)xq->codes, (const uint8_t*)xq->sf, xq->g,
                                       w_fwd->g, M, K, A, B, r, rp, scale, N, gu_half, t, bt, at,
                                       s);
  if (e != cudaSuccess) return cuda_fail(e, "lora down launch");
  return run_gemm(d, xq, w_fwd, M, N, K, t, bt, 2 * rp, residual_opt, y, out_amax_opt, s, gu_half,
                  amax3);
}

int pact_lora_linear_fwd(const pact_nvfp4* xq, const pact_nvfp4* w_fwd, const uint16_t* A,
                         const uint16_t* B, int r, float scale, const uint16_t* residual_opt,
                         uint16_t* y, float* out_amax_opt, void* ws, size_t ws_bytes,
                         pact_stream_t stream) {
  return lora_fwd_impl(xq, w_fwd, A, B, r, scale, residual_opt, y, out_amax_opt, ws, ws_bytes,
                       stream, 0, nullptr);
}

int pact_lora_linear_fwd_gate_up(const pact_nvfp4* xq, const pact_nvfp4* w_fwd_gu,
                                 const uint16_t* A, const uint16_t* B, int r, float scale,
                                 uint16_t* y, float* amax3, void* ws, size_t ws_bytes,
                                 pact_stream_t stream) {
  return lora_fwd_impl(xq, w_fwd_gu, A, B, r, scale, nullptr, y, nullptr, ws, ws_bytes, stream, 1,
                       amax3);
}

int pact_lora_linear_dgrad(const pact_nvfp4* dyq, const uint16_t* dy, const pact_nvfp4* w_bwd,
                           const uint16_t* A, const uint16_t* B, int r, float scale,
                           int accumulate, uint16_t* dx, void* ws, size_t ws_bytes,
                           pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!dyq || !w_bwd) return fail(PACT_ERR_INVALID_ARG, "dyq and w_bwd are required");
  const int64_t M = dyq->rows, N = dyq->cols, K = w_bwd->rows;
  if ((rc = check_gemm_dims(M, N, K, r))) return rc;
  if ((rc = check_nvfp4(dyq, "dyq", M, N, 128)) || (rc = check_nvfp4(w_bwd, "w_bwd", K, N, 128)))
    return rc;
  if (!dy || !A || !B || !dx) return fail(PACT_ERR_INVALID_ARG, "dy, A, B and dx are required");
  if (!aligned(dx, 16) || !aligned(dy, 16) || !aligned(B, 16) || !aligned(A, 2))
    return fail(PACT_ERR_ALIGN, "dx, dy and B must be 16-byte aligned");
  if (!ws || ws_bytes < pact_lora_linear_dgrad_workspace_size(M, N, K, r) || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  const int rp = rp_for(r);
  uint16_t* u = (uint16_t*)ws;
  uint16_t* ap = (uint16_t*)((char*)ws + align256((size_t)M * 2 * rp * 2));
  // A [K, r] with r == rp is already the zero-padded [K, rp] operand the GEMM reads
  const bool a_direct = r == rp && aligned(A, 16);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_lora_down_dgrad(dy, dyq->g, w_bwd->g, M, N, A, B, r, rp, scale, K, u,
                                         a_direct ? nullptr : ap, s);
  if (e != cudaSuccess) return cuda_fail(e, "lora down launch");
  return run_gemm(d, dyq, w_bwd, M, K, N, u, a_direct ? A : ap, 2 * rp, accumulate ? dx : nullptr,
                  dx, nullptr, s);
}

// ---------------------------------------------------------------- dgrad with dY quantisation
size_t pact_lora_linear_dgrad_q_workspace_size(int64_t M, int64_t N, int64_t K, int r) {
  const size_t w = pact_lora_linear_dgrad_workspace_size(M, N, K, r);
  return w ? w + 256 : 0;
}

int pact_lora_linear_dgrad_q(const uint16_t* dy, const float* dy_amax_opt,
                             const pact_nvfp4* w_bwd, const uint16_t* A, const uint16_t* B, int r,
                             float scale, int accumulate, pact_nvfp4* dyq_out, uint16_t* dx,
                             void* ws, size_t ws_bytes, pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!dyq_out || !w_bwd) return fail(PACT_ERR_INVALID_ARG, "dyq_out and w_bwd are required");
  const int64_t M = dyq_out->rows, N = dyq_out->cols, K = w_bwd->rows;
  if ((rc = check_gemm_dims(M, N, K, r))) return rc;
  if (pad_to(M, 128) * (N / 64) >= (int64_t)1 << 31)
    return fail(PACT_ERR_SHAPE, "tensor too large: pad128(M) * N / 64 must be < 2^31");
  if ((rc = check_nvfp4(dyq_out, "dyq_out", M, N, 128)) ||
      (rc = check_nvfp4(w_bwd, "w_bwd", K, N, 128)))
    return rc;
  if (!dy || !A || !B || !dx) return fail(PACT_ERR_INVALID_ARG, "dy, A, B and dx are required");
  if (!aligned(dx, 16) || !aligned(dy, 16) || !aligned(B, 16) || !aligned(A, 2) ||
      (dy_amax_opt && !aligned(dy_amax_opt, 4)))
    return fail(PACT_ERR_ALIGN, "dx, dy and B must be 16-byte aligned");
  if (!ws || ws_bytes < pact_lora_linear_dgrad_q_workspace_size(M, N, K, r) || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  const int rp = rp_for(r);
  uint16_t* u = (uint16_t*)ws;
  uint16_t* ap = (uint16_t*)((char*)ws + align256((size_t)M * 2 * rp * 2));
  unsigned* amax_ws = (unsigned*)((char*)ws + pact_lora_linear_dgrad_workspace_size(M, N, K, r));
  const bool a_direct = r == rp && aligned(A, 16);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_quant_lora_down(dy, M, N, dy_amax_opt, amax_ws, w_bwd->g, A, B, r, rp,
                                         scale, K, (uint8_t*)dyq_out->codes,
                                         (uint8_t*)dyq_out->sf, dyq_out->g, u,
                                         a_direct ? nullptr : ap, d->sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "quant + lora down launch");
  return run_gemm(d, dyq_out, w_bwd, M, K, N, u, a_direct ? A : ap, 2 * rp,
                  accumulate ? dx : nullptr, dx, nullptr, s);
}

// ---------------------------------------------------------------- adapter gradients
size_t pact_lora_adapter_grad_workspace_size(int64_t M, int64_t N, int64_t K, int r) {
  if (M < 1 || N < 1 || K < 1 || r < 1 || r > 64) return 0;
  const int rp = rp_for(r);
  int64_t rps;
  const int64_t part_n = lora_ts_splits(M, N, rp, false, &rps) * N;
  const int64_t part_k = lora_ts_splits(M, K, rp, true, &rps) * K;
  return align256((size_t)rp * K * 2) + align256((size_t)N * rp * 2) +
         2 * align256((size_t)M * 2 * rp * 2) +
         align256((size_t)(part_n > part_k ? part_n : part_k) * rp * 4);
}

int pact_lora_adapter_grad(const pact_nvfp4* xq, const uint16_t* dy, const uint16_t* A,
                           const uint16_t* B, int r, float scale, int64_t N, float* dA, float* dB,
                           void* ws, size_t ws_bytes, pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!xq) return fail(PACT_ERR_INVALID_ARG, "xq is required");
  const int64_t M = xq->rows, K = xq->cols;
  if ((rc = check_gemm_dims(M, N, K, r))) return rc;
  if ((rc = check_nvfp4(xq, "xq", M, K, 16))) return rc;
  if (!dy || !A || !B || !dA || !dB)
    return fail(PACT_ERR_INVALID_ARG, "dy, A, B, dA and dB are required");
  if (!aligned(dy, 16) || !aligned(B, 16) || !aligned(A, 2) || !aligned(dA, 4) || !aligned(dB, 4))
    return fail(PACT_ERR_ALIGN, "dy and B must be 16-byte aligned");
  if (!ws || ws_bytes < pact_lora_adapter_grad_workspace_size(M, N, K, r) || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  const int rp = rp_for(r);
  char* p = (char*)ws;
  uint16_t* at = (uint16_t*)p;
  p += align256((size_t)rp * K * 2);
  uint16_t* bt = (uint16_t*)p;
  p += align256((size_t)N * rp * 2);
  uint16_t* t = (uint16_t*)p;
  p += align256((size_t)M * 2 * rp * 2);
  uint16_t* u = (uint16_t*)p;
  p += align256((size_t)M * 2 * rp * 2);
  float* part = (float*)p;
  cudaError_t e = launch_lora_adapter_grad((const uint8_t*)xq->codes, (const uint8_t*)xq->sf, xq->g,
                                           M, K, dy, N, A, B, r, rp, scale, dA, dB, at, bt, t, u,
                                           part, d->sms, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "adapter gradient launch");
}

// ---------------------------------------------------------------- fused nonlinear ops
size_t pact_rmsnorm_quant_workspace_size(int64_t, int64_t) { return 256; }

int pact_rmsnorm_quant(const uint16_t* x, const uint16_t* gamma, int64_t M, int64_t H, float eps,
                       pact_nvfp4* yq, float* rstd, void* ws, size_t ws_bytes,
                       pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!x || !gamma || !rstd) return fail(PACT_ERR_INVALID_ARG, "x, gamma and rstd are required");
  if (M < 1 || H < 64 || H % 64 || H > 16384)
    return fail(PACT_ERR_SHAPE, "need M >= 1, H %% 64 == 0, H <= 16384");
  if (pad_to(M, 128) * (H / 16) >= (int64_t)1 << 31)
    return fail(PACT_ERR_SHAPE, "tensor too large: pad128(M) * H / 16 must be < 2^31");
  if (!aligned(x, 16) || !aligned(gamma, 16) || !aligned(rstd, 4))
    return fail(PACT_ERR_ALIGN, "x and gamma must be 16-byte aligned");
  if ((rc = check_nvfp4(yq, "yq", M, H, 16))) return rc;
  if (!ws || ws_bytes < 256 || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  CUtensorMap tmx;
  if ((rc = make_map(&tmx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, H, M, 64, 32,
                     CU_TENSOR_MAP_SWIZZLE_128B)))
    return rc;
  cudaError_t e = launch_rmsnorm_quant(tmx, x, gamma, M, H, eps, (uint8_t*)yq->codes, (uint8_t*)yq->sf,
                                       yq->g, rstd, (unsigned*)ws, d->status, d->sms,
                                       (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "rmsnorm launch");
}

size_t pact_silu_mul_quant_workspace_size(int64_t, int64_t) { return 256; }

int pact_silu_mul_quant(const uint16_t* gateup, int64_t M, int64_t I, const float* amax3_opt,
                        pact_nvfp4* hq, pact_nvfp4* gate_q, pact_nvfp4* up_q, void* ws,
                        size_t ws_bytes, pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!gateup) return fail(PACT_ERR_INVALID_ARG, "gateup is null");
  if (M < 1 || I < 64 || I % 64) return fail(PACT_ERR_SHAPE, "need M >= 1 and I %% 64 == 0");
  if (pad_to(M, 128) * (I / 16) >= (int64_t)1 << 31)
    return fail(PACT_ERR_SHAPE, "tensor too large: pad128(M) * I / 16 must be < 2^31");
  if (!aligned(gateup, 16)) return fail(PACT_ERR_ALIGN, "gateup must be 16-byte aligned");
  if ((rc = check_nvfp4(hq, "hq", M, I, 16)) || (rc = check_nvfp4(gate_q, "gate_q", M, I, 16)) ||
      (rc = check_nvfp4(up_q, "up_q", M, I, 16)))
    return rc;
  if (!ws || ws_bytes < 256 || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  uint8_t* codes[3] = {(uint8_t*)hq->codes, (uint8_t*)gate_q->codes, (uint8_t*)up_q->codes};
  uint8_t* sf[3] = {(uint8_t*)hq->sf, (uint8_t*)gate_q->sf, (uint8_t*)up_q->sf};
  float* g[3] = {hq->g, gate_q->g, up_q->g};
  cudaError_t e = launch_silu_mul_quant(gateup, M, I, amax3_opt, codes, sf, g, (unsigned*)ws,
                                        d->sms, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "silu launch");
}

int pact_silu_mul_bwd(const pact_nvfp4* gate_q, const pact_nvfp4* up_q, const uint16_t* dh,
                      uint16_t* dgateup, float* out_amax_opt, pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!gate_q || !up_q || !dh || !dgateup)
    return fail(PACT_ERR_INVALID_ARG, "gate_q, up_q, dh and dgateup are required");
  const int64_t M = gate_q->rows, I = gate_q->cols;
  if (M < 1 || I < 64 || I % 64) return fail(PACT_ERR_SHAPE, "need M >= 1 and I %% 64 == 0");
  if (pad_to(M, 128) * (I / 16) >= (int64_t)1 << 31)
    return fail(PACT_ERR_SHAPE, "tensor too large: pad128(M) * I / 16 must be < 2^31");
  if ((rc = check_nvfp4(gate_q, "gate_q", M, I, 16)) || (rc = check_nvfp4(up_q, "up_q", M, I, 16)))
    return rc;
  if (!aligned(dh, 16) || !aligned(dgateup, 16))
    return fail(PACT_ERR_ALIGN, "dh and dgateup must be 16-byte aligned");
  cudaError_t e = launch_silu_mul_bwd(
      (const uint8_t*)gate_q->codes, (const uint8_t*)gate_q->sf, gate_q->g,
      (const uint8_t*)up_q->codes, (const uint8_t*)up_q->sf, up_q->g, dh, M, I, dgateup,
      (unsigned*)out_amax_opt, d->sms, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "silu bwd launch");
}

int pact_rmsnorm_bwd(const pact_nvfp4* yq, const uint16_t* gamma, const float* rstd,
                     const uint16_t* dy, const uint16_t* dres_opt, uint16_t* dx,
                     float* out_amax_opt, pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!yq || !gamma || !rstd || !dy || !dx)
    return fail(PACT_ERR_INVALID_ARG, "yq, gamma, rstd, dy and dx are required");
  const int64_t M = yq->rows, H = yq->cols;
  if (M < 1 || H < 64 || H % 64 || H > 16384)
    return fail(PACT_ERR_SHAPE, "need M >= 1, H %% 64 == 0, H <= 16384");
  if ((rc = check_nvfp4(yq, "yq", M, H, 16))) return rc;
  if (!aligned(gamma, 16) || !aligned(dy, 16) || !aligned(dx, 16) ||
      (dres_opt && !aligned(dres_opt, 16)) || (out_amax_opt && !aligned(out_amax_opt, 4)))
    return fail(PACT_ERR_ALIGN, "gamma, dy, dres and dx must be 16-byte aligned");
  cudaError_t e = launch_rmsnorm_bwd((const uint8_t*)yq->codes, (const uint8_t*)yq->sf, yq->g,
                                     gamma, rstd, dy, dres_opt, M, H, dx,
                                     (unsigned*)out_amax_opt, d->sms, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "rmsnorm bwd launch");
}

// ---------------------------------------------------------------- FP8, blocks of 128
// Arguments are checked before the device is looked at.
size_t pact_fp8_scale_count(int64_t rows, int64_t cols) {
  return rows > 0 && cols > 0 ? (size_t)(rows * ((cols + 127) / 128)) : 0;
}

size_t pact_fp8_weight_scale_count(int64_t rows, int64_t cols) {
  return rows > 0 && cols > 0 ? (size_t)(((rows + 127) / 128) * ((cols + 127) / 128)) : 0;
}

int pact_quant_fp8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, pact_fp8* out,
                   pact_stream_t stream) {
  int rc;
  if (M < 1 || M > kFp8MaxRows) return fail(PACT_ERR_SHAPE, "need 1 <= M <= 2^30");
  if ((rc = check_fp8_cols(K, "K"))) return rc;
  if (((M + 7) / 8) * ((K + 127) / 128) >= (int64_t)1 << 31)
    return fail(PACT_ERR_SHAPE, "tensor too large: ceil(M / 8) * ceil(K / 128) must be < 2^31");
  if (!x) return fail(PACT_ERR_INVALID_ARG, "x is null");
  if (ldx < K || ldx % 8) return fail(PACT_ERR_SHAPE, "need ldx >= K and ldx %% 8 == 0");
  if (!aligned(x, 16)) return fail(PACT_ERR_ALIGN, "x must be 16-byte aligned");
  if ((rc = check_fp8(out, "out", M, K))) return rc;
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  cudaError_t e = launch_quant_fp8(x, M, K, ldx, (uint8_t*)out->q, out->s, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "fp8 quant launch");
}

static int pack_fp8(const float* W, int64_t N, int64_t K, pact_fp8* out, pact_stream_t stream,
                    int backward) {
  int rc;
  if (!W) return fail(PACT_ERR_INVALID_ARG, "W is null");
  if ((rc = check_fp8_cols(N, "N")) || (rc = check_fp8_cols(K, "K"))) return rc;
  if (((N + 127) / 128) * ((K + 127) / 128) >= (int64_t)1 << 31)
    return fail(PACT_ERR_SHAPE, "weight too large: ceil(N / 128) * ceil(K / 128) must be < 2^31");
  if (!aligned(W, 16)) return fail(PACT_ERR_ALIGN, "W must be 16-byte aligned");
  if ((rc = check_fp8(out, backward ? "out_bwd" : "out_fwd", backward ? K : N, backward ? N : K)))
    return rc;
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  cudaError_t e = launch_pack_fp8(W, N, K, backward, (uint8_t*)out->q, out->s,
                                  (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "fp8 pack launch");
}

int pact_pack_weight_fp8_fwd(const float* W, int64_t N, int64_t K, pact_fp8* out_fwd,
                             pact_stream_t stream) {
  return pack_fp8(W, N, K, out_fwd, stream, 0);
}

int pact_pack_weight_fp8_bwd(const float* W, int64_t N, int64_t K, pact_fp8* out_bwd,
                             pact_stream_t stream) {
  return pack_fp8(W, N, K, out_bwd, stream, 1);
}

// The rules on a product's sizes.
static int check_fp8_product(int64_t M, int64_t N, int64_t K) {
  int rc;
  if (M < 1 || M > kFp8MaxRows) return fail(PACT_ERR_SHAPE, "need 1 <= rows <= 2^30");
  if ((rc = check_fp8_cols(K, "the reduction width")) ||
      (rc = check_fp8_cols(N, "the output width")))
    return rc;
  if (((M + 127) / 128) * ((N + 127) / 128) >= (int64_t)1 << 30)
    return fail(PACT_ERR_SHAPE, "output too large: ceil(M / 128) * ceil(N / 128) must be < 2^30");
  return PACT_OK;
}

static int linear_fp8(const pact_fp8* x, const char* xname, const pact_fp8* w, const char* wname,
                      const uint16_t* add, const char* addname, uint16_t* out,
                      const char* outname, pact_stream_t stream) {
  int rc;
  if (!x || !w) return fail(PACT_ERR_INVALID_ARG, "%s and %s are required", xname, wname);
  const int64_t M = x->rows, K = x->cols, N = w->rows;
  if ((rc = check_fp8_product(M, N, K)) || (rc = check_fp8(x, xname, M, K)) ||
      (rc = check_fp8(w, wname, N, K)))
    return rc;
  if (!out) return fail(PACT_ERR_INVALID_ARG, "%s is required", outname);
  if (!aligned(out, 16) || (add && !aligned(add, 16)))
    return fail(PACT_ERR_ALIGN, "%s and %s must be 16-byte aligned", outname, addname);
  if (partly_same(add, out, 2 * M * N))
    return fail(PACT_ERR_INVALID_ARG, "%s overlaps %s in part", addname, outname);
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  cudaError_t e;
  if (fp8_is_few(M, N, K, d->sms)) {
    e = launch_fp8_few((const uint8_t*)x->q, x->s, (const uint8_t*)w->q, w->s, M, N, K, add, out,
                       d->sms, (cudaStream_t)stream);
  } else {
    Fp8GemmLaunch L;
    std::memset(&L, 0, sizeof(L));
    L.p.box_m = M < 128 ? (int)(M + 7) / 8 * 8 : 128;
    if ((rc = make_map(&L.tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x->q, K, M, 128, L.p.box_m,
                       CU_TENSOR_MAP_SWIZZLE_128B)) ||
        (rc = make_map(&L.tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w->q, K, N, 128, 128,
                       CU_TENSOR_MAP_SWIZZLE_128B)) ||
        (rc = make_map(&L.tmOut, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, N, M, 32, 32,
                       CU_TENSOR_MAP_SWIZZLE_64B)))
      return rc;
    L.p.add32 = add && aligned(add, 32);
    L.p.out = out;
    L.p.sx = x->s;
    L.p.sw = w->s;
    L.p.add = add;
    L.p.status = d->status;
    L.p.M = (int)M;
    L.p.N = (int)N;
    L.p.nkb = (int)((K + 127) / 128);
    L.K = K;
    L.num_sms = d->sms;
    e = launch_fp8_gemm(L, (cudaStream_t)stream);
  }
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "fp8 linear launch");
}

int pact_linear_fp8_fwd(const pact_fp8* xq, const pact_fp8* w_fwd, const uint16_t* residual_opt,
                        uint16_t* y, pact_stream_t stream) {
  return linear_fp8(xq, "xq", w_fwd, "w_fwd", residual_opt, "residual", y, "y", stream);
}

int pact_linear_fp8_dgrad(const pact_fp8* dyq, const pact_fp8* w_bwd, const uint16_t* dx_prev_opt,
                          uint16_t* dx, pact_stream_t stream) {
  return linear_fp8(dyq, "dyq", w_bwd, "w_bwd", dx_prev_opt, "dx_prev", dx, "dx", stream);
}

static int check_norm_dims(int64_t M, int64_t H) {
  if (M < 1 || M > kFp8MaxRows || H < 16 || H % 16 || H > 16384)
    return fail(PACT_ERR_SHAPE, "need 1 <= M <= 2^30, H %% 16 == 0, 16 <= H <= 16384");
  return PACT_OK;
}

int pact_add_rmsnorm_quant_fp8(const uint16_t* x, const uint16_t* residual_opt,
                               const uint16_t* gamma, int64_t M, int64_t H, float eps,
                               uint16_t* h_opt, pact_fp8* yq, float* rstd, pact_stream_t stream) {
  int rc;
  if (!residual_opt != !h_opt)
    return fail(PACT_ERR_INVALID_ARG, "residual and h go together: both or neither");
  if ((rc = check_norm_dims(M, H))) return rc;
  if (!x || !gamma || !rstd) return fail(PACT_ERR_INVALID_ARG, "x, gamma and rstd are required");
  if (!(eps >= 0.0f && eps <= 3.4028235e38f))
    return fail(PACT_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!aligned(x, 16) || !aligned(gamma, 16) || !aligned(residual_opt, 16) ||
      !aligned(h_opt, 16) || !aligned(rstd, 4))
    return fail(PACT_ERR_ALIGN, "x, residual, gamma and h must be 16-byte aligned");
  if ((rc = check_fp8(yq, "yq", M, H))) return rc;
  if (partly_same(h_opt, x, 2 * M * H) || partly_same(h_opt, residual_opt, 2 * M * H))
    return fail(PACT_ERR_INVALID_ARG, "h overlaps x or residual in part");
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  cudaError_t e = launch_add_rmsnorm_fp8(x, residual_opt, gamma, M, H, eps, h_opt,
                                         (uint8_t*)yq->q, yq->s, rstd, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "add rmsnorm launch");
}

size_t pact_add_rmsnorm_bwd_workspace_size(int64_t M, int64_t H) {
  if (M < 1 || M > kFp8MaxRows || H < 16 || H % 16 || H > 16384) return 0;
  return align256((size_t)rmsnorm_bwd_partials(M, H) * (size_t)H * 4);
}

int pact_add_rmsnorm_bwd(const uint16_t* h, const uint16_t* gamma, const float* rstd,
                         const uint16_t* dy, const uint16_t* dres_opt, int64_t M, int64_t H,
                         uint16_t* dh, float* dgamma_opt, void* ws, size_t ws_bytes,
                         pact_stream_t stream) {
  int rc;
  if ((rc = check_norm_dims(M, H))) return rc;
  if (!h || !gamma || !rstd || !dy || !dh)
    return fail(PACT_ERR_INVALID_ARG, "h, gamma, rstd, dy and dh are required");
  if (!aligned(h, 16) || !aligned(gamma, 16) || !aligned(dy, 16) || !aligned(dh, 16) ||
      !aligned(dres_opt, 16) || !aligned(rstd, 4) || !aligned(dgamma_opt, 4))
    return fail(PACT_ERR_ALIGN, "h, gamma, dy, dres and dh must be 16-byte aligned");
  const size_t need = dgamma_opt ? pact_add_rmsnorm_bwd_workspace_size(M, H) : 0;
  if (need && (!ws || ws_bytes < need || !aligned(ws, 256)))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  if (partly_same(dh, h, 2 * M * H) || partly_same(dh, dy, 2 * M * H) ||
      partly_same(dh, dres_opt, 2 * M * H))
    return fail(PACT_ERR_INVALID_ARG, "dh overlaps h, dy or dres in part");
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  cudaError_t e = launch_add_rmsnorm_bwd(h, gamma, rstd, dy, dres_opt, M, H, dh, dgamma_opt,
                                         (float*)ws, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "add rmsnorm bwd launch");
}

// ---------------------------------------------------------------- heads and attention
int pact_rope_turns(const double* inv_freq, int64_t n, int64_t* turns, pact_stream_t stream) {
  if (!inv_freq || !turns) return fail(PACT_ERR_INVALID_ARG, "inv_freq and turns are required");
  if (n < 1 || n > 256) return fail(PACT_ERR_SHAPE, "need 1 <= n <= 256 frequencies");
  if (!aligned(inv_freq, 8) || !aligned(turns, 8))
    return fail(PACT_ERR_ALIGN, "inv_freq and turns must be 8-byte aligned");
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  cudaError_t e = launch_rope_turns(inv_freq, (int)n, turns, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "rope turns launch");
}

// The rules that the rotation's two directions share; fills p but for the tensors' pointers.
static int check_rope(const pact_heads* q, const char* qname, const pact_heads* k,
                      const char* kname, int64_t D, int64_t rot, const int32_t* positions,
                      const int64_t* turns, const uint16_t* gq, const uint16_t* gk, float eps,
                      RopeParams* p) {
  int rc;
  if (D < 16 || D > 256 || D % 16)
    return fail(PACT_ERR_SHAPE, "need D %% 16 == 0 and 16 <= D <= 256");
  if (rot < 16 || rot > D || rot % 16)
    return fail(PACT_ERR_SHAPE, "need rot %% 16 == 0 and 16 <= rot <= D");
  if (!q || !k) return fail(PACT_ERR_INVALID_ARG, "%s and %s are required", qname, kname);
  if ((rc = check_heads(q, qname, q->rows, q->heads, D)) ||
      (rc = check_heads(k, kname, q->rows, k->heads, D)))
    return rc;
  if (!positions || !turns) return fail(PACT_ERR_INVALID_ARG, "positions and turns are required");
  if (!gq != !gk)
    return fail(PACT_ERR_INVALID_ARG, "gamma_q and gamma_k go together: both or neither");
  if (!(eps >= 0.0f && eps <= 3.4028235e38f))
    return fail(PACT_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!aligned(positions, 4) || !aligned(turns, 8) || !aligned(gq, 16) || !aligned(gk, 16))
    return fail(PACT_ERR_ALIGN,
                "positions must be 4-byte, turns 8-byte and the gammas 16-byte aligned");
  std::memset(p, 0, sizeof(*p));
  for (int w = 0; w < 2; ++w) {
    p->side[w].x = w ? k->p : q->p;
    p->side[w].ld = w ? k->ld : q->ld;
    p->side[w].heads = (int)(w ? k->heads : q->heads);
    p->side[w].gamma = w ? gk : gq;
  }
  p->positions = positions;
  p->turns = turns;
  p->T = q->rows;
  p->D = (int)D;
  p->rot = (int)rot;
  p->eps = eps;
  return PACT_OK;
}

int pact_qk_norm_rope(const pact_heads* q, const pact_heads* k, int64_t D, int64_t rot,
                      const int32_t* positions, const int64_t* turns, int interleaved,
                      const uint16_t* gamma_q_opt, const uint16_t* gamma_k_opt, float eps,
                      pact_heads* q_out, pact_heads* k_out, pact_stream_t stream) {
  RopeParams p;
  int rc;
  if ((rc = check_rope(q, "q", k, "k", D, rot, positions, turns, gamma_q_opt, gamma_k_opt, eps,
                       &p)) ||
      (rc = check_heads(q_out, "q_out", q->rows, q->heads, D)) ||
      (rc = check_heads(k_out, "k_out", k->rows, k->heads, D)))
    return rc;
  if (heads_clash(q_out, q, D) || heads_clash(k_out, k, D))
    return fail(PACT_ERR_INVALID_ARG, "q_out overlaps q, or k_out k, in part");
  if (heads_share(q_out, k, D) || heads_share(k_out, q, D) || heads_share(q_out, k_out, D))
    return fail(PACT_ERR_INVALID_ARG, "q_out and k_out share memory, or one does with the other's input");
  for (int w = 0; w < 2; ++w) {
    p.side[w].out = w ? k_out->p : q_out->p;
    p.side[w].ldo = w ? k_out->ld : q_out->ld;
  }
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  cudaError_t e = launch_qk_norm_rope(p, interleaved != 0, d->sms, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "qk norm rope launch");
}

size_t pact_qk_norm_rope_bwd_workspace_size(int64_t T, int64_t heads_q, int64_t heads_k,
                                            int64_t D) {
  if (T < 1 || T > kFp8MaxRows || heads_q < 1 || heads_q > 65536 || heads_k < 1 ||
      heads_k > 65536 || D < 16 || D > 256 || D % 16)
    return 0;
  return align256((size_t)rope_bwd_blocks(T, (int)heads_q, (int)heads_k, (int)D, kRopeSms) * 4 *
                  (size_t)D);
}

int pact_qk_norm_rope_bwd(const pact_heads* dyq, const pact_heads* dyk, const pact_heads* q_opt,
                          const pact_heads* k_opt, int64_t D, int64_t rot,
                          const int32_t* positions, const int64_t* turns, int interleaved,
                          const uint16_t* gamma_q_opt, const uint16_t* gamma_k_opt, float eps,
                          pact_heads* dq, pact_heads* dk, float* dgamma_q_opt,
                          float* dgamma_k_opt, void* ws, size_t ws_bytes, pact_stream_t stream) {
  RopeParams p;
  int rc;
  if ((rc = check_rope(dyq, "dyq", dyk, "dyk", D, rot, positions, turns, gamma_q_opt, gamma_k_opt,
                       eps, &p)) ||
      (rc = check_heads(dq, "dq", dyq->rows, dyq->heads, D)) ||
      (rc = check_heads(dk, "dk", dyk->rows, dyk->heads, D)))
    return rc;
  if (heads_clash(dq, dyq, D) || heads_clash(dk, dyk, D))
    return fail(PACT_ERR_INVALID_ARG, "dq overlaps dyq, or dk dyk, in part");
  if (heads_share(dq, dyk, D) || heads_share(dk, dyq, D) || heads_share(dq, dk, D))
    return fail(PACT_ERR_INVALID_ARG, "dq and dk share memory, or one does with the other's dy");
  if (gamma_q_opt) {
    if ((rc = check_heads(q_opt, "q", dyq->rows, dyq->heads, D)) ||
        (rc = check_heads(k_opt, "k", dyk->rows, dyk->heads, D)))
      return rc;
    if (heads_clash(dq, q_opt, D) || heads_clash(dk, k_opt, D))
      return fail(PACT_ERR_INVALID_ARG, "dq overlaps q, or dk k, in part");
    if (heads_share(dq, k_opt, D) || heads_share(dk, q_opt, D))
      return fail(PACT_ERR_INVALID_ARG, "dq shares memory with k, or dk with q");
    for (int w = 0; w < 2; ++w) {
      p.side[w].xf = w ? k_opt->p : q_opt->p;
      p.side[w].ldxf = w ? k_opt->ld : q_opt->ld;
    }
  }
  if (!dgamma_q_opt != !dgamma_k_opt)
    return fail(PACT_ERR_INVALID_ARG, "dgamma_q and dgamma_k go together: both or neither");
  if (dgamma_q_opt && !gamma_q_opt)
    return fail(PACT_ERR_INVALID_ARG, "dgamma needs gamma_q and gamma_k");
  if (!aligned(dgamma_q_opt, 4) || !aligned(dgamma_k_opt, 4))
    return fail(PACT_ERR_ALIGN, "dgamma_q and dgamma_k must be 4-byte aligned");
  if (dgamma_q_opt) {
    const size_t need = pact_qk_norm_rope_bwd_workspace_size(p.T, dyq->heads, dyk->heads, D);
    if (!ws || ws_bytes < need || !aligned(ws, 256))
      return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  }
  for (int w = 0; w < 2; ++w) {
    p.side[w].out = w ? dk->p : dq->p;
    p.side[w].ldo = w ? dk->ld : dq->ld;
  }
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  cudaError_t e = launch_qk_norm_rope_bwd(p, interleaved != 0, dgamma_q_opt, dgamma_k_opt,
                                          (float*)ws, kRopeSms, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "qk norm rope bwd launch");
}

// The rules that attention's two directions share, on q, k, v and the sequences.
static int check_attention(const pact_heads* q, const pact_heads* k, const pact_heads* v,
                           int64_t D, const int32_t* cu_q, const int32_t* cu_k, int64_t nseq,
                           int causal, float scale, AttnParams* p) {
  int rc;
  if (D < 16 || D > 128 || D % 16)
    return fail(PACT_ERR_SHAPE, "need D %% 16 == 0 and 16 <= D <= 128");
  if (!q || !k) return fail(PACT_ERR_INVALID_ARG, "q and k are required");
  if ((rc = check_heads(q, "q", q->rows, q->heads, D)) ||
      (rc = check_heads(k, "k", k->rows, k->heads, D)) ||
      (rc = check_heads(v, "v", k->rows, k->heads, D)))
    return rc;
  if (q->heads % k->heads) return fail(PACT_ERR_SHAPE, "need hq %% hk == 0");
  if (!cu_q || !cu_k) return fail(PACT_ERR_INVALID_ARG, "cu_q and cu_k are required");
  if (nseq < 1 || nseq > (int64_t)1 << 20) return fail(PACT_ERR_SHAPE, "need 1 <= nseq <= 2^20");
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4))
    return fail(PACT_ERR_ALIGN, "cu_q and cu_k must be 4-byte aligned");
  if (!(scale > 0.0f && scale <= 3.4028235e38f))
    return fail(PACT_ERR_INVALID_ARG, "scale must be finite and positive");
  std::memset(p, 0, sizeof(*p));
  p->cu_q = cu_q;
  p->cu_k = cu_k;
  p->nseq = (int)nseq;
  p->tq = (int)q->rows;
  p->tk = (int)k->rows;
  p->hq = (int)q->heads;
  p->hk = (int)k->heads;
  p->group = p->hq / p->hk;
  p->D = (int)D;
  p->gp = attn_tile_heads(p->group);
  p->tpt = 128 / p->gp;
  p->gp_mul = (uint32_t)((65536 + p->gp - 1) / p->gp);
  p->subs = p->group / p->gp;
  p->units_h = p->hk * p->subs;
  p->units_div = FastDiv::make((uint32_t)p->units_h);
  p->hk_div = FastDiv::make((uint32_t)p->hk);
  const int64_t most = ((int64_t)1 << 31) - 1;
  if (attn_units(p->tq, p->tpt, nseq, p->units_h) >= most ||
      attn_units(p->tk, 128, nseq, p->hk) >= most)
    return fail(PACT_ERR_SHAPE, "too many tiles: tokens times heads must stay below 2^31");
  p->scale = scale;
  p->c = scale * 1.4426950408889634f;
  p->causal = causal != 0;
  return PACT_OK;
}

// The parts' lse, and their rows behind it.
static size_t parts_lse_bytes(int parts, int64_t tq, int64_t hq) {
  return align256((size_t)parts * tq * hq * 4);
}

static bool attention_sizes(int64_t Tq, int64_t heads_q, int64_t Tk, int64_t heads_k, int64_t D,
                            int64_t nseq) {
  const auto in = [](int64_t x, int64_t most) { return x >= 1 && x <= most; };
  return in(Tq, kFp8MaxRows) && in(Tk, kFp8MaxRows) && in(heads_k, 65536) && in(heads_q, 65536) &&
         heads_q % heads_k == 0 && in(D, 128) && D % 16 == 0 && in(nseq, (int64_t)1 << 20);
}

size_t pact_attention_fwd_workspace_size(int64_t Tq, int64_t heads_q, int64_t Tk, int64_t heads_k,
                                         int64_t D, int64_t nseq) {
  if (!attention_sizes(Tq, heads_q, Tk, heads_k, D, nseq)) return 0;
  const int parts = attn_fwd_plan(Tq, Tk, nseq, (int)heads_q, (int)heads_k).parts;
  if (parts == 1) return 0;
  return parts_lse_bytes(parts, Tq, heads_q) + (size_t)parts * Tq * heads_q * D * 4;
}

int pact_attention_fwd(const pact_heads* q, const pact_heads* k, const pact_heads* v, int64_t D,
                       const int32_t* cu_q, const int32_t* cu_k, int64_t nseq, int causal,
                       float scale, pact_heads* o, float* lse, void* ws_opt, size_t ws_bytes,
                       pact_stream_t stream) {
  AttnFwdLaunch L;
  int rc;
  if ((rc = check_attention(q, k, v, D, cu_q, cu_k, nseq, causal, scale, &L.p)) ||
      (rc = check_heads(o, "o", q->rows, q->heads, D)))
    return rc;
  if (!lse) return fail(PACT_ERR_INVALID_ARG, "lse is required");
  if (!aligned(lse, 4)) return fail(PACT_ERR_ALIGN, "lse must be 4-byte aligned");
  const AttnFwdPlan plan = attn_fwd_plan(q->rows, k->rows, nseq, L.p.hq, L.p.hk);
  L.p.parts = 1;
  L.p.unit_tiles = plan.unit_tiles;
  const size_t need =
      pact_attention_fwd_workspace_size(q->rows, q->heads, k->rows, k->heads, D, nseq);
  if (ws_opt) {
    if (ws_bytes < need || !aligned(ws_opt, 256))
      return fail(PACT_ERR_INVALID_ARG, "workspace too small or not 256-byte aligned");
    if (need) {
      L.p.parts = plan.parts;
      L.p.part_lse = (float*)ws_opt;
      L.p.part_o = (float*)((char*)ws_opt + parts_lse_bytes(L.p.parts, q->rows, q->heads));
    }
  }
  // o may be q: the unit that writes a row of heads is the one that has read it
  const Block bl = block_of(lse, (uint64_t)(q->rows * q->heads));
  if (heads_clash(o, q, D) || heads_share(o, k, D) || heads_share(o, v, D) || share(bl, block_of(o, D)) ||
      share(bl, block_of(q, D)) || share(bl, block_of(k, D)) || share(bl, block_of(v, D)))
    return fail(PACT_ERR_INVALID_ARG, "o or lse shares memory with another tensor (o may be q itself)");
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  if ((rc = make_heads_map(&L.tmQ, q, D, L.p.gp, L.p.tpt)) ||
      (rc = make_heads_map(&L.tmK, k, D, 1, 128)) || (rc = make_heads_map(&L.tmV, v, D, 1, 128)))
    return rc;
  L.p.o = o->p;
  L.p.ldo = o->ld;
  L.p.lse = lse;
  L.p.status = d->status;
  L.num_sms = d->sms;
  cudaError_t e = launch_attn_fwd(L, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "attention launch");
}

// The backward's workspace: delta, the parts of dq, those of dv and dk.
struct AttnBwdPlan {
  int parts, parts_q;
  size_t part_o, part_kv, bytes;
};
static AttnBwdPlan attention_bwd_plan(int64_t Tq, int64_t heads_q, int64_t Tk, int64_t heads_k,
                                      int64_t D, int64_t nseq) {
  AttnBwdPlan w;
  w.parts = attn_parts_dq(Tq, Tk, nseq, (int)heads_q, (int)heads_k);
  w.parts_q = attn_parts_dkdv(Tq, Tk, nseq, (int)heads_q, (int)heads_k);
  w.part_o = align256((size_t)Tq * heads_q * 4);
  w.part_kv = w.part_o + (w.parts > 1 ? align256((size_t)w.parts * Tq * heads_q * D * 4) : 0);
  w.bytes = w.part_kv + (w.parts_q > 1 ? align256((size_t)2 * w.parts_q * Tk * heads_k * D * 4) : 0);
  return w;
}

size_t pact_attention_bwd_workspace_size(int64_t Tq, int64_t heads_q, int64_t Tk, int64_t heads_k,
                                         int64_t D, int64_t nseq) {
  if (!attention_sizes(Tq, heads_q, Tk, heads_k, D, nseq)) return 0;
  return attention_bwd_plan(Tq, heads_q, Tk, heads_k, D, nseq).bytes;
}

int pact_attention_bwd(const pact_heads* d_o, const pact_heads* q, const pact_heads* k,
                       const pact_heads* v, const pact_heads* o, const float* lse, int64_t D,
                       const int32_t* cu_q, const int32_t* cu_k, int64_t nseq, int causal,
                       float scale, pact_heads* dq, pact_heads* dk, pact_heads* dv, void* ws,
                       size_t ws_bytes, pact_stream_t stream) {
  AttnBwdLaunch L;
  int rc;
  if ((rc = check_attention(q, k, v, D, cu_q, cu_k, nseq, causal, scale, &L.p)) ||
      (rc = check_heads(d_o, "d_o", q->rows, q->heads, D)) ||
      (rc = check_heads(o, "o", q->rows, q->heads, D)) ||
      (rc = check_heads(dq, "dq", q->rows, q->heads, D)) ||
      (rc = check_heads(dk, "dk", k->rows, k->heads, D)) ||
      (rc = check_heads(dv, "dv", k->rows, k->heads, D)))
    return rc;
  if (!lse) return fail(PACT_ERR_INVALID_ARG, "lse is required");
  if (!aligned(lse, 4)) return fail(PACT_ERR_ALIGN, "lse must be 4-byte aligned");
  const AttnBwdPlan plan =
      attention_bwd_plan(q->rows, q->heads, k->rows, k->heads, D, nseq);
  if (!ws || ws_bytes < plan.bytes || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  // dq and dk|dv run side by side: neither may write what the other reads
  const Block bl = block_of(lse, (uint64_t)(q->rows * q->heads));
  const pact_heads* const outs[3] = {dq, dk, dv};
  const pact_heads* const ins[5] = {q, k, v, o, d_o};
  for (int i = 0; i < 3; ++i) {
    bool meets = share(block_of(outs[i], D), bl) || heads_share(outs[i], outs[(i + 1) % 3], D);
    for (const pact_heads* in : ins) meets = meets || heads_share(outs[i], in, D);
    if (meets)
      return fail(PACT_ERR_INVALID_ARG, "dq, dk or dv shares memory with another tensor");
  }
  DeviceInfo* d;
  if ((rc = device_info(&d))) return rc;
  if ((rc = make_heads_map(&L.tmQ, q, D, L.p.gp, L.p.tpt)) ||
      (rc = make_heads_map(&L.tmdO, d_o, D, L.p.gp, L.p.tpt)) ||
      (rc = make_heads_map(&L.tmK, k, D, 1, 128)) || (rc = make_heads_map(&L.tmV, v, D, 1, 128)))
    return rc;
  L.p.lse_in = lse;
  L.p.o_in = o->p;
  L.p.ldoi = o->ld;
  L.p.dout = d_o->p;
  L.p.lddo = d_o->ld;
  L.p.delta = (float*)ws;
  L.p.parts = plan.parts;
  L.p.parts_q = plan.parts_q;
  L.p.part_o = (float*)((char*)ws + plan.part_o);
  L.p.part_kv = (float*)((char*)ws + plan.part_kv);
  L.p.dq = dq->p;
  L.p.dk = dk->p;
  L.p.dv = dv->p;
  L.p.lddq = dq->ld;
  L.p.lddk = dk->ld;
  L.p.lddv = dv->ld;
  L.p.status = d->status;
  L.num_sms = d->sms;
  cudaError_t e = launch_attn_bwd(L, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "attention bwd launch");
}

int64_t pact_grad_chunks(int64_t numel) {
  return numel < 1 ? 0 : (numel + kGradChunk - 1) / kGradChunk;
}

// the blocks' sums: for the SMs of the GPU that the library is for, whatever the device has
constexpr int kGradSms = 152;
size_t pact_grad_norm_workspace_size(void) { return align256(kGradBlocks * kGradSms * sizeof(double)); }

static int grad_norm(const pact_tensor_list* g, float* const* out, bool clip, double max_norm,
                     float* norm, void* ws, size_t ws_bytes, pact_stream_t stream) {
  if (!g || !g->data || !g->numel || !g->first || !norm || (clip && !out))
    return fail(PACT_ERR_INVALID_ARG, "the lists and norm are required");
  if (g->count < 1 || g->count > (int64_t)1 << 20 || g->chunks < 0 ||
      g->chunks > (int64_t)1 << 40)
    return fail(PACT_ERR_SHAPE, "need 1 <= count <= 2^20 and 0 <= chunks <= 2^40");
  if (!aligned(g->data, 8) || !aligned(g->numel, 8) || !aligned(g->first, 8) ||
      !aligned(out, 8) || !aligned(norm, 4))
    return fail(PACT_ERR_ALIGN, "the lists must be 8-byte and norm 4-byte aligned");
  if (!(max_norm >= 0.0)) return fail(PACT_ERR_INVALID_ARG, "max_norm must not be negative or NaN");
  if (!ws || ws_bytes < pact_grad_norm_workspace_size() || !aligned(ws, 256))
    return fail(PACT_ERR_INVALID_ARG, "workspace missing, too small or not 256-byte aligned");
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  GradTable t = {g->data, g->numel, g->first, g->count, g->chunks};
  cudaError_t e = launch_grad_norm(t, clip ? out : nullptr, max_norm, norm, (double*)ws, kGradSms,
                                   (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "grad norm launch");
}

int pact_grad_norm(const pact_tensor_list* grads, float* norm, void* ws, size_t ws_bytes,
                   pact_stream_t stream) {
  return grad_norm(grads, nullptr, false, 0.0, norm, ws, ws_bytes, stream);
}

int pact_clip_grad_norm(const pact_tensor_list* grads, float* const* out, double max_norm,
                        float* norm, void* ws, size_t ws_bytes, pact_stream_t stream) {
  return grad_norm(grads, out, true, max_norm, norm, ws, ws_bytes, stream);
}

int pact_test_fp8_plan(int64_t rows, int64_t N, int64_t K, int sms, int64_t plan[3]) {
  const int rc = check_fp8_product(rows, N, K);
  if (rc) return rc;
  if (sms < 2 || !plan) return fail(PACT_ERR_INVALID_ARG, "need two SMs or more, and plan");
  fp8_plan_of(rows, N, K, sms, plan);
  return PACT_OK;
}

int pact_test_wait_timeout(uint32_t limit_us, pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (limit_us == 0 || limit_us > 2000000)
    return fail(PACT_ERR_INVALID_ARG, "limit_us must be in [1, 2000000]");
  cudaError_t e = launch_wait_timeout((uint64_t)limit_us * 1000ull, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "wait-timeout launch");
}

int pact_test_bounds_check(pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  cudaError_t e = launch_bounds_check((cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "bounds-check launch");
}

int pact_test_pexp(const float* x, float* y, int64_t n, pact_stream_t stream) {
  DeviceInfo* d;
  int rc = device_info(&d);
  if (rc) return rc;
  if (!x || !y || n < 0) return fail(PACT_ERR_INVALID_ARG, "bad pexp arguments");
  if (n == 0) return PACT_OK;
  cudaError_t e = launch_pexp(x, y, n, (cudaStream_t)stream);
  return e == cudaSuccess ? PACT_OK : cuda_fail(e, "pexp launch");
}

}  // extern "C"
