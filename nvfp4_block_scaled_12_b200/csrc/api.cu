// The library's C ABI (declared in include/nvfp4.h): argument validation,
// device checks, TMA descriptor construction and kernel launch.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <mutex>
#include <string>

#include "internal.h"

namespace nvfp4 {

namespace {

// Fault word: kernels OR a code in here when a barrier wait times out.
__device__ unsigned int g_fault_word;

thread_local std::string t_last_error;

// Grid-wait settings the calling thread's dynamic quantizes launch with
// (changed only by nvfp4_testing_set_grid_wait).
thread_local GridWaitSettings t_grid_wait;

nvfp4_status fail(nvfp4_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
nvfp4_status fail(nvfp4_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return st;
}

nvfp4_status ok() {
  t_last_error.clear();
  return NVFP4_OK;
}

nvfp4_status cuda_fail(cudaError_t e, const char* what) {
  return fail(NVFP4_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

DeviceInfo g_devices[kMaxDevices];
std::mutex g_dev_mutex;

// Properties of the current device (cached); EARCH unless it is cc 10.0.
nvfp4_status current_device(const DeviceInfo** out) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(NVFP4_ECUDA, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  DeviceInfo& d = g_devices[dev];
  if (d.device != dev) {
    cudaDeviceProp prop;
    e = cudaGetDeviceProperties(&prop, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDeviceProperties");
    DeviceInfo n;
    n.device = dev;
    n.num_sms = prop.multiProcessorCount;
    n.cc_major = prop.major;
    n.cc_minor = prop.minor;
    n.max_smem_optin = prop.sharedMemPerBlockOptin;
    if (n.cc_major == 10 && n.cc_minor == 0) {
      void* addr = nullptr;
      e = cudaGetSymbolAddress(&addr, g_fault_word);
      if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(fault word)");
      n.fault = static_cast<unsigned*>(addr);
    }
    d = n;
  }
  if (d.cc_major != 10 || d.cc_minor != 0)
    return fail(NVFP4_EARCH, "device %d has compute capability %d.%d; this library is built for 10.0 (sm_100a)",
                dev, d.cc_major, d.cc_minor);
  *out = &d;
  return NVFP4_OK;
}

// ---------------------------------------------------------------------------
// Scratch of the no-allocation dynamic quantize.  Callers that cannot hand
// the library a workspace (a host program or plugin given only its input and
// output buffers, with no device allocator to draw one from) get the grid
// state from this fixed array in the library's own device memory instead.
// One array per device: calls that overlap in time on a device race on it.
// ---------------------------------------------------------------------------
constexpr size_t kNoAllocScratchBytes = 256;  // the most scratch one call may use
static __device__ __align__(256) uint32_t g_noalloc_scratch[kNoAllocScratchBytes / sizeof(uint32_t)];
uint32_t* g_noalloc_ptr[kMaxDevices];  // device address of g_noalloc_scratch, looked up once per device
std::mutex g_noalloc_mutex;

// Address of the scratch on device `dev`, which must be current.  The first
// call per device looks it up (this may load the module on the device, so it
// belongs outside any stream capture).
nvfp4_status noalloc_scratch(int dev, uint32_t** out) {
  std::lock_guard<std::mutex> lock(g_noalloc_mutex);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* addr = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&addr, g_noalloc_scratch);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(no-allocation scratch)");
    g_noalloc_ptr[dev] = static_cast<uint32_t*>(addr);
  }
  *out = g_noalloc_ptr[dev];
  return NVFP4_OK;
}

// ---------------------------------------------------------------- TMA maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Row-major tensor of `rank` dims (innermost first) with byte strides of
// dims 1.. in `strides`.
nvfp4_status make_tmap_nd(CUtensorMap* m, CUtensorMapDataType dt, const void* base, int rank, const uint64_t* dims,
                          const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle sw, const char* what) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return fail(NVFP4_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t d[4], st[3];
  cuuint32_t bx[4], es[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    bx[i] = box[i];
  }
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  const CUresult r = fn(m, dt, static_cast<cuuint32_t>(rank), const_cast<void*>(base), d, st, bx, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(NVFP4_ECUDA, "cuTensorMapEncodeTiled(%s) failed with %d", what, (int)r);
  return NVFP4_OK;
}

// 2-D row-major tensor [outer, inner] with rows `row_bytes` apart.
nvfp4_status make_tmap(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                       uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw,
                       const char* what) {
  const uint64_t dims[2] = {inner, outer};
  const uint64_t strides[1] = {row_bytes};
  const uint32_t box[2] = {box_inner, box_outer};
  return make_tmap_nd(m, dt, base, 2, dims, strides, box, sw, what);
}

// Swizzled scale buffer of a [rows, k] tensor seen as [row blocks][atoms]
// [128 x u32]; one box = box_atoms atoms (4 = one 256-wide NVFP4 k-tile) of
// box_blocks row blocks.  Out-of-range atoms and blocks read as zero.
nvfp4_status make_sf_tmap(CUtensorMap* m, const void* sf, int64_t rows, int64_t atoms, uint32_t box_atoms,
                          uint32_t box_blocks, const char* what) {
  const uint64_t dims[3] = {128, static_cast<uint64_t>(atoms), static_cast<uint64_t>((rows + 127) / 128)};
  const uint64_t strides[2] = {512, static_cast<uint64_t>(atoms) * 512};
  const uint32_t box[3] = {128, box_atoms, box_blocks};
  return make_tmap_nd(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, sf, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                      what);
}

bool finite_f(float v) { return isfinite(v) != 0; }

// Largest row count and K of any entry point: keeps every row index and TMA
// tile coordinate inside int32.
constexpr int64_t kMaxDim = INT32_MAX / 2;

// 1 <= rows <= kMaxDim; 64 <= K <= kMaxDim with K % 64 == 0.
nvfp4_status check_rows_k(const char* rname, int64_t rows, const char* kname, int64_t K) {
  if (rows < 1 || rows > kMaxDim)
    return fail(NVFP4_EINVAL, "%s=%lld must be in [1, %lld]", rname, (long long)rows, (long long)kMaxDim);
  if (K < 64 || K % 64 != 0 || K > kMaxDim)
    return fail(NVFP4_EINVAL, "%s=%lld must be a positive multiple of 64, at most %lld", kname, (long long)K,
                (long long)kMaxDim);
  return NVFP4_OK;
}

// A one-dimensional grid of `threads`-thread blocks over `items` must fit
// gridDim.x.
bool grid_fits(int64_t items, int threads) { return (items + threads - 1) / threads <= INT32_MAX; }

bool scale_ok(float g) { return finite_f(g) && g >= 0x1p-64f && g <= 0x1p64f; }

// Two per-tensor scales whose fp32 product (the epilogue's alpha) is finite.
bool product_ok(float g_a, float g_b) {
  return finite_f(g_a) && finite_f(g_b) && finite_f(static_cast<float>(static_cast<double>(g_a) * g_b));
}

// Checks shared by the two GEMM entry points; fills the operand part of p
// and the operand tensor maps.
// mx4: MXFP4 operands, E2M1 codes as NVFP4's with E8M0 scales per 32.
// mx: 8-bit operands (one E4M3 byte per element), with E8M0 scales per 32
// (MXFP8) or, with row, one fp32 scale per row passed as sfa / sfb.
// split_y (bf16 [M, N]) non-null: the plain NVFP4 or MXFP4 epilogue, which may split K
// across a cluster (gemm_plan) and then writes y directly from the cluster's
// reduction.
nvfp4_status gemm_common(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb, int64_t M,
                         int64_t N, int64_t K, float alpha, const void* bias, GemmParams* p, GemmTensorMaps* maps,
                         GemmConfig* cfg, const DeviceInfo** dev, bool mx = false, bool row = false,
                         bool fused = false, void* split_y = nullptr, bool mx4 = false) {
  if (!a || !sfa || !b || !sfb) return fail(NVFP4_EINVAL, "null operand pointer");
  nvfp4_status st = check_rows_k("M", M, "K", K);
  if (st != NVFP4_OK) return st;
  if (N < 8 || N % 8 != 0 || N > kMaxDim)
    return fail(NVFP4_EINVAL, "N=%lld must be a positive multiple of 8, at most %lld", (long long)N,
                (long long)kMaxDim);
  if (!finite_f(alpha)) return fail(NVFP4_EINVAL, "alpha must be finite");
  if (!aligned16(a) || !aligned16(sfa) || !aligned16(b) || !aligned16(sfb) || !aligned16(bias))
    return fail(NVFP4_EALIGN, "operand pointers must be 16-byte aligned");
  st = current_device(dev);
  if (st != NVFP4_OK) return st;

  // a k-tile is 128 bytes of every operand row: 256 fp4 or 128 fp8 elements
  const int64_t row_bytes = mx ? K : K / 2;
  const int num_kt = static_cast<int>((row_bytes + 127) / 128);
  int k_split = 1;
  if (split_y != nullptr && !mx && !row && !fused) {
    const GemmPlan plan = gemm_plan(M, N, num_kt, (*dev)->num_sms);
    *cfg = plan.c;
    k_split = plan.k_split;
  } else {
    *cfg = gemm_config(M, N, (*dev)->num_sms);
  }
  const int bn = cfg->tile_n;
  const int cg = cfg->cta_group;
  *p = GemmParams{};
  p->k_split = k_split;
  p->y = static_cast<__nv_bfloat16*>(split_y);
  p->ldy = static_cast<int32_t>(N);
  p->M = static_cast<int32_t>(M);
  p->N = static_cast<int32_t>(N);
  p->K = static_cast<int32_t>(K);
  p->tiles_m = static_cast<int32_t>((M + 128 * cg - 1) / (128 * cg));
  p->tiles_n = static_cast<int32_t>((N + bn - 1) / bn);
  const int64_t tiles = static_cast<int64_t>(p->tiles_m) * p->tiles_n;
  if (tiles > INT32_MAX) return fail(NVFP4_EINVAL, "problem too large");
  p->num_tiles = static_cast<int32_t>(tiles);
  p->num_kt = static_cast<int32_t>(num_kt);
  p->kblocks = static_cast<int32_t>(mx ? K / 32 : K / 64);
  p->alpha = alpha;
  p->alpha_mul = 1.0f;
  p->bias = static_cast<const __nv_bfloat16*>(bias);
  p->fault = (*dev)->fault;

  st = make_tmap(&maps->a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, row_bytes, M, row_bytes, 128, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B, "A");
  if (st != NVFP4_OK) return st;
  st = make_tmap(&maps->b, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, row_bytes, N, row_bytes, 128, bn / cg,
                 CU_TENSOR_MAP_SWIZZLE_128B, "B");
  if (st != NVFP4_OK) return st;
  if (row) {  // no block scales: the kernel reads the row scales in its epilogue
    p->row_scale = reinterpret_cast<const float*>(sfa);
    p->col_scale = reinterpret_cast<const float*>(sfb);
    return NVFP4_OK;
  }
  // scale atoms per 128-row block, and atoms per k-tile
  const int64_t atoms = (mx || mx4) ? (K / 32 + 3) / 4 : K / 64;
  const uint32_t box_atoms = mx ? 1u : (mx4 ? 2u : 4u);
  st = make_sf_tmap(&maps->sfa, sfa, M, atoms, box_atoms, 1, "A scales");
  if (st != NVFP4_OK) return st;
  // 128-row scale blocks one B tile can touch: a width that is not a
  // multiple of 128 may start in the middle of a block
  const uint32_t sfb_blocks = static_cast<uint32_t>(bn % 128 == 0 ? bn / 128 : bn / 128 + 1);
  return make_sf_tmap(&maps->sfb, sfb, N, atoms, box_atoms, sfb_blocks, "B scales");
}

// Checks one heads tensor: extents are those of the call, strides those of
// extents above one.  written: two elements may not share an address, that is,
// each stride goes past all that the smaller ones reach.
nvfp4_status check_heads(const char* name, const nvfp4_heads& t, int64_t batch, int64_t tokens, int64_t heads,
                         int64_t head_dim, bool written) {
  if (!t.data) return fail(NVFP4_EINVAL, "%s: null pointer", name);
  if (!aligned16(t.data)) return fail(NVFP4_EALIGN, "%s must be 16-byte aligned", name);
  const int64_t extent[3] = {batch, tokens, heads};
  const int64_t stride[3] = {t.batch_stride, t.token_stride, t.head_stride};
  for (int i = 0; i < 3; ++i) {
    if (extent[i] == 1) continue;
    if (stride[i] < 0 || stride[i] % 8 != 0 || stride[i] > (int64_t(1) << 38))
      return fail(NVFP4_EINVAL, "%s: stride %lld must be a multiple of 8 in [0, 2^38]", name, (long long)stride[i]);
  }
  if (!written) return NVFP4_OK;
  __int128 reach = head_dim;  // elements from the first one to the last of the strides taken so far
  bool taken[3] = {extent[0] == 1, extent[1] == 1, extent[2] == 1};
  for (;;) {
    int least = -1;
    for (int i = 0; i < 3; ++i)
      if (!taken[i] && (least < 0 || stride[i] < stride[least])) least = i;
    if (least < 0) return NVFP4_OK;
    if (stride[least] < reach)
      return fail(NVFP4_EINVAL, "%s: stride %lld lets two heads overlap", name, (long long)stride[least]);
    reach += static_cast<__int128>(extent[least] - 1) * stride[least];
    taken[least] = true;
  }
}

// Tensor map of a heads tensor, [head_dim, heads, tokens, batch] with boxes of
// 64 elements x box_heads x box_tokens.  *bmul: what a batch index counts for
// (0 when the entries share the tensor).
nvfp4_status make_heads_tmap(CUtensorMap* m, const nvfp4_heads& t, int64_t batch, int64_t tokens, int64_t heads,
                             int64_t head_dim, uint32_t box_heads, uint32_t box_tokens, bool fp16, int32_t* bmul,
                             const char* what) {
  *bmul = batch > 1 && t.batch_stride != 0 ? 1 : 0;
  const uint64_t dims[4] = {static_cast<uint64_t>(head_dim), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(tokens), static_cast<uint64_t>(*bmul ? batch : 1)};
  const uint64_t row = static_cast<uint64_t>(head_dim) * 2;  // stands in for a stride that is not used
  const uint64_t strides[3] = {heads > 1 ? static_cast<uint64_t>(t.head_stride) * 2 : row,
                               tokens > 1 ? static_cast<uint64_t>(t.token_stride) * 2 : row,
                               *bmul ? static_cast<uint64_t>(t.batch_stride) * 2 : row};
  const uint32_t box[4] = {64, box_heads, box_tokens, 1};
  return make_tmap_nd(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, t.data, 4, dims,
                      strides, box, CU_TENSOR_MAP_SWIZZLE_128B, what);
}

// nvfp4_gemm_quant with alpha = fl(alpha * alpha_mul) formed on the device.
nvfp4_status gemm_quant_impl(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb,
                             int64_t M, int64_t N, int64_t K, float alpha, float alpha_mul, const void* bias,
                             const nvfp4_colrange* ranges, int32_t n_ranges, void* y_bf16, int64_t ldy,
                             float g_next, uint8_t* codes_next, uint8_t* sf_next, int64_t k_next, void* stream) {
  if (!ranges || n_ranges < 1 || n_ranges > NVFP4_MAX_RANGES)
    return fail(NVFP4_EINVAL, "n_ranges=%d must be in [1, %d]", n_ranges, NVFP4_MAX_RANGES);
  bool any_bf16 = false, any_fp4 = false;
  for (int i = 0; i < n_ranges; ++i) {
    const nvfp4_colrange& r = ranges[i];
    if (r.begin < 0 || r.end <= r.begin || r.end > N || r.begin % 64 || r.end % 64 || r.dst_col < 0 ||
        r.dst_col % 64)
      return fail(NVFP4_EINVAL, "range %d [%lld, %lld) -> %lld: bounds must be multiples of 64 within [0, N]", i,
                  (long long)r.begin, (long long)r.end, (long long)r.dst_col);
    if (r.act != NVFP4_ACT_NONE && r.act != NVFP4_ACT_GELU_TANH)
      return fail(NVFP4_EINVAL, "range %d: unknown activation %d", i, r.act);
    if (r.dst == NVFP4_DST_BF16) {
      any_bf16 = true;
      if (r.dst_col + (r.end - r.begin) > ldy) return fail(NVFP4_EINVAL, "range %d overruns ldy", i);
    } else if (r.dst == NVFP4_DST_NVFP4) {
      any_fp4 = true;
      if (r.dst_col + (r.end - r.begin) > k_next) return fail(NVFP4_EINVAL, "range %d overruns k_next", i);
    } else {
      return fail(NVFP4_EINVAL, "range %d: unknown destination %d", i, r.dst);
    }
    for (int j = 0; j < i; ++j)
      if (ranges[j].begin < r.end && r.begin < ranges[j].end)
        return fail(NVFP4_EINVAL, "ranges %d and %d overlap", j, i);
  }
  if (any_bf16) {
    if (!y_bf16) return fail(NVFP4_EINVAL, "a BF16 range needs y_bf16");
    if (ldy < 8 || ldy % 8 != 0) return fail(NVFP4_EINVAL, "ldy=%lld must be a positive multiple of 8", (long long)ldy);
    if (!aligned16(y_bf16)) return fail(NVFP4_EALIGN, "y_bf16 must be 16-byte aligned");
  }
  if (any_fp4) {
    if (!codes_next || !sf_next) return fail(NVFP4_EINVAL, "an NVFP4 range needs codes_next and sf_next");
    if (k_next < 64 || k_next % 64 != 0 || k_next > INT32_MAX / 2)
      return fail(NVFP4_EINVAL, "k_next=%lld must be a positive multiple of 64", (long long)k_next);
    if (!scale_ok(g_next)) return fail(NVFP4_EINVAL, "g_next must be finite and in [2^-64, 2^64]");
    if (!aligned16(codes_next) || !aligned16(sf_next))
      return fail(NVFP4_EALIGN, "codes_next and sf_next must be 16-byte aligned");
  }
  GemmParams p;
  GemmTensorMaps maps;
  GemmConfig cg;
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = gemm_common(a, sfa, b, sfb, M, N, K, alpha, bias, &p, &maps, &cg, &dev, false, false, true);
  if (st != NVFP4_OK) return st;
  if (any_bf16) {
    st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y_bf16, ldy, M, ldy * 2, 32, 32,
                   CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  } else {
    // never used for a store; a valid descriptor keeps the prefetch harmless
    st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, 16, 1, 16, 16, 1, CU_TENSOR_MAP_SWIZZLE_NONE,
                   "dummy");
  }
  if (st != NVFP4_OK) return st;
  p.n_ranges = n_ranges;
  for (int i = 0; i < n_ranges; ++i) {
    p.ranges[i].begin = static_cast<int32_t>(ranges[i].begin);
    p.ranges[i].end = static_cast<int32_t>(ranges[i].end);
    p.ranges[i].act = ranges[i].act;
    p.ranges[i].dst = ranges[i].dst;
    p.ranges[i].dst_col = static_cast<int32_t>(ranges[i].dst_col);
  }
  p.g_next = g_next;
  p.codes_next = codes_next;
  p.sf_next = sf_next;
  p.k_next = static_cast<int32_t>(k_next);
  p.alpha_mul = alpha_mul;
  cudaError_t e = launch_gemm(maps, p, cg, true, false, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "gemm_quant launch");
  return ok();
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

static_assert(kDynamicScratchBytes == NVFP4_DYNAMIC_WORKSPACE_BYTES, "workspace size in the header");
static_assert(kNoAllocScratchBytes == NVFP4_NOALLOC_SCRATCH_BYTES, "no-allocation scratch size in the header");

extern "C" {

size_t nvfp4_mxfp8_sf_bytes(int64_t rows, int64_t k) {
  if (rows < 1 || k < 32 || k % 32 != 0) return 0;
  const int64_t rp = (rows + 127) / 128 * 128;
  const int64_t cp = (k / 32 + 3) / 4 * 4;
  return static_cast<size_t>(rp) * static_cast<size_t>(cp);
}

nvfp4_status nvfp4_mxfp8_quantize(const void* x, int64_t M, int64_t K, uint8_t* codes, uint8_t* sf, void* stream) {
  if (!x || !codes || !sf) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("M", M, "K", K) != NVFP4_OK) return NVFP4_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf))
    return fail(NVFP4_EALIGN, "pointers must be 16-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  CUtensorMap tx;
  const int tile_rows = quantize_tile_rows(M, K, dev->num_sms);
  st = make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, K, M, K * 2, 64, static_cast<uint32_t>(tile_rows),
                 CU_TENSOR_MAP_SWIZZLE_128B, "x");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_quantize_mxfp8(tx, tile_rows, M, K, codes, sf, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "mxfp8 quantize launch");
  return ok();
}

nvfp4_status nvfp4_mxfp8_gemm(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb, int64_t M,
                              int64_t N, int64_t K, float alpha, const void* bias, void* y, void* stream) {
  if (!y) return fail(NVFP4_EINVAL, "null output pointer");
  if (!aligned16(y)) return fail(NVFP4_EALIGN, "y must be 16-byte aligned");
  GemmParams p;
  GemmTensorMaps maps;
  GemmConfig cg;
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = gemm_common(a, sfa, b, sfb, M, N, K, alpha, bias, &p, &maps, &cg, &dev, true);
  if (st != NVFP4_OK) return st;
  st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_gemm(maps, p, cg, false, true, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "mxfp8 gemm launch");
  return ok();
}

size_t nvfp4_mxfp4_sf_bytes(int64_t rows, int64_t k) { return nvfp4_mxfp8_sf_bytes(rows, k); }

nvfp4_status nvfp4_mxfp4_quantize(const void* x, int64_t M, int64_t K, uint8_t* codes, uint8_t* sf, void* stream) {
  if (!x || !codes || !sf) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("M", M, "K", K) != NVFP4_OK) return NVFP4_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf))
    return fail(NVFP4_EALIGN, "pointers must be 16-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  CUtensorMap tx;
  const int tile_rows = quantize_tile_rows(M, K, dev->num_sms);
  st = make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, K, M, K * 2, 64, static_cast<uint32_t>(tile_rows),
                 CU_TENSOR_MAP_SWIZZLE_128B, "x");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_quantize_mxfp4(tx, tile_rows, M, K, codes, sf, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "mxfp4 quantize launch");
  return ok();
}

nvfp4_status nvfp4_mxfp4_gemm(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb, int64_t M,
                              int64_t N, int64_t K, float alpha, const void* bias, void* y, void* stream) {
  if (!y) return fail(NVFP4_EINVAL, "null output pointer");
  if (!aligned16(y)) return fail(NVFP4_EALIGN, "y must be 16-byte aligned");
  GemmParams p;
  GemmTensorMaps maps;
  GemmConfig cg;
  const DeviceInfo* dev = nullptr;
  nvfp4_status st =
      gemm_common(a, sfa, b, sfb, M, N, K, alpha, bias, &p, &maps, &cg, &dev, false, false, false, y, true);
  if (st != NVFP4_OK) return st;
  st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_gemm_mxfp4(maps, p, cg, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "mxfp4 gemm launch");
  return ok();
}

nvfp4_status nvfp4_rope(const nvfp4_rope_tensor* tensors, int32_t n_tensors, int64_t batch, int64_t tokens,
                        int64_t head_dim, int32_t dtype, const void* positions, int32_t pos_type,
                        int64_t pos_batch_stride, int32_t n_axes, const int32_t* axis_dims, double theta,
                        int32_t flags, float eps, void* stream) {
  if (!tensors || n_tensors < 1 || n_tensors > 2) return fail(NVFP4_EINVAL, "n_tensors=%d must be 1 or 2", n_tensors);
  if (!positions || !axis_dims) return fail(NVFP4_EINVAL, "null pointer");
  if (batch < 1 || tokens < 1 || batch > kMaxDim || tokens > kMaxDim || batch * tokens > kMaxDim)
    return fail(NVFP4_EINVAL, "batch=%lld and tokens=%lld must be positive, their product at most %lld",
                (long long)batch, (long long)tokens, (long long)kMaxDim);
  if (head_dim < 8 || head_dim % 8 != 0 || head_dim > 2 * kRopeMaxPairs)
    return fail(NVFP4_EINVAL, "head_dim=%lld must be a multiple of 8 in [8, %d]", (long long)head_dim,
                2 * kRopeMaxPairs);
  if (dtype != NVFP4_DTYPE_BF16 && dtype != NVFP4_DTYPE_FP16) return fail(NVFP4_EINVAL, "unknown dtype %d", dtype);
  if (pos_type != NVFP4_POS_INT32 && pos_type != NVFP4_POS_FLOAT32)
    return fail(NVFP4_EINVAL, "unknown pos_type %d", pos_type);
  if (reinterpret_cast<uintptr_t>(positions) % 4 != 0) return fail(NVFP4_EALIGN, "positions must be 4-byte aligned");
  if (pos_batch_stride < 0) return fail(NVFP4_EINVAL, "pos_batch_stride must not be negative");
  if (n_axes < 1 || n_axes > kRopeMaxAxes)
    return fail(NVFP4_EINVAL, "n_axes=%d must be in [1, %d]", n_axes, kRopeMaxAxes);
  if (!(theta > 0.0) || !isfinite(theta)) return fail(NVFP4_EINVAL, "theta must be positive and finite");
  if (flags & ~(NVFP4_ROPE_INTERLEAVED | NVFP4_ROPE_SHARED_LADDER)) return fail(NVFP4_EINVAL, "unknown flags");
  if (!(eps >= 0.0f) || !finite_f(eps)) return fail(NVFP4_EINVAL, "eps must be finite and not negative");
  int64_t rotated = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (axis_dims[a] < 2 || axis_dims[a] % 2 != 0 || axis_dims[a] > head_dim)
      return fail(NVFP4_EINVAL, "axis_dims[%d]=%d must be even, in [2, head_dim]", a, axis_dims[a]);
    rotated += axis_dims[a];
  }
  if (rotated > head_dim || rotated % 8 != 0)
    return fail(NVFP4_EINVAL, "axis_dims add up to %lld: a multiple of 8, at most head_dim, needed",
                (long long)rotated);
  RopeParams p = {};
  bool norm = false;
  for (int i = 0; i < n_tensors; ++i) {
    const nvfp4_rope_tensor& t = tensors[i];
    if (t.heads < 1 || t.heads > 65535) return fail(NVFP4_EINVAL, "heads=%lld must be in [1, 65535]", (long long)t.heads);
    nvfp4_status st = check_heads("in", t.in, batch, tokens, t.heads, head_dim, false);
    if (st == NVFP4_OK) st = check_heads("out", t.out, batch, tokens, t.heads, head_dim, true);
    if (st != NVFP4_OK) return st;
    if (!aligned16(t.norm_weight)) return fail(NVFP4_EALIGN, "norm_weight must be 16-byte aligned");
    // (a stride that is not read, of an extent of one, is passed on as 0)
    p.t[i] = RopeTensor{t.in.data,
                        t.out.data,
                        batch > 1 ? t.in.batch_stride : 0,
                        tokens > 1 ? t.in.token_stride : 0,
                        t.heads > 1 ? t.in.head_stride : 0,
                        batch > 1 ? t.out.batch_stride : 0,
                        tokens > 1 ? t.out.token_stride : 0,
                        t.heads > 1 ? t.out.head_stride : 0,
                        t.norm_weight,
                        static_cast<int32_t>(t.heads),
                        0};
    norm |= t.norm_weight != nullptr;
    const RopeTensor& r = p.t[i];
    if (r.in == r.out && (r.in_batch != r.out_batch || r.in_token != r.out_token || r.in_head != r.out_head))
      return fail(NVFP4_EINVAL, "out in place of in needs in's strides");
    if (i == 1 && (r.out == p.t[0].out || r.out == p.t[0].in || r.in == p.t[0].out))
      return fail(NVFP4_EINVAL, "the second tensor shares its data with what the first one writes, or writes the first's");
  }
  p.positions = positions;
  p.pos_batch_stride = pos_batch_stride;
  p.L = static_cast<int32_t>(tokens);
  p.D = static_cast<int32_t>(head_dim);
  p.R = static_cast<int32_t>(rotated);
  p.n_axes = n_axes;
  p.pos_float = pos_type == NVFP4_POS_FLOAT32;
  p.eps = eps;
  // turns per position of every pair, theta^(-2i/d) / 2 pi: a geometric ladder
  // per axis, or one over all pairs (its steps multiplied up in 64 bits)
  const double per_turn = 0.15915494309189533576888;  // 1 / 2 pi
  int pair = 0;
  double f = per_turn;
  for (int a = 0; a < n_axes; ++a) {
    p.first_pair[a] = pair;
    const bool shared = (flags & NVFP4_ROPE_SHARED_LADDER) != 0;
    if (!shared) f = per_turn;
    const double step = pow(theta, -2.0 / static_cast<double>(shared ? rotated : axis_dims[a]));
    for (int i = 0; i < axis_dims[a] / 2; ++i, f *= step) p.turns[pair++] = f;
  }
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  int64_t blocks = 0;
  if (!rope_plan(&p, batch * tokens, dev->num_sms, &blocks)) return fail(NVFP4_EINVAL, "problem too large");
  cudaError_t e = launch_rope(p, blocks, dtype == NVFP4_DTYPE_FP16, (flags & NVFP4_ROPE_INTERLEAVED) != 0, norm,
                              static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope launch");
  return ok();
}

nvfp4_status nvfp4_attention(const nvfp4_heads* q, const nvfp4_heads* k, const nvfp4_heads* v, const nvfp4_heads* out,
                             int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads, int64_t kv_heads,
                             int64_t head_dim, int32_t dtype, const int32_t* kv_lens, float scale, void* stream) {
  if (!q || !k || !v || !out) return fail(NVFP4_EINVAL, "null pointer");
  const struct {
    const char* name;
    int64_t n, most;
  } extents[] = {{"batch", batch, kMaxDim},      {"q_tokens", q_tokens, kMaxDim}, {"kv_tokens", kv_tokens, kMaxDim},
                 {"q_heads", q_heads, 65535},    {"kv_heads", kv_heads, 65535}};
  for (const auto& x : extents)
    if (x.n < 1 || x.n > x.most)
      return fail(NVFP4_EINVAL, "%s=%lld must be in [1, %lld]", x.name, (long long)x.n, (long long)x.most);
  if (head_dim < 8 || head_dim % 8 != 0 || head_dim > 128)
    return fail(NVFP4_EINVAL, "head_dim=%lld must be a multiple of 8 in [8, 128]", (long long)head_dim);
  if (q_heads % kv_heads != 0 || q_heads / kv_heads > 128)
    return fail(NVFP4_EINVAL, "q_heads=%lld must be a multiple of kv_heads=%lld, at most 128 to each",
                (long long)q_heads, (long long)kv_heads);
  if (dtype != NVFP4_DTYPE_BF16 && dtype != NVFP4_DTYPE_FP16) return fail(NVFP4_EINVAL, "unknown dtype %d", dtype);
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // times log2 e
  if (!finite_f(scale_log2) || scale <= 0.0f) return fail(NVFP4_EINVAL, "scale must be positive and finite");
  if (reinterpret_cast<uintptr_t>(kv_lens) % 4 != 0) return fail(NVFP4_EALIGN, "kv_lens must be 4-byte aligned");
  const struct {
    const char* name;
    const nvfp4_heads* t;
    int64_t tokens, heads;
  } tensors[] = {{"q", q, q_tokens, q_heads}, {"k", k, kv_tokens, kv_heads}, {"v", v, kv_tokens, kv_heads}};
  for (const auto& x : tensors) {
    nvfp4_status st = check_heads(x.name, *x.t, batch, x.tokens, x.heads, head_dim, false);
    if (st != NVFP4_OK) return st;
    if ((x.tokens > 1 && x.t->token_stride == 0) || (x.heads > 1 && x.t->head_stride == 0))
      return fail(NVFP4_EINVAL, "%s: only the batch may share one entry (a stride of 0)", x.name);
  }
  nvfp4_status st = check_heads("out", *out, batch, q_tokens, q_heads, head_dim, true);
  if (st != NVFP4_OK) return st;
  if (out->data == q->data || out->data == k->data || out->data == v->data)
    return fail(NVFP4_EINVAL, "out overlaps an input");

  AttentionParams p = {};
  p.out = out->data;
  p.out_batch = batch > 1 ? out->batch_stride : 0;
  p.out_token = q_tokens > 1 ? out->token_stride : 0;
  p.out_head = q_heads > 1 ? out->head_stride : 0;
  p.q = q->data;
  p.q_batch = batch > 1 ? q->batch_stride : 0;
  p.q_token = q_tokens > 1 ? q->token_stride : 0;
  p.q_head = q_heads > 1 ? q->head_stride : 0;
  p.k = k->data;
  p.k_batch = batch > 1 ? k->batch_stride : 0;
  p.k_token = kv_tokens > 1 ? k->token_stride : 0;
  p.k_head = kv_heads > 1 ? k->head_stride : 0;
  p.v = v->data;
  p.v_batch = batch > 1 ? v->batch_stride : 0;
  p.v_token = kv_tokens > 1 ? v->token_stride : 0;
  p.v_head = kv_heads > 1 ? v->head_stride : 0;
  p.kv_lens = kv_lens;
  p.q_tokens = static_cast<int32_t>(q_tokens);
  p.kv_tokens = static_cast<int32_t>(kv_tokens);
  p.kv_heads = static_cast<int32_t>(kv_heads);
  p.D = static_cast<int32_t>(head_dim);
  p.group = static_cast<int32_t>(q_heads / kv_heads);
  // (queries that fit 32 rows of a tile take a tile of that many: the kernel may keep four copies)
  p.tile_tokens = (q_tokens * p.group <= 32 ? 32 : 128) / p.group;
  p.tile_rows = p.tile_tokens * p.group;
  p.q_tiles = (p.q_tokens + p.tile_tokens - 1) / p.tile_tokens;
  p.pairs = (p.q_tiles + 1) / 2;
  // (half of int32: an item's index plus a grid's worth of CTAs stays inside)
  if (batch * kv_heads > INT32_MAX / 2 / p.pairs) return fail(NVFP4_EINVAL, "problem too large");
  p.items = static_cast<int32_t>(batch * kv_heads * p.pairs);
  p.scale_log2 = scale_log2;
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  p.fault = dev->fault;
  AttentionMaps maps;
  const bool fp16 = dtype == NVFP4_DTYPE_FP16;
  st = make_heads_tmap(&maps.q, *q, batch, q_tokens, q_heads, head_dim, static_cast<uint32_t>(p.group),
                       static_cast<uint32_t>(p.tile_tokens), fp16, &p.q_bmul, "Q");
  if (st == NVFP4_OK)
    st = make_heads_tmap(&maps.k, *k, batch, kv_tokens, kv_heads, head_dim, 1, 128, fp16, &p.k_bmul, "K");
  if (st == NVFP4_OK)
    st = make_heads_tmap(&maps.v, *v, batch, kv_tokens, kv_heads, head_dim, 1, 128, fp16, &p.v_bmul, "V");
  int32_t o_bmul = 0;
  if (st == NVFP4_OK)
    st = make_heads_tmap(&maps.o, *out, batch, q_tokens, q_heads, head_dim, static_cast<uint32_t>(p.group),
                         static_cast<uint32_t>(p.tile_tokens), fp16, &o_bmul, "out");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_attention(maps, p, fp16, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return ok();
}

nvfp4_status nvfp4_fp8row_quantize(const void* x, int64_t M, int64_t K, uint8_t* codes, float* scale,
                                   void* stream) {
  if (!x || !codes || !scale) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("M", M, "K", K) != NVFP4_OK) return NVFP4_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scale))
    return fail(NVFP4_EALIGN, "pointers must be 16-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_quantize_rowwise(x, M, K, codes, scale, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "row-wise fp8 quantize launch");
  return ok();
}

nvfp4_status nvfp4_fp8row_gemm(const uint8_t* a, const float* a_scale, const uint8_t* b, const float* b_scale,
                               int64_t M, int64_t N, int64_t K, const void* bias, void* y, void* stream) {
  if (!y) return fail(NVFP4_EINVAL, "null output pointer");
  if (!aligned16(y)) return fail(NVFP4_EALIGN, "y must be 16-byte aligned");
  GemmParams p;
  GemmTensorMaps maps;
  GemmConfig cg;
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = gemm_common(a, reinterpret_cast<const uint8_t*>(a_scale), b,
                                reinterpret_cast<const uint8_t*>(b_scale), M, N, K, 1.0f, bias, &p, &maps, &cg, &dev,
                                true, true);
  if (st != NVFP4_OK) return st;
  st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_gemm(maps, p, cg, false, true, static_cast<cudaStream_t>(stream), *dev, true);
  if (e != cudaSuccess) return cuda_fail(e, "row-wise fp8 gemm launch");
  return ok();
}

nvfp4_status nvfp4_dequantize(const uint8_t* codes, const uint8_t* sf, float g, int64_t rows, int64_t K, void* out,
                              void* stream) {
  if (!codes || !sf || !out) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("rows", rows, "K", K) != NVFP4_OK) return NVFP4_EINVAL;
  if (!grid_fits(rows * (K / 32), 256)) return fail(NVFP4_EINVAL, "rows*K=%lld is too large", (long long)(rows * K));
  if (!finite_f(g)) return fail(NVFP4_EINVAL, "g must be finite");
  if (!aligned16(codes) || !aligned16(sf) || !aligned16(out))
    return fail(NVFP4_EALIGN, "pointers must be 16-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_dequantize(codes, sf, g, rows, K, out, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dequantize launch");
  return ok();
}

size_t nvfp4_sf_bytes(int64_t rows, int64_t k) {
  if (rows < 1 || k < 16 || k % 16 != 0) return 0;
  const int64_t rp = (rows + 127) / 128 * 128;
  const int64_t cp = (k / 16 + 3) / 4 * 4;
  return static_cast<size_t>(rp) * static_cast<size_t>(cp);
}

nvfp4_status nvfp4_calibrate(const void* x, int64_t n, float* out, void* stream) {
  if (!x || !out) return fail(NVFP4_EINVAL, "null pointer");
  if (n < 8 || n % 8 != 0) return fail(NVFP4_EINVAL, "n=%lld must be a positive multiple of 8", (long long)n);
  if (!aligned16(x)) return fail(NVFP4_EALIGN, "x must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(out) & 3u) != 0) return fail(NVFP4_EALIGN, "out must be 4-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_calibrate(x, n, out, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "calibrate launch");
  return ok();
}

nvfp4_status nvfp4_quantize(const void* x, int64_t M, int64_t K, float g, uint8_t* codes, uint8_t* sf,
                            void* stream) {
  if (!x || !codes || !sf) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("M", M, "K", K) != NVFP4_OK) return NVFP4_EINVAL;
  if (!scale_ok(g)) return fail(NVFP4_EINVAL, "g=%g must be finite and in [2^-64, 2^64]", (double)g);
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf))
    return fail(NVFP4_EALIGN, "pointers must be 16-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  CUtensorMap tx;
  const int tile_rows = quantize_tile_rows(M, K, dev->num_sms);
  st = make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, K, M, K * 2, 64, static_cast<uint32_t>(tile_rows),
                 CU_TENSOR_MAP_SWIZZLE_128B, "x");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_quantize(tx, tile_rows, M, K, g, codes, sf, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
  return ok();
}

nvfp4_status nvfp4_quantize_from_amax(const void* x, int64_t M, int64_t K, const float* amax, uint8_t* codes,
                                      uint8_t* sf, float* scale_out, void* stream) {
  if (!x || !amax || !codes || !sf || !scale_out) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("M", M, "K", K) != NVFP4_OK) return NVFP4_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf))
    return fail(NVFP4_EALIGN, "x, codes and sf must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(amax) & 3u) != 0 || (reinterpret_cast<uintptr_t>(scale_out) & 3u) != 0)
    return fail(NVFP4_EALIGN, "amax and scale_out must be 4-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  CUtensorMap tx;
  const int tile_rows = quantize_tile_rows(M, K, dev->num_sms);
  st = make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, K, M, K * 2, 64, static_cast<uint32_t>(tile_rows),
                 CU_TENSOR_MAP_SWIZZLE_128B, "x");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_quantize_from_amax(tx, tile_rows, M, K, amax, codes, sf, scale_out,
                                            static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
  return ok();
}

nvfp4_status nvfp4_quantize_dynamic(const void* x, int64_t M, int64_t K, uint8_t* codes, uint8_t* sf,
                                    float* scale_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !codes || !sf || !scale_out || !workspace) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("M", M, "K", K) != NVFP4_OK) return NVFP4_EINVAL;
  if (workspace_bytes < kDynamicScratchBytes)
    return fail(NVFP4_EINVAL, "workspace_bytes=%zu is below NVFP4_DYNAMIC_WORKSPACE_BYTES=%zu", workspace_bytes,
                kDynamicScratchBytes);
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf))
    return fail(NVFP4_EALIGN, "pointers must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(scale_out) & 3u) != 0 || (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0)
    return fail(NVFP4_EALIGN, "scale_out and workspace must be 4-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  CUtensorMap tx;
  const int tile_rows = quantize_tile_rows(M, K, dev->num_sms);
  st = make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, K, M, K * 2, 64, static_cast<uint32_t>(tile_rows),
                 CU_TENSOR_MAP_SWIZZLE_128B, "x");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_quantize_dynamic(tx, tile_rows, x, M, K, codes, sf, scale_out, static_cast<uint32_t*>(workspace),
                                          t_grid_wait, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "dynamic quantize launch");
  return ok();
}

nvfp4_status nvfp4_quantize_dynamic_noalloc(const void* x, int64_t M, int64_t K, uint8_t* codes, uint8_t* sf,
                                            float* scale_out, void* stream) {
  if (!x || !codes || !sf || !scale_out) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("M", M, "K", K) != NVFP4_OK) return NVFP4_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf))
    return fail(NVFP4_EALIGN, "pointers must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(scale_out) & 3u) != 0) return fail(NVFP4_EALIGN, "scale_out must be 4-byte aligned");
  // scratch this call needs (the grid-wide maximum and the arrival counter)
  const size_t need = kDynamicScratchBytes;
  if (need > kNoAllocScratchBytes)
    return fail(NVFP4_EINVAL, "this call needs %zu bytes of scratch; the no-allocation scratch holds %zu", need,
                kNoAllocScratchBytes);
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  uint32_t* scratch = nullptr;
  st = noalloc_scratch(dev->device, &scratch);
  if (st != NVFP4_OK) return st;
  CUtensorMap tx;
  const int tile_rows = quantize_tile_rows(M, K, dev->num_sms);
  st = make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, K, M, K * 2, 64, static_cast<uint32_t>(tile_rows),
                 CU_TENSOR_MAP_SWIZZLE_128B, "x");
  if (st != NVFP4_OK) return st;
  // the launch zeroes the scratch on the stream before the kernel
  cudaError_t e = launch_quantize_dynamic(tx, tile_rows, x, M, K, codes, sf, scale_out, scratch, t_grid_wait,
                                          static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "dynamic quantize launch");
  return ok();
}

nvfp4_status nvfp4_swizzle_sf(const uint8_t* sf_linear, int64_t rows, int64_t k, uint8_t* sf_swizzled,
                              void* stream) {
  if (!sf_linear || !sf_swizzled) return fail(NVFP4_EINVAL, "null pointer");
  if (check_rows_k("rows", rows, "k", k) != NVFP4_OK) return NVFP4_EINVAL;
  if (!grid_fits((rows + 127) / 128 * (k / 64) * 32, 256))
    return fail(NVFP4_EINVAL, "rows*k=%lld is too large", (long long)(rows * k));
  if (!aligned16(sf_swizzled)) return fail(NVFP4_EALIGN, "sf_swizzled must be 16-byte aligned");
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_swizzle_sf(sf_linear, rows, k, sf_swizzled, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "swizzle launch");
  return ok();
}

nvfp4_status nvfp4_gemm(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb, int64_t M,
                        int64_t N, int64_t K, float alpha, const void* bias, void* y, void* stream) {
  if (!y) return fail(NVFP4_EINVAL, "null output pointer");
  if (!aligned16(y)) return fail(NVFP4_EALIGN, "y must be 16-byte aligned");
  GemmParams p;
  GemmTensorMaps maps;
  GemmConfig cg;
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = gemm_common(a, sfa, b, sfb, M, N, K, alpha, bias, &p, &maps, &cg, &dev, false, false, false, y);
  if (st != NVFP4_OK) return st;
  st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_gemm(maps, p, cg, false, false, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "gemm launch");
  return ok();
}

nvfp4_status nvfp4_gemm_scaled(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb,
                               int64_t M, int64_t N, int64_t K, float g_a, float g_b, const void* bias, void* y,
                               void* stream) {
  if (!y) return fail(NVFP4_EINVAL, "null output pointer");
  if (!aligned16(y)) return fail(NVFP4_EALIGN, "y must be 16-byte aligned");
  if (!product_ok(g_a, g_b)) return fail(NVFP4_EINVAL, "g_a and g_b must be finite with a finite product");
  GemmParams p;
  GemmTensorMaps maps;
  GemmConfig cg;
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = gemm_common(a, sfa, b, sfb, M, N, K, g_b, bias, &p, &maps, &cg, &dev, false, false, false, y);
  if (st != NVFP4_OK) return st;
  p.alpha_mul = g_a;
  st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_gemm(maps, p, cg, false, false, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "gemm launch");
  return ok();
}

nvfp4_status nvfp4_w4a16_gemm(const void* x, const uint8_t* w_codes, const uint8_t* w_sf, int64_t M, int64_t N,
                              int64_t K, float g_w, const void* bias, void* y, void* stream) {
  if (!x || !w_codes || !w_sf || !y) return fail(NVFP4_EINVAL, "null pointer");
  nvfp4_status st = check_rows_k("M", M, "K", K);
  if (st != NVFP4_OK) return st;
  if (N < 8 || N % 8 != 0 || N > kMaxDim)
    return fail(NVFP4_EINVAL, "N=%lld must be a positive multiple of 8, at most %lld", (long long)N,
                (long long)kMaxDim);
  if (!finite_f(g_w)) return fail(NVFP4_EINVAL, "g_w must be finite");
  if (!aligned16(x) || !aligned16(w_codes) || !aligned16(w_sf) || !aligned16(bias) || !aligned16(y))
    return fail(NVFP4_EALIGN, "pointers must be 16-byte aligned");
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  const GemmPlan plan = gemm_plan(M, N, static_cast<int>(K / 64), dev->num_sms);
  const GemmConfig cg = plan.c;
  GemmParams p{};
  p.k_split = plan.k_split;
  p.y = static_cast<__nv_bfloat16*>(y);
  p.ldy = static_cast<int32_t>(N);
  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.tiles_m = static_cast<int32_t>((M + 128 * cg.cta_group - 1) / (128 * cg.cta_group));
  p.tiles_n = static_cast<int32_t>((N + cg.tile_n - 1) / cg.tile_n);
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > INT32_MAX) return fail(NVFP4_EINVAL, "problem too large");
  p.num_tiles = static_cast<int32_t>(tiles);
  p.num_kt = static_cast<int32_t>(K / 64);    // 64 bf16 elements = 128 bytes of every A row
  p.kblocks = static_cast<int32_t>(K / 16);   // K = 16 per MMA
  p.alpha = 1.0f;
  p.alpha_mul = 1.0f;
  p.w_scale = g_w;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.fault = dev->fault;
  GemmTensorMaps maps;
  st = make_tmap(&maps.a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, K, M, K * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B,
                 "x");
  if (st != NVFP4_OK) return st;
  st = make_tmap(&maps.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_codes, K / 2, N, K / 2, 32,
                 static_cast<uint32_t>(cg.tile_n / cg.cta_group), CU_TENSOR_MAP_SWIZZLE_NONE, "weight codes");
  if (st != NVFP4_OK) return st;
  maps.sfa = maps.b;  // unused (the activations carry no block scales); a valid descriptor
  const uint32_t sfb_blocks = static_cast<uint32_t>(cg.tile_n % 128 == 0 ? cg.tile_n / 128 : cg.tile_n / 128 + 1);
  st = make_sf_tmap(&maps.sfb, w_sf, N, K / 64, 1, sfb_blocks, "weight scales");
  if (st != NVFP4_OK) return st;
  st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_gemm_w4a16(maps, p, cg, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "w4a16 gemm launch");
  return ok();
}

nvfp4_status nvfp4_gemm_dynamic(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb,
                                int64_t M, int64_t N, int64_t K, float g_b, const float* g_a, const void* bias,
                                void* y, void* stream) {
  if (!y || !g_a) return fail(NVFP4_EINVAL, "null output or scale pointer");
  if (!aligned16(y)) return fail(NVFP4_EALIGN, "y must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(g_a) & 3u) != 0) return fail(NVFP4_EALIGN, "g_a must be 4-byte aligned");
  GemmParams p;
  GemmTensorMaps maps;
  GemmConfig cg;
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = gemm_common(a, sfa, b, sfb, M, N, K, g_b, bias, &p, &maps, &cg, &dev, false, false, false, y);
  if (st != NVFP4_OK) return st;
  p.alpha_scale = g_a;
  st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_gemm(maps, p, cg, false, false, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "gemm launch");
  return ok();
}


nvfp4_status nvfp4_gemm_amax(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb,
                             int64_t M, int64_t N, int64_t K, float g_a, const float* g_a_device, float g_b,
                             const void* bias, void* y, float* amax_out, void* stream) {
  if (!y || !amax_out) return fail(NVFP4_EINVAL, "null output pointer");
  if (!aligned16(y)) return fail(NVFP4_EALIGN, "y must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(amax_out) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(g_a_device) & 3u) != 0)
    return fail(NVFP4_EALIGN, "amax_out and g_a_device must be 4-byte aligned");
  if (g_a_device == nullptr && !product_ok(g_a, g_b))
    return fail(NVFP4_EINVAL, "g_a and g_b must be finite with a finite product");
  GemmParams p;
  GemmTensorMaps maps;
  GemmConfig cg;
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = gemm_common(a, sfa, b, sfb, M, N, K, g_b, bias, &p, &maps, &cg, &dev, false, false, false, y);
  if (st != NVFP4_OK) return st;
  p.alpha_mul = g_a;
  p.alpha_scale = g_a_device;
  p.amax_out = reinterpret_cast<unsigned*>(amax_out);
  st = make_tmap(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, N * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, "Y");
  if (st != NVFP4_OK) return st;
  cudaError_t e = launch_gemm(maps, p, cg, false, false, static_cast<cudaStream_t>(stream), *dev);
  if (e != cudaSuccess) return cuda_fail(e, "gemm launch");
  return ok();
}

nvfp4_status nvfp4_gemm_quant(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb,
                              int64_t M, int64_t N, int64_t K, float alpha, const void* bias,
                              const nvfp4_colrange* ranges, int32_t n_ranges, void* y_bf16, int64_t ldy,
                              float g_next, uint8_t* codes_next, uint8_t* sf_next, int64_t k_next, void* stream) {
  return gemm_quant_impl(a, sfa, b, sfb, M, N, K, alpha, 1.0f, bias, ranges, n_ranges, y_bf16, ldy, g_next,
                         codes_next, sf_next, k_next, stream);
}

nvfp4_status nvfp4_gemm_quant_scaled(const uint8_t* a, const uint8_t* sfa, const uint8_t* b, const uint8_t* sfb,
                                     int64_t M, int64_t N, int64_t K, float g_a, float g_b, const void* bias,
                                     const nvfp4_colrange* ranges, int32_t n_ranges, void* y_bf16, int64_t ldy,
                                     float g_next, uint8_t* codes_next, uint8_t* sf_next, int64_t k_next,
                                     void* stream) {
  if (!product_ok(g_a, g_b)) return fail(NVFP4_EINVAL, "g_a and g_b must be finite with a finite product");
  return gemm_quant_impl(a, sfa, b, sfb, M, N, K, g_b, g_a, bias, ranges, n_ranges, y_bf16, ldy, g_next,
                         codes_next, sf_next, k_next, stream);
}

nvfp4_status nvfp4_testing_set_grid_wait(uint64_t limit_ns, uint32_t extra_arrivals) {
  if (limit_ns > kWaitLimitNs) return fail(NVFP4_EINVAL, "limit_ns=%llu exceeds the default %llu",
                                          (unsigned long long)limit_ns, (unsigned long long)kWaitLimitNs);
  if (extra_arrivals > 1024u) return fail(NVFP4_EINVAL, "extra_arrivals=%u exceeds 1024", extra_arrivals);
  t_grid_wait.limit_ns = limit_ns == 0 ? kWaitLimitNs : limit_ns;
  t_grid_wait.extra_arrivals = extra_arrivals;
  return ok();
}

nvfp4_status nvfp4_check_fault(void) {
  const DeviceInfo* dev = nullptr;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  unsigned v = 0;
  e = cudaMemcpyFromSymbol(&v, g_fault_word, sizeof(v));
  if (e != cudaSuccess) return cuda_fail(e, "read fault word");
  if (v != 0u) {
    const unsigned zero = 0u;
    e = cudaMemcpyToSymbol(g_fault_word, &zero, sizeof(zero));
    if (e != cudaSuccess) return cuda_fail(e, "clear fault word");
    return fail(NVFP4_ETIMEOUT, "a kernel gave up waiting on a barrier (fault bits 0x%x)", v);
  }
  return ok();
}

nvfp4_status nvfp4_gemm_tile_shape(int64_t M, int64_t N, int32_t num_sms, int32_t* out) {
  if (!out) return fail(NVFP4_EINVAL, "null output pointer");
  if (M < 1 || M > kMaxDim || N < 8 || N > kMaxDim || num_sms < 2)
    return fail(NVFP4_EINVAL, "M=%lld, N=%lld, num_sms=%d out of range", (long long)M, (long long)N, num_sms);
  const GemmConfig c = gemm_config(M, N, num_sms);
  out[0] = c.cta_group;
  out[1] = c.tile_n;
  out[2] = c.acc_bufs;
  return ok();
}

nvfp4_status nvfp4_gemm_plan(int64_t M, int64_t N, int64_t K, int32_t num_sms, int32_t w4a16, int32_t* out) {
  if (!out) return fail(NVFP4_EINVAL, "null output pointer");
  if (M < 1 || M > kMaxDim || N < 8 || N > kMaxDim || K < 64 || K % 64 != 0 || K > kMaxDim || num_sms < 2)
    return fail(NVFP4_EINVAL, "M=%lld, N=%lld, K=%lld, num_sms=%d out of range", (long long)M, (long long)N,
                (long long)K, num_sms);
  const int num_kt = static_cast<int>(w4a16 ? K / 64 : (K / 2 + 127) / 128);
  const GemmPlan plan = gemm_plan(M, N, num_kt, num_sms);
  out[0] = plan.c.cta_group;
  out[1] = plan.c.tile_n;
  out[2] = plan.c.acc_bufs;
  out[3] = plan.k_split;
  return ok();
}

int32_t nvfp4_quantize_tile_rows(int64_t M, int64_t K, int32_t num_sms) {
  if (M < 1 || M > kMaxDim || K < 64 || K % 64 != 0 || K > kMaxDim || num_sms < 1) return 0;
  return quantize_tile_rows(M, K, num_sms);
}

nvfp4_status nvfp4_rope_plan(int64_t heads0, int64_t heads1, int64_t tokens, int64_t head_dim, int32_t num_sms,
                             int32_t* out) {
  if (!out) return fail(NVFP4_EINVAL, "null output pointer");
  if (heads0 < 1 || heads0 > 65535 || heads1 < 0 || heads1 > 65535 || tokens < 1 || tokens > kMaxDim || head_dim < 8 ||
      head_dim % 8 != 0 || head_dim > 2 * kRopeMaxPairs || num_sms < 1)
    return fail(NVFP4_EINVAL, "heads0=%lld, heads1=%lld, tokens=%lld, head_dim=%lld, num_sms=%d out of range",
                (long long)heads0, (long long)heads1, (long long)tokens, (long long)head_dim, num_sms);
  RopeParams p = {};
  p.t[0].heads = static_cast<int32_t>(heads0);
  p.t[1].heads = static_cast<int32_t>(heads1);
  p.D = static_cast<int32_t>(head_dim);
  int64_t blocks = 0;
  if (!rope_plan(&p, tokens, num_sms, &blocks)) return fail(NVFP4_EINVAL, "problem too large");
  out[0] = p.t[0].heads_per_unit;
  out[1] = p.t[1].heads_per_unit;
  out[2] = p.parts0;
  out[3] = p.units_per_token - p.parts0;
  return ok();
}

const char* nvfp4_last_error(void) { return t_last_error.c_str(); }

}  // extern "C"
