// blocks.cu -- C ABI of the operators around a drafted block: verification from probabilities,
// attention of the drafted nodes, and the commit of the accepted ones. Specified in
// include/psispec.h.
#include <cuda.h>

#include <atomic>
#include <initializer_list>

#include "attend.cuh"
#include "commit.cuh"
#include "host.cuh"
#include "probs.cuh"

namespace psi {
namespace {

constexpr int64_t kMaxV = int64_t(1) << 24;
constexpr int64_t kMaxRows = int64_t(1) << 26;
constexpr int64_t kMaxAttendRows = int64_t(1) << 22;  // (bounds the workspace)

// A kernel's shared-memory attribute, set once per device.
template <typename... A>
bool dynamic_smem(void (*kernel)(A...), int bytes, std::atomic<uint64_t>& ready, int dev) {
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (ready.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  ready.fetch_or(bit, std::memory_order_release);
  return true;
}

template <typename T, int CL>
psispec_status probs_launch(const ProbArgs& a, int dev, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  if (!dynamic_smem(verify_probs_kernel<T, CL>, kProbRing, ready, dev)) return PSISPEC_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * CL);
  cfg.blockDim = dim3(kProbWarps * 32);
  cfg.dynamicSmemBytes = kProbRing;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, verify_probs_kernel<T, CL>, a) == cudaSuccess ? PSISPEC_OK : PSISPEC_ERR_CUDA;
}

// CTAs per request. Three fit on an SM, so 444 run at once; a CTA has a fixed cost of 4 us, and a
// cluster beyond one CTA 0.8 us more. Measured on both sides of each bound (us; fp32 unless said):
// one request of 4096 elements 5.1 (1 CTA) against 5.4 (8), of 16384 7.2 against 5.8; 40 rows of
// 50001 16.8, 12.0, 10.4, 10.3 with 1, 2, 4, 8; 55 rows of 151936 17.0 with 4 against 19.5 with 8;
// 110 rows of 32768 10.1 with 2 against 12.7 with 4, but 100 rows of 151936 29.1 against 25.6;
// 200 rows of 32768 14.2 with 1 against 12.7 with 2, 230 rows 14.2 against 16.6; 512 rows of
// 16384 18.6 with 1 against 32.3 with 4, of 151936 124 against 100 (rows of their own length
// each then even out over four times as many CTAs). Around the bound of 400 KB, for 223, 300, 445 and 512
// rows: of 300 KB (bf16, 151936) 33.6, 40.0, 50.2, 63.5 with 1 against 33.0, 40.0, 55.3, 61.6 with 4; of 400 KB
// (bf16, 204800) 43.4, 47.8, 59.6, 79.2 against 38.2, 45.6, 64.1, 72.6; of 512 KB (fp32, 131072) 42.9, 50.4, 69.7,
// 86.0 against 38.8, 47.6, 65.8, 73.3. (2, which this rule does not take there: 29.0, 38.7, 47.3, 54.1; 36.7,
// 47.3, 58.3, 67.0; 39.8, 50.9, 64.4, 73.3.)
template <typename T>
int prob_cluster(const ProbArgs& a) {
  const bool far = a.V >= (int64_t(400) << 10) / int64_t(sizeof(T));
  if (a.V < 8192) return 1;
  if (a.B <= 40) return 8;
  if (a.B * 4 <= (far ? 444 : 296)) return 4;
  if (a.B * 2 <= 444) return 2;
  return far ? 4 : 1;
}

template <typename T>
psispec_status verify_probs_impl(const ProbArgs& a, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PSISPEC_ERR_CUDA;
  switch (prob_cluster<T>(a)) {
    case 1: return probs_launch<T, 1>(a, dev, st);
    case 2: return probs_launch<T, 2>(a, dev, st);
    case 4: return probs_launch<T, 4>(a, dev, st);
    default: return probs_launch<T, 8>(a, dev, st);
  }
}

// The driver's tensor-map encoder, looked up once.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::atomic<void*> g_encode;

EncodeTiled encoder() {
  void* f = g_encode.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    g_encode.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// Map of a 2-byte tensor with `n` dimensions besides the contiguous one of D elements (innermost
// first in size, stride and box); boxes are 64 columns wide, swizzled by 128 bytes, zeros outside.
// Rows of 64 columns or less are fetched from memory by 128 bytes, not 256: the other 128 belong to
// the next head, which another CTA reads much later (64 requests of 8192 tokens, 8 key heads of 64:
// 190 us by 256 bytes, 168 by 128); of 128 columns the two boxes share the 256.
bool encode(EncodeTiled f, CUtensorMap* map, int dtype, const void* p, int D, int n, const int64_t* size,
            const int64_t* stride, const int* box) {
  cuuint64_t dim[4] = {static_cast<cuuint64_t>(D)}, bytes[3];
  cuuint32_t tile[4] = {64}, step[4] = {1, 1, 1, 1};
  for (int i = 0; i < n; ++i) {
    dim[i + 1] = static_cast<cuuint64_t>(size[i]);
    bytes[i] = static_cast<cuuint64_t>(size[i] > 1 ? stride[i] : D) * 2;
    tile[i + 1] = static_cast<cuuint32_t>(box[i]);
  }
  return f(map, dtype == PSISPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
           static_cast<cuuint32_t>(n + 1), const_cast<void*>(p), dim, bytes, tile, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B,
           D > 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttendWs {
  int4* plan;
  int4* info;
  int2* node_map;
  float2* ml;
  float* part;
  uint4* seen;
};
AttendWs carve_attend(Carver& c, const psispec_attend_tree_args& a) {
  const int64_t rows = max_partial_rows(a.N, a.Hq, a.Hkv, a.prefix_pages > 0);
  AttendWs w;
  w.plan = c.take<int4>(1);
  w.info = c.take<int4>(max_items(a.B, a.N, kTileRows / (a.Hq / a.Hkv), a.Hkv, a.prefix_pages > 0));
  w.node_map = c.take<int2>(a.N);
  w.ml = c.take<float2>(rows);
  w.part = c.take<float>(rows * a.D);
  w.seen = c.take<uint4>(int64_t(kMaxCtas) * 4 * kTileRows);
  return w;
}

template <int DP, bool F16>
psispec_status attend_launch(const AttendParams& p, int dev, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  if (!dynamic_smem(attend_tree_kernel<DP, F16>, attend_smem<DP>(), ready, dev)) return PSISPEC_ERR_CUDA;
  psispec_status s = launch(attend_tree_kernel<DP, F16>, static_cast<unsigned>(p.ctas), kAttendThreads, attend_smem<DP>(),
                            st, p);
  if (s != PSISPEC_OK) return s;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>((int64_t(p.N) * p.Hq + kCombineWarps - 1) / kCombineWarps));
  cfg.blockDim = dim3(kCombineWarps * 32);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* const combine = cfg.gridDim.x <= kMaxCtas       ? attend_combine_kernel<F16, 16, 1>
                        : cfg.gridDim.x <= 4 * kMaxCtas ? attend_combine_kernel<F16, 8, 3>
                                                        : attend_combine_kernel<F16, 4, 5>;
  return cudaLaunchKernelEx(&cfg, combine, p) == cudaSuccess ? PSISPEC_OK : PSISPEC_ERR_CUDA;
}

psispec_status attend_impl(const psispec_attend_tree_args& a, void* ws, cudaStream_t st) {
  EncodeTiled f = encoder();
  if (f == nullptr) return PSISPEC_ERR_CUDA;
  AttendParams p;
  p.shape.G = a.Hq / a.Hkv;
  p.shape.npt = kTileRows / p.shape.G;
  p.shape.Hkv = a.Hkv;
  int box = a.page_size & -a.page_size;  // boxes of a tile start at multiples of their size
  if (box > kTileKeys) box = kTileKeys;
  p.box_log2 = 0;
  while ((1 << p.box_log2) < box) ++p.box_log2;
  p.tile_pages = kTileKeys / a.page_size;
  p.tile_rest = kTileKeys % a.page_size;
  // dimensions innermost first: heads and nodes; tokens of a page, heads and pages
  const int64_t qn[2] = {a.Hq, a.N}, qs[2] = {a.q_stride[1], a.q_stride[0]};
  const int64_t nn[2] = {a.Hkv, a.N}, ks[2] = {a.kn_stride[1], a.kn_stride[0]}, vs[2] = {a.vn_stride[1], a.vn_stride[0]};
  const int64_t cn[3] = {a.page_size, a.Hkv, a.pages};
  const int64_t kcs[3] = {a.kc_stride[1], a.kc_stride[2], a.kc_stride[0]};
  const int64_t vcs[3] = {a.vc_stride[1], a.vc_stride[2], a.vc_stride[0]};
  const int qb[2] = {p.shape.G, p.shape.npt}, nb[2] = {1, kTileKeys}, cb[3] = {box, 1, 1};
  if (!encode(f, &p.q, a.dtype, a.q, a.D, 2, qn, qs, qb) || !encode(f, &p.kn, a.dtype, a.k_nodes, a.D, 2, nn, ks, nb) ||
      !encode(f, &p.vn, a.dtype, a.v_nodes, a.D, 2, nn, vs, nb) ||
      !encode(f, &p.kc, a.dtype, a.k_cache, a.D, 3, cn, kcs, cb) ||
      !encode(f, &p.vc, a.dtype, a.v_cache, a.D, 3, cn, vcs, cb))
    return PSISPEC_ERR_INVALID_ARG;
  int dev = 0, sms = kMaxCtas;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PSISPEC_ERR_CUDA;
  p.ctas = sms < kMaxCtas ? sms : kMaxCtas;
  p.wait_cycles = PSISPEC_ATTEND_WAIT_CYCLES +
                  kUnitCycles * max_units(a.B, a.N, p.shape.npt, a.Hkv,
                                          (int64_t(a.max_pages) + a.prefix_pages) * a.page_size, p.ctas);
  p.B = a.B;
  p.N = a.N;
  p.Hq = a.Hq;
  p.D = a.D;
  p.pages = a.pages;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.prefix_pages = a.prefix_pages;
  p.scale_log2 = static_cast<float>(a.scale * 1.4426950408889634);
  p.node_offsets = a.node_offsets;
  p.parent = a.parent;
  p.page_table = a.page_table;
  p.context_len = a.context_len;
  p.prefix_table = a.prefix_table;
  p.prefix_len = a.prefix_len;
  Carver c(ws);
  const AttendWs w = carve_attend(c, a);
  p.plan = w.plan;
  p.info = w.info;
  p.node_map = w.node_map;
  p.ml = w.ml;
  p.part = w.part;
  p.seen = w.seen;
  p.out = a.out;
  p.lse = a.out_lse;
  if (a.dtype == PSISPEC_F16) return a.D <= 64 ? attend_launch<64, true>(p, dev, st) : attend_launch<128, true>(p, dev, st);
  return a.D <= 64 ? attend_launch<64, false>(p, dev, st) : attend_launch<128, false>(p, dev, st);
}

// Strides (in elements) of a 2-byte tensor whose last dimension of D elements is contiguous and
// whose vectors of 8 elements are 16-byte aligned; a dimension of size 1 has no stride to check.
bool bad_strides(const void* p, const int64_t* stride, const int64_t* size, int n, int D) {
  if (!aligned_to(p, 16)) return true;
  for (int i = 0; i < n; ++i)
    if (size[i] > 1 && (stride[i] < D || stride[i] % 8 != 0 || stride[i] >= (int64_t(1) << 38))) return true;
  return false;
}

// Whether all arrays of 4-byte values start at a multiple of 4 (null ones do).
bool words_aligned(std::initializer_list<const void*> arrays) {
  for (const void* p : arrays)
    if (!aligned_to(p, 4)) return false;
  return true;
}

}  // namespace
}  // namespace psi

using namespace psi;

extern "C" {

psispec_status psispec_verify_probs(const void* target_probs, int64_t target_stride, const void* draft_probs,
                                    int64_t draft_stride, int dtype, int32_t B, int32_t N, int32_t V,
                                    const int32_t* draft_offsets, const int32_t* draft_tokens, const float* u_accept,
                                    const float* u_resid, int32_t* out_tokens, int32_t* out_accept_len, void* stream) {
  if (!target_probs || !draft_offsets || !u_resid || !out_tokens || !out_accept_len ||
      (dtype != PSISPEC_F32 && dtype != PSISPEC_BF16))
    return PSISPEC_ERR_INVALID_ARG;
  if (B <= 0 || N < 0 || V <= 0 || target_stride < V || (draft_probs && draft_stride < V)) return PSISPEC_ERR_INVALID_ARG;
  if (N > 0 && (!draft_tokens || !u_accept)) return PSISPEC_ERR_INVALID_ARG;
  const size_t es = dtype == PSISPEC_BF16 ? 2 : 4;
  if (!aligned_to(target_probs, es) || !aligned_to(draft_probs, es) ||
      !words_aligned({draft_offsets, draft_tokens, u_accept, u_resid, out_tokens, out_accept_len}))
    return PSISPEC_ERR_INVALID_ARG;
  if (int64_t(B) + N > kMaxRows || V > kMaxV || target_stride > (int64_t(1) << 32) || draft_stride > (int64_t(1) << 32))
    return PSISPEC_ERR_UNSUPPORTED;
  ProbArgs a;
  a.target = target_probs;
  a.draft = draft_probs;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.B = B;
  a.N = N;
  a.V = V;
  a.offsets = draft_offsets;
  a.tokens = draft_tokens;
  a.u_acc = u_accept;
  a.u_res = u_resid;
  a.out_tokens = out_tokens;
  a.out_len = out_accept_len;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == PSISPEC_BF16 ? verify_probs_impl<__nv_bfloat16>(a, st) : verify_probs_impl<float>(a, st);
}

static psispec_status check_attend(const psispec_attend_tree_args* a) {
  if (!a || !a->q || !a->k_nodes || !a->v_nodes || !a->k_cache || !a->v_cache || !a->node_offsets || !a->page_table ||
      !a->context_len || !a->out || (a->dtype != PSISPEC_BF16 && a->dtype != PSISPEC_F16))
    return PSISPEC_ERR_INVALID_ARG;
  if (a->B <= 0 || a->N <= 0 || a->Hq <= 0 || a->Hkv <= 0 || a->D <= 0 || a->Hq % a->Hkv != 0 || a->D % 8 != 0 ||
      a->pages <= 0 || a->page_size <= 0 || a->page_size % 8 != 0 || a->max_pages <= 0 || a->prefix_pages < 0)
    return PSISPEC_ERR_INVALID_ARG;
  if (a->prefix_pages > 0 && (!a->prefix_table || !a->prefix_len)) return PSISPEC_ERR_INVALID_ARG;
  if (!(a->scale > 0.0f) || a->scale > 0x1p127f) return PSISPEC_ERR_INVALID_ARG;  // (scale * log2(e) is finite)
  const int64_t qs[2] = {a->N, a->Hq}, ns[2] = {a->N, a->Hkv}, cs[3] = {a->pages, a->page_size, a->Hkv};
  if (bad_strides(a->q, a->q_stride, qs, 2, a->D) || bad_strides(a->k_nodes, a->kn_stride, ns, 2, a->D) ||
      bad_strides(a->v_nodes, a->vn_stride, ns, 2, a->D) || bad_strides(a->k_cache, a->kc_stride, cs, 3, a->D) ||
      bad_strides(a->v_cache, a->vc_stride, cs, 3, a->D) || !aligned_to(a->out, 16) ||
      !words_aligned({a->out_lse, a->node_offsets, a->parent, a->page_table, a->context_len, a->prefix_table, a->prefix_len}))
    return PSISPEC_ERR_INVALID_ARG;
  if (a->D > 128 || a->Hq / a->Hkv > 128 || a->Hkv > 1024 || int64_t(a->N) * a->Hq > kMaxAttendRows || a->B > (1 << 20) ||
      int64_t(a->max_pages) * a->page_size > (1 << 30) || int64_t(a->prefix_pages) * a->page_size > (1 << 30))
    return PSISPEC_ERR_UNSUPPORTED;
  return PSISPEC_OK;
}

size_t psispec_attend_tree_workspace(const psispec_attend_tree_args* args) {
  if (check_attend(args) != PSISPEC_OK) return 0;
  Carver c(nullptr);
  carve_attend(c, *args);
  return c.used;
}

psispec_status psispec_attend_tree(const psispec_attend_tree_args* args, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  psispec_status s = check_attend(args);
  if (s != PSISPEC_OK) return s;
  s = check_ws(workspace, workspace_bytes, psispec_attend_tree_workspace(args));
  if (s != PSISPEC_OK) return s;
  return attend_impl(*args, workspace, static_cast<cudaStream_t>(stream));
}

psispec_status psispec_commit_tree(const psispec_commit_tree_args* a, void* stream) {
  if (!a || !a->k_nodes || !a->v_nodes || !a->k_cache || !a->v_cache || !a->node_offsets || !a->accept_len ||
      !a->page_table || !a->context_len || !a->out_context_len || a->out_context_len == a->context_len ||
      (a->dtype != PSISPEC_BF16 && a->dtype != PSISPEC_F16))
    return PSISPEC_ERR_INVALID_ARG;
  if (a->L <= 0 || a->B <= 0 || a->N <= 0 || a->Hkv <= 0 || a->D <= 0 || a->D % 8 != 0 || a->pages <= 0 ||
      a->page_size <= 0 || a->max_pages <= 0 || (a->path && a->max_depth <= 0))
    return PSISPEC_ERR_INVALID_ARG;
  const int64_t ns[3] = {a->L, a->N, a->Hkv}, cs[4] = {a->L, a->pages, a->page_size, a->Hkv};
  if (bad_strides(a->k_nodes, a->kn_stride, ns, 3, a->D) || bad_strides(a->v_nodes, a->vn_stride, ns, 3, a->D) ||
      bad_strides(a->k_cache, a->kc_stride, cs, 4, a->D) || bad_strides(a->v_cache, a->vc_stride, cs, 4, a->D) ||
      !words_aligned({a->node_offsets, a->path, a->accept_len, a->page_table, a->context_len, a->out_context_len}))
    return PSISPEC_ERR_INVALID_ARG;
  if (a->D > 1024 || a->Hkv > 1024 || a->L > 1024 || a->B > (1 << 20) || a->N > kMaxRows ||
      int64_t(a->max_pages) * a->page_size > (1 << 30))
    return PSISPEC_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a->B), static_cast<unsigned>(2 * a->L));
  cfg.blockDim = dim3(kCommitThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, commit_tree_kernel, *a) == cudaSuccess ? PSISPEC_OK : PSISPEC_ERR_CUDA;
}

}  // extern "C"
