// segpaged_decode.cu -- host side of the decode-side calls (see include/segpaged.h): the 8-bit build, the append
// of new rows, the read back, and single-token attention. Argument checks and launches; allocates no device memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/segpaged.h"
#include "decode_sm100.cuh"
#include "host_common.h"
#include "plan.h"
#include "quant_pages.cuh"

using namespace segpaged;
using namespace segpaged::host;

static_assert(kFmtBf16 == SEGPAGED_KV_BF16 && kFmtE4m3 == SEGPAGED_KV_E4M3 && kFmtInt8 == SEGPAGED_KV_INT8, "pool formats");

namespace {

bool is_8bit(int32_t fmt) { return fmt == SEGPAGED_KV_E4M3 || fmt == SEGPAGED_KV_INT8; }

// The checks every call here shares: dims, the pool format, the pools and their exponent bytes.
int check_pools(const segpaged_dims* dims, int32_t fmt, bool allow_bf16, const void* k_pool, const void* v_pool,
                const uint8_t* kv_scale) {
  const int rc = check_dims(dims);
  if (rc) return rc;
  if (!is_8bit(fmt) && !(allow_bf16 && fmt == SEGPAGED_KV_BF16)) return SEGPAGED_ERR_FORMAT;
  // the kernels index query heads, and three class values a KV head, with 32 bits
  if ((int64_t)dims->num_seqs * dims->num_q_heads > INT32_MAX || (int64_t)dims->num_seqs * dims->num_kv_heads > INT32_MAX / 3)
    return SEGPAGED_ERR_DIMS;
  if (dims->num_seqs == 0) return SEGPAGED_OK;
  if (!k_pool || !v_pool || (is_8bit(fmt) && !kv_scale)) return SEGPAGED_ERR_NULL;
  if (!aligned16(k_pool) || !aligned16(v_pool) || (is_8bit(fmt) && !aligned16(kv_scale))) return SEGPAGED_ERR_ALIGN;
  if (dims->num_pages < 1) return SEGPAGED_ERR_DIMS;
  return SEGPAGED_OK;
}

int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return device_sm_count(dev);
}

// The code of a CUDA call that failed, which is not left behind for the next call's check to find.
int cuda_failed() {
  cudaGetLastError();
  return SEGPAGED_ERR_CUDA;
}

// A launch that may start while the work before it ends; the kernel waits for that before it reads or writes anything,
// so that only its set-up overlaps the last blocks of what came before.
template <typename... Params, typename... Args>
int launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? SEGPAGED_OK : cuda_failed();
}

// Blocks of the kernels that take a slice of a page a warp: a warp for each slice (the kernels loop past the limit).
int slice_blocks(int64_t table_len, int log2_page) {
  const int64_t per_page = (1 << log2_page) / kSliceRows;
  return (int)std::min<int64_t>(ceil_div(std::min<int64_t>(table_len, INT32_MAX) * per_page, kSliceWarps), 1 << 22);
}

template <int D, int FMT>
int launch_build_quant(const BuildQuantParams& p, int grid, cudaStream_t st) {
  return p.b.cos_sin ? launch_early(build_quant_kernel<D, FMT, true>, dim3(grid), 32 * kSliceWarps, 0, st, p)
                     : launch_early(build_quant_kernel<D, FMT, false>, dim3(grid), 32 * kSliceWarps, 0, st, p);
}

template <int D, int FMT>
int launch_append(const AppendParams& p, cudaStream_t st) {
  return launch_early(append_kernel<D, FMT>, dim3(p.total_new, (unsigned)ceil_div(p.Hkv, 512 / D)), 32, 0, st, p);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
constexpr size_t kMetaBytes = 2 * kDecodeMaxCtas * sizeof(int32_t);
constexpr size_t kSlots = 2 * kDecodeMaxCtas;

// A pool [pages][P][D] as boxes of `rows` rows x one column block, in the swizzle of the kernel's stages.
template <int D, int FMT>
bool encode_pool(CUtensorMap* map, const void* base, int P, int64_t pages) {
  using C = DecodeCfg<D, FMT, 1>;
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)P, (cuuint64_t)pages};
  const cuuint64_t strides[2] = {(cuuint64_t)D * C::EB, (cuuint64_t)D * C::EB * P};
  const cuuint32_t box[3] = {(cuuint32_t)(C::ROWB / C::EB), (cuuint32_t)std::min(P, 64), 1}, estr[3] = {1, 1, 1};
  return enc(map, C::EB == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             C::ROWB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Where the table array has room for no more tokens than this (page_table_len is all the host knows of the tables), no (sequence, KV head) is cut into chunks and nothing is left
// to join: even if they are all one pair's, its tiles one after the other take no longer than the second launch. One head
// of 256, 512, 640, 768 tokens (D = 128, e4m3, replayed graphs): 8.1, 9.3, 9.8, 10.3 us whole, 9.9, 10.0, 10.1, 10.0 us
// cut and joined; eight heads of 64: 7.4 against 9.0 us. bf16 and D = 64 cross at or above 640 too.
constexpr int64_t kDecodeWholeTokens = 640;

template <int D, int FMT, int NB>
int launch_decode_nb(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, int grid, cudaStream_t st) {
  using C = DecodeCfg<D, FMT, NB>;
  static std::atomic<bool> configured[kMaxDevices];  // per device; a race only repeats the call
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SEGPAGED_ERR_CUDA;
  if (!configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(decode_kernel<D, FMT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
        cudaSuccess)
      return cuda_failed();
    configured[dev].store(true, std::memory_order_release);
  }
  if (launch_early(decode_kernel<D, FMT, NB>, dim3(grid), C::THREADS, C::SMEM_BYTES, st, tk, tv, p)) return SEGPAGED_ERR_CUDA;
  if (!p.whole && launch_early(decode_combine_kernel<D>, dim3(grid, std::min(p.G, kDecodeGroup)), 32 * kDecodeCombineWarps, 0, st, p))
    return SEGPAGED_ERR_CUDA;
  return SEGPAGED_OK;
}

// Up to eight query heads a KV head fill one column block of the products, up to sixteen two; larger groups take
// several passes of sixteen.
template <int D, int FMT>
int launch_decode(const void* k_pool, const void* v_pool, const DecodeParams& p, int grid, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!encode_pool<D, FMT>(&tk, k_pool, 1 << p.log2_page, p.num_pages) ||
      !encode_pool<D, FMT>(&tv, v_pool, 1 << p.log2_page, p.num_pages))
    return SEGPAGED_ERR_CUDA;
  return p.G <= 8 ? launch_decode_nb<D, FMT, 1>(tk, tv, p, grid, st) : launch_decode_nb<D, FMT, 2>(tk, tv, p, grid, st);
}

}  // namespace

// FN<D, FMT>(args) for the call's head_dim and pool format.
#define SEGPAGED_BY_SHAPE(FN, ...)                                            \
  do {                                                                        \
    if (dims->head_dim == 128) {                                              \
      if (kv_format == SEGPAGED_KV_E4M3) FN<128, kFmtE4m3> __VA_ARGS__;       \
      else if (kv_format == SEGPAGED_KV_INT8) FN<128, kFmtInt8> __VA_ARGS__;  \
      else FN<128, kFmtBf16> __VA_ARGS__;                                     \
    } else {                                                                  \
      if (kv_format == SEGPAGED_KV_E4M3) FN<64, kFmtE4m3> __VA_ARGS__;        \
      else if (kv_format == SEGPAGED_KV_INT8) FN<64, kFmtInt8> __VA_ARGS__;   \
      else FN<64, kFmtBf16> __VA_ARGS__;                                      \
    }                                                                         \
  } while (0)
// The same for the calls that take 8-bit pools only.
#define SEGPAGED_BY_SHAPE_8BIT(FN, ...)                                 \
  do {                                                                  \
    if (dims->head_dim == 128) {                                        \
      if (kv_format == SEGPAGED_KV_E4M3) FN<128, kFmtE4m3> __VA_ARGS__; \
      else FN<128, kFmtInt8> __VA_ARGS__;                               \
    } else {                                                            \
      if (kv_format == SEGPAGED_KV_E4M3) FN<64, kFmtE4m3> __VA_ARGS__;  \
      else FN<64, kFmtInt8> __VA_ARGS__;                                \
    }                                                                   \
  } while (0)

extern "C" int segpaged_build_quant(const segpaged_dims* dims, int32_t kv_format, const void* k_dense, const void* v_dense,
                                 const int32_t* cu_seqlens_k, const int32_t* q_len, const segpaged_head_class* cls,
                                    const int32_t* page_table, int64_t page_table_len, const int32_t* page_table_offs,
                                    const float* rope_cos_sin, void* k_pool, void* v_pool, uint8_t* kv_scale,
                                    int32_t* status, void* stream) {
  int rc = check_pools(dims, kv_format, false, k_pool, v_pool, kv_scale);
  if (rc) return rc;
  if (page_table_len < 0) return SEGPAGED_ERR_DIMS;
  if (dims->num_seqs == 0 || page_table_len == 0) return SEGPAGED_OK;
  if (!k_dense || !v_dense || !cu_seqlens_k || !q_len || !cls || !page_table || !page_table_offs) return SEGPAGED_ERR_NULL;
  if (!aligned16(k_dense) || !aligned16(v_dense) || (rope_cos_sin && !aligned16(rope_cos_sin))) return SEGPAGED_ERR_ALIGN;
  BuildQuantParams p;
  p.b.k_dense = static_cast<const __nv_bfloat16*>(k_dense);
  p.b.v_dense = static_cast<const __nv_bfloat16*>(v_dense);
  p.b.cu_k = cu_seqlens_k;
  p.b.q_len = q_len;
  p.b.cls = reinterpret_cast<const int32_t*>(cls);
  p.b.table = page_table;
  p.b.offs = page_table_offs;
  p.b.cos_sin = rope_cos_sin;
  p.b.k_pool = nullptr;
  p.b.v_pool = nullptr;
  p.b.status = status;
  p.b.B = dims->num_seqs;
  p.b.Hkv = dims->num_kv_heads;
  p.b.P = dims->page_size;
  p.b.num_pages = dims->num_pages;
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.kv_scale = kv_scale;
  p.table_len = page_table_len;
  p.log2_page = log2_int(dims->page_size);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SEGPAGED_BY_SHAPE_8BIT(rc = launch_build_quant, (p, slice_blocks(page_table_len, p.log2_page), st));
  return rc;
}

extern "C" int segpaged_append(const segpaged_dims* dims, int32_t kv_format, const void* k_new, const void* v_new,
                               int32_t total_new, const int32_t* cu_seqlens_new, const int32_t* ctx_len,
                               const int32_t* q_len, const segpaged_head_class* cls, const int32_t* page_table,
                               int64_t page_table_len, const int32_t* page_table_offs, void* k_pool, void* v_pool,
                               uint8_t* kv_scale, int32_t* status, void* stream) {
  int rc = check_pools(dims, kv_format, true, k_pool, v_pool, kv_scale);
  if (rc) return rc;
  if (total_new < 0 || page_table_len < 0) return SEGPAGED_ERR_DIMS;
  if (dims->num_seqs == 0 || total_new == 0) return SEGPAGED_OK;
  if (!k_new || !v_new || !cu_seqlens_new || !ctx_len || !cls || (!page_table && page_table_len > 0) || !page_table_offs) return SEGPAGED_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new)) return SEGPAGED_ERR_ALIGN;
  if (ceil_div(dims->num_kv_heads, 512 / dims->head_dim) > 65535) return SEGPAGED_ERR_DIMS;  // the grid's second extent
  AppendParams p;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.cu_new = cu_seqlens_new;
  p.ctx_len = ctx_len;
  p.q_len = q_len;
  p.cls = reinterpret_cast<const int32_t*>(cls);
  p.table = page_table;
  p.offs = page_table_offs;
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.kv_scale = kv_scale;
  p.status = status;
  p.table_len = page_table_len;
  p.total_new = total_new;
  p.B = dims->num_seqs;
  p.Hkv = dims->num_kv_heads;
  p.log2_page = log2_int(dims->page_size);
  p.num_pages = dims->num_pages;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SEGPAGED_BY_SHAPE(rc = launch_append, (p, st));
  return rc;
}

namespace {
template <int D, int FMT>
int launch_dequant(const DequantParams& p, int grid, cudaStream_t st) {
  return launch_early(dequant_pages_kernel<D, FMT>, dim3(grid), 32 * kSliceWarps, 0, st, p);
}
}  // namespace

extern "C" int segpaged_pages_dequant(const segpaged_dims* dims, int32_t kv_format, const int32_t* ctx_len,
                                      const int32_t* q_len, const segpaged_head_class* cls, const int32_t* page_table,
                                      int64_t page_table_len, const int32_t* page_table_offs, const void* k_pool,
                                      const void* v_pool, const uint8_t* kv_scale, void* k_out, void* v_out,
                                      int32_t* status, void* stream) {
  int rc = check_pools(dims, kv_format, false, k_pool, v_pool, kv_scale);
  if (rc) return rc;
  if (page_table_len < 0) return SEGPAGED_ERR_DIMS;
  if (dims->num_seqs == 0 || page_table_len == 0) return SEGPAGED_OK;
  if (!ctx_len || !cls || !page_table || !page_table_offs || !k_out || !v_out) return SEGPAGED_ERR_NULL;
  if (!aligned16(k_out) || !aligned16(v_out)) return SEGPAGED_ERR_ALIGN;
  DequantParams p;
  p.ctx_len = ctx_len;
  p.q_len = q_len;
  p.cls = reinterpret_cast<const int32_t*>(cls);
  p.table = page_table;
  p.offs = page_table_offs;
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.kv_scale = kv_scale;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.status = status;
  p.table_len = page_table_len;
  p.B = dims->num_seqs;
  p.Hkv = dims->num_kv_heads;
  p.log2_page = log2_int(dims->page_size);
  p.num_pages = dims->num_pages;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SEGPAGED_BY_SHAPE_8BIT(rc = launch_dequant, (p, slice_blocks(page_table_len, p.log2_page), st));
  return rc;
}

// Per CTA the two chunks its run can start and end with, and which pair goes on behind it.
extern "C" size_t segpaged_decode_workspace_bytes(const segpaged_dims* dims) {
  const size_t D = dims && dims->head_dim == 64 ? 64 : 128;
  return align256(kMetaBytes) + align256(kSlots * kDecodeGroup * sizeof(float2)) + kSlots * kDecodeGroup * D * sizeof(float);
}

extern "C" int segpaged_attn_decode(const segpaged_dims* dims, int32_t kv_format, const void* q, const void* k_pool,
                                    const void* v_pool, const uint8_t* kv_scale, const int32_t* page_table,
                                    int64_t page_table_len, const int32_t* page_table_offs, const int32_t* ctx_len,
                                    const int32_t* q_len, const segpaged_head_class* cls, float softmax_scale, void* o,
                                    float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                                    void* stream) {
  int rc = check_pools(dims, kv_format, true, k_pool, v_pool, kv_scale);
  if (rc) return rc;
  if (page_table_len < 0) return SEGPAGED_ERR_DIMS;
  if (dims->num_seqs == 0) return SEGPAGED_OK;
  if (!q || (!page_table && page_table_len > 0) || !page_table_offs || !ctx_len || !cls || !o || !lse || !workspace) return SEGPAGED_ERR_NULL;
  if (workspace_bytes < segpaged_decode_workspace_bytes(dims)) return SEGPAGED_ERR_CAPACITY;
  if (!aligned16(q) || !aligned16(o) || !aligned16(workspace)) return SEGPAGED_ERR_ALIGN;
  // The kernel counts half tiles, and kDecodeMostPairCost for each pair, in 32 bits. Tiles are fewer than table entries.
  const int64_t pairs = (int64_t)dims->num_seqs * dims->num_kv_heads, passes = std::max(dims->num_q_heads / dims->num_kv_heads / kDecodeGroup, 1);
  if (page_table_len > INT32_MAX || (2 * page_table_len + kDecodeMostPairCost * pairs) * passes > UINT32_MAX) return SEGPAGED_ERR_DIMS;
  const float scale_log2 = softmax_scale * 1.4426950408889634f;
  if (!std::isfinite(scale_log2)) return SEGPAGED_ERR_DIMS;
  const int sms = sm_count();
  if (sms <= 0) return SEGPAGED_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.part_meta = reinterpret_cast<int32_t*>(ws);
  p.part_sum = reinterpret_cast<float2*>(ws + align256(kMetaBytes));
  p.part_o = reinterpret_cast<float*>(ws + align256(kMetaBytes) + align256(kSlots * kDecodeGroup * sizeof(float2)));
  p.kv_scale = kv_scale;
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.table = page_table;
  p.offs = page_table_offs;
  p.ctx_len = ctx_len;
  p.q_len = q_len;
  p.cls = reinterpret_cast<const int32_t*>(cls);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.status = status;
  p.table_len = page_table_len;
  p.B = dims->num_seqs;
  p.Hkv = dims->num_kv_heads;
  p.G = dims->num_q_heads / dims->num_kv_heads;
  p.log2_page = log2_int(dims->page_size);
  p.num_pages = dims->num_pages;
  p.log2_hg = p.G > kDecodeGroup ? log2_int(p.G / kDecodeGroup) : 0;
  p.whole = page_table_len <= kDecodeWholeTokens >> p.log2_page;
  p.scale_log2 = scale_log2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = SEGPAGED_OK;
  SEGPAGED_BY_SHAPE(rc = launch_decode, (k_pool, v_pool, p, std::min(sms, kDecodeMaxCtas), st));
  return rc;
}
