// Pages copied inside a cache's tensors: after a fork (the filled entries of
// last pages) and after compaction (whole pages).
//
// A copy: what bounds it is memory.  The work is cut into pieces of one part of
// one page of one layer; the number of pairs is read on the device, CTAs take
// pieces until there are none left.

#include "sd_rows.cuh"
#include "sd_kv.h"

namespace sdv {

constexpr int kCpNT = 256, kCpU = 4;   // a piece: kCpU vectors per thread

struct CopyParams {
  int n_caches, layers, N, parts, page_size, pairs, width;
  int64_t entry_bytes, part_bytes, layer_stride, page_stride;
  int pieces;                 // of a part
  int64_t per_pair;           // pieces of a pair
  const int32_t *src, *dst, *fill, *count;
  int32_t *status;
  uint8_t *caches[SD_MAX_CACHES];
};

template <typename T>
__device__ __forceinline__ void copy_piece(const uint8_t *from, uint8_t *to, int64_t bytes,
                                           T (*load)(const uint8_t *)) {
  const int64_t n = bytes / (int64_t)sizeof(T);
  T v[kCpU];
#pragma unroll
  for (int u = 0; u < kCpU; ++u) {
    const int64_t i = threadIdx.x + u * kCpNT;
    if (i < n) v[u] = load(from + i * sizeof(T));
  }
#pragma unroll
  for (int u = 0; u < kCpU; ++u) {
    const int64_t i = threadIdx.x + u * kCpNT;
    if (i < n) reinterpret_cast<T *>(to)[i] = v[u];
  }
}
__device__ __forceinline__ uint4 load16(const uint8_t *p) { return ld16(p); }
__device__ __forceinline__ uint32_t load4(const uint8_t *p) { return ld4(p); }
__device__ __forceinline__ uint16_t load2(const uint8_t *p) { return (uint16_t)ld2(p); }
__device__ __forceinline__ uint8_t load1(const uint8_t *p) { return (uint8_t)ld1(p); }

__global__ void __launch_bounds__(kCpNT) sd_kv_copy_kernel(const __grid_constant__ CopyParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int pairs = P.count ? min(max(ld_int(P.count), 0), P.pairs) : P.pairs;
  const int64_t total = pairs * P.per_pair;
  const int64_t piece_bytes = (int64_t)kCpNT * kCpU * P.width;
  for (int64_t x = blockIdx.x; x < total; x += gridDim.x) {
    const int pair = (int)(x / P.per_pair);
    int64_t r = x - pair * P.per_pair;
    const int src = ld_int(P.src + pair), dst = ld_int(P.dst + pair);
    if ((unsigned)src >= (unsigned)P.N || (unsigned)dst >= (unsigned)P.N) {
      if ((src != -1 || dst != -1) && r == 0 && threadIdx.x == 0 && P.status)
        atomicOr(P.status, (int)SD_STATUS_BAD_PAGE);
      continue;
    }
    int64_t bytes = P.part_bytes;
    if (P.fill) bytes = min(max(ld_int(P.fill + pair), 0), P.page_size) * P.entry_bytes;
    const int piece = (int)(r % P.pieces);
    r /= P.pieces;
    const int part = (int)(r % P.parts);
    r /= P.parts;
    const int layer = (int)(r % P.layers), cache = (int)(r / P.layers);
    const int64_t at = piece * piece_bytes;
    if (at >= bytes) continue;
    bytes = min(bytes - at, piece_bytes);
    uint8_t *base = P.caches[cache] + layer * P.layer_stride + part * P.part_bytes + at;
    const uint8_t *from = base + src * P.page_stride;
    uint8_t *to = base + dst * P.page_stride;
    if (P.width == 16) copy_piece<uint4>(from, to, bytes, load16);
    else if (P.width == 4) copy_piece<uint32_t>(from, to, bytes, load4);
    else if (P.width == 2) copy_piece<uint16_t>(from, to, bytes, load2);
    else copy_piece<uint8_t>(from, to, bytes, load1);
  }
}

}  // namespace sdv

using namespace sdv;

extern "C" sd_status_t sd_kv_copy(const sd_kv_copy_args *a, void *stream) {
  sdv::NvtxRange nvtx_range("sd_kv_copy");
  if (!a || a->n_caches < 0 || a->n_caches > SD_MAX_CACHES || a->layers < 0 || a->N < 1 ||
      a->N > SD_MAX_PAGES || a->parts < 1 || a->page_size < 1 || a->entry_bytes < 0 || a->pairs < 0)
    return SD_ERR_INVALID_ARG;
  if (a->entry_bytes > ((int64_t)1 << 40) / a->page_size / a->parts) return SD_ERR_INVALID_ARG;
  if (a->n_caches == 0 || a->layers == 0 || a->entry_bytes == 0 || a->pairs == 0) return SD_OK;
  if (!a->caches || !a->src || !a->dst) return SD_ERR_INVALID_ARG;
  CopyParams P = {};
  P.n_caches = a->n_caches;
  P.layers = a->layers;
  P.N = a->N;
  P.parts = a->parts;
  P.page_size = a->page_size;
  P.pairs = a->pairs;
  P.entry_bytes = a->entry_bytes;
  P.part_bytes = a->entry_bytes * a->page_size;
  P.layer_stride = a->layer_stride;
  P.page_stride = a->page_stride;
  P.src = a->src;
  P.dst = a->dst;
  P.fill = a->fill;
  P.count = a->count;
  P.status = a->status;
  // whole entries are copied, so that an entry's bytes bound the vectors' width; without
  // fill whole parts
  uint64_t bits = 16 | (uint64_t)(P.fill ? P.entry_bytes : P.part_bytes) | (uint64_t)P.part_bytes;
  if (P.layers > 1) bits |= (uint64_t)P.layer_stride;
  if (P.N > 1) bits |= (uint64_t)P.page_stride;
  for (int i = 0; i < P.n_caches; ++i) {
    if (!a->caches[i]) return SD_ERR_INVALID_ARG;
    P.caches[i] = static_cast<uint8_t *>(a->caches[i]);
    bits |= (uint64_t)(uintptr_t)a->caches[i];
  }
  const int w = (int)(bits & (~bits + 1));
  P.width = w == 16 ? 16 : w >= 4 ? 4 : w;
  const int64_t piece = (int64_t)kCpNT * kCpU * P.width;
  const int64_t pieces = (P.part_bytes + piece - 1) / piece;
  if (pieces > INT32_MAX) return SD_ERR_INVALID_ARG;
  P.pieces = (int)pieces;
  P.per_pair = pieces * P.parts * P.layers * P.n_caches;
  const int64_t most = std::min<int64_t>(P.per_pair * P.pairs, (int64_t)8 * sm_count());
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)most, 1, 1);
  cfg.blockDim = dim3(kCpNT, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sd_kv_copy_kernel, P);
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}

extern "C" size_t sd_kv_copy_args_size(void) { return sizeof(sd_kv_copy_args); }
