// Pages copied inside a cache's tensors: after a fork (the filled entries of
// last pages) and after compaction (whole pages).
//
// A copy: what bounds it is memory.  Measured on the GPU: 16384 pages of 4 KB in each of
// 4 layers 88.8 us (537 MB, 6.0 TB/s, 90 % of a plain copy's rate); with eight
// CTAs per SM and half the piece 112, with four 89.7, three 89.0, one CTA of
// twice the piece 88.9.  By CTAs of 256 threads, a page each: 194.
// The work is cut into pieces of at most
// 32 kCpU vectors of one part of one page of one layer, one warp each; the number
// of pairs is read on the device, and warps take pieces until there are none
// left, with the next piece's page ids already asked for.  A piece's five
// numbers (pair, cache, layer, part, piece) are counted up by the grid's own,
// digit by digit, without divisions.

#include "sd_rows.cuh"
#include "sd_kv.h"

namespace sdv {

constexpr int kCpNT = 256, kCpCtas = 2;   // threads of a CTA, CTAs per SM
constexpr int kCpU = 8;                   // vectors of a piece per lane
constexpr int kCpWarps = kCpNT / 32;

// A piece's place, and how far apart a warp's pieces are.
struct CopyAt {
  int piece, part, layer, cache, pair;
};

struct CopyParams {
  int n_caches, layers, N, parts, page_size, pairs, width, pieces;
  int64_t entry_bytes, part_bytes, layer_stride, page_stride;
  CopyAt step;
  const int32_t *src, *dst, *fill, *count;
  int32_t *status;
  uint8_t *caches[SD_MAX_CACHES];
};

template <typename T>
__host__ __device__ inline CopyAt copy_at(const CopyParams &P, T x) {
  CopyAt a;
  a.piece = (int)(x % P.pieces);
  x /= P.pieces;
  a.part = (int)(x % P.parts);
  x /= P.parts;
  a.layer = (int)(x % P.layers);
  x /= P.layers;
  a.cache = (int)(x % P.n_caches);
  a.pair = (int)(x / P.n_caches);
  return a;
}
__device__ __forceinline__ CopyAt copy_next(const CopyParams &P, CopyAt a) {
  const auto digit = [](int &at, int more, int end) {
    at += more;
    const bool over = at >= end;
    at -= over ? end : 0;
    return over ? 1 : 0;
  };
  int carry = digit(a.piece, P.step.piece, P.pieces);
  carry = digit(a.part, P.step.part + carry, P.parts);
  carry = digit(a.layer, P.step.layer + carry, P.layers);
  carry = digit(a.cache, P.step.cache + carry, P.n_caches);
  a.pair += P.step.pair + carry;
  return a;
}

template <typename T, typename F>
__device__ __forceinline__ void copy_piece(const uint8_t *from, uint8_t *to, int bytes, F load) {
  const int lane = threadIdx.x & 31, n = bytes / (int)sizeof(T);
  from += lane * sizeof(T);
  to += lane * sizeof(T);
  T v[kCpU];
#pragma unroll
  for (int u = 0; u < kCpU; ++u)
    if (lane + u * 32 < n) v[u] = load(from + u * 32 * sizeof(T));
#pragma unroll
  for (int u = 0; u < kCpU; ++u)
    if (lane + u * 32 < n) *reinterpret_cast<T *>(to + u * 32 * sizeof(T)) = v[u];
  // entries need not end with a vector
  const int rest = bytes - n * (int)sizeof(T);
  if (lane < rest) {
    const int at = n * (int)sizeof(T) + lane - lane * (int)sizeof(T);
    to[at] = (uint8_t)ld1(from + at);
  }
}

__global__ void __launch_bounds__(kCpNT, kCpCtas)
    sd_kv_copy_kernel(const __grid_constant__ CopyParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int pairs = P.count ? min(max(ld_int(P.count), 0), P.pairs) : P.pairs;
  const int piece_bytes = 32 * kCpU * P.width;
  CopyAt a = copy_at(P, (int)(blockIdx.x * kCpWarps + (threadIdx.x >> 5)));
  if (a.pair >= pairs) return;
  int src = ld_int(P.src + a.pair), dst = ld_int(P.dst + a.pair);
  int fill = P.fill ? ld_int(P.fill + a.pair) : P.page_size;
  while (true) {
    const CopyAt next = copy_next(P, a);
    const bool more = next.pair < pairs;
    int src1 = 0, dst1 = 0, fill1 = P.page_size;
    if (more) {
      src1 = ld_int(P.src + next.pair);
      dst1 = ld_int(P.dst + next.pair);
      if (P.fill) fill1 = ld_int(P.fill + next.pair);
    }
    if ((unsigned)src < (unsigned)P.N && (unsigned)dst < (unsigned)P.N) {
      const int64_t at = (int64_t)a.piece * piece_bytes;
      const int64_t end = P.fill ? min(max(fill, 0), P.page_size) * P.entry_bytes : P.part_bytes;
      if (at < end) {
        const int bytes = (int)min(end - at, (int64_t)piece_bytes);
        uint8_t *base = P.caches[a.cache] + a.layer * P.layer_stride + a.part * P.part_bytes + at;
        const uint8_t *from = base + src * P.page_stride;
        uint8_t *to = base + dst * P.page_stride;
        if (P.width == 16)
          copy_piece<uint4>(from, to, bytes, [](const uint8_t *p) { return ld16(p); });
        else if (P.width == 4)
          copy_piece<uint32_t>(from, to, bytes, [](const uint8_t *p) { return ld4(p); });
        else if (P.width == 2)
          copy_piece<uint16_t>(from, to, bytes, [](const uint8_t *p) { return (uint16_t)ld2(p); });
        else
          copy_piece<uint8_t>(from, to, bytes, [](const uint8_t *p) { return (uint8_t)ld1(p); });
      }
    } else if ((src != -1 || dst != -1) && P.status) {
      atomicOr(P.status, (int)SD_STATUS_BAD_PAGE);
    }
    if (!more) return;
    a = next;
    src = src1;
    dst = dst1;
    fill = fill1;
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
  uint64_t bits = 16 | (uint64_t)P.part_bytes;   // what bounds the vectors' width
  if (P.layers > 1) bits |= (uint64_t)P.layer_stride;
  if (P.N > 1) bits |= (uint64_t)P.page_stride;
  for (int i = 0; i < P.n_caches; ++i) {
    if (!a->caches[i]) return SD_ERR_INVALID_ARG;
    P.caches[i] = static_cast<uint8_t *>(a->caches[i]);
    bits |= (uint64_t)(uintptr_t)a->caches[i];
  }
  const int w = (int)(bits & (~bits + 1));
  P.width = w == 16 ? 16 : w >= 4 ? 4 : w;
  const int64_t piece = (int64_t)32 * kCpU * P.width;
  const int64_t pieces = (P.part_bytes + piece - 1) / piece;
  // no digit and no number of pieces overflows
  constexpr int64_t kMost = (int64_t)1 << 30;
  if (pieces > kMost || P.parts > kMost || P.layers > kMost || P.pairs > kMost ||
      pieces * P.parts > kMost || pieces * P.parts * P.layers > kMost * SD_MAX_CACHES)
    return SD_ERR_INVALID_ARG;
  P.pieces = (int)pieces;
  const int64_t per_pair = pieces * P.parts * P.layers * P.n_caches;
  const int64_t most = std::min<int64_t>((per_pair * P.pairs + kCpWarps - 1) / kCpWarps,
                                         (int64_t)kCpCtas * sm_count());
  P.step = copy_at(P, most * kCpWarps);
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
