// Rows of a beam's states (texts, token counts, contiguous caches) in the
// order of their parents.
//
// A copy: what bounds it is memory.  A thread takes the same column of up to 16
// bytes of all rows of a sequence: it reads what their parents hold there, then
// writes.  So a parent of several rows comes from memory once, and a state may
// be reordered where it is, without a copy of it.

#include "sd_rows.cuh"
#include "sd_beam.h"

namespace sdv {

constexpr int kReNT = 256;

struct ReorderState {
  const uint8_t *in;
  uint8_t *out;
  int64_t in_sb, in_sw, out_sb, out_sw;
  int64_t cols;   // columns of a row
  int width;      // bytes of a column: 16, 8, 4, 2 or 1
  int parts;      // CTAs of a sequence
  bool in_place;
};
struct ReorderParams {
  const int32_t *parents;
  int32_t *status;
  int B, W, k, n;
  ReorderState s[SD_MAX_STATES];
};

template <int BYTES>
struct Column;
template <>
struct Column<16> {
  using T = uint4;
  static __device__ __forceinline__ T load(const uint8_t *p) { return ld16(p); }
};
template <>
struct Column<8> {
  using T = uint2;
  static __device__ __forceinline__ T load(const uint8_t *p) {
    uint2 v;
    asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
  }
};
template <>
struct Column<4> {
  using T = uint32_t;
  static __device__ __forceinline__ T load(const uint8_t *p) { return ld4(p); }
};
template <>
struct Column<2> {
  using T = uint16_t;
  static __device__ __forceinline__ T load(const uint8_t *p) { return (uint16_t)ld2(p); }
};
template <>
struct Column<1> {
  using T = uint8_t;
  static __device__ __forceinline__ T load(const uint8_t *p) { return (uint8_t)ld1(p); }
};

// R rows at a time; in place they are all of the sequence's.
template <int BYTES, int R>
__device__ __forceinline__ void reorder_column(const ReorderState &s, const int *from, int k, int b,
                                               int64_t col) {
  using C = Column<BYTES>;
  const uint8_t *in = s.in + b * s.in_sb + col * BYTES;
  uint8_t *out = s.out + b * s.out_sb + col * BYTES;
  for (int k0 = 0; k0 < k; k0 += R) {
    typename C::T v[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (k0 + i < k && from[k0 + i] >= 0) v[i] = C::load(in + from[k0 + i] * s.in_sw);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (k0 + i < k && from[k0 + i] >= 0)
        *reinterpret_cast<typename C::T *>(out + (k0 + i) * s.out_sw) = v[i];
  }
}

template <int R>
__global__ void __launch_bounds__(kReNT) sd_beam_reorder_kernel(const __grid_constant__ ReorderParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int from[SD_MAX_TOP];
  int at = blockIdx.x, i = 0;
  while (i + 1 < P.n && at >= P.s[i].parts * P.B) at -= P.s[i++].parts * P.B;
  const ReorderState &s = P.s[i];
  const int b = at / s.parts, part = at % s.parts;
  for (int j = threadIdx.x; j < P.k; j += kReNT) {
    int p = ld_int(P.parents + (int64_t)b * P.k + j);
    if (p < 0 || p >= P.W) {
      if (p != -1 && P.status) atomicOr(P.status, (int)SD_STATUS_BAD_PARENT);
      p = j < P.W ? j : -1;
    }
    from[j] = s.in_place && p == j ? -1 : p;
  }
  __syncthreads();
  const int64_t col = (int64_t)part * kReNT + threadIdx.x;
  if (col >= s.cols) return;
  switch (s.width) {
    case 16: return reorder_column<16, R>(s, from, P.k, b, col);
    case 8: return reorder_column<8, R>(s, from, P.k, b, col);
    case 4: return reorder_column<4, R>(s, from, P.k, b, col);
    case 2: return reorder_column<2, R>(s, from, P.k, b, col);
    default: return reorder_column<1, R>(s, from, P.k, b, col);
  }
}

}  // namespace sdv

using namespace sdv;

extern "C" sd_status_t sd_beam_reorder(int32_t B, int32_t W, int32_t k, const int32_t *parents,
                                       int32_t n_states, const sd_beam_state *states,
                                       int32_t *status, void *stream) {
  sdv::NvtxRange nvtx_range("sd_beam_reorder");
  if (B < 0 || W < 1 || W > SD_MAX_BEAMS || k < 0 || k > SD_MAX_TOP || n_states < 0 ||
      n_states > SD_MAX_STATES || (n_states > 0 && !states))
    return SD_ERR_INVALID_ARG;
  ReorderParams P = {};
  P.parents = parents;
  P.status = status;
  P.B = B;
  P.W = W;
  P.k = k;
  int64_t grid = 0;
  bool in_place = false;
  for (int i = 0; i < n_states; ++i) {
    const sd_beam_state &a = states[i];
    if (a.row_bytes < 0) return SD_ERR_INVALID_ARG;
    if (B == 0 || k == 0 || a.row_bytes == 0) continue;
    if (!a.in || !a.out) return SD_ERR_INVALID_ARG;
    ReorderState &s = P.s[P.n];
    s.in = static_cast<const uint8_t *>(a.in);
    s.out = static_cast<uint8_t *>(a.out);
    s.in_sb = a.in_sb;
    s.in_sw = a.in_sw;
    s.out_sb = a.out_sb;
    s.out_sw = a.out_sw;
    s.in_place = a.in == a.out;
    if (s.in_place && (k != W || (B > 1 && a.in_sb != a.out_sb) || (W > 1 && a.in_sw != a.out_sw)))
      return SD_ERR_INVALID_ARG;
    in_place |= s.in_place;
    uint64_t bits = (uint64_t)(uintptr_t)a.in | (uintptr_t)a.out | (uint64_t)a.row_bytes | 16;
    if (B > 1) bits |= (uint64_t)a.in_sb | (uint64_t)a.out_sb;
    if (W > 1) bits |= (uint64_t)a.in_sw;
    if (k > 1) bits |= (uint64_t)a.out_sw;
    s.width = (int)(bits & (~bits + 1));
    s.cols = a.row_bytes / s.width;
    const int64_t parts = (s.cols + kReNT - 1) / kReNT;
    grid += parts * B;
    if (grid > INT32_MAX) return SD_ERR_INVALID_ARG;
    s.parts = (int)parts;
    ++P.n;
  }
  if (P.n == 0) return SD_OK;
  if (!parents) return SD_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kReNT, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // rows in registers at once: all of a sequence's in place
  const int need = in_place ? W : 4;
  const cudaError_t e = need <= 4    ? cudaLaunchKernelEx(&cfg, sd_beam_reorder_kernel<4>, P)
                        : need <= 8  ? cudaLaunchKernelEx(&cfg, sd_beam_reorder_kernel<8>, P)
                        : need <= 16 ? cudaLaunchKernelEx(&cfg, sd_beam_reorder_kernel<16>, P)
                                     : cudaLaunchKernelEx(&cfg, sd_beam_reorder_kernel<32>, P);
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}

extern "C" size_t sd_beam_state_size(void) { return sizeof(sd_beam_state); }
