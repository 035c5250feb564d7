// Rows of a beam's states (texts, token counts, contiguous caches) in the
// order of their parents.
//
// A copy: what bounds it is memory.  Where every row starts on the 16-byte grid a
// thread takes the same 16 bytes of all rows of a sequence: it reads what their
// parents hold there, then writes.  Elsewhere a CTA does the same with a tile of
// all rows, by way of shared memory: rows come and go as whole vectors of their
// own place on the grid, and the shift between a row and its parent's is made in
// between.  Either way a parent of several rows comes from memory once, and a
// state may be reordered where it is, without a copy of it.

#include "sd_rows.cuh"
#include "sd_beam.h"

namespace sdv {

constexpr int kReNT = 256;

constexpr int kReTile = 4096;     // bytes of a row in a tile, at most,
constexpr int kReStage = 32768;   // and of all rows

struct ReorderState {
  const uint8_t *in;
  uint8_t *out;
  int64_t in_sb, in_sw, out_sb, out_sw;
  int64_t row_bytes;
  int tile;       // bytes of a tile, 0: columns of 16 bytes
  int parts;      // CTAs of a sequence
  bool in_place;
};
struct ReorderParams {
  const int32_t *parents;
  int32_t *status;
  int B, W, k, n;
  ReorderState s[SD_MAX_STATES];
};

// R rows at a time; in place they are all of the sequence's.
template <int R>
__device__ __forceinline__ void reorder_column(const ReorderState &s, const int *from, int k, int b,
                                               int64_t at) {
  const uint8_t *in = s.in + b * s.in_sb + at;
  uint8_t *out = s.out + b * s.out_sb + at;
  for (int k0 = 0; k0 < k; k0 += R) {
    uint4 v[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (k0 + i < k && from[k0 + i] >= 0) v[i] = ld16(in + from[k0 + i] * s.in_sw);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (k0 + i < k && from[k0 + i] >= 0)
        *reinterpret_cast<uint4 *>(out + (k0 + i) * s.out_sw) = v[i];
  }
}

// 16 bytes from byte `shift` of a, b on.
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, int shift) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
  const int bits = (shift & 3) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes [c0, c0 + n) of all rows; `used`: whether a row is anybody's parent.
__device__ __forceinline__ void reorder_tile(const ReorderState &s, const int *from,
                                             const int *used, int W, int k, int b, int64_t c0,
                                             int n, uint8_t *stage) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pitch = s.tile + 32;
  for (int p = warp; p < W; p += kReNT / 32) {
    if (!used[p]) continue;
    const uint8_t *src = s.in + b * s.in_sb + p * s.in_sw + c0;
    const int off = (int)((uintptr_t)src & 15);   // of the first byte in the row's place
    uint8_t *to = stage + p * pitch;
    const int head = min((16 - off) & 15, n), body = (n - head) & ~15;
    for (int i = lane * 16; i < body; i += 512)
      row_async16(smem_u32(to + off + head + i), src + head + i);
    if (lane < head) to[off + lane] = (uint8_t)ld1(src + lane);
    const int tail = head + body + lane;
    if (tail < n) to[off + tail] = (uint8_t)ld1(src + tail);
  }
  cp_commit();
  cp_wait<0>();
  __syncthreads();
  for (int i = warp; i < k; i += kReNT / 32) {
    const int p = from[i];
    if (p < 0) continue;
    uint8_t *dst = s.out + b * s.out_sb + i * s.out_sw + c0;
    const uint8_t *src =
        stage + p * pitch + ((uintptr_t)(s.in + b * s.in_sb + p * s.in_sw + c0) & 15);
    const int head = min((int)(16 - ((uintptr_t)dst & 15)) & 15, n), body = (n - head) & ~15;
    const uint32_t at = smem_u32(src + head);
    const int shift = at & 15;
#pragma unroll 2
    for (int j = lane * 16; j < body; j += 512) {
      const uint32_t q = at - shift + j;
      *reinterpret_cast<uint4 *>(dst + head + j) = shifted(lds16(q), lds16(q + 16), shift);
    }
    if (lane < head) dst[lane] = src[lane];
    const int tail = head + body + lane;
    if (tail < n) dst[tail] = src[tail];
  }
}

template <int R>
__global__ void __launch_bounds__(kReNT) sd_beam_reorder_kernel(const __grid_constant__ ReorderParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int from[SD_MAX_TOP];
  __shared__ int used[SD_MAX_BEAMS];
  extern __shared__ uint4 stage[];
  int at = blockIdx.x, i = 0;
  while (i + 1 < P.n && at >= P.s[i].parts * P.B) at -= P.s[i++].parts * P.B;
  const ReorderState &s = P.s[i];
  const int b = at / s.parts, part = at % s.parts;
  if (threadIdx.x < SD_MAX_BEAMS) used[threadIdx.x] = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < P.k; j += kReNT) {
    int p = ld_int(P.parents + (int64_t)b * P.k + j);
    if (p < 0 || p >= P.W) {
      if (p != -1 && P.status) atomicOr(P.status, (int)SD_STATUS_BAD_PARENT);
      p = j < P.W ? j : -1;
    }
    if (s.in_place && p == j) p = -1;
    from[j] = p;
    if (p >= 0) used[p] = 1;
  }
  __syncthreads();
  if (s.tile > 0) {
    const int64_t c0 = (int64_t)part * s.tile;
    reorder_tile(s, from, used, P.W, P.k, b, c0, (int)min(s.row_bytes - c0, (int64_t)s.tile),
                 reinterpret_cast<uint8_t *>(stage));
  } else {
    const int64_t col = ((int64_t)part * kReNT + threadIdx.x) * 16;
    if (col < s.row_bytes) reorder_column<R>(s, from, P.k, b, col);
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
  int smem = 0;
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
    uint64_t bits = (uint64_t)(uintptr_t)a.in | (uintptr_t)a.out | (uint64_t)a.row_bytes;
    if (B > 1) bits |= (uint64_t)a.in_sb | (uint64_t)a.out_sb;
    if (W > 1) bits |= (uint64_t)a.in_sw;
    if (k > 1) bits |= (uint64_t)a.out_sw;
    s.row_bytes = a.row_bytes;
    // Measured, us, columns / tiles of rows on the grid: 32 x 8 rows of 304000 bytes 20.3 / 21.7, in
    // place 13.8 / 14.9; 16 x 16 in place 18.8 / 18.1, 8 x 32 in place 24.3 / 24.3.  Off the grid
    // columns of 4, 2 and 1 bytes took 35, 63 and 120 where tiles take 22.
    if (bits & 15 || (s.in_place && W > 8)) {
      s.tile = std::min(kReTile, kReStage / W / 512 * 512);
      smem = std::max(smem, W * (s.tile + 32));
    } else {
      in_place |= s.in_place;
    }
    const int64_t tile = s.tile > 0 ? s.tile : kReNT * 16;
    const int64_t parts = (s.row_bytes + tile - 1) / tile;
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
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // rows in registers at once: all of a sequence's in place, where they are columns
  const cudaError_t e = in_place && W > 4
                            ? cudaLaunchKernelEx(&cfg, sd_beam_reorder_kernel<8>, P)
                            : cudaLaunchKernelEx(&cfg, sd_beam_reorder_kernel<4>, P);
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}

extern "C" size_t sd_beam_state_size(void) { return sizeof(sd_beam_state); }
