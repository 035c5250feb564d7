// Token counts of each sequence, the state that penalties on logits read:
// 16 bits per vocabulary entry, the low 15 the number of times the output
// text holds the token (saturating), the top one set where the prompt does.
//
// Integer work.  sd_token_counts gives each CTA one slice of one sequence's
// vocabulary: a histogram in shared memory, two 16-bit bins per word, fed by
// the whole history (read from L2 by the slices after the first) and written
// out once.  Counts cannot carry into the neighbouring bin: at most 32768
// tokens are added to bins of at most 32767 before every bin is cut back.
// sd_token_counts_add is one thread per emitted token.
// Measured on the GPU: 256 histories of 16384 tokens over 128256 ids 22 us
// (82 MB in and out, 3.7 TB/s); 3 of 131071 over 151936 ids 13 us.  What bounds
// both is that the vocabulary is shared out and the history is not: each of the
// first's four slices reads all of a sequence's tokens, in 2.25 waves of CTAs,
// each of the second's fifty all 131071 of them from L2, four vectors per thread
// in flight.  Without the atomics the first still takes 22 us, and neither
// smaller nor larger slices shorten it.

#include "sd_rows.cuh"

namespace sdv {

constexpr int kCntSlice = 32768;      // most bins of one CTA: 64 KB, three CTAs per SM
constexpr int kCntLeast = 2048;       // fewest, where there are few sequences
constexpr int kCntChunk = 32768;      // tokens added between two cuts

// Calls f(token) for this thread's tokens of h[a .. b): kCntU vectors of four
// in flight where they lie on the 16-byte grid, the ends one by one.
constexpr int kCntU = 4;
template <int NT, typename F>
__device__ __forceinline__ void each_token(const int32_t *h, int a, int b, F f) {
  const int tid = threadIdx.x, off = (int)((uintptr_t)(h + a) >> 2) & 3;
  const int head = min(b, a + ((4 - off) & 3)), nv = (b - head) >> 2, tail = head + nv * 4;
  if (tid < head - a) f(ld_int(h + a + tid));
  if (tid < b - tail) f(ld_int(h + tail + tid));
  for (int i = tid; i < nv; i += kCntU * NT) {
    uint4 v[kCntU];
#pragma unroll
    for (int u = 0; u < kCntU; ++u)
      if (i + u * NT < nv) v[u] = ld16(h + head + 4 * (int64_t)(i + u * NT));
#pragma unroll
    for (int u = 0; u < kCntU; ++u)
      if (i + u * NT < nv) {
        f((int)v[u].x);
        f((int)v[u].y);
        f((int)v[u].z);
        f((int)v[u].w);
      }
  }
}

template <int NT>
__global__ void __launch_bounds__(NT, NT == 512 ? 3 : 1) sd_token_counts_kernel(
    int L, int V, int nslice, int slice, const int32_t *history, const int32_t *lengths,
    const int32_t *prompt_lengths, uint16_t *counts, int32_t *status) {
  // a programmatic dependent of the stream's previous kernel: nothing is read
  // before it has finished; the next launch may be scheduled at once
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint4 bin_vecs[];
  uint32_t *bins = reinterpret_cast<uint32_t *>(bin_vecs);   // bin i: half i & 1 of word i >> 1
  const int b = blockIdx.x / nslice, s0 = (blockIdx.x % nslice) * slice;
  const int n = min(slice, V - s0), nvec = (n + 7) >> 3, tid = threadIdx.x;
  const int32_t *h = history + (int64_t)b * L;
  const int len = min(max(ld_int(lengths + b), 0), L);
  const int pl = prompt_lengths ? min(max(ld_int(prompt_lengths + b), 0), len) : 0;
  for (int i = tid; i < nvec; i += NT) bin_vecs[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  bool bad = false;
  for (int c0 = pl; c0 < len; c0 += min(kCntChunk, len - c0)) {
    each_token<NT>(h, c0, c0 + min(kCntChunk, len - c0), [&](int t) {
      bad |= (unsigned)t >= (unsigned)V;
      const unsigned e = (unsigned)t - (unsigned)s0;
      if (e < (unsigned)n) atomicAdd(&bins[e >> 1], (e & 1u) ? 0x10000u : 1u);
    });
    __syncthreads();
    if (len - pl > 32767) {
      for (int i = tid; i < (n + 1) >> 1; i += NT) {
        const uint32_t w = bins[i];
        bins[i] = min(w & 0xffffu, 32767u) | (min(w >> 16, 32767u) << 16);
      }
      __syncthreads();
    }
  }
  each_token<NT>(h, 0, pl, [&](int t) {
    bad |= (unsigned)t >= (unsigned)V;
    const unsigned e = (unsigned)t - (unsigned)s0;
    if (e < (unsigned)n) atomicOr(&bins[e >> 1], (e & 1u) ? 0x80000000u : 0x8000u);
  });
  __syncthreads();
  uint16_t *out = counts + (int64_t)b * V + s0;
  if (((uintptr_t)out & 15) == 0) {
    for (int i = tid; i < n / 8; i += NT) reinterpret_cast<uint4 *>(out)[i] = bin_vecs[i];
    for (int i = (n & ~7) + tid; i < n; i += NT)
      out[i] = reinterpret_cast<const uint16_t *>(bins)[i];
  } else {
    for (int i = tid; i < n; i += NT) out[i] = reinterpret_cast<const uint16_t *>(bins)[i];
  }
  if (bad && s0 == 0 && status) atomicOr(status, (int)SD_STATUS_BAD_TOKEN);
}

__global__ void __launch_bounds__(256) sd_token_counts_add_kernel(
    int M, int V, const int32_t *tokens, const int32_t *n, uint16_t *counts, int32_t *status,
    int64_t total) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (x >= total) return;
  const int b = (int)(x / M), i = (int)(x % M);
  if (i >= ld_int(n + b)) return;
  const int t = ld_int(tokens + x);
  if (t < 0 || t >= V) {
    if (status) atomicOr(status, (int)SD_STATUS_BAD_TOKEN);
    return;
  }
  // a 16-bit exchange: a row of an odd vocabulary shares words with its neighbours
  unsigned short *p = reinterpret_cast<unsigned short *>(counts + (int64_t)b * V + t);
  unsigned short old = *p, seen;
  do {
    if ((old & 0x7fffu) == 0x7fffu) break;
    seen = old;
    old = atomicCAS(p, seen, (unsigned short)(seen + 1));
  } while (old != seen);
}

// 512 threads, three CTAs per SM; 1024 where there is one at most (a long
// history is then read with twice the loads in flight).
template <int NT>
static cudaError_t launch_counts(int L, int V, int slice, int grid, const int32_t *history,
                                 const int32_t *lengths, const int32_t *prompt_lengths,
                                 uint16_t *counts, int32_t *status, cudaStream_t s) {
  static FuncAttrs attrs;
  attrs.apply((const void *)sd_token_counts_kernel<NT>, 2 * kCntSlice, false, "the count kernel");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.dynamicSmemBytes = (size_t)2 * slice;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sd_token_counts_kernel<NT>, L, V, (V + slice - 1) / slice, slice,
                            history, lengths, prompt_lengths, counts, status);
}

}  // namespace sdv

using namespace sdv;

extern "C" sd_status_t sd_token_counts(int32_t B, int32_t L, int32_t V, const int32_t *history,
                                       const int32_t *lengths, const int32_t *prompt_lengths,
                                       uint16_t *counts, int32_t *status, void *stream) {
  sdv::NvtxRange nvtx_range("sd_token_counts");
  if (B < 0 || L < 0 || V < 1 || V > SD_MAX_V) return SD_ERR_INVALID_ARG;
  if (B == 0) return SD_OK;
  if ((L > 0 && !history) || !lengths || !counts || ((uintptr_t)counts & 1))
    return SD_ERR_INVALID_ARG;
  // few sequences: more and smaller slices, up to one CTA per SM
  const int few = std::min((V + kCntLeast - 1) / kCntLeast, sm_count() / B);
  const int nslice = std::max((V + kCntSlice - 1) / kCntSlice, few);
  const int slice = ((V + nslice - 1) / nslice + 7) & ~7;
  const int64_t grid = (int64_t)B * ((V + slice - 1) / slice);
  if (grid > INT32_MAX) return SD_ERR_INVALID_ARG;
  const cudaError_t e =
      grid <= sm_count()
          ? launch_counts<1024>(L, V, slice, (int)grid, history, lengths, prompt_lengths, counts,
                                status, (cudaStream_t)stream)
          : launch_counts<512>(L, V, slice, (int)grid, history, lengths, prompt_lengths, counts,
                               status, (cudaStream_t)stream);
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}

extern "C" sd_status_t sd_token_counts_add(int32_t B, int32_t M, int32_t V, const int32_t *tokens,
                                           const int32_t *n, uint16_t *counts, int32_t *status,
                                           void *stream) {
  sdv::NvtxRange nvtx_range("sd_token_counts_add");
  if (B < 0 || M < 0 || V < 1 || V > SD_MAX_V) return SD_ERR_INVALID_ARG;
  if (B == 0 || M == 0) return SD_OK;
  if (!tokens || !n || !counts || ((uintptr_t)counts & 1)) return SD_ERR_INVALID_ARG;
  const int64_t total = (int64_t)B * M;
  if ((total + 255) / 256 > INT32_MAX) return SD_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((total + 255) / 256), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sd_token_counts_add_kernel, (int)M, (int)V,
                                           tokens, n, counts, status, total);
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}
