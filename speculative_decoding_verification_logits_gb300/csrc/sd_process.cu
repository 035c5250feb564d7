// Penalties for repeated tokens, biases and a grammar's mask on logits, for
// the rows of a verify round (or a single token's row): the step between the
// model and the verify.
//
// Per logit: c = count + drafts of the round before this row that equal the
// token; seen = c > 0 or in the prompt;
//   y = (seen ? (x > 0 ? x / rep : x rep) : x) - freq c - pres [c > 0] + bias
// or -inf where the mask forbids the token.  fp32, rounded once.
//
// The work is moving memory: a logit is read, written and in most places left
// as it was.  A CTA takes the same NT vectors' worth of vocabulary through
// all R rows of one sequence, so that the counts are read once for all of
// them.  It first makes a bit per token of its window that a count, a draft
// or a bias touches; a vector without a bit is passed on as raw words.
// Logits that the mask forbids are not read.

#include "sd_rows.cuh"

namespace sdv {

constexpr int kProcNT = 256;
constexpr int kProcU = 4;   // rows in flight per thread

struct ProcParams {
  sd_process_args a;
  int nslice;
  int inplace;
};

// Bits e0 .. e0 + VE - 1 of a bit row (word 0 holds bit 0; e0 may be negative
// by less than VE, where the bits come back as zero), at most W words.
template <int VE>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *w, int e0, int W) {
  if (e0 < 0) return (__ldg(w) << -e0) & ((1u << VE) - 1u);
  const int i = e0 >> 5, s = e0 & 31;
  uint32_t r = __ldg(w + i) >> s;
  if (s + VE > 32 && i + 1 < W) r |= __ldg(w + i + 1) << (32 - s);
  return r & ((1u << VE) - 1u);
}

// VEC: rows move as 16-byte vectors (the output's rows lie on the same place
// of the 16-byte grid as the input's); otherwise element by element.
template <typename E, bool VEC>
__global__ void __launch_bounds__(kProcNT) sd_process_kernel(const ProcParams P) {
  constexpr int VE = VEC ? Elt<E>::kPerVec : 1, NT = kProcNT, NW = NT / 32;
  constexpr int SZ = Elt<E>::kSize;
  constexpr int kWin = NT * VE + VE;              // tokens of the window
  constexpr int kBiasPer = SD_MAX_BIAS / NT;      // list entries per thread
  const sd_process_args &a = P.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint16_t cnt[kWin];
  __shared__ uint32_t touch[(kWin + 31) / 32 + 1];
  __shared__ int prev_i[SD_MAX_K], prev_v[SD_MAX_K];   // drafts inside the window, in order
  __shared__ int bias_v[SD_MAX_BIAS];                  // biases inside the window, in order
  __shared__ float bias_x[SD_MAX_BIAS];
  __shared__ int bias_n[kBiasPer][NW];
  __shared__ int n_prev;
  const int b = blockIdx.x / P.nslice, q0 = (blockIdx.x % P.nslice) * NT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = a.V, R = a.R, w0 = q0 * VE - VE;   // first token of the window
  const float rep = a.repetition ? __ldg(a.repetition + b) : 1.f;
  const float pres = a.presence ? __ldg(a.presence + b) : 0.f;
  const float freq = a.frequency ? __ldg(a.frequency + b) : 0.f;
  const bool bad = !(rep > 0.f && rep < INFINITY) || !(fabsf(pres) < INFINITY) ||
                   !(fabsf(freq) < INFINITY);
  // counts of the window, and the tokens they touch
  if (tid == 0) touch[(kWin + 31) / 32] = 0u;
#pragma unroll
  for (int j = tid; j < (kWin + 31) / 32 * 32; j += NT) {
    const int v = w0 + j;
    uint32_t c = 0u;
    if (a.counts && j < kWin && v >= 0 && v < V) c = __ldg(a.counts + (int64_t)b * V + v);
    if (j < kWin) cnt[j] = (uint16_t)c;
    const unsigned m = __ballot_sync(0xffffffffu, c != 0u);
    if (lane == 0) touch[j >> 5] = m;
  }
  // this round's drafts and the biases that fall into the window, in list order
  bool bad_id = false;
  if (warp == 0) {
    int v = -1;
    if (a.prev && lane < a.base + R - 1) {
      v = __ldg(a.prev + (int64_t)b * a.P + lane);
      bad_id = v < 0 || v >= V;
    }
    const bool in = !bad_id && v >= 0 && v >= w0 && v < w0 + kWin;
    const unsigned m = ballot(in);
    if (in) {
      const int at = __popc(m & ((1u << lane) - 1u));
      prev_i[at] = lane;
      prev_v[at] = v;
    }
    if (lane == 0) n_prev = __popc(m);
  }
  int bid[kBiasPer];
  unsigned bhit[kBiasPer];
  if (a.n_bias > 0) {
#pragma unroll
    for (int j = 0; j < kBiasPer; ++j) {
      const int i = j * NT + tid;
      bid[j] = i < a.n_bias ? __ldg(a.bias_ids + (int64_t)b * a.n_bias + i) : -1;
    }
#pragma unroll
    for (int j = 0; j < kBiasPer; ++j) {
      bad_id |= bid[j] < -1 || bid[j] >= V;
      const bool in = bid[j] >= 0 && bid[j] < V && bid[j] >= w0 && bid[j] < w0 + kWin;
      bhit[j] = ballot(in);
      if (!in) bid[j] = -1;
      if (lane == 0) bias_n[j][warp] = __popc(bhit[j]);
    }
  }
  __syncthreads();
  int n_bias = 0;
  if (a.n_bias > 0) {
    int at[kBiasPer];
#pragma unroll
    for (int j = 0; j < kBiasPer; ++j)
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w == warp) at[j] = n_bias;
        n_bias += bias_n[j][w];
      }
#pragma unroll
    for (int j = 0; j < kBiasPer; ++j)
      if (bid[j] >= 0) {
        const int k = at[j] + __popc(bhit[j] & ((1u << lane) - 1u));
        bias_v[k] = bid[j];
        bias_x[k] = __ldg(a.bias_vals + (int64_t)b * a.n_bias + j * NT + tid);
        atomicOr(&touch[(bid[j] - w0) >> 5], 1u << ((bid[j] - w0) & 31));
      }
  }
  if (tid < n_prev) atomicOr(&touch[(prev_v[tid] - w0) >> 5], 1u << ((prev_v[tid] - w0) & 31));
  __syncthreads();
  if (a.status && q0 == 0) {
    if (bad && tid == 0) atomicOr(a.status, (int)SD_STATUS_BAD_PENALTY);
    if (bad_id) atomicOr(a.status, (int)SD_STATUS_BAD_TOKEN);
  }

  const int W = (V + 31) >> 5, q = q0 + tid;
  const uint8_t *xb = (const uint8_t *)a.logits + b * a.logits_sb * SZ;
  uint8_t *yb = (uint8_t *)a.out + b * a.out_sb * SZ;
  for (int r0 = 0; r0 < R; r0 += kProcU) {
    uint4 xv[kProcU];
    int e0[kProcU];
    uint32_t ok[kProcU], valid[kProcU];
#pragma unroll
    for (int u = 0; u < kProcU; ++u) {
      const int r = r0 + u;
      valid[u] = 0u;
      if (r >= R) continue;
      const uint8_t *x = xb + r * a.logits_sr * SZ;
      e0[u] = q * VE - (VEC ? (int)((uintptr_t)x & 15) / SZ : 0);
      uint32_t in = (1u << VE) - 1u;
      if (e0[u] < 0) in &= in << -e0[u];
      if (e0[u] >= V) in = 0u;
      else if (e0[u] + VE > V) in &= (1u << (V - e0[u])) - 1u;
      valid[u] = in;
      ok[u] = in;
      if (a.mask && in)
        ok[u] &= mask_bits<VE>((const uint32_t *)a.mask + b * a.mask_sb + r * a.mask_sr, e0[u], W);
    }
#pragma unroll
    for (int u = 0; u < kProcU; ++u) {
      if (!valid[u] || !ok[u]) continue;
      const uint8_t *x = xb + (r0 + u) * a.logits_sr * SZ;
      if (VEC && valid[u] == (1u << VE) - 1u) {
        xv[u] = __ldcg(reinterpret_cast<const uint4 *>(x + (int64_t)e0[u] * SZ));
      } else {
        float f[Elt<E>::kPerVec] = {};
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if ((valid[u] >> i) & 1u) f[i] = Row<E>::load(x, e0[u] + i);
        Row<E>::pack(f, xv[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kProcU; ++u) {
      if (!valid[u]) continue;
      const int r = r0 + u;
      const int j0 = e0[u] - w0;
      uint32_t hot = touch[j0 >> 5] >> (j0 & 31);
      if ((j0 & 31) + VE > 32) hot |= touch[(j0 >> 5) + 1] << (32 - (j0 & 31));
      hot &= ok[u];
      if (P.inplace && ok[u] == valid[u] && !hot && !bad) continue;
      float f[Elt<E>::kPerVec];
      if (ok[u]) {
        Elt<E>::unpack(xv[u], f);
      } else {
#pragma unroll
        for (int i = 0; i < Elt<E>::kPerVec; ++i) f[i] = neg_inf();
      }
      if (hot) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          if (!((hot >> i) & 1u) || f[i] == neg_inf()) continue;
          const int v = e0[u] + i;
          const uint32_t word = cnt[j0 + i];
          int c = (int)(word & 0x7fffu);
          for (int k = 0; k < n_prev; ++k) c += prev_v[k] == v && prev_i[k] < a.base + r;
          float x = f[i];
          if (c > 0 || (word & 0x8000u)) x = x > 0.f ? x / rep : x * rep;
          if (c > 0) x = x - freq * (float)c - pres;
          for (int k = 0; k < n_bias; ++k)
            if (bias_v[k] == v) x += bias_x[k];
          f[i] = x;
        }
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        if (!((ok[u] >> i) & 1u)) f[i] = neg_inf();
        if (bad) f[i] = __int_as_float(0x7fc00000);
      }
      uint8_t *y = yb + r * a.out_sr * SZ;
      if (VEC && valid[u] == (1u << VE) - 1u) {
        uint4 v;
        Row<E>::pack(f, v);
        *reinterpret_cast<uint4 *>(y + (int64_t)e0[u] * SZ) = v;
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if ((valid[u] >> i) & 1u) Row<E>::store(y, e0[u] + i, f[i]);
      }
    }
  }
}

template <typename E, bool VEC>
static cudaError_t launch_process(ProcParams &P, cudaStream_t s) {
  constexpr int VE = VEC ? Elt<E>::kPerVec : 1;
  // vectors of a row that starts anywhere on the 16-byte grid
  const int64_t nvec = ((int64_t)P.a.V + 2 * VE - 2) / VE;
  P.nslice = (int)((nvec + kProcNT - 1) / kProcNT);
  if ((int64_t)P.a.B * P.nslice > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.a.B * P.nslice), 1, 1);
  cfg.blockDim = dim3(kProcNT, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sd_process_kernel<E, VEC>, (const ProcParams)P);
}

}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_process_args_size(void) { return sizeof(sd_process_args); }

extern "C" sd_status_t sd_process_logits(const sd_process_args *args, void *stream) {
  sdv::NvtxRange nvtx_range("sd_process_logits");
  if (!args) return SD_ERR_INVALID_ARG;
  ProcParams P;
  memset(&P, 0, sizeof(P));
  P.a = *args;
  sd_process_args &a = P.a;
  if (a.B < 0 || a.R < 0 || a.V < 1 || a.V > SD_MAX_V) return SD_ERR_INVALID_ARG;
  if (a.dtype != SD_F32 && a.dtype != SD_BF16) return SD_ERR_INVALID_ARG;
  if (a.n_bias < 0 || a.n_bias > SD_MAX_BIAS || (a.n_bias > 0 && (!a.bias_ids || !a.bias_vals)))
    return SD_ERR_INVALID_ARG;
  if (a.base < 0) return SD_ERR_INVALID_ARG;
  if (a.B == 0 || a.R == 0) return SD_OK;
  if (a.prev && (a.P > SD_MAX_K || a.base > SD_MAX_K || (int64_t)a.base + a.R - 1 > a.P))
    return SD_ERR_INVALID_ARG;
  if (!a.logits || !a.out) return SD_ERR_INVALID_ARG;
  const size_t es = a.dtype == SD_BF16 ? 2 : 4;
  if ((uintptr_t)a.logits % es || (uintptr_t)a.out % es || (uintptr_t)a.counts % 2 ||
      (uintptr_t)a.mask % 4)
    return SD_ERR_INVALID_ARG;
  // rows of the output that share places cannot be written
  if ((a.R > 1 && a.out_sr < a.V) || (a.B > 1 && a.out_sb < a.V)) return SD_ERR_INVALID_ARG;
  if (a.R > 1 && a.B > 1 && a.out_sb < (a.R - 1) * a.out_sr + a.V &&
      a.out_sr < (a.B - 1) * a.out_sb + a.V)
    return SD_ERR_INVALID_ARG;
  P.inplace = a.logits == a.out && (a.R <= 1 || a.logits_sr == a.out_sr) &&
              (a.B <= 1 || a.logits_sb == a.out_sb);
  // 16-byte vectors where every row of the output lies as its row of the input does
  const bool vec = (((uintptr_t)a.logits ^ (uintptr_t)a.out) & 15) == 0 &&
                   ((uint64_t)(a.logits_sb - a.out_sb) * es % 16 == 0 || a.B <= 1) &&
                   ((uint64_t)(a.logits_sr - a.out_sr) * es % 16 == 0 || a.R <= 1);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (a.dtype == SD_BF16)
    e = vec ? launch_process<__nv_bfloat16, true>(P, s) : launch_process<__nv_bfloat16, false>(P, s);
  else
    e = vec ? launch_process<float, true>(P, s) : launch_process<float, false>(P, s);
  return e == cudaSuccess ? SD_OK : e == cudaErrorInvalidValue ? SD_ERR_INVALID_ARG : SD_ERR_CUDA;
}
