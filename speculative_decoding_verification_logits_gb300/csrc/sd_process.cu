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
// as it was.  A CTA takes NT vectors' worth of vocabulary (a window) through
// all R rows of one sequence, in two parts:
//  A. rows are copied as raw words with -inf put where the mask forbids the
//     token; logits that are forbidden all through a vector are not read;
//  B. the window's touched tokens (a count, a draft or a bias) are listed
//     once, from a bit per token, and each (row, listed token) is one thread's
//     work: read the logit again (from L2), compute, write over it.
// Computing touched logits where A meets them is what this replaces: nearly
// every warp then holds a touched one and runs the whole computation for a
// lane or two (64 x 9 x 151936 bf16, masked: 471 us against 81).
// Measured on the GPU, with histories that touch most low ids: that case 81 us
// (66 for part A alone; its bytes alone take 56), 256 x 5 x 128256 bf16 without
// a mask 130 us (99 for part A; 106 of bytes at the copy rate).  Part B is what
// is left above the copy: its instructions, not its bytes (L2 holds them).  A
// single row of 32000 float32: 6 us, nearly all of it part B's chain of
// barriers and dependent loads (2 us without it).

#include "sd_rows.cuh"

#include <type_traits>

namespace sdv {

constexpr int kProcNT = 256;
constexpr int kProcU = 3;   // rows in flight per thread
constexpr int kProcCtas = 6;   // per SM
// part B doubles its groups of threads until one holds the listed tokens or is
// the block (a group larger than the block would have a loop over rows without
// end), the threads share the bias list out evenly, and one warp holds the drafts
static_assert((kProcNT & (kProcNT - 1)) == 0 && kProcNT % 32 == 0, "threads: a power of two");
static_assert(SD_MAX_BIAS % kProcNT == 0 && SD_MAX_K <= 32, "lists as the threads take them");

struct ProcParams {
  sd_process_args a;
  int inplace;
  int rows;   // of a sequence, per CTA
};

// Bits e0 .. e0 + VE - 1 of a bit row (word 0 holds bit 0; e0 may be negative
// by less than VE, where the bits come back as zero), at most W words.
template <int VE>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *w, int e0, int W) {
  if (e0 < 0) return (ld4(w) << -e0) & ((1u << VE) - 1u);
  const int i = e0 >> 5, s = e0 & 31;
  uint32_t r = ld4(w + i) >> s;
  if (s + VE > 32 && i + 1 < W) r |= ld4(w + i + 1) << (32 - s);
  return r & ((1u << VE) - 1u);
}

// VEC: rows move as 16-byte vectors (the output's rows lie on the same place
// of the 16-byte grid as the input's); otherwise element by element.
template <typename E, bool VEC>
__global__ void __launch_bounds__(kProcNT, kProcCtas) sd_process_kernel(const ProcParams P) {
  constexpr int VE = VEC ? Elt<E>::kPerVec : 1, NT = kProcNT, NW = NT / 32;
  constexpr int SZ = Elt<E>::kSize;
  constexpr uint32_t kAll = (1u << VE) - 1u;
  constexpr int kOwn = NT * VE;                    // tokens of a row in this CTA
  // vectors of eight counts that the window (kOwn tokens, VE - 1 more before
  // them for rows off the grid) can meet, and the tokens they hold
  constexpr int kCntVec = (kOwn + VE + 7) / 8 + 1, kWin = kCntVec * 8;
  constexpr int kCntPer = (kCntVec + NT - 1) / NT;
  constexpr int kWords = (kWin + 31) / 32;
  constexpr int kBiasPer = SD_MAX_BIAS / NT;       // list entries per thread
  const sd_process_args &a = P.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint16_t hot[kWin];                       // touched tokens of the window
  __shared__ __align__(16) uint16_t count[kWin];       // the window's counts
  __shared__ float bias[kWin];                         // sum of each token's biases
  __shared__ uint32_t touch[kWords];                   // a bit per token
  __shared__ int prev_i[SD_MAX_K], prev_v[SD_MAX_K];   // drafts inside the window, in order
  __shared__ int bias_v[SD_MAX_BIAS];                  // biases inside the window, in order
  __shared__ float bias_x[SD_MAX_BIAS];
  __shared__ int bias_n[kBiasPer][NW];
  __shared__ int n_prev, n_hot;
  // windows of low ids first: texts have most of their tokens there, so these
  // CTAs' part B is the longest
  const int b = blockIdx.x % a.B, q0 = (blockIdx.x / a.B) * NT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = a.V, r_lo = blockIdx.y * P.rows, R = min(P.rows, a.R - r_lo);
  const int base = a.base + r_lo;   // drafts before this CTA's first row
  const float rep = a.repetition ? ld_float(a.repetition + b) : 1.f;
  const float pres = a.presence ? ld_float(a.presence + b) : 0.f;
  const float freq = a.frequency ? ld_float(a.frequency + b) : 0.f;
  const bool bad = !(rep > 0.f && rep < INFINITY) || !(fabsf(pres) < INFINITY) ||
                   !(fabsf(freq) < INFINITY);
  const int n_draft = a.prev ? base + R - 1 : 0;
  const bool touches = a.counts || n_draft > 0 || a.n_bias > 0;   // part B has work at all

  // the window's counts, this round's drafts and the biases are asked for
  // first and arrive during part A.  Counts come as vectors of their own
  // 16-byte grid; the window's token 0 is the first one of count vector k0.
  const uint16_t *cb = a.counts + (int64_t)b * V;
  const int hpc = a.counts ? (int)((uintptr_t)cb & 15) / 2 : 0;
  const int k0 = (max(q0 * VE - (VE - 1), 0) + hpc) / 8;
  const int w0 = k0 * 8 - hpc;
  uint4 c[kCntPer];
  if (a.counts) {
#pragma unroll
    for (int i = 0; i < kCntPer; ++i) {
      const int k = i * NT + tid, v = w0 + k * 8;
      c[i] = make_uint4(0u, 0u, 0u, 0u);
      if (k >= kCntVec) continue;
      if (v >= 0 && v + 8 <= V) {
        c[i] = ld16(cb + v);
      } else {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = v + e >= 0 && v + e < V ? ld2(cb + v + e) : 0u;
        c[i] = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                          h[6] | (h[7] << 16));
      }
    }
  }
  int draft = -1;
  if (warp == 0 && lane < n_draft) draft = ld_int(a.prev + (int64_t)b * a.P + lane);
  int bid[kBiasPer];
  if (a.n_bias > 0) {
#pragma unroll
    for (int j = 0; j < kBiasPer; ++j) {
      const int i = j * NT + tid;
      bid[j] = i < a.n_bias ? ld_int(a.bias_ids + (int64_t)b * a.n_bias + i) : -1;
    }
  }

  // A. copy and mask this thread's vector of every row
  const int W = (V + 31) >> 5, q = q0 + tid;
  const uint8_t *xb = (const uint8_t *)a.logits + (b * a.logits_sb + r_lo * a.logits_sr) * SZ;
  uint8_t *yb = (uint8_t *)a.out + (b * a.out_sb + r_lo * a.out_sr) * SZ;
  const uint32_t *mb = (const uint32_t *)a.mask + b * a.mask_sb + r_lo * a.mask_sr;
  const int64_t xs = a.logits_sr * SZ, ys = a.out_sr * SZ;
  // INNER: this CTA's vectors lie inside the row whatever its place on the
  // grid; its loop is kept apart from the one with the rows' ends
  auto copy = [&](auto INNER) {
    constexpr bool inner = decltype(INNER)::value;
    // the row at x: its first element in this thread's vector, and which of
    // the vector's places lie in the row
    auto first = [&](const uint8_t *x) {
      return q * VE - (VEC ? (int)((uintptr_t)x & 15) / SZ : 0);
    };
    auto inside = [&](int e0) -> uint32_t {
      uint32_t in = kAll;
      if (inner) return in;
      if (e0 >= V) return 0u;
      if (e0 < 0) in = (kAll << -e0) & kAll;
      if (e0 + VE > V) in &= (1u << (V - e0)) - 1u;
      return in;
    };
    const uint8_t *x = xb;          // row r0
    uint8_t *y = yb;
    const uint32_t *m = mb;         // row r0, then of the rows whose bits are asked for
    uint32_t next[kProcU];          // allowed places of the next rows
    auto ask = [&](const uint8_t *row, int n) {   // of the n rows from `row` and m on
#pragma unroll
      for (int u = 0; u < kProcU; ++u) {
        next[u] = 0u;
        if (u < n) {
          const int e0 = first(row + u * xs);
          next[u] = inside(e0);
          if (a.mask && next[u]) next[u] &= mask_bits<VE>(m + u * a.mask_sr, e0, W);
        }
      }
    };
    ask(x, R);
    for (int left = R; left > 0; left -= kProcU) {
      uint4 xv[kProcU];
      uint32_t ok[kProcU];
#pragma unroll
      for (int u = 0; u < kProcU; ++u) {
        ok[u] = next[u];
        xv[u] = make_uint4(0u, 0u, 0u, 0u);
        if (u < left && ok[u] && !bad) {
          const uint8_t *row = x + u * xs;
          const int e0 = first(row);
          const uint32_t in = inside(e0);
          if (P.inplace && ok[u] == in) continue;
          if (VEC && in == kAll) {
            xv[u] = ld16(row + (int64_t)e0 * SZ);
          } else {
            float f[Elt<E>::kPerVec] = {};
#pragma unroll
            for (int e = 0; e < VE; ++e)
              if ((ok[u] >> e) & 1u) f[e] = Row<E>::load(row, e0 + e);
            Row<E>::pack(f, xv[u]);
          }
        }
      }
      // the mask of the rows after these, so that their loads need not wait for it
      m += kProcU * a.mask_sr;
      ask(x + kProcU * xs, left - kProcU);
#pragma unroll
      for (int u = 0; u < kProcU; ++u) {
        if (u >= left) continue;
        const int e0 = first(x + u * xs);
        const uint32_t in = inside(e0);
        if (in == 0u || (P.inplace && ok[u] == in && !bad)) continue;
        uint4 v = ok[u] == kAll ? xv[u] : mask_vec<E>(xv[u], ok[u]);
        if (bad) {
          const uint32_t nan = SZ == 2 ? 0x7fc07fc0u : 0x7fc00000u;
          v = make_uint4(nan, nan, nan, nan);
        }
        uint8_t *row = y + u * ys;
        if (VEC && in == kAll) {
          *reinterpret_cast<uint4 *>(row + (int64_t)e0 * SZ) = v;
        } else {
          float f[Elt<E>::kPerVec];
          Elt<E>::unpack(v, f);
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if ((in >> e) & 1u) Row<E>::store(row, e0 + e, f[e]);
        }
      }
      x += kProcU * xs;
      y += kProcU * ys;
    }
  };
  if (q0 > 0 && (q0 + NT) * VE <= V)
    copy(std::true_type());
  else
    copy(std::false_type());
  if (bad && tid == 0 && q0 == 0 && a.status) atomicOr(a.status, (int)SD_STATUS_BAD_PENALTY);
  if (!touches) return;

  // B. which tokens of the window are touched
  bool bad_id = false;
#pragma unroll
  for (int i = 0; i < kCntPer; ++i) {
    const int k = i * NT + tid;
    if (k >= kCntVec) continue;
    uint32_t m = 0u;
    if (a.counts) {
      const uint32_t h[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m |= ((h[e] & 0xffffu ? 1u : 0u) | (h[e] >> 16 ? 2u : 0u)) << (2 * e);
      reinterpret_cast<uint4 *>(count)[k] = c[i];
    }
    reinterpret_cast<uint8_t *>(touch)[k] = (uint8_t)m;
  }
  if (tid < kWords * 4 - kCntVec) reinterpret_cast<uint8_t *>(touch)[kCntVec + tid] = 0u;
  if (warp == 0) {
    bad_id = lane < n_draft && (draft < 0 || draft >= V);
    const bool in = lane < n_draft && !bad_id && draft >= w0 && draft < w0 + kWin;
    const unsigned m = ballot(in);
    if (in) {
      const int at = __popc(m & ((1u << lane) - 1u));
      prev_i[at] = lane;
      prev_v[at] = draft;
    }
    if (lane == 0) {
      n_prev = __popc(m);
      n_hot = 0;
    }
  }
  unsigned bhit[kBiasPer];
  if (a.n_bias > 0) {
    for (int j = tid; j < kWin; j += NT) bias[j] = 0.f;
#pragma unroll
    for (int j = 0; j < kBiasPer; ++j) {
      bad_id |= bid[j] < -1 || bid[j] >= V;
      const bool in = bid[j] >= 0 && bid[j] < V && bid[j] >= w0 && bid[j] < w0 + kWin;
      bhit[j] = ballot(in);
      if (!in) bid[j] = -1;
      if (lane == 0) bias_n[j][warp] = __popc(bhit[j]);
    }
  }
  if (bad_id && q0 == 0 && a.status) atomicOr(a.status, (int)SD_STATUS_BAD_TOKEN);
  if (bad) return;   // the same for every CTA of the sequence: its rows are NaN
  __syncthreads();   // also: part A's stores come before part B's to the same places
  if (tid < n_prev) atomicOr(&touch[(prev_v[tid] - w0) >> 5], 1u << ((prev_v[tid] - w0) & 31));
  if (a.n_bias > 0) {
    int n = 0, at[kBiasPer];
#pragma unroll
    for (int j = 0; j < kBiasPer; ++j)
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w == warp) at[j] = n;
        n += bias_n[j][w];
      }
#pragma unroll
    for (int j = 0; j < kBiasPer; ++j)
      if (bid[j] >= 0) {
        const int k = at[j] + __popc(bhit[j] & ((1u << lane) - 1u));
        bias_v[k] = bid[j] - w0;
        bias_x[k] = ld_float(a.bias_vals + (int64_t)b * a.n_bias + j * NT + tid);
        atomicOr(&touch[(bid[j] - w0) >> 5], 1u << ((bid[j] - w0) & 31));
      }
    __syncthreads();
    // a token's biases are summed in list order by the thread of its first one
    for (int k = tid; k < n; k += NT) {
      const int v = bias_v[k];
      int one = k;
      for (int o = 0; o < k && one == k; ++o)
        if (bias_v[o] == v) one = o;
      if (one != k) continue;
      float s = bias_x[k];
      for (int o = k + 1; o < n; ++o)
        if (bias_v[o] == v) s += bias_x[o];
      bias[v] = s;
    }
  }
  __syncthreads();
  for (int w = tid; w < (kWords + 31) / 32 * 32; w += NT) {
    const uint32_t m = w < kWords ? touch[w] : 0u;
    const int n = __popc(m);
    int scan = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, o);
      scan += lane >= o ? y : 0;
    }
    int at = 0;
    if (lane == 31) at = atomicAdd(&n_hot, scan);
    at = __shfl_sync(0xffffffffu, at, 31) + scan - n;
    for (uint32_t left = m; left; left &= left - 1u) hot[at++] = (uint16_t)(w * 32 + __ffs(left) - 1);
  }
  __syncthreads();
  // tpt threads side by side take the listed tokens, NT / tpt such groups the
  // rows; a thread has kProcU rows of its token in flight
  int tpt = 1;
  while (tpt < NT && tpt < n_hot) tpt *= 2;
  const int groups = NT / tpt, r0 = tid / tpt;
  for (int h = tid & (tpt - 1); h < n_hot; h += tpt) {
    const int j = hot[h], v = w0 + j;
    const uint32_t word = a.counts ? count[j] : 0u;
    const int n0 = (int)(word & 0x7fffu);
    const float add = a.n_bias > 0 ? bias[j] : 0.f;
    uint32_t drafts = 0u;   // the drafts that equal the token
    for (int k = 0; k < n_prev; ++k) drafts |= prev_v[k] == v ? 1u << prev_i[k] : 0u;
    for (int r = r0; r < R; r += groups * kProcU) {
      float f[kProcU];
#pragma unroll
      for (int u = 0; u < kProcU; ++u) {
        const int row = r + u * groups;
        f[u] = neg_inf();
        if (row >= R) continue;
        const uint8_t *x = xb + row * xs;
        // a row off the grid leaves up to VE - 1 of the window to a neighbour
        const int lo = q0 * VE - (VEC ? (int)((uintptr_t)x & 15) / SZ : 0);
        if (v < lo || v >= lo + kOwn) continue;
        f[u] = Row<E>::load(x, v);
        if (a.mask && !((ld4(mb + row * a.mask_sr + (v >> 5)) >> (v & 31)) & 1u)) f[u] = neg_inf();
      }
#pragma unroll
      for (int u = 0; u < kProcU; ++u) {
        const int row = r + u * groups;
        float x = f[u];
        if (x == neg_inf()) continue;   // not this CTA's, forbidden, or as it was
        const int before = base + row;
        const int n = n0 + __popc(before >= 32 ? drafts : drafts & ((1u << before) - 1u));
        if (n > 0 || (word & 0x8000u)) x = x > 0.f ? x / rep : x * rep;
        if (n > 0) x = x - freq * (float)n - pres;
        if (a.n_bias > 0) x += add;
        Row<E>::store(yb + row * ys, v, x);
      }
    }
  }
}

template <typename E, bool VEC>
static cudaError_t launch_process(ProcParams &P, cudaStream_t s) {
  constexpr int VE = VEC ? Elt<E>::kPerVec : 1;
  // vectors of a row that starts anywhere on the 16-byte grid
  const int64_t nvec = ((int64_t)P.a.V + 2 * VE - 2) / VE;
  const int64_t grid = (nvec + kProcNT - 1) / kProcNT * P.a.B;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  // where the windows leave SMs idle, several CTAs share a window's rows, up
  // to two waves of them (13 x 7 rows of 50021, tight mask, 300 biases: 19.1 us
  // without, 16.1 with one wave, 14.4 with two, 22.6 with three)
  const int64_t parts = std::min<int64_t>((P.a.R + kProcU - 1) / kProcU,
                                          std::max<int64_t>(2 * kProcCtas * sm_count() / grid, 1));
  P.rows = (int)((P.a.R + parts - 1) / parts);
  cfg.gridDim = dim3((unsigned)grid, (unsigned)((P.a.R + P.rows - 1) / P.rows), 1);
  cfg.blockDim = dim3(kProcNT, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sd_process_kernel<E, VEC>, P);
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
