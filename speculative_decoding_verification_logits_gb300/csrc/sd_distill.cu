// Distillation of the drafter from a teacher's top logits: the loss over the
// k named tokens and one bucket for all others, and its gradient with
// respect to the student's logits.
//
// With p the teacher's shares, q the student's softmax (both over k + 1
// buckets and summing to one) and d = ln(p / q):
//   loss = sum p d = sum [p d - p + q] = sum p h(d),  h(d) = d - 1 + exp(-d).
// The second form is used: its terms are not negative, so nothing cancels
// where the student is near the teacher (h by its series for |d| < 1/2), and
// an error in a normalisation, the same for every d, drops out to first
// order.  The student's share of the others is summed without the named
// tokens (never as 1 - sum q_i), so it keeps its relative precision however
// small it is.
// Gradient: named w/T (q - p) = w/T q (1 - e^d); others w/T (q_r - p_r) e_j / Z_r
// with e_j / Z_r the softmax among the others.
//
// One cluster of cs CTAs per row, each CTA a contiguous share of the row's
// vectors.  Pass 1: running maximum and sum of the others in one read (the
// named tokens' places are bits in shared memory).  The cluster exchanges
// (offset, sum) and every CTA works out the k + 1 buckets.  Pass 2 reads the
// share again (from L2) and writes the gradient; the named places are
// written over last.  HBM-bound: 2 or 4 bytes per logit for the loss, twice
// that with the gradient.

#include "sd_rows.cuh"

namespace sdv {

constexpr int kDistNT = 512;
constexpr int kDistNW = kDistNT / 32;
constexpr int kDistU = 4;         // vectors in flight per thread
constexpr int kDistMaxCS = 8;

struct DistParams {
  sd_distill_args a;
  int cs;
  int bit_words;   // shared-memory words of the named bits
};

// The sum of 2^(x c2 - o) over a share of the others; o = max x c2.
struct DistStat {
  float o, z;
  int bad;
};

__device__ __forceinline__ void dist_merge(float &o, float &z, float o2, float z2) {
  const float m = fmaxf(o, o2);
  const float s = m == neg_inf() ? 0.f : m;   // an empty share leaves its zero sum as it is
  z = z * ex2(o - s) + z2 * ex2(o2 - s);
  o = m;
}

// d - 1 + exp(-d), without cancellation for small d
__device__ __forceinline__ float dist_h(float d) {
  float s = fmaf(d, -1.f / 40320.f, 1.f / 5040.f);
  s = fmaf(-d, s, 1.f / 720.f);
  s = fmaf(-d, s, 1.f / 120.f);
  s = fmaf(-d, s, 1.f / 24.f);
  s = fmaf(-d, s, 1.f / 6.f);
  s = fmaf(-d, s, 0.5f);
  return d * d * s;
}
// p d - p + q for d = ln(p / q)
__device__ __forceinline__ float dist_term(float p, float q, float d) {
  if (p == 0.f) return q;
  return fabsf(d) < 0.5f ? p * dist_h(d) : fmaf(p, d, q - p);
}

template <int NW>
__device__ __forceinline__ float block_sum(float x, float *red) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += red[w];
  __syncthreads();
  return s;
}
template <int NW>
__device__ __forceinline__ float block_max(float x, float *red) {
  x = warp_max(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = neg_inf();
#pragma unroll
  for (int w = 0; w < NW; ++w) s = fmaxf(s, red[w]);
  __syncthreads();
  return s;
}

template <typename E>
__device__ __forceinline__ void store_vec(const RowView<E> &row, int q, const float *f) {
  constexpr int VE = Elt<E>::kPerVec;
  const int e0 = row.first(q);
  uint8_t *y = const_cast<uint8_t *>(row.row);
  if (row.whole(q)) {
    uint4 v;
    Row<E>::pack(f, v);
    *reinterpret_cast<uint4 *>(y + (int64_t)e0 * Elt<E>::kSize) = v;
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (e0 + i >= 0 && e0 + i < row.n) Row<E>::store(y, e0 + i, f[i]);
  }
}

// GRAD: write the gradient; SAME: its rows lie on the 16-byte grid as the
// student's do (whole vectors), otherwise they are written element by element.
template <typename E, bool GRAD, bool SAME>
__global__ void __launch_bounds__(kDistNT, 2) sd_distill_kernel(const DistParams P) {
  constexpr int VE = Elt<E>::kPerVec, NT = kDistNT, NW = kDistNW;
  const sd_distill_args &a = P.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint32_t named[];   // bit per place of this CTA's vectors
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = P.cs, rank = (int)cluster.block_rank(), n = blockIdx.x / cs;
  const int tid = threadIdx.x;
  __shared__ DistStat stat[kDistMaxCS];
  __shared__ float red[NW];
  __shared__ int bad_id;
  const RowView<E> row(a.student, (int64_t)n * a.student_s, a.V);
  const RowView<E> out(GRAD ? a.grad : a.student, (int64_t)n * (GRAD ? a.grad_s : a.student_s),
                       a.V);
  const int per = (row.nvec + cs - 1) / cs;
  const int qa = min(rank * per, row.nvec), qb = min(qa + per, row.nvec);
  const float w = a.weight ? ld_float(a.weight + n) : 1.f;
  const float zero[VE] = {};
  auto write = [&](int q, const float *f) {
    if (SAME) {
      store_vec<E>(out, q, f);
    } else {
      const int e0 = row.first(q);
      uint8_t *y = const_cast<uint8_t *>(out.row);
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (e0 + i >= 0 && e0 + i < row.n) Row<E>::store(y, e0 + i, f[i]);
    }
  };
  if (w == 0.f) {   // the same for every CTA of the row
    if (GRAD)
      for (int q = qa + tid; q < qb; q += NT) write(q, zero);
    if (a.loss && rank == 0 && tid == 0) a.loss[n] = 0.f;
    return;
  }
  row_cluster_arrive();
  // the named tokens: one per thread
  int id = -1;
  float t = neg_inf(), xs = neg_inf();
  if (tid < a.k) {
    id = ld_int(a.ids + (int64_t)n * a.k + tid);
    t = ld_float(a.vals + (int64_t)n * a.k + tid);
  }
  const float rest = a.rest ? ld_float(a.rest + n) : neg_inf();
  for (int i = tid; i < P.bit_words; i += NT) named[i] = 0u;
  if (tid == 0) bad_id = 0;
  __syncthreads();
  bool mine = false;   // this CTA's share holds the token
  if (id < -1 || id >= a.V) {
    bad_id = 1;
  } else if (id >= 0) {
    xs = Row<E>::load(row.row, id);
    const int at = id + row.hp - qa * VE;
    mine = at >= 0 && at < (qb - qa) * VE;
    if (mine && ((atomicOr(&named[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1u)) bad_id = 1;
  }
  if (id < 0) t = neg_inf();
  __syncthreads();

  // pass 1: the others' offset and sum
  const float c2 = log2e_over(a.T);
  float o = neg_inf(), z = 0.f;
  for (int q = qa + tid; q < qb; q += NT * kDistU) {
    uint4 v[kDistU];
#pragma unroll
    for (int u = 0; u < kDistU; ++u)
      if (q + u * NT < qb) v[u] = row.load(q + u * NT);
#pragma unroll
    for (int u = 0; u < kDistU; ++u) {
      const int p = q + u * NT;
      if (p >= qb) continue;
      float f[VE];
      Elt<E>::unpack(v[u], f);
      float m = Elt<E>::vmax(v[u]);
      const int at = (p - qa) * VE;
      const uint32_t bits = (named[at >> 5] >> (at & 31)) & ((1u << VE) - 1u);
      if (bits) {
        m = neg_inf();
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          if ((bits >> i) & 1u) f[i] = neg_inf();
          m = fmaxf(m, f[i]);
        }
      }
      if (m * c2 > o) {
        z *= ex2(o - m * c2);
        o = m * c2;
      }
      const float s = o == neg_inf() ? 0.f : o;
#pragma unroll
      for (int i = 0; i < VE; ++i) z += ex2(fmaf(f[i], c2, -s));
    }
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) {
    const float o2 = __shfl_xor_sync(0xffffffffu, o, i), z2 = __shfl_xor_sync(0xffffffffu, z, i);
    dist_merge(o, z, o2, z2);
  }
  __shared__ float wo[NW], wz[NW];
  if ((tid & 31) == 0) {
    wo[tid >> 5] = o;
    wz[tid >> 5] = z;
  }
  __syncthreads();
  o = wo[0];
  z = wz[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) dist_merge(o, z, wo[i], wz[i]);
  row_cluster_wait();
  if (tid < cs) {
    DistStat *s = cluster.map_shared_rank(&stat[rank], tid);
    s->o = o;
    s->z = z;
    s->bad = bad_id;
  }
  cluster.sync();
  o = neg_inf();
  z = 0.f;
  bool bad = false;
  for (int r = 0; r < cs; ++r) {
    dist_merge(o, z, stat[r].o, stat[r].z);
    bad |= stat[r].bad != 0;
  }
  // the teacher's shares, relative to its largest logit (in units of logits:
  // rest T is exact in the fused products)
  const bool taught = __syncthreads_or((id >= 0 && t != neg_inf()) || rest != neg_inf());
  const float tm = block_max<NW>(fmaxf(t, tid == 0 ? rest * a.T : neg_inf()), red);
  if (bad || !taught) {   // the same for every CTA of the row
    if (GRAD)
      for (int q = qa + tid; q < qb; q += NT) write(q, zero);
    if (rank == 0 && tid == 0) {
      if (a.loss) a.loss[n] = 0.f;
      if (bad && a.status) atomicOr(a.status, (int)SD_STATUS_BAD_TOKEN);
    }
    return;
  }
  const float tl = (t - tm) * c2;
  const float rl = rest == neg_inf() ? neg_inf() : fmaf(rest, a.T, -tm) * c2;
  const float te = ex2(tl), re = ex2(rl);
  const float zt = block_sum<NW>(te, red) + re;
  const float p = te / zt, pr = re / zt;
  // the student's, relative to its largest logit
  const float so = fmaxf(block_max<NW>(xs * c2, red), o);
  const float s0 = so == neg_inf() ? 0.f : so;
  const float sl = fmaf(xs, c2, -s0), se = id >= 0 ? ex2(sl) : 0.f;
  const float ol = o == neg_inf() ? neg_inf() : o - s0 + log2f(z);   // the others' log2 sum
  const float zr = z * ex2(o - s0);
  const float zs = block_sum<NW>(se, red) + zr;
  const float q = se / zs, qr = zr / zs;
  const float ln2 = 0.693147180559945309f;
  const float norm = log2f(zt) - log2f(zs);
  const float d = ((tl - sl) - norm) * ln2, dr = ((rl - ol) - norm) * ln2;
  if (a.loss && rank == 0) {
    float term = id >= 0 ? dist_term(p, q, d) : 0.f;
    if (tid == 0) term += dist_term(pr, qr, dr);
    const float kl = block_sum<NW>(term, red);
    if (tid == 0) a.loss[n] = w * kl;
  }
  if (!GRAD) return;
  // q_r - p_r without cancellation: by expm1 where the others have little of
  // the mass, from the named tokens' sums where they have most of it
  float diff = qr;
  if (pr > 0.f) {
    const float named_diff = block_sum<NW>(p - q, red);
    diff = qr > 0.5f ? named_diff : fabsf(dr) < 0.5f ? -qr * expm1f(dr) : qr - pr;
  }
  const float wt = w / a.T;
  const float coef = z > 0.f || z != z ? wt * diff / z : 0.f;
  const float o0 = o == neg_inf() ? 0.f : o;
  for (int v0 = qa + tid; v0 < qb; v0 += NT * kDistU) {
    uint4 v[kDistU];
#pragma unroll
    for (int u = 0; u < kDistU; ++u)
      if (v0 + u * NT < qb) v[u] = row.load(v0 + u * NT);
#pragma unroll
    for (int u = 0; u < kDistU; ++u) {
      if (v0 + u * NT >= qb) continue;
      float f[VE];
      Elt<E>::unpack(v[u], f);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = coef * ex2(fmaf(f[i], c2, -o0));
      write(v0 + u * NT, f);
    }
  }
  __syncthreads();  // the named places are written over the pass above
  if (mine) {
    const float g = fabsf(d) < 0.5f ? -q * expm1f(d) : q - p;
    Row<E>::store(const_cast<uint8_t *>(out.row), id, wt * g);
  }
}

template <typename E, bool GRAD, bool SAME>
static cudaError_t launch_distill(DistParams &P, cudaStream_t s) {
  constexpr int VE = Elt<E>::kPerVec;
  const int64_t nvec = ((int64_t)P.a.V + 2 * VE - 2) / VE;
  const int64_t slots = 2LL * sm_count();
  int cs = 1;
  while (cs < kDistMaxCS && (int64_t)P.a.N * cs * 2 <= slots && nvec / (2 * cs) >= kDistNT)
    cs *= 2;
  P.cs = cs;
  if ((int64_t)P.a.N * cs > INT32_MAX) return cudaErrorInvalidValue;
  P.bit_words = (int)(((nvec + cs - 1) / cs * VE + 31) / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.a.N * cs), 1, 1);
  cfg.blockDim = dim3(kDistNT, 1, 1);
  cfg.dynamicSmemBytes = (size_t)4 * P.bit_words;   // at most 32 KB
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sd_distill_kernel<E, GRAD, SAME>, (const DistParams)P);
}

template <typename E>
static cudaError_t launch_distill_any(DistParams &P, cudaStream_t s) {
  const sd_distill_args &a = P.a;
  if (!a.grad) return launch_distill<E, false, true>(P, s);
  const bool same = (((uintptr_t)a.student ^ (uintptr_t)a.grad) & 15) == 0 &&
                    (a.N <= 1 || (uint64_t)(a.student_s - a.grad_s) * Elt<E>::kSize % 16 == 0);
  return same ? launch_distill<E, true, true>(P, s) : launch_distill<E, true, false>(P, s);
}

}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_distill_args_size(void) { return sizeof(sd_distill_args); }

extern "C" sd_status_t sd_distill(const sd_distill_args *args, void *stream) {
  sdv::NvtxRange nvtx_range("sd_distill");
  if (!args) return SD_ERR_INVALID_ARG;
  DistParams P;
  memset(&P, 0, sizeof(P));
  P.a = *args;
  const sd_distill_args &a = P.a;
  if (a.N < 0 || a.V < 1 || a.V > SD_MAX_V || a.k < 0 || a.k > SD_MAX_TOP)
    return SD_ERR_INVALID_ARG;
  if (a.dtype != SD_F32 && a.dtype != SD_BF16) return SD_ERR_INVALID_ARG;
  if (!(a.T > 0.f) || !std::isfinite(a.T)) return SD_ERR_INVALID_ARG;
  if (a.N == 0) return SD_OK;
  if (!a.student || (!a.loss && !a.grad) || (a.k > 0 && (!a.ids || !a.vals)))
    return SD_ERR_INVALID_ARG;
  const size_t es = a.dtype == SD_BF16 ? 2 : 4;
  if ((uintptr_t)a.student % es || (uintptr_t)a.grad % es) return SD_ERR_INVALID_ARG;
  if (a.grad && a.N > 1 && a.grad_s < a.V) return SD_ERR_INVALID_ARG;  // rows share places
  const cudaError_t e = a.dtype == SD_BF16
                            ? launch_distill_any<__nv_bfloat16>(P, (cudaStream_t)stream)
                            : launch_distill_any<float>(P, (cudaStream_t)stream);
  return e == cudaSuccess ? SD_OK : e == cudaErrorInvalidValue ? SD_ERR_INVALID_ARG : SD_ERR_CUDA;
}
