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
// One cluster of cs CTAs per row, which holds it in shared memory.  The named
// places are set to -inf there, so that both passes meet only the others.
// Pass 1: running maximum and sum.  The cluster exchanges (offset, sum) and
// every CTA works out the k + 1 buckets.  Pass 2 writes the gradient of its
// share, then the named places over it.  HBM-bound: 2 or 4 bytes per logit
// for the loss, twice that with the gradient.

#include "sd_rows.cuh"

namespace sdv {

constexpr int kDistNT = 256;
constexpr int kDistNW = kDistNT / 32;
constexpr int kDistU = 4;         // vectors at a time per thread

struct DistParams {
  sd_distill_args a;
  int cs;
};

// A share of the others: its largest logit, the sum of 2^((x - m) c2).
struct DistStat {
  float m, z;
};

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

// GRAD: write the gradient; SAME: its rows lie on the 16-byte grid as the
// student's do (whole vectors), otherwise they are written element by element.
template <typename E, bool GRAD, bool SAME>
__global__ void __launch_bounds__(kDistNT, kHeldCtas) sd_distill_kernel(const DistParams P) {
  constexpr int VE = Elt<E>::kPerVec, NT = kDistNT, NW = kDistNW, U = kDistU;
  const sd_distill_args &a = P.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint4 held[];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = P.cs, rank = (int)cluster.block_rank(), n = blockIdx.x / cs;
  const int tid = threadIdx.x;
  __shared__ DistStat stat[kHeldMaxCS];
  __shared__ float red[NW], wm[NW], wz[NW];
  __shared__ __align__(16) int ids[SD_MAX_TOP];
  Held<E> H(a.student, (int64_t)n * a.student_s, a.V, rank, cs, held);
  const float w = a.weight ? ld_float(a.weight + n) : 1.f;
  uint8_t *out = GRAD ? (uint8_t *)a.grad + (int64_t)n * a.grad_s * Elt<E>::kSize : nullptr;
  auto write = [&](int i, const uint4 &v) {   // vector i of the share
    const int e0 = H.row.first(H.qa + i);
    if (SAME && H.row.whole(H.qa + i)) {
      *reinterpret_cast<uint4 *>(out + (int64_t)e0 * Elt<E>::kSize) = v;
    } else {
      float f[VE];
      Elt<E>::unpack(v, f);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (e0 + e >= 0 && e0 + e < a.V) Row<E>::store(out, e0 + e, f[e]);
    }
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (w == 0.f) {   // the same for every CTA of the row
    if (GRAD)
      for (int i = tid; i < H.n; i += NT) write(i, zero);
    if (a.loss && rank == 0 && tid == 0) a.loss[n] = 0.f;
    return;
  }
  row_cluster_arrive();
  H.template fetch<NT>();
  // the named tokens: one per thread
  int id = -1;
  float t = neg_inf(), xs = neg_inf();
  if (tid < a.k) {
    id = ld_int(a.ids + (int64_t)n * a.k + tid);
    t = ld_float(a.vals + (int64_t)n * a.k + tid);
  }
  const float rest = a.rest ? ld_float(a.rest + n) : neg_inf();
  if (tid < SD_MAX_TOP) ids[tid] = id;
  bool bad = id < -1 || id >= a.V;
  const bool is = id >= 0 && !bad;
  if (is) xs = Row<E>::load(H.row.row, id);
  else t = neg_inf();
  cp_wait<0>();
  __syncthreads();   // the share and the ids are there
  const int at = is ? H.place(id) : -1;
  if (at >= 0) {
    if (VE == 8) reinterpret_cast<uint16_t *>(held)[at] = 0xff80u;
    else reinterpret_cast<uint32_t *>(held)[at] = 0xff800000u;
  }
  if (is)   // named before?
    for (int i = 0; i < tid; i += 4) {
      const int4 o = *reinterpret_cast<const int4 *>(ids + i);
      bad |= o.x == id || (o.y == id && i + 1 < tid) || (o.z == id && i + 2 < tid) ||
             (o.w == id && i + 3 < tid);
    }
  bad = __syncthreads_or(bad) != 0;

  // pass 1: the others' largest logit and sum
  const float c2 = log2e_over(a.T);
  ExpSum<E> sum;
  sum.template add_share<NT, U>(held, H.n, c2);
  sum.template block<NW>(c2, wm, wz);
  row_cluster_wait();
  if (tid < cs) {
    DistStat *s = cluster.map_shared_rank(&stat[rank], tid);
    s->m = sum.m;
    s->z = sum.z;
  }
  cluster.sync();
  float m = neg_inf(), z = 0.f;
  for (int r = 0; r < cs; ++r) exp_merge(m, z, stat[r].m, stat[r].z, c2);
  // the teacher's shares, relative to its largest logit (in units of logits:
  // rest T is exact in the fused products)
  const bool taught = __syncthreads_or((is && t != neg_inf()) || rest != neg_inf()) != 0;
  const float tm = block_max<NW>(fmaxf(t, tid == 0 ? rest * a.T : neg_inf()), red);
  if (bad || !taught) {   // the same for every CTA of the row
    if (GRAD)
      for (int i = tid; i < H.n; i += NT) write(i, zero);
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
  const float sm = fmaxf(block_max<NW>(xs, red), m);
  const float s0 = sm == neg_inf() ? 0.f : sm;
  const float sl = (xs - s0) * c2, se = is ? ex2(sl) : 0.f;
  const float ol = m == neg_inf() ? neg_inf() : (m - s0) * c2 + log2f(z);   // the others' log2 sum
  const float zr = z * ex2((m - s0) * c2);
  const float zs = block_sum<NW>(se, red) + zr;
  const float q = se / zs, qr = zr / zs;
  const float ln2 = 0.693147180559945309f;
  const float norm = log2f(zt) - log2f(zs);
  const float d = ((tl - sl) - norm) * ln2, dr = ((rl - ol) - norm) * ln2;
  if (a.loss && rank == 0) {
    float term = is ? dist_term(p, q, d) : 0.f;
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
  const float m0 = m == neg_inf() ? 0.f : m;
  const uint64_t cc = pk2(c2, c2), oo = pk2(-m0, -m0), ss = pk2(coef, coef);
#pragma unroll 4
  for (int i = tid; i < H.n; i += NT) write(i, VecExp<E>::scaled(held[i], cc, oo, ss));
  __syncthreads();  // the named places are written over the pass above
  if (at >= 0) {
    const float g = fabsf(d) < 0.5f ? -q * expm1f(d) : q - p;
    Row<E>::store(out, id, wt * g);
  }
}

template <typename E, bool GRAD, bool SAME>
static cudaError_t launch_distill(DistParams &P, cudaStream_t s) {
  int smem = 0;
  P.cs = held_cluster<E>(P.a.N, P.a.V, kDistNT, &smem);
  static FuncAttrs attrs;
  attrs.apply((const void *)sd_distill_kernel<E, GRAD, SAME>, kHeldBytes + 16, true,
              "the distillation kernel");
  return launch_held(sd_distill_kernel<E, GRAD, SAME>, P, P.a.N, P.cs, kDistNT, smem, s);
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
