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
// Few rows: one cluster of cs CTAs per row, which holds it in shared memory.
// The named places are set to -inf there, so that both passes meet only the
// others.  Pass 1: running maximum and sum.  The cluster exchanges (offset,
// sum) and every CTA works out the k + 1 buckets.  Pass 2 writes the gradient
// of its share, then the named places over it.
// Many rows: one CTA per row, streamed (sd_distill_stream_kernel).
// To move: 2 or 4 bytes per logit for the loss, twice that with the gradient.
// Measured on the GPU: the loss of 576 x 151936 bf16, k 64, 34 us (5.1 TB/s;
// two rows per CTA leave its ends uncovered); loss and gradient of 2048 x
// 128256, 208 us (5.1 TB/s of row bytes; DRAM moves more, since the second
// pass finds only a part of its row in L2: 304 rows of 256 KB are on their way
// beside what is written); 48 x 32000 fp32, k 16, 8.4 us.  A row shared by two
// CTAs, half as many rows on their way, took 228 us, by four 495.

#include "sd_rows.cuh"

namespace sdv {

constexpr int kDistNT = 256;
constexpr int kDistNW = kDistNT / 32;
constexpr int kDistU = 4;         // vectors at a time per thread

struct DistParams {
  sd_distill_args a;
  int cs;          // held rows: cluster size
  int vec_words;   // streamed rows: words with a bit per vector, and
  int bit_words;   // per place, of the named tokens
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

// The named tokens of a row in shared memory: id (-1: empty slot), the
// teacher's and the student's logit, and the gradient that comes out.
struct Named {
  int id[SD_MAX_TOP];
  float t[SD_MAX_TOP], x[SD_MAX_TOP], g[SD_MAX_TOP];
};
// What a row's second pass needs: the others' gradient is
// coef 2^((x - m) c2); not `live`: the row's loss and gradient are zero.
struct Buckets {
  float coef, m;
  int live;
};

// The k + 1 buckets, by one warp: loss, the named tokens' gradients and the
// others' factor from the others' (largest m, sum z of 2^((x - m) c2)).
__device__ __forceinline__ void dist_buckets(Named &N, Buckets &B, int k, float rest, float T,
                                             float c2, float w, float m, float z, bool bad,
                                             float *loss) {
  constexpr int J = SD_MAX_TOP / 32;
  const int lane = threadIdx.x & 31;
  float t[J], x[J];
  bool is[J];
  float tm = neg_inf(), sm = m;   // largest logits: of the teacher's named tokens, of the student
  bool taught = rest != neg_inf();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int i = j * 32 + lane;
    is[j] = i < k && N.id[i] >= 0;
    t[j] = is[j] ? N.t[i] : neg_inf();
    x[j] = is[j] ? N.x[i] : neg_inf();
    tm = fmaxf(tm, t[j]);
    sm = fmaxf(sm, x[j]);
    taught |= t[j] != neg_inf();
  }
  taught = ballot(taught) != 0u;
  if (bad || !taught) {
    if (lane == 0) {
      B.live = 0;
      if (loss) *loss = 0.f;
    }
    return;
  }
  tm = warp_max(tm);
  sm = warp_max(sm);
  const float s0 = sm == neg_inf() ? 0.f : sm;
  // log2 of the teacher's rest beside the largest named token's 2^0: a difference
  // of numbers that may be far larger than itself, and the ratio of the two masses
  // enters the loss to first order, so it is taken to twice fp32's digits where
  // both are in range, and by one fused operation, exact but for its own rounding,
  // where they are not.  Bounded, so that a finite rest has a finite one.
  float rl, rlo = 0.f;
  if (tm == neg_inf()) {   // all of the mass with the others
    tm = 0.f;
    rl = rest < INFINITY ? 0.f : rest - rest;   // NaN has a NaN loss
  } else if (fabsf(tm * c2) < 1e4f && fabsf(rest) < 1e4f) {
    const float l = 1.44269502f, ll = 1.92596299e-8f;           // log2 e = l + ll
    const float cl = (fmaf(-c2, T, l) + ll) / T;                // log2 e / T = c2 + cl
    const float u = rest * l, ul = fmaf(rest, l, -u) + rest * ll;
    const float v = tm * c2, vl = fmaf(tm, c2, -v) + tm * cl;
    rl = u - v;
    const float b = rl - u;
    rlo = ((u - (rl - b)) - (v + b)) + (ul - vl);
  } else {
    rl = fmaf(rest, T, -tm) * c2;
    if (rl > 1e30f && rest < INFINITY) rl = 1e30f;
  }
  // a power of two that keeps the larger of the two in range
  const float n = fmaxf(ceilf(rl), 0.f);
  const float down = n < 126.f ? __int_as_float((127 - (int)n) << 23) : 0.f;
  // the student's likewise: z = zm 2^e, 2^ns is taken out of its masses
  const int e = z >= 1.f && z < INFINITY ? (__float_as_int(z) >> 23) - 127 : 0;
  const float zm = __int_as_float(__float_as_int(z) - (e << 23));
  const float g = m == neg_inf() ? neg_inf() : (m - s0) * c2;
  const int ns = g > -64.f ? max(e + (int)ceilf(g), 0) : 0;
  const float sdown = __int_as_float((127 - ns) << 23);
  float te[J], se[J], tsum = 0.f, ssum = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    t[j] = (t[j] - tm) * c2;
    x[j] = (x[j] - s0) * c2;
    te[j] = ex2(t[j]) * down;
    t[j] -= n;
    se[j] = is[j] ? ex2(x[j]) * sdown : 0.f;
    x[j] -= (float)ns;
    tsum += te[j];
    ssum += se[j];
  }
  const float ol = (log2f(zm) + g) + (float)(e - ns);   // the others' log2 sum
  const float zr = z * sdown * ex2(g);
  const float ln2 = 0.693147180559945309f;
  const float re = ex2(rl - n) * fmaf(rlo, ln2, 1.f);
  const float zt = warp_sum(tsum) + re, zs = warp_sum(ssum) + zr;
  const float pr = re / zt, qr = zr / zs;
  const float norm = log2f(zt) - log2f(zs);
  const float dr = (((rl - n) + rlo - ol) - norm) * ln2;
  const float wt = w / T;
  // a named token's ln(p / q) from the difference of its two logits: the offsets
  // of both sides, far from them where the others hold most of the mass, enter
  // as one number, whose error is the same for all named tokens.  That error, and
  // the difference's own, grow with the distance between the two sides; from 32
  // on (in powers of two: about where they pass those of the logits' distances
  // from their own largest) each side is taken from its own offset instead.
  const float shift = (tm - s0) * c2 + (n - (float)ns);
  const bool direct = fabsf(shift) < 32.f;
  const float off = direct ? shift + norm : norm;
  float kl = lane == 0 ? dist_term(pr, qr, dr) : 0.f, named = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (j * 32 >= k) continue;   // the same for the warp
    const int i = j * 32 + lane;
    const float p = te[j] / zt, q = se[j] / zs;
    if (is[j]) {
      const float d = ((direct ? (N.t[i] - N.x[i]) * c2 : t[j] - x[j]) - off) * ln2;
      kl += dist_term(p, q, d);
      N.g[i] = wt * (p > 0.f && fabsf(d) < 0.5f ? -q * expm1f(d) : q - p);
      named += p - q;
    }
  }
  kl = warp_sum(kl);
  named = warp_sum(named);
  if (lane == 0) {
    if (loss) *loss = w * kl;
    // q_r - p_r without cancellation: by expm1 where the others have little of
    // the mass, from the named tokens' sums where they have most of it
    float diff = qr;
    if (pr > 0.f) diff = qr > 0.5f ? named : fabsf(dr) < 0.5f ? -qr * expm1f(dr) : qr - pr;
    B.live = 1;
    B.coef = z > 0.f || z != z ? wt * diff / z : 0.f;
    B.m = m == neg_inf() ? 0.f : m;
  }
}

// A vector of the gradient: q of a row of n elements at `row` in memory, SAME
// grid or element by element from element e0 on.
template <typename E, bool SAME>
__device__ __forceinline__ void write_grad(uint8_t *out, const RowView<E> &row, int q,
                                           const uint4 &v) {
  constexpr int VE = Elt<E>::kPerVec;
  const int e0 = row.first(q);
  if (SAME && row.whole(q)) {
    *reinterpret_cast<uint4 *>(out + (int64_t)e0 * Elt<E>::kSize) = v;
  } else {
    float f[VE];
    Elt<E>::unpack(v, f);
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (e0 + e >= 0 && e0 + e < row.n) Row<E>::store(out, e0 + e, f[e]);
  }
}

// GRAD: write the gradient; SAME: its rows lie on the 16-byte grid as the
// student's do (whole vectors), otherwise they are written element by element.
// Few rows: one cluster per row, which holds it.
template <typename E, bool GRAD, bool SAME>
__global__ void __launch_bounds__(kDistNT, kHeldCtas) sd_distill_kernel(const DistParams P) {
  constexpr int NT = kDistNT, NW = kDistNW, U = kDistU;
  const sd_distill_args &a = P.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint4 held[];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = P.cs, rank = (int)cluster.block_rank(), n = blockIdx.x / cs;
  const int tid = threadIdx.x;
  __shared__ DistStat stat[kHeldMaxCS];
  __shared__ float wm[NW], wz[NW];
  __shared__ __align__(16) Named named;
  __shared__ Buckets buckets;
  const float c2 = log2e_over(a.T);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const Held<E> H(a.student, (int64_t)n * a.student_s, a.V, rank, cs, smem_u32(held));
  const float w = a.weight ? ld_float(a.weight + n) : 1.f;
  uint8_t *out = GRAD ? (uint8_t *)a.grad + (int64_t)n * a.grad_s * Elt<E>::kSize : nullptr;
  if (w == 0.f) {   // the same for every CTA of the row
    if (GRAD)
      for (int i = tid; i < H.n; i += NT) write_grad<E, SAME>(out, H.row, H.qa + i, zero);
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
  bool bad = id < -1 || id >= a.V;
  const bool is = id >= 0 && !bad;
  if (is) xs = Row<E>::load(H.row.row, id);
  if (tid < SD_MAX_TOP) {
    named.id[tid] = is ? id : -1;
    named.t[tid] = t;
    named.x[tid] = xs;
  }
  cp_wait<0>();
  __syncthreads();   // the share and the named tokens are there
  const int at = is ? H.place(id) : -1;
  if (at >= 0) H.clear(at);
  if (is)   // named before?
    for (int i = 0; i < tid; i += 4) {
      const int4 o = *reinterpret_cast<const int4 *>(named.id + i);
      bad |= o.x == id || (o.y == id && i + 1 < tid) || (o.z == id && i + 2 < tid) ||
             (o.w == id && i + 3 < tid);
    }
  bad = __syncthreads_or(bad) != 0;

  // pass 1: the others' largest logit and sum
  ExpSum<E> sum;
  sum.template add_share<NT, U>(H, c2);
  sum.template block<NW>(c2, wm, wz);
  row_cluster_wait();   // every CTA of the cluster has started
  if (tid < cs) {
    DistStat *s = cluster.map_shared_rank(&stat[rank], tid);
    s->m = sum.m;
    s->z = sum.z;
  }
  cluster.sync();
  if (tid < 32) {
    float m = neg_inf(), z = 0.f;
    for (int r = 0; r < cs; ++r) exp_merge(m, z, stat[r].m, stat[r].z, c2);
    dist_buckets(named, buckets, a.k, rest, a.T, c2, w, m, z, bad,
                 a.loss && rank == 0 ? a.loss + n : nullptr);
    if (bad && rank == 0 && tid == 0 && a.status) atomicOr(a.status, (int)SD_STATUS_BAD_TOKEN);
  }
  if (!GRAD) return;
  __syncthreads();
  const bool live = buckets.live != 0;
  const float coef = live ? buckets.coef : 0.f;
  const ExpBase B(buckets.m, c2);
  const uint64_t ss = pk2(coef * B.fix, coef * B.fix);
  uint8_t *to = out + (int64_t)H.row.first(H.qa) * Elt<E>::kSize;
#pragma unroll 4
  for (int i = tid; i < H.n; i += NT) {
    uint4 v = H.get(i);
    v = !live ? zero : !B.far ? VecExp<E>::template scaled<false>(v, B, ss)
                              : VecExp<E>::template scaled<true>(v, B, ss);
    if (SAME && H.inner(i)) *reinterpret_cast<uint4 *>(to + (int64_t)i * 16) = v;
    else write_grad<E, SAME>(out, H.row, H.qa + i, v);
  }
  __syncthreads();  // the named places are written over the pass above
  if (live && at >= 0) Row<E>::store(out, id, named.g[tid]);
}

// Many rows: one CTA per row, streamed once for the sum and, for the gradient,
// once more (2048 x 128256 bf16: L2 still holds somewhat more than half of
// it).  The named tokens are marked in shared memory, a bit per
// vector (looked at for every vector) and a bit per place.  Nothing but the
// CTA's own barriers lies between the passes.
template <typename E, bool GRAD, bool SAME>
__global__ void __launch_bounds__(kStreamNT, 2) sd_distill_stream_kernel(const DistParams P) {
  constexpr int VE = Elt<E>::kPerVec, NT = kStreamNT, NW = NT / 32, U = kStreamU;
  const sd_distill_args &a = P.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using Stream = RowStream<E, NT, U, kStreamD>;
  extern __shared__ uint4 ring[];
  uint32_t *vecs = reinterpret_cast<uint32_t *>(ring + Stream::kBytes / 16);
  uint32_t *bits = vecs + P.vec_words;
  __shared__ float wm[NW], wz[NW];
  __shared__ Named named;
  __shared__ Buckets buckets;
  __shared__ int dup;
  const int tid = threadIdx.x;
  for (int i = tid; i < P.vec_words + P.bit_words; i += NT) vecs[i] = 0u;
  if (tid == 0) dup = 0;
  Stream S(ring, a.student, a.student_s, a.N, a.V, GRAD ? 2 : 1, a.weight);
  const float c2 = log2e_over(a.T);
  // this row's teacher, asked for a row ahead
  int id_next = -1;
  float t_next = neg_inf(), w_next = 1.f, rest_next = neg_inf();
  auto ahead = [&](int n) {
    if (n >= a.N) return;
    if (tid < a.k) {
      id_next = ld_int(a.ids + (int64_t)n * a.k + tid);
      t_next = ld_float(a.vals + (int64_t)n * a.k + tid);
    }
    if (a.weight) w_next = ld_float(a.weight + n);
    if (a.rest) rest_next = ld_float(a.rest + n);
  };
  ahead(blockIdx.x);
  int late = -1;            // a named place of the row before, still to be written
  uint8_t *late_out = nullptr;
  __syncthreads();
  for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
    const int id = id_next;
    const float t = t_next, w = w_next, rest = rest_next;
    ahead(n + gridDim.x);
    const RowView<E> row(a.student, (int64_t)n * a.student_s, a.V);
    uint8_t *out = GRAD ? (uint8_t *)a.grad + (int64_t)n * a.grad_s * Elt<E>::kSize : nullptr;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    if (w == 0.f) {
      if (GRAD)
        for (int q = tid; q < row.nvec; q += NT) write_grad<E, SAME>(out, row, q, zero);
      if (a.loss && tid == 0) a.loss[n] = 0.f;
      continue;
    }
    bool bad = id < -1 || id >= a.V;
    const bool is = id >= 0 && !bad;
    const int at = id + row.hp;
    float xs = neg_inf();
    if (is) {
      xs = Row<E>::load(row.row, id);
      if ((atomicOr(&bits[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1u) dup = 1;
      atomicOr(&vecs[at / VE >> 5], 1u << (at / VE & 31));
    }
    if (bad) dup = 1;
    __syncthreads();   // the bits are set; the row before is all written
    if (late >= 0) Row<E>::store(late_out, late, named.g[tid]);
    // pass 1
    ExpSum<E> sum;
    for (int q = 0; q < row.nvec; q += Stream::kStep) {
      uint4 v[U];
      S.next(v);
      const int first = q + Stream::at();
      if (q + Stream::kStep > row.nvec) {
        const uint32_t inf = Elt<E>::kNegInfWord;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (first + u * 32 >= row.nvec) v[u] = make_uint4(inf, inf, inf, inf);
      }
      uint32_t w[U], any = 0u;
#pragma unroll
      for (int u = 0; u < U; ++u) any |= w[u] = vecs[(q >> 5) + (tid >> 5) * U + u];
      if (any) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!((w[u] >> (tid & 31)) & 1u)) continue;
          const int at = (first + u * 32) * VE;
          v[u] = mask_vec<E>(v[u], ~(bits[at >> 5] >> (at & 31)) & ((1u << VE) - 1u));
        }
      }
      sum.template add<U>(v, c2);
    }
    if (tid < SD_MAX_TOP) {
      named.id[tid] = is ? id : -1;
      named.t[tid] = t;
      named.x[tid] = xs;
    }
    sum.warp(c2);
    if ((tid & 31) == 0) {
      wm[tid >> 5] = sum.m;
      wz[tid >> 5] = sum.z;
    }
    __syncthreads();   // the warps' sums and the named tokens are there
    if (is) bits[at >> 5] = vecs[at / VE >> 5] = 0u;
    if (tid < 32) {
      const bool any = dup != 0;
      sum.m = tid < NW ? wm[tid] : neg_inf();
      sum.z = tid < NW ? wz[tid] : 0.f;
      sum.warp(c2);
      dist_buckets(named, buckets, a.k, rest, a.T, c2, w, sum.m, sum.z, any,
                   a.loss ? a.loss + n : nullptr);
      if (tid == 0) {
        dup = 0;
        if (any && a.status) atomicOr(a.status, (int)SD_STATUS_BAD_TOKEN);
      }
    }
    __syncthreads();
    late = -1;
    if (!GRAD) continue;
    // pass 2
    const bool live = buckets.live != 0;
    const float coef = live ? buckets.coef : 0.f;
    const ExpBase B(buckets.m, c2);
    const uint64_t ss = pk2(coef * B.fix, coef * B.fix);
    const int last = (row.nvec - 1) / Stream::kStep * Stream::kStep;
    uint8_t *to = out + ((int64_t)(last + Stream::at()) * VE - row.hp) * Elt<E>::kSize;
    for (int q = last; q >= 0; q -= Stream::kStep, to -= Stream::kStep * 16) {
      uint4 v[U];
      S.next(v);
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = !live ? zero : !B.far ? VecExp<E>::template scaled<false>(v[u], B, ss)
                                     : VecExp<E>::template scaled<true>(v[u], B, ss);
      if (SAME && q > 0 && q + Stream::kStep < row.nvec) {
#pragma unroll
        for (int u = 0; u < U; ++u) __stcs(reinterpret_cast<uint4 *>(to + u * 512), v[u]);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = q + Stream::at() + u * 32;
          if (i < row.nvec) write_grad<E, SAME>(out, row, i, v[u]);
        }
      }
    }
    if (is && live) {   // written over the pass above, after the next barrier
      late = id;
      late_out = out;
    }
  }
  if (GRAD) {
    __syncthreads();
    if (late >= 0) Row<E>::store(late_out, late, named.g[tid]);
  }
}

template <typename E, bool GRAD, bool SAME>
static cudaError_t launch_distill(DistParams &P, cudaStream_t s) {
  int smem = 0;
  P.cs = held_cluster<E>(P.a.N, P.a.V, kDistNT, &smem);
  if (P.cs > 0) {
    static FuncAttrs attrs;
    attrs.apply((const void *)sd_distill_kernel<E, GRAD, SAME>, kHeldBytes + 16, true,
                "the distillation kernel");
    return launch_held(sd_distill_kernel<E, GRAD, SAME>, P, P.a.N, P.cs, kDistNT, smem, s);
  }
  constexpr int VE = Elt<E>::kPerVec;
  using Stream = RowStream<E, kStreamNT, kStreamU, kStreamD>;
  const int64_t nvec = ((int64_t)P.a.V + 2 * VE - 2) / VE;
  P.vec_words = (int)((nvec + Stream::kStep - 1) / Stream::kStep * (Stream::kStep / 32));
  P.bit_words = (int)((nvec * VE + 31) / 32);
  static FuncAttrs attrs;
  attrs.apply((const void *)sd_distill_stream_kernel<E, GRAD, SAME>, 200 * 1024, false,
              "the distillation kernel");
  return launch_streamed(sd_distill_stream_kernel<E, GRAD, SAME>, P, P.a.N, kStreamNT,
                         Stream::kBytes + 4 * (P.vec_words + P.bit_words), s);
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
