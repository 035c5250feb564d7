// The k best continuations of each sequence's beams: s + x / T - log sum exp(x / T)
// over W rows of V logits, by two launches.
//
//  1. sd_beam_stream_kernel: every CTA takes one chunk of a row, held in
//     registers.  It writes the chunk's (largest m, sum of 2^((x - m) c)) and the
//     largest logit of every four threads' vectors (a group).  No beam's row is
//     read twice, and nothing depends on other CTAs.
//  2. sd_beam_end_kernel: one CTA per sequence joins the sums of each beam in 64
//     bits, and finds from the groups' largest logits alone a value that k of
//     them reach: no candidate below it is among the k best.  The groups that
//     reach it (little more than k of them) are read again, their logits that
//     do are ranked in 64 bits.
// A sequence of which more groups or logits reach the bound than there is room
// for (thousands of equal logits at the k-th place) takes its beams one by one:
// see each_beam.

#include "sd_rows.cuh"
#include "sd_beam.h"

namespace sdv {

constexpr int kSelNT = 256;      // threads of a streaming CTA
constexpr int kSelSet = 4;       // threads of a group
constexpr int kSelSets = kSelNT / kSelSet;
constexpr int kEndNT = 512;      // threads of a sequence's end
constexpr int kEndU = 4;         // vectors of groups that one of them holds
constexpr int kSelList = 1024;   // listed groups, and candidates, of a sequence

struct SelectParams {
  const void *logits;
  int64_t sb, sw;
  int B, W, V, k, nc, share, eos;
  float T;
  double inv_T;
  const float *scores, *norm;
  const uint8_t *finished;
  float2 *part;      // [B W][nc]: largest logit of a chunk and its sum
  float *gmax;       // [B W][nc][kSelSets]: largest logit of each group
  float *out_scores;
  int32_t *parents, *tokens;
  uint8_t *ended;
  int32_t *status;
};

// How rows are cut: nc chunks of `share` vectors, at most U of them per thread.
struct SelectCut {
  int U, nc, share;
};
static SelectCut select_cut(int64_t rows, int V, int es) {
  const int ve = 16 / es;
  const int nvec = (int)(((int64_t)V + ve - 1) / ve);
  SelectCut c;
  c.U = rows * nvec >= (int64_t)2 * 8 * kSelNT * sm_count() ? 8 : 2;
  c.nc = (nvec + c.U * kSelNT - 1) / (c.U * kSelNT);
  c.share = (nvec + c.nc - 1) / c.nc;
  return c;
}

// A row as vectors of its own elements: vector q holds elements q VE and on, wherever
// the row starts, so that what is computed of a row does not depend on that
// and beams that are alike tie.  Off the 16-byte grid it is cut from the two
// vectors of memory that it lies in.
template <typename E>
struct ElemRow {
  static constexpr int VE = Elt<E>::kPerVec;
  const uint8_t *row;
  int hp, n, nvec;
  __device__ __forceinline__ ElemRow(const void *base, int64_t offset, int n_) {
    row = reinterpret_cast<const uint8_t *>(base) + offset * Elt<E>::kSize;
    hp = (int)((uintptr_t)row & 15) / Elt<E>::kSize;
    n = n_;
    nvec = (n + VE - 1) / VE;
  }
  __device__ __forceinline__ int first(int q) const { return q * VE; }
  // vectors [lo, hi) can be loaded without leaving the row
  __device__ __forceinline__ int lo() const { return hp ? 1 : 0; }
  __device__ __forceinline__ int hi() const { return (n + hp) / VE - (hp ? 1 : 0); }
  __device__ __forceinline__ const uint8_t *grid(int q) const {
    return row + ((int64_t)q * VE - hp) * Elt<E>::kSize;
  }
  __device__ __forceinline__ uint4 cut(const uint4 &a, const uint4 &b) const {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int words = hp * Elt<E>::kSize / 4;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = words & 2 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = words & 1 ? w[i + 1] : w[i];
    if (Elt<E>::kSize == 2 && (hp & 1))
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // vector q < nvec, -inf past the row
  __device__ __forceinline__ uint4 load(int q) const {
    if (q >= lo() && q < hi()) return hp ? cut(ld16(grid(q)), ld16(grid(q + 1))) : ld16(grid(q));
    return load_edge(q);
  }
  __device__ __noinline__ uint4 load_edge(int q) const {
    float f[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i)
      f[i] = q * VE + i < n ? Row<E>::load(row, q * VE + i) : neg_inf();
    uint4 v;
    Row<E>::pack(f, v);
    return v;
  }
};

template <typename E, int U>
__global__ void __launch_bounds__(kSelNT) sd_beam_stream_kernel(const SelectParams P) {
  constexpr int NT = kSelNT, NW = NT / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = blockIdx.x / P.nc, chunk = blockIdx.x % P.nc, tid = threadIdx.x;
  // a beam that is dead or finished has no candidates of its own
  if (!(fabsf(ld_float(P.scores + n)) < INFINITY)) return;
  if (P.finished && ld1(P.finished + n)) return;
  const ElemRow<E> row(P.logits, (n / P.W) * P.sb + (n % P.W) * P.sw, P.V);
  const int q0 = chunk * P.share, q1 = min(q0 + P.share, row.nvec);
  const int lo = max(q0, row.lo()), hi = min(q1, row.hi());
  const uint8_t *src = row.grid(q0 + tid);
  const uint32_t inf = Elt<E>::kNegInfWord;
  uint4 v[U];
  if (row.hp == 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + tid + u * NT;
      v[u] = make_uint4(inf, inf, inf, inf);
      if (q >= lo && q < hi) v[u] = ld16(src + (int64_t)u * NT * 16);
    }
  } else {
    uint4 next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + tid + u * NT;
      v[u] = next[u] = make_uint4(inf, inf, inf, inf);
      if (q >= lo && q < hi) {
        v[u] = ld16(src + (int64_t)u * NT * 16);
        next[u] = ld16(src + (int64_t)u * NT * 16 + 16);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = row.cut(v[u], next[u]);
  }
  if (lo > q0 || hi < q1) {   // the row's first or last vectors
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + tid + u * NT;
      if (q < q1 && (q < lo || q >= hi)) v[u] = row.load_edge(q);
    }
  }
  __shared__ float wm[NW], wz[NW];
  const float best = VecExp<E>::template largest<U>(v);
  float m = best;
#pragma unroll
  for (int o = 1; o < kSelSet; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (tid % kSelSet == 0) P.gmax[((int64_t)n * P.nc + chunk) * kSelSets + tid / kSelSet] = m;
  m = rmax_f(m);
  if ((tid & 31) == 0) wm[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NW; ++i) m = fmaxf(m, wm[i]);
  const float c2 = log2e_over(P.T);
  const ExpBase B(m, c2);
  uint64_t acc = 0ull;
  if (!B.far) {
#pragma unroll
    for (int u = 0; u < U; ++u) acc = VecExp<E>::template sum<false>(v[u], B, acc);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) acc = VecExp<E>::template sum<true>(v[u], B, acc);
  }
  float x, y;
  upk2(acc, x, y);
  const float z = warp_sum((x + y) * B.fix);
  if ((tid & 31) == 0) wz[tid >> 5] = z;
  __syncthreads();
  if (tid == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) t += wz[i];
    P.part[(int64_t)n * P.nc + chunk] = make_float2(m, t);
  }
}

// A double's order as an unsigned integer (never a NaN here).
__device__ __forceinline__ unsigned long long dord(double x) {
  const long long i = __double_as_longlong(x + 0.0);
  return (unsigned long long)i ^ (i < 0 ? ~0ull : 1ull << 63);
}

// What a sequence's end holds on chip.
struct SelectEnd {
  // a beam: 0 offers nothing, 1 live, 2 finished; its score less the log of its sum
  int kind[SD_MAX_BEAMS];
  double base[SD_MAX_BEAMS];
  double over[SD_MAX_BEAMS];          // 1 / norm
  double z[SD_MAX_BEAMS];
  // an fp32 image of the ranked score: max((x - m) c + o, lowest)
  float m[SD_MAX_BEAMS], c[SD_MAX_BEAMS], o[SD_MAX_BEAMS];
  int list[kSelList];                 // groups: beam, chunk, place
  unsigned long long key[kSelList];   // candidates: their order,
  int at[kSelList];                   // w V + v,
  float x[kSelList];                  // and logit
  unsigned long long best_key[SD_MAX_TOP];   // the k best, in order
  int best_at[SD_MAX_TOP];
  float best_x[SD_MAX_TOP];
  unsigned short keys16[kEndNT];
  int warp_n[kEndNT / 32];
  float bound;
  int n_list, n_cand, n_best, count;
};

template <typename E>
struct EndView {
  static constexpr int VE = Elt<E>::kPerVec;
  const SelectParams &P;
  SelectEnd &S;
  int b, U;
  __device__ __forceinline__ EndView(const SelectParams &P_, SelectEnd &S_, int U_)
      : P(P_), S(S_), b(blockIdx.x), U(U_) {}
  __device__ __forceinline__ ElemRow<E> row(int w) const {
    return ElemRow<E>(P.logits, b * P.sb + w * P.sw, P.V);
  }
  __device__ __forceinline__ const float *groups(int w) const {
    return P.gmax + ((int64_t)b * P.W + w) * P.nc * kSelSets;
  }
  // vectors of a group, and the row's vector that is number i of group g, or -1
  __device__ __forceinline__ int size() const { return kSelSet * U; }
  __device__ __forceinline__ int vector(const ElemRow<E> &r, int g, int i) const {
    const int chunk = g / kSelSets;
    const int at = g % kSelSets * kSelSet + i % kSelSet + i / kSelSet * kSelNT;
    const int q = chunk * P.share + at;
    return at < P.share && q < r.nvec ? q : -1;
  }
  __device__ __forceinline__ float approx(int w, float x) const {
    return x > neg_inf() ? fmaxf(fmaf(x - S.m[w], S.c[w], S.o[w]), kLowest) : neg_inf();
  }
  __device__ __forceinline__ double score(int w, float x) const {
    return S.kind[w] == 2 ? S.base[w]
                          : S.base[w] + ((double)x - (double)S.m[w]) * P.inv_T;
  }
  __device__ __forceinline__ void offer(int w, int v, float x) const {
    const int i = atomicAdd(&S.n_cand, 1);
    if (i < kSelList) {
      S.key[i] = dord(score(w, x) * S.over[w]);
      S.at[i] = w * P.V + v;
      S.x[i] = x;
    }
  }
};

// The k best of the candidates, in order, into S.best_*: their places are how
// many are better, and no two are alike.  Begins and ends with a barrier.
__device__ __forceinline__ void rank_candidates(SelectEnd &S, int k) {
  __syncthreads();
  const int n = min(S.n_cand, kSelList);
  for (int i = threadIdx.x; i < n; i += kEndNT) {
    const unsigned long long key = S.key[i];
    const int at = S.at[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += S.key[j] > key || (S.key[j] == key && S.at[j] < at);
    if (above < k) {
      S.best_key[above] = key;
      S.best_at[above] = at;
      S.best_x[above] = S.x[i];
    }
  }
  if (threadIdx.x == 0) S.n_best = min(n, k);
  __syncthreads();
}

// The sum of the threads' counts, in every thread.
__device__ __forceinline__ int block_count(SelectEnd &S, int n) {
  __syncwarp();
  n = __reduce_add_sync(0xffffffffu, n);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) S.warp_n[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int i = 0; i < kEndNT / 32; ++i) n += S.warp_n[i];
  return n;
}

// The beams one by one, whatever their logits: the k best of one by value, then
// by index, join the k best so far.
//  - v*, the k-th largest of its groups' largest, bit by bit;
//  - the logits above v* lie in fewer than k groups.  If they are more than k,
//    the key (value, index) of the k-th is found bit by bit;
//  - if they are fewer, logits equal to v* fill up, lowest index first, from the
//    row's beginning until there are enough.
template <typename E>
__device__ __noinline__ void each_beam(const EndView<E> &X) {
  constexpr int VE = EndView<E>::VE, NT = kEndNT;
  SelectEnd &S = X.S;
  const SelectParams &P = X.P;
  const int tid = threadIdx.x, k = P.k;
  __syncthreads();
  if (tid == 0) S.n_best = 0;
  __syncthreads();
  for (int w = 0; w < P.W; ++w) {
    if (S.kind[w] == 0) continue;
    // the best so far are candidates again
    const int kept = S.n_best;
    for (int i = tid; i < kept; i += NT) {
      S.key[i] = S.best_key[i];
      S.at[i] = S.best_at[i];
      S.x[i] = S.best_x[i];
    }
    if (tid == 0) {
      S.n_cand = kept;
      S.n_list = 0;
    }
    __syncthreads();
    if (S.kind[w] == 2) {
      if (tid == 0) X.offer(w, P.eos, 0.f);
      rank_candidates(S, k);
      continue;
    }
    const ElemRow<E> row = X.row(w);
    const float *gm = X.groups(w);
    const int ng = P.nc * kSelSets;
    const unsigned low = (unsigned)ford(kLowest) ^ 0x80000000u;
    unsigned r = 0u;
    for (int bit = 31; bit >= 0; --bit) {
      const unsigned t = r | (1u << bit);
      int n = 0;
      for (int i = tid; i < ng; i += NT) n += ((unsigned)ford(ld_float(gm + i)) ^ 0x80000000u) >= t;
      if (block_count(S, n) >= k) r = t;
    }
    const float least = fdeord((int)(max(r, low) ^ 0x80000000u));
    for (int i = tid; i < ng; i += NT)
      if (ld_float(gm + i) > least) {   // fewer than k
        const int at = atomicAdd(&S.n_list, 1);
        if (at < kSelList) S.list[at] = i;
      }
    __syncthreads();
    const int items = min(S.n_list, kSelList) * X.size();
    auto above = [&](unsigned long long from, auto f) {
      for (int i = tid; i < items; i += NT) {
        const int q = X.vector(row, S.list[i / X.size()], i % X.size());
        if (q < 0) continue;
        float x[VE];
        Elt<E>::unpack(row.load(q), x);
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (x[e] > least && top_key(x[e], row.first(q) + e) >= from) f(x[e], row.first(q) + e);
      }
    };
    int more = 0;
    above(0ull, [&](float, int) { ++more; });
    more = block_count(S, more);
    unsigned long long from = 0ull;
    if (more > k) {
      for (int bit = 63; bit >= 0; --bit) {
        int n = 0;
        above(from | (1ull << bit), [&](float, int) { ++n; });
        if (block_count(S, n) >= k) from |= 1ull << bit;
      }
    }
    above(from, [&](float x, int v) { X.offer(w, v, x); });
    if (more < k) {
      int need = k - more;
      for (int q0 = 0; q0 < row.nvec && need > 0; q0 += NT) {
        float x[VE];
        int n = 0;
        if (q0 + tid < row.nvec) Elt<E>::unpack(row.load(q0 + tid), x);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          if (q0 + tid >= row.nvec) x[e] = neg_inf();
          n += x[e] == least;
        }
        // places in the order of the threads
        int upto = n;
        __syncwarp();
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          upto += (tid & 31) >= o ? y : 0;
        }
        __syncthreads();
        if ((tid & 31) == 31) S.warp_n[tid >> 5] = upto;
        __syncthreads();
        int before = upto - n, all = 0;
        for (int i = 0; i < NT / 32; ++i) {
          before += i < (tid >> 5) ? S.warp_n[i] : 0;
          all += S.warp_n[i];
        }
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (x[e] == least) {
            if (before < need) X.offer(w, row.first(q0 + tid) + e, x[e]);
            ++before;
          }
        need -= all;
      }
    }
    rank_candidates(S, k);
  }
}

template <typename E>
__global__ void __launch_bounds__(kEndNT) sd_beam_end_kernel(const SelectParams P, int U) {
  constexpr int VE = Elt<E>::kPerVec, NT = kEndNT, NW = NT / 32;
  __shared__ SelectEnd S;
  const EndView<E> X(P, S, U);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = P.W, k = P.k;
  const int64_t b = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) S.n_list = S.n_cand = 0;
  // the groups' largest, kEndU vectors of four per thread at a time
  const int per = P.nc * kSelSets / 4, all = W * per;
  const float *gm = X.groups(0);
  uint4 held[kEndU];
#pragma unroll
  for (int u = 0; u < kEndU; ++u)
    if (tid + u * NT < all) held[u] = ld16(gm + (int64_t)(tid + u * NT) * 4);
  // a warp per beam: the sum over its chunks, in 64 bits
  for (int w = warp; w < W; w += NW) {
    const int64_t n = b * W + w;
    const float2 *part = P.part + n * P.nc;
    float2 p = lane < P.nc ? __ldcg(part + lane) : make_float2(neg_inf(), 0.f);
    const float s = ld_float(P.scores + n), nm = P.norm ? ld_float(P.norm + n) : 1.f;
    int kind = s == neg_inf() ? 0 : P.finished && ld1(P.finished + n) ? 2 : 1;
    int bad = 0;
    if (!(fabsf(s) < INFINITY) && s != neg_inf()) {
      kind = 0;
      bad = SD_STATUS_NONFINITE;
    } else if (kind && !(nm > 0.f && nm < INFINITY)) {
      kind = 0;
      bad = SD_STATUS_BAD_PENALTY;
    }
    float m = neg_inf();
    double z = 1.0;
    if (kind == 1) {   // else the sums were not written
      m = p.x;
      for (int i = lane + 32; i < P.nc; i += 32) m = fmaxf(m, __ldcg(part + i).x);
      m = rmax_f(m);
      const float c2 = log2e_over(P.T);
      z = 0.0;
      for (int i = lane; i < P.nc; i += 32) {
        if (i != lane) p = __ldcg(part + i);
        // a chunk of only -inf has a sum of zero, one with a NaN or +inf a NaN
        if (p.y != 0.f) z += (double)p.y * (double)ex2((p.x - m) * c2);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      if (z != z || m == INFINITY) {
        kind = 0;
        bad = SD_STATUS_NONFINITE;
      } else if (m == neg_inf()) {
        kind = 0;
      }
    }
    if (lane == 0) {
      S.kind[w] = kind;
      S.base[w] = (double)s;
      S.z[w] = kind == 1 ? z : 1.0;
      S.over[w] = (double)nm;
      S.m[w] = m;
      if (bad && P.status) atomicOr(P.status, bad);
    }
  }
  __syncthreads();
  // the slow 64-bit functions, all beams' at once
  if (warp == 0 && lane < W) {
    const double over = P.norm ? 1.0 / S.over[lane] : 1.0, base = S.base[lane] - log(S.z[lane]);
    S.base[lane] = base;
    S.over[lane] = over;
    S.c[lane] = (float)(P.inv_T * over);
    S.o[lane] = (float)(base * over);
  }
  __syncthreads();
  float size = 0.f;
  for (int w = 0; w < W; ++w)
    if (S.kind[w] == 1) size = fmaxf(size, fabsf(S.o[w]));
  // calls f(vector, its place) for the groups' largest
  auto each_vector = [&](auto f) {
#pragma unroll
    for (int u = 0; u < kEndU; ++u)
      if (tid + u * NT < all) f(held[u], tid + u * NT);
    for (int i = tid + kEndU * NT; i < all; i += NT) f(ld16(gm + (int64_t)i * 4), i);
  };
  // the best of each thread's groups, and what k of them reach
  float best = neg_inf();
  each_vector([&](const uint4 &v, int i) {
    const int w = i / per;
    if (S.kind[w] == 1) best = fmaxf(best, X.approx(w, Elt<float>::vmax(v)));
  });
  float bound = top_bound<NT>(best, k, S.keys16, &S.bound, [] {});
  // the fp32 image is off by at most three half steps of its own size and o's: the k groups
  // that reach the bound and the logits held against it by at most six together
  if (bound > kLowest) bound = fmaxf(bound - (fabsf(bound) + size) * 9.5367431640625e-7f, kLowest);
  each_vector([&](const uint4 &v, int i) {
    const int w = i / per;
    if (S.kind[w] != 1 || !(X.approx(w, Elt<float>::vmax(v)) >= bound)) return;
    float f[4];
    Elt<float>::unpack(v, f);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (X.approx(w, f[e]) >= bound) {
        const int at = atomicAdd(&S.n_list, 1);
        if (at < kSelList) S.list[at] = i * 4 + e;
      }
  });
  __syncthreads();
  bool fits = S.n_list <= kSelList;
  if (fits) {
    const int size = X.size(), items = S.n_list * size;
    for (int i = tid; i < items; i += NT) {
      const int g = S.list[i / size], w = g / (per * 4);
      const ElemRow<E> row = X.row(w);
      const int q = X.vector(row, g - w * (per * 4), i % size);
      if (q < 0) continue;
      float x[VE];
      Elt<E>::unpack(row.load(q), x);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (X.approx(w, x[e]) >= bound) X.offer(w, row.first(q) + e, x[e]);
    }
    if (tid < W && S.kind[tid] == 2) X.offer(tid, P.eos, 0.f);
    __syncthreads();
    fits = S.n_cand <= kSelList;
  }
  if (fits) rank_candidates(S, k);
  else each_beam<E>(X);
  for (int i = tid; i < k; i += NT) {
    const int64_t to = b * k + i;
    const bool have = i < S.n_best;
    const int at = have ? S.best_at[i] : -1, w = have ? at / P.V : -1, v = have ? at % P.V : -1;
    P.out_scores[to] = have ? (float)X.score(w, S.best_x[i]) : neg_inf();
    P.parents[to] = w;
    P.tokens[to] = v;
    if (P.ended) P.ended[to] = have && (S.kind[w] == 2 || v == P.eos);
  }
}

template <typename E, int U>
static cudaError_t launch_select_u(const SelectParams &P, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3((unsigned)(P.B * P.W * P.nc), 1, 1);
  cfg.blockDim = dim3(kSelNT, 1, 1);
  cudaError_t e = cudaLaunchKernelEx(&cfg, sd_beam_stream_kernel<E, U>, P);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)P.B, 1, 1);
  cfg.blockDim = dim3(kEndNT, 1, 1);
  return cudaLaunchKernelEx(&cfg, sd_beam_end_kernel<E>, P, U);
}

template <typename E>
static cudaError_t launch_select(const SelectParams &P, int U, cudaStream_t s) {
  return U == 8 ? launch_select_u<E, 8>(P, s) : launch_select_u<E, 2>(P, s);
}

static size_t select_bytes(int64_t rows, int V, int es) {
  const SelectCut c = select_cut(rows, V, es);
  return (size_t)rows * c.nc * (sizeof(float2) + kSelSets * sizeof(float)) + 16;
}

}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t dtype) {
  if (B < 0 || W < 1 || W > SD_MAX_BEAMS || V < 1 || V > SD_MAX_V) return 0;
  if (dtype != SD_F32 && dtype != SD_BF16) return 0;
  return select_bytes((int64_t)B * W, V, dtype == SD_BF16 ? 2 : 4);
}

extern "C" sd_status_t sd_beam_select(const sd_beam_select_args *a, void *stream) {
  sdv::NvtxRange nvtx_range("sd_beam_select");
  if (!a || a->B < 0 || a->W < 1 || a->W > SD_MAX_BEAMS || a->V < 1 || a->V > SD_MAX_V ||
      a->k < 1 || a->k > SD_MAX_TOP)
    return SD_ERR_INVALID_ARG;
  if (a->dtype != SD_F32 && a->dtype != SD_BF16) return SD_ERR_INVALID_ARG;
  if (!(a->T > 0.f) || !std::isfinite(a->T)) return SD_ERR_INVALID_ARG;
  if (a->eos < -1 || a->eos >= a->V || (a->finished && a->eos < 0)) return SD_ERR_INVALID_ARG;
  if (a->B == 0) return SD_OK;
  const int es = a->dtype == SD_BF16 ? 2 : 4;
  if (!a->logits || !a->scores || !a->out_scores || !a->parents || !a->tokens || !a->workspace ||
      (uintptr_t)a->logits % es || (uintptr_t)a->workspace % 16)
    return SD_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)a->B * a->W;
  const SelectCut cut = select_cut(rows, a->V, es);
  if (rows * cut.nc > INT32_MAX || a->workspace_bytes < select_bytes(rows, a->V, es))
    return SD_ERR_INVALID_ARG;
  SelectParams P = {};
  P.logits = a->logits;
  P.sb = a->logits_sb;
  P.sw = a->logits_sw;
  P.B = a->B;
  P.W = a->W;
  P.V = a->V;
  P.k = a->k;
  P.nc = cut.nc;
  P.share = cut.share;
  P.eos = a->eos;
  P.T = a->T;
  P.inv_T = 1.0 / (double)a->T;
  P.scores = a->scores;
  P.norm = a->norm;
  P.finished = a->finished;
  P.gmax = static_cast<float *>(a->workspace);   // whole 16-byte vectors; the sums follow
  P.part = reinterpret_cast<float2 *>(P.gmax + (size_t)rows * cut.nc * kSelSets);
  P.out_scores = a->out_scores;
  P.parents = a->parents;
  P.tokens = a->tokens;
  P.ended = a->ended;
  P.status = a->status;
  const cudaError_t e = es == 2 ? launch_select<__nv_bfloat16>(P, cut.U, (cudaStream_t)stream)
                                : launch_select<float>(P, cut.U, (cudaStream_t)stream);
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}

extern "C" size_t sd_beam_select_args_size(void) { return sizeof(sd_beam_select_args); }
