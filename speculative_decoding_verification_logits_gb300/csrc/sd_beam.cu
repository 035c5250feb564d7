// The k best continuations of each sequence's beams: s + x / T - log sum exp(x / T)
// over W rows of V logits, by two launches.
//
//  1. sd_beam_stream_kernel: a warp per piece of a row, of up to 4 KB.  It writes
//     the piece's (largest m, sum of 2^((x - m) c)) and the largest logit of every
//     two lanes' vectors (a group).  No beam's row is read twice, and no warp
//     waits for another.
//  2. sd_beam_end_kernel: one CTA per sequence joins the sums of each beam in whole
//     units (the same in any order), and finds from the groups' largest logits
//     alone a value that k of them reach: no candidate below it is among the k
//     best.  The groups that reach it (little more than k of them) are read
//     again, their logits that do are ranked in 64 bits.
// A sequence of which more groups or logits reach the bound than there is room
// for finds a better one from the logits of its best groups (narrow); where even
// that is not enough (thousands of equal logits at the k-th place) its beams are
// taken one by one (each_beam).
//
// Measured on the GPU: 64 x 8 rows of 151936 bf16 (a tenth of them finished), k 16,
// 33.3 us: the stream 26 (140 MB, 5.4 TB/s; without the exponentials 25.5), the end
// 7, chains of L2 and DRAM latencies, barriers and one search.  16 x 4 x 128256
// bf16 with norms 10.8 us, 1 x 4 x 32000 fp32 7.7: launches and the end.  Tried: persistent
// warps with a copy ring (40 us for the stream), one CTA of 256 threads per piece
// with block sums (28), pieces of 2, 6 and 8 KB (40, 34.1, 36.6 in all);
// groups of one, four and eight lanes (35.7, 33.5, 35).

#include "sd_rows.cuh"
#include "sd_beam.h"

namespace sdv {

constexpr int kSelNT = 128;      // threads of a streaming CTA
constexpr int kSelSet = 2;       // lanes of a group
constexpr int kSelSets = 32 / kSelSet;
constexpr int kEndNT = 512;      // threads of a sequence's end, at most
constexpr int kEndBins = 256;    // steps of the bound below the best
constexpr int kSelList = 1024;   // listed groups, and candidates, of a sequence

struct SelectParams {
  const void *logits;
  int64_t sb, sw;
  int B, W, V, k, nc, per_row, share, eos;   // per_row: streaming CTAs of a row
  float T;
  double inv_T;
  const float *scores, *norm;
  const uint8_t *finished;
  float2 *part;      // [B W][nc]: largest logit of a piece and its sum
  float *gmax;       // [B W][nc][kSelSets]: largest logit of each group
  float *out_scores;
  int32_t *parents, *tokens;
  uint8_t *ended;
  int32_t *status;
};

__device__ __forceinline__ float ld_near(const float *p) {
  float v;
  asm volatile("ld.global.ca.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int ld_near(const uint8_t *p) {
  unsigned short v;
  asm volatile("ld.global.ca.u8 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

// How rows are cut: nc pieces of `share` vectors, at most U of them per lane: eight, or two
// where that leaves SMs idle (two / eight, us: 8 x 4 x 1000 bf16 7.4 / 11.4, 1 x 4 x 32000 bf16
// 7.5 / 8.1, fp32 7.6 / 7.7, 1 x 4 x 128256 bf16 8.4 / 8.1, 64 x 8 x 151936 57 / 34: the end reads
// four times as much).
struct SelectCut {
  int U, nc, share;
};
static SelectCut select_cut(int64_t rows, int V, int es) {
  const int ve = 16 / es;
  const int nvec = (int)(((int64_t)V + ve - 1) / ve);
  SelectCut c;
  c.U = rows * nvec >= (int64_t)2 * kSelNT * sm_count() ? 8 : 2;
  c.nc = (nvec + c.U * 32 - 1) / (c.U * 32);
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

// From this temperature on x / T is taken as (x / 2) / (T / 2), the same but for logits that are zero
// to it: the difference of two logits may pass fp32's range, and at lower ones its exponential is zero.
constexpr float kFarT = 1.329227995784915872903807060280344576e36f;   // 2^120

// Terms 2^((x - m) c), the differences first: the term of m itself is 1 to the bit.
template <bool HALVES>
struct BeamExp {
  uint64_t o, c;
  __device__ __forceinline__ BeamExp(float m, float T) {
    constexpr float unit = HALVES ? 0.5f : 1.f;
    const float s = m == neg_inf() ? 0.f : -m * unit, k = log2e_over(T * unit);
    o = pk2(s, s);
    c = pk2(k, k);
  }
  template <bool FAR>
  __device__ __forceinline__ void pair(uint64_t x, float &a, float &b) const {
    upk2(mul2(HALVES ? fma2(x, pk2(0.5f, 0.5f), o) : add2(x, o), c), a, b);
    a = ex2(a);
    b = ex2(b);
  }
};

// A warp per piece, in registers: warps share nothing, and CTAs are small, so that an SM asks
// for new pieces whenever one of its warps is done.  The rows' scores come
// through L1, where the CTAs before left them.  Registers for ten CTAs per SM
// (64 x 8 x 151936 bf16 33.1 us; the compiler's eight 1.4 more, eleven 1).
template <typename E, int U, bool HALVES>
__global__ void __launch_bounds__(kSelNT, 10) sd_beam_stream_kernel(const SelectParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x / P.per_row, w = n % P.W;
  const int piece = blockIdx.x % P.per_row * (kSelNT / 32) + (threadIdx.x >> 5);
  if (piece >= P.nc) return;
  // a beam that is dead or finished has no candidates of its own
  if (!(fabsf(ld_near(P.scores + n)) < INFINITY)) return;
  if (P.finished && ld_near(P.finished + n)) return;
  const ElemRow<E> row(P.logits, (n / P.W) * P.sb + w * P.sw, P.V);
  const int q0 = piece * P.share, q1 = min(q0 + P.share, row.nvec);
  const int lo = max(q0, row.lo()), hi = min(q1, row.hi());
  const uint8_t *src = row.grid(q0 + lane);
  const uint32_t inf = Elt<E>::kNegInfWord;
  uint4 v[U];
  if (row.hp == 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + lane + u * 32;
      v[u] = make_uint4(inf, inf, inf, inf);
      if (q >= lo && q < hi) v[u] = ld16(src + u * 512);
    }
  } else {
    uint4 next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + lane + u * 32;
      v[u] = next[u] = make_uint4(inf, inf, inf, inf);
      if (q >= lo && q < hi) {
        v[u] = ld16(src + u * 512);
        next[u] = ld16(src + u * 512 + 16);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = row.cut(v[u], next[u]);
  }
  if (lo > q0 || hi < q1) {   // the row's first or last vectors
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = q0 + lane + u * 32;
      if (q < q1 && (q < lo || q >= hi)) v[u] = row.load_edge(q);
    }
  }
  float m = VecExp<E>::template largest<U>(v);
#pragma unroll
  for (int o = 1; o < kSelSet; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int64_t at = (int64_t)n * P.nc + piece;
  if (lane % kSelSet == 0) P.gmax[at * kSelSets + lane / kSelSet] = m;
  m = rmax_f(m);
  // a beam that is sure of a token has a sum of exactly one
  const BeamExp<HALVES> B(m, P.T);
  uint64_t acc = 0ull;
#pragma unroll
  for (int u = 0; u < U; ++u) acc = VecExp<E>::template sum<true>(v[u], B, acc);
  float x, y;
  upk2(acc, x, y);
  const float z = warp_sum(x + y);
  if (lane == 0) P.part[at] = make_float2(m, z);
}

// A double's order as an unsigned integer (never a NaN here).
__device__ __forceinline__ unsigned long long dord(double x) {
  const long long i = __double_as_longlong(x + 0.0);
  return (unsigned long long)i ^ (i < 0 ? ~0ull : 1ull << 63);
}

// ln z for z >= 1, to 2^-28: z = 2^e m with m in [3/4, 3/2) and, with r = (m - 1) / (m + 1),
// ln m = 2 atanh r = 2 (r + r^3 / 3 + r^5 / 5 + ...), whose terms beyond r^11 / 11 are below
// 2^-33; ln 2 as 11357 / 2^14, whose multiples are exact, and the rest.  The
// same in fp64 took 0.9 us longer.
__device__ __forceinline__ ff ff_log(ff z) {
  const int e = (__float_as_int(z.hi) + 0x00400000 >> 23) - 127;
  const float scale = __int_as_float(127 - e << 23);
  const ff m = ff{z.hi * scale, z.lo * scale};
  const ff num = ff_add_f(m, -1.f), den = ff_add_f(m, 1.f);
  const float r = __fdiv_rn(num.hi, den.hi);
  const float rest = __fdiv_rn(fmaf(-r, den.hi, num.hi) + fmaf(-r, den.lo, num.lo), den.hi);
  const float q = r * r;
  const float p =
      q * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 1.f / 11.f, 1.f / 9.f), 1.f / 7.f), 0.2f), 1.f / 3.f);
  const ff sum = two_sum((float)e * 0.69317626953125f, 2.f * r);
  return fast_two_sum(sum.hi,
                      sum.lo + fmaf((float)e, -2.9088971e-5f, 2.f * fmaf(r, p, rest)));
}

// How far d below the best of a sequence, in bins: of d + 1 the exponent and the four leading bits
// (steps of 1/16 at first, of 1/2 from 7 on, 2^16 in all; the last bin holds the rest).
__device__ __forceinline__ int below_bin(float d) {
  return min(__float_as_int(d + 1.f) - 0x3f800000 >> 19, kEndBins - 1);
}
// What everything in the bins up to this one reaches.
__device__ __forceinline__ float bin_edge(float top, int bin) {
  return bin < kEndBins - 1 ? top - (__int_as_float((bin + 1 << 19) + 0x3f800000) - 1.f) : kLowest;
}

// What a sequence's end holds on chip.
struct SelectEnd {
  // a beam: 0 offers nothing, 1 live, 2 finished; its score less the log of its sum
  int kind[SD_MAX_BEAMS];
  double base[SD_MAX_BEAMS];
  double norm[SD_MAX_BEAMS];          // where there are any
  int top[SD_MAX_BEAMS];              // its largest logit, ordered
  unsigned hi[SD_MAX_BEAMS];          // its sum in units of 2^-10 and of 2^-31
  unsigned lo[SD_MAX_BEAMS];
  int bad[SD_MAX_BEAMS];
  // an fp32 image of the ranked score, max((x - m) c + o, lowest): m, c, o, and the size of
  // what entered o (negative: the beam's logits are not read)
  float4 image[SD_MAX_BEAMS];
  int list[kSelList];                 // groups: beam in the upper half, piece and place
  unsigned long long key[kSelList];   // candidates: the order of their ranked scores,
  int at[kSelList];                   // beam and token (kTokenBits),
  float score[kSelList];
  unsigned long long best_key[SD_MAX_TOP];   // the k best, in order
  int best_at[SD_MAX_TOP];
  float best_score[SD_MAX_TOP];
  int hist[kEndBins];                 // threads by how far their best lies below the best
  int best;
  int warp_n[kEndNT / 32];
  float bound;
  float margin;                       // the largest size of what entered an o
  int n_list, n_cand, n_best;
  int wild;                           // an image leaves fp32: it prunes nothing
  unsigned long long kth;             // of kth_largest: the bits so far
  int rank, count;

  // by the first warp: the bin that holds the k-th of those counted, kEndBins where they are fewer
  __device__ __forceinline__ int bin_of_rank(int k) const {
    constexpr int J = kEndBins / 32;
    const int lane = threadIdx.x & 31;
    int n[J], upto = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) upto += n[j] = hist[lane * J + j];
    const int here = upto;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      upto += lane >= o ? y : 0;
    }
    const unsigned enough = __ballot_sync(0xffffffffu, upto >= k);
    int bin = kEndBins, at = upto - here;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      at += n[j];
      bin = bin == kEndBins && at >= k ? lane * J + j : bin;
    }
    return enough ? __shfl_sync(0xffffffffu, bin, __ffs(enough) - 1) : kEndBins;
  }
};
__device__ __forceinline__ float loosened(float bound, float size) {
  return bound > kLowest ? fmaxf(bound - (fabsf(bound) + size) * 3.814697265625e-6f, kLowest)
                         : bound;
}
constexpr int kTokenBits = 18;
static_assert(SD_MAX_V <= 1 << kTokenBits, "a token and a beam fit an int");

template <typename E, int U, bool NORMS>
struct EndView {
  static constexpr int VE = Elt<E>::kPerVec;
  static constexpr int kSize = kSelSet * U;   // vectors of a group
  const SelectParams &P;
  SelectEnd &S;
  int b;
  __device__ __forceinline__ EndView(const SelectParams &P_, SelectEnd &S_)
      : P(P_), S(S_), b(blockIdx.x) {}
  __device__ __forceinline__ ElemRow<E> row(int w) const {
    return ElemRow<E>(P.logits, b * P.sb + w * P.sw, P.V);
  }
  __device__ __forceinline__ const float *groups(int w) const {
    return P.gmax + ((int64_t)b * P.W + w) * P.nc * kSelSets;
  }
  // the row's vector that is number i of group g, or -1
  __device__ __forceinline__ int vector(const ElemRow<E> &r, int g, int i) const {
    const int at = g % kSelSets * kSelSet + i % kSelSet + i / kSelSet * 32;
    const int q = g / kSelSets * P.share + at;
    return at < P.share && q < r.nvec ? q : -1;
  }
  static __device__ __forceinline__ float approx(const float4 &f, float x) {
    return x > neg_inf() ? fmaxf(fmaf(x - f.x, f.y, f.z), kLowest) : neg_inf();
  }
  // calls f(beam, first token, logits) for the vectors of the listed groups
  template <typename F>
  __device__ __forceinline__ void each_listed(F f) const {
    const int items = S.n_list * kSize;
#pragma unroll 1
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
      const int g = S.list[i / kSize], w = g >> 16;
      const ElemRow<E> r = row(w);
      const int q = vector(r, g & 0xffff, i % kSize);
      if (q < 0) continue;
      float x[VE];
      Elt<E>::unpack(r.load(q), x);
      f(w, r.first(q), x);
    }
  }
  // what reaches the bound in the listed groups, and the finished beams, as candidates;
  // whether there was room for them.  Ends with a barrier.
  __device__ __forceinline__ bool offer_listed(float bound) const {
    each_listed([&](int w, int v, const float(&x)[VE]) {
      const float4 f = S.image[w];
      unsigned pass = 0u;
#pragma unroll
      for (int e = 0; e < VE; ++e) pass |= (approx(f, x[e]) >= bound ? 1u : 0u) << e;
      // once there is no room left nothing more is offered
      while (pass && *(volatile int *)&S.n_cand <= kSelList) {
        const int j = __ffs(pass) - 1;
        pass &= pass - 1;
        float y = x[0];
#pragma unroll
        for (int e = 1; e < VE; ++e) y = j == e ? x[e] : y;
        offer(w, v + j, y);
      }
    });
    if (threadIdx.x < P.W && S.kind[threadIdx.x] == 2) offer(threadIdx.x, P.eos, 0.f);
    __syncthreads();
    return S.n_cand <= kSelList;
  }
  // the score of a live beam's token
  __device__ __forceinline__ double score(int w, float x) const {
    return S.base[w] + ((double)x - (double)S.image[w].x) * P.inv_T;
  }
  // What ranks it: the quotient itself, so that equal ones tie (5 / 5 and 49 / 49, say).  The product
  // with 1 / norm, which may round to a neighbour, is 0.5 us faster (16 x 4 x 128256 bf16).
  __device__ __forceinline__ double ranked(int w, double c) const {
    return NORMS ? c / S.norm[w] : c;
  }
  // a candidate; logits of a finished beam are not looked at
  __device__ __forceinline__ void offer(int w, int v, float x) const {
    const double c = S.kind[w] == 1 ? score(w, x) : S.base[w];
    const int i = atomicAdd(&S.n_cand, 1);
    if (i < kSelList) {
      S.key[i] = dord(ranked(w, c));
      S.at[i] = w << kTokenBits | v;
      S.score[i] = (float)c;
    }
  }
};

// The k best of the candidates, in order, into S.best_*: a warp counts how many are
// better than one, and no two are alike.  Begins and ends with a barrier.
__device__ __forceinline__ void rank_candidates(SelectEnd &S, int k) {
  __syncthreads();
  const int n = min(S.n_cand, kSelList), lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = threadIdx.x >> 5; i < n; i += blockDim.x / 32) {
    const unsigned long long key = S.key[i];
    const int at = S.at[i];
    int above = 0;
#pragma unroll 1
    for (int j = lane; j < n; j += 32) {
      const unsigned long long other = S.key[j];
      above += other > key | (other == key & S.at[j] < at);
    }
    __syncwarp();
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0 && above < k) {
      S.best_key[above] = key;
      S.best_at[above] = at;
      S.best_score[above] = S.score[i];
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
  for (int i = 0; i < blockDim.x / 32; ++i) n += S.warp_n[i];
  return n;
}

// The key of the k-th largest of those that each(f) calls f(key) for, 0 where they are
// fewer: eight bits at a time.
template <typename F>
__device__ __forceinline__ unsigned long long kth_largest(SelectEnd &S, int k, int bits, F each) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    S.kth = 0ull;
    S.rank = k;
  }
#pragma unroll 1
  for (int shift = bits - 8; shift >= 0; shift -= 8) {
    if (tid < kEndBins) S.hist[tid] = 0;
    __syncthreads();
    const unsigned long long known = S.kth;
    const int rank = S.rank;
    each([&](unsigned long long key) {
      // the largest digit in the first bin
      if (((key ^ known) >> shift) >> 8 == 0ull) atomicAdd(&S.hist[255 - (int)(key >> shift & 255u)], 1);
    });
    __syncthreads();
    if (tid < 32) {
      const int bin = S.bin_of_rank(rank);
      int above = 0;
      for (int i = tid; i < min(bin, kEndBins); i += 32) above += S.hist[i];
      __syncwarp();
      above = __reduce_add_sync(0xffffffffu, above);
      if (tid == 0) {
        S.rank = bin < kEndBins ? rank - above : 0;
        S.kth = known | (unsigned long long)(255 - min(bin, 255)) << shift;
      }
    }
    __syncthreads();
    if (S.rank == 0) return 0ull;
  }
  return S.kth;
}
static_assert(kEndBins == 256, "a digit of eight bits per bin");

// Where more groups or logits reach the bound than there is room for: the groups from the best
// down that there is room for, then a bound from their logits instead of their largest.
// Whether that was enough: not where the k-th lies below those groups (or more than 2^16 below
// the best), nor where more logits than there is room for lie in its bin.
template <typename E, int U, bool NORMS>
__device__ __noinline__ bool narrow(const EndView<E, U, NORMS> &X, float top, float margin) {
  constexpr int VE = Elt<E>::kPerVec;
  const int NT = blockDim.x;
  SelectEnd &S = X.S;
  const int tid = threadIdx.x, ng = X.P.nc * kSelSets, W = X.P.W;
  const auto each_group = [&](auto f) {
#pragma unroll 1
    for (int i = tid; i < W * ng; i += NT) {
      const int w = i / ng;
      const float4 g = S.image[w];
      if (g.w >= 0.f) f(w, i - w * ng, X.approx(g, ld_float(X.groups(0) + i)));
    }
  };
  const auto count = [&](float a) {
    const int bin = below_bin(top - a);
    if (bin < kEndBins - 1) atomicAdd(&S.hist[bin], 1);
  };
  const auto clear = [&] {
    __syncthreads();
    if (tid < kEndBins) S.hist[tid] = 0;
    if (tid == 0) S.n_cand = 0;
    __syncthreads();
  };
  // in every thread
  const auto bin_of_rank = [&](int k) {
    __syncthreads();
    const int bin = tid < 32 ? S.bin_of_rank(k) : 0;
    if (tid == 0) S.count = bin;
    __syncthreads();
    return S.count;
  };
  clear();
  if (tid == 0) S.n_list = 0;
  each_group([&](int, int, float a) { count(a); });
  const int past = min(bin_of_rank(kSelList + 1), kEndBins - 1);   // the first bin without room
  if (past == 0) return false;
  const float room = loosened(bin_edge(top, past - 1), margin);
  each_group([&](int w, int g, float a) {
    if (!(a >= room)) return;
    const int at = atomicAdd(&S.n_list, 1);
    if (at < kSelList) S.list[at] = w << 16 | g;
  });
  clear();
  if (S.n_list > kSelList) return false;
  X.each_listed([&](int w, int, const float(&x)[VE]) {
    const float4 f = S.image[w];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float a = X.approx(f, x[e]);
      if (a >= room) count(a);
    }
  });
  const int bin = bin_of_rank(X.P.k);
  if (bin >= kEndBins - 1) return false;
  const float bound = loosened(bin_edge(top, bin), margin);
  return bound >= room && X.offer_listed(bound);
}

// The beams one by one, whatever their logits: the k best of one by value, then
// by index, join the k best so far.
//  - v*, the k-th largest of its groups' largest;
//  - the logits above v* lie in fewer than k groups.  If they are k or more,
//    the key (value, index) of the k-th bounds them;
//  - if they are fewer, logits equal to v* fill up, lowest index first, from the
//    row's beginning until there are enough; so do other logits of the k-th's
//    score, where there are any.
template <typename E, int U, bool NORMS>
__device__ __noinline__ void each_beam(const EndView<E, U, NORMS> &X) {
  constexpr int VE = EndView<E, U, NORMS>::VE, size = EndView<E, U, NORMS>::kSize;
  const int NT = blockDim.x;
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
      S.score[i] = S.best_score[i];
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
    const unsigned r = (unsigned)kth_largest(S, k, 32, [&](auto f) {
      for (int i = tid; i < ng; i += NT) f((unsigned)ford(ld_float(gm + i)) ^ 0x80000000u);
    });
    const float least = fdeord((int)(max(r, low) ^ 0x80000000u));
    for (int i = tid; i < ng; i += NT)
      if (ld_float(gm + i) > least) {   // fewer than k
        const int at = atomicAdd(&S.n_list, 1);
        if (at < kSelList) S.list[at] = i;
      }
    __syncthreads();
    const int items = min(S.n_list, kSelList) * size;
    auto above = [&](unsigned long long from, auto f) {
      for (int i = tid; i < items; i += NT) {
        const int q = X.vector(row, S.list[i / size], i % size);
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
    if (more >= k)
      from = kth_largest(S, k, 64, [&](auto f) {
        above(0ull, [&](float x, int v) { f(top_key(x, v)); });
      });
    // the k-th logit, and those that rank the same in 64 bits: others than itself only where its
    // neighbours do (logits near zero, temperatures that leave no difference)
    const float kth = more >= k ? key_value(from) : least;
    const auto ranked = [&](float x) { return X.ranked(w, X.score(w, x)); };
    const double c = X.score(w, kth), rank = X.ranked(w, c);
    const bool alone = ranked(nextafterf(kth, -INFINITY)) < rank &&
                       ranked(nextafterf(kth, INFINITY)) > rank;
    const double near = alone ? 0.0 : (fabs(S.base[w]) + fabs(c) + 1.0) * 3.6e-15 / P.inv_T;
    const auto ties = [&](float x) {
      return x == kth || (!alone && fabs((double)x - (double)kth) <= near && ranked(x) == rank);
    };
    if (more >= k && alone) {
      above(from, [&](float x, int v) { X.offer(w, v, x); });
    } else {
      int better = 0;
      above(0ull, [&](float x, int v) {
        if (!(x > kth) || ties(x)) return;
        X.offer(w, v, x);
        ++better;
      });
      int need = k - block_count(S, better);
      for (int q0 = 0; q0 < row.nvec && need > 0; q0 += NT) {
        float x[VE];
        unsigned same = 0u;
        if (q0 + tid < row.nvec) {
          Elt<E>::unpack(row.load(q0 + tid), x);
#pragma unroll
          for (int e = 0; e < VE; ++e) same |= (x[e] > neg_inf() && ties(x[e]) ? 1u : 0u) << e;
        }
        // places in the order of the threads
        const int n = __popc(same);
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
          if (same >> e & 1u) {
            if (before < need) X.offer(w, row.first(q0 + tid) + e, x[e]);
            ++before;
          }
        need -= all;
      }
    }
    rank_candidates(S, k);
  }
}

// NT threads, CTAs of them per SM: 512 and one where every sequence has an SM of its own, 256 and
// four where there are more (us: 64 x 8 x 151936 bf16 33 / 44, 256 x 4 x 128256 57 / 53, 2000 x 8 x
// 32000 251 / 201; 512 and two 37, 55, 232).
template <typename E, int U, int NT, int CTAS, bool NORMS>
__global__ void __launch_bounds__(NT, CTAS) sd_beam_end_kernel(const SelectParams P) {
  constexpr int NW = NT / 32, kEndU = NT / 64, kEndPieces = NT / 128;
  static_assert(NT >= kEndBins && NT <= kEndNT, "a thread per bin, a count per warp");
  __shared__ SelectEnd S;
  const EndView<E, U, NORMS> X(P, S);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = P.W, k = P.k;
  const int64_t b = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the groups' largest, vectors of four held by the threads
  const int per = P.nc * kSelSets / 4, all = W * per;
  const float *gm = X.groups(0);
  uint4 held[kEndU];
#pragma unroll
  for (int u = 0; u < kEndU; ++u)
    if (tid + u * NT < all) held[u] = ld16(gm + (int64_t)(tid + u * NT) * 4);
  // a lane of the second warp per beam
  const bool mine = warp == 1 && lane < W;
  float s = neg_inf(), nm = 1.f;
  int ended = 0;
  if (mine) {
    s = ld_float(P.scores + b * W + lane);
    if (NORMS) nm = ld_float(P.norm + b * W + lane);
    if (P.finished) ended = ld1(P.finished + b * W + lane);
  }
  // 32 pieces of a beam per warp.  Of a beam that is not read they may be anything.
  const int blocks = (P.nc + 31) / 32;
  const auto load_piece = [&](int i) {
    const int w = i / blocks, at = i % blocks * 32 + lane;
    return at < P.nc ? __ldcg(P.part + (b * W + w) * P.nc + at) : make_float2(neg_inf(), 0.f);
  };
  float2 piece[kEndPieces];
#pragma unroll
  for (int u = 0; u < kEndPieces; ++u)
    if (warp + u * NW < W * blocks) piece[u] = load_piece(warp + u * NW);
  const auto each_block = [&](auto f) {
#pragma unroll
    for (int u = 0; u < kEndPieces; ++u)
      if (warp + u * NW < W * blocks) f((warp + u * NW) / blocks, piece[u]);
#pragma unroll 1
    for (int i = warp + kEndPieces * NW; i < W * blocks; i += NW) f(i / blocks, load_piece(i));
  };
  if (tid == 0) S.n_list = S.n_cand = S.wild = 0;
  if (tid < kEndBins) S.hist[tid] = 0;
  if (tid < SD_MAX_BEAMS) {
    S.best = ford(neg_inf());
    S.top[tid] = ford(neg_inf());
    S.hi[tid] = S.lo[tid] = 0u;
    S.bad[tid] = 0;
  }
  __syncthreads();
  // their largest logit, then their sums in whole units, which come out the same in any order
  each_block([&](int w, const float2 &p) {
    const int m = __reduce_max_sync(0xffffffffu, ford(p.x));
    if (lane == 0) atomicMax(&S.top[w], m);
  });
  __syncthreads();
  const float unit = P.T >= kFarT ? 0.5f : 1.f, c2 = log2e_over(P.T * unit);
  each_block([&](int w, const float2 &p) {
    // at most 2^11; a piece with a NaN or +inf has a sum of NaN
    const float t = p.y == 0.f ? 0.f : p.y * ex2((p.x * unit - fdeord(S.top[w]) * unit) * c2);
    const float units = t * 1024.f, whole = truncf(units);
    const bool bad = __any_sync(0xffffffffu, !(t <= 4096.f));
    const unsigned hi = __reduce_add_sync(0xffffffffu, __float2uint_rn(whole));
    const unsigned lo = __reduce_add_sync(0xffffffffu, __float2uint_rn((units - whole) * 2097152.f));
    if (lane == 0) {
      atomicAdd(&S.hi[w], hi);
      atomicAdd(&S.lo[w], lo);
      if (bad) S.bad[w] = 1;
    }
  });
  __syncthreads();
  ff z = ff{1.f, 0.f};
  if (mine) {
    int kind = s == neg_inf() ? 0 : ended ? 2 : 1, bad = 0;
    const float m = fdeord(S.top[lane]);
    if (!(fabsf(s) < INFINITY) && s != neg_inf()) {
      kind = 0;
      bad = SD_STATUS_NONFINITE;
    } else if (kind && !(nm > 0.f && nm < INFINITY)) {
      kind = 0;
      bad = SD_STATUS_BAD_PENALTY;
    } else if (kind == 1 && (S.bad[lane] || m == INFINITY)) {
      kind = 0;
      bad = SD_STATUS_NONFINITE;
    } else if (kind == 1 && m == neg_inf()) {
      kind = 0;
    }
    if (kind == 1) {   // the units' first 24 bits, and the others
      const unsigned hi = S.hi[lane];
      const float up = __uint2float_rz(hi), low = __uint2float_rn(hi - (unsigned)up);
      z = fast_two_sum(up * 9.765625e-4f,
                       fmaf(low, 9.765625e-4f, __uint2float_rn(S.lo[lane]) * 4.656612873077393e-10f));
    }
    S.kind[lane] = kind;
    // an fp32 image of what follows in 64 bits
    const float over = __fdividef(1.f, nm);
    const float log_z = 0.693147180559945309f * __log2f(z.hi);
    const float4 f = make_float4(m, __fdividef(over, P.T), (s - log_z) * over,
                                 kind == 1 ? (fabsf(s) + log_z + 1.f) * over : -1.f);
    S.image[lane] = f;
    // where a factor or a difference of logits passes fp32, or a quotient is too small for it (and
    // zero for divisors from 2^126 on), the image says nothing
    if (kind == 1 && !(f.y >= 1.1754943508222875e-38f && f.y < INFINITY && f.w < INFINITY &&
                       m - kLowest < INFINITY))
      S.wild = 1;
    if (bad && P.status) atomicOr(P.status, bad);
  }
  __syncthreads();
  // the best of each thread's groups
  const float inv_per = 1.f / (float)per;
  float best = neg_inf(), size = 0.f;
#pragma unroll
  for (int u = 0; u < kEndU; ++u) {
    const int i = tid + u * NT;
    if (u * NT < all) {
      const float4 f = S.image[min((int)(((float)i + 0.5f) * inv_per), W - 1)];
      const float x = X.approx(f, Elt<float>::vmax(held[u]));
      if (i < all && f.w >= 0.f) best = fmaxf(best, x);
    }
  }
#pragma unroll 1
  for (int i = tid + kEndU * NT; i < all; i += NT) {
    const float4 f = S.image[i / per];
    if (f.w >= 0.f) best = fmaxf(best, X.approx(f, Elt<float>::vmax(ld16(gm + (int64_t)i * 4))));
  }
  if (tid < W) size = S.image[tid].w;
  const int most = __reduce_max_sync(0xffffffffu, ford(best));
  if (lane == 0) atomicMax(&S.best, most);
  __syncthreads();
  // what k of them reach; no bound is known where the k-th lies more than 2^16 below the best
  const float top = fdeord(S.best);
  if (best > neg_inf()) atomicAdd(&S.hist[below_bin(top - best)], 1);
  __syncthreads();
  if (warp == 0) {
    const int bin = S.bin_of_rank(k);
    size = rmax_f(size);
    float bound = bin < kEndBins ? bin_edge(top, bin) : kLowest;
    // the image is off by less than 2^-19 of its own size and of what entered o (quotients of two
    // steps, a logarithm of 2^-22 near one): the groups that reach the bound and the logits
    // held against it by at most twice that
    if (lane == 0) {
      S.margin = size;
      S.bound = loosened(bound, size);
    }
  } else if (mine) {   // meanwhile the beams' numbers in 64 bits
    const ff log_z = ff_log(z);
    S.base[lane] = ((double)s - (double)log_z.hi) - (double)log_z.lo;
    if (NORMS) S.norm[lane] = (double)nm;
  }
  __syncthreads();
  const float bound = S.bound;
  if (best >= bound) {
    const auto list = [&](const uint4 &v, int i, int w) {
      const float4 f = S.image[w];
      if (f.w < 0.f || !(X.approx(f, Elt<float>::vmax(v)) >= bound)) return;
      const float x[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                          __uint_as_float(v.w)};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (X.approx(f, x[e]) >= bound && *(volatile int *)&S.n_list <= kSelList) {
          const int at = atomicAdd(&S.n_list, 1);
          if (at < kSelList) S.list[at] = w << 16 | ((i - w * per) * 4 + e);
        }
    };
#pragma unroll
    for (int u = 0; u < kEndU; ++u)
      if (tid + u * NT < all) list(held[u], tid + u * NT, (int)((tid + u * NT + 0.5f) * inv_per));
#pragma unroll 1
    for (int i = tid + kEndU * NT; i < all; i += NT) list(ld16(gm + (int64_t)i * 4), i, i / per);
  }
  __syncthreads();
  bool fits = S.n_list <= kSelList;
  if (fits) fits = X.offer_listed(bound);
  if (!fits) fits = narrow<E, U, NORMS>(X, top, S.margin);
  if (S.wild) fits = false;
  if (fits) rank_candidates(S, k);
  else each_beam<E, U, NORMS>(X);
  for (int i = tid; i < k; i += NT) {
    const int64_t to = b * k + i;
    const bool have = i < S.n_best;
    const int at = have ? S.best_at[i] : -1;
    const int w = at >> kTokenBits, v = have ? at & ((1 << kTokenBits) - 1) : -1;
    P.out_scores[to] = have ? S.best_score[i] : neg_inf();
    P.parents[to] = w;
    P.tokens[to] = v;
    if (P.ended) P.ended[to] = have && (S.kind[w] == 2 || v == P.eos);
  }
}

template <typename E, int U, bool NORMS>
static cudaError_t launch_select_end(const SelectParams &P, cudaLaunchConfig_t &cfg) {
  cfg.gridDim = dim3((unsigned)P.B, 1, 1);
  if (P.B <= sm_count()) {
    cfg.blockDim = dim3(512, 1, 1);
    return cudaLaunchKernelEx(&cfg, sd_beam_end_kernel<E, U, 512, 1, NORMS>, P);
  }
  cfg.blockDim = dim3(256, 1, 1);
  return cudaLaunchKernelEx(&cfg, sd_beam_end_kernel<E, U, 256, 4, NORMS>, P);
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
  cfg.gridDim = dim3((unsigned)(P.B * P.W * P.per_row), 1, 1);
  cfg.blockDim = dim3(kSelNT, 1, 1);
  const cudaError_t e = P.T >= kFarT ? cudaLaunchKernelEx(&cfg, sd_beam_stream_kernel<E, U, true>, P)
                                     : cudaLaunchKernelEx(&cfg, sd_beam_stream_kernel<E, U, false>, P);
  if (e != cudaSuccess) return e;
  return P.norm ? launch_select_end<E, U, true>(P, cfg) : launch_select_end<E, U, false>(P, cfg);
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
  if (!(a->T >= 1.17549435e-38f) || !std::isfinite(a->T)) return SD_ERR_INVALID_ARG;
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
  P.per_row = (cut.nc + kSelNT / 32 - 1) / (kSelNT / 32);
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
