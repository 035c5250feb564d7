// The top logits of each row and the log-sum-exp of all others: what a
// teacher gives to a distillation step.
//
// One cluster of cs CTAs per row, which holds it in shared memory:
//  1. every thread keeps the best logit of its own vectors; threads side by
//     side form groups.  The k-th best of a set of groups' maxima bounds the
//     k-th best logit from below: k groups hold a logit at least as good.  Two
//     such bounds are taken, the better one is used: the largest over the CTAs
//     of each CTA's k-th best group, and the smallest over the CTAs of each
//     CTA's ceil(k / cs)-th best.
//  2. logits at or above the bound (little more than k of them where the
//     large logits are spread over the row) go to a list and are set to -inf
//     in the share, whose rest is summed: running (largest, sum of
//     2^((x - largest) c)).  The first CTA ranks the list, writes the first k and
//     adds what is left to the sum in rank order, so that nothing depends on
//     the order in which the list was filled.
// A row whose logits at the bound do not fit the list (large logits all in a
// few groups) raises its bound first by halving the range of keys until at
// least k and at most a list of logits are left.
// Keys order logits by value, then by lower index: (ordered image of the
// value, ~index).  HBM-bound: a row is 2 or 4 V bytes, the results 8 k + 4.

#include "sd_rows.cuh"

namespace sdv {

constexpr int kTopNT = 256;
constexpr int kTopNW = kTopNT / 32;
constexpr int kTopU = 4;          // vectors at a time per thread
constexpr int kTopList = 1024;    // listed logits of a row

struct TopParams {
  const void *logits;
  int64_t stride;
  int N, V, k, cs;
  float T;
  float *vals;
  int32_t *ids;
  float *rest;
};

// What the CTAs of a row tell one another.
struct TopStat {
  unsigned long long kth, share;  // keys of the k-th and the ceil(k / cs)-th best group
  float m;                        // largest logit
};

__device__ __forceinline__ unsigned long long top_key(float x, int i) {
  return ((unsigned long long)((unsigned)ford(x) ^ 0x80000000u) << 32) | (unsigned)~i;
}
__device__ __forceinline__ int key_index(unsigned long long key) { return (int)~(unsigned)key; }
__device__ __forceinline__ float key_value(unsigned long long key) {
  return fdeord((int)((unsigned)(key >> 32) ^ 0x80000000u));
}

template <typename E>
__global__ void __launch_bounds__(kTopNT, kHeldCtas) sd_top_kernel(const TopParams P) {
  constexpr int VE = Elt<E>::kPerVec, NT = kTopNT, NW = kTopNW;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  row_cluster_arrive();
  extern __shared__ uint4 held[];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = P.cs, rank = (int)cluster.block_rank(), n = blockIdx.x / cs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ unsigned long long list[kTopList];    // the groups, then this CTA's listed keys
  __shared__ TopStat stat[kHeldMaxCS];
  __shared__ float2 sums[kHeldMaxCS];
  __shared__ int listed[kHeldMaxCS];
  __shared__ int counted[2][kHeldMaxCS];
  __shared__ float red[NW], redz[NW];
  __shared__ unsigned long long kth, share;
  __shared__ int n_list;
  Held<E> H(P.logits, (int64_t)n * P.stride, P.V, rank, cs, smem_u32(held));
  H.template fetch<NT>();
  const float c2 = log2e_over(P.T);
  cp_wait<0>();

  // 1. the best logit of each thread's own vectors, which it copied itself
  float m = neg_inf();
  int mi = -1;
  for (int i = tid; i < H.n; i += NT) {
    const float x = Elt<E>::vmax(H.get(i));
    if (x > m) {
      m = x;
      mi = i;
    }
  }
  // keyed by the last index its vector could give: no better than the logit itself
  unsigned long long key = mi >= 0 ? top_key(m, H.row.first(H.qa + mi) + VE - 1) : 0ull;
  const int side = P.k > 64 ? 1 : P.k > 32 ? 2 : 4;   // threads of a group
  for (int o = 1; o < side; o <<= 1) {
    const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
    key = other > key ? other : key;
  }
  const int groups = NT / side;
  if (tid % side == 0) list[tid / side] = key;
  m = warp_max(m);
  if (lane == 0) red[warp] = m;
  if (tid == 0) {
    kth = share = 0ull;
    n_list = 0;
  }
  __syncthreads();
  const int ks = (P.k + cs - 1) / cs;
  if (tid < groups) {
    const unsigned long long g = list[tid];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < groups; ++j) above += list[j] > g;
    if (g != 0ull) {
      if (above == P.k - 1) kth = g;
      if (above == ks - 1) share = g;
    }
  }
  float cm = neg_inf();
#pragma unroll
  for (int w = 0; w < NW; ++w) cm = fmaxf(cm, red[w]);
  __syncthreads();
  row_cluster_wait();
  if (tid < cs) {
    TopStat *s = cluster.map_shared_rank(&stat[rank], tid);
    s->kth = kth;
    s->share = share;
    s->m = cm;
  }
  cluster.sync();
  unsigned long long bound = 0ull, least = ~0ull;
  float M = neg_inf();
  for (int r = 0; r < cs; ++r) {
    bound = stat[r].kth > bound ? stat[r].kth : bound;
    least = stat[r].share < least ? stat[r].share : least;
    M = fmaxf(M, stat[r].m);
  }
  bound = least > bound ? least : bound;
  // nothing below every finite logit is ever chosen
  const unsigned long long lowest = top_key(-3.402823466e38f, P.V);
  bound = bound > lowest ? bound : lowest;

  // calls f(logit, key, vector, place) for what reaches the bound
  auto reaching = [&](unsigned long long least_key, auto f) {
    const float bx = key_value(least_key);
    for (int i = tid; i < H.n; i += NT) {
      const uint4 v = H.get(i);
      if (!(Elt<E>::vmax(v) >= bx)) continue;
      float x[VE];
      Elt<E>::unpack(v, x);
      const int e0 = H.row.first(H.qa + i);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const unsigned long long k = top_key(x[e], e0 + e);
        if (x[e] >= bx && k >= least_key) f(k, i * VE + e);
      }
    }
  };
  // how many reach it in the whole row
  int step = 0;
  auto count = [&](unsigned long long least_key) {
    int here = 0;
    reaching(least_key, [&](unsigned long long, int) { ++here; });
    here = __reduce_add_sync(0xffffffffu, here);
    if (tid == 0) n_list = 0;
    __syncthreads();
    if (lane == 0) atomicAdd(&n_list, here);
    __syncthreads();
    if (tid < cs) *cluster.map_shared_rank(&counted[step & 1][rank], tid) = n_list;
    cluster.sync();
    int all = 0;
    for (int r = 0; r < cs; ++r) all += counted[step & 1][r];
    ++step;
    return all;
  };
  // 2. list what reaches the bound
  __syncwarp();
  reaching(bound, [&](unsigned long long k, int) {
    const int at = atomicAdd(&n_list, 1);
    if (at < kTopList) list[at] = k;
  });
  __syncthreads();
  if (tid < cs) *cluster.map_shared_rank(&listed[rank], tid) = n_list;
  cluster.sync();
  int total = 0;
  for (int r = 0; r < cs; ++r) total += listed[r];
  if (total > kTopList) {
    // too many: halve the range of keys until k .. kTopList of them are left
    unsigned long long lo = bound, hi = top_key(M, 0) + 1;  // more than a list, none
    for (int i = 0; i < 64; ++i) {
      const unsigned long long mid = lo + (hi - lo) / 2;
      const int c = count(mid);
      if (c < P.k) {
        hi = mid;
      } else {
        lo = mid;
        if (c <= kTopList) break;
      }
    }
    bound = lo;
    if (tid == 0) n_list = 0;
    __syncthreads();
    reaching(bound, [&](unsigned long long k, int) {
      const int at = atomicAdd(&n_list, 1);
      if (at < kTopList) list[at] = k;
    });
    __syncthreads();
    if (tid < cs) *cluster.map_shared_rank(&listed[rank], tid) = min(n_list, kTopList);
    cluster.sync();
  }
  // the listed places leave the share, the rest is summed
  reaching(bound, [&](unsigned long long, int at) { H.clear(at); });
  ExpSum<E> sum;
  sum.template add_share<NT, kTopU>(H, c2);
  sum.template block<NW>(c2, red, redz);
  if (tid == 0) *cluster.map_shared_rank(&sums[rank], 0) = make_float2(sum.m, sum.z);
  cluster.sync();
  if (rank == 0) {
    // the row's list takes the place of the share
    unsigned long long *all = reinterpret_cast<unsigned long long *>(held);
    int at = 0;
    for (int r = 0; r < cs; ++r) {
      const unsigned long long *l = cluster.map_shared_rank(list, r);
      for (int i = tid; i < listed[r] && at + i < kTopList; i += NT) all[at + i] = l[i];
      at += listed[r];
    }
    __syncthreads();
    total = min(at, kTopList);
    // each listed key's rank; the keys are distinct
    constexpr int kPer = kTopList / NT;
    unsigned long long mine[kPer];
    int above[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid + j * NT;
      above[j] = 0;
      mine[j] = 0ull;
      if (i < total) {
        mine[j] = all[i];
#pragma unroll 4
        for (int q = 0; q < total; ++q) above[j] += all[q] > mine[j];
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (tid + j * NT < total) all[above[j]] = mine[j];
    __syncthreads();
    for (int i = tid; i < P.k; i += NT) {
      const bool have = i < total;
      P.vals[(int64_t)n * P.k + i] = have ? key_value(all[i]) : neg_inf();
      P.ids[(int64_t)n * P.k + i] = have ? key_index(all[i]) : -1;
    }
    if (P.rest && warp == 0) {
      // what is left of the list, in rank order: its largest is the first
      float b = P.k < total ? key_value(all[P.k]) : neg_inf(), z = 0.f;
      for (int i = P.k + lane; i < total; i += 32) z += ex2((key_value(all[i]) - b) * c2);
      z = warp_sum(z);
      for (int r = 0; r < cs; ++r) exp_merge(b, z, sums[r].x, sums[r].y, c2);
      if (lane == 0) P.rest[n] = z == 0.f ? neg_inf() : b / P.T + logf(z);
    }
  }
  cluster.sync();  // the lists stay until rank 0 has read them
}

template <typename E>
static cudaError_t launch_top(TopParams &P, cudaStream_t s) {
  int smem = 0;
  P.cs = held_cluster<E>(P.N, P.V, kTopNT, &smem);
  smem = std::max(smem, 8 * kTopList);   // the row's list goes there
  static FuncAttrs attrs;
  attrs.apply((const void *)sd_top_kernel<E>, kHeldBytes + 16, true, "the top-logits kernel");
  return launch_held(sd_top_kernel<E>, P, P.N, false, P.cs, kTopNT, smem, s);
}

}  // namespace sdv

using namespace sdv;

extern "C" sd_status_t sd_top_logits(int32_t N, int32_t V, int32_t dtype, const void *logits,
                                     int64_t stride, int32_t k, float T, float *vals,
                                     int32_t *ids, float *rest, void *stream) {
  sdv::NvtxRange nvtx_range("sd_top_logits");
  if (N < 0 || V < 1 || V > SD_MAX_V || k < 1 || k > SD_MAX_TOP) return SD_ERR_INVALID_ARG;
  if (dtype != SD_F32 && dtype != SD_BF16) return SD_ERR_INVALID_ARG;
  if (!(T > 0.f) || !std::isfinite(T)) return SD_ERR_INVALID_ARG;
  if (N == 0) return SD_OK;
  if (!logits || !vals || !ids || (uintptr_t)logits % (dtype == SD_BF16 ? 2 : 4))
    return SD_ERR_INVALID_ARG;
  TopParams P = {};
  P.logits = logits;
  P.stride = stride;
  P.N = N;
  P.V = V;
  P.k = k;
  P.T = T;
  P.vals = vals;
  P.ids = ids;
  P.rest = rest;
  const cudaError_t e = dtype == SD_BF16 ? launch_top<__nv_bfloat16>(P, (cudaStream_t)stream)
                                         : launch_top<float>(P, (cudaStream_t)stream);
  return e == cudaSuccess ? SD_OK : e == cudaErrorInvalidValue ? SD_ERR_INVALID_ARG : SD_ERR_CUDA;
}
