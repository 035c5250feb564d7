// The top logits of each row and the log-sum-exp of all others: what a
// teacher gives to a distillation step.
//
// One cluster of cs CTAs per row, each CTA a contiguous share of the row's
// vectors, read twice (the second time from L2):
//  1. every thread keeps the best logit of its own vectors.  The k-th best of
//     a set of groups' maxima bounds the k-th best logit from below: k groups
//     hold a logit at least as good.  Two such bounds are taken, the better
//     one is used: the largest over the CTAs of each CTA's k-th best group,
//     and the smallest over the CTAs of each CTA's ceil(k / cs)-th best.
//  2. logits at or above the bound (little more than k of them where the
//     large logits are spread over the row) go to a list, all others into a
//     running (largest, sum of exp((x - largest) / T)).  The first CTA ranks the list, writes the
//     first k and adds what is left to the sum in rank order, so that nothing
//     depends on the order in which the list was filled.
// A row whose logits at the bound do not fit the list (large logits all in a
// few groups) raises its bound first by halving the range of keys until at
// least k and at most a list of logits are left.
// Keys order logits by value, then by lower index: (ordered image of the
// value, ~index).  HBM-bound: a row is 2 or 4 V bytes, the results 8 k + 4.

#include "sd_rows.cuh"

namespace sdv {

constexpr int kTopNT = 512;
constexpr int kTopNW = kTopNT / 32;
constexpr int kTopU = 4;          // vectors in flight per thread
constexpr int kTopGroups = 256;   // groups of a CTA for the bound
constexpr int kTopList = 1024;    // listed logits of a row
constexpr int kTopMaxCS = 8;

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

// (largest logit, sum of exp((x - largest) / T)) of two sets as one
__device__ __forceinline__ void top_merge(float &m, float &z, float m2, float z2, float c2) {
  const float b = fmaxf(m, m2), s = b == neg_inf() ? 0.f : b;
  z = z * ex2((m - s) * c2) + z2 * ex2((m2 - s) * c2);
  m = b;
}

template <typename E>
__global__ void __launch_bounds__(kTopNT, 2) sd_top_kernel(const TopParams P) {
  constexpr int VE = Elt<E>::kPerVec;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  row_cluster_arrive();
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = P.cs, rank = (int)cluster.block_rank(), n = blockIdx.x / cs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ unsigned long long group[kTopGroups];
  __shared__ unsigned long long list[kTopList];    // this CTA's listed keys
  __shared__ unsigned long long all[kTopList];     // rank 0: the row's, then in order
  __shared__ TopStat stat[kTopMaxCS];
  __shared__ float2 sums[kTopMaxCS];
  __shared__ int listed[kTopMaxCS];
  __shared__ int counted[2][kTopMaxCS];
  __shared__ float red[kTopNW], redz[kTopNW];
  __shared__ unsigned long long kth, share;
  __shared__ int n_list;
  const RowView<E> row(P.logits, (int64_t)n * P.stride, P.V);
  const int per = (row.nvec + cs - 1) / cs;
  const int qa = min(rank * per, row.nvec), qb = min(qa + per, row.nvec);
  const float c2 = log2e_over(P.T);

  // 1. the best logit of each thread's vectors
  float m = neg_inf();
  int mq = -1;
  for (int q = qa + tid; q < qb; q += kTopNT * kTopU) {
    uint4 v[kTopU];
#pragma unroll
    for (int u = 0; u < kTopU; ++u)
      if (q + u * kTopNT < qb) v[u] = row.load(q + u * kTopNT);
#pragma unroll
    for (int u = 0; u < kTopU; ++u)
      if (q + u * kTopNT < qb) {
        const float x = Elt<E>::vmax(v[u]);
        if (x > m) {
          m = x;
          mq = q + u * kTopNT;
        }
      }
  }
  // keyed by the last index its vector could give: no better than the logit itself
  unsigned long long key = mq >= 0 ? top_key(m, row.first(mq) + VE - 1) : 0ull;
  {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, key, 1);
    key = o > key ? o : key;
  }
  if ((lane & 1) == 0) group[tid >> 1] = key;
  m = warp_max(m);
  if (lane == 0) red[warp] = m;
  if (tid == 0) {
    kth = share = 0ull;
    n_list = 0;
  }
  __syncthreads();
  const int ks = (P.k + cs - 1) / cs;
  if (tid < kTopGroups) {
    const unsigned long long g = group[tid];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kTopGroups; ++j) above += group[j] > g;
    if (g != 0ull) {
      if (above == P.k - 1) kth = g;
      if (above == ks - 1) share = g;
    }
  }
  float cm = neg_inf();
#pragma unroll
  for (int w = 0; w < kTopNW; ++w) cm = fmaxf(cm, red[w]);
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

  float om = neg_inf(), oz = 0.f;   // the others: largest logit, sum of exp((x - om) / T)
  for (int round = 0;; ++round) {
    // 2. list what reaches the bound, sum the rest
    const float bx = key_value(bound);
    om = neg_inf();
    oz = 0.f;
    for (int q = qa + tid; q < qb; q += kTopNT * kTopU) {
      uint4 v[kTopU];
#pragma unroll
      for (int u = 0; u < kTopU; ++u)
        if (q + u * kTopNT < qb) v[u] = row.load(q + u * kTopNT);
#pragma unroll
      for (int u = 0; u < kTopU; ++u)
        if (q + u * kTopNT < qb) {
          float f[VE];
          Elt<E>::unpack(v[u], f);
          float vm = Elt<E>::vmax(v[u]);
          if (vm >= bx) {
            const int e0 = row.first(q + u * kTopNT);
            vm = neg_inf();
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              const unsigned long long key = top_key(f[i], e0 + i);
              if (f[i] >= bx && key >= bound) {
                const int at = atomicAdd(&n_list, 1);
                if (at < kTopList) list[at] = key;
                f[i] = neg_inf();
              }
              vm = fmaxf(vm, f[i]);
            }
          }
          if (vm > om) {
            oz *= ex2((om - vm) * c2);
            om = vm;
          }
          const float s = om == neg_inf() ? 0.f : om;
#pragma unroll
          for (int i = 0; i < VE; ++i) oz += ex2((f[i] - s) * c2);
        }
    }
    __syncthreads();
    if (tid < cs) *cluster.map_shared_rank(&listed[rank], tid) = n_list;
    cluster.sync();
    int total = 0;
    for (int r = 0; r < cs; ++r) total += listed[r];
    if (total <= kTopList) break;
    // too many: halve the range of keys until k .. kTopList of them are left
    unsigned long long lo = bound, hi = top_key(M, 0) + 1;  // count(lo) > list, count(hi) = 0
    for (int step = 0; step < 64; ++step) {
      const unsigned long long mid = lo + (hi - lo) / 2;
      int here = 0;
      for (int q = qa + tid; q < qb; q += kTopNT) {
        const uint4 v = row.load(q);
        float f[VE];
        Elt<E>::unpack(v, f);
#pragma unroll
        for (int i = 0; i < VE; ++i)
          here += f[i] > neg_inf() && top_key(f[i], row.first(q) + i) >= mid;
      }
      here = __reduce_add_sync(0xffffffffu, here);
      if (tid == 0) n_list = 0;
      __syncthreads();
      if (lane == 0) atomicAdd(&n_list, here);
      __syncthreads();
      if (tid < cs) *cluster.map_shared_rank(&counted[step & 1][rank], tid) = n_list;
      cluster.sync();
      int count = 0;
      for (int r = 0; r < cs; ++r) count += counted[step & 1][r];
      if (count < P.k) {
        hi = mid;
      } else {
        lo = mid;
        if (count <= kTopList) break;
      }
    }
    bound = lo;
    if (tid == 0) n_list = 0;
    __syncthreads();
    if (round > 0) break;   // one narrowing is always enough
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, om, i), z2 = __shfl_xor_sync(0xffffffffu, oz, i);
    top_merge(om, oz, m2, z2, c2);
  }
  if (lane == 0) {
    red[warp] = om;
    redz[warp] = oz;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kTopNW; ++w) top_merge(om, oz, red[w], redz[w], c2);
    *cluster.map_shared_rank(&sums[rank], 0) = make_float2(om, oz);
  }
  cluster.sync();
  if (rank == 0) {
    int at = 0;
    for (int r = 0; r < cs; ++r) {
      const unsigned long long *l = cluster.map_shared_rank(list, r);
      for (int i = tid; i < listed[r] && at + i < kTopList; i += kTopNT) all[at + i] = l[i];
      at += listed[r];
    }
    __syncthreads();
    const int total = min(at, kTopList);
    // each listed key's rank; the keys are distinct
    constexpr int kPer = kTopList / kTopNT;
    unsigned long long mine[kPer];
    int above[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid + j * kTopNT;
      above[j] = 0;
      mine[j] = 0ull;
      if (i < total) {
        mine[j] = all[i];
        for (int o = 0; o < total; ++o) above[j] += all[o] > mine[j];
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (tid + j * kTopNT < total) all[above[j]] = mine[j];
    __syncthreads();
    for (int i = tid; i < P.k; i += kTopNT) {
      const bool have = i < total;
      P.vals[(int64_t)n * P.k + i] = have ? key_value(all[i]) : neg_inf();
      P.ids[(int64_t)n * P.k + i] = have ? key_index(all[i]) : -1;
    }
    if (P.rest && warp == 0) {
      // what is left of the list, in rank order: its largest is the first
      om = P.k < total ? key_value(all[P.k]) : neg_inf();
      oz = 0.f;
      for (int i = P.k + lane; i < total; i += 32) oz += ex2((key_value(all[i]) - om) * c2);
      oz = warp_sum(oz);
      for (int r = 0; r < cs; ++r) top_merge(om, oz, sums[r].x, sums[r].y, c2);
      if (lane == 0) P.rest[n] = oz == 0.f ? neg_inf() : om / P.T + logf(oz);
    }
  }
  cluster.sync();  // the lists stay until rank 0 has read them
}

template <typename E>
static cudaError_t launch_top(TopParams &P, cudaStream_t s) {
  // enough CTAs to fill the device where the rows are few, each with a few
  // vectors per thread at least
  const int64_t nvec = (int64_t)P.V / Elt<E>::kPerVec + 1;
  const int64_t slots = 2LL * sm_count();
  int cs = 1;
  while (cs < kTopMaxCS && (int64_t)P.N * cs * 2 <= slots && nvec / (2 * cs) >= kTopNT) cs *= 2;
  P.cs = cs;
  if ((int64_t)P.N * cs > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.N * cs), 1, 1);
  cfg.blockDim = dim3(kTopNT, 1, 1);
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
  return cudaLaunchKernelEx(&cfg, sd_top_kernel<E>, (const TopParams)P);
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
