// The top logits of each row and the log-sum-exp of all others: what a
// teacher gives to a distillation step.
//
// Few rows: one cluster of cs CTAs per row, which holds it in shared memory:
//  1. every thread keeps the best logit of its own vectors.  A value that k of
//     them reach bounds the k-th best logit from below.  Two such bounds are
//     taken, the better one is used: the largest over the CTAs of what k of
//     their threads reach, and the smallest over the CTAs of what ceil(k / cs)
//     of theirs reach.
//  2. logits at or above the bound (little more than k of them where the
//     large logits are spread over the row) go to a list and are set to -inf
//     in the share, whose rest is summed.  The first CTA ranks the list, writes
//     the first k and adds what is left to the sum in rank order, so that
//     nothing depends on the order in which the list was filled.
// A row whose logits at the bound do not fit the list (large logits all in a
// few groups) raises its bound first by halving the range of keys until at
// least k and at most a list of logits are left.
// Many rows: see sd_top_stream_kernel.
// Keys order logits by value, then by lower index: (ordered image of the
// value, ~index).  A row is 2 or 4 V bytes to read, the results are 8 k + 4.
// Measured on the GPU: 576 rows of 151936 bf16, k 64, 46 us (3.8 TB/s; the
// loss's plain sum over the same rows takes 34): what is above the stream is
// the row's end (bound, list, ranks), which two CTAs per SM overlap only in
// part.  7 rows of 128256, k 32: 9.8 us, 33 rows of 50021 fp32, k 128: 12.3 us,
// chains of one load of the row, two cluster barriers, the ranks.

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

// What the CTAs of a row tell one another: values that k and ceil(k / cs) of
// their threads' best logits reach; what they listed, and the sum of the rest.
struct TopStat {
  float kth, share;
};
struct TopSum {
  float m, z;
  int listed;
};

// Registers for one CTA per SM more than the rule for held rows counts on:
// clusters of eight do not fill every group of SMs to the last place (57 rows
// of 32000 fp32, exactly three CTAs per SM, ran in two waves: 20 us).
template <typename E>
__global__ void __launch_bounds__(kTopNT, kHeldCtas + 1) sd_top_kernel(const TopParams P) {
  constexpr int VE = Elt<E>::kPerVec, NT = kTopNT, NW = kTopNW;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  row_cluster_arrive();
  extern __shared__ uint4 held[];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = P.cs, rank = (int)cluster.block_rank(), n = blockIdx.x / cs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ unsigned long long list[kTopList];    // this CTA's listed keys
  __shared__ TopStat stat[kHeldMaxCS];
  __shared__ TopSum sums[kHeldMaxCS];
  __shared__ int counted[2][kHeldMaxCS];
  __shared__ unsigned short keys[NT];
  __shared__ float wm[NW], wz[NW];
  __shared__ int n_list;
  const Held<E> H(P.logits, (int64_t)n * P.stride, P.V, rank, cs, smem_u32(held));
  H.template fetch<NT>();
  const float c2 = log2e_over(P.T);
  if (tid == 0) n_list = 0;
  cp_wait<0>();

  // 1. the best logit of each thread's own vectors, which it copied itself
  float best = neg_inf();
  for (int i = tid; i < H.n; i += NT) best = fmaxf(best, Elt<E>::vmax(H.get(i)));
  keys[tid] = top_key16(best);
  __syncthreads();
  row_cluster_wait();
  if (warp < 2) {   // a warp for each of the two bounds
    const float b = top_bound_warp<NT>(keys, warp == 0 ? P.k : (P.k + cs - 1) / cs);
    if (lane < cs) {
      TopStat *s = cluster.map_shared_rank(&stat[rank], lane);
      if (warp == 0) s->kth = b;
      else s->share = b;
    }
  }
  cluster.sync();
  float bound = kLowest, least = INFINITY;
  for (int r = 0; r < cs; ++r) {
    bound = fmaxf(bound, stat[r].kth);
    least = fminf(least, stat[r].share);
  }
  bound = fmaxf(bound, least);

  // calls f(key, place) for what has at least this key
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
        const unsigned long long key = top_key(x[e], e0 + e);
        if (x[e] >= bx && key >= least_key) f(key, i * VE + e);
      }
    }
  };
  // 2. what reaches the bound is listed and leaves the share, whose rest is
  // summed; every CTA learns of all lists and sums
  auto list_and_sum = [&](unsigned long long least_key) {
    reaching(least_key, [&](unsigned long long key, int at) {
      const int i = atomicAdd(&n_list, 1);
      if (i < kTopList) list[i] = key;
      H.clear(at);
    });
    __syncwarp();
    ExpSum<E> sum;
    sum.template add_share<NT, kTopU>(H, c2);
    sum.template block<NW>(c2, wm, wz);   // its barrier: the list is complete
    if (tid < cs) {
      TopSum *s = cluster.map_shared_rank(&sums[rank], tid);
      s->m = sum.m;
      s->z = sum.z;
      s->listed = n_list;
    }
    cluster.sync();
    int total = 0;
    for (int r = 0; r < cs; ++r) total += sums[r].listed;
    return total;
  };
  // the bound as the lowest key of its value
  int total = list_and_sum(top_key(bound, INT32_MAX));
  if (total > kTopList) {
    // too many: from the row as it was, halve the range of keys until k ..
    // kTopList of them reach its lower end
    H.template fetch<NT>();
    cp_wait<0>();
    unsigned long long lo = top_key(bound, INT32_MAX), hi = ~0ull;  // more than a list, none
    for (int step = 0; step < 64; ++step) {
      const unsigned long long mid = lo + (hi - lo) / 2;
      int here = 0;
      reaching(mid, [&](unsigned long long, int) { ++here; });
      __syncwarp();
      here = __reduce_add_sync(0xffffffffu, here);
      __syncthreads();
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
    __syncthreads();
    if (tid == 0) n_list = 0;
    __syncthreads();
    total = list_and_sum(lo);
  }
  if (rank == 0) {
    // the row's list takes the place of the share
    unsigned long long *all = reinterpret_cast<unsigned long long *>(held);
    int at = 0;
    for (int r = 0; r < cs; ++r) {
      const unsigned long long *l = cluster.map_shared_rank(list, r);
      for (int i = tid; i < sums[r].listed && at + i < kTopList; i += NT) all[at + i] = l[i];
      at += sums[r].listed;
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
      for (int r = 0; r < cs; ++r) exp_merge(b, z, sums[r].m, sums[r].z, c2);
      if (lane == 0) P.rest[n] = z == 0.f ? neg_inf() : b / P.T + logf(z);
    }
  }
  cluster.sync();  // the lists stay until rank 0 has read them
}

// Many rows: one CTA per row, streamed once.  The bound comes from the
// threads' best logits so far (k of them at or above it) and is raised as the
// row goes by: before the first step, from all the steps in the copy ring,
// when what has gone by is twice that, and then at every fourfold (576 x 151936
// bf16, k 64: 45 us; at every doubling 47, never 49).  Vectors that hold what
// reaches it go to a list, the other ones into the sum.  At the row's end the
// bound from all of the row leaves little more than k logits of the list's
// vectors; these are ranked, the others' exponentials are added as integers
// (fixed point below the largest of them: no order changes the sum).  A row that overflows the list (its
// large logits at its end, or in a few threads' places) is gone over again
// from memory.
constexpr int kTopHeap = 2 * kTopList;   // listed vectors of a streamed row

template <typename E>
__global__ void __launch_bounds__(kStreamNT, 2) sd_top_stream_kernel(const TopParams P) {
  constexpr int VE = Elt<E>::kPerVec, NT = kStreamNT, NW = NT / 32, U = kStreamU;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using Stream = RowStream<E, NT, U, kStreamD>;
  extern __shared__ uint4 ring[];
  // logits that may be chosen; the list of vectors, then the ranked logits
  unsigned long long *kept = reinterpret_cast<unsigned long long *>(ring + Stream::kBytes / 16);
  int *heap = reinterpret_cast<int *>(kept + kTopList);
  unsigned long long *ranked = reinterpret_cast<unsigned long long *>(heap);
  __shared__ unsigned short keys[NT];
  __shared__ float bound_s;
  __shared__ float wm[NW], wz[NW];
  __shared__ unsigned long long less[NW];       // the others' sum, a part per warp
  __shared__ int n_heap, n_kept, less_max;
  const int tid = threadIdx.x, lane = tid & 31, k = P.k;
  const float c2 = log2e_over(P.T);
  const uint32_t inf = Elt<E>::kNegInfWord;
  Stream S(ring, P.logits, P.stride, P.N, P.V, 1, nullptr);
  if (tid == 0) n_heap = 0;
  for (int n = blockIdx.x; n < P.N; n += gridDim.x) {
    const RowView<E> row(P.logits, (int64_t)n * P.stride, P.V);
    // the best of what is in the ring
    float best = neg_inf();
    cp_wait<0>();
#pragma unroll 1
    for (int d = 0; d < kStreamD - 1; ++d)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = d * Stream::kStep + Stream::at() + u * 32;
        if (i < row.nvec) best = fmaxf(best, Elt<E>::vmax(S.peek(d, u)));
      }
    float bound = top_bound<NT>(best, k, keys, &bound_s, [] {});
    int raise = (kStreamD - 1) * Stream::kStep * 2;
    ExpSum<E> sum;
    for (int q = 0; q < row.nvec; q += Stream::kStep) {
      uint4 v[U];
      S.next(v);
      const int first = q + Stream::at();
      if (q + Stream::kStep > row.nvec) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (first + u * 32 >= row.nvec) v[u] = make_uint4(inf, inf, inf, inf);
      }
      float each[U], m = neg_inf();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        each[u] = Elt<E>::vmax(v[u]);
        m = fmaxf(m, each[u]);
      }
      best = fmaxf(best, m);
      if (q >= raise || (bound == kLowest && __syncthreads_count(best > neg_inf()) >= k)) {
        bound = top_bound<NT>(best, k, keys, &bound_s, [] {});
        raise = 4 * q;
      }
      if (m >= bound) {
        m = neg_inf();
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!(each[u] >= bound)) {
            m = fmaxf(m, each[u]);
            continue;
          }
          v[u] = make_uint4(inf, inf, inf, inf);
          const int at = atomicAdd(&n_heap, 1);
          if (at < kTopHeap) heap[at] = first + u * 32;
        }
      }
      sum.template add<U>(v, c2, m);
    }
    // what may be chosen: at or above the bound from the whole row
    int total = 0;
    int h0 = 0;         // the thread's first vector of the list, asked for at once
    uint4 v0 = make_uint4(0u, 0u, 0u, 0u);
    bound = top_bound<NT>(best, k, keys, &bound_s, [&] {   // the list is complete
      total = n_heap;
      if (tid < total) {
        h0 = heap[tid];
        v0 = row.load(h0);
      }
      if (tid == 0) {
        n_kept = 0;
        less_max = (int)0x80000000;
      }
    });
    // calls f(logit, its index) for the listed vectors'
    auto listed = [&](auto f) {
      int h = h0;
      uint4 v = v0;
      for (int i = tid; i < total;) {
        float x[VE];
        Elt<E>::unpack(v, x);
        const int e0 = row.first(h);
#pragma unroll
        for (int e = 0; e < VE; ++e) f(x[e], e0 + e);
        i += NT;
        if (i < total) {
          h = heap[i];
          v = row.load(h);
        }
      }
    };
    if (total <= kTopHeap) {
      int most = (int)0x80000000;
      listed([&](float x, int i) {
        if (x >= bound) {
          const int at = atomicAdd(&n_kept, 1);
          if (at < kTopList) kept[at] = top_key(x, i);
        } else if (x == x) {   // not a NaN
          most = max(most, ford(x));
        }
      });
      __syncwarp();
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) atomicMax(&less_max, most);
    }
    __syncthreads();
    if (total > kTopHeap || n_kept > kTopList) {
      // over the row again: halve the range of keys until k .. kTopList of
      // them reach its lower end (there are more than k logits here)
      unsigned long long lo = top_key(kLowest, P.V), hi = ~0ull;
      for (int step = 0; step < 64; ++step) {
        const unsigned long long mid = lo + (hi - lo) / 2;
        int here = 0;
        for (int q = tid; q < row.nvec; q += NT) {
          float f[VE];
          Elt<E>::unpack(row.load(q), f);
#pragma unroll
          for (int e = 0; e < VE; ++e)
            here += f[e] > neg_inf() && top_key(f[e], row.first(q) + e) >= mid;
        }
        __syncthreads();
        if (tid == 0) n_heap = 0;
        __syncthreads();
        here = __reduce_add_sync(0xffffffffu, here);
        if (lane == 0) atomicAdd(&n_heap, here);
        __syncthreads();
        if (n_heap < k) {
          hi = mid;
        } else {
          lo = mid;
          if (n_heap <= kTopList) break;
        }
      }
      __syncthreads();
      if (tid == 0) {
        n_kept = 0;
        less_max = (int)0x80000000;
      }
      __syncthreads();
      sum = ExpSum<E>();
      for (int q = tid; q < row.nvec; q += NT) {
        uint4 v = row.load(q);
        float f[VE];
        Elt<E>::unpack(v, f);
        uint32_t stay = (1u << VE) - 1u;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const unsigned long long key = top_key(f[e], row.first(q) + e);
          if (f[e] > neg_inf() && key >= lo) {
            const int at = atomicAdd(&n_kept, 1);
            if (at < kTopList) kept[at] = key;
            stay &= ~(1u << e);
          }
        }
        v = mask_vec<E>(v, stay);
        sum.template add<1>(&v, c2);
      }
      total = 0;   // the list is not looked at
      __syncthreads();
    }
    // the others of the list
    const float top_less = fdeord(less_max);
    unsigned long long part = 0ull;
    listed([&](float x, int) {
      if (x >= bound || x == neg_inf()) return;
      if (x == x) part += (unsigned long long)(ex2((x - top_less) * c2) * 17592186044416.f);
      else sum.z = x;
    });
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    sum.warp(c2);
    if (lane == 0) {
      wm[tid >> 5] = sum.m;
      wz[tid >> 5] = sum.z;
      less[tid >> 5] = part;
    }
    // ranks of those kept, four threads to a key: the keys are distinct
    const int nk = min(n_kept, kTopList);
    __syncthreads();   // the list is done with: the ranked ones take its place
    for (int i0 = 0; i0 < nk; i0 += NT / 4) {
      const int i = i0 + (tid >> 2);
      const unsigned long long key = i < nk ? kept[i] : ~0ull;
      int above = 0;
#pragma unroll 4
      for (int o = tid & 3; o < nk; o += 4) above += kept[o] > key;
      __syncwarp();
      above += __shfl_xor_sync(0xffffffffu, above, 1);
      above += __shfl_xor_sync(0xffffffffu, above, 2);
      if ((tid & 3) || i >= nk) continue;
      ranked[above] = key;
      if (above < k) {
        P.vals[(int64_t)n * k + above] = key_value(key);
        P.ids[(int64_t)n * k + above] = key_index(key);
      }
    }
    for (int i = nk + tid; i < k; i += NT) {   // fewer than k finite ones
      P.vals[(int64_t)n * k + i] = neg_inf();
      P.ids[(int64_t)n * k + i] = -1;
    }
    if (tid == 0) n_heap = 0;
    __syncthreads();
    if (P.rest && tid < 32) {
      sum.m = tid < NW ? wm[tid] : neg_inf();
      sum.z = tid < NW ? wz[tid] : 0.f;
      sum.warp(c2);
      // what is left of the ranked ones, and the others of the list
      const float b = k < nk ? key_value(ranked[k]) : neg_inf();
      float z = 0.f;
      for (int i = k + lane; i < nk; i += 32) z += ex2((key_value(ranked[i]) - b) * c2);
      z = warp_sum(z);
      exp_merge(sum.m, sum.z, b, z, c2);
      unsigned long long all = 0ull;
#pragma unroll
      for (int i = 0; i < NW; ++i) all += less[i];
      if (all) exp_merge(sum.m, sum.z, top_less, (float)all * (1.f / 17592186044416.f), c2);
      if (lane == 0) P.rest[n] = sum.z == 0.f ? neg_inf() : sum.m / P.T + logf(sum.z);
    }
  }
}

template <typename E>
static cudaError_t launch_top(TopParams &P, cudaStream_t s) {
  int smem = 0;
  P.cs = held_cluster<E>(P.N, P.V, kTopNT, &smem);
  if (P.cs > 0) {
    smem = std::max(smem, 8 * kTopList);   // the row's list goes there
    static FuncAttrs attrs;
    attrs.apply((const void *)sd_top_kernel<E>, kHeldBytes + 16, true, "the top-logits kernel");
    return launch_held(sd_top_kernel<E>, P, P.N, P.cs, kTopNT, smem, s);
  }
  smem = RowStream<E, kStreamNT, kStreamU, kStreamD>::kBytes + 4 * kTopHeap + 8 * kTopList;
  static FuncAttrs attrs;
  attrs.apply((const void *)sd_top_stream_kernel<E>, smem, false, "the top-logits kernel");
  return launch_streamed(sd_top_stream_kernel<E>, P, P.N, kStreamNT, smem, s);
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
