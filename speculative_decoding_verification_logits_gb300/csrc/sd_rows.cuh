// Device code shared by the logit operators (penalties, top logits,
// distillation): packing to the logits' type, and rows as 16-byte vectors.
//
// A row starts at any element.  Its vectors are those of the 16-byte grid of
// memory: element 0 sits hp elements into vector 0, and element e0(q) =
// q VE - hp + i is element i of vector q.  Vectors wholly inside the row are
// loaded and stored whole, the at most two others element by element, so no
// access leaves the row.
#pragma once

#include "sd_device.cuh"
#include "sd_logits.h"

namespace sdv {

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// A CTA writes into the shared memory of another of its cluster only once that
// one has started: arrive early, wait right before the first such write.
__device__ __forceinline__ void row_cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void row_cluster_wait() {
  asm volatile("barrier.cluster.wait;" ::: "memory");
}

// Global loads that stay where they are written: volatile, so that none is
// moved above the wait for the stream's previous kernel, across a barrier
// after which memory holds something else (outputs in place of inputs), or
// out of the condition that says whether its address is one at all (optional
// arrays, places outside a row).  Through L2 only.
__device__ __forceinline__ uint4 ld16(const void *p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld4(const void *p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld2(const void *p) {
  unsigned short v;
  asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int ld_int(const int32_t *p) { return (int)ld4(p); }
__device__ __forceinline__ float ld_float(const float *p) { return __uint_as_float(ld4(p)); }

// Two floats rounded to nearest-even bf16, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename E>
struct Row;
template <>
struct Row<float> {
  static __device__ __forceinline__ void pack(const float *f, uint4 &v) {
    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float load(const uint8_t *row, int64_t e) {
    return __uint_as_float(ld4(reinterpret_cast<const float *>(row) + e));
  }
  static __device__ __forceinline__ void store(uint8_t *row, int64_t e, float f) {
    reinterpret_cast<float *>(row)[e] = f;
  }
};
template <>
struct Row<__nv_bfloat16> {
  static __device__ __forceinline__ void pack(const float *f, uint4 &v) {
    v = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                   pack_bf16(f[6], f[7]));
  }
  static __device__ __forceinline__ float load(const uint8_t *row, int64_t e) {
    return __uint_as_float(ld2(reinterpret_cast<const unsigned short *>(row) + e) << 16);
  }
  static __device__ __forceinline__ void store(uint8_t *row, int64_t e, float f) {
    reinterpret_cast<unsigned short *>(row)[e] = (unsigned short)pack_bf16(f, 0.f);
  }
};

// A row of n elements at `row`, hp elements into its 16-byte grid.
template <typename E>
struct RowView {
  static constexpr int VE = Elt<E>::kPerVec;
  const uint8_t *row;
  int hp, n, nvec;
  __device__ __forceinline__ RowView(const void *base, int64_t offset, int n_) {
    row = reinterpret_cast<const uint8_t *>(base) + offset * Elt<E>::kSize;
    hp = (int)((uintptr_t)row & 15) / Elt<E>::kSize;
    n = n_;
    nvec = (n + hp + VE - 1) / VE;
  }
  __device__ __forceinline__ int first(int q) const { return q * VE - hp; }
  __device__ __forceinline__ bool whole(int q) const {
    return q * VE >= hp && (q + 1) * VE - hp <= n;
  }
  // vector q (q < nvec), -inf in the places outside the row
  __device__ __forceinline__ uint4 load(int q) const {
    const int e0 = first(q);
    if (whole(q)) return ld16(row + (int64_t)e0 * Elt<E>::kSize);
    return load_edge(e0);
  }
  __device__ __noinline__ uint4 load_edge(int e0) const {
    float f[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i)
      f[i] = e0 + i >= 0 && e0 + i < n ? Row<E>::load(row, e0 + i) : neg_inf();
    uint4 v;
    Row<E>::pack(f, v);
    return v;
  }
};

// -------------------------------------------------- rows held on chip --
// A cluster of cs CTAs holds a row in shared memory, each CTA a contiguous
// share of its vectors, so that the row is read from memory once however
// often it is used.  (Read again through L2, a row's second pass came from
// DRAM: the rows in flight and what is written for them exceed L2.)  Three
// CTAs per SM: while one computes or writes, the others' copies are under way.
constexpr int kHeldCtas = 3;
constexpr int kHeldBytes = 66000;   // largest share: three of them and static arrays per SM
constexpr int kHeldMaxCS = 16;

template <typename E>
struct Held {
  RowView<E> row;
  int qa, n;       // first vector and vectors of this CTA's share
  uint4 *v;        // the share in shared memory, -inf outside the row
  __device__ __forceinline__ Held(const void *base, int64_t offset, int V, int rank, int cs,
                                  uint4 *smem)
      : row(base, offset, V), v(smem) {
    const int per = (row.nvec + cs - 1) / cs;
    qa = min(rank * per, row.nvec);
    n = min(per, row.nvec - qa);
  }
  // asks for every vector of the share; each thread copies its own ones
  template <int NT>
  __device__ __forceinline__ void fetch() {
    for (int i = threadIdx.x; i < n; i += NT) {
      const int q = qa + i;
      if (row.whole(q))
        cp_async16(smem_u32(v + i), row.row + (int64_t)row.first(q) * Elt<E>::kSize);
      else
        v[i] = row.load(q);
    }
    cp_commit();
  }
  // the place of element e in the share, or -1
  __device__ __forceinline__ int place(int e) const {
    const int at = e + row.hp - qa * RowView<E>::VE;
    return at >= 0 && at < n * RowView<E>::VE ? at : -1;
  }
};

// The cluster size for N rows of V elements: the fewest CTAs that hold a row,
// more where N rows would leave SMs without their CTAs (down to two vectors
// per thread).  0: a row does not fit.
template <typename E>
static int held_cluster(int64_t N, int V, int NT, int *share_bytes) {
  constexpr int VE = Elt<E>::kPerVec;
  const int64_t nvec = ((int64_t)V + 2 * VE - 2) / VE;
  int64_t cs = (nvec * 16 + kHeldBytes - 1) / kHeldBytes;
  if (cs > kHeldMaxCS) return 0;
  const int64_t slots = (int64_t)kHeldCtas * sm_count();
  while (cs < 8 && N * (cs + 1) <= slots && nvec / (cs + 1) >= 2 * NT) ++cs;
  *share_bytes = (int)((nvec + cs - 1) / cs * 16);
  return (int)cs;
}

// Launches fn(P) with one cluster of cs CTAs per row, as a programmatic
// dependent of the stream's previous kernel.
template <typename P>
static cudaError_t launch_held(void (*fn)(const P), const P &params, int64_t N, int cs, int NT,
                               int smem, cudaStream_t s) {
  if (N * cs > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(N * cs), 1, 1);
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
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
  return cudaLaunchKernelEx(&cfg, fn, params);
}

// ------------------------------------------------------ rows streamed --
// One CTA takes rows first, first + grid, ... from end to end (each `passes`
// times in a row).  Every thread copies its own vectors, U a step, into its
// own places of a ring of D steps; the copies run on across the ends of
// passes and rows, so that what happens there costs no bandwidth.  Rows of
// weight 0 are left out.  In a step a warp has 32 U vectors side by side:
// its vector u of the step that begins at q is q + at() + 32 u.
template <typename E, int NT, int U, int D>
struct RowStream {
  static constexpr int kStep = NT * U;                  // vectors of a step
  static constexpr int kBytes = D * kStep * 16;
  uint4 *ring;
  const void *base;
  const float *weight;
  int64_t stride;
  int N, V, passes;
  // the next step to ask for
  RowView<E> view;
  const uint8_t *src;   // this thread's first vector of it, where it is inside the row
  int row, pass, q, put, take;
  static __device__ __forceinline__ int at() {
    return (threadIdx.x >> 5) * 32 * U + (threadIdx.x & 31);
  }
  __device__ __forceinline__ RowStream(uint4 *ring_, const void *base_, int64_t stride_, int N_,
                                       int V_, int passes_, const float *weight_)
      : ring(ring_ + threadIdx.x), base(base_), weight(weight_), stride(stride_), N(N_), V(V_),
        passes(passes_), view(base_, 0, V_), row(blockIdx.x), put(0), take(0) {
    open();
#pragma unroll 1
    for (int d = 0; d < D - 1; ++d) ask();
  }
  // at `row` or the next one that counts
  __device__ __forceinline__ void open() {
    if (weight)
      while (row < N && ld_float(weight + row) == 0.f) row += gridDim.x;
    if (row < N) view = RowView<E>(base, (int64_t)row * stride, V);
    pass = 0;
    rewind();
  }
  __device__ __forceinline__ void rewind() {
    q = 0;
    src = view.row + ((int64_t)at() * RowView<E>::VE - view.hp) * Elt<E>::kSize;
  }
  __device__ __forceinline__ void ask() {
    uint4 *to = ring + put * kStep;
    if (row < N) {
      if (q > 0 && q + kStep < view.nvec) {   // no end of the row in the step
#pragma unroll
        for (int u = 0; u < U; ++u) cp_async16(smem_u32(to + u * NT), src + u * 512);
      } else {
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const int i = q + at() + u * 32;
          if (i >= view.nvec) break;
          if (view.whole(i)) cp_async16(smem_u32(to + u * NT), src + u * 512);
          else to[u * NT] = view.load(i);
        }
      }
      q += kStep;
      src += kStep * 16;
      if (q >= view.nvec) {
        if (++pass < passes) {
          rewind();
        } else {
          row += gridDim.x;
          open();
        }
      }
    }
    cp_commit();
    put = put + 1 == D ? 0 : put + 1;
  }
  // the oldest step's vectors; asks for another one
  __device__ __forceinline__ void next(uint4 *v) {
    cp_wait<D - 2>();
    const uint4 *from = ring + take * kStep;
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = from[u * NT];
    take = take + 1 == D ? 0 : take + 1;
    ask();
  }
  // vector u of the step `ahead` (< D - 1) steps after the oldest, once it is there
  __device__ __forceinline__ uint4 peek(int ahead, int u) const {
    int slot = take + ahead;
    slot = slot >= D ? slot - D : slot;
    return ring[slot * kStep + u * NT];
  }
};

// ------------------------------------------------- exponentials of vectors --
// Per vector, with the offset and the scale as packed pairs: the sum of
// 2^((x + o) c), and s 2^((x + o) c).  The offset is a logit and is taken off
// before the scale goes on, so that rows of the type's lowest value (a mask's
// stand-in for -inf) stay finite.
template <typename E>
struct VecExp;
template <>
struct VecExp<__nv_bfloat16> {
  // the largest element of U vectors (packed maxima, exact)
  template <int U>
  static __device__ __forceinline__ float largest(const uint4 *v) {
    const auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
    __nv_bfloat162 m = __hmax2(__hmax2(h(v[0].x), h(v[0].y)), __hmax2(h(v[0].z), h(v[0].w)));
#pragma unroll
    for (int u = 1; u < U; ++u)
      m = __hmax2(m, __hmax2(__hmax2(h(v[u].x), h(v[u].y)), __hmax2(h(v[u].z), h(v[u].w))));
    const uint32_t w = *reinterpret_cast<const uint32_t *>(&m);
    return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint64_t pair(uint32_t w) {
    return pk2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void ex2_pair(uint32_t w, uint64_t c, uint64_t o, float &a,
                                                  float &b) {
    upk2(mul2(add2(pair(w), o), c), a, b);
    a = ex2(a);
    b = ex2(b);
  }
  static __device__ __forceinline__ uint64_t sum(const uint4 &v, uint64_t c, uint64_t o,
                                                 uint64_t acc) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      ex2_pair(w[i], c, o, a, b);
      acc = add2(acc, pk2(a, b));
    }
    return acc;
  }
  static __device__ __forceinline__ uint4 scaled(const uint4 &v, uint64_t c, uint64_t o,
                                                 uint64_t s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      ex2_pair(w[i], c, o, a, b);
      upk2(mul2(pk2(a, b), s), a, b);
      r[i] = pack_bf16(a, b);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};
template <>
struct VecExp<float> {
  template <int U>
  static __device__ __forceinline__ float largest(const uint4 *v) {
    float m = Elt<float>::vmax(v[0]);
#pragma unroll
    for (int u = 1; u < U; ++u) m = fmaxf(m, Elt<float>::vmax(v[u]));
    return m;
  }
  static __device__ __forceinline__ void ex2_pair(uint32_t x, uint32_t y, uint64_t c, uint64_t o,
                                                  float &a, float &b) {
    upk2(mul2(add2(pk2(__uint_as_float(x), __uint_as_float(y)), o), c), a, b);
    a = ex2(a);
    b = ex2(b);
  }
  static __device__ __forceinline__ uint64_t sum(const uint4 &v, uint64_t c, uint64_t o,
                                                 uint64_t acc) {
    float a, b;
    ex2_pair(v.x, v.y, c, o, a, b);
    acc = add2(acc, pk2(a, b));
    ex2_pair(v.z, v.w, c, o, a, b);
    return add2(acc, pk2(a, b));
  }
  static __device__ __forceinline__ uint4 scaled(const uint4 &v, uint64_t c, uint64_t o,
                                                 uint64_t s) {
    float f[4];
    ex2_pair(v.x, v.y, c, o, f[0], f[1]);
    ex2_pair(v.z, v.w, c, o, f[2], f[3]);
    upk2(mul2(pk2(f[0], f[1]), s), f[0], f[1]);
    upk2(mul2(pk2(f[2], f[3]), s), f[2], f[3]);
    uint4 r;
    Row<float>::pack(f, r);
    return r;
  }
};

// Running (largest m, sum z of 2^((x - m) c)) over vectors.
__device__ __forceinline__ void exp_merge(float &m, float &z, float m2, float z2, float c) {
  const float b = fmaxf(m, m2), s = b == neg_inf() ? 0.f : b;   // an empty sum stays zero
  z = z * ex2((m - s) * c) + z2 * ex2((m2 - s) * c);
  m = b;
}
template <typename E>
struct ExpSum {
  float m, z;
  __device__ __forceinline__ ExpSum() : m(neg_inf()), z(0.f) {}
  // U vectors at once: one maximum, one rescaling
  template <int U>
  __device__ __forceinline__ void add(const uint4 *v, float c) {
    const float b = VecExp<E>::template largest<U>(v);
    if (b > m) {
      z *= ex2((m - b) * c);
      m = b;
    }
    const float s = m == neg_inf() ? 0.f : -m;
    const uint64_t c2 = pk2(c, c), s2 = pk2(s, s);
    uint64_t acc = 0ull;
#pragma unroll
    for (int u = 0; u < U; ++u) acc = VecExp<E>::sum(v[u], c2, s2, acc);
    float x, y;
    upk2(acc, x, y);
    z += x + y;
  }
  // this thread's vectors of a share: NT apart, U at a time
  template <int NT, int U>
  __device__ __forceinline__ void add_share(const uint4 *held, int n, float c) {
    int i = threadIdx.x;
    for (; i + (U - 1) * NT < n; i += U * NT) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = held[i + u * NT];
      add<U>(v, c);
    }
    for (; i < n; i += NT) {
      const uint4 v = held[i];
      add<1>(&v, c);
    }
  }
  // the block's, in every thread; wm and wz hold a float per warp
  template <int NW>
  __device__ __forceinline__ void block(float c, float *wm, float *wz) {
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, i), z2 = __shfl_xor_sync(0xffffffffu, z, i);
      exp_merge(m, z, m2, z2, c);
    }
    if ((threadIdx.x & 31) == 0) {
      wm[threadIdx.x >> 5] = m;
      wz[threadIdx.x >> 5] = z;
    }
    __syncthreads();
    m = wm[0];
    z = wz[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) exp_merge(m, z, wm[i], wz[i], c);
  }
};

}  // namespace sdv
