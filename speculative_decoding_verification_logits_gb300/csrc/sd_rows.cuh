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

}  // namespace sdv
