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
__device__ __forceinline__ uint32_t ld1(const void *p) {
  unsigned short v;
  asm volatile("ld.global.cg.u8 %0, [%1];" : "=h"(v) : "l"(p));
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

// Bytes of x picked by the selector's nibbles; 8 + i gives byte i's sign in
// every bit.
__device__ __forceinline__ uint32_t prmt(uint32_t x, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "r"(sel));
  return r;
}

// The words of vector v with -inf where its bit in `ok` is clear: four bits
// are spread to the sign bits of four bytes by one multiply (the partial
// products do not meet), which byte permutes then copy over a half or a word.
template <typename E>
__device__ __forceinline__ uint4 mask_vec(uint4 v, uint32_t ok) {
  const uint32_t lo = ((ok & 15u) * 0x10204080u) & 0x80808080u;
  uint32_t k0, k1, k2, k3;
  if (Elt<E>::kPerVec == 8) {
    const uint32_t hi = ((ok >> 4) * 0x10204080u) & 0x80808080u;
    k0 = prmt(lo, 0x9988);
    k1 = prmt(lo, 0xbbaa);
    k2 = prmt(hi, 0x9988);
    k3 = prmt(hi, 0xbbaa);
  } else {
    k0 = prmt(lo, 0x8888);
    k1 = prmt(lo, 0x9999);
    k2 = prmt(lo, 0xaaaa);
    k3 = prmt(lo, 0xbbbb);
  }
  const uint32_t inf = Elt<E>::kNegInfWord;
  return make_uint4((v.x & k0) | (inf & ~k0), (v.y & k1) | (inf & ~k1), (v.z & k2) | (inf & ~k2),
                    (v.w & k3) | (inf & ~k3));
}

// Shared memory by its 32-bit address.  The copy goes through L1 (.ca): past it
// (.cg) every sector was counted twice between L2 and the SM (576 x 151936
// bf16 rows read once: 352 MB instead of 177 MB).
__device__ __forceinline__ void row_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(p));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t p, const uint4 &v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

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
// For few rows, where latency counts: a cluster of cs CTAs holds a row in
// shared memory, each CTA a contiguous share of its vectors.
constexpr int kHeldCtas = 3;
constexpr int kHeldBytes = 66000;   // largest share: three of them and static arrays per SM
constexpr int kHeldMaxCS = 16;
constexpr int kStreamNT = 384;      // streamed rows: threads, two CTAs per SM
constexpr int kStreamU = 3;         // vectors of a step per thread
constexpr int kStreamD = 4;         // steps of the copy ring

template <typename E>
struct Held {
  RowView<E> row;
  int qa, n;           // first vector and vectors of this CTA's share
  int lo, hi;          // vectors [lo, hi) of the share lie wholly inside the row
  const uint8_t *src;  // vector 0 of the share in memory (if it lies inside the row)
  uint32_t at;         // the share in shared memory, -inf outside the row
  __device__ __forceinline__ Held(const void *base, int64_t offset, int V, int rank, int cs,
                                  uint32_t smem)
      : row(base, offset, V), at(smem) {
    const int per = (row.nvec + cs - 1) / cs;
    qa = min(rank * per, row.nvec);
    n = min(per, row.nvec - qa);
    lo = n > 0 && !row.whole(qa) ? 1 : 0;
    hi = n > 0 && !row.whole(qa + n - 1) ? n - 1 : n;
    src = row.row + (int64_t)row.first(qa) * Elt<E>::kSize;
  }
  __device__ __forceinline__ bool inner(int i) const {
    return (unsigned)(i - lo) < (unsigned)(hi - lo);
  }
  __device__ __forceinline__ uint4 get(int i) const { return lds16(at + i * 16); }
  // asks for vector i < n of the share
  __device__ __forceinline__ void fetch(int i) const {
    if (inner(i)) row_async16(at + i * 16, src + (int64_t)i * 16);
    else sts16(at + i * 16, row.load(qa + i));
  }
  // asks for every vector of the share; each thread copies its own ones
  template <int NT>
  __device__ __forceinline__ void fetch() const {
    for (int i = threadIdx.x; i < n; i += NT) fetch(i);
    cp_commit();
  }
  // the place of element e in the share, or -1
  __device__ __forceinline__ int place(int e) const {
    const int p = e + row.hp - qa * RowView<E>::VE;
    return p >= 0 && p < n * RowView<E>::VE ? p : -1;
  }
  // -inf at place p
  __device__ __forceinline__ void clear(int p) const {
    if (Elt<E>::kSize == 2)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + p * 2), "h"((unsigned short)0xff80)
                   : "memory");
    else
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + p * 4), "r"(0xff800000u) : "memory");
  }
};

// The cluster size that holds rows of V elements, or 0 where N rows are so many
// that streaming them is faster: eight CTAs per row (more for rows that need
// them, fewer for short ones), while the device has room for all of them.
// Measured, us, held / streamed, rows of 128256 bf16: top logits 8 rows 11.3 /
// 16.4, 48 rows 15.3 / 16.7, 76 rows 22.5 / 16.7; loss and gradient 8 rows 8.4 /
// 17.5, 48 rows 11.4 / 17.8, 76 rows 18.1 / 18.0.
template <typename E>
static int held_cluster(int64_t N, int V, int NT, int *share_bytes) {
  constexpr int VE = Elt<E>::kPerVec;
  const int64_t nvec = ((int64_t)V + 2 * VE - 2) / VE;
  int64_t cs = (nvec * 16 + kHeldBytes - 1) / kHeldBytes;   // at most 16: 1 MB + 16 bytes
  if (N * std::max<int64_t>(cs, 8) > (int64_t)kHeldCtas * sm_count()) return 0;
  while (cs < 8 && nvec / (cs + 1) >= 2 * NT) ++cs;
  *share_bytes = (int)((nvec + cs - 1) / cs * 16);
  return (int)cs;
}

// Launches fn(P) with N clusters of cs CTAs, as a programmatic dependent of the
// stream's previous kernel.
template <typename P>
static cudaError_t launch_held(void (*fn)(const P), const P &params, int N, int cs, int NT,
                               int smem, cudaStream_t s) {
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

// Launches fn(P) with two CTAs of NT threads per SM, or one per row.
template <typename P>
static cudaError_t launch_streamed(void (*fn)(const P), const P &params, int N, int NT, int smem,
                                   cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(N, 2 * sm_count()), 1, 1);
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, params);
}

// ------------------------------------------------------ rows streamed --
// For many rows: one CTA takes rows first, first + grid, ... from end to end (each `passes`
// times in a row).  Every thread copies its own vectors, U a step, into its
// own places of a ring of D steps; the copies run on across the ends of
// passes and rows, so that what happens there costs no bandwidth.  The second
// pass goes backwards: what L2 still holds of the row is its end.  Rows of
// weight 0 are left out.  In a step a warp has 32 U vectors side by side:
// its vector u of the step that begins at q is q + at() + 32 u.
template <typename E, int NT, int U, int D>
struct RowStream {
  static constexpr int kStep = NT * U;                  // vectors of a step
  static constexpr int kBytes = D * kStep * 16;
  uint32_t ring;        // this thread's place of the ring
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
      : ring(smem_u32(ring_ + threadIdx.x)), base(base_), weight(weight_), stride(stride_), N(N_), V(V_),
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
    pass = q = 0;
    src = view.row + ((int64_t)at() * RowView<E>::VE - view.hp) * Elt<E>::kSize;
  }
  __device__ __forceinline__ void ask() {
    const uint32_t to = ring + put * (kStep * 16);
    if (row < N) {
      if (q > 0 && q + kStep < view.nvec) {   // no end of the row in the step
#pragma unroll
        for (int u = 0; u < U; ++u) row_async16(to + u * (NT * 16), src + u * 512);
      } else {
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const int i = q + at() + u * 32;
          if (i >= view.nvec) break;
          if (view.whole(i)) row_async16(to + u * (NT * 16), src + u * 512);
          else sts16(to + u * (NT * 16), view.load(i));
        }
      }
      const int way = pass == 0 ? kStep : -kStep;
      q += way;
      src += (int64_t)way * 16;
      if (q >= view.nvec || q < 0) {
        if (++pass < passes) {   // back over the row, from the step just asked for
          q -= kStep;
          src -= kStep * 16;
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
    const uint32_t from = ring + take * (kStep * 16);
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = lds16(from + u * (NT * 16));
    take = take + 1 == D ? 0 : take + 1;
    ask();
  }
  // vector u of the step `ahead` (< D - 1) steps after the oldest, once it is there
  __device__ __forceinline__ uint4 peek(int ahead, int u) const {
    int slot = take + ahead;
    slot = slot >= D ? slot - D : slot;
    return lds16(ring + (slot * kStep + u * NT) * 16);
  }
};

// ------------------------------------------------- exponentials of vectors --
// 2^((x - m) c) for the elements of vectors, in packed pairs.  Where m c is of
// ordinary size: 2^(x c - h) with h = m c rounded, one fused operation.  What
// the rounding of h leaves, m c - h, is as large as 2^-24 |m c| and another
// number for every m (each thread has its own, and the row has one in the second
// pass): `fix` = 2^(h - m c) takes it out of a sum, or of a factor, of such terms.
// From |m c| = kFar on (FAR) the difference comes first: fix, by its first two
// terms, is good to 2^-26 below that, and a finite stand-in for -inf (-1e10,
// the type's lowest value) would leave an h whose rounding passes 2^128.
// Either way the term of m itself is 1.
constexpr float kFar = 4096.f;
struct ExpBase {
  uint64_t o, c;   // FAR: (-m, c), else (-h, c)
  float fix;
  bool far;
  __device__ __forceinline__ ExpBase(float m, float cc) {
    const float s = m == neg_inf() ? 0.f : m, h = s * cc;
    far = fabsf(h) >= kFar;
    fix = far ? 1.f : fmaf(fmaf(-s, cc, h), 0.693147180559945309f, 1.f);
    const float b = far ? -s : -h;
    o = pk2(b, b);
    c = pk2(cc, cc);
  }
  template <bool FAR>
  __device__ __forceinline__ void pair(uint64_t x, float &a, float &b) const {
    upk2(FAR ? mul2(add2(x, o), c) : fma2(x, c, o), a, b);
    a = ex2(a);
    b = ex2(b);
  }
};
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
  static __device__ __forceinline__ uint64_t widen(uint32_t w) {
    return pk2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  template <bool FAR, typename Base>
  static __device__ __forceinline__ uint64_t sum(const uint4 &v, const Base &B, uint64_t acc) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      B.template pair<FAR>(widen(w[i]), a, b);
      acc = add2(acc, pk2(a, b));
    }
    return acc;
  }
  template <bool FAR>
  static __device__ __forceinline__ uint4 scaled(const uint4 &v, const ExpBase &B, uint64_t s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      B.pair<FAR>(widen(w[i]), a, b);
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
  static __device__ __forceinline__ uint64_t two(uint32_t x, uint32_t y) {
    return pk2(__uint_as_float(x), __uint_as_float(y));
  }
  template <bool FAR, typename Base>
  static __device__ __forceinline__ uint64_t sum(const uint4 &v, const Base &B, uint64_t acc) {
    float a, b;
    B.template pair<FAR>(two(v.x, v.y), a, b);
    acc = add2(acc, pk2(a, b));
    B.template pair<FAR>(two(v.z, v.w), a, b);
    return add2(acc, pk2(a, b));
  }
  template <bool FAR>
  static __device__ __forceinline__ uint4 scaled(const uint4 &v, const ExpBase &B, uint64_t s) {
    float f[4];
    B.pair<FAR>(two(v.x, v.y), f[0], f[1]);
    B.pair<FAR>(two(v.z, v.w), f[2], f[3]);
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
  // U vectors at once: one maximum (b), one rescaling
  template <int U>
  __device__ __forceinline__ void add(const uint4 *v, float c) {
    add<U>(v, c, VecExp<E>::template largest<U>(v));
  }
  template <int U>
  __device__ __forceinline__ void add(const uint4 *v, float c, float b) {
    if (b > m) {
      z *= ex2((m - b) * c);
      m = b;
    }
    const ExpBase B(m, c);
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
    z = fmaf(x + y, B.fix, z);
  }
  // this thread's vectors of a share: NT apart, U at a time
  template <int NT, int U>
  __device__ __forceinline__ void add_share(const Held<E> &H, float c) {
    int i = threadIdx.x;
    for (; i + (U - 1) * NT < H.n; i += U * NT) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = H.get(i + u * NT);
      add<U>(v, c);
    }
#pragma unroll 1
    for (; i < H.n; i += NT) {
      const uint4 v = H.get(i);
      add<1>(&v, c);
    }
  }
  // the warp's, in every lane
  __device__ __forceinline__ void warp(float c) {
    const float b = rmax_f(m);
    z = warp_sum(z * ex2((m - (b == neg_inf() ? 0.f : b)) * c));
    m = b;
  }
  // the block's, in every thread; wm and wz hold a float per warp
  template <int NW>
  __device__ __forceinline__ void block(float c, float *wm, float *wz) {
    warp(c);
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

// ------------------------------------------------------- keys and bounds --
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ unsigned long long top_key(float x, int i) {
  return ((unsigned long long)((unsigned)ford(x) ^ 0x80000000u) << 32) | (unsigned)~i;
}
__device__ __forceinline__ int key_index(unsigned long long key) { return (int)~(unsigned)key; }
__device__ __forceinline__ float key_value(unsigned long long key) {
  return fdeord((int)((unsigned)(key >> 32) ^ 0x80000000u));
}

// The upper 16 bits of a value's ordered image.
__device__ __forceinline__ unsigned short top_key16(float x) {
  return (unsigned short)(((unsigned)ford(x) ^ 0x80000000u) >> 16);
}

// The largest value (of the upper 16 bits' grid) that k of NT keys reach, found
// by one warp bit by bit; kLowest where fewer are finite.
template <int NT>
__device__ __forceinline__ float top_bound_warp(const unsigned short *keys, int k) {
  constexpr int J = NT / 32;
  unsigned key[J], lo = 0xffffu, hi = 0u;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    key[j] = keys[j * 32 + (threadIdx.x & 31)];
    lo = min(lo, key[j]);
    hi = max(hi, key[j]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  // the bits that all have in common are known
  const int from = 31 - __clz(lo ^ hi);
  unsigned r = lo & ~((1u << (from + 1)) - 1u);
#pragma unroll 1
  for (int bit = from; bit >= 0; --bit) {
    const unsigned t = r | (1u << bit);
    int n = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) n += key[j] >= t;
    if (__reduce_add_sync(0xffffffffu, n) >= k) r = t;
  }
  // 0x007f is -inf's
  return r > 0x007fu ? fdeord((int)((r << 16) ^ 0x80000000u)) : kLowest;
}

// top_bound_warp of the block's threads by their `best`, in every thread;
// meanwhile() is what the threads do between its barriers.
template <int NT, typename F>
__device__ __forceinline__ float top_bound(float best, int k, unsigned short *keys, float *out,
                                           F meanwhile) {
  keys[threadIdx.x] = top_key16(best);
  __syncthreads();
  meanwhile();
  if (threadIdx.x < 32) {
    const float b = top_bound_warp<NT>(keys, k);
    if (threadIdx.x == 0) *out = b;
  }
  __syncthreads();
  return *out;
}

}  // namespace sdv
