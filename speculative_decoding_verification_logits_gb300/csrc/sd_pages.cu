// Pages of a paged cache: forking and extending block tables, giving pages
// back, moving the pages in use to the front.  Integer work on page ids and
// their counts; the contents are sd_kvcopy.cu's.
//
// Whatever needs the free pages in order goes in two launches: the first
// writes one bit per page and the counts of 8192-page chunks (beside it, one
// CTA plans the rows); in the second every CTA finds the pages of its own ranks
// from the counts and the bits of one chunk.  So no CTA waits for another, and
// nothing depends on the order in which they run.  Small calls take both steps
// in one launch of one cluster (fork_cluster, compact_cluster).
//
// Measured on the GPU: a fork of 512 rows of 513 slots (64 groups of 8 that share 400
// pages) 12.6 us, of one row into 8 8.2; 171 rows of 513 slots given back, half of
// them shared, 3.3; compaction of 65536 pages with 64 tables of 513 slots 9.5, of
// 2000 pages 7.9; 9 entries more in each of 64 rows of 513 slots, in place, 10.3.  None
// of them moves more than 3 MB: what they take are chains of dependent loads
// through L2 (parent, length, last page, its count; counts, bits, page) and
// launches.  A row that gets many pages is slow: one thread counts its empty slots and one warp
// fills them, 513 pages of one row 71 us, 8192 1058.

#include "sd_rows.cuh"
#include "sd_kv.h"

namespace sdv {

constexpr int kPgNT = 1024;              // threads of a chunk's CTA, and of the plan's
constexpr int kPgChunk = 8192;           // pages of a chunk
constexpr int kPgWords = kPgChunk / 32;
constexpr int kRowNT = 128;              // threads for the slots of a row
constexpr int kRowTeam = kRowNT + 32;    // and a warp for its new pages
constexpr int kRowU = 4;                 // slots of one of them in flight
constexpr int64_t kForkCluster = 1 << 15;     // slots of the rows that one cluster takes
constexpr int64_t kCompactCluster = 1 << 14;  // pages, or entries of tables, that one takes
constexpr int kRowSlots = 512;           // slots that get pages at a time

static int page_chunks(int N) { return (N + kPgChunk - 1) / kPgChunk; }

__device__ __forceinline__ void pdl() {
  // a programmatic dependent of the stream's previous kernel: nothing is read
  // before it has finished; the next launch may be scheduled at once
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void set_status(int32_t *status, unsigned bits) {
  if (status) atomicOr(status, (int)bits);
}

// One holder less of U pages at a time, -1 and ids that are none passed over; a page that nobody holds
// stays at zero.  held: how many held each.
template <int U>
__device__ __forceinline__ void give_back(int32_t *refs, int N, const int (&e)[U], int (&held)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    held[u] = 0;
    if ((unsigned)e[u] < (unsigned)N) held[u] = atomicSub(refs + e[u], 1);
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if ((unsigned)e[u] < (unsigned)N && held[u] <= 0) atomicAdd(refs + e[u], 1);
}

// The bits of a chunk's pages that are free (or in use), and how many.
__device__ __forceinline__ void chunk_bits(int chunk, int N, const int32_t *refs, bool free,
                                           uint32_t *bits, int32_t *counts) {
  __shared__ int total;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  int mine = 0;
  int ref[kPgChunk / kPgNT];
#pragma unroll
  for (int u = 0; u < kPgChunk / kPgNT; ++u) {
    const int p = chunk * kPgChunk + u * kPgNT + threadIdx.x;
    ref[u] = p < N ? ld_int(refs + p) : free ? 1 : 0;
  }
#pragma unroll
  for (int u = 0; u < kPgChunk / kPgNT; ++u) {
    const uint32_t word = ballot(free ? ref[u] == 0 : ref[u] > 0);
    if ((threadIdx.x & 31) == 0) {
      bits[(int64_t)chunk * kPgWords + (u * kPgNT + threadIdx.x) / 32] = word;
      mine += __popc(word);
    }
  }
  if ((threadIdx.x & 31) == 0) atomicAdd(&total, mine);
  __syncthreads();
  if (threadIdx.x == 0) counts[chunk] = total;
  __syncthreads();
}

// ------------------------------------------------------------------- fork --
struct ForkRow {
  int parent, len;     // -1: an empty row
  int flags;           // kHeir, kLead, kCopy
  int kids;            // rows with this parent
  int first, pages;    // rank of the first page it gets, and how many
  int pair;            // rank of its copy
  int last;            // the partly filled page
};
constexpr int kHeir = 1, kLead = 2, kCopy = 4;

struct ForkParams {
  int rows_in, R, per_in, per_out, M, page_size, append, keep, N, nchunk;
  const int32_t *parents, *table, *kv_len;
  int32_t *refs, *table_out, *len_out, *src, *dst, *fill, *count, *status;
  // workspace
  uint32_t *bits;
  int32_t *counts, *kids;
  ForkRow *plan;
  unsigned *done;   // CTAs that have seen to their rows, and in the upper half those with doubts
};

__device__ __forceinline__ int fork_parent(const ForkParams &P, int r, bool tell) {
  if (!P.parents) return r;
  const int p = ld_int(P.parents + r);
  if (p == -1) return -1;
  if (p < 0 || p >= P.per_in) {
    if (tell) set_status(P.status, SD_STATUS_BAD_PARENT);
    return -1;
  }
  return r / P.per_out * P.per_in + p;
}

struct ForkSpan {
  int full, part, used, need;   // slots: full pages, entries of the last, all, with room
  bool cut;                     // the table bounds the room
  __device__ __forceinline__ ForkSpan(const ForkParams &P, int len) {
    full = len / P.page_size;
    part = len - full * P.page_size;
    used = full + (part > 0);
    const int64_t want = ((int64_t)len + P.append + P.page_size - 1) / P.page_size;
    cut = want > P.M;
    need = (int)min(want, (int64_t)P.M);
  }
};

// What a row's plan reads of its parent.
struct ForkLook {
  int parent, len, last, refs;   // refs: of the last page
};
__device__ __forceinline__ ForkLook fork_look(const ForkParams &P, int r) {
  ForkLook k = {r < P.R ? fork_parent(P, r, true) : -1, 0, -1, 0};
  if (k.parent >= 0) {
    k.len = (int)min((int64_t)max(ld_int(P.kv_len + k.parent), 0), (int64_t)P.M * P.page_size);
    const ForkSpan s(P, k.len);
    if (s.part) k.last = ld_int(P.table + (int64_t)k.parent * P.M + s.full);
    if ((unsigned)k.last < (unsigned)P.N) k.refs = ld_int(P.refs + k.last);
  }
  return k;
}

// The rows' plan, by one CTA: heirs, and the ranks of the pages and copies that
// the rows need.
__device__ void plan_rows(const ForkParams &P, int *smem) {
  constexpr int NT = kPgNT, NW = NT / 32;
  int *first = smem, *kids = smem + P.rows_in;   // of each old row
  __shared__ unsigned long long warp_sum_s[NW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const ForkLook look0 = fork_look(P, tid);   // under way meanwhile
  for (int p = tid; p < P.rows_in; p += NT) {
    first[p] = INT32_MAX;
    kids[p] = 0;
  }
  __syncthreads();
  for (int r = tid; r < P.R; r += NT) {
    const int p = r == tid ? look0.parent : fork_parent(P, r, false);
    if (p < 0) continue;
    atomicMin(&first[p], r);
    atomicAdd(&kids[p], 1);
  }
  __syncthreads();
  for (int p = tid; p < P.rows_in; p += NT) P.kids[p] = kids[p];
  unsigned long long before = 0ull;   // pages, and copies in the upper half
  for (int r0 = 0; r0 < P.R; r0 += NT) {
    const int r = r0 + tid;
    const ForkLook look = r0 == 0 ? look0 : fork_look(P, r);
    ForkRow row = {look.parent, look.len, 0, 0, 0, 0, 0, look.last};
    if (row.parent >= 0) {
      const int p = row.parent;
      const ForkSpan s(P, row.len);
      const int32_t *old = P.table + (int64_t)p * P.M;
      const bool lead = first[p] == r, heir = lead && !P.keep;
      row.kids = kids[p];
      row.flags = (lead ? kLead : 0) | (heir ? kHeir : 0);
      if (s.cut) set_status(P.status, SD_STATUS_NO_PAGE);
      if (s.part && (unsigned)row.last < (unsigned)P.N && !(heir && look.refs == 1)) {
        row.flags |= kCopy;
        row.pages = 1;
      }
      if (heir) {
#pragma unroll 4
        for (int j = s.used; j < s.need; ++j) row.pages += (unsigned)ld_int(old + j) >= (unsigned)P.N;
      } else {
        row.pages += s.need - s.used;
      }
    }
    // the rows before this one
    const unsigned long long mine =
        (unsigned)row.pages | (unsigned long long)((row.flags & kCopy) != 0) << 32;
    unsigned long long x = mine;
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      x += lane >= o ? y : 0ull;
    }
    if (lane == 31) warp_sum_s[warp] = x;
    __syncthreads();
    unsigned long long all = 0ull, at = before + x - mine;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      at += i < warp ? warp_sum_s[i] : 0ull;
      all += warp_sum_s[i];
    }
    before += all;
    row.first = (int)(unsigned)at;
    row.pair = (int)(at >> 32);
    if (r < P.R) P.plan[r] = row;
    __syncthreads();
  }
  if (tid == 0) {
    *P.count = (int)(before >> 32);
    *P.done = 0u;
  }
}

__global__ void __launch_bounds__(kPgNT) sd_kv_plan_kernel(const ForkParams P) {
  extern __shared__ int plan_smem[];
  pdl();
  if (blockIdx.x == 0) plan_rows(P, plan_smem);
  else chunk_bits(blockIdx.x - 1, P.N, P.refs, true, P.bits, P.counts);
}

// Calls f(rank, page) for the free pages of ranks [q, end), by one warp; returns
// the first rank that there is none for (end if there are all).
template <typename F>
__device__ __forceinline__ int free_pages(const uint32_t *bits, const int32_t *counts, int nchunk,
                                          int q, int end, F f) {
  const int lane = threadIdx.x & 31;
  int before = 0;   // free pages before chunk c0
  for (int c0 = 0; c0 < nchunk && q < end; c0 += 32) {
    const int n = c0 + lane < nchunk ? ld_int(counts + c0 + lane) : 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      upto += lane >= o ? y : 0;
    }
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    while (q < end && q < before + all) {
      // the chunk that holds rank q
      const int k = __popc(__ballot_sync(0xffffffffu, before + upto <= q));
      const int start = before + __shfl_sync(0xffffffffu, upto - n, k);
      const int stop = before + __shfl_sync(0xffffffffu, upto, k);
      const uint4 *w = reinterpret_cast<const uint4 *>(bits + (int64_t)(c0 + k) * kPgWords);
      const uint4 a = ld16(w + lane * 2), b = ld16(w + lane * 2 + 1);
      const uint32_t word[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      int here = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) here += __popc(word[i]);
      int rank = here;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, rank, o);
        rank += lane >= o ? y : 0;
      }
      rank += start - here;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int more = __popc(word[i]);
        if (rank + more > q && rank < end) {
          uint32_t m = word[i];
          for (int at = rank; m && at < end; ++at, m &= m - 1)
            if (at >= q) f(at, (c0 + k) * kPgChunk + (lane * 8 + i) * 32 + __ffs(m) - 1);
        }
        rank += more;
      }
      q = min(end, stop);
      __syncwarp();
    }
    before += all;
  }
  return q;
}

// One holder less of U pages at a time, -1 passed over.  What a call adds to the counts and takes from
// them comes in any order, so nothing is held against zero before all of it is there
// (fork_settle).  A page that was free before the call has nothing to give back, though it may
// have been handed out by now.  Returns whether a count may end below zero.
template <int U>
__device__ __forceinline__ bool fork_give_back(const ForkParams &P, const int (&e)[U], unsigned &bad) {
  int held[U];
  uint32_t word[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool page = (unsigned)e[u] < (unsigned)P.N;
    held[u] = page ? atomicSub(P.refs + e[u], 1) : 1;
    word[u] = page ? ld4(P.bits + (e[u] >> 5)) : 0u;
    if (!page && e[u] != -1) bad |= SD_STATUS_BAD_PAGE;
  }
  bool doubt = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (word[u] >> (e[u] & 31) & 1u) {
      atomicAdd(P.refs + e[u], 1);
      bad |= SD_STATUS_BAD_PAGE;
    } else {
      doubt |= held[u] <= 0;
    }
  }
  return doubt;
}

// At the end of every CTA: the last one raises counts that were given back too often to zero, where
// any CTA saw one at zero.  Takes 1.6 us of a fork of 512 rows of 513 slots (11.0 without).
__device__ __forceinline__ void fork_settle(const ForkParams &P, bool doubt) {
  __shared__ bool settles;
  if (P.keep) return;   // nothing is given back
  doubt = __syncthreads_or(doubt);
  if (threadIdx.x == 0) {
    unsigned before;   // acquires what the CTAs before have done, releases what this one has
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                 : "=r"(before)
                 : "l"(P.done), "r"(doubt ? 0x10001u : 1u)
                 : "memory");
    settles = (before & 0xffffu) == gridDim.x - 1 && (doubt || before >> 16);
  }
  __syncthreads();
  if (!settles) return;
  bool bad = false;
  for (int p = threadIdx.x; p < P.N; p += blockDim.x)
    if (ld_int(P.refs + p) < 0) {
      P.refs[p] = 0;
      bad = true;
    }
  if (bad) set_status(P.status, SD_STATUS_BAD_PAGE);
}
static_assert(SD_MAX_ROWS < 1 << 15, "CTAs are counted in 16 bits");

// Row i, new and old, by five warps (tid in them): four share the new row's slots out and give
// the old one's pages back, the fifth finds the new row's own pages and gives the one back that an
// heir copied.  Returns fork_give_back's doubt.
__device__ __forceinline__ bool fork_row(const ForkParams &P, int i, int tid, int *slots) {
  const int lane = tid & 31;
  unsigned bad = 0u;
  bool doubt = false;
  const int kids = i < P.rows_in ? ld_int(P.kids + i) : 1;
  if (i < P.R) {
    const ForkRow row = P.plan[i];
    ForkSpan s(P, row.len);
    if (row.parent < 0) s.need = 0;   // an empty row has no room either
    const bool in_place = !P.parents, heir = row.flags & kHeir, copy = row.flags & kCopy;
    const int32_t *old = P.table + (int64_t)row.parent * P.M;
    int32_t *out = P.table_out + (int64_t)i * P.M;
    if (tid < kRowNT) {
      // whoever leads a parent's rows counts for all of them
      const int add = !(row.flags & kLead) ? 0 : P.keep ? row.kids : row.kids - 1;
      for (int j0 = tid; j0 < P.M; j0 += kRowU * kRowNT) {
        int e[kRowU];
#pragma unroll
        for (int u = 0; u < kRowU; ++u) {
          const int j = j0 + u * kRowNT;
          e[u] = j < P.M && row.parent >= 0 ? ld_int(old + j) : -1;
        }
#pragma unroll
        for (int u = 0; u < kRowU; ++u) {
          const int j = j0 + u * kRowNT;
          if (j >= P.M) break;
          // a page of its own comes here: in place it may be there already, so that the plan is
          // asked for the old one, which it found to be one
          if (j >= s.full && j < s.used && copy) continue;
          const bool page = (unsigned)e[u] < (unsigned)P.N;
          if (j < s.used && !page) bad |= SD_STATUS_BAD_PAGE;
          if (j < s.full && page && add) atomicAdd(P.refs + e[u], add);
          if (j >= s.used && j < s.need && !(heir && page)) continue;   // gets a page
          if (!in_place) out[j] = j < s.need || heir ? e[u] : -1;
        }
      }
    } else {
      if (lane == 0) {
        if (P.len_out) P.len_out[i] = row.len;
        if (i >= ld_int(P.count)) {
          P.src[i] = -1;
          P.dst[i] = -1;
          P.fill[i] = 0;
        }
        if (copy) P.fill[row.pair] = s.part;
      }
      // slots that get a page, in order, a batch at a time
      int j0 = s.used, done = 0;
      bool first = copy;
      while (done < row.pages) {
        int n = 0;
        if (first) {
          if (lane == 0) slots[0] = s.full;
          n = 1;
        }
        for (; j0 < s.need && n + 32 <= kRowSlots; j0 += 32) {
          const int j = j0 + lane;
          const int e = j < s.need && heir ? ld_int(old + j) : -1;
          const bool want = j < s.need && (unsigned)e >= (unsigned)P.N;
          if (want && e != -1) bad |= SD_STATUS_BAD_PAGE;
          const unsigned m = __ballot_sync(0xffffffffu, want);
          if (want) slots[n + __popc(m & ((1u << lane) - 1u))] = j;
          n += __popc(m);
        }
        __syncwarp();
        if (n == 0) break;
        const int q = row.first + done;
        const int got = free_pages(P.bits, P.counts, P.nchunk, q, q + n, [&](int rank, int page) {
          out[slots[rank - q]] = page;
          atomicAdd(P.refs + page, 1);
          if (first && rank == q) {
            P.src[row.pair] = row.last;
            P.dst[row.pair] = page;
          }
        });
        // the old page of a copy: its row holds it on where no page was found for the copy
        const bool stays = first && heir && got == q;
        if (first && heir && !stays && lane == 0) {
          const int page[1] = {row.last};
          doubt |= fork_give_back(P, page, bad);
        }
        for (int x = got - q + lane; x < n; x += 32) {   // none left
          out[slots[x]] = stays && x == 0 ? row.last : -1;
          bad |= SD_STATUS_NO_PAGE;
          if (first && x == 0) {
            P.src[row.pair] = -1;
            P.dst[row.pair] = -1;
          }
        }
        __syncwarp();
        done += n;
        first = false;
      }
    }
  }
  if (tid < kRowNT && !P.keep && kids == 0) {   // ends without an heir
    const int32_t *old = P.table + (int64_t)i * P.M;
    for (int j0 = tid; j0 < P.M; j0 += kRowU * kRowNT) {
      int e[kRowU];
#pragma unroll
      for (int u = 0; u < kRowU; ++u) e[u] = j0 + u * kRowNT < P.M ? ld_int(old + j0 + u * kRowNT) : -1;
      doubt |= fork_give_back(P, e, bad);
    }
  }
  if (bad) set_status(P.status, bad);
  return doubt;
}

__global__ void __launch_bounds__(kRowTeam) sd_kv_rows_kernel(const ForkParams P) {
  __shared__ int slots[kRowSlots];
  pdl();
  fork_settle(P, fork_row(P, blockIdx.x, threadIdx.x, slots));
}

// Both steps in one launch, for few rows: by one cluster, with its barrier between them.
__global__ void __launch_bounds__(kPgNT) sd_kv_fork_kernel(const ForkParams P) {
  constexpr int kTeams = kPgNT / kRowTeam;
  extern __shared__ int plan_smem[];
  __shared__ int slots[kTeams][kRowSlots];
  pdl();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), cs = (int)cluster.num_blocks();
  if (rank == 0) plan_rows(P, plan_smem);
  else
    for (int c = rank - 1; c < P.nchunk; c += cs - 1)
      chunk_bits(c, P.N, P.refs, true, P.bits, P.counts);
  cluster.sync();
  const int team = threadIdx.x / kRowTeam;
  const int rows = max(P.R, P.rows_in);
  bool doubt = false;
  for (int i = rank * kTeams + team; team < kTeams && i < rows; i += cs * kTeams) {
    doubt |= fork_row(P, i, threadIdx.x % kRowTeam, slots[team]);
    __syncwarp();
  }
  fork_settle(P, doubt);
}

// ------------------------------------------------------------------- free --
constexpr int kFreeNT = 256, kFreeU = 4;

__global__ void __launch_bounds__(kFreeNT) sd_kv_free_kernel(int64_t cols, int parts, int32_t *pages,
                                                             const uint8_t *which,
                                                             const int32_t *count, int clear, int N,
                                                             int32_t *refs, int32_t *status) {
  pdl();
  const int64_t row = blockIdx.x / parts;
  const int64_t c0 = (int64_t)(blockIdx.x % parts) * (kFreeNT * kFreeU) + threadIdx.x;
  if (which && !ld1(which + row)) return;
  int64_t end = cols;
  if (count) end = min(end, (int64_t)ld_int(count) - row * cols);
  int e[kFreeU];
#pragma unroll
  for (int u = 0; u < kFreeU; ++u) {
    const int64_t c = c0 + u * kFreeNT;
    e[u] = c < end ? ld_int(pages + row * cols + c) : -1;
  }
  bool bad = false;
  int held[kFreeU];
  give_back(refs, N, e, held);
#pragma unroll
  for (int u = 0; u < kFreeU; ++u) {
    if (e[u] == -1) continue;
    bad |= held[u] <= 0;
    if (clear) pages[row * cols + c0 + u * kFreeNT] = -1;
  }
  if (bad) set_status(status, SD_STATUS_BAD_PAGE);
}

// ---------------------------------------------------------------- compact --
struct CompactParams {
  int N, nchunk;
  int64_t n_table;
  int32_t *refs, *table, *src, *dst, *count, *live, *new_ids, *status;
  // workspace: bits of the pages in use, counts per chunk, pages in use before
  // each word; pages in use, those below that many, and the moves
  uint32_t *bits;
  int32_t *counts, *before, *meta;
};

__global__ void __launch_bounds__(kPgNT) sd_kv_live_kernel(const CompactParams P) {
  pdl();
  chunk_bits(blockIdx.x, P.N, P.refs, false, P.bits, P.counts);
}

// The block's sum, in every thread.
__device__ __forceinline__ int block_sum(int v, int *warps) {
  __syncwarp();
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kPgNT / 32; ++i) v += warps[i];
  return v;
}

// Of page p: how many pages in use lie before it.
__device__ __forceinline__ int used_before(const CompactParams &P, int p, uint32_t word) {
  return ld_int(P.before + (p >> 5)) + __popc(word & ((1u << (p & 31)) - 1u));
}

// A page in use at or above L is the source of move `used before it` - `used
// before L`, a free one below L the destination of move `free before it`.
__device__ __forceinline__ void chunk_moves(const CompactParams &P, int chunk) {
  __shared__ int warps[kPgNT / 32];
  __shared__ int before_s[kPgWords];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int all = 0, ahead = 0;
  for (int c = tid; c < P.nchunk; c += kPgNT) {
    const int n = ld_int(P.counts + c);
    all += n;
    ahead += c < chunk ? n : 0;
  }
  const int L = block_sum(all, warps);
  ahead = block_sum(ahead, warps);
  int low = 0;   // in use before page L
  const int cL = L / kPgChunk;
  for (int c = tid; c < min(cL, P.nchunk); c += kPgNT) low += ld_int(P.counts + c);
  if (cL < P.nchunk && tid < kPgWords) {
    const int bit0 = tid * 32, cut = L - cL * kPgChunk;
    uint32_t w = ld4(P.bits + (int64_t)cL * kPgWords + tid);
    if (bit0 + 32 > cut) w = bit0 >= cut ? 0u : w & ((1u << (cut - bit0)) - 1u);
    low += __popc(w);
  }
  low = block_sum(low, warps);
  // in use before each word of this chunk
  const uint32_t word = tid < kPgWords ? ld4(P.bits + (int64_t)chunk * kPgWords + tid) : 0u;
  int upto = __popc(word);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    upto += lane >= o ? y : 0;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = upto;
  __syncthreads();
  if (tid < kPgWords) {
    int at = ahead + upto - __popc(word);
    for (int i = 0; i < warp; ++i) at += warps[i];
    before_s[tid] = at;
    P.before[(int64_t)chunk * kPgWords + tid] = at;
  }
  __syncthreads();
  for (int u = 0; u < kPgChunk / kPgNT; ++u) {
    const int w = (u * kPgNT + tid) / 32, p = chunk * kPgChunk + u * kPgNT + tid;
    const uint32_t bits = ld4(P.bits + (int64_t)chunk * kPgWords + w);
    const int used = before_s[w] + __popc(bits & ((1u << lane) - 1u));
    const bool live = bits >> lane & 1u;
    if (p >= P.N) continue;
    if (live && p >= L) P.src[used - low] = p;
    if (!live && p < L) P.dst[p - used] = p;
  }
  if (chunk == 0 && tid == 0) {
    *P.live = L;
    *P.count = L - low;
    P.meta[0] = L;
    P.meta[1] = low;
  }
}

// What becomes of page i, and of entry i of the tables.
__device__ __forceinline__ void page_moved(const CompactParams &P, int64_t i, int L, int low) {
  if (i < P.N) {
    const int p = (int)i;
    const uint32_t word = ld4(P.bits + (p >> 5));
    int to = -1;
    if (word >> (p & 31) & 1u) {
      to = p;
      if (p >= L) {
        to = ld_int(P.dst + used_before(P, p, word) - low);
        P.refs[to] = ld_int(P.refs + p);
        P.refs[p] = 0;
      }
    }
    P.new_ids[p] = to;
    if (p < P.N / 2 && p >= L - low) {
      P.src[p] = -1;
      P.dst[p] = -1;
    }
  }
  if (i < P.n_table) {
    const int e = ld_int(P.table + i);
    if (e == -1) return;
    const uint32_t word = (unsigned)e < (unsigned)P.N ? ld4(P.bits + (e >> 5)) : 0u;
    if (!(word >> (e & 31) & 1u)) set_status(P.status, SD_STATUS_BAD_PAGE);
    else if (e >= L) P.table[i] = ld_int(P.dst + used_before(P, e, word) - low);
  }
}

__global__ void __launch_bounds__(kPgNT) sd_kv_moves_kernel(const CompactParams P) {
  pdl();
  chunk_moves(P, blockIdx.x);
}
__global__ void __launch_bounds__(256) sd_kv_moved_kernel(const CompactParams P) {
  pdl();
  page_moved(P, blockIdx.x * (int64_t)blockDim.x + threadIdx.x, ld_int(P.meta), ld_int(P.meta + 1));
}

// The three steps in one launch, for small pools: by one cluster, with its barrier between them.
__global__ void __launch_bounds__(kPgNT) sd_kv_compact_kernel(const CompactParams P) {
  pdl();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), cs = (int)cluster.num_blocks();
  for (int c = rank; c < P.nchunk; c += cs) chunk_bits(c, P.N, P.refs, false, P.bits, P.counts);
  cluster.sync();
  for (int c = rank; c < P.nchunk; c += cs) chunk_moves(P, c);
  cluster.sync();
  const int L = ld_int(P.meta), low = ld_int(P.meta + 1);
  const int64_t n = max((int64_t)P.N, P.n_table);
  for (int64_t i = rank * kPgNT + threadIdx.x; i < n; i += cs * kPgNT) page_moved(P, i, L, low);
}

// Programmatic dependents of the stream's previous kernel.
struct PageLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  PageLaunch(int64_t grid, int block, int smem, cudaStream_t s, int cluster = 1) {
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
  PageLaunch(const PageLaunch &) = delete;
};

// CTAs of the one cluster that does a small call, 0: several launches are faster.  A launch costs
// the host 3 to 5 us, which is what small calls wait for; on the GPU alone, where the launches
// overlap, the cluster is a little behind.  Measured, us, one launch / several, call (GPU
// alone): fork of one prompt into 8 rows of 513 slots 56 (8.3) / 65 (7.6) with its copies,
// compaction of 2000 pages 67 (8.1) / 77 (7.3) with its copies; compaction of 65536 pages (15.5 / 9.5)
// and a fork of 512 rows (48 / 12.6) are the GPU's.
constexpr int kMaxCluster = 8;
static int fork_cluster(int rows, int M, int nchunk) {
  constexpr int kTeams = kPgNT / kRowTeam;
  if ((int64_t)rows * std::max(M, 1) > kForkCluster || rows > kMaxCluster * kTeams) return 0;
  int cs = 2;
  while (cs < kMaxCluster && (cs * kTeams < rows || cs - 1 < nchunk)) cs *= 2;
  return cs;
}
static int compact_cluster(int nchunk, int64_t places) {
  if (places > kCompactCluster) return 0;
  int cs = 1;
  while (cs < kMaxCluster && (cs < nchunk || (int64_t)cs * kPgNT < places)) cs *= 2;
  return cs;
}

static size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_kv_fork_workspace_size(int32_t rows_in, int32_t R, int32_t N) {
  if (rows_in < 0 || rows_in > SD_MAX_ROWS || R < 0 || R > SD_MAX_ROWS || N < 1 ||
      N > SD_MAX_PAGES)
    return 0;
  const size_t nchunk = (size_t)page_chunks(N);
  return nchunk * kPgWords * 4 + sizeof(ForkRow) * (size_t)R + round16(4 * nchunk) +
         round16(4 * (size_t)rows_in) + 16;
}

extern "C" sd_status_t sd_kv_fork(const sd_kv_fork_args *a, void *stream) {
  sdv::NvtxRange nvtx_range("sd_kv_fork");
  if (!a) return SD_ERR_INVALID_ARG;
  const size_t need = sd_kv_fork_workspace_size(a->rows_in, a->R, a->N);
  if (need == 0 || a->max_pages < 0 || a->page_size < 1 || a->append < 0 || a->groups < 0 ||
      (a->keep != 0 && a->keep != 1))
    return SD_ERR_INVALID_ARG;
  if ((int64_t)a->max_pages * a->page_size > INT32_MAX ||
      (int64_t)a->max_pages * a->R > INT32_MAX)
    return SD_ERR_INVALID_ARG;
  const bool in_place = !a->parents;
  if (in_place && a->R > 0 && (a->R != a->rows_in || a->table_out != a->table || a->keep || a->len_out))
    return SD_ERR_INVALID_ARG;
  if (a->groups > 0 && (a->R % a->groups || a->rows_in % a->groups)) return SD_ERR_INVALID_ARG;
  if (!a->count || !a->refs || !a->workspace || (uintptr_t)a->workspace % 16 ||
      a->workspace_bytes < need)
    return SD_ERR_INVALID_ARG;
  if (a->R > 0 && (!a->src || !a->dst || !a->fill || (!in_place && !a->len_out)))
    return SD_ERR_INVALID_ARG;
  if ((a->rows_in > 0 && !a->kv_len) ||
      (a->max_pages > 0 && ((a->rows_in > 0 && !a->table) || (a->R > 0 && !a->table_out))))
    return SD_ERR_INVALID_ARG;
  ForkParams P = {};
  P.rows_in = a->rows_in;
  P.R = a->R;
  P.per_in = a->groups > 0 ? a->rows_in / a->groups : a->rows_in;
  P.per_out = std::max(1, a->groups > 0 ? a->R / a->groups : a->R);
  P.M = a->max_pages;
  P.page_size = a->page_size;
  P.append = a->append;
  P.keep = a->keep;
  P.N = a->N;
  P.nchunk = page_chunks(a->N);
  P.parents = a->parents;
  P.table = a->table;
  P.kv_len = a->kv_len;
  P.refs = a->refs;
  P.table_out = a->table_out;
  P.len_out = a->len_out;
  P.src = a->src;
  P.dst = a->dst;
  P.fill = a->fill;
  P.count = a->count;
  P.status = a->status;
  uint8_t *ws = static_cast<uint8_t *>(a->workspace);
  P.bits = reinterpret_cast<uint32_t *>(ws);
  ws += (size_t)P.nchunk * kPgWords * 4;
  P.plan = reinterpret_cast<ForkRow *>(ws);
  ws += sizeof(ForkRow) * (size_t)P.R;
  P.counts = reinterpret_cast<int32_t *>(ws);
  P.kids = reinterpret_cast<int32_t *>(ws + round16(4 * (size_t)P.nchunk));
  P.done = reinterpret_cast<unsigned *>(P.kids + round16(4 * (size_t)P.rows_in) / 4);
  const int rows = std::max(P.R, P.rows_in);
  const int cs = fork_cluster(rows, P.M, P.nchunk);
  if (cs > 0) {
    PageLaunch one(cs, kPgNT, 8 * P.rows_in, (cudaStream_t)stream, cs);
    return cudaLaunchKernelEx(&one.cfg, sd_kv_fork_kernel, P) == cudaSuccess ? SD_OK : SD_ERR_CUDA;
  }
  static FuncAttrs attrs;
  attrs.apply((const void *)sd_kv_plan_kernel, 8 * SD_MAX_ROWS, false, "the fork's plan kernel");
  cudaStream_t s = (cudaStream_t)stream;
  PageLaunch plan(1 + P.nchunk, kPgNT, 8 * P.rows_in, s);
  cudaError_t e = cudaLaunchKernelEx(&plan.cfg, sd_kv_plan_kernel, P);
  if (e == cudaSuccess && rows > 0) {
    PageLaunch each(rows, kRowTeam, 0, s);
    e = cudaLaunchKernelEx(&each.cfg, sd_kv_rows_kernel, P);
  }
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}

extern "C" sd_status_t sd_kv_free(int64_t rows, int64_t cols, int32_t *pages, const uint8_t *which,
                                  const int32_t *count, int32_t clear, int32_t N, int32_t *refs,
                                  int32_t *status, void *stream) {
  sdv::NvtxRange nvtx_range("sd_kv_free");
  if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX || N < 1 || N > SD_MAX_PAGES)
    return SD_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return SD_OK;
  if (!pages || !refs) return SD_ERR_INVALID_ARG;
  if (rows > INT64_MAX / 4 / cols) return SD_ERR_INVALID_ARG;
  if (!which) {   // one long row
    cols *= rows;
    rows = 1;
  }
  const int64_t parts = (cols + kFreeNT * kFreeU - 1) / (kFreeNT * kFreeU);
  if (parts > INT32_MAX / rows) return SD_ERR_INVALID_ARG;
  PageLaunch launch(rows * parts, kFreeNT, 0, (cudaStream_t)stream);
  const cudaError_t e = cudaLaunchKernelEx(&launch.cfg, sd_kv_free_kernel, cols, (int)parts, pages,
                                           which, count, (int)clear, (int)N, refs, status);
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}

extern "C" size_t sd_kv_compact_workspace_size(int32_t N) {
  if (N < 1 || N > SD_MAX_PAGES) return 0;
  const size_t nchunk = (size_t)page_chunks(N);
  return nchunk * kPgWords * 8 + round16(4 * nchunk) + 16;
}

extern "C" sd_status_t sd_kv_compact(int32_t N, int32_t *refs, int64_t n_table, int32_t *table,
                                     int32_t *src, int32_t *dst, int32_t *count, int32_t *live,
                                     int32_t *new_ids, int32_t *status, void *workspace,
                                     size_t workspace_bytes, void *stream) {
  sdv::NvtxRange nvtx_range("sd_kv_compact");
  const size_t need = sd_kv_compact_workspace_size(N);
  if (need == 0 || n_table < 0 || n_table > (int64_t)INT32_MAX * 256) return SD_ERR_INVALID_ARG;
  if (!refs || !count || !live || !new_ids || (N > 1 && (!src || !dst)) ||
      (n_table > 0 && !table) || !workspace || (uintptr_t)workspace % 16 || workspace_bytes < need)
    return SD_ERR_INVALID_ARG;
  CompactParams P = {};
  P.N = N;
  P.nchunk = page_chunks(N);
  P.n_table = n_table;
  P.refs = refs;
  P.table = table;
  P.src = src;
  P.dst = dst;
  P.count = count;
  P.live = live;
  P.new_ids = new_ids;
  P.status = status;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  P.bits = reinterpret_cast<uint32_t *>(ws);
  ws += (size_t)P.nchunk * kPgWords * 4;
  P.before = reinterpret_cast<int32_t *>(ws);
  ws += (size_t)P.nchunk * kPgWords * 4;
  P.counts = reinterpret_cast<int32_t *>(ws);
  P.meta = reinterpret_cast<int32_t *>(ws + round16(4 * (size_t)P.nchunk));
  cudaStream_t s = (cudaStream_t)stream;
  if (const int cs = compact_cluster(P.nchunk, std::max<int64_t>(N, n_table))) {
    PageLaunch one(cs, kPgNT, 0, s, cs);
    return cudaLaunchKernelEx(&one.cfg, sd_kv_compact_kernel, P) == cudaSuccess ? SD_OK
                                                                                 : SD_ERR_CUDA;
  }
  PageLaunch chunks(P.nchunk, kPgNT, 0, s);
  cudaError_t e = cudaLaunchKernelEx(&chunks.cfg, sd_kv_live_kernel, P);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&chunks.cfg, sd_kv_moves_kernel, P);
  if (e == cudaSuccess) {
    PageLaunch each((std::max<int64_t>(N, n_table) + 255) / 256, 256, 0, s);
    e = cudaLaunchKernelEx(&each.cfg, sd_kv_moved_kernel, P);
  }
  return e == cudaSuccess ? SD_OK : SD_ERR_CUDA;
}

extern "C" size_t sd_kv_fork_args_size(void) { return sizeof(sd_kv_fork_args); }
