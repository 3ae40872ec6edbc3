// Bookkeeping of a paged cache's pages, and the copies that follow from it.
//
// The state is three int32 arrays (page tables, lengths, reference counts); a page is free when nobody holds
// it, so there is no free list to keep in order: allocation ranks the free pages with a prefix sum over the
// reference counts and hands them out lowest first, in the order of the requests.  That makes every result a
// function of the state alone.  The work is a few hundred KB of integers: bound by latency, not by bandwidth, hence
// one block that ranks and decides, with every read spread over its threads.
#pragma once

#include "layout.cuh"

namespace fa {

struct PagesArgs {
  int* table;
  long long table_stride;
  int* lens;
  int* refs;
  int S, P, page, M;
  int n;                           // requests
  const int* seqs;                 // extend, free: sequences; fork: sources
  const int* arg;                  // extend: tokens; fork: destinations
  int* copies;
  int* status;
  int* claim;                      // workspace: [S] first request that names the sequence
  int* snap;                       // workspace: [n] what a request asks for, by the state before the call; -1: refused
  int* prefix;                     // workspace: [n] pages wanted by the requests before
  int* list;                       // workspace: [P] free pages in order (extend, fork); new places (compact)
  int* info;                       // workspace: [1] pages in use (compact)
  uint32_t* dev_status;
};

constexpr int kPagesThreads = 1024; // at most
constexpr int kPagesPer = 8;       // consecutive pages a thread takes in a scan step

__device__ __forceinline__ int pages_of(int len, int page) { return len / page + (len % page != 0); }

// Sum of the threads before this one over one value per thread; *total is the block's sum.  All threads.  `turn` is 0 or
// 1, another one in the next call: with two buffers one barrier is enough.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* total, int turn) {
  __shared__ T part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T y = x;
  for (int o = 1; o < 32; o <<= 1) {
    const T z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) part[turn][warp] = y;
  __syncthreads();
  T s = lane < blockDim.x / 32 ? part[turn][lane] : 0;
  for (int o = 1; o < 32; o <<= 1) {
    const T z = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += z;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
  return y - x + (warp ? before : 0);
}

// Which of the kPagesPer pages from i on are free.
__device__ __forceinline__ unsigned free_bits(const PagesArgs& a, long long i) {
  unsigned bits = 0;
#pragma unroll
  for (int e = 0; e < kPagesPer; ++e)
    if (i + e < a.P && a.refs[i + e] <= 0) bits |= 1u << e;
  return bits;
}

// put(rank, i) for the pages begin <= i < end that are free (or not), in order, rank counting from 0.  `first` is
// free_bits of this thread's first pages, asked for in good time.  Returns how many there are, or some number >= enough
// when it stopped early.  All threads.
template <typename Put>
__device__ __forceinline__ int ranked(const PagesArgs& a, unsigned first, bool free, int begin, int end, long long enough,
                                      Put put) {
  const int step = blockDim.x * kPagesPer;
  int found = 0, turn = 0;
  __syncthreads();                 // an earlier scan's buffers have been read
  for (long long base = begin / step * step; base < end && found < enough; base += step, turn ^= 1) {
    const long long i0 = base + threadIdx.x * kPagesPer;
    unsigned bits = base == 0 ? first : free_bits(a, i0);
    if (!free) bits = ~bits;
#pragma unroll
    for (int e = 0; e < kPagesPer; ++e)
      if (i0 + e < begin || i0 + e >= end) bits &= ~(1u << e);
    bits &= (1u << kPagesPer) - 1;
    int total;
    int rank = found + block_scan<int>(__popc(bits), &total, turn);
    for (; bits; bits &= bits - 1) put(rank++, static_cast<int>(i0) + __ffs(bits) - 1);
    found += total;
  }
  return found;
}

// The lists of a call lie in shared memory while they fit: every step between two barriers then costs no round trip to L2.
constexpr int kPagesShared = 2048;
struct PagesShared {
  int claim[kPagesShared], snap[kPagesShared], prefix[kPagesShared], list[kPagesShared];
};
__device__ __forceinline__ void use_shared(PagesArgs& a, PagesShared& sh) {
  if (a.S <= kPagesShared) a.claim = sh.claim;
  if (a.n <= kPagesShared) {
    a.snap = sh.snap;
    a.prefix = sh.prefix;
  }
}

// The pages that n requests want, wants(i) each (0 for a bad request): leaves prefix[i], the pages wanted before
// request i (at most 2^30, which no cache has), and in list[] the free pages in order, as far as they are wanted.
// Returns the number of free pages found: request i is granted if prefix[i] + wants(i) is not above it.
template <typename Wants>
__device__ __forceinline__ int plan_pages(PagesArgs& a, PagesShared& sh, unsigned first, Wants wants) {
  long long need = 0;
  int turn = 0;
  for (int base = 0; base < a.n; base += blockDim.x, turn ^= 1) {
    const int i = base + threadIdx.x;
    long long total;
    const long long before = need + block_scan<long long>(i < a.n ? wants(i) : 0, &total, turn);
    if (i < a.n) a.prefix[i] = static_cast<int>(before < (1 << 30) ? before : 1 << 30);
    need += total;
  }
  if (need <= kPagesShared) a.list = sh.list;
  const int found = ranked(a, first, true, 0, a.P, need, [&](int rank, int i) { if (rank < need) a.list[rank] = i; });
  __syncthreads();
  return found;
}

// A sequence length that the table can hold.
__device__ __forceinline__ bool len_ok(const PagesArgs& a, int len) {
  return len >= 0 && len <= static_cast<long long>(a.M) * a.page;
}

// Two requests of a call must not change the same sequence: of the requests with snap[i] >= 0 the first that names a
// sequence keeps it, the others get snap[i] = -1.  snap[] was taken before anything is written.
template <typename Seq>
__device__ __forceinline__ void claim_sequences(const PagesArgs& a, Seq seq) {
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) a.claim[s] = 0x7fffffff;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += blockDim.x)
    if (a.snap[i] >= 0) atomicMin(a.claim + seq(i), i);
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += blockDim.x)
    if (a.snap[i] >= 0 && a.claim[seq(i)] != i) a.snap[i] = -1;
  __syncthreads();
}

// Sequences grow by tokens and get the pages they need.  snap[i]: the pages wanted, -1 for a bad request.
__global__ void __launch_bounds__(kPagesThreads) fa_pages_extend_kernel(PagesArgs a) {
  __shared__ PagesShared sh;
  after_previous_kernel();
  use_shared(a, sh);
  const unsigned first = free_bits(a, threadIdx.x * kPagesPer);
  for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
    const int s = a.seqs[i], t = a.arg[i];
    int w = -1;
    if (s >= 0 && s < a.S && t >= 0) {
      const int len = a.lens[s];
      if (len_ok(a, len) && static_cast<long long>(len) + t <= static_cast<long long>(a.M) * a.page)
        w = pages_of(len + t, a.page) - pages_of(len, a.page);
    }
    a.snap[i] = w;
  }
  claim_sequences(a, [&](int i) { return a.seqs[i]; });
  const int found = plan_pages(a, sh, first, [&](int i) { return max(0, a.snap[i]); });
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < a.n; i += blockDim.x / 32) {      // a warp per request
    const int w = a.snap[i];
    const bool ok = w == 0 || (w > 0 && a.prefix[i] + static_cast<long long>(w) <= found);
    if (ok) {
      const int s = a.seqs[i], len = a.lens[s];
      int* row = a.table + s * a.table_stride + pages_of(len, a.page);
      for (int e = lane; e < w; e += 32) {
        const int p = a.list[a.prefix[i] + e];
        row[e] = p;
        a.refs[p] = 1;
      }
      __syncwarp();                                                        // every lane has read the old length
      if (lane == 0) a.lens[s] = len + a.arg[i];
    }
    if (lane == 0) a.status[i] = ok ? 0 : (w < 0 ? 1 : 4);                 // FA_OK, FA_ERR_INVALID, FA_ERR_WORKSPACE
  }
}

// Empty sequences become copies of others: whole pages shared, the last page, if not full, to be copied.
// snap[i]: the source's length, -1 for a bad request.
__global__ void __launch_bounds__(kPagesThreads) fa_pages_fork_kernel(PagesArgs a) {
  __shared__ PagesShared sh;
  after_previous_kernel();
  use_shared(a, sh);
  const unsigned first = free_bits(a, threadIdx.x * kPagesPer);
  for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
    const int s = a.seqs[i], t = a.arg[i];
    int len = -1;
    if (s >= 0 && s < a.S && t >= 0 && t < a.S && s != t && a.lens[t] == 0 && len_ok(a, a.lens[s])) len = a.lens[s];
    a.snap[i] = len;
  }
  claim_sequences(a, [&](int i) { return a.arg[i]; });
  auto wants = [&](int i) { return a.snap[i] > 0 && a.snap[i] % a.page != 0 ? 1 : 0; };
  const int found = plan_pages(a, sh, first, wants);
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < a.n; i += blockDim.x / 32) {      // a warp per request
    const int len = a.snap[i], w = wants(i);
    const bool ok = len >= 0 && (w == 0 || a.prefix[i] < found);
    if (ok) {
      const int full = len / a.page;
      const int* from = a.table + a.seqs[i] * a.table_stride;
      int* to = a.table + a.arg[i] * a.table_stride;
      for (int e = lane; e < full; e += 32) {
        const int p = from[e];
        to[e] = p;
        if (p >= 0 && p < a.P) atomicAdd(a.refs + p, 1);
        else atomicOr(a.dev_status, DEV_ARGS);
      }
      if (lane == 0) {
        if (w) {
          const int p = a.list[a.prefix[i]], old = from[full];
          const bool good = old >= 0 && old < a.P;
          if (!good) atomicOr(a.dev_status, DEV_ARGS);
          to[full] = p;
          a.refs[p] = 1;
          int* c = a.copies + 3LL * a.prefix[i];      // granted requests come first: the list has no holes
          c[0] = good ? old : p;
          c[1] = p;
          c[2] = good ? len - full * a.page : 0;
        }
        a.lens[a.arg[i]] = len;
      }
    }
    if (lane == 0) a.status[i] = ok ? 0 : (len < 0 ? 1 : 4);
  }
  // everything behind the granted copies: the list's end
  __shared__ int copied;
  if (threadIdx.x == 0) copied = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += blockDim.x)
    if (wants(i) && a.prefix[i] < found) atomicMax(&copied, a.prefix[i] + 1);
  __syncthreads();
  for (long long e = 3LL * copied + threadIdx.x; e < 3LL * a.n; e += blockDim.x) a.copies[e] = -1;
}

// Sequences become empty.  One warp per request; the first to take a sequence's length frees its pages.
__global__ void __launch_bounds__(128) fa_pages_free_kernel(const PagesArgs a) {
  after_previous_kernel();
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= a.n) return;
  const int s = a.seqs[i];
  if (s < 0 || s >= a.S) {
    if (lane == 0) atomicOr(a.dev_status, DEV_ARGS);
    return;
  }
  int len = 0;
  if (lane == 0) {
    len = atomicExch(a.lens + s, 0);
    if (!len_ok(a, len)) {
      atomicOr(a.dev_status, DEV_ARGS);
      len = 0;
    }
  }
  len = __shfl_sync(0xffffffffu, len, 0);
  int* row = a.table + s * a.table_stride;
  for (int e = lane; e < pages_of(len, a.page); e += 32) {
    const int p = row[e];
    row[e] = -1;
    if (p < 0 || p >= a.P || atomicSub(a.refs + p, 1) <= 0) {
      atomicOr(a.dev_status, DEV_ARGS);
      if (p >= 0 && p < a.P) atomicAdd(a.refs + p, 1);
    }
  }
}

// Page p's new number after a compaction to `live` pages; p itself where it names no page.
__device__ __forceinline__ int renamed(const PagesArgs& a, int live, int p) {
  if (p < 0 || p >= a.P) {
    atomicOr(a.dev_status, DEV_ARGS);
    return p;
  }
  return p >= live ? a.list[p] : p;
}

// Entries of all page tables that the planning block renames itself: more take a launch of their own.
constexpr int kPagesRenameHere = 16384;

// Ranks the pages in use and the holes among them; lists the moves; moves the reference counts.
__global__ void __launch_bounds__(kPagesThreads) fa_pages_plan_compact_kernel(const PagesArgs a) {
  after_previous_kernel();
  const unsigned first = free_bits(a, threadIdx.x * kPagesPer);
  int mine = 0, live;
  const int step = blockDim.x * kPagesPer;
  for (long long i = threadIdx.x * kPagesPer; i < a.P; i += step) {
    const int there = a.P - i < kPagesPer ? static_cast<int>(a.P - i) : kPagesPer;
    mine += there - __popc(i < step ? first : free_bits(a, i));
  }
  block_scan<int>(mine, &live, 0);
  int* hole = a.list;              // holes below `live`: at most live of them, in list[0, live)
  const int holes = ranked(a, first, true, 0, live, 1LL << 62, [&](int rank, int i) { hole[rank] = i; });
  // as many pages in use lie at or above `live`; their new places go to list[i], i >= live
  for (int i = live + threadIdx.x; i < a.P; i += blockDim.x) a.list[i] = i;
  __syncthreads();
  ranked(a, first, false, live, a.P, 1LL << 62,
         [&](int rank, int i) {
           const int to = hole[rank];
           a.list[i] = to;
           a.refs[to] = a.refs[i];
           a.refs[i] = 0;
           int* c = a.copies + 3LL * rank;
           c[0] = i;
           c[1] = to;
           c[2] = a.page;
         });
  for (long long e = 3LL * holes + threadIdx.x; e < 3LL * (a.P / 2); e += blockDim.x) a.copies[e] = -1;
  if (1LL * a.S * a.M > kPagesRenameHere) {
    if (threadIdx.x == 0) *a.info = live;
    return;
  }
  __syncthreads();
  for (int x = threadIdx.x; x < a.S * a.M; x += blockDim.x) {
    const int s = x / a.M, e = x - s * a.M, len = a.lens[s];
    int* p = a.table + s * a.table_stride + e;
    const int old = *p;            // asked for together with the length
    if (!len_ok(a, len)) {
      if (e == 0) atomicOr(a.dev_status, DEV_ARGS);
    } else if (e < pages_of(len, a.page)) {
      *p = renamed(a, live, old);
    }
  }
}

// The page tables name the new places.  One warp per sequence.
__global__ void __launch_bounds__(128) fa_pages_rename_kernel(const PagesArgs a) {
  after_previous_kernel();
  const int s = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (s >= a.S) return;
  const int live = *a.info, len = a.lens[s];
  if (!len_ok(a, len)) {
    if (lane == 0) atomicOr(a.dev_status, DEV_ARGS);
    return;
  }
  int* row = a.table + s * a.table_stride;
  for (int e = lane; e < pages_of(len, a.page); e += 32) row[e] = renamed(a, live, row[e]);
}

struct PageCopyArgs {
  __nv_bfloat16 *kp, *vp;
  Strides sk, sv;                  // {page, head, row}
  const int* copies;
  int n, P, page, H_kv, d;
  int tpr;                         // threads of a row
  int rows_per, row_parts;         // a head's rows are copied in row_parts parts of rows_per
  uint32_t* status;
};
constexpr int kPageCopyBytes = 16384;   // of a part: four 16-byte vectors in flight per thread

// A copy is cut into parts (K or V, a head, a piece of its rows).  Block = (team, part): the block copies its part of the
// list's rows team, team + teams, ...; its lanes look at 32 of them at once, so a list that is mostly empty costs one
// read.  16 bytes at a time, a thread has a fixed column.
__global__ void __launch_bounds__(256) fa_pages_copy_kernel(const PageCopyArgs a) {
  after_previous_kernel();
  const int lane = threadIdx.x & 31;
  const int parts = 2 * a.H_kv * a.row_parts, teams = gridDim.x / parts;
  const int team = blockIdx.x / parts, part = blockIdx.x - team * parts;
  const int hk = part / a.row_parts, piece = part - hk * a.row_parts;
  const bool is_v = hk >= a.H_kv;
  const Strides st = is_v ? a.sv : a.sk;
  __nv_bfloat16* base = (is_v ? a.vp : a.kp) + (hk - (is_v ? a.H_kv : 0)) * st.h;
  const int step = 256 / a.tpr, row0 = threadIdx.x / a.tpr, x0 = 8 * (threadIdx.x - row0 * a.tpr);
  const int first = piece * a.rows_per;
  for (long long at = team; at < a.n; at += 32LL * teams) {
    const long long mine = at + static_cast<long long>(lane) * teams;
    int my_src = -1, my_dst = 0, my_rows = 0;
    if (mine < a.n) {
      my_src = a.copies[3 * mine];
      my_dst = a.copies[3 * mine + 1];
      my_rows = a.copies[3 * mine + 2];
    }
    unsigned todo = __ballot_sync(0xffffffffu, my_src >= 0);
    for (; todo; todo &= todo - 1) {
      const int from_lane = __ffs(todo) - 1;
      const int src = __shfl_sync(0xffffffffu, my_src, from_lane), dst = __shfl_sync(0xffffffffu, my_dst, from_lane),
                rows = __shfl_sync(0xffffffffu, my_rows, from_lane);
      if (src >= a.P || dst < 0 || dst >= a.P || rows < 0 || rows > a.page) {
        if (threadIdx.x == 0) atomicOr(a.status, DEV_ARGS);
        continue;
      }
      if (row0 >= step) continue;                  // 256 is no multiple of tpr: the last threads have no row
      const int end = min(rows, first + a.rows_per);
      const __nv_bfloat16* from = base + src * st.b;
      __nv_bfloat16* to = base + dst * st.b;
      for (int x = x0; x < a.d; x += 8 * a.tpr) {
        for (int r = first + row0; r < end; r += 4 * step) {
          uint4 w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (r + u * step < end) w[u] = *reinterpret_cast<const uint4*>(from + (r + u * step) * st.r + x);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (r + u * step < end) *reinterpret_cast<uint4*>(to + (r + u * step) * st.r + x) = w[u];
        }
      }
    }
  }
}

}  // namespace fa
