// Attention of the last N positions of each sequence over a paged key/value
// cache: o = softmax(scale q K^T) V over keys j < seq_len (and j <= seq_len - N + i
// when causal), lse = ln sum exp.
//
// Each key and value is needed once per key/value head by group * N query rows:
// 4 d bytes and 4 d group N flops per key, so a few rows are bound by HBM.  What
// carries the kernel is therefore bytes in flight and an even share for every SM:
//
//  * the keys of all (sequence, key/value head) pairs, in tiles of KT keys, are one
//    line of work that is cut into equal ranges, one per warp (paged_workers of them,
//    all resident at once), whatever the lengths are.  A range covers the end of one
//    pair, whole pairs, and the beginning of another; whole pairs are written out,
//    the cut ones leave (max, sum, O) partials that the merge kernel joins.  The
//    lengths are read on the device: a captured call follows them.  When a table row
//    holds a few tiles only, no pair is cut (paged_share): a warp or a block takes it,
//    there is nothing to plan, and the second launch falls away;
//  * a warp fills its own ring of tiles by TMA, across the ends of pairs, and waits for
//    nobody: no block barrier in the loop.  Beginning and ending a pair (its rows'
//    loads, its outputs) counts as kPagedPairUnits tiles.  A box is 8, 16 or 32 keys of
//    all d columns, the most that divides tile and page; the page numbers of 256 keys
//    are read ahead, and a number that names no page loads zeros (it lies outside the
//    tensor map).  Values behind a sequence's end are zeroed in shared memory, and
//    scores there masked, so what the pages hold there does not matter.  (Gathering
//    with 16-byte asynchronous copies took 150-250 instructions per tile more.);
//  * the products are warp-level matrix instructions (16 rows x 8 columns x 16): rows
//    are few, and the tcgen05 tiles start at 64 rows.  S = Q K^T gives its accumulators
//    in the layout that P V wants its left operand in, so P stays in registers;
//  * P enters the second product as a bf16 and the bf16 of what that rounding left, 16 bits
//    of mantissa, however many rows there are and however a call is cut.  In tiles of 8 rows
//    the remainder rides in the 8 unused rows of the same instruction, in higher ones it
//    takes a second one (32 rows, d 64, 1.07 GB of cache: 182 us without, 211 with it;
//    16 rows, d 128, 0.54 GB: 101 and 103).
//    Everything else is 32-bit; O is rounded once.
//  * O is rescaled only when a row's maximum grows by more than 2^8.
#pragma once

#include "layout.cuh"

namespace fa {

struct PagedArgs {
  const __nv_bfloat16* q;          // (the pages come through the tensor maps)
  __nv_bfloat16* o;
  float* lse;                      // [B, H, N]
  const int* table;
  long long table_stride;
  const int* seq_lens;
  Strides sq, so;
  int B, H, H_kv, N, group;
  int rows;                        // group * N
  int num_pages, page, max_pages;
  int causal;
  float scale_log2;
  int workers;                     // warps that share the work of one row tile
  int min_units;                   // least units of a warp's range
  int whole_units;                 // short tables: units of every pair, none of which is cut; else 0
  int by_block;                    // short tables: a block to a pair, its tiles shared by the four warps; no partials
  int row_tiles;
  int part_rows;                   // rows of a partial
  float* part_o;                   // [row tile][worker][2][part_rows][D]
  unsigned long long wait_limit_ns;
  int box;                         // keys of a TMA box: 8, 16 or 32
  float2* part_ml;                 // [row tile][worker][2][part_rows] maximum (log2 units) and sum
  int2* meta;                      // [row tile][B][H_kv] worker where the pair begins, workers it goes on into
  uint32_t* status;
};

// Keys of sequence b, 0 and flagged when the length makes no sense.
__device__ __forceinline__ int paged_len(const PagedArgs& a, int b) {
  const int n = a.seq_lens[b];
  if (n < 0 || n > static_cast<long long>(a.max_pages) * a.page) {
    atomicOr(a.status, DEV_ARGS);
    return 0;
  }
  return n;
}

// D: head dim.  RM: query rows of a row tile (8, 16 or, d 64, 32).
template <int D_, int RM_>
struct PagedCfg {
  static constexpr int D = D_, RM = RM_;
  static constexpr bool HALF = RM == 8;          // the lo parts of P in rows 8 .. 15
  static constexpr int MT = HALF ? 1 : RM / 16;
  static constexpr int KT = D == 64 ? 32 : 16;   // keys per tile
  static constexpr int NT = KT / 8;
  static constexpr int WARPS = 4, THREADS = 32 * WARPS;
  // A slot of the ring holds the K and the V tile of some keys, or (d = 256, whose tiles are 8 KB) one of them, K and V in
  // turn: two blocks to an SM either way.  (d = 256, 32 rows: 177 us for 536 MB with one block of 48 KB rings, 128 us so;
  // d = 128, 16 x 8192 keys: 95 us with both tiles in a slot, 98 us with slots of one.)
  static constexpr bool SPLIT = D == 256;
  static constexpr int SLOTS = 3;
  static constexpr int PITCH = 2 * D;            // bytes of a key, or of a query
  static constexpr int TILE = KT * PITCH;        // [box][64 columns][key][128 bytes], 128-byte swizzle
  static constexpr int SLOT = (SPLIT ? 1 : 2) * TILE;   // 8 KB
  static constexpr int RING = SLOTS * SLOT;
  static constexpr int SMEM = WARPS * RING + 1024;   // and what aligns it
  static constexpr int CTAS = 2;                 // per SM
};
constexpr int kPagedSms = 148;
constexpr int kPagedMinUnits = 2;                // of a range: what is in flight at once
// How pairs whose table rows hold `tiles` tiles at most are shared out: each to a warp, each to a block's four warps, or
// cut into ranges of equal length.  Uncut pairs take no planning, no partials and no second launch, but one warp's (or
// four warps') time for their tiles.  Measured (device time, us; warp / block / cut; rows R per key/value head):
//   8 pairs, d 128, R 4:     1 tile 4.0 / 4.0 / 7.2, 2 tiles 4.7 / 4.1 / 7.5, 20 tiles 19.1 / 7.4 / 9.5, 32 tiles 28 / 9.4 / 9.4,
//                            36 tiles 32 / 10.4 / 9.6;  d 64: 28 tiles 29 / 9.3 / 9.3, 36 tiles 36 / 11.1 / 9.5
//   8 pairs, d 256, R 8:     16 tiles 24 / 9.6 / 10.4, 20 tiles 29 / 11.0 / 11.3, 24 tiles 34 / 12.0 / 11.2
//   64 pairs, d 128, R 4:    32 tiles 29 / 9.9 / 12.0, 40 tiles 36 / 11.7 / 12.7, 48 tiles 42 / 13.2 / 13.3
//   64 pairs, d 256, R 8:    24 tiles 34 / 12.5 / 13.7, 32 tiles 44 / 15.0 / 13.9;  32 pairs: 24 tiles 33 / 12.5 / 11.9
//   136 pairs, d 128, R 4:   64 tiles 56 / 16.5 / 17.5, 80 tiles 69 / 20.1 / 19.8;  192 pairs: 64 tiles 56 / 20.1 / 22.8
//   320 pairs:               12 tiles 12.8 / 12.3 / 13.3, 16 tiles 16.0 / 14.1 / 14.3, 64 tiles 56 / 42 / 38
//   480 pairs:               12 tiles 13.0 / 13.0 / 16.9, 16 tiles 16.2 / 14.8 / 18.7, 64 tiles 57 / 45 / 52
//   640 pairs:               16 tiles 18.4 / 21 / 19.5, 20 tiles 23.4 / 26 / 24.8;  1280: 16 tiles 36 / 40 / 38, 24 tiles 50 / 53 / 52
//   32-row tiles, d 64 (no joining): 320 pairs: 12 tiles 21.3 / - / 20.3, 16 tiles 26.8 / - / 22.1;  480: 16 tiles 27 / - / 30,
//                            20 tiles 32.9 / - / 32.8;  640: 16 tiles 33 / - / 37, 20 tiles 41 / - / 41
//   16-row tiles, d 128:     320 pairs: 12 tiles 15.0 / 16.9 / 15.6;  480: 12 tiles 15 / 18 / 19, 64 tiles 64 / 52 / 57
//   16-row tiles (pairs times row tiles): 12, d 128: 20 tiles 22 / 10.2 / 10.8, 28 tiles 29 / 11.8 / 10.9;  d 64: 20 tiles
//                            25 / 10.1 / 10.2, 24 tiles 29 / 11.1 / 10.4;  d 256: 12 tiles 33 / 14.1 / 14.9, 16 tiles 42 / 16.4 / 15.2
//   96, d 256:               24 tiles 61 / 21 / 23.5, 32 tiles 80 / 26 / 24;  48, d 256: 24 tiles 61 / 21 / 20.4
enum PagedShare { kPagedCut, kPagedByWarp, kPagedByBlock };
inline PagedShare paged_share(int d, int rm, long long pairs, long long tiles) {
  const bool joins = rm <= 16;                     // blocks join their warps' parts up to 16 rows
  if (pairs < 2 * 148) {
    const int few = pairs >= 32 ? (rm == 16 && d == 256 ? 24 : 32) : d == 256 ? (rm == 8 ? 20 : 12) : rm == 8 ? 32 : 20;
    if (tiles <= 1) return kPagedByWarp;
    return joins && tiles <= (pairs < 128 ? few : 64) ? kPagedByBlock : kPagedCut;
  }
  if (tiles <= (pairs < 4 * 148 && joins ? 12 : 16)) return kPagedByWarp;
  return pairs < 4 * 148 && joins && tiles <= 64 ? kPagedByBlock : kPagedCut;
}
constexpr int kPagedTeam = 32;
constexpr int kPagedPairUnits = 2;               // what beginning and ending a pair costs, in tiles

// Rows of a row tile: 8, 16 or (d 64) 32.  Small row tiles read every key several times, but once only from HBM, and take
// a warp less time per tile: what counts while calls are short and blocks fit the GPU at once.  With d 256, 17 to 24 rows
// fill three tiles of 8 and leave half of a second tile of 16 empty.  `tiles` are those of all pairs.  Device time, us, by
// the rows of a tile (8 / 16, d 64 and 128: / 32):
//   16 rows, d 128, 4 pairs of 64 tiles 11.4 / 12.7 / 14; 64 pairs of 32 tiles 10.9 / 12.9 / 19, of 128 27 / 22.6 / 32;
//                   256 pairs of 4 tiles 7.0 / 7.8 / 12, of 8 10.2 / 9.1 / 21
//   32 rows, d 128, 64 pairs of 32 tiles 12.7 / 13.1 / 24, of 256 64 / 44 / 53, of 1024 215 / 130 / 136; 256 pairs of 256 216 / 131 / 139
//   64 rows, d 128, 64 pairs of 1024 tiles - / 243 / 242; 256 pairs of 64 - / 78 / 86, of 256 - / 247 / 250
//                   (32 rows of d 128 take 255 registers and spill: they win nowhere, and no such kernel is built)
//   24 rows, d 64, 32 pairs of 64 tiles 16.4 / 16.0 / 15.8, of 128 22.1 / 20.8 / 19.4, of 1024 100 / 81 / 64; 256 pairs of 8
//                   12.0 / 12.2 / 16, of 32 34 / 28 / 26
//   16 rows, d 256, 4 pairs of 256 tiles 17.1 / 19.6; 64 pairs of 256 61 / 70, of 1024 197 / 192; 256 pairs of 32 46 / 33
//   32 rows, d 256, 32 pairs of 256 tiles 56 / 58, of 1024 176 / 164; 64 pairs of 256 96 / 94
//   24 rows, d 256, 4 pairs of 1024 tiles 31 / 36; 64 pairs of 256 77 / 93; 256 pairs of 4 11.3 / 15.7, of 256 261 / 324
inline int paged_row_tile(int d, int rows, long long pairs, long long tiles) {
  const int eights = (rows + 7) / 8;
  if (eights == 1 || (d == 256 && eights == 3)) return 8;
  if (eights <= 4 && pairs * eights < 2 * 148 && tiles <= (d == 256 ? 14 : 2) * 1184LL) return 8;
  return rows <= 16 || d > 64 || tiles <= 2 * 1184LL ? 16 : 32;
}
// Warps that share one row tile's work.
__host__ __device__ inline int paged_workers(int row_tiles) {
  const int ctas = kPagedSms * 2 / row_tiles;
  return (ctas < 1 ? 1 : ctas) * 4;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c += a b: a 16 x 16 (row), b 16 x 8 (column), bf16; c fp32.
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
// 16 bytes to shared memory, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// A place in the line: tile `tile` of the `tiles` of (sequence b, key/value head h), which is `unit` of the line.
struct PagedPlace {
  long long unit;
  int b, h, tile, tiles, len;
  template <int KT>
  __device__ __forceinline__ void enter(const PagedArgs& a) {      // sequence b's length; empty ones have a tile too
    len = b < a.B ? paged_len(a, b) : 0;
    tiles = max(1, (len + KT - 1) / KT);
  }
  // units of the line between this pair's tiles and the next one's
  __device__ __forceinline__ int gap(const PagedArgs& a) const { return a.whole_units ? a.whole_units - tiles : kPagedPairUnits; }
  template <int KT>
  __device__ __forceinline__ void next_pair(const PagedArgs& a) {  // unit: already behind this pair's last tile
    unit += gap(a);
    tile = 0;
    if (++h == a.H_kv) {
      h = 0;
      ++b;
      enter<KT>(a);
    }
  }
};

template <int D, int RM>
__global__ void __launch_bounds__(128, (PagedCfg<D, RM>::CTAS))
fa_paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedArgs a) {
  using C = PagedCfg<D, RM>;
  constexpr int KT = C::KT, NT = C::NT, MT = C::MT, RW = C::HALF ? 1 : 2;   // RW: rows of a thread in a 16-row tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ long long before[C::THREADS + 1];
  __shared__ long long warp_sum[C::WARPS];
  __shared__ uint64_t bars[C::WARPS * C::SLOTS];   // a slot's bytes have arrived
  __shared__ uint32_t abort_flag;
  __shared__ float2 team_ml[C::WARPS * RM];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int worker = blockIdx.x * C::WARPS + warp, rt = blockIdx.y;

  const uint32_t bar0 = smem_u32(bars + warp * C::SLOTS);
  if (lane == 0) {
    for (int st = 0; st < C::SLOTS; ++st) mbar_init(bar0 + 8 * st, 1);
    fence_mbar_init();
  }
  if (tid == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (tid == 0) abort_flag = 0u;                   // the barriers below come before every use
  after_previous_kernel();

  long long t0, t1, range;
  PagedPlace in;                                   // the next tile to load
  if (a.by_block) {
    // ---- this warp's quarter of the block's pair
    __syncthreads();                               // abort_flag
    in.b = blockIdx.x / a.H_kv;
    in.h = blockIdx.x - in.b * a.H_kv;
    in.enter<KT>(a);
    in.tile = in.tiles * warp / C::WARPS;
    in.unit = t0 = in.tile;
    t1 = in.tiles * (warp + 1) / C::WARPS;         // t0 == t1: nothing for this warp
    range = 1;
  } else if (a.whole_units) {
    // ---- every pair has its place in the line, whatever its length
    const int pairs = a.B * a.H_kv, mine = (pairs + a.workers - 1) / a.workers;
    range = static_cast<long long>(mine) * a.whole_units;
    t0 = worker * range;
    t1 = min(t0 + range, static_cast<long long>(pairs) * a.whole_units);
    __syncthreads();                               // abort_flag
    if (t0 >= t1) return;
    const int first = worker * mine;               // below pairs
    in.b = first / a.H_kv;
    in.h = first - in.b * a.H_kv;
    in.enter<KT>(a);
    in.tile = 0;
    in.unit = t0 + kPagedPairUnits;
  } else {
    // ---- the line, of one head: thread t sums the units of sequences t q .. t q + q - 1
    const int per_thread = (a.B + C::THREADS - 1) / C::THREADS;
    {
      long long mine = 0;
      for (int b = tid * per_thread; b < min(a.B, (tid + 1) * per_thread); ++b)
        mine += max(1, (paged_len(a, b) + KT - 1) / KT) + kPagedPairUnits;
      long long x = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      long long base = 0;
      for (int w = 0; w < warp; ++w) base += warp_sum[w];
      before[tid] = base + x - mine;
      if (tid == C::THREADS - 1) before[C::THREADS] = base + x;
      __syncthreads();
    }
    const long long total = before[C::THREADS] * a.H_kv;
    const long long share = (total + a.workers - 1) / a.workers;
    range = share > a.min_units ? share : a.min_units;
    t0 = range * worker;
    t1 = min(t0 + range, total);
    if (t0 >= t1) return;

    // ---- the first tile at or behind t0
    {
      const long long s0 = t0 / a.H_kv;
      int slot = 0;
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) slot += __popc(__ballot_sync(0xffffffffu, before[32 * w + lane] <= s0));
      in.b = (slot - 1) * per_thread;
      long long base = before[slot - 1];
      in.enter<KT>(a);
      while (base + in.tiles + kPagedPairUnits <= s0) {   // at most per_thread steps
        base += in.tiles + kPagedPairUnits;
        ++in.b;
        in.enter<KT>(a);
      }
      const long long rest = t0 - base * a.H_kv;     // of this sequence's H_kv (tiles + kPagedPairUnits)
      const long long units = in.tiles + kPagedPairUnits;
      in.h = static_cast<int>(rest / units);
      const int u = static_cast<int>(rest - in.h * units) - kPagedPairUnits;
      in.tile = max(0, u);
      in.unit = t0 + in.tile - u;
    }
  }
  if (in.unit >= t1 && !a.by_block) return;
  // Do the block's four ranges lie inside one pair, and is it cut into kPagedTeam ranges at least?  (The same answer in all
  // four warps.)  Then they leave one partial: 33 MB of cache in 4 pairs (d 256) 23.7 -> 21 us with the merge.  With fewer
  // ranges the block's own joining costs more than it saves, and with 32 rows it takes registers that the loop needs.
  const long long tile0 = in.unit - in.tile, block0 = range * C::WARPS * blockIdx.x;
  const bool team = RM <= 16 && (a.by_block || (!a.whole_units && block0 >= tile0 && block0 + range * C::WARPS <= tile0 + in.tiles &&
                                                in.tiles >= kPagedTeam * range));
  PagedPlace at = in;                              // the next tile to use
  const uint32_t ring = smem_u32(smem) + warp * C::RING;

  // ---- loading
  const int groups_per_page = a.page / 8;
  int pg_next = -1, row_next = 0, pg = -1, row_in = 0;   // this lane's 8 keys: page and first row; the next 256 keys'
  int g0 = -1;                                     // first 8-key group of pg, in sequence in.b
  auto look_up = [&](int g) {                      // page and row of 8-key group g + lane of pair `in`
    const int mine = g + lane;
    pg_next = -1;
    row_next = 0;
    if (8LL * mine < in.len) {
      const int e = mine / groups_per_page;
      row_next = (mine - e * groups_per_page) * 8;
      pg_next = a.table[in.b * a.table_stride + e];
      if (pg_next < 0 || pg_next >= a.num_pages) {
        atomicOr(a.status, DEV_ARGS);
        pg_next = -1;
      }
    }
  };
  int load_slot = 0;
  bool load_v = false;                             // SPLIT: V is next
  auto load_next = [&]() {                         // the tiles of `in`, or (SPLIT) one of them, into the next slot
    if (in.unit >= t1) return;
    const int g = in.tile * (KT / 8), want = g & ~31;
    if (want != g0) {                              // KT / 8 divides 32: a tile's groups are in one look-up
      if (g0 < 0 || want != g0 + 32) look_up(want);
      pg = pg_next;
      row_in = row_next;
      g0 = want;
      look_up(want + 32);
    }
    const uint32_t to = ring + load_slot * C::SLOT, bar = bar0 + 8 * load_slot;
    if (lane == 0) mbar_expect_tx(bar, C::SLOT);
#pragma unroll 1
    for (int key = 0; key < KT; key += a.box) {
      const int p = __shfl_sync(0xffffffffu, pg, (g - g0) + key / 8), row = __shfl_sync(0xffffffffu, row_in, (g - g0) + key / 8);
      if (lane == 0) {
        tma_load_5d(to + key * C::PITCH, C::SPLIT && load_v ? &tm_v : &tm_k, bar, 0, row, 0, in.h, p);
        if constexpr (!C::SPLIT) tma_load_5d(to + C::TILE + key * C::PITCH, &tm_v, bar, 0, row, 0, in.h, p);
      }
    }
    load_slot = load_slot + 1 == C::SLOTS ? 0 : load_slot + 1;
    load_v = C::SPLIT && !load_v;
    if (load_v) return;
    ++in.unit;
    if (++in.tile == in.tiles) {
      if (in.unit + in.gap(a) < t1) {
        const int b = in.b;
        in.next_pair<KT>(a);
        if (in.b != b) g0 = -1;
      } else {
        in.unit = t1;
      }
    }
  };

  // ---- a pair's rows: this thread's rows of the 16-row tiles are lane / 4 and (unless HALF) lane / 4 + 8
  const int quad = lane & 3;
  const float c2 = a.scale_log2;
  uint32_t qf[MT][D / 16][C::HALF ? 2 : 4];
  float acc[MT][D / 8][4];
  float m[MT][RW], l[MT][RW];
  // lane r holds the query head (of the pair's) and position of row r of the row tile; head -1: there is none
  const int my_row = rt * RM + lane, my_i = my_row % a.N, my_g = lane < RM && my_row < a.rows ? my_row / a.N : -1;
  // Q goes through the slot that is loaded next, a 16-row tile at a time, rows without a query as zeros.
  auto begin_pair = [&]() {
    const uint32_t to = ring + load_slot * C::SLOT;
    constexpr int CH = D / 8, RPI = 32 / CH, ROWS = C::HALF ? 8 : 16;   // 16-byte chunks of a row; rows per warp copy
    const int ch = lane % CH;
    const long long q_row = my_g < 0 ? -1 : my_g * a.sq.h + my_i * a.sq.r;
    const __nv_bfloat16* q = a.q + at.b * a.sq.b + static_cast<long long>(at.h) * a.group * a.sq.h + ch * 8;
    const int row = (lane & 7) + (C::HALF ? 0 : ((lane >> 3) & 1) * 8), hi = C::HALF ? lane >> 3 : lane >> 4;
    const uint32_t qa = to + row * C::PITCH + ((hi ^ (row & 7)) << 4);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll 1
      for (int r = 0; r < ROWS; r += RPI) {
        const int rr = r + lane / CH;
        const long long off = __shfl_sync(0xffffffffu, q_row, mt * 16 + rr);
        copy16(to + rr * C::PITCH + ((ch ^ (rr & 7)) << 4), off < 0 ? a.q : q + off, off >= 0);
      }
      copy_commit();
      copy_wait_all();
      __syncwarp();
      if constexpr (C::HALF) {                     // two k-steps at a time: chunks 4 x .. 4 x + 3
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {
          uint32_t w[4];
          ldsm4(qa ^ (32 * k), w);
          qf[0][k][0] = w[0];
          qf[0][k][1] = w[1];
          qf[0][k + 1][0] = w[2];
          qf[0][k + 1][1] = w[3];
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) ldsm4(qa ^ (32 * k), qf[mt][k]);
      }
#pragma unroll
      for (int w = 0; w < RW; ++w) {
        m[mt][w] = -INFINITY;
        l[mt][w] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][n][e] = 0.f;
      __syncwarp();                                // everyone has its Q
    }
    fence_proxy_async_smem();
    __syncwarp();                                  // the slot is free for TMA
  };
  auto end_pair = [&](bool begins, bool ends) {    // of the pair's tiles this warp had the first, the last
    const bool whole = begins && ends && !a.by_block;
    const long long slot = ((static_cast<long long>(rt) * a.workers + worker) * 2 + (begins ? 1 : 0)) * a.part_rows;
    const long long head0 = static_cast<long long>(at.b) * a.H + at.h * a.group;
    const long long o_row = my_g * a.so.h + my_i * a.so.r;
    __nv_bfloat16* o = a.o + at.b * a.so.b + static_cast<long long>(at.h) * a.group * a.so.h + 2 * quad;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int w = 0; w < RW; ++w) {
        float sum = l[mt][w];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int rr = mt * 16 + w * 8 + (lane >> 2);
        const long long off = __shfl_sync(0xffffffffu, o_row, rr);
        if (rt * RM + rr < a.rows) {
          const float top = m[mt][w] == -INFINITY ? -INFINITY : m[mt][w] * c2;
          const float f = !whole ? 1.0f : sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
          char* to = whole ? reinterpret_cast<char*>(o + off)
                     : team ? reinterpret_cast<char*>(reinterpret_cast<float*>(smem + warp * C::RING) + rr * D + 2 * quad)
                            : reinterpret_cast<char*>(a.part_o + (slot + rr) * D + 2 * quad);
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            const float x = f * (C::HALF ? acc[mt][n][0] + acc[mt][n][2] : acc[mt][n][2 * w]);
            const float y = f * (C::HALF ? acc[mt][n][1] + acc[mt][n][3] : acc[mt][n][2 * w + 1]);
            if (whole) *reinterpret_cast<uint32_t*>(to + 16 * n) = pack_bf16x2(x, y);
            else *reinterpret_cast<float2*>(to + 32 * n) = make_float2(x, y);
          }
          if (quad == 0) {
            if (whole)
              a.lse[head0 * a.N + rt * RM + rr] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
            else
              (team ? team_ml + warp * RM : a.part_ml + slot)[rr] = make_float2(top, sum);
          }
        }
      }
    if (begins && !a.whole_units && !a.by_block && lane == 0) {
      const int more = ends ? 0 : static_cast<int>((at.unit + at.tiles - 1 - at.tile) / range) - worker;
      a.meta[(static_cast<long long>(rt) * a.B + at.b) * a.H_kv + at.h] = make_int2(worker, more);
    }
  };

  // One copy of every step in the code: a launch runs each of them a few times only, and what it costs then is fetching
  // the instructions (two more copies of load_next and one of begin_pair took the shortest calls from 7 to 12-30 us).
  bool fresh = true, begins = at.tile == 0, second = false;   // second (SPLIT): P is ready, V is next
  int slot = 0;
  uint32_t phase = 0;                              // bit of each slot: parity of its next arrival
  const WaitCtl ctl{&abort_flag, a.status, a.wait_limit_ns};
  // where key `key` of a tile lies, and the bytes between its 64-column pieces
  const int piece = a.box * 128;
  auto key_at = [&](int key) { return D == 64 ? key * 128 : key / a.box * (a.box * C::PITCH) + key % a.box * 128; };
  const int krow = (lane & 7) + ((lane >> 4) << 3), vrow = lane & 15;
  const uint32_t k_lane = key_at(krow) + ((((lane >> 3) & 1) ^ (krow & 7)) << 4);
  const uint32_t v_lane = key_at(vrow) + (((lane >> 4) ^ (vrow & 7)) << 4);
  const bool busy = in.unit < t1;                  // (by_block: there may be nothing to do)
  if (!busy)
    for (int rr = lane; rr < RM; rr += 32) team_ml[warp * RM + rr] = make_float2(-INFINITY, 0.f);
  uint32_t p[MT][NT / 2][4];                       // per 16 keys: keys 0 .. 7 (rows, rows + 8), then keys 8 .. 15
  uint32_t lo[C::HALF ? 1 : MT][C::HALF ? 1 : NT / 2][4];   // what p's rounding left (HALF: in p's rows 8 .. 15)
#pragma unroll 1
  for (int ahead = C::SLOTS - 1; busy;) {          // tiles to load before the first is used
    if (ahead == 0) {
      if (fresh && !second) {                      // while the pair's first tile is on its way
        __syncwarp();                              // everyone is done with the free slot
        begin_pair();
      }
      if (!mbar_wait_warp(bar0 + 8 * slot, (phase >> slot) & 1, ctl)) {   // (and everyone is done with the last slot)
        // let the copies in flight land (bounded): every slot but the free one
        if (lane == 0)
          for (int st = 0; st < C::SLOTS; ++st)
            if (st != load_slot) mbar_wait_quiet(bar0 + 8 * st, (phase >> st) & 1, 200000000ull);
        if (team) named_bar_and(1, C::THREADS, false);
        return;
      }
    }
    load_next();
    if (ahead > 0) {
      --ahead;
      continue;
    }
    const uint32_t here = ring + slot * C::SLOT, vt = here + (C::SPLIT ? 0 : C::TILE);
    phase ^= 1u << slot;
    slot = slot + 1 == C::SLOTS ? 0 : slot + 1;
    if (!C::SPLIT || !second) {
      // ---- S = Q K^T
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][n][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t ka = (here + k_lane + k / 4 * piece) ^ (32 * (k % 4));
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t kf[4];
          ldsm4(ka + 1024 * n, kf);                // n > 0: d = 64 only, whose keys lie 128 bytes apart
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint32_t a0 = qf[mt][k][0], a1 = C::HALF ? 0u : qf[mt][k][1], a2 = qf[mt][k][RW],
                           a3 = C::HALF ? 0u : qf[mt][k][2 * RW - 1];
            mma_bf16(s[mt][n], a0, a1, a2, a3, kf[0], kf[1]);
            mma_bf16(s[mt][n + 1], a0, a1, a2, a3, kf[2], kf[3]);
          }
        }
      }
      // ---- masks: the tiles at the sequence's end
      if ((at.tile + 1) * KT > at.len - (a.causal ? a.N - 1 : 0)) {
        const int key0 = at.tile * KT + 2 * quad;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int w = 0; w < RW; ++w) {
            const int i = __shfl_sync(0xffffffffu, my_i, mt * 16 + w * 8 + (lane >> 2));
            const int lim = a.causal ? at.len - a.N + i : at.len - 1;   // last key the row sees
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (key0 + 8 * n + e > lim) s[mt][n][2 * w + e] = -INFINITY;
          }
      }
      // ---- online softmax
      bool grew = false;
      float alpha[MT][RW];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int w = 0; w < RW; ++w) {
          float top = fmaxf(s[mt][0][2 * w], s[mt][0][2 * w + 1]);
#pragma unroll
          for (int n = 1; n < NT; ++n) top = fmaxf(top, fmaxf(s[mt][n][2 * w], s[mt][n][2 * w + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const bool grows = (top - m[mt][w]) * c2 > 8.0f;    // false while the row has seen no key
          alpha[mt][w] = 1.0f;
          if (grows) {
            alpha[mt][w] = ex2_approx((m[mt][w] - top) * c2);
            l[mt][w] *= alpha[mt][w];
            m[mt][w] = top;
            grew = true;
          }
          const float nb = m[mt][w] == -INFINITY ? 0.f : m[mt][w] * c2;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = ex2_approx(fmaf(s[mt][n][2 * w + e], c2, -nb));
              s[mt][n][2 * w + e] = x;
              l[mt][w] += x;
            }
        }
      if (!fresh && __any_sync(0xffffffffu, grew)) {   // on a pair's first tile there is nothing to rescale
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][n][e] *= alpha[mt][C::HALF ? 0 : e >> 1];
      }
      fresh = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t* y = &p[mt][n / 2][2 * (n % 2)];
          y[0] = pack_bf16x2(s[mt][n][0], s[mt][n][1]);
          const float2 h = bf16x2_to_float2(y[0]);
          const uint32_t left = pack_bf16x2(s[mt][n][0] - h.x, s[mt][n][1] - h.y);
          if constexpr (C::HALF) {
            y[1] = left;
          } else {
            y[1] = pack_bf16x2(s[mt][n][2], s[mt][n][3]);
            const float2 g = bf16x2_to_float2(y[1]);
            uint32_t* z = &lo[mt][n / 2][2 * (n % 2)];
            z[0] = left;
            z[1] = pack_bf16x2(s[mt][n][2] - g.x, s[mt][n][3] - g.y);
          }
        }
      second = C::SPLIT;
      if constexpr (C::SPLIT) continue;
    }
    second = false;
    // values behind the end: P is 0 there, but 0 * NaN is not
    const int left = at.len - at.tile * KT;
    if (left < KT) {
#pragma unroll 1
      for (int e = lane; e < (KT - left) * (D / 8); e += 32) {
        const int key = left + e / (D / 8), ch = e % (D / 8);
        *reinterpret_cast<uint4*>(smem + (vt - smem_u32(smem)) + key_at(key) + ch / 8 * piece + ch % 8 * 16) =
            make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();                    // before TMA writes the slot again
      __syncwarp();
    }
    // ---- O += P V
#pragma unroll
    for (int kk = 0; kk < NT / 2; ++kk)
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        uint32_t vf[4];
        ldsm4_t(((vt + v_lane + n / 8 * piece) ^ (16 * (n % 8))) + 2048 * kk, vf);   // kk > 0: d = 64 only
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t* y = p[mt][kk];
          mma_bf16(acc[mt][n], y[0], y[1], y[2], y[3], vf[0], vf[1]);
          mma_bf16(acc[mt][n + 1], y[0], y[1], y[2], y[3], vf[2], vf[3]);
          if constexpr (!C::HALF) {
            const uint32_t* z = lo[mt][kk];
            mma_bf16(acc[mt][n], z[0], z[1], z[2], z[3], vf[0], vf[1]);
            mma_bf16(acc[mt][n + 1], z[0], z[1], z[2], z[3], vf[2], vf[3]);
          }
        }
      }
    const bool ends = at.tile + 1 == at.tiles, stop = at.unit + 1 + (ends ? at.gap(a) : 0) >= t1;
    if (ends || stop) end_pair(begins, ends);
    if (stop) break;
    ++at.tile;
    ++at.unit;
    if (ends) {
      at.next_pair<KT>(a);
      fresh = begins = true;
    }
  }
  if (!team || !named_bar_and(1, C::THREADS, true)) return;
  // ---- the block's four partials become one, in the slot of its first warp (the others' slots hold nothing), or, of a
  // block's own pair, the output
  const int head = blockIdx.x * C::WARPS;
  const long long o_row = my_g * a.so.h + my_i * a.so.r;
  for (int rr = warp; rr < min(RM, a.rows - rt * RM); rr += C::WARPS) {
    float2 ml[C::WARPS];
    float top = -INFINITY, sum = 0.f, w[C::WARPS];
#pragma unroll
    for (int x = 0; x < C::WARPS; ++x) {
      ml[x] = team_ml[x * RM + rr];
      top = fmaxf(top, ml[x].x);
    }
#pragma unroll
    for (int x = 0; x < C::WARPS; ++x) {
      w[x] = ml[x].x == -INFINITY ? 0.f : exp2f(ml[x].x - top);
      sum += ml[x].x == -INFINITY ? ml[x].y : w[x] * ml[x].y;   // (0, or NaN from keys that are all NaN)
    }
    auto slot_of = [&](int x) {
      return ((static_cast<long long>(rt) * a.workers + head + x) * 2 + (x == 0 && block0 == tile0 ? 1 : 0)) * a.part_rows + rr;
    };
    const long long off = __shfl_sync(0xffffffffu, o_row, rr);
    float f = 1.0f;
    if (a.by_block) {
      f = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
      if (lane == 0)
        a.lse[(static_cast<long long>(at.b) * a.H + at.h * a.group) * a.N + rt * RM + rr] =
            sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    } else if (lane < C::WARPS) {
      a.part_ml[slot_of(lane)] = lane == 0 ? make_float2(top, sum) : make_float2(-INFINITY, 0.f);
    }
    float* part = a.part_o + slot_of(0) * D;
    __nv_bfloat16* o = a.o + at.b * a.so.b + static_cast<long long>(at.h) * a.group * a.so.h + off;
#pragma unroll
    for (int e = 2 * lane; e < D; e += 64) {
      float2 z = make_float2(0.f, 0.f);
#pragma unroll
      for (int x = 0; x < C::WARPS; ++x) {
        const float2 y = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(smem + x * C::RING) + rr * D + e);
        if (ml[x].x == -INFINITY) continue;        // (a warp without tiles wrote nothing there)
        z.x = fmaf(w[x], y.x, z.x);
        z.y = fmaf(w[x], y.y, z.y);
      }
      if (a.by_block) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16x2(z.x * f, z.y * f);
      else *reinterpret_cast<float2*>(part + e) = z;
    }
  }
}

// Joins the partials of the pairs that several warps shared.  `per_row` warps (1, 2, 4 or 8) take a query row: a lane
// reads the weight of one partial, all lanes its columns.
template <int D>
__global__ void __launch_bounds__(256) fa_paged_merge_kernel(const __grid_constant__ PagedArgs a, int rm, int per_row) {
  constexpr int V = D / 32, W = V < 4 ? V : 4;     // columns of a lane: in pieces of W (8 or 16 bytes)
  auto col = [](int lane, int e) { return e / W * 32 * W + W * lane + e % W; };
  __shared__ float so[8][D];
  __shared__ float2 sml[8];
  __shared__ int2 list[8][32];                     // partial, weight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned rows = static_cast<unsigned>(a.B) * a.H * a.N;
  const unsigned row = blockIdx.x * (8u / per_row) + warp / per_row;
  const int sub = warp % per_row;
  after_previous_kernel();
  float acc[V];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  int more = 0, b = 0, hq = 0, i = 0;
  if (row < rows) {
    i = static_cast<int>(row % a.N);
    const unsigned bh = row / a.N;
    hq = static_cast<int>(bh % a.H);
    b = static_cast<int>(bh / a.H);
    const int h = hq / a.group, rr = (hq - h * a.group) * a.N + i, rt = rr / rm;
    const int2 mt = a.meta[(static_cast<long long>(rt) * a.B + b) * a.H_kv + h];
    // (a warp that gave up waiting left no entry: what stands there may be anything)
    more = mt.x >= 0 && mt.y > 0 && mt.y < a.workers && mt.x < a.workers - mt.y ? mt.y : 0;
    // partial j of the row: the first lies in slot 1 of its worker, the others in slot 0 of the workers behind it
    const long long first = (static_cast<long long>(rt) * a.workers + mt.x) * 2 * a.part_rows + rr - rt * rm;
    for (int j0 = 0; more > 0 && j0 <= more; j0 += 32 * per_row) {
      const int mine = j0 + sub + lane * per_row;  // this lane's partial
      float2 ml = make_float2(-INFINITY, 0.f);
      if (mine <= more) ml = a.part_ml[first + (2LL * mine + (mine == 0 ? 1 : 0)) * a.part_rows];
      float top = ml.x;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mn = fmaxf(m, top), nb = mn == -INFINITY ? 0.f : mn;
      const float old = exp2f(m - nb), w = mine <= more ? exp2f(ml.x - nb) : 0.f;
      float sum = w * ml.y;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l = l * old + sum;
      m = mn;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] *= old;
      // those that hold anything, in order (most of a long pair's are empty: a block leaves one)
      const unsigned there = __ballot_sync(0xffffffffu, !(w == 0.f));
      __syncwarp();                                // the last round's list has been read
      if (!(w == 0.f)) list[warp][__popc(there & ((1u << lane) - 1))] = make_int2(mine, __float_as_int(w));
      __syncwarp();
      const int cnt = __popc(there);
#pragma unroll 8
      for (int j = 0; j < cnt; ++j) {
        const int p = list[warp][j].x;
        const float f = __int_as_float(list[warp][j].y);
        const float* src = a.part_o + (first + (2LL * p + (p == 0 ? 1 : 0)) * a.part_rows) * D;
        struct __align__(4 * W) Piece { float x[W]; };
#pragma unroll
        for (int e = 0; e < V; e += W) {
          const Piece x = *reinterpret_cast<const Piece*>(src + col(lane, e));
#pragma unroll
          for (int u = 0; u < W; ++u) acc[e + u] = fmaf(f, x.x[u], acc[e + u]);
        }
      }
    }
  }
  if (per_row > 1) {                               // the row's warps in order: results do not depend on timing
#pragma unroll
    for (int e = 0; e < V; ++e) so[warp][col(lane, e)] = acc[e];
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (sub != 0) return;
    float top = m;
    for (int w = 1; w < per_row; ++w) top = fmaxf(top, sml[warp + w].x);
    const float nb = top == -INFINITY ? 0.f : top, own = exp2f(m - nb);
    m = top;
    l *= own;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= own;
    for (int w = 1; w < per_row; ++w) {
      const float f = exp2f(sml[warp + w].x - nb);
      l = fmaf(f, sml[warp + w].y, l);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(f, so[warp + w][col(lane, e)], acc[e]);
    }
  }
  if (more == 0) return;                           // written by the warp that had the whole pair
  const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
  __nv_bfloat16* o = a.o + row_offset(a.so, b, hq, i);
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<uint32_t*>(o + col(lane, e)) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace fa
