// Host side of the serving operators: rotary positions, the paged key/value cache, its attention and its pages.
// Included behind fa_api.cu, whose device state and checks it uses.
#pragma once

#include <algorithm>

#include "pages_kernel.cuh"
#include "paged_decode_kernel.cuh"
#include "rotary_kernel.cuh"

namespace fa {
namespace {

bool aligned_to(const void* p, size_t n) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % n == 0; }
bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws != nullptr && have >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0);
}
fa_status launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Launches a kernel that begins with after_previous_kernel(): it comes up while the kernel before it in the stream ends,
// which saves about a microsecond between the small kernels of a serving step.
template <typename... P>
fa_status launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                 const std::common_type_t<P>&... args) {
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  return launched();
}

// Strides of an output: rows of different (batch, head, row) do not coincide on an axis.
bool out_strides_ok(const fa_strides& st, int batch, int heads, int rows) {
  return (batch <= 1 || st.batch > 0) && (heads <= 1 || st.head > 0) && (rows <= 1 || st.row > 0);
}

// Can every row of the operand be moved in vectors of `bytes`?
bool vec_rows(const void* p, const Strides& st, int batch, int heads, int rows, long long bytes, long long es) {
  auto ok = [=](long long x, int extent) { return extent <= 1 || x * es % bytes == 0; };
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ok(st.b, batch) && ok(st.h, heads) && ok(st.r, rows);
}

template <typename T, int V, bool APPEND, bool INTER>
fa_status launch_rotary_vec(const RotArgs& a, dim3 grid, int heads_per, DevState* ds, cudaStream_t stream) {
  constexpr int kMost = kRotHeads * 2 * kRotThreads * V * sizeof(T), id = (sizeof(T) == 4 ? 0 : V == 4 ? 1 : 2) + 3 * APPEND + 6 * INTER;
  if (!ds->rotary_attr[id]) {
    if (cudaFuncSetAttribute(fa_rotary_vec_kernel<T, V, APPEND, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) !=
        cudaSuccess)
      return FA_ERR_CUDA;
    ds->rotary_attr[id] = true;
  }
  return launch(fa_rotary_vec_kernel<T, V, APPEND, INTER>, grid, kRotThreads, kMost / kRotHeads * heads_per, stream, a,
                heads_per);
}

template <typename T, bool APPEND>
fa_status launch_rotary(const RotArgs& a, int interleaved, DevState* ds, cudaStream_t stream) {
  constexpr int es = sizeof(T), V = 16 / es;
  const int heads = a.H + (APPEND ? 2 : 1) * a.H_kv;
  const int rows = APPEND && a.cu != nullptr ? a.total : a.N, nb = APPEND && a.cu != nullptr ? 1 : a.B;
  auto fits = [&](int v) {
    auto rows_ok = [&](const void* p, const Strides& st, int h) { return vec_rows(p, st, nb, h, rows, v * es, es); };
    return a.d % (2 * v) == 0 && a.r % (interleaved ? v : 2 * v) == 0 && (a.H == 0 || (rows_ok(a.q, a.sq, a.H) && rows_ok(a.qo, a.sqo, a.H))) &&
           (a.H_kv == 0 || APPEND || (rows_ok(a.k, a.sk, a.H_kv) && rows_ok(a.ko, a.sko, a.H_kv)));
  };
  const int v = fits(V) ? V : es == 2 && fits(4) ? 4 : 0;
  const long long per = v ? a.d / (2 * v) : a.r / 2 + a.d - a.r, blocks = (a.tokens * per + kRotThreads - 1) / kRotThreads;
  if (blocks >= (1LL << 31)) return FA_ERR_INVALID;
  // heads of a thread: kRotHeads, evenly over the chunks; fewer while there are not two blocks to an SM
  const long long few = std::max(1LL, blocks * heads / (2 * kPagedSms));
  const long long chunks = (heads + std::min<long long>(few, kRotHeads) - 1) / std::min<long long>(few, kRotHeads);
  const int heads_per = static_cast<int>((heads + chunks - 1) / chunks);
  const dim3 grid(static_cast<unsigned>(blocks), (heads + heads_per - 1) / heads_per);
  if (v == 0) return launch(fa_rotary_kernel<T, APPEND>, grid, kRotThreads, 0, stream, a, interleaved, heads_per);
  if (v == V)
    return interleaved ? launch_rotary_vec<T, V, APPEND, true>(a, grid, heads_per, ds, stream)
                       : launch_rotary_vec<T, V, APPEND, false>(a, grid, heads_per, ds, stream);
  return interleaved ? launch_rotary_vec<T, 4, APPEND, true>(a, grid, heads_per, ds, stream)
                     : launch_rotary_vec<T, 4, APPEND, false>(a, grid, heads_per, ds, stream);
}

// The cache and table of a paged layout.
fa_status check_paged(const fa_paged_layout& L) {
  if (L.B < 1 || L.H_kv < 1 || L.num_pages < 1 || L.max_pages < 1 || L.page_size < 1) return FA_ERR_INVALID;
  if (L.d != 64 && L.d != 128 && L.d != 256) return FA_ERR_UNSUPPORTED;
  if (L.page_size % 8 != 0 || L.page_size > 65536 || 1LL * L.max_pages * L.page_size > (1LL << 30) ||
      L.num_pages >= (1 << 30) || (L.B > 1 && L.table_stride < L.max_pages))
    return FA_ERR_INVALID;
  if (!strides_ok(L.k_pages, L.page_size, L.H_kv, L.num_pages) || !strides_ok(L.v_pages, L.page_size, L.H_kv, L.num_pages))
    return FA_ERR_ALIGN;
  return FA_OK;
}

fa_status check_decode(const fa_paged_layout& L) {
  const fa_status st = check_paged(L);
  if (st != FA_OK) return st;
  if (L.N < 1 || L.H < 1 || L.H % L.H_kv != 0 || 1LL * L.B * L.H * L.N >= (1LL << 31) ||
      1LL * (L.H / L.H_kv) * L.N >= (1LL << 19))
    return FA_ERR_INVALID;
  if (!strides_ok(L.q, L.N, L.H, L.B) || !strides_ok(L.o, L.N, L.H, L.B)) return FA_ERR_ALIGN;
  return FA_OK;
}

// How a decode call is cut up, and where its workspace's parts lie.
struct PagedPlan {
  int rm, row_tiles, workers, part_rows, min_units, whole_units, by_block;
  size_t o_bytes, ml_bytes, meta_bytes;            // none is needed when no pair is cut
  size_t bytes() const { return whole_units || by_block ? 256 : o_bytes + ml_bytes + meta_bytes; }
};
PagedPlan paged_plan(const fa_paged_layout& L) {
  PagedPlan p;
  const int rows = L.H / L.H_kv * L.N, kt = L.d == 64 ? 32 : 16;
  // the longest sequences that the table can hold, in tiles
  const long long most = (1LL * L.max_pages * L.page_size + kt - 1) / kt, pairs = 1LL * L.B * L.H_kv;
  p.rm = paged_row_tile(L.d, rows, pairs, most * pairs);
  p.row_tiles = (rows + p.rm - 1) / p.rm;
  p.part_rows = rows < p.rm ? rows : p.rm;
  // A range's partial (4 d bytes a row) should be no more than half of its keys (4 d bytes each)
  p.min_units = std::max(kPagedMinUnits, 2 * p.part_rows / kt);
  // no more warps than those sequences give work to
  const PagedShare share = paged_share(L.d, p.rm, pairs * p.row_tiles, most);
  p.whole_units = share == kPagedByWarp ? static_cast<int>(most) + kPagedPairUnits : 0;
  p.by_block = share == kPagedByBlock;
  const long long units = p.whole_units ? pairs : (most + kPagedPairUnits) * pairs, least = p.whole_units ? 1 : p.min_units;
  const long long ctas = (units + 4 * least - 1) / (4 * least);
  p.workers = paged_workers(p.row_tiles);
  if (ctas < p.workers / 4) p.workers = static_cast<int>(ctas) * 4;
  if (p.by_block) p.workers = static_cast<int>(pairs) * 4;
  const size_t parts = 2 * static_cast<size_t>(p.row_tiles) * p.workers * p.part_rows;
  p.o_bytes = round256(parts * L.d * 4);
  p.ml_bytes = round256(parts * 8);
  p.meta_bytes = round256(8 * static_cast<size_t>(p.row_tiles) * L.B * L.H_kv);
  return p;
}

// 5-D map of a cache's K or V pages, {64 columns, row, 64-column piece, head, page}, so that one box brings `box` keys of
// all d columns as pieces of 128-byte rows.
bool make_map_pages(CUtensorMap* m, const void* base, const fa_paged_layout& L, const fa_strides& st, int box) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dense = static_cast<cuuint64_t>(L.d) * 2;
  cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(L.page_size), static_cast<cuuint64_t>(L.d / 64),
                        static_cast<cuuint64_t>(L.H_kv), static_cast<cuuint64_t>(L.num_pages)};
  cuuint64_t strides[4] = {static_cast<cuuint64_t>(st.row) * 2, 128, L.H_kv > 1 ? static_cast<cuuint64_t>(st.head) * 2 : dense,
                           L.num_pages > 1 ? static_cast<cuuint64_t>(st.batch) * 2 : dense};
  cuuint32_t extent[5] = {64, static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(L.d / 64), 1, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, extent, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int D, int RM>
fa_status launch_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, bool* attr, cudaStream_t s) {
  using C = PagedCfg<D, RM>;
  if (!*attr) {
    if (cudaFuncSetAttribute(fa_paged_decode_kernel<D, RM>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
      return FA_ERR_CUDA;
    *attr = true;
  }
  const fa_status st = launch(fa_paged_decode_kernel<D, RM>, dim3(a.workers / C::WARPS, a.row_tiles), C::THREADS, C::SMEM, s,
                              tk, tv, a);
  if (st != FA_OK || a.whole_units || a.by_block) return st;
  // the merge: 8, 4, 2 or 1 warps to a row, as many as the GPU holds at once
  const long long rows = 1LL * a.B * a.H * a.N;
  const int per_row = rows <= kPagedSms * 8 ? 8 : rows <= kPagedSms * 16 ? 4 : rows <= kPagedSms * 32 ? 2 : 1;
  return launch(fa_paged_merge_kernel<D>, dim3(static_cast<unsigned>((rows * per_row + 7) / 8)), 256, 0, s, a,
                static_cast<int>(RM), per_row);
}

bool pages_layout_ok(const fa_pages_layout* L) {
  return L != nullptr && L->num_seqs >= 1 && L->num_pages >= 1 && L->num_pages < (1 << 30) && L->page_size >= 1 &&
         L->max_pages >= 1 && 1LL * L->max_pages * L->page_size < (1LL << 31) &&
         (L->num_seqs == 1 || L->table_stride >= L->max_pages);
}

// Threads of a planning block: fewer warps take barriers faster, more take long lists in fewer steps.  48 forks and 48
// extensions among 20000 pages: 10.3 + 5.6 us with 256 threads, 8.0 + 4.6 with 512, 9.0 + 5.5 with 1024.
int pages_threads(int items) { return items <= 512 ? 512 : kPagesThreads; }

// Workspace of the page calls: claim [S], snap [n], prefix [n], list [P], info [1].
size_t pages_ws_bytes(const fa_pages_layout& L, int n) {
  return round256(4 * static_cast<size_t>(L.num_seqs)) + 2 * round256(4 * static_cast<size_t>(n)) +
         round256(4 * static_cast<size_t>(L.num_pages)) + 256;
}

fa_status pages_args(PagesArgs* a, int32_t* table, int32_t* lens, int32_t* refs, const fa_pages_layout* L, int n,
                     void* ws, size_t ws_bytes, bool need_ws) {
  if (!pages_layout_ok(L) || n < 0) return FA_ERR_INVALID;
  if (!aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(refs, 4)) return FA_ERR_ALIGN;
  if (need_ws && !workspace_ok(ws, ws_bytes, pages_ws_bytes(*L, n))) return FA_ERR_WORKSPACE;
  DevState* ds = nullptr;
  const fa_status st = device_state(&ds);
  if (st != FA_OK) return st;
  *a = PagesArgs();
  a->table = table;
  a->table_stride = L->table_stride;
  a->lens = lens;
  a->refs = refs;
  a->S = L->num_seqs;
  a->P = L->num_pages;
  a->page = L->page_size;
  a->M = L->max_pages;
  a->n = n;
  if (need_ws) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    a->claim = reinterpret_cast<int*>(w);
    w += round256(4 * static_cast<size_t>(L->num_seqs));
    a->snap = reinterpret_cast<int*>(w);
    w += round256(4 * static_cast<size_t>(n));
    a->prefix = reinterpret_cast<int*>(w);
    w += round256(4 * static_cast<size_t>(n));
    a->list = reinterpret_cast<int*>(w);
    w += round256(4 * static_cast<size_t>(L->num_pages));
    a->info = reinterpret_cast<int*>(w);
  }
  a->dev_status = ds->status;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_rotary(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions,
                    const double* freqs, const fa_rotary_layout* layout, float magnitude, int inverse,
                    fa_dtype dtype, fa_stream_t stream) {
  if (layout == nullptr) return FA_ERR_INVALID;
  const fa_rotary_layout& L = *layout;
  if (L.B < 1 || L.H < 1 || L.H_kv < 0 || L.H >= (1 << 16) || L.H_kv >= (1 << 16) || L.N < 0 || L.d < 1 || L.d > 1024 || L.rotary_dim < 0 || L.rotary_dim > L.d ||
      L.rotary_dim % 2 != 0 || 1LL * L.B * L.N >= (1LL << 31) || !std::isfinite(magnitude) ||
      !out_strides_ok(L.q_out, L.B, L.H, L.N) || (L.H_kv > 0 && !out_strides_ok(L.k_out, L.B, L.H_kv, L.N)))
    return FA_ERR_INVALID;
  if (dtype != FA_BF16 && dtype != FA_F32) return FA_ERR_UNSUPPORTED;
  if (L.N == 0) return FA_OK;   // no row (and perhaps no memory)
  const size_t es = dtype == FA_F32 ? 4 : 2;
  if (!aligned_to(q, es) || !aligned_to(q_out, es) || (L.H_kv > 0 && (!aligned_to(k, es) || !aligned_to(k_out, es))) ||
      (positions != nullptr && !aligned_to(positions, 4)) || (L.rotary_dim > 0 && !aligned_to(freqs, 8)))
    return FA_ERR_ALIGN;
  RotArgs a = {};
  a.q = q;
  a.k = k;
  a.qo = q_out;
  a.ko = k_out;
  a.sq = kstrides(L.q);
  a.sk = kstrides(L.k);
  a.sqo = kstrides(L.q_out);
  a.sko = kstrides(L.k_out);
  a.pos = positions;
  a.pos_b = L.positions_batch;
  a.freqs = freqs;
  a.B = L.B;
  a.N = L.N;
  a.H = L.H;
  a.H_kv = L.H_kv;
  a.d = L.d;
  a.r = L.rotary_dim;
  a.tokens = 1LL * L.B * L.N;
  a.magnitude = magnitude;
  a.inverse = inverse;
  DevState* ds = nullptr;
  const fa_status st = device_state(&ds);
  if (st != FA_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == FA_F32 ? launch_rotary<float, false>(a, L.interleaved, ds, s)
                         : launch_rotary<__nv_bfloat16, false>(a, L.interleaved, ds, s);
}

fa_status fa_paged_append(const void* q, const void* k, const void* v, void* o, void* k_pages, void* v_pages,
                          const int32_t* page_table, const int32_t* seq_lens, const double* freqs,
                          const fa_paged_layout* layout, float magnitude, fa_stream_t stream) {
  if (layout == nullptr) return FA_ERR_INVALID;
  const fa_paged_layout& L = *layout;
  fa_status st = check_paged(L);
  if (st != FA_OK) return st;
  const bool pk = L.cu_seqlens != nullptr;
  const long long tokens = pk ? L.total : 1LL * L.B * L.N;
  if ((pk ? L.total : L.N) < 0 || tokens >= (1LL << 31) || (q != nullptr && (L.H < 1 || L.H >= (1 << 16))) || L.H_kv >= (1 << 16) || !std::isfinite(magnitude) ||
      (freqs != nullptr && (L.rotary_dim < 0 || L.rotary_dim > L.d || L.rotary_dim % 2 != 0)))
    return FA_ERR_INVALID;
  if (tokens == 0) return FA_OK;
  const int nb = pk ? 1 : L.B, rows = pk ? L.total : L.N;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned_to(page_table, 4) ||
      !aligned_to(seq_lens, 4) || (pk && !aligned_to(L.cu_seqlens, 4)) || (L.tokens != nullptr && !aligned_to(L.tokens, 4)) ||
      (L.status != nullptr && !aligned_to(L.status, 4)) || (freqs != nullptr && !aligned_to(freqs, 8)) ||
      (q != nullptr && (!aligned16(q) || !aligned16(o))) || !strides_ok(L.k, rows, L.H_kv, nb) ||
      !strides_ok(L.v, rows, L.H_kv, nb) ||
      (q != nullptr && (!strides_ok(L.q, rows, L.H, nb) || !strides_ok(L.o, rows, L.H, nb))))
    return FA_ERR_ALIGN;
  DevState* ds = nullptr;
  if ((st = device_state(&ds)) != FA_OK) return st;
  RotArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qo = o;
  a.ko = k_pages;
  a.vo = v_pages;
  a.sq = kstrides(L.q);
  a.sk = kstrides(L.k);
  a.sv = kstrides(L.v);
  a.sqo = kstrides(L.o);
  a.sko = kstrides(L.k_pages);
  a.svo = kstrides(L.v_pages);
  a.freqs = freqs;
  a.B = L.B;
  a.N = L.N;
  a.H = q != nullptr ? L.H : 0;
  a.H_kv = L.H_kv;
  a.d = L.d;
  a.r = freqs != nullptr ? L.rotary_dim : 0;
  a.tokens = tokens;
  a.magnitude = magnitude;
  a.table = page_table;
  a.table_stride = L.table_stride;
  a.seq_lens = seq_lens;
  a.cu = L.cu_seqlens;
  a.new_tokens = L.tokens;
  a.refused = L.status;
  a.total = L.total;
  a.num_pages = L.num_pages;
  a.page = L.page_size;
  a.max_pages = L.max_pages;
  a.status = ds->status;
  return launch_rotary<__nv_bfloat16, true>(a, L.interleaved, ds, static_cast<cudaStream_t>(stream));
}

size_t fa_paged_decode_workspace_size(const fa_paged_layout* layout) {
  if (layout == nullptr || check_decode(*layout) != FA_OK) return 0;
  return paged_plan(*layout).bytes();
}

fa_status fa_paged_decode(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                          const int32_t* seq_lens, void* o, float* lse, const fa_paged_layout* layout, float scale,
                          int causal, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (layout == nullptr) return FA_ERR_INVALID;
  const fa_paged_layout& L = *layout;
  fa_status st = check_decode(L);
  if (st != FA_OK) return st;
  if (!scale_ok(scale)) return FA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) || !aligned_to(lse, 4) ||
      !aligned_to(page_table, 4) || !aligned_to(seq_lens, 4))
    return FA_ERR_ALIGN;
  const PagedPlan plan = paged_plan(L);
  if (!workspace_ok(workspace, workspace_bytes, plan.bytes())) return FA_ERR_WORKSPACE;
  DevState* ds = nullptr;
  if ((st = device_state(&ds)) != FA_OK) return st;
  PagedArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.table = page_table;
  a.table_stride = L.table_stride;
  a.seq_lens = seq_lens;
  a.sq = kstrides(L.q);
  a.so = kstrides(L.o);
  a.B = L.B;
  a.H = L.H;
  a.H_kv = L.H_kv;
  a.N = L.N;
  a.group = L.H / L.H_kv;
  a.num_pages = L.num_pages;
  a.page = L.page_size;
  a.max_pages = L.max_pages;
  a.causal = causal ? 1 : 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = ds->status;
  a.rows = a.group * a.N;
  a.workers = plan.workers;
  a.row_tiles = plan.row_tiles;
  a.part_rows = plan.part_rows;
  a.min_units = plan.min_units;
  a.whole_units = plan.whole_units;
  a.by_block = plan.by_block;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + plan.o_bytes);
  a.meta = reinterpret_cast<int2*>(w + plan.o_bytes + plan.ml_bytes);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int kt = L.d == 64 ? 32 : 16;
  a.box = L.page_size % kt == 0 ? kt : L.page_size % 16 == 0 ? 16 : 8;
  a.wait_limit_ns = kWaitLimitNs;
  CUtensorMap tk, tv;
  if (!make_map_pages(&tk, k_pages, L, L.k_pages, a.box) || !make_map_pages(&tv, v_pages, L, L.v_pages, a.box))
    return FA_ERR_CUDA;
  const int di = L.d == 64 ? 0 : L.d == 128 ? 1 : 2, ri = plan.rm == 8 ? 0 : plan.rm == 16 ? 1 : 2;
  bool* attr = &ds->paged_attr[di][ri];
  switch (di * 3 + ri) {
    case 0: return launch_paged<64, 8>(tk, tv, a, attr, s);
    case 1: return launch_paged<64, 16>(tk, tv, a, attr, s);
    case 2: return launch_paged<64, 32>(tk, tv, a, attr, s);
    case 3: return launch_paged<128, 8>(tk, tv, a, attr, s);
    case 4: return launch_paged<128, 16>(tk, tv, a, attr, s);
    case 6: return launch_paged<256, 8>(tk, tv, a, attr, s);
    case 7: return launch_paged<256, 16>(tk, tv, a, attr, s);
    default: return FA_ERR_UNSUPPORTED;              // (32 rows of d 128 or 256: paged_row_tile gives none)
  }
}

size_t fa_pages_workspace_size(const fa_pages_layout* layout, int n) {
  return pages_layout_ok(layout) && n >= 0 ? pages_ws_bytes(*layout, n) : 0;
}

fa_status fa_pages_extend(int32_t* page_table, int32_t* seq_lens, int32_t* refcounts, const fa_pages_layout* layout,
                          const int32_t* seqs, const int32_t* tokens, int n, int32_t* status, void* workspace,
                          size_t workspace_bytes, fa_stream_t stream) {
  PagesArgs a;
  if (n > 0 && (!aligned_to(seqs, 4) || !aligned_to(tokens, 4) || !aligned_to(status, 4))) return FA_ERR_ALIGN;
  const fa_status st = pages_args(&a, page_table, seq_lens, refcounts, layout, n, workspace, workspace_bytes, true);
  if (st != FA_OK || n == 0) return st;
  a.seqs = seqs;
  a.arg = tokens;
  a.status = status;
  return launch(fa_pages_extend_kernel, dim3(1), pages_threads(n), 0, static_cast<cudaStream_t>(stream), a);
}

fa_status fa_pages_fork(int32_t* page_table, int32_t* seq_lens, int32_t* refcounts, const fa_pages_layout* layout,
                        const int32_t* src, const int32_t* dst, int n, int32_t* copies, int32_t* status,
                        void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  PagesArgs a;
  if (n > 0 && (!aligned_to(src, 4) || !aligned_to(dst, 4) || !aligned_to(copies, 4) || !aligned_to(status, 4)))
    return FA_ERR_ALIGN;
  const fa_status st = pages_args(&a, page_table, seq_lens, refcounts, layout, n, workspace, workspace_bytes, true);
  if (st != FA_OK || n == 0) return st;
  a.seqs = src;
  a.arg = dst;
  a.copies = copies;
  a.status = status;
  return launch(fa_pages_fork_kernel, dim3(1), pages_threads(n), 0, static_cast<cudaStream_t>(stream), a);
}

fa_status fa_pages_free(int32_t* page_table, int32_t* seq_lens, int32_t* refcounts, const fa_pages_layout* layout,
                        const int32_t* seqs, int n, fa_stream_t stream) {
  PagesArgs a;
  if (n > 0 && !aligned_to(seqs, 4)) return FA_ERR_ALIGN;
  const fa_status st = pages_args(&a, page_table, seq_lens, refcounts, layout, n, nullptr, 0, false);
  if (st != FA_OK || n == 0) return st;
  a.seqs = seqs;
  return launch(fa_pages_free_kernel, dim3((n + 3LL) / 4), 128, 0, static_cast<cudaStream_t>(stream), a);
}

fa_status fa_pages_compact(int32_t* page_table, const int32_t* seq_lens, int32_t* refcounts,
                           const fa_pages_layout* layout, int32_t* copies, void* workspace, size_t workspace_bytes,
                           fa_stream_t stream) {
  PagesArgs a;
  if (layout != nullptr && layout->num_pages > 1 && !aligned_to(copies, 4)) return FA_ERR_ALIGN;
  const fa_status st = pages_args(&a, page_table, const_cast<int32_t*>(seq_lens), refcounts, layout, 0, workspace,
                                  workspace_bytes, true);
  if (st != FA_OK) return st;
  a.copies = copies;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const fa_status planned = launch(fa_pages_plan_compact_kernel, dim3(1), pages_threads(a.P / kPagesPer), 0, s, a);
  if (planned != FA_OK || 1LL * a.S * a.M <= kPagesRenameHere) return planned;
  return launch(fa_pages_rename_kernel, dim3((a.S + 3LL) / 4), 128, 0, s, a);
}

fa_status fa_pages_copy(void* k_pages, void* v_pages, const int32_t* copies, int n, const fa_paged_layout* layout,
                        fa_stream_t stream) {
  if (layout == nullptr) return FA_ERR_INVALID;
  const fa_paged_layout& L = *layout;
  if (n < 0 || L.H_kv < 1 || L.num_pages < 1 || L.page_size < 1 || L.d < 8 || L.d % 8 != 0 ||
      2LL * L.H_kv * L.page_size * L.d >= (1LL << 31))
    return FA_ERR_INVALID;
  if (!aligned16(k_pages) || !aligned16(v_pages) || (n > 0 && !aligned_to(copies, 4)) ||
      !strides_ok(L.k_pages, L.page_size, L.H_kv, L.num_pages) || !strides_ok(L.v_pages, L.page_size, L.H_kv, L.num_pages))
    return FA_ERR_ALIGN;
  if (n == 0) return FA_OK;
  DevState* ds = nullptr;
  const fa_status st = device_state(&ds);
  if (st != FA_OK) return st;
  PageCopyArgs a;
  a.kp = static_cast<__nv_bfloat16*>(k_pages);
  a.vp = static_cast<__nv_bfloat16*>(v_pages);
  a.sk = kstrides(L.k_pages);
  a.sv = kstrides(L.v_pages);
  a.copies = copies;
  a.n = n;
  a.P = L.num_pages;
  a.page = L.page_size;
  a.H_kv = L.H_kv;
  a.d = L.d;
  a.status = ds->status;
  a.tpr = std::min(L.d / 8, 256);
  // parts of a copy: about kPageCopyBytes each, a head of K or V at most
  const long long unit = 2LL * L.page_size * L.d;
  const int want = static_cast<int>((unit + kPageCopyBytes - 1) / kPageCopyBytes);
  a.rows_per = (L.page_size + want - 1) / want;
  a.row_parts = (L.page_size + a.rows_per - 1) / a.rows_per;
  const long long parts = 2LL * L.H_kv * a.row_parts;
  const long long teams = std::max(1LL, std::min<long long>(n, ds->sms * 16LL / parts));
  if (teams * parts >= (1LL << 31)) return FA_ERR_INVALID;
  return launch(fa_pages_copy_kernel, dim3(static_cast<unsigned>(teams * parts)), 256, 0, static_cast<cudaStream_t>(stream), a);
}

}  // extern "C"
