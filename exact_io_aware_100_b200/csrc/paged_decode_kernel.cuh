// Attention of the last N positions of each sequence over a paged key/value
// cache: o = softmax(scale q K^T) V over keys j < seq_len (and j <= seq_len - N + i
// when causal), lse = ln sum exp.
#pragma once

#include "layout.cuh"

namespace fa {

struct PagedArgs {
  const __nv_bfloat16 *q, *kp, *vp;
  __nv_bfloat16* o;
  float* lse;                      // [B, H, N]
  const int* table;
  long long table_stride;
  const int* seq_lens;
  Strides sq, so, skp, svp;        // skp, svp: {page, head, row}
  int B, H, H_kv, N, group;
  int num_pages, page, max_pages;
  int causal;
  float scale_log2;
  uint32_t* status;
};

// Keys of sequence b, 0 and flagged when the length makes no sense.
__device__ __forceinline__ int paged_len(const PagedArgs& a, int b) {
  const int n = __ldg(a.seq_lens + b);
  if (n < 0 || n > static_cast<long long>(a.max_pages) * a.page) {
    atomicOr(a.status, DEV_ARGS);
    return 0;
  }
  return n;
}

// One warp per query row: lanes over the head's columns, keys one after the other with an online softmax.
template <int D>
__global__ void __launch_bounds__(128) fa_paged_decode_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<long long>(a.B) * a.H * a.N) return;
  const int i = static_cast<int>(w % a.N), h = static_cast<int>(w / a.N % a.H), b = static_cast<int>(w / a.N / a.H);
  const int n = paged_len(a, b);
  const int end = a.causal ? min(n, n - a.N + i + 1) : n;
  float q[E], acc[E];
  for (int e = 0; e < E; ++e) {
    q[e] = static_cast<float>(a.q[row_offset(a.sq, b, h, i) + lane * E + e]) * a.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < end; ++j) {
    const int page = __ldg(a.table + b * a.table_stride + j / a.page);
    if (page < 0 || page >= a.num_pages) {
      atomicOr(a.status, DEV_ARGS);
      break;
    }
    const __nv_bfloat16* k = a.kp + row_offset(a.skp, page, h / a.group, j % a.page) + lane * E;
    const __nv_bfloat16* v = a.vp + row_offset(a.svp, page, h / a.group, j % a.page) + lane * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], static_cast<float>(k[e]), s);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), alpha = exp2f(m - mn), p = exp2f(s - mn);
    l = l * alpha + p;
    for (int e = 0; e < E; ++e) acc[e] = fmaf(p, static_cast<float>(v[e]), acc[e] * alpha);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int e = 0; e < E; ++e) a.o[row_offset(a.so, b, h, i) + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
  if (lane == 0) a.lse[w] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace fa
