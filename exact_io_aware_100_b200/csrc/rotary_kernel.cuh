// Rotary positions, and the append of new tokens to a paged key/value cache.
//
//     y_a = m (x_a cos t - x_b sin t),  y_b = m (x_b cos t + x_a sin t),  t = pos * f_i
//
// for the pairs (a, b) of a head's first r columns; the backward is the same map
// with -t (its transpose).  Both operators read their inputs once and write their
// outputs once, with 3 flops per element: HBM-bound.  The angle depends on the
// token and the pair only, so a thread forms it once and turns that pair in every head.
//
// Angles: t / 2 pi is wanted modulo 1.  f / 2 pi is held as a fixed-point fraction
// of 64 bits and multiplied by the integer position; the product modulo 2^64 is
// the fraction of a turn, exactly, however far the position is.  Its error is
// that of f / 2 pi in double (2^-53 relative) times the position.
#pragma once

#include "layout.cuh"

namespace fa {

struct RotArgs {
  const void *q, *k, *v;
  void *qo, *ko, *vo;              // ko, vo: the outputs, or the pages (append)
  Strides sq, sk, sv, sqo, sko, svo;   // append: sko, svo are {page, head, row}
  const int* pos;                  // rotary: positions (null: the row index)
  long long pos_b;
  const double* freqs;
  int B, N, H, H_kv, d, r;
  long long tokens;                // rows over all batch entries
  float magnitude;
  int inverse;
  // append
  const int* table;
  long long table_stride;
  const int* seq_lens;
  const int* cu;                   // packed offsets, or null
  int total;
  int num_pages, page, max_pages;
  uint32_t* status;
};

// cos and sin (times the magnitude) of the angle pos * f.
__device__ __forceinline__ float2 rot_cos_sin(double f, int pos, float magnitude, int inverse) {
  const double turn = f * 0.15915494309189535;                   // f / 2 pi
  const unsigned long long step = __double2ull_rz((turn - floor(turn)) * 18446744073709551616.0);
  const long long where = static_cast<long long>(step * static_cast<unsigned long long>(static_cast<long long>(pos)));
  const float half_turns = static_cast<float>(static_cast<int>(where >> 32)) * 4.656612873077393e-10f;   // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * magnitude, (inverse ? -s : s) * magnitude);
}

template <typename T>
__device__ __forceinline__ float rot_load(const T* p) { return static_cast<float>(*p); }
template <typename T>
__device__ __forceinline__ void rot_store(T* p, float x) { *p = static_cast<T>(x); }   // to nearest even

// Where a token is: sequence, row within it, row coordinate in the tensors, position; the page row it goes to.
struct RotToken {
  int b, row;
  int pos;
  int page, in_page;               // append; page < 0: padding (not written)
  bool skip;                       // a row of no sequence, or an inconsistent one: nothing but zeros in a separate qo
};

template <bool APPEND>
__device__ __forceinline__ RotToken rot_token(const RotArgs& a, long long t) {
  RotToken k;
  k.skip = false;
  k.page = k.in_page = 0;
  if constexpr (!APPEND) {
    k.b = static_cast<int>(t / a.N);
    k.row = static_cast<int>(t - static_cast<long long>(k.b) * a.N);
    k.pos = a.pos ? __ldg(a.pos + k.b * a.pos_b + k.row) : k.row;
    return k;
  } else {
    int back;                      // tokens of the sequence from this one to its last
    if (a.cu) {
      const int row = static_cast<int>(t);
      int lo = 0, hi = a.B;        // the last b with cu[b] <= row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= row) lo = mid; else hi = mid;
      }
      const int first = __ldg(a.cu + lo), end = __ldg(a.cu + lo + 1);
      k.b = lo;
      k.row = row;
      k.pos = 0;
      back = end - row;
      if (row < first || row >= end) { k.skip = true; return k; }
      if (first < 0 || end > a.total) { atomicOr(a.status, DEV_ARGS); k.skip = true; return k; }
    } else {
      k.b = static_cast<int>(t / a.N);
      k.row = static_cast<int>(t - static_cast<long long>(k.b) * a.N);
      back = a.N - k.row;
    }
    const int len = __ldg(a.seq_lens + k.b);
    k.pos = len - back;
    if (len < 0 || len > static_cast<long long>(a.max_pages) * a.page) {
      atomicOr(a.status, DEV_ARGS);
      k.skip = true;
      return k;
    }
    k.page = -1;
    if (k.pos >= 0) {
      const int slot = k.pos / a.page;
      k.in_page = k.pos - slot * a.page;
      k.page = __ldg(a.table + k.b * a.table_stride + slot);
      if (k.page < 0 || k.page >= a.num_pages) {
        atomicOr(a.status, DEV_ARGS);
        k.skip = true;
      }
    }
    return k;
  }
}

// One thread per (token, pair of columns), any alignment: thread p of a token takes pair p of the r / 2, or column
// r + (p - r / 2) of those that are copied, in every head.
template <typename T, bool APPEND>
__global__ void __launch_bounds__(256) fa_rotary_kernel(const RotArgs a, int interleaved) {
  const int half = a.r / 2, per = half + a.d - a.r;
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long t = idx / per;
  if (t >= a.tokens) return;
  const int p = static_cast<int>(idx - t * per);
  const RotToken tk = rot_token<APPEND>(a, t);
  const bool turn = p < half, pad = APPEND && (tk.skip || tk.page < 0);
  const int ca = turn ? (interleaved ? 2 * p : p) : p + half, cb = turn ? (interleaved ? 2 * p + 1 : p + half) : ca;
  const float2 cs = turn ? rot_cos_sin(__ldg(a.freqs + p), tk.pos, a.magnitude, a.inverse) : make_float2(1.f, 0.f);
  const int bc = APPEND && a.cu ? 0 : tk.b;
  auto move = [&](const void* src, const Strides& ss, int sb, int srow, void* dst, const Strides& sd, int db, int drow,
                  int heads, bool turned) {
    for (int h = 0; h < heads; ++h) {
      const T* x = static_cast<const T*>(src) + row_offset(ss, sb, h, srow);
      T* y = static_cast<T*>(dst) + row_offset(sd, db, h, drow);
      const T va = x[ca], vb = x[cb];
      if (!turn || !turned) {
        y[ca] = va;
        y[cb] = vb;
      } else {
        const float xa = static_cast<float>(va), xb = static_cast<float>(vb);
        rot_store(y + ca, xa * cs.x - xb * cs.y);
        rot_store(y + cb, xb * cs.x + xa * cs.y);
      }
    }
  };
  if (pad) {
    if (a.q && !(tk.skip && a.qo == a.q))
      for (int h = 0; h < a.H; ++h) {
        T* y = static_cast<T*>(a.qo) + row_offset(a.sqo, bc, h, tk.row);
        rot_store(y + ca, 0.f);
        rot_store(y + cb, 0.f);
      }
    return;
  }
  if (a.q) move(a.q, a.sq, bc, tk.row, a.qo, a.sqo, bc, tk.row, a.H, true);
  if (APPEND) {
    move(a.k, a.sk, bc, tk.row, a.ko, a.sko, tk.page, tk.in_page, a.H_kv, true);
    move(a.v, a.sv, bc, tk.row, a.vo, a.svo, tk.page, tk.in_page, a.H_kv, false);
  } else if (a.H_kv > 0) {
    move(a.k, a.sk, bc, tk.row, a.ko, a.sko, bc, tk.row, a.H_kv, true);
  }
}

}  // namespace fa
