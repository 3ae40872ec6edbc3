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
// the fraction of a turn, and the reduction loses nothing however far the position
// is.  What is left is the error of f / 2 pi in double (2^-52 relative: 1 / 2 pi and
// the product are rounded) times the angle: 5e-7 rad at position 2^31 with f = 1.
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
  const int* new_tokens;           // tokens among a sequence's rows (its last ones), or null: all
  const int* refused;              // not 0: none of the sequence's rows is a token; or null
  int total;
  int num_pages, page, max_pages;
  uint32_t* status;
};

// cos and sin (times the magnitude) of the angle pos * f.  FINE (32-bit outputs): the nearest quarter turn comes off as an
// integer first, so that what is rounded to 32 bits is an eighth of a turn at most and not half a one.  (Error of 32-bit
// outputs, relative 2-norm: 4.4e-8 -> 3.4e-8; with 3.2e-8 from sines in 64 bits.  Outputs in bf16 do not show it, and the
// selections took append of prompts from 62.8 to 66.6 us.)
template <bool FINE>
__device__ __forceinline__ float2 rot_cos_sin(double f, int pos, float magnitude, int inverse) {
  const double turn = fabs(f) * 0.15915494309189535;             // |f| / 2 pi (1 - |turn| would round a small one away)
  const bool back = (inverse != 0) != (__double2hiint(f) < 0);
  const unsigned long long step = __double2ull_rz((turn - floor(turn)) * 18446744073709551616.0);
  const long long where = static_cast<long long>(step * static_cast<unsigned long long>(static_cast<long long>(pos)));
  const unsigned at = static_cast<unsigned>(where >> 32), quarters = FINE ? (at + (1u << 29)) >> 30 : 0u;
  const float half_turns = static_cast<float>(static_cast<int>(at - (quarters << 30))) * 4.656612873077393e-10f;   // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  const float x = quarters & 1 ? s : c, y = quarters & 1 ? c : s;
  return make_float2(__fmul_rn((quarters + 1) & 2 ? -x : x, magnitude),
                     __fmul_rn(((quarters & 2) != 0) != back ? -y : y, magnitude));
}

template <typename T>
__device__ __forceinline__ float rot_load(const T* p) { return static_cast<float>(*p); }
template <typename T>
__device__ __forceinline__ void rot_store(T* p, float x) { *p = static_cast<T>(x); }   // to nearest even

// Packed offsets start at 0 or above, do not decrease and end at or below the number of rows.  The threads of the first
// heads look at one each (or at every so many): a token looks up its own sequence only.
template <bool APPEND>
__device__ __forceinline__ void rot_check_offsets(const RotArgs& a) {
  if constexpr (APPEND) {
    if (a.cu == nullptr || blockIdx.y != 0) return;
    const long long threads = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i <= a.B; i += threads) {
      const int at = a.cu[i], before = i > 0 ? a.cu[i - 1] : 0;
      if (at < before || at > a.total) atomicOr(a.status, DEV_ARGS);
    }
  }
}

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
    k.pos = a.pos ? a.pos[k.b * a.pos_b + k.row] : k.row;
    return k;
  } else {
    int back, rows;                // rows of the sequence from this one to its last; all of them
    if (a.cu) {
      const int row = static_cast<int>(t);
      int lo = 0, hi = a.B;        // the last b with cu[b] <= row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= row) lo = mid; else hi = mid;
      }
      const int first = a.cu[lo], end = a.cu[lo + 1];
      const int prev = lo > 0 ? a.cu[lo - 1] : first, next = lo + 2 <= a.B ? a.cu[lo + 2] : end;
      k.b = lo;
      k.row = row;
      k.pos = 0;
      back = end - row;
      rows = end - first;
      if (row < first || row >= end) { k.skip = true; return k; }
      if (first < 0 || end > a.total) { atomicOr(a.status, DEV_ARGS); k.skip = true; return k; }
      // out of order beside this sequence: its rows may be another's too (rot_check_offsets reports it)
      if (prev > first || next < end) { k.skip = true; return k; }
    } else {
      k.b = static_cast<int>(t / a.N);
      k.row = static_cast<int>(t - static_cast<long long>(k.b) * a.N);
      rows = a.N;
      back = rows - k.row;
    }
    // (independent loads: none waits for another)
    const int len = a.seq_lens[k.b], fresh = a.new_tokens ? a.new_tokens[k.b] : rows, no = a.refused ? a.refused[k.b] : 0;
    k.pos = len - back;
    if (no != 0) {
      k.page = -1;
      return k;
    }
    if (fresh < 0 || fresh > rows) {
      atomicOr(a.status, DEV_ARGS);
      k.skip = true;
      return k;
    }
    if (len < 0 || len > static_cast<long long>(a.max_pages) * a.page) {
      atomicOr(a.status, DEV_ARGS);
      k.skip = true;
      return k;
    }
    k.page = -1;
    if (k.pos >= 0 && back <= fresh) {
      const int slot = k.pos / a.page;
      k.in_page = k.pos - slot * a.page;
      k.page = a.table[k.b * a.table_stride + slot];
      if (k.page < 0 || k.page >= a.num_pages) {
        atomicOr(a.status, DEV_ARGS);
        k.skip = true;
      }
    }
    return k;
  }
}

// Heads hh of a launch: q's first, then k's, then (append) v's.
struct RotHead {
  const void* src;
  void* dst;
  bool turned;
};
template <typename T, bool APPEND>
__device__ __forceinline__ RotHead rot_head(const RotArgs& a, const RotToken& tk, int hh) {
  const int bc = APPEND && a.cu ? 0 : tk.b;
  const int ob = APPEND ? tk.page : bc, orow = APPEND ? tk.in_page : tk.row;   // where k and v go
  if (hh < a.H)
    return {static_cast<const T*>(a.q) + row_offset(a.sq, bc, hh, tk.row),
            static_cast<T*>(a.qo) + row_offset(a.sqo, bc, hh, tk.row), true};
  const int h = hh - a.H;
  if (!APPEND || h < a.H_kv)
    return {static_cast<const T*>(a.k) + row_offset(a.sk, bc, h, tk.row),
            static_cast<T*>(a.ko) + row_offset(a.sko, ob, h, orow), true};
  return {static_cast<const T*>(a.v) + row_offset(a.sv, bc, h - a.H_kv, tk.row),
          static_cast<T*>(a.vo) + row_offset(a.svo, ob, h - a.H_kv, orow), false};
}

// The pair of elements (xa, xb) turned, with the roundings fixed, so that every path gives the same bits.
__device__ __forceinline__ float2 rot_turn(float xa, float xb, float2 cs) {
  return make_float2(__fmaf_rn(xa, cs.x, -__fmul_rn(xb, cs.y)), __fmaf_rn(xb, cs.x, __fmul_rn(xa, cs.y)));
}

// Any alignment and any even r: one thread per (token, pair of columns, chunk of heads); thread p of a token takes pair
// p of the r / 2, or column r + (p - r / 2) of those that are copied.
template <typename T, bool APPEND>
__global__ void __launch_bounds__(256) fa_rotary_kernel(const RotArgs a, int interleaved, int heads_per) {
  after_previous_kernel();
  rot_check_offsets<APPEND>(a);
  const int half = a.r / 2, per = half + a.d - a.r;
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long t = idx / per;
  if (t >= a.tokens) return;
  const int p = static_cast<int>(idx - t * per);
  const RotToken tk = rot_token<APPEND>(a, t);
  const bool turn = p < half;
  const int ca = turn ? (interleaved ? 2 * p : p) : p + half, cb = turn ? (interleaved ? 2 * p + 1 : p + half) : ca;
  const float2 cs = turn ? rot_cos_sin<sizeof(T) == 4>(a.freqs[p], tk.pos, a.magnitude, a.inverse) : make_float2(1.f, 0.f);
  const bool pad = APPEND && (tk.skip || tk.page < 0);
  const int heads = pad ? (tk.skip && a.qo == a.q ? 0 : a.H) : a.H + (APPEND ? 2 : 1) * a.H_kv;
  const int h1 = min(heads, (static_cast<int>(blockIdx.y) + 1) * heads_per);
  for (int hh = blockIdx.y * heads_per; hh < h1; ++hh) {
    const RotHead r = rot_head<T, APPEND>(a, tk, hh);
    const T* x = static_cast<const T*>(r.src);
    T* y = static_cast<T*>(r.dst);
    if (pad) {
      rot_store(y + ca, 0.f);
      rot_store(y + cb, 0.f);
    } else if (!turn || !r.turned) {
      const T va = x[ca], vb = x[cb];
      y[ca] = va;
      y[cb] = vb;
    } else {
      const float2 z = rot_turn(rot_load(x + ca), rot_load(x + cb), cs);
      rot_store(y + ca, z.x);
      rot_store(y + cb, z.y);
    }
  }
}

// V elements of T (16 or 8 bytes) as floats, and back (to nearest even).
template <typename T, int V>
struct RotVec;
template <int V_>
struct RotVec<__nv_bfloat16, V_> {
  struct __align__(2 * V_) Word { uint32_t u[V_ / 2]; };
  __device__ static __forceinline__ void unpack(const Word& w, float (&x)[V_]) {
#pragma unroll
    for (int e = 0; e < V_ / 2; ++e) {
      const float2 f = bf16x2_to_float2(w.u[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
  __device__ static __forceinline__ Word pack(const float (&x)[V_]) {
    Word w;
#pragma unroll
    for (int e = 0; e < V_ / 2; ++e) w.u[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
    return w;
  }
};
template <int V_>
struct RotVec<float, V_> {
  struct __align__(4 * V_) Word { uint32_t u[V_]; };
  __device__ static __forceinline__ void unpack(const Word& w, float (&x)[V_]) {
#pragma unroll
    for (int e = 0; e < V_; ++e) x[e] = __uint_as_float(w.u[e]);
  }
  __device__ static __forceinline__ Word pack(const float (&x)[V_]) {
    Word w;
#pragma unroll
    for (int e = 0; e < V_; ++e) w.u[e] = __float_as_uint(x[e]);
    return w;
  }
};

// 16 or 8 bytes to shared memory, in the background.
template <int BYTES>
__device__ __forceinline__ void rot_fetch(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// The vector path: aligned rows whose turned columns fall into whole pairs of vectors of V elements (half layout: r a
// multiple of 2 V), or into whole vectors (interleaved: of V); d a multiple of 2 V.  A thread takes two vectors of a token
// in up to kRotHeads heads: it asks for all of them (through shared memory, where they cost no registers: 32 KB a block; with
// 40, 48 and 58 registers (fp32, bf16, append) 6, 5 and 4 blocks to an SM, 192, 160 and 128 KB in flight), forms the angles meanwhile, once for all heads, and turns and writes head by head.  It
// reads what it fetched itself: no barrier.  Training shape (2 x 40 heads x 8192 x 128, forward and backward): 109 us with
// 4 heads, 110 with 6, 112 with 8; 120 with four heads in flight in registers, 131 with angles shared through a block
// barrier; 111 with the fetches asked for before the token's look-ups (append of prompts 61.6 -> 63.8).
constexpr int kRotThreads = 256, kRotHeads = 4;
template <typename T, int V, bool APPEND, bool INTER>
__global__ void __launch_bounds__(kRotThreads) fa_rotary_vec_kernel(const __grid_constant__ RotArgs a, int heads_per) {
  using R = RotVec<T, V>;
  using Word = typename R::Word;
  extern __shared__ __align__(16) uint8_t rot_smem[];
  after_previous_kernel();
  rot_check_offsets<APPEND>(a);
  Word* buf = reinterpret_cast<Word*>(rot_smem) + threadIdx.x;   // [head][vector][thread]
  const int per = a.d / (2 * V), turning = a.r / (2 * V);      // items of a token, of which these turn
  const long long idx = static_cast<long long>(blockIdx.x) * kRotThreads + threadIdx.x;
  const long long t = idx / per;
  if (t >= a.tokens) return;
  const int p = static_cast<int>(idx - t * per);
  const RotToken tk = rot_token<APPEND>(a, t);
  // columns of the two vectors, far apart, so that a warp's accesses are contiguous: the pairs of the half layout, or
  // (interleaved) any two
  const bool turn = !INTER && p < turning;
  const int ca = turn || INTER ? V * p : a.r + V * (p - turning);
  const int cb = ca + (turn ? a.r : INTER ? a.d : a.d - a.r) / 2;
  const bool turn_a = INTER ? ca < a.r : turn, turn_b = INTER ? cb < a.r : turn;
  const bool pad = APPEND && (tk.skip || tk.page < 0);
  const int heads = pad ? (tk.skip && a.qo == a.q ? 0 : a.H) : a.H + (APPEND ? 2 : 1) * a.H_kv;
  const int h0 = blockIdx.y * heads_per, h1 = min(heads, h0 + heads_per);
  if (pad) {
    for (int h = h0; h < h1; ++h) {
      T* y = static_cast<T*>(rot_head<T, APPEND>(a, tk, h).dst);
      *reinterpret_cast<Word*>(y + ca) = Word{};
      *reinterpret_cast<Word*>(y + cb) = Word{};
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < kRotHeads; ++u)
    if (h0 + u < h1) {
      const T* x = static_cast<const T*>(rot_head<T, APPEND>(a, tk, h0 + u).src);
      rot_fetch<sizeof(Word)>(buf + (2 * u) * kRotThreads, x + ca);
      rot_fetch<sizeof(Word)>(buf + (2 * u + 1) * kRotThreads, x + cb);
    }
  float2 cs[V];                    // half layout: of column ca + e; interleaved: the pairs of one vector, then of the other
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < V / 2 ? turn_a : turn_b) {
      const int pair = INTER ? (e < V / 2 ? ca : cb - V) / 2 + e : ca + e;
      cs[e] = rot_cos_sin<sizeof(T) == 4>(a.freqs[pair], tk.pos, a.magnitude, a.inverse);
    }
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
  for (int h = h0; h < h1; ++h, buf += 2 * kRotThreads) {
    const RotHead r = rot_head<T, APPEND>(a, tk, h);
    T* y = static_cast<T*>(r.dst);
    Word va = buf[0], vb = buf[kRotThreads];
    if (r.turned && (turn_a || turn_b)) {
      float xa[V], xb[V];
      R::unpack(va, xa);
      R::unpack(vb, xb);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float& fa = INTER ? (e < V / 2 ? xa[2 * e] : xb[2 * e - V]) : xa[e];
        float& fb = INTER ? (e < V / 2 ? xa[2 * e + 1] : xb[2 * e + 1 - V]) : xb[e];
        if (e < V / 2 ? turn_a : turn_b) {
          const float2 z = rot_turn(fa, fb, cs[e]);
          fa = z.x;
          fb = z.y;
        }
      }
      if (turn_a) va = R::pack(xa);
      if (turn_b) vb = R::pack(xb);
    }
    *reinterpret_cast<Word*>(y + ca) = va;
    *reinterpret_cast<Word*>(y + cb) = vb;
  }
}

}  // namespace fa
