// One wave's work on 32 cached tokens for 16 query columns (gfx950, wave64): the part that the
// paged attention kernels share.
//
// Scores come transposed, S^T = K Q^T: the A operand's rows are 16 keys and the B operand's columns
// the 16 queries, so after the product lane l holds, for query l % 16, the scores of keys
// 4 (l / 16) + e.  The sum over keys in O^T = V^T P^T may run in any order, so the four values a
// lane holds of each of two 16-key groups are its eight entries of the second product's B
// operand as they stand: p never moves between lanes.  A column's maximum needs two exchanges
// (lanes l, l ^ 16, l ^ 32), its sum none until the end, and rescaling O is per lane.
//
// The A operand of the second product wants, per lane, eight keys of one element d.  A lane reads
// d / 16 neighbouring elements (16 bytes at d = 128 in 16 bits) of each of its eight keys, which is
// a coalesced read of whole rows, and transposes them in registers: operand e takes element e of
// the eight.  Output row r of product e is then element (d / 16) r + e, so the lane ends up with
// d / 4 neighbouring elements of its query's output.  No LDS, no barrier in the loop.
#pragma once

#include "common.h"
#include "dense.h"

namespace fadkv {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

template <int DT, int D> struct AttTile {
  static constexpr int ES = Elem<DT>::bytes;
  static constexpr int ROWB = D * ES;
  static constexpr int CH = ROWB / 64;    // 16-byte chunks of a q or k row per lane
  static constexpr int EP = D / 16;       // neighbouring elements of a v row per lane
  static constexpr int VW = EP * ES / 4;  // their 32-bit words
};

// pages of one kv head: byte offsets of 16-token groups
struct PageView {
  const uint8_t *k, *v;
  const int32_t *table;   // of the row
  int num_pages, page_shift, kv_heads, head, max_pages;
};

// the page of the 16 tokens from t0 (a multiple of 16), -1 past the table
__device__ __forceinline__ int page_of(const PageView &pv, int t0) {
  const int pg = t0 >> pv.page_shift;
  return pg < pv.max_pages ? pv.table[pg] : -1;
}

// byte offset of the 16 tokens from t0 in page id (scalars), or -1 where that is no page
template <int ROWB>
__device__ __forceinline__ int64_t group_at(const PageView &pv, int id, int t0) {
  if (id < 0 || id >= pv.num_pages) return -1;
  const int off = t0 & ((1 << pv.page_shift) - 1);
  return (int64_t)(((((size_t)id * pv.kv_heads + pv.head) << pv.page_shift) + off) * ROWB);
}

template <int DT>
__device__ __forceinline__ void mfma16(const uint4 &a, const uint4 &b, f32x4_t &c) {
  if constexpr (DT == DT_F16) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                               __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  } else if constexpr (DT == DT_BF16) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  } else {
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  }
}

// two floats to one word of 16-bit values, round to nearest even
template <int DT> __device__ __forceinline__ uint32_t round2(float a, float b) {
  if constexpr (DT == DT_F16) {
    half2_t h;
    h[0] = (_Float16)a;
    h[1] = (_Float16)b;
    return __builtin_bit_cast(uint32_t, h);
  } else {
    bf16x2_t h;
    h[0] = (__bf16)a;
    h[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, h);
  }
}

// what a column sees: tokens [lo, hi) and [0, min(sinks, hi))
struct Visible {
  int lo, hi;
};

// (without branches)
__device__ __forceinline__ bool sees(const Visible &s, int sinks, int t) {
  return (t < s.hi) & ((t >= s.lo) | (t < sinks));
}

template <int DT, int D> struct AttState {
  f32x4_t o[AttTile<DT, D>::EP];
  float m, l;   // running maximum (of scores times scale log2 e) and this lane's share of the sum

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < AttTile<DT, D>::EP; ++e) o[e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    m = -__builtin_inff();
    l = 0.f;
  }
};

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// ONCE: what is loaded is not read again soon and leaves the caches to others
template <bool ONCE, class T> __device__ __forceinline__ T load_vec(const void *p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(static_cast<const T *>(p));
  else return *static_cast<const T *>(p);
}

// Keys and values of 32 tokens in registers.  A matrix operand wants 16 bytes of each of 16 keys per
// load; ROWS loads whole rows instead (1 KB of neighbouring bytes), which turn() then exchanges into
// operands through LDS.
template <int DT, int D, bool ONCE, bool ROWS> struct KvTile {
  uint4 k[2][AttTile<DT, D>::CH];
  uint32_t v[8][AttTile<DT, D>::VW];
  bool there[2];

  // id0, id1: pages of the two 16-token groups (scalars).  Groups without a valid page read as
  // zeros and are masked by the caller.
  __device__ __forceinline__ void load(const PageView &pv, int id0, int id1, int t0, int lane) {
    using T = AttTile<DT, D>;
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int64_t at = group_at<T::ROWB>(pv, a ? id1 : id0, t0 + 16 * a);
      there[a] = at >= 0;
      if (there[a]) {
        const u32x4_t *src = reinterpret_cast<const u32x4_t *>(pv.k + at);
#pragma unroll
        for (int i = 0; i < T::CH; ++i)
          k[a][i] = __builtin_bit_cast(uint4, load_vec<ONCE, u32x4_t>(
              src + (ROWS ? 64 * i + lane : r * (T::ROWB / 16) + 4 * i + g)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t *row =
              reinterpret_cast<const uint32_t *>(pv.v + at + (size_t)(4 * g + e) * T::ROWB) + r * T::VW;
          uint32_t *dst = v[4 * a + e];
          if constexpr (T::VW == 2) {
            const u32x2_t w = load_vec<ONCE, u32x2_t>(row);
            dst[0] = w[0]; dst[1] = w[1];
          } else {
#pragma unroll
            for (int c = 0; c < T::VW / 4; ++c) {
              const u32x4_t w = load_vec<ONCE, u32x4_t>(row + 4 * c);
#pragma unroll
              for (int x = 0; x < 4; ++x) dst[4 * c + x] = w[x];
            }
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < T::CH; ++i) k[a][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < T::VW; ++c) v[4 * a + e][c] = 0;
      }
    }
  }

  // ROWS: the keys into operand order, through 32 rows of the wave's own LDS.  Chunk c of row r lies
  // at c ^ f(r), so that 16 rows' reads of one chunk hit distinct banks.
  __device__ __forceinline__ void turn(uint8_t *lds, int lane) {
    using T = AttTile<DT, D>;
    constexpr int CPR = T::ROWB / 16;
    const auto place = [](int row, int c) {
      return (row * CPR + (c ^ (CPR == 16 ? row & 15 : (row >> 1) & 7))) * 16;
    };
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < T::CH; ++i) {
        const int at = 64 * i + lane;
        *reinterpret_cast<uint4 *>(lds + place(16 * a + at / CPR, at % CPR)) = k[a][i];
      }
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < T::CH; ++i)
        k[a][i] = *reinterpret_cast<const uint4 *>(
            lds + place(16 * a + (lane & 15), 4 * i + (lane >> 4)));
  }
};

// Not 0 where a value of the 32-bit word (two in the 16-bit types) is an infinity or NaN: one added
// to an exponent of all ones carries into the sign's place.
template <int DT> __device__ __forceinline__ uint32_t odd_value(uint32_t w) {
  if constexpr (DT == DT_F32) return ((w & 0x7f800000u) + 0x00800000u) & 0x80000000u;
  else if constexpr (DT == DT_F16) return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
  else return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// One tile against the wave's 16 columns.  `whole`: every column sees all 32 tokens (uniform).
// Tokens that no column sees are zeroed in v: p = 0 does not undo an infinity or NaN there.  Where
// the columns see different tokens (MIXED) the same holds for a token that some of them see: then
// nothing is done and the answer is false (attend_column does such blocks).
template <int DT, int D, bool MIXED, bool ONCE, bool ROWS>
__device__ __forceinline__ bool attend_tile(KvTile<DT, D, ONCE, ROWS> &kv, const uint4 (&q)[AttTile<DT, D>::CH],
                                            int t0, bool whole, const Visible &col,
                                            const Visible &any, int sinks, float scale2, int lane,
                                            AttState<DT, D> &st) {
  using T = AttTile<DT, D>;
  const int g = lane >> 4;
  f32x4_t s[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    s[a] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < T::CH; ++i) mfma16<DT>(kv.k[a][i], q[i], s[a]);
  }
  float z[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] = s[j >> 2][j & 3] * scale2;
  if (!whole) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // against offsets from the lane's first token, which leaves constants on this side
      const int k = 16 * (j >> 2) + (j & 3), at = t0 + 4 * g;
      const Visible c = {col.lo - at, kv.there[j >> 2] ? col.hi - at : -1};
      const Visible a = {any.lo - at, any.hi - at};
      z[j] = sees(c, sinks - at, k) ? z[j] : -__builtin_inff();
      const bool used = sees(a, sinks - at, k);
#pragma unroll
      for (int w = 0; w < T::VW; ++w) kv.v[j][w] = used ? kv.v[j][w] : 0;
    }
    if constexpr (MIXED) {
      uint32_t bad = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < T::VW; ++c) bad |= odd_value<DT>(kv.v[j][c]);
      if (__any(bad != 0)) return false;
    }
  }
  float top = z[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) top = fmaxf(top, z[j]);
  top = fmaxf(top, __shfl_xor(top, 16, 64));
  top = fmaxf(top, __shfl_xor(top, 32, 64));
  const float m = fmaxf(st.m, top);
  const float base = m == -__builtin_inff() ? 0.f : m;   // nothing visible yet: all weights are 0
  const float keep = __builtin_amdgcn_exp2f(st.m - base);
  st.m = m;
  float p[8], sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j] = __builtin_amdgcn_exp2f(z[j] - base);
    sum += p[j];
  }
  st.l = fmaf(st.l, keep, sum);
#pragma unroll
  for (int e = 0; e < T::EP; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) st.o[e][i] *= keep;
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < T::EP; ++e)
        st.o[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kv.v[j][e]), p[j], st.o[e], 0, 0, 0);
  } else {
    // p to the type of v: the matrix cores take no other, and half a step of it (2^-9 in bf16, random
    // over the tokens) is what the output's own rounding costs; the sum above is of p itself
    const uint4 pb = make_uint4(round2<DT>(p[0], p[1]), round2<DT>(p[2], p[3]),
                                round2<DT>(p[4], p[5]), round2<DT>(p[6], p[7]));
#pragma unroll
    for (int e = 0; e < T::EP; ++e) {
      // bytes 1:0 (e even) or 3:2 (e odd) of two keys' words
      constexpr uint32_t kLo = 0x05040100u, kHi = 0x07060302u;
      const uint32_t sel = (e & 1) ? kHi : kLo;
      const uint4 va = make_uint4(__builtin_amdgcn_perm(kv.v[1][e / 2], kv.v[0][e / 2], sel),
                                  __builtin_amdgcn_perm(kv.v[3][e / 2], kv.v[2][e / 2], sel),
                                  __builtin_amdgcn_perm(kv.v[5][e / 2], kv.v[4][e / 2], sel),
                                  __builtin_amdgcn_perm(kv.v[7][e / 2], kv.v[6][e / 2], sel));
      mfma16<DT>(va, pb, st.o[e]);
    }
  }
  return true;
}

// c + the products of 16 bytes of two rows
template <int DT> __device__ __forceinline__ float dot16(const uint4 &a, const uint4 &b, float c) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DT_F32) {
      c = fmaf(__uint_as_float(x[i]), __uint_as_float(y[i]), c);
    } else {
      c = fmaf(lo_f<DT>(x[i]), lo_f<DT>(y[i]), c);
      c = fmaf(hi_f<DT>(x[i]), hi_f<DT>(y[i]), c);
    }
  }
  return c;
}

// One column by itself over tiles [i0, i1) of `step` <= 64 tokens, a token per lane: nothing that the
// column does not see is multiplied, whatever it holds.  The path of blocks that
// hold an infinity or NaN where the tiles above cannot keep it from the columns that do not see it.
// Lane l ends up with elements l D / 64 .. of the output, not yet divided by the sum; (m, l) likewise.
template <int DT, int D, class Start>
__device__ __forceinline__ void attend_column(const PageView &pv, const uint8_t *qrow, float scale,
                                              const Visible &see, int sinks, Start start_of, int i0,
                                              int i1, int step, int lane, float (&o)[D / 64],
                                              float &m, float &l) {
  constexpr int E = D / 64, ROWB = D * Elem<DT>::bytes;
  const float scale2 = scale * kLog2e;
  m = -__builtin_inff();
  l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int i = i0; i < i1; ++i) {
    const int t = start_of(i) + lane;
    bool on = lane < step && sees(see, sinks, t);
    const int id = on ? page_of(pv, t) : -1;
    on = id >= 0 && id < pv.num_pages;
    const int off = t & ((1 << pv.page_shift) - 1);
    const int64_t at =
        on ? (int64_t)(((((size_t)id * pv.kv_heads + pv.head) << pv.page_shift) + off) * ROWB) : 0;
    float z = -__builtin_inff();
    if (on) {
      float dot = 0.f;
      const uint4 *qv = reinterpret_cast<const uint4 *>(qrow);
      const uint4 *kv = reinterpret_cast<const uint4 *>(pv.k + at);
#pragma unroll 4
      for (int c = 0; c < ROWB / 16; ++c) dot = dot16<DT>(qv[c], kv[c], dot);
      z = dot * scale2;
    }
    float top = z;
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x, 64));
    const float grown = fmaxf(m, top);
    const float base = grown == -__builtin_inff() ? 0.f : grown;
    const float keep = __builtin_amdgcn_exp2f(m - base);
    m = grown;
    const float p = on ? __builtin_amdgcn_exp2f(z - base) : 0.f;
    l = fmaf(l, keep, wave_sum(p));
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    for (unsigned long long left = __ballot(on); left; left &= left - 1) {
      const int j = __builtin_ctzll(left);
      const float pj = __shfl(p, j, 64);
      const uint8_t *row = pv.v + __shfl((long long)at, j, 64);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(pj, elem_f<DT>(row, lane * E + e), o[e]);
    }
  }
}

// and stores it: a part of a split, or the output
template <int DT, int D, bool SPLIT>
__device__ __forceinline__ void store_column(const AttendArgs &a, size_t qi, int split, int lane,
                                             const float (&o)[D / 64], float m, float l) {
  constexpr int E = D / 64;
  if constexpr (SPLIT) {
    const size_t at = qi * a.splits + split;
#pragma unroll
    for (int e = 0; e < E; ++e) a.part_o[at * D + lane * E + e] = o[e];
    if (lane == 0) a.part_ml[at] = make_float2(m, l);
  } else {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const size_t at = qi * D + lane * E + e;
      if constexpr (DT == DT_F32) static_cast<float *>(a.out)[at] = o[e] * inv;
      else static_cast<uint16_t *>(a.out)[at] = (uint16_t)round2<DT>(o[e] * inv, 0.f);
    }
  }
}

// the 16 queries' B operand; lanes of an absent column hold zeros
template <int DT, int D>
__device__ __forceinline__ void load_queries(const uint8_t *row, bool there, int lane,
                                             uint4 (&q)[AttTile<DT, D>::CH]) {
  const uint4 *src = reinterpret_cast<const uint4 *>(row);
#pragma unroll
  for (int i = 0; i < AttTile<DT, D>::CH; ++i)
    q[i] = there ? src[4 * i + (lane >> 4)] : make_uint4(0, 0, 0, 0);
}

// a column's sum over its four lanes
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// a lane's D / 4 output elements (element i: product i % EP, row entry i / EP) of a row
template <int DT, int D>
__device__ __forceinline__ void store_output(uint8_t *row, int lane, const float (&x)[D / 4]) {
  if constexpr (DT == DT_F32) {
    float4 *dst = reinterpret_cast<float4 *>(row) + (lane >> 4) * (D / 16);
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
      dst[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
  } else {
    uint4 *dst = reinterpret_cast<uint4 *>(row) + (lane >> 4) * (D / 32);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      dst[c] = make_uint4(round2<DT>(x[8 * c], x[8 * c + 1]), round2<DT>(x[8 * c + 2], x[8 * c + 3]),
                          round2<DT>(x[8 * c + 4], x[8 * c + 5]),
                          round2<DT>(x[8 * c + 6], x[8 * c + 7]));
  }
}

}  // namespace fadkv
