// Attention of one new token per row over paged keys and values.
//
// out = sum_t p_t v_t, p = softmax_t(scale <q, k_t>), in one pass over the visible tokens with a
// running maximum and sum.  What bounds it: HBM.  Every visible key and value is read once, by
// one wave, for all query heads of its kv head (up to 16 columns of the matrix instruction), at
// 4 d heads / (4 d kv_heads) = one to a few flops a byte.  8 kv heads of 128 in 16 bits: one row of
// 262144 tokens and 64 of 4096 6.1 to 6.4 TB/s, where a bare read stream reaches 7.2.
//
// Keys are read in whole rows like values: the 64-byte pieces of 16 rows that a matrix operand of keys
// asks for reach 6.1 TB/s in a bare read where whole rows reach 7.0.  A wave holds one tile, and what
// hides the loads is the other waves, three a SIMD (two tiles a wave, loaded in pieces: 64 ragged
// rows 108 us against 99, a window of 1024 18.7 against 17.3, 64 rows of 4096 tokens 171 against 175).
//
// A row's 32-token tiles are split over up to `splits` workgroups, each an equal share of the row's
// own length, and dealt to a workgroup's waves in turn.  The waves' (maximum, sum, output) are joined
// in LDS, the workgroups' through the workspace by a second kernel.
#include "attend_tile.h"

namespace fadkv {

namespace {

// Waves of a workgroup: eight where queries see many tokens, four where they see few and a wave of
// eight would have none or one of the tiles (64 ragged rows to 4096 tokens: 99 us with eight, 101 with
// four; one row of 131072: 91 and 92; a window of 1024: 19.3 and 17.3).
constexpr int AP_SHORT = 2048;
constexpr int AP_FILL = 2048;     // waves in all: two on each SIMD of the 256 CUs
constexpr int AP_ROWS = 8;        // splits of a row of several, at most, beyond those that fill the chip
constexpr int AP_LONG = 2048;     // tokens of such a split, half as many before the chip is full
constexpr int AP_LEAST = 256;     // tokens below which a share is not cut further
constexpr int AP_JOIN = 4;        // waves that join a query's splits
constexpr int AP_FEW = 8;         // splits that one thread joins,
constexpr int AP_MANY = 4096;     // where there are more queries than this

}  // namespace

int attend_paged_waves(int dtype, int64_t visible) {
  return dtype == DT_F32 || visible <= AP_SHORT ? 4 : 8;
}

// As many splits as fill the chip in one round (one row of 131072 tokens: 88 us, 92 in two rounds, 100
// in four).  Several rows are cut further, so that the end does not wait for the longest, where a
// share is long enough to pay for its start and for the join (ragged rows, 1 / 2 / 4 / 8 splits:
// 128 to 1024 tokens 53 / 59 / 64 / 64 us, 48 to 4096 93 / 85 / 84 / 94, 90 to 16384 320 / 291 / 281 / 289,
// 16 to 16384 with two, four and eight 112 / 97 / 91).
int attend_paged_splits(int dtype, int64_t R, int32_t kv_heads, int32_t group, int64_t visible) {
  const int64_t wgs = R * kv_heads * ((group + 15) / 16);
  const int64_t fill = AP_FILL / attend_paged_waves(dtype, visible);
  int64_t s = wgs > 0 ? (fill + wgs - 1) / wgs : 1;
  if (R > 1 && wgs < fill * 8) {   // beyond that the ends even out
    int64_t cut = visible / (wgs < fill ? AP_LONG / 2 : AP_LONG);
    cut = cut < AP_ROWS ? cut : AP_ROWS;
    s = s > cut ? s : cut;
  }
  const int64_t most = (visible + AP_LEAST - 1) / AP_LEAST;
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s);
}

// A window may leave few visible tokens of a long cache, which asks for more splits.
int attend_paged_most_splits(int dtype, int64_t R, int32_t kv_heads, int32_t group, int64_t len) {
  const int far = attend_paged_splits(dtype, R, kv_heads, group, len);
  const int near = attend_paged_splits(dtype, R, kv_heads, group, len < AP_SHORT ? len : AP_SHORT);
  return far > near ? far : near;
}

// the visible tiles of a row: those of the first tokens, then those of the window
struct TileList {
  int first, from, count;   // tiles [0, first), then [from, from + count - first)
};

__device__ __forceinline__ TileList tiles_of(int len, int window, int sinks) {
  TileList tl;
  const int last = (len + 31) >> 5;
  const int lo = window < len ? (len - window) >> 5 : 0;
  const int sk = sinks < len ? sinks : len;
  tl.first = (sk + 31) >> 5;
  if (tl.first >= lo) {   // they meet: one stretch
    tl.first = 0;
    tl.from = sk > 0 ? 0 : lo;
  } else {
    tl.from = lo;
  }
  tl.count = tl.first + last - tl.from;
  return tl;
}

// tiles of a split: an equal share, no less than AP_LEAST tokens
__device__ __forceinline__ int share_of(int count, int splits) {
  const int share = (count + splits - 1) / splits;
  return share < AP_LEAST / 32 ? AP_LEAST / 32 : share;
}

template <int DT, int D, int AP_WAVES, bool SPLIT>
__global__ __launch_bounds__(64 * AP_WAVES, DT == DT_F32 ? 2 : 3) void attend_paged_kernel(AttendArgs a) {
  using T = AttTile<DT, D>;
  using Tile = KvTile<DT, D, true, DT != DT_F32>;
  // a wave's own: its keys on their way to operands, then its output to be joined
  __shared__ __attribute__((aligned(16))) float s_o[AP_WAVES][16][D + 4];
  static_assert(DT == DT_F32 || 32 * T::ROWB <= sizeof(s_o[0]), "32 rows fit");
  __shared__ float s_m[AP_WAVES][16], s_l[AP_WAVES][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // kv head fastest: workgroups of one kv head land on one chiplet (8 heads, 8 chiplets)
  const int blocks = (a.group + 15) >> 4;
  unsigned b = blockIdx.x;
  const int head = (int)(b % a.kv_heads);
  b /= a.kv_heads;
  const int cb = (int)(b % blocks);
  b /= blocks;
  const int split = SPLIT ? (int)(b % a.splits) : 0;
  const int r = (int)(SPLIT ? b / a.splits : b);
  const int heads = a.kv_heads * a.group;

  const int64_t room = (int64_t)a.max_pages << a.page_shift;
  int len = a.lens[r];
  len = len < 0 ? 0 : ((int64_t)len > room ? (int)room : len);
  const TileList tl = tiles_of(len, a.window, a.sinks);
  const int share = SPLIT ? share_of(tl.count, a.splits) : tl.count;
  const int i0 = SPLIT ? split * share : 0;
  const int i1 = i0 + share < tl.count ? i0 + share : tl.count;

  const int col = lane & 15;
  const int gq = cb * 16 + col;
  const bool there = gq < a.group;
  if (SPLIT && i0 >= tl.count) {   // a short row's later splits have nothing
    const size_t qi = (size_t)r * heads + (size_t)head * a.group + gq;
    if (tid < 16 && there) a.part_ml[qi * a.splits + split] = make_float2(-__builtin_inff(), 0.f);
    return;
  }
  const uint8_t *qrow = static_cast<const uint8_t *>(a.q) +
                        ((size_t)r * heads + (size_t)head * a.group + (there ? gq : 0)) * T::ROWB;
  uint4 q[T::CH];
  load_queries<DT, D>(qrow, there, lane, q);
  PageView pv = {static_cast<const uint8_t *>(a.k), static_cast<const uint8_t *>(a.v),
                 a.table + (size_t)r * a.max_pages, a.num_pages, a.page_shift, a.kv_heads, head,
                 a.max_pages};
  const Visible see = {a.window < len ? len - a.window : 0, len};
  const float scale2 = a.scale * kLog2e;

  // Pages of the wave's tiles: lane k holds those of its k-th tile from here, so that a tile's
  // loads wait for no table entry.
  //
  // Every row and split starts at another of its tiles and comes round: rows whose pages follow one
  // another in the pool lie a power of two apart, and workgroups that walk them in step would
  // meet on the same memory channels (64 rows of 4096 tokens in pages of 16, in order: 173 us
  // against 223 us).
  const int mine = i1 > i0 ? i1 - i0 : 1;
  const int turn = (11 * r + 5 * split) % mine;
  const auto start_of = [&](int i) {
    i += i + turn < i1 ? turn : turn - mine;
    return (i < tl.first ? i : tl.from + i - tl.first) << 5;
  };
  int ids0 = -1, ids1 = -1;
  const auto fetch = [&](Tile &kv, int i) {
    const int k = (i - i0) / AP_WAVES;   // the wave's tile number
    if ((k & 63) == 0) {
      const int at = i + lane * AP_WAVES;
      ids0 = at < i1 ? page_of(pv, start_of(at)) : -1;
      ids1 = at < i1 ? page_of(pv, start_of(at) + 16) : -1;
    }
    kv.load(pv, __builtin_amdgcn_readlane(ids0, k & 63), __builtin_amdgcn_readlane(ids1, k & 63),
            start_of(i), lane);
  };
  AttState<DT, D> st;
  st.clear();
  const auto attend = [&](Tile &kv, int i) {
    if constexpr (DT != DT_F32) kv.turn(reinterpret_cast<uint8_t *>(&s_o[wave][0][0]), lane);
    const int t0 = start_of(i);
    const bool whole = kv.there[0] && kv.there[1] && t0 + 32 <= see.hi &&
                       (t0 >= see.lo || t0 + 32 <= a.sinks);
    attend_tile<DT, D, false>(kv, q, t0, whole, see, see, a.sinks, scale2, lane, st);
  };
  int i = i0 + wave;
  Tile kv;
  for (; i < i1; i += AP_WAVES) {
    fetch(kv, i);
    attend(kv, i);
  }

  // join the waves
  const float l = column_sum(st.l);
  const int g = lane >> 4;
#pragma unroll
  for (int e = 0; e < T::EP; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_o[wave][col][T::EP * (4 * g + i) + e] = st.o[e][i];
  if (g == 0) {
    s_m[wave][col] = st.m;
    s_l[wave][col] = l;
  }
  __syncthreads();
  const int here = a.group - cb * 16 < 16 ? a.group - cb * 16 : 16;
  for (int i = tid; i < here * (D / 4); i += 64 * AP_WAVES) {
    const int c = i / (D / 4), d4 = i % (D / 4);
    float m = s_m[0][c];
#pragma unroll
    for (int w = 1; w < AP_WAVES; ++w) m = fmaxf(m, s_m[w][c]);
    const float base = m == -__builtin_inff() ? 0.f : m;
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < AP_WAVES; ++w) {
      const float f = __builtin_amdgcn_exp2f(s_m[w][c] - base);
      const float4 x = *reinterpret_cast<const float4 *>(&s_o[w][c][4 * d4]);
      sum = fmaf(s_l[w][c], f, sum);
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
      o.z = fmaf(x.z, f, o.z);
      o.w = fmaf(x.w, f, o.w);
    }
    const size_t qi = (size_t)r * heads + (size_t)head * a.group + cb * 16 + c;
    if constexpr (SPLIT) {
      const size_t at = qi * a.splits + split;
      reinterpret_cast<float4 *>(a.part_o + at * D)[d4] = o;
      if (d4 == 0) a.part_ml[at] = make_float2(m, sum);
    } else {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;   // no visible token: 0
      if constexpr (DT == DT_F32) {
        reinterpret_cast<float4 *>(a.out)[qi * (D / 4) + d4] =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      } else {
        reinterpret_cast<uint2 *>(a.out)[qi * (D / 4) + d4] =
            make_uint2(round2<DT>(o.x * inv, o.y * inv), round2<DT>(o.z * inv, o.w * inv));
      }
    }
  }
}

// out[query] = the splits' outputs, each scaled from its own maximum to the common one, over the
// sum; parts without a visible token (maximum -inf) are not read.  One workgroup per query: its
// waves take the splits in turn and are joined in LDS.  With cu, queries of no row are left alone.
template <int DT, int D>
__global__ __launch_bounds__(64 * AP_JOIN) void attend_join_kernel(AttendArgs a) {
  __shared__ float s_o[AP_JOIN][D], s_sum[AP_JOIN];
  const size_t qi = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (a.cu) {
    const int64_t tok = (int64_t)(qi / (unsigned)(a.kv_heads * a.group));
    if (tok < a.cu[0] || tok >= a.cu[a.R]) return;
  }
  const float2 *ml = a.part_ml + qi * a.splits;
  float m = -__builtin_inff();
  for (int s = lane; s < a.splits; s += 64) m = fmaxf(m, ml[s].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  const float base = m == -__builtin_inff() ? 0.f : m;
  constexpr int E = D / 64;
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const float *po = a.part_o + qi * a.splits * D + lane * E;
#pragma unroll 4
  for (int s = wave; s < a.splits; s += AP_JOIN) {
    const float2 x = ml[s];
    if (x.x == -__builtin_inff() && x.y == 0.f) continue;
    const float f = __builtin_amdgcn_exp2f(x.x - base);
    sum = fmaf(x.y, f, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(po[(size_t)s * D + e], f, acc[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[wave][lane * E + e] = acc[e];
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  float y[2] = {0.f, 0.f};
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < AP_JOIN; ++w) {
    sum += s_sum[w];
    y[0] += s_o[w][2 * threadIdx.x];
    y[1] += s_o[w][2 * threadIdx.x + 1];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if constexpr (DT == DT_F32)
    static_cast<float2 *>(a.out)[qi * (D / 2) + threadIdx.x] = make_float2(y[0] * inv, y[1] * inv);
  else
    static_cast<uint32_t *>(a.out)[qi * (D / 2) + threadIdx.x] = round2<DT>(y[0] * inv, y[1] * inv);
}

// The same for few splits: D / 4 threads per query, each four elements of it
template <int DT, int D>
__global__ __launch_bounds__(256) void attend_join_few_kernel(AttendArgs a, int64_t queries) {
  constexpr int T = D / 4;
  const int64_t qi = (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T;
  const int d4 = threadIdx.x % T;
  if (qi >= queries) return;
  if (a.cu) {
    const int64_t tok = qi / (a.kv_heads * a.group);
    if (tok < a.cu[0] || tok >= a.cu[a.R]) return;
  }
  const float2 *ml = a.part_ml + qi * a.splits;
  const float4 *po = reinterpret_cast<const float4 *>(a.part_o + qi * a.splits * D) + d4;
  float m = -__builtin_inff();
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, ml[s].x);
  const float base = m == -__builtin_inff() ? 0.f : m;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float2 x = ml[s];
    if (x.x == -__builtin_inff() && x.y == 0.f) continue;
    const float f = __builtin_amdgcn_exp2f(x.x - base);
    const float4 v = po[(size_t)s * T];
    sum = fmaf(x.y, f, sum);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if constexpr (DT == DT_F32)
    static_cast<float4 *>(a.out)[qi * T + d4] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  else
    static_cast<uint2 *>(a.out)[qi * T + d4] =
        make_uint2(round2<DT>(o.x * inv, o.y * inv), round2<DT>(o.z * inv, o.w * inv));
}

template <int DT, int D>
static void attend_join_run(const AttendArgs &a, int64_t queries, hipStream_t stream) {
  constexpr int PER = 256 / (D / 4);
  // A workgroup per query is the shorter chain (512 queries of four splits: 3.9 us against 5.4),
  // until there are more than the chip takes at once (16384 queries of two splits: 18 us against
  // 4.8).
  if (a.splits <= AP_FEW && queries > AP_MANY)
    hipLaunchKernelGGL((attend_join_few_kernel<DT, D>), dim3((unsigned)((queries + PER - 1) / PER)),
                       dim3(256), 0, stream, a, queries);
  else
    hipLaunchKernelGGL((attend_join_kernel<DT, D>), dim3((unsigned)queries), dim3(64 * AP_JOIN), 0,
                       stream, a);
}

hipError_t launch_attend_join(int dtype, int d, const AttendArgs &a, int64_t queries,
                              hipStream_t stream) {
  if (dtype == DT_F32) {
    if (d == 64) attend_join_run<DT_F32, 64>(a, queries, stream);
    else attend_join_run<DT_F32, 128>(a, queries, stream);
  } else if (dtype == DT_F16) {
    if (d == 64) attend_join_run<DT_F16, 64>(a, queries, stream);
    else attend_join_run<DT_F16, 128>(a, queries, stream);
  } else {
    if (d == 64) attend_join_run<DT_BF16, 64>(a, queries, stream);
    else attend_join_run<DT_BF16, 128>(a, queries, stream);
  }
  return hipGetLastError();
}

template <int DT, int D, int WAVES>
static hipError_t attend_paged_run(const AttendArgs &a, hipStream_t stream) {
  const unsigned wgs = (unsigned)((size_t)a.R * a.kv_heads * ((a.group + 15) / 16));
  const dim3 block(64 * WAVES);
  if (a.splits > 1) {
    hipLaunchKernelGGL((attend_paged_kernel<DT, D, WAVES, true>), dim3(wgs * a.splits), block, 0, stream, a);
    return launch_attend_join(DT, D, a, (int64_t)a.R * a.kv_heads * a.group, stream);
  }
  hipLaunchKernelGGL((attend_paged_kernel<DT, D, WAVES, false>), dim3(wgs), block, 0, stream, a);
  return hipGetLastError();
}

template <int DT, int D>
static hipError_t attend_paged_run(const AttendArgs &a, int waves, hipStream_t stream) {
  if constexpr (DT != DT_F32)
    if (waves == 8) return attend_paged_run<DT, D, 8>(a, stream);
  return attend_paged_run<DT, D, 4>(a, stream);
}

hipError_t launch_attend_paged(int dtype, int d, const AttendArgs &a, int waves,
                               hipStream_t stream) {
  if (dtype == DT_F32)
    return d == 64 ? attend_paged_run<DT_F32, 64>(a, waves, stream)
                   : attend_paged_run<DT_F32, 128>(a, waves, stream);
  if (dtype == DT_F16)
    return d == 64 ? attend_paged_run<DT_F16, 64>(a, waves, stream)
                   : attend_paged_run<DT_F16, 128>(a, waves, stream);
  return d == 64 ? attend_paged_run<DT_BF16, 64>(a, waves, stream)
                 : attend_paged_run<DT_BF16, 128>(a, waves, stream);
}

}  // namespace fadkv
