// Causal attention of packed prompt tokens over paged keys and values.
//
// A row's (token, query head of the group) pairs, token by token, are the columns: the `group` query
// heads of a kv head share every key and value read.
//
// attend_prompt_mfma_kernel, 16-bit types: bound by the matrix cores and the vector unit, 4 d flops
// and one exponential per column and visible token.  A wave holds 32 columns, and the workgroup's
// four waves share tiles of 64 tokens that come into LDS by direct copies.  As in attend_tile.h the
// scores are computed transposed (S^T = K Q^T, v_mfma_f32_32x32x16), so that a lane's p are its
// entries of the second product's operand (O^T = V^T P^T) without leaving the lane, and V is read
// from LDS through the transposing load.  The next tile's scores are computed beside this one's
// softmax.  Per score the vector unit does a maximum, a multiply-add, an exponential, a sum and
// half a conversion; O is rescaled only where a column's maximum grows by more than 2^8 (p stays
// below 2^8, which fp32 sums and 16-bit p hold as well as p <= 1).
// 8192 tokens, 32 query and 8 kv heads of 128 in bf16: 540 to 575 us, 0.96 to 1.02 PFLOP/s, where the
// library's 8192^3 product reaches 1.2; two waves a SIMD overlap their matrix and vector instructions
// in part, and the clock falls to 2.0 GHz.
// fp32: the same with tiles of 32 tokens and v_mfma_f32_32x32x2, bound by the matrix cores: a product
// takes two keys, 4 apart as the scores lie, and a lane reads neighbouring elements of a key's value, one
// for each block of d.  4120 us, 133 TFLOP/s at the same shape (the library's product 154), where 16
// columns a wave with tiles in registers, each wave reading keys and values for itself, take 6800.
// Rows of few columns in fp32 (attend_prompt_few_kernel) do take those 16 columns a wave: half a block of
// 32 would be idle, and no tile waits for a barrier.
#include "attend_tile.h"
#include "tiles.h"

namespace fadkv {

namespace {

constexpr int PM_WAVES = 4;     // 32 columns a wave
constexpr int PR_WAVES = 4;     // fp32, few columns: 16 columns a wave
// Columns of a row, on average, up to which they are few (16 and 32 columns a wave: 64 rows of 4 columns
// 73 and 156 us, 5 of 148 35 and 41, 8 of 512 44 and 43 at d = 128, 2 of 500 45 and 55, 3 of 1000 248
// and 188, 3 of 2967 370 and 211).
constexpr int PR_FEW = 512;
// Few columns do not fill the chip: their tokens are then split over workgroups and joined, until
// the two workgroups a CU holds are all there or a share falls to this many tokens.
constexpr int PM_FILL = 512;
constexpr int least_share(int dtype) { return dtype == DT_F32 ? 64 : 256; }

// Workgroup -> (row, block of `per` columns).  Row r's blocks are numbered from
// floor(cu[r] * group / per) + r, which leaves room for all of them (ceil(x) <= floor(b) - floor(a) + 1
// for b - a = x) and, at most, one number without a block; so the row of a number is found by a
// search in cu, 64 rows a step, without adding up the rows before it.  The answer is the
// same for all lanes; tokens = 0 where the number has no block.
struct RowBlock {
  int row, block, begin, tokens;   // first packed token and token count of the row
};

__device__ __forceinline__ int64_t clamped_cu(const AttendArgs &a, int r) {
  const int64_t c = a.cu[r];
  return c < 0 ? 0 : (c > a.n ? a.n : c);
}

__device__ __forceinline__ RowBlock find_row(const AttendArgs &a, int64_t blk, int per, int lane) {
  int lo = 0, len = a.R;   // the row is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 63) >> 6;
    const int r = lo + lane * step;
    const bool at = lane * step < len && clamped_cu(a, r) * a.group / per + r <= blk;
    const unsigned long long hit = __ballot(at);
    const int k = hit ? 63 - __builtin_clzll(hit) : 0;
    lo += k * step;
    len = len - k * step < step ? len - k * step : step;
  }
  RowBlock rb = {lo, 0, 0, 0};
  const int64_t b = clamped_cu(a, lo), e = clamped_cu(a, lo + 1);
  const int64_t block = blk - (b * a.group / per + lo);
  if (e > b && block >= 0 && block < ((e - b) * a.group + per - 1) / per) {
    rb.block = __builtin_amdgcn_readfirstlane((int)block);
    rb.begin = __builtin_amdgcn_readfirstlane((int)b);
    rb.tokens = __builtin_amdgcn_readfirstlane((int)(e - b));
  }
  return rb;
}

}  // namespace

// The visible tiles of columns that some tokens of [lo, hi) and the first `sinks` are visible to:
// tiles [0, first) of the first tokens, then [from, from + count - first).
struct Tiles {
  int first, from, count;
};

__device__ __forceinline__ Tiles tiles_between(const Visible &any, int sinks, int tile) {
  Tiles tl;
  const int hi = any.hi > 0 ? any.hi : 0;
  const int last = (hi + tile - 1) / tile;
  tl.first = ((sinks < hi ? sinks : hi) + tile - 1) / tile;
  tl.from = any.lo / tile;
  if (tl.first >= tl.from) {   // they meet: one stretch
    tl.from = tl.first > 0 ? 0 : tl.from;
    tl.first = 0;
  }
  tl.count = tl.first + (last > tl.from ? last - tl.from : 0);
  return tl;
}

// tiles [i0, i1) of a split: an equal share, `least` at least
__device__ __forceinline__ void split_tiles(int count, int splits, int split, int least, int &i0,
                                            int &i1) {
  int share = (count + splits - 1) / splits;
  share = share < least ? least : share;
  const int64_t begin = (int64_t)split * share;
  i0 = begin < count ? (int)begin : count;
  i1 = i0 + share < count ? i0 + share : count;
}

// `blk` is kv head, then split, then block of columns, the first fastest
template <int DT, int D, bool SPLIT>
__global__ __launch_bounds__(64 * PR_WAVES) void attend_prompt_few_kernel(AttendArgs a) {
  using T = AttTile<DT, D>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  unsigned blk = blockIdx.x;
  const int head = (int)(blk % a.kv_heads);
  blk /= a.kv_heads;
  const int split = SPLIT ? (int)(blk % a.splits) : 0;
  if (SPLIT) blk /= a.splits;
  const RowBlock rb = find_row(a, blk, 16 * PR_WAVES, lane);
  if (rb.tokens == 0) return;
  const int heads = a.kv_heads * a.group;
  const int64_t room = (int64_t)a.max_pages << a.page_shift;
  int len = a.lens[rb.row];
  len = len < 0 ? 0 : ((int64_t)len > room ? (int)room : len);

  const int64_t c0 = ((int64_t)rb.block * PR_WAVES + wave) * 16;   // the wave's first column
  const int64_t cols = (int64_t)rb.tokens * a.group;
  if (c0 >= cols) return;
  const int64_t c = c0 + (lane & 15);
  const bool there = c < cols;
  const int tok = (int)((there ? c : cols - 1) / a.group), gq = (int)((there ? c : cols - 1) % a.group);
  const int pos = len - rb.tokens + tok;
  const Visible see = {a.window <= pos ? pos + 1 - a.window : 0, pos + 1};
  const size_t qi = (size_t)(rb.begin + tok) * heads + (size_t)head * a.group + gq;
  uint4 q[T::CH];
  load_queries<DT, D>(static_cast<const uint8_t *>(a.q) + qi * T::ROWB, there, lane, q);
  PageView pv = {static_cast<const uint8_t *>(a.k), static_cast<const uint8_t *>(a.v),
                 a.table + (size_t)rb.row * a.max_pages, a.num_pages, a.page_shift, a.kv_heads,
                 head, a.max_pages};
  // tokens that the wave's first and last column see bound its tiles
  const int64_t cl = c0 + 15 < cols ? c0 + 15 : cols - 1;
  const int pos0 = len - rb.tokens + (int)(c0 / a.group), pos1 = len - rb.tokens + (int)(cl / a.group);
  const Visible any = {a.window <= pos0 ? pos0 + 1 - a.window : 0, pos1 + 1};
  const Visible all = {a.window <= pos1 ? pos1 + 1 - a.window : 0, pos0 + 1};
  const float scale2 = a.scale * kLog2e;

  const Tiles tl = tiles_between(any, a.sinks, 32);
  const auto start_of = [&](int i) { return (i < tl.first ? i : tl.from + i - tl.first) * 32; };
  int i0 = 0, i1 = tl.count;
  if constexpr (SPLIT) split_tiles(tl.count, a.splits, split, least_share(DT) / 32, i0, i1);

  AttState<DT, D> st;
  st.clear();
  bool fine = true;
  for (int i = i0; i < i1 && fine; ++i) {
    const int t0 = start_of(i);
    KvTile<DT, D, false, false> kv;
    kv.load(pv, __builtin_amdgcn_readfirstlane(page_of(pv, t0)),
            __builtin_amdgcn_readfirstlane(page_of(pv, t0 + 16)), t0, lane);
    const bool whole = kv.there[0] && kv.there[1] && t0 + 32 <= all.hi &&
                       (t0 >= all.lo || t0 + 32 <= a.sinks);
    fine = attend_tile<DT, D, true>(kv, q, t0, whole, see, any, a.sinks, scale2, lane, st);
  }
  if (!fine) {
    for (int c = 0; c < 16 && c0 + c < cols; ++c) {
      const Visible own = {__shfl(see.lo, c, 64), __shfl(see.hi, c, 64)};
      const size_t cq = (size_t)__shfl((long long)qi, c, 64);
      float o[D / 64], m, l;
      attend_column<DT, D>(pv, static_cast<const uint8_t *>(a.q) + cq * T::ROWB, a.scale, own,
                           a.sinks, start_of, i0, i1, 32, lane, o, m, l);
      store_column<DT, D, SPLIT>(a, cq, split, lane, o, m, l);
    }
    return;
  }
  const float l = column_sum(st.l);
  float x[D / 4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < T::EP; ++e) x[T::EP * i + e] = st.o[e][i];
  if (!there) return;
  if constexpr (SPLIT) {
    const size_t at = qi * a.splits + split;
    store_output<DT_F32, D>(reinterpret_cast<uint8_t *>(a.part_o + at * D), lane, x);
    if (lane < 16) a.part_ml[at] = make_float2(st.m, l);
  } else {
    const float inv = l == 0.f ? 0.f : 1.f / l;   // no visible token: 0
#pragma unroll
    for (int i = 0; i < D / 4; ++i) x[i] *= inv;
    store_output<DT, D>(static_cast<uint8_t *>(a.out) + qi * T::ROWB, lane, x);
  }
}

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

template <int DT>
__device__ __forceinline__ void mfma32(const uint4 &a, const uint4 &b, float16_t &c) {
  if constexpr (DT == DT_F32) {
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  } else if constexpr (DT == DT_F16)
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a),
                                               __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  else
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Where the 16-byte chunk c of row r of a tile lies in its row.  Keys: a fragment read takes one
// chunk of 16 rows, values in 16 bits: two 32-byte pieces of 4 rows; both then hit distinct banks.
// Values in fp32 are read in whole rows.
template <int ROWB> __device__ __forceinline__ int key_swz(int r) {
  return ROWB >= 256 ? (r & 15) : ((r >> 1) & 7);
}
template <int DT, int D> __device__ __forceinline__ int value_swz(int r) {
  if (DT == DT_F32) return 0;
  return D == 128 ? ((r & 3) << 1) : (((r >> 1) & 1) << 1);
}

__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, 64); }

// workgroup barrier of LDS alone: the caller has waited for its own copies and LDS accesses
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace

template <int DT, int D, int WAVES, bool SPLIT>
__global__ __launch_bounds__(64 * WAVES, 2) void attend_prompt_mfma_kernel(AttendArgs a) {
  constexpr bool F32 = DT == DT_F32;
  constexpr int PT = F32 ? 32 : 64;      // tokens per tile
  constexpr int SB = PT / 32;            // 32-token score blocks
  constexpr int ROWB = D * Elem<DT>::bytes;
  constexpr int CPR = ROWB / 16;         // chunks per row
  constexpr int NB = D / 32;             // 32-element blocks of d
  constexpr int KC = ROWB / 32;          // 16-byte chunks of a row per lane
  constexpr int TILE = PT * ROWB;        // bytes of a K or V tile
  constexpr int ROWS_W = PT / WAVES;     // rows of a tile that a wave copies
  constexpr int LOADS = ROWS_W * ROWB / 1024;
  static_assert(ROWS_W <= 16 && LOADS >= 1, "a wave copies rows of one 16-token group");
  __shared__ __attribute__((aligned(256))) uint8_t s_kv[2][2][TILE];   // [stage][K, V]
  // [stage][wave's rows]: 1, no valid page; 2, an infinity or NaN that only some columns see
  __shared__ __attribute__((aligned(16))) int s_miss[2][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, h = lane >> 5;

  unsigned blk = blockIdx.x;
  const int head = (int)(blk % a.kv_heads);
  blk /= a.kv_heads;
  const int split = SPLIT ? (int)(blk % a.splits) : 0;
  if (SPLIT) blk /= a.splits;
  RowBlock rb = find_row(a, blk, 32 * WAVES, lane);
  if (rb.tokens == 0) return;
  const int heads = a.kv_heads * a.group;
  const int64_t cols = (int64_t)rb.tokens * a.group;
  // the blocks with the most tokens first
  rb.block = (int)((cols + 32 * WAVES - 1) / (32 * WAVES)) - 1 - rb.block;
  const int64_t room = (int64_t)a.max_pages << a.page_shift;
  int len = __builtin_amdgcn_readfirstlane(a.lens[rb.row]);
  len = len < 0 ? 0 : ((int64_t)len > room ? (int)room : len);
  const int pos_first = len - rb.tokens;   // position of the row's first query

  const int64_t b0 = (int64_t)rb.block * WAVES * 32;            // columns of the workgroup
  const int64_t b1 = (b0 + 32 * WAVES < cols ? b0 + 32 * WAVES : cols) - 1;
  const int64_t c0 = b0 + wave * 32;                            // and of the wave
  const int64_t c1 = c0 + 31 < cols ? c0 + 31 : cols - 1;
  const int64_t cc = c0 + col;
  const bool there = cc < cols;
  const int64_t ccl = there ? cc : cols - 1;
  const int tok = (int)(ccl / a.group), gq = (int)(ccl % a.group);
  const int pos = pos_first + tok;
  const auto lo_of = [&](int p) { return a.window <= p ? p + 1 - a.window : 0; };
  const Visible see = {lo_of(pos), pos + 1};
  const int wg0 = pos_first + (int)(b0 / a.group), wg1 = pos_first + (int)(b1 / a.group);
  const int w0 = pos_first + (int)((c0 < cols ? c0 : b0) / a.group);
  const int w1 = pos_first + (int)((c0 < cols ? c1 : b1) / a.group);
  const Visible any = {lo_of(wg0), wg1 + 1};                    // some column of the workgroup sees
  const Visible each = {lo_of(wg1), wg0 + 1};                   // every column of the workgroup sees
  const Visible all = {lo_of(w1), w0 + 1};                      // every column of the wave sees
  const size_t qi = (size_t)(rb.begin + tok) * heads + (size_t)head * a.group + gq;

  // queries: entry 8 h + j of product i is element 16 i + 8 h + j (fp32: entry h of four products of
  // two, 4 j + i, is element 8 j + 4 h + i).  The score's sign goes into q, so
  // that a column's largest score is its largest product.
  const bool flat = __builtin_fabsf(a.scale) < 1e-37f;   // all scores 0
  uint4 q[KC];
  {
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.q) + qi * ROWB);
    const uint32_t flip = a.scale < 0.f ? (F32 ? 0x80000000u : 0x80008000u) : 0u;
    const bool zero = !there || flat;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const uint4 w = zero ? make_uint4(0, 0, 0, 0) : src[2 * i + h];
      q[i] = make_uint4(w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip);
    }
  }
  const float scale2 = flat ? 1.f : __builtin_fabsf(a.scale) * kLog2e;

  PageView pv = {static_cast<const uint8_t *>(a.k), static_cast<const uint8_t *>(a.v),
                 a.table + (size_t)rb.row * a.max_pages, a.num_pages, a.page_shift, a.kv_heads,
                 head, a.max_pages};

  const Tiles tl = tiles_between(any, a.sinks, PT);
  const auto start_of = [&](int i) { return (i < tl.first ? i : tl.from + i - tl.first) * PT; };
  int i0 = 0, count = tl.count;   // tiles [i0, count)
  if constexpr (SPLIT) split_tiles(tl.count, a.splits, split, least_share(DT) / PT, i0, count);

  // this wave's rows of a tile: ROWS_W of the 16-token group grp
  const int grp = wave * ROWS_W / 16;
  const int row0 = wave * ROWS_W;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&s_kv[0][0][0];
  uint32_t koff[LOADS], voff[LOADS];
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int at = 64 * j + lane;
    const int r = row0 + at / CPR, c = at % CPR;
    koff[j] = (uint32_t)((r - grp * 16) * ROWB + (c ^ key_swz<ROWB>(r)) * 16);
    voff[j] = (uint32_t)((r - grp * 16) * ROWB + (c ^ value_swz<DT, D>(r)) * 16);
  }
  // Byte offset of the wave's group of tile i, or -1; asked for tile after tile.  A lane holds the
  // page of one of the next 64 tiles, so that no tile waits for its table entry.
  int ids = -1;
  const auto group_offset = [&](int i) -> int64_t {
    if (((i - i0) & 63) == 0) ids = i + lane < count ? page_of(pv, start_of(i + lane) + grp * 16) : -1;
    return group_at<ROWB>(pv, __builtin_amdgcn_readlane(ids, (i - i0) & 63), start_of(i) + grp * 16);
  };
  const auto copy_keys = [&](int stage, int64_t at) {
    if (at < 0) return;
    const uint8_t *src = tile::uniform_ptr(pv.k + at);
    const uint32_t dst = lds0 + (uint32_t)stage * 2 * TILE + (uint32_t)row0 * ROWB;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) tile::copy16_to_lds(src, koff[j], dst + 1024u * j);
  };
  const auto copy_values = [&](int stage, int64_t at) {
    if (lane == 0) s_miss[stage][wave] = at < 0;
    if (at < 0) return;
    const uint8_t *src = tile::uniform_ptr(pv.v + at);
    const uint32_t dst = lds0 + (uint32_t)stage * 2 * TILE + TILE + (uint32_t)row0 * ROWB;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) tile::copy16_to_lds(src, voff[j], dst + 1024u * j);
  };
  // After the copies have landed, where not every column sees the whole tile: values that no column
  // sees become zeros, as p = 0 does not undo an infinity or NaN; one that only some columns see
  // cannot be kept from the others here and sends the block to attend_column.
  const auto settle = [&](int i, int stage, int64_t at) {
    tile::wait_vmem();
    asm volatile("" ::: "memory");
    const int t0 = start_of(i);
    if (at < 0 || t0 + PT > each.hi || (t0 < each.lo && t0 + PT > a.sinks)) {
      constexpr int LPR = 64 / ROWS_W;   // lanes per row
      const int r = row0 + lane / LPR;
      const bool seen = at >= 0 && sees(any, a.sinks, t0 + r);
      uint4 *row = reinterpret_cast<uint4 *>(&s_kv[stage][1][r * ROWB]);
      uint32_t bad = 0;
#pragma unroll
      for (int c = 0; c < CPR; c += LPR) {
        uint4 *at16 = row + c + lane % LPR;
        if (seen) {
          const uint4 w = *at16;
          bad |= odd_value<DT>(w.x) | odd_value<DT>(w.y) | odd_value<DT>(w.z) | odd_value<DT>(w.w);
        } else {
          *at16 = make_uint4(0, 0, 0, 0);
        }
      }
      if (__any(bad != 0) && lane == 0) s_miss[stage][wave] = 2;
    }
    tile::wait_lds();
  };

  float16_t o[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[b][e] = 0.f;
  float m = -__builtin_inff(), base = 0.f, l = 0.f;   // m in units of 1 / scale2

  // the lane's byte offsets within a tile
  int kaddr[SB];
#pragma unroll
  for (int kb = 0; kb < SB; ++kb) kaddr[kb] = (32 * kb + col) * ROWB;
  const int kswz = key_swz<ROWB>(col);   // the same for col + 32
  // transposing read: lane 4 j + c of a 16-lane group gives key j's piece c, and gets element lane of
  // the four keys.  Row r of block b of V^T is element D/2 ((r >> 2) & 1) + 16 b + 4 (r >> 3) +
  // (r & 3), which leaves a lane with D/2 neighbouring elements of the output.
  const int vkey = 4 * h + ((lane & 15) >> 2);
  const int vr = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const int vel = (D / 2) * ((vr >> 2) & 1) + 4 * (vr >> 3);     // element of block 0

  // the scores of the tile whose keys lie in `stage`
  const auto scores = [&](int stage, float16_t (&s)[SB]) {
    const uint8_t *kt = s_kv[stage][0];
#pragma unroll
    for (int kb = 0; kb < SB; ++kb) {
#pragma unroll
      for (int e = 0; e < 16; ++e) s[kb][e] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint4 ka = *reinterpret_cast<const uint4 *>(kt + kaddr[kb] + (((2 * c + h) ^ kswz) << 4));
        mfma32<DT>(ka, q[c], s[kb]);
      }
    }
  };

  // Tile i's softmax and second product run while the scores of tile i + 1 are computed: keys are
  // copied two tiles ahead, values one.
  const int64_t at_v = group_offset(i0);
  int64_t at_k = group_offset(i0 + 1);
  float16_t s[SB];
  bool fine = true;
  if (i0 < count) {
    copy_keys(0, at_v);
    copy_values(0, at_v);
    copy_keys(1, at_k);
    settle(i0, 0, at_v);
  }
  lds_barrier();
  if (i0 < count) scores(0, s);
  for (int i = i0; i < count; ++i) {
    const int stage = (i - i0) & 1;
    const int4 miss = *reinterpret_cast<const int4 *>(s_miss[stage]);
    const int gone[4] = {__builtin_amdgcn_readfirstlane(miss.x), __builtin_amdgcn_readfirstlane(miss.y),
                         __builtin_amdgcn_readfirstlane(miss.z), __builtin_amdgcn_readfirstlane(miss.w)};
    if ((gone[0] | gone[1] | gone[2] | gone[3]) & 2) {   // the same for all waves
      fine = false;
      break;
    }
    const int64_t at_now = at_k;             // tile i + 1
    at_k = group_offset(i + 2);
    const int t0 = start_of(i);
    if (i + 2 < count) copy_keys(stage, at_k);
    const bool full = !(gone[0] | gone[1] | gone[2] | gone[3]) && t0 + PT <= all.hi &&
                      (t0 >= all.lo || t0 + PT <= a.sinks);
    if (!full) {
      // against offsets from the lane's first token, which leaves constants on this side
      const int at = t0 + 4 * h;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        constexpr int EG = 4 * SB;   // entries of a wave's rows
        const Visible c = {see.lo - at, gone[g] ? -1 : see.hi - at};
#pragma unroll
        for (int e = EG * g; e < EG * g + EG; ++e) {
          const bool seen = sees(c, a.sinks - at, 8 * (e >> 2) + (e & 3));
          s[e >> 4][e & 15] = seen ? s[e >> 4][e & 15] : -__builtin_inff();
        }
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < SB; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[kb][e]);
    if (__any(top * scale2 > m + 8.f)) {
      top = fmaxf(top, other_half(top)) * scale2;
      const float grown = fmaxf(m, top);
      const float nb = grown == -__builtin_inff() ? 0.f : grown;
      const float keep = __builtin_amdgcn_exp2f(m - nb);
      m = grown;
      base = nb;
      l *= keep;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[b][e] *= keep;
    }
    if (i + 1 < count) copy_values(stage ^ 1, at_now);
    __builtin_amdgcn_iglp_opt(0);   // LDS reads and products in turn: 551 -> 543 us at 8192 tokens
    float16_t next[SB];
    scores(stage ^ 1, next);   // behind the last tile: of old keys, not used
    const uint8_t *vt = s_kv[stage][1];
    if constexpr (F32) {
      // product e takes the two halves' keys 8 (e >> 2) + 4 h + (e & 3), which is where p lies; a lane
      // reads NB neighbouring elements of its key, one for each block of d
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[0][e] = __builtin_amdgcn_exp2f(fmaf(s[0][e], scale2, -base));
        sum += s[0][e];
      }
      l += sum;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint8_t *src = vt + (8 * (e >> 2) + 4 * h + (e & 3)) * ROWB + 4 * NB * col;
        float w[NB];
        if constexpr (NB == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(src);
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(src);
          w[0] = x.x; w[1] = x.y;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
          o[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(w[b], s[0][e], o[b], 0, 0, 0);
      }
    } else {
      uint4 p[4];
#pragma unroll
      for (int kb = 0; kb < SB; ++kb) {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] = __builtin_amdgcn_exp2f(fmaf(s[kb][e], scale2, -base));
          l += x[e];
        }
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2)
          p[2 * kb + g2] = make_uint4(round2<DT>(x[8 * g2], x[8 * g2 + 1]), round2<DT>(x[8 * g2 + 2], x[8 * g2 + 3]),
                                      round2<DT>(x[8 * g2 + 4], x[8 * g2 + 5]), round2<DT>(x[8 * g2 + 6], x[8 * g2 + 7]));
      }
#pragma unroll
      for (int g2 = 0; g2 < 4; ++g2) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint2 w[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = 16 * g2 + 8 * u + vkey;
            const int el = vel + 16 * b;
            const uint8_t *src = vt + r * ROWB + (((el >> 3) ^ value_swz<DT, D>(vkey)) << 4) + ((el & 7) << 1);
            w[u] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t *)src));
          }
          mfma32<DT>(make_uint4(w[0].x, w[0].y, w[1].x, w[1].y), p[g2], o[b]);
        }
      }
    }
    if (i + 1 < count) settle(i + 1, stage ^ 1, at_now);
    lds_barrier();
#pragma unroll
    for (int kb = 0; kb < SB; ++kb) s[kb] = next[kb];
  }
  if (!fine) {
    for (int c = 0; c < 32 && c0 + c < cols; ++c) {
      const Visible own = {__shfl(see.lo, c, 64), __shfl(see.hi, c, 64)};
      const size_t cq = (size_t)__shfl((long long)qi, c, 64);
      float co[D / 64], cm, cl;
      attend_column<DT, D>(pv, static_cast<const uint8_t *>(a.q) + cq * ROWB, a.scale, own, a.sinks,
                           start_of, i0, count, PT, lane, co, cm, cl);
      store_column<DT, D, SPLIT>(a, cq, split, lane, co, cm, cl);
    }
    return;
  }
  if (!there) return;
  l += other_half(l);
  const float inv = SPLIT ? 1.f : (l == 0.f ? 0.f : 1.f / l);   // no visible token: 0
  const size_t at = SPLIT ? qi * a.splits + split : qi;
  if (SPLIT && h == 0) a.part_ml[at] = make_float2(m, l);
  if constexpr (F32) {   // entry e of block b is element NB (8 (e >> 2) + 4 h + (e & 3)) + b
    float *dst = (SPLIT ? a.part_o : static_cast<float *>(a.out)) + at * D + 4 * NB * h;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float *to = dst + NB * (8 * (e >> 2) + (e & 3));
      if constexpr (NB == 4)
        *reinterpret_cast<float4 *>(to) = make_float4(o[0][e] * inv, o[1][e] * inv, o[2][e] * inv, o[3][e] * inv);
      else
        *reinterpret_cast<float2 *>(to) = make_float2(o[0][e] * inv, o[1][e] * inv);
    }
  } else if constexpr (SPLIT) {
    float4 *dst = reinterpret_cast<float4 *>(a.part_o + at * D + h * (D / 2));
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        dst[4 * b + u] = make_float4(o[b][4 * u], o[b][4 * u + 1], o[b][4 * u + 2], o[b][4 * u + 3]);
  } else {
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.out) + at * ROWB + h * D);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = o[b][8 * u + e] * inv;
        dst[2 * b + u] = make_uint4(round2<DT>(x[0], x[1]), round2<DT>(x[2], x[3]),
                                    round2<DT>(x[4], x[5]), round2<DT>(x[6], x[7]));
      }
  }
}

static bool few_columns(int dtype, int64_t R, int64_t n, int32_t group) {
  return dtype == DT_F32 && n * group <= PR_FEW * (R < n ? R : n);
}

// columns per workgroup
static int prompt_columns(int dtype, int64_t R, int64_t n, int32_t group) {
  return few_columns(dtype, R, n, group) ? 16 * PR_WAVES : 32 * PM_WAVES;
}

int attend_prompt_splits(int dtype, int64_t R, int64_t n, int32_t kv_heads, int32_t group,
                         int64_t visible) {
  const int64_t wgs =
      (n * group / prompt_columns(dtype, R, n, group) + (R < n ? R : n)) * kv_heads;
  int64_t s = wgs > 0 ? PM_FILL / wgs : 1;
  const int64_t least = least_share(dtype);
  const int64_t most = (visible + least - 1) / least;
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s);
}

template <int DT, int D, bool SPLIT>
static void attend_prompt_run(const AttendArgs &a, hipStream_t stream) {
  // the blocks' numbers end below floor(n * group / columns) + R (find_row)
  const int64_t wgs = (a.n * a.group / prompt_columns(DT, a.R, a.n, a.group) + a.R) * a.kv_heads;
  const dim3 grid((unsigned)(wgs * a.splits));
  if constexpr (DT == DT_F32)
    if (few_columns(DT, a.R, a.n, a.group)) {
      hipLaunchKernelGGL((attend_prompt_few_kernel<DT, D, SPLIT>), grid, dim3(64 * PR_WAVES), 0, stream, a);
      return;
    }
  hipLaunchKernelGGL((attend_prompt_mfma_kernel<DT, D, PM_WAVES, SPLIT>), grid, dim3(64 * PM_WAVES), 0,
                     stream, a);
}

template <int DT, int D>
static hipError_t attend_prompt_run(const AttendArgs &a, hipStream_t stream) {
  if (a.splits > 1) {
    attend_prompt_run<DT, D, true>(a, stream);
    return launch_attend_join(DT, D, a, a.n * a.kv_heads * a.group, stream);
  }
  attend_prompt_run<DT, D, false>(a, stream);
  return hipGetLastError();
}

hipError_t launch_attend_prompt(int dtype, int d, const AttendArgs &a, hipStream_t stream) {
  if (dtype == DT_F32)
    return d == 64 ? attend_prompt_run<DT_F32, 64>(a, stream) : attend_prompt_run<DT_F32, 128>(a, stream);
  if (dtype == DT_F16)
    return d == 64 ? attend_prompt_run<DT_F16, 64>(a, stream) : attend_prompt_run<DT_F16, 128>(a, stream);
  return d == 64 ? attend_prompt_run<DT_BF16, 64>(a, stream) : attend_prompt_run<DT_BF16, 128>(a, stream);
}

}  // namespace fadkv
