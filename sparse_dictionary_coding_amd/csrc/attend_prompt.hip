// Causal attention of packed prompt tokens over paged keys and values.
//
// A row's (token, query head of the group) pairs, token by token, are the columns: the `group` query
// heads of a kv head share every key and value read.  A wave holds 16 columns and walks the
// visible tiles of 32 tokens (attend_tile.h).
#include "attend_tile.h"

namespace fadkv {

namespace {

constexpr int PR_WAVES = 4;

// Workgroup -> (row, block of `per` columns): rows in order, ceil(tokens * group / per) blocks each.
// Every lane of the wave gets the answer; row = R where the workgroup has none.
struct RowBlock {
  int row, block, begin, tokens;   // first packed token and token count of the row
};

__device__ __forceinline__ RowBlock find_row(const AttendArgs &a, int64_t blk, int per, int lane) {
  RowBlock rb = {a.R, 0, 0, 0};
  int64_t before = 0;
  for (int r0 = 0; r0 < a.R; r0 += 64) {
    const int r = r0 + lane;
    int64_t b = 0, e = 0;
    if (r < a.R) {
      b = a.cu[r];
      e = a.cu[r + 1];
      b = b < 0 ? 0 : (b > a.n ? a.n : b);
      e = e < b ? b : (e > a.n ? a.n : e);
    }
    const int64_t mine = ((e - b) * a.group + per - 1) / per;
    int64_t through = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t u = __shfl_up((long long)through, o, 64);
      if (lane >= o) through += u;
    }
    through += before;
    const unsigned long long hit = __ballot(blk < through);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      rb.row = r0 + src;
      rb.block = (int)(blk - __shfl((long long)(through - mine), src, 64));
      rb.begin = (int)__shfl((long long)b, src, 64);
      rb.tokens = (int)__shfl((long long)(e - b), src, 64);
      return rb;
    }
    before = __shfl((long long)through, 63, 64);
  }
  return rb;
}

}  // namespace

template <int DT, int D>
__global__ __launch_bounds__(64 * PR_WAVES) void attend_prompt_kernel(AttendArgs a) {
  using T = AttTile<DT, D>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int head = (int)(blockIdx.x % a.kv_heads);
  const RowBlock rb = find_row(a, blockIdx.x / a.kv_heads, 16 * PR_WAVES, lane);
  if (rb.row >= a.R) return;
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

  AttState<DT, D> st;
  st.clear();
  for (int t0 = 0; t0 < any.hi; t0 += 32) {
    if (t0 >= a.sinks && t0 + 32 <= any.lo) {   // between the first tokens and the window
      t0 = (any.lo & ~31) - 32;
      continue;
    }
    KvTile<DT, D> kv;
    kv.load(pv, t0, lane);
    const bool whole = kv.there[0] && kv.there[1] && t0 + 32 <= all.hi &&
                       (t0 >= all.lo || t0 + 32 <= a.sinks);
    attend_tile<DT, D>(kv, q, t0, whole, see, any, a.sinks, scale2, lane, st);
  }
  const float l = column_sum(st.l);
  const float inv = l == 0.f ? 0.f : 1.f / l;   // no visible token: 0
  float x[D / 4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < T::EP; ++e) x[T::EP * i + e] = st.o[e][i] * inv;
  if (there) store_output<DT, D>(static_cast<uint8_t *>(a.out) + qi * T::ROWB, lane, x);
}

template <int DT, int D> static void attend_prompt_run(const AttendArgs &a, hipStream_t stream) {
  // at most one started block more per row than the columns fill
  const int64_t blocks = a.n * a.group / (16 * PR_WAVES) + (a.R < a.n ? a.R : a.n);
  hipLaunchKernelGGL((attend_prompt_kernel<DT, D>), dim3((unsigned)(blocks * a.kv_heads)),
                     dim3(64 * PR_WAVES), 0, stream, a);
}

hipError_t launch_attend_prompt(int dtype, int d, const AttendArgs &a, hipStream_t stream) {
  if (dtype == DT_F32) {
    if (d == 64) attend_prompt_run<DT_F32, 64>(a, stream);
    else attend_prompt_run<DT_F32, 128>(a, stream);
  } else if (dtype == DT_F16) {
    if (d == 64) attend_prompt_run<DT_F16, 64>(a, stream);
    else attend_prompt_run<DT_F16, 128>(a, stream);
  } else {
    if (d == 64) attend_prompt_run<DT_BF16, 64>(a, stream);
    else attend_prompt_run<DT_BF16, 128>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace fadkv
