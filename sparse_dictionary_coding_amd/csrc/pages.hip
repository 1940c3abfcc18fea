// Paged-cache bookkeeping: request lengths -> block table, slots, positions.
//
// With P tokens a page, row r needs ceil((len + new) / P) - ceil(len / P) new pages; where they sit
// in the free ring, where the row's tokens sit in the packed batch and where released pages go
// are three prefix sums over the rows.  Released pages are appended behind the free ones, so the
// entries that are read (the ring's head) and written (behind its tail) never meet and the rows
// can be filled in any order.
//
// What bounds it: latency.  A step moves a few KB, so the time is the launches and the chain
// length -> sums -> ring entry -> table and slot.  Up to 1024 rows the sums and row records fit
// LDS: a small step is ONE workgroup that scans and fills everything itself (64 rows of one token:
// 3.6 us), and a large one is many that each scan all rows and fill a part, as long as none of
// them can see the new lengths that the first one stores (lens_out and ring_state_out are
// arrays of their own).  Otherwise one workgroup scans and many fill: tokens by a binary search of
// their row in an LDS copy of cu, pages with one wave per row (256 rows, 262144 tokens: 11.6 us for
// the two launches).
#include "common.h"
#include "dense.h"

namespace fadkv {

namespace {

constexpr int SCAN_THREADS = 1024;
constexpr int FILL_THREADS = 256;
constexpr int FILL_TOKENS = 4 * FILL_THREADS;   // tokens per fill workgroup
constexpr int MAX_ROWS = 8192;                  // rows of one call: their cu fits LDS (32 KB)
constexpr int ONE_ROWS = SCAN_THREADS;          // one-workgroup form: a row per thread,
constexpr int ONE_TOKENS = 4 * SCAN_THREADS;    // and a few tokens per thread
constexpr int MAX_GRID = 1024;                  // workgroups that scan for themselves

// prefix sums over rows; need and back stay below R * max_pages < 2^31
struct Sums {
  long long add;
  uint32_t need, back;
};

__device__ __forceinline__ long long shfl_up_ll(long long v, int o) { return __shfl_up(v, o, 64); }

// inclusive sums over the workgroup's threads of three values, carried in `carry`
__device__ __forceinline__ Sums block_scan(Sums v, Sums &carry, Sums *s_wave) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const Sums u = {shfl_up_ll(v.add, o), (uint32_t)__shfl_up((int)v.need, o, 64),
                    (uint32_t)__shfl_up((int)v.back, o, 64)};
    if (lane >= o) {
      v.add += u.add;
      v.need += u.need;
      v.back += u.back;
    }
  }
  if (lane == 63) s_wave[wave] = v;
  __syncthreads();
  Sums before = carry, total = carry;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    const Sums u = s_wave[w];
    if (w < wave) {
      before.add += u.add;
      before.need += u.need;
      before.back += u.back;
    }
    total.add += u.add;
    total.need += u.need;
    total.back += u.back;
  }
  __syncthreads();
  carry = total;
  return {v.add + before.add, v.need + before.need, v.back + before.back};
}

__device__ __forceinline__ int wrapped(int at, int num) { return at >= num ? at - num : at; }

// slot and position of packed token j, which is in row r (cu[r] <= j < cu[r+1]) or in none
__device__ __forceinline__ void fill_token(const PagesArgs &a, int j, int r, bool in, int begin,
                                           const PageRow &row) {
  int slot = -1, pos = -1;
  if (in) {
    pos = row.old + (j - begin);
    if (row.ok) {
      const int P = 1 << a.page_shift;
      const int held = (int)(((int64_t)row.old + P - 1) >> a.page_shift);
      const int pg = pos >> a.page_shift;
      const int id = pg < held ? a.table[(size_t)r * a.max_pages + pg]
                               : a.ring[wrapped(row.first + (pg - held), a.num_pages)];
      if (id >= 0 && id < a.num_pages) slot = (id << a.page_shift) + (pos & (P - 1));
    }
  }
  a.slots[j] = slot;
  a.positions[j] = pos;
}

// pages i0, i0 + step, ... of the row's new ones into its table, or of its released ones into the ring
__device__ __forceinline__ void fill_pages(const PagesArgs &a, int r, const PageRow &row, int i0,
                                           int step) {
  int32_t *tab = a.table + (size_t)r * a.max_pages;
  if (row.pages > 0) {
    const int held = (int)(((int64_t)row.old + (1 << a.page_shift) - 1) >> a.page_shift);
    for (int i = i0; i < row.pages; i += step)
      tab[held + i] = a.ring[wrapped(row.first + i, a.num_pages)];
  } else {
    for (int i = i0; i < -1 - row.pages; i += step)
      a.ring[wrapped(row.first + i, a.num_pages)] = tab[i];
  }
}

// rows [0, R) of cu that end at or before j: the row of token j
__device__ __forceinline__ int row_of(const int *cu, int R, int j) {
  int lo = 0, hi = R;   // smallest r with cu[r + 1] > j
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] <= j) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

}  // namespace

template <bool ONE>
__global__ __launch_bounds__(SCAN_THREADS) void pages_scan_kernel(PagesArgs a) {
  __shared__ Sums s_wave[SCAN_THREADS / 64];
  __shared__ int s_taken;
  __shared__ int s_cu[ONE ? ONE_ROWS + 1 : 1];
  __shared__ PageRow s_row[ONE ? ONE_ROWS : 1];
  const int tid = threadIdx.x;
  const int P = 1 << a.page_shift;
  const long long room = (long long)a.max_pages << a.page_shift;
  int head = a.ring_state[0], count = a.ring_state[1];
  head = head < 0 || head >= a.num_pages ? 0 : head;
  count = count < 0 ? 0 : (count > a.num_pages ? a.num_pages : count);
  const bool first = blockIdx.x == 0;   // stores what there is one of
  if (tid == 0) {
    s_taken = 0;
    if (first) a.cu[0] = 0;
    if constexpr (ONE) s_cu[0] = 0;
  }
  Sums carry = {0, 0, 0};
  __syncthreads();   // every thread has read ring_state, which ring_state_out may be
  for (int r0 = 0; r0 < a.R; r0 += (int)blockDim.x) {
    const int r = r0 + tid;
    const bool in = r < a.R;
    int len = in ? a.lens[r] : 0;
    const int add_in = in ? a.new_lens[r] : 0;
    len = len < 0 ? 0 : ((long long)len > room ? (int)room : len);
    const bool gone = add_in < 0;
    const long long add = gone ? 0 : add_in;
    const int held = (int)(((long long)len + P - 1) >> a.page_shift);
    const bool fits = len + add <= room;
    const int need = !gone && fits ? (int)((len + add + P - 1) >> a.page_shift) - held : 0;
    // a table cannot name more pages than there are (lens of another table would say so)
    const int back = gone ? (held < a.num_pages ? held : a.num_pages) : 0;
    const Sums s = block_scan({add, (uint32_t)need, (uint32_t)back}, carry, s_wave);
    const bool ok = !gone && (add == 0 || (fits && s.add <= a.max_tokens &&
                                           (need == 0 || s.need <= (uint32_t)count)));
    if (in) {
      PageRow row;
      row.old = len;
      row.pages = gone ? -1 - back : (ok ? need : 0);
      // released pages go behind the free ones, new ones come from the head (below 2^32 both; a row
      // that is ok starts at most num_pages behind the head)
      row.first = gone ? (int)(((uint32_t)head + (uint32_t)count + s.back - (uint32_t)back) %
                               (uint32_t)a.num_pages)
                       : (ok && need > 0 ? wrapped(head + (int)s.need - need, a.num_pages) : 0);
      row.ok = ok;
      if (ok && need > 0) atomicMax(&s_taken, (int)s.need);
      const int end = (int)(s.add < a.max_tokens ? s.add : a.max_tokens);
      if (first) {
        a.lens_out[r] = gone ? 0 : (ok ? (int)(len + add) : len);
        a.status[r] = gone ? FADKV_ROW_RELEASED : (ok ? FADKV_ROW_OK : FADKV_ROW_REFUSED);
        a.cu[r + 1] = end;
      }
      if constexpr (ONE) {
        s_cu[r + 1] = end;
        s_row[r] = row;
      } else {
        a.rows[r] = row;
      }
    }
  }
  __syncthreads();
  if (first && tid == 0) {
    const int taken = s_taken;
    a.ring_state_out[0] = wrapped(head + taken, a.num_pages);
    const long long left = (long long)count - taken + carry.back;
    a.ring_state_out[1] = (int)(left > a.num_pages ? a.num_pages : left);
  }
  if constexpr (ONE) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t j = (int64_t)blockIdx.x * blockDim.x + tid; j < a.max_tokens; j += step) {
      const bool in = j < s_cu[a.R];
      const int r = in ? row_of(s_cu, a.R, (int)j) : 0;
      fill_token(a, (int)j, r, in, s_cu[r], s_row[r]);
    }
    if (gridDim.x > 1) {   // a wave per row
      const int waves = (int)(gridDim.x * (blockDim.x >> 6));
      for (int r = (int)(blockIdx.x * (blockDim.x >> 6)) + (tid >> 6); r < a.R; r += waves)
        fill_pages(a, r, s_row[r], tid & 63, 64);
      return;
    }
    // a thread moves its row's few pages, a wave those of each row with many
    constexpr int FEW = 4;
    int many = 0;
    if (tid < a.R) {
      const PageRow row = s_row[tid];
      const int pages = row.pages >= 0 ? row.pages : -1 - row.pages;
      many = pages > FEW;
      if (!many) fill_pages(a, tid, row, 0, 1);
    }
    for (unsigned long long left = __ballot(many); left; left &= left - 1) {
      const int r = (tid & ~63) + __builtin_ctzll(left);
      fill_pages(a, r, s_row[r], tid & 63, 64);
    }
  }
}

// workgroups [0, token_blocks): FILL_TOKENS tokens each; the others: a row per wave
__global__ __launch_bounds__(FILL_THREADS) void pages_fill_kernel(PagesArgs a, int token_blocks) {
  __shared__ int s_cu[MAX_ROWS + 1];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= token_blocks) {
    const int r = ((int)blockIdx.x - token_blocks) * (FILL_THREADS / 64) + (tid >> 6);
    if (r < a.R) fill_pages(a, r, a.rows[r], tid & 63, 64);
    return;
  }
  for (int r = tid; r <= a.R; r += FILL_THREADS) s_cu[r] = a.cu[r];
  __syncthreads();
  const int j0 = (int)blockIdx.x * FILL_TOKENS;
#pragma unroll
  for (int k = 0; k < FILL_TOKENS / FILL_THREADS; ++k) {
    const int j = j0 + k * FILL_THREADS + tid;
    if (j >= a.max_tokens) break;
    const bool in = j < s_cu[a.R];
    const int r = in ? row_of(s_cu, a.R, j) : 0;
    PageRow row = {0, 0, 0, 0};
    if (in) row = a.rows[r];
    fill_token(a, j, r, in, s_cu[r], row);
  }
}

hipError_t launch_pages_advance(const PagesArgs &a, hipStream_t stream) {
  const bool apart = a.lens_out != a.lens && a.ring_state_out != a.ring_state;
  if (a.R <= ONE_ROWS && (a.max_tokens <= ONE_TOKENS || apart)) {
    const int64_t most = a.R > a.max_tokens ? a.R : a.max_tokens;
    int threads = most <= 64 ? 64 : (most <= 256 ? 256 : SCAN_THREADS);
    int64_t grid = 1;
    if (a.max_tokens > ONE_TOKENS) {
      threads = a.R <= FILL_THREADS ? FILL_THREADS : SCAN_THREADS;
      grid = (a.max_tokens + (int64_t)4 * threads - 1) / (4 * threads);   // four tokens a thread,
      if (grid > MAX_GRID) grid = MAX_GRID;                                // until the chip is full
    }
    hipLaunchKernelGGL(pages_scan_kernel<true>, dim3((unsigned)grid), dim3(threads), 0, stream, a);
    return hipGetLastError();
  }
  const int threads = a.R <= 64 ? 64 : (a.R <= 256 ? 256 : SCAN_THREADS);
  hipLaunchKernelGGL(pages_scan_kernel<false>, dim3(1), dim3(threads), 0, stream, a);
  const int token_blocks = (int)(((int64_t)a.max_tokens + FILL_TOKENS - 1) / FILL_TOKENS);
  const int row_blocks = (a.R + FILL_THREADS / 64 - 1) / (FILL_THREADS / 64);
  if (token_blocks + row_blocks > 0)
    hipLaunchKernelGGL(pages_fill_kernel, dim3((unsigned)(token_blocks + row_blocks)),
                       dim3(FILL_THREADS), 0, stream, a, token_blocks);
  return hipGetLastError();
}

}  // namespace fadkv
