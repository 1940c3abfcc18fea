// Launchers of the paged dense cache's kernels (internal to libfadkv; the public C ABI is in
// include/fadkv.h).  Every launcher enqueues on `stream` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fadkv.h"

namespace fadkv {

// what fadkv_pages_advance knows of a row after the scan, for the part that fills the arrays
struct PageRow {
  int32_t old;     // tokens held before
  int32_t pages;   // new pages (> 0), released pages as -1 - count, or 0
  int32_t first;   // ring entry of the first of them
  int32_t ok;      // its new tokens are mapped
};

struct PagesArgs {
  int32_t num_pages, page_shift, R, max_pages, max_tokens;
  const int32_t *new_lens, *lens;
  int32_t *table, *ring;
  const int32_t *ring_state;
  int32_t *lens_out, *ring_state_out, *cu, *status, *slots, *positions;
  PageRow *rows;
};
hipError_t launch_pages_advance(const PagesArgs &a, hipStream_t stream);

struct NormRopeArgs {
  fadkv_qkv in;
  void *q_out, *k_pages, *v_pages, *k_rows, *v_rows;
  const int32_t *slots;
  int32_t page_shift;
  int32_t num_slots;   // slots of the pages (0 without pages)
};
hipError_t launch_norm_rope(const NormRopeArgs &a, hipStream_t stream);

struct AttendArgs {
  const void *k, *v;        // pages
  int32_t num_pages, page_shift, kv_heads, group, max_pages, R;
  const int32_t *table, *lens, *cu;
  const void *q;
  void *out;
  int64_t n;
  float scale;
  int32_t window, sinks;    // window: INT32_MAX where there is none
  int32_t splits;
  float *part_o;            // [queries][splits][d]: sum p v, not divided
  float2 *part_ml;          // [queries][splits]: maximum (-inf: nothing visible), sum of p
};
// parts that a row's (attend_paged) or a block of columns' (attend_prompt) tokens are split into, at
// most; `visible` bounds the tokens that one query sees
int attend_paged_splits(int dtype, int64_t R, int32_t kv_heads, int32_t group, int64_t visible);
// the largest of it over all windows of a cache of `len` tokens
int attend_paged_most_splits(int dtype, int64_t R, int32_t kv_heads, int32_t group, int64_t len);
int attend_paged_waves(int dtype, int64_t visible);   // per workgroup
int attend_prompt_splits(int dtype, int64_t R, int64_t n, int32_t kv_heads, int32_t group,
                         int64_t visible);
hipError_t launch_attend_paged(int dtype, int d, const AttendArgs &a, int waves,
                               hipStream_t stream);
hipError_t launch_attend_prompt(int dtype, int d, const AttendArgs &a, hipStream_t stream);
// joins the parts of `queries` queries (token times heads plus head) to the output
hipError_t launch_attend_join(int dtype, int d, const AttendArgs &a, int64_t queries,
                              hipStream_t stream);

}  // namespace fadkv
