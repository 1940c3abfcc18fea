// C ABI of the paged dense cache (declared in include/fadkv.h): argument checks on the host and
// kernel dispatch.  As in api.hip, nothing here allocates, synchronises or touches the GPU before
// every argument has been accepted.
#include "fadkv.h"

#include <math.h>

#include "dense.h"

namespace {

constexpr int64_t kMaxRows = 8192;                  // the rows' prefix sums live in LDS
constexpr int64_t kMaxTokens = int64_t(1) << 23;    // a workgroup of 256 per token: 2^31 work-items
constexpr int64_t kMaxRowHeads = int64_t(1) << 22;  // the attention grids
constexpr int64_t kMaxPromptHeads = int64_t(1) << 28;
constexpr int kMaxKvHeads = 256;
constexpr int kMaxGroup = 64;
constexpr int kMaxHeads = kMaxKvHeads * kMaxGroup;
constexpr int64_t kTwo31 = int64_t(1) << 31;
constexpr int64_t kMaxRowTokens = int64_t(1) << 30;  // positions rounded up to tiles stay below 2^31

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t esize(int dtype) { return dtype == FADKV_F32 ? 4 : 2; }

int page_shift(int32_t page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

bool known(int dtype) { return dtype == FADKV_F32 || dtype == FADKV_F16 || dtype == FADKV_BF16; }

int check_pages_shape(const fadkv_pages *p) {
  if (!p) return FADKV_ERR_ARG;
  if (!known(p->dtype)) return FADKV_ERR_DTYPE;
  if (p->d != 64 && p->d != 128) return FADKV_ERR_SHAPE;
  if (p->num_pages < 1 || page_shift(p->page_size) < 0) return FADKV_ERR_SHAPE;
  if ((int64_t)p->num_pages * p->page_size >= kTwo31) return FADKV_ERR_SHAPE;
  if (p->kv_heads < 1 || p->kv_heads > kMaxKvHeads) return FADKV_ERR_SHAPE;
  return FADKV_OK;
}

int check_pages(const fadkv_pages *p) {
  const int st = check_pages_shape(p);
  if (st != FADKV_OK) return st;
  if (!p->k || !p->v || !aligned(p->k, 16) || !aligned(p->v, 16)) return FADKV_ERR_ARG;
  return FADKV_OK;
}

int check_heads(const fadkv_pages *p, int64_t R, int32_t heads) {
  if (heads < 1 || heads % p->kv_heads != 0 || heads / p->kv_heads > kMaxGroup)
    return FADKV_ERR_SHAPE;
  if (R < 0 || R > kMaxRowHeads || R * heads > kMaxRowHeads) return FADKV_ERR_SHAPE;
  return FADKV_OK;
}

// the tables both attention calls take
int check_rows(const fadkv_pages *p, int32_t max_pages, float scale, int32_t window,
               int32_t sinks) {
  if (max_pages < 1 || (int64_t)max_pages * p->page_size > kMaxRowTokens) return FADKV_ERR_SHAPE;
  if (!isfinite(scale) || window < 0 || sinks < 0) return FADKV_ERR_ARG;
  return FADKV_OK;
}

fadkv::AttendArgs attend_args(const fadkv_pages *p, const int32_t *table, int32_t max_pages,
                              const int32_t *lens, int64_t R, const void *q, int32_t heads,
                              float scale, int32_t window, int32_t sinks, void *out) {
  fadkv::AttendArgs a{};
  a.k = p->k;
  a.v = p->v;
  a.num_pages = p->num_pages;
  a.page_shift = page_shift(p->page_size);
  a.kv_heads = p->kv_heads;
  a.group = heads / p->kv_heads;
  a.max_pages = max_pages;
  a.R = (int32_t)R;
  a.table = table;
  a.lens = lens;
  a.q = q;
  a.out = out;
  a.scale = scale;
  a.window = window ? window : INT32_MAX;
  a.sinks = window ? sinks : 0;   // without a window every token up to the query is visible
  a.splits = 1;
  return a;
}

#define FADKV_TRY(expr)        \
  do {                         \
    const int _st = (expr);    \
    if (_st != FADKV_OK) return _st; \
  } while (0)

// [queries][splits] outputs of d floats, then as many (maximum, sum) pairs
size_t attend_part_bytes(int64_t queries, int splits, int32_t d) {
  if (splits <= 1) return 0;
  const size_t parts = (size_t)queries * (size_t)splits;
  return (parts * ((size_t)d * sizeof(float) + 2 * sizeof(float)) + 255) / 256 * 256;
}

int take_parts(fadkv::AttendArgs &a, int64_t queries, int32_t d, void *workspace,
               size_t workspace_bytes) {
  const size_t need = attend_part_bytes(queries, a.splits, d);
  if (need == 0) return FADKV_OK;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return FADKV_ERR_WORKSPACE;
  a.part_o = static_cast<float *>(workspace);
  a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)queries * a.splits * d);
  return FADKV_OK;
}

// tokens that one query can see, at most, rounded out to tiles at both ends
int64_t visible_bound(int32_t max_len, int32_t window, int32_t sinks) {
  const int64_t w = (int64_t)window + sinks + 128;
  return window && w < max_len ? w : max_len;
}

int check_prompt(const fadkv_pages *p, int64_t R, int64_t n, int32_t heads) {
  FADKV_TRY(check_heads(p, R, heads));
  if (n < 0 || n > kMaxPromptHeads || n * heads > kMaxPromptHeads) return FADKV_ERR_SHAPE;
  return FADKV_OK;
}

}  // namespace

extern "C" {

int fadkv_pages_workspace_bytes(int64_t R, size_t *bytes) {
  if (!bytes) return FADKV_ERR_ARG;
  if (R < 0 || R > kMaxRows) return FADKV_ERR_SHAPE;
  *bytes = (size_t)R * sizeof(fadkv::PageRow);
  return FADKV_OK;
}

int fadkv_pages_advance(int32_t num_pages, int32_t page_size, int64_t R, int32_t max_pages,
                        const int32_t *new_lens, const int32_t *lens, int32_t *table,
                        int32_t *ring, const int32_t *ring_state, int64_t max_tokens,
                        int32_t *lens_out, int32_t *ring_state_out, int32_t *cu, int32_t *status,
                        int32_t *slots, int32_t *positions, void *workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  const int shift = page_shift(page_size);
  if (shift < 0 || num_pages < 1 || max_pages < 1 || R < 0 || R > kMaxRows || max_tokens < 0)
    return FADKV_ERR_SHAPE;
  if ((int64_t)num_pages * page_size >= kTwo31 || max_tokens >= kTwo31 ||
      (int64_t)max_pages * page_size + max_tokens >= kTwo31 || R * max_pages >= kTwo31)
    return FADKV_ERR_SHAPE;
  if (!ring || !ring_state || !ring_state_out || !cu) return FADKV_ERR_ARG;
  if (R > 0 && (!new_lens || !lens || !table || !lens_out || !status)) return FADKV_ERR_ARG;
  if (max_tokens > 0 && (!slots || !positions)) return FADKV_ERR_ARG;
  const void *all[] = {new_lens, lens, table, ring, ring_state, lens_out, ring_state_out,
                       cu, status, slots, positions};
  for (const void *p : all)
    if (!aligned(p, 4)) return FADKV_ERR_ARG;
  if (R > 0 && (!workspace || !aligned(workspace, 4) ||
                workspace_bytes < (size_t)R * sizeof(fadkv::PageRow)))
    return FADKV_ERR_WORKSPACE;
  fadkv::PagesArgs a{num_pages, shift, (int32_t)R, max_pages, (int32_t)max_tokens, new_lens, lens,
                     table, ring, ring_state, lens_out, ring_state_out, cu, status, slots,
                     positions, static_cast<fadkv::PageRow *>(workspace)};
  return fadkv::launch_pages_advance(a, stream) == hipSuccess ? FADKV_OK : FADKV_ERR_HIP;
}

int fadkv_rope_freqs(int32_t rot_dim, double base, int32_t kind, double factor, double low,
                     double high, double original_len, double *freqs, double *mscale) {
  if (rot_dim < 2 || rot_dim > 65536 || rot_dim % 2 != 0) return FADKV_ERR_SHAPE;
  if (!freqs || !mscale) return FADKV_ERR_ARG;
  if (!(base > 1.0) || !isfinite(base)) return FADKV_ERR_ARG;
  if (kind < FADKV_ROPE_PLAIN || kind > FADKV_ROPE_YARN) return FADKV_ERR_ARG;
  if (kind != FADKV_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return FADKV_ERR_ARG;
  if (kind == FADKV_ROPE_BANDS || kind == FADKV_ROPE_YARN) {
    if (!(low > 0.0) || !(high > low) || !isfinite(high)) return FADKV_ERR_ARG;
    if (!(original_len >= 1.0) || !isfinite(original_len)) return FADKV_ERR_ARG;
  }
  const double two_pi = 6.28318530717958647692;
  *mscale = kind == FADKV_ROPE_YARN && factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0;
  // YARN: the pair that turns `turns` times within original_len
  const auto pair_of = [&](double turns) {
    return rot_dim * log(original_len / (turns * two_pi)) / (2.0 * log(base));
  };
  double from = 0.0, to = 0.0;
  if (kind == FADKV_ROPE_YARN) {
    from = fmax(floor(pair_of(high)), 0.0);
    to = fmin(ceil(pair_of(low)), (double)rot_dim - 1.0);
    if (to <= from) to = from + 0.001;   // a step, not a division by zero
  }
  for (int32_t i = 0; i < rot_dim / 2; ++i) {
    const double f = pow(base, -2.0 * i / rot_dim);
    double keep = 1.0;   // share of the unscaled frequency
    if (kind == FADKV_ROPE_LINEAR) {
      keep = 0.0;
    } else if (kind == FADKV_ROPE_BANDS) {
      const double turns = original_len * f / two_pi;   // L / wavelength
      keep = fmin(fmax((turns - low) / (high - low), 0.0), 1.0);
    } else if (kind == FADKV_ROPE_YARN) {
      keep = 1.0 - fmin(fmax((i - from) / (to - from), 0.0), 1.0);
    }
    freqs[i] = keep == 1.0 ? f : keep * f + (1.0 - keep) * (f / factor);
  }
  return FADKV_OK;
}

int fadkv_norm_rope(const fadkv_qkv *in, void *q_out, const fadkv_pages *pages,
                    const int32_t *slots, void *k_rows, void *v_rows, hipStream_t stream) {
  if (!in) return FADKV_ERR_ARG;
  if (!known(in->dtype)) return FADKV_ERR_DTYPE;
  if (in->d != 64 && in->d != 128) return FADKV_ERR_SHAPE;
  if (in->n < 0 || in->n > kMaxTokens) return FADKV_ERR_SHAPE;
  if (in->heads < 1 || in->heads > kMaxHeads || in->kv_heads < 1 || in->kv_heads > kMaxKvHeads)
    return FADKV_ERR_SHAPE;
  if (in->rot_dim < 0 || in->rot_dim > in->d || in->rot_dim % 16 != 0) return FADKV_ERR_SHAPE;
  if (in->interleaved != 0 && in->interleaved != 1) return FADKV_ERR_ARG;
  if (!(in->eps >= 0.f) || !isfinite(in->eps) || !isfinite(in->mscale)) return FADKV_ERR_ARG;
  if (in->rot_dim > 0 && (!in->freqs || !aligned(in->freqs, 8))) return FADKV_ERR_ARG;
  const int64_t es = esize(in->dtype);
  const int64_t qrow = (int64_t)in->heads * in->d, krow = (int64_t)in->kv_heads * in->d;
  if (in->q_stride < qrow || in->k_stride < krow || in->v_stride < krow) return FADKV_ERR_SHAPE;
  const int64_t strides[] = {in->q_stride, in->k_stride, in->v_stride};
  for (const int64_t s : strides) {
    if ((s * es) % 16 != 0) return FADKV_ERR_ARG;
    if (s > (int64_t(1) << 36)) return FADKV_ERR_SHAPE;   // n * stride fits 64 bits
  }
  if (pages) {
    FADKV_TRY(check_pages(pages));
    if (pages->dtype != in->dtype) return FADKV_ERR_DTYPE;
    if (pages->d != in->d || pages->kv_heads != in->kv_heads) return FADKV_ERR_SHAPE;
  }
  if (in->n == 0) return FADKV_OK;
  if (pages && (!slots || !aligned(slots, 4))) return FADKV_ERR_ARG;
  if (!in->q || !in->k || !in->v || !in->positions || !q_out) return FADKV_ERR_ARG;
  const void *wide[] = {in->q, in->k, in->v, in->q_weight, in->k_weight, q_out, k_rows, v_rows};
  for (const void *p : wide)
    if (!aligned(p, 16)) return FADKV_ERR_ARG;
  if (!aligned(in->positions, 4)) return FADKV_ERR_ARG;
  if (q_out == in->q && in->q_stride != qrow) return FADKV_ERR_ARG;
  fadkv::NormRopeArgs a{};
  a.in = *in;
  a.q_out = q_out;
  a.k_rows = k_rows;
  a.v_rows = v_rows;
  if (pages) {
    a.k_pages = pages->k;
    a.v_pages = pages->v;
    a.slots = slots;
    a.page_shift = page_shift(pages->page_size);
    a.num_slots = pages->num_pages * pages->page_size;
  }
  return fadkv::launch_norm_rope(a, stream) == hipSuccess ? FADKV_OK : FADKV_ERR_HIP;
}

int fadkv_attend_paged_workspace_bytes(const fadkv_pages *pages, int64_t R, int32_t heads,
                                       int32_t max_len, size_t *bytes) {
  if (!bytes) return FADKV_ERR_ARG;
  FADKV_TRY(check_pages_shape(pages));
  FADKV_TRY(check_heads(pages, R, heads));
  if (max_len < 1) return FADKV_ERR_SHAPE;
  *bytes = attend_part_bytes(
      R * heads,
      fadkv::attend_paged_most_splits(pages->dtype, R, pages->kv_heads, heads / pages->kv_heads,
                                      max_len),
      pages->d);
  return FADKV_OK;
}

int fadkv_attend_paged(const fadkv_pages *pages, const int32_t *table, int32_t max_pages,
                       const int32_t *lens, int64_t R, const void *q, int32_t heads, float scale,
                       int32_t window, int32_t sinks, int32_t max_len, void *out,
                       void *workspace, size_t workspace_bytes, hipStream_t stream) {
  FADKV_TRY(check_pages(pages));
  FADKV_TRY(check_heads(pages, R, heads));
  FADKV_TRY(check_rows(pages, max_pages, scale, window, sinks));
  if (max_len < 1 || (int64_t)max_len > (int64_t)max_pages * pages->page_size)
    return FADKV_ERR_SHAPE;
  if (R == 0) return FADKV_OK;
  if (!table || !lens || !q || !out || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(q, 16) || !aligned(out, 16) || q == out)
    return FADKV_ERR_ARG;
  fadkv::AttendArgs a =
      attend_args(pages, table, max_pages, lens, R, q, heads, scale, window, sinks, out);
  const int64_t visible = visible_bound(max_len, window, sinks);
  a.splits = fadkv::attend_paged_splits(pages->dtype, R, a.kv_heads, a.group, visible);
  FADKV_TRY(take_parts(a, R * heads, pages->d, workspace, workspace_bytes));
  return fadkv::launch_attend_paged(pages->dtype, pages->d, a,
                                    fadkv::attend_paged_waves(pages->dtype, visible),
                                    stream) == hipSuccess
             ? FADKV_OK : FADKV_ERR_HIP;
}

int fadkv_attend_prompt_workspace_bytes(const fadkv_pages *pages, int64_t R, int64_t n,
                                        int32_t heads, int32_t max_len, size_t *bytes) {
  if (!bytes) return FADKV_ERR_ARG;
  FADKV_TRY(check_pages_shape(pages));
  FADKV_TRY(check_prompt(pages, R, n, heads));
  if (max_len < 1) return FADKV_ERR_SHAPE;
  *bytes = attend_part_bytes(n * heads,
                             fadkv::attend_prompt_splits(pages->dtype, R, n, pages->kv_heads,
                                                         heads / pages->kv_heads, max_len),
                             pages->d);
  return FADKV_OK;
}

int fadkv_attend_prompt(const fadkv_pages *pages, const int32_t *table, int32_t max_pages,
                        const int32_t *lens, const int32_t *cu, int64_t R, const void *q,
                        int64_t n, int32_t heads, float scale, int32_t window, int32_t sinks,
                        int32_t max_len, void *out, void *workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  FADKV_TRY(check_pages(pages));
  FADKV_TRY(check_prompt(pages, R, n, heads));
  FADKV_TRY(check_rows(pages, max_pages, scale, window, sinks));
  if (max_len < 1 || (int64_t)max_len > (int64_t)max_pages * pages->page_size)
    return FADKV_ERR_SHAPE;
  if (R == 0 || n == 0) return FADKV_OK;
  if (!table || !lens || !cu || !q || !out || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(cu, 4) || !aligned(q, 16) || !aligned(out, 16) || q == out)
    return FADKV_ERR_ARG;
  fadkv::AttendArgs a =
      attend_args(pages, table, max_pages, lens, R, q, heads, scale, window, sinks, out);
  a.cu = cu;
  a.n = n;
  a.splits = fadkv::attend_prompt_splits(pages->dtype, R, n, a.kv_heads, a.group,
                                         visible_bound(max_len, window, sinks));
  FADKV_TRY(take_parts(a, n * heads, pages->d, workspace, workspace_bytes));
  return fadkv::launch_attend_prompt(pages->dtype, pages->d, a, stream) == hipSuccess
             ? FADKV_OK : FADKV_ERR_HIP;
}

}  // extern "C"
