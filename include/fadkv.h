/*
 * fadkv.h -- C ABI of the FAD-KV screening sparse coder with fixed-size dictionary
 * adaptation, for AMD Instinct MI355X (gfx950).
 *
 * The operations follow "FAD-KV: Adaptive Dictionary KV Caching for Efficient Reasoning
 * Decoding" (arXiv 2610.37921):
 *   - fadkv_encode: abstract and Figure 1 -- each key/value head vector x is screened against
 *     every atom of its dictionary (scores sigma_j = <d_j, x>), a Top-n pool of the largest
 *     |sigma| is kept, s atoms are chosen inside the pool ("GM" greedy pursuit, or "PL" the s
 *     largest scores; Tables 1-4), and coefficients come from the ridge system of Table 5,
 *     (G_SS + diag(ridge_abs + ridge_rel * G_jj)) c = D_S x.  The relative residual
 *     ||x - D_S^T c|| / ||x|| is compared with delta (Table 5: 0.50 keys, 0.70 values).
 *   - fadkv_adapt: Figure 2 -- vectors whose error exceeds delta overwrite an inactive atom
 *     with their own direction instead of growing the dictionary, so N never changes.
 *   - fadkv_reconstruct: the stored sparse code turned back into a vector (abstract).
 *
 * Conventions shared by every call
 *   - Layout.  A "dictionary set" holds num_dicts independent dictionaries; dictionary t of a
 *     model is 2*layer + 0 for keys and 2*layer + 1 for values (delta is chosen by parity).
 *     atoms are row-major [num_dicts][N][d]; vectors X are [num_dicts][M][d] with the rows of
 *     each dictionary in (head, sequence, token) order -- that order is the commit order of
 *     fadkv_adapt.  Codes are [num_dicts][M][s] (idx int32, coef float) plus relerr float and
 *     flags uint8 per vector.  All these are DEVICE pointers, caller-owned; the library keeps
 *     no pointer after a call returns.
 *   - dtypes.  atoms and X share one storage dtype: FADKV_F32, FADKV_F16 or FADKV_BF16.
 *     Scores multiply in that dtype and accumulate in fp32; everything after the screening
 *     (pool scores, Cholesky, residual) is fp32; new atoms are normalised in fp64 and rounded
 *     to the storage dtype (round to nearest even).
 *   - Limits.  d in {64, 128}; 1 <= N <= 65535; 1 <= s <= n <= min(N, 512); s <= 32;
 *     1 <= num_dicts; 0 <= M and num_dicts * M < 2^31 (every accepted size runs: kernels whose
 *     grid grows with the number of vectors are launched in chunks).  atoms, X and X_hat must be 16-byte
 *     aligned, the other arrays 4-byte aligned (flags: any alignment).
 *   - Streams.  Every call only enqueues work on `stream` (0 = the null stream) and never
 *     synchronises.  On one stream, encode of step t+1 sees adapt of step t.  Calls are
 *     capturable into HIP graphs (no memset or allocation is enqueued).
 *   - Memory.  The calls allocate nothing.  Scratch space is the caller's `workspace`, sized
 *     by fadkv_workspace_bytes; one workspace may be reused by consecutive calls on one stream.
 *   - Errors.  Arguments are checked on the host before anything is enqueued; a bad argument
 *     returns a negative fadkv_status and launches nothing.  A failed launch returns
 *     FADKV_ERR_HIP.  Per-vector outcomes (trigger, replacement, exhaustion, non-finite
 *     input) are reported in flags, never as a status.
 *   - Threads.  Calls on disjoint buffers may run concurrently from several host threads.
 */
#ifndef FADKV_H
#define FADKV_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FADKV_ABI_VERSION 1

typedef enum {
  FADKV_OK = 0,
  FADKV_ERR_ARG = -1,       /* null or misaligned pointer, negative count, bad parameter */
  FADKV_ERR_DTYPE = -2,     /* unsupported dtype code */
  FADKV_ERR_SHAPE = -3,     /* d, N, n, s or M outside the limits above */
  FADKV_ERR_WORKSPACE = -4, /* workspace null or smaller than fadkv_workspace_bytes */
  FADKV_ERR_HIP = -5,       /* a HIP runtime call or kernel launch failed */
  FADKV_ERR_SCRATCH = -6    /* fadkv_encode_noalloc: the call needs more than its static
                               scratch (FADKV_NOALLOC_SCRATCH_BYTES) */
} fadkv_status;

typedef enum { FADKV_F32 = 0, FADKV_F16 = 1, FADKV_BF16 = 2 } fadkv_dtype;

/* Support rule inside the pool (Tables 1-4 name both; the pages do not define them):
 * GM = s greedy steps, each taking the pool atom of largest |sigma_j - sum_m G_jm c_m|
 *      (ties to the lowest atom index) and re-solving the ridge system;
 * PL = the s pool atoms of largest |sigma| (ties to the lowest index), one ridge solve. */
typedef enum { FADKV_SELECT_GM = 0, FADKV_SELECT_PL = 1 } fadkv_select;

/* flags byte per vector */
#define FADKV_FLAG_TRIGGER 0x01u   /* relative error > delta                          */
#define FADKV_FLAG_REPLACED 0x02u  /* adapt wrote this vector's direction into an atom */
#define FADKV_FLAG_EXHAUSTED 0x04u /* triggered but no inactive atom was left          */
#define FADKV_FLAG_NONFINITE 0x08u /* input held NaN/Inf: empty code, relerr = NaN     */

typedef struct {
  int32_t num_dicts; /* independent dictionaries in the set                       */
  int32_t N;         /* atoms per dictionary (fixed for the life of the set)      */
  int32_t d;         /* head_dim                                                   */
  int32_t dtype;     /* fadkv_dtype of atoms (and of X)                            */
  void *atoms;       /* device [num_dicts][N][d]; only fadkv_adapt writes it       */
  uint32_t *usage;   /* device [num_dicts][N]; committed codes per atom; only
                        fadkv_adapt writes it (start from zeros)                   */
} fadkv_dict;

typedef struct {
  int32_t n;         /* candidate-pool size (Table 5: 256, or 512 for 8B models)   */
  int32_t s;         /* sparsity (Table 5: 8, or 16 for 8B models)                  */
  float ridge_abs;   /* Table 5: 1e-4                                              */
  float ridge_rel;   /* Table 5: 0.20                                              */
  float delta_key;   /* Table 5: 0.50, used by even dictionaries                    */
  float delta_value; /* Table 5: 0.70, used by odd dictionaries                     */
  uint32_t tau_c;    /* atom inactive iff usage < tau_c (and unselected this step);
                        1 = never referenced by a committed code                    */
  int32_t select;    /* fadkv_select                                               */
} fadkv_params;

typedef struct {
  int32_t *idx;   /* device [num_dicts][M][s]: atom indices in selection order, -1 = empty */
  float *coef;    /* device [num_dicts][M][s]: coefficients, 0 for empty slots             */
  float *relerr;  /* device [num_dicts][M]: ||x - x_hat|| / ||x|| (0 for x = 0)            */
  uint8_t *flags; /* device [num_dicts][M]: FADKV_FLAG_* bits                              */
} fadkv_codes;

/* Bytes of device workspace that fadkv_encode and fadkv_adapt need for M vectors per
 * dictionary (the larger of the two; one buffer serves both).  Writes *bytes and returns
 * FADKV_OK, or a negative status if the shapes are outside the limits. */
int fadkv_workspace_bytes(const fadkv_dict *dict, const fadkv_params *params, int64_t M,
                          size_t *bytes);

/* Encode M vectors per dictionary (abstract; Figure 1; Table 5).
 *   X: device [num_dicts][M][d] in dict->dtype.
 *   out: codes written for every vector; flags get TRIGGER or NONFINITE only.
 * A vector of zeros gets the empty code and relerr 0.  The dictionary is read only. */
int fadkv_encode(const fadkv_dict *dict, const fadkv_params *params, const void *X, int64_t M,
                 const fadkv_codes *out, void *workspace, size_t workspace_bytes,
                 hipStream_t stream);

/* fadkv_encode for callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation): the same kernels and the same
 * results as fadkv_encode, with the candidate pools kept in a static device array of
 * FADKV_NOALLOC_SCRATCH_BYTES instead of a caller workspace.  Each GPU the library runs on
 * holds its own copy of that array until the process ends; the call uses the copy of the
 * current device (make the device of `stream` current before calling).  It allocates
 * nothing, enqueues no memset and never synchronises.
 *   Limit: the call needs fadkv_workspace_bytes(dict, params, M) <= FADKV_NOALLOC_SCRATCH_BYTES
 *   (about num_dicts * M * (6 n + 1) bytes; e.g. 56 x 256 vectors at n = 256, or 64 x 512 at
 *   n = 512); larger calls return FADKV_ERR_SCRATCH and launch nothing.
 *   Concurrency: every call on one GPU shares that GPU's array, so calls that overlap on one
 *   GPU (two streams, two host threads) race; serialise them (one stream) or use fadkv_encode
 *   with separate workspaces.  The array keeps the last call's contents; nothing in it needs
 *   to start at zero. */
#define FADKV_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
int fadkv_encode_noalloc(const fadkv_dict *dict, const fadkv_params *params, const void *X,
                         int64_t M, const fadkv_codes *out, hipStream_t stream);

/* The two stages of fadkv_encode, for callers that want the candidate pool itself (e.g. to
 * measure how much of a full pursuit's support it recalls, Figure 1b) or to time each stage.
 *
 * fadkv_screen -- abstract and Figure 1: scores sigma_j = <d_j, x> of every atom and the pool
 * of the n largest |sigma| (ties to the lowest index).
 *   pool_idx:   device uint16 [num_dicts][M][n], the pool's atom indices (unordered set);
 *   pool_score: device float  [num_dicts][M][n], sigma of each pool atom (fp32 accumulation);
 *   vstatus:    device uint8  [num_dicts][M], 0 = encoded, 1 = zero vector, 2 = non-finite
 *               input (pool rows of status 1 and 2 are left unwritten).
 * Needs no workspace. */
int fadkv_screen(const fadkv_dict *dict, const fadkv_params *params, const void *X, int64_t M,
                 uint16_t *pool_idx, float *pool_score, uint8_t *vstatus, hipStream_t stream);

/* fadkv_select_support -- Tables 1-5: the s-atom support inside each pool (GM or PL), the
 * ridge coefficients and the relative residual against delta, from fadkv_screen's outputs
 * (same dict, params, X and M).  Writes `out` exactly as fadkv_encode does. */
int fadkv_select_support(const fadkv_dict *dict, const fadkv_params *params, const void *X,
                         int64_t M, const uint16_t *pool_idx, const float *pool_score,
                         const uint8_t *vstatus, const fadkv_codes *out, hipStream_t stream);

/* Full-dictionary greedy yardstick: the "full-OMP atoms" Figure 1b compares the screened pool
 * against, and the Cost 1.00 reference of Table 4.  The same greedy steps as GM (largest
 * |rho_j| = |<d_j, x - D_S^T c>|, ties to the lowest index, chosen atoms excluded, the ridge
 * system of Table 5 re-solved at every step) with every atom of the dictionary a candidate
 * instead of the Top-n pool; params->n and params->select are not used.  Writes `out` as
 * fadkv_encode does (same zero and non-finite handling, same trigger against delta).
 * Launches 1 + 2 s kernels on `stream`.  workspace: fadkv_omp_workspace_bytes(), 256-byte
 * aligned, owned by the caller; X: device [num_dicts][M][d], 16-byte aligned. */
int fadkv_omp_workspace_bytes(const fadkv_dict *dict, const fadkv_params *params, int64_t M,
                              size_t *bytes);
int fadkv_encode_omp(const fadkv_dict *dict, const fadkv_params *params, const void *X,
                     int64_t M, const fadkv_codes *out, void *workspace, size_t workspace_bytes,
                     hipStream_t stream);

/* Commit one step's codes and apply fixed-size adaptation (Figure 2), per dictionary:
 *   1. usage[j] += 1 for every atom of every non-triggering code;
 *   2. candidates = atoms with usage < tau_c that no code of this step selected, ordered by
 *      (usage, atom index);
 *   3. the k-th triggering row (row order) takes the k-th candidate j: atom j becomes
 *      x/||x|| rounded to the storage dtype, usage[j] = 1, and the row's code becomes the
 *      single atom j with coefficient <d_j, x> / ((1 + ridge_rel) ||d_j||^2 + ridge_abs)
 *      (relerr recomputed, flag REPLACED);
 *   4. triggering rows beyond the candidates keep their code, commit its usage and get flag
 *      EXHAUSTED.
 * X and codes must be those of the fadkv_encode call of this step (codes is updated in
 * place).  replaced: device [num_dicts][M] int32, the overwritten atom per row or -1.
 * atoms and usage are updated in place; N never changes. */
int fadkv_adapt(const fadkv_dict *dict, const fadkv_params *params, const void *X, int64_t M,
                const fadkv_codes *codes, int32_t *replaced, void *workspace,
                size_t workspace_bytes, hipStream_t stream);

/* Append-only growth: the contrast the abstract draws (an adaptive dictionary that only ever
 * appends keeps growing during generation; FAD-KV, abstract and Fig. 3a), offered to measure it.  Same as fadkv_adapt except where a
 * triggering row's new atom goes: dictionary t uses slots [0, n_atoms[t]) of its capacity N
 * (dict->N; unused slots must hold zeros: they score 0 and are never selected), and its k-th
 * triggering row (row order) writes round(x/||x||) to slot n_atoms[t] + k while slots remain,
 * is re-coded onto it (flag REPLACED, replaced[m] = the slot) and leaves every existing atom
 * untouched; rows past the capacity keep their code, commit its usage and get flag EXHAUSTED.
 * n_atoms: device int32 [num_dicts], read and advanced in place (values clamped to [0, N]).
 * Non-triggering rows commit usage exactly as in fadkv_adapt; tau_c is not used. */
int fadkv_adapt_append(const fadkv_dict *dict, const fadkv_params *params, const void *X,
                       int64_t M, const fadkv_codes *codes, int32_t *replaced, int32_t *n_atoms,
                       void *workspace, size_t workspace_bytes, hipStream_t stream);

/* x_hat[t][m] = sum over non-empty slots k of coef[t][m][k] * atoms[t][idx[t][m][k]],
 * written as out_dtype (fp32 accumulation; 16-bit outputs rounded to nearest even).
 * idx entries must be -1 or in [0, N). */
int fadkv_reconstruct(const fadkv_dict *dict, const int32_t *idx, const float *coef, int32_t s,
                      int64_t M, void *X_hat, int32_t out_dtype, hipStream_t stream);

/* ---- decode attention over the codes ------------------------------------------------------
 * The consumer of the encoder's output.  The abstract stores every token's key and value as a
 * sparse combination of atoms, so a decode query meets the cached keys through the atoms:
 * <q, k_t> = sum_k cK[t][k] <q, d^K_{iK[t][k]}> needs q . D_K^T once per query and s gathers
 * per token, and the weighted values sum to w . D_V with w the softmax weights scattered onto
 * the atoms.  The pages give no formula for this step; the definition taken is standard scaled
 * softmax attention over the rebuilt tokens:
 *   out[r][g] = sum_{t < len[r]} p_t v_t,  p = softmax_t(scale * <q[r][g], k_t>),
 *   k_t = sum_k cK[r][t][k] d^K_{iK[r][t][k]}, v_t = sum_k cV[r][t][k] d^V_{iV[r][t][k]},
 * and out[r][g] = 0 for a row without tokens.
 *
 * Layer `layer` takes its keys from dictionary 2*layer of `dict` and its values from 2*layer+1
 * (0 <= layer, 2*layer + 1 < num_dicts).  Rows r < R are (KV head, sequence) pairs:
 *   k_idx, v_idx  device int32 [R][T][s]  atom per slot; -1 (or anything outside [0, N)) = empty
 *   k_coef, v_coef device fp32 [R][T][s]
 *   lens          device int32 [R]        cached tokens of the row (clamped to [0, T])
 *   q             device [R][G][d] in the dictionary dtype, 16-byte aligned; G query heads
 *                 share row r's keys and values (1 <= G <= 64)
 *   out           device fp32 [R][G][d], overwritten
 *   scale         finite (e.g. 1/sqrt(d))
 * 1 <= s <= 32, N <= 16384, 0 <= R <= 2^22, T >= 0, R*G <= 2^24 (the kernels' grids).
 * Workspace: at least fadkv_attend_workspace_bytes() bytes, 256-byte aligned, caller-owned (it
 * holds q . D_K^T, then the atom weights, fp32 [R*G][N], and partial outputs per range of 128
 * atoms, fp32 [ceil(N/128)][R*G][d]).  Checked synchronously; nothing is launched on error.
 * fp32 throughout after the 16-bit products.  Determinism: for N <= 13311 the value weights
 * are accumulated exactly as 64-bit fixed point, so out is bitwise reproducible; for larger N
 * they are accumulated with fp32 LDS atomics, whose order varies, so the last bits of out may
 * differ between runs. */
int fadkv_attend_workspace_bytes(const fadkv_dict *dict, int64_t R, int32_t G, size_t *bytes);
int fadkv_attend(const fadkv_dict *dict, int32_t layer, int32_t s, const int32_t *k_idx,
                 const float *k_coef, const int32_t *v_idx, const float *v_coef,
                 const int32_t *lens, int64_t R, int32_t T, const void *q, int32_t G,
                 float scale, float *out, void *workspace, size_t workspace_bytes,
                 hipStream_t stream);

/* ---- the dense cache beside the codes -----------------------------------------------------
 * Tokens that are not coded (a prompt while it is prefilled, tokens waiting for the encoder)
 * keep their keys and values in pages: blocks of page_size tokens, handed out to the rows
 * (requests) of a batch as they grow.  Four calls work on them, in the order of a decode step:
 * fadkv_pages_advance (lengths -> block table, slots, positions), fadkv_norm_rope (heads of a
 * projection -> normed, rotated queries; keys and values into the pages and the encoder's rows),
 * fadkv_attend_paged (one new token per row) or fadkv_attend_prompt (many).  They follow the
 * conventions at the top of this file (streams, memory, errors); make the device that holds the
 * buffers current before calling. */

/* One layer's pages.  Token slot t = page * page_size + offset of KV head h is the d elements at
 * k[page][h][offset] (and v). */
typedef struct {
  int32_t num_pages; /* num_pages * page_size < 2^31 */
  int32_t page_size; /* 16, 32, 64, 128 or 256 tokens */
  int32_t kv_heads;  /* 1 .. 256 */
  int32_t d;         /* 64 or 128 */
  int32_t dtype;     /* fadkv_dtype of keys, values and queries */
  void *k;           /* device [num_pages][kv_heads][page_size][d], 16-byte aligned */
  void *v;           /* as k */
} fadkv_pages;

/* row status of fadkv_pages_advance */
#define FADKV_ROW_OK 0
#define FADKV_ROW_REFUSED 1  /* its new tokens did not fit: nothing of the row changed */
#define FADKV_ROW_RELEASED 2 /* ended: its pages are free from the next call on */

/* One step of a paged cache's bookkeeping, on the GPU, from the number of tokens each row adds.
 * Row r held lens[r] tokens in the pages table[r][0 .. ceil(lens[r] / page_size)).
 *   new_lens[r] > 0: its new tokens go behind them, on pages taken from the free ring in row order;
 *   new_lens[r] = 0: nothing changes;
 *   new_lens[r] < 0: the row has ended: its pages go to the ring's tail in row and page order,
 *     to be taken from the next call on, and its length becomes 0.
 * A row is refused (its length and pages stay as they were) if the pages that it and the rows
 * before it need are more than are free, if it would outgrow max_pages, or if its tokens end
 * past max_tokens.  The pages that refused rows need count for the rows behind them too, except
 * those of rows that outgrow max_pages.
 *   new_lens, lens  device int32 [R]; lens is taken as clamped to [0, max_pages * page_size]
 *   table           device int32 [R][max_pages]: entries of new pages are written, no others
 *   ring            device int32 [num_pages]: free page ids in entries ring_state[0],
 *                   ring_state[0] + 1, ... (mod num_pages), ring_state[1] of them
 *   lens_out [R], ring_state_out [2]  the new lengths and state (may be lens and ring_state)
 *   cu              device int32 [R+1]: row r's new tokens are tokens cu[r] .. cu[r+1] - 1 of the
 *                   packed batch (prefix sums of max(new_lens, 0), refused rows included, at
 *                   most max_tokens)
 *   status          device int32 [R]: FADKV_ROW_*
 *   slots, positions  device int32 [max_tokens]: every new token's slot (-1 in a refused row) and
 *                   its position in the row; both -1 behind the last new token (a padded batch)
 * Every page belongs to one row at a time (pages that several rows read, as a common prefix, are the
 * caller's to hand out and take back).  The arrays are distinct except as said.  0 <= R <= 8192, num_pages * page_size < 2^31, 1 <=
 * max_pages, max_pages * page_size + max_tokens < 2^31, R * max_pages < 2^31.
 * workspace: fadkv_pages_workspace_bytes(R), 4-byte aligned. */
int fadkv_pages_workspace_bytes(int64_t R, size_t *bytes);
int fadkv_pages_advance(int32_t num_pages, int32_t page_size, int64_t R, int32_t max_pages,
                        const int32_t *new_lens, const int32_t *lens, int32_t *table,
                        int32_t *ring, const int32_t *ring_state, int64_t max_tokens,
                        int32_t *lens_out, int32_t *ring_state_out, int32_t *cu, int32_t *status,
                        int32_t *slots, int32_t *positions, void *workspace,
                        size_t workspace_bytes, hipStream_t stream);

/* Frequencies of rotary positions, angle = position * freqs[i] for pair i, written to HOST
 * memory (rot_dim / 2 doubles; copy them to the device for fadkv_norm_rope).  base^(-2i/rot_dim),
 * then for long contexts
 *   FADKV_ROPE_LINEAR: divided by factor (position interpolation);
 *   FADKV_ROPE_BANDS:  by wavelength w = 2 pi / f against the original context length L: kept for
 *     w < L / high, divided by factor for w > L / low, between them a mix of both, linear in
 *     L / w (the scaling of the Llama-3.1 and 3.2 models: low 1, high 4, L 8192);
 *   FADKV_ROPE_YARN:   YaRN (arXiv 2309.00071, section 3.2): kept for pairs that turn more than
 *     high times within L, divided by factor below low turns, between them a mix of both, linear
 *     in the pair index between the two rounded outwards (low 1, high 32).
 * *mscale: what queries and keys are multiplied by: 0.1 ln(factor) + 1 for YARN with factor > 1,
 * else 1.  base > 1, factor >= 1, 0 < low < high, original_len >= 1 (the last three for the two
 * kinds that use them). */
typedef enum {
  FADKV_ROPE_PLAIN = 0,
  FADKV_ROPE_LINEAR = 1,
  FADKV_ROPE_BANDS = 2,
  FADKV_ROPE_YARN = 3
} fadkv_rope_kind;
int fadkv_rope_freqs(int32_t rot_dim, double base, int32_t kind, double factor, double low,
                     double high, double original_len, double *freqs, double *mscale);

/* The heads of n tokens, as a projection leaves them. */
typedef struct {
  int64_t n;              /* tokens, padding included, 0 .. 2^23 */
  int32_t heads;          /* query heads, 1 .. 16384 */
  int32_t kv_heads;       /* key and value heads, 1 .. 256 */
  int32_t d;              /* 64 or 128 */
  int32_t dtype;          /* fadkv_dtype */
  const void *q;          /* device [n][heads][d], tokens q_stride elements apart */
  const void *k, *v;      /* device [n][kv_heads][d], tokens k_stride, v_stride apart */
  int64_t q_stride, k_stride, v_stride; /* >= heads * d (kv_heads * d), 16-byte multiples */
  const int32_t *positions; /* device [n]; negative: a padding token, of which nothing is written */
  const void *q_weight, *k_weight; /* device [d] in dtype, or null: no norm */
  float eps;              /* >= 0 */
  const double *freqs;    /* device [rot_dim / 2], radians a position; null if rot_dim is 0 */
  int32_t rot_dim;        /* the first rot_dim elements are rotated: a multiple of 16, 0 .. d */
  int32_t interleaved;    /* pairs (2i, 2i+1) if 1, (i, i + rot_dim/2) if 0 */
  float mscale;           /* factor on the rotated part, finite */
} fadkv_qkv;

/* Norm and rotation of every query and key head, and the cache write, in one pass:
 *   y = w * x / sqrt(mean(x^2) + eps) (where a weight is given), then pair (a, b) becomes
 *   mscale * (a cos - b sin, b cos + a sin) with angle = position * freqs[i].
 *   q_out   device [n][heads][d] (may be q where q_stride = heads * d)
 *   pages, slots  null, or: token i's keys and values go to slot slots[i] (device int32 [n]; a
 *           slot outside [0, num_pages * page_size) is not written; no slot twice)
 *   k_rows, v_rows  null, or device [kv_heads][n][d]: rows in (head, token) order, the encoder's
 *           X of the layer's key and value dictionary
 * All 16-byte aligned.  The outputs must not overlap the inputs (but q_out, as said) or each
 * other.  fp32 throughout (angles are reduced in fp64, for far positions), rounded once. */
int fadkv_norm_rope(const fadkv_qkv *in, void *q_out, const fadkv_pages *pages,
                    const int32_t *slots, void *k_rows, void *v_rows, hipStream_t stream);

/* Attention of one new token per row over the pages:
 *   out[r][h] = sum_t p_t v_t, p = softmax_t(scale * <q[r][h], k_t>) over the visible tokens,
 * k_t and v_t those of KV head h / (heads / kv_heads).  Visible to a query at position i: tokens
 * t <= i with t > i - window or t < sinks (window 0: all t <= i).  The query is the row's last
 * token, i = lens[r] - 1, whose key and value are in the pages already.  A row without tokens
 * gives 0; tokens of a page id outside [0, num_pages) count as not visible.  What lies in pages
 * behind a row's length is never used, whatever it holds.
 *   table device int32 [R][max_pages]; lens device int32 [R], clamped to [0, max_pages * page_size]
 *   q, out  device [R][heads][d] in pages->dtype, 16-byte aligned, distinct
 *   max_len an upper bound of lens that sizes the split over the length (any larger length is
 *           still right, only slower); 1 .. max_pages * page_size
 * heads a multiple of kv_heads, heads / kv_heads <= 64, R * heads <= 2^22, max_pages * page_size
 * <= 2^30, window >= 0, sinks >= 0, scale finite.  Scores and sums are fp32; the weights p are rounded to dtype for the
 * product with v.  Results do not depend on the run (no atomics).  workspace:
 * fadkv_attend_paged_workspace_bytes() bytes (0 where no split is needed), 256-byte aligned. */
int fadkv_attend_paged_workspace_bytes(const fadkv_pages *pages, int64_t R, int32_t heads,
                                       int32_t max_len, size_t *bytes);
int fadkv_attend_paged(const fadkv_pages *pages, const int32_t *table, int32_t max_pages,
                       const int32_t *lens, int64_t R, const void *q, int32_t heads, float scale,
                       int32_t window, int32_t sinks, int32_t max_len, void *out,
                       void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The same for many new tokens per row, packed: tokens cu[r] .. cu[r+1] - 1 of q are the last
 * ones of row r's lens[r] tokens, each attends causally (its visible tokens as above, by its own
 * position); a query whose position would be negative gives 0.
 *   cu device int32 [R+1], non-decreasing, cu[0] >= 0, taken as clamped to [0, n]
 *   q, out device [n][heads][d]; rows of out that belong to no token of a row stay as they were
 * n * heads <= 2^28; the other limits and max_len as above.  What a query does not see never
 * reaches its output, infinities and NaN among other queries' tokens included (a block of queries
 * that meets such a value is computed column by column, many times slower).
 * workspace: fadkv_attend_prompt_workspace_bytes() bytes (0 where no split is needed: there are
 * enough queries to fill the chip), 256-byte aligned. */
int fadkv_attend_prompt_workspace_bytes(const fadkv_pages *pages, int64_t R, int64_t n,
                                        int32_t heads, int32_t max_len, size_t *bytes);
int fadkv_attend_prompt(const fadkv_pages *pages, const int32_t *table, int32_t max_pages,
                        const int32_t *lens, const int32_t *cu, int64_t R, const void *q,
                        int64_t n, int32_t heads, float scale, int32_t window, int32_t sinks,
                        int32_t max_len, void *out, void *workspace, size_t workspace_bytes,
                        hipStream_t stream);

/* Static, NUL-terminated description of a status code. */
const char *fadkv_status_string(int status);

/* FADKV_ABI_VERSION of the built library. */
int fadkv_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FADKV_H */
