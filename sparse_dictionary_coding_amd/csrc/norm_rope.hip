// Norm and rotation of query and key heads, and the cache write, in one pass.
//
//   y = w * x / sqrt(mean(x^2) + eps);   (a, b) -> mscale (a cos t - b sin t, b cos t + a sin t),
//   t = position * f_i, (a, b) = elements (2i, 2i+1) or (i, i + rot/2) of the head.
//
// What bounds it: HBM.  Every value is read once and written once (keys and values twice where the
// encoder's rows are wanted); a token's other data is 8 bytes.  16384 tokens of 32 + 2 * 8 heads of 128
// in bf16 with rows: 470 MB in 79 to 85 us, 5.5 to 6.0 TB/s; 16 tokens: 5 us of latency.  So a head is one 16-byte (two in
// fp32) load per lane, d / 8 lanes a head, a wave's loads contiguous, and everything between load
// and store stays in registers: the sum of squares by DPP within the lanes of the head, the
// partner elements of the half layout by a lane exchange of the packed input.
//
// Angles take 64 bits (at position 10^6 an fp32 product is already 0.06 rad off), which is far too
// much per element; but a token's angles are the same for all its heads, so a workgroup takes one
// token and first computes cos and sin of its angles into LDS, one angle per thread, reduced to
// a part of a turn in fp64 and evaluated in fp32 (two, four and eight tokens a workgroup measured
// 3, 6 and 15 % slower at 16384 tokens).
#include "common.h"
#include "dense.h"

namespace fadkv {

namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_BATCH = 3;   // heads a lane group has in flight
// Outputs beyond the eight L2s' 32 MB are stored around the caches: whatever reads them next would
// not find the first of them there anyway, and the inputs that are still to come stay (16384
// tokens, 302 MB written: 81 us against 106 us with plain stores).
constexpr int64_t NR_STREAM = int64_t(32) << 20;

// 8 elements of a row as they are stored
template <int DT> struct Pack8 {
  uint4 w[DT == DT_F32 ? 2 : 1];
};

template <int DT> __device__ __forceinline__ void unpack(const Pack8<DT> &p, float (&x)[8]) {
  if constexpr (DT == DT_F32) {
    x[0] = __uint_as_float(p.w[0].x); x[1] = __uint_as_float(p.w[0].y);
    x[2] = __uint_as_float(p.w[0].z); x[3] = __uint_as_float(p.w[0].w);
    x[4] = __uint_as_float(p.w[1].x); x[5] = __uint_as_float(p.w[1].y);
    x[6] = __uint_as_float(p.w[1].z); x[7] = __uint_as_float(p.w[1].w);
  } else {
    const uint32_t w[4] = {p.w[0].x, p.w[0].y, p.w[0].z, p.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = lo_f<DT>(w[i]);
      x[2 * i + 1] = hi_f<DT>(w[i]);
    }
  }
}

template <int DT> __device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == DT_F16) {
    return float_to_f16_bits(a) | (float_to_f16_bits(b) << 16);
  } else {
    bf16x2_t v;   // v_cvt_pk_bf16_f32: round to nearest even
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
  }
}

template <int DT> __device__ __forceinline__ Pack8<DT> pack(const float (&x)[8]) {
  Pack8<DT> p;
  if constexpr (DT == DT_F32) {
    p.w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                        __float_as_uint(x[3]));
    p.w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                        __float_as_uint(x[7]));
  } else {
    p.w[0] = make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]),
                        pack2<DT>(x[6], x[7]));
  }
  return p;
}

// sum over the W lanes (8 or 16, aligned) of a head
template <int W> __device__ __forceinline__ float head_sum(float v) {
  v += __int_as_float(dpp_i<0xB1>(__float_as_int(v)));    // quad_perm [1,0,3,2]
  v += __int_as_float(dpp_i<0x4E>(__float_as_int(v)));    // quad_perm [2,3,0,1]
  v += __int_as_float(dpp_i<0x141>(__float_as_int(v)));   // row_half_mirror
  if constexpr (W == 16) v += __int_as_float(dpp_i<0x140>(__float_as_int(v)));   // row_mirror
  return v;
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ Pack8<DT> load8(const uint8_t *row, int lane) {
  Pack8<DT> p;
  const u32x4_t *src = reinterpret_cast<const u32x4_t *>(row) + lane * (DT == DT_F32 ? 2 : 1);
#pragma unroll
  for (int i = 0; i < (DT == DT_F32 ? 2 : 1); ++i) {
    const u32x4_t v = src[i];
    p.w[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
  return p;
}

template <int DT, bool STREAM>
__device__ __forceinline__ void store8(uint8_t *row, int lane, const Pack8<DT> &p) {
  u32x4_t *dst = reinterpret_cast<u32x4_t *>(row) + lane * (DT == DT_F32 ? 2 : 1);
#pragma unroll
  for (int i = 0; i < (DT == DT_F32 ? 2 : 1); ++i) {
    const u32x4_t v = {p.w[i].x, p.w[i].y, p.w[i].z, p.w[i].w};
    if constexpr (STREAM) __builtin_nontemporal_store(v, dst + i);
    else dst[i] = v;
  }
}

__device__ __forceinline__ uint4 shfl4(const uint4 &v, int from) {
  return make_uint4(__shfl((int)v.x, from, 64), __shfl((int)v.y, from, 64),
                    __shfl((int)v.z, from, 64), __shfl((int)v.w, from, 64));
}

}  // namespace

// One token per workgroup, its heads (queries, keys, values in that order) dealt to lane groups
template <int DT, int D, bool STREAM>
__global__ __launch_bounds__(NR_THREADS) void norm_rope_kernel(NormRopeArgs a) {
  constexpr int W = D / 8;                  // lanes a head
  constexpr int GROUPS = NR_THREADS / W;
  constexpr int ES = Elem<DT>::bytes;
  constexpr int ROWB = D * ES;
  __shared__ __attribute__((aligned(16))) float s_cos[D / 2], s_sin[D / 2];
  const fadkv_qkv &in = a.in;
  const int tid = threadIdx.x;
  const int64_t tok = blockIdx.x;
  const int pos = in.positions[tok];
  if (pos < 0) return;   // a padding token
  const int slot = a.k_pages ? a.slots[tok] : -1;
  const int half = in.rot_dim >> 1;
  if (tid < half) {
    // turns = position * f / 2 pi, reduced to [-1/2, 1/2]: 53 bits leave 2^-22 of a turn at 2^31
    double turns = (double)pos * (in.freqs[tid] * 0.15915494309189533577);
    turns -= __builtin_rint(turns);
    float sn, cs;
    sincospif((float)(turns + turns), &sn, &cs);
    s_cos[tid] = cs * in.mscale;
    s_sin[tid] = sn * in.mscale;
  }
  const int li = tid % W, grp = tid / W;
  const int lane = tid & 63;
  const bool turned = 8 * li < in.rot_dim;
  // half layout: this lane's elements pair with those of the lane half / 8 away in the head
  const int hl = half >> 3;
  const bool second = li >= hl;
  const int from = in.interleaved || !turned ? lane : (second ? lane - hl : lane + hl);
  const int partner = from - lane + li;
  Pack8<DT> qw{}, kw{}, qwp{}, kwp{};
  if (in.q_weight) {
    qw = load8<DT>(static_cast<const uint8_t *>(in.q_weight), li);
    qwp = load8<DT>(static_cast<const uint8_t *>(in.q_weight), partner);
  }
  if (in.k_weight) {
    kw = load8<DT>(static_cast<const uint8_t *>(in.k_weight), li);
    kwp = load8<DT>(static_cast<const uint8_t *>(in.k_weight), partner);
  }
  __syncthreads();

  const int heads = in.heads + 2 * in.kv_heads;
  for (int h0 = grp; h0 < heads; h0 += GROUPS * NR_BATCH) {
    Pack8<DT> x[NR_BATCH];
#pragma unroll
    for (int b = 0; b < NR_BATCH; ++b) {
      const int h = h0 + b * GROUPS;
      if (h < heads) {
        const uint8_t *src;
        if (h < in.heads)
          src = static_cast<const uint8_t *>(in.q) + (size_t)(tok * in.q_stride) * ES + (size_t)h * ROWB;
        else if (h < in.heads + in.kv_heads)
          src = static_cast<const uint8_t *>(in.k) + (size_t)(tok * in.k_stride) * ES +
                (size_t)(h - in.heads) * ROWB;
        else
          src = static_cast<const uint8_t *>(in.v) + (size_t)(tok * in.v_stride) * ES +
                (size_t)(h - in.heads - in.kv_heads) * ROWB;
        x[b] = load8<DT>(src, li);
      }
    }
#pragma unroll
    for (int b = 0; b < NR_BATCH; ++b) {
      const int h = h0 + b * GROUPS;
      if (h >= heads) break;
      const bool is_q = h < in.heads, is_v = h >= in.heads + in.kv_heads;
      Pack8<DT> out = x[b];
      if (!is_v) {
        float y[8], z[8];
        unpack<DT>(x[b], y);
        Pack8<DT> xp = x[b];
        if (!in.interleaved) {
          xp.w[0] = shfl4(x[b].w[0], from);
          if constexpr (DT == DT_F32) xp.w[1] = shfl4(x[b].w[1], from);
        }
        unpack<DT>(xp, z);
        if (is_q ? in.q_weight != nullptr : in.k_weight != nullptr) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
          ss = head_sum<W>(ss);
          // 1 / sqrt through the correctly rounded root: v_rsq alone is 1 ulp off, fp32 shows it
          const float r = 1.f / __builtin_sqrtf(ss * (1.f / D) + in.eps);
          float w[8], wp[8];
          unpack<DT>(is_q ? qw : kw, w);
          unpack<DT>(is_q ? qwp : kwp, wp);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = y[e] * r * w[e];
            z[e] = z[e] * r * wp[e];
          }
        }
        if (turned) {
          if (in.interleaved) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float c = s_cos[4 * li + e / 2], s = s_sin[4 * li + e / 2];
              const float p = y[e], q = y[e + 1];
              y[e] = p * c - q * s;
              y[e + 1] = q * c + p * s;
            }
          } else {
            const int f = 8 * (second ? li - hl : li);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float c = s_cos[f + e], s = s_sin[f + e];
              y[e] = y[e] * c + (second ? z[e] : -z[e]) * s;
            }
          }
        }
        out = pack<DT>(y);
      }
      if (is_q) {
        store8<DT, STREAM>(static_cast<uint8_t *>(a.q_out) + (size_t)(tok * in.heads + h) * ROWB, li, out);
      } else {
        const int kh = h - in.heads - (is_v ? in.kv_heads : 0);
        if (slot >= 0 && slot < a.num_slots) {
          const int page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
          uint8_t *pages = static_cast<uint8_t *>(is_v ? a.v_pages : a.k_pages);
          store8<DT, STREAM>(pages + ((((size_t)page * in.kv_heads + kh) << a.page_shift) + off) * ROWB, li, out);
        }
        uint8_t *rows = static_cast<uint8_t *>(is_v ? a.v_rows : a.k_rows);
        if (rows) store8<DT, STREAM>(rows + ((size_t)kh * in.n + tok) * ROWB, li, out);
      }
    }
  }
}

template <int DT, int D> static void norm_rope_run(const NormRopeArgs &a, hipStream_t stream) {
  const int64_t rows = a.in.heads + (int64_t)a.in.kv_heads *
      ((a.k_pages ? 2 : 0) + (a.k_rows ? 1 : 0) + (a.v_rows ? 1 : 0));
  const dim3 grid((unsigned)a.in.n);
  if (a.in.n * rows * D * Elem<DT>::bytes > NR_STREAM)
    hipLaunchKernelGGL((norm_rope_kernel<DT, D, true>), grid, dim3(NR_THREADS), 0, stream, a);
  else
    hipLaunchKernelGGL((norm_rope_kernel<DT, D, false>), grid, dim3(NR_THREADS), 0, stream, a);
}

hipError_t launch_norm_rope(const NormRopeArgs &a, hipStream_t stream) {
  if (a.in.dtype == DT_F32) {
    if (a.in.d == 64) norm_rope_run<DT_F32, 64>(a, stream);
    else norm_rope_run<DT_F32, 128>(a, stream);
  } else if (a.in.dtype == DT_F16) {
    if (a.in.d == 64) norm_rope_run<DT_F16, 64>(a, stream);
    else norm_rope_run<DT_F16, 128>(a, stream);
  } else {
    if (a.in.d == 64) norm_rope_run<DT_BF16, 64>(a, stream);
    else norm_rope_run<DT_BF16, 128>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace fadkv
