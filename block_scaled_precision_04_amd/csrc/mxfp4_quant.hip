// MXFP4 quantisation of activations and weights, and its inverse.
//
// One e8m0 scale per 32 consecutive values of a row (the OCP microscaling
// rule): with m = max |x| over the block,
//   e = clamp(floor(log2 m) - 2, -127, 127)     (2 = exponent of e2m1's largest binade)
//   q = e2m1(x / 2^e), round to nearest even, magnitudes beyond 6 to 6
// and the scale byte is e + 127.  A block that holds an infinity or a NaN gets
// the scale byte 255 (e8m0's NaN) and zero codes: every product that reads it
// is NaN.  All steps but the SiLU product are exact: floor(log2 m) is m's
// exponent field, x * 2^-e only moves the exponent, and the hardware convert
// is the one rounding.  So the codes are the definition's, bit for bit.
//
// Bound by HBM: 2 bytes in and 17/32 out per value (SiLU form: 4 in).  A lane
// owns 8 consecutive values (one 16-byte load, one 4-byte code store), four
// lanes a block; the block maximum is two lane exchanges inside the quad, and
// no LDS or barrier is used.
#include <hip/hip_runtime.h>

#include "common.h"

namespace {

constexpr int kQT = 256;

// scale byte from the bits of the block's largest |x| (fp32; NaN > inf > finite)
BS_INLINE uint32_t e8m0_of(uint32_t amax_bits) {
  const uint32_t f = amax_bits >> 23;
  return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}
// 2^-(byte - 127) for byte <= 252, the largest that a finite block takes
BS_INLINE float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

BS_INLINE uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true)));  // lane ^ 1
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true)));  // lane ^ 2
  return v;
}

// eight fp32 values (already divided by the scale) -> eight e2m1 codes, the
// first in the low nibble
BS_INLINE uint32_t pack_fp4(const float (&t)[8]) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[0], t[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[2], t[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[4], t[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[6], t[7], 1.0f, 3);
  return w;
}

BS_INLINE void unpack_bf16(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

// Chunk i is values [8i, 8i + 8) of the [M, K] matrix in row-major order; nch
// chunks a row, `total` in all.  STRIDED: rows are ldx values apart.
template <int U, bool STRIDED>
__global__ __launch_bounds__(kQT) void k_quant_mxfp4(const uint16_t* __restrict__ x, int64_t ldx,
                                                     uint32_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                     uint32_t nch, uint32_t total) {
  const uint32_t i0 = blockIdx.x * (kQT * U) + threadIdx.x;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = min(i0 + u * kQT, total - 1);
    size_t at = static_cast<size_t>(i) * 8;
    if constexpr (STRIDED) at = static_cast<size_t>(i / nch) * ldx + static_cast<size_t>(i % nch) * 8;
    v[u] = ld_stream16(reinterpret_cast<const uint4*>(x + at));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * kQT;
    float t[8];
    unpack_bf16(v[u], t);
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(t[j]) & 0x7FFFFFFFu);
    amax = quad_max(amax);
    const uint32_t byte = e8m0_of(amax);
    const float inv = inv_scale(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] *= inv;
    const uint32_t w = byte == 255u ? 0u : pack_fp4(t);
    if (i < total) {   // total is a multiple of 4: quads are whole
      q[i] = w;
      if ((i & 3u) == 0) scale[i >> 2] = static_cast<uint8_t>(byte);
    }
  }
}

// SiLU form: h = fp32(g * sigmoid(g) * u), the real value rounded once.  Codes
// and scale are steps of h, so an approximate h is enough wherever the whole
// interval h * (1 +- 2^-20) takes one code (and the block maximum's interval
// one exponent); the hardware exp2 and reciprocal, with the rounding error of
// g * log2(e) added back, stay within 5 fp32 ulps (6e-7 < 2^-20) for
// 2^-100 <= |g| and -87 <= g < 2.35e38.  The few blocks where that does not
// decide -- about one in 10^4 of ordinary data, and those out of that range or
// near the ends of fp32 -- are computed again in fp64.  (From 2.36e38 on
// g * log2(e) overflows and the approximate h is a NaN whatever u is, a zero too,
// so a maximum that is not finite always asks for it.)
constexpr float kEps = 0x1p-20f;

template <int U>
__global__ __launch_bounds__(kQT) void k_silu_quant_mxfp4(const uint4* __restrict__ gu, uint32_t* __restrict__ q,
                                                          uint8_t* __restrict__ scale, uint32_t nch, uint32_t total,
                                                          const int* __restrict__ rows, uint32_t M) {
  if (rows != nullptr) total = min(static_cast<uint32_t>(max(*rows, 0)), M) * nch;
  const uint32_t i0 = blockIdx.x * (kQT * U) + threadIdx.x;
  if (blockIdx.x * (kQT * U) >= total) return;
  uint4 gv[U], uv[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = min(i0 + k * kQT, total - 1);
    const uint4* src = gu + static_cast<size_t>(i / nch) * (2 * nch) + i % nch;
    gv[k] = ld_stream16(src);
    uv[k] = ld_stream16(src + nch);
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = i0 + k * kQT;
    float g[8], u[8], h[8];
    unpack_bf16(gv[k], g);
    unpack_bf16(uv[k], u);
    constexpr float kL = 1.44269502162933349609375f, kLlo = 1.925963033500011e-8f;  // log2(e), high and low
    constexpr float kLn2 = 0.693147180559945f;
    bool redo = false, live = false;
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float p = g[j] * kL;
      const float lo = fmaf(g[j], kL, -p) + g[j] * kLlo;
      const float e0 = __builtin_amdgcn_exp2f(-p);
      const float e = fmaf(e0, -lo * kLn2, e0);
      h[j] = g[j] * __builtin_amdgcn_rcpf(1.0f + e) * u[j];
      amax = max(amax, __float_as_uint(h[j]) & 0x7FFFFFFFu);
      redo |= !(g[j] >= -87.0f && fabsf(g[j]) >= 0x1p-100f) && g[j] != 0.0f;
      live |= g[j] != 0.0f && u[j] != 0.0f;
    }
    amax = quad_max(amax);
    live = quad_max(live ? 1u : 0u) != 0;
    const float am = __uint_as_float(amax);
    uint32_t byte = e8m0_of(__float_as_uint(am * (1.0f - kEps)));
    redo |= e8m0_of(__float_as_uint(am * (1.0f + kEps))) != byte;
    redo |= !(am < 0x1p126f) || (live && am < 0x1p-100f);
    uint32_t w;
    {
      const float inv = inv_scale(byte);
      float a[8], b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = h[j] * (inv * (1.0f - kEps));
        b[j] = h[j] * (inv * (1.0f + kEps));
      }
      w = pack_fp4(a);
      redo |= pack_fp4(b) != w;
    }
    if (quad_max(redo ? 1u : 0u) != 0) {
      amax = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double gd = g[j];
        h[j] = static_cast<float>(gd / (1.0 + exp(-gd)) * static_cast<double>(u[j]));
        amax = max(amax, __float_as_uint(h[j]) & 0x7FFFFFFFu);
      }
      amax = quad_max(amax);
      byte = e8m0_of(amax);
      const float inv = inv_scale(byte);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] *= inv;
      w = pack_fp4(h);
    }
    if (byte == 255u) w = 0;
    if (i < total) {
      q[i] = w;
      if ((i & 3u) == 0) scale[i >> 2] = static_cast<uint8_t>(byte);
    }
  }
}

// Codes and scales back to bf16 (e2m1 times a power of two is a bf16 value;
// beyond bf16's range it becomes an infinity, and a scale byte of 255 a NaN).
template <int U>
__global__ __launch_bounds__(kQT) void k_dequant_mxfp4(const uint32_t* __restrict__ q,
                                                       const uint8_t* __restrict__ scale, uint4* __restrict__ out,
                                                       uint32_t total) {
  const uint32_t i0 = blockIdx.x * (kQT * U) + threadIdx.x;
  uint32_t w[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = min(i0 + u * kQT, total - 1);
    w[u] = q[i];
    b[u] = scale[i >> 2];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * kQT;
    // byte 0 is 2^-127, a subnormal; 255 << 23 would be an infinity
    const float s = __uint_as_float(b[u] == 255u ? 0x7FC00000u : (b[u] == 0u ? 0x00400000u : b[u] << 23));
    typedef float v2f __attribute__((ext_vector_type(2)));
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 0);
    const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 1);
    const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 2);
    const v2f e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 3);
    if (i < total)
      st_stream16(out + i, make_uint4(bf16x2_rne(a.x * s, a.y * s), bf16x2_rne(c.x * s, c.y * s),
                                      bf16x2_rne(d.x * s, d.y * s), bf16x2_rne(e.x * s, e.y * s)));
  }
}

// rows and columns whose chunk count fits the kernels' 32-bit chunk index
// (with room for the last workgroup's overhang)
bool chunks_ok(int M, int K) { return static_cast<uint64_t>(M) * static_cast<uint64_t>(K / 8) < (1ull << 31); }

}  // namespace

extern "C" {

BS_API int quant_mxfp4(const void* x, int64_t ldx, void* q, void* scale, int M, int K, bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(x && q && scale, BS_ERR_NULL);
  BS_CHECK(M >= 1 && K >= 32 && K % 32 == 0 && chunks_ok(M, K), BS_ERR_SHAPE);
  BS_CHECK(ldx >= K && ldx % 8 == 0 && bs_aligned(x, 16) && bs_aligned(q, 4), BS_ERR_ALIGN);
  const uint32_t nch = K / 8, total = static_cast<uint32_t>(M) * nch;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  uint32_t* qp = static_cast<uint32_t*>(q);
  uint8_t* sp = static_cast<uint8_t*>(scale);
#define BS_Q(U_, S_) \
  k_quant_mxfp4<U_, S_><<<(total + kQT * U_ - 1) / (kQT * U_), kQT, 0, st>>>(xp, ldx, qp, sp, nch, total)
  const bool strided = ldx != K && M > 1;
  // two chunks a thread once the grid is large (M = 512 K = 5120 3.15 us with
  // two, 3.56 with four; M = 8192 18.9, 106 MB at 5.6 TB/s; without the
  // streaming hint on the loads 20.9)
  if (total >= 1024u * kQT) {
    if (strided) BS_Q(2, true);
    else BS_Q(2, false);
  } else {
    if (strided) BS_Q(1, true);
    else BS_Q(1, false);
  }
#undef BS_Q
  return bs_launch_status();
}

BS_API int silu_mul_quant_mxfp4(const void* gu, void* q, void* scale, const int32_t* rows, int M, int N,
                                bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(gu && q && scale, BS_ERR_NULL);
  BS_CHECK(M >= 1 && N >= 32 && N % 32 == 0 && chunks_ok(M, N), BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(gu, 16) && bs_aligned(q, 4) && bs_aligned(rows, 4), BS_ERR_ALIGN);
  const uint32_t nch = N / 8, total = static_cast<uint32_t>(M) * nch;
  hipStream_t st = static_cast<hipStream_t>(stream);
#define BS_Q(U_)                                                                         \
  k_silu_quant_mxfp4<U_><<<(total + kQT * U_ - 1) / (kQT * U_), kQT, 0, st>>>(           \
      static_cast<const uint4*>(gu), static_cast<uint32_t*>(q), static_cast<uint8_t*>(scale), nch, total, rows, \
      static_cast<uint32_t>(M))
  // M = 4096 N = 17408: 60.7 us with two chunks a thread, 62.0 with one (323 MB
  // at 5.3 TB/s); M = 512 N = 5120: 5.5 and 4.9
  if (total >= 8192u * kQT) BS_Q(2);
  else BS_Q(1);
#undef BS_Q
  return bs_launch_status();
}

BS_API int dequant_mxfp4(const void* q, const void* scale, void* out, int M, int K, bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(q && scale && out, BS_ERR_NULL);
  BS_CHECK(M >= 1 && K >= 32 && K % 32 == 0 && chunks_ok(M, K), BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(q, 4) && bs_aligned(out, 16), BS_ERR_ALIGN);
  const uint32_t total = static_cast<uint32_t>(M) * (K / 8);
  hipStream_t st = static_cast<hipStream_t>(stream);
#define BS_Q(U_)                                                                  \
  k_dequant_mxfp4<U_><<<(total + kQT * U_ - 1) / (kQT * U_), kQT, 0, st>>>(       \
      static_cast<const uint32_t*>(q), static_cast<const uint8_t*>(scale), static_cast<uint4*>(out), total)
  if (total >= 1024u * kQT) BS_Q(2);
  else BS_Q(1);
#undef BS_Q
  return bs_launch_status();
}

}  // extern "C"
