// Producers of int8 activations and weights for the W8A8 GEMMs, and their inverse.
//
// One scale per row.  For a row h of fp32 values, a = max |h|:
//   s = max(fp32(a / 127), 2^-126),   q = h / s, the exact quotient to nearest even
// s is IEEE fp32 division; q comes from t = h * (1/s) rounded to an integer r, whose
// remainder d = h - r * s is exact in fp32 (a multiple of the smaller operand's
// last place, at most s or so): r is the answer where |d| < s/2, and where it is
// not (the product's rounding took the wrong side, or a tie) r is moved.  |h| / s
// never reaches 127.5, so nothing is clamped.  A row that is not finite gets a
// NaN scale and zero codes.
//
// One workgroup per row; a thread owns chunks of 8 columns (one 16-byte load, one
// 8-byte code store), which stay in registers between the row's reductions, so
// every byte is read once and written once.
#include "common.h"

namespace {

constexpr float kMinNormal = 0x1p-126f;

BS_INLINE uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o, 64)));
  return v;
}
// (each LDS array serves one reduction per kernel: no barrier follows the reads)
template <int W>
BS_INLINE uint32_t block_umax(uint32_t v, uint32_t* red) {
  v = wave_umax(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < W; ++i) v = max(v, red[i]);
  return v;
}
template <int W>
BS_INLINE double block_sum_f64(double v, double* red) {
  v = wave_sum_f64(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < W; ++i) v += red[i];
  return v;
}

BS_INLINE void unpack_bf16(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

// the row's scale from the bits of its largest |h|
struct RowScale {
  float s, inv;
  bool finite;
};
BS_INLINE RowScale row_scale(uint32_t amax_bits) {
  RowScale r;
  r.finite = amax_bits < 0x7F800000u;
  r.s = fmaxf(__uint_as_float(amax_bits) / 127.0f, kMinNormal);
  r.inv = 1.0f / r.s;
  return r;
}

// eight codes.  t + 1.5 * 2^23 rounds t to an integer, which is the sum's low byte.
BS_INLINE uint2 quant8(const float (&h)[8], float s, float inv) {
  constexpr float kMagic = 12582912.0f;
  float r[8], far = 0.0f;
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = fmaf(h[j], inv, kMagic);
    b[j] = __float_as_uint(t);
    r[j] = t - kMagic;
    far = fmaxf(far, fabsf(fmaf(-r[j], s, h[j])));
  }
  if (far + far >= s) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = fmaf(-r[j], s, h[j]), d2 = fabsf(d) + fabsf(d);
      // past the middle, or on it next to an odd code: one step towards h
      if (d2 > s || (d2 == s && (b[j] & 1u))) b[j] += d > 0.0f ? 1u : ~0u;
    }
  }
  uint2 q;
  q.x = (b[0] & 255u) | ((b[1] & 255u) << 8) | ((b[2] & 255u) << 16) | (b[3] << 24);
  q.y = (b[4] & 255u) | ((b[5] & 255u) << 8) | ((b[6] & 255u) << 16) | (b[7] << 24);
  return q;
}

// MODE 0: h = y (rows ldy chunks apart); 1: the norm of y; 2: of y + res.
// The norm: r * r is exact in fp64, the sum and the normalisation are fp64, and h
// is rounded once to fp32.  res and rout may be one buffer (in place), so neither
// is __restrict__; a thread reads its chunks before it writes them.
template <int NC, int T, int MODE>
__global__ __launch_bounds__(T) void k_row_int8(const uint4* __restrict__ y, int64_t ldy, const uint4* res,
                                                const uint4* __restrict__ gamma, float eps, float offset,
                                                uint2* __restrict__ q, float* __restrict__ scale, uint4* rout,
                                                int nch) {
  __shared__ double red_d[T / 64];
  __shared__ uint32_t red_u[T / 64];
  const size_t row = blockIdx.x;
  const int t = threadIdx.x;
  const size_t base = row * nch;
  const uint4* yr = y + row * ldy;
  uint4 yv[NC], rv[NC], gv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int ci = min(c * T + t, nch - 1);
    yv[c] = yr[ci];
    if constexpr (MODE == 2) rv[c] = res[base + ci];
    if constexpr (MODE > 0) gv[c] = gamma[ci];
  }
  float h[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    unpack_bf16(yv[c], h[c]);
    const bool live = c * T + t < nch;
    if constexpr (MODE == 2) {
      float b[8];
      unpack_bf16(rv[c], b);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = bf16x2_rne(h[c][2 * j] + b[2 * j], h[c][2 * j + 1] + b[2 * j + 1]);
        h[c][2 * j] = bf16_lo(w[j]);
        h[c][2 * j + 1] = bf16_hi(w[j]);
      }
      if (live) st_stream16(rout + base + c * T + t, make_uint4(w[0], w[1], w[2], w[3]));
    }
    if (!live)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = 0.0f;
  }
  if constexpr (MODE > 0) {
    double ss = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += static_cast<double>(h[c][j]) * static_cast<double>(h[c][j]);
    const double tot = block_sum_f64<T / 64>(ss, red_d);
    const double inv = 1.0 / sqrt(tot / (8.0 * nch) + static_cast<double>(eps));
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float g[8];
      unpack_bf16(gv[c], g);
      const bool live = c * T + t < nch;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = static_cast<float>(static_cast<double>(h[c][j]) * inv *
                                           (static_cast<double>(offset) + static_cast<double>(g[j])));
        h[c][j] = live ? v : 0.0f;
      }
    }
  }
  uint32_t amax = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(h[c][j]) & 0x7FFFFFFFu);
  amax = block_umax<T / 64>(amax, red_u);
  const RowScale rs = row_scale(amax);
  if (t == 0) scale[row] = rs.finite ? rs.s : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int idx = c * T + t;
    if (idx < nch) {
      uint2 v = quant8(h[c], rs.s, rs.inv);
      if (!rs.finite) v = make_uint2(0, 0);
      st_stream8(q + base + idx, v.x, v.y);
    }
  }
}

// SiLU form, h = fp32(g * sigmoid(g) * u), the real value rounded once.
template <int NC, int T>
__global__ __launch_bounds__(T) void k_silu_int8(const uint4* __restrict__ gu, uint2* __restrict__ q,
                                                 float* __restrict__ scale, const int* __restrict__ rows, int nch) {
  __shared__ uint32_t red_u[T / 64];
  const size_t row = blockIdx.x;
  if (rows != nullptr && static_cast<int>(row) >= *rows) return;
  const int t = threadIdx.x;
  const uint4* g_row = gu + row * 2 * nch;
  uint4 gv[NC], uv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int ci = min(c * T + t, nch - 1);
    gv[c] = ld_stream16(g_row + ci);
    uv[c] = ld_stream16(g_row + nch + ci);
  }
  float h[NC][8];
  uint32_t amax = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float g[8], u[8];
    unpack_bf16(gv[c], g);
    unpack_bf16(uv[c], u);
    const bool live = c * T + t < nch;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double gd = g[j];
      const float v = static_cast<float>(gd / (1.0 + exp(-gd)) * static_cast<double>(u[j]));
      h[c][j] = live ? v : 0.0f;
      amax = max(amax, __float_as_uint(h[c][j]) & 0x7FFFFFFFu);
    }
  }
  amax = block_umax<T / 64>(amax, red_u);
  const RowScale rs = row_scale(amax);
  if (t == 0) scale[row] = rs.finite ? rs.s : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int idx = c * T + t;
    if (idx < nch) {
      uint2 v = quant8(h[c], rs.s, rs.inv);
      if (!rs.finite) v = make_uint2(0, 0);
      st_stream8(q + row * nch + idx, v.x, v.y);
    }
  }
}

// q * s in fp32 is rounded to odd (the lowest bit set where the product is not
// exact), so that the rounding to bf16 is the only one that counts.
BS_INLINE float product_odd(float q, float s) {
  const float p = q * s, e = fmaf(q, s, -p);
  uint32_t b = __float_as_uint(p);
  if (e != 0.0f && fabsf(e) < __builtin_inff() && !(b & 1u)) b += (e < 0.0f) == (p < 0.0f) ? 1u : ~0u;
  return __uint_as_float(b);
}

constexpr int kDT = 256;
__global__ __launch_bounds__(kDT) void k_dequant_int8(const uint2* __restrict__ q, const float* __restrict__ scale,
                                                      uint4* __restrict__ out, uint32_t nch, uint32_t total) {
  const uint32_t i = blockIdx.x * kDT + threadIdx.x;
  if (i >= total) return;
  const uint2 v = q[i];
  const float s = scale[i / nch];
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int w = static_cast<int>(j < 4 ? v.x : v.y);
    f[j] = product_odd(static_cast<float>(static_cast<int8_t>(w >> (8 * (j & 3)))), s);
  }
  st_stream16(out + i, make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                                  bf16x2_rne(f[6], f[7])));
}

constexpr int kMaxRowK = 32768;   // 16 chunks of 8 per thread of 256

template <int MODE>
int launch_rows(const void* y, int64_t ldy, const void* res, const void* gamma, float eps, float offset, void* q,
                float* scale, void* rout, int M, int K, hipStream_t st) {
  const int nch = K / 8, nc = (nch + 255) / 256;
#define BS_ROW(N_)                                                                                            \
  k_row_int8<N_, 256, MODE><<<M, 256, 0, st>>>(static_cast<const uint4*>(y), ldy, static_cast<const uint4*>(res), \
                                               static_cast<const uint4*>(gamma), eps, offset, static_cast<uint2*>(q), \
                                               scale, static_cast<uint4*>(rout), nch)
  if (nc <= 1) BS_ROW(1);
  else if (nc <= 2) BS_ROW(2);
  else if (nc <= 3) BS_ROW(3);
  else if (nc <= 4) BS_ROW(4);
  else if (nc <= 8) BS_ROW(8);
  else BS_ROW(16);
#undef BS_ROW
  return bs_launch_status();
}

}  // namespace

extern "C" {

BS_API int quant_int8_per_token(const void* x, int64_t ldx, void* q, float* scale, int M, int K, bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(x && q && scale, BS_ERR_NULL);
  BS_CHECK(M >= 1 && K >= 8 && K % 8 == 0 && K <= kMaxRowK, BS_ERR_SHAPE);
  BS_CHECK(ldx >= K && ldx % 8 == 0 && bs_aligned(x, 16) && bs_aligned(q, 8) && bs_aligned(scale, 4), BS_ERR_ALIGN);
  return launch_rows<0>(x, ldx / 8, nullptr, nullptr, 0.0f, 0.0f, q, scale, nullptr, M, K,
                        static_cast<hipStream_t>(stream));
}

BS_API int add_rms_quant_int8(const void* y, const void* residual, const void* gamma, float eps, float offset, void* q,
                              float* scale, void* residual_out, int M, int K, bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(y && gamma && q && scale && (!residual || residual_out), BS_ERR_NULL);
  BS_CHECK(M >= 1 && K >= 8 && K % 8 == 0 && K <= kMaxRowK, BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(y, 16) && bs_aligned(residual, 16) && bs_aligned(gamma, 16) && bs_aligned(q, 8) &&
               bs_aligned(scale, 4) && bs_aligned(residual_out, 16),
           BS_ERR_ALIGN);
  BS_CHECK(eps >= 0.0f && offset - offset == 0.0f, BS_ERR_ARG);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (residual)
    return launch_rows<2>(y, K / 8, residual, gamma, eps, offset, q, scale, residual_out, M, K, st);
  return launch_rows<1>(y, K / 8, nullptr, gamma, eps, offset, q, scale, nullptr, M, K, st);
}

BS_API int silu_mul_quant_int8(const void* gu, void* q, float* scale, const int32_t* rows, int M, int N,
                               bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(gu && q && scale, BS_ERR_NULL);
  BS_CHECK(M >= 1 && N >= 8 && N % 8 == 0 && N <= kMaxRowK, BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(gu, 16) && bs_aligned(q, 8) && bs_aligned(scale, 4) && bs_aligned(rows, 4), BS_ERR_ALIGN);
  const int nch = N / 8, nc = (nch + 255) / 256;
  hipStream_t st = static_cast<hipStream_t>(stream);
#define BS_SILU(N_, T_)                                                                                       \
  k_silu_int8<N_, T_><<<M, T_, 0, st>>>(static_cast<const uint4*>(gu), static_cast<uint2*>(q), scale, rows, nch)
  if (nc <= 1) BS_SILU(1, 256);
  else if (nc <= 2) BS_SILU(2, 256);
  else if (nc <= 4) BS_SILU(4, 256);
  else if (nc <= 8) BS_SILU(4, 512);
  else BS_SILU(4, 1024);
#undef BS_SILU
  return bs_launch_status();
}

BS_API int dequant_int8(const void* q, const float* scale, void* out, int M, int K, bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(q && scale && out, BS_ERR_NULL);
  BS_CHECK(M >= 1 && K >= 8 && K % 8 == 0 && static_cast<uint64_t>(M) * static_cast<uint64_t>(K / 8) < (1ull << 31),
           BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(q, 8) && bs_aligned(scale, 4) && bs_aligned(out, 16), BS_ERR_ALIGN);
  const uint32_t nch = K / 8, total = static_cast<uint32_t>(M) * nch;
  k_dequant_int8<<<(total + kDT - 1) / kDT, kDT, 0, static_cast<hipStream_t>(stream)>>>(
      static_cast<const uint2*>(q), scale, static_cast<uint4*>(out), nch, total);
  return bs_launch_status();
}

}  // extern "C"
