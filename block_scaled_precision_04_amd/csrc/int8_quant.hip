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
// One workgroup per row, or one wave of four (short rows: no barriers); a thread owns
// chunks of 8 columns (one 16-byte load, one 8-byte code store), which stay in
// registers between the row's reductions, so every byte is read once and written
// once.
#include <algorithm>

#include "common.h"

namespace {

constexpr float kMinNormal = 0x1p-126f;

BS_INLINE uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o, 64)));
  return v;
}
// The row of this thread, its place in it and the row's threads: the whole workgroup,
// or (WAVE) one wave of kWaveRows.
constexpr int kMaxWaves = 16;
constexpr int kWaveRows = 4;
template <bool WAVE>
BS_INLINE int row_index() {
  return WAVE ? static_cast<int>(blockIdx.x * kWaveRows + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6))
              : static_cast<int>(blockIdx.x);
}
template <bool WAVE>
BS_INLINE int row_thread() {
  return WAVE ? threadIdx.x & 63 : threadIdx.x;
}
template <bool WAVE>
BS_INLINE int row_threads() {
  return WAVE ? 64 : blockDim.x;
}

// Reductions over the row's waves, in wave order.  (Each LDS array serves one
// reduction per kernel: no barrier follows the reads.)
template <bool WAVE>
BS_INLINE uint32_t row_umax(uint32_t v, uint32_t* red) {
  v = wave_umax(v);
  if (WAVE) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < blockDim.x >> 6; ++i) v = max(v, red[i]);
  return v;
}
template <bool WAVE>
BS_INLINE double row_sum_f64(double v, double* red) {
  v = wave_sum_f64(v);
  if (WAVE) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < blockDim.x >> 6; ++i) v += red[i];
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

// low bytes of eight words
BS_INLINE uint2 pack8(const uint32_t (&b)[8]) {
  auto two = [](uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x0C0C0400u); };   // 0, 0, hi, lo
  return make_uint2(__builtin_amdgcn_perm(two(b[2], b[3]), two(b[0], b[1]), 0x05040100u),
                    __builtin_amdgcn_perm(two(b[6], b[7]), two(b[4], b[5]), 0x05040100u));
}

// t + 1.5 * 2^23 rounds t to an integer, which is the sum's low byte.
constexpr float kMagic = 12582912.0f;
// b: the sum's bits for h; one step towards h where it lies past the middle, or on it
// next to an odd code
BS_INLINE uint32_t settle(uint32_t b, float h, float s) {
  const float d = fmaf(kMagic - __uint_as_float(b), s, h), d2 = fabsf(d) + fabsf(d);
  return d2 > s || (d2 == s && (b & 1u)) ? (d > 0.0f ? b + 1u : b - 1u) : b;
}
BS_INLINE uint32_t code_of(float h, float s, float inv) { return settle(__float_as_uint(fmaf(h, inv, kMagic)), h, s); }
BS_INLINE uint2 quant8(const float (&h)[8], float s, float inv) {
  float far = 0.0f;
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u = fmaf(h[j], inv, kMagic);
    b[j] = __float_as_uint(u);
    far = fmaxf(far, fabsf(fmaf(kMagic - u, s, h[j])));
  }
  if (far + far >= s) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = settle(b[j], h[j], s);
  }
  return pack8(b);
}

// ------------------------------------------------ rows of approximate values
// Codes and the scale are those of h = fp32(the real value), and to compute each h
// correctly rounded (in fp64) took most of the kernels' time.  So a row first holds
// h~, an fp32 value within kEps of h, and h itself is computed only where h~ does
// not decide:
//   - the row's largest |h|: of every value whose |h~| is within kMargin of the
//     largest |h~|;
//   - a code whose h~ lies within kEps of the middle between two codes (about one
//     value in 2 * 10^4);
//   - rows whose largest |h~| is not in [2^-40, 2^126): all of it (there h~ may have
//     lost its accuracy to the ends of fp32, or be a NaN).
constexpr float kEps = 0x1p-20f;
constexpr float kMargin = 0x1p-17f;

BS_INLINE uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Scale and codes of a row of h~ (zeros past its end).  exact(c, j): h of element j
// of chunk c, read again from memory, so c and j need not be constants and the rare
// paths are two short loops; odd[c]: chunk c's h~ may be further off than kEps (but
// within kMargin / 4); usable: false where no h~ of this thread is to be trusted.
template <int NC, bool WAVE, typename EXACT>
BS_INLINE void write_row(const float (&h)[NC][8], bool usable, const bool (&odd)[NC], EXACT exact, uint2* q,
                         float* scale, int nch, uint32_t* red) {
  const int t = row_thread<WAVE>(), T = row_threads<WAVE>();
  uint32_t m = usable ? 0u : 0x7FC00000u, live = 0;   // live: a bit for each element of the row
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    live |= c * T + t < nch ? 0xFFu << (8 * c) : 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, mag_bits(h[c][j]));
  }
  const uint32_t top = row_umax<WAVE>(m, red);
  const bool good = top >= 0x2B800000u && top < 0x7E800000u;   // 2^-40, 2^126
  uint32_t todo = live;
  if (good) {
    const float from = __uint_as_float(top) * (1.0f - kMargin);
    todo = 0;
    if (__uint_as_float(m) >= from)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) todo |= fabsf(h[c][j]) >= from ? 1u << (8 * c + j) : 0u;
  }
  uint32_t amax = 0;
  for (; todo != 0; todo &= todo - 1) {
    const int i = __builtin_ctz(todo);
    amax = max(amax, mag_bits(exact(i >> 3, i & 7)));
  }
  const RowScale rs = row_scale(row_umax<WAVE>(amax, red + kMaxWaves));
  if (t == 0) *scale = rs.finite ? rs.s : __uint_as_float(0x7FC00000u);
  uint2 v[NC];
  todo = good ? 0u : live;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float far = 0.0f;
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = fmaf(h[c][j], rs.inv, kMagic), d = fmaf(kMagic - u, rs.s, h[c][j]);
      b[j] = __float_as_uint(u);
      far = fmaxf(far, fmaf(fabsf(h[c][j]), kEps, fabsf(d)));
    }
    v[c] = pack8(b);
    if (far + far >= rs.s) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = fmaf(kMagic - __uint_as_float(b[j]), rs.s, h[c][j]), e = fmaf(fabsf(h[c][j]), kEps, fabsf(d));
        todo |= e + e >= rs.s ? 1u << (8 * c + j) : 0u;
      }
    }
    todo |= odd[c] ? 0xFFu << (8 * c) : 0u;
  }
  for (todo &= rs.finite ? live : 0u; todo != 0; todo &= todo - 1) {
    const int i = __builtin_ctz(todo), sh = 8 * (i & 3);
    const uint32_t code = (code_of(exact(i >> 3, i & 7), rs.s, rs.inv) & 255u) << sh;
#pragma unroll
    for (int c = 0; c < NC; ++c) {   // (no addresses of v: it stays in registers)
      const uint32_t x = (v[c].x & ~(255u << sh)) | code, y = (v[c].y & ~(255u << sh)) | code;
      v[c].x = i >> 2 == 2 * c ? x : v[c].x;
      v[c].y = i >> 2 == 2 * c + 1 ? y : v[c].y;
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int idx = c * T + t;
    if (idx >= nch) break;
    if (!rs.finite) v[c] = make_uint2(0, 0);
    st_stream8(q + idx, v[c].x, v[c].y);
  }
}

// h = y, rows ldy chunks apart: exact as it is.
template <int NC, bool WAVE>
__global__ __launch_bounds__(64 * kMaxWaves) void k_quant_int8(const uint4* __restrict__ y, int64_t ldy,
                                                               uint2* __restrict__ q, float* __restrict__ scale,
                                                               int nch, int M) {
  __shared__ uint32_t red[kMaxWaves];
  const int t = row_thread<WAVE>(), T = row_threads<WAVE>(), row = row_index<WAVE>();
  if (WAVE && row >= M) return;
  const uint4* yr = y + static_cast<int64_t>(row) * ldy;
  uint4 yv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) yv[c] = ld_stream16(yr + min(c * T + t, nch - 1));
  uint32_t amax = 0;   // (a chunk past the row's end repeats its last one)
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const uint32_t w[4] = {yv[c].x, yv[c].y, yv[c].z, yv[c].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFF0000u, (w[j] << 16) & 0x7FFF0000u));
  }
  const RowScale rs = row_scale(row_umax<WAVE>(amax, red));
  if (t == 0) scale[row] = rs.finite ? rs.s : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int idx = c * T + t;
    if (idx >= nch) break;
    float h[8];
    unpack_bf16(yv[c], h);
    const uint2 v = rs.finite ? quant8(h, rs.s, rs.inv) : make_uint2(0, 0);
    st_stream8(q + static_cast<size_t>(row) * nch + idx, v.x, v.y);
  }
}

// The norm of y (+ res): r * r is exact in fp64, the sum and the normalisation are
// fp64, and h is rounded once.  (Values approximated as in write_row need a third
// reduction of the row: 8192 x 5120 56 us with it, 54 without, 8 rows 5.3 and 4.3.)
// res and rout may be one buffer (in place), so neither is __restrict__; a thread
// reads its chunks before it writes them.
template <int NC, bool WAVE, bool RES>
__global__ __launch_bounds__(64 * kMaxWaves) void k_norm_int8(const uint4* __restrict__ y, const uint4* res,
                                                              const uint4* __restrict__ gamma, float eps, float offset,
                                                              uint2* __restrict__ q, float* __restrict__ scale,
                                                              uint4* rout, int nch, int M) {
  __shared__ double red_d[kMaxWaves];
  __shared__ uint32_t red[kMaxWaves];
  const int t = row_thread<WAVE>(), T = row_threads<WAVE>(), row = row_index<WAVE>();
  if (WAVE && row >= M) return;
  const size_t base = static_cast<size_t>(row) * nch;
  uint4 yv[NC], rv[NC], gv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int ci = min(c * T + t, nch - 1);
    yv[c] = ld_stream16(y + base + ci);
    if constexpr (RES) rv[c] = ld_stream16(res + base + ci);
    gv[c] = gamma[ci];
  }
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const bool live = c * T + t < nch;
    if constexpr (RES) {
      // bf16(y + res): the fp32 sum of two bf16 values is exact or far below half a bf16 step off
      const uint32_t a[4] = {yv[c].x, yv[c].y, yv[c].z, yv[c].w}, b[4] = {rv[c].x, rv[c].y, rv[c].z, rv[c].w};
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = bf16x2_rne(bf16_lo(a[j]) + bf16_lo(b[j]), bf16_hi(a[j]) + bf16_hi(b[j]));
      yv[c] = make_uint4(w[0], w[1], w[2], w[3]);
      if (live) st_stream16(rout + base + c * T + t, yv[c]);
    }
    if (!live) yv[c] = make_uint4(0, 0, 0, 0);
    float r[8];
    unpack_bf16(yv[c], r);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += static_cast<double>(r[j]) * static_cast<double>(r[j]);
  }
  const double inv = 1.0 / sqrt(row_sum_f64<WAVE>(ss, red_d) / (8.0 * nch) + static_cast<double>(eps));
  float h[NC][8];
  uint32_t amax = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float r[8], g[8];
    unpack_bf16(yv[c], r);
    unpack_bf16(gv[c], g);
    const bool live = c * T + t < nch;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[c][j] = static_cast<float>(static_cast<double>(r[j]) * inv *
                                   (static_cast<double>(offset) + static_cast<double>(g[j])));
      amax = max(amax, live ? mag_bits(h[c][j]) : 0u);
    }
  }
  const RowScale rs = row_scale(row_umax<WAVE>(amax, red));
  if (t == 0) scale[row] = rs.finite ? rs.s : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int idx = c * T + t;
    if (idx >= nch) break;
    const uint2 v = rs.finite ? quant8(h[c], rs.s, rs.inv) : make_uint2(0, 0);
    st_stream8(q + base + idx, v.x, v.y);
  }
}

// SiLU form.  h~ = g * (u / (1 + 2^(-g log2 e))) from the hardware exp2 and
// reciprocal (an ulp each), the rounding error of g * log2(e) added back; what
// log2(e) itself is short of costs 1.4e-8 |g| of the exponential: in all 7e-7 from g
// = -16 up (1.7e-6 down to -60; below, where 2^x may overflow, a thread's h~ is not
// used).  For g > 17 the quotient is u itself, so a subnormal u costs nothing.
BS_INLINE float silu_exact(float g, float u) {
  const double gd = g;
  return static_cast<float>(gd / (1.0 + exp(-gd)) * static_cast<double>(u));
}
BS_INLINE float silu_near(float g, float u) {
  const float p = g * 1.44269502f, lo = fmaf(g, 1.44269502f, -p);
  const float e0 = __builtin_amdgcn_exp2f(-p);
  const float e = fmaf(e0, lo * -0.693147181f, e0);
  return g * (__builtin_amdgcn_rcpf(1.0f + e) * u);
}

// (six waves a SIMD, 80 registers a lane: two workgroups of 768 threads share a CU, so
// one's loads run under the other's arithmetic: M = 4093 N = 17408 83 us, 117 alone)
template <int NC, bool WAVE>
__global__ __launch_bounds__(64 * kMaxWaves, NC > 3 ? 4 : 6) void k_silu_int8(const uint4* __restrict__ gu, uint2* __restrict__ q,
                                                                 float* __restrict__ scale,
                                                                 const int* __restrict__ rows, int nch, int M) {
  __shared__ uint32_t red[2 * kMaxWaves];
  const int t = row_thread<WAVE>(), T = row_threads<WAVE>(), row = row_index<WAVE>();
  if (rows != nullptr) M = min(M, *rows);
  if (row >= M) return;
  const uint4* g_row = gu + static_cast<size_t>(row) * 2 * nch;
  uint4 gv[NC], uv[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int ci = min(c * T + t, nch - 1);
    gv[c] = ld_stream16(g_row + ci);
    uv[c] = ld_stream16(g_row + nch + ci);
  }
  float h[NC][8], lowest = 0.0f;
  bool odd[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (c * T + t >= nch) gv[c] = uv[c] = make_uint4(0, 0, 0, 0);
    float g[8], u[8], low = 0.0f;
    unpack_bf16(gv[c], g);
    unpack_bf16(uv[c], u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[c][j] = silu_near(g[j], u[j]);
      low = fminf(low, g[j]);
    }
    odd[c] = low < -16.0f;
    lowest = fminf(lowest, low);
  }
  auto exact = [&](int c, int j) {
    const uint16_t* at = reinterpret_cast<const uint16_t*>(g_row + c * T + t) + j;
    return silu_exact(bf16_lo(at[0]), bf16_lo(at[8 * static_cast<size_t>(nch)]));
  };
  write_row<NC, WAVE>(h, lowest >= -60.0f, odd, exact, q + static_cast<size_t>(row) * nch, scale + row, nch, red);
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

constexpr int kMaxRowK = 32768;   // 4 chunks of 8 for each of 1024 threads

// Chunks a thread and threads a row.  Many rows: up to 256 chunks a wave takes a row
// alone (16384 x 2048 without residual 21.8 us, in workgroups of 128 threads 28);
// longer ones take three chunks a thread, which keeps several rows a CU (8192 x 5120
// 52 us, with one chunk 76).  Fewer rows take more threads each (8 x 5120 4.3 us with
// one chunk, 4.7 with four).
struct RowCfg {
  int nc;
  bool wave;
  dim3 grid, block;
};
RowCfg row_cfg(int M, int nch) {
  RowCfg c;
  if (M >= 1024 && nch <= 256) {
    c.nc = (nch + 63) / 64;
    c.wave = true;
    c.grid = dim3((M + kWaveRows - 1) / kWaveRows);
    c.block = dim3(64 * kWaveRows);
    return c;
  }
  c.nc = std::max((nch + 1023) / 1024, M >= 1024 ? 3 : (M >= 256 ? 2 : 1));
  c.wave = false;
  c.grid = dim3(M);
  c.block = dim3(((nch + c.nc - 1) / c.nc + 63) / 64 * 64);
  return c;
}

#define BS_ROWS_(CALL_, W_)     \
  do {                          \
    if (c.nc == 1) CALL_(1, W_); \
    else if (c.nc == 2) CALL_(2, W_); \
    else if (c.nc == 3) CALL_(3, W_); \
    else CALL_(4, W_);          \
  } while (0)
#define BS_ROWS(CALL_)              \
  do {                              \
    if (c.wave) BS_ROWS_(CALL_, true); \
    else BS_ROWS_(CALL_, false);    \
  } while (0)

}  // namespace

extern "C" {

BS_API int quant_int8_per_token(const void* x, int64_t ldx, void* q, float* scale, int M, int K, bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(x && q && scale, BS_ERR_NULL);
  BS_CHECK(M >= 1 && K >= 8 && K % 8 == 0 && K <= kMaxRowK, BS_ERR_SHAPE);
  BS_CHECK(ldx >= K && ldx % 8 == 0 && bs_aligned(x, 16) && bs_aligned(q, 8) && bs_aligned(scale, 4), BS_ERR_ALIGN);
  const int nch = K / 8;
  const RowCfg c = row_cfg(M, nch);
  hipStream_t st = static_cast<hipStream_t>(stream);
#define BS_QUANT(N_, W_) \
  k_quant_int8<N_, W_><<<c.grid, c.block, 0, st>>>(static_cast<const uint4*>(x), ldx / 8, static_cast<uint2*>(q), scale, \
                                                             nch, M)
  BS_ROWS(BS_QUANT);
#undef BS_QUANT
  return bs_launch_status();
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
  const int nch = K / 8;
  const RowCfg c = row_cfg(M, nch);
  const uint4 *yp = static_cast<const uint4*>(y), *rp = static_cast<const uint4*>(residual);
  const uint4* gp = static_cast<const uint4*>(gamma);
  uint2* qp = static_cast<uint2*>(q);
  uint4* op = static_cast<uint4*>(residual_out);
#define BS_NORM(N_, W_)                                                                                \
  do {                                                                                             \
    if (residual) k_norm_int8<N_, W_, true><<<c.grid, c.block, 0, st>>>(yp, rp, gp, eps, offset, qp, scale, op, nch, M); \
    else k_norm_int8<N_, W_, false><<<c.grid, c.block, 0, st>>>(yp, nullptr, gp, eps, offset, qp, scale, nullptr, nch, M); \
  } while (0)
  BS_ROWS(BS_NORM);
#undef BS_NORM
  return bs_launch_status();
}

BS_API int silu_mul_quant_int8(const void* gu, void* q, float* scale, const int32_t* rows, int M, int N,
                               bs_stream_t stream) {
  if (M == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(gu && q && scale, BS_ERR_NULL);
  BS_CHECK(M >= 1 && N >= 8 && N % 8 == 0 && N <= kMaxRowK, BS_ERR_SHAPE);
  BS_CHECK(bs_aligned(gu, 16) && bs_aligned(q, 8) && bs_aligned(scale, 4) && bs_aligned(rows, 4), BS_ERR_ALIGN);
  const int nch = N / 8;
  const RowCfg c = row_cfg(M, nch);
  hipStream_t st = static_cast<hipStream_t>(stream);
#define BS_SILU(N_, W_) \
  k_silu_int8<N_, W_><<<c.grid, c.block, 0, st>>>(static_cast<const uint4*>(gu), static_cast<uint2*>(q), scale, rows, nch, M)
  BS_ROWS(BS_SILU);
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
