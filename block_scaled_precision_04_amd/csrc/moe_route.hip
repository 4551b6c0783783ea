// Routing of tokens to experts: scores, the choice of k experts and their
// weights, and the gradient of the weights.
//
// One wave per token.  ids are discrete, and fp32 scores of different logits meet
// often enough (about one token in 10^4 has two within an ulp or two at the border
// of the choice) that their order would differ from the definition's: where the
// order of scores or of group sums is not clear in fp32, it is decided in fp64.
#include <algorithm>

#include "common.h"

namespace {

constexpr int kWaves = 4;          // tokens per workgroup
constexpr double kNanValue = -1e300;   // where a NaN stands in the order

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  const int* rows;
  int* ids;
  float* weights;
  int T, E, k, groups, keep, top, renorm;
  float scale;
};

template <bool BF16>
BS_INLINE float load_logit(const void* p, size_t i) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  else return static_cast<const float*>(p)[i];
}

// LDS accesses of one wave run in program order; this keeps the compiler from
// moving them.
BS_INLINE void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

BS_INLINE double wave_max_f64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const double u = __shfl_xor(v, o, 64);
    v = u > v ? u : v;
  }
  return v;
}

// The choice and the scores of token t in fp64: lane j's pick and its score (-1, 0
// where there is none).  Expert e = 64 * i + lane sits in register i of its lane;
// s_val: 64 * V doubles of the wave.
template <int V, bool BF16, bool SIGMOID>
BS_INLINE void route_exact(const RouteArgs& p, int t, int l, double* s_val, int& my_id, double& my_s) {
  const double ninf = -__builtin_inf();
  double x[V], sc[V], val[V];
  double mx = ninf;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 64 * i + l;
    const float f = e < p.E ? load_logit<BF16>(p.logits, static_cast<size_t>(t) * p.ld + e) : -__builtin_inff();
    x[i] = f;
    bad |= f != f || f == __builtin_inff();
    mx = x[i] > mx ? x[i] : mx;
  }
  bad = __ballot(bad) != 0;
  double total = 1.0;   // softmax: the sum of exp(x - mx)
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) sc[i] = 1.0 / (1.0 + exp(-x[i]));
  } else {
    mx = wave_max_f64(mx);
    total = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sc[i] = x[i] == ninf ? 0.0 : exp(x[i] - mx);
      total += sc[i];
    }
    total = wave_sum_f64(total);
#pragma unroll
    for (int i = 0; i < V; ++i) sc[i] = bad ? __builtin_nan("") : sc[i] / total;
  }
  // the order of experts: by logits where nothing is added to the scores
  const bool by_logit = p.bias == nullptr;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 64 * i + l;
    const double b = p.bias != nullptr && e < p.E ? p.bias[e] : 0.0;
    double v = by_logit ? x[i] : sc[i] + b;
    v = v != v ? kNanValue : v;
    val[i] = x[i] == ninf || e >= p.E ? ninf : v;
  }
  if (p.groups > 1) {
    // 64 / G2 lanes to a group (G2: groups rounded up to a power of two)
#pragma unroll
    for (int i = 0; i < V; ++i) s_val[64 * i + l] = val[i];
    wave_lds_fence();
    const int size = p.E / p.groups;
    int part = 64;
    while (part * p.groups > 64) part >>= 1;
    const int g = l / part, at = l % part;
    double a = ninf, b = ninf;   // the two largest
    if (g < p.groups)
      for (int i = at; i < size; i += part) {
        const double v = s_val[g * size + i];
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
    for (int s = 1; s < part; s <<= 1) {
      const double a2 = __shfl_xor(a, s, 64), b2 = __shfl_xor(b, s, 64);
      const double lo = a2 > a ? a : a2;
      a = a2 > a ? a2 : a;
      b = b2 > b ? b2 : b;
      b = lo > b ? lo : b;
    }
    if (by_logit && p.top == 2) {   // (a sum is one of scores)
      auto score = [&](double v) {
        if (!(v > kNanValue)) return v;
        if constexpr (SIGMOID) return 1.0 / (1.0 + exp(-v));
        else return bad ? kNanValue : exp(v - mx) / total;
      };
      a = score(a);
      b = score(b);
    }
    double v = p.top == 2 ? a + b : a;
    if (v != v) v = kNanValue;
    int before = 0;
    for (int h = 0; h < p.groups; ++h) {
      const double u = __shfl(v, h * part, 64);
      before += u > v || (u == v && h < g);
    }
    const unsigned long long kept = __ballot(g < p.groups && before < p.keep);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = min(64 * i + l, p.E - 1);
      if (!((kept >> (e / size * part)) & 1)) val[i] = ninf;
    }
  }
  my_id = -1;
  my_s = 0.0;
  for (int j = 0; j < p.k; ++j) {
    double m = ninf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = val[i] > m ? val[i] : m;
    m = wave_max_f64(m);
    if (m == ninf) break;
    int id = 1 << 30;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) id = val[i] == m ? 64 * i + l : id;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) id = min(id, __shfl_xor(id, s, 64));
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (64 * i + l == id) {
        val[i] = ninf;
        s = sc[i];
      }
    s = __shfl(s, id & 63, 64);
    if (l == j) {
      my_id = id;
      my_s = s;
    }
  }
}

// The largest of the wave's values, in all lanes: within rows of 16 by row shifts,
// then across the rows (DPP moves, no LDS round trips).
BS_INLINE float wave_fmax(float v) {
  constexpr int kNinf = static_cast<int>(0xFF800000u);
#define BS_STEP(ctrl_, rows_) \
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(kNinf, __float_as_int(v), ctrl_, rows_, 0xF, false)))
  BS_STEP(0x111, 0xF);   // row_shr:1
  BS_STEP(0x112, 0xF);   // row_shr:2
  BS_STEP(0x114, 0xF);   // row_shr:4
  BS_STEP(0x118, 0xF);   // row_shr:8
  BS_STEP(0x142, 0xA);   // row 0 -> 1, 2 -> 3
  BS_STEP(0x143, 0xC);   // rows 0-1 -> 2-3
#undef BS_STEP
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// fp32 values as unsigned numbers of the same order; 0, below all of them, is "off".
BS_INLINE uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);   // (-0 is 0)
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}
BS_INLINE float value_of(uint32_t key) {
  return __uint_as_float(key ^ (static_cast<int>(key) < 0 ? 0x80000000u : 0xFFFFFFFFu));
}
// The wave's largest key: one instruction a step.
BS_INLINE uint32_t wave_kmax(uint32_t v) {
#define BS_STEP(ctrl_, rows_, zero_) \
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), ctrl_, rows_, 0xF, zero_)))
  BS_STEP(0x111, 0xF, true);
  BS_STEP(0x112, 0xF, true);
  BS_STEP(0x114, 0xF, true);
  BS_STEP(0x118, 0xF, true);
  BS_STEP(0x142, 0xA, false);
  BS_STEP(0x143, 0xC, false);
#undef BS_STEP
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}
BS_INLINE double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// The wave's sum, in all lanes, by the same moves.
BS_INLINE double wave_sum(double v) {
#define BS_STEP(ctrl_, rows_, zero_)                                                       \
  {                                                                                        \
    const uint64_t b = __builtin_bit_cast(uint64_t, v);                                    \
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), ctrl_, rows_, 0xF, zero_);        \
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), ctrl_, rows_, 0xF, zero_);  \
    v += __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);                 \
  }
  BS_STEP(0x111, 0xF, true);
  BS_STEP(0x112, 0xF, true);
  BS_STEP(0x114, 0xF, true);
  BS_STEP(0x118, 0xF, true);
  BS_STEP(0x142, 0xA, false);
  BS_STEP(0x143, 0xC, false);
#undef BS_STEP
  return lane_of(v, 63);
}
BS_INLINE float lane_of(float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); }

// Weights of the picks: lane j's score my_s over the sum of all (renorm), in fp64.
BS_INLINE void store_picks(const RouteArgs& p, size_t o, int l, int my_id, double my_s) {
  double w = my_s;
  if (p.renorm) {
    const double sum = wave_sum(my_s);
    w = sum == 0.0 ? 0.0 : my_s / sum;
  }
  if (l < p.k) {
    p.ids[o + l] = my_id;
    p.weights[o + l] = my_id < 0 ? 0.0f : static_cast<float>(w * static_cast<double>(p.scale));
  }
}

BS_INLINE bool padding(const RouteArgs& p, int t, size_t o, int l) {
  if (p.rows == nullptr || t < *p.rows) return false;
  if (l < p.k) {
    p.ids[o + l] = -1;
    p.weights[o + l] = 0.0f;
  }
  return true;
}

// Any E and groups, all in fp64.
template <int V, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(64 * kWaves) void k_moe_route_f64(RouteArgs p) {
  __shared__ double s_val[kWaves][64 * V];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int t = blockIdx.x * kWaves + wave;
  if (t >= p.T) return;
  const size_t o = static_cast<size_t>(t) * p.k;
  if (padding(p, t, o, l)) return;
  int my_id;
  double my_s;
  route_exact<V, BF16, SIGMOID>(p, t, l, s_val[wave], my_id, my_s);
  store_picks(p, o, l, my_id, my_s);
}

// 2^x of the hardware with the rounding error of the product d * log2(e) added back
BS_INLINE float exp_near(float d) {
  const float p = d * 1.44269502f, lo = fmaf(d, 1.44269502f, -p);
  const float e = __builtin_amdgcn_exp2f(p);
  return fmaf(e, lo * 0.693147181f, e);
}

// The sigmoid to within kTau.  Outside of [-80, 100] it is 0 or 1 to within that, and
// there the product in exp_near passes fp32 for x from 2.36e38 on (its error term is
// then infinite too, and the result a NaN).
BS_INLINE float sigmoid_near(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_near(__builtin_amdgcn_fmed3f(-x, -100.0f, 80.0f)));
}

// e^(x - mx) to about an ulp and a half: the rounding error of the difference (which
// would cost |x - mx| / 2 ulps) and the rest of log2(e) go the same way.
BS_INLINE float exp_diff(float x, float mx) {
  const float d = x - mx, b = d - x, err = (x - (d - b)) - (mx + b);
  const float p = d * 1.44269502f, lo = fmaf(d, 1.44269502f, -p) + fmaf(d, 1.92596299e-8f, err * 1.44269502f);
  const float e = __builtin_amdgcn_exp2f(p);
  return fmaf(e, lo * 0.693147181f, e);
}

// V consecutive logits of a token from expert e0 on (-inf past E).  wide: rows and
// E are whole vectors of V.
template <int V, bool BF16>
BS_INLINE void load_logits(const void* base, size_t row, int e0, int E, bool wide, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = -__builtin_inff();
  if (e0 >= E) return;
  if (wide) {
    if constexpr (BF16) {
      const uint16_t* at = static_cast<const uint16_t*>(base) + row + e0;
      if constexpr (V >= 8) {
#pragma unroll
        for (int i = 0; i < V; i += 8) {
          const uint4 v = *reinterpret_cast<const uint4*>(at + i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[i + 2 * j] = bf16_lo(w[j]);
            x[i + 2 * j + 1] = bf16_hi(w[j]);
          }
        }
      } else if constexpr (V == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
      } else if constexpr (V == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
        x[0] = bf16_lo(w); x[1] = bf16_hi(w);
      } else {
        x[0] = bf16_lo(*at);
      }
    } else {
      const float* at = static_cast<const float*>(base) + row + e0;
      if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const float4 w = *reinterpret_cast<const float4*>(at + i);
          x[i] = w.x; x[i + 1] = w.y; x[i + 2] = w.z; x[i + 3] = w.w;
        }
      } else if constexpr (V == 2) {
        const float2 w = *reinterpret_cast<const float2*>(at);
        x[0] = w.x; x[1] = w.y;
      } else {
        x[0] = *at;
      }
    }
  } else {
    // (all loads at once, those past E of the last value)
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = load_logit<BF16>(base, row + min(e0 + i, E - 1));
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = e0 + i < E ? y[i] : x[i];
  }
}

// The quick form: V consecutive experts a lane, the choice by fp32 values.  Without a
// bias these are the logits themselves, and their order is exact (a group's sum of two
// is one of scores all the same).  Else they are scores within kTau of the real ones;
// where two
// values that the order or the border hangs on are closer than that (about one token
// in 200 of 256 sigmoids), what is close is decided by fp64 values: the groups' sums
// all anew, or the picks together with up to kMore that follow them, ranked.  (The
// whole token anew in fp64 is left to rows with a NaN or +inf and to longer runs of
// close values: the wave takes 8 us, which a launch of 16384 tokens would wait for at
// its end.)  Weights are computed in fp64 from the picks' logits; only the sum over all
// experts, which a softmax without renorm divides by, is one of fp32 exponentials, added
// in fp64: those weights are up to 6 half steps of fp32 off (511 equal logits 4 below the
// largest, whose differences from it round alike).
// A lane keeps its values sorted, in lists of four, so a pick is one reduction over
// the lanes' heads and one shift in the winner's list (16384 tokens, 8 of 256: with
// every value compared anew in fp64 38 us).
// GROUPS: a group is `part` lanes, a power of two.
constexpr float kTau = 0x1p-19f;
constexpr int kMore = 8;

// s_val: 64 * V doubles of the wave (the fp64 form's values; here the logits).
template <int V, bool BF16, bool SIGMOID, bool GROUPS>
BS_INLINE void route_token(const RouteArgs& p, int t, int l, bool wide, int part, double* s_val) {
  constexpr int LS = V < 4 ? V : 4, NL = V / LS;   // lists of LS values
  const size_t o = static_cast<size_t>(t) * p.k;
  const float ninf = -__builtin_inff();
  const int e0 = l * V;
  float x[V], v[V];
  load_logits<V, BF16>(p.logits, static_cast<size_t>(t) * p.ld, e0, p.E, wide, x);
  float* s_x = reinterpret_cast<float*>(s_val);
#pragma unroll
  for (int i = 0; i < V; ++i) s_x[e0 + i] = x[i];

  const bool by_logit = p.bias == nullptr;                      // experts
  const bool by_score = !by_logit || (GROUPS && p.top == 2);    // groups
  float mx = x[0];
  bool odd = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    odd |= !(x[i] < __builtin_inff());
    mx = fmaxf(mx, x[i]);
  }
  bool redo = __ballot(odd) != 0;
  mx = wave_fmax(mx);
  double total = 1.0;     // softmax: the sum of exp(x - mx)
  float largest = 1.0f;   // of the scores
  const bool scored = by_score || (!SIGMOID && !p.renorm);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = x[i];
  if (scored) {
    if constexpr (SIGMOID) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = sigmoid_near(x[i]);
      }
    } else {
      double part_sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = exp_near(fmaxf(x[i] - mx, -100.0f));
        v[i] = x[i] - mx < -100.0f ? 0.0f : v[i];     // (off: -inf)
        part_sum += static_cast<double>(v[i]);
      }
      total = wave_sum(part_sum);
      largest = 1.0f / static_cast<float>(total);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= largest;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!by_score) {
        v[i] = x[i];
      } else {
        if (p.bias != nullptr) {
          const float b = e0 + i < p.E ? p.bias[e0 + i] : 0.0f;
          v[i] += b;
          odd |= !(b < __builtin_inff());
        }
        v[i] = x[i] == ninf ? ninf : v[i];
      }
    }
    redo |= __ballot(odd) != 0;
  }

  // fp64 values of logits f, once the sum is known
  auto exact_total = [&]() {
    if constexpr (SIGMOID) return 1.0;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += x[i] == ninf ? 0.0 : exp(static_cast<double>(x[i]) - static_cast<double>(mx));
    return wave_sum(sum);
  };
  auto exact_value = [&](float f, int e, double sum) {
    const double d = f, b = p.bias != nullptr ? static_cast<double>(p.bias[e]) : 0.0;
    if constexpr (SIGMOID) return 1.0 / (1.0 + exp(-d)) + b;
    else return exp(d - static_cast<double>(mx)) / sum + b;
  };
  int my_id = -1;
  if (!redo) {
    uint32_t key[V], ga = 0u, gb = 0u;   // (ga, gb: the two largest scores where the keys are logits)
    int id[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = v[i] == ninf ? 0u : key_of(v[i]);
      id[i] = e0 + i;
    }
    if constexpr (GROUPS) {
      if (by_logit && by_score) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          gb = max(gb, min(ga, key[i]));
          ga = max(ga, key[i]);
          key[i] = v[i] == ninf ? 0u : key_of(x[i]);
        }
      }
    }
    // each list sorted: downwards, equal ones in the order of their index (only
    // neighbours change places)
#pragma unroll
    for (int q = 0; q < NL; ++q)
#pragma unroll
      for (int i = 1; i < LS; ++i)
#pragma unroll
        for (int j = i; j >= 1; --j) {
          uint32_t &a = key[q * LS + j - 1], &b = key[q * LS + j];
          int &ia = id[q * LS + j - 1], &ib = id[q * LS + j];
          const bool up = b > a;
          const uint32_t hi = max(a, b), lo = min(a, b);
          const int ih = up ? ib : ia, il = up ? ia : ib;
          a = hi;
          b = lo;
          ia = ih;
          ib = il;
        }
    if constexpr (GROUPS) {
      uint32_t a = key[0], b = LS > 1 ? key[LS > 1 ? 1 : 0] : 0u;   // the two largest
      auto join = [&](uint32_t a2, uint32_t b2) {
        b = max(max(b, b2), min(a, a2));
        a = max(a, a2);
      };
      if constexpr (NL == 2) join(key[NL == 2 ? 4 : 0], key[NL == 2 ? 5 : 0]);
      if (by_logit && by_score) {
        a = ga;
        b = gb;
      }
#define BS_JOIN(ctrl_)                                                                                     \
  join(static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(a), ctrl_, 0xF, 0xF, true)),        \
       static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(b), ctrl_, 0xF, 0xF, true)))
      if (part > 1) BS_JOIN(0xB1);    // lane ^ 1
      if (part > 2) BS_JOIN(0x4E);    // lane ^ 2
      if (part > 4) BS_JOIN(0x141);   // the other half of 8 (its lanes are equal by now)
      if (part > 8) BS_JOIN(0x140);   // the other half of 16
#undef BS_JOIN
      for (int s = 16; s < part; s <<= 1)
        join(static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), s, 64)),
             static_cast<uint32_t>(__shfl_xor(static_cast<int>(b), s, 64)));
      const float fa = a == 0u ? ninf : value_of(a), fb = b == 0u ? ninf : value_of(b);
      const float u = p.top == 2 ? fa + fb : fa;
      const int g = l / part;
      int before = 0;
      for (int h = 0; h < p.groups; ++h) {
        const float w = lane_of(u, h * part);
        before += w > u || (w == u && h < g) ? 1 : 0;
      }
      const bool here = g < p.groups;
      if (p.keep < p.groups && by_score) {   // the border
        const float in = lane_of(u, __builtin_ctzll(__ballot(here && before == p.keep - 1)));
        const float out = lane_of(u, __builtin_ctzll(__ballot(here && before == p.keep)));
        // (a sum is off by what its terms are, and those of any group may be large ones
        // that cancel)
        const float terms = p.top == 2 ? fabsf(fa) + fabsf(fb) : fabsf(fa);
        const float most = wave_fmax(terms < __builtin_inff() ? terms : 0.0f);
        if (!(in - out > 4.0f * kTau * (largest + most))) {
          const double sum = exact_total();
          double da = ninf, db = ninf;
          auto add = [&](double a2, double b2) {
            const double lo = a2 > da ? da : a2;
            da = a2 > da ? a2 : da;
            db = b2 > db ? b2 : db;
            db = lo > db ? lo : db;
          };
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (x[i] != ninf) add(exact_value(x[i], e0 + i, sum), ninf);
          for (int s = 1; s < part; s <<= 1) add(__shfl_xor(da, s, 64), __shfl_xor(db, s, 64));
          const double du = p.top == 2 ? da + db : da;
          before = 0;
          for (int h = 0; h < p.groups; ++h) {
            const double w = lane_of(du, h * part);
            before += w > du || (w == du && h < g) ? 1 : 0;
          }
        }
      }
      const bool off = !here || before >= p.keep;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = off ? 0u : key[i];
    }
    int my_key = 0, found = 0;
    // one more pick; false when no expert is left
    auto pick = [&]() {
      const bool second = NL == 2 && key[NL == 2 ? 4 : 0] > key[0];
      const uint32_t head = second ? key[NL == 2 ? 4 : 0] : key[0];
      const uint32_t m = wave_kmax(head);
      if (m == 0u) return false;
      const int w = __builtin_ctzll(__ballot(head == m));
      const int e = __builtin_amdgcn_readlane(second ? id[NL == 2 ? 4 : 0] : id[0], w);
      my_id = l == found ? e : my_id;
      my_key = l == found ? static_cast<int>(m) : my_key;
      ++found;
      if (l == w) {
#pragma unroll
        for (int q = 0; q < NL; ++q)
          if ((q == 1) == second) {
#pragma unroll
            for (int i = 0; i + 1 < LS; ++i) {
              key[q * LS + i] = key[q * LS + i + 1];
              id[q * LS + i] = id[q * LS + i + 1];
            }
            key[q * LS + LS - 1] = 0u;
          }
      }
      return true;
    };
    while (found < p.k && pick()) {
    }
    if (!by_logit) {
      auto best_left = [&]() { return wave_kmax(NL == 2 ? max(key[0], key[NL == 2 ? 4 : 0]) : key[0]); };
      auto clear = [&](float m, float n) { return m - n > kTau * (largest + fabsf(m)); };
      // every pick against the next, the last one against the best that is left
      uint32_t left = best_left();
      const uint32_t next = static_cast<uint32_t>(__shfl_down(my_key, 1, 64));   // (by all lanes: none reads from one that is off)
      const uint32_t below = l == found - 1 ? left : next;
      if (__ballot(l < found && below != 0u && !clear(value_of(my_key), value_of(below))) != 0) {
        const int kept = found;
        while (found < min(p.k + kMore, 64) && pick()) {
        }
        left = best_left();
        const float last = value_of(static_cast<uint32_t>(__builtin_amdgcn_readlane(my_key, kept - 1)));
        if (left != 0u && !clear(last, value_of(left))) {
          redo = true;
        } else {
          wave_lds_fence();
          const double sum = exact_total(), mine = l < found ? exact_value(s_x[max(my_id, 0)], max(my_id, 0), sum) : ninf;
          int rank = 0;
          for (int i = 0; i < found; ++i) {
            const double other = lane_of(mine, i);
            const int e = __builtin_amdgcn_readlane(my_id, i);
            rank += other > mine || (other == mine && e < my_id) ? 1 : 0;
          }
          rank = l < found ? rank : l;
          my_id = __builtin_amdgcn_ds_permute(4 * rank, my_id);
          my_id = l < kept ? my_id : -1;
        }
      }
    }
  }
  double my_s;
  if (redo) {
    wave_lds_fence();
    route_exact<V, BF16, SIGMOID>(p, t, l, s_val, my_id, my_s);
  } else {
    wave_lds_fence();
    const double xj = s_x[max(my_id, 0)];
    const double ref = SIGMOID ? 0.0 : static_cast<double>(mx);
    const double e = exp(SIGMOID ? -xj : xj - ref);
    my_s = my_id < 0 ? 0.0 : (SIGMOID ? 1.0 / (1.0 + e) : (p.renorm ? e : e / total));
  }
  store_picks(p, o, l, my_id, my_s);
}

template <int V, bool BF16, bool SIGMOID, bool GROUPS>
__global__ __launch_bounds__(64 * kWaves) void k_moe_route(RouteArgs p, bool wide, int part) {
  __shared__ double s_val[kWaves][64 * V];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int t = blockIdx.x * kWaves + wave;
  if (t >= p.T || padding(p, t, static_cast<size_t>(t) * p.k, l)) return;
  route_token<V, BF16, SIGMOID, GROUPS>(p, t, l, wide, part, s_val[wave]);
}

// ------------------------------------------------------------ many tokens
// Four tokens a wave, 16 lanes and 16 V experts each, up to kManyK picks: the steps
// that a whole wave does for one token (a pick's reduction, the groups' order, the
// picks' fp64 scores) serve four at once.
// Here the value and its index in the lane share a key, so that sorting moves one
// register: the index, counted down, takes the place of the value's lowest bits (up to
// four), which adds 2^-19 of the value to what is unclear (bf16 logits lose nothing).
// That is decided as above, the picks with kManyMore that follow them in the token's 16
// lanes; a row with a NaN or +inf, or with more close values, by the whole wave in
// fp64.  Loops that few waves run stay rolled: what such a wave waits for, and the
// launch with it at its end, is mostly their instructions' way into the cache.
// 16384 tokens, 8 of 256, us: softmax 7.5 (a token a wave 11.9), sigmoids with bias in
// 8 groups 12 (19); 64 experts 5.0 (9.7) and 8.2 (15).  Bound by VALU instructions and
// by the waves whose order fp32 leaves open, 3 us of the 12 (with the form above for
// those 20; all 16 values of a lane anew in fp64 for a border 16).  Where whole tokens
// are equal sigmoids with a bias, all goes through fp64 (8192 tokens 51 us, a token a
// wave 36).  Its limits are what 16 lanes hold (kManyK + kManyMore candidates, 16
// experts each) and not where it stops to pay: past them a wave takes one token (16384
// x 256, cold, us: softmax with 8 picks 8.7, with 9 13.1, with 12 14.8; 384 experts 18,
// 512 with 10 picks 20).
constexpr int kManyK = 8, kManyMore = 4;
static_assert(kManyK + kManyMore <= 16, "a token's candidates are one to a lane");
// from here on (256 experts, softmax / sigmoids with bias in 8 groups, us: 2048 tokens
// 4.8 / 7.3, a token a wave 4.1 / 7.5; 4096 tokens 4.9 / 7.4 and 5.1 / 9.0)
constexpr int kManyTokens = 4096;

// sorted[LO .. LO + N) downwards: Batcher's odd-even merge sort; compile-time indices
// only, and what nobody reads drops out.
template <int LO, int N, int R, int V>
BS_INLINE void merge_keys(uint32_t (&key)[V]) {
  auto order = [&](int i, int j) {
    const uint32_t a = key[i], b = key[j];
    key[i] = max(a, b);
    key[j] = min(a, b);
  };
  if constexpr (2 * R < N) {
    merge_keys<LO, N, 2 * R>(key);
    merge_keys<LO + R, N, 2 * R>(key);
#pragma unroll
    for (int i = LO + R; i + R < LO + N; i += 2 * R) order(i, i + R);
  } else {
    order(LO, LO + R);
  }
}
template <int LO, int N, int V>
BS_INLINE void sort_keys(uint32_t (&key)[V]) {
  if constexpr (N > 1) {
    sort_keys<LO, N / 2>(key);
    sort_keys<LO + N / 2, N / 2>(key);
    merge_keys<LO, N, 1>(key);
  }
}

// Over the 16 lanes of a token, in all of them.
#define BS_ROR(v_, n_) __builtin_amdgcn_mov_dpp(static_cast<int>(v_), 0x120 + n_, 0xF, 0xF, true)
BS_INLINE uint32_t row_kmax(uint32_t v) {
  v = max(v, static_cast<uint32_t>(BS_ROR(v, 8)));
  v = max(v, static_cast<uint32_t>(BS_ROR(v, 4)));
  v = max(v, static_cast<uint32_t>(BS_ROR(v, 2)));
  return max(v, static_cast<uint32_t>(BS_ROR(v, 1)));
}
BS_INLINE float row_fmax(float v) {
  v = fmaxf(v, __int_as_float(BS_ROR(__float_as_int(v), 8)));
  v = fmaxf(v, __int_as_float(BS_ROR(__float_as_int(v), 4)));
  v = fmaxf(v, __int_as_float(BS_ROR(__float_as_int(v), 2)));
  return fmaxf(v, __int_as_float(BS_ROR(__float_as_int(v), 1)));
}
BS_INLINE double row_sum(double v) {
#define BS_STEP(n_)                                                                                     \
  {                                                                                                     \
    const uint64_t b = __builtin_bit_cast(uint64_t, v);                                                 \
    const uint32_t lo = BS_ROR(b, n_), hi = BS_ROR(b >> 32, n_);                                        \
    v += __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);                              \
  }
  BS_STEP(8)
  BS_STEP(4)
  BS_STEP(2)
  BS_STEP(1)
#undef BS_STEP
  return v;
}
#undef BS_ROR

template <int V, bool BF16, bool SIGMOID, bool GROUPS>
__global__ __launch_bounds__(64 * kWaves) void k_moe_route_many(RouteArgs p, bool wide, bool wide_bias, int part) {
  constexpr uint32_t kLow = V - 1;
  constexpr int D = V < kManyK + 1 ? V : kManyK + 1;   // values of a lane that can matter: the picks and the next
  __shared__ double s_val[kWaves][32 * V];             // logits of the wave's four tokens; then route_exact's
  __shared__ int s_id[kWaves][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int r = l >> 4, c = l & 15;                    // the token's row of lanes, the lane in it
  const int t0 = (blockIdx.x * kWaves + wave) * 4, t = t0 + r;
  if (t0 >= p.T) return;
  const bool live = t < p.T && (p.rows == nullptr || t < *p.rows);
  const float ninf = -__builtin_inff();
  const int e0 = c * V;
  float x[V], v[V];
  float bias[V];
  if (p.bias != nullptr) load_logits<V, false>(p.bias, 0, e0, p.E, wide_bias, bias);
  load_logits<V, BF16>(p.logits, static_cast<size_t>(min(t, p.T - 1)) * p.ld, e0, p.E, wide, x);
  float* s_x = reinterpret_cast<float*>(s_val[wave]) + r * 16 * V;
#pragma unroll
  for (int i = 0; i < V; ++i) s_x[e0 + i] = x[i];

  const bool by_logit = p.bias == nullptr;                      // (as in route_token)
  const bool by_score = !by_logit || (GROUPS && p.top == 2);
  float mx = x[0];
  bool odd = false;
  uint32_t low = 0u;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    odd |= !(x[i] < __builtin_inff());
    low |= __float_as_uint(x[i]);
    mx = fmaxf(mx, x[i]);
  }
  mx = row_fmax(mx);
  double total = 1.0;
  float largest = 1.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = x[i];
  if (by_score || (!SIGMOID && !p.renorm)) {
    if constexpr (SIGMOID) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = sigmoid_near(x[i]);
    } else {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = exp_near(fmaxf(x[i] - mx, -100.0f));
        v[i] = x[i] - mx < -100.0f ? 0.0f : v[i];
        sum += static_cast<double>(v[i]);
      }
      total = row_sum(sum);
      largest = 1.0f / static_cast<float>(total);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= largest;
    }
    if (!by_score) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = x[i];
    } else if (p.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] += bias[i];   // (-inf past E)
        odd |= !(bias[i] < __builtin_inff());
      }
    }
  }
  const uint64_t mine = 0xFFFFull << (16 * r);   // the token's lanes
  bool redo = (__ballot(odd) & mine) != 0;
  const bool lossy = (__ballot((low & kLow) != 0u) & mine) != 0;
  uint32_t key[V], ga = 0u, gb = 0u;   // (as in route_token)
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool off = (x[i] == ninf) | (v[i] == ninf);   // (| : no branch)
    key[i] = off ? 0u : (key_of(v[i]) & ~kLow) | (kLow - i);
  }
  if constexpr (GROUPS) {
    if (by_logit && by_score) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        gb = max(gb, min(ga, key[i]));
        ga = max(ga, key[i]);
        key[i] = x[i] == ninf ? 0u : (key_of(x[i]) & ~kLow) | (kLow - i);
      }
    }
  }
  sort_keys<0, V>(key);

  // what decides in fp64: the sum of the scores, and the value of expert e
  auto exact_total = [&]() {
    if constexpr (SIGMOID) return 1.0;
    double sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
      const float f = s_x[e0 + i];
      sum += f == ninf ? 0.0 : exp(static_cast<double>(f) - static_cast<double>(mx));
    }
    return row_sum(sum);
  };
  auto exact_value = [&](float f, int at, double sum) {
    const double d = f, b = p.bias != nullptr ? static_cast<double>(p.bias[at]) : 0.0;
    if (!by_score) return d;
    if constexpr (SIGMOID) return 1.0 / (1.0 + exp(-d)) + b;
    else return exp(d - static_cast<double>(mx)) / sum + b;
  };

  if constexpr (GROUPS) {
    uint32_t a = key[0], b = key[V > 1 ? 1 : 0];   // the two largest
    auto join = [&](uint32_t a2, uint32_t b2) {
      b = max(max(b, b2), min(a, a2));
      a = max(a, a2);
    };
    if (by_logit && by_score) {
      a = ga;
      b = gb;
    }
#define BS_JOIN(ctrl_)                                                                                     \
  join(static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(a), ctrl_, 0xF, 0xF, true)),        \
       static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(b), ctrl_, 0xF, 0xF, true)))
    if (part > 1) BS_JOIN(0xB1);    // lane ^ 1
    if (part > 2) BS_JOIN(0x4E);    // lane ^ 2
    if (part > 4) BS_JOIN(0x141);   // the other half of 8
    if (part > 8) BS_JOIN(0x140);   // the other half of 16
#undef BS_JOIN
    const float fa = a == 0u ? ninf : value_of(a & ~kLow), fb = b == 0u ? ninf : value_of(b & ~kLow);
    const float u = p.top == 2 ? fa + fb : fa;
    const int g = c / part;
    int before = 0;
    for (int h = 0; h < p.groups; ++h) {
      const float w = __shfl(u, 16 * r + h * part, 64);
      before += w > u || (w == u && h < g) ? 1 : 0;
    }
    const bool here = g < p.groups;
    if (p.keep < p.groups) {   // the border
      const float in = row_fmax(here && before == p.keep - 1 ? u : ninf);
      const float out = row_fmax(here && before == p.keep ? u : ninf);
      const float terms = p.top == 2 ? fabsf(fa) + fabsf(fb) : fabsf(fa);
      const float most = row_fmax(here && terms < __builtin_inff() ? terms : 0.0f);
      // (twice route_token's margin, for the bits that the keys lose)
      const bool anew = by_score ? !(in - out > 8.0f * kTau * (largest + most)) : lossy && in == out && in != ninf;
      if (__ballot(anew && live && !redo) != 0) {
        const double sum = exact_total();
        double da = ninf, db = ninf;
        auto add = [&](double a2, double b2) {
          const double lo = a2 > da ? da : a2;
          da = a2 > da ? a2 : da;
          db = b2 > db ? b2 : db;
          db = lo > db ? lo : db;
        };
        // (of those that may be among the group's two largest)
        const float least = fb - 4.0f * kTau * (largest + fabsf(fb));
        uint32_t which = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) which |= static_cast<uint32_t>(anew & (v[i] >= least) & (v[i] != ninf) & (x[i] != ninf)) << i;
        while (which != 0u) {
          const int i = __builtin_ctz(which);
          which &= which - 1;
          add(exact_value(s_x[e0 + i], e0 + i, sum), ninf);
        }
#pragma unroll 1
        for (int d = 1; d < part; d <<= 1) add(__shfl_xor(da, d, 64), __shfl_xor(db, d, 64));
        const double du = p.top == 2 ? da + db : da;
        int before64 = 0;
#pragma unroll 1
        for (int h = 0; h < p.groups; ++h) {
          const double w = __shfl(du, 16 * r + h * part, 64);
          before64 += w > du || (w == du && h < g) ? 1 : 0;
        }
        before = anew ? before64 : before;
      }
    }
    const bool off = !here || before >= p.keep;
#pragma unroll
    for (int i = 0; i < D; ++i) key[i] = off ? 0u : key[i];
  }

  // the picks: lane j of the token keeps the j-th one's key without its index, its
  // winner writes its number
  const uint64_t lower = mine & ((1ull << l) - 1);
  uint32_t my_key = 0u;
  int* id = s_id[wave] + 16 * r;
  int found = 0, wins = 0;
  auto pick_up_to = [&](int n) {
    for (; found < n; ++found) {
      const uint32_t m = row_kmax(key[0]) & ~kLow;
      const bool tops = key[0] != 0u && (key[0] & ~kLow) == m;
      const bool won = (__ballot(tops) & lower) == 0 && tops;   // equal ones: the lowest lane
      if (won) {
        id[found] = e0 + static_cast<int>(kLow - (key[0] & kLow));
        ++wins;
#pragma unroll
        for (int i = 0; i + 1 < D; ++i) key[i] = key[i + 1];
        key[D - 1] = 0u;
      }
      my_key = c == found ? m : my_key;
    }
    return row_kmax(key[0]) & ~kLow;
  };
  // (m before n, or the last pick before the best that is left)
  auto clear = [&](uint32_t m, uint32_t n) {
    const float fm = value_of(m), fn = value_of(n);
    return by_logit ? !lossy || m != n : fm - fn > 2.0f * kTau * (largest + fabsf(fm) + fabsf(fn));
  };
  bool anew = false;
  {
    const uint32_t left = pick_up_to(p.k);
    const uint32_t next = static_cast<uint32_t>(__shfl_down(static_cast<int>(my_key), 1, 64));
    const uint32_t below = c == p.k - 1 ? left : next;
    anew = (__ballot(c < p.k && my_key != 0u && below != 0u && !clear(my_key, below)) & mine) != 0 && live && !redo;
  }
  const bool some = __ballot(anew) != 0;
  double sum64 = 1.0;
  if (some) {
    const uint32_t left = pick_up_to(p.k + kManyMore);
    const uint32_t last = static_cast<uint32_t>(__shfl(static_cast<int>(my_key), 16 * r + p.k - 1, 64));
    const bool spent = D < V && (__ballot(wins == D) & mine) != 0;
    redo |= anew && (spent || (left != 0u && !clear(last, left)));
    if (!by_logit) sum64 = exact_total();
  }
  wave_lds_fence();
  int my_id = my_key != 0u ? id[c] : -1;
  const double xj = my_id < 0 ? 0.0f : s_x[my_id];
  const double e = exp(SIGMOID ? -xj : xj - static_cast<double>(mx));
  double s = my_id < 0 ? 0.0 : (SIGMOID ? 1.0 / (1.0 + e) : (p.renorm ? e : e / total));
  if (some) {
    double val = ninf;
    if (my_id >= 0) {
      const double b = p.bias != nullptr ? static_cast<double>(p.bias[my_id]) : 0.0;
      val = by_logit ? xj : (SIGMOID ? s : e / sum64) + b;
    }
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const double other = __shfl(val, 16 * r + i, 64);
      const int other_id = __shfl(my_id, 16 * r + i, 64);
      rank += other > val || (other == val && other_id < my_id) ? 1 : 0;
    }
    const int to = 4 * (anew && my_id >= 0 ? 16 * r + rank : l);
    const uint64_t bits = __builtin_bit_cast(uint64_t, s);
    const uint32_t lo = __builtin_amdgcn_ds_permute(to, static_cast<int>(bits));
    const uint32_t hi = __builtin_amdgcn_ds_permute(to, static_cast<int>(bits >> 32));
    s = __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
    my_id = __builtin_amdgcn_ds_permute(to, my_id);
  }
  const bool there = c < p.k && my_id >= 0;
  double w = there ? s : 0.0;
  if (p.renorm) {
    const double sum = row_sum(w);
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  redo &= live;
  if (t < p.T && c < p.k && !redo) {
    const size_t o = static_cast<size_t>(t) * p.k + c;
    p.ids[o] = live && there ? my_id : -1;
    p.weights[o] = live && there ? static_cast<float>(w * static_cast<double>(p.scale)) : 0.0f;
  }
  uint64_t todo = __ballot(redo && c == 0);
  while (todo != 0) {
    const int q = t0 + (__builtin_ctzll(todo) >> 4);
    todo &= todo - 1;
    wave_lds_fence();
    int id64;
    double s64;
    route_exact<V / 4, BF16, SIGMOID>(p, q, l, s_val[wave], id64, s64);
    store_picks(p, static_cast<size_t>(q) * p.k, l, id64, s64);
  }
}

struct RouteBwdArgs {
  const float* dw;
  const void* logits;
  int64_t ld;
  const int* ids;
  void* dl;
  int64_t ldd;
  int T, E, k, renorm;
  float scale;
};

// V consecutive values of a gradient row.
template <int V, bool BF16>
BS_INLINE void store_row(void* base, size_t row, int e0, int E, bool wide, const float (&d)[V]) {
  if (e0 >= E) return;
  if constexpr (BF16) {
    uint32_t w[(V + 1) / 2];
#pragma unroll
    for (int i = 0; i < V; i += 2) w[i / 2] = bf16x2_rne(d[i], i + 1 < V ? d[i + 1 < V ? i + 1 : i] : 0.0f);
    uint16_t* at = static_cast<uint16_t*>(base) + row + e0;
    if (wide && V > 1) {
      if constexpr (V == 2) *reinterpret_cast<uint32_t*>(at) = w[0];
      if constexpr (V == 4) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
      if constexpr (V >= 8)
#pragma unroll
        for (int i = 0; i < V; i += 8)
          *reinterpret_cast<uint4*>(at + i) = make_uint4(w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E) at[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
  } else {
    float* at = static_cast<float*>(base) + row + e0;
    if (wide && V > 1) {
      if constexpr (V == 2) *reinterpret_cast<float2*>(at) = make_float2(d[0], d[1]);
      if constexpr (V >= 4)
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(at + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E) at[i] = d[i];
  }
}

// The gradient: lane j holds choice j (its part in fp64), lane l experts l * V ..
// l * V + V - 1 of the row.  The choices' parts go to their experts' places in LDS;
// where an expert is there twice, one after the other, in the order of j.  Only a
// softmax over all experts needs the row's logits (DENSE), the others those of the
// choices.  16384 x 256 fp32, 8 choices, sigmoids 8.1 us, cold 11: launch 2.6, stores of
// 16.8 MB 3.3, and the VALU, 56% busy with the fp64 exponential, quotients and sums of
// 8 of a wave's 64 lanes.
template <int V, bool BF16, bool SIGMOID, bool DENSE>
__global__ __launch_bounds__(64 * kWaves) void k_moe_route_bwd(RouteBwdArgs p, bool wide) {
  __shared__ __attribute__((aligned(16))) float s_d[kWaves][64 * V];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int t = blockIdx.x * kWaves + wave;
  if (t >= p.T) return;
  float* d = s_d[wave];
  const size_t o = static_cast<size_t>(t) * p.k, row = static_cast<size_t>(t) * p.ld;
  const int e0 = l * V;
  float x[V];
  if constexpr (DENSE) load_logits<V, BF16>(p.logits, row, e0, p.E, wide, x);
  const int id = l < p.k ? p.ids[o + l] : -1;
  const bool there = id >= 0 && id < p.E;
  const double g = there ? p.dw[o + l] : 0.0;
  const float lx = there ? load_logit<BF16>(p.logits, row + id) : -__builtin_inff();
#pragma unroll
  for (int i = 0; i < V; ++i) d[e0 + i] = 0.0f;
  float near = 0.0f;       // DENSE: 1 / the sum of exp(x - mx)
  double s, dot = 0.0, mine;
  const double c = p.scale;
  if constexpr (SIGMOID) {
    s = there ? 1.0 / (1.0 + exp(-static_cast<double>(lx))) : 0.0;
  } else {
    float mx = lx;
    if constexpr (DENSE) {
#pragma unroll
      for (int i = 0; i < V; ++i) mx = fmaxf(mx, x[i]);
    }
    mx = wave_fmax(mx);
    if constexpr (!DENSE) s = lx == -__builtin_inff() ? 0.0 : exp(static_cast<double>(lx) - static_cast<double>(mx));
    if constexpr (DENSE) {
      double part = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // (a NaN stays one; an expert that is off, and the places past E, give 0)
        x[i] = x[i] - mx < -100.0f || x[i] == -__builtin_inff() ? 0.0f : exp_diff(x[i], mx);
        part += static_cast<double>(x[i]);
      }
      // the choices' scores from the very values that the sum is made of: g - dot is
      // then as exact as its terms, where one score is nearly 1 too
      s = lx - mx < -100.0f || lx == -__builtin_inff() ? 0.0 : static_cast<double>(exp_diff(lx, mx));
      const double total = wave_sum(part);
      s = total == 0.0 ? 0.0 : s / total;
      near = total == 0.0 ? 0.0f : static_cast<float>(1.0 / total);
    }
  }
  if constexpr (DENSE) {
    dot = wave_sum(s * g);
    mine = g;
  } else if (SIGMOID && !p.renorm) {
    mine = c * g * s * (1.0 - s);
  } else {
    const double total = wave_sum(s);
    const double q = total == 0.0 ? 0.0 : s / total;
    dot = wave_sum(q * g);
    mine = c * q * (g - dot);
    if (SIGMOID) mine *= 1.0 - s;
  }
  const float add = static_cast<float>(mine);
  // every choice leaves its number at its expert; one that finds another there again
  // shares the expert
  int* tag = reinterpret_cast<int*>(d);
  wave_lds_fence();
  if (there) tag[id] = l;
  wave_lds_fence();
  const bool shared = there && tag[id] != l;
  wave_lds_fence();
  if (__ballot(shared) == 0) {
    if (there) d[id] = add;
  } else {
    if (there) d[id] = 0.0f;
    wave_lds_fence();
    for (int j = 0; j < p.k; ++j) {
      if (l == j && there) d[id] += add;
      wave_lds_fence();
    }
  }
  wave_lds_fence();
  float out[V];
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = d[e0 + i];
  if constexpr (DENSE) {
    // (a token without a choice has no gradient, whatever its logits hold)
    const bool any = __ballot(there) != 0;
    const float cf = p.scale;
#pragma unroll
    for (int i = 0; i < V; ++i)
      out[i] = any ? cf * (x[i] * near) * static_cast<float>(static_cast<double>(out[i]) - dot) : 0.0f;
  }
  store_row<V, BF16>(p.dl, static_cast<size_t>(t) * p.ldd, e0, p.E, wide, out);
}

template <int V>
int launch_route_f64(const RouteArgs& p, bool bf16, bool sigmoid, hipStream_t st) {
  const dim3 grid((p.T + kWaves - 1) / kWaves), block(64 * kWaves);
  if (bf16) {
    if (sigmoid) k_moe_route_f64<V, true, true><<<grid, block, 0, st>>>(p);
    else k_moe_route_f64<V, true, false><<<grid, block, 0, st>>>(p);
  } else {
    if (sigmoid) k_moe_route_f64<V, false, true><<<grid, block, 0, st>>>(p);
    else k_moe_route_f64<V, false, false><<<grid, block, 0, st>>>(p);
  }
  return bs_launch_status();
}
template <int V, bool GROUPS>
int launch_route(const RouteArgs& p, bool bf16, bool sigmoid, bool wide, int part, hipStream_t st) {
  const dim3 grid((p.T + kWaves - 1) / kWaves), block(64 * kWaves);
  if (bf16) {
    if (sigmoid) k_moe_route<V, true, true, GROUPS><<<grid, block, 0, st>>>(p, wide, part);
    else k_moe_route<V, true, false, GROUPS><<<grid, block, 0, st>>>(p, wide, part);
  } else {
    if (sigmoid) k_moe_route<V, false, true, GROUPS><<<grid, block, 0, st>>>(p, wide, part);
    else k_moe_route<V, false, false, GROUPS><<<grid, block, 0, st>>>(p, wide, part);
  }
  return bs_launch_status();
}
template <int V, bool GROUPS>
int launch_many(const RouteArgs& p, bool bf16, bool sigmoid, bool wide, bool wide_bias, int part, hipStream_t st) {
  const dim3 grid((p.T + 4 * kWaves - 1) / (4 * kWaves)), block(64 * kWaves);
  if (bf16) {
    if (sigmoid) k_moe_route_many<V, true, true, GROUPS><<<grid, block, 0, st>>>(p, wide, wide_bias, part);
    else k_moe_route_many<V, true, false, GROUPS><<<grid, block, 0, st>>>(p, wide, wide_bias, part);
  } else {
    if (sigmoid) k_moe_route_many<V, false, true, GROUPS><<<grid, block, 0, st>>>(p, wide, wide_bias, part);
    else k_moe_route_many<V, false, false, GROUPS><<<grid, block, 0, st>>>(p, wide, wide_bias, part);
  }
  return bs_launch_status();
}
// Four tokens a wave with V values a lane, if sizes and groups fit it.
template <int V>
bool try_many(const RouteArgs& p, bool bf16, bool sigmoid, hipStream_t st, int& status) {
  if (p.E > 16 * V || p.k > kManyK || p.T < kManyTokens) return false;
  const int size = p.E / p.groups, part = size / V, b = bf16 ? 2 : 4, bytes = std::min(V * b, 16);
  const bool wide = p.E % V == 0 && p.ld * b % bytes == 0 && bs_aligned(p.logits, bytes), wide_bias = p.E % V == 0 && bs_aligned(p.bias, 16);
  if (p.groups == 1) {
    status = launch_many<V, false>(p, bf16, sigmoid, wide, wide_bias, 16, st);
    return true;
  }
  if (size % V || (part & (part - 1)) || part > 16) return false;
  status = launch_many<V, true>(p, bf16, sigmoid, wide, wide_bias, part, st);
  return true;
}
// The quick form with V values a lane, if the groups fit it; V and BS_OK or an error
// in status.
template <int V>
bool try_route(const RouteArgs& p, bool bf16, bool sigmoid, hipStream_t st, int& status) {
  if (p.E > 64 * V) return false;
  const int size = p.E / p.groups, part = size / V, bytes = V * (bf16 ? 2 : 4);
  const bool wide = p.E % V == 0 && p.ld % V == 0 && bs_aligned(p.logits, std::min(bytes, 16));
  if (p.groups == 1) {
    status = launch_route<V, false>(p, bf16, sigmoid, wide, 64, st);
    return true;
  }
  if (size % V || (part & (part - 1)) || part > 64) return false;
  status = launch_route<V, true>(p, bf16, sigmoid, wide, part, st);
  return true;
}

template <int V>
int launch_route_bwd(const RouteBwdArgs& p, bool bf16, bool sigmoid, hipStream_t st) {
  const dim3 grid((p.T + kWaves - 1) / kWaves), block(64 * kWaves);
  const uintptr_t bytes = std::min(V * (bf16 ? 2 : 4), 16);
  const bool wide = p.E % V == 0 && p.ld % V == 0 && p.ldd % V == 0 && bs_aligned(p.logits, bytes) && bs_aligned(p.dl, bytes);
  if (bf16) {
    if (sigmoid) k_moe_route_bwd<V, true, true, false><<<grid, block, 0, st>>>(p, wide);
    else if (p.renorm) k_moe_route_bwd<V, true, false, false><<<grid, block, 0, st>>>(p, wide);
    else k_moe_route_bwd<V, true, false, true><<<grid, block, 0, st>>>(p, wide);
  } else {
    if (sigmoid) k_moe_route_bwd<V, false, true, false><<<grid, block, 0, st>>>(p, wide);
    else if (p.renorm) k_moe_route_bwd<V, false, false, false><<<grid, block, 0, st>>>(p, wide);
    else k_moe_route_bwd<V, false, false, true><<<grid, block, 0, st>>>(p, wide);
  }
  return bs_launch_status();
}

constexpr int kMaxExperts = 1024, kMaxK = 64;

bool sizes_ok(int T, int E, int k) {
  return T >= 1 && T <= (1 << 24) && E >= 1 && E <= kMaxExperts && k >= 1 && k <= E && k <= kMaxK;
}

}  // namespace

extern "C" {

BS_API int moe_route(const void* logits, int64_t ld, int type, const float* bias, int score, int groups,
                     int topk_groups, int group_top, int renorm, float scale, const int32_t* rows, int32_t* ids,
                     float* weights, int T, int E, int k, bs_stream_t stream) {
  if (T == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(logits && ids && weights, BS_ERR_NULL);
  BS_CHECK(sizes_ok(T, E, k), BS_ERR_SHAPE);
  BS_CHECK(groups >= 1 && groups <= 64 && E % groups == 0 && topk_groups >= 1 && topk_groups <= groups &&
               group_top >= 1 && group_top <= 2 && E / groups >= group_top && topk_groups * (E / groups) >= k,
           BS_ERR_SHAPE);
  BS_CHECK((type == BS_TYPE_F32 || type == BS_TYPE_BF16) && (score == BS_SCORE_SOFTMAX || score == BS_SCORE_SIGMOID),
           BS_ERR_ARG);
  BS_CHECK(ld >= E && bs_aligned(logits, type == BS_TYPE_F32 ? 4 : 2) && bs_aligned(bias, 4) && bs_aligned(rows, 4) &&
               bs_aligned(ids, 4) && bs_aligned(weights, 4),
           BS_ERR_ALIGN);
  const RouteArgs p{logits, ld, bias, rows, ids, weights, T, E, k, groups, topk_groups, group_top, renorm != 0, scale};
  const bool bf16 = type == BS_TYPE_BF16, sigmoid = score == BS_SCORE_SIGMOID;
  hipStream_t st = static_cast<hipStream_t>(stream);
  int status = BS_OK;
  if (try_many<4>(p, bf16, sigmoid, st, status) || try_many<8>(p, bf16, sigmoid, st, status) ||
      try_many<16>(p, bf16, sigmoid, st, status))
    return status;
  if (try_route<1>(p, bf16, sigmoid, st, status) || try_route<2>(p, bf16, sigmoid, st, status) ||
      try_route<4>(p, bf16, sigmoid, st, status) || try_route<8>(p, bf16, sigmoid, st, status))
    return status;
  const int v = (E + 63) / 64;   // more than 512 experts, or groups that are no whole lanes
  if (v <= 2) return launch_route_f64<2>(p, bf16, sigmoid, st);
  if (v <= 4) return launch_route_f64<4>(p, bf16, sigmoid, st);
  if (v <= 8) return launch_route_f64<8>(p, bf16, sigmoid, st);
  return launch_route_f64<16>(p, bf16, sigmoid, st);
}

BS_API int moe_route_backward(const float* dweights, const void* logits, int64_t ld, int type, const int32_t* ids,
                              int score, int renorm, float scale, void* dlogits, int64_t ldd, int T, int E, int k,
                              bs_stream_t stream) {
  if (T == 0) return BS_OK;  // an empty batch: nothing is read or launched
  BS_CHECK(dweights && logits && ids && dlogits, BS_ERR_NULL);
  BS_CHECK(sizes_ok(T, E, k), BS_ERR_SHAPE);
  BS_CHECK((type == BS_TYPE_F32 || type == BS_TYPE_BF16) && (score == BS_SCORE_SOFTMAX || score == BS_SCORE_SIGMOID),
           BS_ERR_ARG);
  const int b = type == BS_TYPE_F32 ? 4 : 2;
  BS_CHECK(ld >= E && ldd >= E && bs_aligned(logits, b) && bs_aligned(dlogits, b) && bs_aligned(dweights, 4) &&
               bs_aligned(ids, 4),
           BS_ERR_ALIGN);
  const RouteBwdArgs p{dweights, logits, ld, ids, dlogits, ldd, T, E, k, renorm != 0, scale};
  const bool bf16 = type == BS_TYPE_BF16, sigmoid = score == BS_SCORE_SIGMOID;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int v = (E + 63) / 64;
  if (v <= 1) return launch_route_bwd<1>(p, bf16, sigmoid, st);
  if (v <= 2) return launch_route_bwd<2>(p, bf16, sigmoid, st);
  if (v <= 4) return launch_route_bwd<4>(p, bf16, sigmoid, st);
  if (v <= 8) return launch_route_bwd<8>(p, bf16, sigmoid, st);
  return launch_route_bwd<16>(p, bf16, sigmoid, st);
}

}  // extern "C"
