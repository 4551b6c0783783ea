// Routing of tokens to experts: scores, the choice of k experts and their
// weights, and the gradient of the weights.
//
// One wave per token.  Scores, group sums and the order of the choice are held in
// fp64: ids are discrete, and fp32 scores of different logits meet often enough
// (about one token in 10^4 has two within an ulp or two at the border of the
// choice) that their order would differ from the definition's.
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

BS_INLINE double wave_max_f64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const double u = __shfl_xor(v, o, 64);
    v = u > v ? u : v;
  }
  return v;
}

// Expert e = 64 * i + lane sits in register i of its lane.
template <int V, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(64 * kWaves) void k_moe_route(RouteArgs p) {
  __shared__ double s_val[kWaves][64 * V];
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int t = blockIdx.x * kWaves + wave;
  const double ninf = -__builtin_inf();
  if (t >= p.T) return;
  const size_t o = static_cast<size_t>(t) * p.k;
  if (p.rows != nullptr && t >= *p.rows) {
    if (l < p.k) {
      p.ids[o + l] = -1;
      p.weights[o + l] = 0.0f;
    }
    return;
  }
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
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) sc[i] = 1.0 / (1.0 + exp(-x[i]));
  } else {
    mx = wave_max_f64(mx);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sc[i] = x[i] == ninf ? 0.0 : exp(x[i] - mx);
      sum += sc[i];
    }
    sum = wave_sum_f64(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) sc[i] = bad ? __builtin_nan("") : sc[i] / sum;
  }
  // the order: by logits where nothing is added to the scores and none summed
  const bool by_logit = p.bias == nullptr && (p.groups == 1 || p.top == 1);
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
    for (int i = 0; i < V; ++i) s_val[wave][64 * i + l] = val[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int size = p.E / p.groups;
    int part = 64;
    while (part * p.groups > 64) part >>= 1;
    const int g = l / part, at = l % part;
    double a = ninf, b = ninf;   // the two largest
    if (g < p.groups)
      for (int i = at; i < size; i += part) {
        const double v = s_val[wave][g * size + i];
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
  int my_id = -1;
  double my_s = 0.0;
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
  double w = my_s;
  if (p.renorm) {
    const double sum = wave_sum_f64(my_s);
    w = sum == 0.0 ? 0.0 : my_s / sum;
  }
  if (l < p.k) {
    p.ids[o + l] = my_id;
    p.weights[o + l] = my_id < 0 ? 0.0f : static_cast<float>(w * static_cast<double>(p.scale));
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

// Lane j holds choice j; the gradients are added up by expert in LDS, in the
// order of j, and the row is written from there.
template <int V, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(64 * kWaves) void k_moe_route_bwd(RouteBwdArgs p) {
  __shared__ double s_d[kWaves][64 * V];
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int t = blockIdx.x * kWaves + wave;
  const double ninf = -__builtin_inf();
  if (t >= p.T) return;
  double* d = s_d[wave];
  double x[V], mx = ninf, sum = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 64 * i + l;
    x[i] = e < p.E ? load_logit<BF16>(p.logits, static_cast<size_t>(t) * p.ld + e) : -__builtin_inff();
    mx = x[i] > mx ? x[i] : mx;
    d[e] = 0.0;
  }
  mx = wave_max_f64(mx);
  const size_t o = static_cast<size_t>(t) * p.k;
  const int id = l < p.k ? p.ids[o + l] : -1;
  const bool there = id >= 0 && id < p.E;
  const double g = there ? p.dw[o + l] : 0.0;
  const double lx = there ? load_logit<BF16>(p.logits, static_cast<size_t>(t) * p.ld + id) : 0.0;
  const bool dense = !SIGMOID && !p.renorm;
  double s;
  if constexpr (SIGMOID) {
    s = there ? 1.0 / (1.0 + exp(-lx)) : 0.0;
  } else {
    s = !there || lx == ninf ? 0.0 : exp(lx - mx);
    if (dense) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[i] = x[i] == ninf ? 0.0 : exp(x[i] - mx);
        sum += x[i];
      }
      sum = wave_sum_f64(sum);
      const double inv = sum == 0.0 ? 0.0 : 1.0 / sum;
      s *= inv;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] *= inv;
    }
  }
  double mine, dot = 0.0;
  const double c = p.scale;
  if (p.renorm) {
    const double total = wave_sum_f64(s);
    const double q = total == 0.0 ? 0.0 : s / total;
    dot = wave_sum_f64(q * g);
    mine = c * q * (g - dot);
    if (SIGMOID) mine *= 1.0 - s;
  } else if (SIGMOID) {
    mine = c * g * s * (1.0 - s);
  } else {
    dot = wave_sum_f64(s * g);
    mine = g;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  for (int j = 0; j < p.k; ++j)
    if (l == j && there) d[id] += mine;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 64 * i + l;
    if (e >= p.E) break;
    const double v = dense ? c * x[i] * (d[e] - dot) : d[e];
    const size_t at = static_cast<size_t>(t) * p.ldd + e;
    if constexpr (BF16) static_cast<uint16_t*>(p.dl)[at] = static_cast<uint16_t>(bf16x2_rne(static_cast<float>(v), 0.0f));
    else static_cast<float*>(p.dl)[at] = static_cast<float>(v);
  }
}

template <int V>
int launch_route(const RouteArgs& p, bool bf16, bool sigmoid, hipStream_t st) {
  const dim3 grid((p.T + kWaves - 1) / kWaves), block(64 * kWaves);
  if (bf16) {
    if (sigmoid) k_moe_route<V, true, true><<<grid, block, 0, st>>>(p);
    else k_moe_route<V, true, false><<<grid, block, 0, st>>>(p);
  } else {
    if (sigmoid) k_moe_route<V, false, true><<<grid, block, 0, st>>>(p);
    else k_moe_route<V, false, false><<<grid, block, 0, st>>>(p);
  }
  return bs_launch_status();
}
template <int V>
int launch_route_bwd(const RouteBwdArgs& p, bool bf16, bool sigmoid, hipStream_t st) {
  const dim3 grid((p.T + kWaves - 1) / kWaves), block(64 * kWaves);
  if (bf16) {
    if (sigmoid) k_moe_route_bwd<V, true, true><<<grid, block, 0, st>>>(p);
    else k_moe_route_bwd<V, true, false><<<grid, block, 0, st>>>(p);
  } else {
    if (sigmoid) k_moe_route_bwd<V, false, true><<<grid, block, 0, st>>>(p);
    else k_moe_route_bwd<V, false, false><<<grid, block, 0, st>>>(p);
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
  const int v = (E + 63) / 64;
  if (v <= 1) return launch_route<1>(p, bf16, sigmoid, st);
  if (v <= 2) return launch_route<2>(p, bf16, sigmoid, st);
  if (v <= 4) return launch_route<4>(p, bf16, sigmoid, st);
  if (v <= 8) return launch_route<8>(p, bf16, sigmoid, st);
  return launch_route<16>(p, bf16, sigmoid, st);
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
