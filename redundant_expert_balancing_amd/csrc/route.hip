// Router on gfx950: scores, balance bias, groups, top-K and gates of every token, and
// the gradient of the logits. The rule is stated in moonep.h (moonep_route).
//
// The choice is made in 64 bits: two experts whose scores differ by less than float32
// resolves must still come out in the order of their values, because a choice is a whole
// number. The gates themselves are float32.
#include <cmath>

#include "common.h"

namespace moonep {

constexpr int kRouteWaves = 4;        // wavefronts (tokens) per workgroup
constexpr int kMaxE = 1024;           // validate() bounds E
constexpr int kMaxPer = kMaxE / 64;   // experts per lane
constexpr float kNegInf = -__builtin_inff();
constexpr double kNegInfD = -__builtin_inf();

template <bool BF16>
__device__ inline float load_logit(const void* p, int64_t i) {
  if (BF16) return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
  return static_cast<const float*>(p)[i];
}

// The logit that counts: -inf where the bias switches the expert off, NaN where the bias
// is NaN.
__device__ inline float effective_logit(float l, float b) {
  if (b == kNegInf) return kNegInf;
  return b != b ? b : l;
}

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ inline double wave_sum_d(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ inline float wave_sum_f(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* gates;
  int N, E, K, groups, top_groups, group_top;
  bool softmax, renorm;
  float scale;
};

// Gates of one token: lane k < K holds the logit l of its k-th choice and whether the
// choice is a live one; m and sum are the row's maximum and softmax sum.
__device__ inline float gate_of(const RouteArgs& a, int lane, float l, bool live, float m,
                                float sum, bool bad) {
  live = live && lane < a.K;
  float w;
  if (!a.renorm) {
    w = a.softmax ? expf(l - m) / sum : 1.0f / (1.0f + expf(-l));
    w = live ? w : 0.f;
  } else {
    const float top = wave_max(live ? l : kNegInf);
    if (a.softmax) {
      w = live ? expf(l - top) : 0.f;
    } else {
      // s_k / sum s_j does not change when every s is divided by e^top: where even the
      // largest score is small, the scores e^l / (1 + e^l) are taken relative to it, so
      // that a row of very low logits does not end as 0 / 0
      w = top >= 0.f ? 1.0f / (1.0f + expf(-l)) : expf(l - top) / (1.0f + expf(l));
      w = live ? w : 0.f;
    }
    const float total = wave_sum_f(w);
    w = total > 0.f ? w / total : 0.f;
  }
  w *= a.scale;
  return bad ? __builtin_nanf("") : w;
}

// One wavefront per token; lane i holds experts i, i + 64, ...
template <bool BF16>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a) {
  __shared__ double s_val[kRouteWaves][kMaxE];
  __shared__ float s_logit[kRouteWaves][kMaxE];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  double* val = s_val[w];
  float* row = s_logit[w];
  const int per_group = a.E / a.groups;
  for (int64_t g = int64_t(blockIdx.x) * kRouteWaves + w; g < a.N;
       g += int64_t(gridDim.x) * kRouteWaves) {
    // effective logits, their maximum and the softmax sum
    float l[kMaxPer];
    float m = kNegInf;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i) {
      const int e = i * 64 + lane;
      l[i] = kNegInf;
      if (e < a.E) {
        l[i] = load_logit<BF16>(a.logits, g * a.E + e);
        if (a.bias) l[i] = effective_logit(l[i], a.bias[e]);
        bad |= l[i] != l[i] || (a.softmax && l[i] == -kNegInf);
        m = fmaxf(m, l[i]);
        row[e] = l[i];
      }
    }
    bad = __any(bad);
    m = wave_max(m);
    float sum = 0.f;
    double sumd = 0.0;
    if (a.softmax) {
#pragma unroll
      for (int i = 0; i < kMaxPer; ++i)
        if (i * 64 + lane < a.E && l[i] != kNegInf) {
          sum += expf(l[i] - m);
          sumd += exp(double(l[i]) - double(m));
        }
      sum = wave_sum_f(sum);
      sumd = wave_sum_d(sumd);
    }
    // keys: the logit itself without a bias (scores keep its order), else score + bias
    double key[kMaxPer];
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i) {
      const int e = i * 64 + lane;
      key[i] = kNegInfD;
      double sc = kNegInfD;
      if (e < a.E && l[i] == l[i] && l[i] != kNegInf) {
        const double ld = double(l[i]);
        const double s = a.softmax ? exp(ld - double(m)) / sumd : 1.0 / (1.0 + exp(-ld));
        sc = a.bias ? s + double(a.bias[e]) : s;
        key[i] = a.bias ? sc : ld;
        if (key[i] != key[i]) key[i] = kNegInfD;
        if (sc != sc) sc = kNegInfD;
      }
      if (e < a.E) val[e] = a.group_top == 1 ? key[i] : sc;
    }
    uint64_t kept = ~uint64_t(0);   // groups whose experts may be chosen
    if (a.groups > 1) {
      // lane j scores group j; rank of a group = groups that precede it
      __builtin_amdgcn_wave_barrier();
      double best = kNegInfD, second = kNegInfD;
      if (lane < a.groups)
        for (int i = 0; i < per_group; ++i) {
          const double v = val[lane * per_group + i];
          if (v > best) { second = best; best = v; }
          else if (v > second) second = v;
        }
      const double score = a.group_top == 2 && second != kNegInfD ? best + second : best;
      int rank = 0;
      for (int j = 0; j < a.groups; ++j) {
        const double o = __shfl(score, j, 64);
        rank += (o > score || (o == score && j < lane)) ? 1 : 0;
      }
      kept = __ballot(lane < a.groups && rank < a.top_groups);
    }
    uint32_t taken = 0;
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i) {
      const int e = i * 64 + lane;
      if (e >= a.E) taken |= 1u << i;
      else if (!((kept >> (e / per_group)) & 1)) key[i] = kNegInfD;
    }
    int my_id = 0;
    bool my_live = false;
    for (int k = 0; k < a.K; ++k) {
      double best = kNegInfD;
      int at = kMaxE;
#pragma unroll
      for (int i = 0; i < kMaxPer; ++i)
        if (!((taken >> i) & 1) && (at == kMaxE || key[i] > best)) {
          best = key[i];
          at = i * 64 + lane;
        }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) {
        const double ob = __shfl_xor(best, d, 64);
        const int oa = __shfl_xor(at, d, 64);
        if (ob > best || (ob == best && oa < at)) {
          best = ob;
          at = oa;
        }
      }
      if ((at & 63) == lane) taken |= 1u << (at >> 6);
      if (lane == k) {
        my_id = at;
        my_live = best != kNegInfD;
      }
    }
    __builtin_amdgcn_wave_barrier();
    const float lk = lane < a.K ? row[my_id] : kNegInf;
    const float gate = gate_of(a, lane, lk, my_live, m, sum, bad);
    if (lane < a.K) {
      a.ids[g * a.K + lane] = my_id;
      a.gates[g * a.K + lane] = gate;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

struct RouteBackwardArgs {
  const void* logits;
  const float* bias;
  const int32_t* ids;
  const float* gates;
  const float* dgates;
  void* dlogits;
  int N, E, K;
  bool softmax, renorm;
  float scale;
};

// One wavefront per token: lane k < K forms the gradient d of its choice's logit, then
// the row is written, each expert adding the choices that name it in k order.
template <bool BF16>
__global__ __launch_bounds__(kRouteWaves * 64) void route_backward_kernel(RouteBackwardArgs a) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const bool dense = a.softmax && !a.renorm;
  for (int64_t g = int64_t(blockIdx.x) * kRouteWaves + w; g < a.N;
       g += int64_t(gridDim.x) * kRouteWaves) {
    int id = -1;
    float gate = 0.f, d = 0.f;
    if (lane < a.K) {
      id = a.ids[g * a.K + lane];
      if (id < 0 || id >= a.E) id = -1;
      gate = id >= 0 ? a.gates[g * a.K + lane] : 0.f;
      d = gate != 0.f ? a.dgates[g * a.K + lane] : 0.f;   // a gate of 0 has no gradient
    }
    const float mean = wave_sum_f(gate * d);
    float v = gate * (a.renorm ? d - mean / a.scale : d);
    if (!a.softmax && gate != 0.f)
      v /= 1.0f + expf(load_logit<BF16>(a.logits, g * a.E + id));   // 1 - sigmoid
    float m = kNegInf, inv = 0.f;
    if (dense) {
      for (int e = lane; e < a.E; e += 64) {
        float l = load_logit<BF16>(a.logits, g * a.E + e);
        if (a.bias) l = effective_logit(l, a.bias[e]);
        m = fmaxf(m, l);
      }
      m = wave_max(m);
      float sum = 0.f;
      for (int e = lane; e < a.E; e += 64) {
        float l = load_logit<BF16>(a.logits, g * a.E + e);
        if (a.bias) l = effective_logit(l, a.bias[e]);
        if (l != kNegInf) sum += expf(l - m);
      }
      sum = wave_sum_f(sum);
      inv = sum != 0.f ? mean / sum : 0.f;
    }
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane;
      float out = 0.f;
      if (dense && e < a.E) {
        float l = load_logit<BF16>(a.logits, g * a.E + e);
        if (a.bias) l = effective_logit(l, a.bias[e]);
        out = l != kNegInf ? -inv * expf(l - m) : 0.f;
      }
      for (int k = 0; k < a.K; ++k) {
        const int ik = __shfl(id, k, 64);
        const float vk = __shfl(v, k, 64);
        if (ik == e) out += vk;
      }
      if (e < a.E) {
        if (BF16) static_cast<uint16_t*>(a.dlogits)[g * a.E + e] = uint16_t(bf16_rne_any(out));
        else static_cast<float*>(a.dlogits)[g * a.E + e] = out;
      }
    }
  }
}

static int check_router(const moonep_shape& s, const moonep_router* r) {
  if (!r) return MOONEP_EINVAL;
  if (r->score != MOONEP_SOFTMAX && r->score != MOONEP_SIGMOID) return MOONEP_EINVAL;
  if (r->dtype != MOONEP_BF16 && r->dtype != MOONEP_FP32) return MOONEP_EINVAL;
  if (r->groups < 1 || s.E % r->groups) return MOONEP_EINVAL;
  const int per_group = s.E / r->groups;
  if (r->top_groups < 1 || r->top_groups > r->groups) return MOONEP_EINVAL;
  if (r->group_top != 1 && r->group_top != 2) return MOONEP_EINVAL;
  if (r->groups > 1 && r->group_top > per_group) return MOONEP_EINVAL;
  if (s.K > r->top_groups * per_group) return MOONEP_EINVAL;
  if (r->renorm != 0 && r->renorm != 1) return MOONEP_EINVAL;
  if (!(r->scale > 0.f) || !std::isfinite(r->scale)) return MOONEP_EINVAL;
  if (r->groups > 64) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

}  // namespace moonep

using namespace moonep;

extern "C" int moonep_route(const moonep_shape* shape, const moonep_router* router,
                            const void* logits, const float* bias, int32_t* topk_idx, float* gates,
                            void* stream) {
  int st = validate(shape);
  if (st) return st;
  st = check_router(*shape, router);
  if (st) return st;
  const moonep_shape& s = *shape;
  const int N = s.R * s.S;
  if (N == 0) return MOONEP_OK;
  if (!aligned16(logits) || (bias && !aligned16(bias)) || !aligned16(topk_idx) || !aligned16(gates))
    return MOONEP_EINVAL;
  const RouteArgs a{logits, bias, topk_idx, gates, N, s.E, s.K, router->groups,
                    router->top_groups, router->group_top, router->score == MOONEP_SOFTMAX,
                    router->renorm != 0, router->scale};
  const int64_t blocks = (int64_t(N) + kRouteWaves - 1) / kRouteWaves;
  const int grid = int(blocks < 65536 ? blocks : 65536);
  if (router->dtype == MOONEP_BF16)
    route_kernel<true><<<grid, kRouteWaves * 64, 0, as_stream(stream)>>>(a);
  else
    route_kernel<false><<<grid, kRouteWaves * 64, 0, as_stream(stream)>>>(a);
  return launch_status();
}

extern "C" int moonep_route_backward(const moonep_shape* shape, const moonep_router* router,
                                     const void* logits, const float* bias,
                                     const int32_t* topk_idx, const float* gates,
                                     const float* dgates, void* dlogits, void* stream) {
  int st = validate(shape);
  if (st) return st;
  st = check_router(*shape, router);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.mode != MOONEP_TRAIN) return MOONEP_EMODE;
  const int N = s.R * s.S;
  if (N == 0) return MOONEP_OK;
  if (!aligned16(logits) || (bias && !aligned16(bias)) || !aligned16(topk_idx) ||
      !aligned16(gates) || !aligned16(dgates) || !aligned16(dlogits))
    return MOONEP_EINVAL;
  const RouteBackwardArgs a{logits, bias, topk_idx, gates, dgates, dlogits, N, s.E, s.K,
                            router->score == MOONEP_SOFTMAX, router->renorm != 0, router->scale};
  const int64_t blocks = (int64_t(N) + kRouteWaves - 1) / kRouteWaves;
  const int grid = int(blocks < 65536 ? blocks : 65536);
  if (router->dtype == MOONEP_BF16)
    route_backward_kernel<true><<<grid, kRouteWaves * 64, 0, as_stream(stream)>>>(a);
  else
    route_backward_kernel<false><<<grid, kRouteWaves * 64, 0, as_stream(stream)>>>(a);
  return launch_status();
}
