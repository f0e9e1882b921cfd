// Router on gfx950: scores, balance bias, groups, top-K and gates of every token, and
// the gradient of the logits. The rule is stated in moonep.h (moonep_route).
//
// The choice is that of 64-bit keys: two experts whose scores differ by less than float32
// resolves must still come out in the order of their values, because a choice is a whole
// number. route_packed_kernel decides in 32 bits what these can decide and the rest in 64;
// route_kernel ranks every key in 64. The gates themselves are float32.
#include <cmath>
#include <type_traits>

#include "common.h"

namespace moonep {

constexpr int kRouteWaves = 4;        // wavefronts (tokens) per workgroup
constexpr int kMaxE = 1024;           // validate() bounds E
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

// Orders this wavefront's LDS accesses for the compiler; its lanes run in step.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* gates;
  int N, E, K, groups, top_groups, group_top;
  bool softmax, renorm;
  float scale;
  bool bf16;
  // packed form: places per lane (a multiple of 4), lanes per group, places without an expert
  // behind each group's
  int epl, run, pad;
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

// One token by one wavefront, every key in float64. `val` is E doubles of LDS of this
// wavefront's own; loops are kept rolled, so that a kernel that seldom comes here does not
// pay for it in registers.
__device__ void route_token(const RouteArgs& a, int64_t g, double* val) {
  const int lane = threadIdx.x & 63;
  const int per_group = a.E / a.groups;
  auto logit = [&](int e) {
    const float l = a.bf16 ? load_logit<true>(a.logits, g * a.E + e)
                           : load_logit<false>(a.logits, g * a.E + e);
    return a.bias ? effective_logit(l, a.bias[e]) : l;
  };
  float m = kNegInf;
  bool bad = false;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const float l = logit(e);
    bad |= l != l || (a.softmax && l == -kNegInf);
    m = fmaxf(m, l);
  }
  bad = __any(bad);
  m = wave_max(m);
  float sum = 0.f;
  double sumd = 0.0;
  if (a.softmax) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      const float l = logit(e);
      if (l == kNegInf) continue;
      sum += expf(l - m);
      sumd += exp(double(l) - double(m));
    }
    sum = wave_sum_f(sum);
    sumd = wave_sum_d(sumd);
  }
  // float64 score + bias of an unmasked expert, -inf of any other or where it is NaN
  auto value = [&](int e, float l) {
    if (!(l > kNegInf)) return kNegInfD;
    const double ld = double(l);
    const double s = a.softmax ? exp(ld - double(m)) / sumd : 1.0 / (1.0 + exp(-ld));
    const double v = a.bias ? s + double(a.bias[e]) : s;
    return v == v ? v : kNegInfD;
  };
  // the ranking's key: without a bias the logit itself, whose order the scores keep
  auto rank_key = [&](int e, float l) {
    if (a.bias) return value(e, l);
    return l > kNegInf ? double(l) : kNegInfD;
  };
  uint64_t kept = ~uint64_t(0);   // groups whose experts may be chosen
  if (a.groups > 1) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64)
      val[e] = a.group_top == 1 ? rank_key(e, logit(e)) : value(e, logit(e));
    wave_sync();
    // lane j scores group j; the rank of a group is the number of groups before it
    double best = kNegInfD, second = kNegInfD;
    if (lane < a.groups)
#pragma unroll 1
      for (int i = 0; i < per_group; ++i) {
        const double v = val[lane * per_group + i];
        if (v > best) { second = best; best = v; }
        else if (v > second) second = v;
      }
    const double score = a.group_top == 2 && second != kNegInfD ? best + second : best;
    int rank = 0;
#pragma unroll 1
    for (int j = 0; j < a.groups; ++j) {
      const double o = __shfl(score, j, 64);
      rank += (o > score || (o == score && j < lane)) ? 1 : 0;
    }
    kept = __ballot(lane < a.groups && rank < a.top_groups);
    wave_sync();
  }
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64)
    val[e] = (kept >> (e / per_group)) & 1 ? rank_key(e, logit(e)) : kNegInfD;
  // K rounds of the best expert left; a taken one's key becomes NaN. Lanes read only what
  // they wrote.
  int my_id = 0;
  bool my_live = false;
#pragma unroll 1
  for (int k = 0; k < a.K; ++k) {
    double best = kNegInfD;
    int at = kMaxE;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      const double v = val[e];
      if (v > best || (v == best && at == kMaxE)) {
        best = v;
        at = e;
      }
    }
#pragma unroll 1
    for (int d = 32; d > 0; d >>= 1) {
      const double ob = __shfl_xor(best, d, 64);
      const int oa = __shfl_xor(at, d, 64);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if ((at & 63) == lane) val[at] = __builtin_nan("");
    if (lane == k) {
      my_id = at;
      my_live = best != kNegInfD;
    }
  }
  const float lk = lane < a.K ? logit(my_id) : kNegInf;
  const float gate = gate_of(a, lane, lk, my_live, m, sum, bad);
  if (lane < a.K) {
    a.ids[g * a.K + lane] = my_id;
    a.gates[g * a.K + lane] = gate;
  }
  wave_sync();
}

// Any E, K and groups: what the packed form does not take (K > 16, groups that need more lanes
// or places than a token has).
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a) {
  __shared__ double s_val[kRouteWaves][kMaxE];
  const int w = threadIdx.x >> 6;
  for (int64_t g = int64_t(blockIdx.x) * kRouteWaves + w; g < a.N;
       g += int64_t(gridDim.x) * kRouteWaves)
    route_token(a, g, s_val[w]);
}

// ---- packed form: 16 lanes per token, four tokens per wavefront, K <= 16.
//
// Ranking by float64 keys costs an exponential and a 64-bit comparison network per expert,
// and almost never decides anything: two scores have to agree to about 2^-21. So each
// expert gets one 32-bit word, its float32 key as a 22-bit fixed-point number between the
// token's lowest and highest key, above its complemented place: unsigned order is (key
// descending, id ascending), a word is its own payload, and one comparator is a max and a
// min. Each lane sorts its experts in columns of 8 and merges them into its best 8; the
// token's best KL (8, or 16 where K is more) are then taken one by one from the heads of its
// lanes' lists (a maximum over 16 lanes is four instructions; merging the lists lane by lane
// took 216 instead of 85). The result stands if no two neighbours of the ranking that could
// change the choice are closer than the keys' error, unless they are equal in logit and
// bias (then the id decides, as it should). Where two are (0.1% of the tokens of a normal
// sigmoid router), the experts in question are ranked by float64 keys, one per lane; so are
// groups that are too close. Tokens with a NaN or +inf, with more than 16 experts in
// question, or with more than 8 of the best 16 in one lane, are done again by route_token; so
// are those whose keys' spread or error the fixed-point range does not suit.
//
// Bound by the vector instructions: 1010 per wavefront at E = 384 with sigmoid, bias and groups
// (759 with softmax and no bias), which issue in 68000 of the 73300 cycles that a CU is busy
// with 65536 tokens. A call among others takes 37 us (softmax bf16 24 us); reading the logits
// alone is 22 us (12).
// Against one float64 wavefront per token (route_kernel): 470 us (410).
// E = 376 in 8 groups, whose places lie apart: 43 us, E = 1024 in 8 groups 131 us, K = 16
// 91 us; route_kernel 535, 1000 and 690 us.
constexpr int kHeads = 8;            // best experts that a lane lists
constexpr int kTokens = 4;           // per wavefront
// Tokens per launch of the kernels of four tokens per wavefront, which do not loop (a loop's
// invariants took 40 registers): a launch holds at most 2^32 threads.
constexpr int kLaunchTokens = 1 << 26;
constexpr uint32_t kIdMask = 1023;
constexpr uint32_t kNearMax = 4096;  // a wider band of doubt sends the token to route_token
constexpr float kQMax = 4186000.f;   // fixed-point range: keys 1 .. below 2^22 - kNearMax, masked 0

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, true));
}
// lane permutations whose pairs span 2, 4, 8 and 16 lanes
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
template <int CTRL>
__device__ inline float dppf(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }

// Larger and smaller of numbers in one instruction: fmaxf also quiets each operand that the
// compiler cannot prove quiet, at an instruction apiece.
__device__ inline float max2(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ inline float min2(float a, float b) {
  float r;
  asm("v_min_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ inline float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ inline float min3(float a, float b, float c) {
  float r;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
// NaN if one of them is.
__device__ inline float nan_min3(float a, float b, float c) {
  return __builtin_elementwise_minimum(__builtin_elementwise_minimum(a, b), c);
}

__device__ inline float row_max(float v) {
  v = max2(v, dppf<kXor1>(v));
  v = max2(v, dppf<kXor2>(v));
  v = max2(v, dppf<kHalfMirror>(v));
  return max2(v, dppf<kMirror>(v));
}
__device__ inline float row_min(float v) { return -row_max(-v); }
__device__ inline float row_sum(float v) {
  v += dppf<kXor1>(v);
  v += dppf<kXor2>(v);
  v += dppf<kHalfMirror>(v);
  return v + dppf<kMirror>(v);
}
__device__ inline uint32_t row_or(uint32_t v) {
  v |= dpp<kXor1>(v);
  v |= dpp<kXor2>(v);
  v |= dpp<kHalfMirror>(v);
  return v | dpp<kMirror>(v);
}

__device__ inline void order(uint32_t& hi, uint32_t& lo) {
  const uint32_t a = max(hi, lo), b = min(hi, lo);
  hi = a;
  lo = b;
}
// Descending sort of 8 (Batcher's odd-even merge sort, 19 comparators).
__device__ inline void sort8(uint32_t* v) {
  order(v[0], v[1]); order(v[2], v[3]); order(v[4], v[5]); order(v[6], v[7]);
  order(v[0], v[2]); order(v[1], v[3]); order(v[4], v[6]); order(v[5], v[7]);
  order(v[1], v[2]); order(v[5], v[6]);
  order(v[0], v[4]); order(v[1], v[5]); order(v[2], v[6]); order(v[3], v[7]);
  order(v[2], v[4]); order(v[3], v[5]);
  order(v[1], v[2]); order(v[3], v[4]); order(v[5], v[6]);
}
// Descending sort of a bitonic sequence of 8.
__device__ inline void bitonic8(uint32_t* v) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) order(v[i], v[i + d]);
}
__device__ inline uint32_t row_max_u(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  return max(v, dpp<kMirror>(v));
}

// 1 / (1 + e^-x), within 2^-22
__device__ inline float fast_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// Unsigned integer of x, saturating: 0 for a negative x or a NaN.
__device__ inline uint32_t saturating_uint(float x) {
  uint32_t r;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(r) : "v"(x));
  return r;
}

// A token's experts have 16 * EPL places, in ascending order. Each group begins at a lane: it has
// a.run lanes (a power of two, 16 without groups) and its last a.pad places are empty, which
// counts as masked. Words, lists and rows go by place; only the loads and the ids that go
// out know experts.
template <int EPL, int KL, bool SOFTMAX, bool BIAS>
__global__ __launch_bounds__(kRouteWaves * 64) void route_packed_kernel(RouteArgs a) {
  constexpr int kRow = 16 * EPL;
  constexpr int kCols = (EPL + 7) / 8 * 8;     // whole columns of 8
  constexpr float kLog2e = 1.44269504f;
  __shared__ __align__(16) float s_row[kRouteWaves][kTokens * kRow];
  __shared__ __align__(16) float s_bias[BIAS ? kRow : 4];
  __shared__ __align__(16) uint32_t s_list[kRouteWaves][kTokens][KL];
  __shared__ uint32_t s_cand[kRouteWaves][kTokens][16];
  const int lane = threadIdx.x & 63, t = lane >> 4, i16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.E, e0 = i16 * EPL, run = a.run, shift = __builtin_ctz(run);
  // the expert at a place; -1 of an empty one
  auto expert_at = [&](int place) {
    const int group = (place / EPL) >> shift, in = place - group * run * EPL;
    const int per_group = run * EPL - a.pad;
    return in < per_group && group < a.groups ? group * per_group + in : -1;
  };
  float* rows = s_row[w];
  bool nan_bias = false;
  if (BIAS) {
    int bad = 0;
    for (int p = threadIdx.x; p < kRow; p += kRouteWaves * 64) {
      const int e = expert_at(p);
      const float b = e >= 0 ? a.bias[e] : 0.f;
      s_bias[p] = b;
      bad |= b != b;
    }
    nan_bias = __syncthreads_or(bad) != 0;
  }
  const int64_t g0 = (int64_t(blockIdx.x) * kRouteWaves + w) * kTokens;
  if (g0 < a.N) {   // uniform per wavefront; no workgroup barrier inside
    const int ntok = int(min(int64_t(kTokens), a.N - g0));
    // the logits as float32, in rows of kRow
    if (E == kRow && ntok == kTokens) {      // the four rows lie together in memory as well
      if (a.bf16) {
        const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + g0 * E);
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) {
          const uint2 u = src[i * 256 / 4 + lane];
          uint2 lo2 = make_uint2(u.x << 16, u.x & 0xFFFF0000u), hi2 = make_uint2(u.y << 16, u.y & 0xFFFF0000u);
          reinterpret_cast<float4*>(rows)[i * 64 + lane] =
              make_float4(__uint_as_float(lo2.x), __uint_as_float(lo2.y), __uint_as_float(hi2.x),
                          __uint_as_float(hi2.y));
        }
      } else {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + g0 * E);
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) reinterpret_cast<float4*>(rows)[i * 64 + lane] = src[i * 64 + lane];
      }
    } else {
      // loads without a branch, so that many are in flight together
      auto spread = [&](auto bf16_c) {
#pragma unroll
        for (int c = 0; c < EPL / 4; ++c) {
          const int p = c * 64 + lane, e = expert_at(p);
#pragma unroll
          for (int r = 0; r < kTokens; ++r) {
            const int64_t first = (g0 + min(r, ntok - 1)) * E;
            const float x = load_logit<decltype(bf16_c)::value>(a.logits, first + max(e, 0));
            rows[r * kRow + p] = e >= 0 ? x : kNegInf;
          }
        }
      };
      if (a.bf16) spread(std::true_type());
      else spread(std::false_type());
    }
    wave_sync();
    const bool on = t < ntok;
    const float* row = rows + t * kRow;
    auto logits4 = [&](int c, float* l) {
      const float4 v = *reinterpret_cast<const float4*>(row + e0 + c);
      l[0] = v.x; l[1] = v.y; l[2] = v.z; l[3] = v.w;
      if (SOFTMAX && BIAS) {     // a switched-off expert has no part in the softmax
        const float4 b = *reinterpret_cast<const float4*>(s_bias + e0 + c);
        l[0] = b.x == kNegInf ? kNegInf : l[0];
        l[1] = b.y == kNegInf ? kNegInf : l[1];
        l[2] = b.z == kNegInf ? kNegInf : l[2];
        l[3] = b.w == kNegInf ? kNegInf : l[3];
      }
    };
    float top = 0.f, inv = 0.f, sum = 0.f;   // the largest logit, 1 / softmax sum, the sum
    // keys of 4 logits: score + bias (a masked expert's, whose score is 0, is made -inf by the
    // callers where the logit is)
    auto keys4 = [&](int c, float* l) {
      if (!BIAS) return;
      const float4 b4 = *reinterpret_cast<const float4*>(s_bias + e0 + c);
      const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = SOFTMAX ? __builtin_amdgcn_exp2f((l[i] - top) * kLog2e) * inv
                                : fast_sigmoid(l[i]);
        l[i] = s + b[i];
      }
    };
    // the same in float64, for the few tokens whose float32 keys are too close: the sum of
    // e^(l - top) over the token, and score + bias of expert e
    auto softmax_sum = [&]() {
      double d = 0.0;
#pragma unroll 1
      for (int c = 0; c < EPL; ++c) {
        float l = row[e0 + c];
        if (BIAS) l = s_bias[e0 + c] == kNegInf ? kNegInf : l;
        d += exp(double(l) - double(top));
      }
      for (int o = 1; o < 16; o <<= 1) d += __shfl_xor(d, o, 64);
      return d;
    };
    auto value = [&](int e, double total) {
      const float l = row[e], b = BIAS ? s_bias[e] : 0.f;
      if (l == kNegInf || b == kNegInf) return kNegInfD;
      const double s = SOFTMAX ? exp(double(l) - double(top)) / total : 1.0 / (1.0 + exp(-double(l)));
      return BIAS ? s + double(b) : s;
    };
    float key[EPL];
    float hi = kNegInf, lo = -kNegInf;
#pragma unroll
    for (int c = 0; c < EPL; c += 4) {
      logits4(c, key + c);
      lo = nan_min3(nan_min3(lo, key[c], key[c + 1]), key[c + 2], key[c + 3]);
      if (SOFTMAX || !BIAS) hi = max3(max3(hi, key[c], key[c + 1]), key[c + 2], key[c + 3]);
    }
    bool unsure = nan_bias || lo != lo;      // a NaN among the logits
    if (SOFTMAX) {
      top = row_max(hi);
      top = top == kNegInf ? 0.f : top;   // nothing left: every e^(l - top) is 0
      if (BIAS || !a.renorm) {
#pragma unroll
        for (int c = 0; c < EPL; ++c) sum += __builtin_amdgcn_exp2f((key[c] - top) * kLog2e);
        sum = row_sum(sum);
        inv = __builtin_amdgcn_rcpf(sum);
      }
    }
    if (BIAS) {
      const bool masked = lo == kNegInf;
      unsure |= SOFTMAX && top == -kNegInf;
#pragma unroll
      for (int c = 0; c < EPL; c += 4) keys4(c, key + c);
      if (__any(masked)) {
#pragma unroll
        for (int c = 0; c < EPL; c += 4) {
          float l[4];
          logits4(c, l);
#pragma unroll
          for (int i = 0; i < 4; ++i) key[c + i] = l[i] == kNegInf ? kNegInf : key[c + i];
        }
      }
      hi = kNegInf;
      lo = -kNegInf;
#pragma unroll
      for (int c = 0; c < EPL; c += 4) {
        hi = max3(max3(hi, key[c], key[c + 1]), key[c + 2], key[c + 3]);
        lo = min3(min3(lo, key[c], key[c + 1]), key[c + 2], key[c + 3]);
      }
    }
    unsure |= hi == -kNegInf;
    if (__any(lo == kNegInf)) {     // masked experts: the lowest of the others
      lo = -kNegInf;
#pragma unroll
      for (int c = 0; c < EPL; ++c) lo = min2(lo, key[c] == kNegInf ? lo : key[c]);
    }
    hi = row_max(hi);
    lo = row_min(lo);
    // float32 keys are off by at most `err`: sigmoid 2^-22, softmax 2^-18 (EPL > 32: 2^-17) of
    // the largest score (at most EPL + 4 roundings of the sum, 6 of the rest, in units of
    // 2^-24), the sum with the bias 2^-23 of itself; logits are exact
    auto key_error = [&](float low) {
      if (!BIAS) return 0.f;
      return (SOFTMAX ? (EPL > 32 ? 7.6293945e-6f : 3.8146973e-6f) * inv : 2.3841858e-7f) +
             1.1920929e-7f * max2(fabsf(hi), fabsf(low));
    };
    const float err = key_error(lo);
    // a long tail of low keys would take the range's resolution: keys more than 64 below the
    // highest get the number of masked ones (where the choice comes down to them, route_token
    // makes it)
    const bool tail = lo < hi - 64.f;
    if (tail) lo = hi - 64.f;
    float f = hi > lo ? kQMax * 0.9999995f * __builtin_amdgcn_rcpf(hi - lo) : 0.f;
    // The error in fixed-point steps, of keys inside the range: where it is too wide, and where
    // the spread is so small that f is not finite, the token goes to route_token. Compared as a
    // float: as a number it would wrap.
    const float steps = BIAS && f > 0.f ? 2.f * key_error(lo) * f : 0.f;
    unsure |= BIAS ? !(steps <= float(kNearMax - 3)) : f == -kNegInf;
    const uint32_t near = BIAS ? saturating_uint(min2(steps, float(kNearMax))) + 3 : 0;

    // groups: runs of the token's lanes; an empty one ranks behind every expert's
    bool kept = true;
    if (a.groups > 1) {
      float m1 = kNegInf, m2 = kNegInf;
#pragma unroll
      for (int c = 0; c < EPL; ++c) {
        m2 = __builtin_amdgcn_fmed3f(m1, m2, key[c]);
        m1 = max2(m1, key[c]);
      }
      auto join = [&](float o1, float o2) {
        m2 = max2(min2(m1, o1), max2(m2, o2));
        m1 = max2(m1, o1);
      };
      if (run >= 2) join(dppf<kXor1>(m1), dppf<kXor1>(m2));
      if (run >= 4) join(dppf<kXor2>(m1), dppf<kXor2>(m2));
      if (run >= 8) join(dppf<kHalfMirror>(m1), dppf<kHalfMirror>(m2));
      float score = m1, tol = 2.f * err;
      if (a.group_top == 2) {
        if (!BIAS) {   // the two best logits' scores (softmax: all by the same factor)
          if (SOFTMAX) {
            m1 = __builtin_amdgcn_exp2f((m1 - top) * kLog2e);
            m2 = __builtin_amdgcn_exp2f((m2 - top) * kLog2e);
          } else {
            m1 = fast_sigmoid(m1);
            m2 = fast_sigmoid(m2);
          }
          // a masked logit's score is 0, which is what it adds; a group with none is last
          score = score == kNegInf ? kNegInf : m1 + m2;
          tol = 3.8146973e-6f;
        } else {
          // half the sum: two biases of the largest value would pass float32's range
          score = 0.5f * m1 + (m2 == kNegInf ? 0.f : 0.5f * m2);
          tol = 2.f * err + 2.3841858e-7f * (score == kNegInf ? 0.f : fabsf(score));
        }
      }
      const int mine = i16 >> shift;
      auto ranked = [&](auto v) {      // groups before mine
        int rank = 0;
        for (int j = 0; j < a.groups; ++j) {
          const auto o = __shfl(v, (lane & 48) + j * run, 64);
          rank += (o > v || (o == v && j < mine)) ? 1 : 0;
        }
        return rank;
      };
      kept = ranked(score) < a.top_groups;
      const float worst = row_min(kept ? score : -kNegInf);
      const float best = row_max(kept ? kNegInf : score);
      // float32 maxima of exact keys decide exactly; sums and biased keys only beyond tol
      if ((BIAS || a.group_top == 2) && __any(on && best != kNegInf && worst - best <= tol)) {
        double d1 = kNegInfD, d2 = kNegInfD;
        const double total = SOFTMAX ? softmax_sum() : 0.0;
#pragma unroll 1
        for (int c = 0; c < EPL; ++c) {
          const double x = value(e0 + c, total);
          d2 = fmax(fmin(d1, x), d2);
          d1 = fmax(d1, x);
        }
        for (int d = 1; d < run; d <<= 1) {
          const double o1 = __shfl_xor(d1, d, 64), o2 = __shfl_xor(d2, d, 64);
          d2 = fmax(fmin(d1, o1), fmax(d2, o2));
          d1 = fmax(d1, o1);
        }
        kept = ranked(a.group_top == 2 && d2 != kNegInfD ? d1 + d2 : d1) < a.top_groups;
      }
    }
    // Key as a fixed-point number from 1; 0 for a masked (or far lower) one and for any of a
    // group that does not stay. Exact keys keep their order exactly; with a bias one fused
    // multiply-add will do, whose rounding of the offset `near` covers.
    const float add = kept ? (BIAS ? float(near) + 1.f - lo * f : 1.f) : 0.f;
    if (!kept) f = 0.f;
    auto fix = [&](float k) {
      if (BIAS) return saturating_uint(fmaf(k, f, add));
      return saturating_uint(fmaf(k - lo, f, add));
    };
    uint32_t v[kCols];
    const uint32_t id0 = kIdMask - uint32_t(e0);
#pragma unroll
    for (int c = 0; c < kCols; ++c) v[c] = c < EPL ? (fix(key[c < EPL ? c : 0]) << 10) | (id0 - c) : 0u;
    if (E != kRow) {     // an empty place comes behind every masked expert
      const int per_group = run * EPL - a.pad, in = (i16 & (run - 1)) * EPL;
      const int there = i16 >> shift < a.groups ? per_group - in : 0;
#pragma unroll
      for (int c = 0; c < EPL; ++c) v[c] = c < there ? v[c] : 0u;
    }
    // the lane's best 8, then the token's
    uint32_t lost = 0;
#pragma unroll
    for (int c = 0; c < kCols; c += 8) sort8(v + c);
#pragma unroll
    for (int c = 8; c < kCols; c += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lost = max(lost, min(v[i], v[c + 7 - i]));
        v[i] = max(v[i], v[c + 7 - i]);
      }
      bitonic8(v);
    }
    // the token's: KL times the best head of its lanes' lists, which then move up
    uint32_t found[KL];
#pragma unroll
    for (int k = 0; k < KL; ++k) {
      found[k] = row_max_u(v[0]);
      const bool mine = v[0] == found[k];
#pragma unroll
      for (int i = 0; i < kHeads && i + k < KL; ++i) v[i] = mine ? (i + 1 < kHeads ? v[i + 1] : 0u) : v[i];
    }
    lost = row_max_u(max(lost, v[0]));
    if (i16 == 0) {
#pragma unroll
      for (int i = 0; i < KL; ++i) s_list[w][t][i] = found[i];
    }
    wave_sync();
    // lane j of a token: its j-th best (from 0) and the next, by place
    const int j = min(i16, KL - 1);
    // (a list of fewer than 8 experts ends in zeros, whose id is cut to a place in the row)
    auto place_of = [&](uint32_t x) { return min(int(kIdMask - (x & kIdMask)), kRow - 1); };
    const uint32_t wl = s_list[w][t][a.K - 1], last = wl >> 10;      // the last chosen
    // the last choice, or a rival within the error below it, may lie under the range
    unsure |= tail && last <= near;
    const uint32_t least = s_list[w][t][KL - 1];
    // a lane has more of the best KL than its list holds
    if (KL > kHeads) unsure |= lost > least && (lost > kIdMask || last == 0);
    bool close = false;
    {
      const uint32_t wj = s_list[w][t][j], wn = s_list[w][t][min(j + 1, KL - 1)];
      const uint32_t qj = wj >> 10, qn = wn >> 10;
      if (j + 1 < KL && qj != 0 && qj - qn <= near && (j < a.K || last - qn <= near)) {
        // too close to tell, unless equal
        const int idj = place_of(wj), idn = place_of(wn);
        close = row[idn] != row[idj] || (BIAS && s_bias[idn] != s_bias[idj]);
      }
    }
    // this lane's experts one by one: calls f(fixed-point key, logit, place)
    auto scan = [&](auto f) {
#pragma unroll 1
      for (int c = 0; c < EPL; c += 4) {
        float l[4], k[4];
        logits4(c, l);
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = l[i];
        keys4(c, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) f(fix(l[i] == kNegInf ? kNegInf : k[i]), l[i], e0 + c + i);
      }
    };
    // experts that did not make the list but are as near to the last chosen one
    if (last != 0 && last - (lost >> 10) <= near) {
      const int idl = place_of(wl);
      const float ll = row[idl], bl = BIAS ? s_bias[idl] : 0.f;
      scan([&](uint32_t q, float l, int e) {
        if (((q << 10) | (kIdMask - uint32_t(e))) < least && q != 0 && last - min(q, last) <= near)
          close |= l != ll || (BIAS && s_bias[e] != bl);
      });
    }
    close = row_or(close ? 1u : 0u) != 0;
    if (__any(on && close)) {
      // Every expert that could be among the best K, one per lane, in the order of float64
      // keys; more than 16 of them are left to route_token.
      const double total = SOFTMAX && BIAS ? softmax_sum() : 0.0;
      const uint32_t bar = last > near ? last - near : 1;
      int n = 0;
      scan([&](uint32_t q, float, int) { n += q >= bar ? 1 : 0; });
      int incl = n;
      for (int d = 1; d < 16; d <<= 1) {
        const int o = __shfl_up(incl, d, 16);
        if (i16 >= d) incl += o;
      }
      const int count = __shfl(incl, 15, 16);
      int at = incl - n;
      scan([&](uint32_t q, float, int e) {
        if (q >= bar) {
          if (at < 16) s_cand[w][t][at] = (q << 10) | (kIdMask - uint32_t(e));
          ++at;
        }
      });
      wave_sync();
      const uint32_t mine = i16 < count ? s_cand[w][t][i16] : 0;
      const int e = place_of(mine);
      const double x = i16 >= count ? kNegInfD : BIAS ? value(e, total) : double(row[e]);
      int rank = 0;
      for (int r = 0; r < 16; ++r) {
        const double o = __shfl(x, r, 16);
        const int oe = __shfl(e, r, 16);
        rank += r < count && (o > x || (o == x && oe < e)) ? 1 : 0;
      }
      if (close && count <= 16 && i16 < count && rank < a.K) s_list[w][t][rank] = mine;
      unsure |= close && count > 16;
      wave_sync();
    }
    const uint32_t wj = s_list[w][t][j], qj = wj >> 10;
    const int id = place_of(wj);
    const float lj = row[id];
    uint32_t again = row_or(unsure && on ? 1u : 0u);
    // gates
    const bool live = on && i16 < a.K && qj != 0;
    float gate;
    if (!a.renorm) {
      gate = SOFTMAX ? expf(lj - top) / sum : 1.0f / (1.0f + expf(-lj));
      gate = live ? gate : 0.f;
    } else {
      const float m = row_max(live ? lj : kNegInf);
      if (SOFTMAX) gate = expf(lj - m);
      else gate = m >= 0.f ? 1.0f / (1.0f + expf(-lj)) : expf(lj - m) / (1.0f + expf(lj));
      gate = live ? gate : 0.f;
      const float total = row_sum(gate);
      gate = total > 0.f ? gate / total : 0.f;
    }
    if (on && i16 < a.K && !again) {
      a.ids[(g0 + t) * a.K + i16] = id - ((id / EPL) >> shift) * a.pad;
      a.gates[(g0 + t) * a.K + i16] = gate * a.scale;
    }
    wave_sync();
    for (uint64_t todo = __ballot(again != 0 && i16 == 0); todo; todo &= todo - 1) {
      const int64_t g = g0 + __builtin_ctzll(todo) / 16;
      route_token(a, g, reinterpret_cast<double*>(rows));
    }
  }
}

template <int EPL, int KL>
static void launch_packed(const RouteArgs& a, int grid, hipStream_t strm) {
  const int threads = kRouteWaves * 64;
  if (a.softmax && a.bias) route_packed_kernel<EPL, KL, true, true><<<grid, threads, 0, strm>>>(a);
  else if (a.softmax) route_packed_kernel<EPL, KL, true, false><<<grid, threads, 0, strm>>>(a);
  else if (a.bias) route_packed_kernel<EPL, KL, false, true><<<grid, threads, 0, strm>>>(a);
  else route_packed_kernel<EPL, KL, false, false><<<grid, threads, 0, strm>>>(a);
}

// Places per lane that have an instance, and a list of 8 or 16.
static int packed_places(int epl, int K) {
  if (K > 8) return epl <= 8 ? 8 : epl <= 16 ? 16 : epl <= 32 ? 32 : 64;
  return epl <= 32 ? epl : epl <= 48 ? 48 : 64;
}

static void launch_packed_any(const RouteArgs& a, hipStream_t strm) {
  const int grid = (a.N + kRouteWaves * kTokens - 1) / (kRouteWaves * kTokens);
  if (a.K > 8) {
    switch (a.epl) {
      case 8: launch_packed<8, 16>(a, grid, strm); break;
      case 16: launch_packed<16, 16>(a, grid, strm); break;
      case 32: launch_packed<32, 16>(a, grid, strm); break;
      default: launch_packed<64, 16>(a, grid, strm); break;
    }
    return;
  }
  switch (a.epl) {
    case 4: launch_packed<4, 8>(a, grid, strm); break;
    case 8: launch_packed<8, 8>(a, grid, strm); break;
    case 12: launch_packed<12, 8>(a, grid, strm); break;
    case 16: launch_packed<16, 8>(a, grid, strm); break;
    case 20: launch_packed<20, 8>(a, grid, strm); break;
    case 24: launch_packed<24, 8>(a, grid, strm); break;
    case 28: launch_packed<28, 8>(a, grid, strm); break;
    case 32: launch_packed<32, 8>(a, grid, strm); break;
    case 48: launch_packed<48, 8>(a, grid, strm); break;
    default: launch_packed<64, 8>(a, grid, strm); break;
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
  bool bf16;
};

// 16 lanes per token, four tokens per wavefront. The row (zeros, or -s sum g dg of the dense
// form) is put into LDS, the choices' gradients are added there, and the row is written out:
// 4 experts to a vector where rows are whole vectors (VEC), else one by one. Each logit is read
// once and each gradient written once; 32768 x 128 softmax bf16 without renorm: 6.8 us for
// 20 MB (2.9 TB/s; 4.2 us at the rate of a large copy, of which a launch this short spends
// the rest on starting and draining), one wavefront per token 25 us.
template <int EPL, bool DENSE, bool VEC>
__global__ __launch_bounds__(kRouteWaves * 64) void route_backward_kernel(RouteBackwardArgs a) {
  constexpr int kRow = 16 * EPL;
  constexpr float kLog2e = 1.44269504f;
  __shared__ __align__(16) float s_row[kRouteWaves][kTokens * kRow];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, t = lane >> 4, i16 = lane & 15;
  const int64_t g = (int64_t(blockIdx.x) * kRouteWaves + w) * kTokens + t;
  const bool on = g < a.N;
  float* row = s_row[w] + t * kRow;
  // this lane's vectors of 4 experts, i16, i16 + 16, ..., or its experts i16, i16 + 16, ...
  float x[EPL];
  if (DENSE && !VEC) {
#pragma unroll
    for (int c = 0; c < EPL; ++c) {
      const int e = c * 16 + i16, at = on && e < a.E ? e : 0;
      const int64_t i = (on ? g : int64_t(a.N) - 1) * a.E + at;
      float l = a.bf16 ? load_logit<true>(a.logits, i) : load_logit<false>(a.logits, i);
      if (a.bias) l = effective_logit(l, a.bias[at]);
      x[c] = on && e < a.E ? l : kNegInf;
    }
  }
  if (DENSE && VEC) {
#pragma unroll
    for (int c = 0; c < EPL; c += 4) {
      const int e = c * 16 + i16 * 4;
      float4 v = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
      if (on && e < a.E) {
        if (a.bf16) {
          const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + g * a.E + e);
          v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                          __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
        } else {
          v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + g * a.E + e);
        }
        if (a.bias) {
          const float4 b = *reinterpret_cast<const float4*>(a.bias + e);
          v = make_float4(effective_logit(v.x, b.x), effective_logit(v.y, b.y),
                          effective_logit(v.z, b.z), effective_logit(v.w, b.w));
        }
      }
      x[c] = v.x; x[c + 1] = v.y; x[c + 2] = v.z; x[c + 3] = v.w;
    }
  }
  // the choices, 16 at a time, K <= 32
  int id[2];
  float gate[2], d[2], mean = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = h * 16 + i16;
    id[h] = -1;
    gate[h] = d[h] = 0.f;
    if (on && k < a.K) {
      id[h] = a.ids[g * a.K + k];
      if (id[h] < 0 || id[h] >= a.E) id[h] = -1;
      gate[h] = id[h] >= 0 ? a.gates[g * a.K + k] : 0.f;
      d[h] = gate[h] != 0.f ? a.dgates[g * a.K + k] : 0.f;   // a gate of 0 has no gradient
    }
    // q exactly 1 for a lone choice, whose gradient is then exactly 0
    mean += (a.renorm ? gate[h] / a.scale : gate[h]) * d[h];
  }
  mean = row_sum(mean);
  if (DENSE) {
    float m = kNegInf, sum = 0.f;
    bool nan = false;
#pragma unroll
    for (int c = 0; c < EPL; ++c) {
      m = max2(m, x[c]);
      nan |= x[c] != x[c];
    }
    m = row_max(m);
    m = m == kNegInf ? 0.f : m;
#pragma unroll
    for (int c = 0; c < EPL; ++c) {
      x[c] = __builtin_amdgcn_exp2f((x[c] - m) * kLog2e);
      sum += x[c];
    }
    sum = row_sum(nan ? __builtin_nanf("") : sum);
    const float f = sum != 0.f ? -mean / sum : 0.f;
#pragma unroll
    for (int c = 0; c < EPL; ++c) x[c] *= f;
  } else {
#pragma unroll
    for (int c = 0; c < EPL; ++c) x[c] = 0.f;
  }
  if (VEC) {
#pragma unroll
    for (int c = 0; c < EPL; c += 4)
      *reinterpret_cast<float4*>(row + c * 16 + i16 * 4) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
  } else {
#pragma unroll
    for (int c = 0; c < EPL; ++c) row[c * 16 + i16] = x[c];
  }
  wave_sync();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (id[h] < 0) continue;
    float v = gate[h] * (a.renorm ? d[h] - mean : d[h]);
    if (!a.softmax && gate[h] != 0.f) {
      const float l = a.bf16 ? load_logit<true>(a.logits, g * a.E + id[h])
                             : load_logit<false>(a.logits, g * a.E + id[h]);
      v /= 1.0f + expf(l);   // 1 - sigmoid
    }
    // lanes of one instruction add in lane order, so a repeated id is summed in k order
    atomicAdd(row + id[h], v);
  }
  wave_sync();
  if (!on) return;
  if (!VEC) {
#pragma unroll
    for (int c = 0; c < EPL; ++c) {
      const int e = c * 16 + i16;
      if (e >= a.E) continue;
      const float v = row[e];
      if (a.bf16) static_cast<uint16_t*>(a.dlogits)[g * a.E + e] = uint16_t(bf16_rne_any(v));
      else static_cast<float*>(a.dlogits)[g * a.E + e] = v;
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < EPL; c += 4) {
    const int e = c * 16 + i16 * 4;
    if (e >= a.E) continue;
    const float4 v = *reinterpret_cast<const float4*>(row + e);
    if (a.bf16) {
      uint2 u;
      u.x = bf16_rne_any(v.x) | (bf16_rne_any(v.y) << 16);
      u.y = bf16_rne_any(v.z) | (bf16_rne_any(v.w) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dlogits) + g * a.E + e) = u;
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + g * a.E + e) = v;
    }
  }
}

template <int EPL>
static void launch_backward(const RouteBackwardArgs& a, int grid, hipStream_t strm) {
  const int threads = kRouteWaves * 64;
  const bool dense = a.softmax && !a.renorm;
  if (a.E % 4 == 0) {
    if (dense) route_backward_kernel<EPL, true, true><<<grid, threads, 0, strm>>>(a);
    else route_backward_kernel<EPL, false, true><<<grid, threads, 0, strm>>>(a);
  } else {
    if (dense) route_backward_kernel<EPL, true, false><<<grid, threads, 0, strm>>>(a);
    else route_backward_kernel<EPL, false, false><<<grid, threads, 0, strm>>>(a);
  }
}

static void launch_backward_any(const RouteBackwardArgs& a, hipStream_t strm) {
  const int grid = (a.N + kRouteWaves * kTokens - 1) / (kRouteWaves * kTokens);
  const int epl = (a.E + 63) / 64 * 4;
  if (epl <= 4) launch_backward<4>(a, grid, strm);
  else if (epl <= 8) launch_backward<8>(a, grid, strm);
  else if (epl <= 16) launch_backward<16>(a, grid, strm);
  else if (epl <= 24) launch_backward<24>(a, grid, strm);
  else if (epl <= 32) launch_backward<32>(a, grid, strm);
  else launch_backward<64>(a, grid, strm);
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
  RouteArgs a{logits, bias, topk_idx, gates, N, s.E, s.K, router->groups, router->top_groups,
              router->group_top, router->score == MOONEP_SOFTMAX, router->renorm != 0,
              router->scale, router->dtype == MOONEP_BF16, 0, 16, 0};
  // packed: a choice has a lane, and every group its lanes and their registers
  const int per_group = s.E / a.groups;
  while (a.run > 0 && a.run * a.groups > 16) a.run /= 2;
  if (a.run > 0) a.epl = packed_places((per_group + 4 * a.run - 1) / (4 * a.run) * 4, s.K);
  a.pad = a.run * a.epl - per_group;
  if (s.K <= 16 && a.run > 0 && a.pad >= 0) {
    for (int n0 = 0; n0 < N; n0 += kLaunchTokens) {
      RouteArgs c = a;
      c.N = N - n0 < kLaunchTokens ? N - n0 : kLaunchTokens;
      c.logits = static_cast<const char*>(logits) + int64_t(n0) * s.E * (a.bf16 ? 2 : 4);
      c.ids += int64_t(n0) * s.K;
      c.gates += int64_t(n0) * s.K;
      launch_packed_any(c, as_stream(stream));
      if (launch_status()) return MOONEP_EHIP;
      if (N - n0 <= kLaunchTokens) break;     // n0 would pass 2^31
    }
    return MOONEP_OK;
  }
  const int64_t blocks = (int64_t(N) + kRouteWaves - 1) / kRouteWaves;
  const int grid = int(blocks < 65536 ? blocks : 65536);
  route_kernel<<<grid, kRouteWaves * 64, 0, as_stream(stream)>>>(a);
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
                            router->score == MOONEP_SOFTMAX, router->renorm != 0, router->scale,
                            router->dtype == MOONEP_BF16};
  for (int n0 = 0; n0 < N; n0 += kLaunchTokens) {
    RouteBackwardArgs c = a;
    c.N = N - n0 < kLaunchTokens ? N - n0 : kLaunchTokens;
    const int64_t at = int64_t(n0) * s.E * (a.bf16 ? 2 : 4), k = int64_t(n0) * s.K;
    c.logits = static_cast<const char*>(logits) + at;
    c.dlogits = static_cast<char*>(dlogits) + at;
    c.ids += k;
    c.gates += k;
    c.dgates += k;
    launch_backward_any(c, as_stream(stream));
    if (launch_status()) return MOONEP_EHIP;
    if (N - n0 <= kLaunchTokens) break;     // n0 would pass 2^31
  }
  return MOONEP_OK;
}
