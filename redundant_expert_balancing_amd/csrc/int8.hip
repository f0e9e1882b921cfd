// Experts in 8-bit integers on gfx950: token rows and weights as whole numbers with a scale per
// row and per column, prefetch and transposition of such weights, the grouped and the dense
// product on them (v_mfma_i32_16x16x64_i8), and the gradient rows for the product back through
// frozen weights. Layouts: moonep.h, "Experts in 8-bit integers"; a 16-column x 64-k block of a
// weight is 1 KiB in the order in which a wavefront's lanes take the operand.
#include <type_traits>

#include "common.h"
#include "lds_dma.h"

namespace moonep {

constexpr int kIntThreads = 256;
constexpr int kIntMaxK = 131072;             // 127 * 127 * 131072 < 2^31: sums stay exact
constexpr int kIntMaxCols = 1 << 24;
constexpr float kIntLeast = 0x1p-126f;       // the smallest scale
constexpr uint32_t kIntNan = 0x7FC00000u;
constexpr int kIntFewRows = 2048;            // fewer rows: as many wavefronts each as it takes
constexpr int kIntChunk = 16;                // positions in a row of the gradient's rounding
// Infinity Cache, 256 MiB: gradient rows beyond it are stored past the caches. 262144 rows of 4096
// 504 -> 456 us, and the product that reads them loses nothing; in int_quantize_kernel 268 MB (65536
// rows of 4096) made no difference, and 117 MB (16384 of 7168) cost the product 25 us.
constexpr int64_t kIntCache = int64_t(1) << 28;
typedef float v4f_t __attribute__((ext_vector_type(4)));

// ---- rounding to 8 bits
//
// Scale of magnitudes up to amax_bits (as bits; integer order ranks Inf and NaN highest).
// The quotient by 127 is the product with the rounded reciprocal and one correction by the exact
// remainder: correctly rounded for every float32 whose quotient is a normal number (checked for
// all mantissas).
__device__ inline float int_scale(uint32_t amax_bits) {
  constexpr float kInv = 1.0f / 127.0f;
  const float m = __uint_as_float(amax_bits), q = m * kInv;
  const float s = fmaxf(fmaf(fmaf(-q, 127.0f, m), kInv, q), kIntLeast);
  return amax_bits >= 0x7F800000u ? __uint_as_float(kIntNan) : s;
}
// 1 / s, off by a unit in the last place (s is normal, and so is this)
__device__ inline float int_inverse(float s) { return __builtin_amdgcn_rcpf(s); }

// The whole number nearest to the exact x / s, ties to even; inv = 1 / s in float32. x * inv is
// off by a few units in its last place, so its nearest whole number is at most one away. The
// remainder x - q s is exact in one FMA: it is a multiple of both numbers' last places and at
// most about s (and a multiple of 2^-149 at the low end). It decides, so the choice is that of
// exact arithmetic and does not depend on how the quotient was formed.
__device__ inline int int_round(float x, float s, float inv) {
  const float q = rintf(x * inv), r = fmaf(-q, s, x), twice = 2.0f * fabsf(r);
  int w = int(q);
  if (twice > s || (twice == s && (w & 1))) w += r > 0.0f ? 1 : -1;
  return w;
}

__device__ inline uint32_t int_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The low bytes of four words
__device__ inline uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(b, a, 0x0c0c0400u) | __builtin_amdgcn_perm(d, c, 0x04000c0cu);
}

// N whole numbers as bytes; STREAM: past the caches
template <int N, bool STREAM = false>
__device__ inline void int_store(int8_t* at, const int* w) {
  uint32_t p[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) p[i] = low_bytes(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  typedef typename std::conditional<N == 8, uint64_t, uint32_t>::type word;
  word all = p[0];
  if constexpr (N == 8) all |= word(p[1]) << 32;
  if constexpr (STREAM) __builtin_nontemporal_store(all, reinterpret_cast<word*>(at));
  else *reinterpret_cast<word*>(at) = all;
}

// N values of a row with scale s, rounded and stored. Adding 1.5 * 2^23 to the quotient leaves
// the whole number in the sum's low bits, so a value takes three more operations than its
// packing: the sum, the whole number back, and the remainder, whose largest magnitude tells
// whether any value of the lane is so near a border that the sum may have chosen the wrong side
// (then, rarely, all of them are rounded the long way). 65536 bfloat16 rows of 4096: 146 us with
// every value the long way, bound by its instructions; 127 us so.
template <int N, bool STREAM = false>
__device__ inline void int_round_store(int8_t* at, const float* v, float s, float inv) {
  constexpr float kMagic = 0x1.8p23f;
  int w[N];
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = fmaf(v[i], inv, kMagic);
    most = fmaxf(most, fabsf(fmaf(kMagic - t, s, v[i])));
    w[i] = int(__float_as_uint(t));
  }
  if (2.0f * most >= s) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = int_round(v[i], s, inv);
  }
  if (s != s) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 0;
  }
  int_store<N, STREAM>(at, w);
}

// The largest of a wavefront's values, uniform: within rows of 16 lanes by DPP, then of the rows.
__device__ inline uint32_t wave_max(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));   // quad_perm 1,0,3,2
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));   // quad_perm 2,3,0,1
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xF, 0xF, false)));  // row_half_mirror
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 0xF, 0xF, false)));  // row_mirror
  const uint32_t a = __builtin_amdgcn_readlane(int(v), 0), b = __builtin_amdgcn_readlane(int(v), 16);
  const uint32_t c = __builtin_amdgcn_readlane(int(v), 32), d = __builtin_amdgcn_readlane(int(v), 48);
  return max(max(a, b), max(c, d));
}

// The largest m of a row that WPR wavefronts share (a whole workgroup, unless it is one
// wavefront), uniform; part: WPR words of LDS, not written again before every wavefront has read
// them.
template <int WPR>
__device__ inline uint32_t row_max(uint32_t m, uint32_t* part) {
  m = wave_max(m);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int i = 0; i < WPR; ++i) m = max(m, part[i]);
    m = __builtin_amdgcn_readfirstlane(int(m));
  }
  return m;
}

// A row's 16-byte vector: 8 bfloat16 or 4 float32.
template <bool BF16>
struct RowVec {
  static constexpr int N = BF16 ? 8 : 4;
  uint4 raw;
  __device__ float at(int i) const {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
    if (BF16) return __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
    return __uint_as_float(u[i]);
  }
};

// Threads of a workgroup whose rows are shared by WPR wavefronts
constexpr int int_threads(int wpr) { return wpr == 1 ? kIntThreads : 64 * wpr; }

// A row is held in registers between the maximum and the rounding: WPR wavefronts per row, VPL
// vectors a lane; VPL 0: rows too wide for that are read twice. Bound by HBM: 65536 bfloat16 rows of
// 4096 123-127 us, 0.81 GB at 6.5 TB/s; 16384 of 7168 55-58 us, 6.3 TB/s (one wavefront a row, 16
// vectors a lane: 116); one row of 4096 2-4 us, most of it the launch (one wavefront: 6.8).
template <bool BF16, int WPR, int VPL>
__global__ __launch_bounds__(int_threads(WPR)) void int_quantize_kernel(const uint4* __restrict__ src,
                                                                        int64_t rows, int nvec, int nout,
                                                                        int8_t* __restrict__ q,
                                                                        float* __restrict__ scales) {
  typedef RowVec<BF16> V;
  constexpr int TPR = 64 * WPR, RPG = int_threads(WPR) / TPR;      // threads per row, rows per workgroup
  __shared__ uint32_t part[2][WPR];
  const int t = threadIdx.x % TPR;
  int turn = 0;
  for (int64_t r = blockIdx.x * int64_t(RPG) + threadIdx.x / TPR; r < rows; r += int64_t(gridDim.x) * RPG) {
    const uint4* in = src + r * nvec;
    int8_t* out = q + r * nout * V::N;
    V held[VPL ? VPL : 1];
    uint32_t m = 0;
    auto take = [&](int c) { return V{c < nvec ? in[c] : make_uint4(0, 0, 0, 0)}; };
    auto most = [&](const V& v) {
#pragma unroll
      for (int i = 0; i < V::N; ++i) m = max(m, int_mag(v.at(i)));
    };
    if constexpr (VPL > 0) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) held[i] = take(t + TPR * i);
#pragma unroll
      for (int i = 0; i < VPL; ++i) most(held[i]);
    } else {
      for (int c = t; c < nvec; c += TPR) most(take(c));
    }
    const float s = int_scale(row_max<WPR>(m, part[turn]));
    turn ^= 1;
    const float inv = int_inverse(s);
    auto put = [&](int c, const V& h) {
      float v[V::N];
#pragma unroll
      for (int i = 0; i < V::N; ++i) v[i] = h.at(i);
      if (c < nout) int_round_store<V::N>(out + c * V::N, v, s, inv);
    };
    if constexpr (VPL > 0) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) put(t + TPR * i, held[i]);
    } else {
      for (int c = t; c < nout; c += TPR) put(c, take(c));
    }
    if (t == 0) scales[r] = s;
  }
}

// ---- gradient rows
struct IntGradArgs {
  const uint4* src;
  const int32_t* src_index;
  const float* gates;
  const float* ws;
  const int32_t* cu;
  int8_t* q;
  float* scales;
  int R, E, B, SK, K, nvec, nout, wscols;
  int64_t NK;
  int chunk;
};

// The view row of position pos of a rank: the last i with cu[i] <= pos, or -1 behind the last
// row and ahead of the first. Each step looks at 64 entries at once.
__device__ inline int segment_of(const int32_t* cu, int EB, int pos, int lane) {
  int lo = 0, n = EB + 1;
  while (n > 1) {
    const int stride = (n + 63) / 64;
    const int at = lane * stride;
    const uint64_t le = __ballot(at < n && cu[min(lo + at, EB)] <= pos);
    if (le == 0) return -1;
    const int c = 63 - __clzll(le);
    lo += c * stride;
    n = min(stride, n - c * stride);
  }
  return lo < EB ? lo : -1;
}

// The upstream row of a position times the scales of its expert's columns, rounded as
// int_quantize_kernel rounds. WPR wavefronts (or each wavefront alone) take a chunk of positions
// in a row: what is looked up per position is looked up by a lane each beforehand, the
// columns' scales stay in registers while the expert is the same, and the next row is on its
// way while one is rounded. VPL as there. 262144 positions of 32768 tokens, 4096 wide: 456 us,
// 1.07 GB written and 2.1 GB of rows read (0.27 GB of them from HBM) at 7 TB/s; 504 us if the
// output goes through the caches, 302 with every position on one token's row (6.5 vector
// instructions a value take 0.2 ms of it; the maximum of magnitudes as integers, one more: 318).
// 128 shares of every expert in turn, so that the workgroups of an XCD read the same tokens:
// 464 us, nine tenths of the requests still miss its L2.
template <bool BF16, int WPR, int VPL, bool STREAM>
__global__ __launch_bounds__(int_threads(WPR)) void int_quantize_grad_kernel(IntGradArgs a) {
  typedef RowVec<BF16> V;
  constexpr int TPR = 64 * WPR, RPG = int_threads(WPR) / TPR, HELD = VPL ? VPL : 1;
  static_assert(kIntChunk <= 64, "a lane per position of a chunk");
  __shared__ uint32_t part[2][WPR];
  const int lane = threadIdx.x & 63, t = threadIdx.x % TPR;
  int turn = 0;
  for (int64_t begin = (blockIdx.x * int64_t(RPG) + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR)) * a.chunk;
       begin < a.NK; begin += int64_t(gridDim.x) * RPG * a.chunk) {
    const int count = int(min(int64_t(a.chunk), a.NK - begin));
    const int p0 = int(begin);
    // lane i: source row of position p0 + i (-1: none), its gate, and in the end its scale
    int my_row = int(uint32_t(p0) + uint32_t(lane));
    float my_gate = 1.0f, my_scale = 0.0f;
    bool my_live = false;
    if (a.src_index) {
      const int u = lane < count ? a.src_index[p0 + lane] : -1;
      const bool there = u >= 0 && u < a.NK;
      my_row = there ? u / a.K : -1;
      if (a.gates && there) my_gate = a.gates[u];
    }
    int wrow = 0;
    int64_t until = p0;             // positions before it belong to weight row wrow (-1: none)
    float ws[HELD][V::N];
    V next[HELD];
    auto source = [&](int i) { return __builtin_amdgcn_readlane(my_row, i); };
    auto fetch = [&](int row) {
      if constexpr (VPL > 0) {
        const uint4* in = a.src + int64_t(row) * a.nvec;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int c = t + TPR * i;
          next[i] = V{row >= 0 && c < a.nvec ? in[c] : make_uint4(0, 0, 0, 0)};
        }
      }
    };
    int row = source(0);
    fetch(row);
    for (int i = 0; i < count; ++i) {
      const int p = p0 + i;
      if (p >= until) {
        wrow = 0;
        until = a.NK;
        if (a.cu) {
          const int rank = p / a.SK, EB = a.E + a.B;
          const int32_t* cu = a.cu + int64_t(rank) * (EB + 1);
          const int pos = p - rank * a.SK, seg = segment_of(cu, EB, pos, lane);
          wrow = __builtin_amdgcn_readfirstlane(seg < 0 ? -1 : seg < a.E ? seg : a.E + rank * a.B + (seg - a.E));
          // outside the rows: up to the first one, or to the end of the rank
          const int end = seg >= 0 ? cu[seg + 1] : pos < cu[0] ? cu[0] : a.SK;
          until = int64_t(rank) * a.SK + __builtin_amdgcn_readfirstlane(end);
        }
        if constexpr (VPL > 0) {
          const v4f_t* from = reinterpret_cast<const v4f_t*>(a.ws + int64_t(max(wrow, 0)) * a.wscols);
#pragma unroll
          for (int k = 0; k < VPL; ++k)
#pragma unroll
            for (int j = 0; j < V::N / 4; ++j) {
              const int c = t + TPR * k;
              const v4f_t s = c < a.nvec ? from[c * (V::N / 4) + j] : v4f_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int e = 0; e < 4; ++e) ws[k][4 * j + e] = s[e];
            }
        }
      }
      const int from_row = row;
      float v[HELD][V::N];
      if constexpr (VPL > 0) {
#pragma unroll
        for (int k = 0; k < VPL; ++k)
#pragma unroll
          for (int e = 0; e < V::N; ++e) v[k][e] = next[k].at(e) * ws[k][e];
      }
      if (i + 1 < count) {
        row = source(i + 1);
        fetch(row);
      }
      if (wrow < 0) continue;       // behind the rank's last row; uniform for the row's wavefronts
      float largest = 0.0f;      // its maximum keeps a NaN
      auto most = [&](const float* h) {
#pragma unroll
        for (int e = 0; e < V::N; ++e) largest = __builtin_elementwise_maximum(largest, fabsf(h[e]));
      };
      auto take = [&](int c, float* h) {       // VPL 0
        const bool in_row = from_row >= 0 && c < a.nvec;
        const V x{in_row ? (a.src + int64_t(from_row) * a.nvec)[c] : make_uint4(0, 0, 0, 0)};
#pragma unroll
        for (int j = 0; j < V::N / 4; ++j) {
          const v4f_t s = in_row ? reinterpret_cast<const v4f_t*>(a.ws + int64_t(wrow) * a.wscols)[c * (V::N / 4) + j]
                                 : v4f_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 4; ++e) h[4 * j + e] = x.at(4 * j + e) * s[e];
        }
      };
      if constexpr (VPL > 0) {
        if (from_row < 0)       // zeros, also where a column's scale is not a number
#pragma unroll
          for (int k = 0; k < VPL; ++k)
#pragma unroll
            for (int e = 0; e < V::N; ++e) v[k][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < VPL; ++k) most(v[k]);
      } else {
        for (int c = t; c < a.nvec; c += TPR) {
          take(c, v[0]);
          most(v[0]);
        }
      }
      const float s = int_scale(row_max<WPR>(int_mag(largest), part[turn]));
      turn ^= 1;
      const float inv = int_inverse(s);
      int8_t* out = a.q + int64_t(p) * a.nout * V::N;
      if constexpr (VPL > 0) {
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
          const int c = t + TPR * k;
          if (c < a.nout) int_round_store<V::N, STREAM>(out + c * V::N, v[k], s, inv);
        }
      } else {
        for (int c = t; c < a.nout; c += TPR) {
          take(c, v[0]);
          int_round_store<V::N, STREAM>(out + c * V::N, v[0], s, inv);
        }
      }
      if (lane == i) {
        my_live = true;
        my_scale = from_row < 0 ? 0.0f : my_gate * s;
      }
    }
    if (t < 64 && my_live) a.scales[p0 + lane] = my_scale;
  }
}

// ---- weights (set-up)
//
// A workgroup has 64 columns of one expert: their maxima over k, then blocks of 64 lanes x 16 k.
template <bool BF16>
__global__ __launch_bounds__(kIntThreads) void int_quantize_weight_kernel(const void* __restrict__ w,
                                                                          int H, int Hp, int KB, int NB,
                                                                          int8_t* __restrict__ wq,
                                                                          float* __restrict__ ws) {
  __shared__ uint32_t s_max[4][64];
  __shared__ float s_scale[64];
  const int64_t e = blockIdx.y;
  const int n0 = blockIdx.x * 64, t = threadIdx.x;
  auto value = [&](int k, int n) {
    if (k >= H || n >= Hp) return 0.0f;
    const int64_t at = (e * H + k) * Hp + n;
    return BF16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(w)[at]) << 16)
                : static_cast<const float*>(w)[at];
  };
  uint32_t m = 0;
  for (int k = t >> 6; k < H; k += 4) m = max(m, int_mag(value(k, n0 + (t & 63))));
  s_max[t >> 6][t & 63] = m;
  __syncthreads();
  if (t < 64) {
    const float s = int_scale(max(max(s_max[0][t], s_max[1][t]), max(s_max[2][t], s_max[3][t])));
    s_scale[t] = s;
    if (n0 + t < NB * 16) ws[e * NB * 16 + n0 + t] = n0 + t < Hp ? s : 0.0f;
  }
  __syncthreads();
  const int j = t >> 6, lane = t & 63, nb = n0 / 16 + j;
  if (nb >= NB) return;
  const int n = nb * 16 + (lane & 15);
  const float s = s_scale[n - n0], inv = int_inverse(s);
  for (int kb = 0; kb < KB; ++kb) {
    int v[16];
#pragma unroll
    for (int b = 0; b < 16; ++b)
      v[b] = s == s ? int_round(value(kb * 64 + 16 * (lane >> 4) + b, n), s, inv) : 0;
    int8_t* at = wq + ((e * NB + nb) * KB + kb) * 1024 + lane * 16;
    int_store<8>(at, v);
    int_store<8>(at + 8, v + 8);
  }
}

// One thread per 16 bytes of the result: lane of block (h / 16, n / 64) has column h of the
// transposed weight and 16 consecutive n, which are byte h % 16 of 16 neighbouring lanes of one
// block of the source.
__global__ __launch_bounds__(kIntThreads) void int_transpose_weight_kernel(const int8_t* __restrict__ wq,
                                                                           int KB, int NB, int KBt,
                                                                           int NBt,
                                                                           int8_t* __restrict__ wqt) {
  const int64_t e = blockIdx.y;
  const int64_t total = int64_t(NBt) * KBt * 64;
  for (int64_t i = blockIdx.x * int64_t(kIntThreads) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kIntThreads) {
    const int lane = int(i & 63), kb = int((i >> 6) % KBt), nb = int((i >> 6) / KBt);
    const int h = nb * 16 + (lane & 15), n16 = kb * 4 + (lane >> 4);     // n = 16 * n16 + b
    int v[16];
    const int8_t* from = wq + ((e * NB + min(n16, NB - 1)) * KB + h / 64) * 1024 +
                         ((h / 16) % 4) * 256 + h % 16;
#pragma unroll
    for (int b = 0; b < 16; ++b) v[b] = n16 < NB ? from[b * 16] : 0;
    int8_t* at = wqt + (e * total + i) * 16;
    int_store<8>(at, v);
    int_store<8>(at + 8, v + 8);
  }
}

// Copies of home rows into used prefetch slots, values and (svec > 0) scales in one launch.
__global__ __launch_bounds__(kIntThreads) void int_prefetch_kernel(const int32_t* __restrict__ replica,
                                                                   int RB, int E, uint4* wq,
                                                                   int64_t qvec, uint4* ws,
                                                                   int64_t svec) {
  const int64_t stride = int64_t(gridDim.x) * kIntThreads;
  const int64_t i0 = int64_t(blockIdx.x) * kIntThreads + threadIdx.x;
  for (int s = 0; s < RB; ++s) {
    const int e = replica[s];
    if (e < 0 || e >= E) continue;
    for (int64_t i = i0; i < qvec + svec; i += stride) {
      if (i < qvec) wq[(int64_t(E) + s) * qvec + i] = wq[int64_t(e) * qvec + i];
      else ws[(int64_t(E) + s) * svec + i - qvec] = ws[int64_t(e) * svec + i - qvec];
    }
  }
}

// ---- products
struct IntArgs {
  const int8_t* xq;
  const float* xs;
  const int32_t* src_index;
  const int8_t* wq;
  const float* ws;       // NULL: 1
  const float* add;      // NULL: nothing added
  float* c;
  void* act;             // SwiGLU: dtype [., W/2], and c is not written
  void* h_saved;         // SwiGLU: NULL or dtype [., W]
  int K, W, NB, KB;      // columns of the weight, blocks of 16 of them, blocks of 64 k
  int64_t NK;            // positions
  const int32_t* cu;     // NULL: NK positions, all of weight row 0
  int R, E, B, SK;
  // the tiled form
  const TileEntry* tiles;   // NULL: 256-row tiles of NK positions, all of weight row 0
  const int32_t* ntiles;
  int32_t* qcnt;            // 8 per-XCD tile-queue counters, zero at launch (NULL: static order)
  int64_t xrows;            // token rows
};

// What a product's epilogue makes of its sums.
enum IntOut { kIntFloat, kIntFloatAdd, kIntSwigluBf16, kIntSwigluF32 };
__host__ __device__ constexpr bool is_swiglu(int out) { return out == kIntSwigluBf16 || out == kIntSwigluF32; }

// (sum * row scale) * column scale, 4 columns of one row
__device__ inline v4f_t int_scaled(v4i_t acc, float sa, v4f_t sw) {
  v4f_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (float(acc[i]) * sa) * sw[i];
  return r;
}

// A sum of its own, not contracted into an FMA with the product before it
__device__ inline v4f_t added(v4f_t a, v4f_t b) {
#pragma clang fp contract(off)
  return a + b;
}

// The activation. float32 layers get swiglu_f32's bits. bfloat16 layers take the exponential and
// the reciprocal from the hardware's instructions, each off by a unit in the last place: off by at
// most (1.25 |g| + 8) * 2^-24 of the value, which the rounding to bfloat16 (2^-8) covers, or
// |g u| * 2^-126 where the reciprocal falls below the normal numbers. The exponent's share is 1.23 |g|:
// the product g * log2(e) is rounded (1) and the constant lies 0.224 * 2^-24 below log2(e). It takes a
// third of swiglu_f32's instructions, with which a tile's epilogue took half as long as its
// products at a reduction of 4096.
template <int OUT>
__device__ inline float int_swiglu(float g, float u) {
  if constexpr (OUT == kIntSwigluF32) return swiglu_f32(g, u);
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -0x1.715476p0f)) * u;
}

// Two values rounded to bfloat16 (nearest even, a NaN stays one)
typedef float v2f_t __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf_t __attribute__((ext_vector_type(2)));
__device__ inline uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f_t{a, b}, v2bf_t));
}

template <int OUT>
__device__ inline void store4(void* base, int64_t at, v4f_t v) {
  if constexpr (OUT == kIntSwigluBf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) =
        make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
  else
    *reinterpret_cast<v4f_t*>(static_cast<float*>(base) + at) = v;
}

// ---- few rows per expert: no list of work. Work items are (share of the rows, segment of the
// view, two blocks of 16 columns), dealt out to the workgroups in turn; a workgroup's threads
// look up one item's cu_seqlens each and list the ones that have rows. A workgroup's eight
// wavefronts take blocks of 16 rows; where there are fewer blocks, the wavefronts of a block
// share its k-blocks in turn and their sums are added. Operands go straight to registers, four
// blocks of 64 k at a time. The call is bound by reading each touched expert's weights once: 16
// tokens, K = 8, 256 experts, H = 4096, H' = 1536: 114 us, 0.63 GB at 5.6 TB/s; 64 tokens, 128
// experts, H = 4096, 2H' = 2816: 237 us, 6.1 TB/s. For one token (12 us, 50 MB) and dense products
// (1 x 2048 x 7168: 4.4 us, 15 MB) its latency counts: two blocks and eight wavefronts took 12.1 and
// 4.4 us, four and four 15.1 and 5.5, one and eight 13.2 and 4.4; 16 tokens 114, 112, 117.
constexpr int kIntRows = 64;      // rows at a time
constexpr int kIntBlocks = 2, kIntDepth = 4, kIntWaves = 8;

// Block j of item t: with SwiGLU a gate block and its up block, 32 columns further.
template <int OUT>
__device__ inline int item_block(int t, int j) {
  return is_swiglu(OUT) ? 4 * (t >> 1) + (t & 1) + 2 * j : 2 * t + j;
}

template <int OUT>
__device__ inline void int_few_rows(const IntArgs& a, int rowbase_v, int wrow_v, int m0_v, int n,
                                    int t_v, v4i_t (*s_part)[kIntBlocks][64]) {
  constexpr int J = kIntBlocks, U = kIntDepth, WAVES = kIntWaves;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kb = lane >> 4, r16 = lane & 15;
  const int rowbase = __builtin_amdgcn_readfirstlane(rowbase_v);
  const int wrow = __builtin_amdgcn_readfirstlane(wrow_v);
  const int m0 = __builtin_amdgcn_readfirstlane(m0_v), t = __builtin_amdgcn_readfirstlane(t_v);
  const int rows = __builtin_amdgcn_readfirstlane(min(kIntRows, n - m0));
  // wavefronts per block of rows, at least two
  const int split = rows <= 16 ? WAVES : rows <= 32 ? WAVES / 2 : WAVES / 4;
  const int part = w % split, r0 = w / split * 16;
  const bool work = r0 < rows;    // uniform
  const int64_t pos = int64_t(rowbase) + m0 + r0 + r16;
  bool in = work && r0 + r16 < rows;
  const bool store = in && part == 0;
  int64_t arow = pos;
  v4i_t acc[J];
#pragma unroll
  for (int j = 0; j < J; ++j) acc[j] = v4i_t{0, 0, 0, 0};
  float sa = 0.0f;
  v4f_t sw[J];
  if (work) {
    const v4i_t* wq[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t blk = int64_t(wrow) * a.NB + min(item_block<OUT>(t, j), a.NB - 1);
      wq[j] = reinterpret_cast<const v4i_t*>(a.wq) + lane + blk * a.KB * 64;
      sw[j] = a.ws ? *reinterpret_cast<const v4f_t*>(a.ws + blk * 16 + 4 * kb) : v4f_t{1.f, 1.f, 1.f, 1.f};
    }
    // a wavefront takes runs of U blocks; weights first, whose addresses wait for nothing
    v4i_t fa[U], fb[U][J];
    auto weights = [&](int c0) {
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < J; ++j)
          fb[k][j] = c0 + k < a.KB ? wq[j][(c0 + k) * 64] : v4i_t{0, 0, 0, 0};    // uniform
    };
    if (part * U < a.KB) weights(part * U);
    if (a.src_index) {
      const int u = in ? a.src_index[pos] : -1;
      in = u >= 0 && u < a.NK;
      arow = in ? u / a.K : 0;
    }
    if (in) sa = a.xs[arow];
    const v4i_t* xq = reinterpret_cast<const v4i_t*>(a.xq) + arow * a.KB * 4 + kb;
    for (int c0 = part * U; c0 < a.KB; c0 += split * U) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        fa[k] = c0 + k < a.KB && in ? xq[(c0 + k) * 4] : v4i_t{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < J; ++j)      // operands swapped: a lane holds 4 columns of one row
          acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[k][j], fa[k], acc[j], 0, 0, 0);
      if (c0 + split * U < a.KB) weights(c0 + split * U);
    }
  }
  if (part > 0)
#pragma unroll
    for (int j = 0; j < J; ++j) s_part[w - 1][j][lane] = acc[j];
  __syncthreads();
  if (part == 0)
    for (int o = 1; o < split; ++o)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[j] += s_part[w + o - 1][j][lane];
  __syncthreads();     // read before the next entry's sums
  if (!store) return;
  v4f_t v[J];
  int col[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    col[j] = item_block<OUT>(t, j) * 16 + 4 * kb;
    v[j] = int_scaled(acc[j], sa, sw[j]);
  }
  if constexpr (!is_swiglu(OUT)) {
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (col[j] < a.W) {
        const int64_t at = pos * a.W + col[j];
        if constexpr (OUT == kIntFloatAdd)
          v[j] = added(v[j], *reinterpret_cast<const v4f_t*>(a.add + at));
        *reinterpret_cast<v4f_t*>(a.c + at) = v[j];
      }
  } else {
    if (a.h_saved)
#pragma unroll
      for (int j = 0; j < J; ++j) store4<OUT>(a.h_saved, pos * a.W + col[j], v[j]);
#pragma unroll
    for (int j = 0; j < J / 2; ++j) {
      v4f_t s;
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = int_swiglu<OUT>(v[j][i], v[j + J / 2][i]);
      // gate column c stands for intermediate column 32 * (c / 64) + c % 32
      store4<OUT>(a.act, pos * (a.W / 2) + col[j] / 64 * 32 + col[j] % 32, s);
    }
  }
}

struct IntItem {
  int32_t rowbase, wrow, m0, n;
};

template <int OUT>
__global__ __launch_bounds__(kIntWaves * 64) void int_gemm_kernel(IntArgs a, int shares) {
  constexpr int J = kIntBlocks, WAVES = kIntWaves;
  constexpr int ITEMS = WAVES * 64;      // items looked up at a time
  __shared__ __align__(16) v4i_t s_part[WAVES - 1][J][64];
  __shared__ IntItem s_item[ITEMS];
  __shared__ int s_t[ITEMS];
  __shared__ int s_wave[WAVES];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int NT = (a.NB + J - 1) / J, EB = a.E + a.B;
  const int64_t segs = a.cu ? int64_t(a.R) * EB : 1;
  const int64_t total = segs * shares * NT;
  for (int64_t t0 = blockIdx.x; t0 < total; t0 += int64_t(gridDim.x) * ITEMS) {
    const int64_t t = t0 + int64_t(threadIdx.x) * gridDim.x;
    IntItem it{0, 0, 0, 0};
    int tn = 0;
    if (t < total) {
      // shares slowest: the empty ones of short segments lie together, over all CUs
      const int64_t rest = t / NT;
      const int seg = int(rest % segs), share = int(rest / segs);
      tn = int(t % NT);
      if (a.cu) {
        const int rank = seg / EB, i = seg % EB;
        const int c0 = a.cu[int64_t(rank) * (EB + 1) + i];
        it = IntItem{rank * a.SK + c0, i < a.E ? i : a.E + rank * a.B + (i - a.E), share * kIntRows,
                     a.cu[int64_t(rank) * (EB + 1) + i + 1] - c0};
      } else {
        it = IntItem{0, 0, share * kIntRows, int(a.NK)};
      }
    }
    const bool some = it.m0 < it.n;
    const uint64_t have = __ballot(some);
    if (lane == 0) s_wave[w] = __popcll(have);
    __syncthreads();
    int at = __popcll(have & ((uint64_t(1) << lane) - 1)), count = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      if (i < w) at += s_wave[i];
      count += s_wave[i];
    }
    if (some) {
      s_item[at] = it;
      s_t[at] = tn;
    }
    __syncthreads();
    for (int i = 0; i < count; ++i) {
      const IntItem te = s_item[i];
      for (int64_t m0 = te.m0; m0 < te.n; m0 += shares * kIntRows)
        int_few_rows<OUT>(a, te.rowbase, te.wrow, int(m0), te.n, s_t[i], s_part);
    }
    __syncthreads();     // the list is read before the next one
  }
}

// ---- tiled form: 256 x 256 output tiles, 8 wavefronts of 128 x 64, 128 k per step. Both operands
// go to LDS by DMA, two stages: token rows (gathered by src_index) as 128-byte rows with
// swizzled chunks, weights as the 1 KiB blocks they are stored in, which a wavefront reads back
// lane by lane. A wavefront holds the fragments of half a step (64 k) and refills them behind
// its MFMAs; the one barrier of a step comes under the MFMAs of its second half, when every read
// of its stage is done, and the DMAs of the step after next are issued between the MFMAs behind
// it (in one burst they held up the wavefront's MFMAs: 3% slower). The next tile's rows and
// scales are looked up during a tile, and its first step is loaded under the tile's epilogue.
//
// Fastest and median pass: 524288 slots of 65536 tokens, 256 experts, H = 4096, H' = 1536 2.93-2.99
// ms, 2.2 Pop/s; gate/up with SwiGLU, 262144 slots, H = 4096, 2H' = 2816, pre-activation kept
// 2.62-2.67 ms, 2.3; dense 16384 x 7168 x 4096 with SwiGLU 353-374 us, 2.6; 262144 x 4096 x 1408
// 1.40-1.44 ms, 2.1; dense 16384 x 2048 x 7168 with an added tile 298-321 us, 1.5; 65536 rows of a
// reduction of 64 to 256 to 2048 columns 90-98 us, 5.5-5.9 TB/s written. (The library's dense int8
// product with an int32 result reached 2.2 at 65536 x 4096 x 1536, 2.0 at 16384 x 7168 x 4096.) Bound
// by power and by the operands' way into LDS together: the matrix pipes are busy 0.575 of the
// cycles at 1.78 GHz (0.67 at 1.92 for the dense product); with operands of zeros the first case
// takes 8% less, with no loads at all two thirds of the time. Short reductions are bound by the output, whose
// stores all tiles of a round send at once: 16384 x 2048 x 7168 takes 235 us without stores.
// No gain or slower: steps of 64 k in four stages (4%), 128 x 256 tiles in two workgroups a CU
// (18%), L2 prefetch of either operand (7 to 12%), cache policies of the loads, other tile
// orders (within 1%), staggered starts (dense with an add 4% faster, others slower).
constexpr int kNonTemporal = 2;   // buffer cache policy: the output is not read back here

struct IntTile {
  static constexpr int BM = 256, BN = 256, WAVES = 8, THREADS = 512;
  static constexpr int FM = 8, FN = 4;                   // 16 x 16 blocks of a wavefront
  static constexpr int STEPB = 128;                      // bytes of a row per step
  static constexpr int A_BYTES = BM * STEPB, B_BYTES = BN * STEPB, STAGE = A_BYTES + B_BYTES;
  static constexpr int A_DMAS = A_BYTES / 1024 / WAVES, B_DMAS = B_BYTES / 1024 / WAVES;
  static constexpr int DMAS = A_DMAS + B_DMAS;           // per wavefront and step
  static constexpr int kBlockE = 8, kBlockN = 4;         // tile-order block
};
static_assert(IntTile::DMAS == IntTile::FM, "one DMA behind each row of the second half step");

// One 4-byte-per-lane DMA into LDS, as dma16.
__device__ inline void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(r), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}

template <bool GATHER, int OUT>
__global__ __launch_bounds__(IntTile::THREADS) void int_gemm_tiled_kernel(IntArgs a) {
  typedef IntTile T;
  constexpr int FM = T::FM, FN = T::FN;
  __shared__ __align__(1024) char smem[2 * T::STAGE];
  __shared__ __align__(256) float s_sw[2][T::BN];        // scales of the tile's columns, and of the next's
  __shared__ __align__(256) float s_sa[2][T::BM];        // the same of its rows
  __shared__ __align__(256) int s_u[T::BM];              // src_index of the next tile's rows
  __shared__ uint32_t s_off[T::BM];                      // byte offsets of its token rows
  __shared__ int s_claim;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  // wavefronts w and w + 4 share a SIMD: of a tile whose last 128 rows or columns are empty each
  // SIMD has one that works
  const int wm = wid / 4, wn = (wid + 2 * wm) % 4;
  const int r16 = lane & 15, kb = lane >> 4;
  const uint32_t lds0 = lds_addr(smem);
  const int NT = (a.W + T::BN - 1) / T::BN;
  const int nent = a.tiles ? *a.ntiles : int((a.NK + T::BM - 1) / T::BM);
  const int total = nent * NT;      // below 2^31 (host)
  const int nsteps = a.KB / 2;
  const uint32_t qrow = uint32_t(a.KB) * 64;             // bytes of a token row
  // The workgroups of one XCD take a contiguous run of tiles per round, first come first
  // served (position q of XCD x is tile (q / per) * G + x * per + q % per), a tile ahead;
  // without a queue in turn.
  const int G = gridDim.x, xcd = blockIdx.x % 8, per = G / 8;      // a multiple of 8 (host)
  const bool dyn = a.qcnt != nullptr;
  auto claim = [&]() { return tid == 0 ? atomicAdd(a.qcnt + xcd, 1) : 0; };
  auto publish = [&](int q) { if (tid == 0) s_claim = (q / per) * G + xcd * per + q % per; };

  struct Place { int rowbase, wrow, rows, n0; };
  auto place = [&](int tau) {
    // blocks of kBlockE entries x kBlockN N-tiles
    const int eb = tau / (T::kBlockE * NT), j = tau % (T::kBlockE * NT);
    const int ge = min(T::kBlockE, nent - eb * T::kBlockE);
    const int nb = j / (ge * T::kBlockN), jj = j % (ge * T::kBlockN);
    const int wb = min(T::kBlockN, NT - nb * T::kBlockN);
    const int ent = eb * T::kBlockE + jj / wb;
    const TileEntry e = a.tiles ? a.tiles[ent] : TileEntry{0, 0, ent * T::BM, int(a.NK)};
    return Place{__builtin_amdgcn_readfirstlane(e.rowbase + e.m0), __builtin_amdgcn_readfirstlane(e.wrow),
                 __builtin_amdgcn_readfirstlane(min(T::BM, e.n - e.m0)), (nb * T::kBlockN + jj % wb) * T::BN};
  };
  // Looking a tile up, in two goes of DMA. First the rows' src_index and the columns' scales ..
  auto look_up = [&](const Place& p, int par) {
    if (GATHER && wid < T::BM / 64)
      dma4(make_rsrc(a.src_index + p.rowbase, uint32_t(p.rows) * 4), uint32_t(tid) * 4,
           lds_addr(s_u) + wid * 256);
    if (wid == T::BM / 64) {
      if (a.ws)
        dma16(make_rsrc(a.ws + int64_t(p.wrow) * a.NB * 16 + p.n0, clamp_bytes((int64_t(a.NB) * 16 - p.n0) * 4)),
              uint32_t(lane) * 16, lds_addr(s_sw[par]));
      else
        *reinterpret_cast<v4f_t*>(&s_sw[par][lane * 4]) = v4f_t{1.f, 1.f, 1.f, 1.f};
    }
  };
  // .. then, behind a barrier, each row's offset and scale.
  auto look_up_rows = [&](const Place& p, int par) {
    if (wid >= T::BM / 64) return;
    uint32_t r = kOffNone;
    if (tid < p.rows) {
      const int u = GATHER ? s_u[tid] : 0;
      if (!GATHER) r = tid;
      else if (u >= 0 && u < a.NK) r = uint32_t(u) / uint32_t(a.K);
    }
    s_off[tid] = r == kOffNone ? kOffNone : r * qrow;
    const int64_t first = GATHER ? 0 : p.rowbase;
    dma4(make_rsrc(a.xs + first, clamp_bytes((GATHER ? a.xrows : p.rows) * 4)),
         r == kOffNone ? kOffNone : r * 4, lds_addr(s_sa[par]) + wid * 256);
  };
  // the operands of the tile whose offsets are in s_off
  __amdgpu_buffer_rsrc_t ars, brs;
  uint32_t va[T::A_DMAS], vb[T::B_DMAS];
  auto operands = [&](const Place& p) {
    const int64_t first = GATHER ? 0 : p.rowbase;
    ars = make_rsrc(a.xq + first * qrow, clamp_bytes((GATHER ? a.xrows : p.rows) * qrow));
    const int nblocks = min(T::BN / 16, a.NB - p.n0 / 16);
    brs = make_rsrc(a.wq + (int64_t(p.wrow) * a.NB + p.n0 / 16) * a.KB * 1024, uint32_t(nblocks * a.KB) * 1024);
#pragma unroll
    for (int i = 0; i < T::A_DMAS; ++i) {
      const int row = (wid + T::WAVES * i) * 8 + (lane >> 3);
      const uint32_t off = s_off[row];
      va[i] = off == kOffNone ? kOffNone : off + ((lane & 7) ^ swz_k(row)) * 16;
    }
#pragma unroll
    for (int i = 0; i < T::B_DMAS; ++i) {
      const int b = wid + T::WAVES * i, j = b >> 1;     // half b % 2 of the step, 16-column block j
      vb[i] = j < nblocks ? uint32_t((j * a.KB + (b & 1)) * 1024 + lane * 16) : kOffNone;
    }
  };
  // DMA i of this wavefront for step k, into stage k % 2
  auto issue = [&](int k, int i) {
    const uint32_t st = lds0 + (k & 1) * T::STAGE;
    if (i < T::A_DMAS)
      dma16(ars, va[i], uint32_t(k) * T::STEPB, st + (wid + T::WAVES * i) * 1024);
    else
      dma16(brs, vb[i - T::A_DMAS], uint32_t(k) * 2048,
            st + T::A_BYTES + (wid + T::WAVES * (i - T::A_DMAS)) * 1024);
  };
  auto issue_all = [&](int k) {
#pragma unroll
    for (int i = 0; i < T::DMAS; ++i) issue(k, i);
  };

  int tau = xcd * per + blockIdx.x / 8;
  if (dyn) {
    publish(claim());
    __syncthreads();
    tau = __builtin_amdgcn_readfirstlane(s_claim);
  }
  if (tau >= total) return;
  Place cur = place(tau);
  int par = 0;
  look_up(cur, par);
  wait_vm<0>();
  __syncthreads();
  if (dyn) publish(claim());
  look_up_rows(cur, par);
  wait_vm<0>();
  __syncthreads();
  operands(cur);
  issue_all(0);
  while (true) {
    __syncthreads();     // the previous tile's LDS is free, and the claim is there
    tau = dyn ? __builtin_amdgcn_readfirstlane(s_claim) : tau + G;
    const bool more = tau < total;
    if (nsteps > 1) {
      issue_all(1);
      wait_vm<T::DMAS>();     // step 0 (and whatever came before it)
    } else {
      wait_vm<0>();
    }
    __syncthreads();
    Place next = cur;
    if (more) {
      next = place(tau);
      look_up(next, par ^ 1);
    }
    const int row0 = wm * 128, col0 = wn * 64;
    const bool idle = row0 >= cur.rows || cur.n0 + col0 >= a.W;    // uniform
    v4i_t acc[FM][FN], fa[FM], fb[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v4i_t{0, 0, 0, 0};
    // fragments of half ks of the step in the stage at st; LDS rows 16 apart swizzle alike
    auto frag_a = [&](const char* st, int ks, int i) {
      return *reinterpret_cast<const v4i_t*>(st + (row0 + r16) * T::STEPB + (((ks * 4 + kb) ^ swz_k(r16)) << 4) +
                                             i * 16 * T::STEPB);
    };
    auto frag_b = [&](const char* st, int ks, int j) {
      return *reinterpret_cast<const v4i_t*>(st + T::A_BYTES + (wn * 8 + ks) * 1024 + lane * 16 + j * 2048);
    };
    // The products of the fragments held: of every row with the first two column blocks, then
    // mid(), then with the other two, each row's fragments refilled from half ks of the
    // stage at st behind its last product, and behind(i).
    auto half = [&](const char* st, int ks, auto mid, auto behind) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j)     // operands swapped: a lane holds 4 columns of one row
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      mid();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 2; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        fa[i] = frag_a(st, ks, i);
        if (i < 2) fb[i] = frag_b(st, ks, i);
        behind(i);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 2; j < 4; ++j) fb[j] = frag_b(st, ks, j);
      __builtin_amdgcn_sched_barrier(0);
    };
    // step k; the stage of step k + 1 has landed for every wavefront behind its barrier
    auto land = [&]() {
      wait_vm<0>();
      __syncthreads();
    };
    auto step = [&](int k, auto fill_c) {
      constexpr bool FILL = decltype(fill_c)::value;
      half(smem + (k & 1) * T::STAGE, 1, []() {}, [](int) {});
      // behind the last step its own stage is read again (not used)
      half(smem + ((FILL || k + 1 < nsteps ? k + 1 : k) & 1) * T::STAGE, 0, land,
           [&](int i) { if constexpr (FILL) issue(k + 2, i); });
    };
    if (idle) {
      for (int k = 0; k < nsteps; ++k) {
        if (k + 1 == nsteps && more) {
          if (nsteps == 1) land();
          look_up_rows(next, par ^ 1);
        }
        land();
        if (k + 2 < nsteps) issue_all(k + 2);
      }
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = frag_a(smem, 0, i);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = frag_b(smem, 0, j);
      int k = 0;
      for (; k + 2 < nsteps; ++k) step(k, std::true_type());
      for (; k < nsteps; ++k) {
        if (k + 1 == nsteps && more) {
          if (nsteps == 1) land();      // what was looked up; longer loops have passed a barrier
          look_up_rows(next, par ^ 1);
        }
        step(k, std::false_type());
      }
    }
    // ---- epilogue. Its addresses are formed from et, which hides them from the code ahead of the
    // loop: kept in registers over the loop they made the accumulators spill.
    int et = tid;
    asm volatile("" : "+v"(et));
    const int er = et & 15, ek = (et & 63) >> 4;
    float sa[FM];
    v4f_t sw[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = s_sa[par][row0 + i * 16 + er];
#pragma unroll
    for (int j = 0; j < FN; ++j) sw[j] = *reinterpret_cast<const v4f_t*>(&s_sw[par][col0 + j * 16 + 4 * ek]);
    // rows of `width` elements of eb bytes from column `col`: descriptor
    auto out_rsrc = [&](const void* base, int64_t width, int64_t col, int eb) {
      return make_rsrc(static_cast<const char*>(base) + (cur.rowbase * width + col) * eb,
                       clamp_bytes((cur.rows * width - col) * eb));
    };
    __syncthreads();     // every wavefront has read the last stage, the claim and the tile's scales
    const int q = dyn ? claim() : 0;
    if (more) {
      operands(next);
      issue_all(0);
    }
    // The lanes' own 16 x 16 blocks would be stored as 16 pieces of 64 bytes; the wavefronts
    // exchange 16 rows of each row group at a time through the second stage and store whole
    // rows. Row R of the 32 is row (R / 16) * 128 + 16 * i + R % 16 of the tile.
    char* const ex = smem + T::STAGE;
    auto put = [&](char* buf, int chunks, int byte, auto v) {
      const int R = wm * 16 + er;
      *reinterpret_cast<decltype(v)*>(buf + R * chunks * 16 + (((byte >> 4) ^ er) << 4) + (byte & 15)) = v;
    };
    // what thread et stores in go h of i: LDS address and offset in rows of ld bytes, of which
    // `left` are left from the tile's first column
    auto spot = [&](auto chunks_c, int h, int i, uint32_t ld, uint32_t left, uint32_t& at, uint32_t& off) {
      constexpr int C = decltype(chunks_c)::value;
      const int id = h * T::THREADS + et, R = id / C, c = id % C;
      at = R * C * 16 + ((c ^ (R & 15)) << 4);
      off = uint32_t(c) * 16 < left ? uint32_t((R >> 4) * 128 + i * 16 + (R & 15)) * ld + c * 16 : kOffNone;
    };
    auto flush = [&](const char* buf, auto chunks_c, int i, __amdgpu_buffer_rsrc_t rs, uint32_t ld,
                     uint32_t left, auto policy_c) {
#pragma unroll
      for (int h = 0; h < 32 * decltype(chunks_c)::value / T::THREADS; ++h) {
        uint32_t at, off;
        spot(chunks_c, h, i, ld, left, at, off);
        __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const v4i_t*>(buf + at), rs, off, 0,
                                               decltype(policy_c)::value);
      }
    };
    const std::integral_constant<int, kNonTemporal> stream;
    if constexpr (!is_swiglu(OUT)) {
      const std::integral_constant<int, 64> chunks;
      constexpr int GOES = 32 * 64 / T::THREADS;
      const uint32_t ld = uint32_t(a.W) * 4, left = uint32_t(a.W - cur.n0) * 4;
      const __amdgpu_buffer_rsrc_t crs = out_rsrc(a.c, a.W, cur.n0, 4);
      const __amdgpu_buffer_rsrc_t drs = out_rsrc(OUT == kIntFloatAdd ? a.add : a.c, a.W, cur.n0, 4);
      v4f_t add[GOES];       // of the next rows, on their way while these are exchanged
      auto fetch = [&](int i) {
        if constexpr (OUT == kIntFloatAdd) {
#pragma unroll
          for (int h = 0; h < GOES; ++h) {
            uint32_t at, off;
            spot(chunks, h, i, ld, left, at, off);
            add[h] = __builtin_bit_cast(v4f_t,
                                        __builtin_amdgcn_raw_buffer_load_b128(drs, off, 0, kNonTemporal));
          }
        }
      };
      fetch(0);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        char* buf = ex + (i & 1) * 32768;
        if (!idle) {
#pragma unroll
          for (int j = 0; j < FN; ++j)
            put(buf, 64, (col0 + j * 16 + 4 * ek) * 4, int_scaled(acc[i][j], sa[i], sw[j]));
        }
        __syncthreads();
        if constexpr (OUT == kIntFloatAdd) {
          v4f_t out[GOES];
          uint32_t at, off[GOES];
#pragma unroll
          for (int h = 0; h < GOES; ++h) {
            spot(chunks, h, i, ld, left, at, off[h]);
            out[h] = added(*reinterpret_cast<const v4f_t*>(buf + at), add[h]);
          }
          if (i + 1 < FM) fetch(i + 1);
#pragma unroll
          for (int h = 0; h < GOES; ++h)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i_t, out[h]), crs, off[h], 0,
                                                   kNonTemporal);
        } else {
          flush(buf, chunks, i, crs, ld, left, stream);
        }
      }
    } else {
      constexpr int EB = OUT == kIntSwigluBf16 ? 2 : 4;
      const std::integral_constant<int, 8 * EB> achunks;
      const std::integral_constant<int, 16 * EB> hchunks;
      const __amdgpu_buffer_rsrc_t ors = out_rsrc(a.act, a.W / 2, cur.n0 / 2, EB);
      const __amdgpu_buffer_rsrc_t hrs = out_rsrc(a.h_saved ? a.h_saved : a.act, a.W, cur.n0, EB);
      auto value = [&](v4f_t v) {
        if constexpr (EB == 2) return uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        else return v;
      };
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        char* abuf = ex + (EB == 2 ? (i & 1) * 24576 : 0);
        char* hbuf = abuf + 32 * 128 * EB;
        if (!idle) {
          v4f_t v[FN];
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            v[j] = int_scaled(acc[i][j], sa[i], sw[j]);
            if (a.h_saved) put(hbuf, 16 * EB, (col0 + j * 16 + 4 * ek) * EB, value(v[j]));
          }
          // blocks 0, 1 of the wavefront's 64 columns are gates, 2, 3 their up columns
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            v4f_t s;
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = int_swiglu<OUT>(v[j][e], v[j + 2][e]);
            put(abuf, 8 * EB, (wn * 32 + j * 16 + 4 * ek) * EB, value(s));
          }
        }
        __syncthreads();
        flush(abuf, achunks, i, ors, uint32_t(a.W / 2) * EB, uint32_t(a.W - cur.n0) / 2 * EB,
              std::integral_constant<int, 0>());
        if (a.h_saved) flush(hbuf, hchunks, i, hrs, uint32_t(a.W) * EB, uint32_t(a.W - cur.n0) * EB, stream);
        if (EB == 4 && i + 1 < FM) __syncthreads();     // one buffer: read before the next rows
      }
    }
    if (!more) break;
    if (dyn) publish(q);
    cur = next;
    par ^= 1;
  }
}

// ---- small tiles: where 256 x 256 tiles would leave CUs without one. BT x BT tiles by eight
// wavefronts, both operands through LDS as in the tiled form, in a ring of four steps that is in
// flight but for one: a tile's time is its loads' latency and what a step takes from barrier to
// barrier. 64 x 64 tiles have two groups of wavefronts, which share a step's 256 k and add their
// sums at the end: half the barriers per k.
template <int BT>
struct IntSmall {
  static constexpr int THREADS = 512, STAGES = 4;
  static constexpr int GROUPS = BT == 64 ? 2 : 1, WAVES_N = BT == 64 ? 2 : 4;   // 2 x WAVES_N wavefronts a group
  static constexpr int FM = BT / 32, FN = 2;
  static constexpr int OP_BYTES = BT * 128, PART = 2 * OP_BYTES, STAGE = GROUPS * PART;
  static constexpr int A_DMAS = OP_BYTES / 1024 / (8 / GROUPS), DMAS = 2 * A_DMAS;   // per wavefront and step
};

template <int BT, bool GATHER, int OUT>
__global__ __launch_bounds__(512) void int_gemm_small_kernel(IntArgs a) {
  typedef IntSmall<BT> T;
  constexpr int FM = T::FM, FN = T::FN, WPG = 8 / T::GROUPS;
  __shared__ __align__(1024) char smem[T::STAGES * T::STAGE];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = wid / WPG, w = wid % WPG;                // group, wavefront in it
  const int wm = w / T::WAVES_N, wn = w % T::WAVES_N;
  const int r16 = lane & 15, kb = lane >> 4;
  const uint32_t lds0 = lds_addr(smem);
  const int NT = (a.W + BT - 1) / BT;
  // A plan's tiles, without a list of them and its launch: thread t counts those of its run of
  // segments and s_upto[t] tells how many come before it.
  __shared__ int s_upto[T::THREADS + 1];
  __shared__ int s_waves[8];
  const int EB = a.E + a.B, segs = a.R * EB, run = (segs + T::THREADS - 1) / T::THREADS;
  auto length = [&](int seg, int& c0) {
    const int32_t* at = a.cu + int64_t(seg / EB) * (EB + 1) + seg % EB;
    c0 = at[0];
    return at[1] - c0;
  };
  int nent = int((a.NK + BT - 1) / BT);
  if (a.cu) {
    int count = 0, c0;
    for (int i = 0; i < run; ++i) {
      const int seg = threadIdx.x * run + i;
      if (seg < segs) count += (max(0, length(seg, c0)) + BT - 1) / BT;
    }
    int upto = count;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    if (lane == 63) s_waves[wid] = upto;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < wid) upto += s_waves[i];
    s_upto[threadIdx.x + 1] = upto;
    if (threadIdx.x == 0) s_upto[0] = 0;
    __syncthreads();
    nent = s_upto[T::THREADS];
  }
  auto entry = [&](int ent) {
    int lo = 0, hi = T::THREADS;       // s_upto[lo] <= ent < s_upto[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_upto[mid] <= ent) lo = mid;
      else hi = mid;
    }
    int before = s_upto[lo], seg = lo * run, c0, n = 0;
    for (int i = 0; i < run; ++i, ++seg) {      // uniform
      n = max(0, length(seg, c0));
      const int t = (n + BT - 1) / BT;
      if (ent < before + t) break;
      before += t;
    }
    const int rank = seg / EB, i = seg % EB;
    return TileEntry{rank * a.SK + c0, i < a.E ? i : a.E + rank * a.B + (i - a.E), (ent - before) * BT, n};
  };
  const int64_t total = int64_t(nent) * NT;
  const int nparts = a.KB / 2, nsteps = (nparts + T::GROUPS - 1) / T::GROUPS;
  const uint32_t qrow = uint32_t(a.KB) * 64;
  // the workgroups of one XCD take a contiguous run of tiles per round: of one weight all its
  // columns' rows, of a list all columns of its entries
  const int G = gridDim.x, per = G / 8;
  for (int64_t tau = (blockIdx.x % 8) * per + blockIdx.x / 8; tau < total; tau += G) {
    const int ent = int(a.cu ? tau / NT : tau % nent), nt = int(a.cu ? tau % NT : tau / nent);
    const TileEntry e = a.cu ? entry(ent) : TileEntry{0, 0, ent * BT, int(a.NK)};
    const int rowbase = __builtin_amdgcn_readfirstlane(e.rowbase + e.m0);
    const int wrow = __builtin_amdgcn_readfirstlane(e.wrow);
    const int rows = __builtin_amdgcn_readfirstlane(min(BT, e.n - e.m0));
    const int n0 = nt * BT;
    const int nblocks = min(BT / 16, a.NB - n0 / 16);
    auto row_of = [&](int row, bool& in) -> int64_t {      // token row of a row of the tile
      in = row < rows;
      if (!GATHER) return int64_t(rowbase) + row;
      const int u = in ? a.src_index[rowbase + row] : -1;
      in = u >= 0 && u < a.NK;
      return in ? u / a.K : 0;
    };
    const int64_t first = GATHER ? 0 : rowbase;
    const __amdgpu_buffer_rsrc_t ars =
        make_rsrc(a.xq + first * qrow, clamp_bytes((GATHER ? a.xrows : rows) * qrow));
    const __amdgpu_buffer_rsrc_t brs =
        make_rsrc(a.wq + (int64_t(wrow) * a.NB + n0 / 16) * a.KB * 1024, uint32_t(nblocks * a.KB) * 1024);
    uint32_t va[T::A_DMAS], vb[T::A_DMAS];
#pragma unroll
    for (int i = 0; i < T::A_DMAS; ++i) {
      const int b = w + WPG * i, row = b * 8 + (lane >> 3), j = b >> 1;
      bool in;
      const int64_t r = row_of(row, in) - first;
      va[i] = in ? uint32_t(r) * qrow + ((lane & 7) ^ swz_k(row)) * 16 : kOffNone;
      vb[i] = j < nblocks ? uint32_t((j * a.KB + (b & 1)) * 1024 + lane * 16) : kOffNone;
    }
    // the group's part of step k; past the last part zeros, so that every step has its DMAs
    auto issue = [&](int k, uint32_t stage) {
      const int p = k * T::GROUPS + g;
      const bool there = T::GROUPS == 1 || p < nparts;
      const uint32_t st = lds0 + stage + g * T::PART;
#pragma unroll
      for (int i = 0; i < T::A_DMAS; ++i)
        dma16(ars, there ? va[i] : kOffNone, uint32_t(p) * 128, st + (w + WPG * i) * 1024);
#pragma unroll
      for (int i = 0; i < T::A_DMAS; ++i)
        dma16(brs, there ? vb[i] : kOffNone, uint32_t(p) * 2048, st + T::OP_BYTES + (w + WPG * i) * 1024);
    };
    auto wait_steps = [&](int n) {     // until at most n later steps are in flight
      if (n >= 2) wait_vm<2 * T::DMAS>();
      else if (n == 1) wait_vm<T::DMAS>();
      else wait_vm<0>();
    };
    __syncthreads();     // every wavefront is done with the previous tile's LDS
#pragma unroll
    for (int k = 0; k < T::STAGES - 1; ++k)
      if (k < nsteps) issue(k, k * T::STAGE);
    v4i_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = v4i_t{0, 0, 0, 0};
    const int row0 = wm * (BT / 2);
    // the wavefront's two blocks of columns lie 32 apart: gate and up
    auto block = [&](int j) { return (wn >> 1) * 4 + (wn & 1) + 2 * j; };
    uint32_t cur = 0, fill = (T::STAGES - 1) * T::STAGE;
    auto after = [](uint32_t s) { return s + T::STAGE == T::STAGES * T::STAGE ? 0u : s + T::STAGE; };
    for (int k = 0; k < nsteps; ++k) {
      wait_steps(min(T::STAGES - 2, nsteps - 1 - k));
      __syncthreads();     // step k has landed, and every wavefront has read step k - 1
      if (k + T::STAGES - 1 < nsteps) issue(k + T::STAGES - 1, fill);
      const char* st = smem + cur + g * T::PART;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        v4i_t fa[FM], fb[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j)
          fb[j] = *reinterpret_cast<const v4i_t*>(st + T::OP_BYTES + (block(j) * 2 + ks) * 1024 + lane * 16);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          fa[i] = *reinterpret_cast<const v4i_t*>(st + (row0 + i * 16 + r16) * 128 +
                                                  (((ks * 4 + kb) ^ swz_k(r16)) << 4));
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
      cur = after(cur);
      fill = after(fill);
    }
    if constexpr (T::GROUPS == 2) {
      // each group takes the other's sums of its row block (FM = 2: block i is group i's)
      v4i_t(*part)[FN][64] = reinterpret_cast<v4i_t(*)[FN][64]>(smem);      // [8][FN][64]
      __syncthreads();
#pragma unroll
      for (int j = 0; j < FN; ++j) part[wid][j][lane] = g ? acc[0][j] : acc[1][j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const v4i_t other = part[wid ^ WPG][j][lane];
        acc[0][j] = (g ? acc[1][j] : acc[0][j]) + other;
      }
    }
    constexpr int ROWS = FM / T::GROUPS;      // row blocks that a wavefront stores
    int col[FN];
    v4f_t sw[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      col[j] = n0 + block(j) * 16 + 4 * kb;
      sw[j] = a.ws && col[j] < a.W ? *reinterpret_cast<const v4f_t*>(a.ws + int64_t(wrow) * a.NB * 16 + col[j])
                                   : v4f_t{1.f, 1.f, 1.f, 1.f};
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int row = row0 + (i + g * ROWS) * 16 + r16;
      if (row >= rows) continue;
      bool in;
      const int64_t r = row_of(row, in);
      const float sa = in ? a.xs[r] : 0.0f;
      const int64_t pos = int64_t(rowbase) + row;
      v4f_t v[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) v[j] = int_scaled(acc[i][j], sa, sw[j]);
      if constexpr (!is_swiglu(OUT)) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
          if (col[j] < a.W) {
            if constexpr (OUT == kIntFloatAdd)
              v[j] = added(v[j], *reinterpret_cast<const v4f_t*>(a.add + pos * a.W + col[j]));
            *reinterpret_cast<v4f_t*>(a.c + pos * a.W + col[j]) = v[j];
          }
      } else if (col[0] < a.W) {
        v4f_t s;
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] = int_swiglu<OUT>(v[0][x], v[1][x]);
        store4<OUT>(a.act, pos * (a.W / 2) + col[0] / 64 * 32 + col[0] % 32, s);
        if (a.h_saved) {
          store4<OUT>(a.h_saved, pos * a.W + col[0], v[0]);
          store4<OUT>(a.h_saved, pos * a.W + col[1], v[1]);
        }
      }
    }
  }
}

static int int_grid(int64_t work, int64_t cap) {
  const int64_t blocks = (work + kIntThreads - 1) / kIntThreads;
  return int(blocks < 1 ? 1 : (blocks > cap ? cap : blocks));
}

inline int64_t int_kb(int width) { return 2 * k_tiles(width); }      // blocks of 64 k
inline int64_t int_nb(int width) { return (int64_t(width) + 15) / 16; }

template <int BT, int OUT>
static int launch_small(const IntArgs& a, int grid, hipStream_t strm) {
  if (OUT != kIntFloatAdd && a.src_index)      // an add comes with dense products alone
    int_gemm_small_kernel<BT, OUT != kIntFloatAdd, OUT><<<grid, IntSmall<BT>::THREADS, 0, strm>>>(a);
  else
    int_gemm_small_kernel<BT, false, OUT><<<grid, IntSmall<BT>::THREADS, 0, strm>>>(a);
  return launch_status();
}

// ws: the layer's workspace, for a grouped product's tile list; s its shape.
//
// Which form, by rows per weight row, and by how many tiles there are to hand out (counting half
// a tile of padding per weight row). us, few rows / 64 x 64 / 128 x 128 / 256 x 256 tiles:
//   grouped 256 x (4096, 1536), rows each: 4: 242/258/259/289, 8: 268/276/267/293, 16:
//     334/289/276/295, 32: 466/317/290/298, 64: 803/416/325/312, 256: 2884/1260/714/509
//   grouped 64 x (7168, 2048): 8: 162/165/166/185, 16: 206/171/168/185, 32: 302/193/174/187, 64:
//     488/242/214/192, 256: 1664/709/388/294
//   grouped 16 x (1024, 512): 8: 4.7/7.3/9.5/22, 32: 6.2/7.8/11/22, 128: 14/13/13/26, 512: 40/30/23/28
//   dense (2048, 7168), rows: 16: 5.4/7.1/12/23, 32: 6.5/7.2/12/23, 48: 7.6/7.4/13/23, 128:
//     16/8.4/17/24, 512: 45/27/19/36, 1024: 86/43/33/39, 2048: 167/93/61/45
//   dense (7168, 4096): 32: 13/15/31/50, 48: 18/15/32/50, 512: 77/28/35/72, 1024: 151/61/38/74,
//     2048: 299/134/74/83, 4096: 595/259/142/89
//   dense (7168, 512): 32: 13/15/31/42, 64: 22/15/33/49, 2048: 43/22/36/71, 4096: 81/40/37/79, 16384:
//     306/145/83/90
//   tiny: grouped 16 x (80, 104), 47 rows: 4.0/6.4, 16 x (64, 136), 32: 4.0/6.2, dense (512, 512), 64:
//     4.8/4.8, 256: 5.2/5.1, 1024: 13/8.4
//   skewed, 256 x (4096, 1536), 8 rows each on average, few rows / 128 x 128: all alike 264/280, a
//     tenth of the rows on one expert 303/285, half 340/288, all of them 367/28 (the rule sees the
//     average alone: the longest segment is known on the device)
// So: few rows up to 8 each (a dense product, which reads its one weight from the caches, up to
// 32), and where the workgroups have at most one item each and a wavefront's share of one is
// short (96 blocks of 16 rows by 64 k); 256-row tiles from 64 rows each on, if they are more than
// half as many as the CUs; below, 128-row tiles if those are, else 64-row tiles.
template <int OUT>
static int int_product(IntArgs a, const moonep_shape& s, void* ws, hipStream_t strm) {
  const int cus = device_cus();
  if (cus <= 0) return MOONEP_EHIP;
  const int64_t segs = a.cu ? int64_t(s.E) + s.R : 1;      // a plan has at most this many segments
  a.xrows = a.src_index ? int64_t(s.R) * s.S : a.NK;
  auto tiles = [&](int64_t bt) {
    return (a.NK + bt / 2 * segs + bt - 1) / bt * ((int64_t(a.W) + bt - 1) / bt);
  };
  // 32-bit offsets of gathered rows, and the order of tiles over the XCDs
  const bool fits = cus % 8 == 0 && (!a.src_index || a.xrows * a.KB * 64 < int64_t(kOffNone));
  const int64_t each = (a.NK + segs - 1) / segs;      // rows per weight row
  const bool few = each <= (a.cu ? 8 : 32) ||
                   (segs * ((a.NB + 1) / 2) * ((each + kIntRows - 1) / kIntRows) <= 4 * cus &&
                    a.KB * ((each + 15) / 16) <= 96);
  if (fits && !few) {
    if (a.NK >= 64 * segs && tiles(IntTile::BM) > cus / 2 &&
        // 32-bit offsets of a tile's outputs, and tile numbers
        int64_t(IntTile::BM) * a.W * 4 <= int64_t(kOffNone) &&
        tiles(IntTile::BM) + int64_t(s.R) * (s.E + s.B) * ((a.W + IntTile::BN - 1) / IntTile::BN) < INT32_MAX) {
      if (a.cu) {
        const int st = launch_tile_list(s, a.cu, IntTile::BM, ws, strm, &a.tiles, &a.ntiles);
        if (st) return st;
        a.qcnt = ws_ptr<int32_t>(ws, ws_layout(s).flags) + kFlagQueue;
      }
      if (OUT != kIntFloatAdd && a.src_index)
        int_gemm_tiled_kernel<OUT != kIntFloatAdd, OUT><<<cus, IntTile::THREADS, 0, strm>>>(a);
      else
        int_gemm_tiled_kernel<false, OUT><<<cus, IntTile::THREADS, 0, strm>>>(a);
      return launch_status();
    }
    return tiles(128) > cus / 2 ? launch_small<128, OUT>(a, cus, strm) : launch_small<64, OUT>(a, cus, strm);
  }
  // a segment's rows are shared out twice as finely as an even plan would need
  const int64_t share = (2 * a.NK + segs * kIntRows - 1) / (segs * kIntRows);
  const int shares = int(share < 64 ? share : 64);
  int_gemm_kernel<OUT><<<cus * 4, kIntWaves * 64, 0, strm>>>(a, shares);
  return launch_status();
}

// How the `nout` vectors of a row are shared out, as arguments of f: wavefronts per row, and
// vectors per lane (0: too many to hold). few: too few rows to fill the card with a wavefront
// each, so that a row's latency counts.
template <typename F>
static void with_row_split(int64_t nout, bool few, F f) {
  const int64_t per = (nout + 63) / 64;       // vectors per lane of one wavefront
#define MOONEP_SPLIT(W, V) f(std::integral_constant<int, W>(), std::integral_constant<int, V>())
  if (per <= 1) MOONEP_SPLIT(1, 1);
  else if (few && per <= 4) MOONEP_SPLIT(4, 1);
  else if (few && per <= 8) MOONEP_SPLIT(8, 1);
  else if (few && per <= 16) MOONEP_SPLIT(16, 1);
  else if (per <= 2) MOONEP_SPLIT(1, 2);
  else if (per <= 4) MOONEP_SPLIT(1, 4);
  else if (per <= 8) MOONEP_SPLIT(4, 2);
  else if (per <= 16) MOONEP_SPLIT(4, 4);
  else if (per <= 64) MOONEP_SPLIT(16, 4);
  else MOONEP_SPLIT(16, 0);
#undef MOONEP_SPLIT
}

// The rules all products share; W the weight's columns. MOONEP_OK leaves *a filled but for the
// outputs, the plan and the add.
static int int_operands(const moonep_shape& s, int64_t W, const int8_t* xq, const float* xscales,
                        const int32_t* src_index, const int8_t* wq, const float* wscales,
                        IntArgs* a) {
  if (!aligned16(xq) || !aligned16(xscales) || !aligned16(wq) ||
      (wscales && !aligned16(wscales)) || (src_index && !aligned16(src_index)))
    return MOONEP_EINVAL;
  *a = IntArgs{};
  a->xq = xq;
  a->xs = xscales;
  a->src_index = src_index;
  a->wq = wq;
  a->ws = wscales;
  a->K = s.K;
  a->W = int(W);
  a->NB = int(int_nb(int(W)));
  a->KB = int(int_kb(s.H));
  return MOONEP_OK;
}

static void int_plan(const moonep_shape& s, const int32_t* cu, IntArgs* a) {
  a->NK = int64_t(s.R) * s.S * s.K;
  a->cu = cu;
  a->R = s.R;
  a->E = s.E;
  a->B = s.B;
  a->SK = s.S * s.K;
}

}  // namespace moonep

using namespace moonep;

extern "C" int moonep_int_quantize(const moonep_shape* shape, int64_t rows, int32_t width,
                                   const void* src, int8_t* q, float* scales, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const bool bf16 = shape->dtype == MOONEP_BF16;
  const int vec = bf16 ? 8 : 4;
  if (rows < 0 || rows > INT32_MAX || width < vec || width % vec) return MOONEP_EINVAL;
  if (width > kIntMaxK) return MOONEP_ELIMIT;
  if (rows == 0) return MOONEP_OK;
  if (!aligned16(src) || !aligned16(q) || !aligned16(scales)) return MOONEP_EINVAL;
  const uint4* in = static_cast<const uint4*>(src);
  const int nvec = width / vec, nout = int(k_tiles(width)) * 128 / vec;
  with_row_split(nout, rows < kIntFewRows, [&](auto w, auto v) {
    constexpr int WPR = decltype(w)::value, VPL = decltype(v)::value, RPG = int_threads(WPR) / (64 * WPR);
    const int64_t groups = (rows + RPG - 1) / RPG;
    const int grid = int(groups < 65536 ? groups : 65536);
    if (bf16)
      int_quantize_kernel<true, WPR, VPL><<<grid, int_threads(WPR), 0, as_stream(stream)>>>(in, rows, nvec, nout, q, scales);
    else
      int_quantize_kernel<false, WPR, VPL><<<grid, int_threads(WPR), 0, as_stream(stream)>>>(in, rows, nvec, nout, q, scales);
  });
  return launch_status();
}

extern "C" int moonep_int_quantize_weight(const moonep_shape* shape, const void* w, int8_t* wq,
                                          float* wscales, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.H > kIntMaxK || s.Hp > kIntMaxCols) return MOONEP_ELIMIT;
  if (!aligned16(w) || !aligned16(wq) || !aligned16(wscales)) return MOONEP_EINVAL;
  const int KB = int(int_kb(s.H)), NB = int(int_nb(s.Hp));
  const dim3 grid((NB + 3) / 4, s.E);
  if (s.dtype == MOONEP_BF16)
    int_quantize_weight_kernel<true><<<grid, kIntThreads, 0, as_stream(stream)>>>(w, s.H, s.Hp, KB, NB, wq, wscales);
  else
    int_quantize_weight_kernel<false><<<grid, kIntThreads, 0, as_stream(stream)>>>(w, s.H, s.Hp, KB, NB, wq, wscales);
  return launch_status();
}

extern "C" int moonep_int_transpose_weight(const moonep_shape* shape, const int8_t* wq, int8_t* wqt,
                                           void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.H > kIntMaxK || s.Hp > kIntMaxK) return MOONEP_ELIMIT;
  if (!aligned16(wq) || !aligned16(wqt)) return MOONEP_EINVAL;
  const int KBt = int(int_kb(s.Hp)), NBt = int(int_nb(s.H));
  const dim3 grid(int_grid(int64_t(KBt) * NBt * 64, 1024), s.E);
  int_transpose_weight_kernel<<<grid, kIntThreads, 0, as_stream(stream)>>>(
      wq, int(int_kb(s.H)), int(int_nb(s.Hp)), KBt, NBt, wqt);
  return launch_status();
}

extern "C" int moonep_int_prefetch_weight(const moonep_shape* shape, const int32_t* replica_expert,
                                          int8_t* wq, float* wscales, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.H > kIntMaxK || s.Hp > kIntMaxCols) return MOONEP_ELIMIT;
  if (s.B == 0) return MOONEP_OK;
  if (!aligned16(replica_expert) || !aligned16(wq) || (wscales && !aligned16(wscales)))
    return MOONEP_EINVAL;
  const int64_t qvec = int_nb(s.Hp) * int_kb(s.H) * 64;
  const int64_t svec = wscales ? int_nb(s.Hp) * 4 : 0;
  int_prefetch_kernel<<<int_grid(qvec + svec, 2048), kIntThreads, 0, as_stream(stream)>>>(
      replica_expert, s.R * s.B, s.E, reinterpret_cast<uint4*>(wq), qvec,
      reinterpret_cast<uint4*>(wscales), svec);
  return launch_status();
}

extern "C" int moonep_int_grouped_gemm(const moonep_shape* shape, const int8_t* xq,
                                       const float* xscales, const int32_t* src_index,
                                       const int8_t* wq, const float* wscales,
                                       const int32_t* cu_seqlens, float* c, void* ws,
                                       size_t ws_bytes, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.H > kIntMaxK || s.Hp > kIntMaxCols) return MOONEP_ELIMIT;
  if (!aligned16(cu_seqlens) || !aligned16(ws)) return MOONEP_EINVAL;
  if (ws_bytes < ws_layout(s).total) return MOONEP_EWORKSPACE;
  if (s.S == 0) return MOONEP_OK;
  IntArgs a;
  st = int_operands(s, s.Hp, xq, xscales, src_index, wq, wscales, &a);
  if (st || !aligned16(c)) return MOONEP_EINVAL;
  int_plan(s, cu_seqlens, &a);
  a.c = c;
  return int_product<kIntFloat>(a, s, ws, as_stream(stream));
}

extern "C" int moonep_int_grouped_gemm_swiglu(const moonep_shape* shape, const int8_t* xq,
                                              const float* xscales, const int32_t* src_index,
                                              const int8_t* wq, const float* wscales,
                                              const int32_t* cu_seqlens, void* act, void* h_saved,
                                              void* ws, size_t ws_bytes, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.Hp % kSwigluBlock) return MOONEP_EINVAL;
  if (s.H > kIntMaxK || s.Hp > kIntMaxCols / 2) return MOONEP_ELIMIT;
  if (!aligned16(cu_seqlens) || !aligned16(ws)) return MOONEP_EINVAL;
  if (ws_bytes < ws_layout(s).total) return MOONEP_EWORKSPACE;
  if (s.S == 0) return MOONEP_OK;
  IntArgs a;
  st = int_operands(s, 2 * int64_t(s.Hp), xq, xscales, src_index, wq, wscales, &a);
  if (st || !aligned16(act) || (h_saved && !aligned16(h_saved))) return MOONEP_EINVAL;
  int_plan(s, cu_seqlens, &a);
  a.act = act;
  a.h_saved = h_saved;
  return s.dtype == MOONEP_BF16 ? int_product<kIntSwigluBf16>(a, s, ws, as_stream(stream))
                                : int_product<kIntSwigluF32>(a, s, ws, as_stream(stream));
}

extern "C" int moonep_int_gemm(const moonep_shape* shape, int64_t rows, const int8_t* xq,
                               const float* xscales, const int8_t* wq, const float* wscales,
                               const float* add, float* c, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (rows < 0 || rows > INT32_MAX) return MOONEP_EINVAL;
  if (s.H > kIntMaxK || s.Hp > kIntMaxCols) return MOONEP_ELIMIT;
  if (rows == 0) return MOONEP_OK;
  IntArgs a;
  st = int_operands(s, s.Hp, xq, xscales, nullptr, wq, wscales, &a);
  if (st || !aligned16(c) || (add && !aligned16(add))) return MOONEP_EINVAL;
  a.NK = rows;
  a.add = add;
  a.c = c;
  return add ? int_product<kIntFloatAdd>(a, s, nullptr, as_stream(stream))
             : int_product<kIntFloat>(a, s, nullptr, as_stream(stream));
}

extern "C" int moonep_int_gemm_swiglu(const moonep_shape* shape, int64_t rows, const int8_t* xq,
                                      const float* xscales, const int8_t* wq, const float* wscales,
                                      void* act, void* h_saved, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (rows < 0 || rows > INT32_MAX || s.Hp % kSwigluBlock) return MOONEP_EINVAL;
  if (s.H > kIntMaxK || s.Hp > kIntMaxCols / 2) return MOONEP_ELIMIT;
  if (rows == 0) return MOONEP_OK;
  IntArgs a;
  st = int_operands(s, 2 * int64_t(s.Hp), xq, xscales, nullptr, wq, wscales, &a);
  if (st || !aligned16(act) || (h_saved && !aligned16(h_saved))) return MOONEP_EINVAL;
  a.NK = rows;
  a.act = act;
  a.h_saved = h_saved;
  return s.dtype == MOONEP_BF16 ? int_product<kIntSwigluBf16>(a, s, nullptr, as_stream(stream))
                                : int_product<kIntSwigluF32>(a, s, nullptr, as_stream(stream));
}

extern "C" int moonep_int_quantize_grad(const moonep_shape* shape, const void* src,
                                        const int32_t* src_index, const float* gates,
                                        const float* wscales, const int32_t* cu_seqlens, int8_t* q,
                                        float* scales, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.mode != MOONEP_TRAIN) return MOONEP_EMODE;
  if (s.Hp > kIntMaxK) return MOONEP_ELIMIT;
  if (s.S == 0) return MOONEP_OK;
  if (!aligned16(src) || !aligned16(wscales) || !aligned16(q) || !aligned16(scales) ||
      (src_index && !aligned16(src_index)) || (gates && !aligned16(gates)) ||
      (cu_seqlens && !aligned16(cu_seqlens)) || (gates && !src_index))
    return MOONEP_EINVAL;
  const bool bf16 = s.dtype == MOONEP_BF16;
  const int vec = bf16 ? 8 : 4;
  IntGradArgs a{static_cast<const uint4*>(src), src_index, gates, wscales, cu_seqlens, q, scales,
                s.R, s.E, s.B, s.S * s.K, s.K, s.Hp / vec, int(k_tiles(s.Hp)) * 128 / vec,
                int(int_nb(s.Hp)) * 16, int64_t(s.R) * s.S * s.K, 0};
  // chunks of at most kIntChunk positions, shorter where there are few
  const int64_t chunk = a.NK / (4 * kIntFewRows);
  a.chunk = int(chunk < 1 ? 1 : chunk < kIntChunk ? chunk : kIntChunk);
  const bool stream_out = a.NK * a.nout * vec > kIntCache;
  with_row_split(a.nout, a.NK < kIntFewRows, [&](auto w, auto v) {
    constexpr int WPR = decltype(w)::value, VPL = decltype(v)::value, RPG = int_threads(WPR) / (64 * WPR);
    const int64_t per = int64_t(RPG) * a.chunk;
    const int64_t groups = (a.NK + per - 1) / per;
    const int grid = int(groups < (1 << 20) ? groups : (1 << 20));
    auto launch = [&](auto type, auto past) {
      int_quantize_grad_kernel<decltype(type)::value, WPR, VPL, decltype(past)::value>
          <<<grid, int_threads(WPR), 0, as_stream(stream)>>>(a);
    };
    const std::true_type yes;
    const std::false_type no;
    if (bf16) stream_out ? launch(yes, yes) : launch(yes, no);
    else stream_out ? launch(no, yes) : launch(no, no);
  });
  return launch_status();
}
