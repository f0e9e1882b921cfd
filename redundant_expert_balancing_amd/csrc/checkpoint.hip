// 8-bit activation checkpoints on gfx950 (format and rounding: moonep.h): quantisation of
// token rows, the permute that reads them back, and the SwiGLU forward and backward with
// the pre-activation kept in 8 bits. All are HBM-bound passes: one read and one write of
// each array, 16-byte vectors of the wide side, the conversions by the hardware's
// float32 <-> e4m3 instructions (round to nearest even; the power-of-two scale is exact).
#include "common.h"

namespace moonep {

constexpr int kCkThreads = kRowThreads;
typedef float v4f_t __attribute__((ext_vector_type(4)));
typedef float v2f_t __attribute__((ext_vector_type(2)));

inline int64_t scale_row(int width) { return 4 * ((int64_t(width) + 127) / 128); }

__device__ inline uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// 4 values scaled by inv as 4 e4m3 bytes
__device__ inline uint32_t pack_e4m3(const float* v, float inv) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(v[0]) * inv, clamp_e4m3(v[1]) * inv, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(v[2]) * inv, clamp_e4m3(v[3]) * inv, w, true));
}

__device__ inline void unpack_e4m3(uint32_t w, float scale, float* v) {
  const v2f_t a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false);
  const v2f_t b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
  v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
}

// V (4 or 8) consecutive values at element idx, a multiple of V
template <bool BF16, int V, bool ONCE = false>
__device__ inline void load_v(const void* base, int64_t idx, float* v) {
  if constexpr (BF16) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const uint2 w = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + idx)[h];
      v[4 * h] = __uint_as_float(w.x << 16);
      v[4 * h + 1] = __uint_as_float(w.x & 0xFFFF0000u);
      v[4 * h + 2] = __uint_as_float(w.y << 16);
      v[4 * h + 3] = __uint_as_float(w.y & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const v4f_t* p = reinterpret_cast<const v4f_t*>(static_cast<const float*>(base) + idx) + h;
      const v4f_t w = ONCE ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = w[i];
    }
  }
}

typedef uint32_t v4u_t __attribute__((ext_vector_type(4)));
typedef uint32_t v2u_t __attribute__((ext_vector_type(2)));

template <bool BF16, int V>
__device__ inline void store_v(void* base, int64_t idx, const float* v) {
  if constexpr (BF16) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = bf16_rne_any(v[2 * i]) | (bf16_rne_any(v[2 * i + 1]) << 16);
    uint16_t* p = static_cast<uint16_t*>(base) + idx;
    if constexpr (V == 8) *reinterpret_cast<v4u_t*>(p) = v4u_t{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<v2u_t*>(p) = v2u_t{w[0], w[1]};
  } else {
#pragma unroll
    for (int h = 0; h < V / 4; ++h)
      reinterpret_cast<v4f_t*>(static_cast<float*>(base) + idx)[h] =
          v4f_t{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
  }
}

template <int V>
__device__ inline void load_q(const uint8_t* p, float scale, float* v) {
  if constexpr (V == 8) {
    const v2u_t w = *reinterpret_cast<const v2u_t*>(p);
    unpack_e4m3(w.x, scale, v);
    unpack_e4m3(w.y, scale, v + 4);
  } else {
    unpack_e4m3(*reinterpret_cast<const uint32_t*>(p), scale, v);
  }
}

// V values of a block that 32 / V neighbouring lanes share, as e4m3 at p (where `in`);
// returns the block's scale byte
template <int V>
__device__ inline uint32_t quantise_v(const float* v, bool in, uint8_t* p) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max(m, mag_bits(v[i]));
#pragma unroll
  for (int d = 1; d < 32 / V; d <<= 1) m = max(m, uint32_t(__shfl_xor(int(m), d, 64)));
  const uint32_t b = scale_byte<E4M3>(m);
  const float inv = b == 255 ? 0.f : scale_inverse(b);
  if (in) {
    // (0 * NaN and 0 * Inf would be NaN codes: the bytes of a NaN block are 0)
    const uint32_t w0 = b == 255 ? 0u : pack_e4m3(v, inv);
    if constexpr (V == 8) *reinterpret_cast<v2u_t*>(p) = v2u_t{w0, b == 255 ? 0u : pack_e4m3(v + 4, inv)};
    else *reinterpret_cast<uint32_t*>(p) = w0;
  }
  return b;
}

// One thread per V columns; a row is padded to whole groups of 128 columns, whose threads
// past the width only write the padding scales. 16384 bfloat16 rows of 7168: 104 us from HBM,
// 66 us where the rows lie in the Infinity Cache (0.36 GB at 3.4 and 5.4 TB/s).
template <bool BF16, int V>
__global__ __launch_bounds__(kCkThreads) void ck_quantize_kernel(const void* __restrict__ src,
                                                                 int64_t rows, int width, RowSplit sp,
                                                                 uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scales) {
  const int srow = (width + 127) / 128 * 4;
  for (int64_t r = int64_t(blockIdx.x) * sp.rows() + sp.row(); r < rows;
       r += int64_t(gridDim.x) * sp.rows()) {
    for (int c = sp.first() * V; c < srow * 32; c += sp.step() * V) {
      const bool in = c < width;
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.f;
      if (in) load_v<BF16, V>(src, r * width + c, v);
      const uint32_t b = quantise_v<V>(v, in, q + r * width + c);
      if ((c & 31) == 0) scales[r * srow + c / 32] = uint8_t(b);
    }
  }
}

// Read and convert a token's row once, write it to the K destinations, whose numbers stay in
// the CU's cache. Bound by its writes: 16384 bfloat16 rows of 7168 to K = 8 places, 383 us,
// 2.0 GB at 5.2 TB/s. Rows that do not fill a workgroup share one: 32768 rows of 32, with
// their quantisation, 12 us against 38 with a workgroup per row; of 256, 37 against 54.
template <bool BF16, int V>
__global__ __launch_bounds__(kCkThreads) void ck_dispatch_kernel(
    const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales, int width, int N, int K,
    RowSplit sp, const int32_t* __restrict__ slot_map, void* __restrict__ dst, int64_t ndst) {
  const int srow = (width + 127) / 128 * 4;
  for (int64_t g = int64_t(blockIdx.x) * sp.rows() + sp.row(); g < N;
       g += int64_t(gridDim.x) * sp.rows()) {
    for (int c = sp.first() * V; c < width; c += sp.step() * V) {
      float v[V];
      load_q<V>(q + g * width + c, scale_value(scales[g * srow + c / 32]), v);
      for (int k = 0; k < K; ++k) {
        const int d = slot_map[g * K + k];
        if (d >= 0 && d < ndst) store_v<BF16, V>(dst, int64_t(d) * width + c, v);
      }
    }
  }
}

// gate column of intermediate column p in a [.., 2H'] row
__device__ inline int gate_at(int p) {
  return 2 * kSwigluBlock * (p / kSwigluBlock) + p % kSwigluBlock;
}

// Exact quotient by a fixed divisor: magic = floor(2^64 / d) + 1, right for n * d < 2^64.
struct Divider {
  uint64_t magic;
  int d;
  __device__ int64_t quotient(int64_t n) const { return d == 1 ? n : int64_t(__umul64hi(uint64_t(n), magic)); }
};
static Divider divider(int d) { return Divider{~uint64_t(0) / uint64_t(d) + 1, d}; }

// One thread per 4 intermediate columns, 8 lanes per (gate, up) block pair, rows and
// columns in one index (a workgroup per row leaves a third of its threads idle at
// H' = 1408, 11% slower; 8 columns per thread split each 128-byte line over two loads).
// 262144 bfloat16 rows, H' = 1408: 832 us, 4.45 GB at 5.3 TB/s.
template <bool BF16>
__global__ __launch_bounds__(kCkThreads) void ck_swiglu_kernel(const float* __restrict__ h,
                                                               int64_t rows, int Hp, Divider per_row,
                                                               void* __restrict__ act,
                                                               uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ scales) {
  const int srow = (2 * Hp + 127) / 128 * 4;
  const int64_t total = rows * per_row.d;
  for (int64_t i = blockIdx.x * int64_t(kCkThreads) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kCkThreads) {
    const int64_t r = per_row.quotient(i);
    const int p = int(i - r * per_row.d) * 4;
    const int gc = gate_at(p);
    const int64_t at = r * 2 * Hp + gc;
    float g[4], u[4], a[4];
    load_v<false, 4, true>(h, at, g);
    load_v<false, 4, true>(h, at + kSwigluBlock, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = swiglu_f32(g[j], u[j]);
    store_v<BF16, 4>(act, r * Hp + p, a);
    const uint32_t bg = quantise_v<4>(g, true, q + at);
    const uint32_t bu = quantise_v<4>(u, true, q + at + kSwigluBlock);
    if (p % kSwigluBlock == 0) {
      uint8_t* s = scales + r * srow + gc / 32;
      *reinterpret_cast<uint16_t*>(s) = uint16_t(bg | (bu << 8));
      if (p + kSwigluBlock == Hp)   // the row's padding scales
        for (int j = gc / 32 + 2; j < srow; ++j) scales[r * srow + j] = 0;
    }
  }
}

// 1 << shift threads of a wavefront per row; the row's dot product is summed over them by
// butterfly. 262144 bfloat16 rows, H' = 1408, with gates: 868-912 us, 4.46 GB at 5 TB/s.
template <bool BF16, bool GATED>
__global__ __launch_bounds__(kCkThreads) void ck_swiglu_backward_kernel(
    const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
    const float* __restrict__ da, int64_t rows, int Hp, RowSplit sp,
    const int32_t* __restrict__ src_index, const float* __restrict__ gates, void* __restrict__ act,
    void* __restrict__ dh, float* __restrict__ dgates) {
  const int srow = (2 * Hp + 127) / 128 * 4;
  for (int64_t r = int64_t(blockIdx.x) * sp.rows() + sp.row(); r < rows;
       r += int64_t(gridDim.x) * sp.rows()) {
    float w = 1.f, dot = 0.f;
    int64_t u = -1;
    if (GATED) {
      u = src_index[r];
      if (u < 0 || u >= rows) u = -1;
      w = u >= 0 ? gates[u] : 0.f;
    }
    for (int p = sp.first() * 4; p < Hp; p += sp.step() * 4) {
      const int gc = gate_at(p);
      const int64_t at = r * 2 * Hp + gc;
      float a[4], dg[4], du[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) a[c] = dg[c] = du[c] = 0.f;
      if (!GATED || u >= 0) {
        const uint32_t s = *reinterpret_cast<const uint16_t*>(scales + r * srow + gc / 32);
        float g[4], v[4], d[4];
        load_q<4>(q + at, scale_value(s & 255), g);
        load_q<4>(q + at + kSwigluBlock, scale_value(s >> 8), v);
        load_v<false, 4, true>(da, r * Hp + p, d);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float sg = 1.0f / (1.0f + expf(-g[c]));
          const float gs = g[c] * sg;
          const float ac = gs * v[c];
          const float dc = d[c] * w;
          if (GATED) dot = fmaf(ac, d[c], dot);
          a[c] = ac * w;
          dg[c] = dc * v[c] * (sg + gs * (1.0f - sg));
          du[c] = dc * gs;
        }
      }
      store_v<BF16, 4>(act, r * Hp + p, a);
      store_v<BF16, 4>(dh, at, dg);
      store_v<BF16, 4>(dh, at + kSwigluBlock, du);
    }
    if (GATED) {
      for (int o = sp.step() / 2; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
      if (sp.first() == 0 && u >= 0) dgates[u] = dot;
    }
  }
}

static int ck_grid(int64_t work, int64_t per_block) {
  const int64_t blocks = (work + per_block - 1) / per_block;
  return int(blocks < 1 ? 1 : (blocks > 65536 ? 65536 : blocks));
}

}  // namespace moonep

using namespace moonep;

extern "C" int moonep_checkpoint_quantize(const moonep_shape* shape, int32_t width,
                                          const void* src, uint8_t* q, uint8_t* scales,
                                          void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.mode != MOONEP_TRAIN) return MOONEP_EMODE;
  if (width != s.H && width != s.Hp) return MOONEP_EINVAL;
  const int64_t N = int64_t(s.R) * s.S;
  if (N == 0) return MOONEP_OK;
  if (!aligned16(src) || !aligned16(q) || !aligned16(scales)) return MOONEP_EINVAL;
  // 8 columns per thread; 4 where a float32 row is no multiple of 8
  const bool eight = width % 8 == 0;
  const RowSplit sp = row_split(scale_row(width) * (eight ? 4 : 8), kCkThreads);
  const int grid = ck_grid(N, sp.rows());
  hipStream_t strm = as_stream(stream);
  if (s.dtype == MOONEP_BF16)
    ck_quantize_kernel<true, 8><<<grid, kCkThreads, 0, strm>>>(src, N, width, sp, q, scales);
  else if (eight)
    ck_quantize_kernel<false, 8><<<grid, kCkThreads, 0, strm>>>(src, N, width, sp, q, scales);
  else
    ck_quantize_kernel<false, 4><<<grid, kCkThreads, 0, strm>>>(src, N, width, sp, q, scales);
  return launch_status();
}

extern "C" int moonep_checkpoint_dispatch(const moonep_shape* shape, int32_t width,
                                          const uint8_t* q, const uint8_t* scales,
                                          const int32_t* slot_map, void* dst, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.mode != MOONEP_TRAIN) return MOONEP_EMODE;
  if (width != s.H && width != s.Hp) return MOONEP_EINVAL;
  const int N = s.R * s.S;
  if (N == 0) return MOONEP_OK;
  if (!aligned16(q) || !aligned16(scales) || !aligned16(slot_map) || !aligned16(dst))
    return MOONEP_EINVAL;
  const int64_t ndst = int64_t(N) * s.K;
  const RowSplit sp = row_split(width / (s.dtype == MOONEP_BF16 ? 8 : 4), kCkThreads);
  const int grid = ck_grid(N, sp.rows());
  hipStream_t strm = as_stream(stream);
  if (s.dtype == MOONEP_BF16)
    ck_dispatch_kernel<true, 8><<<grid, kCkThreads, 0, strm>>>(q, scales, width, N, s.K, sp, slot_map, dst, ndst);
  else
    ck_dispatch_kernel<false, 4><<<grid, kCkThreads, 0, strm>>>(q, scales, width, N, s.K, sp, slot_map, dst, ndst);
  return launch_status();
}

extern "C" int moonep_swiglu_checkpoint(const moonep_shape* shape, const float* h, void* act,
                                        uint8_t* q, uint8_t* scales, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.mode != MOONEP_TRAIN) return MOONEP_EMODE;
  if (s.Hp % kSwigluBlock) return MOONEP_EINVAL;
  const int64_t rows = int64_t(s.R) * s.S * s.K;
  if (rows == 0) return MOONEP_OK;
  if (!aligned16(h) || !aligned16(act) || !aligned16(q) || !aligned16(scales)) return MOONEP_EINVAL;
  const Divider per_row = divider(s.Hp / 4);
  const int grid = ck_grid(rows * (s.Hp / 4), kCkThreads);
  if (s.dtype == MOONEP_BF16)
    ck_swiglu_kernel<true><<<grid, kCkThreads, 0, as_stream(stream)>>>(h, rows, s.Hp, per_row, act, q, scales);
  else
    ck_swiglu_kernel<false><<<grid, kCkThreads, 0, as_stream(stream)>>>(h, rows, s.Hp, per_row, act, q, scales);
  return launch_status();
}

extern "C" int moonep_swiglu_backward_checkpoint(const moonep_shape* shape, const uint8_t* q,
                                                 const uint8_t* scales, const float* da,
                                                 const int32_t* src_index, const float* gates,
                                                 void* act, void* dh, float* dgates,
                                                 void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.mode != MOONEP_TRAIN) return MOONEP_EMODE;
  if (s.Hp % kSwigluBlock) return MOONEP_EINVAL;
  const int64_t rows = int64_t(s.R) * s.S * s.K;
  if (rows == 0) return MOONEP_OK;
  if (!aligned16(q) || !aligned16(scales) || !aligned16(da) || !aligned16(act) || !aligned16(dh))
    return MOONEP_EINVAL;
  if (gates ? !aligned16(gates) || !aligned16(src_index) || !aligned16(dgates)
            : src_index || dgates)
    return MOONEP_EINVAL;
  const RowSplit sp = row_split(s.Hp / 4, 64);
  const int grid = ck_grid(rows, sp.rows());
  hipStream_t strm = as_stream(stream);
#define MOONEP_CK_BACKWARD(BF, G) \
  ck_swiglu_backward_kernel<BF, G><<<grid, kCkThreads, 0, strm>>>(q, scales, da, rows, s.Hp, sp, src_index, gates, act, dh, dgates)
  if (s.dtype == MOONEP_BF16) {
    if (gates) MOONEP_CK_BACKWARD(true, true);
    else MOONEP_CK_BACKWARD(true, false);
  } else {
    if (gates) MOONEP_CK_BACKWARD(false, true);
    else MOONEP_CK_BACKWARD(false, false);
  }
#undef MOONEP_CK_BACKWARD
  return launch_status();
}
