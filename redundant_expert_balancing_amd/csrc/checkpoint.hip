// 8-bit activation checkpoints on gfx950 (format and rounding: moonep.h): quantisation of
// token rows, the permute that reads them back, and the SwiGLU forward and backward with
// the pre-activation kept in 8 bits. All are HBM-bound passes: one read and one write of
// each array, 16-byte vectors of the wide side, the conversions by the hardware's
// float32 <-> e4m3 instructions (round to nearest even; the power-of-two scale is exact).
#include "common.h"

namespace moonep {

constexpr int kCkThreads = 256;
typedef float v4f_t __attribute__((ext_vector_type(4)));
typedef float v2f_t __attribute__((ext_vector_type(2)));

inline int64_t scale_row(int width) { return 4 * ((int64_t(width) + 127) / 128); }

__device__ inline uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ inline uint32_t amax4(v4f_t v) {
  return max(max(mag_bits(v.x), mag_bits(v.y)), max(mag_bits(v.z), mag_bits(v.w)));
}

// 4 values scaled by inv as 4 e4m3 bytes
__device__ inline uint32_t pack_e4m3(v4f_t v, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v.x * inv, v.y * inv, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v.z * inv, v.w * inv, w, true));
}

__device__ inline v4f_t unpack_e4m3(uint32_t w, float scale) {
  const v2f_t a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false);
  const v2f_t b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
  return v4f_t{a.x * scale, a.y * scale, b.x * scale, b.y * scale};
}

template <bool BF16>
__device__ inline v4f_t load4(const void* base, int64_t idx) {
  if (BF16) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + idx);
    return v4f_t{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                 __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
  }
  return *reinterpret_cast<const v4f_t*>(static_cast<const float*>(base) + idx);
}

template <bool BF16>
__device__ inline void store4(void* base, int64_t idx, v4f_t v) {
  if (BF16) {
    uint2 w;
    w.x = bf16_rne_any(v.x) | (bf16_rne_any(v.y) << 16);
    w.y = bf16_rne_any(v.z) | (bf16_rne_any(v.w) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + idx) = w;
  } else {
    *reinterpret_cast<v4f_t*>(static_cast<float*>(base) + idx) = v;
  }
}

// the largest magnitude of the 8 lanes that share a block
__device__ inline uint32_t max_of_8(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) m = max(m, uint32_t(__shfl_xor(int(m), d, 64)));
  return m;
}

// One thread per 4 columns, 8 neighbouring lanes per block; rows padded to whole groups of
// 128 columns, whose threads past the width only write the padding scales.
template <bool BF16>
__global__ __launch_bounds__(kCkThreads) void ck_quantize_kernel(const void* __restrict__ src,
                                                                 int64_t rows, int width,
                                                                 uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scales) {
  const int per_row = (width + 127) / 128 * 32;
  const int64_t total = rows * per_row;
  for (int64_t i = blockIdx.x * int64_t(kCkThreads) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kCkThreads) {
    const int64_t r = i / per_row;
    const int c = int(i - r * per_row) * 4;
    const bool in = c < width;
    const v4f_t v = in ? load4<BF16>(src, r * width + c) : v4f_t{0.f, 0.f, 0.f, 0.f};
    const uint32_t b = scale_byte<E4M3>(max_of_8(amax4(v)));
    if (in)
      *reinterpret_cast<uint32_t*>(q + r * width + c) =
          b == 255 ? 0u : pack_e4m3(v, scale_inverse(b));
    if ((c & 31) == 0) scales[r * (per_row / 8) + c / 32] = uint8_t(b);
  }
}

// One workgroup per token, as the plain dispatch: read and convert the row once, write it
// to the K destinations.
template <bool BF16>
__global__ __launch_bounds__(kCkThreads) void ck_dispatch_kernel(
    const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales, int width, int N, int K,
    const int32_t* __restrict__ slot_map, void* __restrict__ dst, int64_t ndst) {
  __shared__ int32_t s_slot[32];
  const int srow = (width + 127) / 128 * 4;
  for (int64_t g = blockIdx.x; g < N; g += gridDim.x) {
    if (threadIdx.x < K) {
      const int d = slot_map[g * K + threadIdx.x];
      s_slot[threadIdx.x] = (d >= 0 && d < ndst) ? d : -1;
    }
    __syncthreads();
    for (int c = threadIdx.x * 4; c < width; c += kCkThreads * 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(q + g * width + c);
      const v4f_t v = unpack_e4m3(w, scale_value(scales[g * srow + c / 32]));
      for (int k = 0; k < K; ++k) {
        const int d = s_slot[k];
        if (d >= 0) store4<BF16>(dst, int64_t(d) * width + c, v);
      }
    }
    __syncthreads();
  }
}

// One thread per 4 intermediate columns, 8 lanes per (gate, up) block pair.
template <bool BF16>
__global__ __launch_bounds__(kCkThreads) void ck_swiglu_kernel(const float* __restrict__ h,
                                                               int64_t rows, int Hp,
                                                               void* __restrict__ act,
                                                               uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ scales) {
  const int per_row = Hp / 4, srow = (2 * Hp + 127) / 128 * 4;
  const int64_t total = rows * per_row;
  for (int64_t i = blockIdx.x * int64_t(kCkThreads) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kCkThreads) {
    const int64_t r = i / per_row;
    const int p = int(i - r * per_row) * 4;
    const int gc = 2 * kSwigluBlock * (p / kSwigluBlock) + p % kSwigluBlock;
    const int64_t at = r * 2 * Hp + gc;
    const v4f_t g = load4<false>(h, at), u = load4<false>(h, at + kSwigluBlock);
    store4<BF16>(act, r * Hp + p, v4f_t{swiglu_f32(g.x, u.x), swiglu_f32(g.y, u.y),
                                        swiglu_f32(g.z, u.z), swiglu_f32(g.w, u.w)});
    const uint32_t bg = scale_byte<E4M3>(max_of_8(amax4(g)));
    const uint32_t bu = scale_byte<E4M3>(max_of_8(amax4(u)));
    *reinterpret_cast<uint32_t*>(q + at) = bg == 255 ? 0u : pack_e4m3(g, scale_inverse(bg));
    *reinterpret_cast<uint32_t*>(q + at + kSwigluBlock) =
        bu == 255 ? 0u : pack_e4m3(u, scale_inverse(bu));
    if (p % kSwigluBlock == 0) {
      uint8_t* s = scales + r * srow + gc / 32;
      s[0] = uint8_t(bg);
      s[1] = uint8_t(bu);
      if (p + kSwigluBlock == Hp)   // the row's padding scales
        for (int j = gc / 32 + 2; j < srow; ++j) scales[r * srow + j] = 0;
    }
  }
}

// One wavefront per row.
template <bool BF16, bool GATED>
__global__ __launch_bounds__(kCkThreads) void ck_swiglu_backward_kernel(
    const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
    const float* __restrict__ da, int64_t rows, int Hp, const int32_t* __restrict__ src_index,
    const float* __restrict__ gates, void* __restrict__ act, void* __restrict__ dh,
    float* __restrict__ dgates) {
  constexpr int kWaves = kCkThreads / 64;
  const int lane = threadIdx.x & 63;
  const int srow = (2 * Hp + 127) / 128 * 4;
  for (int64_t r = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6); r < rows;
       r += int64_t(gridDim.x) * kWaves) {
    float w = 1.f, dot = 0.f;
    int64_t u = -1;
    if (GATED) {
      u = src_index[r];
      if (u < 0 || u >= rows) u = -1;
      w = u >= 0 ? gates[u] : 0.f;
    }
    for (int p = lane * 4; p < Hp; p += 256) {
      const int gc = 2 * kSwigluBlock * (p / kSwigluBlock) + p % kSwigluBlock;
      const int64_t at = r * 2 * Hp + gc;
      v4f_t a = {0.f, 0.f, 0.f, 0.f}, dg = a, du = a;
      if (!GATED || u >= 0) {
        const uint8_t* s = scales + r * srow + gc / 32;
        const v4f_t g = unpack_e4m3(*reinterpret_cast<const uint32_t*>(q + at), scale_value(s[0]));
        const v4f_t v = unpack_e4m3(*reinterpret_cast<const uint32_t*>(q + at + kSwigluBlock),
                                    scale_value(s[1]));
        const v4f_t d = load4<false>(da, r * Hp + p);
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
      store4<BF16>(act, r * Hp + p, a);
      store4<BF16>(dh, at, dg);
      store4<BF16>(dh, at + kSwigluBlock, du);
    }
    if (GATED) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
      if (lane == 0 && u >= 0) dgates[u] = dot;
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
  const int grid = ck_grid(N * scale_row(width) * 8, kCkThreads);
  if (s.dtype == MOONEP_BF16)
    ck_quantize_kernel<true><<<grid, kCkThreads, 0, as_stream(stream)>>>(src, N, width, q, scales);
  else
    ck_quantize_kernel<false><<<grid, kCkThreads, 0, as_stream(stream)>>>(src, N, width, q, scales);
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
  const int grid = ck_grid(N, 1);
  if (s.dtype == MOONEP_BF16)
    ck_dispatch_kernel<true><<<grid, kCkThreads, 0, as_stream(stream)>>>(q, scales, width, N, s.K,
                                                                         slot_map, dst, ndst);
  else
    ck_dispatch_kernel<false><<<grid, kCkThreads, 0, as_stream(stream)>>>(q, scales, width, N, s.K,
                                                                          slot_map, dst, ndst);
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
  const int grid = ck_grid(rows * (s.Hp / 4), kCkThreads);
  if (s.dtype == MOONEP_BF16)
    ck_swiglu_kernel<true><<<grid, kCkThreads, 0, as_stream(stream)>>>(h, rows, s.Hp, act, q, scales);
  else
    ck_swiglu_kernel<false><<<grid, kCkThreads, 0, as_stream(stream)>>>(h, rows, s.Hp, act, q, scales);
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
  const int grid = ck_grid(rows, kCkThreads / 64);
  hipStream_t strm = as_stream(stream);
#define MOONEP_CK_BACKWARD(BF, G) \
  ck_swiglu_backward_kernel<BF, G><<<grid, kCkThreads, 0, strm>>>(q, scales, da, rows, s.Hp, src_index, gates, act, dh, dgates)
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
