// Experts in 4 bits on gfx950: quantisation of token rows and weights to MXFP4, prefetch of
// 4-bit replicas, and the grouped GEMM on them (v_mfma_scale_f32_16x16x128_f8f6f4, which
// takes e2m1 operands and one scale byte per 32 values). Layouts: moonep.h, "Experts in 4
// bits"; the weight layout is the order in which a wavefront's lanes take an operand, so
// every load of it is 1 KiB in a row.
#include "common.h"

namespace moonep {

constexpr int kMxThreads = 256;
typedef float v4f_t __attribute__((ext_vector_type(4)));
typedef int v4i_t __attribute__((ext_vector_type(4)));
typedef int v8i_t __attribute__((ext_vector_type(8)));

__device__ inline uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// 8 values (scaled to at most 6) as 8 e2m1 nibbles, to nearest even
__device__ inline uint32_t pack_e2m1(const float* v, float inv) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
  return w;
}

template <bool BF16>
__device__ inline void load8(const void* base, int64_t idx, float* v) {
  if (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + idx);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    const v4f_t* p = reinterpret_cast<const v4f_t*>(static_cast<const float*>(base) + idx);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i / 4][i % 4];
  }
}

// One thread per 8 values, 4 neighbouring lanes per block; rows padded to whole chunks of
// 512, whose threads past the k-tiles only write the padding scales.
template <bool BF16>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_kernel(const void* __restrict__ src,
                                                                 int64_t rows, int width, int KT,
                                                                 int KC, uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scales) {
  const int per_row = KC * 64;
  const int64_t total = rows * per_row;
  for (int64_t i = blockIdx.x * int64_t(kMxThreads) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kMxThreads) {
    const int64_t r = i / per_row;
    const int c = int(i - r * per_row);       // 8 values each
    float v[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (c * 8 < width) load8<BF16>(src, r * width + c * 8, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, mag_bits(v[j]));
    m = max(m, uint32_t(__shfl_xor(int(m), 1, 64)));
    m = max(m, uint32_t(__shfl_xor(int(m), 2, 64)));
    const uint32_t b = scale_byte<E2M1>(m);
    if (c * 8 < KT * 128)
      *reinterpret_cast<uint32_t*>(q + r * (KT * 64) + c * 4) =
          b == 255 ? 0u : pack_e2m1(v, scale_inverse(b));
    if ((c & 3) == 0) {
      const int blk = c >> 2;
      scales[r * (KC * 16) + (blk >> 4) * 16 + (blk & 3) * 4 + ((blk >> 2) & 3)] = uint8_t(b);
    }
  }
}

// One thread per (column, block of 32 k), columns across lanes: reads are coalesced rows of
// w, and 16 lanes write 256 bytes in a row. blockIdx.y is the expert.
template <bool BF16>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_weight_kernel(
    const void* __restrict__ w, int H, int Hp, int KT, int KC, uint8_t* __restrict__ wq,
    uint8_t* __restrict__ ws) {
  const int64_t e = blockIdx.y;
  const int nblk = KC * 16;
  const int64_t total = int64_t(nblk) * Hp;
  for (int64_t i = blockIdx.x * int64_t(kMxThreads) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kMxThreads) {
    const int blk = int(i / Hp), n = int(i % Hp);
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = 0.f;
      if (blk * 32 < H) {
        const int64_t at = (e * H + blk * 32 + j) * Hp + n;
        v[j] = BF16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(w)[at]) << 16)
                    : static_cast<const float*>(w)[at];
      }
      m = max(m, mag_bits(v[j]));
    }
    const uint32_t b = scale_byte<E2M1>(m);
    const float inv = b == 255 ? 0.f : scale_inverse(b);
    const int lane = 16 * (blk & 3) + (n & 15);
    const int64_t tile = e * (Hp / 16) + n / 16;
    if (blk < KT * 4) {
      uint4 o = make_uint4(0, 0, 0, 0);
      if (b != 255)
        o = make_uint4(pack_e2m1(v, inv), pack_e2m1(v + 8, inv), pack_e2m1(v + 16, inv),
                       pack_e2m1(v + 24, inv));
      reinterpret_cast<uint4*>(wq)[(tile * KT + blk / 4) * 64 + lane] = o;
    }
    ws[((tile * KC + blk / 16) * 64 + lane) * 4 + (blk / 4) % 4] = uint8_t(b);
  }
}

// Copies of home rows into used prefetch slots, values and scales in one launch.
__global__ __launch_bounds__(kMxThreads) void mx_prefetch_kernel(const int32_t* __restrict__ replica,
                                                                 int RB, int E, uint4* wq,
                                                                 int64_t qvec, uint4* ws,
                                                                 int64_t svec) {
  const int64_t stride = int64_t(gridDim.x) * kMxThreads;
  const int64_t i0 = int64_t(blockIdx.x) * kMxThreads + threadIdx.x;
  for (int s = 0; s < RB; ++s) {
    const int e = replica[s];
    if (e < 0 || e >= E) continue;
    for (int64_t i = i0; i < qvec + svec; i += stride) {
      if (i < qvec) wq[(int64_t(E) + s) * qvec + i] = wq[int64_t(e) * qvec + i];
      else ws[(int64_t(E) + s) * svec + i - qvec] = ws[int64_t(e) * svec + i - qvec];
    }
  }
}

struct MxArgs {
  const uint8_t* xq;
  const uint8_t* xs;
  const int32_t* src_index;
  const uint8_t* wq;
  const uint8_t* ws;
  float* c;
  const TileEntry* tiles;
  const int32_t* ntiles;
  int K, Hp, KT, KC;
  int64_t NK;
};

constexpr int kMxRows = 64;   // rows of a work entry

// One workgroup per (entry, 64 columns): wavefront w multiplies 16 rows with 64 columns,
// operands straight from memory.
__global__ __launch_bounds__(256) void mx_gemm_kernel(MxArgs a) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int NT = a.Hp / 64;
  const int64_t total = int64_t(*a.ntiles) * NT;
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const TileEntry te = a.tiles[t / NT];
    const int n0 = int(t % NT) * 64;
    const int r0 = te.m0 + w * 16;
    if (r0 >= te.n) continue;
    int64_t arow = int64_t(te.rowbase) + r0 + (lane & 15);
    bool in = r0 + (lane & 15) < te.n;
    if (a.src_index) {
      const int u = in ? a.src_index[arow] : -1;
      in = u >= 0 && u < a.NK;
      arow = in ? u / a.K : 0;
    }
    v4f_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = v4f_t{0.f, 0.f, 0.f, 0.f};
    const int kb = lane >> 4;
    for (int kt = 0; kt < a.KT; ++kt) {
      v8i_t fa = {0, 0, 0, 0, 0, 0, 0, 0};
      int sa = 0;
      if (in) {
        const v4i_t x = *reinterpret_cast<const v4i_t*>(a.xq + (arow * a.KT + kt) * 64 + kb * 16);
        fa[0] = x[0]; fa[1] = x[1]; fa[2] = x[2]; fa[3] = x[3];
        sa = a.xs[(arow * a.KC + kt / 4) * 16 + kb * 4 + kt % 4];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t tile = int64_t(te.wrow) * (a.Hp / 16) + n0 / 16 + j;
        const v4i_t x = reinterpret_cast<const v4i_t*>(a.wq)[(tile * a.KT + kt) * 64 + lane];
        const v8i_t fb = {x[0], x[1], x[2], x[3], 0, 0, 0, 0};
        const int sb = a.ws[((tile * a.KC + kt / 4) * 64 + lane) * 4 + kt % 4];
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa, fb, acc[j], 4, 4, 0, sa, 0, sb);
      }
    }
    // lane holds column lane % 16 and rows 4 * (lane / 16) + r of each block
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = r0 + 4 * (lane >> 4) + r;
      if (row >= te.n) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a.c[(int64_t(te.rowbase) + row) * a.Hp + n0 + j * 16 + (lane & 15)] = acc[j][r];
    }
  }
}

static int mx_grid(int64_t work, int64_t cap) {
  const int64_t blocks = (work + kMxThreads - 1) / kMxThreads;
  return int(blocks < 1 ? 1 : (blocks > cap ? cap : blocks));
}

}  // namespace moonep

using namespace moonep;

extern "C" int moonep_mx_quantize(const moonep_shape* shape, int64_t rows, int32_t width,
                                  const void* src, uint8_t* q, uint8_t* scales, void* stream) {
  int st = validate(shape);
  if (st) return st;
  if (rows < 0 || rows > INT32_MAX || width < kScaleBlock || width % kScaleBlock)
    return MOONEP_EINVAL;
  if (rows == 0) return MOONEP_OK;
  if (!aligned16(src) || !aligned16(q) || !aligned16(scales)) return MOONEP_EINVAL;
  const int KT = int(k_tiles(width)), KC = int(k_chunks(width));
  const int grid = mx_grid(rows * KC * 64, 65536);
  if (shape->dtype == MOONEP_BF16)
    mx_quantize_kernel<true><<<grid, kMxThreads, 0, as_stream(stream)>>>(src, rows, width, KT, KC, q, scales);
  else
    mx_quantize_kernel<false><<<grid, kMxThreads, 0, as_stream(stream)>>>(src, rows, width, KT, KC, q, scales);
  return launch_status();
}

extern "C" int moonep_mx_quantize_weight(const moonep_shape* shape, const void* w, uint8_t* wq,
                                         uint8_t* wscales, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.H % kScaleBlock || s.Hp % 16) return MOONEP_EINVAL;
  if (!aligned16(w) || !aligned16(wq) || !aligned16(wscales)) return MOONEP_EINVAL;
  const int KT = int(k_tiles(s.H)), KC = int(k_chunks(s.H));
  const dim3 grid(mx_grid(int64_t(KC) * 16 * s.Hp, 1024), s.E);
  if (s.dtype == MOONEP_BF16)
    mx_quantize_weight_kernel<true><<<grid, kMxThreads, 0, as_stream(stream)>>>(w, s.H, s.Hp, KT, KC, wq, wscales);
  else
    mx_quantize_weight_kernel<false><<<grid, kMxThreads, 0, as_stream(stream)>>>(w, s.H, s.Hp, KT, KC, wq, wscales);
  return launch_status();
}

extern "C" int moonep_mx_prefetch_weight(const moonep_shape* shape, const int32_t* replica_expert,
                                         uint8_t* wq, uint8_t* wscales, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.Hp % 16) return MOONEP_EINVAL;
  if (s.B == 0) return MOONEP_OK;
  if (!aligned16(replica_expert) || !aligned16(wq) || !aligned16(wscales)) return MOONEP_EINVAL;
  const int64_t qvec = int64_t(s.Hp / 16) * k_tiles(s.H) * 64;
  const int64_t svec = int64_t(s.Hp / 16) * k_chunks(s.H) * 16;
  mx_prefetch_kernel<<<mx_grid(qvec + svec, 2048), kMxThreads, 0, as_stream(stream)>>>(
      replica_expert, s.R * s.B, s.E, reinterpret_cast<uint4*>(wq), qvec,
      reinterpret_cast<uint4*>(wscales), svec);
  return launch_status();
}

extern "C" int moonep_mx_grouped_gemm(const moonep_shape* shape, const uint8_t* xq,
                                      const uint8_t* xscales, const int32_t* src_index,
                                      const uint8_t* wq, const uint8_t* wscales,
                                      const int32_t* cu_seqlens, float* c, void* ws,
                                      size_t ws_bytes, void* stream) {
  int st = validate(shape);
  if (st) return st;
  const moonep_shape& s = *shape;
  if (s.H % 64 || s.Hp % 64) return MOONEP_EINVAL;
  if (!aligned16(cu_seqlens) || !aligned16(ws)) return MOONEP_EINVAL;
  if (ws_bytes < ws_layout(s).total) return MOONEP_EWORKSPACE;
  if (s.S == 0) return MOONEP_OK;
  if (!aligned16(xq) || !aligned16(xscales) || !aligned16(wq) || !aligned16(wscales) ||
      !aligned16(c) || (src_index && !aligned16(src_index)))
    return MOONEP_EINVAL;
  const int cus = device_cus();
  if (cus <= 0) return MOONEP_EHIP;
  hipStream_t strm = as_stream(stream);
  MxArgs a{xq, xscales, src_index, wq, wscales, c, nullptr, nullptr, s.K, s.Hp,
           int(k_tiles(s.H)), int(k_chunks(s.H)), int64_t(s.R) * s.S * s.K};
  st = launch_tile_list(s, cu_seqlens, kMxRows, ws, strm, &a.tiles, &a.ntiles);
  if (st) return st;
  mx_gemm_kernel<<<cus * 8, 256, 0, strm>>>(a);
  return launch_status();
}
