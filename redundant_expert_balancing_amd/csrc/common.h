// Internal definitions shared by the HIP sources of the moonep library.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moonep.h"

namespace moonep {

// Router tokens per planning chunk: one 64-wide wavefront owns a chunk, one lane
// per token while counting, 64 consecutive slots per step while assigning.
constexpr int kChunkTokens = 64;
// Chunks per partition of the planner's column scan (16 wavefronts x 4 chunks).
constexpr int kScanPart = 64;
// Layers of at most kFusedMaxChunks chunks count, scan and solve in one launch:
// kFusedChunks chunks (one per wavefront) per workgroup, each workgroup a partition.
constexpr int kFusedChunks = 16;
constexpr int kFusedMaxChunks = 256;
// Smallest GEMM M tile; sizes the tile list in the workspace.
constexpr int kMinTileM = 64;

// Sticky error word and per-call words at the head of the workspace.
enum FlagWord {
  kFlagError = 0, kFlagPlanValid = 1, kFlagTileCount = 2, kFlagTileCountTail = 3,
  kFlagPlanArrive = 4,   // workgroups of the fused planner done counting (back to 0 after)
  kFlagQueue = 16,   // 2 x kQueueWords GEMM tile-queue counters
  kFlagWords = 64
};
constexpr int kQueueWords = 8;   // one tile-queue counter per XCD

struct WsLayout {
  size_t flags, part, counts, piece_ptr, piece_tlo, piece_base, tiles, tiles_tail, total;
  int64_t nchunk, npart, nfused, max_pieces, max_tiles, max_tail;
};

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline WsLayout ws_layout(const moonep_shape& s) {
  WsLayout w{};
  const int64_t N = int64_t(s.R) * s.S;
  const int64_t SK = int64_t(s.S) * s.K;
  w.nchunk = (N + kChunkTokens - 1) / kChunkTokens;
  w.npart = (w.nchunk + kScanPart - 1) / kScanPart;
  w.nfused = w.nchunk > 0 && w.nchunk <= kFusedMaxChunks
                 ? (w.nchunk + kFusedChunks - 1) / kFusedChunks : 0;
  w.max_pieces = int64_t(s.E) + 2 * int64_t(s.R) + 8;
  w.max_tiles = int64_t(s.R) * ((SK + kMinTileM - 1) / kMinTileM + s.E + s.B) + 1;
  w.max_tail = int64_t(s.R) * (s.E + s.B) + 1;   // at most one short tail per segment
  size_t o = 0;
  w.flags = o;      o = align256(o + kFlagWords * 4);
  w.part = o;       o = align256(o + size_t(w.npart > w.nfused ? w.npart : w.nfused) * s.E * 4);
  w.counts = o;     o = align256(o + size_t(w.nchunk) * s.E * 4);
  w.piece_ptr = o;  o = align256(o + size_t(s.E + 1) * 4);
  w.piece_tlo = o;  o = align256(o + size_t(w.max_pieces) * 4);
  w.piece_base = o; o = align256(o + size_t(w.max_pieces) * 4);
  w.tiles = o;      o = align256(o + size_t(w.max_tiles) * 16);
  w.tiles_tail = o; o = align256(o + size_t(w.max_tail) * 16);
  w.total = o;
  return w;
}

template <typename T>
inline T* ws_ptr(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

inline bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// float32 -> bfloat16 bits, round to nearest, ties to even (finite inputs).
__device__ inline uint32_t bf16_rne_bits(float f) {
  uint32_t b = __float_as_uint(f);
  b += 0x7FFFu + ((b >> 16) & 1u);
  return b >> 16;
}

// The same for any input: a NaN stays one (rounding up its mantissa could carry out of it).
__device__ inline uint32_t bf16_rne_any(float f) {
  return f == f ? bf16_rne_bits(f) : 0x7FC0u;
}

// Block scales (E8M0: the byte is the exponent plus 127, 255 is NaN) of small float types.
// The scale of a block is the smallest power of two 2^e, e >= -127, with
// amax <= top * 2^e, so that no value is clipped; top is 448 (e4m3) or 6 (e2m1), given by
// its exponent and mantissa bits. amax_bits: the largest |value| of the block as bits;
// integer order ranks Inf and NaN above every number, and either makes the scale NaN.
struct E4M3 { static constexpr int kTopExp = 8; static constexpr uint32_t kTopMant = 0x600000u; };
struct E2M1 { static constexpr int kTopExp = 2; static constexpr uint32_t kTopMant = 0x400000u; };

template <typename T>
__device__ inline uint32_t scale_byte(uint32_t amax_bits) {
  const int e = int(amax_bits >> 23);
  if (e == 255) return 255;
  const int b = e - T::kTopExp + ((amax_bits & 0x7FFFFFu) > T::kTopMant ? 1 : 0);
  return uint32_t(b < 0 ? 0 : b);
}
// Largest magnitude that e4m3 with a float32 scale is rounded from: 240 * 2^120. What lies above
// (up to float32's largest, 256 * 2^120 less a step) would round to 2^128.
constexpr float kE4m3Max = 0x1.ep127f;
__device__ inline float clamp_e4m3(float v) { return __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max); }
// 2^-e of a scale byte (at most 254 for a finite block), exact
__device__ inline float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^e of a scale byte: byte 0 is the subnormal 2^-127
__device__ inline float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte ? byte << 23 : 0x400000u);
}

// SwiGLU in float32: silu(g) * u with silu(g) = g / (1 + e^-g). Every kernel that
// produces the activation calls this one function, so all of them agree bit for bit.
__device__ inline float swiglu_f32(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Gate/up columns of the FFN's first projection are interleaved in blocks of
// kSwigluBlock: intermediate column p has its gate at 2*kSwigluBlock*(p / kSwigluBlock)
// + p % kSwigluBlock and its up projection kSwigluBlock further.
constexpr int kSwigluBlock = MOONEP_SWIGLU_BLOCK;

// Row-wise kernels of kRowThreads threads: a workgroup has 256 >> shift rows of 1 << shift
// threads, so that rows narrower than a workgroup share one, and no thread divides.
constexpr int kRowThreads = 256;
struct RowSplit {
  int shift;
  __device__ int row() const { return int(threadIdx.x) >> shift; }
  __device__ int first() const { return int(threadIdx.x) & ((1 << shift) - 1); }
  __device__ int step() const { return 1 << shift; }
  __host__ __device__ int rows() const { return kRowThreads >> shift; }
};

// Threads per row for `items` work items of a row, at most `most`.
inline RowSplit row_split(int64_t items, int most) {
  int shift = 0;
  while ((1 << shift) < items && (1 << shift) < most) ++shift;
  return RowSplit{shift};
}

// Layouts of the 4-bit expert operands (moonep.h, "Experts in 4 bits"): tiles of 128 and
// chunks of 512 along the reduction.
constexpr int kScaleBlock = 32;
inline int64_t k_tiles(int width) { return (int64_t(width) + 127) / 128; }
inline int64_t k_chunks(int width) { return (int64_t(width) + 511) / 512; }

// Host-side validation shared by all entry points (defined in api.hip).
int validate(const moonep_shape* s);
int elem_bytes(const moonep_shape& s);
int launch_status();  // MOONEP_OK or MOONEP_EHIP after the last launch

// One work entry of the grouped GEMMs' tile lists (gemm.hip).
struct TileEntry {
  int32_t rowbase;  // global buffer row of the segment's first slot: q*SK + cu[q][i]
  int32_t wrow;     // W_all row (FWD/DGRAD) / grad row (WGRAD: < E grad_home, else reduce_buf+E)
  int32_t m0;       // first segment row of this entry (FWD/DGRAD), 0 for WGRAD
  int32_t n;        // segment length
};

// Enqueues the tile list of `s` and cu_seqlens, M-tiles of bm rows (bm >= kMinTileM), into
// the workspace (gemm.hip); *tiles and *ntiles receive its device addresses.
int launch_tile_list(const moonep_shape& s, const int32_t* cu_seqlens, int bm, void* ws,
                     hipStream_t strm, const TileEntry** tiles, const int32_t** ntiles);
int device_cus();   // compute units of the current device, 0 on failure

}  // namespace moonep
