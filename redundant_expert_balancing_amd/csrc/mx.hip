// Experts in 4 bits on gfx950: quantisation of token rows and weights to MXFP4, prefetch of
// 4-bit replicas, and the grouped GEMM on them (v_mfma_scale_f32_16x16x128_f8f6f4, which
// takes e2m1 operands and one scale byte per 32 values). Layouts: moonep.h, "Experts in 4
// bits"; the weight layout is the order in which a wavefront's lanes take an operand, so
// every load of it is 1 KiB in a row.
#include <type_traits>

#include "common.h"
#include "lds_dma.h"

namespace moonep {

constexpr int kMxThreads = 256;
typedef float v4f_t __attribute__((ext_vector_type(4)));
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
// 512, whose threads past the k-tiles only write the padding scales. 65536 bfloat16 rows of
// 4096: 119-124 us, 0.68 GB at 5.6 TB/s.
template <bool BF16>
__global__ __launch_bounds__(kRowThreads) void mx_quantize_kernel(const void* __restrict__ src,
                                                                  int64_t rows, int width, int KT,
                                                                  int KC, RowSplit sp,
                                                                  uint8_t* __restrict__ q,
                                                                  uint8_t* __restrict__ scales) {
  for (int64_t r = int64_t(blockIdx.x) * sp.rows() + sp.row(); r < rows;
       r += int64_t(gridDim.x) * sp.rows()) {
    for (int c = sp.first(); c < KC * 64; c += sp.step()) {
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
      if (c < KT * 16)
        *reinterpret_cast<uint32_t*>(q + r * (KT * 64) + c * 4) =
            b == 255 ? 0u : pack_e2m1(v, scale_inverse(b));
      if ((c & 3) == 0) {
        const int blk = c >> 2;
        scales[r * (KC * 16) + (blk >> 4) * 16 + (blk & 3) * 4 + ((blk >> 2) & 3)] = uint8_t(b);
      }
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

// Copies of home rows into used prefetch slots, values and scales in one launch. 64 experts of
// H = 4096, H' = 1536: 79 us, 0.43 GB at 5.4 TB/s; no slot used: 9 us.
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
  int64_t NK, xrows;
  int32_t* qcnt;    // 8 per-XCD tile-queue counters, zero at launch
};

// One 16 x 16 x 128 product of e2m1 operands (format 4); byte BYTE of each scale word counts.
template <int BYTE>
__device__ inline v4f_t mfma_e2m1(v8i_t a, v8i_t b, v4f_t c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, BYTE, sa, BYTE, sb);
}

// ---- few rows per expert: the call is bound by reading each touched expert's weights once,
// and, for one token, by its launches; so this form needs no list of work. Its work items
// are (share of the rows, segment of the view, 64 columns), dealt out to the workgroups in
// turn; a workgroup's threads look up one item's cu_seqlens each and list the ones that
// have rows. A workgroup's four wavefronts take blocks of 16 rows; where there are fewer
// than three, the wavefronts of a block share its k-chunks in turn and their sums are added
// in the wavefronts' order. Operands go straight to registers, a chunk (512 k, 17 KiB of
// weights) in flight per wavefront. 16 tokens, K = 8, 256 experts, H = 4096, H' = 1536: 48 us,
// 0.34 GB of weights at 7 TB/s, the Infinity Cache holding a part of them.
constexpr int kMxRows = 64;      // rows at a time
constexpr int kMxItems = 256;    // items looked up at a time

// Rows m0 .. m0 + 63 (at most) of one segment, columns n0 .. n0 + 63, by one workgroup.
__device__ inline void few_rows(const MxArgs& a, int rowbase_v, int wrow_v, int m0_v, int n,
                                int n0_v, v4f_t (*s_part)[4][64]) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kb = lane >> 4, r16 = lane & 15;
  const int rowbase = __builtin_amdgcn_readfirstlane(rowbase_v);
  const int wrow = __builtin_amdgcn_readfirstlane(wrow_v);
  const int m0 = __builtin_amdgcn_readfirstlane(m0_v), n0 = __builtin_amdgcn_readfirstlane(n0_v);
  const int rows = __builtin_amdgcn_readfirstlane(min(kMxRows, n - m0));
  const int split = rows <= 16 ? 4 : rows <= 32 ? 2 : 1;   // wavefronts per block of rows
  const int part = w % split, r0 = w / split * 16;
  const bool work = r0 < rows;    // uniform
  v4f_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = v4f_t{0.f, 0.f, 0.f, 0.f};
  if (work) {
    int64_t arow = int64_t(rowbase) + m0 + r0 + r16;
    bool in = r0 + r16 < rows;
    if (a.src_index) {
      const int u = in ? a.src_index[arow] : -1;
      in = u >= 0 && u < a.NK;
      arow = in ? u / a.K : 0;
    }
    const v4i_t* xq = reinterpret_cast<const v4i_t*>(a.xq) + arow * a.KT * 4 + kb;
    const int* xs = reinterpret_cast<const int*>(a.xs) + arow * a.KC * 4 + kb;
    const int64_t tile = int64_t(wrow) * (a.Hp / 16) + n0 / 16;
    const v4i_t* wq = reinterpret_cast<const v4i_t*>(a.wq) + tile * a.KT * 64 + lane;
    const int* ws = reinterpret_cast<const int*>(a.ws) + tile * a.KC * 64 + lane;
    for (int c = part; c < a.KC; c += split) {
      v4i_t fa[4], fb[4][4];
      int sb[4];
      const int sa = in ? xs[c * 4] : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) sb[j] = ws[(j * a.KC + c) * 64];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool there = c * 4 + k < a.KT;   // uniform
        fa[k] = there && in ? xq[(c * 4 + k) * 4] : v4i_t{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          fb[k][j] = there ? wq[(j * a.KT + c * 4 + k) * 64] : v4i_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const v8i_t xa = {fa[k][0], fa[k][1], fa[k][2], fa[k][3], 0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v8i_t xb = {fb[k][j][0], fb[k][j][1], fb[k][j][2], fb[k][j][3], 0, 0, 0, 0};
          // operands swapped: a lane holds 4 columns of one row
          if (k == 0) acc[j] = mfma_e2m1<0>(xb, xa, acc[j], sb[j], sa);
          else if (k == 1) acc[j] = mfma_e2m1<1>(xb, xa, acc[j], sb[j], sa);
          else if (k == 2) acc[j] = mfma_e2m1<2>(xb, xa, acc[j], sb[j], sa);
          else acc[j] = mfma_e2m1<3>(xb, xa, acc[j], sb[j], sa);
        }
      }
    }
  }
  if (split > 1) {       // uniform
    if (part > 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) s_part[w - 1][j][lane] = acc[j];
    __syncthreads();
    if (part == 0)
      for (int o = 1; o < split; ++o)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += s_part[w + o - 1][j][lane];
    __syncthreads();     // read before the next entry's sums
  }
  if (work && part == 0 && r0 + r16 < rows) {
    float* c = a.c + (int64_t(rowbase) + m0 + r0 + r16) * a.Hp + n0 + 4 * kb;
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<v4f_t*>(c + j * 16) = acc[j];
  }
}

struct MxItem {
  int32_t rowbase, wrow, m0, n;  // as TileEntry, and n0 below
};

__global__ __launch_bounds__(256) void mx_gemm_kernel(MxArgs a, const int32_t* __restrict__ cu,
                                                      int R, int E, int B, int SK, int shares) {
  __shared__ __align__(16) v4f_t s_part[3][4][64];
  __shared__ MxItem s_item[kMxItems];
  __shared__ int s_n0[kMxItems];
  __shared__ int s_wave[4];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int NT = a.Hp / 64, EB = E + B;
  const int64_t total = int64_t(R) * EB * shares * NT;
  for (int64_t t0 = blockIdx.x; t0 < total; t0 += int64_t(gridDim.x) * kMxItems) {
    const int64_t t = t0 + int64_t(threadIdx.x) * gridDim.x;
    MxItem it{0, 0, 0, 0};
    int n0 = 0;
    if (t < total) {
      // shares slowest: the empty ones of short segments lie together, over all CUs
      const int64_t rest = t / NT;
      const int seg = int(rest % (R * EB)), share = int(rest / (R * EB));
      const int rank = seg / EB, i = seg % EB;
      const int c0 = cu[int64_t(rank) * (EB + 1) + i];
      n0 = int(t % NT) * 64;
      it = MxItem{rank * SK + c0, i < E ? i : E + rank * B + (i - E), share * kMxRows,
                  cu[int64_t(rank) * (EB + 1) + i + 1] - c0};
    }
    const bool some = it.m0 < it.n;
    const uint64_t have = __ballot(some);
    if (lane == 0) s_wave[w] = __popcll(have);
    __syncthreads();
    int at = __popcll(have & ((uint64_t(1) << lane) - 1)), count = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < w) at += s_wave[i];
      count += s_wave[i];
    }
    if (some) {
      s_item[at] = it;
      s_n0[at] = n0;
    }
    __syncthreads();
    for (int i = 0; i < count; ++i) {
      const MxItem te = s_item[i];
      for (int m0 = te.m0; m0 < te.n; m0 += shares * kMxRows)
        few_rows(a, te.rowbase, te.wrow, m0, te.n, s_n0[i], s_part);
    }
    __syncthreads();     // the list is read before the next one
  }
}

constexpr int kNonTemporal = 2;   // buffer cache policy: the output is not read back here

// ---- tiled form: 128 x 256 output tiles, four wavefronts side by side in N (128 x 64 each),
// 256 k per step: token rows by DMA into two LDS stages, which all wavefronts read; weights,
// which each wavefront has to itself, straight to registers a step ahead.
//
// 524288 slots, 256 experts, H = 4096, H' = 1536: 1.96-2.1 ms, 3.1-3.3 PFLOP/s; H = 7168,
// H' = 2048, 384 experts 4.5 ms, 3.4 PFLOP/s. The matrix pipes are busy 44% of the cycles, at the
// 1.8 GHz that the card's power allows. The rest are waits: each step begins with all loads
// drained, one step in flight. The same loop without its operand loads runs at 5.1 PFLOP/s, on
// operands of zeros (a higher clock) at 4.7, without its stores (3.2 GB of float32) at 4.0. Of no
// use, or slower: 256 x 256 tiles of 8 wavefronts (same time; with both operands in LDS
// they spill), fragments read 2 or 4 ahead, weights double-buffered by 128 k (spills, 9%
// slower), wave priorities, staggered starts, 64-row tiles (10-20% slower where the card
// is full).
struct MxTile {
  static constexpr int FM = 8, FN = 4;                  // 16 x 16 blocks of a wavefront
  static constexpr int BM = 16 * FM, BN = 256, WAVES = 4;
  static constexpr int STEPB = 128;                     // bytes of a row per step
  static constexpr int A_BYTES = BM * STEPB;            // LDS per stage
  static constexpr int AS_BYTES = BM * 16, BS_BYTES = BN * 16;   // LDS per chunk of scales
  static constexpr int OUT_BYTES = 16 * BN * 4;         // 16 output rows
  static constexpr int RING = 2 * A_BYTES > 2 * OUT_BYTES ? 2 * A_BYTES : 2 * OUT_BYTES;
  static constexpr int DMAS = A_BYTES / 1024 / WAVES;   // per wavefront and step
  static constexpr int kBlockE = 4;                     // entries per tile-order block
};

template <bool GATHER>
__global__ __launch_bounds__(256, 2) void mx_gemm_tiled_kernel(MxArgs a) {
  typedef MxTile T;
  constexpr int FM = T::FM;
  __shared__ __align__(1024) char smem[T::RING + 2 * T::AS_BYTES + 2 * T::BS_BYTES];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = lds_addr(smem);
  const char* s_scale = smem + T::RING;
  const int NT = (a.Hp + T::BN - 1) / T::BN;
  const int nent = *a.ntiles;
  const int total = nent * NT;      // below 2^31 (host)
  const int G = gridDim.x;
  // The workgroups of one XCD take a contiguous run of tiles per round, first come first
  // served (queue position q of XCD x is tile (q / per) * G + x * per + q % per), so that the
  // tiles in flight on an XCD stay together and share operand lines in its L2 however far
  // its workgroups drift apart: 2.57 -> 2.43 ms at 524288 slots, H = 4096, H' = 1536, 5.39
  // -> 5.05 ms at H = 7168, H' = 2048 against the same order taken statically.
  __shared__ int s_claim;
  const int xcd = blockIdx.x % 8, per = G / 8;
  int q = 0;      // thread 0: its claim
  auto claim = [&]() { if (threadIdx.x == 0) q = atomicAdd(a.qcnt + xcd, 1); };
  auto publish = [&]() { if (threadIdx.x == 0) s_claim = (q / per) * G + xcd * per + q % per; };
  auto next = [&]() { return __builtin_amdgcn_readfirstlane(s_claim); };
  claim();
  publish();
  __syncthreads();
  __shared__ uint32_t s_row[T::DMAS + 1][T::WAVES * 64];
  const int nsteps = (a.KT + 1) / 2;
  const uint32_t qrow = uint32_t(a.KT) * 64, srow = uint32_t(a.KC) * 16;   // bytes per A row
  const int r16 = lane & 15, kb = lane >> 4;

  // A tile's place, and in s_row the byte offsets behind this lane's rows of A (DMAS times 8
  // rows a wavefront, then the row of scales): worked out for the next tile before a tile's
  // epilogue, so that the loads they hang on run under other wavefronts' work.
  int rowbase = 0, wrow = 0, rows_valid = 0, n0 = 0;
  auto place = [&](int tau) {
    // blocks of kBlockE entries x all N-tiles, entries fastest
    const int eb = tau / (T::kBlockE * NT), j = tau % (T::kBlockE * NT);
    const int ge = min(T::kBlockE, nent - eb * T::kBlockE);
    const TileEntry e = a.tiles[eb * T::kBlockE + j % ge];
    n0 = j / ge * T::BN;
    rowbase = __builtin_amdgcn_readfirstlane(e.rowbase + e.m0);
    wrow = __builtin_amdgcn_readfirstlane(e.wrow);
    rows_valid = __builtin_amdgcn_readfirstlane(min(T::BM, e.n - e.m0));
    int u[T::DMAS + 1];
#pragma unroll
    for (int i = 0; i <= T::DMAS; ++i) {
      const int row = i < T::DMAS ? (wid + 4 * i) * 8 + (lane >> 3) : (wid & 1) * 64 + lane;
      u[i] = row < rows_valid ? (GATHER ? a.src_index[rowbase + row] : row) : -1;
    }
#pragma unroll
    for (int i = 0; i <= T::DMAS; ++i) {
      uint32_t off = kOffNone;
      if (u[i] >= 0 && (!GATHER || u[i] < a.NK)) {
        const uint32_t r = GATHER ? uint32_t(u[i]) / uint32_t(a.K) : uint32_t(u[i]);
        off = i < T::DMAS ? r * qrow + ((lane & 7) ^ swz_k((wid + 4 * i) * 8 + (lane >> 3))) * 16 : r * srow;
      }
      s_row[i][threadIdx.x] = off;
    }
  };
  int tau = next();
  if (tau < total) place(tau);
  while (tau < total) {
    const int col0 = n0 + wid * 64;
    const bool idle = col0 >= a.Hp;    // uniform
    uint32_t va[T::DMAS];
#pragma unroll
    for (int i = 0; i < T::DMAS; ++i) va[i] = s_row[i][threadIdx.x];
    const uint32_t vs = s_row[T::DMAS][threadIdx.x];
    const int64_t first = GATHER ? 0 : rowbase;
    const int64_t span = GATHER ? a.xrows : rows_valid;
    const __amdgpu_buffer_rsrc_t ars = make_rsrc(a.xq + first * qrow, clamp_bytes(span * qrow));
    const __amdgpu_buffer_rsrc_t srs = make_rsrc(a.xs + first * srow, clamp_bytes(span * srow));
    const int64_t tile16 = int64_t(wrow) * (a.Hp / 16) + (idle ? 0 : col0 / 16);
    const __amdgpu_buffer_rsrc_t brs = make_rsrc(a.wq + tile16 * a.KT * 1024, uint32_t(4 * a.KT) * 1024);
    const __amdgpu_buffer_rsrc_t bss = make_rsrc(a.ws + tile16 * a.KC * 256, uint32_t(4 * a.KC) * 256);

    const uint32_t vbs = (lane >> 4) * uint32_t(a.KC) * 256 + (lane & 15) * 16;
    auto issue_a = [&](int k) {     // step k into stage k % 2
#pragma unroll
      for (int j = 0; j < T::DMAS; ++j)
        dma16(ars, va[j], uint32_t(k) * T::STEPB, lds0 + (k & 1) * T::A_BYTES + (wid + 4 * j) * 1024);
    };
    auto issue_s = [&](int c) {     // scales of chunk c
      if (wid < T::BM / 64)
        dma16(srs, vs, uint32_t(c) * 16, lds0 + T::RING + (c & 1) * T::AS_BYTES + wid * 1024);
      dma16(bss, vbs, uint32_t(c) * 256,
            lds0 + T::RING + 2 * T::AS_BYTES + (c & 1) * T::BS_BYTES + wid * 1024);
    };
    auto load_b = [&](int k, v4i_t (&b)[2][T::FN]) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
          b[t][j] = __builtin_bit_cast(v4i_t, __builtin_amdgcn_raw_buffer_load_b128(
              brs, 2 * k + t < a.KT ? lane * 16 : int(kOffNone), (j * a.KT + 2 * k + t) * 1024, 0));
    };
    v4f_t acc[FM][T::FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < T::FN; ++j) acc[i][j] = v4f_t{0.f, 0.f, 0.f, 0.f};
    v4i_t b0[2][T::FN], b1[2][T::FN];
    int bs[T::FN], as[FM];

    __syncthreads();     // every wavefront has read the previous tile's last stage and its claim
    issue_a(0);
    issue_s(0);
    if (!idle) load_b(0, b0);
    claim();             // the next tile, published at the first step
    // The MFMAs of step k: 2 * FM fragments of 16 rows (both k-tiles), each read from LDS
    // while the MFMAs of the one before it run.
    auto compute = [&](int k, const v4i_t (&b)[2][T::FN], auto odd_c) {
      constexpr int O = decltype(odd_c)::value * 2;
      const char* st = smem + (k & 1) * T::A_BYTES;
      v4i_t f[2];
      auto read = [&](int n) {
        const int row = (n % FM) * 16 + r16;
        f[n & 1] = *reinterpret_cast<const v4i_t*>(
            st + row * T::STEPB + (((n / FM * 4 + kb) ^ swz_k(row)) << 4));
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
      };
      read(0);
#pragma unroll
      for (int n = 0; n < 2 * FM; ++n) {
        if (n + 1 < 2 * FM) read(n + 1);
        const int t = n / FM, i = n % FM;
        const v8i_t fa = {f[n & 1][0], f[n & 1][1], f[n & 1][2], f[n & 1][3], 0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < T::FN; ++j) {
          const v8i_t fb = {b[t][j][0], b[t][j][1], b[t][j][2], b[t][j][3], 0, 0, 0, 0};
          // operands swapped: the block is transposed, a lane holds 4 columns of one row
          if (t == 0) acc[i][j] = mfma_e2m1<O>(fb, fa, acc[i][j], bs[j], as[i]);
          else acc[i][j] = mfma_e2m1<O + 1>(fb, fa, acc[i][j], bs[j], as[i]);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, T::FN, 0);   // its MFMAs
      }
    };
    for (int k = 0; k < nsteps; k += 2) {
      wait_vm<0>();
      if (k == 0) publish();
      __syncthreads();
      if (k + 1 < nsteps) issue_a(k + 1);
      if (!idle) {
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
          bs[j] = *reinterpret_cast<const int*>(s_scale + 2 * T::AS_BYTES + ((k / 2) & 1) * T::BS_BYTES +
                                                 (wid * 4 + j) * 256 + lane * 4);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          as[i] = *reinterpret_cast<const int*>(s_scale + ((k / 2) & 1) * T::AS_BYTES +
                                                (i * 16 + r16) * 16 + kb * 4);
        if (k + 1 < nsteps) load_b(k + 1, b1);
        compute(k, b0, std::integral_constant<int, 0>());
      }
      if (k + 1 < nsteps) {
        wait_vm<0>();
        __syncthreads();
        if (k + 2 < nsteps) {
          issue_a(k + 2);
          issue_s(k / 2 + 1);
        }
        if (!idle) {
          if (k + 2 < nsteps) load_b(k + 2, b0);
          compute(k + 1, b1, std::integral_constant<int, 1>());
        }
      }
    }
    // Epilogue: a store of the lanes' own 16 x 16 block covers 16 rows of 64 bytes, which the
    // memory side takes at a third of the rate of whole rows (11000 cycles per tile against
    // 3800); so the four wavefronts exchange 16 rows at a time through the ring and each
    // stores 4 whole rows of the tile, 1 KiB per instruction: 2.34 -> 2.01 ms at 524288
    // slots, H = 4096, H' = 1536, 4.99 -> 4.63 ms at H = 7168, H' = 2048.
    const __amdgpu_buffer_rsrc_t crs = make_rsrc(a.c + int64_t(rowbase) * a.Hp + n0,
                                                 clamp_bytes((int64_t(rows_valid) * a.Hp - n0) * 4));
    const uint32_t lcol = n0 + lane * 4 < a.Hp ? uint32_t(lane) * 16 : kOffNone;
    tau = next();
    if (tau < total) place(tau);
    __syncthreads();     // every wavefront has read the last stage
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      char* buf = smem + (i & 1) * T::OUT_BYTES;    // 16 rows of 1 KiB, chunks swizzled by row
      if (!idle) {
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
          *reinterpret_cast<v4f_t*>(buf + r16 * 1024 + (((wid * 16 + j * 4 + kb) ^ r16) << 4)) = acc[i][j];
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int row = wid * 4 + h;
        const v4f_t x = *reinterpret_cast<const v4f_t*>(buf + row * 1024 + ((lane ^ row) << 4));
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i_t, x), crs,
                                               lcol + uint32_t(i * 16 + row) * a.Hp * 4, 0, kNonTemporal);
      }
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
  const RowSplit sp = row_split(int64_t(KC) * 64, kRowThreads);
  const int64_t blocks = (rows + sp.rows() - 1) / sp.rows();
  const int grid = int(blocks < 65536 ? blocks : 65536);
  if (shape->dtype == MOONEP_BF16)
    mx_quantize_kernel<true><<<grid, kRowThreads, 0, as_stream(stream)>>>(src, rows, width, KT, KC, sp, q, scales);
  else
    mx_quantize_kernel<false><<<grid, kRowThreads, 0, as_stream(stream)>>>(src, rows, width, KT, KC, sp, q, scales);
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
           int(k_tiles(s.H)), int(k_chunks(s.H)), int64_t(s.R) * s.S * s.K,
           int64_t(s.R) * s.S * (src_index ? 1 : s.K),
           ws_ptr<int32_t>(ws, ws_layout(s).flags) + kFlagQueue};
  // The tiled form reads each weight once per 128 rows, the other once per 64 (and per block
  // of 16 rows from the CU's cache), but needs the card full of tiles. Measured on both
  // sides, tiled / few rows, us (H, H', E; slots): 4096, 1536, 256: 66000 slots and more 5x
  // faster; 2048: 161 / 166, 512: 152 / 136, 128: 95 / 66. 7168, 2048, 64: 1024: 106 / 118,
  // 512: 106 / 104. 1024, 512, 64: 16384 (320 tiles): 34 / 39, 8192 (192 tiles): 33 / 28.
  // 512, 512, 16: 16384 (272 tiles): 33 / 31. So: at least 8 slots per weight row, and a tile
  // for every CU, counting half a tile of padding per weight row.
  const int64_t nt = (s.Hp + MxTile::BN - 1) / MxTile::BN;
  const int64_t held = int64_t(s.E) + s.R;      // a plan has at most this many segments
  const bool tiled = cus % 4 == 0 && a.NK >= 8 * held &&
                     (a.NK + MxTile::BM / 2 * held) / MxTile::BM * nt >= cus &&
                     // 32-bit offsets of gathered rows and of a tile's outputs, and tile numbers
                     (!src_index || a.xrows * a.KT * 64 < int64_t(kOffNone)) &&
                     int64_t(MxTile::BM) * s.Hp * 4 <= int64_t(kOffNone) &&
                     (a.NK / MxTile::BM + int64_t(s.R) * (s.E + s.B)) * nt < INT32_MAX;
  if (tiled) {
    st = launch_tile_list(s, cu_seqlens, MxTile::BM, ws, strm, &a.tiles, &a.ntiles);
    if (st) return st;
    // two workgroups per CU: one's stores and waits run under the other's products
    if (src_index) mx_gemm_tiled_kernel<true><<<cus * 2, 256, 0, strm>>>(a);
    else mx_gemm_tiled_kernel<false><<<cus * 2, 256, 0, strm>>>(a);
    return launch_status();
  }
  // a segment's rows are shared out twice as finely as an even plan would need
  const int64_t share = (2 * a.NK + held * kMxRows - 1) / (held * kMxRows);
  const int shares = int(share < 64 ? share : 64);
  mx_gemm_kernel<<<cus * 8, 256, 0, strm>>>(a, cu_seqlens, s.R, s.E, s.B, s.S * s.K, shares);
  return launch_status();
}
