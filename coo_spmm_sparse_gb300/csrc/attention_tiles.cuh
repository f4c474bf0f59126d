// Attention on tcgen05: 16-bit types, tiles of 128 x 128.
//
// TMA brings tiles of 128 tokens of a head into shared memory; one thread
// issues the MMAs; eight warps read the scores from tensor memory, a thread a
// row, and write the probabilities (forward) or the gradients of the scores
// (backward) back over them as the left operand of the next product, so that
// nothing but inputs and results passes through shared memory.
//
// Tiles of the last tokens of a sequence may bring tokens of the next one, or
// padding.  Scores of them are masked; rows of the operand that meets masked
// (zero) entries in the second product are set to zero, since what lies there
// may not be finite.
#pragma once

#include "attention.cuh"
#include "tcgen05.cuh"

namespace snack {

// Sticky: a wait of one of this file's kernels has run out since the last read.
static __device__ int g_attention_failed = 0;

constexpr int kTile = 128;
// Warps 0-7: rows; 8: copies; 9: MMAs; 10: statistics of
// rows, where they are not a thread's own; 11 only completes the warpgroup.
// 384 threads are launched with 168 registers each: 3 * 168 = 2 * 224 + 56.
constexpr int kTileThreads = 384, kRowRegisters = 224, kOtherRegisters = 56;
constexpr int kCopyWarp = 8, kMmaWarp = 9;

struct TileMaps {
  CUtensorMap q, k, v, dout;
};

// Bytes of a tile: DP / 64 blocks of 128 rows of 128 bytes.
template <int DP>
__host__ __device__ constexpr int tile_bytes() { return kTile * DP * 2; }
constexpr uint32_t kBlock = kTile * 128;

__device__ __forceinline__ unsigned char *align1024(unsigned char *p) {
  return p + ((1024 - (tc::smem_addr(p) & 1023)) & 1023);
}

// Starts the copy of a tile; one thread.
template <int DP>
__device__ __forceinline__ void copy_tile(unsigned char *to, const CUtensorMap *map, uint64_t *bar, int head,
                                          int token, int seq) {
  tc::bar_expect(bar, tile_bytes<DP>());
#pragma unroll
  for (int x = 0; x < DP; x += 64) tc::copy_box(to + x / 64 * kBlock, map, bar, x, head, token, seq);
}

// The whole warp copies a tile and sets the rows from `rows` on to zero;
// `full` is then arrived at by one plain arrival.
template <int DP>
__device__ __forceinline__ bool copy_tile_cut(unsigned char *to, const CUtensorMap *map, uint64_t *full, uint64_t *cut,
                                              int *cut_phase, int head, int token, int seq, int rows,
                                              volatile int *failed) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) copy_tile<DP>(to, map, cut, head, token, seq);
  __syncwarp();
  const bool ok = __all_sync(0xffffffffu, tc::bar_wait(cut, *cut_phase, failed));
  *cut_phase ^= 1;
  if (!ok) return false;
  for (int x = 0; x < DP; x += 64)
    for (int i = rows * 8 + lane; i < kTile * 8; i += 32)
      *reinterpret_cast<uint4 *>(to + x / 64 * kBlock + i * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_async_proxy();
  __syncwarp();
  if (lane == 0) tc::bar_arrive(full);
  return true;
}

// Stores columns [0, d) of a thread's row of sums (DP of them from column
// `from` of tensor memory on) times a factor, or zeros.  Whole warps; `row`
// NULL: nothing; `some`: there are sums (the same in the whole warp).
template <typename T, int DP>
__device__ __forceinline__ void store_sums(uint32_t from, T *row, float factor, int d, bool some, bool zero) {
#pragma unroll
  for (int c = 0; c < DP; c += 32) {
    float v[32];
    if (some) {
      tc::load32(from + c, v);
      tc::wait_loads();
    }
    if (row) {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (some && !zero) {
          u.x = pack2<T>(v[i] * factor, v[i + 1] * factor);
          u.y = pack2<T>(v[i + 2] * factor, v[i + 3] * factor);
          u.z = pack2<T>(v[i + 4] * factor, v[i + 5] * factor);
          u.w = pack2<T>(v[i + 6] * factor, v[i + 7] * factor);
        }
        if (c + i < d) *reinterpret_cast<uint4 *>(row + c + i) = u;
      }
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------ host

using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                            const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                            CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static inline Encode map_encoder() {
  static const Encode f = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    cudaGetLastError();
    return reinterpret_cast<Encode>(p);
  }();
  return f;
}

static inline bool map_of(CUtensorMap *m, int type, const Strided &t, int64_t d, int64_t heads, int64_t tokens, int64_t seqs) {
  const Encode f = map_encoder();
  if (!f) return false;
  const auto bytes = [](int64_t n, int64_t s) { return (cuuint64_t)(n > 1 ? 2 * s : 16); };
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)seqs};
  const cuuint64_t strides[3] = {bytes(heads, t.head), bytes(tokens, t.token), bytes(seqs, t.seq)};
  const cuuint32_t box[4] = {64, 1, kTile, 1}, step[4] = {1, 1, 1, 1};
  return f(m, type == SNACK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, t.p, dims,
           strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What TMA and 16-byte stores need: 16-byte aligned rows, and no dimension
// that repeats the same memory.
static inline bool even(const Strided &t, int64_t heads, int64_t tokens, int64_t seqs) {
  const auto good = [](int64_t n, int64_t s) { return n <= 1 || (s > 0 && s % 8 == 0 && s < (int64_t)1 << 38); };
  return aligned_to(t.p, 16) && good(heads, t.head) && good(tokens, t.token) && good(seqs, t.seq);
}

static inline bool tiles_fit(const AttnCall &c, int type) {
  return type != SNACK_F32 && c.d % 8 == 0 && c.scale > 0.f && c.k_tokens > 0 && c.q_tokens > 0 && c.sequences > 0;
}

}  // namespace snack
