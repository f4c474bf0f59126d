// Attention on tcgen05: tiles of 128 x 128; 16-bit types, and 32-bit floats
// with head sizes up to 64.
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
//
// 32-bit floats arrive as two float16 parts of a tile (128 tokens of a head) scaled
// by a power of two to below 2^15, x = hi + lo (made by split_operands in
// attention.cu): 22 bits of everything above 2^-17 of the tile's largest, and never
// more than 2^-39 of that off.  A power for a tile, not for a tensor, so that nothing
// depends on other sequences and heads; products with a tile of keys, or of queries,
// are brought back as they leave tensor memory.  A row has its 64 high halves, then its 64 low ones, and a product
// is hi*hi + hi*lo + lo*hi; probabilities (2^14 fold) and gradients of scores
// are split the same way.  Three products at the rate of 16 bits cost half of
// three tf32 ones.  The sums leave tensor memory after every tile for 32-bit
// sums in the rows' registers: the matrix unit cuts off what it adds.
#pragma once

#include "attention.cuh"
#include "tcgen05.cuh"

namespace snack {

// Sticky: a wait of one of this file's kernels has run out since the last read.
static __device__ int g_attention_failed = 0;

// Warps 0-7: rows; 8: copies; 9: MMAs; 10: statistics of
// rows, where they are not a thread's own; 11 only completes the warpgroup.
// 384 threads are launched with 168 registers each: 3 * 168 = 2 * 224 + 56.
constexpr int kTileThreads = 384, kRowRegisters = 224, kOtherRegisters = 56;
constexpr int kCopyWarp = 8, kMmaWarp = 9;

struct TileMaps {
  CUtensorMap q, k, v, dout;
};

template <typename T>
struct Operand {
  using type = T;
  static constexpr bool kSplit = false;
};
template <>
struct Operand<float> {
  using type = __half;
  static constexpr bool kSplit = true;
};
// Columns of a tile in shared memory.
template <typename T, int DP>
__host__ __device__ constexpr int wide() { return Operand<T>::kSplit ? 2 * DP : DP; }

// Bytes of a tile: DP / 64 blocks of 128 rows of 128 bytes.
template <int DP>
__host__ __device__ constexpr int tile_bytes() { return kTile * DP * 2; }
constexpr uint32_t kBlock = kTile * 128;

__device__ __forceinline__ unsigned char *align1024(unsigned char *p) {
  return p + ((1024 - (tc::smem_addr(p) & 1023)) & 1023);
}

// A block without a tile returns the tensor memory that it was given.
__device__ __forceinline__ void leave_block(int warp, const uint32_t *tmem) {
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::tmem_free(*tmem, 512);
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
// `full` is then arrived at by one plain arrival, also where the wait gives up.
template <int DP>
__device__ __forceinline__ bool copy_tile_cut(unsigned char *to, const CUtensorMap *map, uint64_t *full, uint64_t *cut,
                                              int *cut_phase, int head, int token, int seq, int rows,
                                              volatile int *failed, int polls) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) copy_tile<DP>(to, map, cut, head, token, seq);
  __syncwarp();
  const bool ok = __all_sync(0xffffffffu, tc::bar_wait(cut, *cut_phase, failed, polls));
  if (!ok) tc::bar_drain(cut, *cut_phase);
  *cut_phase ^= 1;
  for (int x = 0; x < DP; x += 64)
    for (int i = rows * 8 + lane; i < kTile * 8; i += 32)
      *reinterpret_cast<uint4 *>(to + x / 64 * kBlock + i * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_async_proxy();
  __syncwarp();
  if (lane == 0) tc::bar_arrive(full);
  return ok;
}

// What a block whose wait has given up leaves in a row of results.
template <typename T>
__device__ __forceinline__ void poison_row(T *row, int d) {
  for (int e = 0; e < d; ++e) row[e] = from_float<T>(__uint_as_float(0x7fc00000u));
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
      const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0 && d % 8 == 0;
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        if (c + i >= d) break;
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          u[e] = some && !zero ? pack2<T>(v[i + 2 * e] * factor, v[i + 2 * e + 1] * factor) : 0;
        if (vec) {
          *reinterpret_cast<uint4 *>(row + c + i) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
          unsigned short *const to = reinterpret_cast<unsigned short *>(row + c + i);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + i + e < d) to[e] = (unsigned short)(u[e / 2] >> (16 * (e & 1)));
        }
      }
    }
    __syncwarp();
  }
}

// What takes the power of a tile of 32-bit operands out again.
__device__ __forceinline__ float power_back(const int32_t *power, int64_t tile, int heads, int head) {
  return power_of_two(-__ldg(power + tile * heads + head));
}

// Rows a times rows b, over the head size.
template <typename T, int DP>
__device__ __forceinline__ void products(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t kind = tc::mma_kind<typename Operand<T>::type>(kTile, false);
  if constexpr (!Operand<T>::kSplit) {
    tc::mma_rows<DP>(d, a, b, kBlock, kind);
  } else {
    constexpr uint32_t low = kBlock / 16;
#pragma unroll
    for (int k = 0; k < DP; k += 16) tc::mma(d, a + low + k / 8, b + k / 8, kind, k > 0);
#pragma unroll
    for (int k = 0; k < DP; k += 16) tc::mma(d, a + k / 8, b + low + k / 8, kind, true);
#pragma unroll
    for (int k = 0; k < DP; k += 16) tc::mma(d, a + k / 8, b + k / 8, kind, true);
  }
}
// Probabilities (or gradients of scores) in tensor memory, halves of 64 tokens
// 64 columns apart, times rows b: tokens [from, from + K).  Split: every 32
// tokens have their high parts, then their low ones (in the columns that their
// 32 sums had), and the result always begins anew.
template <typename T, int DP, int K>
__device__ __forceinline__ void sums(uint32_t d, uint32_t a, uint32_t b, bool add, int from = 0) {
  constexpr uint32_t kind = tc::mma_kind<typename Operand<T>::type>(DP, true);
  if constexpr (!Operand<T>::kSplit) {
    tc::mma_sums<K>(d, a, kTile / 2, kTile / 2, b, kind, add, from);
  } else {
    constexpr uint32_t low = kBlock / 16;
#pragma unroll
    for (int k = from; k < from + K; k += 16) {
      const uint32_t hi = a + k / 32 * 32 + k % 32 / 2;
      tc::mma_tmem(d, hi + 16, b + k * 8, kind, k > 0);
      tc::mma_tmem(d, hi, b + low + k * 8, kind, true);
      tc::mma_tmem(d, hi, b + k * 8, kind, true);
    }
  }
}

// Probabilities or gradients of scores in two parts of 16-bit type T (laid out as
// above) times rows b in one.
template <typename T, int DP>
__device__ __forceinline__ void fine_sums(uint32_t d, uint32_t a, uint32_t b, bool add) {
  constexpr uint32_t kind = tc::mma_kind<T>(DP, true);
#pragma unroll
  for (int k = 0; k < kTile; k += 16) {
    const uint32_t hi = a + k / 32 * 32 + k % 32 / 2;
    tc::mma_tmem(d, hi + 16, b + k * 8, kind, add || k > 0);
    tc::mma_tmem(d, hi, b + k * 8, kind, true);
  }
}

// 32 values of a row as high and low parts: columns [0, 16) and [16, 32) from `at` on.
template <typename T>
__device__ __forceinline__ void store_parts(uint32_t at, const float *v) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a, b;
    hi[e] = pack2<T>(v[2 * e], v[2 * e + 1]);
    unpack2<T>(hi[e], a, b);
    lo[e] = pack2<T>(v[2 * e] - a, v[2 * e + 1] - b);
  }
  tc::store16(at, hi);
  tc::store16(at + 16, lo);
}

// o += N columns of tensor memory times a factor.
template <int N>
__device__ __forceinline__ void add_sums(float *o, uint32_t from, float by) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    float v[32];
    tc::load32(from + c, v);
    tc::wait_loads();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[c + e] = fmaf(v[e], by, o[c + e]);
  }
}

// Stores N columns of a row, or those of them below d; row NULL: nothing.
template <int N>
__device__ __forceinline__ void store_floats(float *row, const float *v, float factor, int d, bool zero) {
  if (!row) return;
  const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0 && d % 4 == 0;
#pragma unroll
  for (int c = 0; c < N; c += 4) {
    const float4 f = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                          : make_float4(v[c] * factor, v[c + 1] * factor, v[c + 2] * factor, v[c + 3] * factor);
    if (vec) {
      if (c < d) *reinterpret_cast<float4 *>(row + c) = f;
    } else {
      if (c < d) row[c] = f.x;
      if (c + 1 < d) row[c + 1] = f.y;
      if (c + 2 < d) row[c + 2] = f.z;
      if (c + 3 < d) row[c + 3] = f.w;
    }
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

// What TMA needs: 16-byte aligned rows, and no dimension that repeats the same
// memory.
static inline bool even(const Strided &t, int64_t heads, int64_t tokens, int64_t seqs) {
  const auto good = [](int64_t n, int64_t s) { return n <= 1 || (s > 0 && s % 8 == 0 && s < (int64_t)1 << 38); };
  return aligned_to(t.p, 16) && good(heads, t.head) && good(tokens, t.token) && good(seqs, t.seq);
}

// The maps of a call's operands: its tensors, or what was made of them.
static inline bool maps_of(TileMaps *m, const AttnCall &c, int type, const SplitParts &parts, bool backward) {
  const int64_t qn = c.q_offsets ? 1 : c.sequences, kn = c.k_offsets ? 1 : c.sequences;
  const auto map = [&](CUtensorMap *to, const Strided &t, void *part, int64_t heads, int64_t tokens, int64_t seqs) {
    const int64_t row = parts.width;
    return row ? map_of(to, type == SNACK_F32 || parts.halves ? SNACK_F16 : type, Strided{part, tokens * heads * row, heads * row, row}, row, heads, tokens, seqs)
                 : map_of(to, type, t, c.d, heads, tokens, seqs);
  };
  return map(&m->q, c.q, parts.q, c.heads, c.q_tokens, qn) && map(&m->k, c.k, parts.k, c.key_heads, c.k_tokens, kn) &&
         map(&m->v, c.v, parts.v, c.key_heads, c.k_tokens, kn) &&
         (!backward || map(&m->dout, c.dout, parts.dout, c.heads, c.q_tokens, qn));
}

}  // namespace snack
