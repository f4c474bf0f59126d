// Residual norm, rows held in registers: every input is read once, every
// output written once.  Device code that the forward (norm_team_forward.cu)
// and the backward (norm_team_backward.cu) share.
//
// A team of threads takes one row after another; each thread holds 8 columns
// of it, always the same ones.  Rows to come are copied asynchronously into
// shared memory, two ahead.  Rows of 16-byte vectors go to slots that only
// the copying thread reads; of rows that start or end elsewhere, the 16-byte
// pieces that hold them are copied, and every thread picks its elements out
// after a barrier.  Otherwise the team meets only for its sums.  Rows of
// more than 4096 columns are held by a cluster of blocks that exchange
// their sums through each other's shared memory.
#pragma once

#include <cooperative_groups.h>

#include <algorithm>

#include "residual_norm.cuh"

namespace snack {
namespace team {

namespace cg = cooperative_groups;

constexpr int C = kTeamCols;

struct TeamArgs {
  NormArgs n;
  int block_cols;
  int threads;        // of a team in one block
  float *next_parts;  // [teams][2][width]
  float *post_parts;  // [slabs][2][width]
};

// Slots of 16 bytes that C elements of T take.
template <typename T>
__host__ __device__ constexpr int slots_of() { return C * (int)sizeof(T) / 16; }

// Bytes that hold `cols` elements of T from any address on, in 16-byte pieces.
__host__ __device__ constexpr int piece_bytes(int cols, int size) { return (cols * size + 15) / 16 * 16 + 16; }

// The columns of a thread: with vectors, runs of U columns a block's width
// of runs apart, else single columns a block's threads apart.
template <typename TS, typename TB, bool VEC>
struct Columns {
  static constexpr int U = VEC ? (sizeof(TB) == 4 ? 4 : 8) : 1;
  int first;         // the block's first column
  int count;         // its columns
  int tid, threads;  // this thread among those of its team's part in the block
  bool ok[C / U];
  __device__ __forceinline__ Columns(const TeamArgs &q, int rank, int tid_, int threads_)
      : tid(tid_), threads(threads_) {
    const int64_t c0 = (int64_t)rank * q.block_cols, left = q.n.a.width - c0;
    first = (int)c0;
    count = left < 0 ? 0 : (left < q.block_cols ? (int)left : q.block_cols);
#pragma unroll
    for (int k = 0; k < C / U; ++k) ok[k] = local(k * U) < count;
  }
  __device__ __forceinline__ int local(int j) const {  // column of element j within the block
    return ((j / U) * threads + tid) * U + j % U;
  }
  __device__ __forceinline__ int at(int j) const { return first + local(j); }
  __device__ __forceinline__ bool in(int j) const { return ok[j / U]; }
};

// Parameters of the thread's columns (`other` where there is no vector, 0
// beyond the row: what such a column adds to any sum is 0).
template <typename CO>
__device__ __forceinline__ void load_params(const void *p, int type, const CO &co, float other, float (&v)[C]) {
#pragma unroll
  for (int j = 0; j < C; ++j) v[j] = !co.in(j) ? 0.f : (p ? load_as_float(p, type, co.at(j)) : other);
}

// Copies a row of T ahead: vectors into the thread's own slots (16 bytes
// each, the team's side by side), else all of the block's pieces.
template <typename T, bool VEC, typename CO>
__device__ __forceinline__ void copy_row(char *to, const T *row, const CO &co) {
  if (VEC) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < slots_of<T>(); ++k)
      if (co.in(k * E)) copy_async16(to + (k * co.threads + co.tid) * 16, row + co.at(k * E));
  } else {
    const uintptr_t begin = reinterpret_cast<uintptr_t>(row + co.first), base = begin & ~uintptr_t(15);
    const int bytes = (int)(begin - base) + co.count * (int)sizeof(T);
    if (co.count > 0)
      for (int i = co.tid * 16; i < bytes; i += co.threads * 16)
        copy_async16(to + i, reinterpret_cast<const char *>(base) + i, bytes - i < 16 ? bytes - i : 16);
  }
}

// The thread's columns of a row that was copied ahead.  Vectors beyond the
// row read what clear_slots left there.
template <typename T, bool VEC, typename CO>
__device__ __forceinline__ void take_row(const char *from, const T *row, const CO &co, float (&v)[C]) {
  if (VEC) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < slots_of<T>(); ++k) {
      const uint4 raw = *reinterpret_cast<const uint4 *>(from + (k * co.threads + co.tid) * 16);
      if constexpr (sizeof(T) == 4) {
        v[k * E] = __uint_as_float(raw.x);
        v[k * E + 1] = __uint_as_float(raw.y);
        v[k * E + 2] = __uint_as_float(raw.z);
        v[k * E + 3] = __uint_as_float(raw.w);
      } else {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2<T>(w[i], v[k * E + 2 * i], v[k * E + 2 * i + 1]);
      }
    }
  } else {
    const T *at = reinterpret_cast<const T *>(from + (reinterpret_cast<uintptr_t>(row + co.first) & 15));
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = co.in(j) ? to_float(at[co.local(j)]) : 0.f;
  }
}

template <typename T, bool VEC, typename CO>
__device__ __forceinline__ void store_row(T *row, const CO &co, const float (&v)[C]) {
  if (VEC) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < slots_of<T>(); ++k) {
      if (!co.in(k * E)) continue;
      uint4 raw;
      if constexpr (sizeof(T) == 4)
        raw = make_uint4(__float_as_uint(v[k * E]), __float_as_uint(v[k * E + 1]), __float_as_uint(v[k * E + 2]),
                         __float_as_uint(v[k * E + 3]));
      else
        raw = make_uint4(pack2<T>(v[k * E], v[k * E + 1]), pack2<T>(v[k * E + 2], v[k * E + 3]),
                         pack2<T>(v[k * E + 4], v[k * E + 5]), pack2<T>(v[k * E + 6], v[k * E + 7]));
      *reinterpret_cast<uint4 *>(row + co.at(k * E)) = raw;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (co.in(j)) row[co.at(j)] = from_float<T>(v[j]);
  }
}

// Zeros in the ring, where slots beyond the row are read but never copied.
__device__ __forceinline__ void clear_slots(char *ring, int bytes) {
  for (int i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16)
    *reinterpret_cast<uint4 *>(ring + i) = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

// Sums over the team.  One barrier each: consecutive sums use alternate
// halves of `red`.
template <bool CL, bool MULTI>
struct Team {
  static constexpr int kMost = kTeamThreads / 32;  // warps of a block
  static constexpr int kFloats = 2 * 3 * kMost * (CL ? kTeamCluster : 1);
  float *red;
  int flip = 0;
  int rank = 0, size = 1;  // blocks of the team
  int place = 0, warps_ = 0;  // MULTI: the team's place among those of its block, its warps

  __device__ __forceinline__ int index() const { return MULTI ? place : 0; }
  __device__ __forceinline__ int warps() const { return MULTI ? warps_ : (int)blockDim.x >> 5; }
  // The team's threads in this block.
  __device__ __forceinline__ void barrier() const {
    if (!MULTI || (int)blockDim.x == warps() * 32)
      __syncthreads();
    else if (warps() == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(index() + 1), "r"(warps() * 32) : "memory");
  }

  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
    const int lane = threadIdx.x & 31, nw = warps(), w = (int)(threadIdx.x >> 5) - index() * nw;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
    if (!CL && nw == 1) return;
    float *buf = red + flip * (kFloats / 2);
    flip ^= 1;
    if (CL) {
      // every warp's sums to every block of the team
      cg::cluster_group cl = cg::this_cluster();
      const int all = nw * size;
      if (lane < size) {
        float *to = cl.map_shared_rank(buf, lane);
#pragma unroll
        for (int k = 0; k < N; ++k) to[k * all + rank * nw + w] = v[k];
      }
      cl.sync();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        float s = 0.f;
        for (int i = lane; i < all; i += 32) s += buf[k * all + i];
        v[k] = warp_sum(s);
      }
    } else {
      buf += index() * nw;
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) buf[k * kMost + w] = v[k];
      barrier();
      // sixteen lanes hold all warps' sums: four steps
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = (lane & 15) < nw ? buf[k * kMost + (lane & 15)] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
  }

  // Mean and 1/deviation of the row (v is 0 beyond it).
  template <bool LAYER, typename CO>
  __device__ __forceinline__ void stats(const snack_norm_args &a, const CO &co, const float (&v)[C], float &mean,
                                        float &rstd) {
    const float inv = 1.f / (float)a.width;
    float s[1] = {0.f};
    mean = 0.f;
    if (LAYER) {
#pragma unroll
      for (int j = 0; j < C; ++j) s[0] += v[j];
      sum(s);
      mean = s[0] * inv;
      s[0] = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float d = co.in(j) ? v[j] - mean : 0.f;
        s[0] = fmaf(d, d, s[0]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) s[0] = fmaf(v[j], v[j], s[0]);
    }
    sum(s);
    rstd = rsqrtf(fmaf(s[0], inv, a.eps));
  }
};

// `threads`: of a team in this block (MULTI: several teams).
template <bool CL, bool MULTI>
__device__ __forceinline__ Team<CL, MULTI> make_team(float *red, int threads) {
  Team<CL, MULTI> t;
  t.red = red;
  if (MULTI) {
    t.warps_ = threads >> 5;
    t.place = (int)threadIdx.x / threads;
  }
  if (CL) {
    cg::cluster_group cl = cg::this_cluster();
    t.rank = (int)cl.block_rank();
    t.size = (int)cl.num_blocks();
    cl.sync();  // the team's blocks are all there before one writes to another
  }
  return t;
}

// The gate's vector for a row, or null where the gate is one number.
template <typename TB>
__device__ __forceinline__ const TB *gate_row(const snack_norm_args &a, int64_t row) {
  const TB *g = static_cast<const TB *>(a.gate);
  if (a.gate_kind == SNACK_GATE_CHANNEL) return g;
  if (a.gate_kind == SNACK_GATE_SEQUENCE) return g + (row / a.group_rows) * a.width;
  if (a.gate_kind == SNACK_GATE_FULL) return g + row * a.gate_stride;
  return nullptr;
}

// Bytes of one row of an array of T in the ring.
template <typename T, bool VEC>
__device__ __forceinline__ int row_bytes(const TeamArgs &q, int threads) {
  return VEC ? slots_of<T>() * 16 * threads : piece_bytes(q.block_cols, sizeof(T));
}

// ------------------------------------------------------------------ host

inline bool rows16(const void *p, int64_t stride, int type) {
  return !p || (aligned_to(p, 16) && stride * type_bytes(type) % 16 == 0);
}

// The smallest team that holds a row.
inline TeamPlan team_shape(const snack_norm_args &a) {
  TeamPlan p;
  const int64_t most = (int64_t)kTeamThreads * kTeamCols;
  int cluster = 1;
  while (cluster < kTeamCluster && a.width > most * cluster) cluster *= 2;
  if (a.width > most * cluster) return p;
  const int64_t cols = (a.width + cluster - 1) / cluster;
  p.threads = (int)((cols + 32 * kTeamCols - 1) / (32 * kTeamCols)) * 32;
  p.cluster = cluster;
  p.block_cols = cluster > 1 ? (int)((cols + 7) / 8 * 8) : p.threads * kTeamCols;
  return p;
}

// Bytes of a row in the ring, of `ns` arrays of the stream's and `nb` of the branch's type.
inline int ring_row(const TeamPlan &p, const snack_norm_args &a, int ns, int nb) {
  const int ts = (int)type_bytes(a.stream_type), tb = (int)type_bytes(a.branch_type);
  return p.vec ? p.threads * C * (ns * ts + nb * tb)
               : ns * piece_bytes(p.block_cols, ts) + nb * piece_bytes(p.block_cols, tb);
}

// Two rows ahead, or one where two do not fit.
inline void team_ring(TeamPlan *p, const snack_norm_args &a, int ns, int nb) {
  const size_t row = (size_t)ring_row(*p, a, ns, nb) * p->per_block;
  p->stages = 3 * row <= 208 * 1024 ? 3 : 2;
  p->smem = p->stages * row;
}

template <typename K>
cudaError_t launch_team(K kern, const TeamPlan &p, int64_t teams, const TeamArgs &q, cudaStream_t s) {
  const cudaError_t e = allow_smem(kern, p.smem);
  return e != cudaSuccess ? e
                          : launch_clusters(kern, dim3((unsigned)(teams * p.cluster)), p.cluster,
                                            p.threads * p.per_block, p.smem, true, s, q);
}

// The forms of a call that are compiled on their own, because their many
// calls leave no room for the tests and registers of the others: a branch, a
// norm after it, all results wanted, no gate that belongs to a row, no bias
// of an rms norm; rows in one block.
enum Form { kAny = 0, kFast = 1, kFastPost = 2 };

// Returns the launch of KERNEL<TS, TB, stages, vectors, cluster, layer norm,
// form> by the plan p.  Two stages: fp32 rows with a full gate (five arrays).
#define SNACK_TEAM_L(KERNEL, TS, TB, CL, L)                                                       \
  {                                                                                               \
    if (p.stages == 3) {                                                                          \
      if (p.vec) return launch_team(KERNEL<TS, TB, 3, true, CL, L, kAny>, p, teams, q, s);        \
      return launch_team(KERNEL<TS, TB, 3, false, CL, L, kAny>, p, teams, q, s);                  \
    }                                                                                             \
    if constexpr (sizeof(TB) == 4) {                                                              \
      if (p.vec) return launch_team(KERNEL<TS, TB, 2, true, CL, L, kAny>, p, teams, q, s);        \
      return launch_team(KERNEL<TS, TB, 2, false, CL, L, kAny>, p, teams, q, s);                  \
    }                                                                                             \
    return cudaErrorInvalidValue;                                                                 \
  }
#define SNACK_TEAM_F(KERNEL, TS, TB, L)                                                           \
  {                                                                                               \
    if (p.vec) {                                                                                  \
      if (form == kFastPost) return launch_team(KERNEL<TS, TB, 3, true, false, L, kFastPost>, p, teams, q, s); \
      return launch_team(KERNEL<TS, TB, 3, true, false, L, kFast>, p, teams, q, s);               \
    }                                                                                             \
    if (form == kFastPost) return launch_team(KERNEL<TS, TB, 3, false, false, L, kFastPost>, p, teams, q, s); \
    return launch_team(KERNEL<TS, TB, 3, false, false, L, kFast>, p, teams, q, s);                \
  }
#define SNACK_TEAM(KERNEL, TS, TB)                                                                \
  {                                                                                               \
    const bool layer = q.n.a.norm_kind == SNACK_NORM_LAYER;                                       \
    if (form != kAny && p.stages == 3 && p.cluster == 1) {                               \
      if (layer) SNACK_TEAM_F(KERNEL, TS, TB, true)                                               \
      else SNACK_TEAM_F(KERNEL, TS, TB, false)                                                    \
    }                                                                                             \
    if (p.cluster > 1) {                                                                          \
      if (layer) SNACK_TEAM_L(KERNEL, TS, TB, true, true)                                         \
      else SNACK_TEAM_L(KERNEL, TS, TB, true, false)                                              \
    }                                                                                             \
    if (layer) SNACK_TEAM_L(KERNEL, TS, TB, false, true)                                          \
    else SNACK_TEAM_L(KERNEL, TS, TB, false, false)                                               \
  }

// Whether the options allow a form of their own.
inline bool plain_options(const snack_norm_args &a) {
  return a.y && a.next_norm && a.gate_kind != SNACK_GATE_TOKEN && a.gate_kind != SNACK_GATE_FULL &&
         (a.norm_kind == SNACK_NORM_LAYER || (!a.post_bias && !a.next_bias));
}

}  // namespace team
}  // namespace snack
