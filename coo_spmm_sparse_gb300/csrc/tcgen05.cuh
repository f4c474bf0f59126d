// The tensor memory instructions of sm_103a as the attention kernels use them:
// one CTA's MMAs with 128 rows, 16-bit operands and 32-bit sums, operands in
// shared memory in 128-byte swizzled rows (as TMA writes them) or, for the
// left one, in tensor memory; barriers with bounded waits.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "dense_ops.cuh"

namespace snack {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint64_t *b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(b)) : "memory");
}

// One arrival for a whole warp, after what its lanes have read and written
// (256 arrivals one by one took about as long as a product).
__device__ __forceinline__ void bar_arrive_warp(uint64_t *b) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) bar_arrive(b);
}

constexpr int kPolls = 1 << 22;  // of a wait, at most
__device__ __forceinline__ bool bar_done(uint64_t *b, int parity) {
  uint32_t done;
  asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(done)
               : "r"(smem_addr(b)), "r"(parity)
               : "memory");
  return done;
}
// Waits for the phase of that parity, for so many polls at most, or until another
// wait of the block has given up; false: the caller leaves its loop.
__device__ __forceinline__ bool bar_wait(uint64_t *b, int parity, volatile int *failed, int polls) {
  for (int i = 0; i < polls; ++i) {
    if (bar_done(b, parity)) return true;
    if ((i & 63) == 63 && *failed) return false;
  }
  *failed = 1;
  return false;
}
// Waits for copies or products that are in flight after a wait has given up: a block
// does not end before they have.
__device__ __forceinline__ void bar_drain(uint64_t *b, int parity) {
  for (int i = 0; i < kPolls && !bar_done(b, parity); ++i) {
  }
}

// Shared memory written by ordinary stores, seen by the copies and MMAs that follow.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_bar_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

// 64 columns from x on of 128 tokens of one head; what lies outside the tensor
// arrives as zeros.
__device__ __forceinline__ void copy_box(void *to, const CUtensorMap *map, uint64_t *bar, int x, int head, int token,
                                         int seq) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_addr(to)),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(head), "r"(token), "r"(seq)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Whole warps.
__device__ __forceinline__ void tmem_alloc(uint32_t *to, int columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(to)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, int columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the lane that belongs to each thread.
__device__ __forceinline__ void load32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void load32(uint32_t addr, float *v) { load32(addr, reinterpret_cast<uint32_t *>(v)); }

__device__ __forceinline__ void store32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void store16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A matrix in shared memory: blocks of 64 columns, rows of 128 bytes in
// 1024-byte groups of eight, swizzled.  By rows (the summed index runs along a
// row): groups of eight rows are 1024 bytes apart.  By columns (the summed
// index runs down the rows): `block` bytes from one 64-column block to the next.
//
// A descriptor's upper word is the same for both; a step along the matrix adds
// to the lower one.
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_rows(uint32_t addr) { return ((addr & 0x3ffff) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_columns(uint32_t addr, uint32_t block) {
  return ((addr & 0x3ffff) >> 4) | ((block >> 4) << 16);
}

// 128 x n sums in 32 bits of 16-bit operands; b_columns: b is read by columns.
template <typename T>
__host__ __device__ constexpr uint32_t mma_kind(int n, bool b_columns) {
  constexpr uint32_t t = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | (b_columns ? 1u << 16 : 0u) | ((uint32_t)(n / 8) << 17) | (8u << 24);
}

// One thread of the warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
  return yes != 0;
}

// d (tensor memory) = or += a * b over 16 of the summed index.  One thread;
// a and b are lower words of descriptors, or tensor memory.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t kind, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 x, y;\nsetp.ne.b32 p, %4, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(kind), "r"((uint32_t)add), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t kind, bool add) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 y;\nsetp.ne.b32 p, %4, 0;\nmov.b64 y, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(kind), "r"((uint32_t)add), "n"(kDescHigh)
      : "memory");
}
// The barrier is arrived at once all MMAs issued so far by this thread are complete.
__device__ __forceinline__ void commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// Registers of the calling warpgroup from here on, out of what the block was launched with.
template <int N>
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void leave_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two 32-bit operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<uint64_t *>(&d))
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
        "l"(*reinterpret_cast<uint64_t *>(&c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t *>(&d))
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<uint64_t *>(&d))
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// d (128 x n) = or += rows a times rows b: K wide, their 64-column blocks
// `block` bytes apart.  a, b: descriptors of the first columns.
template <int K>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t block, uint32_t kind) {
#pragma unroll
  for (int k = 0; k < K; k += 16) {
    const uint32_t step = ((k / 64) * block + (k % 64) * 2) >> 4;
    mma(d, a + step, b + step, kind, k > 0);
  }
}
// d = or += a (tensor memory, 16-bit values) times b, K rows read by columns, from row `from` on.
// Every `run` values of a lie together, `gap` columns from one run to the next.
template <int K>
__device__ __forceinline__ void mma_sums(uint32_t d, uint32_t a, int run, int gap, uint32_t b, uint32_t kind, bool add,
                                         int from = 0) {
#pragma unroll
  for (int k = from; k < from + K; k += 16)
    mma_tmem(d, a + (k / run) * gap + (k % run) / 2, b + k * 8, kind, add || k > from);
}

}  // namespace tc
}  // namespace snack
