// The global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum_i sum_j g_ij^2)  or  max |g_ij|;   out = g * min(1, max_norm / (norm + eps))
//
// Memory bound: n elements are read once for the norm and once more, after
// the norm is known, to be scaled and written.  The tensors' addresses travel
// as kernel parameters (no table is copied to the device beforehand), cut
// into chunks of equal length that the blocks of a persistent grid take in
// turn.  Every block leaves one partial sum; whoever needs the norm adds the
// partials in their order, so that no atomic decides a result's bits.
//
// Squares leave the range of 32-bit floats long before a norm does.  A thread
// sums its part of a chunk as it is; a sum that is too large or too small to
// be exact is taken again of values scaled by a power of two, and such sums
// are kept apart from the others (three accumulators, after J. L. Blue, "A
// portable Fortran program to find the Euclidean norm of a vector", ACM TOMS
// 4, 1978, chosen here for a thread's part instead of every element).
#include <algorithm>
#include <type_traits>

#include "dense_ops.cuh"

namespace snack {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;
// The last bytes that the norm's pass reads as any kernel does, all before
// them to be evicted first: half of the L2, left for the pass that scales.
// 40.6 M fp32 gradients at 32 / 64 / 96 / 128 MB: 82.1 / 80.7 / 81.0 / 82.6 us,
// without a difference 83.5; 400 M bf16 into fp32 511.3 / 510.6 / 511.8 /
// 512.5, 518.1.  (Evicted last, 505 us; but then they stay when the call is
// over, and four reads of 96 MB after it took 98 us for 75.)
constexpr int64_t kKeepBytes = int64_t(64) << 20;
constexpr int kMostTable = 1024;  // tensors of one launch: 30 KB of the 32 KB that parameters may take

template <int K>
struct TensorTable {
  int count;
  int chunk_elems;
  int64_t chunks;
  int64_t keep_from;  // chunks from here on are read again while they are in the L2
  const void *src[K];
  void *dst[K];
  int64_t n[K];
  uint32_t first[K];  // first chunk of the tensor
  uint8_t stype[K], dtype[K];
};

// The tensor that holds chunk c.
template <int K>
__device__ __forceinline__ int tensor_of(const TensorTable<K> &t, uint32_t c) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// max() that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) { return (a > b || a != a) ? a : b; }

template <bool MAX>
__device__ __forceinline__ void take(float &acc, float v) {
  if (MAX)
    acc = max_nan(fabsf(v), acc);
  else
    acc = fmaf(v, v, acc);
}

template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const auto join = [](float a, float b) { return MAX ? max_nan(a, b) : a + b; };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (lane == 0) red[w] = v;
  __syncthreads();
  v = lane < kThreads / 32 ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  return v;
}

// Sums of squares as they are, and of values times kUp and times kDown.  A
// thread's part of a chunk has at most 160 elements, and there are less than
// 2^30 parts.  Kept as they are, sums of 2^-100 to 2^90: squares that are
// subnormal are off by 2^-150 each, and all parts together stay below 2^120.
// Scaled up, elements of 2^-149 to 2^-50 have squares of 2^-118 to 2^80; the
// largest of a part scaled down, 2^41 to 2^128, has one of 2^-98 to 2^76.
struct Sums {
  float mid, low, high;
};
constexpr float kLeast = 0x1p-100f, kMost = 0x1p90f, kUp = 0x1p90f, kDown = 0x1p-90f;

// Over the block, the same in every thread.
template <bool MAX>
__device__ __forceinline__ Sums block_sums(Sums v, float *red) {
  v.mid = block_reduce<MAX>(v.mid, red);
  if (!MAX && __syncthreads_or(v.low != 0.f || v.high != 0.f)) {
    v.low = block_reduce<false>(v.low, red);
    v.high = block_reduce<false>(v.high, red);
  }
  return v;
}

template <typename T>
struct Vec {  // 16 bytes
  static constexpr int N = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ void load(const T *p, uint64_t policy) {
    asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
                 : "l"(p), "l"(policy));
  }
  __device__ __forceinline__ uint32_t any() const { return raw.x | raw.y | raw.z | raw.w; }
  __device__ __forceinline__ float get(int i) const { return to_float(reinterpret_cast<const T *>(&raw)[i]); }
};

template <typename T, bool MAX>
__device__ __forceinline__ void norm_chunk(const T *p, int n, uint64_t policy, float (&acc)[4], uint32_t &bits) {
  constexpr int V = Vec<T>::N;
  const int tid = threadIdx.x;
  // elements before the first whole vector
  const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T));
  const auto one = [&](T x) {
    const float v = to_float(x);
    take<MAX>(acc[0], v);
    bits |= v != 0.f;
  };
  if (tid < head) one(p[tid]);
  p += head;
  n -= head;
  int done = 0;
  {
    const int nv = n / V;
    int i = tid;
    for (; i + 3 * kThreads < nv; i += 4 * kThreads) {
      Vec<T> v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k].load(p + (int64_t)(i + k * kThreads) * V, policy);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bits |= v[k].any();
#pragma unroll
        for (int j = 0; j < V; ++j) take<MAX>(acc[k], v[k].get(j));
      }
    }
    for (; i < nv; i += kThreads) {
      Vec<T> v;
      v.load(p + (int64_t)i * V, policy);
      bits |= v.any();
#pragma unroll
      for (int j = 0; j < V; ++j) take<MAX>(acc[j & 3], v.get(j));
    }
    done = nv * V;
  }
  for (int i = done + tid; i < n; i += kThreads) one(p[i]);
}

// The same thread's elements again, times `scale`.
template <typename T>
__device__ __noinline__ float norm_chunk_scaled(const T *p, int n, float scale) {
  constexpr int V = Vec<T>::N;
  const int tid = threadIdx.x;
  const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T));
  float s = 0.f;
  const auto add = [&](int i) {
    const float v = to_float(p[i]) * scale;
    s = fmaf(v, v, s);
  };
  if (tid < head) add(tid);
  const int nv = (n - head) / V;
  for (int i = tid; i < nv; i += kThreads)
    for (int j = 0; j < V; ++j) add(head + i * V + j);
  for (int i = head + nv * V + tid; i < n; i += kThreads) add(i);
  return s;
}

// One chunk's part of this thread.
template <typename T, bool MAX>
__device__ __forceinline__ void add_chunk(const void *src, int64_t at, int n, uint64_t policy, Sums &run) {
  const T *p = static_cast<const T *>(src) + at;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t bits = 0;  // of all elements
  norm_chunk<T, MAX>(p, n, policy, acc, bits);
  if (MAX) {
    run.mid = max_nan(max_nan(max_nan(acc[0], acc[1]), max_nan(acc[2], acc[3])), run.mid);
    return;
  }
  const float v = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  if (v >= kLeast && v <= kMost)
    run.mid += v;
  else if (v < kLeast) {
    if (bits & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) run.low += norm_chunk_scaled(p, n, kUp);
  } else {
    run.high += norm_chunk_scaled(p, n, kDown);  // infinities and NaN too
  }
}

template <int K, bool MAX>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_partials(const __grid_constant__ TensorTable<K> t,
                                                          float4 *partial) {
  __shared__ float red[32];
  dependency_wait();
  uint64_t keep, leave;  // in the L2, for the pass that scales
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(leave));
  Sums run = {0.f, 0.f, 0.f};  // over the chunks; within one, four sums of a thread
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const uint64_t policy = c >= t.keep_from ? keep : leave;
    const int k = tensor_of(t, (uint32_t)c);
    const int64_t at = (c - t.first[k]) * (int64_t)t.chunk_elems;
    const int64_t left = t.n[k] - at;
    const int n = left < t.chunk_elems ? (int)left : t.chunk_elems;
    if (t.stype[k] == SNACK_F32)
      add_chunk<float, MAX>(t.src[k], at, n, policy, run);
    else if (t.stype[k] == SNACK_BF16)
      add_chunk<__nv_bfloat16, MAX>(t.src[k], at, n, policy, run);
    else
      add_chunk<__half, MAX>(t.src[k], at, n, policy, run);
  }
  run = block_sums<MAX>(run, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = make_float4(run.mid, run.low, run.high, 0.f);
}

// The norm, root * unit.  unit is 1 unless squares have left the range.
struct Norm {
  float root, unit;
  __device__ __forceinline__ float value() const { return root * unit; }
  // min(1, max_norm / (norm + eps)).  A norm that no float holds, or only as
  // a subnormal, is taken in its own unit.
  __device__ __forceinline__ float factor(float max_norm, float eps) const {
    const float v = value();
    float ratio = max_norm / (v + eps);
    if (unit > 1.f && v > 0x1p120f) ratio = (max_norm * kDown) / (root + eps * kDown);
    if (unit < 1.f && eps < kLeast) ratio = (max_norm * kUp) / (root + eps * kUp);
    return ratio >= 1.f ? 1.f : ratio;  // a NaN stays
  }
};

// The norm from all partials, the same in every thread of every block.
template <bool MAX>
__device__ __forceinline__ Norm whole_norm(const float4 *partial, int parts, float *red) {
  Sums v = {0.f, 0.f, 0.f};
  for (int i = threadIdx.x; i < parts; i += kThreads) {
    const float4 p = partial[i];
    v.mid = MAX ? max_nan(p.x, v.mid) : v.mid + p.x;
    v.low += p.y;
    v.high += p.z;
  }
  v = block_sums<MAX>(v, red);
  if (MAX) return {v.mid, 1.f};
  // all three in the unit of the largest; what is below its last bit may be lost
  if (v.high != 0.f) return {sqrtf(fmaf(v.mid * kDown, kDown, v.high)), kUp};
  if (v.low != 0.f && v.mid < 0x1p-60f) return {sqrtf(fmaf(v.mid * kUp, kUp, v.low)), kDown};
  return {sqrtf(fmaf(v.low * kDown, kDown, v.mid)), 1.f};
}

template <bool MAX>
__global__ void __launch_bounds__(kThreads) norm_finish(const float4 *partial, int parts, float *norm) {
  __shared__ float red[32];
  dependency_wait();
  const Norm v = whole_norm<MAX>(partial, parts, red);
  if (threadIdx.x == 0) *norm = v.value();
}

// Loads that are the last of their bytes and stores that nothing reads soon
// leave the L2 to what the norm's pass left in it.
__device__ __forceinline__ uint2 take_last(const uint2 *p) { return __ldcs(p); }
__device__ __forceinline__ uint4 take_last(const uint4 *p) { return __ldcs(p); }

__device__ __forceinline__ void words_of(uint2 x, uint32_t *w) {
  w[0] = x.x;
  w[1] = x.y;
}
__device__ __forceinline__ void words_of(uint4 x, uint32_t *w) {
  w[0] = x.x;
  w[1] = x.y;
  w[2] = x.z;
  w[3] = x.w;
}

// N pieces of P (8 or 16 bytes) from the address p on, any multiple of the
// element size: the aligned pieces that hold them, moved down by the `off`
// bytes by which p lies above the first.  No piece is read that holds none
// of them.
template <typename P, int N>
__device__ __forceinline__ void load_shifted(const char *p, int off, uint32_t (&w)[N * sizeof(P) / 4]) {
  constexpr int PW = sizeof(P) / 4, W = N * PW;
  const P *at = reinterpret_cast<const P *>(p - off);
  uint32_t v[W + PW];
#pragma unroll
  for (int i = 0; i <= N; ++i) {
    P x = {};
    if (i < N || off) x = at[i];  // its neighbour reads it too
    words_of(x, v + i * PW);
  }
  if (PW == 4)
#pragma unroll
    for (int i = 0; i < W + 2; ++i) v[i] = off & 8 ? v[i + 2] : v[i];
#pragma unroll
  for (int i = 0; i < W + 1; ++i) v[i] = off & 4 ? v[i + 1] : v[i];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = off & 2 ? __funnelshift_r(v[i], v[i + 1], 16) : v[i];
}

// Scales a chunk.  A thread takes the 16 bytes of results at one place;
// where their source does not lie on a boundary of its own size (gradients
// packed end to end), it is moved into place in registers.  (Single elements
// took 773 us for 400 M bf16 packed into fp32; 32 bytes of results for a
// thread, which leaves half sectors to each store, 445 us.)
template <typename S, typename D>
__device__ __forceinline__ void scale_chunk(const S *p, D *q, int n, float coef) {
  constexpr int V = 16 / sizeof(D), SB = V * sizeof(S);  // 8, 16 or 32 bytes of the source
  using P = std::conditional_t<SB == 8, uint2, uint4>;
  constexpr int N = SB / sizeof(P), W = SB / 4;
  const int tid = threadIdx.x;
  // elements before the first whole vector of results
  const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(q) & 15)) & 15) / (int)sizeof(D));
  const int nv = (n - head) / V;
  const char *pv = reinterpret_cast<const char *>(p + head);
  uint4 *qv = reinterpret_cast<uint4 *>(q + head);
  const int off = (int)(reinterpret_cast<uintptr_t>(pv) & (sizeof(P) - 1));
  const auto scale = [&](const uint32_t (&w)[W], int i) {
    float f[V];
    if constexpr (sizeof(S) == 4) {
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = __uint_as_float(w[j]) * coef;
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        unpack2<S>(w[j / 2], f[j], f[j + 1]);
        f[j] *= coef;
        f[j + 1] *= coef;
      }
    }
    if constexpr (sizeof(D) == 4)
      __stcs(qv + i, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
    else
      __stcs(qv + i, make_uint4(pack2<D>(f[0], f[1]), pack2<D>(f[2], f[3]), pack2<D>(f[4], f[5]), pack2<D>(f[6], f[7])));
  };
  constexpr int U = SB == 32 ? 2 : 4;
  if (off == 0) {
    int i = tid;
    for (; i + (U - 1) * kThreads < nv; i += U * kThreads) {
      uint32_t w[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < N; ++b)
          words_of(take_last(reinterpret_cast<const P *>(pv) + (int64_t)(i + u * kThreads) * N + b),
                   w[u] + b * (int)sizeof(P) / 4);
#pragma unroll
      for (int u = 0; u < U; ++u) scale(w[u], i + u * kThreads);
    }
    for (; i < nv; i += kThreads) {
      uint32_t w[W];
#pragma unroll
      for (int b = 0; b < N; ++b)
        words_of(take_last(reinterpret_cast<const P *>(pv) + (int64_t)i * N + b), w + b * (int)sizeof(P) / 4);
      scale(w, i);
    }
  } else {
    int i = tid;
    for (; i + (U - 1) * kThreads < nv; i += U * kThreads) {
      uint32_t w[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u) load_shifted<P, N>(pv + (int64_t)(i + u * kThreads) * SB, off, w[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) scale(w[u], i + u * kThreads);
    }
    for (; i < nv; i += kThreads) {
      uint32_t w[W];
      load_shifted<P, N>(pv + (int64_t)i * SB, off, w);
      scale(w, i);
    }
  }
  // fewer than V elements on either side
  if (tid < head) q[tid] = from_float<D>(to_float(p[tid]) * coef);
  const int tail = head + nv * V;
  if (tid < n - tail) q[tail + tid] = from_float<D>(to_float(p[tail + tid]) * coef);
}

template <typename S>
__device__ __forceinline__ void scale_chunk_to(const S *p, void *q, int dtype, int64_t at, int n, float coef) {
  if (dtype == SNACK_F32)
    scale_chunk(p, static_cast<float *>(q) + at, n, coef);
  else if (dtype == SNACK_BF16)
    scale_chunk(p, static_cast<__nv_bfloat16 *>(q) + at, n, coef);
  else
    scale_chunk(p, static_cast<__half *>(q) + at, n, coef);
}

template <int K, bool MAX>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) scale_tensors(const __grid_constant__ TensorTable<K> t,
                                                          const float4 *partial, int parts, float max_norm,
                                                          float eps, float *norm) {
  __shared__ float red[32];
  dependency_wait();
  const Norm total = whole_norm<MAX>(partial, parts, red);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total.value();
  const float coef = total.factor(max_norm, eps);
  // from the last chunk back: what the norm read last is still in L2
  for (int64_t i = blockIdx.x; i < t.chunks; i += gridDim.x) {
    const int64_t c = t.chunks - 1 - i;
    const int k = tensor_of(t, (uint32_t)c);
    // in place and nothing to clip: what would be written is there already
    if (coef == 1.f && t.dst[k] == t.src[k]) continue;
    const int64_t at = (c - t.first[k]) * (int64_t)t.chunk_elems;
    const int64_t left = t.n[k] - at;
    const int n = left < t.chunk_elems ? (int)left : t.chunk_elems;
    if (t.stype[k] == SNACK_F32)
      scale_chunk_to(static_cast<const float *>(t.src[k]) + at, t.dst[k], t.dtype[k], at, n, coef);
    else if (t.stype[k] == SNACK_BF16)
      scale_chunk_to(static_cast<const __nv_bfloat16 *>(t.src[k]) + at, t.dst[k], t.dtype[k], at, n, coef);
    else
      scale_chunk_to(static_cast<const __half *>(t.src[k]) + at, t.dst[k], t.dtype[k], at, n, coef);
  }
}

struct Request {
  int64_t count;
  const void *const *grads;
  void *const *outs;
  const int64_t *sizes;
  const int32_t *types, *out_types;
  float max_norm, eps;
  float *norm;
  float4 *partial;
  cudaStream_t s;
};

int grid_blocks() { return device_sms() * kBlocksPerSm; }

// Chunk length: about four chunks for every resident block, so that none
// waits long for the last, between 2048 elements (a sweep of the block in
// 16-byte vectors) and 32768 (beyond it the search for the tensor no longer
// shows).
int chunk_length(int64_t total) {
  int c = 2048;
  while (c < 32768 && total > (int64_t)c * 4 * grid_blocks()) c *= 2;
  return c;
}

// Tensors [i, end) of one launch.
template <int K>
int64_t fill(TensorTable<K> &t, const Request &q, int64_t i, int chunk) {
  t.count = 0;
  t.chunks = 0;
  t.chunk_elems = chunk;
  t.keep_from = 0;
  for (; i < q.count && t.count < K; ++i) {
    if (q.sizes[i] == 0) continue;
    const int64_t c = (q.sizes[i] + chunk - 1) / chunk;
    if (t.chunks + c > 0xffffffffLL) break;
    const int k = t.count++;
    t.src[k] = q.grads[i];
    t.dst[k] = q.outs ? q.outs[i] : const_cast<void *>(q.grads[i]);
    t.n[k] = q.sizes[i];
    t.stype[k] = (uint8_t)q.types[i];
    t.dtype[k] = (uint8_t)(q.outs ? q.out_types[i] : q.types[i]);
    t.first[k] = (uint32_t)t.chunks;
    t.chunks += c;
  }
  // the last kKeepBytes of the launch
  int64_t bytes = 0;
  for (int k = t.count - 1; k >= 0; --k) {
    const int64_t e = type_bytes(t.stype[k]);
    if (bytes + t.n[k] * e > kKeepBytes) {
      t.keep_from = t.first[k] + std::max<int64_t>(0, t.n[k] - (kKeepBytes - bytes) / e) / chunk;
      break;
    }
    bytes += t.n[k] * e;
  }
  return i;
}

// launch_kernel() without its copy of the table (6 or 30 KB).
template <int K, typename... P>
cudaError_t launch_table(void (*kern)(TensorTable<K>, P...), int blocks, cudaStream_t s, TensorTable<K> &t, P... rest) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void *args[] = {&t, &rest...};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kern), args);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int K, bool MAX>
cudaError_t run(const Request &q, bool clip) {
  int64_t total = 0;
  for (int64_t i = 0; i < q.count; ++i) total += q.sizes[i];
  const int chunk = chunk_length(total);
  static thread_local TensorTable<K> t;
  int parts = 0, launches = 0;
  cudaError_t e;
  int64_t next = 0;
  while (next < q.count) {
    next = fill(t, q, next, chunk);
    if (t.count == 0) break;
    ++launches;
    const int g = (int)std::min<int64_t>(t.chunks, grid_blocks());
    e = launch_table<K>(norm_partials<K, MAX>, g, q.s, t, q.partial + parts);
    if (e != cudaSuccess) return e;
    parts += g;
  }
  if (!clip || parts == 0)
    return launch_kernel(norm_finish<MAX>, dim3(1), kThreads, 0, true, q.s, (const float4 *)q.partial, parts,
                         q.norm);
  // the table of a list that one launch took whole is still there
  const bool one = launches == 1 && t.count > 0;
  bool first = true;
  next = 0;
  do {
    if (!one) next = fill(t, q, next, chunk);
    if (t.count == 0) break;
    const int g = (int)std::min<int64_t>(t.chunks, grid_blocks());
    e = launch_table<K>(scale_tensors<K, MAX>, g, q.s, t, (const float4 *)q.partial, parts, q.max_norm, q.eps,
                        first ? q.norm : (float *)nullptr);
    if (e != cudaSuccess) return e;
    first = false;
  } while (!one && next < q.count);
  return cudaSuccess;
}

snack_status check(const Request &q, int norm_kind, const void *workspace, bool clip) {
  if (q.count < 0) return refuse(SNACK_ERR_INVALID_ARG, "count must be >= 0");
  if (norm_kind != 0 && norm_kind != 1) return refuse(SNACK_ERR_INVALID_ARG, "norm_kind must be 0 or 1");
  if (!q.norm || !workspace || (q.count > 0 && (!q.grads || !q.sizes || !q.types)))
    return refuse(SNACK_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned_to(workspace, 16) || !aligned_to(q.norm, 4))
    return refuse(SNACK_ERR_INVALID_ARG, "workspace must be 16-byte aligned, norm 4-byte aligned");
  if (q.outs && !q.out_types) return refuse(SNACK_ERR_INVALID_ARG, "outs without out_types");
  if (clip && !(q.max_norm >= 0.f)) return refuse(SNACK_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (clip && !(q.eps >= 0.f)) return refuse(SNACK_ERR_INVALID_ARG, "eps must be >= 0");
  for (int64_t i = 0; i < q.count; ++i) {
    if (q.sizes[i] < 0) return refuse(SNACK_ERR_INVALID_ARG, "a tensor's size is negative");
    if (!known_type(q.types[i]) || (q.outs && !known_type(q.out_types[i])))
      return refuse(SNACK_ERR_INVALID_ARG, "a tensor's type is not one of snack_dtype");
    if (q.sizes[i] == 0) continue;
    if (!q.grads[i] || (q.outs && !q.outs[i])) return refuse(SNACK_ERR_INVALID_ARG, "a tensor is NULL");
    if (!aligned_to(q.grads[i], type_bytes(q.types[i])) ||
        (q.outs && !aligned_to(q.outs[i], type_bytes(q.out_types[i]))))
      return refuse(SNACK_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
    if (q.outs && q.outs[i] == q.grads[i] && q.out_types[i] != q.types[i])
      return refuse(SNACK_ERR_INVALID_ARG, "an output in place must keep its gradient's type");
  }
  return SNACK_OK;
}

snack_status dispatch(const Request &q, int norm_kind, bool clip) {
  cudaError_t e;
  // a short list takes a short parameter block: 30 KB of parameters cost every launch
#define SNACK_CLIP(K) e = norm_kind ? run<K, true>(q, clip) : run<K, false>(q, clip)
  if (q.count <= 32)
    SNACK_CLIP(32);
  else if (q.count <= 192)
    SNACK_CLIP(192);
  else
    SNACK_CLIP(kMostTable);
#undef SNACK_CLIP
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, clip ? "gradient clipping launch" : "gradient norm launch");
}

}  // namespace
}  // namespace snack

extern "C" size_t snack_grad_norm_workspace(int64_t count) {
  // one partial per block and launch
  const int64_t launches = (count < 0 ? 0 : count) / snack::kMostTable + 2;
  return (size_t)launches * snack::grid_blocks() * sizeof(float4);
}

extern "C" snack_status snack_grad_norm(int64_t count, const void *const *grads, const int64_t *sizes,
                                        const int32_t *types, int norm_kind, float *norm, void *workspace,
                                        void *stream) {
  const snack::Request q = {count, grads, nullptr, sizes, types, nullptr, 0.f, 0.f, norm,
                            static_cast<float4 *>(workspace), static_cast<cudaStream_t>(stream)};
  const snack_status st = snack::check(q, norm_kind, workspace, false);
  return st == SNACK_OK ? snack::dispatch(q, norm_kind, false) : st;
}

extern "C" snack_status snack_clip_grad_norm(int64_t count, const void *const *grads, void *const *outs,
                                             const int64_t *sizes, const int32_t *types,
                                             const int32_t *out_types, int norm_kind, float max_norm,
                                             float eps, float *norm, void *workspace, void *stream) {
  const snack::Request q = {count,    grads, outs, sizes, types, out_types,
                            max_norm, eps,   norm, static_cast<float4 *>(workspace),
                            static_cast<cudaStream_t>(stream)};
  const snack_status st = snack::check(q, norm_kind, workspace, true);
  return st == SNACK_OK ? snack::dispatch(q, norm_kind, true) : st;
}
