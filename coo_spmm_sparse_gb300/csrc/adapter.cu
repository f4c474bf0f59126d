// Low-rank adapters of many requests beside one projection:
//
//   H[t] = A_n X[t],  Y[t] += s_n B_n H[t]        n: the adapter of token t's request
//   dH[t] = s_n B_n^T dY[t],  dX[t] += A_n^T dH[t],
//   dA_n = sum_t dH[t] X[t]^T,  dB_n = s_n sum_t dY[t] H[t]^T
#include <algorithm>

#include "dense_ops.cuh"

namespace snack {
namespace {

constexpr int kThreads = 256;

struct AdapterArgs {
  snack_adapter_args a;
  void *Y;
  int64_t y_stride;
  const void *dY;
  int64_t dy_stride;
  void *dX;
  int64_t dx_stride;
  float *H;         // [tokens][rank]
  const float *Hin;
  float *dH;        // [tokens][rank]
  void *dA, *dB;
};

// The adapter of token t, or -1.
__device__ __forceinline__ int adapter_of(const snack_adapter_args &a, int64_t t) {
  // the last request that begins at or before t; requests that hold nothing
  // begin where the next one does
  int lo = 0, hi = (int)a.requests;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  if (lo == 0 || t >= a.offsets[lo]) return -1;
  const int n = a.adapter[lo - 1];
  return n >= 0 && n < a.adapters ? n : -1;
}

__device__ __forceinline__ float scale_of(const snack_adapter_args &a, int n) {
  return a.scale ? a.scale[n] : a.uniform_scale;
}

// A warp for each (token, rank index): the product over `in`.
template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_down(const __grid_constant__ AdapterArgs q) {
  dependency_wait();
  const snack_adapter_args &a = q.a;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; w < a.tokens * a.rank; w += warps) {
    const int64_t t = w / a.rank, j = w % a.rank;
    const int n = adapter_of(a, t);
    float s = 0.f;
    if (n >= 0) {
      const T *x = static_cast<const T *>(a.X) + t * a.x_stride;
      const T *m = static_cast<const T *>(a.A) + ((int64_t)n * a.rank + j) * a.in;
      for (int64_t i = lane; i < a.in; i += 32) s = fmaf(to_float(x[i]), to_float(m[i]), s);
      s = warp_sum(s);
    }
    if (lane == 0) q.H[w] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_up(const __grid_constant__ AdapterArgs q) {
  dependency_wait();
  const snack_adapter_args &a = q.a;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int n = adapter_of(a, t);
    if (n < 0) continue;
    const float scale = scale_of(a, n);
    for (int64_t o = threadIdx.x; o < a.out; o += kThreads) {
      const T *m = static_cast<const T *>(a.B) + ((int64_t)n * a.out + o) * a.rank;
      float s = 0.f;
      for (int64_t j = 0; j < a.rank; ++j) s = fmaf(q.H[t * a.rank + j], to_float(m[j]), s);
      T *y = static_cast<T *>(q.Y) + t * q.y_stride + o;
      *y = from_float<T>(fmaf(scale, s, to_float(*y)));
    }
  }
}

// A warp for each (token, rank index): dH.
template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_back_rank(const __grid_constant__ AdapterArgs q) {
  dependency_wait();
  const snack_adapter_args &a = q.a;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; w < a.tokens * a.rank; w += warps) {
    const int64_t t = w / a.rank, j = w % a.rank;
    const int n = adapter_of(a, t);
    float s = 0.f;
    if (n >= 0) {
      const T *dy = static_cast<const T *>(q.dY) + t * q.dy_stride;
      const T *m = static_cast<const T *>(a.B) + (int64_t)n * a.out * a.rank + j;
      for (int64_t o = lane; o < a.out; o += 32) s = fmaf(to_float(dy[o]), to_float(m[o * a.rank]), s);
      s = warp_sum(s) * scale_of(a, n);
    }
    if (lane == 0) q.dH[w] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) adapter_back_input(const __grid_constant__ AdapterArgs q) {
  dependency_wait();
  const snack_adapter_args &a = q.a;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int n = adapter_of(a, t);
    if (n < 0) continue;
    for (int64_t i = threadIdx.x; i < a.in; i += kThreads) {
      const T *m = static_cast<const T *>(a.A) + (int64_t)n * a.rank * a.in + i;
      float s = 0.f;
      for (int64_t j = 0; j < a.rank; ++j) s = fmaf(q.dH[t * a.rank + j], to_float(m[j * a.in]), s);
      T *dx = static_cast<T *>(q.dX) + t * q.dx_stride + i;
      *dx = from_float<T>(to_float(*dx) + s);
    }
  }
}

// One thread for each element of dA (or dB): the sum over the tokens of the
// adapter's requests.
template <typename T, bool DB>
__global__ void __launch_bounds__(kThreads) adapter_back_weights(const __grid_constant__ AdapterArgs q) {
  dependency_wait();
  const snack_adapter_args &a = q.a;
  const int64_t len = DB ? a.out : a.in, total = a.adapters * a.rank * len;
  const T *big = static_cast<const T *>(DB ? q.dY : a.X);
  const int64_t stride = DB ? q.dy_stride : a.x_stride;
  const float *small = DB ? q.Hin : q.dH;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < total; e += (int64_t)gridDim.x * kThreads) {
    const int64_t n = e / (a.rank * len), rest = e % (a.rank * len);
    const int64_t j = DB ? rest % a.rank : rest / len, i = DB ? rest / a.rank : rest % len;
    float s = 0.f;
    bool used = false;
    for (int64_t r = 0; r < a.requests; ++r) {
      if (a.adapter[r] != n) continue;
      used = true;
      const int64_t t0 = max(0, a.offsets[r]), t1 = min((int64_t)a.offsets[r + 1], a.tokens);
      float part = 0.f;
      for (int64_t t = t0; t < t1; ++t) part = fmaf(small[t * a.rank + j], to_float(big[t * stride + i]), part);
      s += part;
    }
    static_cast<T *>(DB ? q.dB : q.dA)[e] = from_float<T>(DB && used ? s * scale_of(a, (int)n) : s);
  }
}

const char *bad_args(const snack_adapter_args *a) {
  if (!a) return "args is NULL";
  if (a->tokens < 0 || a->tokens > 0x7fffffffLL || a->requests < 0 || a->requests > 0x7ffffffeLL)
    return "tokens and requests must be in [0, 2^31)";
  if (a->adapters < 0 || a->adapters > 65536) return "adapters must be in [0, 65536]";
  if (a->in < 1 || a->out < 1 || a->in > 0x7fffffffLL || a->out > 0x7fffffffLL)
    return "in and out must be in [1, 2^31)";
  if (a->rank < 1 || a->rank > 512) return "rank must be in [1, 512]";
  if (!known_type(a->type)) return "type is not one of snack_dtype";
  if (a->tokens > 0 && a->requests > 0 && (!a->offsets || !a->adapter)) return "offsets or adapter is NULL";
  if (a->tokens > 0 && a->adapters > 0 && (!a->X || !a->A || !a->B)) return "X, A or B is NULL";
  if (a->tokens > 1 && a->x_stride < a->in) return "x_stride is below in";
  const int64_t e = type_bytes(a->type);
  if (!aligned_to(a->X, e) || !aligned_to(a->A, e) || !aligned_to(a->B, e) || !aligned_to(a->offsets, 4) ||
      !aligned_to(a->adapter, 4) || !aligned_to(a->scale, 4))
    return "a pointer is not aligned to its elements";
  return nullptr;
}

bool overlap(const void *p, int64_t pb, const void *q, int64_t qb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
  return p && q && x < y + (uintptr_t)qb && y < x + (uintptr_t)pb;
}

int64_t rows_bytes(int64_t rows, int64_t stride, int64_t width, int type) {
  return rows < 1 ? 0 : ((rows - 1) * stride + width) * type_bytes(type);
}

template <typename K>
cudaError_t go(K kern, int64_t blocks, const AdapterArgs &q, cudaStream_t s) {
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(blocks, (int64_t)device_sms() * 8));
  return launch_kernel(kern, dim3((unsigned)grid), kThreads, 0, true, s, q);
}

template <typename T>
cudaError_t forward(const AdapterArgs &q, cudaStream_t s) {
  cudaError_t e = go(adapter_down<T>, (q.a.tokens * q.a.rank + 7) / 8, q, s);
  return e != cudaSuccess ? e : go(adapter_up<T>, q.a.tokens, q, s);
}

template <typename T>
cudaError_t backward(const AdapterArgs &q, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (q.a.tokens > 0) e = go(adapter_back_rank<T>, (q.a.tokens * q.a.rank + 7) / 8, q, s);
  if (e == cudaSuccess && q.dX && q.a.tokens > 0) e = go(adapter_back_input<T>, q.a.tokens, q, s);
  const int64_t per = q.a.adapters * q.a.rank;
  if (e == cudaSuccess && q.dA && per > 0)
    e = go(adapter_back_weights<T, false>, (per * q.a.in + kThreads - 1) / kThreads, q, s);
  if (e == cudaSuccess && q.dB && per > 0)
    e = go(adapter_back_weights<T, true>, (per * q.a.out + kThreads - 1) / kThreads, q, s);
  return e;
}

#define SNACK_TYPES(type, F)                       \
  ((type) == SNACK_F32 ? F<float>(q, s) : (type) == SNACK_BF16 ? F<__nv_bfloat16>(q, s) : F<__half>(q, s))

}  // namespace
}  // namespace snack

extern "C" size_t snack_adapter_forward_workspace(const snack_adapter_args *args) {
  (void)args;
  return 16;
}

extern "C" snack_status snack_adapter_forward(const snack_adapter_args *args, void *Y, int64_t y_stride,
                                              float *H, void *workspace, void *stream) {
  using namespace snack;
  if (const char *bad = bad_args(args)) return refuse(SNACK_ERR_INVALID_ARG, bad);
  const snack_adapter_args &a = *args;
  if (a.tokens == 0) return SNACK_OK;
  if (!Y || !H) return refuse(SNACK_ERR_INVALID_ARG, "Y or H is NULL");
  if (!workspace || !aligned_to(workspace, 16))
    return refuse(SNACK_ERR_INVALID_ARG, "workspace must be 16-byte aligned device memory");
  if (a.tokens > 1 && y_stride < a.out) return refuse(SNACK_ERR_INVALID_ARG, "y_stride is below out");
  if (!aligned_to(Y, type_bytes(a.type)) || !aligned_to(H, 4))
    return refuse(SNACK_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  if (overlap(a.X, rows_bytes(a.tokens, a.x_stride, a.in, a.type), Y, rows_bytes(a.tokens, y_stride, a.out, a.type)))
    return refuse(SNACK_ERR_INVALID_ARG, "Y overlaps X");
  AdapterArgs q = {};
  q.a = a;
  q.Y = Y;
  q.y_stride = y_stride;
  q.H = H;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = SNACK_TYPES(a.type, forward);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "adapter launch");
}

extern "C" size_t snack_adapter_backward_workspace(const snack_adapter_args *args) {
  return snack::bad_args(args) ? 16 : (size_t)(args->tokens * args->rank * 4 + 16);
}

extern "C" snack_status snack_adapter_backward(const snack_adapter_args *args, const void *dY,
                                               int64_t dy_stride, const float *H, void *dX, int64_t dx_stride,
                                               void *dA, void *dB, void *workspace, void *stream) {
  using namespace snack;
  if (const char *bad = bad_args(args)) return refuse(SNACK_ERR_INVALID_ARG, bad);
  const snack_adapter_args &a = *args;
  if (!workspace || !aligned_to(workspace, 16))
    return refuse(SNACK_ERR_INVALID_ARG, "workspace must be 16-byte aligned device memory");
  if (a.tokens > 0 && (!dY || !H)) return refuse(SNACK_ERR_INVALID_ARG, "dY or H is NULL");
  if (a.tokens > 1 && (dy_stride < a.out || (dX && dx_stride < a.in)))
    return refuse(SNACK_ERR_INVALID_ARG, "a row stride is below its width");
  const int64_t e0 = type_bytes(a.type);
  if (!aligned_to(dY, e0) || !aligned_to(dX, e0) || !aligned_to(dA, e0) || !aligned_to(dB, e0) || !aligned_to(H, 4))
    return refuse(SNACK_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const int64_t dxb = rows_bytes(a.tokens, dx_stride, a.in, a.type);
  if (overlap(a.X, rows_bytes(a.tokens, a.x_stride, a.in, a.type), dX, dxb) ||
      overlap(dY, rows_bytes(a.tokens, dy_stride, a.out, a.type), dX, dxb))
    return refuse(SNACK_ERR_INVALID_ARG, "dX overlaps X or dY");
  AdapterArgs q = {};
  q.a = a;
  q.dY = dY;
  q.dy_stride = dy_stride;
  q.dX = dX;
  q.dx_stride = dx_stride;
  q.Hin = H;
  q.dA = dA;
  q.dB = dB;
  q.dH = static_cast<float *>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = SNACK_TYPES(a.type, backward);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "adapter backward launch");
}
