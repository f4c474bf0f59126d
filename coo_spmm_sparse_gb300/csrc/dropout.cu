// Dropout with the residual's addition: y = residual + M * x, and dx = M * dy.
//
// M is made from the seed and the element's number wherever it is needed.  The
// memory binds: two or three streams, 16 bytes of the narrower type a thread
// and step.
#include <cmath>

#include "counter_random.cuh"
#include "dense_ops.cuh"

namespace snack {
namespace {

struct DropCall {
  const void *x, *residual;
  void *y;
  int64_t n;
  uint32_t drop;
  float scale;
  uint64_t seed;
  const uint64_t *seed_at;
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
    unpack2<T>(u.x, v[0], v[1]);
    unpack2<T>(u.y, v[2], v[3]);
    unpack2<T>(u.z, v[4], v[5]);
    unpack2<T>(u.w, v[6], v[7]);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                                               pack2<T>(v[6], v[7]));
  }
}

// A dropped element adds nothing, whatever x holds there.
template <typename X, typename Y, bool RES, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(const DropCall c) {
  const X *x = static_cast<const X *>(c.x);
  const Y *res = static_cast<const Y *>(c.residual);
  Y *y = static_cast<Y *>(c.y);
  const uint64_t seed = c.seed_at ? *c.seed_at : c.seed;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= c.n) return;
  const uint64_t z[2] = {splitmix(seed, (uint64_t)i >> 2), splitmix(seed, ((uint64_t)i >> 2) + 1)};
  if (VEC && i + 8 <= c.n) {
    float v[8], r[8];
    load8(x + i, v);
    if (RES) load8(res + i, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float kept = draw_lane(z[e >> 2], e & 3) >= c.drop ? v[e] * c.scale : 0.f;
      v[e] = RES ? r[e] + kept : kept;
    }
    store8(y + i, v);
    return;
  }
  for (int e = 0; e < 8 && i + e < c.n; ++e) {
    const float kept = draw_lane(z[e >> 2], e & 3) >= c.drop ? to_float(x[i + e]) * c.scale : 0.f;
    y[i + e] = from_float<Y>(RES ? to_float(res[i + e]) + kept : kept);
  }
}

template <typename X, typename Y>
cudaError_t dropout_typed(const DropCall &c, cudaStream_t s) {
  const dim3 grid((unsigned)((c.n + 2047) / 2048));
  const bool vec = aligned_to(c.x, 16) && aligned_to(c.y, 16) && aligned_to(c.residual, 16);
  if (c.residual)
    return vec ? launch_kernel(dropout_kernel<X, Y, true, true>, grid, 256, 0, false, s, c)
               : launch_kernel(dropout_kernel<X, Y, true, false>, grid, 256, 0, false, s, c);
  return vec ? launch_kernel(dropout_kernel<X, Y, false, true>, grid, 256, 0, false, s, c)
             : launch_kernel(dropout_kernel<X, Y, false, false>, grid, 256, 0, false, s, c);
}

template <typename X>
cudaError_t dropout_from(const DropCall &c, int y_type, cudaStream_t s) {
  return y_type == SNACK_F32    ? dropout_typed<X, float>(c, s)
         : y_type == SNACK_BF16 ? dropout_typed<X, __nv_bfloat16>(c, s)
                                : dropout_typed<X, __half>(c, s);
}

}  // namespace
}  // namespace snack

using namespace snack;

extern "C" snack_status snack_dropout(int64_t n, const void *x, int x_type, const void *residual, void *y, int y_type,
                                      float p, uint64_t seed, const uint64_t *seed_at, void *stream) {
  if (!known_type(x_type) || !known_type(y_type)) return refuse(SNACK_ERR_INVALID_ARG, "unknown element type");
  if (n < 0) return refuse(SNACK_ERR_INVALID_ARG, "negative size");
  if (!(p >= 0.f && p < 1.f) || std::lround(p * 65536.0) > 65535)
    return refuse(SNACK_ERR_INVALID_ARG, "p must be at least 0 and below 1 - 2^-17");
  if (n == 0) return SNACK_OK;
  if (n >= (int64_t)1 << 41) return refuse(SNACK_ERR_UNSUPPORTED, "more than 2^41 elements");
  if (!x || !y) return refuse(SNACK_ERR_INVALID_ARG, "x or y is NULL");
  DropCall c{x, residual, y, n, (uint32_t)std::lround(p * 65536.0), 1.f, seed, seed_at};
  c.scale = 65536.f / (float)(65536 - c.drop);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = x_type == SNACK_F32    ? dropout_from<float>(c, y_type, s)
                        : x_type == SNACK_BF16 ? dropout_from<__nv_bfloat16>(c, y_type, s)
                                               : dropout_from<__half>(c, y_type, s);
  return e == cudaSuccess ? SNACK_OK : cuda_status(e, "dropout");
}
