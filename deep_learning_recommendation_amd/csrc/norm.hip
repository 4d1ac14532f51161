// Residual addition and root-mean-square norm, with the branch's dropout and
// an optional int8 output with one scale per row; and its gradient.
//
//   h = res + dropout(x),  r = 1 / sqrt(mean h^2 + eps),  y = h r w
//   g = dy w,  t = dh + r g - h r^3 mean(g h),  dres = t,  dx = dropout(t),
//   dw = sum over rows of dy h r
#include "common.hpp"
#include "philox.hpp"
#include "rows.hpp"

namespace dlrm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 16384;

// sum (or maximum) over the block's threads, in a fixed order
template <class Op>
__device__ __forceinline__ float block_reduce(float v, float* s, Op op) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = op(v, __shfl_xor(v, o, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) v = op(v, s[w]);
  return v;
}
struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

__device__ __forceinline__ bool kept(const DropState& st, int64_t e, uint32_t cut) {
  return (keep8(st, (uint64_t)(e >> 3), cut) >> (e & 7)) & 1u;
}

// One block per row, element by element, h recomputed in each pass.
template <class T, class TY>
__global__ __launch_bounds__(kThreads) void addnorm_fwd_kernel(const T* x, int64_t x_ld, const T* res, int64_t res_ld,
                                                               const float* __restrict__ w, int64_t n, int d,
                                                               float eps, uint32_t cut, float factor,
                                                               const int64_t* __restrict__ rng, T* h, int64_t h_ld,
                                                               TY* y, int64_t y_ld, float* __restrict__ scale_bias,
                                                               float* __restrict__ rstd) {
  __shared__ float s[kThreads / 64];
  __shared__ float hrow[kMaxD];
  const DropState st = cut ? drop_state(rng) : DropState{0, 0};
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    float sq = 0.f;
    for (int c = threadIdx.x; c < d; c += kThreads) {
      // the factor's product and the addition round once
      float v = to_f32(x[row * x_ld + c]);
      if (cut) v = kept(st, row * d + c, cut) ? v : 0.f;
      v = __builtin_fmaf(v, factor, res ? to_f32(res[row * res_ld + c]) : 0.f);
      hrow[c] = v;
      if (h) h[row * h_ld + c] = from_f32<T>(v);
      sq += v * v;
    }
    const float r = 1.f / sqrtf(block_reduce(sq, s, Add()) / (float)d + eps);
    if (rstd && threadIdx.x == 0) rstd[row] = r;
    if constexpr (sizeof(TY) == 1) {
      float top = 0.f, nan = 0.f;
      for (int c = threadIdx.x; c < d; c += kThreads) {
        const float v = hrow[c] * r * w[c];
        top = fmaxf(top, fabsf(v));
        if (v != v) nan = 1.f;
      }
      top = block_reduce(top, s, Max());
      nan = block_reduce(nan, s, Max());
      const float unit = nan > 0.f ? __uint_as_float(0x7fc00000u) : top / 127.f;
      if (threadIdx.x == 0) {
        scale_bias[2 * row] = unit;
        scale_bias[2 * row + 1] = 0.f;
      }
      for (int c = threadIdx.x; c < d; c += kThreads) {
        const float q = rintf(hrow[c] * r * w[c] / unit);
        y[row * y_ld + c] = unit > 0.f ? (TY)fminf(fmaxf(q, -127.f), 127.f) : (TY)0;
      }
    } else {
      for (int c = threadIdx.x; c < d; c += kThreads) y[row * y_ld + c] = from_f32<TY>(hrow[c] * r * w[c]);
    }
    __syncthreads();
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void addnorm_bwd_kernel(const T* dy, int64_t dy_ld, const T* dh, int64_t dh_ld,
                                                               const T* __restrict__ h, int64_t h_ld,
                                                               const float* __restrict__ w,
                                                               const float* __restrict__ rstd, int64_t n, int d,
                                                               uint32_t cut, float factor,
                                                               const int64_t* __restrict__ rng, T* dx, int64_t dx_ld,
                                                               T* dres, int64_t dres_ld, float* __restrict__ part) {
  __shared__ float s[kThreads / 64];
  __shared__ float dwrow[kMaxD];
  const DropState st = cut ? drop_state(rng) : DropState{0, 0};
  for (int c = threadIdx.x; c < d; c += kThreads) dwrow[c] = 0.f;
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const float r = rstd[row];
    float dot = 0.f;
    for (int c = threadIdx.x; c < d; c += kThreads) {
      const float gy = to_f32(dy[row * dy_ld + c]), hv = to_f32(h[row * h_ld + c]);
      dot += gy * w[c] * hv;
      dwrow[c] += gy * hv * r;
    }
    const float k = block_reduce(dot, s, Add()) / (float)d * r * r * r;
    for (int c = threadIdx.x; c < d; c += kThreads) {
      float t = r * (to_f32(dy[row * dy_ld + c]) * w[c]) - k * to_f32(h[row * h_ld + c]);
      if (dh) t += to_f32(dh[row * dh_ld + c]);
      const float tx = cut ? (kept(st, row * d + c, cut) ? t * factor : 0.f) : t;
      if (dres) dres[row * dres_ld + c] = from_f32<T>(t);
      if (dx) dx[row * dx_ld + c] = from_f32<T>(tx);
    }
  }
  for (int c = threadIdx.x; c < d; c += kThreads) part[(int64_t)blockIdx.x * d + c] = dwrow[c];
}

// dw[c] = the blocks' sums in block order
__global__ __launch_bounds__(kThreads) void dw_kernel(const float* __restrict__ part, int blocks, int d,
                                                      float* __restrict__ dw) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= d) return;
  float a = 0.f;
  for (int b = 0; b < blocks; ++b) a += part[(int64_t)b * d + c];
  dw[c] = a;
}

constexpr int kBwdBlocks = 1024;

template <class T, class TY>
int launch_fwd(const void* x, int64_t x_ld, const void* res, int64_t res_ld, const float* w, int64_t n, int d,
               float eps, uint32_t cut, const int64_t* rng, void* h, int64_t h_ld, void* y, int64_t y_ld,
               float* scale_bias, float* rstd, hipStream_t stream) {
  hipLaunchKernelGGL((addnorm_fwd_kernel<T, TY>), dim3((unsigned)(n < 65536 ? n : 65536)), dim3(kThreads), 0, stream,
                     static_cast<const T*>(x), x_ld, static_cast<const T*>(res), res_ld, w, n, d, eps, cut,
                     drop_factor(cut), rng, static_cast<T*>(h), h_ld, static_cast<TY*>(y), y_ld, scale_bias, rstd);
  return launch_status();
}

template <class T>
int launch_bwd(const void* dy, int64_t dy_ld, const void* dh, int64_t dh_ld, const void* h, int64_t h_ld,
               const float* w, const float* rstd, int64_t n, int d, uint32_t cut, const int64_t* rng, void* dx,
               int64_t dx_ld, void* dres, int64_t dres_ld, float* dw, float* part, hipStream_t stream) {
  const int blocks = (int)(n < kBwdBlocks ? n : kBwdBlocks);
  if (blocks > 0)
    hipLaunchKernelGGL((addnorm_bwd_kernel<T>), dim3(blocks), dim3(kThreads), 0, stream, static_cast<const T*>(dy),
                       dy_ld, static_cast<const T*>(dh), dh_ld, static_cast<const T*>(h), h_ld, w, rstd, n, d, cut,
                       drop_factor(cut), rng, static_cast<T*>(dx), dx_ld, static_cast<T*>(dres), dres_ld, part);
  hipLaunchKernelGGL(dw_kernel, dim3((unsigned)ceil_div(d, kThreads)), dim3(kThreads), 0, stream, part, blocks, d, dw);
  return launch_status();
}

// a nullable row array: absent, or wide enough and aligned to its element
bool rows_fit(const void* p, int64_t ld, int32_t d, size_t e) {
  return !p || (ld >= d && (reinterpret_cast<uintptr_t>(p) % e) == 0);
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" int dlrm_add_rmsnorm_fwd(const void* x, int64_t x_ld, const void* res, int64_t res_ld, int32_t dtype,
                                    const float* w, int64_t n, int32_t d, float eps, float p, const int64_t* rng,
                                    void* h, int64_t h_ld, void* y, int32_t y_dtype, int64_t y_ld, float* scale_bias,
                                    float* rstd, hipStream_t stream) {
  if (!is_activation(dtype) || (y_dtype != dtype && y_dtype != DLRM_I8) || n < 0 || d < 1 || d > kMaxD)
    return DLRM_E_INVALID;
  if (!(p >= 0.f && p <= 1.f) || !(eps >= 0.f)) return DLRM_E_INVALID;
  if (n == 0) return DLRM_OK;
  const bool i8 = y_dtype == DLRM_I8;
  const size_t e = elem_size(dtype);
  if (!x || !w || !y || (p > 0.f && !rng) || (i8 && !scale_bias)) return DLRM_E_INVALID;
  if (!rows_fit(x, x_ld, d, e) || !rows_fit(res, res_ld, d, e) || !rows_fit(h, h_ld, d, e) ||
      !rows_fit(y, y_ld, d, i8 ? 1 : e))
    return DLRM_E_INVALID;
  if ((h && h == x && h_ld != x_ld) || (h && h == res && h_ld != res_ld)) return DLRM_E_INVALID;
  if (n > (1LL << 40) / d) return DLRM_E_UNSUPPORTED;
  const uint32_t cut = drop_cut(p);
  if (dtype == DLRM_F32) {
    if (i8)
      return launch_fwd<float, int8_t>(x, x_ld, res, res_ld, w, n, d, eps, cut, rng, h, h_ld, y, y_ld, scale_bias,
                                       rstd, stream);
    return launch_fwd<float, float>(x, x_ld, res, res_ld, w, n, d, eps, cut, rng, h, h_ld, y, y_ld, nullptr, rstd,
                                    stream);
  }
  if (i8)
    return launch_fwd<uint16_t, int8_t>(x, x_ld, res, res_ld, w, n, d, eps, cut, rng, h, h_ld, y, y_ld, scale_bias,
                                        rstd, stream);
  return launch_fwd<uint16_t, uint16_t>(x, x_ld, res, res_ld, w, n, d, eps, cut, rng, h, h_ld, y, y_ld, nullptr, rstd,
                                        stream);
}

extern "C" size_t dlrm_add_rmsnorm_bwd_workspace_size(int64_t n, int32_t d) {
  if (n < 0 || d < 1 || d > kMaxD) return 0;
  return (size_t)round_up((n < kBwdBlocks ? n : kBwdBlocks) * 4 * (int64_t)d, 256);
}

extern "C" int dlrm_add_rmsnorm_bwd(const void* dy, int64_t dy_ld, const void* dh, int64_t dh_ld, const void* h,
                                    int64_t h_ld, int32_t dtype, const float* w, const float* rstd, int64_t n,
                                    int32_t d, float p, const int64_t* rng, void* dx, int64_t dx_ld, void* dres,
                                    int64_t dres_ld, float* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!is_activation(dtype) || n < 0 || d < 1 || d > kMaxD || !(p >= 0.f && p <= 1.f) || !dw) return DLRM_E_INVALID;
  const size_t e = elem_size(dtype);
  if (n > 0 && (!dy || !h || !w || !rstd || (!dx && !dres) || (p > 0.f && !rng))) return DLRM_E_INVALID;
  if (!rows_fit(dy, dy_ld, d, e) || !rows_fit(dh, dh_ld, d, e) || !rows_fit(h, h_ld, d, e) ||
      !rows_fit(dx, dx_ld, d, e) || !rows_fit(dres, dres_ld, d, e))
    return DLRM_E_INVALID;
  if (dx && dx == dres) return DLRM_E_INVALID;
  for (const void* o : {(const void*)dx, (const void*)dres}) {  // in place only row on row
    const int64_t o_ld = o == dx ? dx_ld : dres_ld;
    if (o && ((o == dy && o_ld != dy_ld) || (o == dh && o_ld != dh_ld) || o == h)) return DLRM_E_INVALID;
  }
  if (n > (1LL << 40) / d) return DLRM_E_UNSUPPORTED;
  if (n > 0 && (!ws || ws_bytes < dlrm_add_rmsnorm_bwd_workspace_size(n, d))) return DLRM_E_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return DLRM_E_INVALID;
  float* part = static_cast<float*>(ws);
  const uint32_t cut = drop_cut(p);
  if (dtype == DLRM_F32)
    return launch_bwd<float>(dy, dy_ld, dh, dh_ld, h, h_ld, w, rstd, n, d, cut, rng, dx, dx_ld, dres, dres_ld, dw,
                             part, stream);
  return launch_bwd<uint16_t>(dy, dy_ld, dh, dh_ld, h, h_ld, w, rstd, n, d, cut, rng, dx, dx_ld, dres, dres_ld, dw,
                              part, stream);
}
