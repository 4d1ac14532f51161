// Dropout from a counter-based generator:
//   y[e] = keep(e) ? x[e] * 65536 / (65536 - cut) : +0
// with keep(e) a function of (seed, offset, e) alone (philox.hpp), so the
// backward pass recomputes the mask instead of reading one.
#include "common.hpp"
#include "philox.hpp"
#include "rows.hpp"

namespace dlrm {
namespace {

// one thread per counter: eight consecutive elements
template <class T>
__global__ __launch_bounds__(256) void dropout_kernel(const T* x, int64_t x_ld, T* y, int64_t y_ld, int64_t total,
                                                      int64_t cols, uint32_t cut, float factor,
                                                      const int64_t* __restrict__ rng) {
  const DropState st = drop_state(rng);
  const int64_t groups = (total + 7) / 8, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g < groups; g += step) {
    const uint32_t keep = keep8(st, (uint64_t)g, cut);
    int64_t r = g * 8 / cols, c = g * 8 - r * cols;
    for (int j = 0; j < 8 && g * 8 + j < total; ++j) {
      y[r * y_ld + c] = (keep >> j) & 1u ? from_f32<T>(to_f32(x[r * x_ld + c]) * factor) : from_f32<T>(0.f);
      if (++c == cols) {
        c = 0;
        ++r;
      }
    }
  }
}

template <class T>
int launch(const void* x, int64_t x_ld, void* y, int64_t y_ld, int64_t rows, int64_t cols, uint32_t cut,
           const int64_t* rng, hipStream_t stream) {
  const int64_t total = rows * cols, blocks = ceil_div(ceil_div(total, 8), 256);
  hipLaunchKernelGGL((dropout_kernel<T>), dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, stream,
                     static_cast<const T*>(x), x_ld, static_cast<T*>(y), y_ld, total, cols, cut, drop_factor(cut),
                     rng);
  return launch_status();
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" int dlrm_dropout(const void* x, int64_t x_ld, void* y, int64_t y_ld, int32_t dtype, int64_t rows,
                            int64_t cols, float p, const int64_t* rng, hipStream_t stream) {
  if (!is_activation(dtype) || rows < 0 || cols < 1 || !(p >= 0.f && p <= 1.f)) return DLRM_E_INVALID;
  if (x_ld < cols || y_ld < cols || (x == y && x_ld != y_ld)) return DLRM_E_INVALID;
  if (rows == 0) return DLRM_OK;
  const size_t e = elem_size(dtype);
  if (!x || !y || !rng || (reinterpret_cast<uintptr_t>(x) % e) || (reinterpret_cast<uintptr_t>(y) % e) ||
      (reinterpret_cast<uintptr_t>(rng) % 8))
    return DLRM_E_INVALID;
  if (rows > (1LL << 40) / cols) return DLRM_E_UNSUPPORTED;
  const uint32_t cut = drop_cut(p);
  if (dtype == DLRM_F32) return launch<float>(x, x_ld, y, y_ld, rows, cols, cut, rng, stream);
  return launch<uint16_t>(x, x_ld, y, y_ld, rows, cols, cut, rng, stream);
}
