// Dropout from a counter-based generator:
//   y[e] = keep(e) ? x[e] * 65536 / (65536 - cut) : +0
// with keep(e) a function of (seed, offset, e) alone (philox.hpp), so the
// backward pass recomputes the mask instead of reading one.  Bound by memory:
// 20 32 x 32-bit products per eight elements hide behind their bytes.
#include "common.hpp"
#include "philox.hpp"
#include "rows.hpp"

namespace dlrm {
namespace {

// Rows without gaps are one flat list: a thread takes one counter, eight
// consecutive elements, with 16-byte accesses.  819200 x 128 bf16: 70 us,
// 6.0 TB/s.
template <class T>
__global__ __launch_bounds__(256) void dropout_flat_kernel(const T* x, T* y, int64_t total, uint32_t cut, float factor,
                                                           const int64_t* __restrict__ rng) {
  const DropState st = drop_state(rng);
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g * 8 < total; g += step) {
    if (g * 8 + 8 <= total) {
      Piece<T, 8> p;
      p.load(x + g * 8);
      const uint32_t keep = keep8(st, (uint64_t)g, cut);
      float v[8];
      p.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (keep >> j) & 1u ? v[j] * factor : 0.f;
      p.set(v);
      p.store(y + g * 8);
    } else {
      const uint32_t keep = keep8(st, (uint64_t)g, cut);
      for (int j = 0; g * 8 + j < total; ++j)
        y[g * 8 + j] = (keep >> j) & 1u ? from_f32<T>(to_f32(x[g * 8 + j]) * factor) : from_f32<T>(0.f);
    }
  }
}

// Rows with gaps: a counter's eight elements may lie in two rows, and a
// row's pieces of VE elements in two counters.  A block takes a tile (as
// many whole rows as kTile elements hold, or kTile columns of one row), puts
// the keep bits of the tile's elements into LDS, one thread per counter,
// then walks the tile's pieces.  16384 x 479 of 512 fp32: 15 us, 4.1 TB/s (one
// thread per counter with single-element accesses: 40 us).
constexpr int kTile = 8192;

template <class T, int VE>
__global__ __launch_bounds__(256) void dropout_rows_kernel(const T* x, int64_t x_ld, T* y, int64_t y_ld, int64_t rows,
                                                           int64_t cols, int tile_rows, int64_t tiles_c,
                                                           int64_t tiles, uint32_t cut, float factor,
                                                           const int64_t* __restrict__ rng) {
  __shared__ uint8_t keep[kTile / 8 + 4];
  const DropState st = drop_state(rng);
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile / tiles_c * tile_rows, c0 = tile % tiles_c * kTile;
    const int nr = (int)(rows - r0 < tile_rows ? rows - r0 : tile_rows);
    const int nc = (int)(cols - c0 < kTile ? cols - c0 : kTile);
    const int64_t e0 = r0 * cols + c0, g0 = e0 >> 3;
    const int lead = (int)(e0 & 7), n = nr * nc;  // the tile's elements lie together: whole rows, or one
    for (int i = threadIdx.x; i * 8 < lead + n; i += 256) keep[i] = (uint8_t)keep8(st, (uint64_t)(g0 + i), cut);
    __syncthreads();
    const int per_row = (nc + VE - 1) / VE;
    for (int i = threadIdx.x; i < nr * per_row; i += 256) {
      const int r = i / per_row, c = (i - r * per_row) * VE;
      const T* src = x + (r0 + r) * x_ld + c0 + c;
      T* dst = y + (r0 + r) * y_ld + c0 + c;
      const int at = lead + r * nc + c;
      if (VE > 1 && c + VE <= nc) {
        const uint32_t k = ((uint32_t)keep[at >> 3] | (uint32_t)keep[(at >> 3) + 1] << 8) >> (at & 7);
        Piece<T, 4> p;
        p.load(src);
        float v[4];
        p.get(v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (k >> j) & 1u ? v[j] * factor : 0.f;
        p.set(v);
        p.store(dst);
      } else {
        for (int j = 0; j < VE && c + j < nc; ++j)
          dst[j] = (keep[(at + j) >> 3] >> ((at + j) & 7)) & 1u ? from_f32<T>(to_f32(src[j]) * factor) : from_f32<T>(0.f);
      }
    }
    __syncthreads();
  }
}

constexpr int64_t kMaxBlocks = 16384;

template <class T>
int launch(const void* x_, int64_t x_ld, void* y_, int64_t y_ld, int64_t rows, int64_t cols, uint32_t cut,
           const int64_t* rng, hipStream_t stream) {
  const T* x = static_cast<const T*>(x_);
  T* y = static_cast<T*>(y_);
  const float factor = drop_factor(cut);
  if (rows == 1 || (x_ld == cols && y_ld == cols)) {  // one flat list
    cols *= rows;
    rows = 1;
    if (aligned16(x) && aligned16(y)) {
      const int64_t blocks = ceil_div(ceil_div(cols, 8), 256);
      hipLaunchKernelGGL((dropout_flat_kernel<T>), dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(256),
                         0, stream, x, y, cols, cut, factor, rng);
      return launch_status();
    }
  }
  const int tile_rows = (int)(cols >= kTile ? 1 : kTile / cols);
  const int64_t tiles_c = ceil_div(cols, kTile), tiles = ceil_div(rows, tile_rows) * tiles_c;
  const dim3 grid((unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks));
  if (rows_aligned(x, x_ld, sizeof(T), 4 * sizeof(T)) && rows_aligned(y, y_ld, sizeof(T), 4 * sizeof(T)))
    hipLaunchKernelGGL((dropout_rows_kernel<T, 4>), grid, dim3(256), 0, stream, x, x_ld, y, y_ld, rows, cols, tile_rows,
                       tiles_c, tiles, cut, factor, rng);
  else
    hipLaunchKernelGGL((dropout_rows_kernel<T, 1>), grid, dim3(256), 0, stream, x, x_ld, y, y_ld, rows, cols, tile_rows,
                       tiles_c, tiles, cut, factor, rng);
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
