// quant8.hip -- a matrix in e4m3 with a scale for each block: by rows, transposed, or both
// from one read.
//
// For a block with magnitudes up to a:  m = max(a, 2^-100), q = e4m3(v (448 / m)) to nearest
// even, scale = m / 448.  A block is 128 elements of a row (of a column, for the transposed
// form), or a tile of 128 x 128 that both forms share.
//
// Bound by HBM: each element is read once and written once or twice as a byte.  2 x 4096 x 5120
// bf16 both ways 41 us (4.1 TB/s of the 5.07 that a large copy reaches), rows alone 29 us; an fp32
// weight of 10576 x 2560 by tiles, both ways, 33 us (4.9 TB/s).
#include "block_device.hpp"
#include "block_host.hpp"

namespace ssd {

// A workgroup of 256 threads takes a tile of 128 x 128; thread t holds the patch of rows
// 8 (t / 16) .. + 8 and columns 8 (t % 16) .. + 8, so that 16 lanes read whole rows of the
// tile, and eight rows of a column are one 8-byte piece of the transposed form.  Held as it was
// read, a bf16 patch takes 32 registers and six waves fit a SIMD (widened: 64, four, 48 us for 42).
template <typename T, bool TILE>
__global__ void __launch_bounds__(256)
quant_tile_kernel(const T* __restrict__ x, Strides xs, unsigned char* __restrict__ q,
                  float* __restrict__ scale, unsigned char* __restrict__ qt,
                  float* __restrict__ scale_t, int64_t L, int64_t rows, int64_t C) {
  __shared__ float col_most[4][kBlock8];
  __shared__ __attribute__((aligned(16))) uint2 turned[kBlock8 * 16];
  const int64_t nc = (C + kBlock8 - 1) / kBlock8, nr = (rows + kBlock8 - 1) / kBlock8;
  const int64_t tr = blockIdx.x / nc, tc = blockIdx.x % nc;
  const int64_t r0 = tr * kBlock8, c0 = tc * kBlock8;
  const int t = threadIdx.x, pr = t / 16, pc = t % 16;
  const int64_t c = c0 + 8 * pc;
  const int n = c < C ? (int)(C - c < 8 ? C - c : 8) : 0;
  Raw8<T> v[8];   // in the registers of its own type, widened where it is used
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + 8 * pr + i;
    v[i] = Raw8<T>{};
    if (n > 0 && row < rows) v[i] = raw8(x + row_at(xs, row, L) + c, n);
  }
  auto row_of = [&](int i, float (&o)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = v[i][e];
  };
  float tile_most = 0.0f;
  if constexpr (TILE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float o[8];
      row_of(i, o);
      tile_most = fmaxf(tile_most, most_of(o));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) tile_most = fmaxf(tile_most, __shfl_xor(tile_most, off, kWave));
    if (t % kWave == 0) col_most[t / kWave][0] = tile_most;
    __syncthreads();
    tile_most = fmaxf(fmaxf(fmaxf(col_most[0][0], col_most[1][0]), fmaxf(col_most[2][0], col_most[3][0])), kLeast8);
    if (t == 0) {
      if (q) scale[tc * nr + tr] = tile_most / kMost8;
      if (qt) scale_t[tr * nc + tc] = tile_most / kMost8;
    }
  }
  if (q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = r0 + 8 * pr + i;
      float m = tile_most, o[8];
      row_of(i, o);
      if constexpr (!TILE) m = fmaxf(most_of_16(most_of(o)), kLeast8);
      if (row < rows) {
        *reinterpret_cast<uint2*>(q + row * nc * kBlock8 + c) = pack8<T>(o, m);
        if (!TILE && pc == 0) scale[tc * rows + row] = m / kMost8;
      }
    }
  }
  if (!qt) return;
  float most[8];
  if constexpr (!TILE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      most[e] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) most[e] = fmaxf(most[e], fabsf(v[i][e]));
      most[e] = fmaxf(most[e], __shfl_xor(most[e], 16, kWave));
      most[e] = fmaxf(most[e], __shfl_xor(most[e], 32, kWave));
    }
    if (t % kWave < 16)
#pragma unroll
      for (int e = 0; e < 8; ++e) col_most[t / kWave][8 * pc + e] = most[e];
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = 8 * pc + e;
    float m = tile_most;
    if constexpr (!TILE) {
      m = fmaxf(fmaxf(fmaxf(col_most[0][k], col_most[1][k]), fmaxf(col_most[2][k], col_most[3][k])), kLeast8);
      if (pr == 0 && e < n) scale_t[tr * C + c + e] = m / kMost8;
    }
    float col[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) col[i] = v[i][e];
    // Column k's 16 pieces lie in places permuted by pc = k / 8, so the 64 lanes of a write
    // touch every bank alike; the permutation keeps pairs of pieces together.
    turned[k * 16 + (pr ^ pc)] = pack8<T>(col, m);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = t / 8 + 32 * i, pair = t % 8, f = k / 8;
    if (c0 + k < C) {
      uint4 w = *reinterpret_cast<const uint4*>(&turned[k * 16 + ((2 * pair) ^ (f & ~1))]);
      if (f & 1) w = make_uint4(w.z, w.w, w.x, w.y);
      *reinterpret_cast<uint4*>(qt + (c0 + k) * nr * kBlock8 + r0 + 16 * pair) = w;
    }
  }
}

// Rows alone: 16 lanes per block of 128.
template <typename T>
__global__ void __launch_bounds__(256)
quant_rows_kernel(const T* __restrict__ x, Strides xs, unsigned char* __restrict__ q,
                  float* __restrict__ scale, int64_t L, int64_t rows, int64_t C) {
  const int64_t nc = (C + kBlock8 - 1) / kBlock8;
  const int64_t block = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
  const int64_t row = block / nc, b = block % nc;
  const int64_t c = b * kBlock8 + 8 * (threadIdx.x % 16);
  if (row >= rows) return;   // all 16 lanes alike
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  if (c < C) load8(x + row_at(xs, row, L) + c, (int)(C - c < 8 ? C - c : 8), v);
  const float m = fmaxf(most_of_16(most_of(v)), kLeast8);
  *reinterpret_cast<uint2*>(q + row * nc * kBlock8 + c) = pack8<T>(v, m);
  if (threadIdx.x % 16 == 0) scale[b * rows + row] = m / kMost8;
}

template <typename T>
static hipError_t quant8_t(const Quant8Args& a, hipStream_t stream) {
  const int64_t rows = a.batch * a.L;
  const int64_t nc = (a.C + kBlock8 - 1) / kBlock8, nr = (rows + kBlock8 - 1) / kBlock8;
  const Strides xs{a.xs[0], a.xs[1]};
  const T* x = static_cast<const T*>(a.x);
  if (!a.tile && !a.qt) {
    hipLaunchKernelGGL(quant_rows_kernel<T>, dim3((unsigned)((rows * nc + 15) / 16)), dim3(256), 0, stream,
                       x, xs, a.q, a.scale, a.L, rows, a.C);
  } else {
    const dim3 grid((unsigned)(nr * nc));
    if (a.tile)
      hipLaunchKernelGGL((quant_tile_kernel<T, true>), grid, dim3(256), 0, stream, x, xs, a.q, a.scale,
                         a.qt, a.scale_t, a.L, rows, a.C);
    else
      hipLaunchKernelGGL((quant_tile_kernel<T, false>), grid, dim3(256), 0, stream, x, xs, a.q, a.scale,
                         a.qt, a.scale_t, a.L, rows, a.C);
  }
  return hipGetLastError();
}

int quant8_grid_ok(int64_t rows, int64_t C) {
  const __int128 nc = (C + kBlock8 - 1) / kBlock8, nr = (rows + kBlock8 - 1) / kBlock8;
  return rows * nc * 16 + 256 < (int64_t(1) << 32) && nr * nc * 256 < (int64_t(1) << 32);
}

hipError_t launch_quant8(const Quant8Args& a, hipStream_t stream) {
  return a.bf16 ? quant8_t<bf16>(a, stream) : quant8_t<float>(a, stream);
}

}  // namespace ssd
