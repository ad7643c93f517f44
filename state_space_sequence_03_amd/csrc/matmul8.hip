// matmul8.hip -- the matrix product of two e4m3 operands with fp32 scales for blocks of 128.
//
//     y[m, n] = sum_b xs[b, m] ws[b, n] p_b[m, n],   p_b = sum_{k in block b} x[m, k] w[n, k]
//
// A block of 128 is one v_mfma_f32_16x16x128_f8f6f4 step: p_b comes out of the matrix core in
// fp32 and is scaled into the sum by one fma per element.  The weight's rows are the A operand
// and x's rows the B operand, so lane l of a 16 x 16 tile holds row m = l % 16 of y and its
// columns n = 4 (l / 16) + 0..3: one scale of x per lane and tile, and stores of four
// consecutive columns.  Lane l supplies bytes 32 (l / 16) .. + 32 of a block of row l % 16.
#include "block_device.hpp"
#include "block_host.hpp"

namespace ssd {

typedef int intx8 __attribute__((ext_vector_type(8)));
typedef int intx4 __attribute__((ext_vector_type(4)));

// p = sum over one block of 128, from zero (operand formats e4m3, no scales).
__device__ __forceinline__ floatx4 mma8(intx8 a, intx8 b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, floatx4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// The same with fp32 accuracy.  The 8-bit matrix instructions, of either shape, add the products
// of a step with about 16 bits (relative error 1.5e-5 of the result's size over 128 products,
// measured against 64 bits), far below the rounding of a bf16 result and far above that of an
// fp32 one.  Every e4m3 value is a bf16 value, and the bf16 instructions add to 9e-9, at half the
// rate: results in fp32 take them.
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
struct Wide8 {
  bf16x8 v[4];
};
__device__ __forceinline__ Wide8 widen8(intx8 a) {
  Wide8 w;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[i], 1.0f, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[i], 1.0f, true);
    w.v[i / 2][4 * (i % 2)] = lo[0];
    w.v[i / 2][4 * (i % 2) + 1] = lo[1];
    w.v[i / 2][4 * (i % 2) + 2] = hi[0];
    w.v[i / 2][4 * (i % 2) + 3] = hi[1];
  }
  return w;
}
__device__ __forceinline__ floatx4 mma8(const Wide8& a, const Wide8& b) {
  floatx4 p = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], p, 0, 0, 0);
  return p;
}
// Operands of one kind or the other, by the type of the result.
template <typename O> struct Frag8 {
  typedef intx8 type;
  static __device__ __forceinline__ intx8 of(intx8 a) { return a; }
};
template <> struct Frag8<float> {
  typedef Wide8 type;
  static __device__ __forceinline__ Wide8 of(intx8 a) { return widen8(a); }
};

__device__ __forceinline__ intx8 frag8(const unsigned char* p) {
  const intx4 a = *reinterpret_cast<const intx4*>(p), b = *reinterpret_cast<const intx4*>(p + 16);
  return intx8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Four consecutive columns of a row of y, the first `n` of them.
__device__ __forceinline__ void store_cols(bf16* p, int n, floatx4 v) {
  typedef bf16 bf16x4_any __attribute__((ext_vector_type(4), aligned(2)));
  if (n >= 4) {
    *reinterpret_cast<bf16x4_any*>(p) = bf16x4_any{static_cast<bf16>(v[0]), static_cast<bf16>(v[1]),
                                                   static_cast<bf16>(v[2]), static_cast<bf16>(v[3])};
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < n) p[r] = static_cast<bf16>(v[r]);
  }
}
__device__ __forceinline__ void store_cols(float* p, int n, floatx4 v) {
  if (n >= 4) {
    *reinterpret_cast<floatx4_any*>(p) = floatx4_any{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < n) p[r] = v[r];
  }
}

// Few rows: a workgroup of eight waves takes 16 NT columns x 16 MT rows; its waves take every
// eighth block of the depth straight from memory, and add their sums through LDS in order.
template <typename O, int NT, int MT, bool TILE>
__global__ void __launch_bounds__(512)
matmul8_few_kernel(const unsigned char* __restrict__ x, const float* __restrict__ xs,
                   const unsigned char* __restrict__ w, const float* __restrict__ ws,
                   O* __restrict__ y, int M, int N, int K, int mtiles) {
  __shared__ floatx4 sums[7][NT * MT][kWave];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int n0 = blockIdx.x / mtiles * (16 * NT), m0 = blockIdx.x % mtiles * (16 * MT);
  const int blocks = K / kBlock8;
  floatx4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const unsigned char *wp[NT], *xp[MT];   // rows past the end read the last one, and are not stored
  int mrow[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i) wp[i] = w + (int64_t)min(n0 + 16 * i + lane % 16, N - 1) * K + 32 * (lane / 16);
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    mrow[j] = min(m0 + 16 * j + lane % 16, M - 1);
    xp[j] = x + (int64_t)mrow[j] * K + 32 * (lane / 16);
  }
  const int wtiles = (N + kBlock8 - 1) / kBlock8;
  for (int b = wave; b < blocks; b += 8) {
    typename Frag8<O>::type a[NT], c[MT];
    float sx[MT], sw[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      a[i] = Frag8<O>::of(frag8(wp[i] + (int64_t)b * kBlock8));
#pragma unroll
      for (int r = 0; r < 4; ++r)
        sw[i][r] = TILE ? ws[(int64_t)b * wtiles + min(n0 + 16 * i, N - 1) / kBlock8]
                        : ws[(int64_t)b * N + min(n0 + 16 * i + 4 * (lane / 16) + r, N - 1)];
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      c[j] = Frag8<O>::of(frag8(xp[j] + (int64_t)b * kBlock8));
      sx[j] = xs[(int64_t)b * M + mrow[j]];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const floatx4 p = mma8(a[i], c[j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(p[r], sx[j] * sw[i][r], acc[i][j][r]);
      }
  }
  if (wave > 0)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) sums[wave - 1][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      for (int v = 0; v < 7; ++v) acc[i][j] += sums[v][i * MT + j][lane];
      const int m = m0 + 16 * j + lane % 16, n = n0 + 16 * i + 4 * (lane / 16);
      if (m < M && n < N) store_cols(y + (int64_t)m * N + n, N - n, acc[i][j]);
    }
}

// ---- host ----

size_t matmul8_workspace(int64_t M, int64_t N, int64_t K) {
  (void)M; (void)N; (void)K;
  return 0;
}

// The smallest tiles, 32 columns by 16 rows, of 512 threads.
int matmul8_grid_ok(int64_t M, int64_t N) {
  return (__int128)((N + 31) / 32) * ((M + 15) / 16) * 512 < (int64_t(1) << 32);
}

template <typename O, int NT, int MT>
static hipError_t few(const Matmul8Args& a, hipStream_t stream) {
  const int mtiles = (int)((a.M + 16 * MT - 1) / (16 * MT));
  const dim3 grid((unsigned)((a.N + 16 * NT - 1) / (16 * NT) * mtiles));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(512), 0, stream, a.x, a.xs, a.w, a.ws, static_cast<O*>(a.y),
                       (int)a.M, (int)a.N, (int)a.K, mtiles);
  };
  if (a.tile) go(matmul8_few_kernel<O, NT, MT, true>);
  else go(matmul8_few_kernel<O, NT, MT, false>);
  return hipGetLastError();
}

template <typename O>
static hipError_t matmul8_o(const Matmul8Args& a, hipStream_t stream) {
  if (a.M <= 16) return few<O, 2, 1>(a, stream);
  return few<O, 2, 4>(a, stream);
}

hipError_t launch_matmul8(const Matmul8Args& a, hipStream_t stream) {
  return a.out_bf16 ? matmul8_o<bf16>(a, stream) : matmul8_o<float>(a, stream);
}

}  // namespace ssd
