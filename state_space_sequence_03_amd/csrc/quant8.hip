// quant8.hip -- a matrix in e4m3 with a scale for each block: by rows, transposed, or both
// from one read.
//
// For a block with magnitudes up to a:  m = max(a, 2^-100), q = e4m3(v (448 / m)) to nearest
// even, scale = m / 448.  A block is 128 elements of a row (of a column, for the transposed
// form), or a tile of 128 x 128 that both forms share.
//
// Bound by HBM: each element is read once and written once or twice as a byte.  2 x 4096 x 5120
// bf16 both ways 39 us (4.3 TB/s of the 5.07 that a large copy reaches), rows alone 27 us; an fp32
// weight of 10576 x 2560 by tiles, both ways, 33 us (4.9 TB/s).
#include "block_device.hpp"
#include "block_host.hpp"

namespace ssd {

// The magnitudes of eight elements, as the bits of their type: pairs of bf16 or single fp32 values, which
// integer maxima compare, two bf16 at once.  `clean`: NaN, above infinity in that order, as 0 (from a copy that
// the compiler cannot tell for one: words kept from the first look at them took 32 to 50 registers more).
template <typename T> struct Bits8;
template <> struct Bits8<bf16> {
  static constexpr int kWords = 4;
  static constexpr uint32_t kInf = 0x7f80;
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
  }
  static __device__ __forceinline__ uint32_t word(const Raw8<bf16>& v, int k, bool clean) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    uint32_t w = __builtin_bit_cast(u32x4, v.v)[k];
    if (clean) asm("" : "+v"(w));
    w &= 0x7fff7fffu;
    if (clean) w = ((w & 0xffff) > kInf ? 0 : w & 0xffff) | ((w >> 16) > kInf ? 0 : w & 0xffff0000u);
    return w;
  }
  static __device__ __forceinline__ uint32_t one(uint32_t w) { return max(w & 0xffff, w >> 16); }
  static __device__ __forceinline__ float value(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
  static __device__ __forceinline__ float of(const uint32_t (&w)[4], int e) {
    return __builtin_bit_cast(float, e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
};
template <> struct Bits8<float> {
  static constexpr int kWords = 8;
  static constexpr uint32_t kInf = 0x7f800000;
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t word(const Raw8<float>& v, int k, bool clean) {
    uint32_t w = __builtin_bit_cast(uint32_t, v[k]);
    if (clean) asm("" : "+v"(w));
    w &= 0x7fffffffu;
    return clean && w > kInf ? 0 : w;
  }
  static __device__ __forceinline__ uint32_t one(uint32_t w) { return w; }
  static __device__ __forceinline__ float value(uint32_t w) { return __builtin_bit_cast(float, w); }
  static __device__ __forceinline__ float of(const uint32_t (&w)[8], int e) { return value(w[e]); }
};

// A workgroup of 256 threads takes a tile of 128 x 128; thread t holds the patch of rows
// 8 (t / 16) .. + 8 and columns 8 (t % 16) .. + 8, so that 16 lanes read whole rows of the
// tile, and eight rows of a column are one 8-byte piece of the transposed form.  Held as it was
// read, a bf16 patch takes 32 registers and eight waves fit a SIMD (widened, an earlier form had four, 48 us for 42).
// The vector ALU is busy for half of the time that the memory takes, so whatever belongs to a row or a column
// (a scale, a column's inverse) is computed once, magnitudes are compared as integers, and addresses are counted
// on from row to row: 39 us in place of 41.  Stores past the caches took 37, and the product that reads them 6 more.
template <typename T, bool TILE>
__global__ void __launch_bounds__(256)
quant_tile_kernel(const T* __restrict__ x, Strides xs, unsigned char* __restrict__ q,
                  float* __restrict__ scale, unsigned char* __restrict__ qt,
                  float* __restrict__ scale_t, int64_t L, int64_t rows, int64_t C) {
  typedef Bits8<T> Bits;
  __shared__ __attribute__((aligned(16))) float col_most[4][kBlock8];
  __shared__ __attribute__((aligned(16))) Inverse8 col_by[kBlock8];
  __shared__ __attribute__((aligned(16))) uint2 turned[kBlock8 * 16];
  const int64_t nc = (C + kBlock8 - 1) / kBlock8, nr = (rows + kBlock8 - 1) / kBlock8;
  const uint32_t tr = blockIdx.x / (uint32_t)nc, tc = blockIdx.x - tr * (uint32_t)nc;   // fewer than 2^24 tiles
  const int64_t r0 = (int64_t)tr * kBlock8, c0 = (int64_t)tc * kBlock8;
  const int t = threadIdx.x, pr = t / 16, pc = t % 16;
  const int64_t c = c0 + 8 * pc;
  const int n = c < C ? (int)(C - c < 8 ? C - c : 8) : 0;
  const int high = rows - r0 < kBlock8 ? (int)(rows - r0) - 8 * pr : 8;   // rows of the patch
  Raw8<T> v[8];   // in the registers of its own type, widened where it is used
  {
    const int64_t row = r0 + 8 * pr < rows ? r0 + 8 * pr : rows - 1;
    const uint32_t b = (uint32_t)row / (uint32_t)L;
    int64_t left = L - (row - (int64_t)b * L);   // tokens to the end of the sequence
    const T* p = x + (int64_t)b * xs.batch + (L - left) * xs.token + c;
    const int64_t next = xs.batch - (L - 1) * xs.token;   // from a sequence's last token to the next one's first
    const bool whole = n == 8 && left >= 8 && high >= 8;
    if (whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = raw8(p + i * xs.token, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = Raw8<T>{};
        if (n > 0 && i < high) v[i] = raw8(p, n);
        const bool end = --left == 0;
        p += end ? next : xs.token;
        if (end) left = L;
      }
    }
  }
  uint32_t row_bits[8], col_bits[Bits::kWords];
  auto magnitudes = [&](bool clean) {
    uint32_t all = 0;
#pragma unroll
    for (int k = 0; k < Bits::kWords; ++k) col_bits[k] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t w = 0;
#pragma unroll
      for (int k = 0; k < Bits::kWords; ++k) {
        const uint32_t a = Bits::word(v[i], k, clean);
        w = Bits::most(w, a);
        col_bits[k] = Bits::most(col_bits[k], a);
      }
      row_bits[i] = Bits::one(w);
      all = max(all, row_bits[i]);
    }
    return all;
  };
  uint32_t all = magnitudes(false);
  if (all > Bits::kInf) all = magnitudes(true);
  Inverse8 tile_by;
  if constexpr (TILE) {
    float most = Bits::value(all);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, kWave));
    if (t % kWave == 0) col_most[t / kWave][0] = most;
    __syncthreads();
    most = fmaxf(fmaxf(fmaxf(col_most[0][0], col_most[1][0]), fmaxf(col_most[2][0], col_most[3][0])), kLeast8);
    tile_by = inverse8(most);
    if (t == 0) {
      if (q) scale[tc * nr + tr] = scale_of(most);
      if (qt) scale_t[tr * nc + tc] = scale_of(most);
    }
  }
  if (q) {
    const int64_t pitch = nc * kBlock8;
    unsigned char* to = q + (r0 + 8 * pr) * pitch + c;
    float mine = 0.0f;   // lane pc keeps the magnitude of row pc
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = v[i][e];
      Inverse8 by = tile_by;
      if constexpr (!TILE) {
        const float m = fmaxf(Bits::value(most_of_16(row_bits[i])), kLeast8);
        by = inverse8(m);
        mine = pc == i ? m : mine;
      }
      if (i < high) *reinterpret_cast<uint2*>(to) = pack8(o, by);
      to += pitch;
    }
    if (!TILE && pc < 8 && pc < high) scale[tc * rows + r0 + 8 * pr + pc] = scale_of(mine);
  }
  if (!qt) return;
  if constexpr (!TILE) {
    // Over a wave's four patches of a column: 32 lanes across, then 16.
#pragma unroll
    for (int k = 0; k < Bits::kWords; ++k) {
      uint32_t w = col_bits[k];
      const auto a = __builtin_amdgcn_permlane32_swap(w, w, false, false);
      w = Bits::most(a[0], a[1]);
      const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
      col_bits[k] = Bits::most(b[0], b[1]);
    }
    if (t % kWave < 16) {
#pragma unroll
      for (int e = 0; e < 8; ++e) col_most[t / kWave][8 * pc + e] = Bits::of(col_bits, e);
    }
    __syncthreads();
    if (t < kBlock8) {
      const float m = fmaxf(fmaxf(fmaxf(col_most[0][t], col_most[1][t]), fmaxf(col_most[2][t], col_most[3][t])), kLeast8);
      col_by[t] = inverse8(m);
      if (c0 + t < C) scale_t[tr * C + c0 + t] = scale_of(m);
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = 8 * pc + e;
    float col[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) col[i] = v[i][e];
    // Column k's 16 pieces lie in places permuted by pc = k / 8, so the 64 lanes of a write
    // touch every bank alike; the permutation keeps pairs of pieces together.
    turned[k * 16 + (pr ^ pc)] = pack8(col, TILE ? tile_by : col_by[k]);
  }
  __syncthreads();
  unsigned char* to = qt + (c0 + t / 8) * nr * kBlock8 + r0 + 16 * (t % 8);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = t / 8 + 32 * i, pair = t % 8, f = k / 8;
    if (c0 + k < C) {
      uint4 w = *reinterpret_cast<const uint4*>(&turned[k * 16 + ((2 * pair) ^ (f & ~1))]);
      if (f & 1) w = make_uint4(w.z, w.w, w.x, w.y);
      *reinterpret_cast<uint4*>(to) = w;
    }
    to += 32 * nr * kBlock8;
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
  *reinterpret_cast<uint2*>(q + row * nc * kBlock8 + c) = pack8(v, m);
  if (threadIdx.x % 16 == 0) scale[b * rows + row] = scale_of(m);
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

// Fewer than 2^32 threads in the launch that quant8_t makes: 16 for each block of a row, or 256 for each tile.
int quant8_grid_ok(int64_t rows, int64_t C, int tile, int transposed) {
  const __int128 nc = (C + kBlock8 - 1) / kBlock8, nr = (rows + kBlock8 - 1) / kBlock8;
  return (!tile && !transposed ? rows * nc * 16 + 256 : nr * nc * 256) < (int64_t(1) << 32);
}

hipError_t launch_quant8(const Quant8Args& a, hipStream_t stream) {
  return a.bf16 ? quant8_t<bf16>(a, stream) : quant8_t<float>(a, stream);
}

}  // namespace ssd
