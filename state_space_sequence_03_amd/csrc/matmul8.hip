// matmul8.hip -- the matrix product of two e4m3 operands with fp32 scales for blocks of 128.
//
//     y[m, n] = sum_b xs[b, m] ws[b, n] p_b[m, n],   p_b = sum_{k in block b} x[m, k] w[n, k]
//
// A block of 128 is one v_mfma_f32_16x16x128_f8f6f4 step: p_b comes out of the matrix core in
// fp32 and is scaled into the sum by one fma per element.  The weight's rows are the A operand
// and x's rows the B operand, so lane l of a 16 x 16 tile holds row m = l % 16 of y and its
// columns n = 4 (l / 16) + 0..3: one scale of x per lane and tile, and stores of four
// consecutive columns.  The order of the 128 within a block is free as long as both operands
// have the same one.
//
// Many rows are bound by the matrix cores and, as closely, by LDS: a tile of 256 x 256 reads
// 192 KB and takes in 66 KB from memory for every 2048 cycles of products.  16384 x 10576 x 2560
// in bf16: 412 us, 2.15 PFLOP/s (without the stores 75 us less, without loads 70, without the
// scaling into the sums 45; a library's product of the same operands with one scale for all 392 us beside
// it; the card's best rate, at 8192 x 8192 x 8192, 2.84 PFLOP/s).  Tiles of 128 x 128: 16384 x 2560 x 5120
// in bf16 213 us, 2.02 PFLOP/s; 10576 x 2560 x 8192 by row in fp32 407 us, 1.09 PFLOP/s.  Few rows are bound by the
// weight's way from memory: one row, 10576 x 2560, 7.1 us, 3.8 TB/s.
#include <type_traits>

#include "block_device.hpp"
#include "block_host.hpp"
#include "matmul8_plan.hpp"

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

__device__ __forceinline__ intx8 frag8(const unsigned char* p, const unsigned char* q) {
  const intx4 a = *reinterpret_cast<const intx4*>(p), b = *reinterpret_cast<const intx4*>(q);
  return intx8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ intx8 frag8(const unsigned char* p) { return frag8(p, p + 16); }

// The tile of a workgroup.  Workgroups go to the eight XCDs in turn; each XCD takes a run of tiles of
// its own, eight tiles of rows at a time and column after column, so that the tiles that run together
// share their operands in its L2.
__device__ __forceinline__ void tile_of(int block, int mtiles, int ntiles, int* mt, int* nt) {
  const int tiles = mtiles * ntiles, each = tiles / 8, more = tiles % 8;
  const int xcd = block % 8;
  const int t = xcd * each + min(xcd, more) + block / 8;
  const int panel = t / (8 * ntiles), high = min(8, mtiles - 8 * panel);
  const int in = t - panel * 8 * ntiles;
  *mt = 8 * panel + in % high;
  *nt = in / high;
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
// eighth block of the depth straight from memory (lane l bytes 32 (l / 16) .. + 32 of a block of row
// l % 16), and add their sums through LDS in order.
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

// One block of both operands and their scales in LDS.
constexpr int matmul8_buffer(int BN, int BM) { return (BN + BM) * (kBlock8 + 4); }

// The tile of y in LDS: bytes from row to row of a wave's part, and all of the workgroup's LDS.
constexpr int matmul8_row(int NT, int size) { return 16 * NT * size + 16; }
constexpr int matmul8_lds(int NT, int MT, int WN, int WM, int size) {
  const int loop = 2 * matmul8_buffer(16 * NT * WN, 16 * MT * WM), out = WN * WM * 16 * MT * matmul8_row(NT, size);
  return loop > out ? loop : out;
}

// Many rows: a workgroup takes BN = 16 NT WN columns x BM = 16 MT WM rows of y, a wave 16 NT x 16 MT
// of them.  Blocks of both operands go straight from memory into two LDS buffers, one block ahead;
// 16-byte piece c of row r lies in place c ^ (r % 8) of the row, so that the sixteen rows of an
// operand read spread over the banks (the permutation is made by the lanes' source addresses).
// Products as for results of type O; y has the type Y, O or (where the depth is split between gridDim.y
// workgroups, `each` blocks to one) fp32: then each leaves its sums [M, N] behind the last one's.
template <typename O, typename Y, int NT, int MT, int WN, int WM, bool TILE>
__global__ void __launch_bounds__(kWave * WN * WM, 2)
matmul8_kernel(const unsigned char* __restrict__ x, const float* __restrict__ xs,
               const unsigned char* __restrict__ w, const float* __restrict__ ws,
               Y* __restrict__ y, int M, int N, int K, int mtiles, int ntiles, int each) {
  constexpr int kWaves = WN * WM, BN = 16 * NT * WN, BM = 16 * MT * WM;
  // 8-row pieces of each half of a wave's columns, and of the rows, that one wave loads
  constexpr int kHalfN = NT / WM, kPiecesM = 2 * MT / WN;
  constexpr int kBuffer = matmul8_buffer(BN, BM);
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wn = wave % WN, wm = wave / WN;
  int mt, nt;
  tile_of(blockIdx.x, mtiles, ntiles, &mt, &nt);
  const int n0 = nt * BN, m0 = mt * BM;
  const int b0 = blockIdx.y * each, blocks = min(each, K / kBlock8 - b0);   // the first block, and how many
  y += (int64_t)blockIdx.y * M * N;
  // Source offsets from the tile's first row, of this lane in a piece's first row and in the last
  // row of the operand: rows past the end read that one, and are not stored.
  const int c0 = 16 * ((lane % 8) ^ (lane / 8));
  const uint32_t from = (uint32_t)(lane / 8) * (uint32_t)K + c0;
  auto last_of = [&](int rows) {
    const uint64_t at = (uint64_t)(rows - 1) * (uint32_t)K + c0;
    return at < UINT32_MAX ? (uint32_t)at : UINT32_MAX;
  };
  const uint32_t last_n = last_of(N - n0), last_m = last_of(M - m0);
  const unsigned char* wb = w + (int64_t)n0 * K + (int64_t)b0 * kBlock8;
  const unsigned char* xb = x + (int64_t)m0 * K + (int64_t)b0 * kBlock8;
  auto rows8 = [&](const unsigned char* base, uint32_t last, int piece, unsigned char* to) {
    dma16_so(base, min(from + (uint32_t)(8 * piece) * (uint32_t)K, last), to + piece * 1024);
  };
  // Each wave's columns fall into a lower and an upper half.  The i-th piece of one, of this wave's:
  auto load_half = [&](int b, int half, int i) {
    const int l = wave + kWaves * i;
    rows8(wb + min(b, blocks - 1) * kBlock8, last_n, l / NT * 2 * NT + half * NT + l % NT, lds + (b % 2) * kBuffer);
  };
  // The scales of a block, 64 by each wave (more than once where there are more waves than that).
  const int wtiles = (N + kBlock8 - 1) / kBlock8;
  constexpr int kScaleParts = BM / 64 + (TILE ? 1 : BN / 64);
  const int spart = wave % kScaleParts;
  const bool for_m = spart < BM / 64;
  const float* sbase = for_m ? xs + m0 : TILE ? ws + n0 / kBlock8 : ws + n0;
  const int64_t srow = for_m ? M : TILE ? wtiles : N;
  sbase += b0 * srow;
  const int sleft = (int)(for_m ? M - m0 : TILE ? wtiles - n0 / kBlock8 : N - n0);
  const uint32_t sat = 4 * min(64 * (for_m ? spart : spart - BM / 64) + lane, sleft - 1);
  // The rows of x, the scales and the lower half: the i-th of kFirst loads.
  constexpr int kFirst = kPiecesM + 1 + kHalfN;
  auto load_first = [&](int b, int i) {
    unsigned char* to = lds + (b % 2) * kBuffer;
    if (i < kPiecesM)
      rows8(xb + min(b, blocks - 1) * kBlock8, last_m, wave + kWaves * i, to + BN * kBlock8);
    else if (i == kPiecesM)
      dma4_so(sbase + min(b, blocks - 1) * srow, sat, to + (BN + BM) * kBlock8 + 256 * spart);
    else
      load_half(b, 0, i - kPiecesM - 1);
  };
  // Waits until every wave's loads but those of the latest `kAhead` have arrived, and its LDS reads are done.
  constexpr int kAhead = kFirst + kHalfN;
  auto arrived = [&](floatx4& behind) {   // behind the work that gives `behind`
    asm volatile("s_waitcnt vmcnt(%1) lgkmcnt(0)" : "+v"(behind) : "n"(kAhead) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const int row = lane % 16, part = lane / 16;
  const int nbase = n0 + 16 * NT * wn;
  floatx4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int first = row * kBlock8 + 16 * (part ^ (row % 8));   // of the two 16-byte pieces; the other is 64 bytes across
  auto read_n = [&](int b, int i) {
    const unsigned char* p = lds + (b % 2) * kBuffer + (NT * wn + i) * 2048;
    return frag8(p + first, p + (first ^ 64));
  };
  auto read_m = [&](int b, int j) {
    const unsigned char* p = lds + (b % 2) * kBuffer + BN * kBlock8 + (MT * wm + j) * 2048;
    return frag8(p + first, p + (first ^ 64));
  };
  float by[MT];
  floatx4 sw[TILE ? 1 : NT];
  auto read_scales = [&](int b) {
    const float* s = reinterpret_cast<const float*>(lds + (b % 2) * kBuffer + (BN + BM) * kBlock8);
#pragma unroll
    for (int j = 0; j < MT; ++j) by[j] = s[16 * (MT * wm + j) + row];
    if constexpr (TILE) {
      const float one = s[BM + 16 * NT * wn / kBlock8];
#pragma unroll
      for (int j = 0; j < MT; ++j) by[j] *= one;
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i) sw[i] = *reinterpret_cast<const floatx4*>(s + BM + 16 * (NT * wn + i) + 4 * part);
    }
  };
  typedef typename Frag8<O>::type Frag;
  // 8-bit operands are read into the registers that products take them from; operands to be
  // widened wait as they are.
  constexpr bool kWide = !std::is_same<Frag, intx8>::value;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
#pragma unroll
    for (int i = 0; i < kFirst; ++i) load_first(b, i);
#pragma unroll
    for (int i = 0; i < (b == 0 ? kHalfN : 1); ++i) load_half(b, 1, i);
  }
  arrived(acc[0][0]);
  intx8 an = read_n(0, 0), cn[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) cn[j] = read_m(0, j);
  read_scales(0);
  // The operands of a block's first products are in registers when it begins; products are scaled into
  // the sums kLag products later, so that neither the matrix core nor the vector ALU waits for the other.
  // What the second half of a block's products needs is waited for in front of that half's first read,
  // what the next block begins with in front of the last products, and is read while they run.  Behind
  // each of the two waits every wave is done with a part of this block's buffer, and the same part of the
  // block after the next is loaded there: each load has one and a half blocks' time.  Past the last
  // block the last one is loaded again, which keeps the counts of the waits the same and branches out of
  // the loop (sums in front of a branch would move behind it), and what is read is not used.
  constexpr int kLag = 2;
  for (int b = 0; b < blocks; ++b) {
    Frag c[kWide ? MT : 1], a;
    if constexpr (kWide)
#pragma unroll
      for (int j = 0; j < MT; ++j) c[j] = Frag8<O>::of(cn[j]);
    floatx4 p[kLag + 1];
    auto add = [&](int t) {
      const int i = t / MT, j = t % MT;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[i][j][r] = fmaf(p[t % (kLag + 1)][r], TILE ? by[j] : by[j] * sw[TILE ? 0 : i][r], acc[i][j][r]);
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      a = Frag8<O>::of(an);
      if (i + 1 == NT / 2) arrived(acc[NT / 2 > 2 ? NT / 2 - 2 : 0][0]);
      if (i + 1 == NT) arrived(acc[NT - 2][0]);
      an = i + 1 < NT ? read_n(b, i + 1) : read_n(b + 1, 0);
      // loads, a few between any two reads: many in a row would hold the wave up
      if (i + 1 >= NT / 2 && i + 1 < NT) {
        constexpr int kEach = (kFirst + NT / 2 - 1) / (NT / 2);
        const int g = i + 1 - NT / 2;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          if (g * kEach + k < kFirst) load_first(b + 2, g * kEach + k);
      } else if (i + 1 < kHalfN) {
        load_half(b + 1, 1, i + 1);
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int t = i * MT + j;
        if constexpr (kWide) p[t % (kLag + 1)] = mma8(a, c[j]);
        else p[t % (kLag + 1)] = mma8(a, cn[j]);
        if (i + 1 == NT) cn[j] = read_m(b + 1, j);
        if (t >= kLag) add(t - kLag);
      }
    }
#pragma unroll
    for (int t = NT * MT - kLag; t < NT * MT; ++t) add(t);
    read_scales(b + 1);
    load_half(b + 2, 1, 0);
    // the order of the above, which the scheduler is held to: reads, one product, the sums of an earlier one
    constexpr int kSums = (TILE ? 4 : 8) + (kWide ? 16 / MT : 0);
#pragma unroll
    for (int t = 0; t < NT * MT; ++t) {
      if (t % MT == 0) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kWide ? 4 : 1, 0);
      if (t / MT + 1 == NT) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      if (t >= kLag) __builtin_amdgcn_sched_group_barrier(0x002, kSums, 0);
    }
  }
  // The tile of y goes through LDS, so that whole rows of a wave's columns are stored: 16 bytes a lane,
  // 256 in a row.  Rows lie 16 bytes further apart than they are long, and their pieces in all banks.
  // The largest tiles, taken for large y alone, are stored past the caches (16384 x 10576 x 2560: 417 us in
  // place of 448).
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();   // no load is on its way to LDS, and nothing is read from it any more
  asm volatile("" ::: "memory");
  constexpr int kRow = matmul8_row(NT, sizeof(Y)), kEach = 16 / sizeof(Y), kLanes = 16 * NT / kEach;
  unsigned char* mine = lds + wave * (16 * MT * kRow);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
      store_cols(reinterpret_cast<Y*>(mine + (16 * j + row) * kRow) + 16 * i + 4 * part, 4, acc[i][j]);
  wave_sync();
  const int n = nbase + lane % kLanes * kEach;
#pragma unroll
  for (int r = 0; r < 16 * MT; r += kWave / kLanes) {
    const int at = r + lane / kLanes, m = m0 + 16 * MT * wm + at;
    const Y* from_lds = reinterpret_cast<const Y*>(mine + at * kRow) + lane % kLanes * kEach;
    if (m < M && n < N) {
      Y* to = y + (int64_t)m * N + n;
      typedef Y Piece __attribute__((ext_vector_type(16 / sizeof(Y))));
      typedef Y PieceAny __attribute__((ext_vector_type(16 / sizeof(Y)), aligned(sizeof(Y))));
      const Piece v = *reinterpret_cast<const Piece*>(from_lds);
      if (n + kEach <= N) {
        if constexpr (NT * MT > 16) __builtin_nontemporal_store(v, reinterpret_cast<PieceAny*>(to));
        else *reinterpret_cast<PieceAny*>(to) = v;
      } else {
#pragma unroll
        for (int e = 0; e < kEach; ++e)
          if (n + e < N) to[e] = v[e];
      }
    }
  }
}

// The sums of the parts of a split depth, in order.
template <typename O>
__global__ void __launch_bounds__(256)
matmul8_join_kernel(const float* __restrict__ part, int parts, int64_t n, O* __restrict__ y) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const int left = (int)(n - i < 4 ? n - i : 4);
  floatx4 s = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float* q = part + p * n + i;
    if (left == 4) {
      s += *reinterpret_cast<const floatx4_any*>(q);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) s[e] += q[e];
    }
  }
  store_cols(y + i, left, s);
}

// ---- host ----

size_t matmul8_workspace(int64_t M, int64_t N, int64_t K, int out_bf16) {
  const Matmul8Plan p = matmul8_plan(M, N, K, out_bf16);
  return p.parts > 1 ? size_t(p.parts) * M * N * sizeof(float) : 0;
}

// Fewer than 2^32 threads along the first axis of the plan's launch: 512 for 16 columns x 16 rows (of more than 16 rows,
// 16 x 32) or 256 x 256, 256 for 64 x 64 or 128 x 128.  (The parts of a depth lie along the second, and what joins
// them has fewer.)
int matmul8_grid_ok(int64_t M, int64_t N, int64_t K, int out_bf16) {
  const Matmul8Form form = matmul8_plan(M, N, K, out_bf16).form;
  const int64_t side = form == kTile64 ? 64 : form == kTile128 ? 128 : 256;
  const __int128 groups = form == kFew ? (__int128)((N + 15) / 16) : (__int128)((N + side - 1) / side) * ((M + side - 1) / side);
  return groups * (form == kFew || form == kTile256 ? 512 : 256) < (int64_t(1) << 32);
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

template <typename O, typename Y, int NT, int MT, int WN, int WM, bool TILE>
static hipError_t tiles(const Matmul8Args& a, const Matmul8Plan& p, Y* y, hipStream_t stream) {
  constexpr int kLds = matmul8_lds(NT, MT, WN, WM, sizeof(Y));
  constexpr auto kernel = matmul8_kernel<O, Y, NT, MT, WN, WM, TILE>;
  const hipError_t e = ensure_dyn_lds<kernel>(kLds);
  if (e != hipSuccess) return e;
  const int mtiles = (int)((a.M + 16 * MT * WM - 1) / (16 * MT * WM)), ntiles = (int)((a.N + 16 * NT * WN - 1) / (16 * NT * WN));
  hipLaunchKernelGGL(kernel, dim3((unsigned)(mtiles * ntiles), (unsigned)p.parts), dim3(kWave * WN * WM), kLds, stream,
                     a.x, a.xs, a.w, a.ws, y, (int)a.M, (int)a.N, (int)a.K, mtiles, ntiles, p.each);
  return hipGetLastError();
}

template <typename O, bool TILE>
static hipError_t matmul8_o(const Matmul8Args& a, hipStream_t stream) {
  const Matmul8Plan p = matmul8_plan(a.M, a.N, a.K, a.out_bf16);
  O* y = static_cast<O*>(a.y);
  if (p.form == kFew) return a.M <= 16 ? few<O, 1, 1>(a, stream) : few<O, 1, 2>(a, stream);
  if constexpr (sizeof(O) == 2)
    if (p.form == kTile256) return tiles<O, O, 8, 4, 2, 4, TILE>(a, p, y, stream);
  if (p.parts == 1)
    return p.form == kTile128 ? tiles<O, O, 4, 4, 2, 2, TILE>(a, p, y, stream) : tiles<O, O, 2, 2, 2, 2, TILE>(a, p, y, stream);
  float* part = static_cast<float*>(a.workspace);
  const hipError_t e = p.form == kTile128 ? tiles<O, float, 4, 4, 2, 2, TILE>(a, p, part, stream)
                                          : tiles<O, float, 2, 2, 2, 2, TILE>(a, p, part, stream);
  if (e != hipSuccess) return e;
  const int64_t n = a.M * a.N;
  hipLaunchKernelGGL(matmul8_join_kernel<O>, dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0, stream, part, p.parts, n, y);
  return hipGetLastError();
}

hipError_t launch_matmul8(const Matmul8Args& a, hipStream_t stream) {
  if (a.out_bf16) return a.tile ? matmul8_o<bf16, true>(a, stream) : matmul8_o<bf16, false>(a, stream);
  return a.tile ? matmul8_o<float, true>(a, stream) : matmul8_o<float, false>(a, stream);
}

}  // namespace ssd
