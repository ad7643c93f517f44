// add_norm.hip -- the residual addition with the RMS norm in front of a layer, its
// gradients, and the gated norm behind the layer with its output in 8 bits.
//
// Over the C channels of a token:  h = x + residual, rounded to the residual's type;
// r = (mean(h^2) + eps)^(-1/2);  y = w h r.  In 8 bits, per block of 128 channels:
// m = max |y|, q = e4m3(y 448 / m), scale = m / 448, with no rounding of y between.
// Gated, in each of G groups, with s(z) = z sigmoid(z):  u = x s(z) or x,  y = w u r or
// w u r s(z).
// Gradients, with n = h r and t = w dy:  dh' = dh + r (t - n mean(t n)),  dw = sum over
// tokens of dy n;  mean(t n) = r mean(t h), so one reduction gives both sums.
//
// Bound by HBM: every input is read once, a token's elements stay in registers between
// the sum and the outputs, in pieces of eight channels, NV per thread.  The gates (an exp2
// and a reciprocal per element, quarter rate) keep the vector ALU busy beside it.
// bf16 with an fp32 residual, 2 x 8192 x 2560 to 8 bits 86 us (5.4 TB/s; a large copy, half of
// which is written, 5.07), gradients over 2 x 4096 65 us (5.1 TB/s, 5 of them part sums); gated
// norm of 2 x 8192 x 5120 to 8 bits 90 us (4.7 TB/s), of 2 groups of 128 24 us (0.9 TB/s: see item_grid).
#include "block_device.hpp"
#include "block_host.hpp"

namespace ssd {

enum NormForm { kAdd = 0, kGateFirst = 1, kNormFirst = 2 };

// A workgroup takes `each` tokens in a row: blockDim.x / tg of them at a time, or, with several groups,
// as many groups of one (blockIdx.y tells which).  The next token's elements are loaded while this one's
// are worked on, and the weights stay in registers.
template <typename T, typename R, int NV, int FORM>
__global__ void __launch_bounds__(512)
block_norm_kernel(const T* __restrict__ x, Strides xs, const R* r, Strides zs,
                  const float* __restrict__ w, R* h, T* __restrict__ y,
                  unsigned char* __restrict__ q, float* __restrict__ scale, int64_t L, int64_t rows,
                  int C, int G, float eps, int tg, int each) {
  __shared__ float lds[8];
  const int S = C / G;
  const int slot = threadIdx.x / tg, slots = blockDim.x / tg, lane = threadIdx.x % tg;
  const int grp = G == 1 ? 0 : blockIdx.y * slots + slot, step = G == 1 ? slots : 1;
  const int c0 = grp * S;
  const int64_t first = (int64_t)blockIdx.x * each;
  const int64_t last = grp < G ? (first + each < rows ? first + each : rows) : 0;
  const int64_t P = (int64_t)(C + kBlock8 - 1) / kBlock8 * kBlock8;
  const int padded = (S + kBlock8 - 1) / kBlock8 * kBlock8;   // S itself with several groups
  float wt[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) wt[i][e] = 0.0f;
    if (grp < G && c < S) load8(w + c0 + c, S - c, wt[i]);
  }
  Raw8<T> xn[NV];
  Raw8<R> rn[NV];
  auto load = [&](int64_t row) {
    const T* xp = x + row_at(xs, row, L) + c0;
    const R* rp = FORM != kAdd ? r + row_at(zs, row, L) + c0 : r ? r + row * C : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * 8;
      if (c < S) {
        xn[i] = raw8(xp + c, S - c);
        if (FORM != kAdd || r) rn[i] = raw8(rp + c, S - c);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    xn[i] = Raw8<T>{};
    rn[i] = Raw8<R>{};
  }
  const int64_t mine = first + (G == 1 ? slot : 0);
  if (mine < last) load(mine);
  for (int k = 0; k < each; k += step) {   // as often in every thread: the sums have barriers
    const int64_t row = mine + k;
    const bool live = row < last;
    float u[NV][8], gate[FORM == kAdd ? 1 : NV][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[i][e] = xn[i][e];
        if constexpr (FORM == kAdd) {
          if (r) u[i][e] = to_f32(to_io<R>(u[i][e] + rn[i][e]));
        } else {
          const float z = rn[i][e];
          gate[i][e] = z * sigmoid_f32(z);
          if (FORM == kGateFirst) u[i][e] *= gate[i][e];
        }
        sum[0] = fmaf(u[i][e], u[i][e], sum[0]);
      }
      if (FORM == kAdd && h && live && c < S) store8(h + row * C + c, S - c, u[i]);
    }
    if (row + step < last) load(row + step);
    group_sum(sum, tg, lds);
    float root = sqrtf(sum[0] / (float)S + eps), rr = 1.0f / root;
    if (q && root < 0x1p-9f) {
      // Far below 1 (with an eps below 2^-18) t, and with it the least magnitude of a block, would leave the range in
      // which 448 / m is finite and values are normal; brought to [1, 2) by a power of two, which changes no digit.
      const uint32_t power = __builtin_bit_cast(uint32_t, root) >> 23;   // biased; 0 for a root of 0 alone
      const float up = __builtin_bit_cast(float, (254 - power) << 23);
      root *= up;
      rr = 1.0f / root;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= up;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * 8;
      if (FORM == kAdd && y && live && c < S) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = u[i][e] * rr * wt[i][e];
        store8(y + row * C + c, S - c, o);
      }
      if (q) {
        // y / m does not depend on r: what is quantised is t = y / r, and r joins the scale.  Behind a gate,
        // whose own roundings are of the size of its product's, t is one number; else it is two.
        float t[8], rest[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          t[e] = u[i][e] * wt[i][e];
          if constexpr (FORM == kAdd) rest[e] = fmaf(u[i][e], wt[i][e], -t[e]);
          if constexpr (FORM == kNormFirst) t[e] *= gate[i][e];
        }
        const float m = fmaxf(most_of_16(most_of(t)), kLeast8 * root);
        if (live && c < padded) {
          *reinterpret_cast<uint2*>(q + row * P + c0 + c) = FORM == kAdd ? pack8(t, rest, m) : pack8_once(t, m);
          if (lane % 16 == 0) scale[(int64_t)((c0 + c) / kBlock8) * rows + row] = scale_of(m * rr);
        }
      }
    }
  }
}

// A workgroup takes blockDim.x / tg rows at a time, the next ones loaded ahead, and keeps its sums of dw in
// registers; it leaves one row of part sums [C] in the workspace.
template <typename T, typename R, int NV>
__global__ void __launch_bounds__(512)
add_norm_bwd_kernel(const R* h, const float* __restrict__ w, const T* __restrict__ dy, const R* dh,
                    T* __restrict__ dx, R* dres, float* __restrict__ part, int64_t rows, int C,
                    float eps, int tg) {
  __shared__ float lds[16];
  __shared__ float joined[2048];   // several rows at a time have at most 256 threads of 8 channels each
  const int slot = threadIdx.x / tg, slots = blockDim.x / tg, lane = threadIdx.x % tg;
  const int64_t step = (int64_t)gridDim.x * slots, mine = (int64_t)blockIdx.x * slots + slot;
  const int64_t turns = (rows + step - 1) / step;   // as many in every thread: the sums have barriers
  float wt[NV][8], dw[NV][8];
  Raw8<R> hn[NV], un[NV];
  Raw8<T> gn[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) wt[i][e] = dw[i][e] = 0.0f;
    if (c < C) load8(w + c, C - c, wt[i]);
    hn[i] = un[i] = Raw8<R>{};
    gn[i] = Raw8<T>{};
  }
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * 8;
      if (c < C) {
        hn[i] = raw8(h + row * C + c, C - c);
        gn[i] = raw8(dy + row * C + c, C - c);
        if (dh) un[i] = raw8(dh + row * C + c, C - c);
      }
    }
  };
  if (mine < rows) load(mine);
  for (int64_t k = 0; k < turns; ++k) {
    const int64_t row = mine + k * step;
    const bool live = row < rows;
    float u[NV][8], g[NV][8], up[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[i][e] = hn[i][e];
        g[i][e] = live ? gn[i][e] : 0.0f;   // past the last row: nothing for dw
        up[i][e] = un[i][e];
      }
    if (row + step < rows) load(row + step);
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[0] = fmaf(u[i][e], u[i][e], sum[0]);
        sum[1] = fmaf(g[i][e] * wt[i][e], u[i][e], sum[1]);
      }
    group_sum(sum, tg, lds);
    const float r = 1.0f / sqrtf(sum[0] / (float)C + eps);
    const float m = r * (sum[1] / (float)C);   // mean(t n)
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tg + lane) * 8;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = u[i][e] * r;
          dw[i][e] = fmaf(g[i][e], n, dw[i][e]);
          o[e] = fmaf(r, g[i][e] * wt[i][e] - n * m, up[i][e]);
        }
        if (c < C) {
          if (dx) store8(dx + row * C + c, C - c, o);
          if (dres) store8(dres + row * C + c, C - c, o);
        }
      }
    }
  }
  if (slots == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * 8;
      if (c < C) store8(part + (int64_t)blockIdx.x * C + c, C - c, dw[i]);
    }
    return;
  }
  if constexpr (NV == 1) {   // the rows side by side, added in order
    for (int q = 0; q < slots; ++q) {
      if (slot == q)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = lane * 8 + e;
          joined[c] = q == 0 ? dw[0][e] : joined[c] + dw[0][e];
        }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < C; c += blockDim.x) part[(int64_t)blockIdx.x * C + c] = joined[c];
  }
}

__global__ void __launch_bounds__(256)
add_norm_reduce_kernel(const float* __restrict__ part, int64_t n, int64_t C, float* __restrict__ dw) {
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
  const float v = column_sum(c < C ? part + c : nullptr, n, C);
  if (threadIdx.x < 32 && c < C) dw[c] = v;
}

// ---- host ----

namespace {

struct ItemGrid {
  int tg, nv, threads, each;   // threads per item and workgroup, pieces per thread, tokens per workgroup
  int64_t sets;                // of groups
};

// Pieces of 8 channels, padded to whole blocks.  16 or 32 lanes hold an item of up to 32; beyond that:
//   the addition, which waits for memory alone, takes as many waves as give each thread one piece (two
//   past 512), and one token for each: 16384 x 2560 to 8 bits 93 us; 2 pieces 95, 3 pieces and half the
//   threads 100, 5 pieces in one wave 109; four tokens in a row 94, sixteen 100;
//   gates also keep the vector ALU busy: 1, 2, 4 or 8 waves (three or five leave a SIMD with less) of up to
//   three pieces per thread, the fewest idle lanes first (256 threads of 3 pieces 92 us, 128 of 5 95, 512 of 2
//   114, 320 of 2 105), and two tokens in a row: more of them make whole rounds of workgroups that load, compute
//   and store in step (256 of 3: four 90, but 16384 x 8 x 512 70 in place of 67, 2048 x 5120 17 in place of 16).
// With several groups a workgroup's places are for groups of one token, and those past the last group stand idle
// (16384 x 2 x 128 24 us, 8 x 128 27, 2 x 1024 45, 8 x 512 72).
ItemGrid item_grid(int64_t rows, int64_t S, int64_t G, bool gate) {
  ItemGrid g;
  const int pieces = (int)((S + kBlock8 - 1) / kBlock8 * (kBlock8 / 8));
  const bool many = gate && rows * G >= 1024;
  if (pieces <= 32) {
    g.tg = pieces;
  } else if (!many) {
    const int most = pieces > 512 ? 2 : 1;
    g.tg = (pieces + kWave * most - 1) / (kWave * most) * kWave;
  } else {
    g.tg = 0;
    for (int tg = 512; tg >= kWave; tg /= 2) {
      const int nv = (pieces + tg - 1) / tg;
      if (nv > 3 || (nv == 1 && tg > kWave)) continue;
      if (g.tg == 0 || tg * nv < g.tg * g.nv) {
        g.tg = tg;
        g.nv = nv;
      }
    }
  }
  g.nv = (pieces + g.tg - 1) / g.tg;
  int slots = g.tg >= 256 || many ? (g.tg < kWave ? 256 / g.tg : 1) : 256 / g.tg;
  if (many && g.tg == kWave) slots = 4;
  g.threads = g.tg * slots;
  g.sets = G == 1 ? 1 : (G + slots - 1) / slots;
  g.each = (G == 1 ? slots : 1) * (many ? 2 : 1);
  return g;
}

// The gradients: one piece per thread up to 512 of them, two beyond; small rows side by side in workgroups of
// up to 512 threads; and workgroups until 20 KB of inputs are on their way to each CU, at most 1280 threads:
// more only make more part sums (8192 x 2560 with an fp32 residual, one workgroup per CU 66 us, two 73,
// four 82; one row of 128 channels at a time, 145388 x 128 in bf16 181 us, 32 at a time 39).
struct BwdGrid {
  int nv, tg, threads;
  int64_t stripes;
};
BwdGrid bwd_grid(int64_t rows, int64_t C, int bf16, int res_bf16) {
  BwdGrid g;
  const int pieces = (int)((C + 7) / 8);
  g.nv = pieces > 512 ? 2 : 1;
  g.tg = pieces <= 16 ? 16 : pieces <= 32 ? 32 : (pieces + g.nv * kWave - 1) / (g.nv * kWave) * kWave;
  const int slots = g.tg <= 256 ? 512 / g.tg : 1;
  g.threads = g.tg * slots;
  const int64_t bytes = ((bf16 ? 2 : 4) + (res_bf16 ? 4 : 8)) * C * slots;
  int64_t each = (20 * 1024 + bytes - 1) / bytes;
  if (each * g.threads > 1280) each = 1280 / g.threads;
  g.stripes = 256 * each;
  const int64_t most = (rows + slots - 1) / slots;
  if (g.stripes > most) g.stripes = most;
  return g;
}

}  // namespace

// 512 threads hold 2 x 8 elements each.
int64_t block_norm_limit() { return 8192; }

// Rows are counted in 31 bits, and the launch has fewer than 2^32 threads along its first axis.
int block_norm_grid_ok(int64_t batch, int64_t L, int64_t C, int64_t G, int gate) {
  if (C > (1 << 24) || batch > INT32_MAX / L) return 0;
  const int64_t rows = batch * L;
  const ItemGrid g = item_grid(rows, C / G, G, gate != 0);
  return (rows + g.each - 1) / g.each * g.threads < (int64_t(1) << 32) && g.sets <= 65535;
}

size_t add_norm_bwd_workspace(int64_t rows, int64_t C, int bf16, int res_bf16) {
  return size_t(bwd_grid(rows, C, bf16, res_bf16).stripes) * C * sizeof(float);
}

template <typename T, typename R, int FORM>
static hipError_t block_norm_f(const BlockNormArgs& a, hipStream_t stream) {
  const int64_t rows = a.batch * a.L;
  const ItemGrid g = item_grid(rows, a.C / a.G, a.G, FORM != kAdd);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((rows + g.each - 1) / g.each), (unsigned)g.sets), dim3(g.threads), 0, stream,
                       static_cast<const T*>(a.x), Strides{a.xs[0], a.xs[1]},
                       static_cast<const R*>(a.r), Strides{a.zs[0], a.zs[1]}, a.w,
                       static_cast<R*>(a.h), static_cast<T*>(a.y), a.q, a.scale, a.L, rows, (int)a.C,
                       (int)a.G, a.eps, g.tg, g.each);
  };
  if (g.nv == 1) go(block_norm_kernel<T, R, 1, FORM>);
  else if (g.nv == 2) go(block_norm_kernel<T, R, 2, FORM>);
  else if constexpr (FORM != kAdd) {
    go(block_norm_kernel<T, R, 3, FORM>);
  }
  return hipGetLastError();
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream) {
  if (a.gate == 0) {
    if (!a.bf16) return block_norm_f<float, float, kAdd>(a, stream);
    return a.res_bf16 ? block_norm_f<bf16, bf16, kAdd>(a, stream) : block_norm_f<bf16, float, kAdd>(a, stream);
  }
  if (a.gate == 1)
    return a.bf16 ? block_norm_f<bf16, bf16, kGateFirst>(a, stream) : block_norm_f<float, float, kGateFirst>(a, stream);
  return a.bf16 ? block_norm_f<bf16, bf16, kNormFirst>(a, stream) : block_norm_f<float, float, kNormFirst>(a, stream);
}

template <typename T, typename R>
static hipError_t add_norm_bwd_t(const AddNormBwdArgs& a, hipStream_t stream) {
  const BwdGrid g = bwd_grid(a.rows, a.C, a.bf16, a.res_bf16);
  float* part = static_cast<float*>(a.workspace);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)g.stripes), dim3(g.threads), 0, stream,
                       static_cast<const R*>(a.h), a.w, static_cast<const T*>(a.dy),
                       static_cast<const R*>(a.dh), static_cast<T*>(a.dx), static_cast<R*>(a.dres),
                       part, a.rows, (int)a.C, a.eps, g.tg);
  };
  if (g.nv == 1) go(add_norm_bwd_kernel<T, R, 1>);
  else go(add_norm_bwd_kernel<T, R, 2>);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(add_norm_reduce_kernel, dim3((unsigned)((a.C + 31) / 32)), dim3(256), 0, stream,
                     part, g.stripes, a.C, a.dw);
  return hipGetLastError();
}

hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t stream) {
  if (!a.bf16) return add_norm_bwd_t<float, float>(a, stream);
  return a.res_bf16 ? add_norm_bwd_t<bf16, bf16>(a, stream) : add_norm_bwd_t<bf16, float>(a, stream);
}

}  // namespace ssd
