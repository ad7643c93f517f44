// add_norm.hip -- the residual addition with the RMS norm in front of a layer, its
// gradients, and the gated norm behind the layer with its output in 8 bits.
//
// Over the C channels of a token:  h = x + residual, rounded to the residual's type;
// r = (mean(h^2) + eps)^(-1/2);  y = w h r.  In 8 bits, per block of 128 channels:
// m = max |y|, q = e4m3(y 448 / m), scale = m / 448, from h and w with no rounding of y between.
// Gated, in each of G groups, with s(z) = z sigmoid(z):  u = x s(z) or x,  y = w u r or
// w u r s(z).
// Gradients, with n = h r and t = w dy:  dh' = dh + r (t - n mean(t n)),  dw = sum over
// tokens of dy n;  mean(t n) = r mean(t h), so one reduction gives both sums.
//
// Bound by HBM: every input is read once, a token's elements stay in registers between
// the sum and the outputs.  Pieces of eight channels, NV per thread; a token is held by
// 16 or 32 lanes, one wave, or several.
#include "block_device.hpp"
#include "block_host.hpp"

namespace ssd {

enum NormForm { kAdd = 0, kGateFirst = 1, kNormFirst = 2 };

// blockDim.x / tg items (a token, or a group of one) per workgroup.
template <typename T, typename R, int NV, int FORM>
__global__ void __launch_bounds__(512)
block_norm_kernel(const T* __restrict__ x, Strides xs, const R* r, Strides zs,
                  const float* __restrict__ w, R* h, T* __restrict__ y,
                  unsigned char* __restrict__ q, float* __restrict__ scale, int64_t L, int64_t rows,
                  int C, int G, float eps, int tg) {
  __shared__ float lds[8];
  const int S = C / G;
  const int per = blockDim.x / tg;
  const int64_t item = (int64_t)blockIdx.x * per + threadIdx.x / tg;
  const int lane = threadIdx.x % tg;
  const bool live = item < rows * G;
  const int64_t row = live ? item / G : 0;
  const int c0 = live ? (int)(item % G) * S : 0;
  const T* xp = x + row_at(xs, row, L) + c0;
  const R* rp = r;
  if (FORM == kAdd) {
    if (r) rp = r + row * C;
  } else {
    rp = r + row_at(zs, row, L) + c0;
  }
  float u[NV][8], other[NV][8];
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * 8;
    const int n = live ? S - c : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) u[i][e] = other[i][e] = 0.0f;
    if (n > 0) {
      load8(xp + c, n, u[i]);
      if (FORM != kAdd || r) load8(rp + c, n, other[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * 8;
    const int n = live ? S - c : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (FORM == kAdd) {
        if (r) u[i][e] = to_f32(to_io<R>(u[i][e] + other[i][e]));
      } else {
        other[i][e] *= sigmoid_f32(other[i][e]);
        if (FORM == kGateFirst) u[i][e] *= other[i][e];
      }
      sum[0] = fmaf(u[i][e], u[i][e], sum[0]);
    }
    if (FORM == kAdd && h && n > 0) store8(h + row * C + c, n, u[i]);
  }
  group_sum(sum, tg, lds);
  const float rr = 1.0f / sqrtf(sum[0] / (float)S + eps);
  const int64_t P = (int64_t)(C + kBlock8 - 1) / kBlock8 * kBlock8;
  const int padded = (S + kBlock8 - 1) / kBlock8 * kBlock8;   // S itself with several groups
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * 8;
    const int n = live ? S - c : 0;
    float wt[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) wt[e] = 0.0f;
    if (n > 0) load8(w + c0 + c, n, wt);
    if (FORM == kAdd && y && n > 0) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = u[i][e] * rr * wt[e];
      store8(y + row * C + c, n, o);
    }
    if (q) {
      // y / m does not depend on r: what is quantised is y / r, and r joins the scale.
      double t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t[e] = (double)u[i][e] * (double)wt[e];
        if (FORM == kNormFirst) t[e] *= (double)other[i][e];
      }
      const double m = fmax(most_of_16(most_of(t)) * (double)rr, (double)kLeast8);
      if (live && c < padded) {
        *reinterpret_cast<uint2*>(q + row * P + c0 + c) = pack8(t, (double)kMost8 * (double)rr / m);
        if (lane % 16 == 0) scale[(int64_t)((c0 + c) / kBlock8) * rows + row] = (float)(m / (double)kMost8);
      }
    }
  }
}

// A workgroup takes rows first, first + stride, ... and keeps its sums of dw in
// registers; it leaves one row of part sums [C] in the workspace.
template <typename T, typename R, int NV>
__global__ void __launch_bounds__(512)
add_norm_bwd_kernel(const R* h, const float* __restrict__ w, const T* __restrict__ dy, const R* dh,
                    T* __restrict__ dx, R* dres, float* __restrict__ part, int64_t rows, int C,
                    float eps) {
  __shared__ float lds[16];
  const int tg = blockDim.x, lane = threadIdx.x;
  float wt[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) wt[i][e] = dw[i][e] = 0.0f;
    if (c < C) load8(w + c, C - c, wt[i]);
  }
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    float u[NV][8], g[NV][8], up[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] = g[i][e] = up[i][e] = 0.0f;
      if (c < C) {
        load8(h + row * C + c, C - c, u[i]);
        load8(dy + row * C + c, C - c, g[i]);
        if (dh) load8(dh + row * C + c, C - c, up[i]);
      }
    }
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
    const float k = r * (sum[1] / (float)C);   // mean(t n)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * 8;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = u[i][e] * r;
        dw[i][e] = fmaf(g[i][e], n, dw[i][e]);
        o[e] = fmaf(r, g[i][e] * wt[i][e] - n * k, up[i][e]);
      }
      if (c < C) {
        if (dx) store8(dx + row * C + c, C - c, o);
        if (dres) store8(dres + row * C + c, C - c, o);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * 8;
    if (c < C) store8(part + (int64_t)blockIdx.x * C + c, C - c, dw[i]);
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
  int tg, nv, threads;
};

// 16 or 32 lanes hold an item of up to 32 pieces; beyond that whole waves.
ItemGrid item_grid(int64_t items, int64_t S) {
  ItemGrid g;
  const int pieces = (int)((S + kBlock8 - 1) / kBlock8 * (kBlock8 / 8));
  if (pieces <= 32) {
    g.tg = pieces;
  } else {
    const int most = items < 1024 ? 2 : 4;
    g.tg = (pieces + kWave * most - 1) / (kWave * most) * kWave;
  }
  g.nv = (pieces + g.tg - 1) / g.tg;
  g.threads = g.tg >= 256 ? g.tg : 256 / g.tg * g.tg;
  return g;
}

constexpr int kStripes = 1024;
int64_t stripes_of(int64_t rows) { return rows < kStripes ? rows : kStripes; }

}  // namespace

// 512 threads hold 2 x 8 elements each.
int64_t block_norm_limit() { return 8192; }

int block_norm_grid_ok(int64_t batch, int64_t L, int64_t C, int64_t G) {
  const ItemGrid g = item_grid(1, C / G);
  return C <= (1 << 24) && (__int128)batch * L * G * g.tg + 512 < (int64_t(1) << 32);
}

size_t add_norm_bwd_workspace(int64_t rows, int64_t C) {
  return size_t(stripes_of(rows)) * C * sizeof(float);
}

template <typename T, typename R, int FORM>
static hipError_t block_norm_f(const BlockNormArgs& a, hipStream_t stream) {
  const int64_t rows = a.batch * a.L, items = rows * a.G;
  const ItemGrid g = item_grid(items, a.C / a.G);
  const int64_t per = g.threads / g.tg;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((items + per - 1) / per)), dim3(g.threads), 0, stream,
                       static_cast<const T*>(a.x), Strides{a.xs[0], a.xs[1]},
                       static_cast<const R*>(a.r), Strides{a.zs[0], a.zs[1]}, a.w,
                       static_cast<R*>(a.h), static_cast<T*>(a.y), a.q, a.scale, a.L, rows, (int)a.C,
                       (int)a.G, a.eps, g.tg);
  };
  if (g.nv == 1) go(block_norm_kernel<T, R, 1, FORM>);
  else if (g.nv == 2) go(block_norm_kernel<T, R, 2, FORM>);
  else if (g.nv == 3) go(block_norm_kernel<T, R, 3, FORM>);
  else go(block_norm_kernel<T, R, 4, FORM>);
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
  const int pieces = (int)((a.C + 7) / 8);
  const int nv = pieces > 512 ? 2 : 1;
  const int threads = (pieces + nv * kWave - 1) / (nv * kWave) * kWave;
  const int64_t stripes = stripes_of(a.rows);
  float* part = static_cast<float*>(a.workspace);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)stripes), dim3(threads), 0, stream,
                       static_cast<const R*>(a.h), a.w, static_cast<const T*>(a.dy),
                       static_cast<const R*>(a.dh), static_cast<T*>(a.dx), static_cast<R*>(a.dres),
                       part, a.rows, (int)a.C, a.eps);
  };
  if (nv == 1) go(add_norm_bwd_kernel<T, R, 1>);
  else go(add_norm_bwd_kernel<T, R, 2>);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(add_norm_reduce_kernel, dim3((unsigned)((a.C + 31) / 32)), dim3(256), 0, stream,
                     part, stripes, a.C, a.dw);
  return hipGetLastError();
}

hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t stream) {
  if (!a.bf16) return add_norm_bwd_t<float, float>(a, stream);
  return a.res_bf16 ? add_norm_bwd_t<bf16, bf16>(a, stream) : add_norm_bwd_t<bf16, float>(a, stream);
}

}  // namespace ssd
