// gated_norm.hip -- the grouped RMS norm with a SiLU gate that follows the scan,
// and its gradients.
//
// A row's D channels fall into G groups of S = D / G.  With s(z) = z sigmoid(z)
// (1 without z) and, in each group, r = (mean(u^2) + eps)^(-1/2):
//     gate first (norm_before_gate = 0):  u = x s(z),  y = w u r
//     norm first (norm_before_gate = 1):  u = x,       y = w u r s(z)
// Gradients: with t = w dy (times s(z) where the norm comes first),
//     du = r (t - n mean(t n)), n = u r,    dw = sum over rows of dy (s(z)) n,
//     gate first:  dx = du s(z),  dz = du x s'(z)
//     norm first:  dx = du,       dz = dy w n s'(z)
// With n in place of u r^3 nothing leaves fp32 that its factors and the result fit: r^3
// does for |u| above 1e13 or below 1e-13.
//
// Bound by HBM: 3 elements moved per output forwards, 5 backwards.  A group's
// elements stay in registers between the sums and the outputs, so every input
// is read once: TG threads hold a group, NV pieces of V elements each (TG at most one
// wave where a group fits one, so that no barrier is needed and small groups share
// a wave; otherwise as many waves as the group fills).  The backward pass sums
// mean(u^2) and mean(t u) = mean(t n) / r in one reduction: neither needs the other.
// bf16: 2 x 8192 rows of 5120 channels 107 us forwards (4.7 TB/s of the 5.15 that a large
// copy reaches), 2 x 4096 rows of 8 x 512 channels 76 us backwards (4.4 TB/s; the part
// sums take 6 of them).
#include "layer_device.hpp"
#include "layer_host.hpp"

namespace ssd {

constexpr int kNormThreads = 256;

// blockDim.x / tg groups per workgroup.
template <typename T, int V, int NV, bool GATE, int NT>
__global__ void __launch_bounds__(NT)
norm_fwd_kernel(const T* __restrict__ x, const T* __restrict__ z, Strides zs,
                const float* __restrict__ w, T* __restrict__ y, int64_t L, int64_t rows, int D,
                int G, float eps, int before, int tg) {
  __shared__ float lds[16];
  const int S = D / G;
  const int per = blockDim.x / tg;
  const int64_t item = (int64_t)blockIdx.x * per + threadIdx.x / tg;   // (row, group)
  const int lane = threadIdx.x % tg;
  const bool live = item < rows * G;
  const int64_t row = live ? item / G : 0;
  const int c0 = live ? (int)(item % G) * S : 0;
  const T* xp = x + row * D + c0;
  const T* zp = GATE ? z + (row / L) * zs.batch + (row % L) * zs.token + c0 : nullptr;
  float u[NV][V], gate[GATE ? NV : 1][V];
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) u[i][v] = 0.0f;
    if (live && c < S) {
      load_v<V>(xp + c, u[i]);
      if constexpr (GATE) load_v<V>(zp + c, gate[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (live && (i * tg + lane) * V < S) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (GATE) {
          gate[i][v] *= sigmoid_f32(gate[i][v]);
          if (!before) u[i][v] *= gate[i][v];
        }
        sum[0] = fmaf(u[i][v], u[i][v], sum[0]);
      }
    }
  }
  group_sum(sum, tg, lds);
  const float r = rsqrtf(sum[0] / (float)S + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * V;
    if (live && c < S) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v] = u[i][v] * r * w[c0 + c + v];
        if constexpr (GATE)
          if (before) o[v] *= gate[i][v];
      }
      store_v<V>(y + row * D + c0 + c, o);
    }
  }
}

// A workgroup takes rows first, first + stride, ... of its groups and keeps
// their sums of dw in registers; it leaves one row of part sums [D] in the
// workspace, and norm_reduce_kernel adds those in order.
template <typename T, int V, int NV, bool GATE, int NT>
__global__ void __launch_bounds__(NT)
norm_bwd_kernel(const T* __restrict__ x, const T* __restrict__ z, Strides zs,
                const float* __restrict__ w, const T* __restrict__ dy, T* __restrict__ dx,
                T* __restrict__ dz, Strides dzs, float* __restrict__ part, int64_t L, int64_t rows,
                int D, int G, float eps, int before, int tg) {
  __shared__ float lds[32];
  const int S = D / G;
  const int per = blockDim.x / tg;
  const int grp = blockIdx.y * per + threadIdx.x / tg;
  const int lane = threadIdx.x % tg;
  const bool live = grp < G;
  const int c0 = live ? grp * S : 0;
  float wt[NV][V], dw[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (i * tg + lane) * V;
      wt[i][v] = live && c < S ? w[c0 + c + v] : 0.0f;
      dw[i][v] = 0.0f;
    }
  typedef typename RawV<T, V>::type Raw;
  Raw xn[NV], gn[NV], zn[GATE ? NV : 1];   // the next row, loaded while this one is worked on
  auto load = [&](int64_t row) {
    const T* xp = x + row * D + c0;
    const T* gp = dy + row * D + c0;
    const T* zp = GATE ? z + (row / L) * zs.batch + (row % L) * zs.token + c0 : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * V;
      xn[i] = gn[i] = zero_raw<T, V>();
      if constexpr (GATE) zn[i] = zero_raw<T, V>();
      if (live && c < S) {
        xn[i] = load_raw<T, V>(xp + c);
        gn[i] = load_raw<T, V>(gp + c);
        if constexpr (GATE) zn[i] = load_raw<T, V>(zp + c);
      }
    }
  };
  if (blockIdx.x < rows) load(blockIdx.x);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    T* dzp = GATE ? dz + (row / L) * dzs.batch + (row % L) * dzs.token + c0 : nullptr;
    Raw xr[NV], gr[NV], zr[GATE ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xr[i] = xn[i];
      gr[i] = gn[i];
      if constexpr (GATE) zr[i] = zn[i];
    }
    if (row + gridDim.x < rows) load(row + gridDim.x);
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float xv[V], gv[V], zv[V];
      widen<T, V>(xr[i], xv);
      widen<T, V>(gr[i], gv);
      if constexpr (GATE) widen<T, V>(zr[i], zv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float u = xv[v], t = gv[v] * wt[i][v];
        if constexpr (GATE) {
          const float s = zv[v] * sigmoid_f32(zv[v]);
          if (before) t *= s; else u *= s;
        }
        sum[0] = fmaf(u, u, sum[0]);
        sum[1] = fmaf(t, u, sum[1]);
      }
    }
    group_sum(sum, tg, lds);
    const float r = rsqrtf(sum[0] / (float)S + eps);
    const float k = r * (sum[1] / (float)S);   // mean(t n)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tg + lane) * V;
      float xv[V], gv[V], zv[V], ox[V], oz[V];
      widen<T, V>(xr[i], xv);
      widen<T, V>(gr[i], gv);
      if constexpr (GATE) widen<T, V>(zr[i], zv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float s = 1.0f, slope = 0.0f;
        if constexpr (GATE) {
          const float sg = sigmoid_f32(zv[v]);
          s = zv[v] * sg;
          slope = silu_slope(zv[v], sg);
        }
        if (before) {
          const float n = xv[v] * r, dn = gv[v] * s;
          dw[i][v] = fmaf(dn, n, dw[i][v]);
          ox[v] = r * (dn * wt[i][v] - n * k);
          oz[v] = gv[v] * wt[i][v] * n * slope;
        } else {
          const float n = xv[v] * s * r;
          const float du = r * (gv[v] * wt[i][v] - n * k);
          dw[i][v] = fmaf(gv[v], n, dw[i][v]);
          ox[v] = du * s;
          oz[v] = du * xv[v] * slope;
        }
      }
      if (live && c < S) {
        store_v<V>(dx + row * D + c0 + c, ox);
        if constexpr (GATE) store_v<V>(dzp + c, oz);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tg + lane) * V;
    if (live && c < S)
#pragma unroll
      for (int v = 0; v < V; ++v) part[(int64_t)blockIdx.x * D + c0 + c + v] = dw[i][v];
  }
}

__global__ void __launch_bounds__(256)
norm_reduce_kernel(const float* __restrict__ part, int64_t n, int64_t D, float* __restrict__ dw) {
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
  const float v = column_sum(c < D ? part + c : nullptr, n, D);
  if (threadIdx.x < 32 && c < D) dw[c] = v;
}

// ---- host ----

namespace {

struct NormGrid {
  int tg, threads, nv;   // threads per group and workgroup, pieces per thread
  int64_t stripes;       // backward: workgroups sharing the rows of one set of groups
  int64_t sets;          // sets of groups
};

// Pieces per thread before a group takes more threads: 16 elements in fp32
// registers either way, a few single ones where nothing is aligned.
constexpr int kNormStripes = 1024;   // workgroups of the backward pass (75 us; 512: 85, 2048: 81)
constexpr int norm_wide(int V) { return V == 8 ? 2 : 4; }

NormGrid norm_grid(int64_t rows, int64_t D, int64_t G, int V) {
  NormGrid g;
  const int64_t S = D / G, pieces = (S + V - 1) / V;
  if (pieces <= kWave) {
    g.tg = 1;
    while (g.tg < pieces) g.tg *= 2;
  } else {
    const int64_t wide = V == 1 && pieces > 4096 ? 8 : norm_wide(V);
    g.tg = (int)((pieces + kWave * wide - 1) / (kWave * wide)) * kWave;
  }
  g.nv = (int)((pieces + g.tg - 1) / g.tg);
  // small groups share a workgroup of four waves, or of one where there are few
  const int few = rows * G * g.tg <= 64 * 256 ? kWave : kNormThreads;
  const int64_t per = g.tg < few ? few / g.tg : 1;
  g.threads = (int)(g.tg * per);
  g.sets = (G + per - 1) / per;
  g.stripes = kNormStripes / g.sets;
  if (g.stripes < 1) g.stripes = 1;
  if (g.stripes > rows) g.stripes = rows;
  return g;
}

}  // namespace

// The largest group: 512 threads hold 2 x 8 bf16 or 4 x 4 fp32 each, or 1024
// hold 8 single elements.
int64_t norm_group_limit() { return 8192; }

// Every launch has fewer than 2^32 threads (V = 1 takes the most).
int norm_grid_ok(int64_t batch, int64_t L, int64_t D, int64_t G) {
  if (D > (1 << 24)) return 0;
  const NormGrid g = norm_grid(batch * L, D, G, 1);
  return (__int128)batch * L * G * g.tg + 1024 < (int64_t(1) << 32) && g.sets <= 65535;
}

size_t norm_bwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t G, int io_bf16) {
  size_t most = 0;
  for (int V : {1, io_bf16 ? 8 : 4}) {
    const NormGrid g = norm_grid(batch * L, D, G, V);
    const size_t n = size_t(g.stripes) * D * sizeof(float);
    if (n > most) most = n;
  }
  return most;
}

template <typename T, int V, bool GATE>
static hipError_t norm_fwd_v(const NormArgs& a, hipStream_t stream) {
  const int64_t rows = a.batch * a.L;
  const NormGrid g = norm_grid(rows, a.D, a.G, V);
  const int64_t per = g.threads / g.tg;
  const dim3 grid((unsigned)((rows * a.G + per - 1) / per));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(g.threads), 0, stream, static_cast<const T*>(a.x),
                       static_cast<const T*>(a.z), Strides{a.zs[0], a.zs[1]}, a.w,
                       static_cast<T*>(a.y), a.L, rows, (int)a.D, (int)a.G, a.eps, a.before, g.tg);
  };
  if (g.threads <= kNormThreads) {
    if (g.nv == 1) go(norm_fwd_kernel<T, V, 1, GATE, kNormThreads>);
    else if (g.nv == 2) go(norm_fwd_kernel<T, V, 2, GATE, kNormThreads>);
    else if constexpr (norm_wide(V) > 2) {
      if (g.nv == 3) go(norm_fwd_kernel<T, V, 3, GATE, kNormThreads>);
      else go(norm_fwd_kernel<T, V, 4, GATE, kNormThreads>);
    }
  } else if constexpr (V > 1) {
    go(norm_fwd_kernel<T, V, norm_wide(V), GATE, 512>);
  } else {
    if (g.nv <= 4) go(norm_fwd_kernel<T, 1, 4, GATE, 1024>);
    else go(norm_fwd_kernel<T, 1, 8, GATE, 1024>);
  }
  return hipGetLastError();
}

template <typename T, int V>
static hipError_t norm_fwd_g(const NormArgs& a, hipStream_t stream) {
  return a.z ? norm_fwd_v<T, V, true>(a, stream) : norm_fwd_v<T, V, false>(a, stream);
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream) {
  if (a.bf16) return a.vec ? norm_fwd_g<bf16, 8>(a, stream) : norm_fwd_g<bf16, 1>(a, stream);
  return a.vec ? norm_fwd_g<float, 4>(a, stream) : norm_fwd_g<float, 1>(a, stream);
}

template <typename T, int V, bool GATE>
static hipError_t norm_bwd_v(const NormArgs& a, hipStream_t stream) {
  const int64_t rows = a.batch * a.L;
  const NormGrid g = norm_grid(rows, a.D, a.G, V);
  const dim3 grid((unsigned)g.stripes, (unsigned)g.sets);
  float* part = static_cast<float*>(a.workspace);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(g.threads), 0, stream, static_cast<const T*>(a.x),
                       static_cast<const T*>(a.z), Strides{a.zs[0], a.zs[1]}, a.w,
                       static_cast<const T*>(a.dy), static_cast<T*>(a.dx), static_cast<T*>(a.dz),
                       Strides{a.dzs[0], a.dzs[1]}, part, a.L, rows, (int)a.D, (int)a.G, a.eps,
                       a.before, g.tg);
  };
  if (g.threads <= kNormThreads) {
    if (g.nv == 1) go(norm_bwd_kernel<T, V, 1, GATE, kNormThreads>);
    else if (g.nv == 2) go(norm_bwd_kernel<T, V, 2, GATE, kNormThreads>);
    else if constexpr (norm_wide(V) > 2) {
      if (g.nv == 3) go(norm_bwd_kernel<T, V, 3, GATE, kNormThreads>);
      else go(norm_bwd_kernel<T, V, 4, GATE, kNormThreads>);
    }
  } else if constexpr (V > 1) {
    go(norm_bwd_kernel<T, V, norm_wide(V), GATE, 512>);
  } else {
    if (g.nv <= 4) go(norm_bwd_kernel<T, 1, 4, GATE, 1024>);
    else go(norm_bwd_kernel<T, 1, 8, GATE, 1024>);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((a.D + 31) / 32)), dim3(256), 0, stream,
                     part, g.stripes, a.D, a.dw);
  return hipGetLastError();
}

template <typename T, int V>
static hipError_t norm_bwd_g(const NormArgs& a, hipStream_t stream) {
  return a.z ? norm_bwd_v<T, V, true>(a, stream) : norm_bwd_v<T, V, false>(a, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream) {
  if (a.bf16) return a.vec ? norm_bwd_g<bf16, 8>(a, stream) : norm_bwd_g<bf16, 1>(a, stream);
  return a.vec ? norm_bwd_g<float, 4>(a, stream) : norm_bwd_g<float, 1>(a, stream);
}

}  // namespace ssd
