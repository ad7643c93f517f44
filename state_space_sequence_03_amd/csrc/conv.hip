// conv.hip -- the short depthwise causal convolution that makes a layer's x, B
// and C out of its projection, its gradients, and its single-token form.
//
// For every batch b, channel c and token t, with width W:
//     u[t] = bias[c] + sum_{k < W} w[c, k] x[t - (W - 1) + k]
//     y[t] = u[t]                (no activation)  or  u[t] sigmoid(u[t])
// where x at t < 0 is the caller's state of the W - 1 inputs before the first
// (zero without one).  The gradients, with du = dy act'(u):
//     dx[t] = sum_k w[c, k] du[t + (W - 1) - k]     (du = 0 past the last token)
//     dw[c, k] = sum_{b, t} du[t] x[t - (W - 1) + k],   dbias[c] = sum du[t]
//
// Both directions are bound by HBM: 2 elements moved per output forwards, 3
// backwards, against ~20 and ~40 VALU operations.  A thread owns V channels
// (four where sizes and alignment allow, else one) of a run of tokens and slides a
// window of W - 1 rows in registers, so each row is loaded once per run plus W - 1
// rows of overlap.  Four channels a thread keep enough waves in flight (eight: 87 us
// against 80 forwards, 102 against 86 backwards).  bf16, width 4: 2 x 8192 tokens of
// 5376 channels 75 us forwards (4.7 TB/s of the 5.15 that a large copy reaches; runs of
// 16 tokens, of 8 and 64 tokens 3 us more), 2 x 4096 tokens 65 us backwards (4.1 TB/s;
// the part sums take 5 of them).  Both have a path without conditions for the rows
// inside a run: with them 78 and 72 us.
#include <type_traits>

#include "layer_device.hpp"
#include "layer_host.hpp"

namespace ssd {

// Up to three outputs (or upstream gradients) side by side along the channels,
// each a contiguous [batch, seqlen, size] tensor; `end` are running channel counts.
struct ConvParts {
  void* p[3];
  int64_t end[3];
};

template <typename T>
struct PartRow {
  T* p;        // element (b, 0, c)
  int64_t ld;  // elements per token
};
template <typename T>
__device__ __forceinline__ PartRow<T> part_of(const ConvParts& q, int64_t b, int64_t L, int64_t c) {
  const int s = (c >= q.end[0]) + (c >= q.end[1]);
  T* const p = static_cast<T*>(s == 0 ? q.p[0] : s == 1 ? q.p[1] : q.p[2]);
  const int64_t lo = s == 0 ? 0 : s == 1 ? q.end[0] : q.end[1];
  const int64_t hi = s == 0 ? q.end[0] : s == 1 ? q.end[1] : q.end[2];
  return {p + (b * L * (hi - lo) + (c - lo)), hi - lo};
}

constexpr int kConvThreads = 256;
constexpr int kFwdAhead = 4, kBwdAhead = 2;   // rows loaded ahead of those in use

// Workgroup -> (channels, tokens).  Workgroups go to the 8 XCDs in turn; each XCD
// takes a run of tokens, channels fastest, so that rows are read whole and the
// W - 1 rows that neighbouring tiles share come from one L2.  The grid is rounded up to
// a multiple of 8: tiles past the last are empty.
struct ConvTiles {
  int64_t bx, by;   // workgroups along the channels and the tokens
};
__device__ __forceinline__ bool conv_tile(const ConvTiles& n, int64_t* ix, int64_t* iy) {
  const int64_t t = (int64_t)(blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;
  *ix = t % n.bx;
  *iy = t / n.bx;
  return t < n.bx * n.by;
}

// Threads of a workgroup: lc lanes along the channels (a power of two up to
// 64), kConvThreads / lc runs of tokens.
template <typename T, int V, int W, bool ACT>
__global__ void __launch_bounds__(kConvThreads)
conv_fwd_kernel(const T* __restrict__ x, Strides xs, const float* __restrict__ w,
                const float* __restrict__ bias, const T* init, ConvParts y, T* fin, int64_t L, int64_t C, ConvTiles tiles, int lc_log, int64_t run) {
  constexpr int M = kFwdAhead;
  int64_t ix, iy;
  if (!conv_tile(tiles, &ix, &iy)) return;
  const int lane = threadIdx.x & ((1 << lc_log) - 1);
  const int64_t c = (ix * (1 << lc_log) + lane) * V;
  const int64_t t0 = (iy * (blockDim.x >> lc_log) + (threadIdx.x >> lc_log)) * run;
  const int64_t b = blockIdx.y;
  if (c >= C || t0 >= L) return;
  const int64_t t1 = t0 + run < L ? t0 + run : L;
  float wt[W][V], bs[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bs[v] = bias ? bias[c + v] : 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) wt[k][v] = w[(c + v) * W + k];
  }
  typedef typename RawV<T, V>::type Raw;
  const T* xp = x + b * xs.batch + c;
  Raw win[W - 1];   // rows t - (W - 1) .. t - 1
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int64_t t = t0 - (W - 1) + k;
    if (t >= 0)
      win[k] = load_raw<T, V>(xp + t * xs.token);
    else if (init)
      win[k] = load_raw<T, V>(init + (b * (W - 1) + (t + W - 1)) * C + c);
    else
      win[k] = zero_raw<T, V>();
  }
  const PartRow<T> o = part_of<T>(y, b, L, c);
  Raw next[M];
#pragma unroll
  for (int a = 0; a < M; ++a)
    next[a] = t0 + a < t1 ? load_raw<T, V>(xp + (t0 + a) * xs.token) : zero_raw<T, V>();
  auto form = [&](const Raw& cur, int64_t t) {
    float u[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = bs[v];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      widen<T, V>(win[k], r);
#pragma unroll
      for (int v = 0; v < V; ++v) u[v] = fmaf(wt[k][v], r[v], u[v]);
    }
    widen<T, V>(cur, r);
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = fmaf(wt[W - 1][v], r[v], u[v]);
    if constexpr (ACT) {
#pragma unroll
      for (int v = 0; v < V; ++v) u[v] *= sigmoid_f32(u[v]);
    }
    store_v<V>(o.p + t * o.ld, u);
#pragma unroll
    for (int k = 0; k + 1 < W - 1; ++k) win[k] = win[k + 1];
    win[W - 2] = cur;
  };
  for (int64_t t = t0; t < t1; t += M) {   // whole groups of M rows without conditions
    Raw cur[M];
#pragma unroll
    for (int a = 0; a < M; ++a) cur[a] = next[a];
    if (t + 2 * M <= t1) {
#pragma unroll
      for (int a = 0; a < M; ++a) next[a] = load_raw<T, V>(xp + (t + M + a) * xs.token);
    } else {
#pragma unroll
      for (int a = 0; a < M; ++a)
        if (t + M + a < t1) next[a] = load_raw<T, V>(xp + (t + M + a) * xs.token);
    }
    if (t + M <= t1) {
#pragma unroll
      for (int a = 0; a < M; ++a) form(cur[a], t + a);
    } else {
#pragma unroll
      for (int a = 0; a < M; ++a) {
        if (t + a >= t1) break;
        form(cur[a], t + a);
      }
    }
  }
  if (fin && t1 == L) {   // the run that ends the sequence holds the last W - 1 inputs
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      *reinterpret_cast<Raw*>(fin + (b * (W - 1) + k) * C + c) = win[k];
  }
}

// Gradients.  A run of tokens [t0, t1) forms dx there (and, at the sequence's
// start, the W - 1 rows of dinit) and adds its tokens to dw and dbias, which
// needs du up to W - 1 tokens past the run.  The runs of a workgroup add up
// their dw and dbias in LDS, in order, and leave one row of part sums
// [W + 1][C] in the workspace; conv_reduce_kernel adds those rows in order, so the
// same call gives the same bits.
template <typename T, int V, int W, bool ACT>
__global__ void __launch_bounds__(kConvThreads)
conv_bwd_kernel(const T* __restrict__ x, Strides xs, const float* __restrict__ w,
                const float* __restrict__ bias, const T* __restrict__ init, ConvParts dy,
                const T* __restrict__ dfin, T* __restrict__ dx, Strides dxs, T* __restrict__ dinit,
                float* __restrict__ part, int64_t L, int64_t C, ConvTiles tiles,
                int lc_log, int64_t run) {
  const int lanes = 1 << lc_log;
  const int lane = threadIdx.x & (lanes - 1);
  const int row = threadIdx.x >> lc_log;
  const int rows = blockDim.x >> lc_log;
  int64_t ix, iy;
  if (!conv_tile(tiles, &ix, &iy)) return;
  const int64_t c0 = ix * lanes * V;   // the workgroup's first channel
  const int64_t c = c0 + lane * V;
  const int64_t t0 = (iy * rows + row) * run;
  const int64_t b = blockIdx.y;
  typedef typename RawV<T, V>::type Raw;
  float dw[W][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][v] = 0.0f;
  }
  if (c < C && t0 < L) {
    const int64_t t1 = t0 + run < L ? t0 + run : L;
    float wt[W][V], bs[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bs[v] = bias ? bias[c + v] : 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) wt[k][v] = w[(c + v) * W + k];
    }
    const T* xp = x + b * xs.batch + c;
    T* dxp = dx + b * dxs.batch + c;
    const PartRow<const T> g = part_of<const T>(dy, b, L, c);
    float xw[W - 1][V], gw[W - 1][V];   // the W - 1 rows of x and of du before the current one
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int64_t t = t0 - (W - 1) + k;
      Raw r = zero_raw<T, V>();
      if (t >= 0)
        r = load_raw<T, V>(xp + t * xs.token);
      else if (init)
        r = load_raw<T, V>(init + (b * (W - 1) + (t + W - 1)) * C + c);
      widen<T, V>(r, xw[k]);
#pragma unroll
      for (int v = 0; v < V; ++v) gw[k][v] = 0.0f;
    }
    const int64_t first = t0 == 0 ? -(int64_t)(W - 1) : t0;   // first row of dx (or dinit) formed here
    const int64_t end = t1 + W - 1;                            // rows of x and dy looked at
    constexpr int M = kBwdAhead;
    Raw xn[M], gn[M];
    auto load = [&](int64_t t) {
#pragma unroll
      for (int a = 0; a < M; ++a)
        if (t + a < L && t + a < end) {
          xn[a] = load_raw<T, V>(xp + (t + a) * xs.token);
          gn[a] = load_raw<T, V>(g.p + (t + a) * g.ld);
        }
    };
    // Row t: du there (zero where not IN: past the last token), the sums of dw and
    // dbias (ADD: rows of this run), and row s = t - (W - 1) of dx, which takes du[s ..
    // s + W - 1] = gw[0 .. W - 2], du (OUT; before the first token it is dinit's).
    auto form = [&](auto IN, auto ADD, auto OUT, const Raw& xr, const Raw& gr, int64_t t) {
      float xc[V], du[V];
      if constexpr (decltype(IN)::value) {
        float gc[V];
        widen<T, V>(xr, xc);
        widen<T, V>(gr, gc);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float u = fmaf(wt[W - 1][v], xc[v], bs[v]);
#pragma unroll
          for (int k = 0; k < W - 1; ++k) u = fmaf(wt[k][v], xw[k][v], u);
          du[v] = ACT ? gc[v] * silu_slope(u, sigmoid_f32(u)) : gc[v];
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) xc[v] = du[v] = 0.0f;
      }
      if constexpr (decltype(ADD)::value) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          db[v] += du[v];
          dw[W - 1][v] = fmaf(du[v], xc[v], dw[W - 1][v]);
#pragma unroll
          for (int k = 0; k < W - 1; ++k) dw[k][v] = fmaf(du[v], xw[k][v], dw[k][v]);
        }
      }
      if constexpr (decltype(OUT)::value) {
        const int64_t s = t - (W - 1);
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o[v] = wt[0][v] * du[v];
#pragma unroll
          for (int k = 0; k < W - 1; ++k) o[v] = fmaf(wt[W - 1 - k][v], gw[k][v], o[v]);
        }
        const int64_t f = s - (L - (W - 1));   // this input's row in the final state
        if (f >= 0 && dfin) {
          float d[V];
          load_v<V>(dfin + (b * (W - 1) + f) * C + c, d);
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] += d[v];
        }
        if (s >= 0)
          store_v<V>(dxp + s * dxs.token, o);
        else if (dinit)
          store_v<V>(dinit + (b * (W - 1) + s + (W - 1)) * C + c, o);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) {
          xw[k][v] = xw[k + 1][v];
          gw[k][v] = gw[k + 1][v];
        }
        xw[W - 2][v] = xc[v];
        gw[W - 2][v] = du[v];
      }
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    // the run's own rows; the first W - 1 complete no row of dx, but for the sequence's
    // first run, whose dinit they are
#pragma unroll
    for (int a = 0; a < M; ++a) xn[a] = gn[a] = zero_raw<T, V>();
    load(t0);
    for (int64_t tt = t0; tt < end; tt += M) {
      Raw xr[M], gr[M];
#pragma unroll
      for (int a = 0; a < M; ++a) {
        xr[a] = xn[a];
        gr[a] = gn[a];
      }
      load(tt + M);
      if (tt >= t0 + W - 1 && tt + M <= t1) {
#pragma unroll
        for (int a = 0; a < M; ++a) form(yes, yes, yes, xr[a], gr[a], tt + a);
      } else {
#pragma unroll
        for (int a = 0; a < M; ++a) {
          const int64_t t = tt + a;
          if (t >= end) break;
          const bool out = t - (W - 1) >= first;
          if (t < t1) {
            if (out) form(yes, yes, yes, xr[a], gr[a], t);
            else form(yes, yes, no, xr[a], gr[a], t);
          } else if (t < L) {
            if (out) form(yes, no, yes, xr[a], gr[a], t);
            else form(yes, no, no, xr[a], gr[a], t);
          } else {
            if (out) form(no, no, yes, xr[a], gr[a], t);
            else form(no, no, no, xr[a], gr[a], t);
          }
        }
      }
    }
  }
  __shared__ float sums[kConvThreads][V];
  float* out = part + (b * tiles.by + iy) * (W + 1) * C;
#pragma unroll
  for (int k = 0; k <= W; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) sums[threadIdx.x][v] = k < W ? dw[k < W ? k : 0][v] : db[v];
    __syncthreads();
    for (int i = threadIdx.x; i < lanes * V; i += blockDim.x) {
      const int64_t cc = c0 + i;
      if (cc < C) {
        float s = 0.0f;
        for (int r = 0; r < rows; ++r) s += sums[r * lanes + i / V][i % V];
        out[k * C + cc] = s;
      }
    }
    __syncthreads();
  }
}

// dweight [C, W] and dbias [C] from `n` rows of part sums [W + 1][C].
__global__ void __launch_bounds__(256)
conv_reduce_kernel(const float* __restrict__ part, int64_t n, int64_t C, int W,
                   float* __restrict__ dw, float* __restrict__ db) {
  const int64_t cols = (W + 1) * C, i = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
  const float v = column_sum(i < cols ? part + i : nullptr, n, cols);
  if (threadIdx.x >= 32 || i >= cols) return;
  const int64_t k = i / C, c = i % C;
  if (k < W)
    dw[c * W + k] = v;
  else if (db)
    db[c] = v;
}

// ---- host ----

namespace {

struct ConvGrid {
  int lc_log, rows;     // lanes along the channels (their log2) and runs per workgroup
  int64_t run, bx, by;  // tokens per run; workgroups along the channels and the tokens
  int threads() const { return rows << lc_log; }
};

// Lanes along the channels and tokens per run.  Runs are long (fewer
// overlapping rows) as long as the launch keeps `enough` waves.
ConvGrid conv_grid(int64_t batch, int64_t L, int64_t C, int V, int longest, int64_t enough) {
  ConvGrid g;
  const int64_t cv = (C + V - 1) / V;
  g.lc_log = 0;
  while (g.lc_log < 6 && (int64_t(1) << g.lc_log) < cv) ++g.lc_log;
  g.bx = (cv + (int64_t(1) << g.lc_log) - 1) >> g.lc_log;
  g.run = longest;
  while (g.run > 4 && batch * g.bx * (int64_t(1) << g.lc_log) * ((L + g.run - 1) / g.run) < enough * 64)
    g.run /= 2;
  g.by = 1;
  g.rows = kConvThreads >> g.lc_log;
  const int64_t runs = (L + g.run - 1) / g.run;
  while (g.rows > 1 && g.rows / 2 >= runs && g.threads() > 64) g.rows /= 2;
  g.by = (runs + g.rows - 1) / g.rows;
  return g;
}
ConvGrid conv_bwd_grid(int64_t batch, int64_t L, int64_t C, int V) {
  return conv_grid(batch, L, C, V, 64, 2048);
}

}  // namespace

size_t conv_bwd_workspace(int64_t batch, int64_t L, int64_t C, int W) {
  // either vector width may be taken, by the call's pointers and strides
  size_t most = 0;
  for (int V : {1, 4}) {
    const ConvGrid g = conv_bwd_grid(batch, L, C, V);
    const size_t n = size_t(batch) * g.by * (W + 1) * C * sizeof(float);
    if (n > most) most = n;
  }
  return most;
}

// Every launch has fewer than 2^32 threads along x (V = 1 has the most).
int conv_grid_ok(int64_t batch, int64_t L, int64_t C) {
  if (batch > 65535 || C > (1 << 24) || L > (int64_t(1) << 32)) return 0;
  const ConvGrid g = conv_grid(batch, L, C, 1, 16, 4096);
  return ((__int128)g.bx * g.by + 7) * kConvThreads < (int64_t(1) << 32);
}

template <typename T, int V>
static hipError_t conv_fwd_v(const ConvArgs& a, hipStream_t stream) {
  ConvGrid g = conv_grid(a.batch, a.L, a.C, V, 16, 4096);
  if (a.one_run) {   // the state is updated in place: one thread per (b, c) reads and writes it
    g.run = a.L;
    g.by = 1;
    g.rows = g.lc_log < 6 ? 64 >> g.lc_log : 1;
  }
  const ConvParts y{{a.y[0], a.y[1], a.y[2]}, {a.end[0], a.end[1], a.end[2]}};
  const dim3 grid((unsigned)((g.bx * g.by + 7) / 8 * 8), (unsigned)a.batch);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(g.threads()), 0, stream, static_cast<const T*>(a.x),
                       Strides{a.xs[0], a.xs[1]}, a.w, a.bias, static_cast<const T*>(a.init), y,
                       static_cast<T*>(a.fin), a.L, a.C, ConvTiles{g.bx, g.by}, g.lc_log, g.run);
  };
  if (a.W == 2) a.silu ? go(conv_fwd_kernel<T, V, 2, true>) : go(conv_fwd_kernel<T, V, 2, false>);
  else if (a.W == 3) a.silu ? go(conv_fwd_kernel<T, V, 3, true>) : go(conv_fwd_kernel<T, V, 3, false>);
  else a.silu ? go(conv_fwd_kernel<T, V, 4, true>) : go(conv_fwd_kernel<T, V, 4, false>);
  return hipGetLastError();
}

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t stream) {
  if (a.bf16)
    return a.vec ? conv_fwd_v<bf16, 4>(a, stream) : conv_fwd_v<bf16, 1>(a, stream);
  return a.vec ? conv_fwd_v<float, 4>(a, stream) : conv_fwd_v<float, 1>(a, stream);
}

template <typename T, int V>
static hipError_t conv_bwd_v(const ConvArgs& a, hipStream_t stream) {
  const ConvGrid g = conv_bwd_grid(a.batch, a.L, a.C, V);
  const ConvParts dy{{a.y[0], a.y[1], a.y[2]}, {a.end[0], a.end[1], a.end[2]}};
  const dim3 grid((unsigned)((g.bx * g.by + 7) / 8 * 8), (unsigned)a.batch);
  float* part = static_cast<float*>(a.workspace);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(g.threads()), 0, stream, static_cast<const T*>(a.x),
                       Strides{a.xs[0], a.xs[1]}, a.w, a.bias, static_cast<const T*>(a.init), dy,
                       static_cast<const T*>(a.dfin), static_cast<T*>(a.dx),
                       Strides{a.dxs[0], a.dxs[1]}, static_cast<T*>(a.dinit), part, a.L,
                       a.C, ConvTiles{g.bx, g.by}, g.lc_log, g.run);
  };
  if (a.W == 2) a.silu ? go(conv_bwd_kernel<T, V, 2, true>) : go(conv_bwd_kernel<T, V, 2, false>);
  else if (a.W == 3) a.silu ? go(conv_bwd_kernel<T, V, 3, true>) : go(conv_bwd_kernel<T, V, 3, false>);
  else a.silu ? go(conv_bwd_kernel<T, V, 4, true>) : go(conv_bwd_kernel<T, V, 4, false>);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t cols = (a.W + 1) * a.C;
  hipLaunchKernelGGL(conv_reduce_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, stream,
                     part, a.batch * g.by, a.C, (int)a.W, a.dw, a.db);
  return hipGetLastError();
}

hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t stream) {
  if (a.bf16)
    return a.vec ? conv_bwd_v<bf16, 4>(a, stream) : conv_bwd_v<bf16, 1>(a, stream);
  return a.vec ? conv_bwd_v<float, 4>(a, stream) : conv_bwd_v<float, 1>(a, stream);
}

}  // namespace ssd
