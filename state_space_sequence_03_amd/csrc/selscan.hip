// selscan.hip -- the selective scan, with a decay of its own for every channel and
// state, over prompts and for single tokens.
//
// For every batch b, channel c (in group g = c / (D / G)) and state n:
//     h_t = exp(dt_t A[c, n]) h_{t-1} + dt_t x_t B_t[g, n]
//     s_t = sum_n C_t[g, n] h_t[n] + D[c] x_t,    y_t = s_t z_t sigmoid(z_t)
// (y = s without z).  The decay differs in every (c, n), so no matrix product
// evaluates a chunk, as it does for one decay per head: each (t, c, n) costs a
// product, an exp2, a product and two fmas on the vector ALU, which is the bound
// (7 issue slots of ALU work per 16th of ~8 bytes moved, at dstate 16).
//
// One wave walks tokens with its channels x states tile in registers.  Where
// batch x channels do not fill the chip, the sequence is cut into K chunks:
// selscan_kernel<states> runs chunks 0 .. K-2 from a zero state and leaves their end
// states and step-size sums, selscan_pass_kernel chains them (the decay of
// a whole chunk is exp(A sum dt)), and selscan_kernel<out> runs every chunk again from
// its true start state.  Only then is a decay formed twice.
#include <type_traits>

#include "layer_host.hpp"
#include "selscan_device.hpp"

namespace ssd {

constexpr int kScanThreads = 256;
constexpr int kScanTile = 32;    // tokens of B and C staged in LDS at a time
constexpr int kScanAhead = 8;    // tokens loaded ahead

enum { kStates = 0, kOut = 1, kBoth = 2 };

// What a wave of the chunked kernels reads and writes.  kStates: end states of
// chunks.  kOut: y (and the final state).  kBoth: end states, and the gradient that
// chunk k's own outputs send to its start state (R = sum_t (prod_{s<=t} a_s)
// ds_t C_t), for the backward pass.
template <typename T>
struct ScanIo {
  const T *x, *dt;
  const float* A;
  const T* B;
  Strides bs;
  const T* C;
  Strides cs;
  const float* Dv;
  const T* z;
  Strides zs;
  const T* dy;
  const float* init;
  float* H;       // [batch][K][D][NP]: start state of each chunk
  float* R;       // [batch][K][D][NP]: gradient at each chunk's end
  float* sumdt;   // [batch][K][D]
  T* y;
  float* fin;
  DtXform xf;
};

template <typename T, int RN, int MODE, bool GATE>
__global__ void __launch_bounds__(kScanThreads)
selscan_kernel(ScanIo<T> io, ScanShape sh) {
  constexpr int NP = 4 * RN, CW = 256 / RN;   // padded states, channels per wave
  constexpr int PER = kScanTile * NP / kScanThreads;
  __shared__ float sB[2][kScanTile][NP];
  __shared__ float sC[MODE == kStates ? 1 : 2][kScanTile][NP];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int64_t tile = blockIdx.x % (sh.tiles * sh.G);
  const int64_t k = blockIdx.x / (sh.tiles * sh.G);
  const int64_t b = blockIdx.y;
  const int64_t g = tile / sh.tiles;
  const int64_t base = ((tile % sh.tiles) * (kScanThreads / kWave) + wave) * CW;
  const bool live = base < sh.Dg;             // whole waves past the group only stage
  const int nl = lane % RN, dl = lane / RN;
  const int n0 = 4 * nl;
  const int64_t own = base + dl * 4 + (lane & 3);   // the channel this lane prepares
  const int64_t c = g * sh.Dg + (own < sh.Dg ? own : sh.Dg - 1);
  const bool mine = own < sh.Dg && nl < 4;
  const int64_t t0 = k * sh.T, t1 = t0 + sh.T < sh.L ? t0 + sh.T : sh.L;

  float A2[4][4], h[4][4], P[4][4], R[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t lc = base + dl * 4 + j;
    const int64_t cj = g * sh.Dg + (lc < sh.Dg ? lc : sh.Dg - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + i;
      A2[j][i] = n < sh.N ? io.A[cj * sh.N + n] * kLog2e : 0.0f;
      h[j][i] = 0.0f;
      P[j][i] = 1.0f;
      R[j][i] = 0.0f;
      if (k == 0) {
        if (io.init && n < sh.N) h[j][i] = io.init[(b * sh.D + cj) * sh.N + n];
      } else if (MODE == kOut) {
        h[j][i] = io.H[((b * sh.K + k) * sh.D + cj) * NP + n];
      }
    }
  }
  const DtLane f = dt_lane(io.xf, c);
  const float Dc = MODE == kOut && io.Dv ? io.Dv[c] : 0.0f;
  float sum = 0.0f;

  const T* xp = io.x + b * sh.L * sh.D + c;
  const T* dp = io.dt + b * sh.L * sh.D + c;
  const T* gp = MODE == kBoth ? io.dy + b * sh.L * sh.D + c : nullptr;
  const T* zp = GATE ? io.z + b * io.zs.batch + c : nullptr;
  const T* Bp = io.B + b * io.bs.batch + g * sh.N;
  const T* Cp = MODE == kStates ? nullptr : io.C + b * io.cs.batch + g * sh.N;

  // B and C of one tile, held in registers from their load to their place in LDS
  float rb[PER], rc[MODE == kStates ? 1 : PER];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int i = q * kScanThreads + tid;
      const int64_t tok = t + i / NP;
      const int n = i % NP;
      const bool in = tok < t1 && n < sh.N;
      rb[q] = in ? to_f32(Bp[tok * io.bs.token + n]) : 0.0f;
      if constexpr (MODE != kStates) rc[q] = in ? to_f32(Cp[tok * io.cs.token + n]) : 0.0f;
    }
  };
  auto place = [&](int buf) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int i = q * kScanThreads + tid;
      sB[buf][i / NP][i % NP] = rb[q];
      if constexpr (MODE != kStates) sC[buf][i / NP][i % NP] = rc[q];
    }
  };

  T xr[kScanAhead], dr[kScanAhead], zr[kScanAhead], gr[kScanAhead];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int u = 0; u < kScanAhead; ++u) {
      const int64_t tok = t + u < t1 ? t + u : t1 - 1;
      xr[u] = xp[tok * sh.D];
      dr[u] = dp[tok * sh.D];
      if constexpr (GATE && MODE != kStates) zr[u] = zp[tok * io.zs.token];
      if constexpr (MODE == kBoth) gr[u] = gp[tok * sh.D];
    }
  };

  fetch(t0);
  load(t0);
  place(0);
  __syncthreads();
  int buf = 0;
  for (int64_t tt = t0; tt < t1; tt += kScanTile, buf ^= 1) {
    const bool more = tt + kScanTile < t1;
    if (more) fetch(tt + kScanTile);
    if (live) {
      for (int s = 0; s < kScanTile && tt + s < t1; s += kScanAhead) {
        const int64_t ts = tt + s;
        float xv[kScanAhead], dv[kScanAhead], zv[kScanAhead], gv[kScanAhead];
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u) {
          xv[u] = to_f32(xr[u]);
          dv[u] = to_f32(dr[u]);
          zv[u] = GATE && MODE != kStates ? to_f32(zr[u]) : 0.0f;
          gv[u] = MODE == kBoth ? to_f32(gr[u]) : 0.0f;
        }
        if (ts + kScanAhead < t1) load(ts + kScanAhead);
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u) {
          const bool in = ts + u < t1;
          const float d = in ? dt_value(f, dv[u]) : 0.0f;
          const float dx = in ? d * xv[u] : 0.0f;
          float gate = 1.0f;
          if constexpr (GATE && MODE != kStates) gate = zv[u] * sigmoid_f32(zv[u]);
          const float ds = MODE == kBoth && in ? gv[u] * gate : 0.0f;
          if constexpr (MODE != kOut) sum += d;
          const floatx4 Bv = *reinterpret_cast<const floatx4*>(&sB[buf][s + u][n0]);
          floatx4 Cv = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (MODE != kStates) Cv = *reinterpret_cast<const floatx4*>(&sC[buf][s + u][n0]);
          float yp[4];
          auto channel = [&](auto J) {
            constexpr int j = decltype(J)::value;
            const float dj = quad_bcast<j>(d), xj = quad_bcast<j>(dx);
            const float sj = MODE == kBoth ? quad_bcast<j>(ds) : 0.0f;
            yp[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = fast_exp2(dj * A2[j][i]);
              h[j][i] = fmaf(a, h[j][i], xj * Bv[i]);
              if constexpr (MODE == kOut) yp[j] = fmaf(Cv[i], h[j][i], yp[j]);
              if constexpr (MODE == kBoth) {
                P[j][i] *= a;
                R[j][i] = fmaf(P[j][i], sj * Cv[i], R[j][i]);
              }
            }
          };
          channel(std::integral_constant<int, 0>{});
          channel(std::integral_constant<int, 1>{});
          channel(std::integral_constant<int, 2>{});
          channel(std::integral_constant<int, 3>{});
          if constexpr (MODE == kOut) {
            float o = quads_sum<RN>(quad_fold(yp, lane));
            o = fmaf(Dc, xv[u], o) * gate;
            if (in && mine) io.y[(b * sh.L + ts + u) * sh.D + c] = to_io<T>(o);
          }
        }
      }
    }
    if (more) place(buf ^ 1);
    __syncthreads();
  }
  if (!live) return;
  const bool last = k == sh.K - 1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t lc = base + dl * 4 + j;
    if (lc >= sh.Dg) continue;
    const int64_t cj = g * sh.Dg + lc;
    if constexpr (MODE == kOut) {
      if (last && io.fin)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < sh.N) io.fin[(b * sh.D + cj) * sh.N + n0 + i] = h[j][i];
    } else {
      if (!last)
        *reinterpret_cast<floatx4*>(io.H + ((b * sh.K + k + 1) * sh.D + cj) * NP + n0) =
            floatx4{h[j][0], h[j][1], h[j][2], h[j][3]};
      if constexpr (MODE == kBoth)
        if (k > 0)
          *reinterpret_cast<floatx4*>(io.R + ((b * sh.K + k - 1) * sh.D + cj) * NP + n0) =
              floatx4{R[j][0], R[j][1], R[j][2], R[j][3]};
    }
  }
  if constexpr (MODE != kOut)
    if (mine) io.sumdt[(b * sh.K + k) * sh.D + c] = sum;
}

// Chains the chunks, one thread per (b, c, n).  Forwards, slot k of H holds chunk
// k - 1's end state from a zero start (chunk 0's from the caller's state) and
// becomes chunk k's start state; backwards, slot k of R holds what chunk k + 1
// sends to its start and becomes the gradient at chunk k's end.
__global__ void __launch_bounds__(256)
selscan_pass_kernel(float* __restrict__ H, const float* __restrict__ A,
                    const float* __restrict__ sumdt, const float* __restrict__ last, int64_t batch,
                    int64_t K, int64_t D, int64_t N, int NP, int reverse) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= batch * D * NP) return;
  const int64_t n = i % NP, c = i / NP % D, b = i / NP / D;
  const float a2 = n < N ? A[c * N + n] * kLog2e : 0.0f;
  float* p = H + (b * K * D + c) * NP + n;
  const float* sp = sumdt + b * K * D + c;
  if (!reverse) {
    float run = p[D * NP];
    for (int64_t k = 2; k < K; ++k) {
      run = fmaf(fast_exp2(a2 * sp[(k - 1) * D]), run, p[k * D * NP]);
      p[k * D * NP] = run;
    }
  } else {
    float run = last && n < N ? last[(b * D + c) * N + n] : 0.0f;
    p[(K - 1) * D * NP] = run;
    for (int64_t k = K - 2; k >= 0; --k) {
      run = fmaf(fast_exp2(a2 * sp[(k + 1) * D]), run, p[k * D * NP]);
      p[k * D * NP] = run;
    }
  }
}

// Single tokens: the recurrence from a resident state, in place.  Bound by the
// state's bytes (8 per element against ~8 slots of ALU work), so every lane holds
// four consecutive states of one channel and takes all of the call's tokens.
template <typename T, int RN, bool GATE, bool VEC>
__global__ void __launch_bounds__(256)
selscan_step_kernel(float* __restrict__ state, const T* __restrict__ x, const T* __restrict__ dt,
                    const float* __restrict__ A, const T* __restrict__ B, Strides bs,
                    const T* __restrict__ C, Strides cs, const float* __restrict__ Dv,
                    const T* __restrict__ z, Strides zs, T* __restrict__ y, DtXform xf, int64_t batch,
                    int64_t L, int64_t D, int64_t N, int64_t Dg) {
  const int nl = threadIdx.x % RN;
  const int n0 = 4 * nl;
  const int64_t item = (int64_t)blockIdx.x * (256 / RN) + threadIdx.x / RN;
  const bool live = item < batch * D;
  const int64_t b = live ? item / D : 0, c = live ? item % D : 0;
  const int64_t g = c / Dg;
  float* sp = state + (b * D + c) * N + n0;
  const float* ap = A + c * N + n0;
  float h[4], A2[4];
  if constexpr (VEC) {
    const bool in = n0 < N;
    const floatx4 hv = in ? *reinterpret_cast<const floatx4*>(sp) : floatx4{0, 0, 0, 0};
    const floatx4 av = in ? *reinterpret_cast<const floatx4*>(ap) : floatx4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = hv[i];
      A2[i] = av[i] * kLog2e;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = n0 + i < N ? sp[i] : 0.0f;
      A2[i] = n0 + i < N ? ap[i] * kLog2e : 0.0f;
    }
  }
  const DtLane f = dt_lane(xf, c);
  const float Dc = Dv ? Dv[c] : 0.0f;
  const T* Bp = B + b * bs.batch + g * N + n0;
  const T* Cp = C + b * cs.batch + g * N + n0;
  for (int64_t t = 0; t < L; ++t) {
    const int64_t at = (b * L + t) * D + c;
    const float xv = to_f32(x[at]);
    const float d = dt_value(f, to_f32(dt[at]));
    const float dx = d * xv;
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = n0 + i < N;
      const float bv = in ? to_f32(Bp[t * bs.token + i]) : 0.0f;
      const float cv = in ? to_f32(Cp[t * cs.token + i]) : 0.0f;
      h[i] = fmaf(fast_exp2(d * A2[i]), h[i], dx * bv);
      part = fmaf(cv, h[i], part);
    }
#pragma unroll
    for (int off = RN / 2; off >= 1; off >>= 1) part += __shfl_xor(part, off, kWave);
    float o = fmaf(Dc, xv, part);
    if constexpr (GATE) {
      const float zv = to_f32(z[b * zs.batch + t * zs.token + c]);
      o *= zv * sigmoid_f32(zv);
    }
    if (live && nl == 0) y[at] = to_io<T>(o);
  }
  if (!live) return;
  if constexpr (VEC) {
    if (n0 < N) *reinterpret_cast<floatx4*>(sp) = floatx4{h[0], h[1], h[2], h[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < N) sp[i] = h[i];
  }
}

// ---- host ----

// Chunks of the forward pass.  One chunk where its waves fill the chip;
// otherwise as many as give about three waves per SIMD, of at least 64 tokens.
ScanShape selscan_fwd_shape(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
  ScanShape s;
  const int rn = selscan_rn(N);
  const int64_t cw = 256 / rn, per = cw * (kScanThreads / kWave);
  s.L = L; s.D = D; s.N = N; s.G = G; s.Dg = D / G;
  s.tiles = (s.Dg + per - 1) / per;
  const int64_t waves = batch * G * ((s.Dg + cw - 1) / cw);
  s.K = 1;
  s.T = L;
  if (waves < 640 && L > 128) {
    int64_t k = (3072 + waves - 1) / waves;
    if (k > L / 64) k = L / 64;
    s.T = ((L + k - 1) / k + kScanTile - 1) / kScanTile * kScanTile;
    s.K = (L + s.T - 1) / s.T;
  }
  return s;
}

static size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
size_t selscan_state_bytes(int64_t batch, const ScanShape& s) {
  return up256(size_t(batch) * s.K * s.D * 4 * selscan_rn(s.N) * sizeof(float));
}
size_t selscan_sum_bytes(int64_t batch, const ScanShape& s) {
  return up256(size_t(batch) * s.K * s.D * sizeof(float));
}

size_t selscan_fwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
  const ScanShape s = selscan_fwd_shape(batch, L, D, N, G);
  return s.K == 1 ? 0 : selscan_state_bytes(batch, s) + selscan_sum_bytes(batch, s);
}

template <typename T>
static ScanIo<T> scan_io(const ScanArgs& a) {
  ScanIo<T> io{};
  io.x = static_cast<const T*>(a.x);
  io.dt = static_cast<const T*>(a.dt);
  io.A = a.A;
  io.B = static_cast<const T*>(a.B);
  io.bs = {a.bs[0], a.bs[1]};
  io.C = static_cast<const T*>(a.C);
  io.cs = {a.cs[0], a.cs[1]};
  io.Dv = a.Dv;
  io.z = static_cast<const T*>(a.z);
  io.zs = {a.zs[0], a.zs[1]};
  io.dy = static_cast<const T*>(a.dy);
  io.init = a.init;
  io.y = static_cast<T*>(a.y);
  io.fin = a.fin;
  io.xf = a.xf ? *a.xf : DtXform{nullptr, 0, -INFINITY, INFINITY};
  return io;
}

template <typename T, int RN, int MODE>
static void launch_scan(const ScanIo<T>& io, const ScanShape& s, int64_t batch, int64_t chunks,
                        hipStream_t stream) {
  const dim3 grid((unsigned)(s.tiles * s.G * chunks), (unsigned)batch);
  if constexpr (MODE != kStates) {
    if (io.z) {
      hipLaunchKernelGGL((selscan_kernel<T, RN, MODE, true>), grid, dim3(kScanThreads), 0, stream, io, s);
      return;
    }
  }
  hipLaunchKernelGGL((selscan_kernel<T, RN, MODE, false>), grid, dim3(kScanThreads), 0, stream, io, s);
}

void launch_selscan_pass(float* H, const float* A, const float* sumdt, const float* last,
                         int64_t batch, const ScanShape& s, int reverse, hipStream_t stream) {
  const int np = 4 * selscan_rn(s.N);
  hipLaunchKernelGGL(selscan_pass_kernel, dim3((unsigned)((batch * s.D * np + 255) / 256)), dim3(256), 0,
                     stream, H, A, sumdt, last, batch, s.K, s.D, s.N, np, reverse);
}

template <typename T, int RN>
static hipError_t fwd_rn(const ScanArgs& a, hipStream_t stream) {
  const ScanShape s = selscan_fwd_shape(a.batch, a.L, a.D, a.N, a.G);
  ScanIo<T> io = scan_io<T>(a);
  if (s.K > 1) {
    io.H = static_cast<float*>(a.workspace);
    io.sumdt = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + selscan_state_bytes(a.batch, s));
    launch_scan<T, RN, kStates>(io, s, a.batch, s.K - 1, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (s.K > 2) {
      launch_selscan_pass(io.H, a.A, io.sumdt, nullptr, a.batch, s, 0, stream);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  launch_scan<T, RN, kOut>(io, s, a.batch, s.K, stream);
  return hipGetLastError();
}

template <typename T>
static hipError_t fwd_t(const ScanArgs& a, hipStream_t stream) {
  const int rn = selscan_rn(a.N);
  if (rn == 4) return fwd_rn<T, 4>(a, stream);
  if (rn == 8) return fwd_rn<T, 8>(a, stream);
  return fwd_rn<T, 16>(a, stream);
}

hipError_t launch_selscan_fwd(const ScanArgs& a, hipStream_t stream) {
  return a.bf16 ? fwd_t<bf16>(a, stream) : fwd_t<float>(a, stream);
}

// First stage of the backward pass: every chunk's end state and the gradient it sends
// to its start, then both chains.
template <typename T, int RN>
static hipError_t both_rn(const ScanArgs& a, const ScanShape& s, float* H, float* R, float* sumdt,
                          hipStream_t stream) {
  ScanIo<T> io = scan_io<T>(a);
  io.H = H;
  io.R = R;
  io.sumdt = sumdt;
  if (s.K > 1) {
    launch_scan<T, RN, kBoth>(io, s, a.batch, s.K, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (s.K > 2) launch_selscan_pass(H, a.A, sumdt, nullptr, a.batch, s, 0, stream);
  launch_selscan_pass(R, a.A, sumdt, a.dfin, a.batch, s, 1, stream);
  return hipGetLastError();
}
hipError_t launch_selscan_both(const ScanArgs& a, const ScanShape& s, float* H, float* R,
                               float* sumdt, hipStream_t stream) {
  const int rn = selscan_rn(a.N);
  if (a.bf16)
    return rn == 4 ? both_rn<bf16, 4>(a, s, H, R, sumdt, stream)
           : rn == 8 ? both_rn<bf16, 8>(a, s, H, R, sumdt, stream)
                     : both_rn<bf16, 16>(a, s, H, R, sumdt, stream);
  return rn == 4 ? both_rn<float, 4>(a, s, H, R, sumdt, stream)
         : rn == 8 ? both_rn<float, 8>(a, s, H, R, sumdt, stream)
                   : both_rn<float, 16>(a, s, H, R, sumdt, stream);
}

template <typename T, int RN, bool GATE>
static hipError_t step_g(const ScanArgs& a, hipStream_t stream) {
  const int64_t items = a.batch * a.D;
  const dim3 grid((unsigned)((items + 256 / RN - 1) / (256 / RN)));
  const DtXform xf = a.xf ? *a.xf : DtXform{nullptr, 0, -INFINITY, INFINITY};
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a.state, static_cast<const T*>(a.x),
                       static_cast<const T*>(a.dt), a.A, static_cast<const T*>(a.B),
                       Strides{a.bs[0], a.bs[1]}, static_cast<const T*>(a.C),
                       Strides{a.cs[0], a.cs[1]}, a.Dv, static_cast<const T*>(a.z),
                       Strides{a.zs[0], a.zs[1]}, static_cast<T*>(a.y), xf, a.batch, a.L, a.D, a.N,
                       a.D / a.G);
  };
  if (a.N % 4 == 0) go(selscan_step_kernel<T, RN, GATE, true>);
  else go(selscan_step_kernel<T, RN, GATE, false>);
  return hipGetLastError();
}
template <typename T>
static hipError_t step_t(const ScanArgs& a, hipStream_t stream) {
  const int rn = selscan_rn(a.N);
  if (rn == 4) return a.z ? step_g<T, 4, true>(a, stream) : step_g<T, 4, false>(a, stream);
  if (rn == 8) return a.z ? step_g<T, 8, true>(a, stream) : step_g<T, 8, false>(a, stream);
  return a.z ? step_g<T, 16, true>(a, stream) : step_g<T, 16, false>(a, stream);
}
hipError_t launch_selscan_step(const ScanArgs& a, hipStream_t stream) {
  return a.bf16 ? step_t<bf16>(a, stream) : step_t<float>(a, stream);
}

}  // namespace ssd
