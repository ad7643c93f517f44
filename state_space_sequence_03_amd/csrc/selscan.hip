// selscan.hip -- the selective scan, with a decay of its own for every channel and
// state, over prompts and for single tokens.
//
// For every batch b, channel c (in group g = c / (D / G)) and state n:
//     h_t = exp(dt_t A[c, n]) h_{t-1} + dt_t x_t B_t[g, n]
//     s_t = sum_n C_t[g, n] h_t[n] + D[c] x_t,    y_t = s_t z_t sigmoid(z_t)
// (y = s without z).  The decay differs in every (c, n), so no matrix product
// evaluates a chunk, as it does for one decay per head: each (t, c, n) costs a
// product, an exp2, a product and two fmas on the vector ALU, which is the bound:
// a wave's exp2 takes 3.5 ns of its SIMD and the five together 9.4, at one wave
// per SIMD as at four, so 2048 tokens of 5120 channels x 16 states need 24 us of it
// against 16 us of HBM.
//
// One wave walks tokens with its channels x states tile in registers.  Where
// batch x channels do not fill the chip, the sequence is cut into K chunks:
// selscan_kernel<states> runs chunks 0 .. K-2 from a zero state and leaves their end
// states and step-size sums (the decay of a whole chunk is exp(A sum dt)), and
// selscan_kernel<out> chains those before its own chunk and runs it again from its
// true start state.  Only then is a decay formed twice: 44 us of the vector ALU at
// the size above, which takes 98 us.  Of those the exp2s cost 20, the step sizes 9,
// the chains 6 (each measured by leaving it out).
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
// ds_t C_t), for the backward pass, and the states every 8 tokens.
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
  float* ckpt;    // [batch][ceil(L / 8)][D][NP]: kBoth, states every 8 tokens from a zero start
  float* sumsub;  // [batch][ceil(L / 8)][D]: the chunk's step sizes before them
  T* y;
  float* fin;
  DtXform xf;
};

template <typename T, int RN, int SN, int MODE, bool GATE>
__global__ void __launch_bounds__(kScanThreads, 3)
selscan_kernel(ScanIo<T> io, ScanShape sh) {
  constexpr int NP = RN * SN, CW = 128 / RN;   // padded states, channels per wave
  constexpr int VS = SN % 4 == 0 ? 4 : 2;      // states per access
  constexpr int PER = kScanTile * NP / kScanThreads;
  constexpr int U = kScanAhead;
  __shared__ float sB[2][kScanTile][NP];
  __shared__ float sC[MODE == kStates ? 1 : 2][kScanTile][NP];
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int tiles = (int)sh.tiles, groups = (int)sh.G;
  const int tile = blockIdx.x % (tiles * groups);
  const int k = blockIdx.x / (tiles * groups);
  const int64_t b = blockIdx.y;
  const int g = tile / tiles;
  const int base = ((tile % tiles) * (kScanThreads / kWave) + wave) * CW;
  const int Dg = (int)sh.Dg, N = (int)sh.N;
  const bool live = base < Dg;             // whole waves past the group only stage
  const int nl = lane % RN, dl = lane / RN;
  const int n0 = SN * nl;
  const int own = base + dl * 2 + (lane & 1);   // the channel this lane prepares
  const int c = g * Dg + (own < Dg ? own : Dg - 1);
  const bool mine = own < Dg && nl < 2;
  // byte offsets of the lane's channel in U rows of x, dt, dy and y, and of z; lanes
  // that share a channel store the same value
  unsigned ox[U], oz[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    ox[u] = own < Dg ? (unsigned)(u * sh.D + c) * (unsigned)sizeof(T) : kOutside;
    oz[u] = GATE && own < Dg ? (unsigned)(u * io.zs.token + c) * (unsigned)sizeof(T) : kOutside;
  }
  // kBoth has no registers for them: each offset is formed from the first where it is used
  auto offset = [&](const unsigned* o, unsigned first, int u, int64_t stride) {
    return MODE == kBoth ? first + (unsigned)u * (unsigned)(stride * sizeof(T)) : o[u];
  };
  const int64_t t0 = k * sh.T;
  const int len = (int)(t0 + sh.T < sh.L ? sh.T : sh.L - t0);   // tokens of this chunk

  float A2[2][SN], h[2][SN], P[2][SN], R[2][SN];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lc = base + dl * 2 + j;
    const int64_t cj = g * Dg + (lc < Dg ? lc : Dg - 1);
#pragma unroll
    for (int i = 0; i < SN; ++i) {
      const int n = n0 + i;
      A2[j][i] = n < N ? io.A[cj * N + n] * kLog2e : 0.0f;
      h[j][i] = 0.0f;
      P[j][i] = 1.0f;
      R[j][i] = 0.0f;
      if (k == 0) {
        if (io.init && n < N) h[j][i] = io.init[(b * sh.D + cj) * N + n];
      }
    }
  }
  if constexpr (MODE == kOut) {
    // the start state: the chunks before this one, chained.  Slot m of H holds chunk
    // m - 1's end state from a zero start, chunk 0's from the caller's
    if (k > 0) {
      constexpr int M = 4;   // chunks loaded at a time
      for (int m0 = 1; m0 <= k; m0 += M) {
        float s[M][2], v[M][2][SN];
#pragma unroll
        for (int u = 0; u < M; ++u) {
          const int m = m0 + u <= k ? m0 + u : k;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int lc = base + dl * 2 + j;
            const int64_t at = (b * sh.K + m) * sh.D + g * Dg + (lc < Dg ? lc : Dg - 1);
            s[u][j] = io.sumdt[at - sh.D];
#pragma unroll
            for (int q = 0; q < SN; q += VS) load_v<VS>(io.H + at * NP + n0 + q, v[u][j] + q);
          }
        }
#pragma unroll
        for (int u = 0; u < M; ++u)
          if (m0 + u <= k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < SN; ++i)
                h[j][i] = m0 + u == 1 ? v[u][j][i]
                                      : fmaf(fast_exp2(A2[j][i] * s[u][j]), h[j][i], v[u][j][i]);
      }
    }
  }
  const DtLane f = dt_lane(io.xf, c);
  const float Dc = MODE == kOut && io.Dv ? io.Dv[c] : 0.0f;
  float sum = 0.0f;

  // rows: a uniform pointer to the chunk's first token, the lane's channel as offset
  const int64_t row = (b * sh.L + t0) * sh.D;
  const T* const xp = io.x + row;
  const T* const dp = io.dt + row;
  const T* const gp = MODE == kBoth ? io.dy + row : nullptr;
  T* const yp0 = MODE == kOut ? io.y + row : nullptr;
  const T* const zp = GATE ? io.z + b * io.zs.batch + t0 * io.zs.token : nullptr;
  const T* const Bp = io.B + b * io.bs.batch + t0 * io.bs.token + g * N;
  const T* const Cp = MODE == kStates ? nullptr : io.C + b * io.cs.batch + t0 * io.cs.token + g * N;

  unsigned oc[2];   // byte offsets of the lane's states in a row of checkpoints
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lc = base + dl * 2 + j;
    oc[j] = lc < Dg ? (unsigned)((g * Dg + lc) * NP + n0) * 4u : kOutside;
  }
  // B and C of one tile, held in registers from their load to their place in LDS, and
  // widened there: a conversion here would wait for them, and for the rows ahead
  T rb[PER], rc[MODE == kStates ? 1 : PER];
  auto fetch = [&](int t) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int i = q * kScanThreads + tid;
      const int tok = t + i / NP, n = i % NP;
      const bool in = tok < len && n < N;
      rb[q] = in ? Bp[tok * io.bs.token + n] : T(0.0f);
      if constexpr (MODE != kStates) rc[q] = in ? Cp[tok * io.cs.token + n] : T(0.0f);
    }
  };
  auto place = [&](int buf) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int i = q * kScanThreads + tid;
      sB[buf][i / NP][i % NP] = to_f32(rb[q]);
      if constexpr (MODE != kStates) sC[buf][i / NP][i % NP] = to_f32(rc[q]);
    }
  };

  T xr[U], dr[U], zr[U], gr[U];
  auto load = [&](int t) {
    const int valid = t + U <= len ? U : len - t;
    const Rows rx = rows_at(xp + t * sh.D, valid, sh.D, sh.D);
    const Rows rd = rows_at(dp + t * sh.D, valid, sh.D, sh.D);
    const unsigned fx = MODE == kBoth ? fresh(ox[0]) : 0, fz = MODE == kBoth && GATE ? fresh(oz[0]) : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xr[u] = row_load<T>(rx, offset(ox, fx, u, sh.D));
      dr[u] = row_load<T>(rd, offset(ox, fx, u, sh.D));
    }
    if constexpr (GATE && MODE != kStates) {
      const Rows rz = rows_at(zp + t * io.zs.token, valid, io.zs.token, sh.D);
#pragma unroll
      for (int u = 0; u < U; ++u) zr[u] = row_load<T>(rz, offset(oz, fz, u, io.zs.token));
    }
    if constexpr (MODE == kBoth) {
      const Rows rg = rows_at(gp + t * sh.D, valid, sh.D, sh.D);
#pragma unroll
      for (int u = 0; u < U; ++u) gr[u] = row_load<T>(rg, offset(ox, fx, u, sh.D));
    }
  };

  fetch(0);
  load(0);
  place(0);
  __syncthreads();
  int buf = 0;
  for (int tt = 0; tt < len; tt += kScanTile, buf ^= 1) {
    const bool more = tt + kScanTile < len;
    if (more) fetch(tt + kScanTile);
    if (live) {
      for (int s = 0; s < kScanTile && tt + s < len; s += U) {
        const int ts = tt + s;
        // the lane's own channel at U tokens
        float d[U], dx[U], xv[U], gate[U], ds[U], none[1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          xv[u] = to_f32(xr[u]);
          d[u] = to_f32(dr[u]);
          gate[u] = GATE && MODE != kStates ? to_f32(zr[u]) : 1.0f;
          ds[u] = MODE == kBoth ? to_f32(gr[u]) : 0.0f;
        }
        load(ts + U);   // past the chunk's last token an empty resource: zeros, and no branch
        if constexpr (MODE == kBoth) {
          if (ts > 0) {   // the state and the step sizes so far, before these 8 tokens
            const int64_t at = (b * ((sh.L + kSub - 1) / kSub) + (t0 + ts) / kSub) * sh.D;
            const Rows rs = rows_at(io.ckpt + at * NP, 1, 0, sh.D * NP);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int q = 0; q < SN; q += VS) row_store4(rs, oc[j] + 4 * q, h[j] + q);
            row_store<float>(rows_at(io.sumsub + at, 1, 0, sh.D), own < Dg ? (unsigned)c * 4u : kOutside, sum);
          }
        }
        dt_values<U, false>(f, d, none);
        if (ts + U > len) {   // past the last token x and dy are zero; the decays have to be one
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (ts + u >= len) d[u] = 0.0f;
        }
        const Rows ry = rows_at(MODE == kOut ? yp0 + ts * sh.D : nullptr, ts + U <= len ? U : len - ts,
                                sh.D, sh.D);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          dx[u] = d[u] * xv[u];
          if constexpr (GATE && MODE != kStates) gate[u] *= sigmoid_f32(gate[u]);
          if constexpr (MODE == kBoth) ds[u] *= gate[u];
          if constexpr (MODE != kOut) sum += d[u];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float Bv[SN], Cv[SN], part[2];
#pragma unroll
          for (int q = 0; q < SN; q += VS) {
            load_v<VS>(&sB[buf][s + u][n0 + q], Bv + q);
            if constexpr (MODE != kStates) load_v<VS>(&sC[buf][s + u][n0 + q], Cv + q);
          }
          auto channel = [&](auto J) {
            constexpr int j = decltype(J)::value;
            const float dj = pair_bcast<j>(d[u]), xj = pair_bcast<j>(dx[u]);
            const float sj = MODE == kBoth ? pair_bcast<j>(ds[u]) : 0.0f;
            part[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < SN; ++i) {
              const float a = fast_exp2(dj * A2[j][i]);
              h[j][i] = fmaf(a, h[j][i], xj * Bv[i]);
              if constexpr (MODE == kOut) part[j] = fmaf(Cv[i], h[j][i], part[j]);
              if constexpr (MODE == kBoth) {
                P[j][i] *= a;
                R[j][i] = fmaf(P[j][i], sj * Cv[i], R[j][i]);
              }
            }
          };
          channel(std::integral_constant<int, 0>{});
          channel(std::integral_constant<int, 1>{});
          if constexpr (MODE == kOut) {
            const float o = pairs_sum<RN>(pair_fold(part[0], part[1], lane));
            row_store<T>(ry, ox[u], to_io<T>(fmaf(Dc, xv[u], o) * gate[u]));
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
  for (int j = 0; j < 2; ++j) {
    const int lc = base + dl * 2 + j;
    if (lc >= Dg) continue;
    const int64_t cj = g * Dg + lc;
    if constexpr (MODE == kOut) {
      if (last && io.fin)
#pragma unroll
        for (int i = 0; i < SN; ++i)
          if (n0 + i < N) io.fin[(b * sh.D + cj) * N + n0 + i] = h[j][i];
    } else {
      if (!last)
#pragma unroll
        for (int q = 0; q < SN; q += VS)
          store_v<VS>(io.H + ((b * sh.K + k + 1) * sh.D + cj) * NP + n0 + q, h[j] + q);
      if constexpr (MODE == kBoth)
        if (k > 0)
#pragma unroll
          for (int q = 0; q < SN; q += VS)
            store_v<VS>(io.R + ((b * sh.K + k - 1) * sh.D + cj) * NP + n0 + q, R[j] + q);
    }
  }
  if constexpr (MODE != kOut)
    if (mine) io.sumdt[(b * sh.K + k) * sh.D + c] = sum;
}

// Chains the chunks for the backward pass, one thread per (b, c, n) and direction.
// Forwards, slot k of H holds chunk k - 1's end state from a zero start (chunk
// 0's from the caller's state) and becomes chunk k's start state; backwards, slot k
// of R holds what chunk k + 1 sends to its start and becomes the gradient at chunk
// k's end.
__global__ void __launch_bounds__(256)
selscan_pass_kernel(float* __restrict__ H, float* __restrict__ R, const float* __restrict__ A,
                    const float* __restrict__ sumdt, const float* __restrict__ last, int64_t batch,
                    int64_t K, int64_t D, int64_t N, int NP) {
  const bool reverse = blockIdx.y == 0;
  if (!reverse && K < 3) return;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= batch * D * NP) return;
  const int64_t n = i % NP, c = i / NP % D, b = i / NP / D;
  const float a2 = n < N ? A[c * N + n] * kLog2e : 0.0f;
  float* const p = (reverse ? R : H) + (b * K * D + c) * NP + n;
  const float* const sp = sumdt + b * K * D + c;
  const int64_t step = D * NP;
  // slots `at` from `first` on, `dir` apart, the decay of slot k being chunk
  // k - dir's; eight slots are loaded before the first of them is used
  float run = reverse ? (last && n < N ? last[(b * D + c) * N + n] : 0.0f) : p[step];
  if (reverse) p[(K - 1) * step] = run;
  const int64_t first = reverse ? K - 2 : 2, count = reverse ? K - 1 : K - 2, dir = reverse ? -1 : 1;
  constexpr int M = 8;
  for (int64_t q = 0; q < count; q += M) {
    float v[M], s[M];
#pragma unroll
    for (int u = 0; u < M; ++u) {
      const int64_t k = first + dir * (q + u < count ? q + u : count - 1);
      v[u] = p[k * step];
      s[u] = sp[(k - dir) * D];
    }
#pragma unroll
    for (int u = 0; u < M; ++u) {
      if (q + u < count) {
        run = fmaf(fast_exp2(a2 * s[u]), run, v[u]);
        p[(first + dir * (q + u)) * step] = run;
      }
    }
  }
}

// Single tokens: the recurrence from a resident state, in place.  Bound by the
// state's bytes (8 per element).  A lane holds four consecutive states of one
// channel for NB batches, whose loads are all in flight before the first is used
// and which share the channel's A, D and bias, and takes all of the call's tokens.
// VEC: dstate is a multiple of 4 and B and C allow accesses of 4 elements.
constexpr int kStepThreads = 256;
template <typename T, int RN, bool VEC, int NB>
__global__ void __launch_bounds__(kStepThreads)
selscan_step_kernel(float* __restrict__ state, const T* __restrict__ x, const T* __restrict__ dt,
                    const float* __restrict__ A, const T* __restrict__ B, Strides bs,
                    const T* __restrict__ C, Strides cs, const float* __restrict__ Dv,
                    const T* __restrict__ z, Strides zs, T* __restrict__ y, DtXform xf, int batch,
                    int64_t L, int D, int N, int Dg) {
  const int nl = threadIdx.x % RN, n0 = 4 * nl;
  const int own = blockIdx.x * (kStepThreads / RN) + threadIdx.x / RN;
  const bool live = own < D;
  const int c = live ? own : D - 1;
  const int g = c / Dg;
  const int b0 = blockIdx.y * NB;
  const bool states = n0 < N;
  auto load4 = [&](const float* p, float* v) {
    if constexpr (VEC) {
      v[0] = v[1] = v[2] = v[3] = 0.0f;
      if (states) load_v<4>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = n0 + i < N ? p[i] : 0.0f;
    }
  };
  auto load_bc = [&](const T* p, float* v) {
    if constexpr (VEC) {
      v[0] = v[1] = v[2] = v[3] = 0.0f;
      if (states) load_v<4>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = n0 + i < N ? to_f32(p[i]) : 0.0f;
    }
  };
  float h[NB][4], A2[4];
#pragma unroll
  for (int u = 0; u < NB; ++u) {
    const int64_t b = b0 + u < batch ? b0 + u : batch - 1;
    load4(state + (b * D + c) * N + n0, h[u]);
  }
  load4(A + (int64_t)c * N + n0, A2);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
  const DtLane f = dt_lane(xf, c);
  const float Dc = Dv ? Dv[c] : 0.0f;
  for (int64_t t = 0; t < L; ++t) {
    float xv[NB], d[NB], zv[NB], Bv[NB][4], Cv[NB][4], none[1];
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const int64_t b = b0 + u < batch ? b0 + u : batch - 1;
      xv[u] = to_f32(x[(b * L + t) * D + c]);
      d[u] = to_f32(dt[(b * L + t) * D + c]);
      zv[u] = z ? to_f32(z[b * zs.batch + t * zs.token + c]) : 0.0f;
      load_bc(B + b * bs.batch + t * bs.token + (int64_t)g * N + n0, Bv[u]);
      load_bc(C + b * cs.batch + t * cs.token + (int64_t)g * N + n0, Cv[u]);
    }
    dt_values<NB, false>(f, d, none);
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const float dx = d[u] * xv[u];
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[u][i] = fmaf(fast_exp2(d[u] * A2[i]), h[u][i], dx * Bv[u][i]);
        part = fmaf(Cv[u][i], h[u][i], part);
      }
      part += dpp_move<0xB1>(part);                          // the four lanes of a quad, then RN
      part += dpp_move<0x4E>(part);
      part = quads_sum<RN>(part);
      float o = fmaf(Dc, xv[u], part);
      if (z) o *= zv[u] * sigmoid_f32(zv[u]);
      if (live && nl == 0 && b0 + u < batch) y[((int64_t)(b0 + u) * L + t) * D + c] = to_io<T>(o);
    }
  }
#pragma unroll
  for (int u = 0; u < NB; ++u) {
    if (!live || b0 + u >= batch) continue;
    float* p = state + ((int64_t)(b0 + u) * D + c) * N + n0;
    if constexpr (VEC) {
      if (states) store_v<4>(p, h[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + i < N) p[i] = h[u][i];
    }
  }
}

// ---- host ----

// Chunks of the forward pass.  One where its waves nearly fill the chip (1024 tokens
// of 5120 channels: for 8 batches, 640 waves, chunks take 306 us and one chunk 334, for
// 10 batches 399 and 340); otherwise as many as give about two waves per SIMD
// (2048 tokens of 5120 channels x 16 states: 24 chunks 98 us, 12 chunks 110, 37 chunks
// 103, 43 chunks 118: more chunks cost more starts and longer chains), of at
// least 16 tokens (300 tokens of 2560 channels: at least 16 28 us, 32 35, 64 54), and
// 64 to 128 of them at most (64 channels: 8192 tokens in 128 chunks 80 us, in 64 95;
// 2048 tokens 56 and 44).
ScanShape selscan_fwd_shape(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
  ScanShape s;
  const int np = selscan_fwd_np(N);
  const int64_t cw = np <= 16 ? 64 : np <= 32 ? 32 : 16, per = cw * (kScanThreads / kWave);
  s.L = L; s.D = D; s.N = N; s.G = G; s.Dg = D / G;
  s.tiles = (s.Dg + per - 1) / per;
  const int64_t waves = batch * G * ((s.Dg + cw - 1) / cw);
  s.K = 1;
  s.T = L;
  if (waves < 720 && L > 64) {
    int64_t k = 2000 / waves;
    if (k > L / 16) k = L / 16;
    const int64_t most = L / 64 < 64 ? 64 : L / 64 < 128 ? L / 64 : 128;
    if (k > most) k = most;
    if (k < 1) k = 1;
    s.T = ((L + k - 1) / k + 7) / 8 * 8;
    s.K = (L + s.T - 1) / s.T;
  }
  return s;
}

static size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
size_t selscan_state_bytes(int64_t batch, const ScanShape& s, int np) {
  return up256(size_t(batch) * s.K * s.D * np * sizeof(float));
}
size_t selscan_sum_bytes(int64_t batch, const ScanShape& s) {
  return up256(size_t(batch) * s.K * s.D * sizeof(float));
}

size_t selscan_fwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
  const ScanShape s = selscan_fwd_shape(batch, L, D, N, G);
  return s.K == 1 ? 0 : selscan_state_bytes(batch, s, selscan_fwd_np(N)) + selscan_sum_bytes(batch, s);
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

template <typename T, int RN, int SN, int MODE>
static void launch_scan(const ScanIo<T>& io, const ScanShape& s, int64_t batch, int64_t chunks,
                        hipStream_t stream) {
  const dim3 grid((unsigned)(s.tiles * s.G * chunks), (unsigned)batch);
  if constexpr (MODE != kStates) {
    if (io.z) {
      hipLaunchKernelGGL((selscan_kernel<T, RN, SN, MODE, true>), grid, dim3(kScanThreads), 0, stream, io, s);
      return;
    }
  }
  hipLaunchKernelGGL((selscan_kernel<T, RN, SN, MODE, false>), grid, dim3(kScanThreads), 0, stream, io, s);
}

template <typename T, int RN, int SN>
static hipError_t fwd_np(const ScanArgs& a, hipStream_t stream) {
  const ScanShape s = selscan_fwd_shape(a.batch, a.L, a.D, a.N, a.G);
  ScanIo<T> io = scan_io<T>(a);
  if (s.K > 1) {
    io.H = static_cast<float*>(a.workspace);
    io.sumdt = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + selscan_state_bytes(a.batch, s, RN * SN));
    launch_scan<T, RN, SN, kStates>(io, s, a.batch, s.K - 1, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  launch_scan<T, RN, SN, kOut>(io, s, a.batch, s.K, stream);
  return hipGetLastError();
}

template <typename T>
static hipError_t fwd_t(const ScanArgs& a, hipStream_t stream) {
  switch (selscan_fwd_np(a.N)) {
    case 8: return fwd_np<T, 2, 4>(a, stream);
    case 16: return fwd_np<T, 2, 8>(a, stream);
    case 24: return fwd_np<T, 4, 6>(a, stream);
    case 32: return fwd_np<T, 4, 8>(a, stream);
    case 48: return fwd_np<T, 8, 6>(a, stream);
    default: return fwd_np<T, 8, 8>(a, stream);
  }
}

hipError_t launch_selscan_fwd(const ScanArgs& a, hipStream_t stream) {
  return a.bf16 ? fwd_t<bf16>(a, stream) : fwd_t<float>(a, stream);
}

// First stage of the backward pass: every chunk's end state and the gradient it sends
// to its start, then both chains.
template <typename T, int NP>
static hipError_t both_np(const ScanArgs& a, const ScanShape& s, float* H, float* R, float* sumdt,
                          float* ckpt, float* sumsub, hipStream_t stream) {
  ScanIo<T> io = scan_io<T>(a);
  io.H = H;
  io.R = R;
  io.sumdt = sumdt;
  io.ckpt = ckpt;
  io.sumsub = sumsub;
  launch_scan<T, NP / 8, 8, kBoth>(io, s, a.batch, s.K, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(selscan_pass_kernel, dim3((unsigned)((a.batch * s.D * NP + 255) / 256), s.K > 2 ? 2 : 1),
                     dim3(256), 0, stream, H, R, a.A, sumdt, a.dfin, a.batch, s.K, s.D, s.N, NP);
  return hipGetLastError();
}
hipError_t launch_selscan_both(const ScanArgs& a, const ScanShape& s, float* H, float* R,
                               float* sumdt, float* ckpt, float* sumsub, hipStream_t stream) {
  const int np = selscan_np(a.N);
  if (a.bf16)
    return np == 16 ? both_np<bf16, 16>(a, s, H, R, sumdt, ckpt, sumsub, stream)
           : np == 32 ? both_np<bf16, 32>(a, s, H, R, sumdt, ckpt, sumsub, stream)
                      : both_np<bf16, 64>(a, s, H, R, sumdt, ckpt, sumsub, stream);
  return np == 16 ? both_np<float, 16>(a, s, H, R, sumdt, ckpt, sumsub, stream)
         : np == 32 ? both_np<float, 32>(a, s, H, R, sumdt, ckpt, sumsub, stream)
                    : both_np<float, 64>(a, s, H, R, sumdt, ckpt, sumsub, stream);
}

template <typename T, int RN, int NB>
static hipError_t step_nb(const ScanArgs& a, hipStream_t stream) {
  constexpr int per = kStepThreads / RN;
  const dim3 grid((unsigned)((a.D + per - 1) / per), (unsigned)((a.batch + NB - 1) / NB));
  const DtXform xf = a.xf ? *a.xf : DtXform{nullptr, 0, -INFINITY, INFINITY};
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kStepThreads), 0, stream, a.state, static_cast<const T*>(a.x),
                       static_cast<const T*>(a.dt), a.A, static_cast<const T*>(a.B),
                       Strides{a.bs[0], a.bs[1]}, static_cast<const T*>(a.C),
                       Strides{a.cs[0], a.cs[1]}, a.Dv, static_cast<const T*>(a.z),
                       Strides{a.zs[0], a.zs[1]}, static_cast<T*>(a.y), xf, (int)a.batch, a.L, (int)a.D,
                       (int)a.N, (int)(a.D / a.G));
  };
  if (a.vec) go(selscan_step_kernel<T, RN, true, NB>);
  else go(selscan_step_kernel<T, RN, false, NB>);
  return hipGetLastError();
}
template <typename T, int RN>
static hipError_t step_rn(const ScanArgs& a, hipStream_t stream) {
  // two batches per lane where that still leaves eight waves per SIMD (128 x 5120 x 16
  // states: 20.5 us, one 22.2, four 25.1; smaller calls need the waves)
  return a.batch * a.D * RN / 64 >= 2 * 8192 ? step_nb<T, RN, 2>(a, stream) : step_nb<T, RN, 1>(a, stream);
}
template <typename T>
static hipError_t step_t(const ScanArgs& a, hipStream_t stream) {
  const int rn = selscan_np(a.N) / 4;
  if (rn == 4) return step_rn<T, 4>(a, stream);
  if (rn == 8) return step_rn<T, 8>(a, stream);
  return step_rn<T, 16>(a, stream);
}
hipError_t launch_selscan_step(const ScanArgs& a, hipStream_t stream) {
  return a.bf16 ? step_t<bf16>(a, stream) : step_t<float>(a, stream);
}

}  // namespace ssd
