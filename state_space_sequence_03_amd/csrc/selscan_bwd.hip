// selscan_bwd.hip -- gradients of the selective scan.
//
// With ds_t = dy_t z_t sigmoid(z_t) (dy without z), a_t = exp(dt_t A) and g_t the
// gradient of the loss with respect to h_t:
//     g_t = ds_t C_t + a_{t+1} g_{t+1}          (dfinal enters after the last token)
//     q_t = sum_n g_t B_t,   r_t = sum_n A a_t g_t h_{t-1}
//     dx_t = dt_t q_t + D ds_t,                 ddt_t = (x_t q_t + r_t) d(dt)/d(raw)
//     dB_t[g] = sum_c dt_t x_t g_t,             dC_t[g] = sum_c ds_t h_t
//     dA = sum_t dt_t a_t g_t h_{t-1},          dD = sum_t ds_t x_t
//     dz_t = dy_t s_t silu'(z_t)                dinit = a_0 g_0
//
// The states are needed from the last token to the first.  selscan_kernel<both> and
// its chains (selscan.hip) give each chunk's start state, the gradient at its end
// and, every 8 tokens, the state from a zero start of the chunk; the true state
// there is that plus the decayed start state.  selscan_bwd_kernel walks a chunk
// backwards 8 tokens at a time and forms their states and decays again in
// registers (a quarter of the decays a third time), and the checkpoints move N
// bytes per (t, c): 16 at dstate 16, beside the 22 of bf16 operands.
//
// Bound by the issue of vector ALU instructions: about 1600 per wave and 8 tokens
// (64 elements a lane), 860 of them the sums above, the rest the step sizes, the
// sums across lanes and the broadcasts; counters show the vector ALU busy 75% of
// the time.  2 x 2048 tokens x 5120 channels x 16 states, bf16 with gate: 423 us in
// all, 276 of them here, 119 in selscan_kernel<both>, 19 in the chains and 9 in
// the last sums (kernel trace).  Walking each chunk forwards once more in place of the checkpoints took
// the same 472 us when both were measured, and 81 against 69 us for 2 x 515 x 770
// channels in fp32.
//
// dB and dC are sums over channels: over the lane groups of a wave by lane
// swaps, over a workgroup's waves in LDS, and over workgroups by
// selscan_reduce_kernel from the workspace, each in a fixed order.  dA, dD and the
// bias gradient are sums over tokens: per chunk in registers, then over chunks by
// the same kernel.
#include <type_traits>

#include "layer_host.hpp"
#include "selscan_device.hpp"

namespace ssd {

constexpr int kBwdThreads = 256;
constexpr int kBwdWaves = kBwdThreads / kWave;
constexpr int kPairs = kSub / 2;    // lanes prepare two tokens of two channels at a time
// The decays of the last tokens of each 8 stay in registers, those of the first
// kAgain are formed a second time: all of them would not fit beside the states
// (0 and 1, which spill: 513 and 453 us, 2: 429, 3: 432, 4: 436 for all kernels at the
// size above).
constexpr int kAgain = 2;

// Tokens per chunk at most: B and C of all of it, and the waves' parts of dB and
// dC, fit LDS for two workgroups per CU (dstate up to 32), so that the waves meet
// at two barriers only: one barrier per 8 tokens, with chunks three times as long,
// took 505 us against 472 for 2 x 2048 x 5120 channels x 16 states; chunks of 32
// tokens 517, of 80 485, of 112 496.
__host__ __device__ constexpr int bwd_tokens(int NP) { return NP == 16 ? 64 : 32; }
constexpr int bwd_smem_bytes(int NP) {
  return (bwd_tokens(NP) * 2 * NP * (1 + kBwdWaves) + kBwdThreads * 8) * (int)sizeof(float);
}

template <typename T>
struct ScanBwdIo {
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
  const float *H, *R;   // [batch][K][D][NP]
  const float *ckpt, *sumsub;   // [batch][ceil(L / 8)][D][NP], [batch][ceil(L / 8)][D]
  float* dApart;        // [batch][K][D][NP]: H's slots, each read before it is written
  float *dDpart, *dbpart;   // [batch][K][D]
  float* bcpart;        // [batch][L][G][tiles][2][NP]
  T *dx, *ddt, *dz;
  Strides dzs;
  float* dinit;
  DtXform xf;
};

template <typename T, int RN, bool GATE>
__global__ void __launch_bounds__(kBwdThreads, 2)
selscan_bwd_kernel(ScanBwdIo<T> io, ScanShape sh) {
  constexpr int NP = 4 * RN, CW = 128 / RN;
  constexpr int ROW = kSub * 2 * NP;           // B and C, or dB and dC, of 8 tokens: [token][2][NP]
  constexpr int SUBS = bwd_tokens(NP) / kSub;
  extern __shared__ float smem[];
  float* const bc = smem;                      // [SUBS][ROW], the chunk's B and C
  float* const sums = bc + SUBS * ROW;         // [wave][SUBS][ROW], the waves' parts of dB and dC
  float* const start = sums + kBwdWaves * SUBS * ROW + threadIdx.x * 4;   // [2][thread][4]: start states
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int tiles = (int)sh.tiles, groups = (int)sh.G, Dg = (int)sh.Dg, N = (int)sh.N;
  const int tile = blockIdx.x % (tiles * groups);
  const int k = blockIdx.x / (tiles * groups);
  const int64_t b = blockIdx.y;
  const int g = tile / tiles;
  const int base = ((tile % tiles) * kBwdWaves + wave) * CW;
  const bool live = base < Dg;                       // whole waves past the group only stage and sum
  const int nl = lane % RN, dl = lane / RN, n0 = 4 * nl;
  const int par = (lane >> 1) & 1;                   // which token of a pair this lane prepares
  const int own = base + dl * 2 + (lane & 1);        // and which channel
  const int c = g * Dg + (own < Dg ? own : Dg - 1);
  const bool mine = own < Dg && nl < 4;
  const int64_t t0 = k * sh.T;
  const int len = (int)(t0 + sh.T < sh.L ? sh.T : sh.L - t0);   // tokens of this chunk
  const int subs = (len + kSub - 1) / kSub;

  float A2[2][4], gr[2][4], dA[2][4];
  unsigned oc[2];                        // byte offsets of the lane's states in a row of checkpoints
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lc = base + dl * 2 + j;
    const int64_t cj = g * Dg + (lc < Dg ? lc : Dg - 1);
    const int64_t at = ((b * sh.K + k) * sh.D + cj) * NP + n0;
    oc[j] = (unsigned)(cj * NP + n0) * 4u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + i;
      A2[j][i] = n < N ? io.A[cj * N + n] * kLog2e : 0.0f;
      start[j * kBwdThreads * 4 + i] = k > 0 ? io.H[at + i]
                              : io.init && n < N ? io.init[(b * sh.D + cj) * N + n] : 0.0f;
      gr[j][i] = io.R[at + i];
      dA[j][i] = 0.0f;
    }
  }
  const DtLane f = dt_lane(io.xf, c);
  const float Dc = io.Dv ? io.Dv[c] : 0.0f;
  float dD = 0.0f, dbias = 0.0f;

  // this chunk's rows, and byte offsets of the lane's channel and token in 8 of them;
  // lanes that share both store the same values
  const int64_t row = (b * sh.L + t0) * sh.D;
  const T* const xp = io.x + row;
  const T* const dp = io.dt + row;
  const T* const gp = io.dy + row;
  const T* const zp = GATE ? io.z + b * io.zs.batch + t0 * io.zs.token : nullptr;
  T* const zo = GATE ? io.dz + b * io.dzs.batch + t0 * io.dzs.token : nullptr;
  const int64_t sub0 = b * ((sh.L + kSub - 1) / kSub) + t0 / kSub;
  const unsigned xrow = (unsigned)(sh.D * sizeof(T)), zrow = GATE ? (unsigned)(io.zs.token * sizeof(T)) : 0;
  const unsigned zorow = GATE ? (unsigned)(io.dzs.token * sizeof(T)) : 0;
  const unsigned cb = own < Dg ? (unsigned)c * (unsigned)sizeof(T) : kOutside;
  const unsigned ox = cb + par * xrow, oz = cb + par * zrow, ozo = cb + par * zorow;
  // what 8 tokens need, loaded while the 8 after them are worked on
  T xr[kPairs], dr[kPairs], zr[kPairs], yr[kPairs];
  float ck[2][4], cs[2];
  auto load = [&](int s) {
    const int more = (s * kSub + kSub <= len ? kSub : len - s * kSub) - 1;   // valid rows after the first
    const int64_t t = (int64_t)s * kSub * sh.D;
    const unsigned bytes = (more + 1) * xrow;
    const Rows rx = rows_bytes(xp + t, bytes), rd = rows_bytes(dp + t, bytes), rg = rows_bytes(gp + t, bytes);
    const unsigned o = fresh(ox);
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      xr[p] = row_load<T>(rx, o + 2 * p * xrow);
      dr[p] = row_load<T>(rd, o + 2 * p * xrow);
      yr[p] = row_load<T>(rg, o + 2 * p * xrow);
    }
    if constexpr (GATE) {
      const Rows rz = rows_bytes(zp + s * kSub * io.zs.token, more * zrow + xrow);
      const unsigned q = fresh(oz);
#pragma unroll
      for (int p = 0; p < kPairs; ++p) zr[p] = row_load<T>(rz, q + 2 * p * zrow);
    }
    if (s > 0) {
      const Rows rc = rows_bytes(io.ckpt + (sub0 + s) * sh.D * NP, (unsigned)(sh.D * NP) * 4u);
      const Rows rs = rows_bytes(io.sumsub + (sub0 + s) * sh.D, (unsigned)sh.D * 4u);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        row_load4(rc, oc[j], ck[j]);
        cs[j] = row_load<float>(rs, fresh(oc[j]) / (4 * NP) * 4);
      }
    }
  };
  if (live) load(subs - 1);
  {
    const T* const Bp = io.B + b * io.bs.batch + t0 * io.bs.token + g * N;
    const T* const Cp = io.C + b * io.cs.batch + t0 * io.cs.token + g * N;
    for (int i = tid; i < SUBS * ROW / 2; i += kBwdThreads) {
      const int tok = i / NP, n = i % NP;
      const bool in = tok < len && n < N;
      bc[tok * 2 * NP + n] = in ? to_f32(Bp[tok * io.bs.token + n]) : 0.0f;
      bc[(tok * 2 + 1) * NP + n] = in ? to_f32(Cp[tok * io.cs.token + n]) : 0.0f;
    }
  }
  __syncthreads();
  if (live) {
    for (int s = subs - 1; s >= 0; --s) {
      const float* const sBC = bc + s * ROW + n0;
      float* const slot = sums + (wave * SUBS + s) * ROW;
      float h0[2][4], hist[kSub][2][4], dec[kSub - kAgain + (kAgain == kSub)][2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) load_v<4>(start + j * kBwdThreads * 4, h0[j]);
      if (s > 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)   // (chunk 0's checkpoints start from the caller's state)
            h0[j][i] = k > 0 ? fmaf(fast_exp2(A2[j][i] * cs[j]), h0[j][i], ck[j][i]) : ck[j][i];
      }
      float d[kPairs], dx[kPairs], ds[kPairs], xv[kPairs], slope[kPairs], yv[kPairs], zv[kPairs];
#pragma unroll
      for (int p = 0; p < kPairs; ++p) d[p] = to_f32(dr[p]);
      dt_values<kPairs, true>(f, d, slope);
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        xv[p] = to_f32(xr[p]);
        yv[p] = to_f32(yr[p]);   // x and dy are zero past the last token and the last channel
        zv[p] = GATE ? to_f32(zr[p]) : 0.0f;
        ds[p] = GATE ? yv[p] * (zv[p] * sigmoid_f32(zv[p])) : yv[p];
      }
      if (s * kSub + kSub > len) {
#pragma unroll
        for (int p = 0; p < kPairs; ++p)
          if (s * kSub + 2 * p + par >= len) d[p] = slope[p] = 0.0f;
      }
#pragma unroll
      for (int p = 0; p < kPairs; ++p) dx[p] = d[p] * xv[p];
      if (s > 0) load(s - 1);
      const int more = (s * kSub + kSub <= len ? kSub : len - s * kSub) - 1;
      const int64_t t8 = row + (int64_t)s * kSub * sh.D;
      const Rows wx = rows_bytes(io.dx + t8, (more + 1) * xrow), wd = rows_bytes(io.ddt + t8, (more + 1) * xrow);
      // (rows of dz are at least a row apart, also where there is one: rows past the last end behind it)
      const Rows wz = rows_bytes(GATE ? zo + s * kSub * io.dzs.token : nullptr, more * zorow + xrow);
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        float yp[4];
        auto token = [&](auto Q) {
          constexpr int q = decltype(Q)::value;
          const int t = 2 * p + q;
          const floatx4 Bv = *reinterpret_cast<const floatx4*>(sBC + 2 * t * NP);
          const floatx4 Cv = *reinterpret_cast<const floatx4*>(sBC + (2 * t + 1) * NP);
          const float dj[2] = {quad_bcast<2 * q>(d[p]), quad_bcast<2 * q + 1>(d[p])};
          const float xj[2] = {quad_bcast<2 * q>(dx[p]), quad_bcast<2 * q + 1>(dx[p])};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = fast_exp2(dj[j] * A2[j][i]);
              if (t >= kAgain) dec[t >= kAgain ? t - kAgain : 0][j][i] = a;
              hist[t][j][i] = fmaf(a, t ? hist[t ? t - 1 : 0][j][i] : h0[j][i], xj[j] * Bv[i]);
              if constexpr (GATE) y = i ? fmaf(Cv[i], hist[t][j][i], y) : Cv[i] * hist[t][j][i];
            }
            if constexpr (GATE) yp[2 * q + j] = y;
          }
        };
        token(std::integral_constant<int, 0>{});
        token(std::integral_constant<int, 1>{});
        if constexpr (GATE) {
          const float o = fmaf(Dc, xv[p], quads_sum<RN>(quad_fold(yp, lane)));
          row_store<T>(wz, fresh(ozo) + 2 * p * zorow, to_io<T>(yv[p] * o * silu_slope(zv[p], sigmoid_f32(zv[p]))));
        }
      }
#pragma unroll
      for (int p = kPairs - 1; p >= 0; --p) {
        float vq[4], vr[4], vB[8], vC[8];
        auto token = [&](auto Q) {
          constexpr int q = decltype(Q)::value;
          const int t = 2 * p + q;
          const floatx4 Bv = *reinterpret_cast<const floatx4*>(sBC + 2 * t * NP);
          const floatx4 Cv = *reinterpret_cast<const floatx4*>(sBC + (2 * t + 1) * NP);
          const float dj[2] = {quad_bcast<2 * q>(d[p]), quad_bcast<2 * q + 1>(d[p])};
          const float xj[2] = {quad_bcast<2 * q>(dx[p]), quad_bcast<2 * q + 1>(dx[p])};
          const float sj[2] = {quad_bcast<2 * q>(ds[p]), quad_bcast<2 * q + 1>(ds[p])};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float qs, rs;
            const float da = __builtin_bit_cast(float, fresh(__builtin_bit_cast(unsigned, dj[j])));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float gt = fmaf(sj[j], Cv[i], gr[j][i]);
              // the first term of each sum is a product of its own
              vC[4 * q + i] = j ? fmaf(sj[j], hist[t][j][i], vC[4 * q + i]) : sj[j] * hist[t][j][i];
              vB[4 * q + i] = j ? fmaf(xj[j], gt, vB[4 * q + i]) : xj[j] * gt;
              qs = i ? fmaf(gt, Bv[i], qs) : gt * Bv[i];
              const float a = t >= kAgain ? dec[t >= kAgain ? t - kAgain : 0][j][i] : fast_exp2(da * A2[j][i]);
              const float ag = a * gt;
              const float flow = ag * (t ? hist[t ? t - 1 : 0][j][i] : h0[j][i]);
              dA[j][i] = fmaf(dj[j], flow, dA[j][i]);
              rs = i ? fmaf(A2[j][i], flow, rs) : A2[j][i] * flow;
              gr[j][i] = ag;
            }
            vq[2 * q + j] = qs;
            vr[2 * q + j] = rs;
          }
        };
        token(std::integral_constant<int, 1>{});
        token(std::integral_constant<int, 0>{});
        const float qv = quads_sum<RN>(quad_fold(vq, lane));
        const float rv = quads_sum<RN>(quad_fold(vr, lane)) * 0.6931471805599453f;   // A2 = A log2 e
        const float ddt = fmaf(xv[p], qv, rv) * slope[p];   // (past the end x, ds and slope are zero)
        dbias += ddt;
        dD = fmaf(ds[p], xv[p], dD);
        const unsigned o = fresh(ox) + 2 * p * xrow;
        row_store<T>(wx, o, to_io<T>(fmaf(d[p], qv, Dc * ds[p])));
        row_store<T>(wd, o, to_io<T>(ddt));
        // the wave's sums over channels: the lower half of the wave gets the pair's
        // first token, even rows states 0 and 1 of the four, odd rows 2 and 3
        auto channels = [&](const float (&v)[8], int which) {
          float w[4], o[2];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = halves_fold(v[i], v[4 + i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            o[i] = rows_fold(w[i], w[i + 2]);
            if constexpr (RN <= 8) o[i] += dpp_move<0x128>(o[i]);   // row_ror:8
            if constexpr (RN <= 4) o[i] += dpp_move<0x124>(o[i]);   // row_ror:4
          }
          const int tok = 2 * p + (lane >> 5);
          if ((lane & 15) < RN) {
            float* q = slot + (tok * 2 + which) * NP + n0 + ((lane >> 4) & 1) * 2;
            q[0] = o[0];
            q[1] = o[1];
          }
        };
        channels(vB, 0);
        channels(vC, 1);
      }
    }
  }
  __syncthreads();
  // the workgroup's sums of dB and dC: live waves in order
  const int left = Dg - (tile % tiles) * kBwdWaves * CW;
  const int waves = left >= kBwdWaves * CW ? kBwdWaves : (left + CW - 1) / CW;
  for (int i = tid; i < len * 2 * NP; i += kBwdThreads) {
    float v = 0.0f;
    for (int w = 0; w < waves; ++w) v += sums[w * SUBS * ROW + i];
    io.bcpart[(((b * sh.L + t0 + i / (2 * NP)) * groups + g) * tiles + tile % tiles) * 2 * NP + i % (2 * NP)] = v;
  }
  if (!live) return;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lc = base + dl * 2 + j;
    if (lc >= Dg) continue;
    const int64_t cj = g * Dg + lc;
    store_v<4>(io.dApart + ((b * sh.K + k) * sh.D + cj) * NP + n0, dA[j]);
    if (k == 0 && io.dinit)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + i < N) io.dinit[(b * sh.D + cj) * N + n0 + i] = gr[j][i];
  }
  dD += dpp_move<0x4E>(dD);         // both tokens of the pairs
  dbias += dpp_move<0x4E>(dbias);
  if (mine && par == 0) {
    io.dDpart[(b * sh.K + k) * sh.D + c] = dD;
    io.dbpart[(b * sh.K + k) * sh.D + c] = dbias;
  }
}

// The last sums.  The first `bc_blocks` workgroups form dB and dC [rows, N] (rows =
// batch x tokens x groups) from the scan's workgroups' sums, `tiles` for each row;
// the others dA [D, N], dD [D] and the bias gradient [D] from `n` (batch x chunks)
// rows of sums.
template <typename T>
__global__ void __launch_bounds__(256)
selscan_reduce_kernel(const float* __restrict__ part, T* __restrict__ dB, T* __restrict__ dC,
                      int64_t rows, int64_t tiles, unsigned bc_blocks, const float* __restrict__ dAp,
                      const float* __restrict__ dDp, const float* __restrict__ dbp, int64_t n, int64_t D,
                      int64_t N, int NP, float* __restrict__ dA, float* __restrict__ dD,
                      float* __restrict__ db) {
  if (blockIdx.x < bc_blocks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t r = i / (2 * NP);
    const int e = (int)(i % (2 * NP)), m = e % NP;
    if (r >= rows || m >= N) return;
    float v = 0.0f;
    const float* p = part + r * tiles * 2 * NP + e;
    int64_t t = 0;
    for (; t + 8 <= tiles; t += 8) {   // eight loads in flight
      float q[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) q[u] = p[(t + u) * 2 * NP];
#pragma unroll
      for (int u = 0; u < 8; ++u) v += q[u];
    }
    for (; t < tiles; ++t) v += p[t * 2 * NP];
    (e < NP ? dB : dC)[r * N + m] = to_io<T>(v);
    return;
  }
  const int64_t per = D * NP, cols = per + 2 * D;
  const int64_t i = (int64_t)(blockIdx.x - bc_blocks) * 32 + threadIdx.x % 32;
  const float* p = i >= cols ? nullptr : i < per ? dAp + i : i < per + D ? dDp + (i - per) : dbp + (i - per - D);
  const float v = column_sum(p, n, i < per ? per : D);
  if (threadIdx.x >= 32 || i >= cols) return;
  if (i < per) {
    if (i % NP < N) dA[i / NP * N + i % NP] = v;
  } else if (i < per + D) {
    if (dD) dD[i - per] = v;
  } else if (db) {
    db[i - per - D] = v;
  }
}

// ---- host ----

// Chunks: as long as LDS allows, half that where their waves would not fill the chip
// (512 tokens of 5120 channels: halved from 2048 waves down 104 us, from 1024 down
// 114; 2 x 512 x 2048 channels x 4 states: 75 and 92).
static ScanShape bwd_shape(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
  ScanShape s;
  const int np = selscan_np(N);
  const int64_t cw = 512 / np, per = cw * kBwdWaves;
  s.L = L; s.D = D; s.N = N; s.G = G; s.Dg = D / G;
  s.tiles = (s.Dg + per - 1) / per;
  const int64_t waves = batch * G * ((s.Dg + cw - 1) / cw);
  s.T = bwd_tokens(np);
  if (waves * ((L + s.T - 1) / s.T) < 2048) s.T /= 2;
  s.K = (L + s.T - 1) / s.T;
  return s;
}
static size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

struct ScanBwdLayout {
  size_t h, r, sum, dd, db, ckpt, sumsub, bc, bytes;
};
static ScanBwdLayout bwd_layout(int64_t batch, const ScanShape& s) {
  ScanBwdLayout w;
  const size_t st = selscan_state_bytes(batch, s, selscan_np(s.N)), sm = selscan_sum_bytes(batch, s);
  const size_t subs = size_t(batch) * ((s.L + kSub - 1) / kSub) * s.D * sizeof(float);
  w.h = 0;
  w.r = st;
  w.sum = 2 * st;
  w.dd = w.sum + sm;
  w.db = w.dd + sm;
  w.ckpt = w.db + sm;
  w.sumsub = w.ckpt + up256(subs * selscan_np(s.N));
  w.bc = w.sumsub + up256(subs);
  w.bytes = w.bc + up256(size_t(batch) * s.L * s.G * s.tiles * 2 * selscan_np(s.N) * sizeof(float));
  return w;
}

size_t selscan_bwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
  return bwd_layout(batch, bwd_shape(batch, L, D, N, G)).bytes;
}

// Whether every launch of the scan stays within a grid: workgroups along x
// (channels x chunks, rows of the reductions), batches along y.
int selscan_grid_ok(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
  const ScanShape s = bwd_shape(batch, L, D, N, G);
  const __int128 most = (1 << 24) - 1;   // of 256 threads each: a launch has fewer than 2^32
  const int np = selscan_np(N);
  return batch <= 65535 && D * np < (1 << 29) && (__int128)s.tiles * G * s.K <= most &&
         (__int128)batch * L * G * 2 * np / 256 + (__int128)D * (np + 2) / 32 + 2 < most &&
         (__int128)batch * D * np / 256 < most;
}

// The forward kernels tile channels more widely than the backward one.
static ScanShape fwd_tiles(ScanShape s) {
  const int64_t per = 1024 / selscan_np(s.N) * 4;
  s.tiles = (s.Dg + per - 1) / per;
  return s;
}

template <typename T, int RN, bool GATE>
static hipError_t bwd_g(const ScanArgs& a, hipStream_t stream) {
  const ScanShape s = bwd_shape(a.batch, a.L, a.D, a.N, a.G);
  const ScanBwdLayout w = bwd_layout(a.batch, s);
  char* ws = static_cast<char*>(a.workspace);
  float* H = reinterpret_cast<float*>(ws + w.h);
  float* R = reinterpret_cast<float*>(ws + w.r);
  float* ckpt = reinterpret_cast<float*>(ws + w.ckpt);
  float* sumsub = reinterpret_cast<float*>(ws + w.sumsub);
  hipError_t e = launch_selscan_both(a, fwd_tiles(s), H, R, reinterpret_cast<float*>(ws + w.sum), ckpt,
                                     sumsub, stream);
  if (e != hipSuccess) return e;
  ScanBwdIo<T> io{};
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
  io.H = H;
  io.R = R;
  io.ckpt = ckpt;
  io.sumsub = sumsub;
  io.dApart = H;
  io.dDpart = reinterpret_cast<float*>(ws + w.dd);
  io.dbpart = reinterpret_cast<float*>(ws + w.db);
  io.bcpart = reinterpret_cast<float*>(ws + w.bc);
  io.dx = static_cast<T*>(a.dx);
  io.ddt = static_cast<T*>(a.ddt);
  io.dz = static_cast<T*>(a.dz);
  io.dzs = {a.dzs[0], a.dzs[1]};
  io.dinit = a.dinit;
  io.xf = a.xf ? *a.xf : DtXform{nullptr, 0, -INFINITY, INFINITY};
  constexpr int smem = bwd_smem_bytes(4 * RN);
  e = ensure_dyn_lds<selscan_bwd_kernel<T, RN, GATE>>(smem);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((selscan_bwd_kernel<T, RN, GATE>),
                     dim3((unsigned)(s.tiles * s.G * s.K), (unsigned)a.batch), dim3(kBwdThreads), smem,
                     stream, io, s);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t rows = a.batch * a.L * a.G;
  const int np = 4 * RN;
  const unsigned bc_blocks = (unsigned)((rows * 2 * np + 255) / 256);
  const unsigned a_blocks = (unsigned)((a.D * (np + 2) + 31) / 32);
  hipLaunchKernelGGL(selscan_reduce_kernel<T>, dim3(bc_blocks + a_blocks), dim3(256), 0, stream, io.bcpart,
                     static_cast<T*>(a.dB), static_cast<T*>(a.dC), rows, s.tiles, bc_blocks, io.dApart,
                     io.dDpart, io.dbpart, a.batch * s.K, a.D, a.N, np, a.dA, a.dD, a.dbias);
  return hipGetLastError();
}

template <typename T, int RN>
static hipError_t bwd_rn(const ScanArgs& a, hipStream_t stream) {
  return a.z ? bwd_g<T, RN, true>(a, stream) : bwd_g<T, RN, false>(a, stream);
}
template <typename T>
static hipError_t bwd_t(const ScanArgs& a, hipStream_t stream) {
  const int rn = selscan_np(a.N) / 4;
  if (rn == 4) return bwd_rn<T, 4>(a, stream);
  if (rn == 8) return bwd_rn<T, 8>(a, stream);
  return bwd_rn<T, 16>(a, stream);
}

hipError_t launch_selscan_bwd(const ScanArgs& a, hipStream_t stream) {
  return a.bf16 ? bwd_t<bf16>(a, stream) : bwd_t<float>(a, stream);
}

}  // namespace ssd
