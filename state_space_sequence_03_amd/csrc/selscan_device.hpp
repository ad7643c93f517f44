// selscan_device.hpp -- lane layout and cross-lane sums of the selective-scan
// kernels.
//
// A wave holds a tile of channels x states.  RN lanes (4, 8 or 16, consecutive)
// share the states: lane r = l % RN holds states 4 r .. 4 r + 3, padded with zero B
// and C beyond dstate; the 64 / RN lane groups hold consecutive channels, a few
// per lane.  With few channels per lane and few states per lane both sums of the
// scan are cheap: the sum over states (y, dx, ddt) runs over RN neighbouring lanes,
// the sum over channels (dB, dC) over the lane groups, and what belongs to a
// channel alone (step size, gate) is prepared once per channel, by one lane of
// each group of four, and read by the others as a DPP quad broadcast.
#pragma once
#include "layer_device.hpp"

namespace ssd {

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// lane J of each group of four lanes
template <int J> __device__ __forceinline__ float quad_bcast(float v) { return dpp_move<J * 0x55>(v); }

// Four values summed over the four lanes of a quad: lane q gets the sum of v[q].
__device__ __forceinline__ float quad_fold(const float (&v)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
  const float w0 = (b0 ? v[1] : v[0]) + dpp_move<0xB1>(b0 ? v[0] : v[1]);   // lane ^ 1
  const float w1 = (b0 ? v[3] : v[2]) + dpp_move<0xB1>(b0 ? v[2] : v[3]);
  return (b1 ? w1 : w0) + dpp_move<0x4E>(b1 ? w0 : w1);                     // lane ^ 2
}
// The rest of a sum over RN lanes, after quad_fold.
template <int RN> __device__ __forceinline__ float quads_sum(float v) {
#pragma unroll
  for (int off = 4; off < RN; off *= 2) v += __shfl_xor(v, off, kWave);
  return v;
}

// v0 and v1 each summed over the lane pairs 32 apart: the lower half of the
// wave gets v0's sums, the upper half v1's.
__device__ __forceinline__ float halves_fold(float v0, float v1) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v0),
                                                  __builtin_bit_cast(unsigned, v1), false, false);
  const unsigned lo = r[0], hi = r[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
// The same between neighbouring rows of 16: even rows get v0's sums, odd rows v1's.
__device__ __forceinline__ float rows_fold(float v0, float v1) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v0),
                                                  __builtin_bit_cast(unsigned, v1), false, false);
  const unsigned lo = r[0], hi = r[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}

// The step size of one channel and token: dt_prepare with the bias in a register.
struct DtLane {
  float bias, lo, hi;
  int has_bias, softplus;
};
__device__ __forceinline__ DtLane dt_lane(const DtXform& f, int64_t c) {
  return {f.bias ? f.bias[c] : 0.0f, f.lo, f.hi, f.bias != nullptr, f.softplus};
}
__device__ __forceinline__ float dt_value(const DtLane& f, float v) {
  if (f.has_bias) v += f.bias;
  if (f.softplus) v = softplus_f32(v);
  return fminf(fmaxf(v, f.lo), f.hi);
}
// d(step size)/d(raw): the logistic of the raw value where softplus is on, and
// zero where the clamp holds (its ends pass the gradient).
__device__ __forceinline__ float dt_slope(const DtLane& f, float v) {
  if (f.has_bias) v += f.bias;
  float s = 1.0f;
  if (f.softplus) {
    s = sigmoid_f32(v);
    v = softplus_f32(v);
  }
  return v >= f.lo && v <= f.hi ? s : 0.0f;
}

// Workspace rows of the chunked passes: [batch][chunks][channels][NP] fp32
// states (NP = 4 RN) and [batch][chunks][channels] step-size sums.
struct ScanShape {
  int64_t L, D, N, G, Dg;   // Dg = channels per group
  int64_t K, T;             // chunks and tokens per chunk
  int64_t tiles;            // workgroups per group of channels
};

// Lanes that share the states, and what the two source files of the scan share on
// the host: chained start states and end gradients of every chunk, workspace sizes.
inline int selscan_rn(int64_t N) { return N <= 16 ? 4 : N <= 32 ? 8 : 16; }
struct ScanArgs;
hipError_t launch_selscan_both(const ScanArgs& a, const ScanShape& s, float* H, float* R,
                               float* sumdt, hipStream_t stream);
size_t selscan_state_bytes(int64_t batch, const ScanShape& s);
size_t selscan_sum_bytes(int64_t batch, const ScanShape& s);

}  // namespace ssd
