// block_host.hpp -- between block_api.cpp (argument checks) and the kernels'
// launchers: one plain struct of checked arguments per operator.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ssd_block.h"

namespace ssd {

// The norms in front of and behind a layer (add_norm.hip).
struct BlockNormArgs {
  int64_t batch, L, C, G;
  float eps;
  int bf16, res_bf16;   // io and residual types
  int gate;             // 0: residual addition; 1, 2: gate before, behind the norm
  const void* x;
  int64_t xs[2];
  const void* r;        // residual, or the gate z
  int64_t zs[2];
  const float* w;
  void* h;
  void* y;
  unsigned char* q;
  float* scale;
};
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream);
int block_norm_grid_ok(int64_t batch, int64_t L, int64_t C, int64_t G, int gate);
int64_t block_norm_limit();

struct AddNormBwdArgs {
  int64_t rows, C;
  float eps;
  int bf16, res_bf16;
  const void* h;
  const float* w;
  const void *dy, *dh;
  void *dx, *dres;
  float* dw;
  void* workspace;
};
hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t stream);
size_t add_norm_bwd_workspace(int64_t rows, int64_t C, int bf16, int res_bf16);

struct Quant8Args {
  int64_t batch, L, C;
  int bf16, tile;
  const void* x;
  int64_t xs[2];
  unsigned char *q, *qt;
  float *scale, *scale_t;
};
hipError_t launch_quant8(const Quant8Args& a, hipStream_t stream);
int quant8_grid_ok(int64_t rows, int64_t C, int tile, int transposed);

struct Matmul8Args {
  int64_t M, N, K;
  int tile, out_bf16;
  const unsigned char* x;
  const float* xs;
  const unsigned char* w;
  const float* ws;
  void* y;
  void* workspace;
};
hipError_t launch_matmul8(const Matmul8Args& a, hipStream_t stream);
size_t matmul8_workspace(int64_t M, int64_t N, int64_t K, int out_bf16);
int matmul8_grid_ok(int64_t M, int64_t N, int64_t K, int out_bf16);

hipError_t launch_clip(const ssd_grad* grads, int64_t n, const ssd_clip_options& opt, float* norm,
                       void* workspace, hipStream_t stream);
size_t clip_workspace(const ssd_grad* grads, int64_t n);

}  // namespace ssd
