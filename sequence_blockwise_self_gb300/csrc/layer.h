// layer.h -- launch interface of the layer operators around the attention:
// rotary positions (rope.cu), the norms before and after a block with its
// gate and residual scale (block_norm_fwd.cu, block_norm_bwd*.cu), the
// gradient norm and clipping (grad_clip.cu).
#pragma once
#include "kernels.h"

namespace ra {

// Element types of the layer operators (RING_ATTN_DTYPE_* of the C ABI).
enum LayerDtype : int { kBf16 = 0, kFp16 = 1, kFp32 = 2 };
inline int dtype_bytes(int t) { return t == kFp32 ? 4 : 2; }

// ------------------------------------------------------- rotary positions
// One of q, k, v: [B][H][L][d] views, strides in elements, last one 1.
struct RopeTensor {
  const void* in = nullptr;
  void* out = nullptr;
  int H = 0;  // 0: absent
  long long ib = 0, ih = 0, il = 0, ob = 0, oh = 0, ol = 0;
};

struct RopeArgs {
  RopeTensor t[3];  // q, k (rotated), v (copied)
  int B = 0, L = 0, d = 0, R = 0;
  int dtype = 0, interleaved = 0, inverse = 0;
  const uint64_t* phase = nullptr;  // [R/2] turns a position, as 64-bit fractions
  float factor = 1.f;               // of cos and sin
  // positions: device [B or 1][L] (32 or 64 bits), or the affine map
  const void* pos = nullptr;
  int pos64 = 0;
  long long pos_b = 0;
  int split = 0;
  long long base0 = 0, base1 = 0, step = 1;
  int n_sms = 0;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream);

// ------------------------------------------- norms, gate and residual scale
enum NormFlags : int { kNormLayer = 1, kNormPost = 2, kNormPre = 4, kNormGateSigmoid = 8 };
constexpr int kNormMaxD = 8192;

struct BlockNormArgs {
  // forward: x, a -> y, h, stats; a null: y = x is not written
  // backward: dy, dh, y, a, stats -> dx, da, dgate and the weight gradients
  const void *x = nullptr, *a = nullptr, *gate = nullptr;
  const float *post_w = nullptr, *post_b = nullptr, *pre_w = nullptr, *pre_b = nullptr;
  void *y = nullptr, *h = nullptr;
  float* stats = nullptr;  // [2 or 4][M]: rstd post, rstd pre, mean post, mean pre
  const void *dy = nullptr, *dh = nullptr;
  void *dx = nullptr, *da = nullptr, *dgate = nullptr;
  float *dpost_w = nullptr, *dpost_b = nullptr, *dpre_w = nullptr, *dpre_b = nullptr;
  long long ld_x = 0, ld_a = 0, ld_gate = 0, ld_y = 0, ld_h = 0, ld_dy = 0, ld_dh = 0, ld_dx = 0, ld_da = 0;
  long long M = 0, gate_rows = 0;  // gate_rows 0: no gate; row m uses gate row m / (M / gate_rows)
  int D = 0, flags = 0, dt_x = 0, dt_a = 0, dt_gate = 0;
  float scale = 1.f, eps = 0.f;
  float* partial = nullptr;  // backward workspace
  int n_sms = 0;             // (forward)
};
cudaError_t launch_block_norm_fwd(const BlockNormArgs& a, cudaStream_t stream);
cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, cudaStream_t stream);
size_t block_norm_bwd_workspace(long long M, int D, long long gate_rows, int flags);

// ------------------------------------------- gradient norm and clipping
struct GradTensor {
  const void* in;
  void* out;
  long long n;
  int dt_in, dt_out;
};
struct GradArgs {
  const GradTensor* tensors = nullptr;  // host array
  int n_tensors = 0;
  float max_norm = 0.f;
  float* norm = nullptr;
  double* partial = nullptr;  // workspace
};
size_t grad_workspace_bytes(int n_tensors);
cudaError_t launch_grad_norm(const GradArgs& a, cudaStream_t stream);
cudaError_t launch_grad_scale(const GradArgs& a, cudaStream_t stream);
cudaError_t launch_grad_clip(const GradArgs& a, cudaStream_t stream);

}  // namespace ra
