// Host-side declarations of the per-head calls: rotation and norms
// (rope_norm.cu) and attention under masks (masked_attention.cu).
#pragma once

#include "internal.h"

namespace jb {

constexpr int kMaxHeadDim = 256;  // of the rotation and the norms

enum { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

struct RopeParams {
  int rot_dim, half_layout, n_axes, pos_i64;
  const void* pos;
  long long pos_stride_axis, pos_stride_b;
  float factor;
  unsigned char axis[kMaxHeadDim / 2];
  unsigned long long turns[kMaxHeadDim / 2];  // by value: a plan needs no device memory
};

// One tensor of a call: heads == 0 for a call that has only one.
struct HeadTensor {
  const void* in;
  void* out;
  long long in_b, in_n, in_h, out_b, out_n, out_h;
  int heads;
  const float* weight;
  const float* bias;
  long long weight_h, bias_h;
};

// x / d for 0 <= x < 2^31 by a multiplication (Granlund and Montgomery's
// division by an invariant): d <= 2^s, m = 2^32 (2^s - d) / d + 1.
struct Div {
  unsigned d, m, s;
  void set(unsigned by) {
    d = by;
    s = 0;
    while ((1ull << s) < by) ++s;
    m = static_cast<unsigned>(((1ull << 32) * ((1ull << s) - by)) / by + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ unsigned operator()(unsigned x) const {
    return static_cast<unsigned>((static_cast<unsigned long long>(__umulhi(x, m)) + x) >> s);
  }
#endif
};

struct HeadOpParams {
  HeadTensor t[2];
  int B, N, d, norm;
  float eps;
  RopeParams rope;
};

int launch_head_op(const HeadOpParams& p, int dtype, cudaStream_t st);

struct MaskedAttnParams {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  long long q_b, q_n, q_h, k_b, k_n, k_h, v_b, v_n, v_h, o_b, o_n, o_h;
  int B, Nq, Nk, hq, hk, d;
  float scale, cap;  // cap 0: none
  int causal, n_docs;
  const float* slopes;
  const int *prefix, *doc_offsets, *kv_len, *q_start;
  unsigned long long timeout_ns;
};

int launch_masked_attention(const MaskedAttnParams& p, bool bf16, cudaStream_t st);
// The status word of the masked-attention kernels on the current device:
// read and cleared.
int masked_attention_take_error(unsigned* code);

}  // namespace jb
