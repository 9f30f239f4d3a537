// Rotary positions of heads, and norms of query and key heads with the
// rotation in the same pass.
//
// A head's d values are normalised (none, RMS or LayerNorm) and its first
// rot dims turned in pairs:
//   (x0, x1) -> factor * (x0 cos - x1 sin, x0 sin + x1 cos).
// The angle is exact: a pair's frequency is a 64-bit binary fraction of a
// turn, its product with the integer position modulo 2^64 is the phase, and
// the upper 32 bits of that, as a signed number of half-turns in [-1, 1),
// go to sincospif.
#include "internal.h"
#include "head_ops.h"

namespace jb {

namespace {

__device__ __forceinline__ float2 pair_cos_sin(const RopeParams& r, int pair, int b, int n) {
  const int a = r.axis ? r.axis[pair] : 0;
  const long long at = (a < r.n_axes ? a : 0) * r.pos_stride_axis + b * r.pos_stride_b + n;
  const long long pos = r.pos_i64 ? static_cast<const long long*>(r.pos)[at] : static_cast<const int*>(r.pos)[at];
  const unsigned long long phase = static_cast<unsigned long long>(pos) * r.turns[pair];
  const float half_turns = static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * r.factor, s * r.factor);
}

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace

// One warp per head of a token, whatever the strides: lane l holds elements
// l, l + 32, ...; the row passes through shared memory for the pairs.
template <typename T>
__global__ void __launch_bounds__(128) head_rows_kernel(const HeadOpParams p) {
  __shared__ float rows[4][kMaxHeadDim];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * 4 + warp;
  const int heads = p.t[0].heads + p.t[1].heads;
  const long long token = unit / heads;
  if (token >= static_cast<long long>(p.B) * p.N) return;
  int h = static_cast<int>(unit - token * heads);
  const int w = h >= p.t[0].heads ? 1 : 0;
  if (w) h -= p.t[0].heads;
  const HeadTensor& x = p.t[w];
  const int b = static_cast<int>(token / p.N), n = static_cast<int>(token - static_cast<long long>(b) * p.N);
  const T* src = static_cast<const T*>(x.in) + b * x.in_b + n * x.in_n + h * x.in_h;
  T* dst = static_cast<T*>(x.out) + b * x.out_b + n * x.out_n + h * x.out_h;
  float* row = rows[warp];
  float sum = 0.f;
  for (int i = lane; i < p.d; i += 32) {
    const float v = widen<T>(src[i]);
    row[i] = v;
    sum += v;
  }
  if (p.norm != NORM_NONE) {
    const float mean = p.norm == NORM_LAYER ? warp_sum(sum) / p.d : 0.f;
    float sq = 0.f;
    for (int i = lane; i < p.d; i += 32) {
      const float c = row[i] - mean;
      sq = fmaf(c, c, sq);
    }
    const float inv = rsqrtf(warp_sum(sq) / p.d + p.eps);
    for (int i = lane; i < p.d; i += 32) {
      const float y = (row[i] - mean) * inv * x.weight[h * x.weight_h + i];
      row[i] = x.bias ? y + x.bias[h * x.bias_h + i] : y;
    }
  }
  __syncwarp();
  const int half = p.rope.rot_dim / 2;
  for (int i = lane; i < p.d; i += 32)
    if (i >= p.rope.rot_dim) dst[i] = narrow<T>(row[i]);
  for (int i = lane; i < half; i += 32) {
    const float2 cs = pair_cos_sin(p.rope, i, b, n);
    const int i0 = p.rope.half_layout ? i : 2 * i, i1 = p.rope.half_layout ? i + half : 2 * i + 1;
    const float x0 = row[i0], x1 = row[i1];
    dst[i0] = narrow<T>(x0 * cs.x - x1 * cs.y);
    dst[i1] = narrow<T>(x0 * cs.y + x1 * cs.x);
  }
}

namespace {
template <typename T>
int launch_rows(const HeadOpParams& p, cudaStream_t st) {
  const long long units = static_cast<long long>(p.B) * p.N * (p.t[0].heads + p.t[1].heads);
  const long long blocks = (units + 3) / 4;
  if (blocks > 0x7fffffffll) return JEPA_B200_ERR_SHAPE;
  return launch_pdl(head_rows_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, st, 1, p) == cudaSuccess
             ? JEPA_B200_OK
             : JEPA_B200_ERR_CUDA;
}
}  // namespace

int launch_head_op(const HeadOpParams& p, int dtype, cudaStream_t st) {
  switch (dtype) {
    case JEPA_B200_F32: return launch_rows<float>(p, st);
    case JEPA_B200_F16: return launch_rows<__half>(p, st);
    default: return launch_rows<__nv_bfloat16>(p, st);
  }
}

}  // namespace jb
