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
#include "head_ops.h"
#include "internal.h"

namespace jb {

namespace {

__device__ __forceinline__ float2 pair_cos_sin(const RopeParams& r, int pair, int b, int n) {
  const long long at = r.axis[pair] * r.pos_stride_axis + b * r.pos_stride_b + n;
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
// l, l + 32, ...; the row passes through shared memory for the pairs.  For
// operands that the kernel below cannot read in wide pieces.
template <typename T>
__global__ void __launch_bounds__(128) head_rows_kernel(const __grid_constant__ HeadOpParams p) {
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

// The wide form.  A head's d values are cut into chunks of VEC elements (16
// or 8 bytes); `lanes` threads share a head and each holds two chunks, for
// the half layout the two that hold the partners of its pairs, so that a
// value's partner is in the thread that turns it.  A thread takes R heads of
// one token: it starts their loads, the block makes its tokens' cosines and
// sines in shared memory meanwhile (once for all heads), and each thread reads
// its own ones, its weights and its addresses once for the R heads.  Bound by
// memory.
struct WideParams {
  HeadOpParams op;
  int tokens_per, tokens;  // tokens a block takes, all of them
  int lanes, lanes_log2;   // threads a head: a power of two
  int pairs_split;         // half layout: chunks of the first half of the turned dims
  int chunks;              // chunks a head
  int slots0, slots;       // groups of R heads a token: of t[0], of both
  Div by_slots, by_n, by_pairs;
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Chunk {
  T v[VEC];
};

constexpr int kWideThreads = 128;
// Blocks an SM is to hold at least (0: no bound).  The norms of 16-bit heads
// would else take 156 registers (12548 x 32 heads of 64: 31 us, with four
// blocks 28); the other instances lose 5 to 20 % by a bound.
template <int VEC, int R, int NORM>
constexpr int kWideBlocks = NORM != NORM_NONE && VEC == 8 && R == 4 ? 4 : 0;

template <typename T, int VEC, int R, int NORM, bool SPLIT>
__global__ void __launch_bounds__(kWideThreads, kWideBlocks<VEC, R, NORM>) head_wide_kernel(const __grid_constant__ WideParams wp) {
  using C = Chunk<T, VEC>;
  extern __shared__ float2 cs[];  // [tokens_per][pairs]
  const HeadOpParams& p = wp.op;
  pdl_wait();
  pdl_trigger();
  const int tok0 = blockIdx.x * wp.tokens_per;
  const int n_tok = min(wp.tokens_per, wp.tokens - tok0);
  const int lane = threadIdx.x & (wp.lanes - 1);
  const int half = p.rope.rot_dim >> 1;
  int ca, cb;  // this thread's chunks
  if (SPLIT) {
    const bool turned = lane < wp.pairs_split;
    ca = turned ? lane : 2 * lane;
    cb = turned ? lane + wp.pairs_split : 2 * lane + 1;
  } else {
    const int mid = (wp.chunks + 1) >> 1;
    ca = lane < mid ? lane : wp.chunks;
    cb = lane + mid;
  }
  const bool has_a = ca < wp.chunks, has_b = has_a && cb < wp.chunks;
  const int ea = ca * VEC, eb = cb * VEC;
  const int units = n_tok * wp.slots;
  const int first = threadIdx.x >> wp.lanes_log2, step = kWideThreads >> wp.lanes_log2;
  for (int u0 = 0; u0 < units; u0 += step) {
    const int u = u0 + first;
    const bool on = u < units;
    const int tok = on ? static_cast<int>(wp.by_slots(u)) : 0;
    const int slot = on ? u - tok * wp.slots : 0;
    const bool second = slot >= wp.slots0;
    const HeadTensor& x = p.t[second ? 1 : 0];
    const int h0 = second ? slot - wp.slots0 : slot, h_step = second ? wp.slots - wp.slots0 : wp.slots0;
    const int token = tok0 + tok;
    const int b = static_cast<int>(wp.by_n(token)), n = token - b * p.N;
    C xa[R], xb[R];
    {
      const T* src = static_cast<const T*>(x.in) + b * x.in_b + n * x.in_n + h0 * x.in_h;
      const long long by = h_step * x.in_h;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (on && has_a) xa[r] = *reinterpret_cast<const C*>(src + ea);
        if (on && has_b) xb[r] = *reinterpret_cast<const C*>(src + eb);
        src += by;
      }
    }
    if (u0 == 0 && half > 0) {
      for (int i = threadIdx.x; i < n_tok * half; i += kWideThreads) {
        const int t = static_cast<int>(wp.by_pairs(i));
        const int tk = tok0 + t;
        const int tb = static_cast<int>(wp.by_n(tk));
        cs[i] = pair_cos_sin(p.rope, i - t * half, tb, tk - tb * p.N);
      }
      __syncthreads();
    }
    // cosines and sines: of pairs ea .. ea + VEC - 1 (half layout), or of the
    // pairs inside the two chunks; a pair that is not turned keeps (1, 0) and
    // is passed by below
    float2 ta[VEC];
    bool turn_a = false, turn_b = false;  // any pair of the chunk is turned
    if (on && has_a && half > 0) {
      const float2* row = cs + tok * half;
      if (SPLIT) {
        turn_a = lane < wp.pairs_split;
        if (turn_a) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) ta[e] = row[ea + e];
        }
      } else {
        turn_a = ea < p.rope.rot_dim;
        turn_b = has_b && eb < p.rope.rot_dim;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          if ((ea >> 1) + e < half) ta[e] = row[(ea >> 1) + e];
          if (has_b && (eb >> 1) + e < half) ta[VEC / 2 + e] = row[(eb >> 1) + e];
        }
      }
    }
    float wa[VEC], wb[VEC], ba[VEC], bb[VEC];
    T* dst = static_cast<T*>(x.out) + b * x.out_b + n * x.out_n + h0 * x.out_h;
    const long long out_by = h_step * x.out_h;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float a[VEC], c[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        a[e] = on && has_a ? widen<T>(xa[r].v[e]) : 0.f;
        c[e] = on && has_b ? widen<T>(xb[r].v[e]) : 0.f;
      }
      if constexpr (NORM != NORM_NONE) {
        if (r == 0 || x.weight_h != 0) {
          const float* wt = x.weight + (h0 + r * h_step) * x.weight_h;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            wa[e] = on && has_a ? __ldg(wt + ea + e) : 0.f;
            wb[e] = on && has_b ? __ldg(wt + eb + e) : 0.f;
          }
        }
        if (r == 0 || x.bias_h != 0) {
          const float* bs = x.bias ? x.bias + (h0 + r * h_step) * x.bias_h : nullptr;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            ba[e] = bs && on && has_a ? __ldg(bs + ea + e) : 0.f;
            bb[e] = bs && on && has_b ? __ldg(bs + eb + e) : 0.f;
          }
        }
        const float inv_d = 1.0f / p.d;
        if (NORM == NORM_LAYER) {
          float mean = 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) mean += a[e] + c[e];
          for (int o = wp.lanes >> 1; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
          mean *= inv_d;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            a[e] = has_a ? a[e] - mean : 0.f;
            c[e] = has_b ? c[e] - mean : 0.f;
          }
        }
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) sq = fmaf(a[e], a[e], fmaf(c[e], c[e], sq));
        for (int o = wp.lanes >> 1; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        const float inv = rsqrtf(fmaf(sq, inv_d, p.eps));
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          a[e] = fmaf(a[e] * inv, wa[e], ba[e]);
          c[e] = fmaf(c[e] * inv, wb[e], bb[e]);
        }
      }
      if (SPLIT) {
        if (turn_a) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float x0 = a[e], x1 = c[e];
            a[e] = x0 * ta[e].x - x1 * ta[e].y;
            c[e] = x0 * ta[e].y + x1 * ta[e].x;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          if (turn_a && (ea >> 1) + e < half) {
            const float x0 = a[2 * e], x1 = a[2 * e + 1];
            a[2 * e] = x0 * ta[e].x - x1 * ta[e].y;
            a[2 * e + 1] = x0 * ta[e].y + x1 * ta[e].x;
          }
          if (turn_b && (eb >> 1) + e < half) {
            const float2 t = ta[VEC / 2 + e];
            const float x0 = c[2 * e], x1 = c[2 * e + 1];
            c[2 * e] = x0 * t.x - x1 * t.y;
            c[2 * e + 1] = x0 * t.y + x1 * t.x;
          }
        }
      }
      if (on && has_a) {
        C y;
#pragma unroll
        for (int e = 0; e < VEC; ++e) y.v[e] = narrow<T>(a[e]);
        *reinterpret_cast<C*>(dst + ea) = y;
        if (has_b) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) y.v[e] = narrow<T>(c[e]);
          *reinterpret_cast<C*>(dst + eb) = y;
        }
      }
      dst += out_by;
    }
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

// Whether every chunk of `vec` elements of the call's operands is aligned and
// holds whole pairs, or whole runs of a half's pairs.
template <typename T>
bool chunks_fit(const HeadOpParams& p, int vec) {
  const int half = p.rope.rot_dim / 2;
  if (p.d % vec != 0 || (half > 0 && (p.rope.half_layout ? half % vec != 0 : vec % 2 != 0))) return false;
  for (const HeadTensor& t : p.t) {
    if (t.heads == 0) continue;
    const uintptr_t mask = sizeof(T) * vec - 1;
    if ((reinterpret_cast<uintptr_t>(t.in) & mask) || (reinterpret_cast<uintptr_t>(t.out) & mask)) return false;
    for (const long long s : {p.B > 1 ? t.in_b : 0, p.N > 1 ? t.in_n : 0, t.heads > 1 ? t.in_h : 0,
                              p.B > 1 ? t.out_b : 0, p.N > 1 ? t.out_n : 0, t.heads > 1 ? t.out_h : 0})
      if (s % vec != 0) return false;
  }
  return true;
}

template <typename T, int VEC, int R, int NORM, bool SPLIT>
int launch_wide_as(const WideParams& wp, cudaStream_t st) {
  const unsigned blocks = static_cast<unsigned>((wp.tokens + wp.tokens_per - 1) / wp.tokens_per);
  const size_t smem = static_cast<size_t>(wp.tokens_per) * (wp.op.rope.rot_dim / 2) * sizeof(float2);
  return launch_pdl(head_wide_kernel<T, VEC, R, NORM, SPLIT>, dim3(blocks), dim3(kWideThreads), smem, st, 1, wp) ==
                 cudaSuccess
             ? JEPA_B200_OK
             : JEPA_B200_ERR_CUDA;
}

template <typename T, int VEC, int R>
int launch_wide_r(WideParams& wp, cudaStream_t st) {
  const HeadOpParams& p = wp.op;
  wp.slots0 = p.t[0].heads / R;
  wp.slots = wp.slots0 + p.t[1].heads / R;
  wp.by_slots.set(wp.slots);
  const long long per_token = static_cast<long long>(wp.slots) * wp.lanes;
  const long long fit = kWideThreads / per_token;
  wp.tokens_per = static_cast<int>(fit < 1 ? 1 : (fit > 32 ? 32 : fit));
  const bool split = wp.pairs_split > 0;
  switch (p.norm) {
    case NORM_NONE:
      return split ? launch_wide_as<T, VEC, R, NORM_NONE, true>(wp, st) : launch_wide_as<T, VEC, R, NORM_NONE, false>(wp, st);
    case NORM_RMS:
      return split ? launch_wide_as<T, VEC, R, NORM_RMS, true>(wp, st) : launch_wide_as<T, VEC, R, NORM_RMS, false>(wp, st);
    default:
      return split ? launch_wide_as<T, VEC, R, NORM_LAYER, true>(wp, st) : launch_wide_as<T, VEC, R, NORM_LAYER, false>(wp, st);
  }
}

template <typename T, int VEC>
int launch_wide(const HeadOpParams& p, cudaStream_t st) {
  WideParams wp;
  wp.op = p;
  const int h0 = p.t[0].heads, h1 = p.t[1].heads, half = p.rope.rot_dim / 2;
  wp.chunks = p.d / VEC;
  wp.pairs_split = half > 0 && p.rope.half_layout ? half / VEC : 0;
  const int need = wp.pairs_split + (wp.chunks - 2 * wp.pairs_split + 1) / 2;
  wp.lanes = 1;
  wp.lanes_log2 = 0;
  while (wp.lanes < need) wp.lanes *= 2, ++wp.lanes_log2;
  if (wp.lanes > 32) return launch_rows<T>(p, st);
  wp.tokens = p.B * p.N;
  wp.by_n.set(p.N);
  wp.by_pairs.set(half > 0 ? half : 1);
  // several heads a thread once that still gives every SM several blocks
  const long long threads = static_cast<long long>(h0 + h1) * wp.lanes * wp.tokens;
  const long long enough = static_cast<long long>(num_sms()) * 4 * kWideThreads;
  if (threads >= 4 * enough && h0 % 4 == 0 && h1 % 4 == 0) return launch_wide_r<T, VEC, 4>(wp, st);
  if (threads >= 2 * enough && h0 % 2 == 0 && h1 % 2 == 0) return launch_wide_r<T, VEC, 2>(wp, st);
  return launch_wide_r<T, VEC, 1>(wp, st);
}

template <typename T>
int launch_typed(const HeadOpParams& p, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  if (chunks_fit<T>(p, kVec)) return launch_wide<T, kVec>(p, st);
  if (chunks_fit<T>(p, kVec / 2)) return launch_wide<T, kVec / 2>(p, st);
  return launch_rows<T>(p, st);
}
}  // namespace

int launch_head_op(const HeadOpParams& p, int dtype, cudaStream_t st) {
  switch (dtype) {
    case JEPA_B200_F32: return launch_typed<float>(p, st);
    case JEPA_B200_F16: return launch_typed<__half>(p, st);
    default: return launch_typed<__nv_bfloat16>(p, st);
  }
}

}  // namespace jb
