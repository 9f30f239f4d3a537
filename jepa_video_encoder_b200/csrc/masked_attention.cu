// Attention under masks: capped scores, a distance bias, causal and prefix
// masks, packed documents, padded and cached clips, shared key heads.
//
// Every mask here leaves each query row one interval [lo, hi) of keys
// (row_keys), so a kernel visits keys between the smallest lo and the largest
// hi of its rows and compares positions only in tiles that an interval cuts.
#include "head_ops.h"

namespace jb {

namespace {

__device__ DevErr g_masked_err;

struct RowKeys {
  int lo, hi;     // allowed keys [lo, hi)
  int pos;        // the row's own position among the keys
  bool written;   // false: a row outside every document
};

__device__ __forceinline__ RowKeys row_keys(const MaskedAttnParams& p, int b, int i) {
  RowKeys r;
  if (p.n_docs > 0) {
    const int* off = p.doc_offsets + static_cast<long long>(b) * (p.n_docs + 1);
    int t = 0, n = p.n_docs + 1;  // t: offsets <= i
    while (n > 0) {
      const int half = n >> 1;
      if (__ldg(off + t + half) <= i) {
        t += half + 1;
        n -= half + 1;
      } else {
        n = half;
      }
    }
    r.pos = i;
    r.written = t > 0 && t <= p.n_docs;
    r.lo = r.hi = 0;
    if (r.written) {
      r.lo = max(__ldg(off + t - 1), 0);
      r.hi = min(__ldg(off + t), p.Nk);
      if (p.causal) {
        const int pre = p.prefix ? max(0, min(__ldg(p.prefix + static_cast<long long>(b) * p.n_docs + t - 1), p.Nk)) : 0;
        r.hi = min(r.hi, max(i + 1, r.lo + pre));
      }
    }
  } else {
    const long long start = p.q_start ? __ldg(p.q_start + b) : p.Nk - p.Nq;
    const long long pos = start + i;
    r.written = true;
    r.pos = static_cast<int>(max(min(pos, 0x7ffffffell), -0x7fffffffll));
    r.lo = 0;
    r.hi = p.kv_len ? min(__ldg(p.kv_len + b), p.Nk) : p.Nk;
    if (p.causal) r.hi = min(r.hi, max(r.pos + 1, p.prefix ? __ldg(p.prefix + b) : 0));
  }
  if (r.hi < r.lo) r.hi = r.lo;
  return r;
}

// Score of one key in the exp2 domain: capped, biased, times log2 e.
__device__ __forceinline__ float finish_score(const MaskedAttnParams& p, float dot, float slope, int pos, int j) {
  float s = dot * p.scale;
  if (p.cap > 0.f) s = p.cap * tanhf(s / p.cap);
  s -= slope * fabsf(static_cast<float>(static_cast<long long>(pos) - j));
  return s * 1.4426950408889634f;
}

// One query row by one warp, straight from the definition: 32 keys at a
// time, one per lane, for the scores; then each lane sums its own output
// dims over the 32 probabilities.  Keys outside [lo, hi) are never read.
template <bool BF>
__device__ void attend_row(const MaskedAttnParams& p, int b, int i, int h, const RowKeys& r, int lane) {
  const int hk = h / (p.hq / p.hk);
  const uint16_t* q = p.q + b * p.q_b + i * p.q_n + h * p.q_h;
  const uint16_t* k = p.k + b * p.k_b + hk * p.k_h;
  const uint16_t* v = p.v + b * p.v_b + hk * p.v_h;
  uint16_t* o = p.out + b * p.o_b + i * p.o_n + h * p.o_h;
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};  // dims lane, lane + 32, ...
  for (int j0 = r.lo; j0 < r.hi; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < r.hi) {
      const uint16_t* kr = k + j * p.k_n;
      float dot = 0.f;
      for (int c = 0; c < p.d; c += 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(q + c), w = *reinterpret_cast<const uint4*>(kr + c);
        const uint32_t au[4] = {a.x, a.y, a.z, a.w}, wu[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dot = fmaf(widen1<BF>(au[e] & 0xffffu), widen1<BF>(wu[e] & 0xffffu), dot);
          dot = fmaf(widen1<BF>(au[e] >> 16), widen1<BF>(wu[e] >> 16), dot);
        }
      }
      s = finish_score(p, dot, slope, r.pos, j);
    }
    float mx = s;
    bool nan = s != s;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
    if (__any_sync(0xffffffffu, nan)) mx = NAN;
    const float m_new = (m != m || mx != mx) ? NAN : fmaxf(m, mx);
    const float alpha = m == m_new ? 1.f : exp2f(m - m_new);
    // while every score is -inf nothing is added: a row of such scores ends as 0 / 0, as the definition has it
    const float pr = j < r.hi && m_new != -INFINITY ? exp2f(s - m_new) : 0.f;
    m = m_new;
    float sum = pr;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
    l = l * alpha + sum;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] *= alpha;
    const int n = min(32, r.hi - j0);
    for (int t = 0; t < n; ++t) {
      const float pt = __shfl_sync(0xffffffffu, pr, t);
      const uint16_t* vr = v + (j0 + t) * p.v_n;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (lane + 32 * c < p.d) acc[c] = fmaf(pt, widen1<BF>(vr[lane + 32 * c]), acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < p.d) o[lane + 32 * c] = pack1<BF>(r.hi > r.lo ? acc[c] / l : 0.f);
}

}  // namespace

template <bool BF>
__global__ void __launch_bounds__(128) masked_rows_kernel(const MaskedAttnParams p) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + warp;
  if (row >= static_cast<long long>(p.B) * p.Nq * p.hq) return;
  const int h = static_cast<int>(row % p.hq);
  const long long bi = row / p.hq;
  const int b = static_cast<int>(bi / p.Nq), i = static_cast<int>(bi % p.Nq);
  const RowKeys r = row_keys(p, b, i);
  if (r.written) attend_row<BF>(p, b, i, h, r, lane);
}

int masked_attention_take_error(unsigned* code) {
  DevErr h{0, 0};
  if (cudaMemcpyFromSymbol(&h, g_masked_err, sizeof(h)) != cudaSuccess) return JEPA_B200_ERR_CUDA;
  *code = h.code;
  if (h.code != DERR_NONE) {
    const DevErr zero{0, 0};
    if (cudaMemcpyToSymbol(g_masked_err, &zero, sizeof(zero)) != cudaSuccess) return JEPA_B200_ERR_CUDA;
  }
  return JEPA_B200_OK;
}

int launch_masked_attention(const MaskedAttnParams& p, bool bf16, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.B) * p.Nq * p.hq;
  const long long blocks = (rows + 3) / 4;
  if (blocks > 0x7fffffffll) return JEPA_B200_ERR_SHAPE;
  const auto kern = bf16 ? masked_rows_kernel<true> : masked_rows_kernel<false>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, st, 1, p) == cudaSuccess
             ? JEPA_B200_OK
             : JEPA_B200_ERR_CUDA;
}

}  // namespace jb
