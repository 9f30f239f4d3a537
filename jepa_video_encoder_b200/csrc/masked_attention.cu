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
// dims over the 32 probabilities.  Keys outside [lo, hi) are never read.  The
// time that it takes goes to *spent as it passes, for warps that wait meanwhile.
template <bool BF>
__device__ void attend_row(const MaskedAttnParams& p, int b, int i, int h, const RowKeys& r, int lane,
                           unsigned long long* spent = nullptr) {
  unsigned long long since = spent ? globaltimer() : 0;
  const int hk = h / (p.hq / p.hk);
  const uint16_t* q = p.q + b * p.q_b + i * p.q_n + h * p.q_h;
  const uint16_t* k = p.k + b * p.k_b + hk * p.k_h;
  const uint16_t* v = p.v + b * p.v_b + hk * p.v_h;
  uint16_t* o = p.out + b * p.o_b + i * p.o_n + h * p.o_h;
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};  // dims lane, lane + 32, ...
  for (int j0 = r.lo; j0 < r.hi; j0 += 32) {
    if (spent && lane == 0) {
      const unsigned long long now = globaltimer();
      atomicAdd(spent, now - since);
      since = now;
    }
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

// One warp a row.  For more than a few queries over no keys, or over keys that
// no tensor map describes (one key broadcast along the token axis).
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

// ------------------------------------------------------------ tensor cores --
// 128-query tiles on tcgen05.  A work item is 256 query rows (two tiles) of
// one head.  One CTA an SM (registers, TMEM and shared memory are its own);
// the grid has a CTA for every item, and a running CTA takes over items of
// CTAs that have not started, so that items of unequal length even out.
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1, one thread a row: the
//                   row's 128 scores of a key tile come from TMEM into
//                   registers at once, so maxima and sums need no exchange;
//   warp 8          TMA: Q tiles, then K and V tiles of 128 keys (V as it
//                   lies, keys by dims: the MN-major B operand of P V);
//   warps 9, 10     MMA: S = Q K^T and O += P V, P from TMEM;
//   warp 11         the items.
// Heads up to 64 dims: S, P and O of both tiles lie side by side in TMEM and
// S of the next key tile is computed during the softmax of this one.  Heads
// up to 128: P takes the place of S, whose product is issued behind P V.
// O is rescaled only when a row's maximum grew by more than 2^8 (P stays <=
// 256, the division by the row sum makes it exact again).  P is rounded to
// the 16-bit type for its product; the row sum is of the unrounded values.
//
// What bounds it: heads of 128, the tensor cores (9472 keys, 8 heads, bf16:
// 287 us, 1280 TFLOP/s, beside 1378 for a matrix product sustained under the
// power limit); heads of 64, the softmax (252 us in f16, 729 TFLOP/s; 259 in
// bf16, whose part of the exponentials costs a product more): a pair of
// key tiles takes 2900 clocks, in which the special-function unit is busy for
// half, the issue slots for half and the tensor cores for a third, and the
// rest is the two softmax warps of a scheduler waiting on the same things.
// Sixteen softmax warps with two or four threads a row fit only with spilled
// registers, or read the scores twice, and gained nothing (251 to 292 us);
// the next tile's scores loaded early, with the exponentials (255 to 278 us).
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;
constexpr int kBlockBytes = 128 * 128;  // [128 rows x 64 dims] of 16 bits

// Score transforms of a kernel instance.
constexpr int kCap = 1, kBias = 2;

constexpr int kOutBytes = 32 * 128;

template <int NB>  // 64-dim blocks of a head: 1 or 2
struct TileCfg {
  static constexpr int kStages = NB == 1 ? 4 : 2;
  static constexpr int kQBufs = NB == 1 ? 2 : 1;
  static constexpr int kTileBytes = NB * kBlockBytes;
  static constexpr int kOffQ = 0;  // [buffer][tile]
  static constexpr int kOffK = kOffQ + kQBufs * 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffOut = kOffV + kStages * kTileBytes;  // [softmax warp] 32 rows of 64 dims on their way out
  static constexpr int kSmem = kOffOut + 8 * kOutBytes + 1024;
  static constexpr bool kAliasP = NB == 2;
  static constexpr uint32_t kColS = 0, kColO = 256, kColP = NB == 1 ? 384 : 0;
  static constexpr uint32_t kStepO = 64 * NB, kStepP = NB == 1 ? 64 : 128;
};
// Three warpgroups; the softmax ones take registers from the third: 2 * 128 *
// 224 + 128 * 56 = 384 * 168, what the launch gives.
constexpr int kTileThreads = 12 * 32;
constexpr int kRegsSoftmax = 224, kRegsOther = 56;

struct TileParams {
  MaskedAttnParams a;
  int n_pairs, n_items;        // 256-row groups of a head; items = B * hq * n_pairs
  int q_step, k_step, v_step, o_step;  // bit 0: batch, bit 1: token, bit 2: head axis has a stride (0: broadcast)
};

// The key tiles of one item: tile j holds keys lo + 128 j ..; query tile g
// needs tiles [first[g], last[g]).
struct Item {
  int b, h, q0, lo, hi, n, first[2], last[2];
};

__device__ __forceinline__ Item load_item(const TileParams& p, int idx, int lane) {
  const MaskedAttnParams& a = p.a;
  Item it;
  const int bh_all = a.B * a.hq;
  int pair, bh;
  if (a.causal) {  // the longest rows of every head first
    pair = p.n_pairs - 1 - idx / bh_all;
    bh = idx % bh_all;
  } else {         // neighbours share a head's keys
    bh = idx / p.n_pairs;
    pair = idx - bh * p.n_pairs;
  }
  it.b = bh / a.hq;
  it.h = bh - it.b * a.hq;
  it.q0 = pair * 256;
  // lanes 0..3: first key of tile 0's first row, end of its last row, the same of tile 1
  int v = 0;
  const int g = (lane >> 1) & 1;
  int r0 = it.q0 + 128 * g, r1 = min(r0 + 128, a.Nq) - 1;
  if (a.n_docs > 0) {
    const int* off = a.doc_offsets + static_cast<long long>(it.b) * (a.n_docs + 1);
    r0 = max(r0, __ldg(off));
    r1 = min(r1, __ldg(off + a.n_docs) - 1);
  }
  if (lane < 4 && r0 <= r1) {
    const RowKeys r = row_keys(a, it.b, (lane & 1) ? r1 : r0);
    v = (lane & 1) ? r.hi : r.lo;
  }
  int lo[2], hi[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    lo[t] = __shfl_sync(0xffffffffu, v, 2 * t);
    hi[t] = __shfl_sync(0xffffffffu, v, 2 * t + 1);
  }
  const bool any0 = hi[0] > lo[0], any1 = hi[1] > lo[1];
  it.lo = any0 ? (any1 ? min(lo[0], lo[1]) : lo[0]) : lo[1];
  it.hi = max(any0 ? hi[0] : 0, any1 ? hi[1] : 0);
  it.n = any0 || any1 ? (it.hi - it.lo + 127) >> 7 : 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const bool any = t ? any1 : any0;
    it.first[t] = any ? (lo[t] - it.lo) >> 7 : 0;
    it.last[t] = any ? (hi[t] - it.lo + 127) >> 7 : 0;
  }
  return it;
}

// tanh(z) = z P(z^2) for |z| <= 1; P by weighted least squares driven to equal
// ripple (softmax_fit.py): relative error 6.9e-6 with 5 terms (bf16
// probabilities), 5.9e-7 with 6.
template <bool BF>
struct TanhPoly;
template <>
struct TanhPoly<true> {
  static constexpr int kTerms = 5;
  static __device__ __forceinline__ float c(int k) {
    constexpr float v[5] = {0.999993089590493f, -0.3329806545269403f, 0.13036811735219106f, -0.04481755800903122f,
                            0.009036424468049704f};
    return v[k];
  }
};
template <>
struct TanhPoly<false> {
  static constexpr int kTerms = 6;
  static __device__ __forceinline__ float c(int k) {
    constexpr float v[6] = {0.9999994136209384f, -0.3332904241225214f, 0.13281434020653068f,
                            -0.051605676150095f, 0.016743116205360516f, -0.0030670603865920864f};
    return v[k];
  }
};

// How the exponent of a score is made from its register: s * c - m of a raw
// dot product, s - m of a finished score, or the capped score of a raw dot
// product by its polynomial, s * Q(s^2) - m.
enum { FROM_DOT = 0, FROM_SCORE = 1, FROM_CAP = 2 };

// cap * log2 e * tanh(z) of a raw dot product s, z = s scale / cap, in two forms:
// s scale log2 e P(z^2) for |z| <= 1, cap * log2 e * (1 - 2 / (1 + e^2z)) beyond.
// The second alone would lose a small score in the cap's rounding, cap * 2^-23:
// at a cap of 1e6 a score of 1 came out as 0.95.
struct CapScore {
  float zs, c, kl;  // scale / cap, scale * log2 e, cap * log2 e
  __device__ __forceinline__ void init(float scale, float cap) {
    zs = scale / cap;
    c = scale * kLog2e;
    kl = cap * kLog2e;
  }
  __device__ __forceinline__ float operator()(float s) const {
    const float z = s * zs, t = z * z;
    float y = TanhPoly<false>::c(TanhPoly<false>::kTerms - 1);
#pragma unroll
    for (int k = TanhPoly<false>::kTerms - 2; k >= 0; --k) y = fmaf(y, t, TanhPoly<false>::c(k));
    const float far = fmaf(-2.0f * kl, rcp_approx(1.0f + ex2_approx(z * (2.0f * kLog2e))), kl);
    return fabsf(z) <= 1.0f ? s * c * y : far;
  }
};

// Coefficients of the first form as a polynomial s Q(s^2), and the largest |s|
// that it serves.  That is the one of |z| = 1; where scale / cap is so small
// that the last coefficients leave f32's normal range they are dropped, and it
// is the z whose first dropped term is 2^-21 of the score (0.0012 for the linear
// term alone, caps of 1e17 and more).  None (-1) where they would be infinite.
template <bool BF>
struct CapPoly {
  uint64_t q[TanhPoly<BF>::kTerms];
  float most;
  __device__ __forceinline__ void init(float scale, float cap) {
    constexpr float kDropped[5] = {0.0012f, 0.043f, 0.14f, 0.26f, 0.37f};
    const float zs = scale / cap;
    float f = scale * kLog2e, z = 1.0f;
    bool overflow = !(fabsf(f) < 1e36f);
#pragma unroll
    for (int k = 0; k < TanhPoly<BF>::kTerms; ++k) {
      if (k > 0) {
        f *= zs * zs;
        if (z == 1.0f && !(fabsf(f) > 1e-35f)) z = kDropped[k - 1];
      }
      const float v = z < 1.0f ? 0.0f : TanhPoly<BF>::c(k) * f;
      q[k] = f2_pack(v, v);
    }
    overflow |= !(fabsf(f) < 1e36f);
    most = overflow ? -1.0f : z / fabsf(zs);
  }
  __device__ __forceinline__ bool fits(float big) const { return big <= most; }
  // Q(s^2) of two scores
  __device__ __forceinline__ uint64_t slope(uint64_t s) const {
    const uint64_t t = f2_mul(s, s);
    uint64_t y = q[TanhPoly<BF>::kTerms - 1];
#pragma unroll
    for (int k = TanhPoly<BF>::kTerms - 2; k >= 0; --k) y = f2_fma(y, t, q[k]);
    return y;
  }
};

// Raw dot products in s[] to scores in the exp2 domain.
template <int MODE, bool BF>
__device__ __forceinline__ void finish_scores(float (&s)[128], const MaskedAttnParams& a, const CapPoly<BF>& cap, bool poly,
                                              float c, float slope2, float dist0) {
  if constexpr ((MODE & kCap) != 0) {
    if (poly) {
#pragma unroll
      for (int e = 0; e < 128; e += 2) {
        const uint64_t v = f2_pack(s[e], s[e + 1]);
        f2_unpack(f2_mul(v, cap.slope(v)), s[e], s[e + 1]);
      }
    } else {
      CapScore any;
      any.init(a.scale, a.cap);
#pragma unroll
      for (int e = 0; e < 128; ++e) s[e] = any(s[e]);
    }
  }
  if constexpr ((MODE & kBias) != 0) {
    const bool left = __all_sync(0xffffffffu, dist0 >= 127.f), right = __all_sync(0xffffffffu, dist0 <= 0.f);
    if (left || right) {
      // every key of the tile on one side of every row: the bias is linear in the key
      const float g = left ? slope2 : -slope2;
      const uint64_t g2 = f2_pack(g, g), b2 = f2_pack(-g * dist0, -g * dist0), c2 = f2_pack(c, c);
#pragma unroll
      for (int e = 0; e < 128; e += 2) {
        const uint64_t v = f2_pack(s[e], s[e + 1]);
        const uint64_t bias = f2_fma(f2_pack(static_cast<float>(e), static_cast<float>(e + 1)), g2, b2);
        f2_unpack((MODE & kCap) ? f2_add(v, bias) : f2_fma(v, c2, bias), s[e], s[e + 1]);
      }
    } else {
      // slope * |p - j| as the magnitude of slope * (p - j), with the sign of -slope
      const uint32_t sign = slope2 > 0.f ? 0x80000000u : 0u;
      const float b0 = slope2 * dist0;
#pragma unroll
      for (int e = 0; e < 128; ++e) {
        const float t = fmaf(-slope2, static_cast<float>(e), b0);
        const float bias = __uint_as_float((__float_as_uint(t) & 0x7fffffffu) | sign);
        s[e] = (MODE & kCap) ? s[e] + bias : fmaf(s[e], c, bias);
      }
    }
  }
}

// 2^x of two arguments without the special-function unit (Cody and Waite's
// reduction: x = n + f, n the nearest integer, taken from the low bits of x +
// 1.5 * 2^23; a polynomial on [-1/2, 1/2], least squares driven to equal
// ripple, softmax_fit.py: relative error 7.5e-5 of degree 3 for bf16
// probabilities, 2.6e-6 of degree 4 for f16; n added to the exponent).
// Arguments stop at -126, where both polynomials are just under 1.  f16: 2^-126
// is left to the conversion, which makes it zero; a NaN does not come out as a
// NaN but as a value that overflows the type.  bf16 holds 2^-126, which would
// count for a value of 1e35 that its row may not read: there the polynomial is
// multiplied by 2^n, so that results under 2^-126 flush to zero as ex2.approx
// has them, and a NaN stays one.  (f16 with the product: 266 us, 258 without,
// 9472 keys, 8 heads of 64; bf16 262 and 261.)
template <bool BF>
__device__ __forceinline__ void ex2_poly2(uint64_t x, float& pa, float& pb) {
  constexpr float kMagic = 12582912.0f + (BF ? 127.0f : 0.0f);  // bf16: the low bits are the exponent of 2^n
  float xa, xb;
  f2_unpack(x, xa, xb);
  x = f2_pack(max_nan(xa, -126.0f), max_nan(xb, -126.0f));
  const uint64_t t = f2_add(x, f2_pack(kMagic, kMagic));
  const uint64_t f = f2_fma(f2_add(t, f2_pack(-kMagic, -kMagic)), f2_pack(-1.0f, -1.0f), x);
  uint64_t y;
  if constexpr (BF) {
    y = f2_fma(f, f2_pack(0.055171669359523244f, 0.055171669359523244f), f2_pack(0.24261113138277252f, 0.24261113138277252f));
    y = f2_fma(y, f, f2_pack(0.6932609862029608f, 0.6932609862029608f));
    y = f2_fma(y, f, f2_pack(0.9999280729973522f, 0.9999280729973522f));
  } else {
    y = f2_fma(f, f2_pack(0.009570101946824233f, 0.009570101946824233f), f2_pack(0.055917861585536834f, 0.055917861585536834f));
    y = f2_fma(y, f, f2_pack(0.24024744837984294f, 0.24024744837984294f));
    y = f2_fma(y, f, f2_pack(0.6931218145829672f, 0.6931218145829672f));
    y = f2_fma(y, f, f2_pack(0.9999992614392345f, 0.9999992614392345f));
  }
  float ya, yb, ta, tb;
  f2_unpack(t, ta, tb);
  if constexpr (BF) {
    y = f2_mul_ftz(y, f2_pack(__uint_as_float(__float_as_uint(ta) << 23), __uint_as_float(__float_as_uint(tb) << 23)));
    f2_unpack(y, pa, pb);
  } else {
    f2_unpack(y, ya, yb);
    pa = __uint_as_float(__float_as_uint(ya) + (__float_as_uint(ta) << 23));
    pb = __uint_as_float(__float_as_uint(yb) + (__float_as_uint(tb) << 23));
  }
}

// Largest of s[A..B) and of `top`, in four chains; of the magnitudes with ABS.
template <int A, int B, bool ABS = false>
__device__ __forceinline__ float row_max(const float (&s)[128], float top) {
  const auto v = [&](int e) { return ABS ? fabsf(s[e]) : s[e]; };
  float mx[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) mx[t] = fmaxf(v(A + t), v(A + 4 + t));
#pragma unroll
  for (int e = A + 8; e < B; e += 8) {
#pragma unroll
    for (int t = 0; t < 4; ++t) mx[t] = fmax3(mx[t], v(e + t), v(e + 4 + t));
  }
  return fmaxf(fmax3(mx[0], mx[1], mx[2]), fmaxf(mx[3], top));
}

// P of the tile's 128 keys into TMEM (two to a word), and their sum: one
// straight run of code, so that exponentials of either kind overlap.
template <int KIND, int POLY, bool BF>
__device__ __forceinline__ float exp_tile(const float (&s)[128], uint64_t c2, uint64_t nm2, const CapPoly<BF>& cap,
                                          uint32_t tP) {
  uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t v = f2_pack(s[32 * q + 2 * e], s[32 * q + 2 * e + 1]);
      const uint64_t x = KIND == FROM_DOT ? f2_fma(v, c2, nm2)
                                          : (KIND == FROM_CAP ? f2_fma(v, cap.slope(v), nm2) : f2_add(v, nm2));
      float pa, pb;
      if ((e * POLY) % 16 + POLY < 16) {
        f2_unpack(x, pa, pb);
        pa = ex2_approx(pa);
        pb = ex2_approx(pb);
      } else {
        ex2_poly2<BF>(x, pa, pb);
      }
      sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(pa, pb));
      pk[e] = pack2<BF>(pa, pb);
    }
    tmem_st16_nowait(tP + 16 * q, pk);
  }
  float sa, sb;
  f2_unpack(f2_add(sum2[0], sum2[1]), sa, sb);
  return sa + sb;
}

// The lowest n of 32 bits, n outside 0 .. 32 taken as the nearer end.
__device__ __forceinline__ uint32_t key_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// mbar_wait whose thread sleeps; a bound of 0 gives up at once as there.  The
// time that the CTA's warps have spent on rows computed anew (attend_row: up to
// 32 rows a warp at some 4.7 us for 32 keys) is added to the bound.
struct TileWait : WaitCtl {
  volatile unsigned long long* spent;
};
constexpr uint32_t kSleepNs = 20000;
__device__ __forceinline__ bool sleep_wait(uint64_t* bar, uint32_t parity, const TileWait& w) {
  if (mbar_try_wait(bar, parity)) return true;
  if (w.timeout_ns == 0) {
    raise_error(w, DERR_TIMEOUT);
    return false;
  }
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait_for(bar, parity, kSleepNs)) {
    if (*w.abort) return false;
    if (globaltimer() - t0 > w.timeout_ns + *w.spent) {
      raise_error(w, DERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// The same by a whole warp, its lanes together again behind it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const TileWait& w) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, sleep_wait(bar, parity, w));
}

// Pairs of every 16 whose exponential is the polynomial: the special-function
// unit alone would be the bound.
template <int MODE>
constexpr int kPolyPairs = MODE == 0 ? 4 : (MODE == kBias ? 3 : 0);

}  // namespace

template <int NB, bool BF, int MODE>
__global__ void __launch_bounds__(kTileThreads, 1)
    masked_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                        const __grid_constant__ TileParams p) {
  using C = TileCfg<NB>;
  constexpr int kStages = C::kStages, kQBufs = C::kQBufs;
  extern __shared__ uint8_t dsmem[];
  __shared__ uint64_t q_full[kQBufs][2], q_empty[kQBufs][2];
  __shared__ uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  __shared__ uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], drain_bar[2];
  __shared__ uint64_t item_full, item_empty, steal_bar;
  __shared__ alignas(16) uint4 steal_answer;
  // The item that the CTA's warps are at, and the next; n < 0: none.  A slot is
  // written again only when every warp has taken the item behind it.
  __shared__ Item item_sh[2];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ unsigned long long spent_sh;  // ns, in rows computed anew

  const uint32_t raw = smem_u32(dsmem);
  uint8_t* sm = dsmem + ((1024u - (raw & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MaskedAttnParams& a = p.a;

  if (threadIdx.x == 0) {
    for (int g = 0; g < 2; ++g) {
      for (int i = 0; i < kQBufs; ++i) {
        mbar_init(&q_full[i][g], 1);
        mbar_init(&q_empty[i][g], 1);
      }
      mbar_init(&s_full[g], 1);
      mbar_init(&s_free[g], 4);  // one arrival a softmax warp
      mbar_init(&p_full[g], 4);
      mbar_init(&pv_done[g], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(&drain_bar[0], 1);
    mbar_init(&drain_bar[1], 1);
    mbar_init(&item_full, 1);
    mbar_init(&item_empty, 1 + (C::kAliasP ? 1 : 2) + 8);  // TMA, MMA and softmax warps
    mbar_init(&steal_bar, 1);
    abort_sh = 0;
    spent_sh = 0;
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_wait();
  pdl_trigger();

  TileWait w;
  w.abort = reinterpret_cast<volatile int*>(&abort_sh);
  w.spent = reinterpret_cast<volatile unsigned long long*>(&spent_sh);
  w.err = &g_masked_err;
  w.timeout_ns = a.timeout_ns;
  w.where = (KID_ATTN << 8) | static_cast<unsigned>(warp);

  if (warp >= 8) {
    regs_lower<kRegsOther>();
    if (warp == 8) {
      // ---------------------------------------------------------------- TMA
      bool ok = true;
      uint32_t items = 0, kv = 0;  // items taken, key tiles loaded so far
      uint32_t qc[2] = {0, 0};     // Q tiles loaded so far
      uint32_t karmed = 0, varmed = 0;
      while (ok) {
        ok = warp_wait(&item_full, items & 1, w);
        if (!ok) break;
        const Item it = item_sh[items++ & 1];
        if (it.n < 0) break;
        if (lane == 0) {
          const int hk = it.h / (a.hq / a.hk);
          const int qb = (p.q_step & 1) ? it.b : 0, qh = (p.q_step & 4) ? it.h : 0;
          const int kb = (p.k_step & 1) ? it.b : 0, kh = (p.k_step & 4) ? hk : 0;
          const int vb = (p.v_step & 1) ? it.b : 0, vh = (p.v_step & 4) ? hk : 0;
          for (int g = 0; ok && g < 2; ++g) {
            if (it.last[g] == 0) continue;
            const int buf = static_cast<int>(qc[g] % kQBufs);
            if (!sleep_wait(&q_empty[buf][g], ((qc[g] / kQBufs) & 1) ^ 1, w)) {
              ok = false;
              break;
            }
            mbar_expect_tx(&q_full[buf][g], C::kTileBytes);
            for (int c = 0; c < NB; ++c)
              tma_load_4d(sm + C::kOffQ + (buf * 2 + g) * C::kTileBytes + c * kBlockBytes, &tmQ, &q_full[buf][g], 64 * c,
                          qh, it.q0 + 128 * g, qb);
            ++qc[g];
          }
          for (int j = 0; ok && j < it.n; ++j, ++kv) {
            const int s = static_cast<int>(kv % kStages);
            const uint32_t ph = (kv / kStages) & 1;
            const int key = it.lo + 128 * j;
            if (!sleep_wait(&k_empty[s], ph ^ 1, w)) {
              ok = false;
              break;
            }
            mbar_expect_tx(&k_full[s], C::kTileBytes);
            for (int c = 0; c < NB; ++c)
              tma_load_4d(sm + C::kOffK + s * C::kTileBytes + c * kBlockBytes, &tmK, &k_full[s], 64 * c, kh, key, kb);
            karmed = (karmed & ~(3u << (2 * s))) | ((1u | (ph << 1)) << (2 * s));
            if (!sleep_wait(&v_empty[s], ph ^ 1, w)) {
              ok = false;
              break;
            }
            mbar_expect_tx(&v_full[s], C::kTileBytes);
            for (int c = 0; c < NB; ++c)
              tma_load_4d(sm + C::kOffV + s * C::kTileBytes + c * kBlockBytes, &tmV, &v_full[s], 64 * c, vh, key, vb);
            varmed = (varmed & ~(3u << (2 * s))) | ((1u | (ph << 1)) << (2 * s));
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        // the next item is fetched once this one's loads are on their way: no
        // earlier, since an item once taken stays with its CTA
        if (lane == 0) mbar_arrive(&item_empty);
      }
      if (lane == 0) {  // whatever happened to the readers: the copies issued land before the CTA exits
        for (int g = 0; g < 2; ++g)
          for (uint32_t i = 0; i < kQBufs; ++i)
            if (qc[g] > i) {
              const uint32_t last = qc[g] - 1 - i;
              mbar_wait_drain(&q_full[last % kQBufs][g], (last / kQBufs) & 1);
            }
        for (int s = 0; s < kStages; ++s) {
          if ((karmed >> (2 * s)) & 1u) mbar_wait_drain(&k_full[s], (karmed >> (2 * s + 1)) & 1u);
          if ((varmed >> (2 * s)) & 1u) mbar_wait_drain(&v_full[s], (varmed >> (2 * s + 1)) & 1u);
        }
      }
    } else if (warp == 9 || (warp == 10 && !C::kAliasP)) {
      // ---------------------------------------------------------------- MMA
      // Both query tiles in a fixed turn: the tensor core works for one tile
      // while the other is in its softmax.  P beside S: warp 9 issues S and warp
      // 10 P V, each at its own pace.  P in S's place: warp 9 issues P V and the
      // S that follows it, in order.  The whole warp walks
      // the loop and one elected lane issues, on descriptors that differ by
      // constants: operands then stay in uniform registers (a lane's own branch
      // issues a 128 x 64 x 16 product every 60 to 104 clocks, this one every
      // 32, the tensor core's own pace).
      const bool lead = elect_one();
      const uint32_t idesc_s = idesc_f16_f32(128, 128, BF);
      const int ksteps = (a.d + 15) >> 4;  // 16 dims each: zeros behind d
      const uint32_t idesc_o = idesc_f16_f32(128, 16 * ksteps, BF) | kIdescBMnMajor;
      const uint64_t qdesc = sdesc_kmajor_sw128(smem_u32(sm + C::kOffQ));
      const uint64_t kdesc = sdesc_kmajor_sw128(smem_u32(sm + C::kOffK));
      const uint64_t vdesc = sdesc_mnmajor_sw128(smem_u32(sm + C::kOffV), kBlockBytes);
      constexpr uint64_t kTile16 = C::kTileBytes / 16, kBlock16 = kBlockBytes / 16;  // descriptors count 16 bytes
      bool ok = true;
      uint32_t items = 0;
      uint32_t ks = 0, kph = 0, vs = 0, vph = 0;        // stage and phase of the next K and V tile
      uint32_t qc[2] = {0, 0}, sc[2] = {0, 0}, pc[2] = {0, 0};  // Q tiles, S and P V products so far
      while (ok) {
        ok = warp_wait(&item_full, items & 1, w);
        if (!ok) break;
        const Item it = item_sh[items++ & 1];
        if (it.n < 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty);
        if (it.n == 0) continue;
        uint32_t buf[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          buf[g] = qc[g] % kQBufs;
          if (it.last[g] > 0 && warp == 9) {
            ok = ok && warp_wait(&q_full[buf[g]][g], (qc[g] / kQBufs) & 1, w);
            ++qc[g];
          }
        }
        // S of key tile j
        const auto issue_s = [&](int j, int g) {
          if (j < it.first[g] || j >= it.last[g]) return true;
          // P beside S: S may be overwritten once the softmax has taken the tile
          // before; P in S's place: the product that reads it was issued before
          if (!C::kAliasP && sc[g] > 0 && !warp_wait(&s_free[g], (sc[g] - 1) & 1, w)) return false;
          ++sc[g];
          tc_fence_after();
          const uint64_t qd = qdesc + (buf[g] * 2 + g) * kTile16, kd = kdesc + ks * kTile16;
          if (lead) {
#pragma unroll
            for (int t = 0; t < 4 * NB; ++t)
              if (t < ksteps)
                tc_mma_f16_ss(tmem + C::kColS + 128 * g, qd + (t >> 2) * kBlock16 + (t & 3) * 2,
                              kd + (t >> 2) * kBlock16 + (t & 3) * 2, idesc_s, t > 0 ? 1u : 0u);
            tc_commit(&s_full[g]);
            if (j == it.last[g] - 1) tc_commit(&q_empty[buf[g]][g]);
          }
          return true;
        };
        // O += P V of key tile j
        const auto issue_pv = [&](int j, int g) {
          if (j < it.first[g] || j >= it.last[g]) return true;
          if (!warp_wait(&p_full[g], pc[g] & 1, w)) return false;
          ++pc[g];
          tc_fence_after();
          const uint64_t vd = vdesc + vs * kTile16;
          if (lead) {
#pragma unroll
            for (int t = 0; t < 8; ++t)  // 16 keys each
              tc_mma_f16_ts(tmem + C::kColO + C::kStepO * g, tmem + C::kColP + C::kStepP * g + 8 * t, vd + t * 128,
                            idesc_o, (j > it.first[g] || t > 0) ? 1u : 0u);
            tc_commit(&pv_done[g]);
          }
          return true;
        };
        const auto k_release = [&] {
          if (lead) tc_commit(&k_empty[ks]);
          if (++ks == kStages) ks = 0, kph ^= 1;
        };
        const auto v_release = [&] {
          if (lead) tc_commit(&v_empty[vs]);
          if (++vs == kStages) vs = 0, vph ^= 1;
        };
        if constexpr (!C::kAliasP) {
          if (warp == 9) {
            for (int j = 0; ok && j < it.n; ++j) {
              ok = warp_wait(&k_full[ks], kph, w) && issue_s(j, 0) && issue_s(j, 1);
              if (ok) k_release();
            }
          } else {
            for (int j = 0; ok && j < it.n; ++j) {
              ok = warp_wait(&v_full[vs], vph, w) && issue_pv(j, 0) && issue_pv(j, 1);
              if (ok) v_release();
            }
          }
        } else {
          ok = ok && warp_wait(&k_full[ks], kph, w) && issue_s(0, 0) && issue_s(0, 1);
          if (ok) k_release();
          for (int j = 0; ok && j < it.n; ++j) {
            const bool more = j + 1 < it.n;
            if (more) ok = warp_wait(&k_full[ks], kph, w);
            ok = ok && warp_wait(&v_full[vs], vph, w);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              ok = ok && issue_pv(j, g);
              if (more) ok = ok && issue_s(j + 1, g);
            }
            if (!ok) break;
            v_release();
            if (more) k_release();
          }
        }
      }
      if (lead) {
        tc_commit(&drain_bar[warp - 9]);
        mbar_wait_drain(&drain_bar[warp - 9], 0);
      }
      __syncwarp();
    } else if (warp == 11) {
      // -------------------------------------------------------------- items
      // The CTA's own item, then those of CTAs that have not started: items
      // differ in length (documents, causal rows), and this evens them out
      // without a counter in memory.
      int idx = static_cast<int>(blockIdx.x);
      for (uint32_t n = 0;; ++n) {
        Item it;
        it.n = -1;
        if (idx >= 0) it = load_item(p, idx, lane);
        if (lane == 0) item_sh[n & 1] = it;
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_full);
        if (idx < 0) break;
        // not before every warp has taken this one
        if (!warp_wait(&item_empty, n & 1, w)) break;
        if (lane == 0) {
          fence_proxy_async_smem();
          mbar_expect_tx(&steal_bar, 16);
          clc_try_cancel(&steal_answer, &steal_bar);
        }
        __syncwarp();
        if (!warp_wait(&steal_bar, n & 1, w)) {
          mbar_wait_drain(&steal_bar, n & 1);
          __syncwarp();
          break;
        }
        idx = clc_cancelled(&steal_answer);
      }
      __syncwarp();
    }
  } else {
    regs_raise<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    const int g = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + C::kColS + 128 * g + lane_off, tO = tmem + C::kColO + C::kStepO * g + lane_off,
                   tP = tmem + C::kColP + C::kStepP * g + lane_off;
    const float c = a.scale * kLog2e;
    CapPoly<BF> cap;
    if constexpr ((MODE & kCap) != 0) cap.init(a.scale, a.cap);
    bool ok = true;
    uint32_t items = 0, cnt = 0, kv = 0;  // items taken, this tile's key tiles so far, the CTA's
    while (ok) {
      ok = warp_wait(&item_full, items & 1, w);
      if (!ok) break;
      const Item& it = item_sh[items++ & 1];  // what the key loop does not need stays there
      const int n_tiles = it.n, lo_all = it.lo;
      if (n_tiles < 0) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty);
      // A row that is not written reads everything: it must not make tiles look
      // cut (1000 queries took 17 % longer than 1024 when it did).
      int klo = -(1 << 30), khi = 0x7fffffff, kpos;
      bool written;
      {
        const int i = it.q0 + 128 * g + r;
        const RowKeys k = row_keys(a, it.b, min(i, a.Nq - 1));
        kpos = k.pos;
        written = k.written && i < a.Nq;
        if (written) klo = k.lo, khi = k.hi;
      }
      const float slope2 = (MODE & kBias) && a.slopes ? __ldg(a.slopes + it.h) * kLog2e : 0.f;
      const int first = it.first[g], last = it.last[g];
      float m_run = -INFINITY, l_run = 0.f;
      float s[128];  // the key tile's scores of this row
      for (int j = first; j < last; ++j, ++cnt) {
        const int base = lo_all + 128 * j;
        const int rlo = klo - base, rhi = khi - base;
        const bool cut = !__all_sync(0xffffffffu, rlo <= 0 && rhi >= 128);
        if (!warp_wait(&s_full[g], cnt & 1, w)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the second half on its way while the first one's maximum is taken
        tmem_ld32_nowait(tS, s);
        tmem_ld32_nowait(tS + 32, s + 32);
        tmem_wait_ld();
        tmem_landed(s);
        tmem_landed(s + 32);
        tmem_ld32_nowait(tS + 64, s + 64);
        tmem_ld32_nowait(tS + 96, s + 96);
        const bool early = MODE == 0 && !cut;
        float top = -INFINITY;
        if (early) top = row_max<0, 64>(s, top);
        tmem_wait_ld();
        tmem_landed(s + 64);
        tmem_landed(s + 96);
        if (!C::kAliasP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[g]);
        }
        bool raw = MODE == 0;  // exponents straight from the dot products
        [[maybe_unused]] const float dist0 = static_cast<float>(static_cast<long long>(kpos) - base);
        if constexpr ((MODE & kCap) != 0) {
          const bool poly = __all_sync(0xffffffffu, cap.fits(row_max<0, 128, true>(s, 0.f)));
          raw = MODE == kCap && poly && !cut;
          if (!raw) finish_scores<MODE, BF>(s, a, cap, poly, c, slope2, dist0);
        } else if constexpr (MODE == kBias) {
          finish_scores<MODE, BF>(s, a, cap, false, c, slope2, dist0);
        }
        if (cut) {
          // the allowed keys as bits, 32 at a time: one select a key, its bit
          // turned into a predicate for several keys at once
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t keep = key_bits(rhi - 32 * q) & ~key_bits(rlo - 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[32 * q + e] = ((keep >> e) & 1u) ? s[32 * q + e] : -INFINITY;
          }
        }
        top = early ? row_max<64, 128>(s, top) : row_max<0, 128>(s, top);
        if (MODE == 0) top *= c;
        if constexpr (MODE == kCap) {
          if (raw) {
            if (a.scale < 0.f) {  // the smallest product gives the largest score
              top = INFINITY;
#pragma unroll
              for (int e = 0; e < 128; ++e) top = fminf(top, s[e]);
            }
            const uint64_t t2 = f2_pack(top, top);
            float unused;
            f2_unpack(f2_mul(t2, cap.slope(t2)), top, unused);
          }
        }
        const float m_new = fmaxf(m_run, top);
        const bool grow = m_new > m_run + kRescale;
        const bool any_grow = __any_sync(0xffffffffu, grow);
        float alpha = 1.0f;
        if (any_grow) {
          if (grow) {
            alpha = ex2_approx(m_run - m_new);  // exp2(-inf) = 0 on the first tile
            l_run *= alpha;
            m_run = m_new;
          }
          __syncwarp();  // (the TMEM instructions behind want the lanes together)
        }
        // a row that has seen no allowed key yet keeps m = -inf: all its p are 0
        const float m_use = m_run == -INFINITY ? 0.0f : m_run;
        const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-m_use, -m_use);
        if (j > first) {
          // O is stable (and, beside S, P free) once the product of the tile before is done
          if (!warp_wait(&pv_done[g], (cnt - 1) & 1, w)) {
            ok = false;
            break;
          }
          if (any_grow) {
            tc_fence_after();
#pragma unroll 1
            for (int t = 0; t < a.d; t += 16) {
              uint32_t o[16];
              tmem_ld16(tO + t, o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tmem_st16(tO + t, o);
            }
          }
        }
        if constexpr (MODE == kCap) {
          if (raw)
            l_run += exp_tile<FROM_CAP, 0, BF>(s, c2, nm2, cap, tP);
          else
            l_run += exp_tile<FROM_SCORE, 0, BF>(s, c2, nm2, cap, tP);
        } else {
          l_run += exp_tile<MODE == 0 ? FROM_DOT : FROM_SCORE, kPolyPairs<MODE>, BF>(s, c2, nm2, cap, tP);
        }
        tmem_wait_st();
        if (j == n_tiles - 1 && it.hi - base < 128 && it.hi < a.Nk) {
          // values behind the last key that any row reads: zeros, since P's
          // zeros would not hide a NaN or an infinity there
          const uint32_t t = kv + static_cast<uint32_t>(j);
          if (!warp_wait(&v_full[t % kStages], (t / kStages) & 1, w)) {
            ok = false;
            break;
          }
          if (r >= it.hi - base) {
            const uint32_t at = smem_u32(sm + C::kOffV + (t % kStages) * C::kTileBytes) + r * 128;
            for (int x = 0; x < NB * 8; ++x) st_shared_v4(at + (x >> 3) * kBlockBytes + (x & 7) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g]);
      }
      kv += static_cast<uint32_t>(n_tiles);
      if (!ok) break;
      const bool some = last > first;
      if (some && !warp_wait(&pv_done[g], (cnt - 1) & 1, w)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int i = it.q0 + 128 * g + r;
      const bool row = i < a.Nq, full_row = written && khi > klo;
      const float inv = full_row ? 1.0f / l_run : 0.f;
      // The rows go out through shared memory and TMA, 64 dims at a time: a
      // store instruction over 32 rows of their own took 32 passes, 2000 to
      // 4000 clocks an item.  Where a row must be left as it is (no document),
      // each thread stores its own.
      uint16_t* dst = a.out + it.b * a.o_b + static_cast<long long>(i) * a.o_n + it.h * a.o_h;
      uint8_t* stage = sm + C::kOffOut + warp * kOutBytes;
      const bool by_tma = __all_sync(0xffffffffu, !row || written);
      const int row0 = it.q0 + 128 * g + quad * 32;  // the warp's first row
      float odd = 0.f;  // 0 unless a value of the row is not finite
#pragma unroll 1
      for (int blk = 0; 64 * blk < a.d; ++blk) {
        if (lane == 0) bulk_wait_read0();  // the rows staged before have been read
        __syncwarp();
#pragma unroll 1
        for (int t = 64 * blk; t < min(a.d, 64 * blk + 64); t += 32) {
          uint32_t o[32];
          __syncwarp();
          if (some) tmem_ld32(tO + t, o);
          uint32_t h[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = some && full_row ? __uint_as_float(o[2 * e]) * inv : 0.f;
            const float y = some && full_row ? __uint_as_float(o[2 * e + 1]) * inv : 0.f;
            if (t + 2 * e < a.d) odd = fmaf(x, 0.f, fmaf(y, 0.f, odd));  // (columns behind the dims hold anything)
            h[e] = pack2<BF>(x, y);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (by_tma)
              st_shared_v4(smem_u32(stage) + sw128_offset(lane, (t & 32) + 8 * u), h[4 * u], h[4 * u + 1], h[4 * u + 2],
                           h[4 * u + 3]);
            else if (written && t + 8 * u < a.d)
              *reinterpret_cast<uint4*>(dst + t + 8 * u) = make_uint4(h[4 * u], h[4 * u + 1], h[4 * u + 2], h[4 * u + 3]);
          }
        }
        if (by_tma && row0 < a.Nq) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_4d(&tmO, stage, 64 * blk, (p.o_step & 4) ? it.h : 0, row0, (p.o_step & 1) ? it.b : 0);
            bulk_commit();
          }
        }
      }
      // A value that is not finite may have come from a key that the row does
      // not read (0 * inf in the tile's product), and a row whose scores are all
      // -inf may have nothing but the polynomial's 2^-126: such rows anew, by the
      // definition.  One warp a row, and slow: an infinity among the values of
      // 8192 keys that every row reads makes 16 heads of 64 take 153 ms in place
      // of 0.47 (of one head alone 40).
      unsigned again =
          __ballot_sync(0xffffffffu, full_row && (!(odd == 0.f) || m_run == -INFINITY));
      if (again) {  // (not before the rows written above have landed)
        if (lane == 0) bulk_wait0();
        __syncwarp();
      }
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        RowKeys o;
        o.lo = __shfl_sync(0xffffffffu, klo, src);
        o.hi = __shfl_sync(0xffffffffu, khi, src);
        o.pos = __shfl_sync(0xffffffffu, kpos, src);
        o.written = true;
        attend_row<BF>(a, it.b, it.q0 + 128 * g + quad * 32 + src, it.h, o, lane, &spent_sh);
      }
      tc_fence_before();
    }
    __syncwarp();
    tmem_wait_ld();  // nothing in flight when the columns are given back
    if (lane == 0) bulk_wait0();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem_sh, 512);
  }
}

namespace {

// [B, N, heads, d] as a map of (d, heads, N, B) with tiles of `rows` tokens by
// 64 dims, zeros outside; an axis without a stride has length 1.  Returns the
// axes that have one (TileParams::q_step).
bool make_tile_map(CUtensorMap* m, const uint16_t* data, int d, int H, int N, int B, long long sh, long long sn,
                   long long sb, int rows, int* step) {
  const bool hb = B > 1 && sb > 0, hh = H > 1 && sh > 0, hn = N > 1 && sn > 0;
  if (N > 1 && !hn) return false;
  const uint64_t dims[4] = {static_cast<uint64_t>(d), hh ? static_cast<uint64_t>(H) : 1u, static_cast<uint64_t>(N),
                            hb ? static_cast<uint64_t>(B) : 1u};
  const uint64_t one = static_cast<uint64_t>(d) * 2;
  const uint64_t str[3] = {hh ? static_cast<uint64_t>(sh) * 2 : one, hn ? static_cast<uint64_t>(sn) * 2 : one,
                           hb ? static_cast<uint64_t>(sb) * 2 : one};
  const uint32_t box[4] = {64, 1, static_cast<uint32_t>(rows), 1};
  *step = (hb ? 1 : 0) | (hn ? 2 : 0) | (hh ? 4 : 0);
  return make_tmap_f16(m, data, 4, dims, str, box);
}

template <int NB, bool BF, int MODE>
int launch_tiles(const TileParams& p, const CUtensorMap* tm, cudaStream_t st) {
  using C = TileCfg<NB>;
  auto kern = masked_tiles_kernel<NB, BF, MODE>;
  static std::atomic<unsigned long long> attr_done{0};
  if (!smem_attr_once(attr_done, kern, C::kSmem)) return JEPA_B200_ERR_CUDA;
  return launch_pdl(kern, dim3(p.n_items), dim3(kTileThreads), C::kSmem, st, 1, tm[0], tm[1], tm[2], tm[3], p) == cudaSuccess
             ? JEPA_B200_OK
             : JEPA_B200_ERR_CUDA;
}

template <int NB, bool BF>
int launch_tiles_mode(const TileParams& p, const CUtensorMap* tm, cudaStream_t st) {
  // a scale that is not positive turns maxima of dot products into minima:
  // the instance that scales first
  const int mode = (p.a.cap > 0.f ? kCap : 0) | (p.a.slopes || !(p.a.scale > 0.f || p.a.cap > 0.f) ? kBias : 0);
  switch (mode) {
    case 0: return launch_tiles<NB, BF, 0>(p, tm, st);
    case kCap: return launch_tiles<NB, BF, kCap>(p, tm, st);
    case kBias: return launch_tiles<NB, BF, kBias>(p, tm, st);
    default: return launch_tiles<NB, BF, kCap | kBias>(p, tm, st);
  }
}

}  // namespace

// -------------------------------------------------------------- few queries --
// One to a few query rows of each clip against a long cache: bound by the
// bytes of K and V.  The rows that share a key head (Nq query positions by
// heads_q / heads_kv heads) are the 8-wide N of m16n8k16 products, with the
// keys (S^T = K Q^T) and then the dims (O^T = V^T P^T) as M: K and V go from
// global memory straight into the A fragments, 16 bytes a load.  For K that
// works because a dot product may take its dims in any order: a lane's 8
// consecutive dims serve as the pairs of two products, Q's alike.  For V a
// lane loads the same 8 dims of two neighbouring keys and interleaves them
// (one byte permutation a fragment word).  P^T comes from S^T's accumulators
// by a transposing move of 8 x 8 blocks.
// A cluster of CTAs shares a clip's key head and splits its keys; each warp
// keeps its own running maximum and sums over tiles of 32 keys, K of the next
// tile in flight while this one's softmax runs; the parts are joined through
// shared memory, then through the cluster's, so that no workspace is needed
// and the order of the sums is fixed.
namespace {

constexpr int kStepKeys = 32;  // keys of a warp's tile (64 for heads of 64: 41 us in place of 34 at 32 x 12 heads, 2048 keys)

// CTAs an SM holds, by the registers of K and V in flight.
template <int NB, int NR, int WARPS>
constexpr int kStepResident = WARPS == 8 ? 1 : (NB == 1 && NR == 1 ? 3 : 2);

struct StepParams {
  MaskedAttnParams a;
  int chunks;  // groups of 8 NR rows of a key head
  int splits;  // CTAs of a cluster
};

template <bool BF>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 matrix of 16-bit values, a row a lane quad: transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// What a part with maximum m and sum l counts for against the maximum `top`
// of all parts: 0 where it has no key (or only scores of -inf), NaN where its
// only scores are NaN.
__device__ __forceinline__ float part_factor(float m, float l, float top) {
  if (m == -INFINITY) return l == 0.f ? 0.f : NAN;
  return ex2_approx(m - top);
}

__device__ __forceinline__ uint4 load_16(const uint16_t* p, bool on) {
  return on ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace

template <int NB, bool BF, int NR, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, kStepResident<NB, NR, WARPS>) masked_step_kernel(const __grid_constant__ StepParams p) {
  constexpr int kRows = 8 * NR, kDims = 64 * NB, kKeys = kStepKeys, kH = kKeys / 16;
  __shared__ float part_o[WARPS][kRows][kDims];
  __shared__ float part_m[WARPS][kRows], part_l[WARPS][kRows];
  __shared__ float cta_m[kRows], cta_l[kRows];
  __shared__ unsigned again;    // rank 0: rows whose result is not finite
  __shared__ int row_some[kRows];  // the row has keys (1), has none (0), is not written (-1)
  const MaskedAttnParams& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, c4 = lane & 3;
  const int rank = blockIdx.x % p.splits;
  int unit = blockIdx.x / p.splits;
  const int chunk = unit % p.chunks;
  unit /= p.chunks;
  const int hk = unit % a.hk, b = unit / a.hk;
  const int group = a.hq / a.hk, row0 = chunk * kRows;
  if (threadIdx.x == 0) again = 0u;
  pdl_wait();
  pdl_trigger();

  // row lane of the chunk: query position i, its keys; all warps alike
  RowKeys rk;
  rk.lo = rk.hi = rk.pos = 0;
  rk.written = false;
  const bool row_on = lane < kRows && row0 + lane < a.Nq * group;
  if (row_on) rk = row_keys(a, b, (row0 + lane) / group);
  const bool any = rk.hi > rk.lo;
  if (warp == 0 && lane < kRows) row_some[lane] = rk.written ? (any ? 1 : 0) : -1;
  const int lo = __reduce_min_sync(0xffffffffu, any ? rk.lo : 0x7fffffff);
  const int hi = __reduce_max_sync(0xffffffffu, any ? rk.hi : 0);
  const int total = hi > lo ? hi - lo : 0;
  const int per = ((total + p.splits - 1) / p.splits + kKeys - 1) / kKeys * kKeys;
  const int k0 = lo + rank * per, k1 = min(hi, k0 + per);
  const int tiles = total > 0 && k1 > k0 ? (k1 - k0 + kKeys - 1) / kKeys : 0;

  // this lane's rows of S^T and O^T: 2 c4 and 2 c4 + 1 of each group of 8
  int rlo[NR][2], rhi[NR][2], rpos[NR][2];
  float slope2[NR][2];
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int src = 8 * x + 2 * c4 + y;
      // a row that is not there reads everything: it must not make tiles look cut
      rlo[x][y] = __shfl_sync(0xffffffffu, row_on ? rk.lo : 0, src);
      rhi[x][y] = __shfl_sync(0xffffffffu, row_on ? rk.hi : 0x7fffffff, src);
      rpos[x][y] = __shfl_sync(0xffffffffu, rk.pos, src);
      slope2[x][y] = a.slopes ? __ldg(a.slopes + hk * group + (row0 + src) % group) * kLog2e : 0.f;
    }
  // Q: row quad of each group, dims 8 (4 s + c4) .. + 7
  uint4 qf[NR][2 * NB];
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    const int r = row0 + 8 * x + quad;
    const bool on = r < a.Nq * group;
    const uint16_t* q = a.q + b * a.q_b + (on ? r / group : 0) * a.q_n + (hk * group + (on ? r % group : 0)) * a.q_h;
#pragma unroll
    for (int s = 0; s < 2 * NB; ++s) qf[x][s] = load_16(q + 8 * (4 * s + c4), on && 8 * (4 * s + c4) < a.d);
  }

  // Loads need no bounds but the clamps here: a key behind the last one is
  // read as the last (its score is masked), dims behind d as the first ones
  // (Q has zeros there, and O's are not stored).
  int koff[2 * NB], voff[NB];
#pragma unroll
  for (int s = 0; s < 2 * NB; ++s) koff[s] = 8 * (4 * s + c4) < a.d ? 8 * (4 * s + c4) : 0;
#pragma unroll
  for (int n = 0; n < NB; ++n) voff[n] = 8 * (8 * n + quad) < a.d ? 8 * (8 * n + quad) : 0;
  const uint16_t* kbase = a.k + b * a.k_b + hk * a.k_h;
  const uint16_t* vbase = a.v + b * a.v_b + hk * a.v_h;
  uint4 kf[kH][2][2 * NB];  // [16 keys][key quad, quad + 8][32 dims]
  uint4 vf[kH][4][NB];      // [16 keys][key 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9][64 dims]
  const auto load_k = [&](int key0) {
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint16_t* src = kbase + min(key0 + 16 * h + 8 * y + quad, k1 - 1) * a.k_n;
#pragma unroll
        for (int s = 0; s < 2 * NB; ++s) kf[h][y][s] = __ldg(reinterpret_cast<const uint4*>(src + koff[s]));
      }
  };
  const auto load_v = [&](int key0) {
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint16_t* src = vbase + min(key0 + 16 * h + 2 * c4 + (y & 1) + 8 * (y >> 1), k1 - 1) * a.v_n;
#pragma unroll
        for (int n = 0; n < NB; ++n) vf[h][y][n] = __ldg(reinterpret_cast<const uint4*>(src + voff[n]));
      }
  };

  float m[NR][2], l[NR][2], o[NR][NB][4][4];
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    m[x][0] = m[x][1] = -INFINITY;
    l[x][0] = l[x][1] = 0.f;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int t = 0; t < 4; ++t) o[x][n][t][0] = o[x][n][t][1] = o[x][n][t][2] = o[x][n][t][3] = 0.f;
  }
  const float c = a.scale * kLog2e;
  CapPoly<BF> cap;
  if (a.cap > 0.f) cap.init(a.scale, a.cap);
  if (warp < tiles) {
    load_k(k0 + warp * kKeys);
    load_v(k0 + warp * kKeys);
  }
  for (int t = warp; t < tiles; t += WARPS) {
    const int key0 = k0 + t * kKeys;
    const bool more = t + WARPS < tiles;
    float s[NR][kH][4];
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        s[x][h][0] = s[x][h][1] = s[x][h][2] = s[x][h][3] = 0.f;
#pragma unroll
        for (int d = 0; d < 2 * NB; ++d) {
          const uint4 u = kf[h][0][d], w = kf[h][1][d], q = qf[x][d];
          const uint32_t a0[4] = {u.x, w.x, u.y, w.y}, a1[4] = {u.z, w.z, u.w, w.w};
          mma_16816<BF>(s[x][h], a0, q.x, q.y);
          mma_16816<BF>(s[x][h], a1, q.z, q.w);
        }
      }
    if (more) load_k(key0 + WARPS * kKeys);
    if (a.cap > 0.f) {
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * kH * NR; ++i) big = fmaxf(big, fabsf(s[i / (4 * kH)][(i >> 2) % kH][i & 3]));
      if (__all_sync(0xffffffffu, cap.fits(big))) {
#pragma unroll
        for (int i = 0; i < 4 * kH * NR; i += 2) {
          float(&v)[4] = s[i / (4 * kH)][(i >> 2) % kH];
          const uint64_t d = f2_pack(v[i & 3], v[(i & 3) + 1]);
          f2_unpack(f2_mul(d, cap.slope(d)), v[i & 3], v[(i & 3) + 1]);
        }
      } else {
        CapScore any;
        any.init(a.scale, a.cap);
#pragma unroll
        for (int i = 0; i < 4 * kH * NR; ++i) {
          float& v = s[i / (4 * kH)][(i >> 2) % kH][i & 3];
          v = any(v);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * kH * NR; ++i) s[i / (4 * kH)][(i >> 2) % kH][i & 3] *= c;
    }
    if (a.slopes) {
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float far = static_cast<float>(static_cast<long long>(rpos[x][y]) - key0 - quad);
#pragma unroll
          for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[x][h][2 * e + y] -= slope2[x][y] * fabsf(far - static_cast<float>(16 * h + 8 * e));
        }
    }
    bool whole = true;  // no row's interval cuts the tile
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) whole = whole && rlo[x][y] <= key0 && rhi[x][y] >= key0 + kKeys;
    if (!__all_sync(0xffffffffu, whole)) {
#pragma unroll
      for (int i = 0; i < 4 * kH * NR; ++i) {
        const int x = i / (4 * kH), h = (i >> 2) % kH, e = i & 3, key = key0 + 16 * h + 8 * (e >> 1) + quad;
        if (key < rlo[x][e & 1] || key >= rhi[x][e & 1]) s[x][h][e] = -INFINITY;
      }
    }
    bool grow = false;
    float top[NR][2];
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y)
        {
          top[x][y] = fmaxf(s[x][0][y], s[x][0][y + 2]);
#pragma unroll
          for (int h = 1; h < kH; ++h) top[x][y] = fmax3(top[x][y], s[x][h][y], s[x][h][y + 2]);
          grow |= top[x][y] > m[x][y] + kRescale;
        }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float mx = top[x][y];
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
          if (mx > m[x][y] + kRescale) {
            const float alpha = ex2_approx(m[x][y] - mx);  // 0 while there was none
            m[x][y] = mx;
            l[x][y] *= alpha;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                o[x][n][u][y] *= alpha;
                o[x][n][u][y + 2] *= alpha;
              }
          }
        }
      __syncwarp();  // (the matrix instructions behind want the lanes together)
    }
    uint32_t pf[NR][kH][2];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const float m0 = m[x][0] == -INFINITY ? 0.f : m[x][0], m1 = m[x][1] == -INFINITY ? 0.f : m[x][1];
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const float p0 = ex2_approx(s[x][h][0] - m0), p1 = ex2_approx(s[x][h][1] - m1);
        const float p2 = ex2_approx(s[x][h][2] - m0), p3 = ex2_approx(s[x][h][3] - m1);
        l[x][0] += p0 + p2;
        l[x][1] += p1 + p3;
        pf[x][h][0] = transpose_8x8(pack2<BF>(p0, p1));
        pf[x][h][1] = transpose_8x8(pack2<BF>(p2, p3));
      }
    }
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint4 e0 = vf[h][0][n], e1 = vf[h][1][n], e2 = vf[h][2][n], e3 = vf[h][3][n];
        const uint32_t w0[4] = {e0.x, e0.y, e0.z, e0.w}, w1[4] = {e1.x, e1.y, e1.z, e1.w};
        const uint32_t w2[4] = {e2.x, e2.y, e2.z, e2.w}, w3[4] = {e3.x, e3.y, e3.z, e3.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t af[4] = {__byte_perm(w0[u], w1[u], 0x5410), __byte_perm(w0[u], w1[u], 0x7632),
                                  __byte_perm(w2[u], w3[u], 0x5410), __byte_perm(w2[u], w3[u], 0x7632)};
#pragma unroll
          for (int x = 0; x < NR; ++x) mma_16816<BF>(o[x][n][u], af, pf[x][h][0], pf[x][h][1]);
        }
      }
    if (more) load_v(key0 + WARPS * kKeys);
  }

  // the warp's part: lane holds dims 64 n + 8 quad + 2 u, + 1 of its rows
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float sum = l[x][y];
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
      const int r = 8 * x + 2 * c4 + y;
      if (quad == 0) {
        part_m[warp][r] = m[x][y];
        part_l[warp][r] = sum;
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<float2*>(&part_o[warp][r][64 * n + 8 * quad + 2 * u]) = make_float2(o[x][n][u][y], o[x][n][u][y + 2]);
    }
  __syncthreads();
  // the CTA's part, in place of warp 0's
  if (threadIdx.x < kRows) {
    const int r = threadIdx.x;
    float mm = part_m[0][r];
#pragma unroll
    for (int v = 1; v < WARPS; ++v) mm = fmaxf(mm, part_m[v][r]);
    float ll = 0.f;
#pragma unroll
    for (int v = 0; v < WARPS; ++v) {
      const float f = part_factor(part_m[v][r], part_l[v][r], mm);
      ll += part_l[v][r] * f;
      part_m[v][r] = f;  // from here on the part's factor
    }
    cta_m[r] = mm;
    cta_l[r] = ll;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kDims; i += WARPS * 32) {
    const int r = i / kDims, d = i % kDims;
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < WARPS; ++x)
      if (!(part_m[x][r] == 0.f)) v = fmaf(part_o[x][r][d], part_m[x][r], v);
    part_o[0][r][d] = v;
  }
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  // Each CTA of the cluster joins and writes its share of the values.
  const int share = (kRows * kDims / 8 + p.splits - 1) / p.splits;  // pieces of 8 dims
  const uint32_t at_o = smem_u32(&part_o[0][0][0]), at_m = smem_u32(cta_m), at_l = smem_u32(cta_l);
  const uint32_t at_again = p.splits > 1 ? mapa_shared(smem_u32(&again), 0) : smem_u32(&again);
  for (int i = rank * share + threadIdx.x; i < min((rank + 1) * share, kRows * kDims / 8); i += WARPS * 32) {
    const int r = i / (kDims / 8), d = i % (kDims / 8) * 8;
    const int row = row0 + r;
    if (row_some[r] < 0 || d >= a.d) continue;  // (a row behind the last one neither)
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, ll = 0.f, mm = -INFINITY;
    for (int x = 0; x < p.splits; ++x)
      mm = fmaxf(mm, p.splits > 1 ? ld_cluster_f32(mapa_shared(at_m + 4 * r, x)) : cta_m[r]);
    for (int x = 0; x < p.splits; ++x) {
      const float mx = p.splits > 1 ? ld_cluster_f32(mapa_shared(at_m + 4 * r, x)) : cta_m[r];
      const float lx = p.splits > 1 ? ld_cluster_f32(mapa_shared(at_l + 4 * r, x)) : cta_l[r];
      const float f = part_factor(mx, lx, mm);
      if (f == 0.f) continue;
      ll = fmaf(lx, f, ll);
      const uint32_t from = p.splits > 1 ? mapa_shared(at_o + 4 * (r * kDims + d), x) : 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = fmaf(p.splits > 1 ? ld_cluster_f32(from + 4 * e) : part_o[0][r][d + e], f, v[e]);
    }
    const bool some = row_some[r] > 0;
    const float inv = some ? 1.0f / ll : 0.f;
    float odd = 0.f;
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = some ? v[2 * e] * inv : 0.f, y = some ? v[2 * e + 1] * inv : 0.f;
      odd = fmaf(x, 0.f, fmaf(y, 0.f, odd));
      h[e] = pack2<BF>(x, y);
    }
    *reinterpret_cast<uint4*>(a.out + b * a.o_b + (row / group) * a.o_n + (hk * group + row % group) * a.o_h + d) =
        make_uint4(h[0], h[1], h[2], h[3]);
    // as in the tiles: a value that is not finite may have come from a key
    // that its row does not read
    if (some && !(odd == 0.f))
      asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(at_again), "r"(1u << r) : "memory");
  }
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  if (rank == 0 && again != 0u) {
    for (int r = warp; r < kRows; r += WARPS) {
      if (!((again >> r) & 1u)) continue;
      const int row = row0 + r;
      const RowKeys k = row_keys(a, b, row / group);
      attend_row<BF>(a, b, row / group, hk * group + row % group, k, lane);
    }
  }
}

namespace {

// CTAs of one instance that the current device holds at once in clusters of
// 2^log2s (a cluster lies within one of its groups of SMs, so that large ones
// leave SMs over); asked once per device and size.  0: the size cannot run.
template <int NB, bool BF, int NR, int WARPS>
int step_slots(int log2s) {
  static std::atomic<int> known[64][5] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][log2s].load(std::memory_order_acquire);
  if (n == 0) {
    auto kern = masked_step_kernel<NB, BF, NR, WARPS>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1u << log2s);
    cfg.blockDim = dim3(WARPS * 32);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << log2s;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // beyond 8 CTAs: not portable, but this device's
    if (log2s > 3 && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) n = -1;
    if (n == 0 && (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1)) n = -1;
    if (n < 0) cudaGetLastError();  // not an error of the call
    n = n < 0 ? -1 : n << log2s;
    known[dev][log2s].store(n, std::memory_order_release);
  }
  return n < 0 ? 0 : n;
}

template <int NB, bool BF, int NR, int WARPS>
int launch_step_as(const StepParams& p, long long units, cudaStream_t st) {
  return launch_pdl(masked_step_kernel<NB, BF, NR, WARPS>, dim3(static_cast<unsigned>(units * p.splits)),
                    dim3(WARPS * 32), 0, st, p.splits, p) == cudaSuccess
             ? JEPA_B200_OK
             : JEPA_B200_ERR_CUDA;
}

template <int NB, bool BF, int NR>
int launch_step(const MaskedAttnParams& a, cudaStream_t st) {
  StepParams p;
  p.a = a;
  const int rows = a.Nq * (a.hq / a.hk);
  p.chunks = (rows + 8 * NR - 1) / (8 * NR);
  const long long units = static_cast<long long>(a.B) * a.hk * p.chunks;
  if (units > 0x7fffffffll / 16) return JEPA_B200_ERR_SHAPE;
  // The cluster size s and the warps w of a CTA that end first, by rounds of
  // CTAs over the device times what one takes: its keys a warp, and a fixed
  // part worth 40 + 8 s keys (about 14 keys a microsecond and warp; joining a
  // cluster of 16 costs some 10 us).  16 x 8 key heads of 128 over 8192 keys:
  // s w = 1 x 8 76 us, 2 x 4 76 us, 4 x 4 84 us, 8 x 4 106 us, 16 x 4 203 us.
  double best = 1e30;
  int warps = 4;
  p.splits = 1;
  for (int i = 0; i <= 4 && (i == 0 || a.Nk >= (2 * kStepKeys << i)); ++i)
    for (int w = 4; w <= (NR == 1 ? 8 : 4); w *= 2) {
      const int slots = w == 8 ? step_slots<NB, BF, 1, 8>(i) : step_slots<NB, BF, NR, 4>(i);
      if (slots == 0) continue;
      const int s = 1 << i;
      const long long rounds = (units * s + slots - 1) / slots;
      const double cost = static_cast<double>(rounds) * (static_cast<double>(a.Nk) / (s * w) + 40 + 8 * s);
      if (cost < best) {
        best = cost;
        p.splits = s;
        warps = w;
      }
    }
  if constexpr (NR == 1) {
    if (warps == 8) return launch_step_as<NB, BF, 1, 8>(p, units, st);
  }
  return launch_step_as<NB, BF, NR, 4>(p, units, st);
}

template <int NB, bool BF>
int launch_step_rows(const MaskedAttnParams& a, cudaStream_t st) {
  return a.Nq * (a.hq / a.hk) <= 8 ? launch_step<NB, BF, 1>(a, st) : launch_step<NB, BF, 2>(a, st);
}

}  // namespace

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

// Which kernel: the few-query one up to 32 query positions, and up to 64 where
// the tiles would leave three quarters of the SMs without an item.  Few-query
// kernel against tiles, us, at 16, 32 and 64 positions: 2 clips, 4096 keys, 32
// heads on 8 of 128: 37, 55, 99 against 59; 16 clips, 512 keys, 16 heads of 64:
// 10, 19, 36 against 21; 64 clips, 300 keys, 12 heads of 64: 24, 45, 85 against
// 46 to 49; one clip, 16384 keys, 16 heads of 64: 29, 31, 49 against 151.
static bool few_queries(const MaskedAttnParams& p) {
  return p.Nq <= 32 || (p.Nq <= 64 && 4ll * p.B * p.hq <= num_sms());
}

int launch_masked_attention(const MaskedAttnParams& p, bool bf16, cudaStream_t st) {
  if (few_queries(p)) {
    if (p.d <= 64) return bf16 ? launch_step_rows<1, true>(p, st) : launch_step_rows<1, false>(p, st);
    return bf16 ? launch_step_rows<2, true>(p, st) : launch_step_rows<2, false>(p, st);
  } else {
    TileParams tp;
    tp.a = p;
    tp.n_pairs = (p.Nq + 255) / 256;
    const long long items = static_cast<long long>(p.B) * p.hq * tp.n_pairs;
    if (items > 0x7fffffffll) return JEPA_B200_ERR_SHAPE;
    tp.n_items = static_cast<int>(items);
    CUtensorMap tm[4];
    if (p.Nk > 0 && make_tile_map(&tm[0], p.q, p.d, p.hq, p.Nq, p.B, p.q_h, p.q_n, p.q_b, 128, &tp.q_step) &&
        make_tile_map(&tm[1], p.k, p.d, p.hk, p.Nk, p.B, p.k_h, p.k_n, p.k_b, 128, &tp.k_step) &&
        make_tile_map(&tm[2], p.v, p.d, p.hk, p.Nk, p.B, p.v_h, p.v_n, p.v_b, 128, &tp.v_step) &&
        make_tile_map(&tm[3], p.out, p.d, p.hq, p.Nq, p.B, p.o_h, p.o_n, p.o_b, 32, &tp.o_step)) {
      if (p.d <= 64) return bf16 ? launch_tiles_mode<1, true>(tp, tm, st) : launch_tiles_mode<1, false>(tp, tm, st);
      return bf16 ? launch_tiles_mode<2, true>(tp, tm, st) : launch_tiles_mode<2, false>(tp, tm, st);
    }
  }
  const long long rows = static_cast<long long>(p.B) * p.Nq * p.hq;
  const long long blocks = (rows + 3) / 4;
  if (blocks > 0x7fffffffll) return JEPA_B200_ERR_SHAPE;
  const auto kern = bf16 ? masked_rows_kernel<true> : masked_rows_kernel<false>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, st, 1, p) == cudaSuccess
             ? JEPA_B200_OK
             : JEPA_B200_ERR_CUDA;
}

}  // namespace jb
