// Single-kernel entry points of the C ABI: each validates its arguments on
// the host and enqueues exactly the kernel the forward pass uses.
#include <string.h>

#include <cmath>
#include <mutex>

#include "head_ops.h"
#include "internal.h"
#include "patchify.h"

using namespace jb;

namespace {

unsigned long long g_timeout_ns = kDefaultTimeoutNs;
std::mutex g_err_mu;
DevErr* g_err[64] = {nullptr};

// The per-device error word of the op entry points (allocated on first use).
DevErr* op_err() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lk(g_err_mu);
  if (!g_err[dev]) {
    void* p = nullptr;
    if (cudaMalloc(&p, sizeof(DevErr)) != cudaSuccess) return nullptr;
    if (cudaMemset(p, 0, sizeof(DevErr)) != cudaSuccess) {
      cudaFree(p);
      return nullptr;
    }
    g_err[dev] = static_cast<DevErr*>(p);
  }
  return g_err[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int bmode_of(int dtype) {
  switch (dtype) {
    case JEPA_B200_F16: return B_F16;
    case JEPA_B200_Q8_0: return B_Q8;
    case JEPA_B200_Q4_0: return B_Q4;
    default: return -1;
  }
}

int make_matrix(DevMatrix* W, const void* w, const void* scales, int dtype, int N, int K) {
  const int bm = bmode_of(dtype);
  if (bm < 0) return JEPA_B200_ERR_DTYPE;
  if (!w || (bm != B_F16 && !scales)) return JEPA_B200_ERR_ARG;
  if (!aligned16(w)) return JEPA_B200_ERR_ARG;
  W->bmode = bm;
  W->N = N;
  W->K = K;
  W->data = const_cast<void*>(w);
  W->scales = static_cast<__half*>(const_cast<void*>(scales));
  // the caller's [N, K/32] scales serve the CTA-pair kernel's staged loader
  // when their rows are whole 16-byte groups (K a multiple of 256) and 16-byte aligned
  if (bm != B_F16 && (K / 32) % 8 == 0 && aligned16(scales)) {
    W->scales_pad = W->scales;
    W->sc_ld = K / 32;
  }
  return JEPA_B200_OK;
}

// ---- per-head calls --------------------------------------------------------
int dtype_bytes(int dtype) {
  switch (dtype) {
    case JEPA_B200_F32: return 4;
    case JEPA_B200_F16:
    case JEPA_B200_BF16: return 2;
    default: return 0;
  }
}

// The strides a [B, N, heads, d] operand can be read by; an axis of length 1
// has no stride.
bool heads_ok(const jepa_b200_heads& t, int elem_bytes) {
  return t.data && (reinterpret_cast<uintptr_t>(t.data) & (elem_bytes - 1)) == 0 && t.stride_b >= 0 &&
         t.stride_n >= 0 && t.stride_h >= 0 && t.stride_b < (1ll << 40) && t.stride_n < (1ll << 40) &&
         t.stride_h < (1ll << 40);
}
// Outputs besides: no two elements in one place along a single axis.
bool heads_out_ok(const jepa_b200_heads& t, int elem_bytes, int B, int N, int H, int d) {
  return heads_ok(t, elem_bytes) && (B == 1 || t.stride_b >= d) && (N == 1 || t.stride_n >= d) &&
         (H == 1 || t.stride_h >= d);
}

int fill_rope(RopeParams* r, const jepa_b200_rope& a, int d, int B) {
  memset(r, 0, sizeof(*r));
  if (a.rot_dim == 0) return JEPA_B200_OK;
  if (a.layout != JEPA_B200_ROPE_HALF && a.layout != JEPA_B200_ROPE_INTERLEAVED) return JEPA_B200_ERR_ARG;
  if (a.rot_dim < 0 || a.rot_dim % 2 != 0 || a.rot_dim > d || a.n_axes < 1 || a.n_axes > 3) return JEPA_B200_ERR_SHAPE;
  if (!a.pos || !a.turns || (a.n_axes > 1 && !a.axis)) return JEPA_B200_ERR_ARG;
  if ((a.pos_i64 != 0 && a.pos_i64 != 1) || (reinterpret_cast<uintptr_t>(a.pos) & (a.pos_i64 ? 7u : 3u)) != 0)
    return JEPA_B200_ERR_ARG;
  if (a.pos_stride_axis < 0 || a.pos_stride_b < 0) return JEPA_B200_ERR_ARG;
  r->rot_dim = a.rot_dim;
  r->half_layout = a.layout == JEPA_B200_ROPE_HALF ? 1 : 0;
  r->n_axes = a.n_axes;
  r->pos_i64 = a.pos_i64;
  r->pos = a.pos;
  r->pos_stride_axis = a.n_axes > 1 ? a.pos_stride_axis : 0;
  r->pos_stride_b = B > 1 ? a.pos_stride_b : 0;
  r->factor = a.factor;
  for (int i = 0; i < a.rot_dim / 2; ++i) {
    r->turns[i] = a.turns[i];
    r->axis[i] = a.n_axes > 1 ? a.axis[i] : 0;
    if (r->axis[i] >= a.n_axes) return JEPA_B200_ERR_ARG;
  }
  return JEPA_B200_OK;
}

int fill_tensor(HeadTensor* t, const jepa_b200_heads& in, const jepa_b200_heads& out, int elem_bytes, int B, int N,
                int H, int d) {
  if (!heads_ok(in, elem_bytes) || !heads_out_ok(out, elem_bytes, B, N, H, d)) return JEPA_B200_ERR_ARG;
  t->in = in.data;
  t->out = out.data;
  t->in_b = in.stride_b;
  t->in_n = in.stride_n;
  t->in_h = in.stride_h;
  t->out_b = out.stride_b;
  t->out_n = out.stride_n;
  t->out_h = out.stride_h;
  t->heads = H;
  return JEPA_B200_OK;
}

bool float_ptr_ok(const float* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

void jepa_b200_op_set_timeout_ns(unsigned long long ns) { g_timeout_ns = ns; }

int jepa_b200_op_sync_status(void* stream) {
  DevErr* e = op_err();
  if (!e) return JEPA_B200_ERR_CUDA;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return JEPA_B200_ERR_CUDA;
  // both words are read and cleared before either decides: the calls before
  // this one leave nothing for the next
  DevErr h{0, 0};
  if (cudaMemcpy(&h, e, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return JEPA_B200_ERR_CUDA;
  if (h.code != DERR_NONE) cudaMemset(e, 0, sizeof(DevErr));
  unsigned masked = 0;
  if (masked_attention_take_error(&masked) != JEPA_B200_OK) return JEPA_B200_ERR_CUDA;
  for (const unsigned code : {h.code, masked})
    if (code != DERR_NONE && code != DERR_TIMEOUT) return JEPA_B200_ERR_CUDA;
  return h.code == DERR_NONE && masked == DERR_NONE ? JEPA_B200_OK : JEPA_B200_ERR_TIMEOUT;
}

int jepa_b200_op_layernorm(const float* x, int rows, int D, int in_row_stride, const float* gamma,
                           const float* beta, float eps, void* out, int out_dtype, void* stream) {
  if (out_dtype != JEPA_B200_F16 && out_dtype != JEPA_B200_F32) return JEPA_B200_ERR_DTYPE;
  if (!aligned16(x) || !aligned16(out) || !aligned16(gamma) || !aligned16(beta)) return JEPA_B200_ERR_ARG;
  if (!(eps > 0.0f)) return JEPA_B200_ERR_ARG;
  return launch_layernorm(x, rows, D, in_row_stride, gamma, beta, eps, out, out_dtype == JEPA_B200_F16,
                          static_cast<cudaStream_t>(stream));
}

int jepa_b200_op_repack(int dtype, const void* blocks, int N, int K, void* qs, void* scales, void* stream) {
  const int bm = bmode_of(dtype);
  if (bm != B_Q8 && bm != B_Q4) return JEPA_B200_ERR_DTYPE;
  return launch_repack(bm, static_cast<const uint8_t*>(blocks), N, K, qs, static_cast<__half*>(scales),
                       static_cast<cudaStream_t>(stream));
}

int jepa_b200_op_dequant_f16(int dtype, const void* qs, const void* scales, int N, int K, void* out, void* stream) {
  const int bm = bmode_of(dtype);
  if (bm != B_Q8 && bm != B_Q4) return JEPA_B200_ERR_DTYPE;
  if (!qs || !scales || !out || !aligned16(out)) return JEPA_B200_ERR_ARG;
  return launch_dequant_f16(bm, qs, static_cast<const __half*>(scales), N, K, static_cast<__half*>(out),
                            static_cast<cudaStream_t>(stream));
}

int jepa_b200_op_linear(const void* A, int M, int K, const void* w, const void* w_scales, int w_dtype, int N,
                        const float* bias, int epilogue, void* out, int ldo, void* stream) {
  if (!A || !out) return JEPA_B200_ERR_ARG;
  if (epilogue < JEPA_B200_EPI_F16 || epilogue > JEPA_B200_EPI_F32) return JEPA_B200_ERR_ARG;
  if (!aligned16(A) || !aligned16(out) || (bias && !aligned16(bias)) || ldo % 8 != 0) return JEPA_B200_ERR_ARG;
  DevMatrix W;
  int s = make_matrix(&W, w, w_scales, w_dtype, N, K);
  if (s) return s;
  DevErr* e = op_err();
  if (!e) return JEPA_B200_ERR_CUDA;
  GemmOp op;
  if ((s = gemm_prepare(&op, static_cast<const __half*>(A), M, K, W, bias, epilogue, out, ldo, nullptr, nullptr)))
    return s;
  return gemm_launch(op, static_cast<cudaStream_t>(stream), e, g_timeout_ns);
}

int jepa_b200_op_linear_qkv(const void* A, int M, int K, const void* w, const void* w_scales, int w_dtype, int N,
                            const float* bias, int ntok, int heads, int npad, int first_part, void* q, void* k,
                            void* vt, void* stream) {
  if (!A || heads < 1 || ntok < 1 || first_part < 0 || first_part > 2) return JEPA_B200_ERR_ARG;
  const int D = 64 * heads;
  if (N % D != 0 || N / D + first_part > 3 || M % ntok != 0 || npad < ntok || npad % 128 != 0)
    return JEPA_B200_ERR_SHAPE;
  if (!aligned16(A) || (bias && !aligned16(bias)) || (q && !aligned16(q)) || (k && !aligned16(k)))
    return JEPA_B200_ERR_ARG;
  DevMatrix W;
  int s = make_matrix(&W, w, w_scales, w_dtype, N, K);
  if (s) return s;
  DevErr* e = op_err();
  if (!e) return JEPA_B200_ERR_CUDA;
  QkvDst qd;
  qd.q = static_cast<__half*>(q);
  qd.k = static_cast<__half*>(k);
  qd.vt = static_cast<__half*>(vt);
  qd.ntok = ntok;
  qd.heads = heads;
  qd.npad = npad;
  qd.first_part = first_part;
  qd.dim = D;
  void* anyout = q ? q : (k ? k : vt);
  if (!anyout) return JEPA_B200_ERR_ARG;
  GemmOp op;
  if ((s = gemm_prepare(&op, static_cast<const __half*>(A), M, K, W, bias, EPI_QKV, anyout, N, &qd, nullptr)))
    return s;
  return gemm_launch(op, static_cast<cudaStream_t>(stream), e, g_timeout_ns);
}

int jepa_b200_op_attention(const void* q, const void* k, const void* vt, int B, int heads, int ntok, int npad,
                           int mask, int has_cls, int patches_per_slot, void* out, void* stream) {
  if (!aligned16(q) || !aligned16(k) || !aligned16(vt) || !aligned16(out)) return JEPA_B200_ERR_ARG;
  DevErr* e = op_err();
  if (!e) return JEPA_B200_ERR_CUDA;
  AttnOp op;
  int s = attn_prepare(&op, static_cast<const __half*>(q), static_cast<const __half*>(k),
                       static_cast<const __half*>(vt), B, heads, ntok, npad, mask, has_cls, patches_per_slot,
                       static_cast<__half*>(out));
  if (s) return s;
  return attn_launch(op, static_cast<cudaStream_t>(stream), e, g_timeout_ns);
}

int jepa_b200_op_patch_embed(const float* pixels, int B, int T, int H, int W, int patch, int tubelet,
                             const void* w_pe, int D, const float* bias, const float* pos, const float* cls,
                             int has_cls, float* x, void* stream) {
  if (!pixels || !w_pe || !pos || !x || (has_cls && !cls)) return JEPA_B200_ERR_ARG;
  if (B < 1 || patch < 1 || tubelet < 1 || T < tubelet || T % tubelet || H % patch || W % patch || H < patch ||
      W < patch || D < 64 || D % 32 != 0)
    return JEPA_B200_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(pos) || (bias && !aligned16(bias))) return JEPA_B200_ERR_ARG;
  // the limits of the model loader: K = 3 * kt * p^2 <= 32768, B * ntok * 4096 < 2^31
  if (D > 4096 || 3ll * tubelet * patch * patch > 32768 ||
      static_cast<long long>(B) * ((static_cast<long long>(T / tubelet) * (H / patch) * (W / patch)) + 1) >
          (1ll << 31) / 4096)
    return JEPA_B200_ERR_SHAPE;
  const int k_real = 3 * tubelet * patch * patch;
  const int kpad = (k_real + 63) / 64 * 64;
  const int n_patches = (T / tubelet) * (H / patch) * (W / patch);
  const int ntok = n_patches + (has_cls ? 1 : 0);
  DevMatrix Wm;
  int s = make_matrix(&Wm, w_pe, nullptr, JEPA_B200_F16, D, kpad);
  if (s) return s;
  DevErr* e = op_err();
  if (!e) return JEPA_B200_ERR_CUDA;
  PatchSrc ps;
  ps.pixels = pixels;
  ps.T = T;
  ps.H = H;
  ps.W = W;
  ps.patch = patch;
  ps.tubelet = tubelet;
  ps.n_patches = n_patches;
  ps.k_real = k_real;
  ps.pos = pos;
  ps.ntok = ntok;
  ps.has_cls = has_cls ? 1 : 0;
  // the unfolded patch matrix goes to a per-device scratch buffer that grows
  // on demand (growing waits for the device to be idle)
  static std::mutex mu;
  static void* scratch[64] = {nullptr};
  static size_t scratch_bytes[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return JEPA_B200_ERR_CUDA;
  const size_t need = static_cast<size_t>(B) * n_patches * kpad * 2;
  void* a = nullptr;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (scratch_bytes[dev] < need) {
      cudaDeviceSynchronize();
      if (scratch[dev]) cudaFree(scratch[dev]);
      scratch[dev] = nullptr;
      scratch_bytes[dev] = 0;
      if (cudaMalloc(&scratch[dev], need) != cudaSuccess) return JEPA_B200_ERR_CUDA;
      scratch_bytes[dev] = need;
    }
    a = scratch[dev];
  }
  GemmOp op;
  if ((s = gemm_prepare(&op, static_cast<const __half*>(a), B * n_patches, kpad, Wm, bias, EPI_PATCH, x, D, nullptr,
                        &ps)))
    return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = launch_patchify(pixels, ps, B, kpad, a, st, false))) return s;
  if ((s = gemm_launch(op, st, e, g_timeout_ns))) return s;
  if (has_cls) return launch_cls_rows(x, B, ntok, D, cls, pos, st);
  return JEPA_B200_OK;
}

int jepa_b200_op_gemv(const float* x, int M, int K, const void* w, const void* w_scales, int w_dtype, int N,
                      const float* bias, int epi, const float* resid, int resid_row_stride, float* y, void* stream) {
  if (epi < 0 || epi > 2 || M > 64) return JEPA_B200_ERR_ARG;
  DevMatrix W;
  int s = make_matrix(&W, w, w_scales, w_dtype, N, K);
  if (s) return s;
  return launch_gemv(x, M, K, W, bias, epi, resid, resid_row_stride, y, static_cast<cudaStream_t>(stream));
}

int jepa_b200_op_xattn_1q(const float* q, const void* k, const void* vt, int B, int heads, int ntok, int npad,
                          float* out, void* stream) {
  if (!aligned16(k)) return JEPA_B200_ERR_ARG;
  return launch_xattn_1q(q, static_cast<const __half*>(k), static_cast<const __half*>(vt), B, heads, ntok, npad, out,
                         static_cast<cudaStream_t>(stream));
}

int jepa_b200_op_rope(const jepa_b200_rope_args* a, void* stream) {
  if (!a) return JEPA_B200_ERR_ARG;
  const int es = dtype_bytes(a->dtype);
  if (!es) return JEPA_B200_ERR_DTYPE;
  if (a->B < 0 || a->N < 0 || a->heads < 0 || a->head_dim < 1 || a->head_dim > kMaxHeadDim ||
      static_cast<long long>(a->B) * a->N > 0x7fffffffll)
    return JEPA_B200_ERR_SHAPE;
  if (a->B == 0 || a->N == 0 || a->heads == 0) return JEPA_B200_OK;
  HeadOpParams p;
  memset(&p, 0, sizeof(p));
  int s = fill_rope(&p.rope, a->rope, a->head_dim, a->B);
  if (s) return s;
  if ((s = fill_tensor(&p.t[0], a->x, a->out, es, a->B, a->N, a->heads, a->head_dim))) return s;
  p.B = a->B;
  p.N = a->N;
  p.d = a->head_dim;
  p.norm = NORM_NONE;
  return launch_head_op(p, a->dtype, static_cast<cudaStream_t>(stream));
}

int jepa_b200_op_qk_norm_rope(const jepa_b200_qk_norm_rope_args* a, void* stream) {
  if (!a) return JEPA_B200_ERR_ARG;
  const int es = dtype_bytes(a->dtype);
  if (!es) return JEPA_B200_ERR_DTYPE;
  if (a->B < 0 || a->N < 0 || a->heads_q < 0 || a->heads_k < 0 || a->head_dim < 1 || a->head_dim > kMaxHeadDim ||
      static_cast<long long>(a->B) * a->N > 0x7fffffffll ||
      static_cast<long long>(a->heads_q) + a->heads_k > 0x7fffffffll)
    return JEPA_B200_ERR_SHAPE;
  if (a->norm != JEPA_B200_NORM_RMS && a->norm != JEPA_B200_NORM_LAYER) return JEPA_B200_ERR_ARG;
  if (!(a->eps >= 0.0f)) return JEPA_B200_ERR_ARG;
  if (a->B == 0 || a->N == 0 || (a->heads_q == 0 && a->heads_k == 0)) return JEPA_B200_OK;
  HeadOpParams p;
  memset(&p, 0, sizeof(p));
  int s = fill_rope(&p.rope, a->rope, a->head_dim, a->B);
  if (s) return s;
  int n = 0;
  const struct {
    const jepa_b200_heads *in, *out;
    int heads;
    const float *weight, *bias;
    int64_t weight_h, bias_h;
  } side[2] = {{&a->q, &a->q_out, a->heads_q, a->q_weight, a->q_bias, a->q_weight_stride_h, a->q_bias_stride_h},
               {&a->k, &a->k_out, a->heads_k, a->k_weight, a->k_bias, a->k_weight_stride_h, a->k_bias_stride_h}};
  for (const auto& x : side) {
    if (x.heads == 0) continue;
    if (!x.weight || !float_ptr_ok(x.weight) || !float_ptr_ok(x.bias) || x.weight_h < 0 || x.bias_h < 0)
      return JEPA_B200_ERR_ARG;
    HeadTensor& t = p.t[n++];
    if ((s = fill_tensor(&t, *x.in, *x.out, es, a->B, a->N, x.heads, a->head_dim))) return s;
    t.weight = x.weight;
    t.bias = x.bias;
    t.weight_h = x.weight_h;
    t.bias_h = x.bias_h;
  }
  p.B = a->B;
  p.N = a->N;
  p.d = a->head_dim;
  p.norm = a->norm == JEPA_B200_NORM_RMS ? NORM_RMS : NORM_LAYER;
  p.eps = a->eps;
  return launch_head_op(p, a->dtype, static_cast<cudaStream_t>(stream));
}

int jepa_b200_op_masked_attention(const jepa_b200_masked_attention_args* a, void* stream) {
  if (!a) return JEPA_B200_ERR_ARG;
  if (a->dtype != JEPA_B200_F16 && a->dtype != JEPA_B200_BF16) return JEPA_B200_ERR_DTYPE;
  if (a->B < 0 || a->Nq < 0 || a->Nk < 0 || a->heads_q < 1 || a->heads_kv < 1 || a->heads_q % a->heads_kv != 0 ||
      a->head_dim < 8 || a->head_dim > 128 || a->head_dim % 8 != 0 || a->B > 65535 || a->heads_q > 65535 ||
      static_cast<long long>(a->B) * a->heads_q > 0x7fffffffll || a->Nq > 0x3fffffff || a->Nk > 0x3fffffff)
    return JEPA_B200_ERR_SHAPE;
  if (!std::isfinite(a->scale) || !std::isfinite(a->cap) || a->cap < 0.0f || (a->causal != 0 && a->causal != 1)) return JEPA_B200_ERR_ARG;
  if (a->n_docs < 0 || (a->n_docs > 0) != (a->doc_offsets != nullptr) || (a->prefix && !a->causal))
    return JEPA_B200_ERR_ARG;
  if (a->n_docs > 0 && (a->Nq != a->Nk || a->kv_len || a->q_start)) return JEPA_B200_ERR_ARG;
  for (const void* x : {static_cast<const void*>(a->slopes), static_cast<const void*>(a->prefix),
                        static_cast<const void*>(a->doc_offsets), static_cast<const void*>(a->kv_len),
                        static_cast<const void*>(a->q_start)})
    if ((reinterpret_cast<uintptr_t>(x) & 3u) != 0) return JEPA_B200_ERR_ARG;
  if (a->B == 0 || a->Nq == 0) return JEPA_B200_OK;
  for (const jepa_b200_heads* t : {&a->q, &a->k, &a->v, &a->out}) {
    if (a->Nk == 0 && (t == &a->k || t == &a->v)) continue;  // nothing to read
    if (!heads_ok(*t, 2) || !aligned16(t->data) || t->stride_b % 8 != 0 || t->stride_n % 8 != 0 || t->stride_h % 8 != 0)
      return JEPA_B200_ERR_ARG;
  }
  if (!heads_out_ok(a->out, 2, a->B, a->Nq, a->heads_q, a->head_dim)) return JEPA_B200_ERR_ARG;
  MaskedAttnParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(a->q.data);
  p.k = static_cast<const uint16_t*>(a->k.data);
  p.v = static_cast<const uint16_t*>(a->v.data);
  p.out = static_cast<uint16_t*>(a->out.data);
  p.q_b = a->q.stride_b;
  p.q_n = a->q.stride_n;
  p.q_h = a->q.stride_h;
  p.k_b = a->k.stride_b;
  p.k_n = a->k.stride_n;
  p.k_h = a->k.stride_h;
  p.v_b = a->v.stride_b;
  p.v_n = a->v.stride_n;
  p.v_h = a->v.stride_h;
  p.o_b = a->out.stride_b;
  p.o_n = a->out.stride_n;
  p.o_h = a->out.stride_h;
  p.B = a->B;
  p.Nq = a->Nq;
  p.Nk = a->Nk;
  p.hq = a->heads_q;
  p.hk = a->heads_kv;
  p.d = a->head_dim;
  p.scale = a->scale;
  p.cap = a->cap;
  p.causal = a->causal;
  p.n_docs = a->n_docs;
  p.slopes = a->slopes;
  p.prefix = a->prefix;
  p.doc_offsets = a->doc_offsets;
  p.kv_len = a->kv_len;
  p.q_start = a->q_start;
  p.timeout_ns = g_timeout_ns;
  return launch_masked_attention(p, a->dtype == JEPA_B200_BF16, static_cast<cudaStream_t>(stream));
}

int jepa_b200_op_mean_pool(const float* y, int B, int ntok, int D, int first, float* out, void* stream) {
  if (!y || !out) return JEPA_B200_ERR_ARG;
  if (B < 1 || D < 1) return JEPA_B200_ERR_SHAPE;
  // partial column sums go to a per-device scratch buffer that grows on demand
  static std::mutex mu;
  static float* scratch[64] = {nullptr};
  static size_t scratch_n[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return JEPA_B200_ERR_CUDA;
  const size_t need = static_cast<size_t>(mean_pool_partial_floats(B, D));
  {
    std::lock_guard<std::mutex> lk(mu);
    if (scratch_n[dev] < need) {
      cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
      if (scratch[dev]) cudaFree(scratch[dev]);
      scratch[dev] = nullptr;
      scratch_n[dev] = 0;
      if (cudaMalloc(&scratch[dev], need * 4) != cudaSuccess) return JEPA_B200_ERR_CUDA;
      scratch_n[dev] = need;
    }
  }
  return launch_mean_pool(y, B, ntok, D, first, scratch[dev], out, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
