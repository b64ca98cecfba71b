// C ABI of the block's backward pass (declarations and contracts:
// include/h3.h), included by h3_api.cu, whose checks it uses.
#include "backward.cu"
#include "gemm_bwd.cu"
#include "attention_bwd.cu"

namespace {

// Workspaces are cut into 256-byte-aligned parts in the order they are taken.
struct Carve {
  uint8_t* base;
  size_t used = 0;
  explicit Carve(void* b) : base(static_cast<uint8_t*>(b)) {}
  template <typename T>
  T* take(size_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += (n * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

struct GatedWs {  // h3_gated_residual_backward and the outer half of h3_ffn_swiglu_backward
  bf16 *plain, *gated;
  float *gate_part, *split;  // split: partials of the split products, one after another
};
GatedWs carve_gated(Carve& c, const h3_dims* d, int L_pad, int K, size_t more_split) {
  using gemm_bwd::split_bytes;
  GatedWs w;
  w.plain = c.take<bf16>((size_t)L_pad * d->D);
  w.gated = c.take<bf16>((size_t)L_pad * d->D);
  w.gate_part = c.take<float>((size_t)3 * gate_parts(d->D, K, L_pad) * d->D);
  w.split = c.take<float>((split_bytes(d->D, K, L_pad / 64) + more_split) / 4);
  return w;
}
GatedWs carve_out(Carve& c, const h3_dims* d, int L_pad) {
  return carve_gated(c, d, L_pad, d->I, gemm_bwd::split_bytes(L_pad, d->I, d->D / 64));
}
GatedWs carve_ffn(Carve& c, const h3_dims* d, int L_pad) {
  using gemm_bwd::split_bytes;
  return carve_gated(c, d, L_pad, d->F,
                     split_bytes(L_pad, d->D, 2 * d->F / 64) + split_bytes(2 * d->F, d->D, L_pad / 64));
}
struct QkvWs {
  bf16* dqkv;
  float *norm_part, *split;
};
QkvWs carve_qkv(Carve& c, const h3_dims* d, int L_pad) {
  using gemm_bwd::split_bytes;
  QkvWs w;
  w.dqkv = c.take<bf16>((size_t)L_pad * 3 * d->I);
  w.norm_part = c.take<float>((size_t)QKNORM_PARTS * 2 * 128);
  w.split = c.take<float>((split_bytes(L_pad, d->D, 3 * d->I / 64) + split_bytes(3 * d->I, d->D, L_pad / 64)) / 4);
  return w;
}

int check_branch(int branch, const char* fn) {
  if (branch != H3_MSA && branch != H3_MLP) return fail(H3_ERR_SHAPE, "%s: branch must be H3_MSA or H3_MLP", fn);
  return H3_OK;
}

// a pointer that may be NULL but not misaligned
#define H3_OPTIONAL_PTR(p)                                                  \
  do {                                                                      \
    if (!aligned16(p)) return fail(H3_ERR_ALIGN, "%s: argument '%s' is not 16-byte aligned", __func__, #p); \
  } while (0)

bf16* b16(h3_bf16* p) { return reinterpret_cast<bf16*>(p); }
const bf16* b16(const h3_bf16* p) { return reinterpret_cast<const bf16*>(p); }

}  // namespace

extern "C" {

size_t h3_backward_workspace_bytes(const h3_dims* dims, int L_pad, int op) {
  if (check_dims(dims, __func__) != H3_OK || L_pad <= 0 || L_pad % 128 != 0) return 0;
  Carve c(nullptr);
  switch (op) {
    case H3_BWD_ADALN: c.take<float>((size_t)adaln_bwd_parts(dims->D) * 2 * dims->D); break;
    case H3_BWD_QKV: carve_qkv(c, dims, L_pad); break;
    case H3_BWD_ATTENTION: c.take<float>((size_t)2 * dims->H * L_pad); break;
    case H3_BWD_GATED_RESIDUAL: carve_out(c, dims, L_pad); break;
    case H3_BWD_FFN:
      carve_ffn(c, dims, L_pad);
      c.take<bf16>((size_t)L_pad * 3 * dims->F);
      break;
    default: return 0;
  }
  return c.used;
}

int h3_adaln_norm_modulate_backward(const h3_dims* dims, const h3_ranges* ranges, const float* x, const float* mod,
                                    int branch, const h3_bf16* dxm, const float* dres, float* dx, h3_bf16* dmod,
                                    void* ws, void* stream) {
  H3_TRACE();
  H3_CHECK(check_dims(dims, __func__));
  H3_CHECK(check_ranges(ranges, __func__));
  H3_CHECK(check_branch(branch, __func__));
  H3_REQUIRE_PTR(x);
  H3_REQUIRE_PTR(mod);
  H3_REQUIRE_PTR(dxm);
  H3_REQUIRE_PTR(dres);
  H3_REQUIRE_PTR(dx);
  H3_OPTIONAL_PTR(dmod);
  H3_REQUIRE_PTR(ws);
  if (dx == x) return fail(H3_ERR_SHAPE, "%s: dx must not be x (it may be dres)", __func__);
  cudaError_t e = launch_adaln_bwd(x, mod, branch, b16(dxm), dres, dx, ranges->start, ranges->count, ranges->L,
                                   ranges->L_pad, dims->D, dims->eps_ln, static_cast<float*>(ws), b16(dmod),
                                   static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "h3_adaln_norm_modulate_backward");
  return ok();
}

int h3_qkv_qknorm_mrope_backward(const h3_dims* dims, const h3_ranges* ranges, const h3_bf16* xm,
                                 const h3_bf16* Wqkv, const h3_bf16* qn_w, const h3_bf16* kn_w, const float* pos,
                                 const h3_bf16* dq, const h3_bf16* dk, const h3_bf16* dv, h3_bf16* dxm,
                                 h3_bf16* dWqkv, h3_bf16* dqn_w, h3_bf16* dkn_w, void* ws, void* stream) {
  H3_TRACE();
  H3_CHECK(check_dims(dims, __func__));
  H3_CHECK(check_ranges(ranges, __func__));
  H3_REQUIRE_PTR(xm);
  H3_REQUIRE_PTR(Wqkv);
  H3_REQUIRE_PTR(qn_w);
  H3_REQUIRE_PTR(kn_w);
  H3_REQUIRE_PTR(pos);
  H3_REQUIRE_PTR(dq);
  H3_REQUIRE_PTR(dk);
  H3_REQUIRE_PTR(dv);
  H3_REQUIRE_PTR(dxm);
  H3_OPTIONAL_PTR(dWqkv);
  H3_OPTIONAL_PTR(dqn_w);
  H3_OPTIONAL_PTR(dkn_w);
  H3_REQUIRE_PTR(ws);
  const int D = dims->D, I = dims->I, L = ranges->L, Lp = ranges->L_pad;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Carve c(ws);
  const QkvWs w = carve_qkv(c, dims, Lp);
  const int rope[3] = {dims->rope_t, dims->rope_h, dims->rope_w};
  int n_parts = 0;
  cudaError_t e = launch_qknorm_bwd(b16(xm), b16(Wqkv), b16(dq), b16(dk), b16(qn_w), b16(kn_w), pos, L, Lp, D, I, rope,
                                    dims->theta, dims->eps_qk, w.dqkv, w.norm_part, &n_parts, st);
  if (e != cudaSuccess) return cuda_fail(e, "h3_qkv_qknorm_mrope_backward: norm and RoPE");
  e = launch_dv_rows(b16(dv), dims->H, L, Lp, w.dqkv, st);
  if (e != cudaSuccess) return cuda_fail(e, "h3_qkv_qknorm_mrope_backward: dv");
  Products g(w.split);
  g.input_gradient(w.dqkv, b16(Wqkv), L, Lp, D, 3 * I, b16(dxm));
  if (dWqkv) g.weight_gradient(w.dqkv, b16(xm), L, Lp, 3 * I, D, b16(dWqkv));
  if (dqn_w || dkn_w) {  // norm_part [n_parts][2][128]
    g.fin.n_reduce = 2;
    g.fin.reduce.end[0] = g.fin.reduce.end[1] = n_parts;
    g.fin.reduce.out[0] = b16(dqn_w);
    g.fin.reduce.out[1] = b16(dkn_w);
    g.fin.reduce_part = w.norm_part;
    g.fin.reduce_stride = 256;
    g.fin.reduce_offset = 128;
    g.fin.reduce_cols = 128;
  }
  e = g.run(st);
  if (e != cudaSuccess) return cuda_fail(e, "h3_qkv_qknorm_mrope_backward: dxm, dWqkv");
  return ok();
}

int h3_attention_lse(const h3_dims* dims, const h3_ranges* ranges, const h3_bf16* q, const h3_bf16* k,
                     const h3_bf16* v, const h3_bf16* qn_w, const h3_bf16* kn_w, h3_bf16* o, float* lse,
                     void* stream) {
  H3_TRACE();
  H3_CHECK(check_dims(dims, __func__));
  H3_CHECK(check_ranges(ranges, __func__));
  H3_REQUIRE_PTR(q);
  H3_REQUIRE_PTR(k);
  H3_REQUIRE_PTR(v);
  if (qn_w || kn_w) {
    H3_REQUIRE_PTR(qn_w);
    H3_REQUIRE_PTR(kn_w);
  }
  H3_REQUIRE_PTR(o);
  H3_REQUIRE_PTR(lse);
  AttnProblem p;
  memset(&p, 0, sizeof(p));
  p.qn_w = b16(qn_w);
  p.kn_w = b16(kn_w);
  p.q = b16(q);
  p.k = b16(k);
  p.v = b16(v);
  p.o = b16(o);
  p.lse = lse;
  p.H = dims->H;
  p.L = ranges->L;
  p.L_pad = ranges->L_pad;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)dims->head_dim));
  cudaError_t e = launch_attention(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "h3_attention_lse");
  return ok();
}

int h3_attention_backward(const h3_dims* dims, const h3_ranges* ranges, const h3_bf16* q, const h3_bf16* k,
                          const h3_bf16* v, const h3_bf16* o, const float* lse, const h3_bf16* d_o, h3_bf16* dq,
                          h3_bf16* dk, h3_bf16* dv, void* ws, void* stream) {
  H3_TRACE();
  H3_CHECK(check_dims(dims, __func__));
  H3_CHECK(check_ranges(ranges, __func__));
  H3_REQUIRE_PTR(q);
  H3_REQUIRE_PTR(k);
  H3_REQUIRE_PTR(v);
  H3_REQUIRE_PTR(o);
  H3_REQUIRE_PTR(lse);
  H3_REQUIRE_PTR(d_o);
  H3_REQUIRE_PTR(dq);
  H3_REQUIRE_PTR(dk);
  H3_REQUIRE_PTR(dv);
  H3_REQUIRE_PTR(ws);
  const double scale = 1.0 / sqrt((double)dims->head_dim);
  cudaError_t e = launch_attention_bwd(b16(q), b16(k), b16(v), b16(o), lse, b16(d_o), dims->H, ranges->L,
                                       ranges->L_pad, (float)scale, (float)(1.4426950408889634 * scale), b16(dq),
                                       b16(dk), b16(dv), static_cast<float*>(ws), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "h3_attention_backward");
  return ok();
}

int h3_gated_residual_backward(const h3_dims* dims, const h3_ranges* ranges, const float* dx, const h3_bf16* o,
                               const h3_bf16* Wo, const float* mod, int branch, h3_bf16* d_o, h3_bf16* dWo,
                               h3_bf16* dmod, void* ws, void* stream) {
  H3_TRACE();
  H3_CHECK(check_dims(dims, __func__));
  H3_CHECK(check_ranges(ranges, __func__));
  H3_CHECK(check_branch(branch, __func__));
  H3_REQUIRE_PTR(dx);
  H3_REQUIRE_PTR(o);
  H3_REQUIRE_PTR(Wo);
  H3_REQUIRE_PTR(mod);
  H3_REQUIRE_PTR(d_o);
  H3_OPTIONAL_PTR(dWo);
  H3_OPTIONAL_PTR(dmod);
  H3_REQUIRE_PTR(ws);
  const int D = dims->D, I = dims->I, L = ranges->L, slot = 3 * branch + 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Carve c(ws);
  const GatedWs w = carve_out(c, dims, ranges->L_pad);
  cudaError_t e = launch_gate_cast(dx, mod, slot, ranges->start, ranges->count, L, D, dWo || dmod ? w.plain : nullptr,
                                   w.gated, st);
  if (e != cudaSuccess) return cuda_fail(e, "h3_gated_residual_backward: gate");
  Products g(w.split);
  g.input_gradient(w.gated, b16(Wo), L, ranges->L_pad, I, D, b16(d_o));
  if (dWo || dmod)
    g.gated_weight_gradient(w.plain, b16(o), ranges->start, ranges->count, ranges->L_pad, D, I, mod, slot, b16(Wo),
                            b16(dWo), b16(dmod), w.gate_part);
  e = g.run(st);
  if (e != cudaSuccess) return cuda_fail(e, "h3_gated_residual_backward: do, dWo");
  return ok();
}

int h3_ffn_swiglu_backward(const h3_dims* dims, const h3_ranges* ranges, const float* dx, const h3_bf16* xm,
                           const h3_bf16* Wgu, const h3_bf16* Wd, const float* mod, h3_bf16* dxm, h3_bf16* dWgu,
                           h3_bf16* dWd, h3_bf16* dmod, void* ws, void* stream) {
  H3_TRACE();
  H3_CHECK(check_dims(dims, __func__));
  H3_CHECK(check_ranges(ranges, __func__));
  H3_REQUIRE_PTR(dx);
  H3_REQUIRE_PTR(xm);
  H3_REQUIRE_PTR(Wgu);
  H3_REQUIRE_PTR(Wd);
  H3_REQUIRE_PTR(mod);
  H3_REQUIRE_PTR(dxm);
  H3_OPTIONAL_PTR(dWgu);
  H3_OPTIONAL_PTR(dWd);
  H3_OPTIONAL_PTR(dmod);
  H3_REQUIRE_PTR(ws);
  const int D = dims->D, F = dims->F, L = ranges->L, Lp = ranges->L_pad, slot = 5;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Carve c(ws);
  const GatedWs w = carve_ffn(c, dims, Lp);
  bf16* h = c.take<bf16>((size_t)Lp * 3 * F);
  bf16* dgu = h + (size_t)Lp * F;
  cudaError_t e = launch_gate_cast(dx, mod, slot, ranges->start, ranges->count, L, D, dWd || dmod ? w.plain : nullptr,
                                   w.gated, st);
  if (e != cudaSuccess) return cuda_fail(e, "h3_ffn_swiglu_backward: gate");
  e = launch_ffn_bwd(b16(xm), w.gated, b16(Wgu), b16(Wd), L, D, F, h, dgu, st);
  if (e != cudaSuccess) return cuda_fail(e, "h3_ffn_swiglu_backward: hidden state");
  Products g(w.split);  // the longest contraction first
  g.input_gradient(dgu, b16(Wgu), L, Lp, D, 2 * F, b16(dxm));
  if (dWgu) g.weight_gradient(dgu, b16(xm), L, Lp, 2 * F, D, b16(dWgu));
  if (dWd || dmod)
    g.gated_weight_gradient(w.plain, h, ranges->start, ranges->count, Lp, D, F, mod, slot, b16(Wd), b16(dWd), b16(dmod),
                            w.gate_part);
  e = g.run(st);
  if (e != cudaSuccess) return cuda_fail(e, "h3_ffn_swiglu_backward: dxm, dWgu, dWd");
  return ok();
}

}  // extern "C"
