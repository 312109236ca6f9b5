// C-ABI of the companion operators: host-side validation and error mapping.
// Every check runs before anything is enqueued, so a rejected call writes
// nothing.  See include/libkda.h for the contract of each entry point.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "kda_host.hpp"
#include "kda_ops.hpp"

namespace {

using kda::api_fail;
using kda::api_ok;
using kda::Str3;

const long long kMaxElems = 1LL << 40;

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define OPS_TRY(expr)                       \
  do {                                      \
    const kda_status st_ = (expr);          \
    if (st_ != KDA_OK) return st_;          \
  } while (0)

kda_status need(const void* p, const char* name) {
  if (!p) return api_fail(KDA_ERR_NULL, "%s is NULL", name);
  if (!aligned(p)) return api_fail(KDA_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return KDA_OK;
}
kda_status too_large() { return api_fail(KDA_ERR_SHAPE, "problem too large"); }
kda_status need_any(const void* p, const char* name) {
  return p ? KDA_OK : api_fail(KDA_ERR_NULL, "%s is NULL", name);
}
kda_status maybe(const void* p, const char* name) { return p ? need(p, name) : KDA_OK; }

kda_status hip_fail(hipError_t e, const char* what) {
  return api_fail(KDA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

kda_status check_dtype(kda_dtype dt) {
  if (dt != KDA_F32 && dt != KDA_BF16) return api_fail(KDA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dt);
  return KDA_OK;
}

// Strides of [B, H, T, d] (contiguous without s) into *out.  row16: rows start on
// 16-byte boundaries.  Strides of dimensions of size 1, and of
// tensors without elements, are not looked at.
kda_status take_strides(const kda_strides* s, int B, int H, int T, int d, int es, bool row16, bool output,
                        const char* name, Str3* out) {
  // (a chunk's rows are addressed with 32-bit offsets from its first one)
  const long long most[3] = {kMaxElems, kMaxElems, 1 << 23};
  Str3 r{(long long)H * T * d, (long long)T * d, d};
  if (s) r = Str3{s->b, s->h, s->t};
  const long long v[3] = {r.b, r.h, r.t};
  const int n[3] = {B, H, T};
  const bool empty = B == 0 || H == 0 || T == 0;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1 || empty) continue;
    if (v[i] < 0 || v[i] > most[i] || (output && v[i] == 0))
      return api_fail(KDA_ERR_SHAPE, "%s: stride %lld of dimension %d is not usable", name, v[i], i);
    if (row16 && v[i] * es % 16)
      return api_fail(KDA_ERR_ALIGN, "%s: stride %lld of dimension %d is not a multiple of 16 bytes", name, v[i], i);
  }
  if (B <= 1) r.b = 0;
  if (H <= 1) r.h = 0;
  if (T <= 1) r.t = 0;
  *out = r;
  return KDA_OK;
}

kda_status conv_dims(int B, int H, int T, int d, int K, kda_activation act, kda_dtype dtype) {
  if (B < 0 || H < 0 || T < 0 || d < 0)
    return api_fail(KDA_ERR_SHAPE, "negative size B=%d H=%d T=%d d=%d", B, H, T, d);
  OPS_TRY(check_dtype(dtype));
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return api_fail(KDA_ERR_UNSUPPORTED, "unknown activation %d", (int)act);
  if (K < 2 || K > 4) return api_fail(KDA_ERR_UNSUPPORTED, "%d taps not supported (2, 3 or 4)", K);
  const int es = dtype == KDA_BF16 ? 2 : 4;
  if ((long long)d * es % 16) return api_fail(KDA_ERR_UNSUPPORTED, "rows of %d elements are not a multiple of 16 bytes", d);
  const long long C = (long long)H * d;
  // (a kernel's token index may pass the end by a block's runs)
  if (C > (1 << 28) || T > (1 << 30) || (long long)B * C > kMaxElems || (long long)B * C * T > kMaxElems ||
      (long long)B * C * (T / 8 + 1) / 8 / 64 > INT32_MAX)
    return api_fail(KDA_ERR_SHAPE, "problem too large");
  return KDA_OK;
}

kda_status ssm_dims(int B, int H, int G, int T, int dk, int dv, kda_dtype dtype) {
  if (B < 0 || H < 0 || G < 0 || T < 0)
    return api_fail(KDA_ERR_SHAPE, "negative size B=%d H=%d G=%d T=%d", B, H, G, T);
  OPS_TRY(check_dtype(dtype));
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128))
    return api_fail(KDA_ERR_UNSUPPORTED, "head sizes dk=%d dv=%d not supported (64 or 128)", dk, dv);
  if (H > 0 && (G == 0 || H % G)) return api_fail(KDA_ERR_SHAPE, "G=%d does not divide H=%d", G, H);
  const long long BH = (long long)B * H;
  if (BH > (1 << 24) || T > (1 << 30) || BH * T > kMaxElems / 128) return api_fail(KDA_ERR_SHAPE, "problem too large");
  return KDA_OK;
}

struct Plan {
  int nseg, chunks;
};
Plan ssm_plan(int B, int H, int G, int T, int dk, int dv, kda_dtype dtype, bool gradients) {
  Plan p;
  p.nseg = kda::ssm_plan(B, H, G, T, dk, dv, dtype == KDA_BF16, gradients, kda::api_cu_count(), &p.chunks);
  return p;
}

kda_status check_gates(const void* la, Str3 ls, const void* beta, Str3 bs, const int* lens, int B, int H, int T,
                       kda_dtype dtype, hipStream_t stream) {
  if (!kda::api_check_on()) return KDA_OK;
  unsigned int bits = 0u;
  const hipError_t e = kda::check_ssm_gates(la, ls, beta, bs, lens, B, H, T, dtype == KDA_BF16, stream, &bits);
  if (e != hipSuccess) return hip_fail(e, "input check");
  if (bits & 1u) return api_fail(KDA_ERR_PRECONDITION, "log_alpha has values above 0 or NaN (check mode)");
  if (bits & 2u) return api_fail(KDA_ERR_PRECONDITION, "beta has values that are not finite (check mode)");
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_conv_prefill(const void* x, const kda_strides* xs, const void* weight, const void* bias,
                            const void* state_in, const int* lens, void* o, const kda_strides* os, void* state_out,
                            int B, int H, int T, int d, int K, kda_activation act, kda_dtype dtype,
                            hipStream_t stream) {
  OPS_TRY(conv_dims(B, H, T, d, K, act, dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  kda::ConvArgs a{};
  OPS_TRY(take_strides(xs, B, H, T, d, es, true, false, "x", &a.xs));
  OPS_TRY(take_strides(os, B, H, T, d, es, true, true, "o", &a.os));
  if ((long long)B * H * d == 0 || (T == 0 && !state_out)) return api_ok();
  if (T > 0) {
    OPS_TRY(need(x, "x"));
    OPS_TRY(need_any(weight, "weight"));
    OPS_TRY(need(o, "o"));
  }
  OPS_TRY(maybe(state_in, "state_in"));
  OPS_TRY(maybe(state_out, "state_out"));
  if (state_out && state_out == state_in) return api_fail(KDA_ERR_UNSUPPORTED, "state_out must not be state_in");
  if (T > 0 && o == x) return api_fail(KDA_ERR_UNSUPPORTED, "o must not be x");
  a.x = x; a.w = weight; a.bias = bias; a.state = state_in; a.lens = lens; a.o = o; a.state_out = state_out;
  a.B = B; a.H = H; a.T = T; a.d = d; a.K = K; a.silu = act == KDA_ACT_SILU;
  const hipError_t e = kda::launch_conv(a, dtype == KDA_BF16, kda::api_cu_count(), stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_conv_prefill launch");
}

kda_status kda_conv_step(const void* x, const kda_strides* xs, void* state, const void* weight, const void* bias,
                         void* o, const kda_strides* os, int N, int H, int d, int K, kda_activation act,
                         kda_dtype dtype, hipStream_t stream) {
  OPS_TRY(conv_dims(N, H, 1, d, K, act, dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  kda::ConvArgs a{};
  OPS_TRY(take_strides(xs, N, H, 1, d, es, true, false, "x", &a.xs));
  OPS_TRY(take_strides(os, N, H, 1, d, es, true, true, "o", &a.os));
  if ((long long)N * H * d == 0) return api_ok();
  OPS_TRY(need(x, "x"));
  OPS_TRY(need(state, "state"));
  OPS_TRY(need_any(weight, "weight"));
  OPS_TRY(need(o, "o"));
  for (const void* in : {x, static_cast<const void*>(state), weight, bias})
    if (o == in) return api_fail(KDA_ERR_UNSUPPORTED, "o must not be an input");
  for (const void* in : {x, weight, bias})
    if (state == in) return api_fail(KDA_ERR_UNSUPPORTED, "state must not be another input");
  a.x = x; a.w = weight; a.bias = bias; a.state_out = state; a.o = o;
  a.B = N; a.H = H; a.T = 1; a.d = d; a.K = K; a.silu = act == KDA_ACT_SILU;
  const hipError_t e = kda::launch_conv_step(a, dtype == KDA_BF16, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_conv_step launch");
}

size_t kda_conv_backward_workspace_bytes(int B, int H, int T, int d, int K, kda_dtype dtype) {
  if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || conv_dims(B, H, T, d, K, KDA_ACT_NONE, dtype) != KDA_OK) return 0;
  return kda::conv_backward_ws_floats(B, H, T, d, K, dtype == KDA_BF16, kda::api_cu_count()) * sizeof(float);
}

kda_status kda_conv_backward(const void* x, const kda_strides* xs, const void* weight, const void* bias,
                             const void* state_in, const void* dO, const kda_strides* dos, const void* dstate_out,
                             void* dx, const kda_strides* dxs, void* dweight, void* dbias, void* dstate_in, int B,
                             int H, int T, int d, int K, kda_activation act, kda_dtype dtype, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  OPS_TRY(conv_dims(B, H, T, d, K, act, dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  kda::ConvArgs a{};
  OPS_TRY(take_strides(xs, B, H, T, d, es, true, false, "x", &a.xs));
  OPS_TRY(take_strides(dos, B, H, T, d, es, true, false, "dO", &a.dos));
  OPS_TRY(take_strides(dxs, B, H, T, d, es, true, true, "dx", &a.dxs));
  if ((long long)H * d == 0) return api_ok();
  if (B == 0 || T == 0) return api_fail(KDA_ERR_SHAPE, "the gradients need B >= 1 and T >= 1 (B=%d T=%d)", B, T);
  OPS_TRY(need(x, "x"));
  OPS_TRY(need_any(weight, "weight"));
  OPS_TRY(maybe(state_in, "state_in"));
  OPS_TRY(need(dO, "dO"));
  OPS_TRY(maybe(dstate_out, "dstate_out"));
  OPS_TRY(need(dx, "dx"));
  OPS_TRY(need_any(dweight, "dweight"));
  OPS_TRY(maybe(dstate_in, "dstate_in"));
  if (dx == x || dx == dO) return api_fail(KDA_ERR_UNSUPPORTED, "dx must not be x or dO");
  const size_t bytes = kda_conv_backward_workspace_bytes(B, H, T, d, K, dtype);
  if (!workspace) return api_fail(KDA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", bytes);
  if (!aligned(workspace)) return api_fail(KDA_ERR_ALIGN, "workspace is not 16-byte aligned");
  if (workspace_bytes < bytes)
    return api_fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, bytes);
  a.x = x; a.w = weight; a.bias = bias; a.state = state_in; a.dO = dO; a.dstate_out = dstate_out;
  a.dx = dx; a.dw = dweight; a.dbias = dbias; a.dstate = dstate_in; a.ws = static_cast<float*>(workspace);
  a.B = B; a.H = H; a.T = T; a.d = d; a.K = K; a.silu = act == KDA_ACT_SILU;
  const hipError_t e = kda::launch_conv_backward(a, dtype == KDA_BF16, kda::api_cu_count(), stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_conv_backward launch");
}

size_t kda_ssm_prefill_workspace_bytes(int B, int H, int G, int T, int dk, int dv, kda_dtype dtype) {
  if (B <= 0 || H <= 0 || T <= 0 || ssm_dims(B, H, G, T, dk, dv, dtype) != KDA_OK) return 0;
  const Plan p = ssm_plan(B, H, G, T, dk, dv, dtype, false);
  return kda::ssm_ws_floats(B, H, dk, dv, p.nseg) * sizeof(float);
}

kda_status kda_ssm_prefill(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                           const void* D, const float* S0, const int* lens, void* o, float* S_T,
                           const kda_ssm_strides* st, int B, int H, int G, int T, int dk, int dv, kda_dtype dtype,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  OPS_TRY(ssm_dims(B, H, G, T, dk, dv, dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  kda::SsmArgs a{};
  OPS_TRY(take_strides(st ? &st->q : nullptr, B, G, T, dk, es, true, false, "q", &a.qs));
  OPS_TRY(take_strides(st ? &st->k : nullptr, B, G, T, dk, es, true, false, "k", &a.ks));
  OPS_TRY(take_strides(st ? &st->v : nullptr, B, H, T, dv, es, true, false, "v", &a.vs));
  OPS_TRY(take_strides(st ? &st->log_alpha : nullptr, B, H, T, 1, es, false, false, "log_alpha", &a.ls));
  OPS_TRY(take_strides(st ? &st->beta : nullptr, B, H, T, 1, es, false, false, "beta", &a.bs));
  OPS_TRY(take_strides(st ? &st->o : nullptr, B, H, T, dv, es, true, true, "o", &a.os));
  if ((long long)B * H == 0) return api_ok();
  OPS_TRY(maybe(S0, "S0"));
  OPS_TRY(need(S_T, "S_T"));
  if (T > 0) {
    OPS_TRY(need(q, "q"));
    OPS_TRY(need(k, "k"));
    OPS_TRY(need(v, "v"));
    OPS_TRY(need_any(log_alpha, "log_alpha"));
    OPS_TRY(need_any(beta, "beta"));
    OPS_TRY(need(o, "o"));
    OPS_TRY(maybe(workspace, "workspace"));
    if (o == q || o == k || o == v) return api_fail(KDA_ERR_UNSUPPORTED, "o must not be an input");
    OPS_TRY(check_gates(log_alpha, a.ls, beta, a.bs, lens, B, H, T, dtype, stream));
  }
  a.q = q; a.k = k; a.v = v; a.la = log_alpha; a.beta = beta; a.D = D; a.S0 = S0; a.lens = lens; a.o = o; a.S_T = S_T;
  a.B = B; a.H = H; a.G = G; a.T = T; a.dk = dk; a.dv = dv;
  if (T > 0) {
    Plan p = ssm_plan(B, H, G, T, dk, dv, dtype, false);
    if (p.nseg > 1 && (!workspace || workspace_bytes < kda::ssm_ws_floats(B, H, dk, dv, p.nseg) * sizeof(float)))
      p = Plan{1, (T + kda::kSsmChunk - 1) / kda::kSsmChunk};
    a.nseg = p.nseg;
    a.seg_chunks = p.chunks;
    a.ws = static_cast<float*>(workspace);
    if (kda::api_log_on())
      fprintf(stderr, "[kda] ssm_prefill B=%d H=%d G=%d T=%d dk=%d dv=%d: %d segments of %d chunks\n", B, H, G, T, dk, dv,
              p.nseg, p.chunks);
  }
  const hipError_t e = kda::launch_ssm_prefill(a, dtype == KDA_BF16, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_ssm_prefill launch");
}

kda_status kda_ssm_step(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                        const void* D, float* S, void* o, int N, int H, int G, int dk, int dv, kda_dtype dtype,
                        hipStream_t stream) {
  OPS_TRY(ssm_dims(N, H, G, 1, dk, dv, dtype));
  if ((long long)N * H == 0) return api_ok();
  OPS_TRY(need(q, "q"));
  OPS_TRY(need(k, "k"));
  OPS_TRY(need(v, "v"));
  OPS_TRY(need_any(log_alpha, "log_alpha"));
  OPS_TRY(need_any(beta, "beta"));
  OPS_TRY(need(S, "S"));
  OPS_TRY(need(o, "o"));
  // (a group's q and k are read by the workgroups of all its heads)
  for (const void* in : {q, k, v, log_alpha, beta, static_cast<const void*>(S)})
    if (o == in) return api_fail(KDA_ERR_UNSUPPORTED, "o must not be an input");
  for (const void* in : {q, k, v})
    if (S == in) return api_fail(KDA_ERR_UNSUPPORTED, "S must not be another input");
  const Str3 gs{H, 1, 0};
  OPS_TRY(check_gates(log_alpha, gs, beta, gs, nullptr, N, H, 1, dtype, stream));
  const hipError_t e = kda::launch_ssm_step(q, k, v, log_alpha, beta, D, S, o, N, H, G, dk, dv, dtype == KDA_BF16, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_ssm_step launch");
}

size_t kda_ssm_backward_workspace_bytes(int B, int H, int G, int T, int dk, int dv, kda_dtype dtype) {
  if (B <= 0 || H <= 0 || T <= 0 || ssm_dims(B, H, G, T, dk, dv, dtype) != KDA_OK) return 0;
  const Plan p = ssm_plan(B, H, G, T, dk, dv, dtype, true);
  return kda::ssm_backward_ws_floats(B, H, G, T, dk, dv, p.nseg, dtype == KDA_BF16) * sizeof(float);
}

kda_status kda_ssm_backward(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                            const void* D, const float* S0, const void* dO, const float* dS_T, void* dq, void* dk_,
                            void* dv_, void* dlog_alpha, void* dbeta, void* dD, float* dS0, const kda_ssm_strides* st,
                            const kda_ssm_grad_strides* gst, int B, int H, int G, int T, int dk, int dv,
                            kda_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  OPS_TRY(ssm_dims(B, H, G, T, dk, dv, dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  kda::SsmArgs a{};
  OPS_TRY(take_strides(st ? &st->q : nullptr, B, G, T, dk, es, true, false, "q", &a.qs));
  OPS_TRY(take_strides(st ? &st->k : nullptr, B, G, T, dk, es, true, false, "k", &a.ks));
  OPS_TRY(take_strides(st ? &st->v : nullptr, B, H, T, dv, es, true, false, "v", &a.vs));
  OPS_TRY(take_strides(st ? &st->log_alpha : nullptr, B, H, T, 1, es, false, false, "log_alpha", &a.ls));
  OPS_TRY(take_strides(st ? &st->beta : nullptr, B, H, T, 1, es, false, false, "beta", &a.bs));
  OPS_TRY(take_strides(gst ? &gst->dO : nullptr, B, H, T, dv, es, true, false, "dO", &a.dos));
  OPS_TRY(take_strides(gst ? &gst->dq : nullptr, B, G, T, dk, es, true, true, "dq", &a.dqs));
  OPS_TRY(take_strides(gst ? &gst->dk : nullptr, B, G, T, dk, es, true, true, "dk_", &a.dks));
  OPS_TRY(take_strides(gst ? &gst->dv : nullptr, B, H, T, dv, es, true, true, "dv_", &a.dvs));
  OPS_TRY(take_strides(gst ? &gst->dlog_alpha : nullptr, B, H, T, 1, es, false, true, "dlog_alpha", &a.dls));
  OPS_TRY(take_strides(gst ? &gst->dbeta : nullptr, B, H, T, 1, es, false, true, "dbeta", &a.dbs));
  if (H == 0) return api_ok();
  if (B == 0 || T == 0) return api_fail(KDA_ERR_SHAPE, "the gradients need B >= 1 and T >= 1 (B=%d T=%d)", B, T);
  OPS_TRY(need(q, "q"));
  OPS_TRY(need(k, "k"));
  OPS_TRY(need(v, "v"));
  OPS_TRY(need_any(log_alpha, "log_alpha"));
  OPS_TRY(need_any(beta, "beta"));
  OPS_TRY(maybe(S0, "S0"));
  OPS_TRY(need(dO, "dO"));
  OPS_TRY(maybe(dS_T, "dS_T"));
  OPS_TRY(need(dq, "dq"));
  OPS_TRY(need(dk_, "dk_"));
  OPS_TRY(need(dv_, "dv_"));
  OPS_TRY(need_any(dlog_alpha, "dlog_alpha"));
  OPS_TRY(need_any(dbeta, "dbeta"));
  if (D) OPS_TRY(need_any(dD, "dD"));
  OPS_TRY(maybe(dS0, "dS0"));
  // (later launches read the inputs again)
  for (const void* out : {dq, dk_, dv_, dlog_alpha, dbeta})
    for (const void* in : {q, k, v, log_alpha, beta, dO})
      if (out == in) return api_fail(KDA_ERR_UNSUPPORTED, "a gradient must not be an input");
  if (dS0 && (dS0 == S0 || dS0 == dS_T)) return api_fail(KDA_ERR_UNSUPPORTED, "dS0 must not be S0 or dS_T");
  const Plan p = ssm_plan(B, H, G, T, dk, dv, dtype, true);
  const size_t bytes = kda::ssm_backward_ws_floats(B, H, G, T, dk, dv, p.nseg, dtype == KDA_BF16) * sizeof(float);
  if (!workspace) return api_fail(KDA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", bytes);
  if (!aligned(workspace)) return api_fail(KDA_ERR_ALIGN, "workspace is not 16-byte aligned");
  if (workspace_bytes < bytes)
    return api_fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, bytes);
  OPS_TRY(check_gates(log_alpha, a.ls, beta, a.bs, nullptr, B, H, T, dtype, stream));
  a.q = q; a.k = k; a.v = v; a.la = log_alpha; a.beta = beta; a.D = D; a.S0 = S0; a.dO = dO; a.dS_T = dS_T;
  a.dq = dq; a.dkk = dk_; a.dvv = dv_; a.dla = dlog_alpha; a.dbeta = dbeta; a.dD = D ? dD : nullptr; a.dS0 = dS0;
  a.B = B; a.H = H; a.G = G; a.T = T; a.dk = dk; a.dv = dv;
  a.nseg = p.nseg;
  a.seg_chunks = p.chunks;
  a.ws = static_cast<float*>(workspace);
  if (kda::api_log_on())
    fprintf(stderr, "[kda] ssm_backward B=%d H=%d G=%d T=%d dk=%d dv=%d: %d segments of %d chunks\n", B, H, G, T, dk, dv,
            p.nseg, p.chunks);
  const hipError_t e = kda::launch_ssm_backward(a, dtype == KDA_BF16, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_ssm_backward launch");
}

namespace {
kda_status cache_dims(int n, int nslots, int H, int dk, int dv, kda_cache_format f) {
  if (n < 0 || nslots < 0 || H < 0 || dk < 0 || dv < 0)
    return api_fail(KDA_ERR_SHAPE, "negative size n=%d nslots=%d H=%d dk=%d dv=%d", n, nslots, H, dk, dv);
  if (f != KDA_CACHE_INT8 && f != KDA_CACHE_E4M3) return api_fail(KDA_ERR_UNSUPPORTED, "unknown cache format %d", (int)f);
  if (dv % 32) return api_fail(KDA_ERR_UNSUPPORTED, "rows of %d values are not whole blocks of 32", dv);
  const long long e = (long long)dk * dv, nh = (long long)n * H;
  // (store looks each entry's slot up among the later ones)
  if (n > (1 << 16) || e > (1 << 24) || nh >= (1 << 24) || nh * e > kMaxElems || (long long)nslots * H > kMaxElems)
    return api_fail(KDA_ERR_SHAPE, "problem too large");
  return KDA_OK;
}
}  // namespace

kda_status kda_state_store(const float* S, const int* slots, void* cache, void* scales, int n, int nslots, int H,
                           int dk, int dv, kda_cache_format format, hipStream_t stream) {
  OPS_TRY(cache_dims(n, nslots, H, dk, dv, format));
  if ((long long)n * H * dk * dv == 0 || nslots == 0) return api_ok();
  OPS_TRY(need(S, "S"));
  OPS_TRY(need_any(slots, "slots"));
  OPS_TRY(need(cache, "cache"));
  OPS_TRY(need_any(scales, "scales"));
  const hipError_t e = kda::launch_state_store(S, slots, cache, static_cast<unsigned char*>(scales), n, nslots, H, dk,
                                               dv, format == KDA_CACHE_E4M3, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_state_store launch");
}

kda_status kda_state_load(const void* cache, const void* scales, const int* slots, float* S, int n, int nslots, int H,
                          int dk, int dv, kda_cache_format format, hipStream_t stream) {
  OPS_TRY(cache_dims(n, nslots, H, dk, dv, format));
  if ((long long)n * H * dk * dv == 0) return api_ok();
  if (nslots > 0) {
    OPS_TRY(need(cache, "cache"));
    OPS_TRY(need_any(scales, "scales"));
  }
  OPS_TRY(need_any(slots, "slots"));
  OPS_TRY(need(S, "S"));
  const hipError_t e = kda::launch_state_load(cache, static_cast<const unsigned char*>(scales), slots, S, n, nslots, H,
                                              dk, dv, format == KDA_CACHE_E4M3, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_state_load launch");
}

// ------------------------------------------------ gated linear recurrence
namespace {
kda_status glr_dims(int B, int H, int T, int d, kda_dtype dtype) {
  if (B < 0 || H < 0 || T < 0 || d < 0)
    return api_fail(KDA_ERR_SHAPE, "negative size B=%d H=%d T=%d d=%d", B, H, T, d);
  OPS_TRY(check_dtype(dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  if ((long long)d * es % 16) return api_fail(KDA_ERR_UNSUPPORTED, "rows of %d elements are not a multiple of 16 bytes", d);
  const long long C = (long long)H * d;
  if (C > (1 << 28) || T > (1 << 30) || (long long)B * C > kMaxElems || (long long)B * C * T > kMaxElems ||
      ((long long)B * ((C + 63) / 64) + 8) * (T / 32 + 1) > INT32_MAX)
    return too_large();
  return KDA_OK;
}

kda_status glr_inputs(kda::GlrArgs& a, const kda_glr_strides* st, int B, int H, int T, int d, bool has_beta, bool o_out,
                      kda_dtype dtype) {
  OPS_TRY(glr_dims(B, H, T, d, dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  OPS_TRY(take_strides(st ? &st->x : nullptr, B, H, T, d, es, true, false, "x", &a.xs));
  OPS_TRY(take_strides(st ? &st->log_alpha : nullptr, B, H, T, d, es, true, false, "log_alpha", &a.ls));
  if (has_beta) OPS_TRY(take_strides(st ? &st->beta : nullptr, B, H, T, d, es, true, false, "beta", &a.bs));
  OPS_TRY(take_strides(st ? &st->o : nullptr, B, H, T, d, es, true, o_out, "o", &a.os));
  a.B = B; a.H = H; a.T = T; a.d = d;
  return KDA_OK;
}

kda_status glr_check(const kda::GlrArgs& a, kda_dtype dtype, hipStream_t stream) {
  if (!kda::api_check_on()) return KDA_OK;
  unsigned int bits = 0u;
  const hipError_t e = kda::check_glr_gates(a, dtype == KDA_BF16, stream, &bits);
  if (e != hipSuccess) return hip_fail(e, "input check");
  if (bits & 1u) return api_fail(KDA_ERR_PRECONDITION, "log_alpha has values above 0 or NaN (check mode)");
  if (bits & 2u) return api_fail(KDA_ERR_PRECONDITION, "beta has values that are not finite (check mode)");
  return KDA_OK;
}

kda_status need_workspace(const void* workspace, size_t have, size_t bytes) {
  if (!bytes) return KDA_OK;
  if (!workspace) return api_fail(KDA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", bytes);
  if (!aligned(workspace)) return api_fail(KDA_ERR_ALIGN, "workspace is not 16-byte aligned");
  if (have < bytes) return api_fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", have, bytes);
  return KDA_OK;
}
}  // namespace

size_t kda_glr_prefill_workspace_bytes(int B, int H, int T, int d, kda_dtype dtype) {
  if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || glr_dims(B, H, T, d, dtype) != KDA_OK) return 0;
  return kda::glr_ws_bytes(B, H, T, d, dtype == KDA_BF16, false);
}

kda_status kda_glr_prefill(const void* x, const void* log_alpha, const void* beta, const float* h0, const int* lens,
                           void* o, float* h_T, const kda_glr_strides* st, int B, int H, int T, int d, int normalise,
                           kda_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::GlrArgs a{};
  OPS_TRY(glr_inputs(a, st, B, H, T, d, beta != nullptr, true, dtype));
  if ((long long)B * H * d == 0) return api_ok();
  if (!kda::glr_fits(B, H, T, d, beta != nullptr, normalise != 0, dtype == KDA_BF16, false)) return too_large();
  OPS_TRY(maybe(h0, "h0"));
  OPS_TRY(need(h_T, "h_T"));
  if (T > 0) {
    OPS_TRY(need(x, "x"));
    OPS_TRY(need(log_alpha, "log_alpha"));
    OPS_TRY(maybe(beta, "beta"));
    OPS_TRY(need(o, "o"));
    if (o == x || o == log_alpha || o == beta) return api_fail(KDA_ERR_UNSUPPORTED, "o must not be an input");
    OPS_TRY(need_workspace(workspace, workspace_bytes, kda_glr_prefill_workspace_bytes(B, H, T, d, dtype)));
  }
  a.x = x; a.la = log_alpha; a.beta = beta; a.h0 = h0; a.lens = lens; a.o = o; a.h_T = h_T;
  a.norm = normalise != 0;
  a.ws = workspace;
  if (T > 0) OPS_TRY(glr_check(a, dtype, stream));
  const hipError_t e = kda::launch_glr(a, dtype == KDA_BF16, kda::api_glr_polls(), stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_glr_prefill launch");
}

kda_status kda_glr_step(const void* x, const void* log_alpha, const void* beta, float* h, void* o,
                        const kda_glr_strides* st, int N, int H, int d, int normalise, kda_dtype dtype,
                        hipStream_t stream) {
  kda::GlrArgs a{};
  OPS_TRY(glr_inputs(a, st, N, H, 1, d, beta != nullptr, true, dtype));
  if ((long long)N * H * d == 0) return api_ok();
  if (!kda::glr_step_fits(N, H, d, dtype == KDA_BF16)) return too_large();
  OPS_TRY(need(x, "x"));
  OPS_TRY(need(log_alpha, "log_alpha"));
  OPS_TRY(maybe(beta, "beta"));
  OPS_TRY(need(h, "h"));
  OPS_TRY(need(o, "o"));
  for (const void* in : {x, log_alpha, beta, static_cast<const void*>(h)})
    if (o == in) return api_fail(KDA_ERR_UNSUPPORTED, "o must not be an input");
  for (const void* in : {x, log_alpha, beta})
    if (h == in) return api_fail(KDA_ERR_UNSUPPORTED, "h must not be another input");
  a.x = x; a.la = log_alpha; a.beta = beta; a.h_T = h; a.o = o;
  a.norm = normalise != 0;
  OPS_TRY(glr_check(a, dtype, stream));
  const hipError_t e = kda::launch_glr_step(a, dtype == KDA_BF16, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_glr_step launch");
}

size_t kda_glr_backward_workspace_bytes(int B, int H, int T, int d, kda_dtype dtype) {
  if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || glr_dims(B, H, T, d, dtype) != KDA_OK) return 0;
  return kda::glr_ws_bytes(B, H, T, d, dtype == KDA_BF16, true);
}

kda_status kda_glr_backward(const void* x, const void* log_alpha, const void* beta, const float* h0, const void* o,
                            const void* dO, const float* dh_T, const int* lens, void* dx, void* dlog_alpha, void* dbeta,
                            float* dh0, const kda_glr_strides* st, const kda_glr_grad_strides* gst, int B, int H, int T,
                            int d, int normalise, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  kda::GlrArgs a{};
  OPS_TRY(glr_inputs(a, st, B, H, T, d, beta != nullptr, false, dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  OPS_TRY(take_strides(gst ? &gst->dO : nullptr, B, H, T, d, es, true, false, "dO", &a.dos));
  OPS_TRY(take_strides(gst ? &gst->dx : nullptr, B, H, T, d, es, true, true, "dx", &a.dxs));
  OPS_TRY(take_strides(gst ? &gst->dlog_alpha : nullptr, B, H, T, d, es, true, true, "dlog_alpha", &a.dls));
  if (beta) OPS_TRY(take_strides(gst ? &gst->dbeta : nullptr, B, H, T, d, es, true, true, "dbeta", &a.dbs));
  if ((long long)H * d == 0) return api_ok();
  if (B == 0 || T == 0) return api_fail(KDA_ERR_SHAPE, "the gradients need B >= 1 and T >= 1 (B=%d T=%d)", B, T);
  if (!kda::glr_fits(B, H, T, d, beta != nullptr, normalise != 0, dtype == KDA_BF16, true)) return too_large();
  OPS_TRY(need(x, "x"));
  OPS_TRY(need(log_alpha, "log_alpha"));
  OPS_TRY(maybe(beta, "beta"));
  OPS_TRY(maybe(h0, "h0"));
  OPS_TRY(need(o, "o"));
  OPS_TRY(need(dO, "dO"));
  OPS_TRY(maybe(dh_T, "dh_T"));
  OPS_TRY(need(dx, "dx"));
  OPS_TRY(need(dlog_alpha, "dlog_alpha"));
  if (beta) OPS_TRY(need(dbeta, "dbeta"));
  OPS_TRY(maybe(dh0, "dh0"));
  for (const void* out : {dx, dlog_alpha, beta ? dbeta : dx})
    for (const void* in : {x, log_alpha, beta, o, dO})
      if (out == in) return api_fail(KDA_ERR_UNSUPPORTED, "a gradient must not be an input");
  if (dx == dlog_alpha || (beta && (dbeta == dx || dbeta == dlog_alpha)))
    return api_fail(KDA_ERR_UNSUPPORTED, "gradients must not share memory");
  if (dh0 && (dh0 == h0 || dh0 == dh_T)) return api_fail(KDA_ERR_UNSUPPORTED, "dh0 must not be h0 or dh_T");
  OPS_TRY(need_workspace(workspace, workspace_bytes, kda_glr_backward_workspace_bytes(B, H, T, d, dtype)));
  a.x = x; a.la = log_alpha; a.beta = beta; a.h0 = h0; a.lens = lens; a.o = const_cast<void*>(o); a.dO = dO; a.dh_T = dh_T;
  a.dx = dx; a.dla = dlog_alpha; a.dbeta = beta ? dbeta : nullptr; a.dh0 = dh0;
  a.norm = normalise != 0;
  a.ws = workspace;
  OPS_TRY(glr_check(a, dtype, stream));
  const hipError_t e = kda::launch_glr_backward(a, dtype == KDA_BF16, kda::api_glr_polls(), stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_glr_backward launch");
}

// ------------------------------------------------------------------- norm
namespace {
kda_status norm_dims(int B, int H, int T, int d, float eps, kda_gate gate_activation, kda_dtype dtype) {
  if (B < 0 || H < 0 || T < 0 || d < 0)
    return api_fail(KDA_ERR_SHAPE, "negative size B=%d H=%d T=%d d=%d", B, H, T, d);
  OPS_TRY(check_dtype(dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  if ((long long)d * es % 16) return api_fail(KDA_ERR_UNSUPPORTED, "rows of %d elements are not a multiple of 16 bytes", d);
  if (d > 32768) return api_fail(KDA_ERR_UNSUPPORTED, "rows of %d elements, at most 32768 are supported", d);
  if (gate_activation != KDA_GATE_SIGMOID && gate_activation != KDA_GATE_SILU)
    return api_fail(KDA_ERR_UNSUPPORTED, "unknown gate activation %d", (int)gate_activation);
  if (!(eps >= 0.f && eps < 1e30f)) return api_fail(KDA_ERR_UNSUPPORTED, "eps = %g is not a finite number of at least 0", eps);
  if ((long long)B * H > INT32_MAX || (long long)B * H * T > INT32_MAX - 65536 || (long long)H * d > (1 << 28))
    return too_large();
  return KDA_OK;
}
}  // namespace

kda_status kda_rms_norm(const void* x, const void* residual, const void* gate, const void* weight, void* y,
                        void* scales, void* residual_out, const kda_norm_strides* st, int B, int H, int T, int d,
                        int weight_per_head, float eps, kda_gate gate_activation, kda_norm_output output,
                        kda_dtype dtype, hipStream_t stream) {
  OPS_TRY(norm_dims(B, H, T, d, eps, gate_activation, dtype));
  if (output < KDA_OUT_SAME || output > KDA_OUT_E4M3_BLOCKS) return api_fail(KDA_ERR_UNSUPPORTED, "unknown output %d", (int)output);
  const bool bits8 = output != KDA_OUT_SAME, blocks = output == KDA_OUT_INT8_BLOCKS || output == KDA_OUT_E4M3_BLOCKS;
  if (blocks && d % 32) return api_fail(KDA_ERR_UNSUPPORTED, "rows of %d values are not whole blocks of 32", d);
  const int es = dtype == KDA_BF16 ? 2 : 4;
  kda::NormArgs a{};
  OPS_TRY(take_strides(st ? &st->x : nullptr, B, H, T, d, es, true, false, "x", &a.xs));
  if (residual) OPS_TRY(take_strides(st ? &st->residual : nullptr, B, H, T, d, es, true, false, "residual", &a.rs));
  if (gate) OPS_TRY(take_strides(st ? &st->gate : nullptr, B, H, T, d, es, true, false, "gate", &a.gs));
  // (8-bit rows are written 8 or 4 bytes at a time)
  OPS_TRY(take_strides(st ? &st->y : nullptr, B, H, T, d, es, true, true, "y", &a.ys));
  if (residual_out) OPS_TRY(take_strides(st ? &st->residual_out : nullptr, B, H, T, d, es, true, true, "residual_out", &a.ss));
  if (bits8) OPS_TRY(take_strides(st ? &st->scales : nullptr, B, H, T, blocks ? d / 32 : 1, 4, false, true, "scales", &a.cs));
  if ((long long)B * H * T * d == 0) return api_ok();
  if (!kda::norm_fits(B * H * T, d, dtype == KDA_BF16)) return too_large();
  OPS_TRY(need(x, "x"));
  OPS_TRY(maybe(residual, "residual"));
  OPS_TRY(maybe(gate, "gate"));
  OPS_TRY(maybe(weight, "weight"));
  OPS_TRY(need(y, "y"));
  OPS_TRY(maybe(residual_out, "residual_out"));
  if (bits8) OPS_TRY(need_any(scales, "scales"));
  if (bits8 && !blocks && (reinterpret_cast<uintptr_t>(scales) & 3u))
    return api_fail(KDA_ERR_ALIGN, "scales is not aligned to its floats");
  if (residual_out && !residual) return api_fail(KDA_ERR_UNSUPPORTED, "residual_out without a residual");
  for (const void* in : {x, residual, gate, weight})
    if (y == in || (bits8 && scales == in)) return api_fail(KDA_ERR_UNSUPPORTED, "y must not be an input");
  for (const void* in : {x, gate, weight})
    if (residual_out && residual_out == in) return api_fail(KDA_ERR_UNSUPPORTED, "residual_out must not be an input but residual");
  if (residual_out && residual_out == residual && (a.ss.b != a.rs.b || a.ss.h != a.rs.h || a.ss.t != a.rs.t))
    return api_fail(KDA_ERR_UNSUPPORTED, "residual_out in the place of residual has other strides");
  if (residual_out && residual_out == y) return api_fail(KDA_ERR_UNSUPPORTED, "residual_out must not be y");
  a.x = x; a.residual = residual; a.gate = gate; a.w = weight; a.y = y; a.scales = scales; a.s = residual_out;
  if (weight && weight_per_head && H > 1) a.ws.h = d;
  a.rows = B * H * T; a.d = d; a.eps = eps; a.inv_d = 1.f / (float)d;
  a.silu = gate_activation == KDA_GATE_SILU;
  a.e4m3 = output == KDA_OUT_E4M3_ROWS || output == KDA_OUT_E4M3_BLOCKS;
  a.blocks = blocks;
  const hipError_t e = kda::launch_norm(a, B, H, T, bits8, dtype == KDA_BF16, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_rms_norm launch");
}

size_t kda_rms_norm_backward_workspace_bytes(int B, int H, int T, int d, int weight_per_head, kda_dtype dtype) {
  if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || norm_dims(B, H, T, d, 0.f, KDA_GATE_SIGMOID, dtype) != KDA_OK) return 0;
  const int heads = weight_per_head ? H : 1;
  return (size_t)kda::norm_parts(B * H * T, d, heads, dtype == KDA_BF16, kda::api_cu_count()) * heads * d * sizeof(float);
}

kda_status kda_rms_norm_backward(const void* x, const void* gate, const void* weight, const void* dy,
                                 const void* dresidual_out, void* dx, void* dgate, void* dweight,
                                 const kda_norm_grad_strides* st, int B, int H, int T, int d, int weight_per_head,
                                 float eps, kda_gate gate_activation, kda_dtype dtype, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  OPS_TRY(norm_dims(B, H, T, d, eps, gate_activation, dtype));
  const int es = dtype == KDA_BF16 ? 2 : 4;
  kda::NormArgs a{};
  OPS_TRY(take_strides(st ? &st->x : nullptr, B, H, T, d, es, true, false, "x", &a.xs));
  if (gate) OPS_TRY(take_strides(st ? &st->gate : nullptr, B, H, T, d, es, true, false, "gate", &a.gs));
  OPS_TRY(take_strides(st ? &st->dy : nullptr, B, H, T, d, es, true, false, "dy", &a.dys));
  if (dresidual_out)
    OPS_TRY(take_strides(st ? &st->dresidual_out : nullptr, B, H, T, d, es, true, false, "dresidual_out", &a.dss));
  OPS_TRY(take_strides(st ? &st->dx : nullptr, B, H, T, d, es, true, true, "dx", &a.dxs));
  if (gate) OPS_TRY(take_strides(st ? &st->dgate : nullptr, B, H, T, d, es, true, true, "dgate", &a.dgs));
  if ((long long)H * d == 0) return api_ok();
  if (B == 0 || T == 0) return api_fail(KDA_ERR_SHAPE, "the gradients need B >= 1 and T >= 1 (B=%d T=%d)", B, T);
  const int heads = weight_per_head ? H : 1, nparts = kda::norm_parts(B * H * T, d, heads, dtype == KDA_BF16, kda::api_cu_count());
  if (!kda::norm_backward_fits(nparts, d, heads, weight != nullptr, dtype == KDA_BF16)) return too_large();
  OPS_TRY(need(x, "x"));
  OPS_TRY(maybe(gate, "gate"));
  OPS_TRY(maybe(weight, "weight"));
  OPS_TRY(need(dy, "dy"));
  OPS_TRY(maybe(dresidual_out, "dresidual_out"));
  OPS_TRY(need(dx, "dx"));
  if (gate) OPS_TRY(need(dgate, "dgate"));
  if (weight) OPS_TRY(need_any(dweight, "dweight"));
  for (const void* out : {dx, gate ? dgate : dx, weight ? dweight : dx})
    for (const void* in : {x, gate, weight, dy, dresidual_out})
      if (out == in) return api_fail(KDA_ERR_UNSUPPORTED, "a gradient must not be an input");
  if ((gate && dgate == dx) || (weight && (dweight == dx || (gate && dweight == dgate))))
    return api_fail(KDA_ERR_UNSUPPORTED, "gradients must not share memory");
  if (weight)
    OPS_TRY(need_workspace(workspace, workspace_bytes,
                           kda_rms_norm_backward_workspace_bytes(B, H, T, d, weight_per_head, dtype)));
  a.x = x; a.gate = gate; a.w = weight; a.dy = dy; a.ds = dresidual_out; a.dx = dx;
  a.dgate = gate ? dgate : nullptr;
  a.dw = weight ? dweight : nullptr;
  a.rows = B * H * T; a.d = d; a.w_heads = heads; a.eps = eps; a.inv_d = 1.f / (float)d;
  a.silu = gate_activation == KDA_GATE_SILU;
  a.scratch = static_cast<float*>(workspace);
  a.nparts = nparts;
  const hipError_t e = kda::launch_norm_backward(a, B, H, T, dtype == KDA_BF16, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_rms_norm_backward launch");
}

// ----------------------------------------------------------------- drafts
namespace {
kda_status verify_dims(int N, int K, int V, kda_dtype dtype) {
  if (N < 0 || K < 0 || V < 0) return api_fail(KDA_ERR_SHAPE, "negative size N=%d K=%d V=%d", N, K, V);
  OPS_TRY(check_dtype(dtype));
  if (N > (1 << 24) || K > (1 << 16) || V > (1 << 30) || !kda::verify_fits(N, V)) return too_large();
  return KDA_OK;
}

// The strides of rows of V probabilities, with the largest distances that sums in 64 bits hold.
kda_status row_strides(const kda_strides* s, int N, int K, int V, const char* name, long long* n, long long* t) {
  *n = s ? s->b : (long long)K * V;
  *t = s ? s->t : V;
  if (N <= 1) *n = 0;
  if (K <= 1) *t = 0;
  if (*n < 0 || *t < 0 || *n > kMaxElems || *t > kMaxElems)
    return api_fail(KDA_ERR_SHAPE, "%s: strides %lld and %lld are not usable", name, *n, *t);
  return KDA_OK;
}
}  // namespace

size_t kda_draft_verify_workspace_bytes(int N, int K, int V, kda_dtype dtype) {
  if (N <= 0 || V <= 0 || verify_dims(N, K, V, dtype) != KDA_OK) return 0;
  return kda::verify_ws_bytes(N, V);
}

kda_status kda_draft_verify(const void* target, const kda_strides* target_strides, const void* draft,
                            const kda_strides* draft_strides, const int* tokens, const float* uniforms,
                            const int* counts, int* accepted, int* out, int N, int K, int V, kda_dtype dtype,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  OPS_TRY(verify_dims(N, K, V, dtype));
  kda::VerifyArgs a{};
  OPS_TRY(row_strides(target_strides, N, K + 1, V, "target", &a.pn, &a.pt));
  OPS_TRY(row_strides(draft_strides, N, K, V, "draft", &a.qn, &a.qt));
  if (N == 0) return api_ok();
  if (V == 0) return api_fail(KDA_ERR_SHAPE, "no vocabulary (V = 0)");
  OPS_TRY(need_any(target, "target"));
  if (K > 0) OPS_TRY(need_any(tokens, "tokens"));
  OPS_TRY(need_any(uniforms, "uniforms"));
  OPS_TRY(need_any(accepted, "accepted"));
  OPS_TRY(need_any(out, "out"));
  const uintptr_t es = dtype == KDA_BF16 ? 2 : 4;
  for (const void* p : {target, draft})
    if (reinterpret_cast<uintptr_t>(p) % es) return api_fail(KDA_ERR_ALIGN, "probabilities are not aligned to their elements");
  for (const void* p : {static_cast<const void*>(tokens), static_cast<const void*>(uniforms), static_cast<const void*>(counts),
                        static_cast<const void*>(accepted), static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return api_fail(KDA_ERR_ALIGN, "an array of 32-bit values is not aligned to them");
  // (a second launch reads the inputs again)
  for (const void* o : {static_cast<const void*>(accepted), static_cast<const void*>(out)})
    for (const void* in : {target, draft, static_cast<const void*>(tokens), static_cast<const void*>(uniforms),
                           static_cast<const void*>(counts)})
      if (o == in) return api_fail(KDA_ERR_UNSUPPORTED, "an output must not be an input");
  if (accepted == out) return api_fail(KDA_ERR_UNSUPPORTED, "accepted must not be out");
  OPS_TRY(need_workspace(workspace, workspace_bytes, kda_draft_verify_workspace_bytes(N, K, V, dtype)));
  a.p = target; a.q = draft; a.tokens = tokens; a.u = uniforms; a.counts = counts; a.accepted = accepted; a.out = out;
  a.N = N; a.K = K; a.V = V;
  a.ws = workspace;
  const hipError_t e = kda::launch_verify(a, dtype == KDA_BF16, stream);
  return e == hipSuccess ? api_ok() : hip_fail(e, "kda_draft_verify launch");
}

kda_status kda_state_commit(const float* S_pos, const int* index, float* S, int N, int ntok, int H, int dk, int dv,
                            hipStream_t stream) {
  if (N < 0 || ntok < 0 || H < 0 || dk < 0 || dv < 0)
    return api_fail(KDA_ERR_SHAPE, "negative size N=%d ntok=%d H=%d dk=%d dv=%d", N, ntok, H, dk, dv);
  const long long e = (long long)dk * dv;
  if (N >= (1 << 24) || ntok > (1 << 16) || e > (1 << 24) || (long long)H * e > (1LL << 36) ||
      (long long)N * ntok > kMaxElems / ((long long)H * e + 1))
    return too_large();
  if ((long long)H * e % 4) return api_fail(KDA_ERR_UNSUPPORTED, "states of %lld floats are not a multiple of 16 bytes", (long long)H * e);
  if (N == 0 || ntok == 0 || H * e == 0) return api_ok();
  OPS_TRY(need(S_pos, "S_pos"));
  OPS_TRY(need_any(index, "index"));
  OPS_TRY(need(S, "S"));
  if (S == S_pos) return api_fail(KDA_ERR_UNSUPPORTED, "S must not be S_pos");
  const hipError_t err = kda::launch_state_commit(S_pos, index, S, N, ntok, H * e, stream);
  return err == hipSuccess ? api_ok() : hip_fail(err, "kda_state_commit launch");
}

}  // extern "C"
