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

}  // extern "C"
