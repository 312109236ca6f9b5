// Internal launch interface of the companion operators (short convolution,
// selective scan, quantised state cache).  Host-side only; no validation here.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "kda_device.hpp"

namespace kda {

// Element strides of a [B, H, T, d] array whose rows of d are contiguous.
struct Str3 {
  long long b = 0, h = 0, t = 0;
};

// ------------------------------------------------------------ convolution
struct ConvArgs {
  const void* x;
  const void* w;      // [H, d, K]
  const void* bias;   // [H, d] or null
  const void* state;  // [B, H, K-1, d] or null (zero)
  const int* lens;    // [B] or null (T)
  void* o;
  void* state_out;    // [B, H, K-1, d] or null
  Str3 xs, os;
  int B, H, T, d, K;
  bool silu;
  // backward
  const void* dO = nullptr;
  const void* dstate_out = nullptr;
  void* dx = nullptr;
  void* dw = nullptr;
  void* dbias = nullptr;
  void* dstate = nullptr;
  Str3 dos, dxs;
  float* ws = nullptr;
};
hipError_t launch_conv(const ConvArgs& a, bool bf16_io, int cus, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs& a, bool bf16_io, hipStream_t stream);
size_t conv_backward_ws_floats(int B, int H, int T, int d, int K, bool bf16_io, int cus);
hipError_t launch_conv_backward(const ConvArgs& a, bool bf16_io, int cus, hipStream_t stream);

// ---------------------------------------------------- quantised state cache
// n states of H heads, dk x dv fp32, to or from slots of the cache; rows = dk.
hipError_t launch_state_store(const float* S, const int* slots, void* cache, unsigned char* scales, int n,
                              int nslots, int H, int dk, int dv, bool e4m3, hipStream_t stream);
hipError_t launch_state_load(const void* cache, const unsigned char* scales, const int* slots, float* S, int n,
                             int nslots, int H, int dk, int dv, bool e4m3, hipStream_t stream);

// -------------------------------------------------------- selective scan
struct SsmArgs {
  const void* q;    // [B, G, T, dk]
  const void* k;
  const void* v;    // [B, H, T, dv]
  const void* la;   // [B, H, T]
  const void* beta;
  const void* D;    // [H] or null
  const float* S0;  // [B, H, dk, dv] or null
  const int* lens;  // [B] or null
  void* o;
  float* S_T;
  Str3 qs, ks, vs, ls, bs, os;
  int B, H, G, T, dk, dv;
  // the sequence in nseg runs of seg_chunks 64-token chunks (the last may be shorter)
  int nseg = 1, seg_chunks = 0;
  float* ws = nullptr;
  // backward
  const void* dO = nullptr;
  const float* dS_T = nullptr;
  void* dq = nullptr;
  void* dkk = nullptr;
  void* dvv = nullptr;
  void* dla = nullptr;
  void* dbeta = nullptr;
  void* dD = nullptr;
  float* dS0 = nullptr;
  Str3 dos, dqs, dks, dvs, dls, dbs;
};
constexpr int kSsmChunk = 64;
// segments for a call (1: none), chunks per segment
int ssm_plan(int B, int H, int G, int T, int dk, int dv, bool bf16_io, bool gradients, int cus, int* seg_chunks);
size_t ssm_ws_floats(int B, int H, int dk, int dv, int nseg);
size_t ssm_backward_ws_floats(int B, int H, int G, int T, int dk, int dv, int nseg, bool bf16_io);
hipError_t launch_ssm_prefill(const SsmArgs& a, bool bf16_io, hipStream_t stream);
hipError_t launch_ssm_backward(const SsmArgs& a, bool bf16_io, hipStream_t stream);
hipError_t launch_ssm_step(const void* q, const void* k, const void* v, const void* la, const void* beta,
                           const void* D, float* S, void* o, int N, int H, int G, int dk, int dv, bool bf16_io,
                           hipStream_t stream);
// bit 0: a log_alpha above 0 or NaN, bit 1: a beta not finite.  Synchronises `stream`.
hipError_t check_ssm_gates(const void* la, Str3 ls, const void* beta, Str3 bs, const int* lens, int B, int H, int T, bool bf16_io,
                           hipStream_t stream, unsigned int* bits_out);

}  // namespace kda
