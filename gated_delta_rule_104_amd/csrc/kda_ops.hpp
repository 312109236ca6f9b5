// Internal launch interface of the companion operators (short convolution,
// selective scan, quantised state cache, gated linear recurrence, norm, drafts).
// Host-side only; no validation here.
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


// Whether an output of n rows of `bytes` bytes is written past the caches: rows that are whole 128-byte lines (parts
// of lines are joined in the caches only: a norm's rows of 2000 bytes 84 us against 112) of an output that they would
// not keep until it is read (32 MiB of L2).
inline bool whole_lines(const void* p, Str3 s, long long rows, long long bytes, long long elem) {
  return rows * bytes >= (32LL << 20) && bytes % 128 == 0 && reinterpret_cast<uintptr_t>(p) % 128 == 0 &&
         s.b * elem % 128 == 0 && s.h * elem % 128 == 0 && s.t * elem % 128 == 0;
}

// A launch holds fewer than 2^32 threads.  The *_fits say whether a call's launches do.
inline bool launchable(long long blocks, int threads) { return blocks * threads < (1LL << 32); }

// ------------------------------------------------ gated linear recurrence
struct GlrArgs {
  const void* x;     // [B, H, T, d]
  const void* la;
  const void* beta;  // or null (1)
  const float* h0;   // [B, H, d] or null (zero)
  const int* lens;   // [B] or null (T)
  void* o;           // (backward: the outputs, read)
  float* h_T;
  Str3 xs, ls, bs, os;
  int B, H, T, d;
  bool norm;
  // backward
  const void* dO = nullptr;
  const float* dh_T = nullptr;
  void* dx = nullptr;
  void* dla = nullptr;
  void* dbeta = nullptr;
  float* dh0 = nullptr;
  Str3 dos, dxs, dls, dbs;
  void* ws = nullptr;
  bool lines = false;  // outputs are written past the caches (set by the launch)
};
size_t glr_ws_bytes(int B, int H, int T, int d, bool bf16_io, bool gradients);
bool glr_fits(int B, int H, int T, int d, bool beta, bool norm, bool bf16_io, bool gradients);
bool glr_step_fits(int N, int H, int d, bool bf16_io);
// polls: how often a run of tokens looks for the state in front of it before it walks the sequence itself
hipError_t launch_glr(const GlrArgs& a, bool bf16_io, int polls, hipStream_t stream);
hipError_t launch_glr_step(const GlrArgs& a, bool bf16_io, hipStream_t stream);
hipError_t launch_glr_backward(const GlrArgs& a, bool bf16_io, int polls, hipStream_t stream);
// bit 0: a log_alpha above 0 or NaN, bit 1: a beta not finite.  Synchronises `stream`.
hipError_t check_glr_gates(const GlrArgs& a, bool bf16_io, hipStream_t stream, unsigned int* bits_out);

// ------------------------------------------------------------------- norm
struct NormArgs {
  const void* x;         // [B, H, T, d] (backward: the rows that were normalised)
  const void* residual;  // or null
  const void* gate;      // or null
  const void* w;         // [d], [H, d] or null (1)
  void* y;
  void* scales;          // 8 bits: a float per row, or a byte per 32 values
  void* s;               // x + residual, or null
  Str3 xs, rs, gs, ys, ss, ws, cs;  // ws: the weight's, 0 but for one row per head
  int rows, d, n1, n2;   // rows = n0 n1 n2
  int w_heads;           // rows of the weight
  float eps, inv_d;
  bool silu, e4m3, blocks;
  // backward
  const void* dy = nullptr;
  const void* ds = nullptr;  // or null
  void* dx = nullptr;
  void* dgate = nullptr;
  void* dw = nullptr;        // or null
  Str3 dys, dss, dxs, dgs;
  float* scratch = nullptr;
  int nparts = 0;
  // set by the launches
  bool lines = false;                                 // outputs are written past the caches
  long long hx = 0, hg = 0, hdy = 0, hds = 0, hdx = 0, hdg = 0;  // backward: from one row of the weight to the next
};
bool norm_fits(int rows, int d, bool bf16_io);
bool norm_backward_fits(int nparts, int d, int w_heads, bool weight, bool bf16_io);
int norm_parts(int rows, int d, int w_heads, bool bf16_io, int cus);
hipError_t launch_norm(NormArgs a, int B, int H, int T, bool bits8, bool bf16_io, hipStream_t stream);
hipError_t launch_norm_backward(NormArgs a, int B, int H, int T, bool bf16_io, hipStream_t stream);

// ----------------------------------------------------------------- drafts
struct VerifyArgs {
  const void* p;       // [N, K + 1, V]
  const void* q;       // [N, K, V] or null (one at the token)
  const int* tokens;   // [N, K]
  const float* u;      // [N, K + 1]
  const int* counts;   // [N] or null (K)
  int* accepted;       // [N]
  int* out;            // [N, K + 1]
  long long pn, pt, qn, qt;  // elements between sequences and tokens
  int N, K, V;
  void* ws;
};
size_t verify_ws_bytes(int N, int V);
bool verify_fits(int N, int V);
hipError_t launch_verify(const VerifyArgs& a, bool bf16_io, hipStream_t stream);
hipError_t launch_state_commit(const float* S_pos, const int* index, float* S, int N, int ntok, long long elems,
                               hipStream_t stream);

}  // namespace kda
