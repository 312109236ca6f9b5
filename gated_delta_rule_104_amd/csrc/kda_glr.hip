// Gated linear recurrence: one decay per channel and token, a vector as state,
//     h_t = a_t h_{t-1} + n_t beta_t x_t,   o_t = h_t,   a = e^{log_alpha} <= 1,   n = 1 or sqrt(1 - a^2)
// and its gradients, with lam the gradient that reaches h_t:
//     lam_t = dO_t + a_{t+1} lam_{t+1} (+ dh_T at the end),   dx = n beta lam,   dbeta = n x lam,
//     dlog_alpha = a h_{t-1} lam - (a^2 / n) beta x lam,   dh0 = a_1 lam_1,
// where h_{t-1} is read back from the forward pass's outputs.
#include <mutex>
#include <type_traits>

#include "kda_ops.hpp"
#include "kda_vec.hpp"

namespace kda {

namespace {

// A decay a = e^x, x <= 0, in one float: a itself (sign bit clear) for strong decays, a - 1 (sign bit
// set, zero included) for x above -1/4.  A slow decay next to 1 keeps all its digits that way:
// as a float it would be off by up to 2^-25 a token, which a state that lasts 1/|x| tokens adds up
// to 2^-25 / |x| of itself, and so would 1 - a^2.
template <typename T>
__device__ __forceinline__ float decay_of(float x) {
  constexpr float c = 1.44269504088896340736f, c_low = 1.92596299e-8f;  // log2(e) in two floats
  float a;
  if constexpr (sizeof(T) == 2) {
    a = __builtin_amdgcn_exp2f(c * x);
  } else {
    // the rounding of x log2(e) is taken back (below -128 both forms give 0)
    const float y = fmaxf(x, -128.f), t = c * y, r = fmaf(c_low, y, fmaf(c, y, -t));
    a = __builtin_amdgcn_exp2f(t);
    a = x == x ? fmaf(a * r, 0.69314718055994530942f, a) : x;
  }
  // the series of (e^x - 1) / x; what follows is below x^6 / 5040, 2^-24 of it
  float p = fmaf(x, 1.f / 720, 1.f / 120);
  p = fmaf(x, p, 1.f / 24);
  p = fmaf(x, p, 1.f / 6);
  p = fmaf(x, p, 0.5f);
  p = x * fmaf(x, p, 1.f);
  return fabsf(x) < 0.25f ? __uint_as_float(__float_as_uint(p) | 0x80000000u) : a;
}
__device__ __forceinline__ bool slow(float e) { return (int)__float_as_uint(e) < 0; }

// a h + b; a decay of exactly zero clears the state whatever it holds.
template <typename A>
__device__ __forceinline__ A advance(float e, A h, float b) {
  const A keep = slow(e) ? h : (A)0;
  const A old = __float_as_uint(e) == 0u ? (A)0 : h;
  if constexpr (sizeof(A) == 4) return fmaf(old, e, b) + keep;
  else return fma(old, (double)e, (double)b) + keep;
}

// n = sqrt(1 - a^2) = sqrt((1 - a)(1 + a)).
__device__ __forceinline__ float unit_of(float e) {
  const float d = slow(e) ? -e : 1.f - e, s = slow(e) ? 2.f + e : 1.f + e;
  return __builtin_amdgcn_sqrtf(d * s);
}

// The state between tokens: fp32 inputs carry it in 64 bits, since its own rounding, 2^-25 a token,
// would be the largest error of outputs that are stored with 24 bits.
template <typename T> using State = typename std::conditional<sizeof(T) == 2, float, double>::type;

template <typename T>
__device__ __forceinline__ Row<T> ones() {
  Row<T> r;
#pragma unroll
  for (int c = 0; c < kVec<T>; ++c) r.v[c] = 1.f;
  return r;
}

// One lane per 16 bytes of channels, token after token.
template <typename T>
__global__ __launch_bounds__(256) void kda_glr_kernel(GlrArgs a, int nvec) {
  constexpr int V = kVec<T>, U = 8;
  const long long f = (long long)blockIdx.x * 256 + threadIdx.x;
  const int vec = (int)(f % nvec), b = (int)(f / nvec);
  if (b >= a.B) return;
  const int c0 = vec * V, hd = c0 / a.d, j0 = c0 % a.d;
  const T* x = static_cast<const T*>(a.x) + b * a.xs.b + hd * a.xs.h + j0;
  const T* la = static_cast<const T*>(a.la) + b * a.ls.b + hd * a.ls.h + j0;
  const T* beta = a.beta ? static_cast<const T*>(a.beta) + b * a.bs.b + hd * a.bs.h + j0 : nullptr;
  T* o = static_cast<T*>(a.o) + b * a.os.b + hd * a.os.h + j0;
  const long long at = ((long long)b * a.H + hd) * a.d + j0;
  const int len = seq_len(a.lens, b, a.T);
  State<T> h[V];
#pragma unroll
  for (int c = 0; c < V; ++c) h[c] = a.h0 ? a.h0[at + c] : 0.f;
  for (int t = 0; t < len; t += U) {
    u32x4 rx[U], rl[U], rb[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const long long tt = min(t + i, len - 1);
      rx[i] = ld16(x + tt * a.xs.t);
      rl[i] = ld16(la + tt * a.ls.t);
      if (beta) rb[i] = ld16(beta + tt * a.bs.t);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (t + i >= len) break;
      const Row<T> xv = unpack<T>(rx[i]), lv = unpack<T>(rl[i]), bv = beta ? unpack<T>(rb[i]) : ones<T>();
      Row<T> y;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float e = decay_of<T>(lv.v[c]);
        float in = bv.v[c] * xv.v[c];
        if (a.norm) in *= unit_of(e);
        h[c] = advance(e, h[c], in);
        y.v[c] = (float)h[c];
      }
      st16(o + (long long)(t + i) * a.os.t, pack<T>(y));
    }
  }
  if (a.h_T) {
#pragma unroll
    for (int c = 0; c < V; ++c) a.h_T[at + c] = (float)h[c];
  }
}

// One token per sequence, the state in place.
template <typename T>
__global__ __launch_bounds__(256) void kda_glr_step_kernel(GlrArgs a, int nvec) {
  constexpr int V = kVec<T>;
  const long long f = (long long)blockIdx.x * 256 + threadIdx.x;
  const int vec = (int)(f % nvec);
  const long long b = f / nvec;
  if (b >= a.B) return;
  const int c0 = vec * V, hd = c0 / a.d, j0 = c0 % a.d;
  float* h = a.h_T + (b * a.H + hd) * a.d + j0;
  f32x4 hv[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) hv[i] = *reinterpret_cast<const f32x4*>(h + 4 * i);
  const Row<T> xv = unpack<T>(ld16(static_cast<const T*>(a.x) + b * a.xs.b + hd * a.xs.h + j0));
  const Row<T> lv = unpack<T>(ld16(static_cast<const T*>(a.la) + b * a.ls.b + hd * a.ls.h + j0));
  const Row<T> bv = a.beta ? unpack<T>(ld16(static_cast<const T*>(a.beta) + b * a.bs.b + hd * a.bs.h + j0)) : ones<T>();
  Row<T> y;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const float e = decay_of<T>(lv.v[c]);
    float in = bv.v[c] * xv.v[c];
    if (a.norm) in *= unit_of(e);
    y.v[c] = (float)advance(e, (State<T>)hv[c / 4][c % 4], in);
    hv[c / 4][c % 4] = y.v[c];
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) *reinterpret_cast<f32x4*>(h + 4 * i) = hv[i];
  st16(static_cast<T*>(a.o) + b * a.os.b + hd * a.os.h + j0, pack<T>(y));
}

template <typename T>
__global__ __launch_bounds__(256) void kda_glr_bwd_kernel(GlrArgs a, int nvec) {
  constexpr int V = kVec<T>;
  const long long f = (long long)blockIdx.x * 256 + threadIdx.x;
  const int vec = (int)(f % nvec), b = (int)(f / nvec);
  if (b >= a.B) return;
  const int c0 = vec * V, hd = c0 / a.d, j0 = c0 % a.d;
  const T* x = static_cast<const T*>(a.x) + b * a.xs.b + hd * a.xs.h + j0;
  const T* la = static_cast<const T*>(a.la) + b * a.ls.b + hd * a.ls.h + j0;
  const T* beta = a.beta ? static_cast<const T*>(a.beta) + b * a.bs.b + hd * a.bs.h + j0 : nullptr;
  const T* o = static_cast<const T*>(a.o) + b * a.os.b + hd * a.os.h + j0;
  const T* dO = static_cast<const T*>(a.dO) + b * a.dos.b + hd * a.dos.h + j0;
  T* dx = static_cast<T*>(a.dx) + b * a.dxs.b + hd * a.dxs.h + j0;
  T* dla = static_cast<T*>(a.dla) + b * a.dls.b + hd * a.dls.h + j0;
  T* dbeta = a.dbeta ? static_cast<T*>(a.dbeta) + b * a.dbs.b + hd * a.dbs.h + j0 : nullptr;
  const long long at = ((long long)b * a.H + hd) * a.d + j0;
  const int len = seq_len(a.lens, b, a.T);
  State<T> lam[V];
#pragma unroll
  for (int c = 0; c < V; ++c) lam[c] = a.dh_T ? a.dh_T[at + c] : 0.f;
  const u32x4 zero{0u, 0u, 0u, 0u};
  for (int t = a.T - 1; t >= len; --t) {
    st16(dx + (long long)t * a.dxs.t, zero);
    st16(dla + (long long)t * a.dls.t, zero);
    if (dbeta) st16(dbeta + (long long)t * a.dbs.t, zero);
  }
  for (int t = len - 1; t >= 0; --t) {
    const Row<T> xv = unpack<T>(ld16(x + (long long)t * a.xs.t)), lv = unpack<T>(ld16(la + (long long)t * a.ls.t));
    const Row<T> bv = beta ? unpack<T>(ld16(beta + (long long)t * a.bs.t)) : ones<T>();
    const Row<T> g = unpack<T>(ld16(dO + (long long)t * a.dos.t));
    Row<T> before, gx, gl, gb;
    if (t > 0) {
      before = unpack<T>(ld16(o + (long long)(t - 1) * a.os.t));
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) before.v[c] = a.h0 ? a.h0[at + c] : 0.f;
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float e = decay_of<T>(lv.v[c]);
      lam[c] += (State<T>)g.v[c];
      const float l = (float)lam[c], al = slow(e) ? 1.f + e : e;
      float n = 1.f, slope = 0.f;
      if (a.norm) {
        n = unit_of(e);
        slope = n > 0.f ? al * al / n * (bv.v[c] * xv.v[c]) : 0.f;
      }
      gx.v[c] = n * bv.v[c] * l;
      gb.v[c] = n * xv.v[c] * l;
      gl.v[c] = al == 0.f ? 0.f : (al * before.v[c] - slope) * l;
      lam[c] = advance(e, lam[c], 0.f);
    }
    st16(dx + (long long)t * a.dxs.t, pack<T>(gx));
    st16(dla + (long long)t * a.dls.t, pack<T>(gl));
    if (dbeta) st16(dbeta + (long long)t * a.dbs.t, pack<T>(gb));
  }
  if (a.dh0) {
#pragma unroll
    for (int c = 0; c < V; ++c) a.dh0[at + c] = (float)lam[c];
  }
}

// ------------------------------------------------------------- input check
__device__ unsigned int g_glr_check_bits;

__global__ void kda_glr_check_clear_kernel(unsigned int* bits) { *bits = 0u; }

template <typename T>
__global__ __launch_bounds__(256) void kda_glr_check_kernel(GlrArgs a, int nvec, unsigned int* bits) {
  constexpr int V = kVec<T>;
  const long long n = (long long)a.B * a.T * nvec;
  unsigned int bad = 0u;
  for (long long f = (long long)blockIdx.x * 256 + threadIdx.x; f < n; f += (long long)gridDim.x * 256) {
    const int c0 = (int)(f % nvec) * V, hd = c0 / a.d, j0 = c0 % a.d;
    const long long bt = f / nvec;
    const int b = (int)(bt / a.T), t = (int)(bt % a.T);
    if (t >= seq_len(a.lens, b, a.T)) continue;
    const Row<T> l = unpack<T>(ld16(static_cast<const T*>(a.la) + b * a.ls.b + hd * a.ls.h + t * a.ls.t + j0));
    const Row<T> g = a.beta ? unpack<T>(ld16(static_cast<const T*>(a.beta) + b * a.bs.b + hd * a.bs.h + t * a.bs.t + j0)) : ones<T>();
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if (!(l.v[c] <= 0.f)) bad |= 1u;
      if (!(fabsf(g.v[c]) < __builtin_inff())) bad |= 2u;
    }
  }
  if (bad) atomicOr(bits, bad);
}

template <typename T>
hipError_t glr_fwd(const GlrArgs& a, hipStream_t stream) {
  const int nvec = a.H * a.d / kVec<T>;
  const dim3 grid((unsigned)(((long long)nvec * a.B + 255) / 256));
  hipLaunchKernelGGL((kda_glr_kernel<T>), grid, dim3(256), 0, stream, a, nvec);
  return hipGetLastError();
}

template <typename T>
hipError_t glr_step(const GlrArgs& a, hipStream_t stream) {
  const int nvec = a.H * a.d / kVec<T>;
  const dim3 grid((unsigned)(((long long)nvec * a.B + 255) / 256));
  hipLaunchKernelGGL((kda_glr_step_kernel<T>), grid, dim3(256), 0, stream, a, nvec);
  return hipGetLastError();
}

template <typename T>
hipError_t glr_bwd(const GlrArgs& a, hipStream_t stream) {
  const int nvec = a.H * a.d / kVec<T>;
  const dim3 grid((unsigned)(((long long)nvec * a.B + 255) / 256));
  hipLaunchKernelGGL((kda_glr_bwd_kernel<T>), grid, dim3(256), 0, stream, a, nvec);
  return hipGetLastError();
}

}  // namespace

size_t glr_ws_bytes(int, int, int, int, bool, bool, int) { return 0; }

hipError_t launch_glr(const GlrArgs& a, bool bf16_io, int, hipStream_t stream) {
  return bf16_io ? glr_fwd<bf16>(a, stream) : glr_fwd<float>(a, stream);
}

hipError_t launch_glr_step(const GlrArgs& a, bool bf16_io, hipStream_t stream) {
  return bf16_io ? glr_step<bf16>(a, stream) : glr_step<float>(a, stream);
}

hipError_t launch_glr_backward(const GlrArgs& a, bool bf16_io, int, hipStream_t stream) {
  return bf16_io ? glr_bwd<bf16>(a, stream) : glr_bwd<float>(a, stream);
}

hipError_t check_glr_gates(const GlrArgs& a, bool bf16_io, hipStream_t stream, unsigned int* bits_out) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);  // one check at a time: the flag is the device's only one
  void* p = nullptr;
  hipError_t e;
  if ((e = hipGetSymbolAddress(&p, HIP_SYMBOL(g_glr_check_bits))) != hipSuccess) return e;
  unsigned int* f = static_cast<unsigned int*>(p);
  hipLaunchKernelGGL(kda_glr_check_clear_kernel, dim3(1), dim3(1), 0, stream, f);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int nvec = a.H * a.d / (bf16_io ? 8 : 4);
  const long long nb = ((long long)a.B * a.T * nvec + 255) / 256;
  const dim3 grid((unsigned)(nb < 2048 ? nb : 2048));
  if (bf16_io) hipLaunchKernelGGL(kda_glr_check_kernel<bf16>, grid, dim3(256), 0, stream, a, nvec, f);
  else hipLaunchKernelGGL(kda_glr_check_kernel<float>, grid, dim3(256), 0, stream, a, nvec, f);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  unsigned int h = 0u;
  if ((e = hipMemcpyAsync(&h, f, sizeof(h), hipMemcpyDeviceToHost, stream)) != hipSuccess) return e;
  if ((e = hipStreamSynchronize(stream)) != hipSuccess) return e;
  *bits_out = h;
  return hipSuccess;
}

}  // namespace kda
