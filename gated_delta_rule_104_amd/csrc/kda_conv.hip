// Short causal convolution per channel, K = 2 .. 4 taps:
//     e = [state; x],   pre[t] = bias + sum_k w[k] e[t + k],   o[t] = act(pre[t]),
// state_out = the K - 1 rows of e that precede token T (or lens[b]).  act is the
// identity or SiLU, x sigma(x).  Gradients, with dpre = dO act'(pre):
//     de[t + k] += w[k] dpre[t],  dw[k] = sum_t dpre[t] e[t + k],  dbias = sum_t dpre[t].
//
// All of it is bound by HBM: a row element is read once and written once for K
// multiply-adds.  A lane owns one 16-byte group of channels of a run of tokens
// and keeps the K - 1 rows before the current one in registers, so only the
// first rows of a run are read twice.  Sums are fp32, rounded once on the store.
// Measured: four 8192-token sequences of 4096 channels, bf16 with SiLU, 113 us (4.9
// TB/s), gradients 181 us (4.8 TB/s); fp32 217 and 346 us (twice the bytes); one token of 256
// sequences 6.6 us, a chain of latencies (index divisions, taps, one row) and not HBM.
#include "kda_ops.hpp"
#include "kda_vec.hpp"

namespace kda {

namespace {

// The taps (w[c][k] for the lane's channels) and bias.
template <typename T, int K>
struct Taps {
  float w[K][kVec<T>];
  float b[kVec<T>];
  __device__ __forceinline__ void load(const T* wt, const T* bias, int c0) {
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][i] = to_f32(wt[(size_t)(c0 + i) * K + k]);
      b[i] = bias ? to_f32(bias[c0 + i]) : 0.f;
    }
  }
};

// Row r of e, r = token + K - 1: the state's rows come first.
template <typename T, int K>
__device__ __forceinline__ u32x4 ext_row(const T* x, long long st, const T* state, int d, int r) {
  if (r >= K - 1) return ld16(x + (long long)(r - (K - 1)) * st);
  if (state) return ld16(state + (long long)r * d);
  return u32x4{0u, 0u, 0u, 0u};
}

// One lane: 16 bytes of channels (vector vec of H * d) of tokens [t0, t0 + TT) of
// sequence b.  Groups of U tokens are loaded before they are used, so that a
// lane has U rows in flight.
template <typename T, int K, bool SILU>
__global__ __launch_bounds__(256) void kda_conv_kernel(ConvArgs a, int nvec, int ntiles, int TT) {
  constexpr int V = kVec<T>, U = 8;
  const long long f = (long long)blockIdx.x * 256 + threadIdx.x;
  const int vec = (int)(f % nvec);
  const long long bt = f / nvec;
  const int b = (int)(bt / ntiles), tile = (int)(bt % ntiles);
  if (b >= a.B) return;
  const int c0 = vec * V, h = c0 / a.d, j0 = c0 % a.d;
  const int len = seq_len(a.lens, b, a.T);
  const T* x = static_cast<const T*>(a.x) + b * a.xs.b + h * a.xs.h + j0;
  T* o = static_cast<T*>(a.o) + b * a.os.b + h * a.os.h + j0;
  const long long sbase = (((long long)b * a.H + h) * (K - 1)) * a.d + j0;
  const T* state = a.state ? static_cast<const T*>(a.state) + sbase : nullptr;
  if (tile == 0 && a.state_out) {
    T* so = static_cast<T*>(a.state_out) + sbase;
#pragma unroll
    for (int r = 0; r < K - 1; ++r) st16(so + (long long)r * a.d, ext_row<T, K>(x, a.xs.t, state, a.d, len + r));
  }
  const int t0 = tile * TT, t1 = min(t0 + TT, len);
  if (t0 >= t1) return;
  Taps<T, K> taps;
  taps.load(static_cast<const T*>(a.w), static_cast<const T*>(a.bias), c0);
  Row<T> e[K + U - 1];
#pragma unroll
  for (int r = 0; r < K - 1; ++r) e[r] = unpack<T>(ext_row<T, K>(x, a.xs.t, state, a.d, t0 + r));
  for (int t = t0; t < t1; t += U) {
    u32x4 raw[U];
    // past the end the last row is read again; its outputs are not stored
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i] = ld16(x + (long long)min(t + i, t1 - 1) * a.xs.t);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      e[K - 1 + i] = unpack<T>(raw[i]);
      Row<T> y;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        float s = taps.b[c];
#pragma unroll
        for (int k = 0; k < K; ++k) s += taps.w[k][c] * e[i + k].v[c];
        y.v[c] = SILU ? s * sigmoid<T>(s) : s;
      }
      if (t + i < t1) st16(o + (long long)(t + i) * a.os.t, pack<T>(y));
    }
#pragma unroll
    for (int r = 0; r < K - 1; ++r) e[r] = e[U + r];
  }
}

// One token per sequence: the state's rows and x are the K rows of the token;
// the state moves on by one row in place.
template <typename T, int K, bool SILU>
__global__ __launch_bounds__(256) void kda_conv_step_kernel(ConvArgs a, int nvec) {
  constexpr int V = kVec<T>;
  const long long f = (long long)blockIdx.x * 256 + threadIdx.x;
  const int vec = (int)(f % nvec);
  const long long b = f / nvec;
  if (b >= a.B) return;
  const int c0 = vec * V, h = c0 / a.d, j0 = c0 % a.d;
  T* state = static_cast<T*>(a.state_out) + ((b * a.H + h) * (K - 1)) * a.d + j0;
  u32x4 raw[K];
#pragma unroll
  for (int r = 0; r < K - 1; ++r) raw[r] = ld16(state + (long long)r * a.d);
  raw[K - 1] = ld16(static_cast<const T*>(a.x) + b * a.xs.b + h * a.xs.h + j0);
  Taps<T, K> taps;
  taps.load(static_cast<const T*>(a.w), static_cast<const T*>(a.bias), c0);
  Row<T> y;
#pragma unroll
  for (int c = 0; c < V; ++c) y.v[c] = taps.b[c];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Row<T> e = unpack<T>(raw[k]);
#pragma unroll
    for (int c = 0; c < V; ++c) y.v[c] += taps.w[k][c] * e.v[c];
  }
  if constexpr (SILU) {
#pragma unroll
    for (int c = 0; c < V; ++c) y.v[c] *= sigmoid<T>(y.v[c]);
  }
  st16(static_cast<T*>(a.o) + b * a.os.b + h * a.os.h + j0, pack<T>(y));
#pragma unroll
  for (int r = 0; r < K - 1; ++r) st16(state + (long long)r * a.d, raw[r + 1]);
}

// Gradients.  A block takes VB channel vectors (a power of two) and 256 / VB
// runs of TT tokens of one sequence.  A lane walks its run with the last K rows
// of e and of dpre in registers: at token t it forms dpre[t], adds its taps'
// gradients and emits de for row t (token t - K + 1), whose K contributions are
// then complete.  The walk goes K - 1 tokens past the run for the last rows.
// The taps' sums are joined over the block in LDS and written as one partial
// per block; a second kernel adds the partials in a fixed order.
template <typename T, int K, bool SILU>
__global__ __launch_bounds__(256) void kda_conv_bwd_kernel(ConvArgs a, int nvec, int VB, int nvb, int nrun, int TT) {
  constexpr int V = kVec<T>, U = 4;
  __shared__ float red[V * (K + 1)][256];
  const int tid = threadIdx.x;
  const int vb = blockIdx.x % nvb, part = blockIdx.x / nvb;  // part = b * nrun + run block
  const int b = part / nrun;
  const int nsub = 256 / VB;
  const int vec = vb * VB + (tid & (VB - 1));
  const int t0 = ((part % nrun) * nsub + tid / VB) * TT;
  const int t1 = min(t0 + TT, a.T);
  float dw[K][V], db[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    db[c] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][c] = 0.f;
  }
  if (vec < nvec && t0 < t1) {
    const int c0 = vec * V, h = c0 / a.d, j0 = c0 % a.d;
    const T* x = static_cast<const T*>(a.x) + b * a.xs.b + h * a.xs.h + j0;
    const T* dO = static_cast<const T*>(a.dO) + b * a.dos.b + h * a.dos.h + j0;
    T* dx = static_cast<T*>(a.dx) + b * a.dxs.b + h * a.dxs.h + j0;
    const long long sbase = (((long long)b * a.H + h) * (K - 1)) * a.d + j0;
    const T* state = a.state ? static_cast<const T*>(a.state) + sbase : nullptr;
    const T* dso = a.dstate_out ? static_cast<const T*>(a.dstate_out) + sbase : nullptr;
    T* ds = a.dstate ? static_cast<T*>(a.dstate) + sbase : nullptr;
    Taps<T, K> taps;
    taps.load(static_cast<const T*>(a.w), static_cast<const T*>(a.bias), c0);
    Row<T> e[K + U - 1], g[K + U - 1];  // rows of e and dpre before and at the current tokens
#pragma unroll
    for (int r = 0; r < K - 1; ++r) {
      e[r] = unpack<T>(ext_row<T, K>(x, a.xs.t, state, a.d, t0 + r));
#pragma unroll
      for (int c = 0; c < V; ++c) g[r].v[c] = 0.f;
    }
    for (int t = t0; t < t1 + K - 1; t += U) {
      u32x4 rx[U], rg[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long tt = min(t + i, a.T - 1);
        rx[i] = ld16(x + tt * a.xs.t);
        rg[i] = ld16(dO + tt * a.dos.t);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        e[K - 1 + i] = unpack<T>(rx[i]);
        Row<T> gy = unpack<T>(rg[i]);
        const bool have = t + i < a.T, mine = t + i < t1;
#pragma unroll
        for (int c = 0; c < V; ++c) {
          if constexpr (SILU) {
            float s = taps.b[c];
#pragma unroll
            for (int k = 0; k < K; ++k) s += taps.w[k][c] * e[i + k].v[c];
            const float sg = sigmoid<T>(s);
            gy.v[c] *= sg * (1.f + s * (1.f - sg));
          }
          if (!have) gy.v[c] = 0.f;
          if (mine) {
            db[c] += gy.v[c];
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][c] += gy.v[c] * e[i + k].v[c];
          }
        }
        g[K - 1 + i] = gy;
        const int u = t + i - (K - 1);  // the token whose gradient is complete
        if ((u >= t0 || t0 == 0) && u < t1) {
          Row<T> de;
#pragma unroll
          for (int c = 0; c < V; ++c) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) s += taps.w[k][c] * g[K - 1 + i - k].v[c];
            de.v[c] = s;
          }
          const int r = u - (a.T - (K - 1));  // row of state_out that token u became
          if (dso && r >= 0) {
            const Row<T> q = unpack<T>(ld16(dso + (long long)r * a.d));
#pragma unroll
            for (int c = 0; c < V; ++c) de.v[c] += q.v[c];
          }
          if (u >= 0) st16(dx + (long long)u * a.dxs.t, pack<T>(de));
          else if (ds) st16(ds + (long long)(u + K - 1) * a.d, pack<T>(de));
        }
      }
#pragma unroll
      for (int r = 0; r < K - 1; ++r) {
        e[r] = e[U + r];
        g[r] = g[U + r];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < V; ++c) {
#pragma unroll
    for (int k = 0; k < K; ++k) red[k * V + c][tid] = dw[k][c];
    red[K * V + c][tid] = db[c];
  }
  __syncthreads();
  // partial [part][k][channel], row K the bias
  const int C = nvec * V;
  float* out = a.ws + (size_t)part * (K + 1) * C;
  for (int i = tid; i < VB * V * (K + 1); i += 256) {
    const int k = i / (VB * V), ch = i % (VB * V), vl = ch / V, c = ch % V;
    if (vb * VB + vl >= nvec) continue;
    float s = 0.f;
    for (int u = 0; u < nsub; ++u) s += red[k * V + c][u * VB + vl];
    out[(size_t)k * C + vb * VB * V + ch] = s;
  }
}

// dw[c][k] and dbias[c]: sums of the partials, four interleaved runs of them per
// value, joined in a fixed order.
template <typename T>
__global__ __launch_bounds__(256) void kda_conv_taps_kernel(const float* ws, T* dw, T* dbias, int C, int K, int nparts) {
  __shared__ float red[4][64];
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n = (K + 1) * C;
  const int i = blockIdx.x * 64 + l;
  float s = 0.f;
  if (i < n) {
#pragma unroll 8
    for (int p = w; p < nparts; p += 4) s += ws[(size_t)p * n + i];
  }
  red[w][l] = s;
  __syncthreads();
  if (w == 0 && i < n) {
    s = (red[0][l] + red[1][l]) + (red[2][l] + red[3][l]);
    const int k = i / C, c = i % C;
    if (k < K) dw[(size_t)c * K + k] = from_f32<T>(s);
    else if (dbias) dbias[c] = from_f32<T>(s);
  }
}

struct ConvBwdPlan {
  int nvec, VB, nvb, nsub, TT, nrun, nparts;
};
// Runs of 64 tokens, or fewer (at least 8) where that would leave the chip with
// less than about 4 blocks a compute unit.
ConvBwdPlan conv_bwd_plan(int B, int H, int T, int d, bool bf16_io, int cus) {
  ConvBwdPlan p;
  const int V = bf16_io ? 8 : 4;
  p.nvec = H * d / V;
  p.VB = 1;
  while (p.VB < 64 && p.VB < p.nvec) p.VB *= 2;
  p.nvb = (p.nvec + p.VB - 1) / p.VB;
  p.nsub = 256 / p.VB;
  long long TT = (long long)B * T * p.nvb / (4LL * cus * p.nsub);
  TT = TT / 8 * 8;
  p.TT = (int)(TT < 8 ? 8 : (TT > 64 ? 64 : TT));
  p.nrun = (T + p.TT * p.nsub - 1) / (p.TT * p.nsub);
  p.nparts = B * p.nrun;
  return p;
}

template <typename T>
hipError_t conv_fwd(const ConvArgs& a, int cus, hipStream_t stream) {
  const int nvec = a.H * a.d / kVec<T>;
  // runs of 64 tokens, or fewer (at least 8) where that leaves the chip with
  // less than 16 waves a compute unit
  long long TT = (long long)a.B * nvec * a.T / (1024LL * cus) / 8 * 8;
  TT = TT < 8 ? 8 : (TT > 64 ? 64 : TT);
  const int ntiles = a.T > 0 ? (int)((a.T + TT - 1) / TT) : 1;
  const long long nthr = (long long)nvec * ntiles * a.B;
  const dim3 grid((unsigned)((nthr + 255) / 256));
#define KDA_CONV(KK)                                                                                             \
  do {                                                                                                           \
    if (a.silu) hipLaunchKernelGGL((kda_conv_kernel<T, KK, true>), grid, dim3(256), 0, stream, a, nvec, ntiles, (int)TT); \
    else hipLaunchKernelGGL((kda_conv_kernel<T, KK, false>), grid, dim3(256), 0, stream, a, nvec, ntiles, (int)TT); \
  } while (0)
  if (a.K == 2) KDA_CONV(2);
  else if (a.K == 3) KDA_CONV(3);
  else KDA_CONV(4);
#undef KDA_CONV
  return hipGetLastError();
}

template <typename T>
hipError_t conv_step(const ConvArgs& a, hipStream_t stream) {
  const int nvec = a.H * a.d / kVec<T>;
  const dim3 grid((unsigned)(((long long)nvec * a.B + 255) / 256));
#define KDA_CONV(KK)                                                                                          \
  do {                                                                                                        \
    if (a.silu) hipLaunchKernelGGL((kda_conv_step_kernel<T, KK, true>), grid, dim3(256), 0, stream, a, nvec); \
    else hipLaunchKernelGGL((kda_conv_step_kernel<T, KK, false>), grid, dim3(256), 0, stream, a, nvec);       \
  } while (0)
  if (a.K == 2) KDA_CONV(2);
  else if (a.K == 3) KDA_CONV(3);
  else KDA_CONV(4);
#undef KDA_CONV
  return hipGetLastError();
}

template <typename T>
hipError_t conv_bwd(const ConvArgs& a, int cus, hipStream_t stream) {
  const ConvBwdPlan p = conv_bwd_plan(a.B, a.H, a.T, a.d, sizeof(T) == 2, cus);
  const dim3 grid((unsigned)((long long)p.nvb * p.nparts));
#define KDA_CONV(KK)                                                                                            \
  do {                                                                                                          \
    if (a.silu)                                                                                                 \
      hipLaunchKernelGGL((kda_conv_bwd_kernel<T, KK, true>), grid, dim3(256), 0, stream, a, p.nvec, p.VB, p.nvb, p.nrun, p.TT); \
    else                                                                                                        \
      hipLaunchKernelGGL((kda_conv_bwd_kernel<T, KK, false>), grid, dim3(256), 0, stream, a, p.nvec, p.VB, p.nvb, p.nrun, p.TT); \
  } while (0)
  if (a.K == 2) KDA_CONV(2);
  else if (a.K == 3) KDA_CONV(3);
  else KDA_CONV(4);
#undef KDA_CONV
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int C = a.H * a.d;
  hipLaunchKernelGGL((kda_conv_taps_kernel<T>), dim3((unsigned)(((long long)(a.K + 1) * C + 63) / 64)), dim3(256), 0,
                     stream, a.ws, static_cast<T*>(a.dw), static_cast<T*>(a.dbias), C, a.K, p.nparts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_conv(const ConvArgs& a, bool bf16_io, int cus, hipStream_t stream) {
  return bf16_io ? conv_fwd<bf16>(a, cus, stream) : conv_fwd<float>(a, cus, stream);
}

hipError_t launch_conv_step(const ConvArgs& a, bool bf16_io, hipStream_t stream) {
  return bf16_io ? conv_step<bf16>(a, stream) : conv_step<float>(a, stream);
}

size_t conv_backward_ws_floats(int B, int H, int T, int d, int K, bool bf16_io, int cus) {
  return (size_t)conv_bwd_plan(B, H, T, d, bf16_io, cus).nparts * (K + 1) * H * d;
}

hipError_t launch_conv_backward(const ConvArgs& a, bool bf16_io, int cus, hipStream_t stream) {
  return bf16_io ? conv_bwd<bf16>(a, cus, stream) : conv_bwd<float>(a, cus, stream);
}

}  // namespace kda
