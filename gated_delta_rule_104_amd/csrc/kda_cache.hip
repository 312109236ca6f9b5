// The quantised state cache: fp32 states held in 8 bits.
//
// A state row (dv values) is cut into blocks of 32 values that share a scale
// 2^p, stored as the byte p + 127.  p is the smallest power, at least -126, with
// max|x| 2^-p <= 127 (int8) or 448 (e4m3), so nothing saturates, the scaling is
// exact and only the rounding of each value to nearest even loses anything.  A
// block with an infinity or NaN gets the byte 255 and reads back as NaN.
//
// Both directions are bound by HBM (5 bytes a value and 1/32 byte of scale): 64 states
// of 32 heads of 128 x 128 are stored in 33 us (25 when the states lie in the last-level
// cache), 256 loaded in 127 (5.3 TB/s).  On the
// way in four neighbouring lanes own a block, 8 values each: the block's largest
// value takes two quad moves, and a lane's 8 bytes are one store.
#include "kda_ops.hpp"

namespace kda {

namespace {

__device__ __forceinline__ float quad_max(float m) {
  m = fmaxf(m, __uint_as_float(dppu<DPP_QUAD_SWAP1>(__float_as_uint(m))));
  return fmaxf(m, __uint_as_float(dppu<DPP_QUAD_SWAP2>(__float_as_uint(m))));
}

template <bool E4M3>
__device__ __forceinline__ u32x2 quantise8(const float* x, float s) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = x[4 * i] * s, b = x[4 * i + 1] * s, c = x[4 * i + 2] * s, d = x[4 * i + 3] * s;
    if constexpr (E4M3) {
      int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    } else {
      w[i] = ((uint32_t)(int)rintf(a) & 255u) | (((uint32_t)(int)rintf(b) & 255u) << 8) |
             (((uint32_t)(int)rintf(c) & 255u) << 16) | ((uint32_t)(int)rintf(d) << 24);
    }
  }
  return u32x2{w[0], w[1]};
}

// One block of threads per (entry, head) and share of its values.  An entry
// whose slot is outside the cache, or that a later entry of the call names too,
// writes nothing.
template <bool E4M3>
__global__ __launch_bounds__(256) void kda_state_store_kernel(const float* __restrict__ S, const int* __restrict__ slots,
                                                              unsigned char* __restrict__ cache,
                                                              unsigned char* __restrict__ scales, int n, int nslots,
                                                              int H, int elems, int share) {
  const int part = blockIdx.x % share;
  const long long ih = blockIdx.x / share;
  const int i = (int)(ih / H), h = (int)(ih % H);
  const int slot = slots[i];
  if (slot < 0 || slot >= nslots) return;
  int later = 0;
  for (int j = i + 1 + (int)threadIdx.x; j < n; j += 256) later |= slots[j] == slot;
  if (__syncthreads_or(later)) return;
  const float* src = S + (size_t)ih * elems;
  const size_t dst = ((size_t)slot * H + h) * elems;
  for (int e = (part * 256 + (int)threadIdx.x) * 8; e < elems; e += share * 2048) {
    const f32x4 lo = *reinterpret_cast<const f32x4*>(src + e), hi = *reinterpret_cast<const f32x4*>(src + e + 4);
    float x[8], m = 0.f;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[c] = lo[c];
      x[4 + c] = hi[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      m = fmaxf(m, fabsf(x[c]));
      bad |= !(fabsf(x[c]) < __builtin_inff());
    }
    m = quad_max(bad ? __builtin_inff() : m);
    const bool block_bad = m == __builtin_inff();
    // m = f 2^ex with f in [1, 2): 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8
    const uint32_t mb = __float_as_uint(m);
    const int ex = (int)(mb >> 23) - 127;
    const uint32_t frac = mb & 0x7fffffu;
    int p = E4M3 ? ex - 8 + (frac > 0x600000u) : ex - 6 + (frac > 0x7e0000u);
    p = p < -126 ? -126 : p;
    u32x2 w = quantise8<E4M3>(x, block_bad ? 0.f : __uint_as_float((uint32_t)(127 - p) << 23));
    if (block_bad) w = u32x2{0u, 0u};
    *reinterpret_cast<u32x2*>(cache + dst + e) = w;
    if ((threadIdx.x & 3) == 0) scales[(dst + e) >> 5] = block_bad ? 255 : (unsigned char)(p + 127);
  }
}

// A lane reads four values at a time and writes 16 bytes, so that a wave's store is 1
// KiB of one run; four of them are in flight.
template <bool E4M3>
__global__ __launch_bounds__(256) void kda_state_load_kernel(const unsigned char* __restrict__ cache,
                                                             const unsigned char* __restrict__ scales,
                                                             const int* __restrict__ slots, float* __restrict__ S,
                                                             int nslots, int H, int elems, int share) {
  const int part = blockIdx.x % share;
  const long long ih = blockIdx.x / share;
  const int i = (int)(ih / H), h = (int)(ih % H);
  const int slot = slots[i];
  const bool have = slot >= 0 && slot < nslots;
  const size_t src = ((size_t)(have ? slot : 0) * H + h) * elems;
  float* dst = S + (size_t)ih * elems;
  constexpr int U = 4;
  for (int e0 = part * (1024 * U) + (int)threadIdx.x * 4; e0 < elems; e0 += share * (1024 * U)) {
    uint32_t w[U], sb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * 1024;
      w[u] = sb[u] = 0u;
      if (have && e < elems) {
        w[u] = *reinterpret_cast<const uint32_t*>(cache + src + e);
        sb[u] = scales[(src + e) >> 5];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * 1024;
      if (e >= elems) break;
      const float s = sb[u] == 255u ? __builtin_nanf("") : __uint_as_float(sb[u] << 23);
      f32x4 x;
      if constexpr (E4M3) {
        typedef float v2 __attribute__((ext_vector_type(2)));
        const v2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u], true);
        x = f32x4{a[0] * s, a[1] * s, b[0] * s, b[1] * s};
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = (float)(int)(signed char)(w[u] >> (8 * c)) * s;
      }
      *reinterpret_cast<f32x4*>(dst + e) = x;
    }
  }
}

// Blocks per (entry, head): one for every per_block values while there are few
// states, fewer where that would give more than 8192 blocks.
int state_share(long long nh, int elems, int per_block) {
  int share = (elems + per_block - 1) / per_block;
  while (share > 1 && nh * share > 8192) share = (share + 1) / 2;
  return share;
}

}  // namespace

hipError_t launch_state_store(const float* S, const int* slots, void* cache, unsigned char* scales, int n, int nslots,
                              int H, int dk, int dv, bool e4m3, hipStream_t stream) {
  const long long nh = (long long)n * H;
  const int elems = dk * dv, share = state_share(nh, elems, 2048);
  const dim3 grid((unsigned)(nh * share));
  unsigned char* c = static_cast<unsigned char*>(cache);
  if (e4m3)
    hipLaunchKernelGGL(kda_state_store_kernel<true>, grid, dim3(256), 0, stream, S, slots, c, scales, n, nslots, H, elems, share);
  else
    hipLaunchKernelGGL(kda_state_store_kernel<false>, grid, dim3(256), 0, stream, S, slots, c, scales, n, nslots, H, elems, share);
  return hipGetLastError();
}

hipError_t launch_state_load(const void* cache, const unsigned char* scales, const int* slots, float* S, int n,
                             int nslots, int H, int dk, int dv, bool e4m3, hipStream_t stream) {
  const long long nh = (long long)n * H;
  const int elems = dk * dv, share = state_share(nh, elems, 4096);
  const dim3 grid((unsigned)(nh * share));
  const unsigned char* c = static_cast<const unsigned char*>(cache);
  if (e4m3)
    hipLaunchKernelGGL(kda_state_load_kernel<true>, grid, dim3(256), 0, stream, c, scales, slots, S, nslots, H, elems, share);
  else
    hipLaunchKernelGGL(kda_state_load_kernel<false>, grid, dim3(256), 0, stream, c, scales, slots, S, nslots, H, elems, share);
  return hipGetLastError();
}

}  // namespace kda
