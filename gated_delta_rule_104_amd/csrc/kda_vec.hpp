// Rows of 16-byte vectors, as the memory-bound companion operators take them.
#pragma once

#include "kda_device.hpp"

namespace kda {

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

template <typename T>
struct Row {
  float v[kVec<T>];
};

template <typename T>
__device__ __forceinline__ Row<T> unpack(u32x4 w) {
  Row<T> r;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = __uint_as_float(w[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = __uint_as_float(w[i]);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ u32x4 pack(const Row<T>& r) {
  if constexpr (sizeof(T) == 2)
    return u32x4{cvt2(r.v[0], r.v[1]), cvt2(r.v[2], r.v[3]), cvt2(r.v[4], r.v[5]), cvt2(r.v[6], r.v[7])};
  else
    return u32x4{__float_as_uint(r.v[0]), __float_as_uint(r.v[1]), __float_as_uint(r.v[2]),
                 __float_as_uint(r.v[3])};
}

template <typename T>
__device__ __forceinline__ u32x4 ld16(const T* p) {
  return *reinterpret_cast<const u32x4*>(p);
}
template <typename T>
__device__ __forceinline__ void st16(T* p, u32x4 w) {
  *reinterpret_cast<u32x4*>(p) = w;
}

// The same for values that nothing reads again soon: they pass the caches without pushing out others.
template <typename T>
__device__ __forceinline__ u32x4 ld_once(const T* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}
template <typename V>
__device__ __forceinline__ void st_once(void* p, V w) {
  __builtin_nontemporal_store(w, static_cast<V*>(p));
}

// Either, by a choice that is the same for all lanes.  (Two stores to one place in two branches would be joined to
// one plain store; the empty statements keep them apart.)
template <typename V>
__device__ __forceinline__ void store_by(void* p, V w, bool once) {
  if (once) {
    asm volatile("");
    st_once(p, w);
    asm volatile("");
  } else {
    *static_cast<V*>(p) = w;
  }
}

// Registers whose contents the compiler must take as new: what it has computed from them before is then
// computed again where it is used again, instead of being kept.
template <int N>
__device__ __forceinline__ void forget(u32x4 (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(r[i]));
}
template <int N, int M>
__device__ __forceinline__ void forget(float (&r)[N][M]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < M; ++j) asm volatile("" : "+v"(r[i][j]));
}

__device__ __forceinline__ int seq_len(const int* lens, int b, int T) {
  if (!lens) return T;
  const int n = lens[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// The short convolution's SiLU: x times this.  The hardware's exponential and reciprocal, each within a unit in the last
// place of fp32: with the correctly rounded division and expf its four prompts of 8192 tokens (4096 channels, bf16) took 145
// us, bound by vector instructions.  The exponent's own rounding is |x| 2^-24 of the
// result, nothing beside bf16's; fp32 takes it back: t = x c is rounded, r what that and c's
// rounding left, e^-x = 2^t (1 + r ln 2).  (Past 128 the result is 0 or 1 whatever x
// is, and r of an infinity would be NaN; a NaN is held too, but x multiplies the result.)
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
  constexpr float c = -1.44269504088896340736f, c_low = -1.92596299e-8f;  // -log2(e) in two floats
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(c * x));
  } else {
    x = fminf(fmaxf(x, -128.f), 128.f);
    const float t = c * x, r = fmaf(c_low, x, fmaf(c, x, -t));
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t) * fmaf(r, 0.69314718055994530942f, 1.f));
  }
}

}  // namespace kda
