// Selective state space scan with one decay per head and token, prefill and
// gradients, in 64-token chunks on the matrix cores.
//
// One form serves every pass.  For row vectors Q_i, K_i (the contracted ones) and
// V_i of a chunk, decays x_i <= 0 and weights rho_i, kappa_j, with l_i the sum of
// x up to and including i,
//     Y_i  = rho_i ( e^{l_i} S^T Q_i + sum_{j <= i} e^{l_i - l_j} kappa_j (Q_i.K_j) V_j )
//     S   <- e^{l_end} S + sum_j e^{l_end - l_j} kappa_j K_j V_j^T.
//   pass                Q   K   V   kappa  rho   result
//   outputs             q   k   v   beta   1     o (+ D v)
//   reversed outputs    k   q   dO  1      1     z = dS^T k: dv = beta z + D dO, dbeta = v.z
//   dq (heads summed)   dO  v   k   beta   1     dq
//   dk (heads summed)   v   dO  q   1      beta  dk
// The reversed passes walk the tokens backwards; a position's decay is then the
// one of the token after it (1 at the last token).
//
// Decays.  e^{l_i - l_j} is never formed from sums over the chunk, whose
// difference would lose digits: sums run inside blocks of 16 tokens only, from
// the block's start (u_i), to its end (w_j) and over whole blocks (E_J), so that
// e^{l_i - l_j} = w_j E.. u_i across blocks is a product of factors <= 1, and
// inside a block the exponential of a difference of 16-token sums.  Nothing
// overflows for any log_alpha <= 0; -inf is held at 2^-180, which is zero in fp32.
// That difference still loses digits behind a strong decay or a reset in the block: up
// to 16 times 180 in fp32, whose step there is 2.4e-4.  With fp32 inputs the sums are
// formed in 64 bits and kept in two floats (48 bits), whose differences are exact to the
// difference's own digits.  With bf16 inputs, whose scores are rounded by up to 2^-8 of
// themselves, one float is enough: it costs a decay 2e-4 or so, with a reset every second token.
//
// Tiles.  v_mfma 16x16: the accumulator's rows 4g + e (g = lane / 16) are also the
// contraction order of the next product's operand, so the scores (formed
// transposed) and the state feed it from registers.  Rows of the state are taken in
// the order 32c + 8(r / 4) + 4(odd) + r % 4 for row r of an (even, odd) pair of
// tiles, which makes a lane's share of a pair eight consecutive channels, so that
// the rows it is multiplied with are read in their natural order.  A wave owns NC
// column tiles of a state: two with bf16 (64 registers a lane for 128 rows, two waves
// a SIMD; the columns taken in the same paired order, so that results are stored 16
// bytes a lane), one with fp32, whose tiles fill the LDS and whose products are long.
// bf16 with one column tile and twice the waves took 580 us where this took 561, for
// the outputs of 64K tokens, 64 heads of 128 x 64 (now 464 in the same trace, of a
// process's first calls; 375 after some tens of calls).
//
// Precision.  bf16 inputs are exact operands.  The scores and the state are
// rounded once to bf16 where they multiply V and Q (both times one rounding in
// front of an fp32 sum, like the output's own); the weighted V that updates the
// fp32 state is carried in three bf16 terms (24 bits) where the state is a result,
// in two (16 bits) where it only multiplies Q afterwards, rounded to fewer.  The
// gradient of log_alpha sums what pairs of tokens owe each other, so the score sums it
// needs are taken from fp32 scores and the state terms from a two-term (16-bit)
// state.  fp32 inputs run the same kernels on the fp32 matrix instructions.
//
// Measured (bf16): 64K tokens, 64 heads of 128 x 64 in 8 groups 0.59 ms, of that
// outputs 0.375 (1.4 GB, 3.75 TB/s), the state pass 0.198 and the merge 0.016; gradients
// of four 8K sequences, 32 heads in 4 groups 0.67 ms (dq and dk 0.285, reversed outputs
// 0.167, states 0.109, the sums of partial results 0.080, merges and dD 0.029).  Bound by
// the latency of a chunk's chain (scores, products, state, with a barrier between) at the
// two waves a SIMD that the states' registers leave: vector issue 52% and matrix cores 34%
// of a SIMD's cycles in the outputs, a third of a wave's cycles waiting for LDS.  fp32: one
// sequence of 8192 tokens, 8 heads of 128 x 64 in 2 groups 0.078 ms, gradients 0.198.
// Figures of variants against each other below are of the first calls of a process, in
// which these kernels take a fifth longer (what HBM bounds does not).
#include <mutex>
#include <type_traits>

#include "kda_ops.hpp"

namespace kda {

namespace {

constexpr int CH = kSsmChunk;
constexpr float kLog2e = 1.44269504088896340736f;

// --------------------------------------------------------------- operands
// column tiles of 16 a wave owns
template <typename T> constexpr int kNC = sizeof(T) == 2 ? 2 : 1;

template <typename T> struct Op;
template <> struct Op<bf16> {
  typedef bf16x8 F;
  static __device__ __forceinline__ f32x4 mma(f32x4 acc, F a, F b) { return mfma_bf16_k32(acc, a, b); }
  static __device__ __forceinline__ F round(f32x4 lo, f32x4 hi) {
    return __builtin_bit_cast(F, u32x4{cvt2(lo[0], lo[1]), cvt2(lo[2], lo[3]), cvt2(hi[0], hi[1]), cvt2(hi[2], hi[3])});
  }
  static __device__ __forceinline__ float at(F f, int i) { return (float)f[i]; }
};
template <> struct Op<float> {
  struct F { float v[8]; };
  static __device__ __forceinline__ f32x4 mma(f32x4 acc, const F& a, const F& b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = mfma_f32_k4(acc, a.v[i], b.v[i]);
    return acc;
  }
  static __device__ __forceinline__ F round(f32x4 lo, f32x4 hi) {
    return F{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
  static __device__ __forceinline__ float at(const F& f, int i) { return f.v[i]; }
};

// The terms of an fp32 operand: NT bf16 values whose sum is x to 8 NT bits
// (fp32: x itself).
template <typename T, int NT>
struct Split {
  typename Op<T>::F t[sizeof(T) == 2 ? NT : 1];
  __device__ __forceinline__ Split(f32x4 lo, f32x4 hi) {
    t[0] = Op<T>::round(lo, hi);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int n = 1; n < NT; ++n) {
        // the remainder of each rounding is exact in fp32
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] -= (float)t[n - 1][e];
          hi[e] -= (float)t[n - 1][4 + e];
        }
        t[n] = Op<T>::round(lo, hi);
      }
    }
  }
  static constexpr int N = sizeof(T) == 2 ? NT : 1;
};

// ------------------------------------------------------------- LDS tiles
// [64 tokens][COLS] of T, 16-byte granules XORed with a function of the row, f: the
// row's low bits, or, in rows of 256 bytes, its low four bits with the two pairs
// exchanged.  The transposing reads take four neighbouring rows of four lanes each,
// which that sends to four different parts of the banks (1.8 ns a wave's read and
// compute unit, 3.4 with the plain bits; rows of 128 bytes: 1.8 plain, 3.4
// exchanged).  Reads take
// a lane's base offset, row_off or col_off, computed afresh for every chunk
// (fresh_lane): a granule's number enters an address by XOR and a row tile by
// addition, so that one register serves every read of a kind, where addresses
// hoisted out of the chunk loop would not leave enough for the tiles in flight.
template <typename T, int COLS>
struct Tile {
  static constexpr int R = COLS * (int)sizeof(T);
  static constexpr int BYTES = CH * R;
  static constexpr int GPR = R / 16;  // granules per row
  static constexpr uint32_t MASK = GPR < 16 ? GPR - 1 : 15;
  static constexpr int GB = 32 * (int)sizeof(T);  // bytes of 32 channels
  static __host__ __device__ __forceinline__ constexpr uint32_t f(uint32_t row) {
    return GPR == 16 ? ((row & 3) << 2) | ((row >> 2) & 3) : row & MASK;
  }
  static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t byte) {
    return row * R + ((((byte >> 4) ^ f(row)) << 4) | (byte & 15u));
  }

  static __device__ __forceinline__ uint32_t row_off(int g, int i) { return i * R + ((((GB / 64) * g) ^ f(i)) << 4); }
  // channels 32m + 8g .. + 7 of row 16 I + i
  static __device__ __forceinline__ typename Op<T>::F row(const char* s, uint32_t off, int I, int m) {
    const char* p = s + I * 16 * R;
    if constexpr (sizeof(T) == 2) return lds_ld<bf16x8>(p, off ^ (m * GB));
    else return Op<T>::round(lds_ld<f32x4>(p, off ^ (m * GB)), lds_ld<f32x4>(p, off ^ (m * GB) ^ 16));
  }
  // Contraction over tokens: lane (g, i) gets tokens 32m + 4g + e and 32m + 16 +
  // 4g + e of channel 32c + 8(i / 4) + 4 odd + i % 4 (col) or i (vcol).  bf16: the transposing read
  // takes lane i's 8 bytes as row i of a 16 x 4 matrix and returns element
  // [4e + i / 4][i % 4] as lane i's e-th.
  static __device__ __forceinline__ uint32_t col_off(int g, int i) {
    if constexpr (sizeof(T) == 2) {
      const int r = 4 * g + (i >> 2);
      return r * R + (((i & 3) ^ f(r)) << 4);
    } else {
      return 4 * g * R + (((2 * (i >> 2)) ^ f(4 * g)) << 4) + 4 * (i & 3);
    }
  }
  static __device__ __forceinline__ typename Op<T>::F col(const char* s, uint32_t off, int m, int c, int odd) {
    const char* p = s + 32 * m * R;
    if constexpr (sizeof(T) == 2) {
      const uint32_t o = (off ^ (c * GB)) + 8 * odd;
      const bf16x4 lo = lds_tr16(p, o), hi = lds_tr16(p + 16 * R, o);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      typename Op<T>::F x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t o = off ^ (c * GB) ^ (odd * 16) ^ (f(e) << 4);
        x.v[e] = lds_ld<float>(p + e * R, o);
        x.v[4 + e] = lds_ld<float>(p + (16 + e) * R, o);
      }
      return x;
    }
  }
  static __device__ __forceinline__ uint32_t vcol_off(int g, int i) {
    if constexpr (sizeof(T) == 2) {
      const int r = 4 * g + (i >> 2);
      return r * R + ((((i & 3) >> 1) ^ f(r)) << 4) + 8 * (i & 1);
    } else {
      return 4 * g * R + (((i >> 2) ^ f(4 * g)) << 4) + 4 * (i & 3);
    }
  }
  static __device__ __forceinline__ typename Op<T>::F vcol(const char* s, uint32_t off, int m) {
    const char* p = s + 32 * m * R;
    if constexpr (sizeof(T) == 2) {
      const bf16x4 lo = lds_tr16(p, off), hi = lds_tr16(p + 16 * R, off);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      typename Op<T>::F x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t o = off ^ (f(e) << 4);
        x.v[e] = lds_ld<float>(p + e * R, o);
        x.v[4 + e] = lds_ld<float>(p + (16 + e) * R, o);
      }
      return x;
    }
  }
  // a lane's place in a result, row 16 I + i: 4 NC channels from 16 NC w + 4 NC g on
  template <int NC>
  static __device__ __forceinline__ void place(const char* s, int I, int i, int w, int g, float (&x)[4 * NC]) {
#pragma unroll
    for (int b = 0; b < NC * (int)sizeof(T) / 4; ++b) {  // 16 bytes (or one 8-byte read)
      if constexpr (sizeof(T) == 2) {
        if constexpr (NC == 2) {
          const bf16x8 v = lds_ld<bf16x8>(s, at(16 * I + i, (32 * w + 8 * g) * 2));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
        }
      } else {
        const f32x4 v = lds_ld<f32x4>(s, at(16 * I + i, (16 * NC * w + 4 * NC * g + 4 * b) * 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * b + e] = v[e];
      }
    }
  }
  // V's column tile of a wave as an operand, half m of the tokens, tile p of NC
  template <int NC>
  static __device__ __forceinline__ uint32_t vtile_off(int g, int i, int w) {
    return NC == 2 ? col_off(g, i) ^ (w * GB) : vcol_off(g, i) ^ (w * (GB / 2));
  }
  template <int NC>
  static __device__ __forceinline__ typename Op<T>::F vtile(const char* s, uint32_t off, int m, int p) {
    return NC == 2 ? col(s, off, m, 0, p) : vcol(s, off, m);
  }
};

// A tile on its way from HBM: NT threads hold 16-byte granules of it.
template <typename T, int COLS, int NT>
struct Fetch {
  typedef Tile<T, COLS> L;
  static constexpr int STEP = NT / L::GPR;  // rows between a thread's granules
  static constexpr int N = CH / STEP;
  static_assert(STEP >= 1 && (STEP & (STEP - 1)) == 0 && STEP * L::GPR == NT, "whole rows");
  u32x4 r[N];
  // Byte offset of the thread's first granule from the chunk's base: a uniform base
  // and a 32-bit offset are all that a load needs, so that a full chunk's addresses
  // cost no vector instructions.  Position p is token p, or CH - 1 - p reversed.
  template <bool REV>
  static __device__ __forceinline__ uint32_t lane_off(long long st, int tid) {
    const int row = tid / L::GPR, c = tid % L::GPR;
    return ((uint32_t)(REV ? CH - 1 - row : row) * (uint32_t)st) * (uint32_t)sizeof(T) + 16u * c;
  }
  // position p of the chunk is token tok0 + p, or tok0 + n - 1 - p reversed; rows past n are zero
  template <bool REV>
  __device__ __forceinline__ void get(const T* p, long long st, int tok0, int n, uint32_t off, int tid) {
    off = fresh_lane(off);  // (or its sum with the tensor's address would be kept, in two registers)
    const char* b = reinterpret_cast<const char*>(p + (long long)(REV ? tok0 + n - CH : tok0) * st);
    const long long d = (REV ? -STEP : STEP) * st * (long long)sizeof(T);
    if (n == CH) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = *reinterpret_cast<const u32x4*>(b + i * d + off);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        r[i] = u32x4{0u, 0u, 0u, 0u};
        if (tid / L::GPR + i * STEP < n) r[i] = *reinterpret_cast<const u32x4*>(b + i * d + off);
      }
    }
  }
  // nothing: a fetch that is left out would keep the last tile's registers alive
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void put(char* s, int tid) const {
    tid = fresh_lane(tid);  // (formed again for every chunk rather than kept in a register)
    const int row = tid / L::GPR, c = tid % L::GPR;
    const uint32_t off = L::at(row, 16 * c);
#pragma unroll
    for (int i = 0; i < N; ++i) lds_st<u32x4>(s + i * STEP * L::R, off ^ (L::f(i * STEP) << 4), r[i]);
  }
};

// ---------------------------------------------------------------- decays
// Per head of the chunk, floats.  PB: sums from the block's start; U: u rho; W: w
// kappa; RH: rho (or, in the reversed outputs, beta); IN: rho e^{l_i}; WS: kappa
// e^{l_end - l_j}; ET: E of the four blocks; GM: e^{l_end}; KP: kappa, where it is not
// one; behind them, with fp32, what PB's rounding left.  All but RH, IN, WS and GM are
// read only while the scores are formed.
enum { V_PB = 0, V_U = 64, V_W = 128, V_RH = 192, V_IN = 256, V_WS = 320, V_ET = 384, V_GM = 388, V_KP = 392 };
template <bool KAPPA> constexpr int kVecLow = KAPPA ? V_KP + 64 : V_KP;
template <typename T, bool KAPPA> constexpr int kVecSize = kVecLow<KAPPA> + (sizeof(T) == 4 ? 64 : 0);  // floats of a head's vectors

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// 2^x to fp32's digits: the exponent's own rounding would cost |x| 2^-24 of the result.
__device__ __forceinline__ float ex2(double x) {
  const float hi = (float)x, e = ex2(hi);
  return fmaf(e, (float)(x - hi) * 0.69314718055994530942f, e);
}
using kda::dpp;
constexpr int DPP_ROW_SHL = 0x100;
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  return __builtin_bit_cast(double, u32x2{dppu<CTRL>(w[0]), dppu<CTRL>(w[1])});
}

// The binary logarithm of a decay from log_alpha, held at -180, in the type that decays
// are summed in.  A NaN passes, which a maximum of the two would not let it.
__device__ __forceinline__ float log2_decay(bf16 la) {
  const float x = to_f32(la) * kLog2e;
  return x < -180.f ? -180.f : x;
}
__device__ __forceinline__ double log2_decay(float la) {
  const double x = la * 1.44269504088896340736;
  return x < -180. ? -180. : x;
}

// One wave fills a head's vectors; lane r is position r with gate la.  WS is also
// multiplied by run.  Returns e^{l_end}.
template <typename T, bool KAPPA>
__device__ __forceinline__ float fill_vec(float* v, int r, T la, float kappa, float rho, float rh, float run = 1.f) {
  const auto x = log2_decay(la);
  auto pre = x;
  pre += dpp<DPP_ROW_SHR + 1>(pre);
  pre += dpp<DPP_ROW_SHR + 2>(pre);
  pre += dpp<DPP_ROW_SHR + 4>(pre);
  pre += dpp<DPP_ROW_SHR + 8>(pre);
  auto suf = dpp<DPP_ROW_SHL + 1>(x);
  suf += dpp<DPP_ROW_SHL + 1>(suf);
  suf += dpp<DPP_ROW_SHL + 2>(suf);
  suf += dpp<DPP_ROW_SHL + 4>(suf);
  suf += dpp<DPP_ROW_SHL + 8>(suf);
  const float et = ex2(__shfl(pre, r | 15));
  const float e0 = __shfl(et, 0), e1 = __shfl(et, 16), e2 = __shfl(et, 32), e3 = __shfl(et, 48);
  const int blk = r >> 4;
  const float before = (blk > 0 ? e0 : 1.f) * (blk > 1 ? e1 : 1.f) * (blk > 2 ? e2 : 1.f);
  const float after = (blk < 1 ? e1 : 1.f) * (blk < 2 ? e2 : 1.f) * (blk < 3 ? e3 : 1.f);
  const float u = ex2(pre), w = ex2(suf);
  v[V_PB + r] = (float)pre;
  if (sizeof(T) == 4) v[kVecLow<KAPPA> + r] = (float)(pre - (float)pre);
  v[V_U + r] = u * rho;
  v[V_W + r] = w * kappa;
  if (KAPPA) v[V_KP + r] = kappa;
  v[V_RH + r] = rh;
  v[V_IN + r] = u * before * rho;
  v[V_WS + r] = w * after * kappa * run;
  if ((r & 15) == 0) v[V_ET + blk] = et;
  const float gm = e0 * e1 * e2 * e3;
  if (r == 0) v[V_GM] = gm;
  return gm;
}

// The gate of position p as it is stored: the token's own, or reversed the next
// token's (0 behind the last).  It is converted where it is used: a conversion here
// would wait for the tiles on their way too.
template <typename T, bool REV>
__device__ __forceinline__ T decay_at(const T* la, long long st, int tok0, int n, int Ttot, int p) {
  p = fresh_lane(p);
  const int t = REV ? tok0 + n - p : tok0 + p;
  T x = T(0.f);
  const T* b = la + (long long)(REV ? tok0 + n - CH + 1 : tok0) * st;
  if (p < n && !(REV && t >= Ttot)) x = b[(uint32_t)(REV ? CH - 1 - p : p) * (uint32_t)st];
  return x;
}
template <typename T, bool REV>
__device__ __forceinline__ T weight_at(const T* beta, long long st, int tok0, int n, int p, bool on) {
  p = fresh_lane(p);
  T x = T(0.f);
  const T* b = beta + (long long)(REV ? tok0 + n - CH : tok0) * st;
  if (p < n && on) x = b[(uint32_t)(REV ? CH - 1 - p : p) * (uint32_t)st];
  return x;
}

// ---------------------------------------------------------------- scores
// Transposed score tiles (I, J <= I), bf16 or fp32, lane by lane, as half of an
// operand of the product with V.
template <typename T>
struct Scores {
  static constexpr int LANE = 4 * (int)sizeof(T);  // bytes of a lane in a tile
  static constexpr int TILE = 64 * LANE;
  static constexpr int BYTES = 10 * TILE;
  typedef typename std::conditional<sizeof(T) == 2, bf16x4, f32x4>::type H;
  static __device__ __forceinline__ int tile(int I, int J) { return I * (I + 1) / 2 + J; }
  static __device__ __forceinline__ void put(char* s, int I, int J, int l, f32x4 v) {
    H h;
    if constexpr (sizeof(T) == 2) h = pack4(v);
    else h = v;
    *reinterpret_cast<H*>(s + tile(I, J) * TILE + l * LANE) = h;
  }
  // tiles (I, 2m) and (I, 2m + 1), the latter zero above the diagonal
  static __device__ __forceinline__ typename Op<T>::F get(const char* s, int I, int m, int l) {
    const char* p = s + tile(I, 2 * m) * TILE + l * LANE;
    const H a = *reinterpret_cast<const H*>(p);
    H b = {};
    if (2 * m < I) b = *reinterpret_cast<const H*>(p + TILE);
    if constexpr (sizeof(T) == 2) return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    else return Op<T>::round(a, b);
  }
};

// Sums over the four rows of 16 lanes, of one, two or four values.  The exchanges are
// vector moves (a shuffle goes through the LDS and waits for it), and halves of two
// values share them: of N values a lane ends up with the sum of value rows_value<N>(g),
// the same for N = 1 in every row, for N = 2 in two.
__device__ __forceinline__ float swap_sum16(float x, float y) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float swap_sum32(float x, float y) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
template <int N>
__device__ __forceinline__ float rows_sum(const float (&x)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "values");
  // lanes 0 .. 31: x[0] over rows g and g + 2; lanes 32 .. 63: x[1]
  const float a = swap_sum32(x[0], x[N > 1 ? 1 : 0]);
  // even rows: a over rows g and g + 1; odd rows: the other pair's
  return swap_sum16(a, N == 4 ? swap_sum32(x[N == 4 ? 2 : 0], x[N == 4 ? 3 : 0]) : a);
}
template <int N>
__device__ __forceinline__ int rows_value(int g) { return N == 4 ? (g >> 1) | ((g & 1) << 1) : N == 2 ? g >> 1 : 0; }
// whether lane row g is the first with its value
template <int N>
__device__ __forceinline__ bool rows_first(int g) { return N == 4 || (N == 2 ? (g & 1) == 0 : g == 0); }
// The total x of a lane row (the same in its 16 lanes): sums of the rows before and behind, and of all.
struct RowTotals {
  float before, behind, all;
};
__device__ __forceinline__ RowTotals row_totals(float x, int g) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float even = __uint_as_float(a[0]), odd = __uint_as_float(a[1]), pair = even + odd;
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(pair), __float_as_uint(pair), false, false);
  const float lo = __uint_as_float(b[0]), hi = __uint_as_float(b[1]);
  return RowTotals{(g & 1 ? even : 0.f) + (g > 1 ? lo : 0.f), (g & 1 ? 0.f : odd) + (g > 1 ? 0.f : hi), lo + hi};
}
// sum over a row of 16 lanes, in every lane of it
__device__ __forceinline__ float row16_sum(float x) {
  x += dpp<DPP_QUAD_SWAP1>(x);
  x += dpp<DPP_QUAD_SWAP2>(x);
  x += dpp<0x124>(x);  // rotations by 4 and 8 within the row
  x += dpp<DPP_ROW_ROR8>(x);
  return x;
}

// sums over the lanes of a row of 16 up to this one, and behind it
__device__ __forceinline__ float row16_prefix(float x) {
  x += dpp<DPP_ROW_SHR + 1>(x);
  x += dpp<DPP_ROW_SHR + 2>(x);
  x += dpp<DPP_ROW_SHR + 4>(x);
  x += dpp<DPP_ROW_SHR + 8>(x);
  return x;
}
__device__ __forceinline__ float row16_behind(float x) {
  x = dpp<DPP_ROW_SHL + 1>(x);
  x += dpp<DPP_ROW_SHL + 1>(x);
  x += dpp<DPP_ROW_SHL + 2>(x);
  x += dpp<DPP_ROW_SHL + 4>(x);
  x += dpp<DPP_ROW_SHL + 8>(x);
  return x;
}
// Of a 16 x 16 tile, rows j = 4g + e and column i in a lane: row p becomes its sum over
// rows j <= p, in the columns i > p, and zero in the others.
__device__ __forceinline__ void crossing(float (&x)[4], int g, int i) {
#pragma unroll
  for (int e = 1; e < 4; ++e) x[e] += x[e - 1];
  const float before = row_totals(x[3], g).before;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = i > 4 * g + e ? x[e] + before : 0.f;
}

// tile t of the ten (I, J <= I), diagonal first
__device__ __forceinline__ int tile_i(int t) { return (int)((0x0fe9e4u >> (2 * t)) & 3u); }  // 0 1 2 3 1 2 2 3 3 3
__device__ __forceinline__ int tile_j(int t) { return (int)((0x0910e4u >> (2 * t)) & 3u); }  // 0 1 2 3 0 0 1 0 1 2

// Decayed, weighted scores of a transposed tile: rows j = 16J + 4g + e, column
// i = 16I + r16; on the diagonal and below it.
template <typename T, bool KAPPA>
__device__ __forceinline__ f32x4 weigh_diag(f32x4 acc, const float* v, int I, int g, int r16) {
  f32x4 m;
  const float pi = v[V_PB + 16 * I + r16];
  const f32x4 pj = *reinterpret_cast<const f32x4*>(v + V_PB + 16 * I + 4 * g);
  f32x4 x;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = pi - pj[e];
  if constexpr (sizeof(T) == 4) {
    const float li = v[kVecLow<KAPPA> + 16 * I + r16];
    const f32x4 lj = *reinterpret_cast<const f32x4*>(v + kVecLow<KAPPA> + 16 * I + 4 * g);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += li - lj[e];
  }
  f32x4 kp = {1.f, 1.f, 1.f, 1.f};
  if (KAPPA) kp = *reinterpret_cast<const f32x4*>(v + V_KP + 16 * I + 4 * g);
#pragma unroll
  for (int e = 0; e < 4; ++e) m[e] = 4 * g + e <= r16 ? acc[e] * (KAPPA ? ex2(x[e]) * kp[e] : ex2(x[e])) : 0.f;
  return m;
}
__device__ __forceinline__ f32x4 weigh_below(f32x4 acc, const float* v, int I, int J, int g, int r16) {
  const f32x4 et = *reinterpret_cast<const f32x4*>(v + V_ET);
  const f32x4 wj = *reinterpret_cast<const f32x4*>(v + V_W + 16 * J + 4 * g);
  // the whole blocks between: 1 and 2 of (3, 0), 1 of (2, 0), 2 of (3, 1)
  const float c = v[V_U + 16 * I + r16] * (I - J > 1 && J == 0 ? et[1] : 1.f) * (I - J > 1 && I == 3 ? et[2] : 1.f);
  f32x4 m;
#pragma unroll
  for (int e = 0; e < 4; ++e) m[e] = acc[e] * (c * wj[e]);
  return m;
}

// The ten score tiles dealt to NW waves, tile n of a wave; eight waves: the two left
// over go to waves 4 and 5.  At most four waves take the diagonal's first.
template <int NW> constexpr int kTiles = NW == 8 ? 2 : (10 + NW - 1) / NW;
template <int NW>
__device__ __forceinline__ int wave_tile(int wave, int n) {
  if (NW == 8) return n == 0 ? wave : (wave < 4 ? 10 : wave + 4);
  return wave + n * NW;
}

// -------------------------------------------------------- state and results
// A wave's state: NK = rows / 16 by NC column tiles.
template <int NK, int NC>
struct State {
  f32x4 t[NK][NC];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int a = 0; a < NK; ++a)
#pragma unroll
      for (int p = 0; p < NC; ++p) t[a][p] = zero4();
  }
  // Makes the compiler take the values as new, so that operands formed from them
  // before are formed again rather than kept in registers.
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int a = 0; a < NK; ++a)
#pragma unroll
      for (int p = 0; p < NC; ++p) asm volatile("" : "+v"(t[a][p]));
  }
};
__device__ __forceinline__ int pair_chan(int tile, int r) { return 32 * (tile >> 1) + 8 * (r >> 2) + 4 * (tile & 1) + (r & 3); }
// column of lane i's column tile p, from the wave's first
template <int NC>
__device__ __forceinline__ int col_chan(int p, int i) { return NC == 2 ? pair_chan(p, i) : i; }

// One word (two elements) of the TERMS bf16 terms of w V.
template <int TERMS>
__device__ __forceinline__ void split_word(uint32_t x, float wa, float wb, uint32_t (&t)[TERMS]) {
  float a = __uint_as_float(x << 16) * wa, b = __uint_as_float(x & 0xffff0000u) * wb;
#pragma unroll
  for (int n = 0; n < TERMS; ++n) {
    if (n > 0) {  // (exact)
      a -= __uint_as_float(t[n - 1] << 16);
      b -= __uint_as_float(t[n - 1] & 0xffff0000u);
    }
    t[n] = cvt2(a, b);
  }
}

// S <- gm S + K^T (w V) (without SCALE: S + ..): w the per-token weights, V the wave's
// column tiles (two 32-token halves each).  bf16: 2 TERMS products a step; the
// state's scaling and the second half's terms are dealt over the first half's
// products, whose time on the matrix cores they fit into.
template <typename T, int NK, int NC, int TERMS, bool SCALE, typename KT>
__device__ __forceinline__ void update(State<NK, NC>& S, const char* ktile, const typename Op<T>::F (&vf)[NC][2], const float* ws,
                                       float gm, uint32_t kcol, int g) {
  if constexpr (sizeof(T) == 2) {
    constexpr int AP = 2 / NC, NS = NK / AP, NW = 4 * NC;  // row tiles a step, steps, words a half
    u32x4 t[2][NC][TERMS];                                 // [half][column tile][term]
    auto word = [&](int m, int n) {
      const int p = n % NC, q = n / NC;
      const f32x2 w = *reinterpret_cast<const f32x2*>(ws + 32 * m + 16 * (q >> 1) + 4 * g + 2 * (q & 1));
      uint32_t r[TERMS];
      split_word<TERMS>(__builtin_bit_cast(u32x4, vf[p][m])[q], w[0], w[1], r);
#pragma unroll
      for (int x = 0; x < TERMS; ++x) t[m][p][x][q] = r[x];
    };
#pragma unroll
    for (int n = 0; n < NW; ++n) word(0, n);
    bf16x8 kn[AP];
#pragma unroll
    for (int b = 0; b < AP; ++b) kn[b] = KT::col(ktile, kcol, 0, b >> 1, b & 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        bf16x8 kc[AP];
        const int sn = st + 1 < NS ? st + 1 : 0, mn = st + 1 < NS ? m : 1;
#pragma unroll
        for (int b = 0; b < AP; ++b) {
          kc[b] = kn[b];
          const int a = sn * AP + b;
          if (m == 0 || st + 1 < NS) kn[b] = KT::col(ktile, kcol, mn, a >> 1, a & 1);
        }
        if (m == 0) {
          if (SCALE) {
#pragma unroll
            for (int b = 0; b < AP; ++b)
#pragma unroll
              for (int p = 0; p < NC; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) S.t[st * AP + b][p][e] *= gm;
          }
#pragma unroll
          for (int n = st * NW / NS; n < (st + 1) * NW / NS; ++n) word(1, n);
        }
#pragma unroll
        for (int x = TERMS - 1; x >= 0; --x)
#pragma unroll
          for (int b = 0; b < AP; ++b)
#pragma unroll
            for (int p = 0; p < NC; ++p)
              S.t[st * AP + b][p] = mfma_bf16_k32(S.t[st * AP + b][p], kc[b], __builtin_bit_cast(bf16x8, t[m][p][x]));
        __builtin_amdgcn_sched_barrier(0);
      }
  } else {
    if (SCALE) {
#pragma unroll
      for (int a = 0; a < NK; ++a)
#pragma unroll
        for (int p = 0; p < NC; ++p)
#pragma unroll
          for (int e = 0; e < 4; ++e) S.t[a][p][e] *= gm;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(ws + 32 * m + 4 * g);
      const f32x4 w1 = *reinterpret_cast<const f32x4*>(ws + 32 * m + 16 + 4 * g);
      typename Op<T>::F y[NC];
#pragma unroll
      for (int p = 0; p < NC; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[p].v[e] = vf[p][m].v[e] * w0[e];
          y[p].v[4 + e] = vf[p][m].v[4 + e] * w1[e];
        }
#pragma unroll
      for (int a = 0; a < NK; ++a) {
        const typename Op<T>::F k = KT::col(ktile, kcol, m, a >> 1, a & 1);
#pragma unroll
        for (int p = 0; p < NC; ++p) S.t[a][p] = Op<T>::mma(S.t[a][p], k, y[p]);
      }
    }
  }
}

// Y^T[p][I] = S^T Q^T (rows: the wave's columns, columns: tokens) for the NI row
// tiles from I0 on, NT terms of S
template <typename T, int NK, int NC, int NT, int NI, typename QT>
__device__ __forceinline__ void inter(f32x4 (&y)[NC][NI], const State<NK, NC>& S, const char* qtile, uint32_t qrow, int I0) {
#pragma unroll
  for (int p = 0; p < NC; ++p)
#pragma unroll
    for (int I = 0; I < NI; ++I) y[p][I] = zero4();
#pragma unroll
  for (int m = 0; m < NK / 2; ++m) {
    typename Op<T>::F qf[NI];
#pragma unroll
    for (int I = 0; I < NI; ++I) qf[I] = QT::row(qtile, qrow, I0 + I, m);
#pragma unroll
    for (int p = 0; p < NC; ++p) {
      const Split<T, NT> s(S.t[2 * m][p], S.t[2 * m + 1][p]);
#pragma unroll
      for (int n = Split<T, NT>::N - 1; n >= 0; --n)
#pragma unroll
        for (int I = 0; I < NI; ++I) y[p][I] = Op<T>::mma(y[p][I], s.t[n], qf[I]);
    }
    if ((m & 1) || NT > 1 || NC == 1) __builtin_amdgcn_sched_barrier(0);  // (operands of a step or two in registers)
  }
}

// Y^T += V^T M^T
template <typename T, int NC, int I0, int NI>
__device__ __forceinline__ void intra(f32x4 (&y)[NC][NI], const typename Op<T>::F (&vf)[NC][2], const char* scores, int l) {
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int I = 0; I < NI; ++I)
      if (2 * m <= I0 + I) {
        const typename Op<T>::F mf = Scores<T>::get(scores, I0 + I, m, l);
#pragma unroll
        for (int p = 0; p < NC; ++p) y[p][I] = Op<T>::mma(y[p][I], vf[p][m], mf);
      }
}

// N consecutive values
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&x)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int b = 0; b < N; b += 4) *reinterpret_cast<f32x4*>(p + b) = f32x4{x[b], x[b + 1], x[b + 2], x[b + 3]};
  } else if constexpr (N == 8) {
    *reinterpret_cast<u32x4*>(p) = u32x4{cvt2(x[0], x[1]), cvt2(x[2], x[3]), cvt2(x[4], x[5]), cvt2(x[6], x[7])};
  } else {
    *reinterpret_cast<u32x2*>(p) = u32x2{cvt2(x[0], x[1]), cvt2(x[2], x[3])};
  }
}
// The values of a lane in row tile I of a result, in channel order.
template <int NC, int NI>
__device__ __forceinline__ void gather(const f32x4 (&y)[NC][NI], int I, float (&x)[4 * NC]) {
#pragma unroll
  for (int p = 0; p < NC; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * p + e] = y[p][I][e];
}

// sum over channels of A row tile J by B row tile I (both [64][COLS]), the operands
// read before the first product
template <typename T, int COLS>
__device__ __forceinline__ f32x4 score_tile(const char* at, const char* bt, uint32_t off, int I, int J) {
  typedef Tile<T, COLS> L;
  typename Op<T>::F x[COLS / 32], y[COLS / 32];
#pragma unroll
  for (int m = 0; m < COLS / 32; ++m) {
    x[m] = L::row(at, off, J, m);
    y[m] = L::row(bt, off, I, m);
  }
  __builtin_amdgcn_sched_barrier(0);
  f32x4 acc = zero4();
#pragma unroll
  for (int m = 0; m < COLS / 32; ++m) acc = Op<T>::mma(acc, x[m], y[m]);
  return acc;
}
// acc[n] = the same for a
// wave's tiles; the operands of PRE tiles are read before the first product, so that
// one LDS latency is exposed and not one each (fp32: its products are long, none).
template <typename T, int COLS, int NW, int PRE>
__device__ __forceinline__ void score_tiles(f32x4 (&acc)[kTiles<NW>], const char* at, const char* bt, uint32_t off, int wave) {
  typedef Tile<T, COLS> L;
  constexpr int N = kTiles<NW>, ST = PRE > 0 ? PRE : 1;
#pragma unroll
  for (int n0 = 0; n0 < N; n0 += ST) {
    if constexpr (PRE == 0) {
      const int t = wave_tile<NW>(wave, n0);
      if (t >= 10) continue;
      acc[n0] = zero4();
#pragma unroll
      for (int m = 0; m < COLS / 32; ++m) acc[n0] = Op<T>::mma(acc[n0], L::row(at, off, tile_j(t), m), L::row(bt, off, tile_i(t), m));
      continue;
    }
    typename Op<T>::F x[ST][COLS / 32], y[ST][COLS / 32];
#pragma unroll
    for (int k = 0; k < ST; ++k) {
      const int t = wave_tile<NW>(wave, n0 + k);
      if (n0 + k >= N || t >= 10) continue;
#pragma unroll
      for (int m = 0; m < COLS / 32; ++m) {
        x[k][m] = L::row(at, off, tile_j(t), m);
        y[k][m] = L::row(bt, off, tile_i(t), m);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < ST; ++k) {
      const int t = wave_tile<NW>(wave, n0 + k);
      if (n0 + k >= N || t >= 10) continue;
      f32x4 s = zero4();
#pragma unroll
      for (int m = 0; m < COLS / 32; ++m) s = Op<T>::mma(s, x[k][m], y[k][m]);
      acc[n0 + k] = s;
    }
  }
}
// f(n, I, J, diagonal) for each of a wave's tiles, the last argument an
// integral_constant where it is known
template <int NW, typename F>
__device__ __forceinline__ void each_tile(int wave, F f) {
  auto one = [&](auto n) {
    const int t = wave_tile<NW>(wave, n.value);
    if (t >= 10) return;
    if constexpr (NW == 8) {
      if (n.value == 0 && wave < 4) f(n.value, t, t, std::true_type());
      else f(n.value, tile_i(t), tile_j(t), std::false_type());
    } else if constexpr (n.value * NW < 4) {
      f(n.value, t, t, std::true_type());
    } else {
      f(n.value, tile_i(t), tile_j(t), std::false_type());
    }
  };
  one(std::integral_constant<int, 0>());
  one(std::integral_constant<int, 1>());
  if constexpr (kTiles<NW> > 2) one(std::integral_constant<int, 2>());
  if constexpr (kTiles<NW> > 3) {
    one(std::integral_constant<int, 3>());
    one(std::integral_constant<int, 4>());
  }
}

// A wave's row tiles I0 .. of results, row 16 I + i at p + I * d + off, rows below n.
template <typename T, int NC, int NI>
__device__ __forceinline__ void store_rows(const f32x4 (&y)[NC][NI], char* p, long long d, uint32_t off, int n, int i, int I0) {
#pragma unroll
  for (int I = 0; I < NI; ++I) {
    float x[4 * NC];
    gather(y, I, x);
    if (16 * (I0 + I) + i < n) store_n<T>(reinterpret_cast<T*>(p + (I0 + I) * d + off), x);
  }
}

__device__ __forceinline__ int clamp_len(const int* lens, int b, int T) {
  if (!lens) return T;
  const int n = lens[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// Work items: `sub` of np workgroups that share one (b, group, segment), which are
// placed on one XCD (workgroups go to the eight in turn) so that the tiles they
// share come from its L2.
struct Item {
  int b, g, seg, sub;
  bool valid;
};
__device__ __forceinline__ Item item_of(int block, int B, int G, int nseg, int np) {
  const int x = block & 7, y = block >> 3;
  const int grp = (y / np) * 8 + x;
  Item it;
  it.sub = y % np;
  it.valid = grp < B * G * nseg;
  it.seg = grp % nseg;
  const int bg = grp / nseg;
  it.g = bg % G;
  it.b = bg / G;
  return it;
}
unsigned item_grid(long long B, long long G, long long nseg, long long np) { return (unsigned)((B * G * nseg + 7) / 8 * 8 * np); }

// What a pass over [B, G] groups of 64-column units reads.
struct PassArgs {
  const void* Q;     // contracted rows, [B, G, T, DK]
  const void* K;
  const void* V;     // [B, H, T, dv]
  const void* V2;    // reversed outputs: v
  const void* la;
  const void* beta;
  const void* D;
  const int* lens;
  Str3 qs, ks, vs, v2s, ls, bs, os;
  void* o;
  const float* start;  // start state of order o at start + o * B * H * dk * dv, or null (zero)
  float* end;          // end state of the last order [B, H, dk, dv], or null
  float* dec;          // state pass: e^{sum of decays} of order o at dec + o * B * H
  float* c;            // reversed outputs: [B, H * dv / 64, T] each
  float* x;
  float* d;
  float* xe;           // [B, H * dv / 64, chunks]
  int B, H, G, T, dk, dv, nseg, seg_chunks;
  int norders;  // state pass: orders walked (the last ones' end states may not be needed)
};

// The state's rows and columns of a lane in global memory, [dk][dv] row-major.
template <int NK, int NC>
__device__ __forceinline__ void load_state(State<NK, NC>& S, const float* p, int ld, int col0, int g, int i) {
#pragma unroll
  for (int a = 0; a < NK; ++a)
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) S.t[a][c][e] = p[(size_t)pair_chan(a, 4 * g + e) * ld + col0 + col_chan<NC>(c, i)];
}
template <int NK, int NC>
__device__ __forceinline__ void store_state(const State<NK, NC>& S, float* p, int ld, int col0, int g, int i, float s) {
#pragma unroll
  for (int a = 0; a < NK; ++a)
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) p[(size_t)pair_chan(a, 4 * g + e) * ld + col0 + col_chan<NC>(c, i)] = s * S.t[a][c][e];
}

// ------------------------------------------------------------- state pass
// End state of every segment from zero.  Workgroup = two 64-column units of one
// group, wave = 16 NC columns of one.  The weight of a token is the decay from it to
// the segment's end, so the chunks are walked from that end on and the state needs no
// scaling; once the decay to the end is exactly zero for a unit, every token before
// adds exactly zero (for finite inputs): its waves only keep step with the other
// unit's, and the walk stops when both have come to zero.  The slowest decays set the
// kernel's end: 198 us for 64K tokens, 64 heads (239 in a process's first calls).
// Two buffers for the tiles took longer (268 us against 253, 64K tokens, 64 heads).
template <typename T, int DK> constexpr int kStateLds = Tile<T, DK>::BYTES + 2 * Tile<T, 64>::BYTES + 4 * kVecSize<T, false> * 4;
template <typename T, int DK, bool REV>
__device__ __forceinline__ void state_pass(const PassArgs& a, int block, char* smem) {
  typedef Tile<T, DK> KT;
  typedef Tile<T, 64> VT;
  constexpr int NC = kNC<T>, NWV = 8 / NC, NT = 64 * NWV, VS = kVecSize<T, false>;
  char* const sk = smem;
  char* const sv = smem + KT::BYTES;
  float* const vecs = reinterpret_cast<float*>(sv + 2 * VT::BYTES);  // two buffers, two units
  const int cpu = a.dv / 64, nu = a.H / a.G * cpu;  // column units per head, units per group
  const Item it = item_of(block, a.B, a.G, a.norders, (nu + 1) / 2);
  if (!it.valid) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int len = clamp_len(a.lens, it.b, a.T);
  const int nch = (len + CH - 1) / CH;
  const int seg = REV ? a.nseg - 1 - it.seg : it.seg;
  const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, nch);
  const int uw = wave / (NWV / 2), part = wave % (NWV / 2);
  const T* K = static_cast<const T*>(a.K) + it.b * a.ks.b + it.g * a.ks.h;
  int head[2];
  const T* V[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int un = min(2 * it.sub + u, nu - 1);
    head[u] = it.g * (a.H / a.G) + un / cpu;
    V[u] = static_cast<const T*>(a.V) + it.b * a.vs.b + head[u] * a.vs.h + (un % cpu) * 64;
  }
  const int fu = wave - (NWV - 2);  // the last two waves fill the units' decay vectors
  const bool filler = fu >= 0;
  const int hv = fu == 1 ? head[1] : head[0];
  const T* la = static_cast<const T*>(a.la) + it.b * a.ls.b + hv * a.ls.h;
  const T* beta = static_cast<const T*>(a.beta) + it.b * a.bs.b + hv * a.bs.h;
  State<DK / 16, NC> S;
  S.zero();
  float dec[2] = {1.f, 1.f};  // decays of the chunks walked
  Fetch<T, DK, NT> fk;
  Fetch<T, 64, NT> fv[2];
  const uint32_t ofk = fk.template lane_off<REV>(a.ks.t, tid), ofv = fv[0].template lane_off<REV>(a.vs.t, tid);
  T fx = T(0.f), fb = T(0.f);
  float run = 1.f;  // filler: decay from the chunk's end to the segment's
  auto chunk = [&](int step) { return REV ? c0 + step : c1 - 1 - step; };  // the order's last chunk first
  auto fetch = [&](int step) {
    const int tok0 = chunk(step) * CH, n = min(CH, len - tok0);
    fk.template get<REV>(K, a.ks.t, tok0, n, ofk, tid);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (dec[u] != 0.f) fv[u].template get<REV>(V[u], a.vs.t, tok0, n, ofv, tid);
  };
  auto fetch_gates = [&](int step) {
    if (!filler || step >= c1 - c0) return;
    const int tok0 = chunk(step) * CH, n = min(CH, len - tok0);
    fx = decay_at<T, REV>(la, a.ls.t, tok0, n, a.T, l);
    fb = weight_at<T, false>(beta, a.bs.t, tok0, n, l, !REV);
  };
  auto fill = [&](int step) {
    if (!filler || step >= c1 - c0) return;
    float* v = vecs + ((step & 1) * 2 + fu) * VS;
    run *= fill_vec<T, false>(v, l, fx, REV ? 1.f : to_f32(fb), 1.f, 1.f, run);
    if (l == 0) v[V_GM] = run;
  };
  fetch_gates(0);
  if (c0 < c1) fetch(0);
  fill(0);
  fetch_gates(1);
  for (int step = 0; step < c1 - c0; ++step) {
    const float* const vec = vecs + (step & 1) * 2 * VS;
    fk.put(sk, tid);
#pragma unroll
    for (int u = 0; u < 2; ++u) fv[u].put(sv + u * VT::BYTES, tid);
    if (step + 1 < c1 - c0) fetch(step + 1);
    sync_lds();
    fill(step + 1);
    fetch_gates(step + 2);
    const int ln = fresh_lane(l), g = ln >> 4, i = ln & 15;
    const uint32_t vcol = VT::template vtile_off<NC>(g, i, part);
    if ((uw ? dec[1] : dec[0]) != 0.f) {
      typename Op<T>::F vf[NC][2];
#pragma unroll
      for (int p = 0; p < NC; ++p)
#pragma unroll
        for (int m = 0; m < 2; ++m) vf[p][m] = VT::template vtile<NC>(sv + uw * VT::BYTES, vcol, m, p);
      update<T, DK / 16, NC, 3, false, KT>(S, sk, vf, vec + uw * VS + V_WS, 1.f, KT::col_off(g, i), g);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      dec[u] = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(vec[u * VS + V_GM])));
    if (dec[0] == 0.f && dec[1] == 0.f) break;
    sync_lds();
  }
  const int un = 2 * it.sub + uw;
  if (un >= nu) return;
  const size_t bh = (size_t)it.b * a.H + (uw ? head[1] : head[0]);
  // order o's end state lies in slot o + 1
  float* out = a.end + ((size_t)(it.seg + 1) * a.B * a.H + bh) * a.dk * a.dv;
  store_state(S, out, a.dv, (un % cpu) * 64 + part * 16 * NC, l >> 4, l & 15, 1.f);
  if (part == 0 && un % cpu == 0 && l == 0) a.dec[(size_t)it.seg * a.B * a.H + bh] = uw ? dec[1] : dec[0];
}

template <typename T, int DK>
__global__ __launch_bounds__(512 / kNC<T>, 4 / kNC<T>) void kda_ssm_state_kernel(PassArgs a) {
  __shared__ __attribute__((aligned(16))) char smem[kStateLds<T, DK>];
  state_pass<T, DK, false>(a, blockIdx.x, smem);
}

// Both directions of the gradients: blocks from nf on walk the reversed orders.  One
// launch, so that the second direction starts where the first one's blocks end.
template <typename T, int DK>
__global__ __launch_bounds__(512 / kNC<T>, 4 / kNC<T>) void kda_ssm_states_kernel(PassArgs f, PassArgs r, int nf) {
  __shared__ __attribute__((aligned(16))) char smem[kStateLds<T, DK>];
  if ((int)blockIdx.x < nf) state_pass<T, DK, false>(f, blockIdx.x, smem);
  else state_pass<T, DK, true>(r, blockIdx.x - nf, smem);
}

// slots[0] = start; slots[o + 1] = dec[o] slots[o] + slots[o + 1], o = 0 .. n - 1.  The
// last one also goes to out (which may be start), with la times the decay of token 0.
struct MergeArgs {
  const float* start;
  float* slots;
  const float* dec;
  int n;
  float* out;
  const void* la;
  Str3 ls;
};
template <typename T>
__device__ __forceinline__ void merge_at(const MergeArgs& a, long long f, long long BH, int elems, int H) {
  if (f >= BH * elems) return;
  const long long bh = f / elems;
  f32x4 s = a.start ? *reinterpret_cast<const f32x4*>(a.start + f) : zero4();
  *reinterpret_cast<f32x4*>(a.slots + f) = s;
  for (int o = 0; o < a.n; ++o) {
    float* p = a.slots + (o + 1) * BH * elems + f;
    const f32x4 z = *reinterpret_cast<const f32x4*>(p);
    const float d = a.dec[o * BH + bh];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = d * s[e] + z[e];
    *reinterpret_cast<f32x4*>(p) = s;
  }
  if (!a.out) return;
  if (a.la) {
    const float d = ex2(log2_decay(static_cast<const T*>(a.la)[(bh / H) * a.ls.b + (bh % H) * a.ls.h]));
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] *= d;
  }
  *reinterpret_cast<f32x4*>(a.out + f) = s;
}
// (blocks from nf on: the other direction)
template <typename T>
__global__ __launch_bounds__(256) void kda_ssm_merge_kernel(MergeArgs x, MergeArgs y, int nf, long long BH, int elems, int H) {
  const bool first = (int)blockIdx.x < nf;
  const long long f = ((long long)(first ? blockIdx.x : blockIdx.x - nf) * 256 + threadIdx.x) * 4;
  if (first) merge_at<T>(x, f, BH, elems, H);
  else merge_at<T>(y, f, BH, elems, H);
}

__global__ __launch_bounds__(256) void kda_ssm_copy_kernel(const float* src, float* dst, long long n4) {
  const long long f = (long long)blockIdx.x * 256 + threadIdx.x;
  if (f < n4) reinterpret_cast<f32x4*>(dst)[f] = src ? reinterpret_cast<const f32x4*>(src)[f] : zero4();
}

// ----------------------------------------------------------------- outputs
// Workgroup = two 64-column units of one group over a segment's chunks, wave = 16 NC
// columns of one unit.  Per chunk: the scores are formed once (Q.K once for both
// units) and left in LDS; every wave then forms its columns of Y and moves its
// state on.  The next chunk's tiles are loaded to registers meanwhile.
// TERMS: of the state's updates; three where the state is written at the end.
// BWD: the reversed pass, which also leaves, per unit and token, what the
// gradients of beta, log_alpha and D need, with P_ij = (dO_i.v_j) (q_i.k_j) e^{l_i - l_j}
// inside the chunk and s_j the same with the state, for the tokens behind the chunk:
//   c[j] = sum_i P_ij + s_j,   d[i] = dO_i.v_i,
//   x[t] = sum_{i >= t > j} beta_j P_ij + sum_{j < t} beta_j s_j,   xe = sum_j beta_j s_j.
// x are the pairs that t's decay lies between.
template <typename T, int DK, bool BWD, int TERMS>
__global__ __launch_bounds__(512 / kNC<T>, 2) void kda_ssm_out_kernel(PassArgs a) {
  typedef Tile<T, DK> KT;
  typedef Tile<T, 64> VT;
  typedef Scores<T> SC;
  constexpr int NC = kNC<T>, NWV = 8 / NC, NT = 64 * NWV, NPU = NWV / 2;  // waves, threads, waves per unit
  constexpr bool KAPPA = !BWD;
  constexpr int VS = kVecSize<T, KAPPA>;
  constexpr int OV = 2 * KT::BYTES, OV2 = OV + 2 * VT::BYTES, OM = OV2 + (BWD ? 2 * VT::BYTES : 0);
  // two buffers of decay vectors, the next chunk's filled beside this one's products
  // (one where two would leave a compute unit with one workgroup)
  constexpr int NB = sizeof(T) == 2 && BWD && DK == 128 ? 1 : 2;
  constexpr int OVEC = OM + 2 * SC::BYTES, ORED = OVEC + NB * 2 * VS * 4;
  constexpr int RED = 160 + 160;  // column and row sums of the ten tiles
  __shared__ __attribute__((aligned(16))) char smem[ORED + (BWD ? 2 * RED * 4 : 0)];
  char* const sq = smem;
  char* const sk = smem + KT::BYTES;
  char* const sv = smem + OV;
  char* const sv2 = smem + OV2;
  char* const sm = smem + OM;
  float* const vecs = reinterpret_cast<float*>(smem + OVEC);
  float* const red = reinterpret_cast<float*>(smem + ORED);
  const int cpu = a.dv / 64, nu = a.H / a.G * cpu;
  const Item it = item_of(blockIdx.x, a.B, a.G, a.nseg, (nu + 1) / 2);
  if (!it.valid) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int len = clamp_len(a.lens, it.b, a.T);
  const int nch = (len + CH - 1) / CH;
  const int seg = BWD ? a.nseg - 1 - it.seg : it.seg;
  const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, nch);
  const int uw = wave / NPU, part = wave % NPU;
  const T* Q = static_cast<const T*>(a.Q) + it.b * a.qs.b + it.g * a.qs.h;
  const T* K = static_cast<const T*>(a.K) + it.b * a.ks.b + it.g * a.ks.h;
  int head[2], colu[2];
  const T *V[2], *V2[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int un = min(2 * it.sub + u, nu - 1);
    head[u] = it.g * (a.H / a.G) + un / cpu;
    colu[u] = (un % cpu) * 64;
    V[u] = static_cast<const T*>(a.V) + it.b * a.vs.b + head[u] * a.vs.h + colu[u];
    V2[u] = BWD ? static_cast<const T*>(a.V2) + it.b * a.v2s.b + head[u] * a.v2s.h + colu[u] : nullptr;
  }
  const bool mine = 2 * it.sub + uw < nu;
  const int hw = uw ? head[1] : head[0], cw = (uw ? colu[1] : colu[0]) + part * 16 * NC;  // the wave's head and column
  const int fu = wave - (NWV - 2);  // the last two waves fill the units' decay vectors
  const bool filler = fu >= 0;
  const int hv = fu == 1 ? head[1] : head[0];
  const T* la = static_cast<const T*>(a.la) + it.b * a.ls.b + hv * a.ls.h;
  const T* beta = static_cast<const T*>(a.beta) + it.b * a.bs.b + hv * a.bs.h;
  float skip[2] = {0.f, 0.f};
  if (a.D) {
#pragma unroll
    for (int u = 0; u < 2; ++u) skip[u] = to_f32(static_cast<const T*>(a.D)[head[u]]);
  }
  const float skip_w = uw ? skip[1] : skip[0];
  T* o = static_cast<T*>(a.o) + it.b * a.os.b + hw * a.os.h + cw;
  const size_t bh = (size_t)it.b * a.H + hw;
  State<DK / 16, NC> S;
  if (a.start) load_state(S, a.start + ((size_t)it.seg * a.B * a.H + bh) * a.dk * a.dv, a.dv, cw, l >> 4, l & 15);
  else S.zero();

  Fetch<T, DK, NT> fq, fk;
  Fetch<T, 64, NT> fv[2], fw[2];
  const uint32_t ofq = fq.template lane_off<BWD>(a.qs.t, tid), ofk = fk.template lane_off<BWD>(a.ks.t, tid);
  const uint32_t ofv = fv[0].template lane_off<BWD>(a.vs.t, tid), ofw = BWD ? fw[0].template lane_off<BWD>(a.v2s.t, tid) : 0u;
  T fx = T(0.f), fb = T(0.f);
  // the next chunk's loads, in three parts between this one's products: together they
  // held the issuing wave up for a sixth of the chunk's cycles (64K tokens: 501 us, in
  // parts 480)
  auto fetch_q = [&](int step) {
    if (step >= c1 - c0) {
      fq.none();
      return;
    }
    const int c = BWD ? c1 - 1 - step : c0 + step;
    fq.template get<BWD>(Q, a.qs.t, c * CH, min(CH, len - c * CH), ofq, tid);
  };
  auto fetch_k = [&](int step) {
    if (step >= c1 - c0) {
      fk.none();
      return;
    }
    const int c = BWD ? c1 - 1 - step : c0 + step;
    fk.template get<BWD>(K, a.ks.t, c * CH, min(CH, len - c * CH), ofk, tid);
  };
  auto fetch_v = [&](int step) {
    if (step >= c1 - c0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        fv[u].none();
        if constexpr (BWD) fw[u].none();
      }
      return;
    }
    const int c = BWD ? c1 - 1 - step : c0 + step;
    const int tok0 = c * CH, n = min(CH, len - tok0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      fv[u].template get<BWD>(V[u], a.vs.t, tok0, n, ofv, tid);
      if constexpr (BWD) fw[u].template get<BWD>(V2[u], a.v2s.t, tok0, n, ofw, tid);
    }
  };
  // decays and weights of a chunk, lane = position
  auto fetch_gates = [&](int step) {
    if (!filler || step >= c1 - c0) return;
    const int c = BWD ? c1 - 1 - step : c0 + step;
    const int tok0 = c * CH, n = min(CH, len - tok0);
    fx = decay_at<T, BWD>(la, a.ls.t, tok0, n, a.T, l);
    fb = weight_at<T, BWD>(beta, a.bs.t, tok0, n, l, true);
  };
  auto fill = [&](int step) {
    if (filler && step < c1 - c0)
      fill_vec<T, KAPPA>(vecs + ((step % NB) * 2 + fu) * VS, l, fx, BWD ? 1.f : to_f32(fb), 1.f, to_f32(fb));
  };
  fetch_gates(0);
  fetch_q(0);
  fetch_k(0);
  fetch_v(0);
  if (NB == 2) {
    fill(0);
    fetch_gates(1);
  }
  for (int step = 0; step < c1 - c0; ++step) {
    const int c = BWD ? c1 - 1 - step : c0 + step;
    const int tok0 = c * CH, n = min(CH, len - tok0);
    float* const vec = vecs + (step % NB) * 2 * VS;
    fq.put(sq, tid);
    fk.put(sk, tid);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      fv[u].put(sv + u * VT::BYTES, tid);
      if constexpr (BWD) fw[u].put(sv2 + u * VT::BYTES, tid);
    }
    if (NB == 1) {
      fill(step);
      fetch_gates(step + 1);
    }
    fetch_q(step + 1);
    sync_lds();

    const int ln = fresh_lane(l), g = ln >> 4, i = ln & 15;
    const uint32_t krow = KT::row_off(g, i);
    if constexpr (!BWD) {
      f32x4 acc[kTiles<NWV>];
      score_tiles<T, DK, NWV, sizeof(T) == 2 ? 2 : 0>(acc, sk, sq, krow, wave);
      fetch_k(step + 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float* v = vec + u * VS;
        each_tile<NWV>(wave, [&](int nt, int I, int J, auto diag) {
          f32x4 mm;
          if constexpr (decltype(diag)::value) {
            mm = weigh_diag<T, KAPPA>(acc[nt], v, I, g, i);
            if constexpr (sizeof(T) == 4) {
#pragma unroll
              for (int e = 0; e < 4; ++e) mm[e] += 4 * g + e == i ? skip[u] : 0.f;
            }
          } else {
            mm = weigh_below(acc[nt], v, I, J, g, i);
          }
          SC::put(sm + u * SC::BYTES, I, J, l, mm);
        });
      }
    } else {
      // tile by tile, the operands of its three products read together
#pragma unroll 1
      for (int n = 0; n < kTiles<NWV>; ++n) {
        const int t = wave_tile<NWV>(wave, n);
        if (t >= 10) break;
        const int I = tile_i(t), J = tile_j(t);
        f32x4 acc, dd[2], mm[2];
        if constexpr (sizeof(T) == 2) {
          const uint32_t vrow = VT::row_off(g, i);
          typename Op<T>::F x[DK / 32], z[DK / 32], dx[2][2], dz[2][2];
#pragma unroll
          for (int m = 0; m < DK / 32; ++m) {
            x[m] = KT::row(sk, krow, J, m);
            z[m] = KT::row(sq, krow, I, m);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              dx[u][m] = VT::row(sv + u * VT::BYTES, vrow, J, m);
              dz[u][m] = VT::row(sv2 + u * VT::BYTES, vrow, I, m);
            }
          __builtin_amdgcn_sched_barrier(0);
          acc = zero4();
#pragma unroll
          for (int m = 0; m < DK / 32; ++m) acc = Op<T>::mma(acc, x[m], z[m]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            dd[u] = zero4();
#pragma unroll
            for (int m = 0; m < 2; ++m) dd[u] = Op<T>::mma(dd[u], dx[u][m], dz[u][m]);
          }
        } else {
          acc = score_tile<T, DK>(sk, sq, krow, I, J);
        }
        if (I == J) {
#pragma unroll
          for (int u = 0; u < 2; ++u) mm[u] = weigh_diag<T, KAPPA>(acc, vec + u * VS, I, g, i);
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u) mm[u] = weigh_below(acc, vec + u * VS, I, J, g, i);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (sizeof(T) == 4) dd[u] = score_tile<T, 64>(sv + u * VT::BYTES, sv2 + u * VT::BYTES, VT::row_off(g, i), I, J);
          float* rd = red + u * RED + 16 * SC::tile(I, J);
          const float bi = vec[u * VS + V_RH + 16 * I + i];
          float cs = 0.f, rs[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float pp = mm[u][e] * dd[u][e];
            cs += pp;
            rs[e] = bi * pp;
          }
          const float c1[1] = {cs};
          cs = rows_sum(c1);
          if (g == 0) rd[i] = cs;
          if (I == J) crossing(rs, g, i);
#pragma unroll
          for (int e = 0; e < 4; ++e) rs[e] = row16_sum(rs[e]);
          if (i == 0) *reinterpret_cast<f32x4*>(rd + 160 + 4 * g) = f32x4{rs[0], rs[1], rs[2], rs[3]};
          SC::put(sm + u * SC::BYTES, I, J, l, mm[u]);
        }
      }
      fetch_k(step + 1);
    }
    if (NB == 2) {
      fill(step + 1);
      fetch_gates(step + 2);
    }
    float* const v = vec + uw * VS;
    f32x4 y[NC][4];
    inter<T, DK / 16, NC, BWD ? 2 : 1, 4, KT>(y, S, sq, krow, 0);
#pragma unroll
    for (int I = 0; I < 4; ++I) {
      const float s = v[V_IN + 16 * I + i];
#pragma unroll
      for (int p = 0; p < NC; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[p][I][e] *= s;
    }
    fetch_v(step + 1);
    sync_lds();
    if constexpr (BWD) {
      // the state's part of c, z.v before the chunk's own part joins z, one sum per
      // wave, left in the dead Q tile: its u-th KiB is wave u's to put, which adds unit
      // u's sums before it does
      float zv[4];
#pragma unroll
      for (int I = 0; I < 4; ++I) {
        float x[4 * NC], z[4 * NC];
        VT::template place<NC>(sv2 + uw * VT::BYTES, I, i, part, g, x);
        gather(y, I, z);
        zv[I] = 0.f;
#pragma unroll
        for (int e = 0; e < 4 * NC; ++e) zv[I] += z[e] * x[e];
      }
      reinterpret_cast<float*>(sq + 1024 * uw)[64 * part + 16 * rows_value<4>(g) + i] = rows_sum(zv);
    }
    typename Op<T>::F vf[NC][2];
    const uint32_t vcol = VT::template vtile_off<NC>(g, i, part);
#pragma unroll
    for (int p = 0; p < NC; ++p)
#pragma unroll
      for (int m = 0; m < 2; ++m) vf[p][m] = VT::template vtile<NC>(sv + uw * VT::BYTES, vcol, m, p);
    intra<T, NC, 0, 4>(y, vf, sm + uw * SC::BYTES, l);
    if constexpr (!BWD && sizeof(T) == 2) {
      // D v as products with a diagonal operand of its own: D is exact in bf16, its sum
      // with a score would not be (and D is often just above one, where rounding is
      // coarsest).  fp32 adds it to the scores.
      if (a.D) {
        bf16x4 dg;
#pragma unroll
        for (int e = 0; e < 4; ++e) dg[e] = (bf16)(4 * g + e == i ? skip_w : 0.f);
#pragma unroll
        for (int I = 0; I < 4; ++I)
#pragma unroll
          for (int p = 0; p < NC; ++p) {
            const bf16x8 x = vf[p][I >> 1];
            y[p][I] = mfma_bf16_k16(y[p][I], (I & 1) ? __builtin_shufflevector(x, x, 4, 5, 6, 7) : __builtin_shufflevector(x, x, 0, 1, 2, 3), dg);
          }
      }
    }
    if constexpr (BWD) {
#pragma unroll
      for (int I = 0; I < 4; ++I) {
        const float bi = v[V_RH + 16 * I + i];
        float gy[4 * NC];
        VT::template place<NC>(sv + uw * VT::BYTES, I, i, part, g, gy);
#pragma unroll
        for (int p = 0; p < NC; ++p)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[p][I][e] = bi * y[p][I][e] + skip_w * gy[4 * p + e];
      }
    }
    char* const ob = reinterpret_cast<char*>(o + (long long)(BWD ? tok0 + n - CH : tok0) * a.os.t);
    const long long od = (BWD ? -16 : 16) * a.os.t * (long long)sizeof(T);
    const uint32_t oo = ((uint32_t)(BWD ? CH - 1 - i : i) * (uint32_t)a.os.t + 4u * NC * g) * (uint32_t)sizeof(T);
    store_rows<T>(y, ob, od, oo, mine ? n : 0, i, 0);
    __builtin_amdgcn_sched_barrier(0);
    update<T, DK / 16, NC, TERMS, true, KT>(S, sk, vf, v + V_WS, v[V_GM], KT::col_off(g, i), g);
    if constexpr (BWD) {
      // dO.v of the unit's rows, 64 / NPU rows a wave
      if (a.D) {
        constexpr int RI = 4 / NPU;
        float d[RI];
#pragma unroll
        for (int r = 0; r < RI; ++r) {
          d[r] = 0.f;
#pragma unroll
          for (int w = 0; w < 4 / NC; ++w) {
            float x[4 * NC], gy[4 * NC];
            VT::template place<NC>(sv2 + uw * VT::BYTES, part * RI + r, i, w, g, x);
            VT::template place<NC>(sv + uw * VT::BYTES, part * RI + r, i, w, g, gy);
#pragma unroll
            for (int e = 0; e < 4 * NC; ++e) d[r] += x[e] * gy[e];
          }
        }
        const int p = 16 * (part * RI + rows_value<RI>(g)) + i;
        const float s = rows_sum(d);
        if (rows_first<RI>(g) && p < n && mine)
          a.d[((size_t)it.b * a.H * cpu + (size_t)hw * cpu + (cw >> 6)) * a.T + tok0 + n - 1 - p] = s;
      }
    }
    float bl = 0.f;  // (the vectors may be filled anew behind the barrier)
    if (BWD && wave < 2) bl = vec[wave * VS + V_RH + l];
    sync_lds();
    if constexpr (BWD) {
      // one wave writes a unit's sums (not one of those that fill the vectors meanwhile)
      if (wave < 2 && 2 * it.sub + wave < nu) {
        const float* rd = red + wave * RED + i;
        const float* w = reinterpret_cast<const float*>(sq + 1024 * wave);
        float st = 0.f;
#pragma unroll
        for (int q = 0; q < NPU; ++q) st += w[64 * q + l];
        // lane = position p: of the tiles, p as a key in front of other blocks' queries,
        // p as a query behind other blocks' keys, whole tiles across p's block, and p's own
        float cs = st, key = 0.f, query = 0.f, across = 0.f;
#pragma unroll
        for (int J = 0; J < 3; ++J)
          if (J < g) {
            const float x = rd[16 * SC::tile(g, J)];
            cs += x;
            key += x;
            for (int I = g + 1; I < 4; ++I) across += rd[160 + 16 * SC::tile(I, J)];
          }
        cs += rd[16 * SC::tile(g, g)];
        for (int I = g + 1; I < 4; ++I) query += rd[160 + 16 * SC::tile(I, g)];
        st = l < n ? bl * st : 0.f;  // (a row behind the last token has no key, but may have met an infinite state)
        key = l < n ? bl * key : 0.f;
        const RowTotals ends = row_totals(row16_sum(st), g);
        const float x = rd[160 + 16 * SC::tile(g, g)] + row16_prefix(query) + row16_behind(key + st) + row16_sum(across) + ends.behind;
        const size_t un = (size_t)it.b * a.H * cpu + (size_t)(wave == 1 ? head[1] : head[0]) * cpu + (2 * it.sub + wave) % cpu;
        if (l < n) {
          const size_t at = un * a.T + tok0 + n - 1 - l;
          a.c[at] = cs;
          a.x[at] = x;
        }
        if (l == 0) a.xe[un * ((a.T + CH - 1) / CH) + c] = ends.all;
      }
    }
  }
  if (it.seg == a.nseg - 1 && a.end && mine) {
    // reversed: the state before the first token owes its own decay too
    float s = 1.f;
    if (BWD) s = ex2(log2_decay((static_cast<const T*>(a.la) + it.b * a.ls.b + hw * a.ls.h)[0]));
    store_state(S, a.end + bh * a.dk * a.dv, a.dv, cw, l >> 4, l & 15, s);
  }
}

// ---------------------------------------------------------- summed over heads
// dq (REV = false) and dk (REV): V is the group's shared row (k or q, DK
// columns), Q and K are the heads' rows (dO and v, DV).  Workgroup = HG heads of
// one group, wave = 16 NC of the DK columns for all of them, so that the sum over
// the heads stays in its accumulators; groups with more heads leave one partial
// result per workgroup.  The forward pass also leaves, per head and token,
// rs[i] = q_i . (the state's part of dq_i), what the tokens before the chunk owe i.
struct GroupArgs : PassArgs {
  const void* qin;  // forward: the q rows
  Str3 qrs;
  float* rs;
  float* parts;
};
// LDS (rs: one sum per wave, head and token; four waves' where the score vectors were, four more)
// Heads of a workgroup, and column tiles of a wave.  The states of two heads of 64
// columns fill the registers of waves with two column tiles.  WIDE doubles the heads
// and gives each wave one column tile (twice the waves, the same registers): half the
// partial results, against operands read from LDS for one product instead of two.
// Measured (bf16, 32 heads in 4 groups): four 8192-token sequences, 128 x 64 states, 770
// us for the whole call and 738 wide (the partials' sum 140 -> 79 us, this kernel 354 ->
// 386, since then 360, or 285 after some tens of calls); two of them with 128 x 128 states
// 720 and 671; 64 x 64 602 and 602.
template <typename T, int DV, bool WIDE> constexpr int kGroupHeads = (WIDE ? 256 : 128) / DV;
template <typename T, bool WIDE> constexpr int kGroupNC = WIDE ? 1 : kNC<T>;
template <typename T, int DV, int DK, bool WIDE, bool REV>
constexpr int kGroupLds = Tile<T, DK>::BYTES + kGroupHeads<T, DV, WIDE> * (2 * Tile<T, DV>::BYTES + Scores<T>::BYTES + 2 * kVecSize<T, !REV> * 4) +
                          (!REV && DK / 16 / kGroupNC<T, WIDE> > 4 ? kGroupHeads<T, DV, WIDE> * 256 * 4 : 0);
template <typename T, int DV, int DK, bool WIDE, bool REV>
__device__ __forceinline__ void group_pass(const GroupArgs& a, int block, char* smem) {
  constexpr int NC = kGroupNC<T, WIDE>, HG = kGroupHeads<T, DV, WIDE>, NW = DK / 16 / NC, NT = 64 * NW;
  constexpr int NI = NC == 2 ? 2 : 4;  // row tiles at a time: with two column tiles a half of the tokens
  constexpr bool KAPPA = !REV;
  constexpr int VS = kVecSize<T, KAPPA>;
  typedef Tile<T, DV> QT;
  typedef Tile<T, DK> VT;
  typedef Scores<T> SC;
  constexpr int OQ = VT::BYTES, OK = OQ + HG * QT::BYTES, OM = OK + HG * QT::BYTES;
  constexpr int OVEC = OM + HG * SC::BYTES, ORS = OVEC + 2 * HG * VS * 4;
  static_assert(ORS + (!REV && NW > 4 ? HG * 256 * 4 : 0) == kGroupLds<T, DV, DK, WIDE, REV>, "layout");
  const Str3 qrs = a.qrs;
  float* const parts = a.parts;
  char* const sv = smem;
  char* const sq = smem + OQ;
  char* const sk = smem + OK;
  char* const sm = smem + OM;
  float* const vecs = reinterpret_cast<float*>(smem + OVEC);
  float* const rsx = reinterpret_cast<float*>(smem + ORS);
  const int R = a.H / a.G, np = (R + HG - 1) / HG;
  const Item it = item_of(block, a.B, a.G, a.nseg, np);
  if (!it.valid) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int nch = (a.T + CH - 1) / CH;
  const int seg = REV ? a.nseg - 1 - it.seg : it.seg;
  const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, nch);
  const T* V = static_cast<const T*>(a.V) + it.b * a.vs.b + it.g * a.vs.h;
  const T* W = REV ? nullptr : static_cast<const T*>(a.qin) + it.b * qrs.b + it.g * qrs.h;
  const int nh = min(HG, R - it.sub * HG);  // heads of this workgroup
  int head[HG];
  const T *Q[HG], *K[HG];
  State<DV / 16, NC> S[HG];
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    head[h] = it.g * R + it.sub * HG + min(h, nh - 1);
    Q[h] = static_cast<const T*>(a.Q) + it.b * a.qs.b + head[h] * a.qs.h;
    K[h] = static_cast<const T*>(a.K) + it.b * a.ks.b + head[h] * a.ks.h;
    S[h].zero();
    if (a.start && h < nh) {
      // the transposed state: rows are dv channels
      const float* p = a.start + ((size_t)it.seg * a.B * a.H + (size_t)it.b * a.H + head[h]) * DK * DV;
#pragma unroll
      for (int t = 0; t < DV / 16; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c)
          S[h].t[t][c] = *reinterpret_cast<const f32x4*>(p + (size_t)(16 * NC * wave + col_chan<NC>(c, l & 15)) * DV +
                                                         pair_chan(t, 4 * (l >> 4)));
    }
  }
  // HG waves fill the heads' decay vectors: the last ones, or of eight the first, which
  // are ahead of the others that share their SIMDs
  const int fh = NW == 8 ? wave : wave - (NW - HG);
  const bool filler = fh >= 0 && fh < HG;
  const int hv = it.g * R + it.sub * HG + max(0, min(fh, nh - 1));
  const T* la = static_cast<const T*>(a.la) + it.b * a.ls.b + hv * a.ls.h;
  const T* beta = static_cast<const T*>(a.beta) + it.b * a.bs.b + hv * a.bs.h;

  Fetch<T, DK, NT> fv;
  Fetch<T, DV, NT> fq[HG], fk[HG];
  const uint32_t ofv = fv.template lane_off<REV>(a.vs.t, tid), ofq = fq[0].template lane_off<REV>(a.qs.t, tid),
                 ofk = fk[0].template lane_off<REV>(a.ks.t, tid);
  T fx = T(0.f), fb = T(0.f);
  // (in three parts, as above)
  auto fetch_q = [&](int step) {
    if (step >= c1 - c0) {
#pragma unroll
      for (int h = 0; h < HG; ++h) fq[h].none();
      return;
    }
    const int c = REV ? c1 - 1 - step : c0 + step;
#pragma unroll
    for (int h = 0; h < HG; ++h) fq[h].template get<REV>(Q[h], a.qs.t, c * CH, min(CH, a.T - c * CH), ofq, tid);
  };
  auto fetch_k = [&](int step) {
    if (step >= c1 - c0) {
#pragma unroll
      for (int h = 0; h < HG; ++h) fk[h].none();
      return;
    }
    const int c = REV ? c1 - 1 - step : c0 + step;
#pragma unroll
    for (int h = 0; h < HG; ++h) fk[h].template get<REV>(K[h], a.ks.t, c * CH, min(CH, a.T - c * CH), ofk, tid);
  };
  auto fetch_v = [&](int step) {
    if (step >= c1 - c0) {
      fv.none();
      return;
    }
    const int c = REV ? c1 - 1 - step : c0 + step;
    fv.template get<REV>(V, a.vs.t, c * CH, min(CH, a.T - c * CH), ofv, tid);
  };
  auto fetch_gates = [&](int step) {
    if (!filler || step >= c1 - c0) return;
    const int c = REV ? c1 - 1 - step : c0 + step;
    const int tok0 = c * CH, n = min(CH, a.T - tok0);
    fx = decay_at<T, REV>(la, a.ls.t, tok0, n, a.T, l);
    // a head past the group's last one gets no weight
    fb = weight_at<T, REV>(beta, a.bs.t, tok0, n, l, fh < nh);
  };
  auto fill = [&](int step) {
    if (filler && step < c1 - c0)
      fill_vec<T, KAPPA>(vecs + ((step & 1) * HG + fh) * VS, l, fx, REV ? 1.f : to_f32(fb), REV ? to_f32(fb) : 1.f, to_f32(fb));
  };
  fetch_gates(0);
  fetch_q(0);
  fetch_k(0);
  fetch_v(0);
  fill(0);
  fetch_gates(1);
  for (int step = 0; step < c1 - c0; ++step) {
    const int c = REV ? c1 - 1 - step : c0 + step;
    const int tok0 = c * CH, n = min(CH, a.T - tok0);
    float* const vec = vecs + (step & 1) * HG * VS;
    fv.put(sv, tid);
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      fq[h].put(sq + h * QT::BYTES, tid);
      fk[h].put(sk + h * QT::BYTES, tid);
    }
    // the wave's columns of the q rows, for rs: straight from memory, in the layout of its results
    typedef typename std::conditional<4 * NC * sizeof(T) == 16, u32x4, u32x2>::type XQ;  // a lane's columns
    XQ xq[4];
    const uint32_t oxq = ((uint32_t)(l & 15) * (uint32_t)qrs.t + 4u * NC * (l >> 4)) * (uint32_t)sizeof(T);
    if constexpr (!REV) {
#pragma unroll
      for (int I = 0; I < 4; ++I) {
        const int p = 16 * I + (l & 15);
        xq[I] = XQ{};
        if (p < n) xq[I] = *reinterpret_cast<const XQ*>(reinterpret_cast<const char*>(W + (tok0 + 16 * I) * qrs.t + 16 * NC * wave) + oxq);
      }
    }
    fetch_q(step + 1);
    sync_lds();

    const int ln = fresh_lane(l), g = ln >> 4, i = ln & 15;
    const uint32_t qrow = QT::row_off(g, i);
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      f32x4 acc[kTiles<NW>];
      // (eight waves share ten tiles: with several heads each wave has its turn at two)
      const int turn = NW == 8 ? (wave + 2 * h) & 7 : wave;
      score_tiles<T, DV, NW, sizeof(T) == 2 ? 2 : 0>(acc, sk + h * QT::BYTES, sq + h * QT::BYTES, qrow, turn);
      const float* v = vec + h * VS;
      if (h == 0) fetch_k(step + 1);
      each_tile<NW>(turn, [&](int nt, int I, int J, auto diag) {
        f32x4 mm;
        if constexpr (decltype(diag)::value) {
          mm = weigh_diag<T, KAPPA>(acc[nt], v, I, g, i);
          if constexpr (REV) {
            const float rho = v[V_RH + 16 * I + i];
#pragma unroll
            for (int e = 0; e < 4; ++e) mm[e] *= rho;
          }
        } else {
          mm = weigh_below(acc[nt], v, I, J, g, i);
        }
        SC::put(sm + h * SC::BYTES, I, J, l, mm);
      });
    }
    fill(step + 1);
    fetch_gates(step + 2);
    sync_lds();

    typename Op<T>::F vf[NC][2];
    const uint32_t vcol = VT::template vtile_off<NC>(g, i, wave);
    const long long row0 = REV ? tok0 + n - CH : tok0;  // as in Fetch
    const int ri = REV ? CH - 1 - i : i;
    auto some = [&](auto B) {
      constexpr int I0 = decltype(B)::value;
      f32x4 y[NC][NI];
#pragma unroll
      for (int p = 0; p < NC; ++p)
#pragma unroll
        for (int I = 0; I < NI; ++I) y[p][I] = zero4();
#pragma unroll
      for (int h = 0; h < HG; ++h) {
        float* v = vec + h * VS;
        f32x4 z[NC][NI];
        float dots[NI];
        inter<T, DV / 16, NC, REV ? 1 : 2, NI, QT>(z, S[h], sq + h * QT::BYTES, qrow, I0);
#pragma unroll
        for (int I = 0; I < NI; ++I) {
          const float s = h < nh ? v[V_IN + 16 * (I0 + I) + i] : 0.f;
          if constexpr (!REV) {
            float zz[4 * NC], dot = 0.f;
            gather(z, I, zz);
#pragma unroll
            for (int e = 0; e < 4 * NC; ++e) {
              const uint32_t w = xq[I0 + I][e * (int)sizeof(T) / 4];
              dot += zz[e] * __uint_as_float(sizeof(T) == 4 ? w : (e & 1 ? w & 0xffff0000u : w << 16));
            }
            dots[I] = s * dot;
          }
#pragma unroll
          for (int p = 0; p < NC; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[p][I][e] += s * z[p][I][e];
        }
        if constexpr (!REV) {
          // (the score vectors are no longer needed)
          const float dot = rows_sum(dots);
          if (rows_first<NI>(g)) (wave < 4 ? v + 64 * wave : rsx + 256 * h + 64 * (wave - 4))[16 * (I0 + rows_value<NI>(g)) + i] = dot;
        }
        __builtin_amdgcn_sched_barrier(0);
        if (h == 0 && I0 == 0) {
#pragma unroll
          for (int p = 0; p < NC; ++p)
#pragma unroll
            for (int m = 0; m < 2; ++m) vf[p][m] = VT::template vtile<NC>(sv, vcol, m, p);
        }
        intra<T, NC, I0, NI>(y, vf, sm + h * SC::BYTES, l);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (np == 1) {
        char* const ob = reinterpret_cast<char*>(static_cast<T*>(a.o) + it.b * a.os.b + it.g * a.os.h + row0 * a.os.t + 16 * NC * wave);
        store_rows<T>(y, ob, (REV ? -16 : 16) * a.os.t * (long long)sizeof(T),
                      ((uint32_t)ri * (uint32_t)a.os.t + 4u * NC * g) * (uint32_t)sizeof(T), n, i, I0);
      } else {
        char* const ob = reinterpret_cast<char*>(parts + (((long long)it.sub * a.B * a.G + (long long)it.b * a.G + it.g) * a.T + row0) * DK +
                                                 16 * NC * wave);
        store_rows<float>(y, ob, (REV ? -16 : 16) * DK * 4, (uint32_t)(ri * DK + 4 * NC * g) * 4u, n, i, I0);
      }
    };
    some(std::integral_constant<int, 0>());
    fetch_v(step + 1);
    if constexpr (NI == 2) {
#pragma unroll
      for (int h = 0; h < HG; ++h) S[h].renew();
      some(std::integral_constant<int, 2>());
    }
    // after the stores, when the results' registers are free
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      __builtin_amdgcn_sched_barrier(0);
      const float* v = vec + h * VS;
      update<T, DV / 16, NC, 2, true, QT>(S[h], sk + h * QT::BYTES, vf, v + V_WS, v[V_GM], QT::col_off(g, i), g);
    }
    sync_lds();
    if constexpr (!REV) {
      if (wave < nh && l < n) {
        const float* v = vec + wave * VS;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += w < 4 ? v[64 * w + l] : rsx[256 * wave + 64 * (w - 4) + l];
        a.rs[((size_t)it.b * a.H + it.g * R + it.sub * HG + wave) * a.T + tok0 + l] = s;
      }
    }
  }
}

// dq and dk in one launch: blocks from nf on are dk's.
template <typename T, int DV, int DK, bool WIDE>
__global__ __launch_bounds__((4 * DK / kGroupNC<T, WIDE>), DK == 128 ? 2 : 1) void kda_ssm_group_kernel(GroupArgs q, GroupArgs k, int nf) {
  constexpr int F = kGroupLds<T, DV, DK, WIDE, false>, R = kGroupLds<T, DV, DK, WIDE, true>;
  __shared__ __attribute__((aligned(16))) char smem[F > R ? F : R];
  if ((int)blockIdx.x < nf) group_pass<T, DV, DK, WIDE, false>(q, blockIdx.x, smem);
  else group_pass<T, DV, DK, WIDE, true>(k, blockIdx.x - nf, smem);
}

// out[row] = sum of np partials, rows of dk values
template <typename T>
__device__ __forceinline__ void sum_parts(const float* parts, int np, T* out, Str3 os, int B, int G, int T_, int dk, int block) {
  const long long rows = (long long)B * G * T_;
  const long long f = (long long)block * 256 + threadIdx.x;
  const int vpr = dk / 8;
  const long long row = f / vpr;
  if (row >= rows) return;
  const int c = (int)(f % vpr) * 8;
  float x[8] = {};
  for (int p = 0; p < np; ++p) {
    const float* s = parts + ((size_t)p * rows + row) * dk + c;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(s), hi = *reinterpret_cast<const f32x4*>(s + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] += lo[e];
      x[4 + e] += hi[e];
    }
  }
  const int t = (int)(row % T_);
  const long long bg = row / T_;
  store_n<T>(out + (bg / G) * os.b + (bg % G) * os.h + (long long)t * os.t + c, x);
}

// dlog_alpha and dbeta of one (b, h, segment), and the segment's share of dD.
// dlog_alpha[t] is what lies on both sides of t's decay: the pairs (i >= t > j) in t's
// chunk, the tokens from t on with the chunk's start state, the tokens before t with the
// gradient that enters at its end, and those two with each other, X = e^{l_end} <S, dS>:
//     dlog_alpha[t] = x[t] + sum_{i >= t} rs_i + X.
// Of a segment of one chunk, X is formed from its states.  Else the sum N = sum_i rs_i + X
// at a chunk's first token is also the chunk before's xe + X, so that X = N - xe, from
// <S, dS> at the segment's end on and chunk by chunk to its start.  X is zero where the
// chunk's decay is zero in fp32 or there is no start state.  Where the decay is below 2^-20
// and N - xe no more than the rounding of the two (bf16: states of 16 bits; fp32) it is
// taken as zero too, which is off by that rounding at most and leaves none of it to the
// chunks before.  Otherwise each chunk adds its own: fp32 segments end after 16 (ssm_plan).
// (One sum of q.dq - beta dbeta over the segment's tokens is shorter, but leaves all its
// rounding in every gradient before it: 8e-5 after 2048 tokens with decays of e^-3, and
// anything but zero at resets.)
// slots_f, slots_r: start states of the segments in both directions.
struct GateArgs {
  const float *slots_f, *slots_r, *rs;
  void *dla, *dbeta;
  Str3 dls, dbs;
  float* dDp;
  bool from_zero;  // no start state
};
template <typename T>
__device__ __forceinline__ void gate_gradients(const PassArgs& a, const GateArgs& x_) {
  const float *slots_f = x_.slots_f, *slots_r = x_.slots_r, *rs = x_.rs;
  T *dla = static_cast<T*>(x_.dla), *dbeta = static_cast<T*>(x_.dbeta);
  const Str3 dls = x_.dls, dbs = x_.dbs;
  float* const dDp = x_.dDp;
  __shared__ float sh[12];
  const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63;
  const int seg = blockIdx.x % a.nseg;
  const long long bh = blockIdx.x / a.nseg;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H), cpu = a.dv / 64;
  const int nch = (a.T + CH - 1) / CH, c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, nch);
  const bool one = c1 - c0 == 1;
  const size_t elems = (size_t)a.dk * a.dv, all = (size_t)a.B * a.H * elems;
  const T* la = static_cast<const T*>(a.la) + b * a.ls.b + h * a.ls.h;
  auto block_sum = [&](float s) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    __syncthreads();
    if (l == 0) sh[wave] = s;
    __syncthreads();
    return (sh[0] + sh[1]) + (sh[2] + sh[3]);
  };
  float dot = 0.f;
  {
    const float* p = slots_f + (seg + (one ? 0 : 1)) * all + bh * elems;
    const float* q = slots_r + (a.nseg - 1 - seg) * all + bh * elems;
    for (size_t e = tid * 4; e < elems; e += 1024) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p + e), y = *reinterpret_cast<const f32x4*>(q + e);
      dot += (x[0] * y[0] + x[1] * y[1]) + (x[2] * y[2] + x[3] * y[3]);
    }
  }
  float N = block_sum(dot);
  if (c1 < nch) N *= ex2(log2_decay(la[(long long)c1 * CH * a.ls.t]));
  constexpr float kSmall = sizeof(T) == 2 ? 0x1p-12f : 0x1p-18f;
  float dsum = 0.f;
  // four chunks at a time, one a wave, last ones first; lane order is token order reversed
  for (int ce = c1; ce > c0; ce -= 4) {
    const int c = ce - 1 - wave, n = min(CH, a.T - c * CH), t = c * CH + n - 1 - l;
    float s = 0.f, x = 0.f, xe = 0.f;
    decltype(log2_decay(T())) dec = 0;
    if (c >= c0 && l < n) {
      float db = 0.f;
      s = rs[bh * a.T + t];
      dec = log2_decay(la[(long long)t * a.ls.t]);
      for (int u = 0; u < cpu; ++u) {
        const size_t un = (size_t)bh * cpu + u, at = un * a.T + t;
        db += a.c[at];
        x += a.x[at];
        xe += a.xe[un * nch + c];
        if (dDp) dsum += a.d[at];
      }
      dbeta[b * dbs.b + h * dbs.h + (long long)t * dbs.t] = from_f32<T>(db);
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const float y = __shfl_up(s, off);
      s += l >= off ? y : 0.f;
      dec += __shfl_xor(dec, off);
    }
    __syncthreads();
    if (l == 63) sh[wave] = s;
    if (l == 0) {
      sh[4 + wave] = xe;
      sh[8 + wave] = c == 0 && x_.from_zero ? -180.f : (float)dec;
    }
    __syncthreads();
    float X = one ? N * ex2(dec) : 0.f;
#pragma unroll
    for (int w = 0; w < 4 && !one; ++w) {
      float y = N - sh[4 + w];
      if (sh[8 + w] < -150.f || (sh[8 + w] < -20.f && fabsf(y) <= kSmall * fabsf(N))) y = 0.f;
      if (w == wave) X = y;
      N = sh[w] + y;
    }
    if (c >= c0 && l < n) dla[b * dls.b + h * dls.h + (long long)t * dls.t] = from_f32<T>(x + s + X);
  }
  dsum = block_sum(dsum);
  if (tid == 0 && dDp) dDp[((size_t)b * a.nseg + seg) * a.H + h] = dsum;
}

// What is left when the passes are done, in one launch: the gates' gradients (blocks
// below ng), then the sums of dq's and dk's partials (npart blocks each).
template <typename T>
__global__ __launch_bounds__(256) void kda_ssm_finish_kernel(GroupArgs q, GroupArgs k, GateArgs gate, int ng, int npart, int np) {
  const int b = (int)blockIdx.x - ng;
  if (b < 0) gate_gradients<T>(q, gate);
  else if (b < npart) sum_parts<T>(q.parts, np, static_cast<T*>(q.o), q.os, q.B, q.G, q.T, q.dk, b);
  else sum_parts<T>(k.parts, np, static_cast<T*>(k.o), k.os, k.B, k.G, k.T, k.dk, b - npart);
}

// dD of 64 heads: four waves share the partials.
template <typename T>
__global__ __launch_bounds__(256) void kda_ssm_skip_kernel(const float* dDp, T* dD, int H, int n) {
  __shared__ float sh[4][64];
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, h = blockIdx.x * 64 + l;
  float s = 0.f;
  if (h < H)
    for (int p = wave; p < n; p += 4) s += dDp[(size_t)p * H + h];
  sh[wave][l] = s;
  __syncthreads();
  if (wave == 0 && h < H) dD[h] = from_f32<T>((sh[0][l] + sh[1][l]) + (sh[2][l] + sh[3][l]));
}

// ----------------------------------------------------------------- one token
// S = a S + k (beta v)^T, o = S^T q + D v.  256 sequences of 32 heads, 128 x 128: 198
// us, 5.4 TB/s, the rate of a copy.  Workgroup = one (sequence, head), four
// waves of dv / 4 columns each; lane = 4 columns of consecutive rows.  Bound by
// the state, which is read and written once, past the caches.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(256) void kda_ssm_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                                                           const T* __restrict__ la, const T* __restrict__ beta,
                                                           const T* __restrict__ D, float* S, T* __restrict__ o, int H, int G) {
  constexpr int CPW = DV / 4, LPR = CPW / 4, RG = 64 / LPR, RPL = DK / RG;
  const int nh = blockIdx.x, n = nh / H, h = nh - n * H;
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int c0 = wave * CPW + 4 * (l % LPR), r0 = (l / LPR) * RPL;
  float* s = S + (size_t)nh * DK * DV + (size_t)r0 * DV + c0;
  f32x4 st[RPL];
#pragma unroll
  for (int r = 0; r < RPL; ++r) st[r] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(s + r * DV));
  const size_t row = ((size_t)n * G + h / (H / G)) * DK + r0;
  float kk[RPL], qq[RPL];
#pragma unroll
  for (int r = 0; r < RPL; ++r) {
    kk[r] = to_f32(k[row + r]);
    qq[r] = to_f32(q[row + r]);
  }
  const float al = expf(to_f32(la[nh])), b = to_f32(beta[nh]);
  float vv[4], y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) vv[c] = to_f32(v[(size_t)nh * DV + c0 + c]);
#pragma unroll
  for (int r = 0; r < RPL; ++r) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      st[r][c] = al * st[r][c] + kk[r] * (b * vv[c]);
      y[c] += qq[r] * st[r][c];
    }
    __builtin_nontemporal_store(st[r], reinterpret_cast<f32x4*>(s + r * DV));
  }
#pragma unroll
  for (int off = LPR; off < 64; off <<= 1)
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] += __shfl_xor(y[c], off);
  if (l < LPR) {
    const float d = D ? to_f32(D[h]) : 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[(size_t)nh * DV + c0 + c] = from_f32<T>(y[c] + d * vv[c]);
  }
}

// ------------------------------------------------------------------- check
__device__ unsigned int g_ssm_check_bits;

__global__ void kda_ssm_check_clear_kernel(unsigned int* bits) { *bits = 0u; }

template <typename T>
__global__ __launch_bounds__(256) void kda_ssm_check_kernel(const T* la, Str3 ls, const T* beta, Str3 bs, const int* lens, int H,
                                                            int T_, long long n, unsigned int* bits) {
  unsigned int b = 0u;
  for (long long f = (long long)blockIdx.x * 256 + threadIdx.x; f < n; f += (long long)gridDim.x * 256) {
    const int t = (int)(f % T_);
    const long long bh = f / T_, bb = bh / H, h = bh % H;
    if (t >= clamp_len(lens, (int)bb, T_)) continue;
    if (!(to_f32(la[bb * ls.b + h * ls.h + t * ls.t]) <= 0.f)) b |= 1u;
    if (!(fabsf(to_f32(beta[bb * bs.b + h * bs.h + t * bs.t])) < __builtin_inff())) b |= 2u;
  }
  if (b) atomicOr(bits, b);
}

// ------------------------------------------------------------------ launch
template <typename T>
hipError_t run_state(const PassArgs& a, hipStream_t s) {
  const int nu = a.H / a.G * (a.dv / 64);
  const dim3 grid(item_grid(a.B, a.G, a.norders, (nu + 1) / 2)), block(512 / kNC<T>);
  if (a.dk == 128) hipLaunchKernelGGL((kda_ssm_state_kernel<T, 128>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((kda_ssm_state_kernel<T, 64>), grid, block, 0, s, a);
  return hipGetLastError();
}
template <typename T>
hipError_t run_states(const PassArgs& f, const PassArgs& r, hipStream_t s) {
  const int nu = f.H / f.G * (f.dv / 64);
  const unsigned nf = item_grid(f.B, f.G, f.norders, (nu + 1) / 2), nr = item_grid(r.B, r.G, r.norders, (nu + 1) / 2);
  const dim3 block(512 / kNC<T>);
  if (f.dk == 128) hipLaunchKernelGGL((kda_ssm_states_kernel<T, 128>), dim3(nf + nr), block, 0, s, f, r, (int)nf);
  else hipLaunchKernelGGL((kda_ssm_states_kernel<T, 64>), dim3(nf + nr), block, 0, s, f, r, (int)nf);
  return hipGetLastError();
}

// (fp32 operands are whole: one variant)
template <typename T, bool BWD, int TERMS>
hipError_t run_out_terms(const PassArgs& a, hipStream_t s) {
  const int nu = a.H / a.G * (a.dv / 64);
  const dim3 grid(item_grid(a.B, a.G, a.nseg, (nu + 1) / 2)), block(512 / kNC<T>);
  if (a.dk == 128) hipLaunchKernelGGL((kda_ssm_out_kernel<T, 128, BWD, TERMS>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((kda_ssm_out_kernel<T, 64, BWD, TERMS>), grid, block, 0, s, a);
  return hipGetLastError();
}
template <typename T, bool BWD>
hipError_t run_out(const PassArgs& a, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (!a.end) return run_out_terms<T, BWD, 2>(a, s);
  }
  return run_out_terms<T, BWD, 3>(a, s);
}

bool group_wide(int H, int G, int dv, bool bf16_io) { return bf16_io && H / G > 128 / dv; }
int group_parts(int H, int G, int dv, bool bf16_io) {
  const int hg = (group_wide(H, G, dv, bf16_io) ? 256 : 128) / dv;
  return (H / G + hg - 1) / hg;
}
template <typename T, bool WIDE>
hipError_t run_groups_of(const GroupArgs& q, const GroupArgs& k, hipStream_t s) {
  const unsigned n = item_grid(q.B, q.G, q.nseg, group_parts(q.H, q.G, q.dv, sizeof(T) == 2));
#define KDA_GROUP(DV, DK) \
  hipLaunchKernelGGL((kda_ssm_group_kernel<T, DV, DK, WIDE>), dim3(2 * n), dim3(4 * DK / kGroupNC<T, WIDE>), 0, s, q, k, (int)n)
  if (q.dv == 64 && q.dk == 64) KDA_GROUP(64, 64);
  else if (q.dv == 64) KDA_GROUP(64, 128);
  else if (q.dk == 64) KDA_GROUP(128, 64);
  else KDA_GROUP(128, 128);
#undef KDA_GROUP
  return hipGetLastError();
}
template <typename T>
hipError_t run_groups(const GroupArgs& q, const GroupArgs& k, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (group_wide(q.H, q.G, q.dv, true)) return run_groups_of<T, true>(q, k, s);
  }
  return run_groups_of<T, false>(q, k, s);
}

template <typename T>
hipError_t run_merge(const MergeArgs& x, const MergeArgs* y, const PassArgs& a, hipStream_t s) {
  const long long BH = (long long)a.B * a.H;
  const int elems = a.dk * a.dv;
  const unsigned n = (unsigned)((BH * elems / 4 + 255) / 256);
  hipLaunchKernelGGL((kda_ssm_merge_kernel<T>), dim3(y ? 2 * n : n), dim3(256), 0, s, x, y ? *y : x, (int)n, BH, elems, a.H);
  return hipGetLastError();
}

#define SSM_TRY(expr)                       \
  do {                                      \
    const hipError_t e_ = (expr);           \
    if (e_ != hipSuccess) return e_;        \
  } while (0)

template <typename T>
hipError_t prefill(const SsmArgs& x, hipStream_t s) {
  PassArgs a{};
  a.Q = x.q; a.K = x.k; a.V = x.v; a.la = x.la; a.beta = x.beta; a.D = x.D; a.lens = x.lens; a.o = x.o;
  a.qs = x.qs; a.ks = x.ks; a.vs = x.vs; a.ls = x.ls; a.bs = x.bs; a.os = x.os;
  a.B = x.B; a.H = x.H; a.G = x.G; a.T = x.T; a.dk = x.dk; a.dv = x.dv;
  a.nseg = x.nseg; a.seg_chunks = x.seg_chunks;
  if (x.nseg == 1) {
    a.start = x.S0;
    a.end = x.S_T;
    return run_out<T, false>(a, s);
  }
  // every segment's end state from zero, the states at the cuts and S_T from those,
  // then the outputs, whose own states need not be results
  a.dec = x.ws + (size_t)(x.nseg + 1) * x.B * x.H * x.dk * x.dv;
  a.end = x.ws;
  a.norders = x.nseg;
  SSM_TRY(run_state<T>(a, s));
  SSM_TRY(run_merge<T>(MergeArgs{x.S0, x.ws, a.dec, x.nseg, x.S_T, nullptr, Str3()}, nullptr, a, s));
  a.start = x.ws;
  a.end = nullptr;
  return run_out<T, false>(a, s);
}

struct BwdWs {
  size_t slots_f, slots_r, dec_f, dec_r, c, x, d, xe, rs, dDp, parts_q, parts_k, total;
};
BwdWs backward_ws(int B, int H, int G, int T, int dk, int dv, int nseg, bool bf16_io) {
  BwdWs w;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += (n + 3) / 4 * 4;  // 16-byte aligned
    return p;
  };
  const size_t st = (size_t)B * H * dk * dv, bht = (size_t)B * H * T, cpu = dv / 64;
  w.slots_f = take((nseg + 1) * st);
  w.slots_r = take((nseg + 1) * st);
  w.dec_f = take((size_t)nseg * B * H);
  w.dec_r = take((size_t)nseg * B * H);
  w.c = take(bht * cpu);
  w.x = take(bht * cpu);
  w.d = take(bht * cpu);
  w.xe = take((size_t)B * H * cpu * ((T + CH - 1) / CH));
  w.rs = take(bht);
  w.dDp = take((size_t)nseg * B * H);
  const int np = group_parts(H, G, dv, bf16_io);
  w.parts_q = take(np > 1 ? (size_t)np * B * G * T * dk : 0);
  w.parts_k = take(np > 1 ? (size_t)np * B * G * T * dk : 0);
  w.total = at;
  return w;
}

template <typename T>
hipError_t backward(const SsmArgs& x, hipStream_t s) {
  const BwdWs w = backward_ws(x.B, x.H, x.G, x.T, x.dk, x.dv, x.nseg, sizeof(T) == 2);
  float* const ws = x.ws;
  PassArgs a{};
  a.la = x.la; a.beta = x.beta; a.D = x.D;
  a.ls = x.ls; a.bs = x.bs;
  a.B = x.B; a.H = x.H; a.G = x.G; a.T = x.T; a.dk = x.dk; a.dv = x.dv;
  a.nseg = x.nseg; a.seg_chunks = x.seg_chunks;
  a.c = ws + w.c; a.x = ws + w.x; a.d = ws + w.d; a.xe = ws + w.xe;
  // start states of the segments, forwards (with the end state) and reversed; of one
  // segment dS0 comes from the outputs' pass
  PassArgs f = a, r = a;
  f.K = x.k; f.ks = x.ks; f.V = x.v; f.vs = x.vs;
  f.end = ws + w.slots_f;
  f.dec = ws + w.dec_f;
  f.norders = x.nseg;
  r.K = x.q; r.ks = x.qs; r.V = x.dO; r.vs = x.dos;
  r.end = ws + w.slots_r;
  r.dec = ws + w.dec_r;
  r.norders = x.nseg == 1 ? 0 : x.dS0 ? x.nseg : x.nseg - 1;
  SSM_TRY(run_states<T>(f, r, s));
  const MergeArgs mr{x.dS_T, r.end, r.dec, r.norders, x.nseg > 1 ? x.dS0 : nullptr, x.la, x.ls};
  SSM_TRY(run_merge<T>(MergeArgs{x.S0, f.end, f.dec, x.nseg, nullptr, nullptr, Str3()}, &mr, a, s));
  // dv, dbeta's and dlog_alpha's sums, dS0
  PassArgs v = r;
  v.Q = x.k; v.qs = x.ks;
  v.V2 = x.v; v.v2s = x.vs;
  v.o = x.dvv; v.os = x.dvs;
  v.start = r.end;
  v.end = x.nseg == 1 ? x.dS0 : nullptr;
  SSM_TRY((run_out<T, true>(v, s)));
  // dq and dk
  GroupArgs q{}, k{};
  static_cast<PassArgs&>(q) = a;
  q.Q = x.dO; q.qs = x.dos; q.K = x.v; q.ks = x.vs; q.V = x.k; q.vs = x.ks;
  q.o = x.dq; q.os = x.dqs;
  q.start = f.end;
  q.qin = x.q; q.qrs = x.qs;
  q.rs = ws + w.rs;
  q.parts = ws + w.parts_q;
  static_cast<PassArgs&>(k) = a;
  k.Q = x.v; k.qs = x.vs; k.K = x.dO; k.ks = x.dos; k.V = x.q; k.vs = x.qs;
  k.o = x.dkk; k.os = x.dks;
  k.start = r.end;
  k.parts = ws + w.parts_k;
  SSM_TRY(run_groups<T>(q, k, s));
  const GateArgs gate{f.end, r.end, q.rs, x.dla, x.dbeta, x.dls, x.dbs, x.dD ? ws + w.dDp : nullptr, x.S0 == nullptr};
  const int np = group_parts(x.H, x.G, x.dv, sizeof(T) == 2);
  const long long ng = (long long)x.B * x.H * x.nseg, npart = np > 1 ? ((long long)x.B * x.G * x.T * (x.dk / 8) + 255) / 256 : 0;
  hipLaunchKernelGGL((kda_ssm_finish_kernel<T>), dim3((unsigned)(ng + 2 * npart)), dim3(256), 0, s, q, k, gate, (int)ng, (int)npart, np);
  SSM_TRY(hipGetLastError());
  if (x.dD) {
    hipLaunchKernelGGL((kda_ssm_skip_kernel<T>), dim3((x.H + 63) / 64), dim3(256), 0, s, ws + w.dDp, static_cast<T*>(x.dD), x.H,
                       x.B * x.nseg);
    SSM_TRY(hipGetLastError());
  }
  return hipSuccess;
}

}  // namespace

// Two workgroups a compute unit (one with fp32 tiles) fill the device; where the
// sequences and heads alone give fewer, the sequence is cut.  A chunk walked alone
// takes 3 to 8 us, the two launches that a cut adds about 8, so runs may be one chunk
// long from four chunks on (fp32 three).  Measured against runs of at least four
// chunks: 16 heads, 512 tokens, bf16 37 -> 23 us; 8 heads, 333 tokens, fp32 55 -> 26;
// gradients of 8 heads, 256 tokens, bf16 128 -> 68.  Past 16 bf16 chunks runs of two
// are as good or better (8 heads, 2048 tokens: 30 us, 32 with runs of one).
// The gradients of fp32 inputs cut every sequence after 16 chunks, however many there are:
// the gradient of log_alpha takes <S, dS> at the cuts, and between them its rounding adds up
// chunk by chunk (512 heads, 8192 tokens, decays of 0.999: 4e-6 of a head's norm and 1.1e-5
// over its first tokens, with the cuts 1.2e-6; the call takes 10.9 ms, uncut 9.4, for the
// reversed states at the cuts).  bf16's own rounding hides that.
int ssm_plan(int B, int H, int G, int T, int dk, int dv, bool bf16_io, bool gradients, int cus, int* seg_chunks) {
  const int nch = (T + CH - 1) / CH;
  const long long np = ((long long)H / G * (dv / 64) + 1) / 2, base = (long long)B * G * np;
  const int least = bf16_io && nch > 16 ? 2 : 1;
  long long nseg = base > 0 ? (bf16_io ? 2 : 1) * (long long)cus / base : 1;
  if (nseg > nch / least) nseg = nch / least;
  if (nseg < 1 || nch < (bf16_io ? 4 : 3)) nseg = 1;
  int sc = (int)((nch + nseg - 1) / nseg);
  if (gradients && !bf16_io && sc > 16) sc = 16;
  *seg_chunks = sc > 0 ? sc : 1;
  return nch > 0 ? (nch + *seg_chunks - 1) / *seg_chunks : 1;
}

size_t ssm_ws_floats(int B, int H, int dk, int dv, int nseg) {
  if (nseg <= 1) return 0;
  return (size_t)(nseg + 1) * B * H * dk * dv + ((size_t)nseg * B * H + 3) / 4 * 4;
}

size_t ssm_backward_ws_floats(int B, int H, int G, int T, int dk, int dv, int nseg, bool bf16_io) {
  return backward_ws(B, H, G, T, dk, dv, nseg, bf16_io).total;
}

hipError_t launch_ssm_prefill(const SsmArgs& a, bool bf16_io, hipStream_t stream) {
  if (a.T == 0) {
    if (a.S_T == a.S0) return hipSuccess;
    const long long n4 = (long long)a.B * a.H * a.dk * a.dv / 4;
    hipLaunchKernelGGL(kda_ssm_copy_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, stream, a.S0, a.S_T, n4);
    return hipGetLastError();
  }
  return bf16_io ? prefill<bf16>(a, stream) : prefill<float>(a, stream);
}

hipError_t launch_ssm_backward(const SsmArgs& a, bool bf16_io, hipStream_t stream) {
  return bf16_io ? backward<bf16>(a, stream) : backward<float>(a, stream);
}

hipError_t launch_ssm_step(const void* q, const void* k, const void* v, const void* la, const void* beta, const void* D,
                           float* S, void* o, int N, int H, int G, int dk, int dv, bool bf16_io, hipStream_t stream) {
#define KDA_STEP(TY, DK, DV)                                                                                              \
  hipLaunchKernelGGL((kda_ssm_step_kernel<TY, DK, DV>), dim3((unsigned)((long long)N * H)), dim3(256), 0, stream,         \
                     (const TY*)q, (const TY*)k, (const TY*)v, (const TY*)la, (const TY*)beta, (const TY*)D, S, (TY*)o, H, G)
#define KDA_STEP_T(TY)                                    \
  do {                                                    \
    if (dk == 128 && dv == 128) KDA_STEP(TY, 128, 128);   \
    else if (dk == 128) KDA_STEP(TY, 128, 64);            \
    else if (dv == 128) KDA_STEP(TY, 64, 128);            \
    else KDA_STEP(TY, 64, 64);                            \
  } while (0)
  if (bf16_io) KDA_STEP_T(bf16);
  else KDA_STEP_T(float);
#undef KDA_STEP_T
#undef KDA_STEP
  return hipGetLastError();
}

hipError_t check_ssm_gates(const void* la, Str3 ls, const void* beta, Str3 bs, const int* lens, int B, int H, int T,
                           bool bf16_io, hipStream_t stream, unsigned int* bits_out) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);  // one check at a time: the flag is the device's only one
  void* p = nullptr;
  hipError_t e;
  if ((e = hipGetSymbolAddress(&p, HIP_SYMBOL(g_ssm_check_bits))) != hipSuccess) return e;
  unsigned int* f = static_cast<unsigned int*>(p);
  hipLaunchKernelGGL(kda_ssm_check_clear_kernel, dim3(1), dim3(1), 0, stream, f);
  SSM_TRY(hipGetLastError());
  const long long n = (long long)B * H * T;
  const long long nb = (n + 255) / 256;
  const dim3 grid((unsigned)(nb < 2048 ? nb : 2048));
  if (bf16_io)
    hipLaunchKernelGGL(kda_ssm_check_kernel<bf16>, grid, dim3(256), 0, stream, static_cast<const bf16*>(la), ls,
                       static_cast<const bf16*>(beta), bs, lens, H, T, n, f);
  else
    hipLaunchKernelGGL(kda_ssm_check_kernel<float>, grid, dim3(256), 0, stream, static_cast<const float*>(la), ls,
                       static_cast<const float*>(beta), bs, lens, H, T, n, f);
  SSM_TRY(hipGetLastError());
  unsigned int h = 0u;
  if ((e = hipMemcpyAsync(&h, f, sizeof(h), hipMemcpyDeviceToHost, stream)) != hipSuccess) return e;
  if ((e = hipStreamSynchronize(stream)) != hipSuccess) return e;
  *bits_out = h;
  return hipSuccess;
}

}  // namespace kda
