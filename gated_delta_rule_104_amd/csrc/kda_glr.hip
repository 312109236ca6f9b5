// Gated linear recurrence: one decay per channel and token, a vector as state,
//     h_t = a_t h_{t-1} + n_t beta_t x_t,   o_t = h_t,   a = e^{log_alpha} <= 1,   n = 1 or sqrt(1 - a^2)
// and its gradients, with lam the gradient that reaches h_t:
//     lam_t = dO_t + a_{t+1} lam_{t+1} (+ dh_T at the end),   dx = n beta lam,   dbeta = n x lam,
//     dlog_alpha = a h_{t-1} lam - (a^2 / n) beta x lam,   dh0 = a_1 lam_1,
// where h_{t-1} is read back from the forward pass's outputs.
//
// Nothing but the inputs and outputs has to move, so HBM bounds long calls: four prompts of 8192 tokens, 4096 channels, bf16,
// with beta and normalised, 198-203 us for 1.07 GB (5.3-5.4 TB/s); one of 65536 tokens, 2560 channels, without either 187-193
// for 1.01 GB; the gradients of the former 387-436, by card and place in memory, for 2.15 GB.  Vector instructions take 70% of
// the SIMDs' cycles beside that in the first and the last of these: 41 a value in the prompt and 82 in the gradients, whose
// lanes hold half as many tokens for the same joining and relay.  Every token
// waits for the one before it; the relay below keeps that to a few microseconds a tile, behind other tiles' loads.  One token of 256 sequences
// x 4096 channels: 7.4 us, 5.4 of them the kernel.  Short prompts are bounded by their launches: 9 us with one, 13 with two.
#include <cstdio>
#include <mutex>
#include <type_traits>

#include "kda_host.hpp"
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
__device__ __forceinline__ A advance(float e, A h, A b) {
  const A keep = slow(e) ? h : (A)0;
  const A old = __float_as_uint(e) == 0u ? (A)0 : h;
  if constexpr (sizeof(A) == 4) return fmaf(old, e, b) + keep;
  else return fma(old, (double)e, b) + keep;
}

// The state between tokens: fp32 inputs carry it in 64 bits, since its own rounding, 2^-25 a token,
// would be the largest error of outputs that are stored with 24 bits.
template <typename T> using State = typename std::conditional<sizeof(T) == 2, float, double>::type;

// A single token's decay.  bf16 takes it as a float: inside a lane's few tokens its rounding does not add up, and what
// passes from one lane's tokens to the next one's takes the decay of the sum of their logs (above).
template <typename T>
__device__ __forceinline__ float token_decay(float x) {
  if constexpr (sizeof(T) == 2) return __builtin_amdgcn_exp2f(1.44269504088896340736f * x);
  else return decay_of<T>(x);
}
template <typename T>
__device__ __forceinline__ float factor_of(float e) {  // a itself
  if constexpr (sizeof(T) == 2) return e;
  else return slow(e) ? 1.f + e : e;
}

// What a lane keeps of its tokens' log decays until the second walk: bf16 as they are, and takes the exponential
// again (half the registers), fp32 the decays in their place.
template <typename T, int NT>
__device__ __forceinline__ void hold_decays(u32x4 (&r)[NT]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) r[i][c] = __float_as_uint(decay_of<T>(__uint_as_float(r[i][c])));
  } else {
    forget(r);
  }
}
// Sums of log decays: a decay of zero makes a run's decay zero, also next to a gate of NaN (NaN - inf is NaN).
__device__ __forceinline__ float add_log(float sum, float x, bool clears) {
  return clears || sum == -__builtin_inff() ? -__builtin_inff() : sum + x;
}
template <typename T, int NT>
__device__ __forceinline__ void add_logs(const u32x4 (&r)[NT], float (&l)[kVec<T>]) {
#pragma unroll
  for (int c = 0; c < kVec<T>; ++c) {
    l[c] = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float x = unpack<T>(r[i]).v[c];
      l[c] = add_log(l[c], x, __float_as_uint(token_decay<T>(x)) == 0u);
    }
  }
}
template <typename T>
__device__ __forceinline__ float held_decay(u32x4 r, int c) {
  const float x = unpack<T>(r).v[c];
  return sizeof(T) == 2 ? token_decay<T>(x) : x;
}

// a h + b for one token.  CAREFUL: a decay of zero clears an infinity or NaN too; bf16 calls look at the last
// state of a run and walk it again if it has become one (the look costs less than the choice at every token).
template <typename T, bool CAREFUL>
__device__ __forceinline__ State<T> walk(float e, State<T> h, State<T> b) {
  if constexpr (sizeof(T) == 2) return fmaf(CAREFUL && e == 0.f ? 0.f : h, e, b);
  else return advance<State<T>>(e, h, b);
}
template <typename T>
__device__ __forceinline__ bool all_finite(const State<T> (&h)[kVec<T>]) {
  if constexpr (sizeof(T) == 4) return true;  // fp32 is always careful
  float zero = 0.f;
#pragma unroll
  for (int c = 0; c < kVec<T>; ++c) zero = fmaf((float)h[c], 0.f, zero);
  return zero == 0.f;
}

// n = sqrt(1 - a^2) from x = log a and the token's decay: bf16 from the series of 1 - e^2x above -1/16 (what follows is below
// y^5 / 720 of it, y = 2x, 2^-24), fp32 as sqrt((1 - a)(1 + a)) with 1 - a in all its digits.
template <typename T>
__device__ __forceinline__ float unit_of(float x, float e) {
  if constexpr (sizeof(T) == 2) {
    float p = fmaf(x, 2.f / 15, 1.f / 3);
    p = fmaf(x, p, 2.f / 3);
    p = fmaf(x, p, 1.f);
    p = fmaf(x, p, 1.f);
    return __builtin_amdgcn_sqrtf(fabsf(x) < 0.0625f ? -2.f * x * p : fmaf(-e, e, 1.f));
  } else {
    const float d = slow(e) ? -e : 1.f - e;
    return __builtin_amdgcn_sqrtf(d * (2.f - d));
  }
}

template <typename T>
__device__ __forceinline__ Row<T> ones() {
  Row<T> r;
#pragma unroll
  for (int c = 0; c < kVec<T>; ++c) r.v[c] = 1.f;
  return r;
}

// ------------------------------------------------------- runs of tokens
// A workgroup takes a tile: a slab of 64 channels of a run of tokens, one 16-byte group of channels of
// NT neighbouring tokens per lane.  It reads the inputs once and keeps decay and input of every
// token in registers while the state that enters the tile is found:
//   - a lane's tokens from a zero state give z and the sum l of their log decays; the state behind
//     them is e^l h + z.  They are joined over the lanes and waves in LDS, lane = channel;
//   - the tile publishes its (l, z), looks back at the tiles before it in the sequence for the nearest one
//     whose end state is known, goes forwards from there through the (l, z) in between, and publishes its
//     own end state as (-inf, end): a tile that clears what comes in and ends in that state.  A state is always
//     carried through tile after tile in order, so that it has the same bits however far a tile had to look;
//   - every lane's first state follows, and its tokens are walked again from registers.
// What is published are single 64-bit words that are valid once they are not the empty one, so no order
// between them is needed.  Waiting is bounded: a tile whose predecessors do not answer walks the
// sequence from its start by itself, so the call ends whatever order workgroups run in.

constexpr int kSlab = 64;                // channels of a tile
constexpr uint32_t kEmpty = 0xffffffffu;    // in the place of l (a NaN that no published value has)
constexpr uint32_t kCleared = 0xff800000u;  // -inf

// A channel's word of a tile: l below, z above.
__device__ __forceinline__ void publish(uint64_t* p, float l, float z) {
  const uint32_t low = l == l ? __float_as_uint(l) : 0x7fc00000u;
  __hip_atomic_store(p, (uint64_t)__float_as_uint(z) << 32 | low, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t published(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Lanes of a tile: a row of 64 channels takes LPR lanes, a wave holds SUB groups of NT tokens.
template <typename T> constexpr int kLpr = kSlab / kVec<T>;
template <typename T> constexpr int kSub = 64 / kLpr<T>;

template <typename T, int WAVES>
struct RelayMem {
  static constexpr int SUBS = WAVES * kSub<T>, WINDOW = SUBS / 2;
  alignas(16) float e[SUBS][kSlab];  // decays of the lanes' tokens
  // the sums of their logs; later decays and end states from zero of the tiles looked back at
  union {
    float l[SUBS][kSlab];
    float past[2][WINDOW][kSlab];
  };
  alignas(16) State<T> z[SUBS][kSlab];  // end states from zero; later the states in front
  float we[WAVES][kSlab], wl[WAVES][kSlab], h[kSlab];
  State<T> wz[WAVES][kSlab];
  uint32_t sums_there[WAVES], end_there[WAVES];
};

// The state in front of tile s >= 1 of a chain, lane = channel, for wave 0; false if the tiles before it did
// not answer.  words: the chain's tile 0, hop words to the next one (tile 0 publishes its end state alone);
// window: how many tiles to look at, shared out over the waves, which have nothing else to do.
template <typename T, int WAVES>
__device__ __forceinline__ bool look_back(RelayMem<T, WAVES>& m, const uint64_t* words, long long hop, int s, int window,
                                          int polls, float* state) {
  constexpr int W = RelayMem<T, WAVES>::WINDOW, OWN = W / WAVES;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int poll = 0; poll < polls; ++poll) {
    uint32_t sums = 0u, ends = 0u;
    uint64_t word[OWN];
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int i = k * WAVES + w;
      word[k] = kEmpty;
      if (i < window && i < s) word[k] = published(words + (long long)(s - 1 - i) * hop + lane);
    }
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int i = k * WAVES + w;
      const uint32_t l = (uint32_t)word[k];
      if (__ballot(l == kEmpty) == 0ull) sums |= 1u << i;
      if (__ballot(l != kCleared) == 0ull) ends |= 1u << i;
      m.past[0][i][lane] = decay_of<T>(__uint_as_float(l));
      m.past[1][i][lane] = __uint_as_float((uint32_t)(word[k] >> 32));
    }
    if (lane == 0) {
      m.sums_there[w] = sums;
      m.end_there[w] = ends;
    }
    __syncthreads();
    sums = ends = 0u;
#pragma unroll
    for (int u = 0; u < WAVES; ++u) {
      sums |= m.sums_there[u];
      ends |= m.end_there[u];
    }
    // the nearest tile whose end state is known, if everything in between is
    const int found = __ffs(ends) - 1;
    if (found >= 0 && (~sums & ((1u << found) - 1u)) == 0u) {
      if (w == 0) {
        float h = m.past[1][found][lane];
        for (int i = found - 1; i >= 0; --i) h = advance(m.past[0][i][lane], h, m.past[1][i][lane]);
        *state = h;
      }
      return true;
    }
    __builtin_amdgcn_s_sleep(1);
    __syncthreads();
  }
  return false;
}

// The state in front of a lane's tokens, once relay has found it.
template <typename T, int WAVES>
__device__ __forceinline__ void front_state(const RelayMem<T, WAVES>& m, State<T> (&h)[kVec<T>]) {
  const int lane = threadIdx.x & 63, sub = (threadIdx.x >> 6) * kSub<T> + lane / kLpr<T>;
#pragma unroll
  for (int c = 0; c < kVec<T>; ++c) h[c] = m.z[sub][lane % kLpr<T> * kVec<T> + c];
}

// N neighbouring values to LDS, 16 bytes at a time: single ones, which the compiler would make of them, have the lanes
// of eight groups of tokens on the same banks.
template <int N, typename A>
__device__ __forceinline__ void put(A* p, const A (&v)[N]) {
  using Vec = A __attribute__((ext_vector_type(16 / sizeof(A))));
  constexpr int W = 16 / sizeof(A);
#pragma unroll
  for (int i = 0; i < N / W; ++i) {
    Vec w;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = v[i * W + k];
    reinterpret_cast<Vec*>(p)[i] = w;
  }
}

// From each lane's (l, z) to the state in front of its tokens, h.  s: the tile's number in its chain;
// self: the state in front of the tile without the others' help; end: where the chain's end state goes
// (lane = channel), or null.
template <typename T, int WAVES, typename Self>
__device__ __forceinline__ void relay(RelayMem<T, WAVES>& m, const float (&l)[kVec<T>], const State<T> (&z)[kVec<T>],
                                      State<T> (&h)[kVec<T>], uint64_t* words, long long hop, int s, bool last, float first,
                                      int window, int polls, float* end, Self self) {
  constexpr int V = kVec<T>, LPR = kLpr<T>, SUB = kSub<T>;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, sub = w * SUB + lane / LPR, c0 = lane % LPR * V;
  float e[V];
#pragma unroll
  for (int c = 0; c < V; ++c) e[c] = decay_of<T>(l[c]);
  put<V>(&m.e[sub][c0], e);
  put<V>(&m.l[sub][c0], l);
  put<V>(&m.z[sub][c0], z);
  wave_lds_fence();
  float lw = 0.f;
  State<T> zw = 0;
#pragma unroll
  for (int r = 0; r < SUB; ++r) {
    const float e = m.e[w * SUB + r][lane];
    zw = advance(e, zw, m.z[w * SUB + r][lane]);
    lw = add_log(lw, m.l[w * SUB + r][lane], __float_as_uint(e) == 0u);
  }
  m.we[w][lane] = decay_of<T>(lw);
  m.wl[w][lane] = lw;
  m.wz[w][lane] = zw;
  __syncthreads();
  float lt = 0.f, front = first;
  State<T> zt = 0;
  uint64_t* own = words + s * hop + lane;
  if (w == 0) {
#pragma unroll
    for (int u = 0; u < WAVES; ++u) {
      const float e = m.we[u][lane];
      zt = advance(e, zt, m.wz[u][lane]);
      lt = add_log(lt, m.wl[u][lane], __float_as_uint(e) == 0u);
    }
    if (s > 0 && !last) publish(own, lt, (float)zt);
  }
  const bool known = s == 0 || look_back<T, WAVES>(m, words, hop, s, window, polls, &front);
  if (w == 0) {
    if (!known) front = self();
    const float out = advance(decay_of<T>(lt), front, (float)zt);
    if (!last) publish(own, -__builtin_inff(), out);
    else if (end) *end = out;
    m.h[lane] = front;
  }
  __syncthreads();
  State<T> run = m.h[lane];
  for (int u = 0; u < w; ++u) run = advance(m.we[u][lane], run, m.wz[u][lane]);
#pragma unroll
  for (int r = 0; r < SUB; ++r) {
    const State<T> zr = m.z[w * SUB + r][lane];
    m.z[w * SUB + r][lane] = run;
    run = advance(m.e[w * SUB + r][lane], run, zr);
  }
  wave_lds_fence();
  front_state(m, h);
}

// Which tile a workgroup has.  Tiles are handed out run by run, so that the ones in front of a tile are
// under way before it.  Consecutive workgroups go to the 8 XCDs in turn; with enough chains (or a
// multiple of 8) every XCD gets neighbouring ones, whose rows of 128 bytes lie side by side
// in memory (four 8K prompts 228 -> 206 us); with few chains all XCDs share each.
struct GlrGrid {
  int nslab, ntile, nchain, blocks;  // blocks: workgroups per run of all chains
  bool spread;
  bool place;  // the first states are in the words of the last tiles
};
struct GlrTile {
  int b, slab, s, len, ntile;  // sequence, slab, number in the chain, tokens and tiles of the sequence
  int chain;
  bool none;
  __device__ __forceinline__ GlrTile(const GlrArgs& a, const GlrGrid& n, int run) {
    s = blockIdx.x / n.blocks;
    chain = blockIdx.x % n.blocks;
    none = false;
    if (n.spread) {
      const int x = chain & 7, first = x * n.nchain / 8;
      chain = first + (chain >> 3);
      none = chain >= (x + 1) * n.nchain / 8;
    }
    b = chain / n.nslab;
    slab = chain % n.nslab;
    len = none ? 0 : seq_len(a.lens, b, a.T);
    ntile = max(1, (len + run - 1) / run);
  }
};

// NT rows of a lane's 16 bytes, at tokens t0, t0 + STEP, ...  Where not all of a tile's rows and channels are
// there (full false), rows outside [0, len) are read from inside and set to zero.
template <typename T, int NT, int STEP>
__device__ __forceinline__ void load_rows(u32x4 (&r)[NT], const T* p, long long st, int t0, int len, bool on, bool full) {
  if (full) {
    p += t0 * st;
#pragma unroll
    for (int i = 0; i < NT; ++i) r[i] = ld_once(p + i * (STEP * st));
  } else {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = t0 + i * STEP;
      r[i] = ld_once(p + min(max(t, 0), len - 1) * st);
      if (!on || t < 0 || t >= len) r[i] = u32x4{0u, 0u, 0u, 0u};
    }
  }
}

// Waves per SIMD that the registers have to leave room for.
template <typename T, int NT, bool GRADIENTS, bool BETA>
constexpr int kResident = GRADIENTS ? (sizeof(T) == 4 || NT == 2 ? 4 : (NT == 3 || !BETA ? 3 : 2))
                                    : (sizeof(T) == 2 && NT == 4 ? 4 : 3);

template <typename T, int NT, int WAVES, bool NORM, bool BETA>
__global__ __launch_bounds__(64 * WAVES, (kResident<T, NT, false, BETA>)) void kda_glr_kernel(GlrArgs a, GlrGrid n, int window, int polls) {
  constexpr int V = kVec<T>, LPR = kLpr<T>, SUB = kSub<T>, RUN = WAVES * SUB * NT;
  __shared__ RelayMem<T, WAVES> mem;
  const GlrTile g(a, n, RUN);
  if (g.none || g.s >= g.ntile) return;
  const int lane = threadIdx.x & 63, C = a.H * a.d, first_t = g.s * RUN;
  const int t0 = first_t + ((int)(threadIdx.x >> 6) * SUB + lane / LPR) * NT;
  const int c0 = g.slab * kSlab + lane % LPR * V;
  const bool on = c0 < C;
  const int hd = on ? c0 / a.d : 0, j0 = on ? c0 % a.d : 0;
  const T* x = static_cast<const T*>(a.x) + g.b * a.xs.b + hd * a.xs.h + j0;
  const T* la = static_cast<const T*>(a.la) + g.b * a.ls.b + hd * a.ls.h + j0;
  const T* beta = BETA ? static_cast<const T*>(a.beta) + g.b * a.bs.b + hd * a.bs.h + j0 : nullptr;
  const int cl = g.slab * kSlab + lane;  // lane = channel
  const long long at = (long long)g.b * C + cl;
  uint64_t* words = static_cast<uint64_t*>(a.ws) + (long long)g.chain * kSlab;
  const float first = a.h0 && cl < C ? (n.place ? __uint_as_float((uint32_t)words[(long long)(n.ntile - 1) * n.nchain * kSlab + lane]) : a.h0[at]) : 0.f;
  if (g.len == 0) {
    if (threadIdx.x < 64 && cl < C) a.h_T[at] = first;
    return;
  }
  const bool full = first_t + RUN <= g.len && (g.slab + 1) * kSlab <= C;
  u32x4 rx[NT], rl[NT], rb[NT];
  load_rows<T, NT, 1>(rl, la, a.ls.t, t0, g.len, on, full);
  load_rows<T, NT, 1>(rx, x, a.xs.t, t0, g.len, on, full);
  if constexpr (BETA) load_rows<T, NT, 1>(rb, beta, a.bs.t, t0, g.len, on, full);
  // longer runs of bf16 are kept as they were read, and their inputs are formed again: fewer registers
  constexpr bool AGAIN = sizeof(T) == 2 && NT > 4;
  float in[AGAIN ? 1 : NT][V], l[V];
  State<T> h[V], z[V];
  const auto input = [&](int i, int c, float e) {
    if constexpr (!AGAIN) {
      return in[i][c];
    } else {
      float v = unpack<T>(rx[i]).v[c];
      if constexpr (BETA) v *= unpack<T>(rb[i]).v[c];
      return NORM ? v * unit_of<T>(unpack<T>(rl[i]).v[c], e) : v;
    }
  };
#pragma unroll
  for (int c = 0; c < V; ++c) l[c] = 0.f;
  if constexpr (sizeof(T) == 4) {
    add_logs<T>(rl, l);
    hold_decays<T>(rl);
  }
#pragma unroll
  for (int c = 0; c < V; ++c) z[c] = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const Row<T> xv = unpack<T>(rx[i]), bv = BETA ? unpack<T>(rb[i]) : ones<T>();
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float e = held_decay<T>(rl[i], c);
      float v = BETA ? bv.v[c] * xv.v[c] : xv.v[c];
      if constexpr (NORM) v *= unit_of<T>(unpack<T>(rl[i]).v[c], e);
      if constexpr (!AGAIN) in[i][c] = v;
      z[c] = walk<T, false>(e, z[c], v);
      if constexpr (sizeof(T) == 2) l[c] += unpack<T>(rl[i]).v[c];
    }
    __builtin_amdgcn_sched_barrier(0);  // (token by token: interleaved, they would hold all decays at once)
  }
  if (__builtin_expect(!all_finite<T>(z), 0)) {
    forget(rl);
    if constexpr (AGAIN) forget(rx);
    if constexpr (AGAIN && BETA) forget(rb);
    add_logs<T>(rl, l);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      z[c] = 0;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float e = held_decay<T>(rl[i], c);
        z[c] = walk<T, true>(e, z[c], input(i, c, e));
      }
    }
  }
  if constexpr (sizeof(T) == 2) hold_decays<T>(rl);
  if constexpr (AGAIN) forget(rx);
  if constexpr (AGAIN && BETA) forget(rb);
  const auto self = [&]() {
    if (cl >= C) return 0.f;
    const int hh = cl / a.d, jj = cl % a.d;
    const T* px = static_cast<const T*>(a.x) + g.b * a.xs.b + hh * a.xs.h + jj;
    const T* pl = static_cast<const T*>(a.la) + g.b * a.ls.b + hh * a.ls.h + jj;
    const T* pb = BETA ? static_cast<const T*>(a.beta) + g.b * a.bs.b + hh * a.bs.h + jj : nullptr;
    State<T> run = first;
    for (long long t = 0; t < first_t; ++t) {
      const float x1 = to_f32(pl[t * a.ls.t]);
      float v = to_f32(px[t * a.xs.t]);
      if constexpr (BETA) v *= to_f32(pb[t * a.bs.t]);
      if constexpr (NORM) v *= unit_of<T>(x1, token_decay<T>(x1));
      run = advance<State<T>>(decay_of<T>(x1), run, v);
    }
    return (float)run;
  };
  relay<T, WAVES>(mem, l, z, h, words, (long long)n.nchain * kSlab, g.s, g.s == g.ntile - 1, first, window, polls,
                  cl < C ? a.h_T + at : nullptr, self);
  if (!on) return;
  if constexpr (sizeof(T) == 4) {  // (what was kept in 64 bits)
    forget(rl);
    forget(in);
  }
  T* o = static_cast<T*>(a.o) + g.b * a.os.b + hd * a.os.h + j0;
  const auto outputs = [&](auto careful) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      Row<T> y;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float e = held_decay<T>(rl[i], c);
        h[c] = walk<T, decltype(careful)::value>(e, h[c], input(i, c, e));
        y.v[c] = (float)h[c];
      }
      if (full || t0 + i < g.len) store_by(o + (t0 + i) * a.os.t, pack<T>(y), a.lines);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  outputs(std::false_type());
  if (__builtin_expect(!all_finite<T>(h), 0)) {
    forget(rl);
    if constexpr (AGAIN) forget(rx);
    if constexpr (AGAIN && BETA) forget(rb);
    front_state(mem, h);
    outputs(std::true_type());
  }
}

// Empties the n / 2 words of a call's tiles, 64 bytes a thread.  With h0 the first states, of C channels a sequence, are
// put into the words of the chains' last tiles, which publish nothing.
__global__ __launch_bounds__(256) void kda_glr_clear_kernel(u32x4* words, long long n, const float* h0, int nchain, int nslab, int C) {
  const long long last = n - (long long)nchain * (kSlab / 2);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const long long i = (long long)blockIdx.x * 1024 + u * 256 + threadIdx.x;
    if (i >= n) continue;
    u32x4 v{kEmpty, kEmpty, kEmpty, kEmpty};
    if (h0 && i >= last) {
      const int chain = (int)((i - last) / (kSlab / 2)), c = chain % nslab * kSlab + (int)((i - last) % (kSlab / 2)) * 2;
      if (c < C) {  // (C is even)
        const float* h = h0 + (long long)(chain / nslab) * C + c;
        v[0] = __float_as_uint(h[0]);
        v[2] = __float_as_uint(h[1]);
      }
    }
    words[i] = v;
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
    if (a.norm) in *= unit_of<T>(lv.v[c], token_decay<T>(lv.v[c]));
    y.v[c] = (float)advance<State<T>>(e, hv[c / 4][c % 4], in);
    hv[c / 4][c % 4] = y.v[c];
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) *reinterpret_cast<f32x4*>(h + 4 * i) = hv[i];
  st16(static_cast<T*>(a.o) + b * a.os.b + hd * a.os.h + j0, pack<T>(y));
}

// The gradients' chain runs from the last token to the first: mu_t = a_t (dO_t + mu_{t+1}), the same relay
// with the tiles, and the tokens in them, in reverse.
template <typename T, int NT, int WAVES, bool NORM, bool BETA>
__global__ __launch_bounds__(64 * WAVES, (kResident<T, NT, true, BETA>)) void kda_glr_bwd_kernel(GlrArgs a, GlrGrid n, int window, int polls) {
  constexpr int V = kVec<T>, LPR = kLpr<T>, SUB = kSub<T>, RUN = WAVES * SUB * NT;
  __shared__ RelayMem<T, WAVES> mem;
  const GlrTile g(a, n, RUN);
  if (g.none) return;
  const int lane = threadIdx.x & 63, C = a.H * a.d;
  const int tile = g.s < g.ntile ? g.ntile - 1 - g.s : g.s;  // behind the sequence: only zeros
  const int t0 = (tile + 1) * RUN - 1 - ((int)(threadIdx.x >> 6) * SUB + lane / LPR) * NT;  // a lane's tokens: t0, t0 - 1, ...
  const int c0 = g.slab * kSlab + lane % LPR * V;
  const bool on = c0 < C;
  const int hd = on ? c0 / a.d : 0, j0 = on ? c0 % a.d : 0;
  const u32x4 zero{0u, 0u, 0u, 0u};
  T* dx = static_cast<T*>(a.dx) + g.b * a.dxs.b + hd * a.dxs.h + j0;
  T* dla = static_cast<T*>(a.dla) + g.b * a.dls.b + hd * a.dls.h + j0;
  T* dbeta = BETA ? static_cast<T*>(a.dbeta) + g.b * a.dbs.b + hd * a.dbs.h + j0 : nullptr;
  if ((tile + 1) * RUN > g.len && on) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const long long t = t0 - i;
      if (t < g.len || t >= a.T) continue;
      st16(dx + t * a.dxs.t, zero);
      st16(dla + t * a.dls.t, zero);
      if constexpr (BETA) st16(dbeta + t * a.dbs.t, zero);
    }
  }
  if (g.s >= g.ntile) return;
  const T* x = static_cast<const T*>(a.x) + g.b * a.xs.b + hd * a.xs.h + j0;
  const T* la = static_cast<const T*>(a.la) + g.b * a.ls.b + hd * a.ls.h + j0;
  const T* beta = BETA ? static_cast<const T*>(a.beta) + g.b * a.bs.b + hd * a.bs.h + j0 : nullptr;
  const T* o = static_cast<const T*>(a.o) + g.b * a.os.b + hd * a.os.h + j0;
  const T* dO = static_cast<const T*>(a.dO) + g.b * a.dos.b + hd * a.dos.h + j0;
  const int cl = g.slab * kSlab + lane;  // lane = channel
  const long long at = (long long)g.b * C;
  const float first = a.dh_T && cl < C ? a.dh_T[at + cl] : 0.f;
  if (g.len == 0) {
    if (threadIdx.x < 64 && cl < C && a.dh0) a.dh0[at + cl] = first;
    return;
  }
  const bool full = (tile + 1) * RUN <= g.len && (g.slab + 1) * kSlab <= C;
  u32x4 rx[NT], rl[NT], rb[NT], rg[NT], ro[NT];
  load_rows<T, NT, -1>(rl, la, a.ls.t, t0, g.len, on, full);
  load_rows<T, NT, -1>(rg, dO, a.dos.t, t0, g.len, on, full);
  if constexpr (NORM || BETA) load_rows<T, NT, -1>(rx, x, a.xs.t, t0, g.len, on, full);
  if constexpr (BETA) load_rows<T, NT, -1>(rb, beta, a.bs.t, t0, g.len, on, full);
  load_rows<T, NT, -1>(ro, o, a.os.t, t0 - 1, g.len, on, full && tile > 0);
  float l[V];
  State<T> mu[V], z[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    l[c] = 0.f;
    z[c] = 0;
  }
  if constexpr (sizeof(T) == 4) {
    add_logs<T>(rl, l);
    hold_decays<T>(rl);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const Row<T> gv = unpack<T>(rg[i]);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      z[c] = walk<T, false>(held_decay<T>(rl[i], c), z[c] + gv.v[c], 0);
      if constexpr (sizeof(T) == 2) l[c] += unpack<T>(rl[i]).v[c];
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (__builtin_expect(!all_finite<T>(z), 0)) {
    forget(rl);
    add_logs<T>(rl, l);
    forget(rg);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      z[c] = 0;
#pragma unroll
      for (int i = 0; i < NT; ++i) z[c] = walk<T, true>(held_decay<T>(rl[i], c), z[c] + unpack<T>(rg[i]).v[c], 0);
    }
  }
  if constexpr (sizeof(T) == 2) hold_decays<T>(rl);
  const auto self = [&]() {
    if (cl >= C) return 0.f;
    const int hh = cl / a.d, jj = cl % a.d;
    const T* pl = static_cast<const T*>(a.la) + g.b * a.ls.b + hh * a.ls.h + jj;
    const T* pg = static_cast<const T*>(a.dO) + g.b * a.dos.b + hh * a.dos.h + jj;
    State<T> run = first;
    for (long long t = g.len - 1; t >= (long long)(tile + 1) * RUN; --t)
      run = advance<State<T>>(decay_of<T>(to_f32(pl[t * a.ls.t])), run + to_f32(pg[t * a.dos.t]), 0);
    return (float)run;
  };
  uint64_t* words = static_cast<uint64_t*>(a.ws) + (long long)g.chain * kSlab;
  relay<T, WAVES>(mem, l, z, mu, words, (long long)n.nchain * kSlab, g.s, g.s == g.ntile - 1, first, window, polls,
                  a.dh0 && cl < C ? a.dh0 + at + cl : nullptr, self);
  if (!on) return;
  forget(rl);
  forget(rg);
  const auto gradients = [&](auto careful) {
    constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const long long t = t0 - i;
      const Row<T> xv = NORM || BETA ? unpack<T>(rx[i]) : ones<T>(), bv = BETA ? unpack<T>(rb[i]) : ones<T>();
      const Row<T> gv = unpack<T>(rg[i]);
      Row<T> before = unpack<T>(ro[i]), gx, gl, gb;
      if (t == 0 && a.h0) {
#pragma unroll
        for (int c = 0; c < V; ++c) before.v[c] = a.h0[at + c0 + c];
      }
#pragma unroll
      for (int c = 0; c < V; ++c) {
        mu[c] += (State<T>)gv.v[c];
        const float lam = (float)mu[c], ee = held_decay<T>(rl[i], c), al = factor_of<T>(ee);
        float nl = lam, part = 0.f;
        if constexpr (NORM) {
          const float n = unit_of<T>(unpack<T>(rl[i]).v[c], ee);
          nl *= n;
          part = n > 0.f ? al * al * __builtin_amdgcn_rcpf(n) * (BETA ? bv.v[c] * xv.v[c] : xv.v[c]) : 0.f;
        }
        gx.v[c] = BETA ? nl * bv.v[c] : nl;
        gb.v[c] = nl * xv.v[c];
        gl.v[c] = (al * before.v[c] - part) * lam;
        gl.v[c] = al == 0.f ? 0.f : gl.v[c];  // (also where the state in front is not finite)
        mu[c] = walk<T, CAREFUL>(ee, mu[c], 0);
      }
      if (!full && t >= g.len) continue;
      store_by(dx + t * a.dxs.t, pack<T>(gx), a.lines);
      store_by(dla + t * a.dls.t, pack<T>(gl), a.lines);
      if constexpr (BETA) store_by(dbeta + t * a.dbs.t, pack<T>(gb), a.lines);
    }
  };
  gradients(std::false_type());
  if (__builtin_expect(!all_finite<T>(mu), 0)) {
    forget(rl);
    if constexpr (NORM || BETA) forget(rx);
    if constexpr (BETA) forget(rb);
    forget(rg);
    forget(ro);
    front_state(mem, mu);
    gradients(std::true_type());
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

constexpr int kWaves = 4;

// Tokens per lane.  More of them make a tile longer, and a chain's way through its tiles shorter, but take
// registers, and with them the waves that hide each other's latency, and leave short sequences with few tiles.  So long
// sequences, and few chains, whose way bounds the call, take more than others, and calls without beta, which hold a tensor
// less, more than calls with it.  Prompts form their inputs again with more than 4 tokens (fewer registers), which a
// normaliser makes dearer.  bf16, us; prompts by chains of 64 channels and tokens:
//   with beta, normalised    4 / 8 tokens       4 x 32000 45 / 33   40 x 32000 143 / 135   64 x 32000 209 / 204   128 x 32000 386 / 392
//                                               4 x 8000 18 / 19    40 x 8000 42 / 44      64 x 8000 60 / 63      256 x 8000 192 / 203
//   without, normalised      4 / 8 / 12         4 x 32000 43 / 30 / 29   64 x 32000 177 / 172 / 169   256 x 32000 625 / 651 / 626
//                                               4 x 8000 17 / 17 / 19    64 x 8000 50 / 52 / 55       256 x 8000 161 / 172 / 164
//   without either           4 / 8 / 12         4 x 32000 43 / 28 / 26   64 x 32000 170 / 152 / 149   256 x 32000 564 / 555 / 543
//                                               4 x 8000 17 / 15 / 15    64 x 8000 48 / 46 / 48       256 x 2000 44 / 44 / 47
// (The joining of lanes and the relay cost a lane the same whatever its tokens: with 2 a lane the gradients' share of it is
// twice the prompts' with 4.)
// gradients of 134M values with beta (268M without) in up to 64K tokens by chains, with 2 / 3 / 4 tokens:
//   with beta                256 439 / 444 / 468   64 443 / 456 / 468   40 453 / 429 / 456   4 141 / 105 / 86
//   without                  256 310 / 272 / 273   64 323 / 293 / 285   40 340 / 292 / 282   4 133 / 95 / 73
// Where the longer run is the whole sequence, the call needs no second launch: prompts with beta of 200 tokens, 4 / 8:
// 64 chains 14.5 / 12.1, 128 13.5 / 12.8, 512 19.3 / 20.5; without either of 300, 8 / 12: 64 chains 12.9 / 10.6, 512
// 22.2 / 17.0 (normalised, 4 / 12: 13.3 / 13.1, 22.4 / 24.2); gradients with beta of 100, 3 or 2 / 4: 15 chains 18.1 / 13.9,
// 512 20.8 / 17.1.
// fp32 holds half as many values per lane and token: prompts of 128 chains 234 / 201 / 199 with 2 / 4 / 8, gradients 403 /
// 377 with 2 / 4, and the longer ones win with fewer chains too.
int glr_tokens(bool bf16_io, bool gradients, bool beta, bool norm, int nchain, int len) {
  if (!bf16_io) return gradients ? 4 : 8;
  const bool longer = len >= 16384;
  if (gradients) return !beta || nchain <= 8 || (len > 64 && len <= 128) ? 4 : (nchain < 64 ? 3 : 2);
  if (beta) return nchain < 128 && (longer || (len > 128 && len <= 256)) ? 8 : 4;
  if (norm) return longer ? 12 : 4;
  return longer || (len > 256 && len <= 384) ? 12 : 8;
}

GlrGrid glr_grid(int B, int H, int len, int d, bool bf16_io, bool gradients, bool beta, bool norm, int* tokens) {
  GlrGrid n;
  n.nslab = (H * d + kSlab - 1) / kSlab;
  n.nchain = n.nslab * B;
  *tokens = glr_tokens(bf16_io, gradients, beta, norm, n.nchain, len);
  const int run = kWaves * (bf16_io ? kSub<bf16> : kSub<float>) * *tokens;
  n.ntile = len > 0 ? (len + run - 1) / run : 1;
  n.spread = n.nchain >= 64 || (n.nchain % 8 == 0 && n.nchain > 0);
  n.blocks = n.spread ? (n.nchain + 7) / 8 * 8 : n.nchain;
  n.place = false;
  return n;
}

template <typename T, bool GRADIENTS, int NT, bool BETA, bool NORM>
hipError_t glr_launch(const GlrArgs& a, GlrGrid n, int polls, hipStream_t stream) {
  if (n.ntile > 1) {
    const long long words = (long long)n.nchain * n.ntile * (kSlab / 2);  // 16 bytes each
    // a chain's last tile may write h_T before another one has read h0: in place, the tiles read a copy
    n.place = !GRADIENTS && a.h0 && a.h0 == a.h_T;
    hipLaunchKernelGGL(kda_glr_clear_kernel, dim3((unsigned)((words + 1023) / 1024)), dim3(256), 0, stream,
                       static_cast<u32x4*>(a.ws), words, n.place ? a.h0 : nullptr, n.nchain, n.nslab, a.H * a.d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (api_log_on())
    fprintf(stderr, "[kda] %s B=%d H=%d T=%d d=%d: %d chains of %d runs of %d tokens\n", GRADIENTS ? "glr_backward" : "glr_prefill",
            a.B, a.H, a.T, a.d, n.nchain, n.ntile, kWaves * kSub<T> * NT);
  const dim3 grid((unsigned)((long long)n.blocks * n.ntile)), threads(64 * kWaves);
  // tiles of a chain that are under way together, and one more: about 1024 workgroups fit the device
  const int window = 1 + 1024 / n.nchain;
  if constexpr (GRADIENTS) hipLaunchKernelGGL((kda_glr_bwd_kernel<T, NT, kWaves, NORM, BETA>), grid, threads, 0, stream, a, n, window, polls);
  else hipLaunchKernelGGL((kda_glr_kernel<T, NT, kWaves, NORM, BETA>), grid, threads, 0, stream, a, n, window, polls);
  return hipGetLastError();
}
template <typename T, bool GRADIENTS, int NT, bool BETA>
hipError_t glr_launch(const GlrArgs& a, const GlrGrid& n, int polls, hipStream_t stream) {
  return a.norm ? glr_launch<T, GRADIENTS, NT, BETA, true>(a, n, polls, stream) : glr_launch<T, GRADIENTS, NT, BETA, false>(a, n, polls, stream);
}

template <typename T>
hipError_t glr_step(const GlrArgs& a, hipStream_t stream) {
  const int nvec = a.H * a.d / kVec<T>;
  const dim3 grid((unsigned)(((long long)nvec * a.B + 255) / 256));
  hipLaunchKernelGGL((kda_glr_step_kernel<T>), grid, dim3(256), 0, stream, a, nvec);
  return hipGetLastError();
}

}  // namespace

size_t glr_ws_bytes(int B, int H, int T, int d, bool bf16_io, bool gradients) {
  size_t most = 0;
  for (int k = 0; k < 4; ++k) {
    int nt;
    const GlrGrid n = glr_grid(B, H, T, d, bf16_io, gradients, k & 1, k & 2, &nt);
    const size_t bytes = n.ntile > 1 ? (size_t)n.nchain * n.ntile * kSlab * sizeof(uint64_t) : 0;
    most = bytes > most ? bytes : most;
  }
  return most;
}

bool glr_fits(int B, int H, int T, int d, bool beta, bool norm, bool bf16_io, bool gradients) {
  int nt;
  const GlrGrid n = glr_grid(B, H, T, d, bf16_io, gradients, beta, norm, &nt);
  return launchable((long long)n.blocks * n.ntile, 64 * kWaves);
}
bool glr_step_fits(int N, int H, int d, bool bf16_io) {
  return launchable(((long long)N * (H * d / (bf16_io ? 8 : 4)) + 255) / 256, 256);
}

// (a tile's rows are 64 channels of heads that may lie apart)
bool glr_lines(const GlrArgs& a, const void* p, Str3 s, bool bf16_io) {
  const int es = bf16_io ? 2 : 4;
  return whole_lines(p, s, (long long)a.B * a.H * a.T, (long long)a.d * es, es);
}

hipError_t launch_glr(const GlrArgs& args, bool bf16_io, int polls, hipStream_t stream) {
  GlrArgs a = args;
  a.lines = glr_lines(a, a.o, a.os, bf16_io);
  int nt;
  const GlrGrid n = glr_grid(a.B, a.H, a.T, a.d, bf16_io, false, a.beta != nullptr, a.norm, &nt);
  if (!bf16_io) return a.beta ? glr_launch<float, false, 8, true>(a, n, polls, stream) : glr_launch<float, false, 8, false>(a, n, polls, stream);
  if (a.beta) return nt == 8 ? glr_launch<bf16, false, 8, true>(a, n, polls, stream) : glr_launch<bf16, false, 4, true>(a, n, polls, stream);
  if (nt == 12) return glr_launch<bf16, false, 12, false>(a, n, polls, stream);
  return a.norm ? glr_launch<bf16, false, 4, false, true>(a, n, polls, stream) : glr_launch<bf16, false, 8, false, false>(a, n, polls, stream);
}

hipError_t launch_glr_backward(const GlrArgs& args, bool bf16_io, int polls, hipStream_t stream) {
  GlrArgs a = args;
  a.lines = glr_lines(a, a.dx, a.dxs, bf16_io) && glr_lines(a, a.dla, a.dls, bf16_io) &&
            (!a.dbeta || glr_lines(a, a.dbeta, a.dbs, bf16_io));
  int nt;
  const GlrGrid n = glr_grid(a.B, a.H, a.T, a.d, bf16_io, true, a.beta != nullptr, a.norm, &nt);
  if (!bf16_io) return a.beta ? glr_launch<float, true, 4, true>(a, n, polls, stream) : glr_launch<float, true, 4, false>(a, n, polls, stream);
  if (!a.beta) return glr_launch<bf16, true, 4, false>(a, n, polls, stream);
  if (nt == 2) return glr_launch<bf16, true, 2, true>(a, n, polls, stream);
  return nt == 3 ? glr_launch<bf16, true, 3, true>(a, n, polls, stream) : glr_launch<bf16, true, 4, true>(a, n, polls, stream);
}

hipError_t launch_glr_step(const GlrArgs& a, bool bf16_io, hipStream_t stream) {
  return bf16_io ? glr_step<bf16>(a, stream) : glr_step<float>(a, stream);
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
