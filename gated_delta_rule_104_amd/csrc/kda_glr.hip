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
__device__ __forceinline__ A advance(float e, A h, A b) {
  const A keep = slow(e) ? h : (A)0;
  const A old = __float_as_uint(e) == 0u ? (A)0 : h;
  if constexpr (sizeof(A) == 4) return fmaf(old, e, b) + keep;
  else return fma(old, (double)e, b) + keep;
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

// ------------------------------------------------------- runs of tokens
// A workgroup takes a tile: a slab of 64 channels of a run of tokens, one 16-byte group of channels of
// NT neighbouring tokens per lane.  It reads the inputs once and keeps decay and input of every
// token in registers while the state that enters the tile is found:
//   - a lane's tokens from a zero state give z and the sum l of their log decays; the state behind
//     them is e^l h + z.  They are joined over the lanes and waves in LDS, lane = channel;
//   - the tile publishes its (l, z), looks back at the tiles before it in the sequence for the nearest one
//     whose end state is known, goes forwards from there through the (l, z) in between, and publishes its
//     own end state.  A state is always carried through tile after tile in order, so that it has the
//     same bits however far a tile had to look;
//   - every lane's first state follows, and its tokens are walked again from registers.
// What is published are single 32-bit words that are valid once they are not the empty one, so no order
// between them is needed.  Waiting is bounded: a tile whose predecessors do not answer walks the
// sequence from its start by itself, so the call ends whatever order workgroups run in.

constexpr int kSlab = 64;                // channels of a tile
constexpr int kWords = 3 * kSlab;        // of a tile: l, z and the end state of each channel
constexpr uint32_t kEmpty = 0xffffffffu;  // (a NaN that no published value has)

__device__ __forceinline__ void publish(uint32_t* p, float v) {
  __hip_atomic_store(p, v == v ? __float_as_uint(v) : 0x7fc00000u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t published(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Lanes of a tile: a row of 64 channels takes LPR lanes, a wave holds SUB groups of NT tokens.
template <typename T> constexpr int kLpr = kSlab / kVec<T>;
template <typename T> constexpr int kSub = 64 / kLpr<T>;

template <typename T, int WAVES>
struct RelayMem {
  float e[WAVES * kSub<T>][kSlab], l[WAVES * kSub<T>][kSlab];
  State<T> z[WAVES * kSub<T>][kSlab];
  float we[WAVES][kSlab], wl[WAVES][kSlab], h[kSlab];
  State<T> wz[WAVES][kSlab];
};

// The state in front of tile s >= 1 of a chain, lane = channel; false if the tiles before it did not
// answer.  words: the chain's tile 0, hop words to the next one; first: the state in front of tile 0.
template <typename T>
__device__ __forceinline__ bool look_back(const uint32_t* words, long long hop, int s, float first, int polls, float* state) {
  constexpr int W = 8;  // tiles looked at together
  const int lane = threadIdx.x & 63;
  for (int poll = 0; poll < polls; ++poll) {
    uint32_t p[W], l[W], z[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t* q = words + (long long)max(s - 1 - i, 0) * hop + lane;
      p[i] = published(q + 2 * kSlab);
      l[i] = published(q);
      z[i] = published(q + kSlab);
    }
    int found = -1;
    bool open = true;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (!open || found >= 0) continue;
      if (i >= s || __ballot(p[i] == kEmpty) == 0ull) found = i;
      else if (__ballot(l[i] == kEmpty || z[i] == kEmpty) != 0ull) open = false;
    }
    if (found >= 0) {
      float h = first;
#pragma unroll
      for (int i = W - 1; i >= 0; --i) {
        if (i == found && i < s) h = __uint_as_float(p[i]);
        if (i < found) h = advance(decay_of<T>(__uint_as_float(l[i])), h, __uint_as_float(z[i]));
      }
      *state = h;
      return true;
    }
    __builtin_amdgcn_s_sleep(4);
  }
  return false;
}

// From each lane's (l, z) to the state in front of its tokens, h.  s: the tile's number in its chain;
// self: the state in front of the tile without the others' help; end: where the chain's end state goes
// (lane = channel), or null.
template <typename T, int WAVES, typename Self>
__device__ __forceinline__ void relay(RelayMem<T, WAVES>& m, const float (&l)[kVec<T>], const State<T> (&z)[kVec<T>],
                                      State<T> (&h)[kVec<T>], uint32_t* words, long long hop, int s, bool last, float first,
                                      int polls, float* end, Self self) {
  constexpr int V = kVec<T>, LPR = kLpr<T>, SUB = kSub<T>;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, sub = w * SUB + lane / LPR, c0 = lane % LPR * V;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    m.e[sub][c0 + c] = decay_of<T>(l[c]);
    m.l[sub][c0 + c] = l[c];
    m.z[sub][c0 + c] = z[c];
  }
  wave_lds_fence();
  float lw = 0.f;
  State<T> zw = 0;
#pragma unroll
  for (int r = 0; r < SUB; ++r) {
    zw = advance(m.e[w * SUB + r][lane], zw, m.z[w * SUB + r][lane]);
    lw += m.l[w * SUB + r][lane];
  }
  m.we[w][lane] = decay_of<T>(lw);
  m.wl[w][lane] = lw;
  m.wz[w][lane] = zw;
  __syncthreads();
  if (w == 0) {
    float lt = 0.f;
    State<T> zt = 0;
#pragma unroll
    for (int u = 0; u < WAVES; ++u) {
      zt = advance(m.we[u][lane], zt, m.wz[u][lane]);
      lt += m.wl[u][lane];
    }
    uint32_t* own = words + s * hop + lane;
    float front = first;
    if (s > 0) {
      if (!last) {
        publish(own, lt);
        publish(own + kSlab, (float)zt);
      }
      if (!look_back<T>(words, hop, s, first, polls, &front)) front = self();
    }
    const float out = advance(decay_of<T>(lt), front, (float)zt);
    if (!last) publish(own + 2 * kSlab, out);
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
#pragma unroll
  for (int c = 0; c < V; ++c) h[c] = m.z[sub][c0 + c];
}

// Which tile a workgroup has, and a lane's place in it.
struct GlrTile {
  int b, slab, s, len, ntile;  // sequence, slab, number in the chain, tokens and tiles of the sequence
  int chain;
  __device__ __forceinline__ GlrTile(const GlrArgs& a, int nslab, int run) {
    const int nchain = nslab * a.B;
    s = blockIdx.x / nchain;
    chain = blockIdx.x % nchain;
    b = chain / nslab;
    slab = chain % nslab;
    len = seq_len(a.lens, b, a.T);
    ntile = max(1, (len + run - 1) / run);
  }
};

template <typename T, int NT, int WAVES, bool NORM, bool BETA>
__global__ __launch_bounds__(64 * WAVES) void kda_glr_kernel(GlrArgs a, int nslab, int polls) {
  constexpr int V = kVec<T>, LPR = kLpr<T>, SUB = kSub<T>, RUN = WAVES * SUB * NT;
  __shared__ RelayMem<T, WAVES> mem;
  const GlrTile g(a, nslab, RUN);
  if (g.s >= g.ntile) return;
  const int lane = threadIdx.x & 63, C = a.H * a.d, first_t = g.s * RUN;
  const int t0 = first_t + ((int)(threadIdx.x >> 6) * SUB + lane / LPR) * NT;
  const int c0 = g.slab * kSlab + lane % LPR * V;
  const bool on = c0 < C;
  const int hd = on ? c0 / a.d : 0, j0 = on ? c0 % a.d : 0;
  const T* x = static_cast<const T*>(a.x) + g.b * a.xs.b + hd * a.xs.h + j0;
  const T* la = static_cast<const T*>(a.la) + g.b * a.ls.b + hd * a.ls.h + j0;
  const T* beta = BETA ? static_cast<const T*>(a.beta) + g.b * a.bs.b + hd * a.bs.h + j0 : nullptr;
  u32x4 rx[NT], rl[NT], rb[NT];
  const u32x4 zero{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    rx[i] = rl[i] = rb[i] = zero;
    if (on && t0 + i < g.len) {
      const long long t = t0 + i;
      rl[i] = ld16(la + t * a.ls.t);
      rx[i] = ld16(x + t * a.xs.t);
      if constexpr (BETA) rb[i] = ld16(beta + t * a.bs.t);
    }
  }
  float e[NT][V], in[NT][V], l[V];
  State<T> h[V], z[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    l[c] = 0.f;
    z[c] = 0;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const Row<T> xv = unpack<T>(rx[i]), lv = unpack<T>(rl[i]), bv = unpack<T>(rb[i]);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      e[i][c] = decay_of<T>(lv.v[c]);
      float v = BETA ? bv.v[c] * xv.v[c] : xv.v[c];
      if constexpr (NORM) v *= unit_of(e[i][c]);
      in[i][c] = v;
      z[c] = advance<State<T>>(e[i][c], z[c], v);
      l[c] += lv.v[c];
    }
  }
  const int cl = g.slab * kSlab + lane;  // lane = channel
  const long long at = (long long)g.b * C + cl;
  const float first = a.h0 && cl < C ? a.h0[at] : 0.f;
  const auto self = [&]() {
    if (cl >= C) return 0.f;
    const int hh = cl / a.d, jj = cl % a.d;
    const T* px = static_cast<const T*>(a.x) + g.b * a.xs.b + hh * a.xs.h + jj;
    const T* pl = static_cast<const T*>(a.la) + g.b * a.ls.b + hh * a.ls.h + jj;
    const T* pb = BETA ? static_cast<const T*>(a.beta) + g.b * a.bs.b + hh * a.bs.h + jj : nullptr;
    State<T> run = first;
    for (long long t = 0; t < first_t; ++t) {
      const float ee = decay_of<T>(to_f32(pl[t * a.ls.t]));
      float v = to_f32(px[t * a.xs.t]);
      if constexpr (BETA) v *= to_f32(pb[t * a.bs.t]);
      if constexpr (NORM) v *= unit_of(ee);
      run = advance<State<T>>(ee, run, v);
    }
    return (float)run;
  };
  uint32_t* words = static_cast<uint32_t*>(a.ws) + (long long)g.chain * kWords;
  relay<T, WAVES>(mem, l, z, h, words, (long long)nslab * a.B * kWords, g.s, g.s == g.ntile - 1, first, polls,
                  cl < C ? a.h_T + at : nullptr, self);
  if (!on) return;
  T* o = static_cast<T*>(a.o) + g.b * a.os.b + hd * a.os.h + j0;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    Row<T> y;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      h[c] = advance<State<T>>(e[i][c], h[c], in[i][c]);
      y.v[c] = (float)h[c];
    }
    if (t0 + i < g.len) st16(o + (long long)(t0 + i) * a.os.t, pack<T>(y));
  }
}

// Empties the words of a call's tiles.
__global__ __launch_bounds__(256) void kda_glr_clear_kernel(u32x4* words, long long n) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i < n) words[i] = u32x4{kEmpty, kEmpty, kEmpty, kEmpty};
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
__global__ __launch_bounds__(64 * WAVES) void kda_glr_bwd_kernel(GlrArgs a, int nslab, int polls) {
  constexpr int V = kVec<T>, LPR = kLpr<T>, SUB = kSub<T>, RUN = WAVES * SUB * NT;
  __shared__ RelayMem<T, WAVES> mem;
  const GlrTile g(a, nslab, RUN);
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
  u32x4 rx[NT], rl[NT], rb[NT], rg[NT], ro[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    rx[i] = rl[i] = rb[i] = rg[i] = ro[i] = zero;
    if (on && t0 - i < g.len) {
      const long long t = t0 - i;
      rl[i] = ld16(la + t * a.ls.t);
      rg[i] = ld16(dO + t * a.dos.t);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (on && t0 - i < g.len) {
      const long long t = t0 - i;
      rx[i] = ld16(x + t * a.xs.t);
      if constexpr (BETA) rb[i] = ld16(beta + t * a.bs.t);
      if (t > 0) ro[i] = ld16(o + (t - 1) * a.os.t);
    }
  }
  float e[NT][V], l[V];
  State<T> mu[V], z[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    l[c] = 0.f;
    z[c] = 0;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const Row<T> lv = unpack<T>(rl[i]), gv = unpack<T>(rg[i]);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      e[i][c] = decay_of<T>(lv.v[c]);
      z[c] = advance<State<T>>(e[i][c], z[c] + gv.v[c], 0);
      l[c] += lv.v[c];
    }
  }
  const int cl = g.slab * kSlab + lane;  // lane = channel
  const long long at = (long long)g.b * C;
  const float first = a.dh_T && cl < C ? a.dh_T[at + cl] : 0.f;
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
  uint32_t* words = static_cast<uint32_t*>(a.ws) + (long long)g.chain * kWords;
  relay<T, WAVES>(mem, l, z, mu, words, (long long)nslab * a.B * kWords, g.s, g.s == g.ntile - 1, first, polls,
                  a.dh0 && cl < C ? a.dh0 + at + cl : nullptr, self);
  if (!on) return;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const long long t = t0 - i;
    const Row<T> xv = unpack<T>(rx[i]), bv = BETA ? unpack<T>(rb[i]) : ones<T>(), gv = unpack<T>(rg[i]);
    Row<T> before = unpack<T>(ro[i]), gx, gl, gb;
    if (t == 0 && a.h0) {
#pragma unroll
      for (int c = 0; c < V; ++c) before.v[c] = a.h0[at + c0 + c];
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      mu[c] += (State<T>)gv.v[c];
      const float lam = (float)mu[c], ee = e[i][c], al = slow(ee) ? 1.f + ee : ee;
      float n = 1.f, part = 0.f;
      if constexpr (NORM) {
        n = unit_of(ee);
        part = n > 0.f ? al * al / n * (bv.v[c] * xv.v[c]) : 0.f;
      }
      gx.v[c] = n * bv.v[c] * lam;
      gb.v[c] = n * xv.v[c] * lam;
      gl.v[c] = al == 0.f ? 0.f : (al * before.v[c] - part) * lam;
      mu[c] = advance<State<T>>(ee, mu[c], 0);
    }
    if (t >= g.len) continue;
    st16(dx + t * a.dxs.t, pack<T>(gx));
    st16(dla + t * a.dls.t, pack<T>(gl));
    if constexpr (BETA) st16(dbeta + t * a.dbs.t, pack<T>(gb));
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

#ifndef GLR_NT
#define GLR_NT 8
#endif
#ifndef GLR_NTB
#define GLR_NTB 4
#endif
#ifndef GLR_WAVES
#define GLR_WAVES 4
#endif
struct GlrPlan {
  int nslab, ntile;
  long long chains;
};
template <typename T>
GlrPlan glr_plan(int B, int H, int T_, int d, int nt, int waves) {
  GlrPlan p;
  p.nslab = (H * d + kSlab - 1) / kSlab;
  p.chains = (long long)p.nslab * B;
  const int run = waves * kSub<T> * nt;
  p.ntile = T_ > 0 ? (int)(((long long)T_ + run - 1) / run) : 1;
  return p;
}

template <typename T, int NT, int WAVES, bool BWD>
hipError_t glr_launch(const GlrArgs& a, int polls, hipStream_t stream) {
  const GlrPlan p = glr_plan<T>(a.B, a.H, a.T, a.d, NT, WAVES);
  if (p.ntile > 1) {
    const long long n = p.chains * p.ntile * kWords / 4;
    hipLaunchKernelGGL(kda_glr_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, static_cast<u32x4*>(a.ws), n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)(p.chains * p.ntile));
#define KDA_GLR(NO, BE)                                                                                                        \
  do {                                                                                                                         \
    if constexpr (BWD) hipLaunchKernelGGL((kda_glr_bwd_kernel<T, NT, WAVES, NO, BE>), grid, dim3(64 * WAVES), 0, stream, a, p.nslab, polls); \
    else hipLaunchKernelGGL((kda_glr_kernel<T, NT, WAVES, NO, BE>), grid, dim3(64 * WAVES), 0, stream, a, p.nslab, polls);     \
  } while (0)
  if (a.norm && a.beta) KDA_GLR(true, true);
  else if (a.norm) KDA_GLR(true, false);
  else if (a.beta) KDA_GLR(false, true);
  else KDA_GLR(false, false);
#undef KDA_GLR
  return hipGetLastError();
}

template <typename T>
hipError_t glr_step(const GlrArgs& a, hipStream_t stream) {
  const int nvec = a.H * a.d / kVec<T>;
  const dim3 grid((unsigned)(((long long)nvec * a.B + 255) / 256));
  hipLaunchKernelGGL((kda_glr_step_kernel<T>), grid, dim3(256), 0, stream, a, nvec);
  return hipGetLastError();
}

}  // namespace

size_t glr_ws_bytes(int B, int H, int T, int d, bool bf16_io, bool gradients, int) {
  const int nt = gradients ? GLR_NTB : GLR_NT;
  const GlrPlan p = bf16_io ? glr_plan<bf16>(B, H, T, d, nt, GLR_WAVES) : glr_plan<float>(B, H, T, d, nt, GLR_WAVES);
  return p.ntile > 1 ? (size_t)p.chains * p.ntile * kWords * sizeof(uint32_t) : 0;
}

hipError_t launch_glr(const GlrArgs& a, bool bf16_io, int polls, hipStream_t stream) {
  return bf16_io ? glr_launch<bf16, GLR_NT, GLR_WAVES, false>(a, polls, stream) : glr_launch<float, GLR_NT, GLR_WAVES, false>(a, polls, stream);
}

hipError_t launch_glr_backward(const GlrArgs& a, bool bf16_io, int polls, hipStream_t stream) {
  return bf16_io ? glr_launch<bf16, GLR_NTB, GLR_WAVES, true>(a, polls, stream) : glr_launch<float, GLR_NTB, GLR_WAVES, true>(a, polls, stream);
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
