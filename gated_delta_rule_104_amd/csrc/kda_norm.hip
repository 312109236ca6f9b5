// Root-mean-square norm of rows of d values, with the residual's addition in front and a
// gate behind, in the input's type or in 8 bits, and its gradients:
//     s = x + residual (rounded to its type),  r = (mean s^2 + eps)^-1/2,  y = s r w g(gate)
//     dn = dy w g,  ds = r (dn - s r mean(dn s r)) + ds_out,  dw = sum dy s r g,  dgate = dy s r w g'
//
// Every value is read and written once, so HBM bounds long rows; short ones with a gate are bound by vector instructions (an
// exponential and a reciprocal a value, and a row's addresses in every lane for few values).  A row stays in the
// registers of the lanes that share it: 8 to 64 lanes of a wave for short rows, whose sums
// then take lane exchanges only, and 4 or 16 waves for long ones, whose sums meet in LDS.
// Sums are fp32 in a fixed order (lanes by a butterfly, waves in order), results rounded once.
//
// 32K rows of 4096 bf16 values: with a residual in front and e4m3 blocks behind 143-146 us for 943 MB (in rows 149-151, fp32
// 274 and 280 for 1.75 GB), gradients 184-195 us for 1.07 GB (fp32 390): 5.5-6.5 TB/s (a large copy reaches 5.4).  1M rows of
// 128 with a gate 142 us for 805 MB, 1268 vector instructions a wave or 135 us of the SIMDs' cycles; in e4m3 blocks 166 and in
// rows 196 us for 675 MB; gradients 252-258 for 1.34 GB.  256 rows of 4096 with
// e4m3 rows: 10.6 us, of which the kernel, one chain of load, two sums and store, 5.9 and the call the rest.
#include "kda_ops.hpp"
#include "kda_vec.hpp"

namespace kda {

namespace {

constexpr int DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140;

// Over a group of 4, 8, 16, 32 or 64 neighbouring lanes; all of them get the same bits.  (In a
// row of 16 lanes a mirror reaches the other half, whose lanes are equal by then.)
template <int LANES, bool MAX>
__device__ __forceinline__ float across(float v) {
  const auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  v = join(v, dpp<DPP_QUAD_SWAP1>(v));
  v = join(v, dpp<DPP_QUAD_SWAP2>(v));
  if constexpr (LANES >= 8) v = join(v, dpp<DPP_HALF_MIRROR>(v));
  if constexpr (LANES >= 16) v = join(v, dpp<DPP_MIRROR>(v));
  if constexpr (LANES >= 32) v = join(v, __shfl_xor(v, 16));
  if constexpr (LANES >= 64) v = join(v, __shfl_xor(v, 32));
  return v;
}

// NR values of as many rows, over the lanes and waves that share a row.
template <int LANES, int WAVES, int NR, bool MAX = false>
__device__ __forceinline__ void row_reduce(float (&v)[NR], float* red) {
#pragma unroll
  for (int j = 0; j < NR; ++j) v[j] = across<LANES, MAX>(v[j]);
  if constexpr (WAVES > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // (red may still be read from the sum before)
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int j = 0; j < NR; ++j) red[j * WAVES + w] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      v[j] = red[j * WAVES];
#pragma unroll
      for (int u = 1; u < WAVES; ++u) v[j] = MAX ? fmaxf(v[j], red[j * WAVES + u]) : v[j] + red[j * WAVES + u];
    }
  }
}

// The gate's factor g(z) and its derivative, from sigma(z) and 1 - sigma(z) = e^-z sigma(z), which has all its
// digits that way.  Below -88 or so e^-z is infinite and sigma zero; z is held to finite numbers where it meets
// them, and e^-z to 2^126.  (sigma of a NaN is one.)  bf16's exponent is rounded, |z| 2^-24 of sigma; fp32's has that taken back.
template <typename T>
struct Gate {
  float g, dg;
  __device__ __forceinline__ Gate(float z, bool silu) {
    constexpr float c = -1.44269504088896340736f, c_low = -1.92596299e-8f;  // -log2(e) in two floats
    constexpr float most = 3.402823466e38f;
    float e;
    if constexpr (sizeof(T) == 2) {
      e = __builtin_amdgcn_exp2f(c * z);
    } else {  // the exponent's own rounding is taken back
      const float y = __builtin_amdgcn_fmed3f(z, -128.f, 128.f), t = c * y, r = fmaf(c_low, y, fmaf(c, y, -t));
      e = z == z ? __builtin_amdgcn_exp2f(t) * fmaf(r, 0.69314718055994530942f, 1.f) : z;
    }
    const float s = __builtin_amdgcn_rcpf(1.f + e), one_less = fminf(e, 0x1p126f) * s;
    // (-inf, the largest bits but for negative NaN, to the lowest number: one instruction less than a maximum)
    const float low = __uint_as_float(min(__float_as_uint(z), 0xff7fffffu));
    g = silu ? low * s : s;
    dg = silu ? s * fmaf(__builtin_amdgcn_fmed3f(z, -most, most), one_less, 1.f) : s * one_less;
  }
};

// Offsets of a row in each tensor: its place (i0, i1, i2) in the dimensions that are left
// after neighbouring ones have been joined.
struct Place {
  int i[3];
  __device__ __forceinline__ Place(int row, int n1, int n2) {
    i[2] = n2 > 1 ? row % n2 : 0;
    const int q = n2 > 1 ? row / n2 : row;
    i[1] = n1 > 1 ? q % n1 : 0;
    i[0] = n1 > 1 ? q / n1 : q;
  }
  __device__ __forceinline__ long long at(const Str3& s) const { return i[0] * s.b + i[1] * s.h + i[2] * s.t; }
};

template <bool E4M3>
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    const int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  } else {
    return ((uint32_t)(int)rintf(a) & 255u) | (((uint32_t)(int)rintf(b) & 255u) << 8) |
           (((uint32_t)(int)rintf(c) & 255u) << 16) | ((uint32_t)(int)rintf(d) << 24);
  }
}

// 8 or 4 values of a lane in 8 bits.
template <typename T>
__device__ __forceinline__ void store8(unsigned char* p, const Row<T>& y, float scale, bool e4m3) {
  uint32_t w[kVec<T> / 4];
#pragma unroll
  for (int i = 0; i < kVec<T> / 4; ++i) {
    const float a = y.v[4 * i] * scale, b = y.v[4 * i + 1] * scale, c = y.v[4 * i + 2] * scale, d = y.v[4 * i + 3] * scale;
    w[i] = e4m3 ? quant4<true>(a, b, c, d) : quant4<false>(a, b, c, d);
  }
  if constexpr (kVec<T> == 8) {
    *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
  } else {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

template <typename T>
__device__ __forceinline__ float most(const Row<T>& y, bool* bad) {
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < kVec<T>; ++c) {
    m = fmaxf(m, fabsf(y.v[c]));
    *bad |= !(fabsf(y.v[c]) < __builtin_inff());
  }
  return m;
}

// NR groups of rows per block; a row is shared by LANES lanes of WAVES waves, NV vectors of 16
// bytes each (vector i * LANES * WAVES + lane: neighbouring lanes read neighbouring 16 bytes).
template <typename T, int LANES, int WAVES, int NV, int NR, bool BITS8>
__global__ __launch_bounds__(WAVES > 4 ? 64 * WAVES : 256) void kda_norm_kernel(NormArgs a) {
  constexpr int V = kVec<T>, THREADS = WAVES > 4 ? 64 * WAVES : 256;
  constexpr int PER = LANES * WAVES, GROUPS = THREADS / PER;  // lanes of a row, rows at once
  __shared__ float red[WAVES > 1 ? NR * WAVES : 1];
  const int lane = threadIdx.x % PER;
  const int row0 = (int)blockIdx.x * (GROUPS * NR) + threadIdx.x / PER;
  const int nvec = a.d / V;
  u32x4 xr[NR][NV], rr[NR][NV], gr[NR][NV];
  bool have[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int row = row0 + j * GROUPS;
    have[j] = row < a.rows;
    const Place p(have[j] ? row : 0, a.n1, a.n2);
    const T* x = static_cast<const T*>(a.x) + p.at(a.xs);
    const T* r = a.residual ? static_cast<const T*>(a.residual) + p.at(a.rs) : nullptr;
    const T* g = a.gate ? static_cast<const T*>(a.gate) + p.at(a.gs) : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * PER + lane;
      const bool on = have[j] && vec < nvec;
      xr[j][i] = rr[j][i] = gr[j][i] = u32x4{0u, 0u, 0u, 0u};
      if (on) xr[j][i] = ld_once(x + vec * V);
      if (on && r) rr[j][i] = ld_once(r + vec * V);
      if (on && g) gr[j][i] = ld_once(g + vec * V);
    }
  }
  float sum[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    sum[j] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Row<T> s = unpack<T>(xr[j][i]);
      if (a.residual) {
        const Row<T> r = unpack<T>(rr[j][i]);
#pragma unroll
        for (int c = 0; c < V; ++c) s.v[c] += r.v[c];
        // (what is normalised is what later layers and the gradients read)
        xr[j][i] = pack<T>(s);
        s = unpack<T>(xr[j][i]);
      }
#pragma unroll
      for (int c = 0; c < V; ++c) sum[j] = fmaf(s.v[c], s.v[c], sum[j]);
    }
  }
  row_reduce<LANES, WAVES, NR>(sum, red);
  // Rows in 8 bits without a gate leave their factor to their scale: its rounding would put quotients value / largest
  // that lie on a border between two 8-bit values (3 or 4 in 10,000 of rows of 4096 in bf16) to either side of it.
  const bool later = BITS8 && !a.blocks && !a.gate;
  float scale[NR], top[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    scale[j] = 1.f / sqrtf(sum[j] * a.inv_d + a.eps);
    top[j] = 0.f;
  }
  const auto value = [&](int j, int i, const T* w) {
    Row<T> y = unpack<T>(xr[j][i]);
    const int vec = i * PER + lane;
    if (w) {  // (of bf16 values this product is exact)
      const Row<T> k = unpack<T>(vec < nvec ? ld16(w + vec * V) : u32x4{0u, 0u, 0u, 0u});
#pragma unroll
      for (int c = 0; c < V; ++c) y.v[c] *= k.v[c];
    }
    if (!later) {
#pragma unroll
      for (int c = 0; c < V; ++c) y.v[c] *= scale[j];
    }
    if (a.gate) {
      const Row<T> g = unpack<T>(gr[j][i]);
#pragma unroll
      for (int c = 0; c < V; ++c) y.v[c] *= Gate<T>(g.v[c], a.silu).g;
    }
    return y;
  };
  Row<T> keep[BITS8 ? NR : 1][BITS8 ? NV : 1];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const Place p(have[j] ? row0 + j * GROUPS : 0, a.n1, a.n2);
    const T* w = a.w ? static_cast<const T*>(a.w) + p.at(a.ws) : nullptr;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * PER + lane;
      const bool on = have[j] && vec < nvec;
      if (a.s && on) store_by(static_cast<T*>(a.s) + p.at(a.ss) + vec * V, xr[j][i], a.lines);
      Row<T> y = value(j, i, w);
      if constexpr (!BITS8) {
        if (on) store_by(static_cast<T*>(a.y) + p.at(a.ys) + vec * V, pack<T>(y), a.lines);
      } else {
        // (lanes behind the row's end have y = 0 r, NaN where the row's factor is not finite, as it is for the others)
        unsigned char* out = static_cast<unsigned char*>(a.y) + p.at(a.ys) + vec * V;
        if (a.blocks) {
          bool off = false;
          float m = most<T>(y, &off);
          m = across<kVec<T> == 8 ? 4 : 8, true>(off ? __builtin_inff() : m);
          const bool none = m == __builtin_inff();
          // m = f 2^ex with f in [1, 2): 127 = 1.984375 2^6, 448 = 1.75 2^8
          const uint32_t mb = __float_as_uint(m), frac = mb & 0x7fffffu;
          const int ex = (int)(mb >> 23) - 127;
          int e = a.e4m3 ? ex - 8 + (frac > 0x600000u) : ex - 6 + (frac > 0x7e0000u);
          e = e < -126 ? -126 : e;
          if (on) {
            if (none) y = unpack<T>(u32x4{0u, 0u, 0u, 0u});
            store8<T>(out, y, __uint_as_float((uint32_t)(127 - e) << 23), a.e4m3);
            if ((vec * V & 31) == 0)
              static_cast<unsigned char*>(a.scales)[p.at(a.cs) + (vec * V >> 5)] = none ? 255 : (unsigned char)(e + 127);
          }
        } else {
          keep[j][i] = y;
          top[j] = fmaxf(top[j], most<T>(y, &bad));
        }
      }
    }
    if (bad) top[j] = __builtin_inff();
  }
  if constexpr (BITS8) {
    if (a.blocks) return;
    row_reduce<LANES, WAVES, NR, true>(top, red);
    const float limit = a.e4m3 ? 448.f : 127.f;
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const Place p(have[j] ? row0 + j * GROUPS : 0, a.n1, a.n2);
      // (a row of zeros, or one so small that its scale would not be a normal number, takes the smallest
      // scale; its values are then rounded to multiples of that, like a block's)
      const float most_y = later ? top[j] * scale[j] : top[j], sc_y = most_y / limit;
      const bool none = !(most_y < __builtin_inff());
      const float sc = none ? __builtin_nanf("") : fmaxf(sc_y, 1.17549435e-38f);
      // y / sc; without the factor v limit / top, as v (limit 2^-ex) / m with top = m 2^ex, of which bf16 rounds the
      // quotient alone
      float m = sc, by = 1.f;
      if (later) {
        const bool least = sc_y < 1.17549435e-38f;
        const int ex = max(__builtin_amdgcn_frexp_expf(top[j]), -100);
        m = least ? 0x1p-126f : ldexpf(top[j], -ex);
        by = least ? scale[j] : ldexpf(limit, -ex);
      }
      const float inv = __builtin_amdgcn_rcpf(m);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int vec = i * PER + lane;
        if (!have[j] || vec >= nvec) continue;
        Row<T>& y = keep[j][i];
#pragma unroll
        for (int c = 0; c < V; ++c) {  // a quotient, what it is off by taken back once
          const float v = y.v[c] * by, q = v * inv;
          y.v[c] = none ? 0.f : fmaf(fmaf(-q, m, v), inv, q);
        }
        store8<T>(static_cast<unsigned char*>(a.y) + p.at(a.ys) + vec * V, y, 1.f, a.e4m3);
      }
      if (have[j] && lane == 0) static_cast<float*>(a.scales)[p.at(a.cs)] = sc;
    }
  }
}

// NV vectors of a row, zeros outside.
template <typename T, int PER, int NV, bool ONCE>
__device__ __forceinline__ void load_row(u32x4 (&r)[NV], const T* p, int lane, int nvec, bool on) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = i * PER + lane;
    r[i] = u32x4{0u, 0u, 0u, 0u};
    if (on && vec < nvec) r[i] = ONCE ? ld_once(p + vec * kVec<T>) : ld16(p + vec * kVec<T>);
  }
}

// Gradients.  A block walks rows part, part + nparts, ... of one weight row's rows, so that a lane's columns
// stay the same and dw is summed in registers; one partial row of sums per block goes to the workspace,
// and a second kernel adds the partials in a fixed order.  AGAIN: rows too long for the registers are read
// a second time, from the caches.
template <typename T, int LANES, int WAVES, int NV, bool GATE, bool AGAIN>
__global__ __launch_bounds__(WAVES > 4 ? 64 * WAVES : 256) void kda_norm_bwd_kernel(NormArgs a) {
  constexpr int V = kVec<T>, THREADS = WAVES > 4 ? 64 * WAVES : 256;
  constexpr int PER = LANES * WAVES, GROUPS = THREADS / PER;
  __shared__ float red[WAVES > 1 ? 2 * WAVES : 1];
  __shared__ float cols[GROUPS > 1 ? THREADS * NV * V : 1];
  const int lane = threadIdx.x % PER, group = threadIdx.x / PER;
  const int part = blockIdx.x % a.nparts, hw = blockIdx.x / a.nparts;
  const int nvec = a.d / V;
  const int rows = a.rows / a.w_heads;  // of this row of the weight
  u32x4 wr[NV];
  float dw[NV][V];
  if (a.w) {
    load_row<T, PER, NV, false>(wr, static_cast<const T*>(a.w) + (long long)hw * a.d, lane, nvec, true);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) wr[i] = sizeof(T) == 2 ? u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}
                                                       : u32x4{0x3f800000u, 0x3f800000u, 0x3f800000u, 0x3f800000u};  // ones
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < V; ++c) dw[i][c] = 0.f;
  for (long long base = (long long)part * GROUPS; base < rows; base += (long long)a.nparts * GROUPS) {
    const long long row = base + group;
    const bool have = row < rows;
    const Place p(have ? (int)row : 0, a.n1, a.n2);
    const T* s_p = static_cast<const T*>(a.x) + hw * a.hx + p.at(a.xs);
    const T* y_p = static_cast<const T*>(a.dy) + hw * a.hdy + p.at(a.dys);
    const T* g_p = GATE ? static_cast<const T*>(a.gate) + hw * a.hg + p.at(a.gs) : nullptr;
    const T* d_p = a.ds ? static_cast<const T*>(a.ds) + hw * a.hds + p.at(a.dss) : nullptr;
    u32x4 sr[NV], yr[NV], gr[NV], dr[NV];
    load_row<T, PER, NV, !AGAIN>(sr, s_p, lane, nvec, have);
    load_row<T, PER, NV, !AGAIN>(yr, y_p, lane, nvec, have);
    if constexpr (GATE) load_row<T, PER, NV, !AGAIN>(gr, g_p, lane, nvec, have);
    if constexpr (!AGAIN) load_row<T, PER, NV, !AGAIN>(dr, d_p, lane, nvec, have && a.ds);
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Row<T> s = unpack<T>(sr[i]), dy = unpack<T>(yr[i]), w = unpack<T>(wr[i]);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        float dn = dy.v[c] * w.v[c];
        if constexpr (GATE) dn *= Gate<T>(unpack<T>(gr[i]).v[c], a.silu).g;
        sum[0] = fmaf(s.v[c], s.v[c], sum[0]);
        sum[1] = fmaf(dn, s.v[c], sum[1]);
      }
    }
    row_reduce<LANES, WAVES, 2>(sum, red);
    const float r = have ? 1.f / sqrtf(sum[0] * a.inv_d + a.eps) : 0.f;
    const float back = r * (r * (r * (sum[1] * a.inv_d)));
    if constexpr (AGAIN) {
      asm volatile("" ::: "memory");
      load_row<T, PER, NV, true>(sr, s_p, lane, nvec, have);
      load_row<T, PER, NV, true>(yr, y_p, lane, nvec, have);
      if constexpr (GATE) load_row<T, PER, NV, true>(gr, g_p, lane, nvec, have);
      load_row<T, PER, NV, true>(dr, d_p, lane, nvec, have && a.ds);
    } else {
      // (else the fp32 forms, twice the registers, would be kept from the sums to the gradients)
      forget(sr);
      forget(yr);
      if constexpr (GATE && NV > 1) forget(gr);  // (a single vector's gates are kept)
    }
    forget(wr);
    T* dx_p = static_cast<T*>(a.dx) + hw * a.hdx + p.at(a.dxs);
    T* dz_p = GATE ? static_cast<T*>(a.dgate) + hw * a.hdg + p.at(a.dgs) : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * PER + lane;
      const Row<T> s = unpack<T>(sr[i]), dy = unpack<T>(yr[i]), w = unpack<T>(wr[i]);
      Row<T> dx = unpack<T>(dr[i]), dz;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float n = s.v[c] * r, yn = dy.v[c] * n;
        if constexpr (GATE) {
          const Gate<T> f(unpack<T>(gr[i]).v[c], a.silu);
          dx.v[c] += r * (dy.v[c] * w.v[c] * f.g) - s.v[c] * back;
          dz.v[c] = yn * w.v[c] * f.dg;
          dw[i][c] = fmaf(yn, f.g, dw[i][c]);
        } else {
          dx.v[c] += r * (dy.v[c] * w.v[c]) - s.v[c] * back;
          dw[i][c] += yn;
        }
      }
      if (!have || vec >= nvec) continue;
      store_by(dx_p + vec * V, pack<T>(dx), a.lines);
      if constexpr (GATE) store_by(dz_p + vec * V, pack<T>(dz), a.lines);
    }
  }
  if (!a.dw) return;
  float* out = a.scratch + ((size_t)part * a.w_heads + hw) * a.d;
  if constexpr (GROUPS > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < V; ++c) cols[(group * NV * PER + i * PER + lane) * V + c] = dw[i][c];
    __syncthreads();
    for (int k = threadIdx.x; k < a.d; k += THREADS) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < GROUPS; ++g) s += cols[g * NV * PER * V + k];
      out[k] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * PER + lane;
      if (vec >= nvec) continue;
#pragma unroll
      for (int c = 0; c < V; c += 4) *reinterpret_cast<f32x4*>(out + vec * V + c) = f32x4{dw[i][c], dw[i][c + 1], dw[i][c + 2], dw[i][c + 3]};
    }
  }
}

// dw[k]: the sum of the partials, 32 interleaved runs of them per column, joined in a fixed order.
template <typename T>
__global__ __launch_bounds__(1024) void kda_norm_dw_kernel(const float* ws, T* dw, int n, int nparts) {
  __shared__ float red[32][32];
  const int l = threadIdx.x & 31, u = threadIdx.x >> 5, k = blockIdx.x * 32 + l;
  float s = 0.f;
  if (k < n) {
#pragma unroll 8
    for (int p = u; p < nparts; p += 32) s += ws[(size_t)p * n + k];
  }
  red[u][l] = s;
  __syncthreads();
  if (u == 0 && k < n) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += red[i][l];
    dw[k] = from_f32<T>(s);
  }
}

// Puts the dimensions in the order of the output (the first of `all`) in memory, joins neighbouring ones whose rows
// lie evenly in every tensor, and drops those of size 1: blocks then walk memory in order (heads of a token-major
// tensor 193 -> 161 us), a row's place takes few divisions, and single tokens of many sequences fill whole blocks.
template <int N>
void join_dims(NormArgs& a, Str3* const (&all)[N], int B, int H, int T) {
  struct Dim {
    long long n = 1, st[N] = {};
  } in[3], out[3];
  int k = 0;
  for (int i = 0; i < 3; ++i) {
    Dim d;
    d.n = i == 0 ? B : (i == 1 ? H : T);
    if (d.n == 1) continue;
    for (int j = 0; j < N; ++j) d.st[j] = i == 0 ? all[j]->b : (i == 1 ? all[j]->h : all[j]->t);
    int at = k++;
    for (; at > 0 && in[at - 1].st[0] < d.st[0]; --at) in[at] = in[at - 1];
    in[at] = d;
  }
  int m = 0;
  for (int i = 0; i < k; ++i) {
    Dim d = in[i];
    bool even = m > 0;
    for (int j = 0; j < N; ++j) even = even && out[m - 1].st[j] == d.n * d.st[j];
    if (even) d.n *= out[--m].n;
    out[m++] = d;
  }
  const Dim none;
  const Dim &d0 = m > 2 ? out[0] : none, &d1 = m > 1 ? out[m - 2] : none, &d2 = m > 0 ? out[m - 1] : none;
  for (int j = 0; j < N; ++j) *all[j] = Str3{d0.st[j], d1.st[j], d2.st[j]};
  a.n1 = (int)d1.n;
  a.n2 = (int)d2.n;
}

// Calls f(lanes, waves, vectors a lane, rows at once) with the shape for rows of nvec vectors, as
// integral constants.  Rows of up to 64 vectors stay inside a wave, and a lane reads from four of
// them at once so that its loads cover the latency; longer ones give a lane up to 8 vectors.
template <int N> struct Int { static constexpr int value = N; };
template <typename T, typename F>
auto with_shape(int d, F f) {
  const int nvec = d / kVec<T>;
  if (nvec <= 8) return f(Int<8>(), Int<1>(), Int<1>(), Int<4>());
  if (nvec <= 16) return f(Int<16>(), Int<1>(), Int<1>(), Int<4>());
  if (nvec <= 32) return f(Int<32>(), Int<1>(), Int<1>(), Int<4>());
  if (nvec <= 64) return f(Int<64>(), Int<1>(), Int<1>(), Int<4>());
  if (nvec <= 128) return f(Int<64>(), Int<1>(), Int<2>(), Int<2>());
  if (nvec <= 256) return f(Int<64>(), Int<4>(), Int<1>(), Int<2>());
  if (nvec <= 512) return f(Int<64>(), Int<4>(), Int<2>(), Int<1>());
  if (nvec <= 1024) return f(Int<64>(), Int<4>(), Int<4>(), Int<1>());
  if (nvec <= 2048) return f(Int<64>(), Int<16>(), Int<2>(), Int<1>());
  if (sizeof(T) == 2 || nvec <= 4096) return f(Int<64>(), Int<16>(), Int<4>(), Int<1>());
  return f(Int<64>(), Int<16>(), Int<sizeof(T) == 2 ? 4 : 8>(), Int<1>());
}

template <typename T, bool BITS8>
hipError_t norm_fwd(const NormArgs& a, hipStream_t stream) {
  return with_shape<T>(a.d, [&](auto l, auto w, auto nv, auto nr) {
    constexpr int LANES = decltype(l)::value, WAVES = decltype(w)::value, NV = decltype(nv)::value, NR = decltype(nr)::value;
    constexpr int THREADS = WAVES > 4 ? 64 * WAVES : 256, per = THREADS / (LANES * WAVES) * NR;
    hipLaunchKernelGGL((kda_norm_kernel<T, LANES, WAVES, NV, NR, BITS8>), dim3((unsigned)((a.rows + per - 1) / per)),
                       dim3(THREADS), 0, stream, a);
    return hipGetLastError();
  });
}

// The gradients' shapes: one row per group of lanes, fewer vectors per lane.
template <typename T, typename F>
auto with_bwd_shape(int d, F f) {
  const int nvec = d / kVec<T>;
  if (nvec <= 8) return f(Int<8>(), Int<1>(), Int<1>());
  if (nvec <= 16) return f(Int<16>(), Int<1>(), Int<1>());
  if (nvec <= 32) return f(Int<32>(), Int<1>(), Int<1>());
  if (nvec <= 64) return f(Int<64>(), Int<1>(), Int<1>());
  if (nvec <= 128) return f(Int<64>(), Int<1>(), Int<2>());
  if (nvec <= 256) return f(Int<64>(), Int<4>(), Int<1>());
  if (nvec <= 512) return f(Int<64>(), Int<4>(), Int<2>());
  if (nvec <= 1024) return f(Int<64>(), Int<8>(), Int<2>());
  if (nvec <= 2048) return f(Int<64>(), Int<16>(), Int<2>());
  if (sizeof(T) == 2 || nvec <= 4096) return f(Int<64>(), Int<16>(), Int<4>());
  return f(Int<64>(), Int<16>(), Int<sizeof(T) == 2 ? 4 : 8>());
}

template <typename T>
hipError_t norm_bwd(const NormArgs& a, hipStream_t stream) {
  const hipError_t e = with_bwd_shape<T>(a.d, [&](auto l, auto w, auto nv) {
    constexpr int LANES = decltype(l)::value, WAVES = decltype(w)::value, NV = decltype(nv)::value;
    constexpr int THREADS = WAVES > 4 ? 64 * WAVES : 256;
    const dim3 grid((unsigned)(a.nparts * a.w_heads));
    if (a.gate) hipLaunchKernelGGL((kda_norm_bwd_kernel<T, LANES, WAVES, NV, true, (NV > 2)>), grid, dim3(THREADS), 0, stream, a);
    else hipLaunchKernelGGL((kda_norm_bwd_kernel<T, LANES, WAVES, NV, false, (NV > 2)>), grid, dim3(THREADS), 0, stream, a);
    return hipGetLastError();
  });
  if (e != hipSuccess || !a.dw) return e;
  const int n = a.w_heads * a.d;
  hipLaunchKernelGGL((kda_norm_dw_kernel<T>), dim3((unsigned)((n + 31) / 32)), dim3(1024), 0, stream, a.scratch,
                     static_cast<T*>(a.dw), n, a.nparts);
  return hipGetLastError();
}

}  // namespace

bool norm_fits(int rows, int d, bool bf16_io) {
  const auto fits = [&](auto l, auto w, auto, auto nr) {
    constexpr int LANES = decltype(l)::value, WAVES = decltype(w)::value, THREADS = WAVES > 4 ? 64 * WAVES : 256;
    constexpr int per = THREADS / (LANES * WAVES) * decltype(nr)::value;
    return launchable(((long long)rows + per - 1) / per, THREADS);
  };
  return bf16_io ? with_shape<bf16>(d, fits) : with_shape<float>(d, fits);
}
bool norm_backward_fits(int nparts, int d, int w_heads, bool weight, bool bf16_io) {
  const auto fits = [&](auto, auto w, auto) {
    constexpr int WAVES = decltype(w)::value, THREADS = WAVES > 4 ? 64 * WAVES : 256;
    return launchable((long long)nparts * w_heads, THREADS) && (!weight || launchable(((long long)w_heads * d + 31) / 32, 1024));
  };
  return bf16_io ? with_bwd_shape<bf16>(d, fits) : with_bwd_shape<float>(d, fits);
}

// Blocks per weight row: three of 256 threads a compute unit, two of 512 or one of 1024 (32K rows of 4096 bf16 values,
// blocks of 256: 262, 178, 182-186, 195 us with one to four; heads of 128 with a gate 437, 280, 257, 269), no more than there
// are units of rows.
int norm_parts(int rows, int d, int w_heads, bool bf16_io, int cus) {
  const auto parts = [&](auto l, auto w, auto) {
    constexpr int LANES = decltype(l)::value, WAVES = decltype(w)::value;
    constexpr int THREADS = WAVES > 4 ? 64 * WAVES : 256, per = THREADS / (LANES * WAVES);
    const int own = rows / w_heads;
    int most = (THREADS > 512 ? 1 : (THREADS > 256 ? 2 : 3)) * cus / w_heads;
    most = most < 1 ? 1 : most;
    const int units = (own + per - 1) / per;
    return units < most ? (units < 1 ? 1 : units) : most;
  };
  return bf16_io ? with_bwd_shape<bf16>(d, parts) : with_bwd_shape<float>(d, parts);
}

hipError_t launch_norm(NormArgs a, int B, int H, int T, bool bits8, bool bf16_io, hipStream_t stream) {
  const long long es = bf16_io ? 2 : 4;
  // (8-bit rows go through the caches in any case: 143 us against 154 for 32K rows of 4096)
  a.lines = (bits8 || whole_lines(a.y, a.ys, a.rows, a.d * es, es)) && (!a.s || whole_lines(a.s, a.ss, a.rows, a.d * es, es));
  Str3* const all[] = {&a.ys, &a.xs, &a.rs, &a.gs, &a.ss, &a.ws, &a.cs};
  join_dims(a, all, B, H, T);
  if (bits8) return bf16_io ? norm_fwd<bf16, true>(a, stream) : norm_fwd<float, true>(a, stream);
  return bf16_io ? norm_fwd<bf16, false>(a, stream) : norm_fwd<float, false>(a, stream);
}

hipError_t launch_norm_backward(NormArgs a, int B, int H, int T, bool bf16_io, hipStream_t stream) {
  const long long es = bf16_io ? 2 : 4;
  // (rows of a wave or less; longer ones are slower that way: 173 us against 182 for 32K rows of 4096)
  a.lines = a.d * es <= 1024 && whole_lines(a.dx, a.dxs, a.rows, a.d * es, es) &&
            (!a.dgate || whole_lines(a.dgate, a.dgs, a.rows, a.d * es, es));
  Str3* const all[] = {&a.dxs, &a.xs, &a.gs, &a.dys, &a.dss, &a.dgs};
  if (a.w_heads > 1) {  // a block stays with one head
    a.hx = a.xs.h; a.hg = a.gs.h; a.hdy = a.dys.h; a.hds = a.dss.h; a.hdx = a.dxs.h; a.hdg = a.dgs.h;
    H = 1;
    for (Str3* s : all) s->h = 0;
  }
  join_dims(a, all, B, H, T);
  return bf16_io ? norm_bwd<bf16>(a, stream) : norm_bwd<float>(a, stream);
}

}  // namespace kda
