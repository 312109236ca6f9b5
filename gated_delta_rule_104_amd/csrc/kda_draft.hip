// Drafted tokens: how many the target's probabilities accept, the token behind them, and the
// states that go with them.
//
// Token j is accepted while u_j q_j(tok_j) < p_j(tok_j).  At the first refusal the next token is drawn
// from max(p_j - q_j, 0), behind the last accepted one from p: the smallest i whose running sum is above
// u times the whole one.  Products of fp32 numbers are exact in fp64, and sums are fp64, so that the
// choice is the one of the exact sums but for a threshold within about 1e-14 of a border.
//
// One row of V probabilities (two after a refusal) is all that has to be read, and HBM bounds that.
// A row is cut into chunks that fill the chip with few sequences too: one launch adds every chunk up,
// a second one finds the chunk that holds the threshold and walks it alone.
#include "kda_ops.hpp"
#include "kda_vec.hpp"

namespace kda {

namespace {

constexpr int kChunk = 8192;  // probabilities of a row per workgroup

struct Choice {
  int accepted, count, token;  // token: the refused one
};

// Every wave finds out for itself how far sequence n is accepted.
template <typename T>
__device__ __forceinline__ Choice accept(const VerifyArgs& a, int n) {
  const int lane = lane_id();
  int count = a.K;
  if (a.counts) {
    count = a.counts[n];
    count = count < 0 ? 0 : (count > a.K ? a.K : count);
  }
  Choice c{count, count, -1};
  for (int j0 = 0; j0 < count; j0 += 64) {
    const int j = j0 + lane;
    bool ok = true;
    int tok = -1;
    if (j < count) {
      tok = a.tokens[(long long)n * a.K + j];
      ok = false;
      if (tok >= 0 && tok < a.V) {
        const double p = (double)to_f32(static_cast<const T*>(a.p)[n * a.pn + j * a.pt + tok]);
        const double q = a.q ? (double)to_f32(static_cast<const T*>(a.q)[n * a.qn + j * a.qt + tok]) : 1.0;
        ok = (double)a.u[(long long)n * (a.K + 1) + j] * q < p;
      }
    }
    const unsigned long long no = __ballot(!ok);
    if (no) {
      const int first = __ffsll((unsigned long long)no) - 1;
      c.accepted = j0 + first;
      c.token = __shfl(tok, first);
      break;
    }
  }
  return c;
}

// The row that sequence n draws from, V probabilities of any alignment.
template <typename T>
struct Rows {
  const T* p;
  const T* q;  // after a refusal
  int token;   // after a refusal without q: the token whose q is one, else -1
  __device__ __forceinline__ Rows(const VerifyArgs& a, int n, const Choice& c) {
    const bool refused = c.accepted < c.count;
    p = static_cast<const T*>(a.p) + n * a.pn + c.accepted * a.pt;
    q = refused && a.q ? static_cast<const T*>(a.q) + n * a.qn + c.accepted * a.qt : nullptr;
    token = refused && !a.q ? c.token : -1;
  }
};

// 16 bytes at any element's address.
template <typename T>
__device__ __forceinline__ Row<T> load_any(const T* p) {
  u32x4 w;
  __builtin_memcpy(&w, p, 16);
  return unpack<T>(w);
}

// A lane's vector of both rows: what is left of p behind q, and p, in fp64; NaN and what is negative
// count as no mass.
template <typename T>
__device__ __forceinline__ void masses(const Rows<T>& r, int i0, int end, double* w, double* whole) {
  constexpr int V = kVec<T>;
  Row<T> p, q;
  if (i0 + V <= end) {
    p = load_any(r.p + i0);
    if (r.q) q = load_any(r.q + i0);
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      p.v[c] = i0 + c < end ? to_f32(r.p[i0 + c]) : 0.f;
      q.v[c] = r.q && i0 + c < end ? to_f32(r.q[i0 + c]) : 0.f;
    }
  }
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const double x = (double)p.v[c];
    double y = r.q ? (double)q.v[c] : 0.0;
    if (i0 + c == r.token) y = 1.0;
    whole[c] = x > 0.0 ? x : 0.0;
    w[c] = x > y ? x - y : 0.0;
    if (!(y > 0.0)) w[c] = whole[c];
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// The sums of every chunk: what is left, and the whole.  The first chunk's block writes how far the
// sequence is accepted.
template <typename T>
__global__ __launch_bounds__(256) void kda_verify_sum_kernel(VerifyArgs a, int nchunk) {
  __shared__ double red[2][4];
  const int n = blockIdx.x / nchunk, chunk = blockIdx.x % nchunk;
  const Choice choice = accept<T>(a, n);
  if (chunk == 0 && threadIdx.x == 0) a.accepted[n] = choice.accepted;
  const Rows<T> r(a, n, choice);
  const int c0 = chunk * kChunk, end = min(c0 + kChunk, a.V);
  double s = 0.0, whole = 0.0;
  constexpr int V = kVec<T>;
#pragma unroll 4
  for (int i = c0 + (int)threadIdx.x * V; i < end; i += 256 * V) {
    double w[V], z[V];
    masses<T>(r, i, end, w, z);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      s += w[c];
      whole += z[c];
    }
  }
  s = wave_sum(s);
  whole = wave_sum(whole);
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = s;
    red[1][threadIdx.x >> 6] = whole;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const double* v = red[threadIdx.x];
    a.ws[((size_t)n * nchunk + chunk) * 2 + threadIdx.x] = ((v[0] + v[1]) + v[2]) + v[3];
  }
}

// The sum in front of each of the block's 256 threads, and the whole one.
__device__ __forceinline__ double block_scan(double v, double* red, double* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  double s = v;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double u = __shfl_up(s, m);
    if (lane >= m) s += u;
  }
  double front = __shfl_up(s, 1);
  if (lane == 0) front = 0.0;
  __syncthreads();  // (red may still be read from the scan before)
  if (lane == 63) red[w] = s;
  __syncthreads();
  for (int u = 0; u < w; ++u) front += red[u];
  *total = ((red[0] + red[1]) + red[2]) + red[3];
  return front;
}

// One workgroup per sequence: which chunk the threshold lies in, and which token.  Where rounding
// leaves no sum above the threshold, the last token that has mass is taken.
template <typename T>
__global__ __launch_bounds__(256) void kda_verify_pick_kernel(VerifyArgs a, int nchunk) {
  constexpr int V = kVec<T>, OWN = kChunk / 256;  // a thread's neighbouring probabilities of the chunk
  constexpr int NONE = 0x7fffffff;
  __shared__ double red[4], front_s;
  __shared__ int first, last;
  const int n = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) {
    first = NONE;
    last = -1;
  }
  Choice c{a.accepted[n], a.K, -1};
  if (a.counts) c.count = min(max(a.counts[n], 0), a.K);
  if (c.accepted < c.count) c.token = a.tokens[(long long)n * a.K + c.accepted];
  const double* sums = a.ws + (size_t)n * nchunk * 2;
  double left = 0.0, whole = 0.0, total_left, total;
  for (int i = tid; i < nchunk; i += 256) {
    left += sums[2 * i];
    whole += sums[2 * i + 1];
  }
  block_scan(left, red, &total_left);
  block_scan(whole, red, &total);
  Rows<T> r(a, n, c);
  const bool rest = total_left > 0.0;
  if (rest) {
    total = total_left;
  } else {  // q covers all of p: the token is drawn from p
    r.q = nullptr;
    r.token = -1;
  }
  const double goal = (double)a.u[(long long)n * (a.K + 1) + a.K] * total;
  double base = 0.0;
  for (int i0 = 0; i0 < nchunk; i0 += 256) {
    const int i = i0 + tid;
    const double v = i < nchunk ? sums[2 * i + (rest ? 0 : 1)] : 0.0;
    double all;
    const double before = base + block_scan(v, red, &all);
    if (v > 0.0) {
      atomicMax(&last, i);
      if (before + v > goal) atomicMin(&first, i);
    }
    __syncthreads();
    if (i == first) front_s = before;
    base += all;
    const bool done = first != NONE;
    __syncthreads();
    if (done) break;
  }
  const int chunk = first != NONE ? first : last;
  const bool sure = first != NONE;
  const double front = front_s;
  int token = -1;
  if (chunk >= 0) {
    __syncthreads();
    if (tid == 0) {
      first = NONE;
      last = -1;
    }
    const int c0 = chunk * kChunk, end = min(c0 + kChunk, a.V), mine = c0 + tid * OWN;
    double w[OWN], s = 0.0;
#pragma unroll
    for (int i = 0; i < OWN; i += V) {
      double z[V];
#pragma unroll
      for (int k = 0; k < V; ++k) w[i + k] = 0.0;
      if (mine + i < end) masses<T>(r, mine + i, end, w + i, z);
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) s += w[i];
    double all, run = front + block_scan(s, red, &all);  // (its barriers order the reset above)
    int hit = NONE, behind = -1;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      run += w[i];
      if (w[i] > 0.0) {
        behind = mine + i;
        if (hit == NONE && run > goal) hit = mine + i;
      }
    }
    if (sure && hit != NONE) atomicMin(&first, hit);
    if (behind >= 0) atomicMax(&last, behind);
    __syncthreads();
    token = first != NONE ? first : last;
  }
  for (int j = tid; j <= a.K; j += 256)
    a.out[(long long)n * (a.K + 1) + j] =
        j < c.accepted ? a.tokens[(long long)n * a.K + j] : (j == c.accepted ? token : -1);
}

// S[n] = S_pos[n][index[n]], by shares of a state's values; an index outside leaves S[n] as it is.
__global__ __launch_bounds__(256) void kda_state_commit_kernel(const float* __restrict__ S_pos, const int* __restrict__ index,
                                                               float* __restrict__ S, int ntok, long long elems, int share) {
  const int n = blockIdx.x / share;
  const int t = index[n];
  if (t < 0 || t >= ntok) return;
  const float* src = S_pos + ((size_t)n * ntok + t) * elems;
  float* dst = S + (size_t)n * elems;
  constexpr int U = 4;
  for (long long e0 = ((long long)(blockIdx.x % share) * (256 * U) + threadIdx.x) * 4; e0 < elems; e0 += (long long)share * (1024 * U)) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e0 + u * 1024 < elems) v[u] = ld16(src + e0 + u * 1024);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e0 + u * 1024 < elems) st16(dst + e0 + u * 1024, v[u]);
  }
}

int verify_chunks(int V) { return (V + kChunk - 1) / kChunk; }

template <typename T>
hipError_t verify(const VerifyArgs& a, hipStream_t stream) {
  const int nchunk = verify_chunks(a.V);
  hipLaunchKernelGGL((kda_verify_sum_kernel<T>), dim3((unsigned)((long long)a.N * nchunk)), dim3(256), 0, stream, a, nchunk);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((kda_verify_pick_kernel<T>), dim3((unsigned)a.N), dim3(256), 0, stream, a, nchunk);
  return hipGetLastError();
}

}  // namespace

size_t verify_ws_bytes(int N, int V) { return (size_t)N * verify_chunks(V) * 2 * sizeof(double); }

hipError_t launch_verify(const VerifyArgs& a, bool bf16_io, hipStream_t stream) {
  return bf16_io ? verify<bf16>(a, stream) : verify<float>(a, stream);
}

hipError_t launch_state_commit(const float* S_pos, const int* index, float* S, int N, int ntok, long long elems,
                               hipStream_t stream) {
  // blocks per state: one for every 4096 values, fewer where that would give more than 8192 blocks
  long long share = (elems + 4095) / 4096;
  while (share > 1 && N * share > 8192) share = (share + 1) / 2;
  hipLaunchKernelGGL(kda_state_commit_kernel, dim3((unsigned)(N * share)), dim3(256), 0, stream, S_pos, index, S, ntok, elems, (int)share);
  return hipGetLastError();
}

}  // namespace kda
