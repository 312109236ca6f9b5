// Drafted tokens: how many the target's probabilities accept, the token behind them, and the
// states that go with them.
//
// Token j is accepted while u_j q_j(tok_j) < p_j(tok_j), both as they count below.  At the first refusal the next token is drawn
// from max(p_j - q_j, 0), behind the last accepted one from p: the smallest i whose running sum is above
// u times the whole one.  Products of fp32 numbers are exact in fp64, and sums are fp64, so that the
// choice is the one of the exact sums but for a threshold within about 1e-14 of a border.
//
// One row of V probabilities (two after a refusal) is all that has to be read, and HBM bounds that where
// there are many long ones.  A row is cut into chunks that fill the chip with few sequences too: one launch adds every
// chunk up, a second one finds the chunk that holds the threshold and walks it alone.  Short rows
// take one launch, a workgroup each, since what two launches cost the host is more than they save.
// fp32, 4 drafts: 256 rows of 128K 39-41 us for 188 MB (the sums at HBM's rate, then the choice, 6); 1 row of 50K 15 us, 4.4 + 4.5
// of it kernels; 64 rows of 20K 11 us, bounded by the host's launch.
// Choosing 64 states of 32 x 128 x 128 out of 5 takes 51-54 us for 268 MB, 5.0-5.2 TB/s.
#include "kda_ops.hpp"
#include "kda_vec.hpp"

namespace kda {

namespace {

constexpr int kChunk = 4096;  // probabilities of a row per workgroup
constexpr int kRowChunks = 16;  // of a row that one workgroup takes

// A probability as it counts: NaN and what is negative as none, an infinity as the largest number.
__device__ __forceinline__ float mass(float p) { return fminf(fmaxf(p, 0.f), 3.402823466e38f); }

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
        const float p = to_f32(static_cast<const T*>(a.p)[n * a.pn + j * a.pt + tok]);
        const float q = a.q ? to_f32(static_cast<const T*>(a.q)[n * a.qn + j * a.qt + tok]) : 1.f;
        // (a NaN is not below or above anything: refused)
        ok = q == q && (double)a.u[(long long)n * (a.K + 1) + j] * (double)mass(q) < (double)mass(p);
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
  __device__ __forceinline__ Rows(const VerifyArgs& a, int n, int accepted, int refused_token, bool refused) {
    p = static_cast<const T*>(a.p) + n * a.pn + accepted * a.pt;
    q = refused && a.q ? static_cast<const T*>(a.q) + n * a.qn + accepted * a.qt : nullptr;
    token = refused && !a.q ? refused_token : -1;
  }
};

// 16 bytes at any element's address; ONCE: past the caches (256 rows of 128K 43.7 -> 41.4 us).
template <typename T, bool ONCE>
__device__ __forceinline__ Row<T> load_any(const T* p) {
  using Any = uint32_t __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  const Any* at = reinterpret_cast<const Any*>(p);
  const u32x4 w = ONCE ? __builtin_nontemporal_load(at) : *at;
  return unpack<T>(w);
}

// A lane's vector of both rows: what is left of p behind q, and p, in fp64.  The clamps are in fp32, whose instructions
// are cheaper; p - min(q, p) of fp32 numbers is exact in fp64 unless one is 2^28 times the other.
template <typename T, bool ONCE>
__device__ __forceinline__ void masses(const Rows<T>& r, int i0, int end, double* w, double* whole) {
  constexpr int V = kVec<T>;
  Row<T> p, q;
  if (i0 + V <= end) {
    p = load_any<T, ONCE>(r.p + i0);
    if (r.q) q = load_any<T, ONCE>(r.q + i0);
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      p.v[c] = i0 + c < end ? to_f32(r.p[i0 + c]) : 0.f;
      q.v[c] = r.q && i0 + c < end ? to_f32(r.q[i0 + c]) : 0.f;
    }
  }
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const float x = mass(p.v[c]);
    float y = r.q ? q.v[c] : 0.f;
    if (i0 + c == r.token) y = 1.f;
    whole[c] = (double)x;
    w[c] = whole[c] - (double)fminf(fmaxf(y, 0.f), x);
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// A thread's share of the sums over [c0, end), THREADS of them together, DEEP vectors at a time.
template <typename T, int THREADS, int DEEP, bool ONCE>
__device__ __forceinline__ void add_up(const Rows<T>& r, int c0, int end, int thread, double* left, double* whole) {
  constexpr int V = kVec<T>;
  double s = 0.0, t = 0.0;
#pragma unroll DEEP
  for (int i = c0 + thread * V; i < end; i += THREADS * V) {
    double w[V], z[V];
    masses<T, ONCE>(r, i, end, w, z);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      s += w[c];
      t += z[c];
    }
  }
  *left = s;
  *whole = t;
}

// A sequence's record in the workspace: (accepted, refused token or -1, refused, 0), then the chunks' sums.
struct Record {
  int4* choice;
  double2* sums;  // of every chunk: what is left, and the whole
  __device__ __forceinline__ Record(const VerifyArgs& a, int n, int nchunk)
      : choice(reinterpret_cast<int4*>(a.ws) + (size_t)n * (nchunk + 1)), sums(reinterpret_cast<double2*>(choice + 1)) {}
};

// The first chunk's block writes how far the sequence is accepted.
template <typename T>
__global__ __launch_bounds__(256) void kda_verify_sum_kernel(VerifyArgs a, int nchunk) {
  __shared__ double red[2][4];
  const int n = blockIdx.x / nchunk, chunk = blockIdx.x % nchunk;
  const Choice choice = accept<T>(a, n);
  const Record rec(a, n, nchunk);
  if (chunk == 0 && threadIdx.x == 0) {
    a.accepted[n] = choice.accepted;
    *rec.choice = int4{choice.accepted, choice.token, choice.accepted < choice.count, 0};
  }
  const Rows<T> r(a, n, choice.accepted, choice.token, choice.accepted < choice.count);
  const int c0 = chunk * kChunk;
  double s, whole;
  // (more vectors at a time take registers, and with them waves: 1024 rows of 50257 in bf16 70, 62, 56 us with 4, 2, 1,
  // 256 of 128K in fp32 41.4, 41.2, 41.8)
  add_up<T, 256, sizeof(T) == 2 ? 1 : 2, true>(r, c0, min(c0 + kChunk, a.V), threadIdx.x, &s, &whole);
  s = wave_sum(s);
  whole = wave_sum(whole);
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = s;
    red[1][threadIdx.x >> 6] = whole;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const double* v = red[threadIdx.x];
    reinterpret_cast<double*>(rec.sums + chunk)[threadIdx.x] = ((v[0] + v[1]) + v[2]) + v[3];
  }
}

// The sum up to and including each lane's v.
__device__ __forceinline__ double wave_scan(double v) {
  const int lane = lane_id();
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double u = __shfl_up(v, m);
    if (lane >= m) v += u;
  }
  return v;
}

// The token, by a workgroup of WAVES waves: every wave finds the chunk that the threshold lies in (lane = chunk), then
// 512 threads walk it, 8 probabilities each.  Where rounding leaves no sum above the threshold, the last token that
// has mass is taken.  choice and sums: a sequence's record.
template <typename T, int WAVES>
__device__ __forceinline__ void pick(const VerifyArgs& a, int n, int4 choice, float u, const double2* sums, int nchunk, int size) {
  constexpr int V = kVec<T>, OWN = kChunk / 512;  // a thread's neighbouring probabilities of the chunk
  constexpr int NONE = 0x7fffffff;
  __shared__ double front_of[WAVES];
  __shared__ int first, last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  double2 v{0.0, 0.0};
  if (lane < nchunk) v = sums[lane];
  if (tid == 0) {
    first = NONE;
    last = -1;
  }
  double left = v.x, whole = v.y;
  for (int i = lane + 64; i < nchunk; i += 64) {
    const double2 x = sums[i];
    left += x.x;
    whole += x.y;
  }
  left = wave_sum(left);
  whole = wave_sum(whole);
  const bool rest = left > 0.0;  // else q covers all of p: the token is drawn from p
  const Rows<T> r(a, n, choice.x, rest ? choice.y : -1, rest && choice.z);
  const double goal = (double)u * (rest ? left : whole);
  int chunk = -1;  // the first one whose running sum is above the goal, or the last that has mass
  bool sure = false;
  double front = 0.0, base = 0.0;
  for (int i0 = 0; i0 < nchunk; i0 += 64) {
    if (i0 > 0) v = i0 + lane < nchunk ? sums[i0 + lane] : double2{0.0, 0.0};
    const double mine = rest ? v.x : v.y, sum = base + wave_scan(mine);
    const unsigned long long above = __ballot(mine > 0.0 && sum > goal), any = __ballot(mine > 0.0);
    if (above) {
      const int at = __ffsll(above) - 1;
      chunk = i0 + at;
      sure = true;
      front = at ? __shfl(sum, at - 1) : base;
      break;
    }
    if (any) chunk = i0 + 63 - __clzll(any);
    base = __shfl(sum, 63);
  }
  int token = -1;
  if (chunk >= 0) {
    const int c0 = chunk * size, end = min(c0 + size, a.V), mine = c0 + tid * OWN;
    double w[OWN], s = 0.0;
#pragma unroll
    for (int i = 0; i < OWN; i += V) {
      double z[V];
#pragma unroll
      for (int k = 0; k < V; ++k) w[i + k] = 0.0;
      if (mine + i < end) masses<T, false>(r, mine + i, end, w + i, z);
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) s += w[i];
    const double upto = wave_scan(s);
    if (lane == 63) front_of[wave] = upto;
    __syncthreads();
    double run = __shfl_up(upto, 1);
    run = (lane ? run : 0.0) + front;
    for (int k = 0; k < wave; ++k) run += front_of[k];
    int hit = NONE, behind = -1;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      run += w[i];
      if (w[i] > 0.0) {
        behind = mine + i;
        if (hit == NONE && run > goal) hit = mine + i;
      }
    }
    const unsigned long long hits = __ballot(hit != NONE), some = __ballot(behind >= 0);
    if (sure && hits && lane == __ffsll(hits) - 1) atomicMin(&first, hit);
    if (some && lane == 63 - __clzll(some)) atomicMax(&last, behind);
    __syncthreads();
    token = first != NONE ? first : last;
  }
  for (int j = tid; j <= a.K; j += 64 * WAVES)
    a.out[(long long)n * (a.K + 1) + j] =
        j < choice.x ? a.tokens[(long long)n * a.K + j] : (j == choice.x ? token : -1);
}

// One workgroup per sequence, a chain of latencies: the record, the chunk, the sums over lanes and waves.
template <typename T>
__global__ __launch_bounds__(512) void kda_verify_pick_kernel(VerifyArgs a, int nchunk) {
  const int n = blockIdx.x;
  const Record rec(a, n, nchunk);
  const float u = a.u[(long long)n * (a.K + 1) + a.K];
  pick<T, 8>(a, n, *rec.choice, u, rec.sums, nchunk, kChunk);
}

// Short rows in one launch: a workgroup per sequence, a chunk per wave.  Only what is left is added up; where that is
// nothing, p itself.
template <typename T>
__global__ __launch_bounds__(1024) void kda_verify_row_kernel(VerifyArgs a, int nchunk, int size) {
  __shared__ double2 sums[kRowChunks];
  const int n = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const float u = a.u[(long long)n * (a.K + 1) + a.K];
  const Choice choice = accept<T>(a, n);
  if (threadIdx.x == 0) a.accepted[n] = choice.accepted;
  for (bool refused = choice.accepted < choice.count;; refused = false) {
    if (wave < nchunk) {
      const Rows<T> r(a, n, choice.accepted, choice.token, refused);
      double left, whole;
      add_up<T, 64, 1, false>(r, wave * size, min((wave + 1) * size, a.V), lane, &left, &whole);
      left = wave_sum(left);
      if (lane == 0) sums[wave] = double2{left, left};
    }
    __syncthreads();
    bool any = !refused;
    for (int i = 0; i < nchunk; ++i) any = any || sums[i].x > 0.0;
    if (any) {
      pick<T, 16>(a, n, int4{choice.accepted, refused ? choice.token : -1, refused, 0}, u, sums, nchunk, size);
      return;
    }
    __syncthreads();
  }
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
// Whether a workgroup takes a whole row: one launch less and no workspace, but a row's sums then are one CU's work.
// With a draft, fp32, us in one launch / two: 1 row of 4K 10.6 / 14.3, 32K 11.2 / 15.0, 64K 14.7 / 14.3; 64 rows 10.7 / 14.7,
// 13.2 / 14.1, 18.9 / 14.7; 256 rows 10.7 / 14.7, 16.7 / 20.1; with more rows than CUs, 1024 of 1K, 34 / 15.
bool verify_row(int N, int V) { return N <= 256 && V <= 32768; }

template <typename T>
hipError_t verify(const VerifyArgs& a, hipStream_t stream) {
  const int nchunk = verify_chunks(a.V);
  if (verify_row(a.N, a.V)) {
    const int size = ((a.V + kRowChunks - 1) / kRowChunks + 511) / 512 * 512;
    hipLaunchKernelGGL((kda_verify_row_kernel<T>), dim3((unsigned)a.N), dim3(1024), 0, stream, a, (a.V + size - 1) / size, size);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((kda_verify_sum_kernel<T>), dim3((unsigned)((long long)a.N * nchunk)), dim3(256), 0, stream, a, nchunk);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((kda_verify_pick_kernel<T>), dim3((unsigned)a.N), dim3(512), 0, stream, a, nchunk);
  return hipGetLastError();
}

}  // namespace

size_t verify_ws_bytes(int N, int V) {
  const int nchunk = verify_chunks(V);
  return verify_row(N, V) ? 0 : (size_t)N * (nchunk + 1) * 16;
}

bool verify_fits(int N, int V) {
  return verify_row(N, V) || (launchable((long long)N * verify_chunks(V), 256) && launchable(N, 512));
}

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
