// Gated delta rule, one token of many sequences (sm_100a): the decode step.
//
// Per head with the state S (value channel i x key channel j), decay a = e^g:
//   e = v - a S k,   S <- a S + beta e k^T,   y = scale S q.
// The rows of S never meet: row i needs v_i, the whole of k and q, and two dot products over
// its own columns. 16 lanes hold a row, a warp 16 rows (two at a time), all of them loaded
// before the first is used, so that a warp has its 4 KiB (N = 64) or 8 KiB (N = 128) of state
// in flight at once. Bound by HBM: a token reads and writes the state once, 8 N^2 bytes a head
// against 6 N^2 flops. Measured: 256 rows x 64 heads x 64, fp32: 87 us, 0.96 of the copy rate;
// 87 rows of a pool x 32 x 128, bf16: 62 us, 0.91; one row of 12 heads: 4 us, the launch.
#include "wkv_device.cuh"
#include "wkv_internal.h"

namespace wkv {

namespace {

constexpr int kRows = 16;           // rows of S per warp
constexpr int kPairs = kRows / 2;   // row pairs: lanes 0-15 the even row, 16-31 the odd one
constexpr int kWarps = 4;

// Below this a log-decay counts as a decay of zero: e^-200 is far below the smallest float.
constexpr float kLeastG = -200.f;

__device__ __forceinline__ float decay_of(float g) { return expf(g < kLeastG ? kLeastG : g); }

__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
  const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float acc) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, acc))));
}

// Sum over the 16 lanes of a half warp, in every lane.
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

template <typename T, int N>
__global__ void __launch_bounds__(kWarps * 32) gdr_decode_kernel(GdrArgs a) {
  constexpr int V = N / 64;  // float4s of a row per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = lane >> 4, l16 = lane & 15;
  constexpr int kSplit = N / (kRows * kWarps) > 0 ? N / (kRows * kWarps) : 1;
  const int part = blockIdx.x % kSplit;
  const int64_t sh = blockIdx.x / kSplit;
  const int seq = int(sh / a.H), h = int(sh % a.H), hk = h / (a.H / a.Hk);
  const int r0 = (part * kWarps + warp) * kRows;
  int64_t slot = seq;
  if (a.slots != nullptr) {
    slot = a.slots[seq];
    if (slot < 0 || slot >= a.n_slots) return;
  }
  const T* q = static_cast<const T*>(a.q);
  const T* k = static_cast<const T*>(a.k);
  const T* v = static_cast<const T*>(a.v);
  T* y = static_cast<T*>(a.y);
  const int64_t state_at = ((slot * a.H + h) * N + r0) * N;

  float4 S[kPairs][V];
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
#pragma unroll
    for (int c = 0; c < V; ++c)
      S[i][c] = load4(a.s0 + state_at + (2 * i + half) * N + 64 * c + 4 * l16);

  const int64_t t = seq;
  float4 kv[V], qv[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    kv[c] = load4(k + (t * a.Hk + hk) * N + 64 * c + 4 * l16);
    qv[c] = load4(q + (t * a.Hk + hk) * N + 64 * c + 4 * l16);
  }
  const float vv = Elem<T>::to_f(v[(t * a.H + h) * N + r0 + l16]);
  const float al = decay_of(a.g[t * a.H + h]), be = a.beta[t * a.H + h];
  float mine = 0.f;  // y of row r0 + l16
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    float d = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      S[i][c].x *= al; S[i][c].y *= al; S[i][c].z *= al; S[i][c].w *= al;
      d = dot4(S[i][c], kv[c], d);
    }
    const float u = be * (__shfl_sync(0xffffffffu, vv, 2 * i + half) - sum16(d));
    float o = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      S[i][c].x = fmaf(u, kv[c].x, S[i][c].x);
      S[i][c].y = fmaf(u, kv[c].y, S[i][c].y);
      S[i][c].z = fmaf(u, kv[c].z, S[i][c].z);
      S[i][c].w = fmaf(u, kv[c].w, S[i][c].w);
      o = dot4(S[i][c], qv[c], o);
    }
    o = sum16(o);
    // row 2 i + half is in this half's lanes; lane l16 < 16 of half 0 collects row l16
    const float other = __shfl_xor_sync(0xffffffffu, o, 16);
    if (l16 == 2 * i) mine = half == 0 ? o : other;
    if (l16 == 2 * i + 1) mine = half == 1 ? o : other;
  }
  if (half == 0) y[(t * a.H + h) * N + r0 + l16] = Elem<T>::from_f(a.scale * mine);
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
#pragma unroll
    for (int c = 0; c < V; ++c)
      *reinterpret_cast<float4*>(a.s1 + state_at + (2 * i + half) * N + 64 * c + 4 * l16) = S[i][c];
}

template <typename T>
int launch(const GdrArgs& a, cudaStream_t stream) {
  const int split = a.N / (kRows * kWarps);
  const unsigned grid = unsigned(int64_t(a.n_seqs) * a.H * split);
  if (a.N == 64)
    return launch_kernel(gdr_decode_kernel<T, 64>, grid, kWarps * 32, 0, stream, a);
  return launch_kernel(gdr_decode_kernel<T, 128>, grid, kWarps * 32, 0, stream, a);
}

}  // namespace

int launch_gdr_decode(const GdrArgs& a, cudaStream_t stream) {
  return a.bf16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace wkv
