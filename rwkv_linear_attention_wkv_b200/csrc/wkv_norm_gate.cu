// Norm, gate, scaled residual and next norm around a block, forward and backward (sm_100a).
//
// Per row of C channels, r1 = 1 / RMS over a group of channels, r2 = 1 / RMS over the row:
//   m   = act(z) w h r1,   out = x + s m,   y = w' out r2.
// Backward, with d = dout + r2 (dy w' - out r2^2 <dy w', out> / C):
//   dx = d,  ds = sum_rows d m,  dz = d s w h r1 act'(z),  dw = sum_rows d s act(z) h r1,
//   dh = r1 (n - h r1^2 <n, h>_group / group),  n = d s act(z) w,   dw' = sum_rows dy out r2.
//
// A team of ceil(C / 256) warps holds a row, eight channels a thread, and walks rows; the three
// weights wait in shared memory in the order of the threads. A thread meets the same channels in
// every row, so its sums of dw, ds and dw' stay in registers (one line per CTA into the workspace
// at the end, added up in a fixed order by a second kernel). The next row's inputs are loaded
// before this row's sums, so that a row is always in flight. Group sums are shuffles where a group
// is 8 x a power of two channels up to 256 (the heads), the row sum where it is the row, and go
// through shared memory otherwise.
// Bound by HBM: 32768 x 4096 bf16 with gate, residual and next norm in 267 us, 5.0 TB/s, 0.76 of
// the copy rate; 16384 x 4096 fp32 in 230 us, 0.89. The backward (16384 x 768 in 58 us, 3.5 TB/s) by
// latency: its sums leave 12 warps an SM. Few rows by the launch (256 x 4096: 6 us).
#include <algorithm>

#include "wkv_device.cuh"
#include "wkv_internal.h"

namespace wkv {

namespace {

constexpr int kE = 8;             // channels per thread
constexpr int kMaxC = 8192;       // 1024 threads a row
constexpr int kTeamsMax = 8;      // rows a CTA works on at once

enum GroupMode { kRow, kLanes, kAny };

// CTAs on an SM at once. Forward, bf16: two of 512 threads, so that one loads while the other sums
// (64 registers hold the next row and this one; fp32 rows need twice as many, and one CTA has as
// many bytes in flight). Backward: one; its sums over rows and five inputs take 128 to 168.
constexpr int fwd_ctas(bool bf16, int threads) { return bf16 && threads <= 512 ? 2 : 1; }

struct Eight {
  float v[kE];
};

// Eight at a time, two to an instruction.
__device__ __forceinline__ float2 two(const Eight& a, int i) {
  return make_float2(a.v[2 * i], a.v[2 * i + 1]);
}
__device__ __forceinline__ void put(Eight& a, int i, float2 x) {
  a.v[2 * i] = x.x;
  a.v[2 * i + 1] = x.y;
}
__device__ __forceinline__ Eight operator*(const Eight& a, const Eight& b) {
  Eight r;
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) put(r, i, __fmul2_rn(two(a, i), two(b, i)));
  return r;
}
__device__ __forceinline__ Eight operator*(const Eight& a, float b) {
  Eight r;
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) put(r, i, __fmul2_rn(two(a, i), make_float2(b, b)));
  return r;
}
__device__ __forceinline__ Eight fma(const Eight& a, const Eight& b, const Eight& c) {
  Eight r;
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) put(r, i, __ffma2_rn(two(a, i), two(b, i), two(c, i)));
  return r;
}
__device__ __forceinline__ Eight fma(const Eight& a, float b, const Eight& c) {
  Eight r;
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) put(r, i, __ffma2_rn(two(a, i), make_float2(b, b), two(c, i)));
  return r;
}
// sum of a b over the eight
__device__ __forceinline__ float dot(const Eight& a, const Eight& b) {
  float2 s = __fmul2_rn(two(a, 0), two(b, 0));
#pragma unroll
  for (int i = 1; i < kE / 2; ++i) s = __ffma2_rn(two(a, i), two(b, i), s);
  return s.x + s.y;
}

// Raw values as loaded (four or eight registers), so that a prefetched row costs little.
template <typename T> struct Raw;
template <> struct Raw<float> {
  float4 a, b;
};
template <> struct Raw<__nv_bfloat16> {
  uint4 a;
};

// Where a thread's eight channels are: adjacent (VEC), or a row's width apart (any C, any
// alignment).
template <bool VEC>
struct Place {
  int c0, step, C;
  __device__ int at(int i) const { return VEC ? c0 + i : c0 + i * step; }
  __device__ bool in(int i) const { return VEC ? c0 < C : c0 + i * step < C; }
};

template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load_raw(const T* p, const Place<VEC>& pl) {
  Raw<T> r;
  T* e = reinterpret_cast<T*>(&r);
  if (VEC) {
    if (pl.c0 < pl.C) {
      r = *reinterpret_cast<const Raw<T>*>(p + pl.c0);
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) e[i] = Elem<T>::from_f(0.f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i) e[i] = pl.in(i) ? p[pl.at(i)] : Elem<T>::from_f(0.f);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ Eight widen(const Raw<T>& r) {
  const T* e = reinterpret_cast<const T*>(&r);
  Eight x;
#pragma unroll
  for (int i = 0; i < kE; ++i) x.v[i] = Elem<T>::to_f(e[i]);
  return x;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store(T* p, const Eight& x, const Place<VEC>& pl) {
  Raw<T> r;
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < kE; ++i) e[i] = Elem<T>::from_f(x.v[i]);
  if (VEC) {
    if (pl.c0 < pl.C) *reinterpret_cast<Raw<T>*>(p + pl.c0) = r;
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (pl.in(i)) p[pl.at(i)] = e[i];
  }
}

// A weight's row in shared memory, in the order in which a team's threads take it: [8][threads],
// or, for adjacent channels, [2][threads][4].
template <bool VEC>
__device__ __forceinline__ Eight params(const float* row, const Place<VEC>& pl) {
  Eight x;
  if (VEC) {
    const float4 a = *reinterpret_cast<const float4*>(row + pl.c0 / 2);
    const float4 b = *reinterpret_cast<const float4*>(row + 4 * pl.step + pl.c0 / 2);
    x.v[0] = a.x; x.v[1] = a.y; x.v[2] = a.z; x.v[3] = a.w;
    x.v[4] = b.x; x.v[5] = b.y; x.v[6] = b.z; x.v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i) x.v[i] = row[pl.c0 + i * pl.step];
  }
  return x;
}
// The three weights' rows, ones where there is none, zeros past C.
template <bool VEC>
__device__ __forceinline__ void put_params(float* rows, const float* w, const float* s,
                                           const float* n, int step, int C) {
  for (int i = threadIdx.x; i < 3 * step; i += blockDim.x) {
    const int j = i / step, at = i % step;
    const float* const p = j == 0 ? w : j == 1 ? s : n;
    float* const row = rows + j * kE * step;
    if (VEC && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (at * kE < C)
          v = p ? *reinterpret_cast<const float4*>(p + at * kE + 4 * half)
                : make_float4(1.f, 1.f, 1.f, 1.f);
        *reinterpret_cast<float4*>(row + half * 4 * step + 4 * at) = v;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int c = VEC ? at * kE + e : e * step + at;
        const int to = VEC ? e / 4 * 4 * step + 4 * at + e % 4 : c;
        row[to] = c >= C ? 0.f : p ? p[c] : 1.f;
      }
    }
  }
}

// The warps that hold one row: their sums go through shared memory (two slots in turn, so that
// one barrier a sum is enough).
struct Team {
  int warps, warp, lane, id;
  float* weights;    // [3][8 x threads of a team]: weight, scale, next weight
  float2* slots;     // [2][32]
  float* parts;      // kAny: one value per channel (VEC: per eight) and one per group
  int turn = 0;

  __device__ void sync() const {
    if (warps == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(warps * 32) : "memory");
  }

  __device__ static void lanes(float& a) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
  }

  __device__ float sum(float a) {
    lanes(a);
    if (warps == 1) return a;
    float2* s = slots + 32 * turn;
    turn ^= 1;
    if (lane == 0) s[warp].x = a;
    sync();
    a = lane < warps ? s[lane].x : 0.f;
    lanes(a);
    return a;
  }

  __device__ float2 sum(float a, float b) {
    lanes(a);
    lanes(b);
    if (warps == 1) return make_float2(a, b);
    float2* s = slots + 32 * turn;
    turn ^= 1;
    if (lane == 0) s[warp] = make_float2(a, b);
    sync();
    const float2 mine = lane < warps ? s[lane] : make_float2(0.f, 0.f);
    a = mine.x;
    b = mine.y;
    lanes(a);
    lanes(b);
    return make_float2(a, b);
  }
};

// For each of a thread's channels the sum of x over the channel's group.
template <bool VEC, GroupMode MODE>
__device__ __forceinline__ Eight group_sum(const Eight& x, Team& t, const Place<VEC>& pl,
                                           int group) {
  Eight out;
  if (MODE != kAny) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) s += x.v[i];
    if (MODE == kRow) {
      s = t.sum(s);
    } else {
      for (int m = group / kE / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    }
#pragma unroll
    for (int i = 0; i < kE; ++i) out.v[i] = s;
    return out;
  }
  float* sums = t.parts + pl.C;
  t.sync();  // the last sums have been read
#pragma unroll
  for (int i = 0; i < kE; ++i)
    if (pl.in(i)) t.parts[pl.at(i)] = x.v[i];
  t.sync();
  for (int g = t.warp; g < pl.C / group; g += t.warps) {
    float s = 0.f;
    for (int c = t.lane; c < group; c += 32) s += t.parts[g * group + c];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (t.lane == 0) sums[g] = s;
  }
  t.sync();
#pragma unroll
  for (int i = 0; i < kE; ++i) out.v[i] = pl.in(i) ? sums[pl.at(i) / group] : 0.f;
  return out;
}

__device__ __forceinline__ Eight inverse_rms(const Eight& sum, float inv, float eps) {
  Eight r;
#pragma unroll
  for (int i = 0; i < kE; ++i) r.v[i] = rsqrtf(fmaf(sum.v[i], inv, eps));
  return r;
}

// e^-z by the exponential instruction: off by less than |z| 2^-23 of itself, the roundings of its
// argument and of log2(e), and by the instruction's 2^-22.
__device__ __forceinline__ float exp_minus(float z) { return ex2(z * -1.4426950408889634f); }

// s = sigmoid(z) by the exponential and reciprocal instructions: 1 - s times what e^-z is off by, the
// sum's rounding of 2^-24 and the reciprocal's 2^-23; 2^-21 of s at most for z >= 0, |z| 2^-23 more
// below. (expf and a division: 15 instructions more, a third of a forward row.)
__device__ __forceinline__ float sigmoid_of(float z) { return rcp(1.f + exp_minus(z)); }
// 1 - sigmoid(z) from s = sigmoid(z), without the difference where s is close to one.
__device__ __forceinline__ float off_of(float z, float s) {
  return z > 0.f ? exp_minus(z) * s : 1.f - s;
}

template <bool VEC>
__device__ __forceinline__ void make_team(int team_warps, int C, Team& t, Place<VEC>& pl) {
  extern __shared__ float smem_ng[];
  const int warp = threadIdx.x >> 5;
  t.warps = team_warps;
  t.id = warp / team_warps;
  t.warp = warp % team_warps;
  t.lane = threadIdx.x & 31;
  const int teams = (blockDim.x >> 5) / team_warps;
  const int wide = team_warps * 32 * kE;
  t.weights = smem_ng;
  t.slots = reinterpret_cast<float2*>(smem_ng + 3 * wide) + 64 * t.id;
  t.parts = smem_ng + 3 * wide + 128 * teams + 2 * C * t.id;
  const int at = t.warp * 32 + t.lane;
  pl.C = C;
  pl.step = team_warps * 32;
  pl.c0 = VEC ? at * kE : at;
}

template <typename T, bool VEC, GroupMode MODE, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS, fwd_ctas(sizeof(T) == 2, MAX_THREADS))
    norm_gate_fwd_kernel(NormGateArgs a, int team_warps) {
  Team t;
  Place<VEC> pl;
  make_team<VEC>(team_warps, a.C, t, pl);
  const int teams = (blockDim.x >> 5) / team_warps;
  const int wide = pl.step * kE;
  const T *h = static_cast<const T*>(a.h), *z = static_cast<const T*>(a.gate),
          *x = static_cast<const T*>(a.x);
  const float inv_group = 1.f / a.group, inv_c = 1.f / a.C;
  int64_t row = int64_t(blockIdx.x) * teams + t.id;
  const int64_t stride = int64_t(gridDim.x) * teams;
  Raw<T> hr, zr, xr;
  auto fetch = [&](int64_t r) {
    hr = load_raw<T, VEC>(h + r * a.C, pl);
    if (z) zr = load_raw<T, VEC>(z + r * a.C, pl);
    if (x) xr = load_raw<T, VEC>(x + r * a.C, pl);
  };
  if (row < a.R) fetch(row);
  put_params<VEC>(t.weights, a.weight, a.scale, a.next_weight, pl.step, a.C);
  __syncthreads();
  for (; row < a.R; row += stride) {
    const Eight hv = widen<T>(hr);
    Eight m = params<VEC>(t.weights, pl) * hv;
    if (z) {
      const Eight zv = widen<T>(zr);
      Eight sig;
#pragma unroll
      for (int i = 0; i < kE; ++i) sig.v[i] = sigmoid_of(zv.v[i]);
      m = m * sig;
      if (a.act == WKV_ACT_SILU) m = m * zv;
    }
    Eight xv{};
    if (x) xv = widen<T>(xr);
    if (row + stride < a.R) fetch(row + stride);
    m = m * inverse_rms(group_sum<VEC, MODE>(hv * hv, t, pl, a.group), inv_group, a.eps);
    if (x) m = fma(params<VEC>(t.weights + wide, pl), m, xv);
    store<T, VEC>(static_cast<T*>(a.out) + row * a.C, m, pl);
    if (a.y) {
      const float r2 = rsqrtf(fmaf(t.sum(dot(m, m)), inv_c, a.eps));
      m = m * r2 * params<VEC>(t.weights + 2 * wide, pl);
      store<T, VEC>(static_cast<T*>(a.y) + row * a.C, m, pl);
    }
  }
}

template <typename T, bool VEC, GroupMode MODE, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS, 1) norm_gate_bwd_kernel(NormGateArgs a, int team_warps) {
  Team t;
  Place<VEC> pl;
  make_team<VEC>(team_warps, a.C, t, pl);
  const int teams = (blockDim.x >> 5) / team_warps;
  const int wide = pl.step * kE;
  const T *h = static_cast<const T*>(a.h), *z = static_cast<const T*>(a.gate),
          *x = static_cast<const T*>(a.x), *dout = static_cast<const T*>(a.dout),
          *dy = static_cast<const T*>(a.dy);
  const float inv_group = 1.f / a.group, inv_c = 1.f / a.C;
  const int64_t first = int64_t(blockIdx.x) * teams + t.id;
  const int64_t stride = int64_t(gridDim.x) * teams;
  Eight dw{}, ds{}, dwn{};
  Raw<T> hr, zr, xr, dor, dyr;
  auto fetch = [&](int64_t r) {
    hr = load_raw<T, VEC>(h + r * a.C, pl);
    if (z) zr = load_raw<T, VEC>(z + r * a.C, pl);
    if (x) xr = load_raw<T, VEC>(x + r * a.C, pl);
    if (dout) dor = load_raw<T, VEC>(dout + r * a.C, pl);
    if (dy) dyr = load_raw<T, VEC>(dy + r * a.C, pl);
  };
  if (first < a.R) fetch(first);
  put_params<VEC>(t.weights, a.weight, a.scale, a.next_weight, pl.step, a.C);
  __syncthreads();
  for (int64_t row = first; row < a.R; row += stride) {
    Eight hn = widen<T>(hr), sig{}, d{}, out{};
    const Raw<T> zk = zr;
    if (z) {
      const Eight zv = widen<T>(zk);
#pragma unroll
      for (int i = 0; i < kE; ++i) sig.v[i] = sigmoid_of(zv.v[i]);
    }
    const bool silu = a.act == WKV_ACT_SILU;
    auto act_of = [&] {
      Eight act = silu ? widen<T>(zk) : sig;
#pragma unroll
      for (int i = 0; i < kE; ++i) act.v[i] = !z ? 1.f : silu ? act.v[i] * sig.v[i] : act.v[i];
      return act;
    };
    if (x) out = widen<T>(xr);
    if (dout) d = widen<T>(dor);
    Eight dn{};
    if (dy) dn = widen<T>(dyr);
    if (row + stride < a.R) fetch(row + stride);
    const Eight r1 =
        inverse_rms(group_sum<VEC, MODE>(hn * hn, t, pl, a.group), inv_group, a.eps);
    hn = hn * r1;
    const Eight w = params<VEC>(t.weights, pl);
    if (dy) {
      const Eight wn = params<VEC>(t.weights + 2 * wide, pl);
      out = fma(params<VEC>(t.weights + wide, pl), act_of() * w * hn, out);
      const Eight dw_n = dn * wn;
      const float2 both = t.sum(dot(out, out), dot(out, dw_n));
      const float r2 = rsqrtf(fmaf(both.x, inv_c, a.eps));
      const float pull = r2 * r2 * both.y * inv_c;  // <dy w', out r2> r2 / C
      dwn = fma(dn, out * r2, dwn);
      d = fma(fma(out, -pull, dw_n), r2, d);
    }
    if (a.dx) store<T, VEC>(static_cast<T*>(a.dx) + row * a.C, d, pl);
    const Eight s = params<VEC>(t.weights + wide, pl), act = act_of();
    const Eight dm = d * s, ah = act * hn;
    ds = fma(d, ah * w, ds);
    dw = fma(dm, ah, dw);
    Eight n = dm * w;
    if (a.dgate) {
      // silu' = sig + z sig (1 - sig), sigmoid' = sig (1 - sig)
      Eight slope;
      const Eight zv = widen<T>(zk);
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const float off = off_of(zv.v[i], sig.v[i]);
        slope.v[i] = silu ? ::fmaf(act.v[i], off, sig.v[i]) : sig.v[i] * off;
      }
      store<T, VEC>(static_cast<T*>(a.dgate) + row * a.C, n * hn * slope, pl);
    }
    n = n * act;
    const Eight p = group_sum<VEC, MODE>(n * hn, t, pl, a.group) * -inv_group;
    store<T, VEC>(static_cast<T*>(a.dh) + row * a.C, fma(hn, p, n) * r1, pl);
  }
  // the teams' sums added up in order where the weights were, a line a CTA
  float* const sums = t.weights;
  for (int id = 0; id < teams; ++id) {
    __syncthreads();
    if (t.id != id) continue;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const int c = pl.at(i);
      if (!pl.in(i)) continue;
      sums[c] = id == 0 ? dw.v[i] : sums[c] + dw.v[i];
      sums[wide + c] = id == 0 ? ds.v[i] : sums[wide + c] + ds.v[i];
      sums[2 * wide + c] = id == 0 ? dwn.v[i] : sums[2 * wide + c] + dwn.v[i];
    }
  }
  __syncthreads();
  float* line = a.partial + int64_t(blockIdx.x) * 3 * a.C;  // [dw, ds, dw'] of this CTA
  for (int c = threadIdx.x; c < a.C; c += blockDim.x)
#pragma unroll
    for (int j = 0; j < 3; ++j) line[j * a.C + c] = sums[j * wide + c];
}

// The CTAs' lines added up: 32 columns x kSlices slices of the lines a CTA, the slices in order.
constexpr int kSlices = 16;
__global__ void __launch_bounds__(32 * kSlices)
    norm_gate_sum_kernel(const float* partial, int lines, int C, float* dw, float* ds, float* dwn) {
  __shared__ float part[kSlices][32];
  float* const to = blockIdx.y == 0 ? dw : blockIdx.y == 1 ? ds : dwn;
  if (to == nullptr) return;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < C) {
    const float* p = partial + int64_t(blockIdx.y) * C + c;
#pragma unroll 8
    for (int l = slice; l < lines; l += kSlices) s += p[int64_t(l) * 3 * C];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < C) {
    for (int i = 1; i < kSlices; ++i) s += part[i][lane];
    to[c] = s;
  }
}

struct Plan {
  int team_warps, teams, grid;
  GroupMode mode;
  size_t smem;
};

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// Rows of a CTA: as many as make 512 threads (forward) or 384 (backward), CTAs: as many as the
// GPU holds at once, as long as each team has a row.
Plan plan_of(int64_t R, int C, int group, bool vec, bool bf16, bool backward, int sms) {
  Plan p;
  p.team_warps = (C + 32 * kE - 1) / (32 * kE);
  p.teams = std::max(1, std::min(kTeamsMax, (backward ? 12 : 16) / p.team_warps));
  const int threads = 32 * p.team_warps * p.teams;
  const int per_sm = backward ? 1 : fwd_ctas(bf16, threads);
  p.grid = int(std::min<int64_t>((R + p.teams - 1) / p.teams, int64_t(sms) * per_sm));
  const int lanes = group / kE;
  const bool pow2 = (lanes & (lanes - 1)) == 0;
  p.mode = group == C ? kRow
           : vec && group % kE == 0 && lanes <= 32 && pow2 ? kLanes
                                                           : kAny;
  p.smem = size_t(p.teams) * (512 + (p.mode == kAny ? 8 * size_t(C) : 0)) +
           size_t(p.team_warps) * 32 * kE * 12;
  return p;
}

// Backward: rows of up to 12 warps fit 384 threads, which leaves a thread 168 registers for
// the sums over rows, this row and the next; up to 16 warps take 512 threads and 128; wider
// ones take 1024 threads and spill (forward and backward of 4096 x 4096 bf16: 156 us, 0.33 of HBM;
// of 2048 x 8192: 339 us, 0.15).
template <typename T, bool VEC, GroupMode MODE>
int run(const NormGateArgs& a, const Plan& p, bool backward, cudaStream_t stream) {
  const int warps = p.team_warps * p.teams;
  auto* kernel = backward ? (warps <= 12   ? norm_gate_bwd_kernel<T, VEC, MODE, 384>
                             : warps <= 16 ? norm_gate_bwd_kernel<T, VEC, MODE, 512>
                                           : norm_gate_bwd_kernel<T, VEC, MODE, 1024>)
                          : (warps <= 16 ? norm_gate_fwd_kernel<T, VEC, MODE, 512>
                                         : norm_gate_fwd_kernel<T, VEC, MODE, 1024>);
  if (p.smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(p.smem)) !=
          cudaSuccess)
    return WKV_ERR_CUDA;
  return launch_kernel(kernel, p.grid, p.team_warps * p.teams * 32, p.smem, stream, a,
                       p.team_warps);
}

template <typename T>
int pick(const NormGateArgs& a, const Plan& p, bool vec, bool backward, cudaStream_t stream) {
  if (vec) {
    if (p.mode == kRow) return run<T, true, kRow>(a, p, backward, stream);
    if (p.mode == kLanes) return run<T, true, kLanes>(a, p, backward, stream);
    return run<T, true, kAny>(a, p, backward, stream);
  }
  if (p.mode == kRow) return run<T, false, kRow>(a, p, backward, stream);
  return run<T, false, kAny>(a, p, backward, stream);
}

bool vectors(const NormGateArgs& a) {
  uintptr_t all = 0;
  for (const void* q : {a.h, a.gate, a.x, (const void*)a.out, (const void*)a.y, a.dout, a.dy,
                        (const void*)a.dh, (const void*)a.dgate, (const void*)a.dx})
    all |= reinterpret_cast<uintptr_t>(q);
  return a.C % kE == 0 && all % 16 == 0;
}

}  // namespace

int64_t norm_gate_max_c() { return kMaxC; }

// Lines of partial sums: no more teams than the widest grid has (a 160-SM bound, so that the
// size does not depend on the device that is current).
size_t norm_gate_workspace_bytes(int64_t R, int64_t C) {
  if (R <= 0 || C <= 0 || C > kMaxC) return 0;
  const Plan p = plan_of(R, int(C), int(C), true, true, true, 160);
  return size_t(p.grid) * 3 * size_t(C) * sizeof(float);
}

int launch_norm_gate_forward(const NormGateArgs& a, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return WKV_ERR_CUDA;
  const bool vec = vectors(a);
  const Plan p = plan_of(a.R, a.C, a.group, vec, a.bf16, false, sms);
  return a.bf16 ? pick<__nv_bfloat16>(a, p, vec, false, stream)
                : pick<float>(a, p, vec, false, stream);
}

int launch_norm_gate_backward(const NormGateArgs& a, cudaStream_t stream) {
  const int sms = std::min(sm_count(), 160);
  if (sms <= 0) return WKV_ERR_CUDA;
  const bool vec = vectors(a);
  const Plan p = plan_of(a.R, a.C, a.group, vec, a.bf16, true, sms);
  const int rc = a.bf16 ? pick<__nv_bfloat16>(a, p, vec, true, stream)
                        : pick<float>(a, p, vec, true, stream);
  if (rc != WKV_OK) return rc;
  if (!a.dweight && !a.dscale && !a.dnext_weight) return WKV_OK;
  return launch_kernel(norm_gate_sum_kernel, dim3((a.C + 31) / 32, 3), 32 * kSlices, 0, stream,
                       a.partial, p.grid, a.C, a.dweight, a.dscale, a.dnext_weight);
}

}  // namespace wkv
