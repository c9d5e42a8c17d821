// Building blocks of the chunked gated delta rule (sm_100a): warp matrix instructions on bf16
// parts of fp32 values, the tokens' tiles in shared memory, and the small matrices of a group
// of 16 tokens.
//
// Warp matrix instructions (mma.sync). A head's state is N x N and every product of the rule has a
// side of 64 or 128 and one of 16 tokens; the results feed the next product at once. The state stays
// in a warp's registers as the accumulator of one product and, since an accumulator tile and an
// operand tile are laid out alike, turns into the operand of the next by splitting it in place, and
// so do the group's small matrices. mma.sync m16n8k16 runs at 549 TFLOP/s here (8 cycles an
// instruction and scheduler), a third of tcgen05's rate; few heads are bound by the chain of a
// group's products, many by issue slots. tcgen05 takes its first operand from tensor memory, where
// the state could stay as well (tf32: the high part in place, the rest as a second operand), in
// chunks of 64 tokens; that form is not built and not measured here. (The matrix-state kernel, which
// takes every operand through shared memory, keeps the tensor pipe busy a sixth of the time: a
// property of its phases, one after the other, not of the unit.)
//
// Precision: a state, and what is derived from it, is fp32; as an operand it is split into three
// bf16 parts (24 bits), so that products with bf16 inputs (one part) take 3 instructions and
// products of two split values 6 (hi hi, hi mid, mid hi, hi lo, lo hi, mid mid: what is left out is
// below 2^-22). fp32 inputs are split into three parts as well. So a bf16 result is an fp32 result
// rounded once. (The read-outs of bf16 problems with two parts a factor, 2^-15 of a value: 754 us
// instead of 848 at 8 x 4096 x 64 x 64, and forty times as many of them on the other side of a
// rounding.)
#pragma once

#include <cstdint>

#include "wkv_async.cuh"
#include "wkv_device.cuh"
#include "wkv_internal.h"
#include "wkv_tc.cuh"

namespace wkv {
namespace gdr {

constexpr int kStagePitch = 24;  // bf16 staging of a warp's 16 x 16 outputs
constexpr int kG = 16;  // tokens of a group: one k step of the matrix instruction

// Below this a log-decay counts as a decay of zero: e^-200 is far below the smallest float.
constexpr float kLeastG = -200.f;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Four 8 x 8 tiles of bf16 pairs, each stored transposed.
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                       uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

// c (16 x 8) += a (16 x 16) b (16 x 8), bf16 with fp32 sums. Thread (g, t) = (lane / 4, lane % 4)
// holds c: rows g, g + 8, columns 2t, 2t + 1; a: the same of two column tiles; b: rows (k) 2t,
// 2t + 1 and 8 on, column g.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two values as three packed bf16 parts that add up to them, 8 bits each: mid and lo by cutting
// off, hi to the nearest, or cut off as well (CUT: two instructions less, for operands of a product
// with exact bf16 values, where no part pair is left out; two parts are then good to 2^-15). With
// integer adds, masks and byte permutes: packed conversions and fp32x2 arithmetic take as many
// instructions, but wait for one another and for the matrix instructions (16 such splits beside 16
// matrix instructions, cycles a scheduler: 435 with conversions, 298 this way; 129 for the matrix
// instructions alone).
template <bool CUT = false>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  constexpr uint32_t kTop = 0xffff0000u, kHalf = CUT ? 0u : 0x8000u;
  const uint32_t xh = __float_as_uint(x) + kHalf, yh = __float_as_uint(y) + kHalf;
  hi = __byte_perm(xh, yh, 0x7632);
  const float xr = __fsub_rn(x, __uint_as_float(xh & kTop));
  const float yr = __fsub_rn(y, __uint_as_float(yh & kTop));
  const uint32_t xm = __float_as_uint(xr), ym = __float_as_uint(yr);
  mid = __byte_perm(xm, ym, 0x7632);
  lo = __byte_perm(__float_as_uint(__fsub_rn(xr, __uint_as_float(xm & kTop))),
                   __float_as_uint(__fsub_rn(yr, __uint_as_float(ym & kTop))), 0x7632);
}

// Two adjacent 16 x 8 accumulator tiles as a 16 x 16 operand in three parts.
template <bool CUT = false>
__device__ __forceinline__ void split_tiles(const float (&t0)[4], const float (&t1)[4],
                                            uint32_t (&a)[3][4]) {
  split2<CUT>(t0[0], t0[1], a[0][0], a[1][0], a[2][0]);
  split2<CUT>(t0[2], t0[3], a[0][1], a[1][1], a[2][1]);
  split2<CUT>(t1[0], t1[1], a[0][2], a[1][2], a[2][2]);
  split2<CUT>(t1[2], t1[3], a[0][3], a[1][3], a[2][3]);
}

__device__ __forceinline__ void zero(float (&c)[4]) { c[0] = c[1] = c[2] = c[3] = 0.f; }

// s = c s + d (fp32x2 arithmetic keeps the matrix instructions waiting, see split2).
__device__ __forceinline__ void scale_add(float (&s)[4], float c, const float (&d)[4]) {
#pragma unroll
  for (int x = 0; x < 4; ++x) s[x] = fmaf(c, s[x], d[x]);
}

// The part pairs of a product, largest first: P operand parts of b (1: exact bf16, 3: split).
// Each pair is two digits, a's part and b's, in the packed lists.
template <int P>
struct Pairs {
  static constexpr int n = P == 1 ? 3 : 6;
  static constexpr uint32_t as = P == 1 ? 0x210u : 0x120100u;
  static constexpr uint32_t bs = P == 1 ? 0x000u : 0x102010u;
  __device__ static constexpr int a(int i) { return int(as >> (4 * i)) & 15; }
  __device__ static constexpr int b(int i) { return int(bs >> (4 * i)) & 15; }
};

// main += hi hi, corr += the other pairs, over two column tiles whose b parts are b[p][0..3]
// (tile 0: registers 0, 1; tile 1: 2, 3). Separate sums, so that the small products are not
// rounded into the large sum one by one.
template <int P>
__device__ __forceinline__ void mma_pairs(float (&main)[2][4], float (&corr)[2][4],
                                          const uint32_t (&a)[3][4], const uint32_t (&b)[P][4]) {
  using X = Pairs<P>;
#pragma unroll
  for (int i = 0; i < X::n; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n)
      mma(i == 0 ? main[n] : corr[n], a[X::a(i)], b[X::b(i)][2 * n], b[X::b(i)][2 * n + 1]);
}

// One sum, the small products first.
template <int P>
__device__ __forceinline__ void mma_up(float (&c)[2][4], const uint32_t (&a)[3][4],
                                       const uint32_t (&b)[P][4]) {
  using X = Pairs<P>;
#pragma unroll
  for (int i = X::n - 1; i >= 0; --i)
#pragma unroll
    for (int n = 0; n < 2; ++n)
      mma(c[n], a[X::a(i)], b[X::b(i)][2 * n], b[X::b(i)][2 * n + 1]);
}

// ---- operands from token tiles in shared memory ([token][channel] bf16, PITCH elements) ----

// b operand of (., 16 channels) x (16 channels, 16 tokens): columns are tokens.
__device__ __forceinline__ uint32_t at_tokens(int lane, int pitch) {
  const int m = lane >> 3, r = lane & 7;
  return uint32_t(((m >> 1) * 8 + r) * pitch + (m & 1) * 8) * 2u;
}
// b operand of (., 16 tokens) x (16 tokens, 16 channels): columns are channels (transposed load).
__device__ __forceinline__ uint32_t at_channels(int lane, int pitch) {
  const int m = lane >> 3, r = lane & 7;
  return uint32_t(((m & 1) * 8 + r) * pitch + (m >> 1) * 8) * 2u;
}
// 16 channels x 16 tokens as two accumulator tiles (transposed load): registers 0, 1 are tile 0's
// rows g and g + 8, 2, 3 tile 1's. Also the a operand of (channels, tokens) as registers 0..3.
__device__ __forceinline__ uint32_t at_transposed(int lane, int pitch) {
  const int m = lane >> 3, r = lane & 7;
  return uint32_t(((m >> 1) * 8 + r) * pitch + (m & 1) * 8) * 2u;
}

__device__ __forceinline__ float2 unpack(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// One 16-byte copy that leaves zeros where `ok` is false.
__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
template <int LEFT>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// ---- the tokens of a problem ----------------------------------------------------------------

// First token (over all rows) and length of sequence `seq`.
__device__ __forceinline__ int64_t sequence(const GdrArgs& a, int seq, int& len) {
  if (a.offsets == nullptr) {
    len = a.T;
    return int64_t(seq) * a.T;
  }
  const int t0 = min(max(a.offsets[seq], 0), a.T), t1 = min(max(a.offsets[seq + 1], 0), a.T);
  len = max(t1 - t0, 0);
  return t0;
}

// The sequence that comes `rank`-th when the longest come first: a walk is as long as its sequence,
// and a long one that starts last leaves the SMs idle (17 sequences of 9001 tokens, 32 x 128 heads:
// 428 us, 330 longest first). Up to 64 packed sequences; more are taken as they come. Whole warps.
__device__ __forceinline__ int by_length(const GdrArgs& a, int rank, int lane) {
  if (a.offsets == nullptr || a.n_seqs > 64) return rank;
  int len[2] = {-1, -1}, before[2] = {0, 0};
#pragma unroll
  for (int p = 0; p < 2; ++p)
    if (p * 32 + lane < a.n_seqs) sequence(a, p * 32 + lane, len[p]);
  for (int j = 0; j < a.n_seqs; ++j) {
    const int other = __shfl_sync(0xffffffffu, j < 32 ? len[0] : len[1], j & 31);
#pragma unroll
    for (int p = 0; p < 2; ++p)
      before[p] += other > len[p] || (other == len[p] && j < p * 32 + lane) ? 1 : 0;
  }
  const unsigned lo = __ballot_sync(0xffffffffu, lane < a.n_seqs && before[0] == rank);
  const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < a.n_seqs && before[1] == rank);
  return lo != 0 ? __ffs(lo) - 1 : 31 + __ffs(hi);
}

// Segments of a sequence: none of up to three, which three passes would not gain anything.
__device__ __forceinline__ int spans_of(int len, int tokens) {
  return len <= 3 * int64_t(tokens) ? 1 : (len - 1) / tokens + 1;
}

// What a CTA walks: a sequence, or segment `s` of its `count`.
struct Span {
  int seq, s, count, slot;
  int64_t t_seq, t0;  // first token of the sequence, of the span
  int len;
};
// The span of number `index` (by rank of length, or of segment); false where there is none. Whole
// warps.
__device__ __forceinline__ bool find_span(const GdrArgs& a, const GdrSegs& g, int index, int lane,
                                          Span& sp) {
  sp.s = 0;
  sp.count = 1;
  sp.slot = index;
  if (g.tokens == 0) {
    sp.seq = by_length(a, index, lane);
    sp.t_seq = sp.t0 = sequence(a, sp.seq, sp.len);
    return true;
  }
  if (a.offsets == nullptr) {
    sp.count = spans_of(a.T, g.tokens);
    sp.seq = index / sp.count;
    sp.s = index % sp.count;
  } else {  // up to 64 sequences
    int count[2] = {0, 0}, upto[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      int len = 0;
      if (p * 32 + lane < a.n_seqs) {
        sequence(a, p * 32 + lane, len);
        count[p] = spans_of(len, g.tokens);
      }
      upto[p] = count[p];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, upto[p], d);
        if (lane >= d) upto[p] += below;
      }
    }
    upto[1] += __shfl_sync(0xffffffffu, upto[0], 31);
    int found = -1, first = 0;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const unsigned who = __ballot_sync(0xffffffffu, index >= upto[p] - count[p] && index < upto[p]);
      if (who != 0) {
        found = p * 32 + __ffs(who) - 1;
        first = __shfl_sync(0xffffffffu, upto[p] - count[p], __ffs(who) - 1);
        sp.count = __shfl_sync(0xffffffffu, count[p], __ffs(who) - 1);
      }
    }
    if (found < 0) return false;
    sp.seq = found;
    sp.s = index - first;
  }
  int len;
  sp.t_seq = sequence(a, sp.seq, len);
  sp.t0 = sp.t_seq + int64_t(sp.s) * g.tokens;
  sp.len = sp.count == 1 ? len : min(len - sp.s * g.tokens, g.tokens);
  return true;
}

// A running log2-decay as an unevaluated sum of two floats (48 bits): decays between two tokens
// are differences of such sums, and a strong decay earlier must not cost later ones their digits.
// (fp64 took 4 times as long here: its unit is slow and its shuffles come in pairs.)
struct Decay {
  float hi, lo;
};
__device__ __forceinline__ Decay add(Decay a, Decay b) {
  const float s = __fadd_rn(a.hi, b.hi), v = __fsub_rn(s, a.hi);
  const float err = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, v)), __fsub_rn(b.hi, v));
  const float lo = err + (a.lo + b.lo);
  const float hi = __fadd_rn(s, lo);
  return {hi, __fsub_rn(lo, __fsub_rn(hi, s))};
}
// exp of the decay from one running sum to a later one.
__device__ __forceinline__ float decay_between(Decay to, Decay from) {
  return ex2((to.hi - from.hi) + (to.lo - from.lo));
}
// 2^d. The exponential's argument is rounded to 32 bits, up to 2^-19 of a decay of e^-40; what the
// rounding left out is put back. decay_between() goes without, 16 x 16 times a group.
__device__ __forceinline__ float power(Decay d) {
  const float e = ex2(d.hi);
  return fmaf(e, d.lo * 0.693147180559945f, e);
}
__device__ __forceinline__ float power_between(Decay to, Decay from) {
  return power(add(to, {-from.hi, -from.lo}));
}
__device__ __forceinline__ Decay shfl(Decay d, int lane) {
  return {__shfl_sync(0xffffffffu, d.hi, lane), __shfl_sync(0xffffffffu, d.lo, lane)};
}

// Inclusive sums of g log2(e) over each WIDTH adjacent lanes.
template <int WIDTH>
__device__ __forceinline__ Decay decay_sums(float g, int lane) {
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kLog2eLo = float(1.4426950408889634 - double(kLog2e));
  if (g < kLeastG) g = kLeastG;
  Decay s;
  s.hi = __fmul_rn(g, kLog2e);
  s.lo = fmaf(g, kLog2eLo, fmaf(g, kLog2e, -s.hi));
#pragma unroll
  for (int d = 1; d < WIDTH; d <<= 1) {
    const Decay below = {__shfl_up_sync(0xffffffffu, s.hi, d, WIDTH),
                         __shfl_up_sync(0xffffffffu, s.lo, d, WIDTH)};
    const Decay sum = add(s, below);
    if ((lane & (WIDTH - 1)) >= d) s = sum;
  }
  return s;
}

// The strictly lower part of (I + L)^-1 for a strictly lower 16 x 16 L in shared memory (pitch
// 20), left in the same place. The two diagonal 8 x 8 blocks A and B by forward substitution, one
// column a lane; the block below them is -B^-1 (L21 A^-1). `tmp`: 8 x 8 floats.
constexpr int kLP = 20;
constexpr int kLTmp = 64;
__device__ __forceinline__ void invert_group(float* L, float* tmp, int lane) {
  const int b = (lane >> 3) & 1, c = lane & 7;
  const float* const D = L + b * 8 * (kLP + 1);
  __syncwarp();
  float r[8][8];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    const float4 lo = *reinterpret_cast<const float4*>(D + i * kLP);
    r[i][0] = lo.x; r[i][1] = lo.y; r[i][2] = lo.z; r[i][3] = lo.w;
    if (i > 4) {
      const float4 hi = *reinterpret_cast<const float4*>(D + i * kLP + 4);
      r[i][4] = hi.x; r[i][5] = hi.y; r[i][6] = hi.z; r[i][7] = hi.w;
    }
  }
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < i; ++j) {
      if (j & 1)
        s1 = fmaf(r[i][j], x[j], s1);
      else
        s0 = fmaf(r[i][j], x[j], s0);
    }
    x[i] = i < c ? 0.f : i == c ? 1.f : -(s0 + s1);
  }
  __syncwarp();
  // A^-1 and B^-1 with their unit diagonals
  if (lane < kG) {
#pragma unroll
    for (int i = 0; i < 8; ++i) L[(b * 8 + i) * kLP + b * 8 + c] = x[i];
  }
  __syncwarp();
  const int row = lane >> 2, col = (lane & 3) * 2;
  auto times = [&](const float* left, const float* right, int pitch) {
    const float4 l0 = *reinterpret_cast<const float4*>(left);
    const float4 l1 = *reinterpret_cast<const float4*>(left + 4);
    const float l[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 y = *reinterpret_cast<const float2*>(right + k * pitch + col);
      s = make_float2(fmaf(l[k], y.x, s.x), fmaf(l[k], y.y, s.y));
    }
    return s;
  };
  *reinterpret_cast<float2*>(tmp + row * 8 + col) = times(L + (8 + row) * kLP, L, kLP);
  __syncwarp();
  const float2 t = times(L + (8 + row) * kLP + 8, tmp, 8);
  *reinterpret_cast<float2*>(L + (8 + row) * kLP + col) = make_float2(-t.x, -t.y);
  if (lane < kG) L[lane * (kLP + 1)] = 0.f;
  __syncwarp();
}

// One tensor's tile of a step: kStep rows of ROW bytes into rows PITCH bytes apart, 16 bytes a
// copy, by THREADS threads. src: the step's first row; rows past `left` become zeros.
template <int STEP, int ROW, int PITCH, int THREADS>
__device__ __forceinline__ void load_tile(uint32_t dst, const void* src, int64_t stride, int left,
                                          int thread) {
  constexpr int kChunks = ROW / 16, kAtOnce = THREADS / kChunks;
  static_assert(THREADS % kChunks == 0 && STEP % kAtOnce == 0, "whole rows a pass");
  const int t = thread / kChunks, c = thread % kChunks;
  const char* p = static_cast<const char*>(src) + t * stride + c * 16;
  dst += uint32_t(t * PITCH + c * 16);
  if (left >= STEP) {
#pragma unroll
    for (int j = 0; j < STEP / kAtOnce; ++j)
      cp_async_16z(dst + j * kAtOnce * PITCH, p + j * kAtOnce * stride, true);
  } else {
#pragma unroll 1
    for (int j = 0; j < STEP / kAtOnce; ++j) {
      const bool ok = t + j * kAtOnce < left;
      cp_async_16z(dst + j * kAtOnce * PITCH, ok ? p + j * kAtOnce * stride : src, ok);
    }
  }
}

// A warp's 16 tokens x N of fp32 (pitch N + 4) into three bf16 parts (pitch N + 8, PART bytes
// apart).
template <int N, int PART>
__device__ __forceinline__ void split_tokens(const float* src, unsigned char* dst, int lane) {
#pragma unroll 8
  for (int j = 0; j < kG * N / 128; ++j) {
    const int at = j * 32 + lane, r = at / (N / 4), c = (at % (N / 4)) * 4;
    const float4 x = *reinterpret_cast<const float4*>(src + r * (N + 4) + c);
    uint2 p0, p1, p2;
    split2(x.x, x.y, p0.x, p1.x, p2.x);
    split2(x.z, x.w, p0.y, p1.y, p2.y);
    unsigned char* d = dst + (r * (N + 8) + c) * 2;
    *reinterpret_cast<uint2*>(d) = p0;
    *reinterpret_cast<uint2*>(d + PART) = p1;
    *reinterpret_cast<uint2*>(d + 2 * PART) = p2;
  }
}

// What the producers hand over for a group of 16 tokens: operand fragments (three parts, a uint4
// a lane) of an inverse less its diagonal and of a read matrix, and vectors over the tokens.
struct GroupMats {
  uint4 inv[3][32];
  uint4 read[3][32];
  float decay[kG];  // C_i
  float out[kG];    // scale C_i
  float write[kG];  // forward: exp(c_16 - c_j) beta_j; reverse: exp(c_16 - c_j)
  float beta[kG];   // reverse only
  float end;        // C
  float pad[3];
};

// Sizes of the two kernels that walk sequences in groups: steps of NG groups, prepared by NP
// producer warps (NG, or 2 NG: two a group), and NC consumer warps of 16 value channels each. "v"
// is whatever comes per value head: v, or dy.
template <typename T, int N, int NC, int NG, int NP>
struct Shape {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kParts = kBf16 ? 1 : 3;      // operand parts of q and k
  static constexpr int kGroups = NG, kProducers = NP;
  static constexpr bool kPairs = NP == 2 * NG;      // of producers
  static_assert(kPairs || (NP == NG && kBf16), "one or two producers a group");
  static constexpr int kStep = NG * kG;             // tokens of a step
  static constexpr int kPitch = N + 8;              // bf16 tiles (16-byte rows, no conflicts)
  static constexpr int kPitchF = N + 4;             // fp32 tiles
  static constexpr int kTile = kStep * kPitch * 2;  // bytes of a bf16 tile
  static constexpr int kTileF = kStep * kPitchF * 4;
  static constexpr int kVRows = 16 * NC;            // value channels of the CTA
  static constexpr int kVPitch = kBf16 ? kVRows + 8 : kVRows + 4;
  static constexpr int kVTile = kStep * kVPitch * int(sizeof(T));
  // bf16: rings of three for q, k, v. fp32: q and k arrive in a ring of two and are split into
  // two sets of parts; v in a ring of three.
  static constexpr int kQK = kBf16 ? 3 * 2 * kTile : 2 * 2 * kTileF;
  static constexpr int kSplit = kBf16 ? 0 : 2 * 2 * 3 * kTile;
  static constexpr int kOffSplit = kQK;
  static constexpr int kOffV = kOffSplit + kSplit;
  static constexpr int kOffMats = kOffV + 3 * kVTile;
  static constexpr int kOffL = kOffMats + 2 * NG * int(sizeof(GroupMats));
  static constexpr int kOffY = kOffL + NG * (kG * kLP + kLTmp) * 4;
  static constexpr int kSmem = kOffY + (kBf16 ? NC * kG * kStagePitch * 2 : 0);
  static constexpr int kThreads = 32 * (NC + NP);
};


// A B^T over the channels of a group's tokens; A and B: 0 for k, 1 for q, at byte offset `off` of
// every part's tile.
template <int N, int P, class Tile>
__device__ __forceinline__ void group_product(float (&c)[2][4], Tile tile, int A, int B,
                                              uint32_t off) {
  float corr[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n) zero(c[n]), zero(corr[n]);
#pragma unroll
  for (int ch = 0; ch < N; ch += 16) {
    uint32_t b[P][4], a[3][4], r[4];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      ldsm4(r, tile(A, p) + off + ch * 2);
      // the same four 8 x 8 blocks in the order of an a operand
      a[p][0] = r[0]; a[p][1] = r[2]; a[p][2] = r[1]; a[p][3] = r[3];
      ldsm4(b[p], tile(B, p) + off + ch * 2);
    }
    if constexpr (P == 1) {
#pragma unroll
      for (int n = 0; n < 2; ++n) mma(c[n], a[0], b[0][2 * n], b[0][2 * n + 1]);
    } else {
      mma_pairs<P>(c, corr, a, b);
    }
  }
  if (P > 1) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) c[n][x] += corr[n][x];
  }
}

// Two pairs of adjacent accumulator tiles (rows: the product's columns) as the b operand of a
// 16 x 16 product, three parts of a uint4 a lane.
__device__ __forceinline__ void put_fragment(uint4 (*to)[32], const float2& t00, const float2& t01,
                                             const float2& t10, const float2& t11, int lane) {
  uint4 f[3];
  split2(t00.x, t00.y, f[0].x, f[1].x, f[2].x);
  split2(t01.x, t01.y, f[0].y, f[1].y, f[2].y);
  split2(t10.x, t10.y, f[0].z, f[1].z, f[2].z);
  split2(t11.x, t11.y, f[0].w, f[1].w, f[2].w);
#pragma unroll
  for (int p = 0; p < 3; ++p) to[p][lane] = f[p];
}

// A warp's 16 channels x 16 tokens (accumulator tiles) to rows of tokens in global memory:
// fp32 eight channels of a token at a time, bf16 through 16 x 24 elements of shared memory.
template <typename T>
__device__ __forceinline__ void put_tokens(T* to, int64_t row, const float (&x)[2][4], int left,
                                           __nv_bfloat16* stage, int lane) {
  if constexpr (sizeof(T) == 2) {
    uint32_t r[2][2];  // token tile, channel half
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int z = 0; z < 2; ++z)
        r[n][z] = bits(__float22bfloat162_rn(make_float2(x[n][2 * z], x[n][2 * z + 1])));
    __syncwarp();
    // tile m of the four: tokens 8 (m / 2).., channels 8 (m % 2)..
    stsm4t(smem_u32(stage) + uint32_t(((lane >> 4) * 8 + (lane & 7)) * kStagePitch +
                                      ((lane >> 3) & 1) * 8) * 2u,
           r[0][0], r[0][1], r[1][0], r[1][1]);
    __syncwarp();
    const int tok = lane >> 1, c = (lane & 1) * 8;
    if (tok < left)
      *reinterpret_cast<uint4*>(to + tok * row + c) =
          *reinterpret_cast<const uint4*>(stage + tok * kStagePitch + c);
  } else {
    const int g4 = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int tok = n * 8 + 2 * t4 + y;
        if (tok < left) {
          to[tok * row + g4] = x[n][y];
          to[tok * row + g4 + 8] = x[n][2 + y];
        }
      }
  }
}

// 16 channels x 16 tokens of v (or dy) as accumulator values; for bf16 also the raw operand.
template <typename T, class X>
__device__ __forceinline__ void get_tokens(float (&vv)[2][4], uint32_t (&raw)[4],
                                           const unsigned char* tile, int token, int channel,
                                           int lane) {
  if constexpr (sizeof(T) == 2) {
    ldsm4t(raw, smem_u32(tile) + uint32_t(token * X::kVPitch + channel) * 2u +
                    at_transposed(lane, X::kVPitch));
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float2 lo = unpack(raw[2 * n]), hi = unpack(raw[2 * n + 1]);
      vv[n][0] = lo.x; vv[n][1] = lo.y; vv[n][2] = hi.x; vv[n][3] = hi.y;
    }
  } else {
    const float* vp = reinterpret_cast<const float*>(tile) + token * X::kVPitch + channel;
    const int g4 = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        vv[n][x] = vp[(n * 8 + 2 * t4 + (x & 1)) * X::kVPitch + g4 + (x >> 1) * 8];
  }
}

// A warp's 16 rows x N of a state, as accumulator tiles, from and to global memory.
template <int N>
__device__ __forceinline__ void get_state(float (&S)[N / 8][4], const float* from, int lane) {
  const int g4 = lane >> 2, t4 = lane & 3;
#pragma unroll
  for (int n = 0; n < N / 8; ++n) {
    zero(S[n]);
    if (from != nullptr) {
      const float2 x = *reinterpret_cast<const float2*>(from + g4 * N + n * 8 + 2 * t4);
      const float2 z = *reinterpret_cast<const float2*>(from + (g4 + 8) * N + n * 8 + 2 * t4);
      S[n][0] = x.x; S[n][1] = x.y; S[n][2] = z.x; S[n][3] = z.y;
    }
  }
}
template <int N>
__device__ __forceinline__ void put_state(float* to, const float (&S)[N / 8][4], int lane) {
  const int g4 = lane >> 2, t4 = lane & 3;
#pragma unroll
  for (int n = 0; n < N / 8; ++n) {
    *reinterpret_cast<float2*>(to + g4 * N + n * 8 + 2 * t4) = make_float2(S[n][0], S[n][1]);
    *reinterpret_cast<float2*>(to + (g4 + 8) * N + n * 8 + 2 * t4) = make_float2(S[n][2], S[n][3]);
  }
}

// Rows r0.. of the identity.
template <int N>
__device__ __forceinline__ void unit_state(float (&S)[N / 8][4], int r0, int lane) {
  const int row = r0 + (lane >> 2), col = 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < N / 8; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      S[n][x] = row + (x >> 1) * 8 == n * 8 + col + (x & 1) ? 1.f : 0.f;
}

// Where a span's walk starts and what a summary (see GdrSegs) is of: S_in of this warp's rows.
// False: the CTA has nothing to walk. `first` and `last`: of the walk's spans.
template <int N, bool SUMMARY>
__device__ __forceinline__ bool start_state(float (&S)[N / 8][4], const GdrArgs& a,
                                            const GdrSegs& g, const Span& sp, bool first, bool last,
                                            bool unit, int back, const float* given, int h, int r0,
                                            int lane) {
  const int64_t at = (int64_t(sp.seq) * a.H + h) * N * N + int64_t(r0) * N;
  const int64_t slot_at = (int64_t(sp.slot) * a.H + h) * N * N + int64_t(r0) * N;
  const float* const start = given == nullptr ? nullptr : given + at;
  if (!SUMMARY) {
    get_state<N>(S,
                 g.tokens == 0 ? start
                 : first       ? g.unit + slot_at
                               : g.leave + slot_at - int64_t(back) * a.H * N * N,
                 lane);
    return true;
  }
  if (unit && first) {
    // kept where the last span's result cannot overwrite it
    get_state<N>(S, start, lane);
    put_state<N>(g.unit + slot_at, S, lane);
    return false;
  }
  if (last) return false;
  if (unit)
    unit_state<N>(S, r0, lane);
  else
    get_state<N>(S, first ? start : nullptr, lane);
  return true;
}

// Four consumers and steps of two groups everywhere (heads of 128 are two CTAs). bf16: two
// producers, 168 registers and two CTAs an SM where there is work for them, or four producers and
// one CTA, which is quicker alone (us, singles / pairs: 1 x 2048 x 8 x 64: 134 / 119, 1 x 2048 x 8
// x 128: 203 / 177) and slower where CTAs queue (8 x 4096 x 64 x 64: 849 / 932, 16 x 1024 x 32 x
// 128: 587 / 625). fp32 splits q and k on the way, which takes four producers always (two / four:
// 8 x 1024 x 64 x 64: 496 / 379, 1 x 2048 x 8 x 64: 253 / 186).
enum GdrWalkForm { kGdrWalkSingles, kGdrWalkPairs, kGdrWalkError };
inline GdrWalkForm gdr_walk_form(const GdrArgs& a, int64_t spans) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return kGdrWalkError;
  return spans * a.H * (a.N / 64) <= sms ? kGdrWalkPairs : kGdrWalkSingles;
}

// The producers' part of both kernels. Step s of a walk has the tokens from s kStep, counted from
// the sequence's first token forwards, or (REVERSE) from its last step backwards. While the
// consumers work on step i the producers copy step i + 2 in and prepare step i + 1: everything that
// does not depend on the state. One barrier a step. A pair of warps shares a group where
// X::kPairs: one makes the inverse, the other the read matrix and the vectors.
//   forward: (I + A)^-1 - I with A_ij = D_ij (k_i . k_j) beta_j, and scale D_ij (q_i . k_j) beta_j,
//   reverse: the transpose of (I + A')^-1 - I with A'_ij = D_ij (k_i . k_j) beta_i, and
//            scale D_ij (q_i . k_j),
// as operands whose columns are the tokens that the product is for.
struct Walk {
  int h, hk, part, len, steps;
  int64_t t0;
};

// bf16 part p of q (which = 1) or k (0) of step s
template <class X>
__device__ __forceinline__ uint32_t tile_of(uint32_t sb, int s, int which, int p) {
  if (X::kBf16) return sb + ((s % 3) * 2 + which) * X::kTile;
  return sb + X::kOffSplit + (((s & 1) * 2 + which) * 3 + p) * X::kTile;
}

template <typename T, int N, class X, bool REVERSE>
__device__ __forceinline__ void produce(const GdrArgs& a, const void* vals, const Walk& w,
                                        unsigned char* smem, int pw, int lane) {
  constexpr int P = X::kParts, NP = X::kProducers, kSize = int(sizeof(T));
  const int group = X::kPairs ? pw >> 1 : pw;
  const bool inverts = !X::kPairs || (pw & 1) == 0, reads = !X::kPairs || (pw & 1) == 1;
  const uint32_t sb = smem_u32(smem);
  const int g4 = lane >> 2, t4 = lane & 3, pt = pw * 32 + lane;
  const int64_t qk_row = int64_t(a.Hk) * N, v_row = int64_t(a.H) * N;
  const T* const q = static_cast<const T*>(a.q) + w.t0 * qk_row + int64_t(w.hk) * N;
  const T* const k = static_cast<const T*>(a.k) + w.t0 * qk_row + int64_t(w.hk) * N;
  const T* const v =
      static_cast<const T*>(vals) + w.t0 * v_row + int64_t(w.h) * N + w.part * X::kVRows;
  const float* const gp = a.g + w.t0 * a.H + w.h;
  const float* const bp = a.beta + w.t0 * a.H + w.h;
  GroupMats* const mats = reinterpret_cast<GroupMats*>(smem + X::kOffMats);  // [2][groups]
  float* const Ls = reinterpret_cast<float*>(smem + X::kOffL);
  float* const L = Ls + group * kG * kLP;
  float* const tmp = Ls + X::kGroups * kG * kLP + group * kLTmp;
  auto first_of = [&](int s) { return (REVERSE ? w.steps - 1 - s : s) * X::kStep; };

  auto load = [&](int s) {
    if (s < w.steps) {
      const int first = first_of(s), left = w.len - first;
      constexpr int kPitch = X::kBf16 ? X::kPitch * 2 : X::kPitchF * 4;
      const uint32_t kd = X::kBf16 ? tile_of<X>(sb, s, 0, 0) : sb + (s & 1) * 2 * X::kTileF;
      const uint32_t qd = X::kBf16 ? tile_of<X>(sb, s, 1, 0) : kd + X::kTileF;
      load_tile<X::kStep, N * kSize, kPitch, NP * 32>(kd, k + first * qk_row, qk_row * kSize, left,
                                                      pt);
      load_tile<X::kStep, N * kSize, kPitch, NP * 32>(qd, q + first * qk_row, qk_row * kSize, left,
                                                      pt);
      load_tile<X::kStep, X::kVRows * kSize, X::kVPitch * kSize, NP * 32>(
          sb + X::kOffV + (s % 3) * X::kVTile, v + first * v_row, v_row * kSize, left, pt);
    }
    cp_async_commit();
  };
  // g and beta of this lane's token of the next step
  float g_next = 0.f, b_next = 0.f;
  auto load_g = [&](int s) {
    const int tok = first_of(s) + group * kG + (lane & 15);
    const bool ok = s < w.steps && tok < w.len;
    g_next = ok ? gp[int64_t(tok) * a.H] : 0.f;
    b_next = ok ? bp[int64_t(tok) * a.H] : 0.f;
  };

  load(0);
  load_g(0);
  load(1);
  for (int i = -1; i < w.steps; ++i) {
    const int s = i + 1;  // the step to prepare
    if (i >= 0) load(i + 2);
    if (s < w.steps) {
      const float gv = g_next, bv = b_next;
      load_g(s + 1);
      cp_async_wait<1>();
      asm volatile("bar.sync 1, %0;" ::"n"(NP * 32) : "memory");
      if (!X::kBf16) {
        // the group's k (one warp) and q (the other) into three parts
        const int which = pw & 1, row = group * kG;
        split_tokens<N, X::kTile>(
            reinterpret_cast<const float*>(smem + ((s & 1) * 2 + which) * X::kTileF) +
                row * X::kPitchF,
            smem + (tile_of<X>(sb, s, which, 0) - sb) + row * X::kPitch * 2, lane);
        asm volatile("bar.sync 1, %0;" ::"n"(NP * 32) : "memory");
      }
      auto tile = [&](int which, int p) { return tile_of<X>(sb, s, which, p); };
      const uint32_t off =
          at_tokens(lane, X::kPitch) + uint32_t(group * kG * X::kPitch) * 2u;
      const Decay cs = decay_sums<kG>(gv, lane);
      const Decay cr[2] = {shfl(cs, g4), shfl(cs, g4 + 8)};
      GroupMats& m = mats[(s & 1) * X::kGroups + group];
      if (inverts) {
        float kk[2][4];
        group_product<N, P>(kk, tile, 0, 0, off);
        const float br[2] = {__shfl_sync(0xffffffffu, bv, g4),
                             __shfl_sync(0xffffffffu, bv, g4 + 8)};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int col = n * 8 + 2 * t4 + y;
            const Decay cc = shfl(cs, col);
            const float bc = __shfl_sync(0xffffffffu, bv, col);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float d = decay_between(cr[z], cc) * (REVERSE ? br[z] : bc);
              kk[n][2 * z + y] = g4 + z * 8 > col ? d * kk[n][2 * z + y] : 0.f;
            }
          }
#pragma unroll
          for (int z = 0; z < 2; ++z)
            *reinterpret_cast<float2*>(L + (g4 + z * 8) * kLP + n * 8 + 2 * t4) =
                make_float2(kk[n][2 * z], kk[n][2 * z + 1]);
        }
        invert_group(L, tmp, lane);
        // operand entry (contraction j or j + 1, column i): the inverse's (i, j), or (j, i)
        auto pair = [&](int i, int j) {
          return REVERSE ? make_float2(L[j * kLP + i], L[(j + 1) * kLP + i])
                         : *reinterpret_cast<const float2*>(L + i * kLP + j);
        };
        put_fragment(m.inv, pair(g4, 2 * t4), pair(g4, 8 + 2 * t4), pair(g4 + 8, 2 * t4),
                        pair(g4 + 8, 8 + 2 * t4), lane);
        __syncwarp();
      }
      if (reads) {
        // q_i . k_j, rows i; reverse: rows j
        float qk[2][4];
        group_product<N, P>(qk, tile, REVERSE ? 0 : 1, REVERSE ? 1 : 0, off);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int col = n * 8 + 2 * t4 + y;
            const Decay cc = shfl(cs, col);
            const float bc = REVERSE ? 1.f : __shfl_sync(0xffffffffu, bv, col);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int row = g4 + z * 8, x = 2 * z + y;
              const float d =
                  REVERSE ? col >= row ? decay_between(cc, cr[z]) : 0.f
                          : row >= col ? decay_between(cr[z], cc) * bc : 0.f;
              qk[n][x] = a.scale * (d * qk[n][x]);
            }
          }
        auto two = [](const float(&t)[4], int j) { return make_float2(t[j], t[j + 1]); };
        put_fragment(m.read, two(qk[0], 0), two(qk[1], 0), two(qk[0], 2), two(qk[1], 2), lane);
        const Decay last = shfl(cs, 15);
        if (lane < kG) {
          const float d = power(cs), to_end = power_between(last, cs);
          m.decay[lane] = d;
          m.out[lane] = a.scale * d;
          m.write[lane] = REVERSE ? to_end : to_end * bv;
          if (REVERSE) m.beta[lane] = bv;
          if (lane == 15) m.end = d;
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace gdr
}  // namespace wkv
