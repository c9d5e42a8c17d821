// Building blocks of the chunked gated delta rule (sm_100a): warp matrix instructions on bf16
// parts of fp32 values, the tokens' tiles in shared memory, and the small matrices of a group
// of 16 tokens.
//
// Why warp matrix instructions (mma.sync) and not tcgen05 here. A head's state is N x N and every
// product of the rule has a side of 64 or 128 and one of 16 tokens; the results feed the next
// product at once. With mma.sync the state stays in a warp's registers as the accumulator of one
// product and, since an accumulator tile and an operand tile are laid out alike, turns into the
// operand of the next by splitting it in place. tcgen05 would take every operand through shared
// memory (split, stored, fenced, waited for) twice a chunk: the matrix-state kernel, which does
// that with 64-token chunks, spends 34,000 cycles a chunk of which the tensor pipe is busy a
// sixth. mma.sync m16n8k16 runs at 549 TFLOP/s here (8 cycles an instruction and scheduler), a
// third of tcgen05's rate, and the rule at 16 tokens a group needs no more than the chain of
// latencies leaves time for.
//
// Precision: a state, and what is derived from it, is fp32; as an operand it is split into three
// bf16 parts (24 bits), so that products with bf16 inputs (one part) take 3 instructions and
// products of two split values 6 (hi hi, hi mid, mid hi, hi lo, lo hi, mid mid). fp32 inputs are
// split into three parts as well. What only bf16 outputs see leaves out the third part (2^-17 of
// a value against their own rounding of 2^-9).
#pragma once

#include <cstdint>

#include "wkv_async.cuh"
#include "wkv_device.cuh"
#include "wkv_internal.h"
#include "wkv_tc.cuh"

namespace wkv {
namespace gdr {

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

// c (16 x 8) += a (16 x 16) b (16 x 8), bf16 with fp32 sums. Thread (g, t) = (lane / 4, lane % 4)
// holds c: rows g, g + 8, columns 2t, 2t + 1; a: the same of two column tiles; b: rows (k) 2t,
// 2t + 1 and 8 on, column g.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two values as three packed bf16 parts.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  __nv_bfloat162 h, m, l;
  bf16_split3x2(make_float2(x, y), h, m, l);
  hi = bits(h);
  mid = bits(m);
  lo = bits(l);
}

// Two adjacent 16 x 8 accumulator tiles as a 16 x 16 operand in three parts.
__device__ __forceinline__ void split_tiles(const float (&t0)[4], const float (&t1)[4],
                                            uint32_t (&a)[3][4]) {
  split2(t0[0], t0[1], a[0][0], a[1][0], a[2][0]);
  split2(t0[2], t0[3], a[0][1], a[1][1], a[2][1]);
  split2(t1[0], t1[1], a[0][2], a[1][2], a[2][2]);
  split2(t1[2], t1[3], a[0][3], a[1][3], a[2][3]);
}

__device__ __forceinline__ void zero(float (&c)[4]) { c[0] = c[1] = c[2] = c[3] = 0.f; }

// The part pairs of a product, largest first: P operand parts of b (1: exact bf16, 3: split).
// FULL leaves out none of the six (three with P = 1) that fp32 accuracy takes; without it the
// pairs below 2^-16 go.
// Each pair is two digits, a's part and b's, in the packed lists.
template <int P, bool FULL>
struct Pairs {
  static constexpr int n = P == 1 ? (FULL ? 3 : 2) : (FULL ? 6 : 3);
  static constexpr uint32_t as = P == 1 ? 0x210u : 0x120100u;
  static constexpr uint32_t bs = P == 1 ? 0x000u : 0x102010u;
  __device__ static constexpr int a(int i) { return int(as >> (4 * i)) & 15; }
  __device__ static constexpr int b(int i) { return int(bs >> (4 * i)) & 15; }
};

// main += hi hi, corr += the other pairs, over two column tiles whose b parts are b[p][0..3]
// (tile 0: registers 0, 1; tile 1: 2, 3). Separate sums, so that the small products are not
// rounded into the large sum one by one.
template <int P, bool FULL>
__device__ __forceinline__ void mma_pairs(float (&main)[2][4], float (&corr)[2][4],
                                          const uint32_t (&a)[3][4], const uint32_t (&b)[P][4]) {
  using X = Pairs<P, FULL>;
#pragma unroll
  for (int i = 0; i < X::n; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n)
      mma(i == 0 ? main[n] : corr[n], a[X::a(i)], b[X::b(i)][2 * n], b[X::b(i)][2 * n + 1]);
}

// One sum, the small products first.
template <int P, bool FULL>
__device__ __forceinline__ void mma_up(float (&c)[2][4], const uint32_t (&a)[3][4],
                                       const uint32_t (&b)[P][4]) {
  using X = Pairs<P, FULL>;
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

// Inclusive sums over the group's 16 tokens of g log2(e), in every lane for token lane % 16, in
// fp64: decays between two tokens are differences of these, and a strong decay earlier in the
// group must not cost the later ones their digits.
__device__ __forceinline__ double decay_sums(float g, int lane) {
  double s = double(g < kLeastG ? kLeastG : g) * 1.4426950408889634;
#pragma unroll
  for (int d = 1; d < kG; d <<= 1) {
    const double below = __shfl_up_sync(0xffffffffu, s, d, 16);
    if ((lane & 15) >= d) s += below;
  }
  return s;
}

// The strictly lower part of (I + L)^-1 for a strictly lower 16 x 16 L in shared memory (pitch
// 20), by forward substitution, one column a lane; left in the same place.
constexpr int kLP = 20;
__device__ __forceinline__ void invert_group(float* L, int lane) {
  const int c = lane & 15;
  float x[kG];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kG; ++i) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < i; j += 4) {
      const float4 l = *reinterpret_cast<const float4*>(L + i * kLP + j);
      s0 = fmaf(l.x, x[j], s0);
      if (j + 1 < i) s1 = fmaf(l.y, x[j + 1], s1);
      if (j + 2 < i) s0 = fmaf(l.z, x[j + 2], s0);
      if (j + 3 < i) s1 = fmaf(l.w, x[j + 3], s1);
    }
    x[i] = i < c ? 0.f : i == c ? 1.f : -(s0 + s1);
  }
  __syncwarp();
  if (lane < kG) {
#pragma unroll
    for (int i = 0; i < kG; ++i) L[i * kLP + c] = i == c ? 0.f : x[i];
  }
  __syncwarp();
}

}  // namespace gdr
}  // namespace wkv
