// Gated delta rule over long sequences with few heads: segments side by side (sm_100a).
//
// Over a segment the rule is linear in the state that enters: S_out = S_in M + B, with M and B
// from the segment's tokens (M: the walk that starts from the identity, without values; B: from
// zero). So one pass walks every segment for its M and B, this file's kernel passes the states
// from segment to segment, and a second pass walks the segments from the right states for the
// outputs. Three times the work of one pass, over as many times the CTAs. The reverse walk is the
// same with the segments in the other order (its M is the transpose).
//
// Measured, 1 x 16384 x 8 x 64 fp32 in 18 segments: 151 + 41 + 99 us against 1,480 whole. With
// four segments a sequence (the fewest taken), whole / in segments, us: 1 x 1024 x 8 x 64 bf16 62 /
// 46, fp32 95 / 60; 1 x 4096 x 37 x 64 bf16 235 / 157; 1 x 2048 x 16 x 128 bf16 178 / 141; 1 x 1024
// x 18 x 128 bf16 92 / 88.
#include <algorithm>

#include "wkv_gdr.cuh"

namespace wkv {

using namespace gdr;

namespace {

// leave[s] = leave[s - 1] M_s + B_s, one CTA for 64 rows of a head, 16 a warp in registers. M_s
// goes through shared memory in three bf16 parts; the next one comes in meanwhile.
template <int N>
__global__ void __launch_bounds__(128) gdr_combine_kernel(GdrArgs a, GdrSegs g, bool reverse) {
  constexpr int kPitch = N + 8, kPart = N * kPitch * 2, kQuads = N / 4;
  constexpr int kPer = N * kQuads / 128;  // float4s of M a thread
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.x % (N / 64) * 64 + warp * 16;
  const int sh = blockIdx.x / (N / 64), seq = sh / a.H, h = sh % a.H;
  // the sequence's segments
  int len, base = 0, count = 0;
  for (int s = 0; s <= seq; ++s) {
    sequence(a, s, len);
    base += count;
    count = spans_of(len, g.tokens);
    if (a.offsets == nullptr) {
      base = seq * count;
      break;
    }
  }
  if (base + count > g.slots) return;
  const int64_t head = int64_t(a.H) * N * N;
  auto slot_at = [&](int k) {
    return int64_t(reverse ? base + count - 1 - k : base + k) * head + int64_t(h) * N * N;
  };
  if (count <= 2) return;
  const float4* const raw = reinterpret_cast<const float4*>(smem + 3 * kPart);
  auto fetch = [&](int k) {
    const float4* const M = reinterpret_cast<const float4*>(g.unit + slot_at(k));
#pragma unroll 8
    for (int x = 0; x < kPer; ++x) {
      const int i = threadIdx.x + x * 128;
      cp_async_16z(sb + 3 * kPart + i * 16, M + i, true);
    }
  };
  fetch(1);
  float S[N / 8][4];
  get_state<N>(S, g.leave + slot_at(0) + r0 * N, lane);
  for (int k = 1; k < count - 1; ++k) {
    float B[N / 8][4];
    get_state<N>(B, g.leave + slot_at(k) + r0 * N, lane);
    cp_async_wait_all();
    __syncthreads();  // M is there, the last one's parts have been read
#pragma unroll 8
    for (int x = 0; x < kPer; ++x) {
      const int i = threadIdx.x + x * 128;
      const float4 m = raw[i];
      unsigned char* d = smem + (i / kQuads * kPitch + (i % kQuads) * 4) * 2;
      uint2 p0, p1, p2;
      split2(m.x, m.y, p0.x, p1.x, p2.x);
      split2(m.z, m.w, p0.y, p1.y, p2.y);
      *reinterpret_cast<uint2*>(d) = p0;
      *reinterpret_cast<uint2*>(d + kPart) = p1;
      *reinterpret_cast<uint2*>(d + 2 * kPart) = p2;
    }
    __syncthreads();
    if (k + 1 < count - 1) fetch(k + 1);
    // B += S M, every 16 of the contraction summed on their own and added in fp32
    const uint32_t ch = sb + at_channels(lane, kPitch);
#pragma unroll
    for (int c = 0; c < N; c += 16) {
      uint32_t sp[3][4];
      split_tiles(S[c / 8], S[c / 8 + 1], sp);
#pragma unroll
      for (int n = 0; n < N / 8; n += 2) {
        uint32_t mb[3][4];
#pragma unroll
        for (int p = 0; p < 3; ++p) ldsm4t(mb[p], ch + p * kPart + c * kPitch * 2 + n * 16);
        float d[2][4];
        zero(d[0]);
        zero(d[1]);
        mma_up<3>(d, sp, mb);
#pragma unroll
        for (int x = 0; x < 4; ++x) B[n][x] += d[0][x], B[n + 1][x] += d[1][x];
      }
    }
#pragma unroll
    for (int n = 0; n < N / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) S[n][x] = B[n][x];
    put_state<N>(g.leave + slot_at(k) + r0 * N, S, lane);
  }
}

template <int N>
int combine(const GdrArgs& a, const GdrSegs& segs, bool reverse, cudaStream_t stream) {
  constexpr int kSmem = 3 * N * (N + 8) * 2 + N * N * 4;
  auto* kernel = gdr_combine_kernel<N>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
      cudaSuccess)
    return WKV_ERR_CUDA;
  return launch_kernel(kernel, unsigned(a.n_seqs * a.H * (N / 64)), 128, kSmem, stream, a, segs,
                       reverse);
}

}  // namespace

int64_t gdr_plan_segments(const GdrArgs& a, GdrSegs* segs) {
  *segs = GdrSegs();
  constexpr int kLeast = 256;  // tokens of a segment: passing a state on costs as much as 64 to 128
  constexpr int kGain = 4;     // segments of a sequence that make three passes' work worth it
  if (int64_t(a.T) < int64_t(kGain) * kLeast) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  const int cap = sms / (a.H * (a.N / 64));  // spans that fit the GPU at once
  const bool packed = a.offsets != nullptr;
  if (packed && a.n_seqs > 64) return 0;  // find_span
  // Packed lengths are not known here: one span a sequence, the rest cut from whatever is long.
  // Where nothing is, every sequence is one span, and the two other passes are for nothing; so they
  // have to be short enough for twice the gain. (8 x 64, whole / in segments, us: 3700, 100, 100 and
  // 100 tokens bf16 211 / 82, fp32 328 / 115; four of 1000 bf16 62 / 64, fp32 95 / 97.)
  const int want = packed ? cap - a.n_seqs : cap / a.n_seqs, least = packed ? 2 * kGain : kGain;
  if (want < least) return 0;
  int tokens = (a.T + want - 1) / want;
  tokens = (std::max(tokens, kLeast) + 63) / 64 * 64;
  const int count = (a.T + tokens - 1) / tokens;
  if (count < least) return 0;
  segs->tokens = tokens;
  segs->slots = packed ? a.T / tokens + a.n_seqs : a.n_seqs * count;
  return int64_t(segs->slots) * a.H * a.N * a.N * 4 * 2;
}

int launch_gdr_combine(const GdrArgs& a, const GdrSegs& segs, bool reverse, cudaStream_t stream) {
  return a.N == 64 ? combine<64>(a, segs, reverse, stream) : combine<128>(a, segs, reverse, stream);
}

}  // namespace wkv
