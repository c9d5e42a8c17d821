// Gated delta rule over sequences, in groups of 16 tokens (sm_100a).
//
// With c_i the sum of g over the group up to token i, D_ij = exp(c_i - c_j) (j <= i), C_i =
// exp(c_i), C the whole group's decay, and S_0 the state that enters:
//   e = (I + A)^-1 (V - C_i K S_0^T),   A_ij = D_ij (k_i . k_j) beta_j  (j < i)
//   y = scale (C_i Q S_0^T + (D_ij q_i . k_j beta_j)_{j <= i} e)
//   S = C S_0 + (exp(c_16 - c_j) beta_j e_j)^T K.
// No row of S (value channel) needs another, so a warp keeps 16 rows for the whole sequence in
// registers, and the products run transposed (channels x tokens): S_0 K^T and S_0 Q^T take the
// state as operand a in place, e^T and the weighted e^T become operands as they come out.
//
// Bound by issue slots: a group of a head takes 3,080 warp instructions, 400 of them matrix
// instructions of 8 cycles that hold the issue port for about 4.5, so that the matrix time adds to
// the rest instead of hiding behind it (8 x 4096 x 64 x 64 bf16: 848 us, matrix pipe half busy,
// 0.20 of HBM). More warps do not help (three CTAs of 96 registers took 8 % longer), fewer
// instructions do.
// Few heads are bound by a group's chain of products, 0.9 us (bf16, 64): see wkv_gdr_seg.cu.
//
// A CTA has 64 value channels of one head of one sequence (or of a segment of it): two or four
// producer warps, see produce(), and four consumer warps.
#include "wkv_gdr.cuh"

namespace wkv {

using namespace gdr;

namespace {

// SUMMARY: not the outputs but what a segment does to the state that enters it: the state leaving
// it from zero (from s0 in a sequence's first segment), and from the identity without values.
template <typename T, int N, int NC, int NG, int NP, int CTAS, bool SUMMARY>
__global__ void __launch_bounds__(Shape<T, N, NC, NG, NP>::kThreads, CTAS)
    gdr_fwd_kernel(GdrArgs a, GdrSegs segs, float* e_out, float* checkpoints) {
  using X = Shape<T, N, NC, NG, NP>;
  constexpr int P = X::kParts;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t4 = lane & 3;
  constexpr int kSplitRows = N / X::kVRows, kParts = SUMMARY ? 2 * kSplitRows : kSplitRows;
  const int part = blockIdx.x % kParts % kSplitRows;
  const bool unit = SUMMARY && blockIdx.x % kParts >= kSplitRows;
  const int sh = blockIdx.x / kParts;
  const int h = sh % a.H, hk = h / (a.H / a.Hk);
  Span sp;
  if (!find_span(a, segs, sh / a.H, lane, sp)) return;
  const int len = sp.len;
  const int64_t t0 = sp.t0;
  const bool first_span = sp.s == 0, last_span = sp.s == sp.count - 1;
  if (SUMMARY && warp >= NC && (unit ? first_span || last_span : last_span)) return;
  const int steps = (len + X::kStep - 1) / X::kStep;
  const GroupMats* const mats = reinterpret_cast<GroupMats*>(smem + X::kOffMats);  // [2][NG]
  const int64_t v_row = int64_t(a.H) * N;

  auto tile = [&](int s, int which, int p) { return tile_of<X>(sb, s, which, p); };

  if (warp >= NC) {
    produce<T, N, X, false>(a, a.v, {h, hk, part, len, steps, t0}, smem, warp - NC, lane);
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int r0 = part * X::kVRows + warp * 16;  // this warp's value channels
  float S[N / 8][4];  // 16 rows x N columns: accumulator tiles of 8 columns
  if (!start_state<N, SUMMARY>(S, a, segs, sp, first_span, last_span, unit, 1, a.s0, h, r0, lane))
    return;
  T* y = static_cast<T*>(a.y) + t0 * v_row + int64_t(h) * N + r0;
  float* eo = e_out == nullptr ? nullptr : e_out + t0 * v_row + int64_t(h) * N + r0;
  __nv_bfloat16* const stage =
      reinterpret_cast<__nv_bfloat16*>(smem + X::kOffY) + warp * kG * kStagePitch;

  constexpr int kChunk = gdr_chunk(X::kBf16, N);
  if (checkpoints != nullptr)
    checkpoints += ((gdr_chunk_base(a, sp.seq, sp.t_seq) + (t0 - sp.t_seq) / kChunk) * a.H + h) * N *
                       N + r0 * N;

  __syncthreads();  // the first step is prepared
  for (int i = 0; i < steps; ++i) {
#pragma unroll 1
    for (int gi = 0; gi < NG; ++gi) {
      const int first = i * X::kStep + gi * kG;
      if (first >= len) break;
      if (!SUMMARY && checkpoints != nullptr && first % kChunk == 0)
        put_state<N>(checkpoints + int64_t(first / kChunk) * a.H * N * N, S, lane);
      const GroupMats& m = mats[(i & 1) * NG + gi];
      const uint32_t grp = uint32_t(gi * kG * X::kPitch) * 2u;
      // S_0 K^T and S_0 Q^T
      float xm[2][4], xc[2][4], om[2][4], oc[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) zero(xm[n]), zero(xc[n]), zero(om[n]), zero(oc[n]);
      const uint32_t to = at_tokens(lane, X::kPitch) + grp;
#pragma unroll
      for (int c = 0; c < N; c += 16) {
        uint32_t parts[3][4], kb[P][4], qb[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p) {
          ldsm4(kb[p], tile(i, 0, p) + to + c * 2);
          if (!SUMMARY) ldsm4(qb[p], tile(i, 1, p) + to + c * 2);
        }
        split_tiles<X::kBf16>(S[c / 8], S[c / 8 + 1], parts);
        mma_pairs<P>(xm, xc, parts, kb);
        // (one sum where only a bf16 y sees it: 8 registers less)
        if constexpr (!SUMMARY && X::kBf16) mma_up<P>(om, parts, qb);
        if constexpr (!SUMMARY && !X::kBf16) mma_pairs<P>(om, oc, parts, qb);
      }
      // e: V^T - C_i X as accumulator, plus its product with (I + A)^-1 - I
      float e[2][4], ec[2][4];
      {
        float vv[2][4];
        uint32_t raw[4];
        get_tokens<T, X>(vv, raw, smem + X::kOffV + (i % 3) * X::kVTile, gi * kG, warp * 16, lane);
        if (SUMMARY && unit) zero(vv[0]), zero(vv[1]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float2 d = *reinterpret_cast<const float2*>(m.decay + n * 8 + 2 * t4);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            e[n][x] = fmaf(-((x & 1) ? d.y : d.x), xm[n][x] + xc[n][x], vv[n][x]);
          zero(ec[n]);
        }
      }
      uint32_t ep[3][4], fb[3][4];
      split_tiles(e[0], e[1], ep);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(fb[p]) = m.inv[p][lane];
      mma_up<3>(ec, ep, fb);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) e[n][x] += ec[n][x];
      // y: scale C_i S_0 Q^T plus the read matrix times e
      split_tiles(e[0], e[1], ep);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(fb[p]) = m.read[p][lane];
      float o[2][4];
      zero(o[0]);
      zero(o[1]);
      if (!SUMMARY) mma_up<3>(o, ep, fb);
      float w[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float2 d = *reinterpret_cast<const float2*>(m.out + n * 8 + 2 * t4);
        const float2 f = *reinterpret_cast<const float2*>(m.write + n * 8 + 2 * t4);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          o[n][x] = fmaf((x & 1) ? d.y : d.x, X::kBf16 ? om[n][x] : om[n][x] + oc[n][x], o[n][x]);
          w[n][x] = e[n][x] * ((x & 1) ? f.y : f.x);
        }
      }
      // S = C S_0 + W^T K, the products summed on their own
      uint32_t wp[3][4];
      split_tiles<X::kBf16>(w[0], w[1], wp);
      const float end = m.end;
      const uint32_t ch = at_channels(lane, X::kPitch) + grp;
#pragma unroll
      for (int c = 0; c < N; c += 16) {
        uint32_t kb[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p) ldsm4t(kb[p], tile(i, 0, p) + ch + c * 2);
        float d[2][4];
        zero(d[0]);
        zero(d[1]);
        mma_up<P>(d, wp, kb);
#pragma unroll
        for (int n = 0; n < 2; ++n) scale_add(S[c / 8 + n], end, d[n]);
      }
      if (!SUMMARY && eo != nullptr)
        put_tokens<float>(eo + first * v_row, v_row, e, len - first, nullptr, lane);
      if (!SUMMARY) put_tokens<T>(y + first * v_row, v_row, o, len - first, stage, lane);
    }
    __syncthreads();
  }
  if (SUMMARY) {
    put_state<N>((unit ? segs.unit : segs.leave) + (int64_t(sp.slot) * a.H + h) * N * N + r0 * N, S,
                 lane);
    return;
  }
  if (!last_span) return;
  if (a.s1 != nullptr)
    put_state<N>(a.s1 + (int64_t(sp.seq) * a.H + h) * N * N + r0 * N, S, lane);
}

template <bool SUMMARY, typename T, int N, int NC, int NG, int NP, int CTAS>
int launch(const GdrArgs& a, const GdrSegs& segs, float* e, float* checkpoints,
           cudaStream_t stream) {
  using X = Shape<T, N, NC, NG, NP>;
  auto* kernel = gdr_fwd_kernel<T, N, NC, NG, NP, CTAS, SUMMARY>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, X::kSmem) !=
      cudaSuccess)
    return WKV_ERR_CUDA;
  const int64_t spans = segs.tokens == 0 ? a.n_seqs : segs.slots;
  return launch_kernel(kernel, unsigned(spans * a.H * (N / X::kVRows) * (SUMMARY ? 2 : 1)),
                       X::kThreads, X::kSmem, stream, a, segs, e, checkpoints);
}

template <typename T, int N, int NP, int CTAS>
int walk(const GdrArgs& a, const GdrSegs& segs, float* e, float* checkpoints, cudaStream_t stream) {
  return launch<false, T, N, 4, 2, NP, CTAS>(a, segs, e, checkpoints, stream);
}
template <typename T, int N, int NP, int CTAS>
int summary(const GdrArgs& a, const GdrSegs& segs, cudaStream_t stream) {
  return launch<true, T, N, 4, 2, NP, CTAS>(a, segs, nullptr, nullptr, stream);
}

}  // namespace

int launch_gdr_chunked(const GdrArgs& a, const GdrSegs& segs, float* e, float* checkpoints,
                       cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  const GdrWalkForm form = gdr_walk_form(a, segs.tokens == 0 ? a.n_seqs : segs.slots);
  if (form == kGdrWalkError) return WKV_ERR_CUDA;
  if (segs.tokens > 0) {
    int rc = a.bf16 ? (a.N == 64 ? summary<bf16, 64, 2, 2>(a, segs, stream)
                                 : summary<bf16, 128, 2, 2>(a, segs, stream))
                    : (a.N == 64 ? summary<float, 64, 4, 1>(a, segs, stream)
                                 : summary<float, 128, 4, 1>(a, segs, stream));
    if (rc == WKV_OK) rc = launch_gdr_combine(a, segs, false, stream);
    if (rc != WKV_OK) return rc;
  }
  if (!a.bf16)
    return a.N == 64 ? walk<float, 64, 4, 1>(a, segs, e, checkpoints, stream)
                     : walk<float, 128, 4, 1>(a, segs, e, checkpoints, stream);
  if (form == kGdrWalkPairs)
    return a.N == 64 ? walk<bf16, 64, 4, 1>(a, segs, e, checkpoints, stream)
                     : walk<bf16, 128, 4, 1>(a, segs, e, checkpoints, stream);
  return a.N == 64 ? walk<bf16, 64, 2, 2>(a, segs, e, checkpoints, stream)
                   : walk<bf16, 128, 2, 2>(a, segs, e, checkpoints, stream);
}

}  // namespace wkv
