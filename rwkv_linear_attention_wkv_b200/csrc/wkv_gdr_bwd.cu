// Gradients of the gated delta rule (sm_100a), in two kernels.
//
// With u_j = beta_j e_j what a token writes, D the gradient of the state after it, and per group
// of 16 tokens c_i, D_ij, C_i, C as in the forward, dD the gradient of the state that leaves:
//   R_j  = exp(c_16 - c_j) dD k_j + scale sum_{i >= j} D_ij (q_i . k_j) dy_i
//   du_j = R_j - sum_{i > j} D_ij (k_i . k_j) beta_i du_i,     de = beta du = dv
//   dD  <- C dD + sum_i (scale C_i dy_i) q_i^T - (C_i de_i) k_i^T
// 1. The chain walks a sequence's groups from the last to the first. It is the forward with dy in
//    the place of v: rows of dD (value channels) stay in registers, 16 a warp, the system is the
//    forward's transposed. It leaves du, and dD after every chunk of 64 tokens.
// 2. Everything else needs sums over value channels, but no chain: a CTA takes a chunk of one
//    query/key head, with the state S that enters it (the forward's checkpoint), the gradient dD
//    of the one that leaves, e and du, and per value head
//      P_ij = scale D_ij (dy_i . u_j) (i >= j),   Z_ij = D_ij (de_i . u_j) (i > j)
//      dq = scale C S^T dy + P K
//      dk = [exp(c_L - c) dD^T u + P^T Q - Z^T K] + [-C S^T de - Z K]
//      dbeta_j = du_j . e_j
//      dg_t = sum_{i >= t} R_i + sum_{j < t} W_j + sum_{i >= t > j} X_ij + C_L <dD, S>
//      R_i = q_i . scale C_i S^T dy_i - k_i . C_i S^T de_i,   W_j = k_j . exp(c_L - c_j) dD^T u_j
//      X_ij = P_ij (q_i . k_j) - Z_ij (k_i . k_j)
//    These are the terms whose decays pass t: read from the state or written to it on this side of
//    t or that, or both. Each carries e^{g_t} itself. (The gradient of every running sum c_i, added
//    up from the end, is shorter, but there the terms on one side of t have to cancel: nothing but
//    rounding was left of dg_t at g_t = -16, and something at -inf.)
//
// Rounding: both kernels keep the full three-part products everywhere, so that a bf16 gradient is
// an fp32 gradient rounded once. What only the bf16 dk sees is added up by the matrix instructions
// alone (see product()).
//
// Measured, 16 x 1024 x 12 x 64 bf16: chain 127 us, second kernel 275 us (198 with two parts for dk
// and dg from the running sums). The chain is bound like the forward (wkv_gdr_fwd.cu). The second
// kernel issues a third of the time and has its matrix pipe busy a third: 16 warps an SM wait for
// each other's tiles (barriers) and for e, du and states, 1.6 KB a token and head, which HBM
// delivers in 50 us.
#include "wkv_gdr.cuh"

namespace wkv {

using namespace gdr;

namespace {

// c += a b with a of one exact part and b of three, the small products first.
__device__ __forceinline__ void mma_exact_a(float (&c)[2][4], const uint32_t (&a)[4],
                                            const uint32_t (&b)[3][4]) {
#pragma unroll
  for (int p = 2; p >= 0; --p)
#pragma unroll
    for (int n = 0; n < 2; ++n) mma(c[n], a, b[p][2 * n], b[p][2 * n + 1]);
}

// SUMMARY: as the forward's, of the gradient that enters a segment at its end.
template <typename T, int N, int NC, int NG, int NP, int CTAS, bool SUMMARY>
__global__ void __launch_bounds__(Shape<T, N, NC, NG, NP>::kThreads, CTAS)
    gdr_chain_kernel(GdrBwdArgs b, GdrSegs segs) {
  using X = Shape<T, N, NC, NG, NP>;
  constexpr int P = X::kParts;
  extern __shared__ __align__(128) unsigned char smem[];
  const GdrArgs& a = b.p;
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
  const bool first_span = sp.s == sp.count - 1, last_span = sp.s == 0;  // of the walk
  if (SUMMARY && warp >= NC && (unit ? first_span || last_span : last_span)) return;
  const int steps = (len + X::kStep - 1) / X::kStep;
  GroupMats* const mats = reinterpret_cast<GroupMats*>(smem + X::kOffMats);  // [2][NG]
  const int64_t v_row = int64_t(a.H) * N;

  // Steps are counted in the order they are taken: step i has the tokens from `first_of(i)`.
  auto first_of = [&](int i) { return (steps - 1 - i) * X::kStep; };
  auto tile = [&](int s, int which, int p) { return tile_of<X>(sb, s, which, p); };

  if (warp >= NC) {
    produce<T, N, X, true>(a, b.dy, {h, hk, part, len, steps, t0}, smem, warp - NC, lane);
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int r0 = part * X::kVRows + warp * 16;  // this warp's value channels
  float S[N / 8][4];  // dD: 16 rows x N columns
  if (!start_state<N, SUMMARY>(S, a, segs, sp, first_span, last_span, unit, -1, b.ds1, h, r0, lane))
    return;
  T* dv = static_cast<T*>(b.dv) + t0 * v_row + int64_t(h) * N + r0;
  float* du = b.du + t0 * v_row + int64_t(h) * N + r0;
  __nv_bfloat16* const stage =
      reinterpret_cast<__nv_bfloat16*>(smem + X::kOffY) + warp * kG * kStagePitch;
  constexpr int kChunk = gdr_chunk(X::kBf16, N);
  float* const dstates =
      b.dstates + (gdr_chunk_base(a, sp.seq, sp.t_seq) + (t0 - sp.t_seq) / kChunk) * a.H * N * N +
      (int64_t(h) * N + r0) * N;

  __syncthreads();  // the first step is prepared
  for (int i = 0; i < steps; ++i) {
#pragma unroll 1
    for (int gi = NG - 1; gi >= 0; --gi) {
      const int first = first_of(i) + gi * kG;
      if (first >= len) continue;
      if (!SUMMARY && ((first + kG) % kChunk == 0 || first + kG >= len))
        put_state<N>(dstates + int64_t(first / kChunk) * a.H * N * N, S, lane);
      const GroupMats& m = mats[(i & 1) * NG + gi];
      const uint32_t grp = uint32_t(gi * kG * X::kPitch) * 2u;
      // dD K^T
      float xm[2][4], xc[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) zero(xm[n]), zero(xc[n]);
      const uint32_t to = at_tokens(lane, X::kPitch) + grp;
#pragma unroll
      for (int c = 0; c < N; c += 16) {
        uint32_t parts[3][4], kb[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p) ldsm4(kb[p], tile(i, 0, p) + to + c * 2);
        split_tiles<X::kBf16>(S[c / 8], S[c / 8 + 1], parts);
        mma_pairs<P>(xm, xc, parts, kb);
      }
      // R^T
      float vv[2][4], r[2][4];
      uint32_t raw[4], ap[3][4], fb[3][4];
      get_tokens<T, X>(vv, raw, smem + X::kOffV + (i % 3) * X::kVTile, gi * kG, warp * 16, lane);
      if (SUMMARY && unit) {
        zero(vv[0]);
        zero(vv[1]);
        raw[0] = raw[1] = raw[2] = raw[3] = 0u;
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(fb[p]) = m.read[p][lane];
      zero(r[0]);
      zero(r[1]);
      if constexpr (X::kBf16) {
        mma_exact_a(r, raw, fb);
      } else {
        split_tiles(vv[0], vv[1], ap);
        mma_up<3>(r, ap, fb);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float2 w = *reinterpret_cast<const float2*>(m.write + n * 8 + 2 * t4);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          r[n][x] = fmaf((x & 1) ? w.y : w.x, xm[n][x] + xc[n][x], r[n][x]);
      }
      // du^T = R^T (inverse)^T
      split_tiles(r[0], r[1], ap);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(fb[p]) = m.inv[p][lane];
      float ec[2][4];
      zero(ec[0]);
      zero(ec[1]);
      mma_up<3>(ec, ap, fb);
      float de[2][4], w1[2][4], w2[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float2 be = *reinterpret_cast<const float2*>(m.beta + n * 8 + 2 * t4);
        const float2 dc = *reinterpret_cast<const float2*>(m.decay + n * 8 + 2 * t4);
        const float2 ou = *reinterpret_cast<const float2*>(m.out + n * 8 + 2 * t4);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          r[n][x] += ec[n][x];
          de[n][x] = r[n][x] * ((x & 1) ? be.y : be.x);
          w1[n][x] = vv[n][x] * ((x & 1) ? ou.y : ou.x);
          w2[n][x] = -de[n][x] * ((x & 1) ? dc.y : dc.x);
        }
      }
      // dD = C dD + W1^T Q + W2^T K, each product summed on its own (in one sum the matrix
      // instructions cut it seven times instead of twice: 3e-7 of dD instead of 1.2e-7)
      uint32_t bp[3][4];
      split_tiles<X::kBf16>(w1[0], w1[1], ap);
      split_tiles<X::kBf16>(w2[0], w2[1], bp);
      const float end = m.end;
      const uint32_t ch = at_channels(lane, X::kPitch) + grp;
#pragma unroll
      for (int c = 0; c < N; c += 16) {
        uint32_t kb[P][4], qb[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p) {
          ldsm4t(kb[p], tile(i, 0, p) + ch + c * 2);
          ldsm4t(qb[p], tile(i, 1, p) + ch + c * 2);
        }
        float d1[2][4], d2[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) zero(d1[n]), zero(d2[n]);
        mma_up<P>(d1, ap, qb);
        mma_up<P>(d2, bp, kb);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          scale_add(S[c / 8 + n], end, d1[n]);
#pragma unroll
          for (int x = 0; x < 4; ++x) S[c / 8 + n][x] += d2[n][x];
        }
      }
      if (SUMMARY) continue;
      put_tokens<float>(du + first * v_row, v_row, r, len - first, nullptr, lane);
      put_tokens<T>(dv + first * v_row, v_row, de, len - first, stage, lane);
    }
    __syncthreads();
  }
  if (SUMMARY)
    put_state<N>((unit ? segs.unit : segs.leave) + (int64_t(sp.slot) * a.H + h) * N * N + r0 * N, S,
                 lane);
  else if (last_span && b.ds0 != nullptr)
    put_state<N>(b.ds0 + (int64_t(sp.seq) * a.H + h) * N * N + r0 * N, S, lane);
}

// ---- the second kernel ----------------------------------------------------------------------

template <typename T, int N>
struct Chunk {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kLen = gdr_chunk(kBf16, N);    // tokens
  static constexpr int kIn = kBf16 ? 1 : 3;           // parts of q, k, dy
  static constexpr int kParts = 3;                    // parts of u, de, states, P, Z
  // Columns of a warp: such that an SM holds 16 warps (two CTAs of 8 for bf16 heads of 64, else one
  // of 16) at 128 registers.
  static constexpr int kCols = kBf16 ? 32 : 16;
  static constexpr int kCtas = kBf16 && N == 64 ? 2 : 1;
  static constexpr int kSlices = N / kCols;           // warps that share a strip of 16 tokens
  static constexpr int kWarps = kLen / 16 * kSlices;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPitch = N + 8;
  static constexpr int kTile = kLen * kPitch * 2;
  static constexpr int kRows = 64;                    // rows of a state staged at once
  static constexpr int kState = kRows * kPitch * 2;
  static constexpr int kPPitch = kLen + 8;
  static constexpr int kPTile = kLen * kPPitch * 2;
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kOffK + kIn * kTile;
  static constexpr int kOffDy = kOffQ + kIn * kTile;
  static constexpr int kOffU = kOffDy + kIn * kTile;
  static constexpr int kOffDe = kOffU + kParts * kTile;   // later Z
  static constexpr int kOffS = kOffDe + kParts * kTile;  // 64 rows of a state; later P
  static constexpr int kOffF = kOffS + kParts * kState;    // floats
  static_assert(kPTile <= kTile && kPTile <= kState, "Z and P fit where de and the states were");
  static constexpr int kShares = kSlices < kLen / 16 ? kSlices : kLen / 16;  // of P's columns
  static constexpr int kShare = kLen / kShares;
  struct Floats {
    Decay c[kLen];
    float beta[kLen];
    float to_end[kLen];           // exp(c_L - c_j)
    float since[kLen];            // C_i
    float read[kSlices][kLen];    // R_i by slice of the columns
    float wrote[kSlices][kLen];   // W_j, the same
    float across[kLen / 16][kLen];  // sum of X_ij over i >= t of a strip and j < t of t's share
    float rows[kShares][kLen];    // sum of X_ij over a share's j
    float inner[kWarps];          // <dD, S> by warp
  };
  static constexpr int kSmem = kOffF + int(sizeof(Floats));
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "the CTAs' shared memory fits an SM");
};

// One value as three bf16 parts, four at a time, PART bytes apart.
template <int PART>
__device__ __forceinline__ void put_parts(unsigned char* d, float4 x) {
  uint2 p[3];
  split2(x.x, x.y, p[0].x, p[1].x, p[2].x);
  split2(x.z, x.w, p[0].y, p[1].y, p[2].y);
#pragma unroll
  for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(d + i * PART) = p[i];
}

// Products of operands of PA and PB parts: what a factor's parts leave out, the pairs do too.
template <int PA, int PB, int NT>
__device__ __forceinline__ void mma_parts(float (&c)[NT][4], int n, const uint32_t (&a)[PA][4],
                                          const uint32_t (&b)[PB][4]) {
  constexpr int kMost = PA > PB ? PA : PB;
#pragma unroll
  for (int sum = kMost - 1; sum >= 0; --sum)
#pragma unroll
    for (int i = PA - 1; i >= 0; --i) {
      const int j = sum - i;
      if (j < 0 || j >= PB) continue;
      mma(c[n], a[i], b[j][0], b[j][1]);
      mma(c[n + 1], a[i], b[j][2], b[j][3]);
    }
}

// c (16 rows x 8 NT columns) += A B over LEN: A's fragments at `a` + 32 bytes a step, B's rows at
// `b` + 16 rows a step, columns 32 bytes apart a tile pair. TA: A stored transposed. EXACT: every
// step of 16 is summed on its own and added in fp32 (the matrix instruction truncates as it adds
// to a large sum: over the 24 to 48 adds of a product that costs two bits).
// Only the steps of [l0, l1) and the first `cols` column tiles are taken.
template <int PA, int PB, int NT, bool TA, bool TB, bool EXACT>
__device__ __forceinline__ void product(float (&c)[NT][4], int l0, int l1, uint32_t a, int a_part,
                                        int a_pitch, uint32_t b, int b_part, int b_pitch,
                                        int cols = NT) {
#pragma unroll 2
  for (int l = l0; l < l1; l += 16) {
    uint32_t ap[PA][4];
#pragma unroll
    for (int p = 0; p < PA; ++p) {
      if (TA)
        ldsm4t(ap[p], a + p * a_part + l * a_pitch * 2);
      else
        ldsm4(ap[p], a + p * a_part + l * 2);
    }
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      if (n >= cols) continue;
      uint32_t bp[PB][4];
#pragma unroll
      for (int p = 0; p < PB; ++p) {
        if (TB)  // rows are the contraction
          ldsm4t(bp[p], b + p * b_part + l * b_pitch * 2 + n * 16);
        else     // rows are the product's columns
          ldsm4(bp[p], b + p * b_part + n * 8 * b_pitch * 2 + l * 2);
      }
      if (EXACT) {
        float d[2][4];
        zero(d[0]);
        zero(d[1]);
        mma_parts<PA, PB, 2>(d, 0, ap, bp);
#pragma unroll
        for (int x = 0; x < 4; ++x) c[n][x] += d[0][x], c[n + 1][x] += d[1][x];
      } else {
        mma_parts<PA, PB, NT>(c, n, ap, bp);
      }
    }
  }
}

// a operand of 16 rows x 16 columns stored by rows (plain load) or by columns (transposed load).
__device__ __forceinline__ uint32_t at_rows(int lane, int pitch) {
  const int m = lane >> 3, r = lane & 7;
  return uint32_t(((m & 1) * 8 + r) * pitch + (m >> 1) * 8) * 2u;
}

// SHARED: several value heads share the query/key head, whose dq and dk are summed over them (32
// more registers).
template <typename T, int N, bool SHARED>
__global__ void __launch_bounds__(Chunk<T, N>::kThreads, Chunk<T, N>::kCtas)
    gdr_chunk_kernel(GdrBwdArgs b) {
  using X = Chunk<T, N>;
  constexpr int PI = X::kIn, PP = X::kParts, NT = X::kCols / 8, L = X::kLen;
  constexpr bool kExact = !X::kBf16;  // of what only dk sees
  extern __shared__ __align__(128) unsigned char smem[];
  typename X::Floats& F = *reinterpret_cast<typename X::Floats*>(smem + X::kOffF);
  const GdrArgs& a = b.p;
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g4 = lane >> 2, t4 = lane & 3;
  const int strip = warp / X::kSlices, slice = warp % X::kSlices;
  const int G = a.H / a.Hk;
  const int hk = blockIdx.x % a.Hk;
  const int64_t slot = blockIdx.x / a.Hk;
  // the sequence and chunk of this slot
  int seq, chunk, len;
  int64_t t0 = 0;
  if (a.offsets == nullptr) {
    const int per = (a.T + L - 1) / L + 1;
    seq = int(slot / per);
    chunk = int(slot % per);
    t0 = sequence(a, seq, len);
    if (chunk == per - 1) return;
  } else {
    // The last sequence whose first chunk is not behind this slot, 32 candidates at a time (first
    // chunks increase with the sequence; whatever the offsets are, the sequence found is checked).
    int lo = 0, hi = a.n_seqs;
    do {
      const int step = (hi - lo + 31) / 32, s = lo + lane * step;
      bool before = false;
      if (s < hi) before = gdr_chunk_base(a, s, sequence(a, s, len)) <= slot;
      const unsigned who = __ballot_sync(0xffffffffu, before);
      if (who == 0) return;
      lo += (31 - __clz(who)) * step;
      hi = min(hi, lo + step);
    } while (hi - lo > 1);
    seq = lo;
    t0 = sequence(a, seq, len);
    const int64_t at = slot - gdr_chunk_base(a, seq, t0);
    if (at < 0 || at * L >= len) return;
    chunk = int(at);
  }
  t0 += int64_t(chunk) * L;
  len = min(len - chunk * L, L);
  const int64_t qk_row = int64_t(a.Hk) * N, v_row = int64_t(a.H) * N;
  constexpr int kQuads = N / 4;

  // the chunk's rows of an input into PI parts, zeros past `len`
  auto load_input = [&](const T* src, int64_t row, int off) {
    if constexpr (X::kBf16) {
      for (int i = threadIdx.x; i < L * (N / 8); i += X::kThreads) {
        const int t = i / (N / 8), c = (i % (N / 8)) * 8;
        const bool ok = t < len;
        cp_async_16z(sb + off + uint32_t(t * X::kPitch + c) * 2u, src + (ok ? t : 0) * row + c, ok);
      }
    } else {
#pragma unroll 4
      for (int i = threadIdx.x; i < L * kQuads; i += X::kThreads) {
        const int t = i / kQuads, c = (i % kQuads) * 4;
        float4 x = *reinterpret_cast<const float4*>(src + min(t, len - 1) * row + c);
        if (t >= len) x = make_float4(0.f, 0.f, 0.f, 0.f);
        put_parts<X::kTile>(smem + off + (t * X::kPitch + c) * 2, x);
      }
    }
  };
  load_input(static_cast<const T*>(a.k) + t0 * qk_row + int64_t(hk) * N, qk_row, X::kOffK);
  load_input(static_cast<const T*>(a.q) + t0 * qk_row + int64_t(hk) * N, qk_row, X::kOffQ);

  // sum over a warp's columns of x times an input's rows, for the two tokens of a thread
  auto dot_rows = [&](const float(&x)[NT][4], int off, float(&out)[2]) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const unsigned char* r = smem + off + ((strip * 16 + g4 + z * 8) * X::kPitch +
                                             slice * X::kCols + 2 * t4) * 2;
      float s = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int p = PI - 1; p >= 0; --p) {
          const float2 w = unpack(*reinterpret_cast<const uint32_t*>(r + p * X::kTile + n * 16));
          v.x += w.x;
          v.y += w.y;
        }
        s = fmaf(x[n][2 * z], v.x, s);
        s = fmaf(x[n][2 * z + 1], v.y, s);
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      out[z] = s;
    }
  };

  auto put_rows = [&](void* to, const float(&x)[NT][4]) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int t = strip * 16 + g4 + z * 8;
      if (t >= len) continue;
      T* const row =
          static_cast<T*>(to) + (t0 + t) * qk_row + int64_t(hk) * N + slice * X::kCols + 2 * t4;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 v = make_float2(x[n][2 * z], x[n][2 * z + 1]);
        if constexpr (X::kBf16)
          *reinterpret_cast<__nv_bfloat162*>(row + n * 8) = __float22bfloat162_rn(v);
        else
          *reinterpret_cast<float2*>(row + n * 8) = v;
      }
    }
  };

  float dq[SHARED ? NT : 1][4], dk[SHARED ? NT : 1][4];  // sums over the value heads
#pragma unroll
  for (int n = 0; n < (SHARED ? NT : 1); ++n) zero(dq[n]), zero(dk[n]);

#pragma unroll 1
  for (int h = hk * G; h < hk * G + G; ++h) {
    const int64_t state_at = (slot * a.H + h) * N * N;
    // what the head needs first, on its way before anything is waited for
    constexpr int kTok = L * kQuads / X::kThreads, kSt = X::kRows * kQuads / X::kThreads;
    float4 er[kTok], dr[kTok], sr[kSt];
    // (rows past the end read the last one: a branch would put the loads one after the other)
#pragma unroll
    for (int x = 0; x < kTok; ++x) {
      const int i = threadIdx.x + x * X::kThreads;
      const int64_t at =
          (t0 + min(i / kQuads, len - 1)) * v_row + int64_t(h) * N + (i % kQuads) * 4;
      er[x] = *reinterpret_cast<const float4*>(b.e + at);
      dr[x] = *reinterpret_cast<const float4*>(b.du + at);
    }
    // 64 rows of a state, from global memory and into parts
    auto fetch_state = [&](const float* src, int r0) {
#pragma unroll
      for (int x = 0; x < kSt; ++x)
        sr[x] = reinterpret_cast<const float4*>(src + r0 * N)[threadIdx.x + x * X::kThreads];
    };
    auto store_state = [&] {
#pragma unroll
      for (int x = 0; x < kSt; ++x) {
        const int i = threadIdx.x + x * X::kThreads;
        put_parts<X::kState>(smem + X::kOffS + (i / kQuads * X::kPitch + (i % kQuads) * 4) * 2,
                             sr[x]);
      }
    };
    fetch_state(b.checkpoints + state_at, 0);
    __syncthreads();  // the last head's tiles have been read
    load_input(static_cast<const T*>(b.dy) + t0 * v_row + int64_t(h) * N, v_row, X::kOffDy);
    if (threadIdx.x < 32) {
      // decays over the chunk, L / 32 adjacent stretches of 32 tokens
      Decay carry = {0.f, 0.f};
#pragma unroll
      for (int s = 0; s < L; s += 32) {
        const int t = s + lane;
        const float g = t < len ? a.g[(t0 + t) * a.H + h] : 0.f;
        const Decay c = add(decay_sums<32>(g, lane), carry);
        F.c[t] = c;
        F.since[t] = power(c);
        carry = shfl(c, 31);
      }
#pragma unroll
      for (int s = 0; s < L; s += 32) F.to_end[s + lane] = power_between(carry, F.c[s + lane]);
    } else if (threadIdx.x < 32 + L) {
      const int t = threadIdx.x - 32;
      F.beta[t] = t < len ? a.beta[(t0 + t) * a.H + h] : 0.f;
    }
    __syncthreads();
    // u, de, dbeta: a token's row lies in kQuads adjacent lanes
#pragma unroll
    for (int x = 0; x < kTok; ++x) {
      const int i = threadIdx.x + x * X::kThreads, t = i / kQuads, c = (i % kQuads) * 4;
      const bool in = t < len;
      const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 e = in ? er[x] : zero4, d = in ? dr[x] : zero4;
      const float be = F.beta[t];
      float s = fmaf(e.x, d.x, fmaf(e.y, d.y, fmaf(e.z, d.z, e.w * d.w)));
#pragma unroll
      for (int m = kQuads / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      if (c == 0 && in) b.dbeta[(t0 + t) * a.H + h] = s;
      const int to = (t * X::kPitch + c) * 2;
      put_parts<X::kTile>(smem + X::kOffU + to,
                          make_float4(be * e.x, be * e.y, be * e.z, be * e.w));
      put_parts<X::kTile>(smem + X::kOffDe + to,
                          make_float4(be * d.x, be * d.y, be * d.z, be * d.w));
    }
    const uint32_t rows = at_rows(lane, X::kPitch) + uint32_t(strip * 16 * X::kPitch) * 2u;
    const uint32_t cols = at_channels(lane, X::kPitch) + uint32_t(slice * X::kCols) * 2u;
    float q1[NT][4], k1[NT][4], k2[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) zero(q1[n]), zero(k1[n]), zero(k2[n]);
    // S^T dy, S^T de; while a block of rows is at work the next is fetched
#pragma unroll 1
    for (int r0 = 0; r0 < N; r0 += X::kRows) {
      if (r0 > 0) __syncthreads();
      store_state();
      cp_async_wait_all();
      __syncthreads();
      if (r0 + X::kRows < N)
        fetch_state(b.checkpoints + state_at, r0 + X::kRows);
      else
        fetch_state(b.dstates + state_at, 0);
      product<PI, PP, NT, false, true, true>(q1, 0, X::kRows, sb + X::kOffDy + rows + r0 * 2,
                                             X::kTile, X::kPitch, sb + X::kOffS + cols, X::kState,
                                             X::kPitch);
      product<PP, PP, NT, false, true, true>(k1, 0, X::kRows, sb + X::kOffDe + rows + r0 * 2,
                                               X::kTile, X::kPitch, sb + X::kOffS + cols, X::kState,
                                               X::kPitch);
    }
    // dD^T u, and <dD, S>
    float inner = 0.f;
#pragma unroll 1
    for (int r0 = 0; r0 < N; r0 += X::kRows) {
      float4 nr[kSt];
#pragma unroll
      for (int x = 0; x < kSt; ++x)
        nr[x] = reinterpret_cast<const float4*>(b.checkpoints + state_at +
                                                r0 * N)[threadIdx.x + x * X::kThreads];
      __syncthreads();
      store_state();
#pragma unroll
      for (int x = 0; x < kSt; ++x)
        inner = fmaf(sr[x].x, nr[x].x, fmaf(sr[x].y, nr[x].y,
                     fmaf(sr[x].z, nr[x].z, fmaf(sr[x].w, nr[x].w, inner))));
      __syncthreads();
      if (r0 + X::kRows < N) fetch_state(b.dstates + state_at, r0 + X::kRows);
      product<PP, PP, NT, false, true, true>(k2, 0, X::kRows, sb + X::kOffU + rows + r0 * 2,
                                               X::kTile, X::kPitch, sb + X::kOffS + cols, X::kState,
                                               X::kPitch);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, m);
    if (lane == 0) F.inner[warp] = inner;
    {
      // dk = k2 - k1 from here on
      const int t = strip * 16 + g4;
      const float since[2] = {F.since[t], F.since[t + 8]};
      const float to_end[2] = {F.to_end[t], F.to_end[t + 8]};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          q1[n][x] *= a.scale * since[x >> 1];
          k1[n][x] *= since[x >> 1];
          k2[n][x] *= to_end[x >> 1];
        }
      // what dg needs of them, before the chunk's own tokens join
      float rq[2], rk[2], wk[2];
      dot_rows(q1, X::kOffQ, rq);
      dot_rows(k1, X::kOffK, rk);
      dot_rows(k2, X::kOffK, wk);
      if (t4 == 0) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          F.read[slice][t + z * 8] = rq[z] - rk[z];
          F.wrote[slice][t + z * 8] = wk[z];
        }
      }
    }
    // P and Z: this warp's tokens i, its share of the columns j
    constexpr int NW = X::kShare / 8;  // column tiles of a warp
    const bool shares = slice < X::kShares;
    float pw[NW][4], zw[NW][4];
#pragma unroll
    for (int n = 0; n < NW; ++n) zero(pw[n]), zero(zw[n]);
    const int j0 = slice * X::kShare;
    // (16 x 16 blocks above the diagonal are neither made nor read)
    const int tiles = shares ? (strip + 1) * 2 - j0 / 8 : 0;
    if (tiles > 0) {
      const uint32_t us =
          sb + X::kOffU + at_tokens(lane, X::kPitch) + uint32_t(j0 * X::kPitch) * 2u;
      product<PI, PP, NW, false, false, true>(pw, 0, N, sb + X::kOffDy + rows, X::kTile, X::kPitch,
                                              us, X::kTile, X::kPitch, tiles);
      product<PP, PP, NW, false, false, true>(zw, 0, N, sb + X::kOffDe + rows, X::kTile,
                                              X::kPitch, us, X::kTile, X::kPitch, tiles);
      // P and Z by elements, and X: sums over the columns before t, added up over the rows from t
      const uint32_t ks =
          sb + X::kOffK + at_tokens(lane, X::kPitch) + uint32_t(j0 * X::kPitch) * 2u;
      float before[2] = {0.f, 0.f};  // this row's sums over the columns so far
#pragma unroll
      for (int n = 0; n < NW; n += 2) {
        if (n >= tiles) continue;
        float qk[2][4], kk[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) zero(qk[m]), zero(kk[m]);
        const uint32_t kn = ks + uint32_t(n * 8 * X::kPitch) * 2u;
        product<PI, PI, 2, false, false, true>(qk, 0, N, sb + X::kOffQ + rows, X::kTile, X::kPitch,
                                               kn, X::kTile, X::kPitch);
        product<PI, PI, 2, false, false, true>(kk, 0, N, sb + X::kOffK + rows, X::kTile, X::kPitch,
                                               kn, X::kTile, X::kPitch);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int j = j0 + (n + m) * 8 + 2 * t4;
          float from[2] = {0.f, 0.f};  // columns j and j + 1: over this thread's rows
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int i = strip * 16 + g4 + z * 8;
            float x[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float d = i >= j + y ? decay_between(F.c[i], F.c[j + y]) : 0.f;
              float& p = pw[n + m][2 * z + y];
              float& q = zw[n + m][2 * z + y];
              p = i >= j + y ? a.scale * d * p : 0.f;
              q = i > j + y ? d * q : 0.f;
              x[y] = i > j + y ? fmaf(p, qk[m][2 * z + y], -q * kk[m][2 * z + y]) : 0.f;
            }
            float upto = x[0] + x[1];
#pragma unroll
            for (int s = 1; s < 4; s <<= 1) {
              const float below = __shfl_up_sync(0xffffffffu, upto, s, 4);
              if (t4 >= s) upto += below;
            }
            const float here = __shfl_up_sync(0xffffffffu, upto, 1, 4);
            const float start = before[z] + (t4 > 0 ? here : 0.f);
            if (i >= j) from[0] += start;
            if (i >= j + 1) from[1] += start + x[0];
            before[z] += __shfl_sync(0xffffffffu, upto, 3, 4);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) from[y] += __shfl_xor_sync(0xffffffffu, from[y], s);
            if (g4 == 0) F.across[strip][j + y] = from[y];
          }
        }
      }
      if (t4 == 0) {
#pragma unroll
        for (int z = 0; z < 2; ++z) F.rows[slice][strip * 16 + g4 + z * 8] = before[z];
      }
    }
    __syncthreads();  // dD's rows and de have been read: P and Z take their places
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        if (n >= tiles) continue;
        const int i = strip * 16 + g4 + z * 8, j = j0 + n * 8 + 2 * t4;
        uint32_t p[3];
        const int to = (i * X::kPPitch + j) * 2;
        split2(pw[n][2 * z], pw[n][2 * z + 1], p[0], p[1], p[2]);
#pragma unroll
        for (int x = 0; x < PP; ++x)
          *reinterpret_cast<uint32_t*>(smem + X::kOffS + x * X::kPTile + to) = p[x];
        split2(zw[n][2 * z], zw[n][2 * z + 1], p[0], p[1], p[2]);
#pragma unroll
        for (int x = 0; x < PP; ++x)
          *reinterpret_cast<uint32_t*>(smem + X::kOffDe + x * X::kPTile + to) = p[x];
      }
    __syncthreads();
    // dq: + P K; k2: + P^T Q; k1: + Z K + Z^T K
    const uint32_t prow = at_rows(lane, X::kPPitch) + uint32_t(strip * 16 * X::kPPitch) * 2u;
    const uint32_t pcol = at_tokens(lane, X::kPPitch) + uint32_t(strip * 16) * 2u;
    const int below = strip * 16, upto = strip * 16 + 16;
    product<PP, PI, NT, false, true, kExact>(q1, 0, upto, sb + X::kOffS + prow, X::kPTile,
                                             X::kPPitch, sb + X::kOffK + cols, X::kTile, X::kPitch);
    product<PP, PI, NT, true, true, kExact>(k2, below, L, sb + X::kOffS + pcol, X::kPTile,
                                            X::kPPitch, sb + X::kOffQ + cols, X::kTile, X::kPitch);
    product<PP, PI, NT, false, true, kExact>(k1, 0, upto, sb + X::kOffDe + prow, X::kPTile,
                                             X::kPPitch, sb + X::kOffK + cols, X::kTile, X::kPitch);
    product<PP, PI, NT, true, true, kExact>(k1, below, L, sb + X::kOffDe + pcol, X::kPTile,
                                            X::kPPitch, sb + X::kOffK + cols, X::kTile, X::kPitch);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        k2[n][x] -= k1[n][x];
        if constexpr (SHARED) {
          dq[n][x] += q1[n][x];
          dk[n][x] += k2[n][x];
        }
      }
    if constexpr (!SHARED) {
      put_rows(b.dq, q1);
      put_rows(b.dk, k2);
    }
    // (everything that dg takes was written before the last two barriers)
    if (warp == 0) {
      constexpr int kHalves = L / 32;  // 32 tokens at a time, one a lane
      float dg[kHalves], inner_all = 0.f;
      for (int w = 0; w < X::kWarps; ++w) inner_all += F.inner[w];
      const float through = F.since[L - 1] * inner_all;
      auto from_here = [&](float x) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const float above = __shfl_down_sync(0xffffffffu, x, d);
          if (lane + d < 32) x += above;
        }
        return x;
      };
      // R over the tokens from t, X over the rows from t and the shares before t's
      float later = 0.f, later_rows[X::kShares];
#pragma unroll
      for (int r = 0; r < X::kShares; ++r) later_rows[r] = 0.f;
#pragma unroll
      for (int s = kHalves - 1; s >= 0; --s) {
        const int t = s * 32 + lane;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < X::kSlices; ++w) x += F.read[w][t];
        x = from_here(x) + later;
        later = __shfl_sync(0xffffffffu, x, 0);
        for (int w = t / 16; w < L / 16; ++w) x += F.across[w][t];
#pragma unroll
        for (int r = 0; r < X::kShares - 1; ++r) {
          const float over = from_here(F.rows[r][t]) + later_rows[r];
          later_rows[r] = __shfl_sync(0xffffffffu, over, 0);
          if (t / X::kShare > r) x += over;
        }
        dg[s] = x + through;
      }
      // W over the tokens before t
      float earlier = 0.f;
#pragma unroll
      for (int s = 0; s < kHalves; ++s) {
        const int t = s * 32 + lane;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < X::kSlices; ++w) x += F.wrote[w][t];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const float below = __shfl_up_sync(0xffffffffu, x, d);
          if (lane >= d) x += below;
        }
        const float before = __shfl_up_sync(0xffffffffu, x, 1);
        dg[s] += earlier + (lane > 0 ? before : 0.f);
        earlier += __shfl_sync(0xffffffffu, x, 31);
        if (t < len) b.dg[(t0 + t) * a.H + h] = dg[s];
      }
    }
  }

  if constexpr (SHARED) {
    put_rows(b.dq, dq);
    put_rows(b.dk, dk);
  }
}

template <typename K>
bool allow_smem(K* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
         cudaSuccess;
}

template <bool SUMMARY, typename T, int N, int NP, int CTAS>
int chain(const GdrBwdArgs& b, const GdrSegs& segs, cudaStream_t stream) {
  using X = Shape<T, N, 4, 2, NP>;
  auto* kernel = gdr_chain_kernel<T, N, 4, 2, NP, CTAS, SUMMARY>;
  if (!allow_smem(kernel, X::kSmem)) return WKV_ERR_CUDA;
  const int64_t spans = segs.tokens == 0 ? b.p.n_seqs : segs.slots;
  return launch_kernel(kernel, unsigned(spans * b.p.H * (N / X::kVRows) * (SUMMARY ? 2 : 1)),
                       X::kThreads, X::kSmem, stream, b, segs);
}

template <typename T, int N>
int rest(const GdrBwdArgs& b, cudaStream_t stream) {
  using X = Chunk<T, N>;
  auto* kernel =
      b.p.H == b.p.Hk ? gdr_chunk_kernel<T, N, false> : gdr_chunk_kernel<T, N, true>;
  if (!allow_smem(kernel, X::kSmem)) return WKV_ERR_CUDA;
  return launch_kernel(kernel, unsigned(gdr_chunks(b.p) * b.p.Hk), X::kThreads, X::kSmem, stream,
                       b);
}

template <typename T, int N>
int backward(const GdrBwdArgs& b, const GdrSegs& segs, cudaStream_t stream) {
  constexpr bool kBf16 = sizeof(T) == 2;
  const GdrWalkForm form = gdr_walk_form(b.p, segs.tokens == 0 ? b.p.n_seqs : segs.slots);
  if (form == kGdrWalkError) return WKV_ERR_CUDA;
  int rc = WKV_OK;
  if (segs.tokens > 0) {
    if constexpr (kBf16)
      rc = chain<true, T, N, 2, 2>(b, segs, stream);
    else
      rc = chain<true, T, N, 4, 1>(b, segs, stream);
    if (rc == WKV_OK) rc = launch_gdr_combine(b.p, segs, true, stream);
  }
  if (rc != WKV_OK) return rc;
  if (!kBf16 || form == kGdrWalkPairs) {
    rc = chain<false, T, N, 4, 1>(b, segs, stream);
  } else {
    if constexpr (kBf16) rc = chain<false, T, N, 2, 2>(b, segs, stream);
  }
  return rc == WKV_OK ? rest<T, N>(b, stream) : rc;
}

}  // namespace

int launch_gdr_backward(const GdrBwdArgs& b, const GdrSegs& segs, cudaStream_t stream) {
  if (b.p.bf16)
    return b.p.N == 64 ? backward<__nv_bfloat16, 64>(b, segs, stream)
                       : backward<__nv_bfloat16, 128>(b, segs, stream);
  return b.p.N == 64 ? backward<float, 64>(b, segs, stream) : backward<float, 128>(b, segs, stream);
}

}  // namespace wkv
