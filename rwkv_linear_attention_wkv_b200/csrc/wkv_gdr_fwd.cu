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
// A CTA has one head of one sequence (or 64 of 128 rows of it): one producer warp per group of a
// step of 16 or 32 tokens, and 4 or 8 consumer warps. While the consumers work on step i the
// producers copy step i + 2 in (cp.async), and form A, its inverse and the masked read matrix of
// step i + 1: everything that does not depend on the state. One barrier a step.
#include <algorithm>

#include "wkv_gdr.cuh"

namespace wkv {

using namespace gdr;

namespace {

// What the producers hand over for a group: operand fragments of (I + A)^-1 - I and of the read
// matrix (three parts, a uint4 a lane), and four vectors over the tokens.
struct GroupMats {
  uint4 inv[3][32];
  uint4 read[3][32];
  float decay[kG];    // C_i
  float out[kG];      // scale C_i
  float write[kG];    // exp(c_16 - c_j) beta_j
  float end;          // C
  float pad[3];
};

template <typename T, int N, int NC, int NG>
struct Shape {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kParts = kBf16 ? 1 : 3;      // operand parts of q and k
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
  static constexpr int kOffY = kOffL + NG * kG * kLP * 4;
  static constexpr int kYPitch = 24;                // bf16 staging of a warp's 16 x 16 outputs
  static constexpr int kSmem = kOffY + (kBf16 ? NC * kG * kYPitch * 2 : 0);
  static constexpr int kThreads = 32 * (NC + NG);
};

template <typename T, int N, int NC, int NG>
__global__ void __launch_bounds__(Shape<T, N, NC, NG>::kThreads)
    gdr_fwd_kernel(GdrArgs a, float* e_out, float* checkpoints) {
  using X = Shape<T, N, NC, NG>;
  constexpr int P = X::kParts;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g4 = lane >> 2, t4 = lane & 3;
  constexpr int kSplitRows = N / X::kVRows;
  const int part = blockIdx.x % kSplitRows;
  const int sh = blockIdx.x / kSplitRows;
  const int seq = sh / a.H, h = sh % a.H, hk = h / (a.H / a.Hk);
  int len;
  const int64_t t0 = sequence(a, seq, len);
  const int steps = (len + X::kStep - 1) / X::kStep;
  GroupMats* const mats = reinterpret_cast<GroupMats*>(smem + X::kOffMats);  // [2][NG]
  const int64_t qk_row = int64_t(a.Hk) * N, v_row = int64_t(a.H) * N;

  // bf16 part p of q (which = 1) or k (0) of step s
  auto tile = [&](int s, int which, int p) -> uint32_t {
    if (X::kBf16) return sb + ((s % 3) * 2 + which) * X::kTile;
    return sb + X::kOffSplit + (((s & 1) * 2 + which) * 3 + p) * X::kTile;
  };

  if (warp >= NC) {
    // ------------------------------------------------------------------ producers
    const int pw = warp - NC, pt = pw * 32 + lane;
    const T* q = static_cast<const T*>(a.q) + t0 * qk_row + int64_t(hk) * N;
    const T* k = static_cast<const T*>(a.k) + t0 * qk_row + int64_t(hk) * N;
    const T* v = static_cast<const T*>(a.v) + t0 * v_row + int64_t(h) * N + part * X::kVRows;
    const float* gp = a.g + t0 * a.H + h;
    const float* bp = a.beta + t0 * a.H + h;
    float* const L = reinterpret_cast<float*>(smem + X::kOffL) + pw * kG * kLP;
    constexpr int kPer = 16 / int(sizeof(T));  // elements of a 16-byte copy

    auto load = [&](int s) {
      if (s < steps) {
        const int first = s * X::kStep;
        const uint32_t kd = X::kBf16 ? tile(s, 0, 0) : sb + ((s & 1) * 2 + 0) * X::kTileF;
        const uint32_t qd = X::kBf16 ? tile(s, 1, 0) : sb + ((s & 1) * 2 + 1) * X::kTileF;
        constexpr int pitch = X::kBf16 ? X::kPitch : X::kPitchF;
        for (int i = pt; i < X::kStep * (N / kPer); i += NG * 32) {
          const int tok = i / (N / kPer), c = (i % (N / kPer)) * kPer;
          const bool ok = first + tok < len;
          const int64_t at = (ok ? first + tok : 0) * qk_row + c;
          const uint32_t to = uint32_t(tok * pitch + c) * uint32_t(sizeof(T));
          cp_async_16z(kd + to, k + at, ok);
          cp_async_16z(qd + to, q + at, ok);
        }
        const uint32_t vd = sb + X::kOffV + (s % 3) * X::kVTile;
        for (int i = pt; i < X::kStep * (X::kVRows / kPer); i += NG * 32) {
          const int tok = i / (X::kVRows / kPer), c = (i % (X::kVRows / kPer)) * kPer;
          const bool ok = first + tok < len;
          cp_async_16z(vd + uint32_t(tok * X::kVPitch + c) * uint32_t(sizeof(T)),
                       v + (ok ? first + tok : 0) * v_row + c, ok);
        }
      }
      cp_async_commit();
    };
    auto sync_producers = [&] {
      if (NG == 1)
        __syncwarp();
      else
        asm volatile("bar.sync 1, %0;" ::"n"(NG * 32) : "memory");
    };

    load(0);
    load(1);
    for (int i = -1; i < steps; ++i) {
      const int s = i + 1;  // the step to prepare
      if (i >= 0) load(i + 2);
      if (s < steps) {
        const int tok = s * X::kStep + pw * kG + (lane & 15);
        const float gv = tok < len ? gp[int64_t(tok) * a.H] : 0.f;
        const float bv = tok < len ? bp[int64_t(tok) * a.H] : 0.f;
        cp_async_wait<1>();
        sync_producers();
        if (!X::kBf16) {
          // this warp's 16 tokens of q and k into three parts
#pragma unroll 2
          for (int w = 0; w < 2; ++w) {
            const float* src = reinterpret_cast<const float*>(smem + ((s & 1) * 2 + w) * X::kTileF) +
                               pw * kG * X::kPitchF;
            unsigned char* dst = smem + (tile(s, w, 0) - sb) + pw * kG * X::kPitch * 2;
            for (int j = lane; j < kG * N / 4; j += 32) {
              const int r = j / (N / 4), c = (j % (N / 4)) * 4;
              const float4 x = *reinterpret_cast<const float4*>(src + r * X::kPitchF + c);
              uint2 p0, p1, p2;
              split2(x.x, x.y, p0.x, p1.x, p2.x);
              split2(x.z, x.w, p0.y, p1.y, p2.y);
              unsigned char* d = dst + (r * X::kPitch + c) * 2;
              *reinterpret_cast<uint2*>(d) = p0;
              *reinterpret_cast<uint2*>(d + X::kTile) = p1;
              *reinterpret_cast<uint2*>(d + 2 * X::kTile) = p2;
            }
          }
          __syncwarp();
        }
        // k k^T and q k^T over the group
        float kk[2][4], qk[2][4], kc[2][4], qc[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) zero(kk[n]), zero(qk[n]), zero(kc[n]), zero(qc[n]);
        const uint32_t off = at_tokens(lane, X::kPitch) + uint32_t(pw * kG * X::kPitch) * 2u;
#pragma unroll
        for (int c = 0; c < N; c += 16) {
          uint32_t kb[P][4], qb[P][4], ka[3][4], qa[3][4];
#pragma unroll
          for (int p = 0; p < P; ++p) {
            ldsm4(kb[p], tile(s, 0, p) + off + c * 2);
            ldsm4(qb[p], tile(s, 1, p) + off + c * 2);
            // the same four 8 x 8 blocks in the order of an a operand
            ka[p][0] = kb[p][0]; ka[p][1] = kb[p][2]; ka[p][2] = kb[p][1]; ka[p][3] = kb[p][3];
            qa[p][0] = qb[p][0]; qa[p][1] = qb[p][2]; qa[p][2] = qb[p][1]; qa[p][3] = qb[p][3];
          }
          if (P == 1) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              mma(kk[n], ka[0], kb[0][2 * n], kb[0][2 * n + 1]);
              mma(qk[n], qa[0], kb[0][2 * n], kb[0][2 * n + 1]);
            }
          } else {
            mma_pairs<P, true>(kk, kc, ka, kb);
            mma_pairs<P, true>(qk, qc, qa, kb);
          }
        }
        // decays between tokens, the two matrices
        const double cs = decay_sums(gv, lane);
        GroupMats& m = mats[(s & 1) * NG + pw];
        float read[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = g4 + (x >> 1) * 8, col = n * 8 + 2 * t4 + (x & 1);
            const double ci = __shfl_sync(0xffffffffu, cs, row);
            const double cj = __shfl_sync(0xffffffffu, cs, col);
            const float bj = __shfl_sync(0xffffffffu, bv, col);
            const float d = row >= col ? exp2f(float(ci - cj)) * bj : 0.f;
            read[n][x] = a.scale * (d * (qk[n][x] + qc[n][x]));
            L[row * kLP + col] = row > col ? d * (kk[n][x] + kc[n][x]) : 0.f;
          }
        {
          uint4 f[3];
          // columns of the product are the rows (i) of the read matrix
          split2(read[0][0], read[0][1], f[0].x, f[1].x, f[2].x);
          split2(read[1][0], read[1][1], f[0].y, f[1].y, f[2].y);
          split2(read[0][2], read[0][3], f[0].z, f[1].z, f[2].z);
          split2(read[1][2], read[1][3], f[0].w, f[1].w, f[2].w);
#pragma unroll
          for (int p = 0; p < 3; ++p) m.read[p][lane] = f[p];
        }
        invert_group(L, lane);
        {
          auto pair = [&](int i, int j) {
            return *reinterpret_cast<const float2*>(L + i * kLP + j);
          };
          const float2 x0 = pair(g4, 2 * t4), x1 = pair(g4, 8 + 2 * t4),
                       x2 = pair(g4 + 8, 2 * t4), x3 = pair(g4 + 8, 8 + 2 * t4);
          uint4 f[3];
          split2(x0.x, x0.y, f[0].x, f[1].x, f[2].x);
          split2(x1.x, x1.y, f[0].y, f[1].y, f[2].y);
          split2(x2.x, x2.y, f[0].z, f[1].z, f[2].z);
          split2(x3.x, x3.y, f[0].w, f[1].w, f[2].w);
#pragma unroll
          for (int p = 0; p < 3; ++p) m.inv[p][lane] = f[p];
        }
        const double last = __shfl_sync(0xffffffffu, cs, 15);
        if (lane < kG) {
          const float d = exp2f(float(cs));
          m.decay[lane] = d;
          m.out[lane] = a.scale * d;
          m.write[lane] = exp2f(float(last - cs)) * bv;
          if (lane == 15) m.end = d;
        }
      }
      __syncthreads();
    }
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int r0 = part * X::kVRows + warp * 16;  // this warp's value channels
  const int64_t state_at = ((int64_t(seq) * a.H + h) * N + r0) * N;
  float S[N / 8][4];  // 16 rows x N columns: accumulator tiles of 8 columns
#pragma unroll
  for (int n = 0; n < N / 8; ++n) {
    zero(S[n]);
    if (a.s0 != nullptr) {
      const float2 x = *reinterpret_cast<const float2*>(a.s0 + state_at + g4 * N + n * 8 + 2 * t4);
      const float2 z =
          *reinterpret_cast<const float2*>(a.s0 + state_at + (g4 + 8) * N + n * 8 + 2 * t4);
      S[n][0] = x.x; S[n][1] = x.y; S[n][2] = z.x; S[n][3] = z.y;
    }
  }
  T* y = static_cast<T*>(a.y) + t0 * v_row + int64_t(h) * N + r0;
  float* eo = e_out == nullptr ? nullptr : e_out + t0 * v_row + int64_t(h) * N + r0;
  auto put_state = [&](float* to) {
#pragma unroll
    for (int n = 0; n < N / 8; ++n) {
      *reinterpret_cast<float2*>(to + g4 * N + n * 8 + 2 * t4) = make_float2(S[n][0], S[n][1]);
      *reinterpret_cast<float2*>(to + (g4 + 8) * N + n * 8 + 2 * t4) =
          make_float2(S[n][2], S[n][3]);
    }
  };

  __syncthreads();  // the first step is prepared
  for (int i = 0; i < steps; ++i) {
#pragma unroll 1
    for (int gi = 0; gi < NG; ++gi) {
      const int first = i * X::kStep + gi * kG;
      if (first >= len) break;
      if (checkpoints != nullptr && first % kGdrChunk == 0)
        put_state(checkpoints +
                  ((gdr_chunk_base(a, seq, t0) + first / kGdrChunk) * a.H + h) * N * N + r0 * N);
      const GroupMats& m = mats[(i & 1) * NG + gi];
      const uint32_t grp = uint32_t(gi * kG * X::kPitch) * 2u;
      // S_0 K^T and S_0 Q^T
      float xm[2][4], xc[2][4], om[2][4], oc[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) zero(xm[n]), zero(xc[n]), zero(om[n]), zero(oc[n]);
      const uint32_t to = at_tokens(lane, X::kPitch) + grp;
#pragma unroll
      for (int c = 0; c < N; c += 16) {
        uint32_t sp[3][4], kb[P][4], qb[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p) {
          ldsm4(kb[p], tile(i, 0, p) + to + c * 2);
          ldsm4(qb[p], tile(i, 1, p) + to + c * 2);
        }
        split_tiles(S[c / 8], S[c / 8 + 1], sp);
        mma_pairs<P, true>(xm, xc, sp, kb);
        mma_pairs<P, !X::kBf16>(om, oc, sp, qb);
      }
      // e: V^T - C_i X as accumulator, plus its product with (I + A)^-1 - I
      float e[2][4], ec[2][4];
      {
        float vv[2][4];
        if (X::kBf16) {
          uint32_t r[4];
          ldsm4t(r, sb + X::kOffV + (i % 3) * X::kVTile +
                        uint32_t(gi * kG * X::kVPitch + warp * 16) * 2u +
                        at_transposed(lane, X::kVPitch));
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float2 lo = unpack(r[2 * n]), hi = unpack(r[2 * n + 1]);
            vv[n][0] = lo.x; vv[n][1] = lo.y; vv[n][2] = hi.x; vv[n][3] = hi.y;
          }
        } else {
          const float* vp = reinterpret_cast<const float*>(smem + X::kOffV + (i % 3) * X::kVTile) +
                            gi * kG * X::kVPitch + warp * 16;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              vv[n][x] = vp[(n * 8 + 2 * t4 + (x & 1)) * X::kVPitch + g4 + (x >> 1) * 8];
        }
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
      mma_up<3, true>(ec, ep, fb);
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
      mma_up<3, !X::kBf16>(o, ep, fb);
      float w[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float2 d = *reinterpret_cast<const float2*>(m.out + n * 8 + 2 * t4);
        const float2 f = *reinterpret_cast<const float2*>(m.write + n * 8 + 2 * t4);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          o[n][x] = fmaf((x & 1) ? d.y : d.x, om[n][x] + oc[n][x], o[n][x]);
          w[n][x] = e[n][x] * ((x & 1) ? f.y : f.x);
        }
      }
      // S = C S_0 + W^T K, the products summed on their own
      uint32_t wp[3][4];
      split_tiles(w[0], w[1], wp);
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
        mma_up<P, true>(d, wp, kb);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) S[c / 8 + n][x] = fmaf(end, S[c / 8 + n][x], d[n][x]);
      }
      // out: fp32 eight channels of a token at a time, bf16 through shared memory in 32-byte rows
      if (eo != nullptr) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int tok = first + n * 8 + 2 * t4 + (x & 1);
            if (tok < len) eo[tok * v_row + g4 + (x >> 1) * 8] = e[n][x];
          }
      }
      if (X::kBf16) {
        __nv_bfloat16* st =
            reinterpret_cast<__nv_bfloat16*>(smem + X::kOffY) + warp * kG * X::kYPitch;
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            st[(n * 8 + 2 * t4 + (x & 1)) * X::kYPitch + g4 + (x >> 1) * 8] =
                __float2bfloat16_rn(o[n][x]);
        __syncwarp();
        const int tok = lane >> 1, c = (lane & 1) * 8;
        if (first + tok < len)
          *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(y) +
                                    int64_t(first + tok) * v_row + c) =
              *reinterpret_cast<const uint4*>(st + tok * X::kYPitch + c);
      } else {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int tok = first + n * 8 + 2 * t4 + (x & 1);
            if (tok < len) reinterpret_cast<float*>(y)[tok * v_row + g4 + (x >> 1) * 8] = o[n][x];
          }
      }
    }
    __syncthreads();
  }
  if (a.s1 != nullptr) put_state(a.s1 + state_at);
}

template <typename T, int N, int NC, int NG>
int launch(const GdrArgs& a, float* e, float* checkpoints, cudaStream_t stream) {
  using X = Shape<T, N, NC, NG>;
  auto* kernel = gdr_fwd_kernel<T, N, NC, NG>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, X::kSmem) !=
      cudaSuccess)
    return WKV_ERR_CUDA;
  const unsigned grid = unsigned(int64_t(a.n_seqs) * a.H * (N / X::kVRows));
  kernel<<<grid, X::kThreads, X::kSmem, stream>>>(a, e, checkpoints);
  return cudaPeekAtLastError() == cudaSuccess ? WKV_OK : WKV_ERR_CUDA;
}

}  // namespace

int launch_gdr_chunked(const GdrArgs& a, float* e, float* checkpoints, cudaStream_t stream) {
  if (a.bf16)
    return a.N == 64 ? launch<__nv_bfloat16, 64, 4, 2>(a, e, checkpoints, stream)
                     : launch<__nv_bfloat16, 128, 8, 2>(a, e, checkpoints, stream);
  return a.N == 64 ? launch<float, 64, 4, 2>(a, e, checkpoints, stream)
                   : launch<float, 128, 8, 1>(a, e, checkpoints, stream);
}

}  // namespace wkv
