// C-ABI entry points of the gated delta rule: argument checks, plan selection, launches.
// Declarations and their documentation: include/wkv.h.
#include <algorithm>
#include <cstdint>

#include "wkv_internal.h"

namespace wkv {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Sizes of a problem. WKV_OK with *empty set where there is nothing to index.
int check_problem(const wkv_gdr_problem* p, bool* empty) {
  *empty = false;
  if (p == nullptr) return WKV_ERR_INVALID_ARG;
  if (p->B < 0 || p->T < 0 || p->Hk < 0 || p->H < 0 || p->N < 0) return WKV_ERR_INVALID_ARG;
  if (p->dtype != WKV_DTYPE_F32 && p->dtype != WKV_DTYPE_BF16) return WKV_ERR_INVALID_ARG;
  const bool packed = p->seq_offsets != nullptr;
  if (packed && (p->n_seqs < 0 || p->B != 1)) return WKV_ERR_INVALID_ARG;
  if (!aligned(p->seq_offsets, 4) || !aligned(p->workspace, 16)) return WKV_ERR_ALIGNMENT;
  const int64_t seqs = packed ? p->n_seqs : p->B;
  if (seqs == 0 || p->H == 0) {
    *empty = true;
    return WKV_OK;
  }
  if (p->N != 64 && p->N != 128) return WKV_ERR_UNSUPPORTED;
  if (p->Hk == 0 || p->H % p->Hk != 0) return WKV_ERR_UNSUPPORTED;
  // Tokens (rounded up to a kernel's step, or to what segments there may be) and heads are indexed in
  // int32, elements in int64; a grid is 31 bits wide.
  constexpr int64_t kMax = int64_t(1) << 31;
  if (p->T > kMax - 1024 || p->H >= (int64_t(1) << 20) || p->B >= kMax || seqs >= kMax / 8 / p->H)
    return WKV_ERR_UNSUPPORTED;
  if (p->T > 0 && (p->B > (int64_t(1) << 40) / p->T ||
                   p->B * p->T > INT64_MAX / 16 / (p->H * p->N)))
    return WKV_ERR_UNSUPPORTED;
  return WKV_OK;
}

GdrArgs args_of(const wkv_gdr_problem* p) {
  GdrArgs a{};
  a.B = int(p->B); a.T = int(p->T); a.Hk = int(p->Hk); a.H = int(p->H); a.N = int(p->N);
  a.offsets = p->seq_offsets;
  a.n_seqs = p->seq_offsets ? int(p->n_seqs) : a.B;
  a.bf16 = p->dtype == WKV_DTYPE_BF16;
  a.scale = p->scale;
  return a;
}

int pass_state(const float* s0, float* s1, size_t bytes, cudaStream_t stream) {
  if (s1 == nullptr || s1 == s0) return WKV_OK;
  const cudaError_t e = s0 ? cudaMemcpyAsync(s1, s0, bytes, cudaMemcpyDeviceToDevice, stream)
                           : cudaMemsetAsync(s1, 0, bytes, stream);
  return e == cudaSuccess ? WKV_OK : WKV_ERR_CUDA;
}

// Checkpoints: every token's e, then the state entering every chunk. Workspace: the same shapes.
struct Saved {
  size_t tokens, states;  // floats
};
Saved saved_of(const GdrArgs& a) {
  return {size_t(a.B) * a.T * a.H * a.N, size_t(gdr_chunks(a)) * a.H * a.N * a.N};
}
size_t saved_bytes(const wkv_gdr_problem* p) {
  bool empty;
  if (check_problem(p, &empty) != WKV_OK || empty || p->T == 0) return 0;
  const Saved s = saved_of(args_of(p));
  return (s.tokens + s.states) * sizeof(float);
}

// The plan of segments for a walk with `bytes` of scratch at hand: none where they do not fit.
int segments_in(const GdrArgs& a, void* scratch, size_t bytes, GdrSegs* segs) {
  const int64_t need = gdr_plan_segments(a, segs);
  if (need < 0) return WKV_ERR_CUDA;
  if (need == 0 || scratch == nullptr || size_t(need) > bytes) {
    *segs = GdrSegs();
    return WKV_OK;
  }
  segs->leave = static_cast<float*>(scratch);
  segs->unit = segs->leave + size_t(segs->slots) * a.H * a.N * a.N;
  return WKV_OK;
}
size_t segment_bytes(const wkv_gdr_problem* p) {
  bool empty;
  if (check_problem(p, &empty) != WKV_OK || empty || p->T == 0) return 0;
  GdrSegs segs;
  return size_t(std::max<int64_t>(0, gdr_plan_segments(args_of(p), &segs)));
}

// Forward, with somewhere to put the checkpoints or without.
int forward(const wkv_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
            const float* beta, void* y, const float* s0, float* s1, bool keep, void* saved,
            size_t saved_size, cudaStream_t stream) {
  bool empty;
  if (int rc = check_problem(p, &empty)) return rc;
  if (empty) return WKV_OK;
  if (p->T > 0 && (!q || !k || !v || !g || !beta || !y)) return WKV_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, (const void*)y, (const void*)s0, (const void*)s1,
                        (const void*)saved})
    if (!aligned(x, 16)) return WKV_ERR_ALIGNMENT;
  if (!aligned(g, 4) || !aligned(beta, 4)) return WKV_ERR_ALIGNMENT;
  GdrArgs a = args_of(p);
  if (a.T == 0) return pass_state(s0, s1, size_t(a.n_seqs) * a.H * a.N * a.N * 4, stream);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.y = y; a.s0 = s0; a.s1 = s1;
  if (keep && (saved == nullptr || saved_size < saved_bytes(p))) return WKV_ERR_INVALID_ARG;
  float* const e = keep ? static_cast<float*>(saved) : nullptr;
  float* const states = keep ? e + saved_of(a).tokens : nullptr;
  GdrSegs segs;
  if (int rc = segments_in(a, p->workspace, p->workspace_bytes, &segs)) return rc;
  return launch_gdr_chunked(a, segs, e, states, stream);
}

}  // namespace

extern "C" {

WKV_API int wkv_gdr_forward(const wkv_gdr_problem* p, const void* q, const void* k,
                            const void* v, const float* g, const float* beta, void* y,
                            const float* s0, float* s1, cudaStream_t stream) {
  return forward(p, q, k, v, g, beta, y, s0, s1, false, nullptr, 0, stream);
}

WKV_API size_t wkv_gdr_checkpoint_bytes(const wkv_gdr_problem* p) { return saved_bytes(p); }
WKV_API size_t wkv_gdr_forward_workspace_bytes(const wkv_gdr_problem* p) {
  return segment_bytes(p);
}
WKV_API size_t wkv_gdr_backward_workspace_bytes(const wkv_gdr_problem* p) {
  return saved_bytes(p) + segment_bytes(p);
}

WKV_API int wkv_gdr_forward_checkpointed(const wkv_gdr_problem* p, const void* q, const void* k,
                                         const void* v, const float* g, const float* beta, void* y,
                                         const float* s0, float* s1, void* checkpoints,
                                         size_t checkpoint_bytes, cudaStream_t stream) {
  return forward(p, q, k, v, g, beta, y, s0, s1, true, checkpoints, checkpoint_bytes, stream);
}

WKV_API int wkv_gdr_backward(const wkv_gdr_problem* p, const void* q, const void* k,
                             const void* v, const float* g, const float* beta, const void* dy,
                             const void* checkpoints, size_t checkpoint_bytes, const float* ds1,
                             void* dq, void* dk, void* dv, float* dg, float* dbeta, float* ds0,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  bool empty;
  if (int rc = check_problem(p, &empty)) return rc;
  if (empty) return WKV_OK;
  for (const void* x : {q, k, v, dy, checkpoints, (const void*)dq, (const void*)dk, (const void*)dv,
                        (const void*)ds1, (const void*)ds0, (const void*)workspace})
    if (!aligned(x, 16)) return WKV_ERR_ALIGNMENT;
  for (const void* x : {(const void*)g, (const void*)beta, (const void*)dg, (const void*)dbeta})
    if (!aligned(x, 4)) return WKV_ERR_ALIGNMENT;
  GdrBwdArgs b{};
  b.p = args_of(p);
  if (p->T == 0)
    return pass_state(ds1, ds0, size_t(b.p.n_seqs) * b.p.H * b.p.N * b.p.N * 4, stream);
  for (const void* x : {q, k, v, (const void*)g, (const void*)beta, dy, checkpoints, (const void*)dq,
                        (const void*)dk, (const void*)dv, (const void*)dg, (const void*)dbeta,
                        (const void*)workspace})
    if (x == nullptr) return WKV_ERR_INVALID_ARG;
  if (checkpoint_bytes < saved_bytes(p) || workspace_bytes < saved_bytes(p))
    return WKV_ERR_INVALID_ARG;
  if (gdr_chunks(b.p) > ((int64_t(1) << 31) - 1) / b.p.Hk) return WKV_ERR_UNSUPPORTED;
  const Saved s = saved_of(b.p);
  b.p.q = q; b.p.k = k; b.p.v = v; b.p.g = g; b.p.beta = beta;
  b.dy = dy;
  b.e = static_cast<const float*>(checkpoints);
  b.checkpoints = b.e + s.tokens;
  b.ds1 = ds1;
  b.du = static_cast<float*>(workspace);
  b.dstates = b.du + s.tokens;
  b.dq = dq; b.dk = dk; b.dv = dv; b.dg = dg; b.dbeta = dbeta; b.ds0 = ds0;
  GdrSegs segs;
  const size_t used = saved_bytes(p);
  if (int rc = segments_in(b.p, static_cast<char*>(workspace) + used, workspace_bytes - used, &segs))
    return rc;
  return launch_gdr_backward(b, segs, stream);
}

WKV_API int wkv_gdr_decode_step(const wkv_gdr_problem* p, const void* q, const void* k,
                                const void* v, const float* g, const float* beta, void* y,
                                float* state, int64_t n_slots, const int32_t* slots,
                                cudaStream_t stream) {
  bool empty;
  if (int rc = check_problem(p, &empty)) return rc;
  if (p->T != 1 || p->seq_offsets != nullptr || n_slots < 0) return WKV_ERR_INVALID_ARG;
  if (empty) return WKV_OK;
  if (!q || !k || !v || !g || !beta || !y || !state) return WKV_ERR_INVALID_ARG;
  if (slots == nullptr && n_slots < p->B) return WKV_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, (const void*)y, (const void*)state})
    if (!aligned(x, 16)) return WKV_ERR_ALIGNMENT;
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(slots, 4)) return WKV_ERR_ALIGNMENT;
  if (n_slots >= (int64_t(1) << 31)) return WKV_ERR_UNSUPPORTED;
  GdrArgs a = args_of(p);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.y = y; a.s0 = state; a.s1 = state;
  a.n_slots = int(n_slots);
  a.slots = slots;
  return launch_gdr_decode(a, stream);
}

}  // extern "C"

}  // namespace wkv
