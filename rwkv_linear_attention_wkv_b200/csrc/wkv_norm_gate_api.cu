// C-ABI entry points of the norms around a block: argument checks and launches. Declarations
// and their documentation: include/wkv.h.
#include <cstdint>

#include "wkv_internal.h"

namespace wkv {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check(const wkv_norm_gate_problem* p, const void* gate, const void* x, const float* scale) {
  if (p == nullptr || p->R < 0 || p->C < 0) return WKV_ERR_INVALID_ARG;
  if (p->dtype != WKV_DTYPE_F32 && p->dtype != WKV_DTYPE_BF16) return WKV_ERR_INVALID_ARG;
  if (!(p->eps > 0.f)) return WKV_ERR_INVALID_ARG;
  if (gate && p->act != WKV_ACT_SIGMOID && p->act != WKV_ACT_SILU) return WKV_ERR_INVALID_ARG;
  if (p->C == 0) return WKV_OK;
  if (scale && !x && p->R > 0) return WKV_ERR_INVALID_ARG;  // empty arrays may have no address
  if (p->group <= 0 || p->C % p->group != 0) return WKV_ERR_INVALID_ARG;
  if (p->C > norm_gate_max_c() || p->R > (int64_t(1) << 40)) return WKV_ERR_UNSUPPORTED;
  return WKV_OK;
}

NormGateArgs args_of(const wkv_norm_gate_problem* p) {
  NormGateArgs a{};
  a.R = p->R; a.C = int(p->C); a.group = int(p->group); a.act = p->act;
  a.bf16 = p->dtype == WKV_DTYPE_BF16;
  a.eps = p->eps;
  return a;
}

}  // namespace

extern "C" {

WKV_API int wkv_norm_gate_forward(const wkv_norm_gate_problem* p, const void* h,
                                  const float* weight, const void* gate, const void* x,
                                  const float* scale, const float* next_weight, void* out,
                                  void* y, cudaStream_t stream) {
  if (int rc = check(p, gate, x, scale)) return rc;
  if (p->R == 0 || p->C == 0) return WKV_OK;
  if ((next_weight == nullptr) != (y == nullptr)) return WKV_ERR_INVALID_ARG;
  if (!h || !out) return WKV_ERR_INVALID_ARG;
  const size_t e = p->dtype == WKV_DTYPE_BF16 ? 2 : 4;
  for (const void* q : {h, gate, x, (const void*)out, (const void*)y})
    if (!aligned(q, e)) return WKV_ERR_ALIGNMENT;
  if (!aligned(weight, 4) || !aligned(scale, 4) || !aligned(next_weight, 4))
    return WKV_ERR_ALIGNMENT;
  NormGateArgs a = args_of(p);
  a.h = h; a.weight = weight; a.gate = gate; a.x = x; a.scale = scale;
  a.next_weight = next_weight; a.out = out; a.y = y;
  return launch_norm_gate_forward(a, stream);
}

WKV_API size_t wkv_norm_gate_workspace_bytes(int64_t R, int64_t C) {
  return norm_gate_workspace_bytes(R, C);
}

WKV_API int wkv_norm_gate_backward(const wkv_norm_gate_problem* p, const void* h,
                                   const float* weight, const void* gate, const void* x,
                                   const float* scale, const float* next_weight,
                                   const void* dout, const void* dy, void* dh, float* dweight,
                                   void* dgate, void* dx, float* dscale, float* dnext_weight,
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (int rc = check(p, gate, x, scale)) return rc;
  if (p->C == 0) return WKV_OK;
  if (!aligned(weight, 4) || !aligned(scale, 4) || !aligned(next_weight, 4) ||
      !aligned(dweight, 4) || !aligned(dscale, 4) || !aligned(dnext_weight, 4))
    return WKV_ERR_ALIGNMENT;
  if (p->R == 0) {
    for (float* q : {dweight, dscale, dnext_weight})
      if (q && cudaMemsetAsync(q, 0, size_t(p->C) * 4, stream) != cudaSuccess) return WKV_ERR_CUDA;
    return WKV_OK;
  }
  if (dy && !next_weight) return WKV_ERR_INVALID_ARG;
  if ((dgate && !gate) || (dx && !x) || (dscale && !scale) || (dnext_weight && !dy))
    return WKV_ERR_INVALID_ARG;
  if (!h || !dh || (!dout && !dy)) return WKV_ERR_INVALID_ARG;
  const size_t e = p->dtype == WKV_DTYPE_BF16 ? 2 : 4;
  for (const void* q : {h, gate, x, dout, dy, (const void*)dh, (const void*)dgate, (const void*)dx})
    if (!aligned(q, e)) return WKV_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < norm_gate_workspace_bytes(p->R, p->C))
    return WKV_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return WKV_ERR_ALIGNMENT;
  NormGateArgs a = args_of(p);
  a.h = h; a.weight = weight; a.gate = gate; a.x = x; a.scale = scale;
  a.next_weight = next_weight; a.dout = dout; a.dy = dy;
  a.dh = dh; a.dweight = dweight; a.dgate = dgate; a.dx = dx; a.dscale = dscale;
  a.dnext_weight = dnext_weight;
  a.partial = static_cast<float*>(workspace);
  return launch_norm_gate_backward(a, stream);
}

}  // extern "C"

}  // namespace wkv
