// Internal interfaces between the C-ABI layer (wkv_api.cu) and the kernel files.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include <utility>

#include "wkv.h"

namespace wkv {

// For tests: launches of this thread that are still to report a failure (after they were made).
inline thread_local int failing_launches = 0;

// A launch and how that launch went. (After <<<>>> one can only ask for the thread's last error,
// which may be an earlier call's: CUDA keeps it until somebody takes it.)
template <typename... Params, typename... Args>
int launch_kernel(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                  cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = block;
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  if (cudaLaunchKernelEx(&config, kernel, std::forward<Args>(args)...) != cudaSuccess)
    return WKV_ERR_CUDA;
  if (failing_launches > 0) {
    --failing_launches;
    return WKV_ERR_CUDA;
  }
  return WKV_OK;
}

// Arguments of one forward pass over (B, T, C). k, v, r, y are fp32 or bf16 according to
// the entry point; r may be null (no gate); a0/b0/p0 null = empty initial state; a1/b1/p1
// null = final state not wanted.
struct FwdArgs {
  int64_t B, T, C;
  const float* w;
  const float* u;
  const void* k;
  const void* v;
  const void* r;
  void* y;
  const float* a0;
  const float* b0;
  const float* p0;
  float* a1;
  float* b1;
  float* p1;
  unsigned* err;  // device error word
};

// Device address of this library's error word on the current device (nullptr on error).
unsigned* device_error_word();

// 3-D tiled tensor map over a (B, T, C) tensor (C fastest) with a box of
// [box_c channels x box_t tokens x 1 batch row]. Returns a wkv_status.
int encode_btc_map(CUtensorMap* map, const void* base, CUtensorMapDataType dtype,
                   int elem_bytes, int64_t B, int64_t T, int64_t C, int box_c, int box_t);

// Whether the TMA streaming kernel can describe this problem (alignment, extents).
bool fwd_tma_ok(const FwdArgs& a, int elem_bytes);

// Whole-sequence forward, one thread per channel (streaming TMA kernel, or the plain
// kernel when the TMA kernel cannot be used or force_plain is set).
int launch_fwd_stream(const FwdArgs& a, bool bf16, bool force_plain, cudaStream_t stream);

// Chunked (time-parallel) forward for problems with few channels; fp32 only.
// scratch: device memory of chunked_scratch_bytes(); its first flag_bytes must be
// zero on entry (the caller clears them).
size_t chunked_scratch_bytes(int64_t B, int64_t T, int64_t C, int64_t* flag_bytes,
                             int* n_segments);
int launch_fwd_chunked(const FwdArgs& a, void* scratch, int n_segments, cudaStream_t stream);
// Same, with the wait limit (ns) given and, for tests of the bounded wait, segment 0
// optionally withholding its published aggregate so that its successors give up.
int launch_fwd_chunked_ex(const FwdArgs& a, void* scratch, int n_segments,
                          unsigned long long wait_ns, int withhold_seg0, cudaStream_t stream);

// One decode step over N x L x C states.
struct DecodeArgs {
  int64_t N, L, C;
  const float* w;
  const float* u;
  const float* k;
  const float* v;
  const float* r;
  float* y;
  float* a;
  float* b;
  float* p;
};
int launch_decode(const DecodeArgs& a, cudaStream_t stream);
// S chained tokens: k, v, r, y are [S, N, L, C]; the state stays on chip between tokens.
int launch_decode_steps(const DecodeArgs& a, int64_t S, cudaStream_t stream);

// Matrix-valued-state forward (heads of 64), chunked on the tensor cores. scratch: device
// memory of mstate_scratch_bytes(B, H) bytes (cleared in part by the launcher).
size_t mstate_scratch_bytes(int64_t B, int64_t H);
int launch_mstate(int64_t B, int64_t T, int64_t H, const float* r, const float* w,
                  const float* k, const float* v, float* y, const float* s0, float* s1,
                  void* scratch, unsigned* err, cudaStream_t stream);

// Backward over (B, T, C), fp32. r null: no gate (dr must be null). ws: device workspace of
// backward_workspace_bytes(B, T, C) bytes, 256-byte aligned; no part needs clearing.
struct BwdArgs {
  int64_t B, T, C;
  const float* w;
  const float* u;
  const float* k;
  const float* v;
  const float* r;
  const float* dy;
  float* dk;
  float* dv;
  float* dw;
  float* du;
  float* dr;
  void* ws;
  unsigned* err;
  // Backward through a state (all may be NULL): the initial state (a0, b0, p0) [B, C];
  // the gradients (ga1, gb1) of a later loss with respect to the final state's a1, b1,
  // whose log-scale is p1 [B, C]; and the outputs (da0, db0, dp0) [B, C].
  const float* a0 = nullptr;
  const float* b0 = nullptr;
  const float* p0 = nullptr;
  const float* ga1 = nullptr;
  const float* gb1 = nullptr;
  const float* p1 = nullptr;
  float* da0 = nullptr;
  float* db0 = nullptr;
  float* dp0 = nullptr;
  // Chain waits of the time-parallel passes: their limit (ns) and, for tests of the
  // bounded wait only, the last segment of the reverse pass withholding its published map.
  unsigned long long wait_ns = 2000000000ull;
  int withhold_last_map = 0;
  // The workspace already holds the checkpoints (written by launch_fwd_ckpt over the same
  // w, k, v and initial state): the checkpoint pass is skipped and the reverse pass
  // recomputes in the streaming forward's arithmetic. Time-parallel path only.
  int have_ckpt = 0;
};
size_t backward_workspace_bytes(int64_t B, int64_t T, int64_t C);
// Where the backward's workspace keeps the checkpoints ([B, ceil(T/16), C] float4: the state
// (a, b, Q, pl) entering every chunk of 16 tokens) and the state after the last token
// ([B, C] float4).
void backward_checkpoint_ptrs(void* ws, int64_t B, int64_t T, int64_t C, float4** ckpt,
                              float4** ckend);
// Whether the backward takes its time-parallel (checkpointed) path for these arguments.
bool backward_time_parallel_ok(const BwdArgs& a);
// Forward (fp32, TMA shapes only: else WKV_ERR_UNSUPPORTED) that also writes the backward's
// checkpoints into its workspace ws: the streaming kernel in its checkpointing mode
// (wkv_fwd.cu); a backward with have_ckpt set recomputes in the same arithmetic.
int launch_fwd_ckpt(const FwdArgs& a, void* ws, cudaStream_t stream);
int launch_backward(const BwdArgs& a, bool force_plain, cudaStream_t stream);
// Which reverse pass the TMA path takes: 0 automatic, 1 time-parallel segments, 2 one CTA
// per channel group, 3 one CTA of four warps per channel group (a test hook; process-wide).
void set_backward_path(int path);
// T == 0 with the state's gradients wanted: they pass straight through.
int launch_backward_no_tokens(const BwdArgs& a, cudaStream_t stream);

// RWKV-7 recurrence (wkv7.cu), head size 64, all pointers 16-byte aligned.
int launch_wkv7(int64_t B, int64_t T, int64_t H, const float* r, const float* w, const float* k,
                const float* v, const float* a, const float* b, float* y, const float* s0,
                float* s1, unsigned* err, cudaStream_t stream);

// Gated delta rule (wkv_gdr_*.cu). Sequences are batch rows, or spans of one packed row.
struct GdrArgs {
  int B, T, Hk, H, N;
  int n_seqs;               // batch rows, or packed sequences
  const int32_t* offsets;   // packed: n_seqs + 1 token offsets (device), else null
  bool bf16;
  float scale;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  void* y;
  const float* s0;
  float* s1;
  // decode: states picked by slot
  int n_slots = 0;
  const int32_t* slots = nullptr;
};
// One token a row, the states in place.
int launch_gdr_decode(const GdrArgs& a, cudaStream_t stream);
// Walks in segments, side by side, where a few heads would leave most SMs idle (wkv_gdr_seg.cu).
// A state leaves a segment as S M + B, M and B from the segment's tokens alone.
struct GdrSegs {
  int tokens = 0;  // of a segment (a multiple of every chunk's); 0: sequences are walked whole
  int slots = 0;   // segments, numbered through the sequences (packed: as many as there may be)
  float* leave = nullptr;  // (slots, H, N, N): B, then the state leaving a segment
  float* unit = nullptr;   // (slots, H, N, N): M; for a walk's first segment the state it starts from
};
// The plan for a problem; reverse or not, the same. < 0 on a CUDA error, else the scratch in bytes.
int64_t gdr_plan_segments(const GdrArgs& a, GdrSegs* segs);
// leave[s] for the inner segments of every walk, from the walk's first to its last but one.
int launch_gdr_combine(const GdrArgs& a, const GdrSegs& segs, bool reverse, cudaStream_t stream);
// In groups of 16 tokens on the matrix units. e (tokens, H, N) and checkpoints (chunks, H, N, N)
// are what the backward reads: every token's error before its write, and the state entering
// every chunk of gdr_chunk() tokens of every sequence; null = not wanted.
int launch_gdr_chunked(const GdrArgs& a, const GdrSegs& segs, float* e, float* checkpoints,
                       cudaStream_t stream);
// Tokens of a chunk: 32 where the chunk's operands would not fit shared memory at 64.
__host__ __device__ constexpr int gdr_chunk(bool bf16, int N) { return !bf16 && N == 128 ? 32 : 64; }
// Number of a sequence's first chunk. A packed sequence has two numbers more than whole chunks, so
// that they follow from the offsets alone (which must not decrease); a batch row has one more than
// chunks, which nothing is kept under.
__host__ __device__ inline int64_t gdr_chunk_base(const GdrArgs& a, int seq, int64_t first_token) {
  const int chunk = gdr_chunk(a.bf16, a.N);
  return a.offsets == nullptr ? int64_t(seq) * ((int64_t(a.T) + chunk - 1) / chunk + 1)
                              : first_token / chunk + 2 * int64_t(seq);
}
__host__ __device__ inline int64_t gdr_chunks(const GdrArgs& a) {
  const int chunk = gdr_chunk(a.bf16, a.N);
  return a.offsets == nullptr ? int64_t(a.n_seqs) * ((int64_t(a.T) + chunk - 1) / chunk + 1)
                              : a.T / chunk + 2 * int64_t(a.n_seqs) + 1;
}
// Gradients. e, checkpoints: the forward's. du (tokens, H, N) and dstates (chunks, H, N, N):
// scratch for the gradients of the written values and of the state leaving every chunk.
struct GdrBwdArgs {
  GdrArgs p;  // q, k, v, g, beta and sizes
  const void* dy;
  const float* e;
  const float* checkpoints;
  const float* ds1;
  float* du;
  float* dstates;
  void* dq;
  void* dk;
  void* dv;
  float* dg;
  float* dbeta;
  float* ds0;
};
int launch_gdr_backward(const GdrBwdArgs& a, const GdrSegs& segs, cudaStream_t stream);

// Norm, gate, residual and next norm around a block (wkv_norm_gate.cu); null pointers are what
// the entry points let a caller leave out.
struct NormGateArgs {
  int64_t R;
  int C, group, act;
  bool bf16;
  float eps;
  const void* h;
  const float* weight;
  const void* gate;
  const void* x;
  const float* scale;
  const float* next_weight;
  void* out;
  void* y;
  // backward
  const void* dout = nullptr;
  const void* dy = nullptr;
  void* dh = nullptr;
  float* dweight = nullptr;
  void* dgate = nullptr;
  void* dx = nullptr;
  float* dscale = nullptr;
  float* dnext_weight = nullptr;
  float* partial = nullptr;  // norm_gate_workspace_bytes(R, C)
};
int64_t norm_gate_max_c();
size_t norm_gate_workspace_bytes(int64_t R, int64_t C);
int launch_norm_gate_forward(const NormGateArgs& a, cudaStream_t stream);
int launch_norm_gate_backward(const NormGateArgs& a, cudaStream_t stream);

}  // namespace wkv
