// Internal launch interfaces between the C ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr {

// Records the device time of the enclosed launch(es) on `s` when tracing is
// enabled (kda_trace_enable); does nothing otherwise.
class TraceScope {
 public:
  TraceScope(const char *name, cudaStream_t s);
  ~TraceScope();
  TraceScope(const TraceScope &) = delete;
  TraceScope &operator=(const TraceScope &) = delete;

 private:
  const char *name_;
  cudaStream_t stream_;
  void *start_ = nullptr;
  void *stop_ = nullptr;
};

// Sets the text kda_last_error() returns on the calling host thread.
void set_last_error(const char *msg);

// Multiprocessor count of the current device.
int sm_count();

// Bounds-checked build: violations counted by each translation unit's
// kernels since the last read (0 in the normal build; ~0u if unreadable).
unsigned int oob_count_prefill_tc();
unsigned int oob_count_prefill_simt();
unsigned int oob_count_decode();
unsigned int oob_count_api();
unsigned int oob_count_glr();
unsigned int oob_count_gated_norm();
unsigned int oob_count_add_norm();

// Token-by-token form: T tokens for each of N sequences ([N, T, H, d]
// layout), state updated in place.  T = 1 is one decode step.
struct DecodeArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  void *o;
  float *state;
  const int32_t *slots;  // device [N] state-pool slots, or nullptr (slot n = n)
  int64_t num_slots;     // pool capacity; slots outside [0, num_slots) are padding
  int N, T, H_qk, H_v, d_k, d_v;
  bool channel_gate;  // KDA (per-channel) or Gated DeltaNet (scalar)
  bool decay_first;   // decay before the erase (KDA only)
  bool bf16;          // io dtype
};

cudaError_t launch_recurrent(const DecodeArgs &a, cudaStream_t stream);

// dst[dst_slots[n]] = src[src_slots[n]] for n < N, per_seq_floats floats per
// entry (a multiple of 4, 16-byte aligned buffers); NULL slots = identity.
// A source slot outside [0, src_limit) copies zeros (as does src == NULL); a
// destination slot outside [0, dst_limit) is skipped.
cudaError_t launch_state_copy(const float *src, const int32_t *src_slots, int64_t src_limit,
                              float *dst, const int32_t *dst_slots, int64_t dst_limit, int N,
                              int64_t per_seq_floats, cudaStream_t stream);

// One bounded on-device wait that expires: writes KDA_DEVICE_TIMEOUT to *status.
cudaError_t launch_wait_timeout(int32_t *status, uint32_t max_polls, cudaStream_t stream);

// Chunk length of the prefill kernels (tokens per chunk).
constexpr int kChunk = 64;

struct PrefillArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  void *o;
  const float *initial_state;
  float *final_state;
  const int32_t *state_slots;  // device [num_seqs] pool slots of the states, or nullptr
  int64_t num_slots;           // pool capacity (slots outside [0, num_slots): no state)
  const int32_t *cu_seqlens;  // device, or nullptr (dense)
  int num_seqs;               // N
  int B, T, H_qk, H_v, d_k, d_v;
  bool channel_gate;
  bool decay_first;  // decay before the erase (KDA only)
  bool bf16;
  // workspace (device); status word at offset 0
  void *workspace;
  size_t workspace_bytes;
  // chunks: an upper bound on the total number of chunks over all sequences
  int64_t max_chunks;
};

// Bytes of workspace a prefill call needs (includes the 256-byte status block).
size_t prefill_workspace_bytes(int T, int H_v, int d_k, int d_v, int num_seqs, bool bf16);

cudaError_t launch_prefill_f32(const PrefillArgs &a, cudaStream_t stream);
cudaError_t launch_prefill_tc(const PrefillArgs &a, cudaStream_t stream);

// Gated linear recurrence over a vector state.  Tokens are numbered along one
// axis (sequence b of a dense batch begins at b T).
constexpr int kGlrChunk = 64;         // tokens between two saved states
constexpr int kGlrShortestGroup = 8;  // tiles of a group of the chain, at least (tiles are a chunk or longer)

struct GlrArgs {
  const void *x;
  const float *g;
  int64_t ld_x, ld_g;  // elements from one token's row to the next
  void *h;
  const float *initial_state;
  float *final_state;          // glr_step: the states, updated in place
  const int32_t *state_slots;  // device [num_seqs] pool slots, or nullptr
  int64_t num_slots;
  float *chunk_states;  // [chunks, D]: the state that enters each chunk
  // backward
  const void *dh;
  int64_t ld_dh;
  const float *dfinal;
  void *dx;
  float *dg, *dinitial;
  const int32_t *cu_seqlens;  // device [num_seqs + 1], or nullptr (dense)
  int num_seqs, T, D;
  int64_t tokens, chunks;
  bool complement, bf16;
  // workspace
  int32_t *status;
  int32_t *ticket;
  uint64_t *tile_map;   // [tiles][pitch], then the groups' words [groups][pitch]
  int64_t pitch;        // D, rounded up to whole tiles
  int32_t *tile_marks;  // packed: whether a sequence begins or ends in the tile
  bool own_chunks;  // backward: chunk_states is workspace, to be filled first
  // set at the launch
  uint64_t *carry;
  int stripes, tile_tokens;
  int64_t tiles, groups;
  bool chained;
  bool keep_status;       // the second pass of a call: an error of the first one stays
  uint32_t first_ticket;  // 0; the self-test leaves out the tiles before it ...
  uint32_t max_polls;     // ... and gives up waiting for them after these
};
constexpr int kGlrGroup = 16;                  // tiles of a group of the chain
constexpr uint32_t kGlrMaxPolls = 1u << 20;    // of one wait in the chain: about a second

cudaError_t launch_glr_fwd(const GlrArgs &a, cudaStream_t stream);
cudaError_t launch_glr_bwd(const GlrArgs &a, cudaStream_t stream);
cudaError_t launch_glr_step(const GlrArgs &a, cudaStream_t stream);

// RMS norm of each head's d channels, a weight, and a gate.
struct GatedNormArgs {
  const void *dy, *x, *z;
  int64_t ld_dy, ld_x, ld_z;  // elements from one token's row to the next
  const float *weight;        // [d] or nullptr
  void *y, *dx, *dz;
  float *dweight;
  float *partial;  // workspace: [norm_blocks(), d] sums of the weight's gradient
  int64_t tokens;
  int H, d, gate;
  float eps;
  bool bf16;
};
cudaError_t launch_gated_norm_fwd(const GatedNormArgs &a, cudaStream_t stream);
cudaError_t launch_gated_norm_bwd(const GatedNormArgs &a, cudaStream_t stream);

// residual + scale y and the RMS norm of the sum.
struct AddNormArgs {
  const void *residual, *y;
  const float *scale, *weight;  // [D] or nullptr
  void *residual_out, *n;
  // backward
  const void *dn, *dresidual_out;
  void *dresidual, *dy;
  float *dscale, *dweight;
  float *partial;  // workspace: [2][norm_blocks(), D]
  int64_t rows;
  int D;
  float eps;
  bool res_bf16, bf16;
};
cudaError_t launch_add_norm_fwd(const AddNormArgs &a, cudaStream_t stream);
cudaError_t launch_add_norm_bwd(const AddNormArgs &a, cudaStream_t stream);

// Most blocks that a norm's backward pass launches, i.e. the rows of its
// partial column sums.  The same on every device, so that a workspace size does
// not depend on the current one.
constexpr int kNormBlocks = 1184;
// Longest row of the norms.
constexpr int kNormMaxRow = 16384;

// Device-side check of cu_seqlens; writes KDA_DEVICE_BAD_CU_SEQLENS into the
// status word on failure (kernels then skip all work).
cudaError_t launch_check_cu_seqlens(const int32_t *cu, int num_seqs, int T, int32_t *status,
                                    cudaStream_t stream);

}  // namespace gdr
