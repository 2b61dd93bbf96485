// Entry points shared between translation units of libvt (not exported).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace vt {

// cuTensorMapEncodeTiled of the loaded driver, or nullptr
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// 2-D tensor map of rows of dims[0] elements, ld_bytes apart, dims[1] of them:
// boxes of box[0] x box[1] elements, 128-byte swizzle, zeros outside.  false: failed.
bool encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr,
                       const cuuint64_t (&dims)[2], cuuint64_t ld_bytes,
                       const cuuint32_t (&box)[2]);

// Multiprocessors of the current device (152 where that cannot be asked)
int num_sms();

// Clears the status word of a call whose one kernel would otherwise need a
// memset before it (which costs the call 2.5 us more).  The kernel behind it
// is launched with programmatic stream serialization, so the two launches
// overlap; it has to wait (griddepcontrol.wait) in the threads that raise
// flags, and needs to for nothing else: the clearing kernel is launched
// without that attribute, so everything before the call has completed when
// either starts.
int clear_status(cudaStream_t s, int32_t* dev_status);

constexpr int kDraftTopkMax = 32;  // largest k of the drafter's top-k

// The second half of a drafting step, after a projection that left z (scaled
// by log2(e) / T; raw when greedy) in q and one partial per tile_rows rows in
// part[G][B]: softmax and draw, or the one-hot q and argmax when greedy.
int draft_finish(cudaStream_t s, int B, int K, bool greedy, const float2* part, int G,
                 int tile_rows, const float* uniforms, const int32_t* trim_ids, float* q,
                 int64_t ldq, int32_t* tokens, int64_t ld_tokens, int32_t* dev_status);

// The second half of the drafter's top-k: z2 [B, K] = z log2(e) / T and the
// softmax partials part[G][B] of a projection.
int draft_topk_finish(cudaStream_t s, const float* z2, int B, int K, int k, const float2* part,
                      int G, const int32_t* trim_ids, int32_t* out_ids, float* out_logq,
                      int32_t* dev_status);

// vt_draft_step with two choices: status_reset = 1 zeroes *dev_status first
// (vt_draft_step), 0 adds this step's flags to it (later steps of a block);
// hidden_ready = 1 promises that no kernel still running in the stream writes
// the hidden states (they were complete before the previous kernel started),
// so the projection may stage them before its dependency wait.
int draft_step_impl(const uint16_t* hidden, int32_t B, int32_t H, const uint16_t* W_trim,
                    const int32_t* trim_ids, int32_t K, const float* uniforms, float temperature,
                    float* q, int64_t ldq, int32_t* tokens, int64_t ld_tokens,
                    int32_t* dev_status, void* workspace, size_t workspace_bytes, void* stream,
                    int status_reset, int hidden_ready);

// vt_draft_step_fp8 with the same choice of status_reset.
int draft_step_fp8_impl(const uint16_t* hidden, int32_t B, int32_t H, const uint8_t* W8,
                        int64_t ldw, const float* w_scale, const int32_t* trim_ids, int32_t K,
                        const float* uniforms, float temperature, float* q, int64_t ldq,
                        int32_t* tokens, int64_t ld_tokens, int32_t* dev_status, void* workspace,
                        size_t workspace_bytes, void* stream, int status_reset);

}  // namespace vt
