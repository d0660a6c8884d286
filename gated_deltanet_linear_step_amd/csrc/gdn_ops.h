// gdn_ops.h -- kernel parameter blocks and launchers of the operators beside the delta rule: decayed
// linear attention, RMS norm with residual and 8-bit output, int8 product. They have a header of their
// own so that the sources that the delta-rule kernels' counters were taken at do not change with them.
#pragma once

#include "gdn_kernels.h"

namespace gdn {

enum : uint32_t { F_HEAD_DECAY = 16u };  // beside gdn_device.h's flags

// Decayed linear attention (gdn_linattn.hip). Decode: cu is NULL, sequence b has the
// T rows from b * T on. Prefill: sequence b has the rows [cu[b], cu[b + 1]).
struct LinattnParams {
    ActInputs in;  // q, k, v and g or decay_param
    HeadCfg hc;
    float *state;
    const int32_t *slots;  // decode only; NULL: slot b
    int num_slots;
    void *out;
    int out_dt;
    int N, T;  // sequences; tokens per sequence (decode) or the longest sequence (prefill)
    int total;
    const int32_t *cu;
    void *workspace;
    // prefill: sequences longer than seg_tokens are split into segments, the first of
    // seg_first_tokens, the others of seg_tokens; how many segments come first of a
    // sequence, and between first and last; states after (and summed log decays of)
    // each segment but a sequence's last, [slot][Hv]
    int seg_tokens, seg_first_tokens, segs_first, segs_between;
    float *seg_state, *seg_decay;
};
bool linattn_supported(int dk, int dv);
bool linattn_grid_fits(int N, int Hv, int dk, int dv);
hipError_t launch_linattn_decode(const LinattnParams &p, hipStream_t s);
size_t linattn_prefill_workspace_bytes(int Hk, int Hv, int dk, int dv, int N, int64_t total_tokens);
// cu: the offsets on the host
hipError_t launch_linattn_prefill(const LinattnParams &p, const int32_t *cu, hipStream_t s);
// The chunk kernels per activation dtype (gdn_linattn_chunk.h): `second` the later segments
hipError_t launch_linattn_chunk_bf16(const LinattnParams &p, int64_t segments, bool second, hipStream_t s);
hipError_t launch_linattn_chunk_f16(const LinattnParams &p, int64_t segments, bool second, hipStream_t s);
hipError_t launch_linattn_chunk_f32(const LinattnParams &p, int64_t segments, bool second, hipStream_t s);

// RMS norm with residual and 8-bit output (gdn_norm.hip). Strides in elements.
struct NormParams {
    int rows, hidden, dt, out_dt;
    const void *x, *residual;  // residual may be NULL
    int64_t x_stride, residual_stride;
    void *residual_out;  // NULL: not stored
    int64_t residual_out_stride;
    const float *weight;
    float eps;
    void *out;  // NULL: not stored
    int64_t out_stride;
    int8_t *out_q;  // NULL: not stored; with it out_scale [rows]
    int64_t out_q_stride;
    float *out_scale;
};
hipError_t launch_norm(const NormParams &p, hipStream_t s);

// Product of 8-bit integers with row scales (gdn_matmul.hip).
struct MatmulParams {
    int M, N, K, out_dt;
    const int8_t *a, *w;
    int64_t a_stride, w_stride, out_stride;
    const float *a_scale, *w_scale;
    void *out;
};
// The kernel that launch_matmul takes, M, N >= 1.
struct MatmulPlan {
    int workgroups, threads;
};
MatmulPlan matmul_plan(int M, int N);
hipError_t launch_matmul(const MatmulParams &p, hipStream_t s);

}  // namespace gdn
