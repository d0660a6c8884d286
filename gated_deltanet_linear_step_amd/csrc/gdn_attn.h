// gdn_attn.h -- kernel parameter blocks and launchers of the softmax attention layer's operators: rotary positions,
// attention over prompts and in decode steps, and the pages of their cache.
#pragma once

#include "gdn_kernels.h"

namespace gdn {

constexpr int kCus = 256;  // of an MI355X

// Rotary positions (gdn_rope.hip). Strides in elements.
struct RopeParams {
    int tokens, Hq, Hkv, D, rot, layout, dt;
    float magnitude;
    const int32_t *positions;
    const double *w;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    void *q_out, *k_out, *k_pages, *v_pages;  // NULL: not stored
    int64_t q_out_stride, k_out_stride, page_stride;
    int64_t num_slots;
    int page_shift;
    const int32_t *slots;
};
hipError_t launch_rope(const RopeParams &p, hipStream_t s);

// Keys and values of an attention call: packed rows, or pools of pages [Hkv][page size][D].
struct KvSource {
    const void *k, *v;
    int64_t k_stride, v_stride;  // elements from row to row, or from page to page
    int page_shift, num_pages;   // log2 of the page size; page_shift < 0: packed rows
    const int32_t *table;
    int64_t table_stride;
};

// What the attention kernels share. Partial results go to `part` where a query's keys are
// split: [token][head][slot] rows of D f32, with pairs in `stat`: the score,
// not scaled, that the weights are relative to, and their sum.
struct AttnParams {
    int Hq, Hkv, D, dt;
    float scale;
    const void *q;
    int64_t q_stride;
    void *out;
    int64_t out_stride;
    float *lse;
    KvSource kv;
    float *part;
    float2 *stat;
    int slots;  // partial results of a query; 0: the outputs are written at once
};

// Blocks of queries against runs of keys (gdn_attn_prefill.h). Sequences: packed and causal by cu_q and cu_k (device);
// or, cu_q NULL, N of T queries each, causal against lens[s] keys of table row s (lens on the device, at most max_keys
// count), or, lens NULL too, N = 1 against max_keys keys that every query sees.
struct AttnPrefillParams {
    AttnParams a;
    int N, T, total;  // sequences, queries of each without cu_q, queries in all
    const int32_t *cu_q, *cu_k, *lens;
    int max_keys;
    int splits, split_tiles, first_slot;  // runs of keys of a block of queries, their tiles, and the slot of the first
    bool whole;              // rows whose keys are one run are written at once
    int blocks;              // of rows, for each key head (this and the next are set by the launcher)
    bool one_round;          // all workgroups are on the device at once
};
bool attn_supported(int D);
// Runs of keys that a call is split into, and their length: by the offsets, or (cu_q NULL) one sequence against `keys` keys;
// and the most that any offsets of as many queries give
void attn_prefill_splits(int Hq, int Hkv, int D, int N, int64_t total, const int32_t *cu_q, const int32_t *cu_k, int keys, int *splits,
                         int *split_tiles);
int attn_prefill_most_splits(int Hq, int Hkv, int64_t total);
// Workgroups for each run of keys
int64_t attn_prefill_blocks(int Hq, int Hkv, int N, int64_t total, bool packed);
hipError_t launch_attn_prefill(const AttnPrefillParams &p, hipStream_t s);
hipError_t launch_attn_prefill_bf16(const AttnPrefillParams &p, unsigned grid, hipStream_t s);
hipError_t launch_attn_prefill_f16(const AttnPrefillParams &p, unsigned grid, hipStream_t s);

// Keys of one run: an output is an f32 sum that 16 keys are added to at a time, and drifts where all weights and values are alike, as each
// addition is then rounded the same way. Measured with five such weights: at most 2^-8 (bf16's half step) at 2^20 and 2^-7 at 2^22 keys, 2^-5.4
// at 2^24.
constexpr int kMostKeys = 1 << 21;

// Keys that a workgroup of the decode kernel takes at a time, and the most that a run has of that
constexpr int kDecodeRound = 128, kDecodeRounds = 32;

// A few queries of each sequence against its own pages (gdn_attn_decode.h).
struct AttnDecodeParams {
    AttnParams a;
    int B, T;
    const int32_t *lens;
    int max_len;
    int splits, split_keys, first_slot;  // runs of split_keys keys each (of split_keys tiles where blocks of rows take it)
};
int64_t attn_decode_blocks(int Hq, int Hkv, int D, int B, int T);  // workgroups for each run of keys
void attn_decode_splits(int Hq, int Hkv, int D, int B, int T, int max_len, int *splits, int *split_keys);
hipError_t launch_attn_decode(const AttnDecodeParams &p, hipStream_t s);
hipError_t launch_attn_decode_bf16(const AttnDecodeParams &p, unsigned grid, hipStream_t s);
hipError_t launch_attn_decode_f16(const AttnDecodeParams &p, unsigned grid, hipStream_t s);

// Joins the partial results of `rows` rows (queries times heads) into outputs; its workgroups.
int64_t attn_join_blocks(int D, int slots, int64_t rows);
hipError_t launch_attn_join(const AttnParams &p, int64_t rows, hipStream_t s);

// Pages of a cache (gdn_pages.hip).
struct PageParams {
    int32_t *table;
    int64_t table_stride;
    int rows, width;
    int32_t *refs;
    int num_pages, page_size;
    unsigned char *data;
    int num_planes;
    int64_t plane_stride, page_stride, page_bytes;
    int n;
    const int32_t *row, *src, *len;  // requests: rows (fork: dst), fork's sources, lengths or entries to keep
    int32_t *status;
    int32_t *page_map, *used;
    int32_t *workspace;
};
constexpr int kPageRequests = 1024;
size_t pages_workspace_bytes(int num_pages);
hipError_t launch_pages_free(const PageParams &p, hipStream_t s);
hipError_t launch_pages_reserve(const PageParams &p, hipStream_t s);
hipError_t launch_pages_fork(const PageParams &p, hipStream_t s);
hipError_t launch_pages_compact(const PageParams &p, hipStream_t s);

}  // namespace gdn
