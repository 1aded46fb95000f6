// Launch parameters of the fused rotary append (append_rope.cu).
#pragma once

#include "rope.cuh"

namespace duo {

struct AppendRopeParams {
    duo_rows in[3];               // q, k, v
    uint16_t* q_out;              // may be null: keys and values only
    const int32_t* len_before;
    // a ragged batch (map_seq != null): one entry per row
    const int32_t* map_seq;
    const int32_t* map_pos;
    const int64_t* map_slot;      // may be null
    const int32_t* len_after;
    // a padded batch: n rows per sequence
    const int32_t* n_new;         // may be null
    int n;
    int64_t T;                    // rows in all
    uint16_t* kr;
    uint16_t* vr;
    uint16_t* ks;
    uint16_t* vs;
    int32_t* pos;
    int32_t* status;
    int64_t cap;
    int B, hq, n_kv, n_r, n_s, S, W;
    int fp8, int4;
    int page_tokens;              // > 0: paged retrieval caches
    int64_t num_pages;
    int max_pages;
    const int32_t* page_table;
    int per_thread;               // heads per thread
    int groups;                   // of heads, each a block per 8 tokens
    RopeTable table;
    int32_t rank[kMaxKvHeads];
    uint8_t is_r[kMaxKvHeads];
    float k_scale[kMaxKvHeads], v_scale[kMaxKvHeads];
};

cudaError_t launch_append_rope(const AppendRopeParams& p, int d, int num_sms, cudaStream_t s);

}  // namespace duo
