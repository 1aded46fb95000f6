// Launch parameters of the windowed attention and its gradient (window_attn.cu).
#pragma once

#include <cuda.h>

#include "duo_internal.cuh"

namespace duo {

struct HeadTensor {          // [batch][heads][tokens][128] by strides in elements
    void* data;
    int64_t b, h, t;
};

struct WindowAttnParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;
    CUtensorMap tm_out, tm_dq, tm_dk, tm_dv;   // of results: whole tiles are stored through them
    HeadTensor v, out, dout, dk, dv;
    float* stats;            // [B][hq][Tp]: minus each row's log2-sum-exp of the scaled scores (plus kWeightShift in
                             // fp16), -inf for no row
    uint8_t* low;            // [B][hq][Tp / 128][128 / 16][128][16]: what the rounding of the output took
                             // away, e5m2, 16 columns of 128 rows together
    float* delta;            // [B][hq][Tp]: minus the dot of each output row with its gradient
    float* peak;             // fp16: [B][hq][Tp / 64] largest |g_i|^2 of 64 rows, then [B][n_kv][Tp / 64] of |v_j|^2
    float* part;             // partial dK, dV of key tiles whose rows are shared out
    const int32_t* lengths;  // may be null
    int32_t* status;         // may be null
    int B, hq, n_kv, G, T, Tp, n_t;
    int S, W, full;          // S, W <= T; full: no window
    float scale, scale_log2;
    int pairs;               // forward: work items of two query tiles; those of one follow
    int n_long;              // key tiles of the first class (those that hold sinks), each in p_long pieces;
    int p_long, p_short;     // the others in p_short
    int items_kv;            // work items of the key tiles; those of the query tiles follow
    unsigned long long timeout_ns;
};

}  // namespace duo
