// Rotary positions and KV append of one layer in one launch, from the
// projections' token-major outputs.
//
// Queries: q_out = R(p) q.  Keys: the cache's row of position p receives
// R(p) k (and the codes of R(p) k / scale in quantised caches, rounded once
// from fp32), values as given.  R(p) is the rotation of rope.cuh; where a row
// goes, which rows the rings keep and what the position table holds are
// append.cu's rules.  Fused, a key is read once and written once (rotating
// first and appending then reads and writes it twice, with a second launch).
//
// Bound by HBM for long batches and by latency for a decode step.  A block
// owns 8 tokens and a group of heads: the cosines and sines of its tokens are
// worked out once, into shared memory.  A thread owns 16 elements of a token
// (8 pairs) and walks over heads of one kind after the other, two heads' loads
// in flight and four blocks per SM.  Keys and values of streaming heads that
// the ring will not hold are not read.
// Measured: 8 prompts of 8192 tokens, 32 query / 8 KV heads of 128, bf16:
// 238 us for 1.34 GB (86% of the copy rate); 6205 ragged tokens into FP8
// pages: 31 us for 122 MB, where address arithmetic, code conversion and the
// map's dependent loads count.  Angles per thread and group of heads instead
// of per block: 248 and 48 us; four heads in flight with three blocks per SM:
// 244 and 36 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "append_rope.cuh"

namespace duo {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;     // heads whose loads are in flight
constexpr int kTokens = 8;     // per block

// Eight fp32 values -> their E4M3 codes of value / scale (append.cu's rule).
template <bool DIVIDE>
__device__ __forceinline__ uint2 e4m3_codes8(const float* x, float scale) {
    uint16_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = DIVIDE ? __fdiv_rn(x[2 * i], scale) : x[2 * i];
        const float hi = DIVIDE ? __fdiv_rn(x[2 * i + 1], scale) : x[2 * i + 1];
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c[i]) : "f"(hi), "f"(lo));
    }
    return make_uint2(uint32_t(c[0]) | (uint32_t(c[1]) << 16), uint32_t(c[2]) | (uint32_t(c[3]) << 16));
}

// Eight fp32 values -> their packed INT4 codes (append.cu's rule).
__device__ __forceinline__ uint32_t int4_codes8(const float* x, float scale) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = __float2int_rn(__fdiv_rn(x[i], scale));
        out |= (uint32_t(min(max(c, -8), 7)) & 0xFu) << (4 * i);
    }
    return out;
}

// Codes of 16 values.  A scale of one (the usual one of FP8 caches) divides
// nothing: the same codes without sixteen divisions.
__device__ __forceinline__ void store_codes(const AppendRopeParams& p, uint8_t* base, int64_t row, int d, const RopeUnit& unit,
                                            float* x, float scale) {
    if (p.int4) {
        uint8_t* y = base + row * (d / 2);
        *reinterpret_cast<uint32_t*>(y + unit.e0 / 2) = int4_codes8(x, scale);
        *reinterpret_cast<uint32_t*>(y + unit.e1 / 2) = int4_codes8(x + 8, scale);
        return;
    }
    uint8_t* y = base + row * d;
    const bool one = scale == 1.f;
    *reinterpret_cast<uint2*>(y + unit.e0) = one ? e4m3_codes8<false>(x, 1.f) : e4m3_codes8<true>(x, scale);
    *reinterpret_cast<uint2*>(y + unit.e1) = one ? e4m3_codes8<false>(x + 8, 1.f) : e4m3_codes8<true>(x + 8, scale);
}

// Token t of the launch: its sequence, position and the sequence's tokens
// after the step; false: no token.  Reported by the thread with `lead`.
__device__ __forceinline__ bool token_of(const AppendRopeParams& p, int64_t t, bool lead, int& b, int& pos, int& t_new) {
    if (p.map_seq) {
        b = p.map_seq[t];
        pos = p.map_pos[t];
        if (b < 0) return false;
        if (b >= p.B || pos < 0) {
            if (lead) set_status(p.status, DUO_STATUS_BAD_LENGTH);
            return false;
        }
        t_new = -1;      // read where it is needed
        return true;
    }
    b = int(uint32_t(t) / uint32_t(p.n));       // rows are counted in 31 bits
    const int i = int(t) - b * p.n;
    const int nb = p.n_new ? p.n_new[b] : p.n;
    const int lb = p.len_before[b];
    if (lb < 0 || nb < 0 || nb > p.n || lb > 0x7fffffff - nb) {
        if (lead && i == 0) set_status(p.status, DUO_STATUS_BAD_LENGTH);
        return false;
    }
    if (i >= nb) return false;
    pos = lb + i;
    t_new = lb + nb;
    return true;
}

// Position of token t where it has one (any number where not).
__device__ __forceinline__ int position_of(const AppendRopeParams& p, int64_t t) {
    if (p.map_seq) return p.map_pos[t];
    const int b = int(uint32_t(t) / uint32_t(p.n));
    return int(uint32_t(p.len_before[b]) + uint32_t(int(t) - b * p.n));
}

// Where a token's keys and values go.
struct Place {
    int64_t row;    // first retrieval head's row of the token, -1: none
    int64_t ring;   // first streaming head's row, -1: the ring does not keep it
    int slot;       // of the ring
};

__device__ __forceinline__ Place place_of(const AppendRopeParams& p, int64_t t, bool lead, int b, int pos, int t_new) {
    Place pl;
    // the loads that depend on the sequence alone go out together
    const bool mapped = p.map_seq && p.map_slot;
    const int64_t slot = mapped && p.page_tokens > 0 ? p.map_slot[t] : -1;
    if (p.map_seq) t_new = p.len_after[b];
    const bool survives = pos < p.S || pos >= int64_t(t_new) - p.W;
    pl.slot = !survives ? -1 : (pos < p.S ? pos : p.S + (pos - p.S) % p.W);
    pl.ring = survives ? int64_t(b) * p.n_s * (p.S + p.W) + pl.slot : -1;
    pl.row = -1;
    if (p.n_r == 0) return pl;
    if (pos >= p.cap) {
        if (lead) set_status(p.status, DUO_STATUS_OVER_CAPACITY);
    } else if (p.page_tokens > 0) {
        int64_t page;
        int off = 0;
        if (mapped) {
            if (slot < 0) {
                page = -1;
            } else if (slot >> 32) {
                page = slot / p.page_tokens;
                off = int(slot - page * p.page_tokens);
            } else {
                page = uint32_t(slot) / uint32_t(p.page_tokens);
                off = int(uint32_t(slot) - uint32_t(page) * uint32_t(p.page_tokens));
            }
        } else {
            const int j = int(uint32_t(pos) / uint32_t(p.page_tokens));
            page = j < p.max_pages ? p.page_table[size_t(b) * p.max_pages + j] : -1;
            off = pos - j * p.page_tokens;
        }
        if (page < 0 || page >= p.num_pages) {
            if (lead) set_status(p.status, DUO_STATUS_NO_PAGE);
        } else {
            pl.row = page * p.n_r * p.page_tokens + off;
        }
    } else {
        pl.row = int64_t(b) * p.n_r * p.cap + pos;
    }
    return pl;
}

template <int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 4) append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    constexpr int UPH = D / 16;                          // units (16 elements) per head
    constexpr int kLanes = kThreads / (UPH * kTokens);   // heads of a token in work at a time
    constexpr int kPairs = D / 2;
    using Vec = Vec8<__nv_bfloat16>;
    __shared__ __align__(16) float turns[2][kTokens][kPairs];   // cosines, sines of the block's tokens
    // as in append.cu: a programmatic dependent that lets a decode start once
    // everything before this launch has completed
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int tiles = int((p.T + kTokens - 1) / kTokens), SW = p.S + p.W;
    const int group = int(blockIdx.x) / tiles;
    if (group >= p.groups) {
        // position-table reset for sequences that start from empty: the slots
        // that this call does not fill
        const int64_t r = (int64_t(blockIdx.x) - int64_t(tiles) * p.groups) * kThreads + threadIdx.x;
        if (r >= int64_t(p.B) * SW) return;
        const int b = int(r / SW), slot = int(r % SW);
        if (p.len_before[b] != 0) return;
        const int nb = p.map_seq ? p.len_after[b] : (p.n_new ? p.n_new[b] : p.n);
        if (slot >= nb) p.pos[r] = -1;
        return;
    }
    const int64_t t0 = int64_t(int(blockIdx.x) - group * tiles) * kTokens;
    const int u = threadIdx.x % UPH, token = threadIdx.x / UPH % kTokens, lane = threadIdx.x / (UPH * kTokens);
    const int64_t t = t0 + token;
    const RopeUnit unit = rope_unit(p.table, u);
    // the heads in order: keys, values, queries
    const int heads = 2 * p.n_kv + (p.q_out ? p.hq : 0);
    const int first = group * p.per_thread * kLanes + lane, last = min((group + 1) * p.per_thread * kLanes, heads);
    const int64_t head_rows = p.page_tokens > 0 ? p.page_tokens : p.cap;
    // one thread per token reports it and writes the position table
    const bool lead = group == 0 && lane == 0 && u == 0;
    int b = 0, pos = 0, t_new = 0;
    const bool live = t < p.T && token_of(p, t, lead, b, pos, t_new);
    Place pl{-1, -1, -1};
    if (live && first < 2 * p.n_kv) {
        pl = place_of(p, t, lead, b, pos, t_new);
        if (lead && pl.slot >= 0) p.pos[size_t(b) * SW + pl.slot] = pos;
        // a map whose lengths have advanced in place (len_before is len_after) still says by its token 0 that
        // the sequence starts from empty
        if (lead && pos == 0 && p.map_seq && p.len_before[b] != 0)
            for (int r = max(p.len_after[b], 1); r < SW; ++r) p.pos[size_t(b) * SW + r] = -1;      // whatever a map says
    }

    for (int x = threadIdx.x; x < kTokens * kPairs; x += kThreads) {
        const int64_t at = t0 + x / kPairs;
        const int pair = x % kPairs;
        if (at >= p.T || pair >= 8 * p.table.rot_units) continue;
        rope_angle(p.table, pair, position_of(p, at), 1.f, turns[0][x / kPairs][pair], turns[1][x / kPairs][pair]);
    }
    __syncthreads();
    if (!live) return;
    float c[8], s[8];
    if (unit.rotates) {
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            *reinterpret_cast<float4*>(c + k) = *reinterpret_cast<const float4*>(&turns[0][token][8 * u + k]);
            *reinterpret_cast<float4*>(s + k) = *reinterpret_cast<const float4*>(&turns[1][token][8 * u + k]);
        }
    }
    // this thread's heads of one kind: keys (1), values (2), queries (0)
    const auto walk = [&](auto kind, int begin, int end) {
        constexpr int w = decltype(kind)::value;
        const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(p.in[w].data) + t * p.in[w].token_stride;
        const int from = first + max(0, (begin - first + kLanes - 1) / kLanes) * kLanes, to = min(end, last);
        for (int h = from; h < to; h += kUnroll * kLanes) {
            Vec v[kUnroll][2];
            int row[kUnroll];          // cache row of the head (a cache on one GPU has fewer than 2^31), -1: not stored
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int g = h + k * kLanes - begin;
                row[k] = -1;
                if (h + k * kLanes >= to) continue;
                if (w == 0)
                    row[k] = 0;
                else if (p.is_r[g])
                    row[k] = pl.row < 0 ? -1 : int(pl.row + p.rank[g] * head_rows);
                else
                    row[k] = pl.ring < 0 ? -1 : int(pl.ring + int64_t(p.rank[g]) * SW);
                if (row[k] < 0) continue;
                v[k][0].load(x + g * p.in[w].head_stride + unit.e0);
                v[k][1].load(x + g * p.in[w].head_stride + unit.e1);
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                if (row[k] < 0) continue;
                const int g = h + k * kLanes - begin;
                uint16_t* const y = w == 0 ? p.q_out + (t * p.hq + g) * D
                                           : (p.is_r[g] ? (w == 1 ? p.kr : p.vr) : (w == 1 ? p.ks : p.vs));
                const bool turn = w != 2 && unit.rotates;
                if (w != 0 && p.fp8) {
                    float e[16];
                    widen(v[k][0], e);
                    widen(v[k][1], e + 8);
                    if (turn) rope_rotate<HALF>(e, c, s);
                    store_codes(p, reinterpret_cast<uint8_t*>(y), row[k], D, unit, e, w == 1 ? p.k_scale[g] : p.v_scale[g]);
                    continue;
                }
                if (turn) {
                    float e[16];
                    widen(v[k][0], e);
                    widen(v[k][1], e + 8);
                    rope_rotate<HALF>(e, c, s);
                    narrow(v[k][0], e);
                    narrow(v[k][1], e + 8);
                }
                __nv_bfloat16* const z = reinterpret_cast<__nv_bfloat16*>(y) + int64_t(row[k]) * D;
                v[k][0].store(z + unit.e0);
                v[k][1].store(z + unit.e1);
            }
        }
    };
    walk(std::integral_constant<int, 1>{}, 0, p.n_kv);
    walk(std::integral_constant<int, 2>{}, p.n_kv, 2 * p.n_kv);
    walk(std::integral_constant<int, 0>{}, 2 * p.n_kv, heads);
}

}  // namespace

cudaError_t launch_append_rope(const AppendRopeParams& p0, int d, int num_sms, cudaStream_t s) {
    AppendRopeParams p = p0;
    const int64_t tiles = (p.T + kTokens - 1) / kTokens;
    const int heads = 2 * p.n_kv + (p.q_out ? p.hq : 0), lanes = kThreads / (d / 16 * kTokens);
    // heads per thread: as many as leave the GPU eight blocks per SM
    int n = 1;
    while (n < 16 && n * lanes < heads && tiles * ((heads + 2 * n * lanes - 1) / (2 * n * lanes)) >= int64_t(num_sms) * 8)
        n *= 2;
    p.per_thread = n;
    p.groups = (heads + n * lanes - 1) / (n * lanes);
    const int64_t reset = (int64_t(p.B) * (p.S + p.W) + kThreads - 1) / kThreads;
    const int64_t blocks = tiles * p.groups + reset;
    if (blocks > 0x7fffffff || p.T > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (d == 128)
        e = p.table.half ? cudaLaunchKernelEx(&cfg, append_rope_kernel<128, true>, p)
                         : cudaLaunchKernelEx(&cfg, append_rope_kernel<128, false>, p);
    else
        e = p.table.half ? cudaLaunchKernelEx(&cfg, append_rope_kernel<64, true>, p)
                         : cudaLaunchKernelEx(&cfg, append_rope_kernel<64, false>, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace duo
