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
// Bound by HBM for long batches and by latency for a decode step.  A thread
// owns one token's 16 elements of a head and walks over heads_per_thread of
// the batch's query, key and value heads (in that order), four heads' loads
// in flight; the angles of a token are computed once per thread.  Keys and
// values of streaming heads that the ring will not hold are not read.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "append_rope.cuh"

namespace duo {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// Eight fp32 values -> their E4M3 codes of value / scale (append.cu's rule).
__device__ __forceinline__ uint2 e4m3_codes8(const float* x, float scale) {
    uint16_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __fdiv_rn(x[2 * i], scale), hi = __fdiv_rn(x[2 * i + 1], scale);
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

// Where one token's rows go.
struct Place {
    int b;          // sequence
    int64_t row;    // first retrieval head's row of the token, -1: none
    int slot;       // ring slot, -1: the ring does not keep it
};

// Token t of the launch: its sequence, position and rows; false: no token.
// Flagged once per token (by the thread with `lead`).
template <int D>
__device__ __forceinline__ bool place_of(const AppendRopeParams& p, int64_t t, bool lead, int& pos, Place& pl) {
    int64_t slot = -1;
    int t_new;                    // the sequence's tokens after this step
    if (p.map_seq) {
        pl.b = p.map_seq[t];
        pos = p.map_pos[t];
        slot = p.map_slot ? p.map_slot[t] : -1;
        if (pl.b < 0) return false;
        if (pl.b >= p.B || pos < 0) {
            if (lead) set_status(p.status, DUO_STATUS_BAD_LENGTH);
            return false;
        }
        t_new = p.len_after[pl.b];
    } else {
        pl.b = int(t / p.n);
        const int i = int(t - int64_t(pl.b) * p.n);
        const int nb = p.n_new ? p.n_new[pl.b] : p.n;
        const int lb = p.len_before[pl.b];
        if (lb < 0 || nb < 0 || nb > p.n || lb > 0x7fffffff - nb) {
            if (lead && i == 0) set_status(p.status, DUO_STATUS_BAD_LENGTH);
            return false;
        }
        if (i >= nb) return false;
        pos = lb + i;
        t_new = lb + nb;
    }
    const bool survives = pos < p.S || pos >= int64_t(t_new) - p.W;
    pl.slot = !survives ? -1 : (pos < p.S ? pos : p.S + (pos - p.S) % p.W);
    pl.row = -1;
    if (p.n_r > 0) {
        if (pos >= p.cap) {
            if (lead) set_status(p.status, DUO_STATUS_OVER_CAPACITY);
        } else if (p.page_tokens > 0) {
            int64_t page;
            int off;
            if (p.map_seq && p.map_slot) {
                if (slot < 0 || uint64_t(slot) >> 32) {
                    page = slot < 0 ? -1 : slot / p.page_tokens;
                } else {
                    page = uint32_t(slot) / uint32_t(p.page_tokens);
                }
                off = page < 0 ? 0 : int(slot - page * p.page_tokens);
            } else {
                const int j = pos / p.page_tokens;
                page = j < p.max_pages ? p.page_table[size_t(pl.b) * p.max_pages + j] : -1;
                off = pos - j * p.page_tokens;
            }
            if (page < 0 || page >= p.num_pages) {
                if (lead) set_status(p.status, DUO_STATUS_NO_PAGE);
            } else {
                pl.row = page * p.n_r * p.page_tokens + off;
            }
        } else {
            pl.row = int64_t(pl.b) * p.n_r * p.cap + pos;
        }
    }
    return true;
}

template <int D, bool HALF>
__global__ void __launch_bounds__(kThreads) append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    constexpr int UPH = D / 16;                    // units (16 elements) per head
    constexpr int kTokens = kThreads / UPH;        // tokens per block
    using Vec = Vec8<__nv_bfloat16>;
    // as in append.cu: a programmatic dependent that lets a decode start once
    // everything before this launch has completed
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t token_blocks = (p.T + kTokens - 1) / kTokens;
    const int groups = (p.hq + 2 * p.n_kv + p.heads_per_thread - 1) / p.heads_per_thread;
    const int SW = p.S + p.W;
    if (blockIdx.x >= token_blocks * groups) {
        // position-table reset for sequences that start from empty: the slots
        // that this call does not fill
        const int64_t r = (int64_t(blockIdx.x) - token_blocks * groups) * kThreads + threadIdx.x;
        if (r >= int64_t(p.B) * SW) return;
        const int b = int(r / SW), slot = int(r % SW);
        if (p.len_before[b] != 0) return;
        const int nb = p.map_seq ? p.len_after[b] : (p.n_new ? p.n_new[b] : p.n);
        if (slot >= nb) p.pos[r] = -1;
        return;
    }
    const int64_t group = blockIdx.x / token_blocks;
    const int64_t t = (blockIdx.x - group * token_blocks) * kTokens + threadIdx.x / UPH;
    const int u = threadIdx.x % UPH;
    if (t >= p.T) return;
    const int h0 = int(group) * p.heads_per_thread;
    const int h1 = min(h0 + p.heads_per_thread, p.hq + 2 * p.n_kv);
    int pos;
    Place pl;
    // one thread per token reports it and writes the position table: unit 0
    // of the group that holds KV head 0's keys
    const bool lead = u == 0 && h0 <= p.hq && p.hq < h1;
    if (!place_of<D>(p, t, lead, pos, pl)) return;
    if (lead && pl.slot >= 0) p.pos[size_t(pl.b) * SW + pl.slot] = pos;

    const RopeUnit unit = rope_unit(p.table, u);
    float c[8], s[8];
    if (unit.rotates && h0 < p.hq + p.n_kv) rope_angles(p.table, u, pos, 1.f, c, s);

    for (int h = h0; h < h1; h += kUnroll) {
        Vec v[kUnroll][2];
        int64_t row[kUnroll];                      // cache row of the head, -1: not stored
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (h + k >= h1) break;
            const int hh = h + k;
            const int g = hh < p.hq ? -1 : (hh - p.hq) % p.n_kv;     // KV head of keys and values
            const int w = hh < p.hq ? 0 : (hh < p.hq + p.n_kv ? 1 : 2);
            const uint16_t* x = p.in[w].data + t * p.in[w].token_stride + (w == 0 ? hh : g) * p.in[w].head_stride;
            row[k] = 0;
            if (w > 0) {
                if (p.is_r[g])
                    row[k] = pl.row < 0 ? -1
                                        : pl.row + int64_t(p.rank[g]) * (p.page_tokens > 0 ? p.page_tokens : p.cap);
                else
                    row[k] = pl.slot < 0 ? -1 : (int64_t(pl.b) * p.n_s + p.rank[g]) * SW + pl.slot;
            } else if (!p.q_out) {
                row[k] = -1;
            }
            if (row[k] >= 0) {
                v[k][0].load(reinterpret_cast<const __nv_bfloat16*>(x + unit.e0));
                v[k][1].load(reinterpret_cast<const __nv_bfloat16*>(x + unit.e1));
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (h + k >= h1) break;
            if (row[k] < 0) continue;
            const int hh = h + k;
            const int w = hh < p.hq ? 0 : (hh < p.hq + p.n_kv ? 1 : 2);
            const bool turn = unit.rotates && w < 2;
            if (w == 0 || !p.fp8) {
                if (turn) {
                    float x[16];
                    widen(v[k][0], x);
                    widen(v[k][1], x + 8);
                    rope_rotate<HALF>(x, c, s);
                    narrow(v[k][0], x);
                    narrow(v[k][1], x + 8);
                }
                uint16_t* y;
                if (w == 0) {
                    y = p.q_out + (t * p.hq + hh) * D;
                } else {
                    const int g = (hh - p.hq) % p.n_kv;
                    y = (p.is_r[g] ? (w == 1 ? p.kr : p.vr) : (w == 1 ? p.ks : p.vs)) + row[k] * D;
                }
                v[k][0].store(reinterpret_cast<__nv_bfloat16*>(y + unit.e0));
                v[k][1].store(reinterpret_cast<__nv_bfloat16*>(y + unit.e1));
            } else {
                float x[16];
                widen(v[k][0], x);
                widen(v[k][1], x + 8);
                if (turn) rope_rotate<HALF>(x, c, s);
                const int g = (hh - p.hq) % p.n_kv;
                const float scale = w == 1 ? p.k_scale[g] : p.v_scale[g];
                uint8_t* y = reinterpret_cast<uint8_t*>(p.is_r[g] ? (w == 1 ? p.kr : p.vr) : (w == 1 ? p.ks : p.vs));
                if (p.int4) {
                    y += row[k] * (D / 2);
                    *reinterpret_cast<uint32_t*>(y + unit.e0 / 2) = int4_codes8(x, scale);
                    *reinterpret_cast<uint32_t*>(y + unit.e1 / 2) = int4_codes8(x + 8, scale);
                } else {
                    y += row[k] * D;
                    *reinterpret_cast<uint2*>(y + unit.e0) = e4m3_codes8(x, scale);
                    *reinterpret_cast<uint2*>(y + unit.e1) = e4m3_codes8(x + 8, scale);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_append_rope(const AppendRopeParams& p0, int d, int num_sms, cudaStream_t s) {
    AppendRopeParams p = p0;
    const int heads = p.hq + 2 * p.n_kv;
    const int tokens = kThreads / (d / 16);
    const int64_t token_blocks = (p.T + tokens - 1) / tokens;
    // heads per thread: as many as leave a full wave of threads
    int hpt = 1;
    while (hpt < 8 && hpt < heads && token_blocks * ((heads + 2 * hpt - 1) / (2 * hpt)) >= int64_t(num_sms) * 8) hpt *= 2;
    p.heads_per_thread = hpt;
    const int64_t reset = (int64_t(p.B) * (p.S + p.W) + kThreads - 1) / kThreads;
    const int64_t blocks = token_blocks * ((heads + hpt - 1) / hpt) + reset;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
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
