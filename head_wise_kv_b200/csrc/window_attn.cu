// Causal attention with a sliding window and sinks, forward and backward, on
// the 5th-generation tensor cores (tcgen05), for training the two branches of
// the gated forward: row i of a sequence sees the keys
//   j <= i with (j < S or j > i - W),          or every j <= i (full branch).
//
// Forward:   s_ij = scale q_i.k_j,  p_ij = exp(s_ij) / sum_j exp(s_ij),  o_i = sum_j p_ij v_j.
// Backward, with g_i the gradient of o_i and D_i = o_i.g_i:
//   dv_j = sum_i p_ij g_i
//   ds_ij = p_ij (g_i.v_j - D_i)
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i
// (sums over the query heads that share a key head for dk and dv).
//
// Every tile is 128 rows x 128 keys x 128 dims.  p_ij comes back in the
// backward from the scores and one saved number per row (minus its
// log2-sum-exp), so nothing of size T^2 is kept.  Only tiles that hold a
// visible pair are visited.
//
// Precision: products take bf16 (fp16) operands and sum in fp32; scores,
// softmax statistics, sums and D are fp32
// (D from the result before its rounding, as far as 8 more bits hold it).  p_ij and ds_ij are rounded to the
// inputs' type because a tcgen05 product needs both operands in one 16-bit
// type: at most 2^-8 (bf16) or 2^-11 (fp16) of each element, averaged over the
// sums, the size of the rounding of the result.
//
// fp16 is that exact from 2^-14 to 65504 only, and weights of long rows and
// gradients lie anywhere.  There they are held times powers of two, which the
// results take out again: the forward's weights 2^7 (below 2^15, the running
// maximum may lag by 2^8), the backward's 2^14 (at most 1 before), ds a factor
// f of each (sequence, key head).  |g_i.v_j - D_i| p_ij =
// p (1 - p) |g_i.(v_j - the other keys' mean)| <= M / 2 with M = max |g_i| max |v_j|, so f
// is the power of two that brings M into 2^14 .. 2^15.  What then falls below
// 2^-14 is off by at most 2^-32 of the row's largest weight, 2^-39, and 2^-39 M.
//
// No atomics: the backward visits each tile pair twice, once for the key
// tile's owner (dK, dV) and once for the query tile's (dQ).  That is 7
// products per pair instead of 5, and every sum is taken in one fixed order.
//
// Measured, 32 query / 8 KV heads, 4096 tokens, bf16, every key: forward 153 us
// (137 GFLOP, 900 TFLOP/s), backward 454 us (344 GFLOP in five products, 760
// TFLOP/s; 1060 counting the seven that are done), at the board's power limit.
// 16 / 4 heads, 8192 tokens, window 1024, 64 sinks: 113 and 294 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "duo_internal.cuh"
#include "tcgen05.cuh"
#include "window_attn.cuh"

namespace duo {

namespace {

constexpr int kTile = 128;                    // rows, keys and dims of a tile
constexpr uint32_t kSlab = 128 * 128;         // bytes: 128 rows x 64 16-bit elements
constexpr uint32_t kTileBytes = 2 * kSlab;
constexpr float kNegBig = -1.0e30f;
constexpr float kRescaleThreshold = 8.0f;     // log2 units

template <typename T>
struct Elem;
constexpr int kWeightShift = 14;              // fp16: log2 of the factor of the backward's weights
template <>
struct Elem<__nv_bfloat16> {
    static constexpr bool bf16 = true;
    static constexpr float kForwardShift = 0.f, kStatsShift = 0.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 wide(uint32_t x) { return bf2_to_f2(x); }
};
template <>
struct Elem<__half> {
    static constexpr bool bf16 = false;
    static constexpr float kForwardShift = 7.f, kStatsShift = float(kWeightShift);   // log2 of the weights' factors
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 wide(uint32_t x) {
        return __half22float2(*reinterpret_cast<const __half2*>(&x));
    }
};

// ------------------------------------------------------------------ small helpers
__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {      // bits lo .. hi of 0 .. 31
    lo = max(lo, 0);
    hi = min(hi, 31);
    if (lo > hi) return 0u;
    const uint32_t upto = hi == 31 ? 0xffffffffu : ((2u << hi) - 1u);
    return upto & ~((1u << lo) - 1u);
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    unsigned long long av = *reinterpret_cast<unsigned long long*>(&a);
    unsigned long long bv = *reinterpret_cast<unsigned long long*>(&b);
    unsigned long long dv;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(dv) : "l"(av), "l"(bv));
    return *reinterpret_cast<float2*>(&dv);
}

// Bounded waits of one CTA: the first that runs out marks the CTA, and every
// role leaves at its next wait.  A warp waits with all its lanes: a wait by
// one lane and the reconvergence behind it take about 500 cycles even where
// the phase has completed, one by all lanes about 120 (backward of 4096
// tokens x 32 heads: 587 us with the former in every role).
struct Waiter {
    int32_t* status;
    unsigned long long limit;
    volatile int* abort_flag;

    __device__ __forceinline__ bool gave_up(unsigned long long t0) const {
        if (*abort_flag) return true;
        if (global_ns() - t0 <= limit) return false;
        if (status) set_status(status, DUO_STATUS_WAIT_TIMEOUT);
        *abort_flag = 1;
        return true;
    }
    // one thread, alone in its warp's path
    __device__ __forceinline__ bool thread(uint32_t bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return true;
        const unsigned long long t0 = global_ns();
        while (!mbar_try_wait(bar, parity))
            if (gave_up(t0)) return false;
        return true;
    }
    // a converged warp
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const unsigned long long t0 = global_ns();
        while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
            if (__any_sync(0xffffffffu, gave_up(t0))) return false;
        return true;
    }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int t, int h, int b,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(t), "r"(h), "r"(b), "r"(bar)
        : "memory");
}

// 128 tokens x 128 dims: two 64-dim slabs, 128-byte swizzled.  Tokens behind
// the tensor's last one arrive as zeros.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int t, int h, int b, uint32_t bar) {
    tma_load_4d(dst, map, 0, t, h, b, bar);
    tma_load_4d(dst + kSlab, map, 64, t, h, b, bar);
}

// 128 consecutive floats.
__device__ __forceinline__ void bulk_row(uint32_t dst, const float* src, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(uint32_t(kTile * 4)), "r"(bar)
        : "memory");
}

// Rows [first, 128) of a tile become zeros, by `warps` warps of which this is
// number w: a product must not meet what lies behind a sequence's last token,
// since 0 x NaN is NaN.  The products must wait for these warps.
__device__ __forceinline__ void zero_rows(uint32_t tile, int first, int w, int warps) {
    for (int off = first * 128 + (w * 32 + int(threadIdx.x & 31)) * 16; off < int(kSlab); off += warps * 32 * 16) {
        st_shared_v4(tile + off, make_uint4(0, 0, 0, 0));
        st_shared_v4(tile + kSlab + off, make_uint4(0, 0, 0, 0));
    }
    fence_proxy_async_smem();
}

// D (+)= A B^T: both tiles with their 128 dims along K.
__device__ __forceinline__ void mma_dims(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t off = (k >> 2) * kSlab + (k & 3) * 32;
        umma_f16(d, smem_desc(a + off, 16, 1024), smem_desc(b + off, 16, 1024), idesc, k > 0);
    }
}

// D (+)= A B: A in TMEM (16-bit pairs, K steps of 8 columns from column a),
// B a tile with its 128 rows along K; K steps k0 .. k1 - 1.
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, int k0, int k1, uint32_t b, uint32_t idesc, bool add) {
#pragma unroll
    for (int k = k0; k < k1; ++k)
        umma_f16_ts(d, a + k * 8, smem_desc(b + k * 2048, kSlab, 1024), idesc, (add || k > k0) ? 1u : 0u);
}

__device__ __forceinline__ int length_of(const WindowAttnParams& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// The key tiles that query tile qt visits, in order: sinks first.
struct KeyTiles {
    int lo, sinks, n;
    __device__ __forceinline__ KeyTiles(const WindowAttnParams& p, int qt) {
        lo = p.full ? 0 : max(0, qt * kTile - p.W + 1) / kTile;
        sinks = p.full ? 0 : min((p.S + kTile - 1) / kTile, lo);
        n = sinks + qt - lo + 1;
    }
    __device__ __forceinline__ int at(int j) const { return j < sinks ? j : lo + j - sinks; }
};

// Whether every row of query tile qt sees every key of key tile kt < qt.
__device__ __forceinline__ bool whole(const WindowAttnParams& p, int qt, int kt) {
    return p.full || kt * kTile + kTile - 1 < p.S || kt * kTile > qt * kTile + kTile - 1 - p.W;
}

// Keys first .. first + 31 that row i sees.
__device__ __forceinline__ uint32_t row_sees(const WindowAttnParams& p, int i, int first) {
    const uint32_t causal = range_bits(0, i - first);
    if (p.full) return causal;
    return causal & (range_bits(i - p.W + 1 - first, 31) | range_bits(0, p.S - 1 - first));
}

// Eight results of a row -> 16 bytes in the tensor's type.
template <typename T>
__device__ __forceinline__ uint4 pack8(const uint32_t* u, float f) {
    uint32_t w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
        w[x] = Elem<T>::pack(__uint_as_float(u[2 * x]) * f, __uint_as_float(u[2 * x + 1]) * f);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ T* row_at(const HeadTensor& x, int b, int h, int t) {
    return static_cast<T*>(x.data) + b * x.b + h * x.h + t * x.t;
}

// ------------------------------------------------------------------ shared memory
// Both kernels use seven tiles and a little more, of the 227 KB that a CTA
// may have.  The dynamic region starts at a multiple of 1024 bytes (there is
// no static one before it); the kernels leave with a status bit if not.
constexpr int kThreads = 352;                        // warps 0-7 elementwise, 8 TMA, 9 and 10 products
constexpr uint32_t kStatsAt = 7 * kTileBytes;        // [3][128] minus D, [2][128] row statistics
constexpr uint32_t kBarsAt = kStatsAt + 5 * kTile * 4;
constexpr int kRing3 = 3, kRing2 = 2;                // stages of the two rings of tiles

struct Bars {
    uint64_t once, full3[kRing3], empty3[kRing3], full2[kRing2], empty2[kRing2];
    uint64_t s_full[2], s_read, dp_full, dp_read, p_half[2], p_full[2], ds_full[2], trimmed, done[2], fin;
    uint32_t tmem;
    int abort_flag;
    float peak[2][8];
};
constexpr uint32_t kSmem = kBarsAt + sizeof(Bars);
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");

__device__ __forceinline__ Bars& bars_of(unsigned char* raw) { return *reinterpret_cast<Bars*>(raw + kBarsAt); }

// Barriers (one arrival each unless said) and TMEM, by every warp of the CTA.
__device__ __forceinline__ void set_up(Bars& sh, int p_arrivals, int empty3_arrivals, int empty2_arrivals) {
    if (threadIdx.x == 0) {
        for (uint64_t* bar : {&sh.once, &sh.full3[0], &sh.full3[1], &sh.full3[2], &sh.full2[0], &sh.full2[1], &sh.s_full[0],
                              &sh.s_full[1], &sh.dp_full, &sh.done[0], &sh.done[1], &sh.fin})
            mbar_init(smem_addr(bar), 1);
        for (uint64_t* bar : {&sh.s_read, &sh.dp_read, &sh.ds_full[0], &sh.ds_full[1], &sh.trimmed}) mbar_init(smem_addr(bar), 8);
        for (uint64_t* bar : {&sh.p_half[0], &sh.p_half[1], &sh.p_full[0], &sh.p_full[1]})
            mbar_init(smem_addr(bar), p_arrivals);
        for (uint64_t& bar : sh.empty3) mbar_init(smem_addr(&bar), empty3_arrivals);
        for (uint64_t& bar : sh.empty2) mbar_init(smem_addr(&bar), empty2_arrivals);
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x >> 5 == 9) tmem_alloc(smem_addr(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

__device__ __forceinline__ void fetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void tear_down(Bars& sh) {
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x >> 5 == 9) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 512);
    }
}

// The last copies of a ring have landed (a CTA must not leave before).
template <int STAGES>
__device__ __forceinline__ void drain(uint64_t* full, int issued, unsigned long long limit) {
    for (int k = 1; k <= STAGES && k <= issued; ++k)
        mbar_wait(smem_addr(&full[(issued - k) % STAGES]), ((issued - k) / STAGES) & 1, limit);
}

// A finished tile leaves through shared memory and one TMA store: a thread
// owns a row, and rows written straight to global memory would be 32 separate
// lines per instruction (5000 cycles for a CTA's two tiles against 1500).
// put_row: 32 columns of a row in the layout of a 128-byte swizzled box.
__device__ __forceinline__ void put_row(uint32_t tile, int r, int col, const uint4* v) {
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        const int c = col / 8 + z;              // 16-byte piece of the row
        st_shared_v4(tile + (c >> 3) * kSlab + r * 128 + ((c & 7) ^ (r & 7)) * 16, v[z]);
    }
}

__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint32_t tile, int t, int h, int b) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
        asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(x * 64), "r"(t), "r"(h), "r"(b), "r"(tile + x * kSlab)
                     : "memory");
}

// Whether every thread of a named barrier says yes (a warp whose wait ran out
// says no, and none of them goes on).
__device__ __forceinline__ bool all_agree(int id, int threads, bool yes) {
    uint32_t out;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.u32 pi, %1, 0;\n\t"
        "bar.red.and.pred po, %2, %3, pi;\n\t"
        "selp.u32 %0, 1, 0, po;\n\t}"
        : "=r"(out)
        : "r"(uint32_t(yes)), "r"(id), "r"(threads)
        : "memory");
    return out != 0;
}

// The stores that this thread issued have read shared memory.
__device__ __forceinline__ void stores_read() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The end of a product warp: all that it issued has completed.
__device__ __forceinline__ void finish_products(uint64_t* bar, unsigned long long limit) {
    if ((threadIdx.x & 31) == 0) {
        umma_commit(smem_addr(bar));
        mbar_wait(smem_addr(bar), 0, limit);
    }
    __syncwarp();
}

// This thread's warp has reached a point: one arrival, predicated (a branch
// for one lane would cost its reconvergence).
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
    tc_fence_before();
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar)),
        "r"(threadIdx.x & 31)
        : "memory");
}

// ------------------------------------------------------------------ forward
// One CTA per (sequence, query head, two query tiles a and b), which share
// the key tiles that pass: Q stays, K in a ring of three tiles, V of two (a
// load takes about 2500 cycles under load, so each is asked for a whole tile
// pair ahead).
//   products: S = Q K_j^T, O += P_j V_j, P_j over S in TMEM as the A operand:
//     PV_a(j), S_a(j+1), PV_b(j), S_b(j+1), so that one tile's products run
//     under the other's softmax
//   warps 0-3, 4-7: softmax of a and b, a thread per row: running maximum
//     with lazy rescaling (O is rescaled only where the maximum grows by more
//     than 2^8), P_j, O / l at the end.
// Beside the result each row leaves its statistics and what the rounding of
// the result took away (in 8 bits), for D_i in the backward.
// Bound by the chain scores - softmax - P V of each tile: a step of both tiles
// has 2048 cycles of products and, at 16 a cycle, 2048 of exponentials; 153 us
// over the steps of an SM is about twice that.  One query tile per CTA with
// waits by whole warps measured 171 us, two tiles 169, and 153 with the weights
// handed over in halves and results that leave through TMA.
constexpr float kLowScale = 1024.f;      // of the rounding's remainder: 2^-26 .. 56 without loss of its leading bits

// The key tiles of two neighbouring query tiles: those of the first and of
// the second one in one list.
struct PairTiles {
    int qa, lo_b, sink_tiles, sinks, lo, hi, n;
    __device__ __forceinline__ PairTiles(const WindowAttnParams& p, int first, int count, int len) {
        qa = first;
        hi = count == 2 && (qa + 1) * kTile < len ? qa + 1 : qa;
        sink_tiles = p.full ? 0 : (p.S + kTile - 1) / kTile;
        lo = p.full ? 0 : max(0, qa * kTile - p.W + 1) / kTile;
        lo_b = p.full ? 0 : max(0, (qa + 1) * kTile - p.W + 1) / kTile;
        sinks = min(sink_tiles, lo);
        n = sinks + hi - lo + 1;
    }
    __device__ __forceinline__ int at(int j) const { return j < sinks ? j : lo + j - sinks; }
    // whether query tile qa + x visits key tile kt of the list
    __device__ __forceinline__ bool visits(int x, int kt) const {
        return x == 0 ? kt <= qa : hi > qa && (kt >= lo_b || kt < sink_tiles);
    }
    __device__ __forceinline__ bool last(int x, int kt) const { return kt == qa + x; }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) window_fwd_kernel(const __grid_constant__ WindowAttnParams p) {
    extern __shared__ __align__(1024) unsigned char raw[];
    constexpr uint32_t kQK = idesc_f16(kTile, kTile, Elem<T>::bf16, false, false);
    constexpr uint32_t kPV = idesc_f16(kTile, kTile, Elem<T>::bf16, false, true);
    Bars& sh = bars_of(raw);
    const uint32_t smem = smem_addr(raw), sQ = smem, sK = sQ + 2 * kTileBytes, sV = sK + kRing3 * kTileBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem & 1023u) {
        if (p.status && threadIdx.x == 0) set_status(p.status, DUO_STATUS_WAIT_TIMEOUT);
        return;
    }
    if (warp == 8 && lane < 4) fetch_map(lane == 0 ? &p.tm_q : lane == 1 ? &p.tm_k : lane == 2 ? &p.tm_v : &p.tm_out);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // the query tiles with most keys first; those of the last pairs one by one
    const int heads = p.B * p.hq, alone = int(blockIdx.x) - p.pairs, count = alone < 0 ? 2 : 1;
    const int item = alone < 0 ? int(blockIdx.x) : p.pairs + alone / 2;
    const int first = 2 * ((p.n_t + 1) / 2 - 1 - item / heads) + (alone < 0 ? 0 : 1 - alone % 2);
    const int b = item % heads / p.hq, h = item % p.hq, g = h / p.G;
    const int len = length_of(p, b), i0 = first * kTile;
    const int64_t row0 = (int64_t(b) * p.hq + h) * p.Tp;
    if (i0 >= len) {        // no row of a sequence: zeros
        for (int x = threadIdx.x; x < count * kTile * 16; x += kThreads) {
            const int t = i0 + x / 16;
            if (t < p.T) *reinterpret_cast<uint4*>(row_at<T>(p.out, b, h, t) + x % 16 * 8) = make_uint4(0, 0, 0, 0);
        }
        for (int t = i0 + threadIdx.x; t < min(i0 + count * kTile, p.Tp); t += kThreads) p.stats[row0 + t] = -CUDART_INF_F;
        return;
    }
    const PairTiles tiles(p, first, count, len);
    set_up(sh, 4, 1, 1);
    const uint32_t tmem = sh.tmem;
    const Waiter wait{p.status, p.timeout_ns, &sh.abort_flag};

    if (warp == 8) {
        if (lane == 0) {
            const bool two = tiles.hi > tiles.qa;
            mbar_arrive_expect_tx(smem_addr(&sh.once), (two ? 2 : 1) * kTileBytes);
            tma_tile(sQ, &p.tm_q, i0, h, b, smem_addr(&sh.once));
            if (two) tma_tile(sQ + kTileBytes, &p.tm_q, i0 + kTile, h, b, smem_addr(&sh.once));
            int ks = 0, vs = 0;
            for (int j = 0; j < tiles.n; ++j) {
                const int t = tiles.at(j) * kTile;
                if (!wait.thread(smem_addr(&sh.empty3[j % kRing3]), ((j / kRing3) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(smem_addr(&sh.full3[j % kRing3]), kTileBytes);
                tma_tile(sK + j % kRing3 * kTileBytes, &p.tm_k, t, g, b, smem_addr(&sh.full3[j % kRing3]));
                ++ks;
                if (!wait.thread(smem_addr(&sh.empty2[j % kRing2]), ((j / kRing2) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(smem_addr(&sh.full2[j % kRing2]), kTileBytes);
                tma_tile(sV + j % kRing2 * kTileBytes, &p.tm_v, t, g, b, smem_addr(&sh.full2[j % kRing2]));
                ++vs;
            }
            mbar_wait(smem_addr(&sh.once), 0, p.timeout_ns);
            drain<kRing3>(sh.full3, ks, p.timeout_ns);
            drain<kRing2>(sh.full2, vs, p.timeout_ns);
        }
    } else if (warp >= 9) {
        // one thread issues for both tiles (a warp for each: 163 us instead of 153, the
        // two tiles' products then take turns and each lasts twice as long)
        if (warp == 9 && lane == 0) {
            bool ok = wait.thread(smem_addr(&sh.once), 0);
            int seen[2] = {0, 0};               // key tiles that a and b have been through
            // S of both tiles' next key tile and P V of this one, a before b; the
            // products run in the order of issue, so S may take the place of a P
            // whose product has been issued
            for (int j = -1; ok && j < tiles.n; ++j) {
                const int kt = j < 0 ? -1 : tiles.at(j), next = j + 1 < tiles.n ? tiles.at(j + 1) : -1;
                const uint32_t k = sK + (j + 1) % kRing3 * kTileBytes, v = sV + max(j, 0) % kRing2 * kTileBytes;
                // the tiles' own waits come before those for the softmax, which is later
                if (next >= 0) ok = wait.thread(smem_addr(&sh.full3[(j + 1) % kRing3]), ((j + 1) / kRing3) & 1);
                if (ok && j >= 0) ok = wait.thread(smem_addr(&sh.full2[j % kRing2]), (j / kRing2) & 1);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (ok && j >= 0 && tiles.visits(x, kt)) {
                        // the first half of the keys while the second half's weights are worked out
                        ok = wait.thread(smem_addr(&sh.p_half[x]), seen[x] & 1);
                        if (!ok) break;
                        tc_fence_after();
                        mma_rows(tmem + 256 + x * 128, tmem + x * 128, 0, 4, v, kPV, seen[x] > 0);
                        ok = wait.thread(smem_addr(&sh.p_full[x]), seen[x] & 1);
                        if (!ok) break;
                        tc_fence_after();
                        mma_rows(tmem + 256 + x * 128, tmem + x * 128, 4, 8, v, kPV, true);
                        if (tiles.last(x, kt)) umma_commit(smem_addr(&sh.done[x]));
                        ++seen[x];
                    }
                    if (ok && next >= 0 && tiles.visits(x, next)) {
                        mma_dims(tmem + x * 128, sQ + x * kTileBytes, k, kQK);
                        umma_commit(smem_addr(&sh.s_full[x]));
                    }
                }
                if (!ok) break;
                if (next >= 0) umma_commit(smem_addr(&sh.empty3[(j + 1) % kRing3]));
                if (j >= 0) umma_commit(smem_addr(&sh.empty2[j % kRing2]));
            }
            // every product has completed before TMEM is freed
            umma_commit(smem_addr(&sh.dp_full));
            mbar_wait(smem_addr(&sh.dp_full), 0, p.timeout_ns);
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, x = warp >> 2, qt = tiles.qa + x, r = quarter * 32 + lane, i = qt * kTile + r;
        const uint32_t at = tmem + (uint32_t(quarter * 32) << 16) + x * 128;
        float m = kNegBig, l = 0.f;
        bool ok = true;
        int seen = 0;
        for (int j = 0; j < tiles.n; ++j) {
            const int kt = tiles.at(j);
            if (!tiles.visits(x, kt)) continue;
            ok = wait.warp(smem_addr(&sh.s_full[x]), seen & 1);
            if (!ok) break;
            tc_fence_after();
            float s[128];
            uint32_t* u = reinterpret_cast<uint32_t*>(s);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32p(at + q * 32, u + q * 32);
            tmem_wait_ld();
            if (kt == qt || !whole(p, qt, kt)) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t keep = row_sees(p, i, kt * kTile + q * 32);
#pragma unroll
                    for (int c = 0; c < 32; ++c) s[q * 32 + c] = (keep >> c) & 1u ? s[q * 32 + c] : -CUDART_INF_F;
                }
            }
            float t8[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) t8[c] = s[c];
#pragma unroll
            for (int c = 8; c < 128; c += 2) t8[(c >> 1) & 7] = fmax3(t8[(c >> 1) & 7], s[c], s[c + 1]);
            const float mx = fmax3(fmax3(t8[0], t8[1], t8[2]), fmax3(t8[3], t8[4], t8[5]), fmaxf(t8[6], t8[7]));
            const float mt = mx * p.scale_log2;          // a scale above zero keeps the order
            const bool grow = mt > m + kRescaleThreshold;
            const float m_new = grow ? mt : m;
            const float alpha = fast_exp2(m - m_new);
            m = m_new;
            // s_full follows O += P V of the tile before in the order of issue
            if (seen > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tmem_ld32(at + 256 + c * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int z = 0; z < 32; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * alpha);
                    tmem_st32(at + 256 + c * 32, o);
                }
            }
            float2 acc[4] = {};
            const float nm = Elem<T>::kForwardShift - m;
            const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(nm, nm);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t ph[16];
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float2 y = ffma2(make_float2(s[q * 32 + c], s[q * 32 + c + 1]), sc2, nm2);
                    const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    acc[(c >> 1) & 3] = fadd2(acc[(c >> 1) & 3], e);
                    ph[c / 2] = Elem<T>::pack(e.x, e.y);
                }
                tmem_stn<16>(at + q * 16, ph);
                if (q == 1) {
                    if (kt * kTile + kTile > len && len < p.T) {
                        // the sequence ends inside its last key tile (which one query tile visits)
                        ok = wait.warp(smem_addr(&sh.full2[j % kRing2]), (j / kRing2) & 1);
                        if (!ok) break;
                        zero_rows(sV + j % kRing2 * kTileBytes, len - kt * kTile, quarter, 4);
                    }
                    tmem_wait_st();
                    arrive_warp(&sh.p_half[x]);
                }
            }
            if (!ok) break;
            const float2 sum = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
            l = l * alpha + (sum.x + sum.y);
            tmem_wait_st();
            arrive_warp(&sh.p_full[x]);
            ++seen;
        }
        if (x >= count) {                   // another CTA's tile
        } else if (qt > tiles.hi) {         // the second tile lies behind the sequence
            if (i < p.T)
                for (int c = 0; c < kTile; c += 8)
                    *reinterpret_cast<uint4*>(row_at<T>(p.out, b, h, i) + c) = make_uint4(0, 0, 0, 0);
            if (i < p.Tp) p.stats[row0 + i] = -CUDART_INF_F;
        } else if (all_agree(1 + x, 128, ok && wait.warp(smem_addr(&sh.done[x]), 0))) {
            tc_fence_after();
            const bool row = i < len;
            const float inv = row && l > 0.f ? 1.f / l : 0.f;
            p.stats[row0 + i] =
                row && l > 0.f ? Elem<T>::kForwardShift + Elem<T>::kStatsShift - (m + __log2f(l)) : -CUDART_INF_F;
            // through this tile's Q, which no product reads any more
            const uint32_t tile = sQ + x * kTileBytes;
            uint4* low = reinterpret_cast<uint4*>(p.low + (row0 + qt * kTile) * kTile) + r;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32], hi[16], lo[8];
                tmem_ld32(at + 256 + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int z = 0; z < 32; z += 2) {
                    const float2 y = make_float2(__uint_as_float(o[z]) * inv, __uint_as_float(o[z + 1]) * inv);
                    hi[z / 2] = row ? Elem<T>::pack(y.x, y.y) : 0;
                    const float2 w = Elem<T>::wide(hi[z / 2]);
                    uint16_t f8;
                    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;"
                        : "=h"(f8)
                        : "f"((y.y - w.y) * kLowScale), "f"((y.x - w.x) * kLowScale));
                    lo[z / 4] = z % 4 == 0 ? f8 : lo[z / 4] | uint32_t(f8) << 16;
                }
                const uint4 v[4] = {make_uint4(hi[0], hi[1], hi[2], hi[3]), make_uint4(hi[4], hi[5], hi[6], hi[7]),
                                    make_uint4(hi[8], hi[9], hi[10], hi[11]), make_uint4(hi[12], hi[13], hi[14], hi[15])};
                put_row(tile, r, c * 32, v);
                // the remainders lie 16 of 128 rows together: whole lines
                low[c * 2 * kTile] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                low[(c * 2 + 1) * kTile] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
            }
            fence_proxy_async_smem();
            named_bar_sync(1 + x, 128);
            if ((warp & 3) == 0 && lane == 0) {
                store_tile(&p.tm_out, tile, qt * kTile, h, b);
                stores_read();
            }
        }
    }
    tear_down(sh);
}

// ------------------------------------------------------------------ D_i = o_i . g_i
// Bound by HBM: reads each output row, its remainder and the gradient's row
// once; writes minus D.  The remainder matters where few keys share a row:
// the rounding of o_i is then as large beside D_i as that of ds.  Sixteen
// threads per row, four rows per thread.  Measured: 17 us for 84 MB from cold
// caches (32 heads x 4096 tokens), 0.75 of the copy rate.  In fp16 each block
// also leaves the largest |g_i|^2 of its rows, and blocks behind these that of
// the values' rows: what ds is scaled by.
constexpr int kDeltaRows = 4;

// The largest of 256 threads' numbers (not below zero), by one of them.
__device__ __forceinline__ void store_largest(float x, float* to) {
    __shared__ float top[8];
    const float w = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
    if (threadIdx.x % 32 == 0) top[threadIdx.x / 32] = w;
    __syncthreads();
    if (threadIdx.x == 0)
        *to = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7])));
}

// The sum of 8 elements' squares.
template <typename T>
__device__ __forceinline__ float squares(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float s = 0.f;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        const float2 u = Elem<T>::wide(w[z]);
        s = fmaf(u.x, u.x, fmaf(u.y, u.y, s));
    }
    return s;
}

// Of 16 threads' numbers that make up a row.
__device__ __forceinline__ float row_sum(float d) {
#pragma unroll
    for (int z = 8; z > 0; z >>= 1) d += __shfl_xor_sync(0xffffffffu, d, z);
    return d;
}

template <typename T>
__global__ void __launch_bounds__(256) window_delta_kernel(const __grid_constant__ WindowAttnParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // blockIdx.x: 64 rows of a (sequence, head); Tp is a multiple of 64
    const int blocks = p.Tp / (16 * kDeltaRows);
    if (!Elem<T>::bf16 && int(blockIdx.x) >= blocks * p.B * p.hq) {       // 64 rows of the values
        const int bg = int(blockIdx.x) / blocks - p.B * p.hq, b = bg / p.n_kv, len = length_of(p, b);
        const int t0 = int(blockIdx.x) % blocks * (16 * kDeltaRows) + threadIdx.x / 16;
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kDeltaRows; ++k) {
            const int t = t0 + 16 * k;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (t < len) x = *reinterpret_cast<const uint4*>(row_at<const T>(p.v, b, bg - b * p.n_kv, t) + threadIdx.x % 16 * 8);
            top = fmaxf(top, row_sum(squares<T>(x)));
        }
        store_largest(top, p.peak + blockIdx.x);
        return;
    }
    const int bh = int(blockIdx.x) / blocks, b = bh / p.hq, h = bh - b * p.hq;
    const int t0 = (int(blockIdx.x) - bh * blocks) * (16 * kDeltaRows) + threadIdx.x / 16, part = threadIdx.x % 16;
    const int len = length_of(p, b);
    uint4 x[kDeltaRows], y[kDeltaRows];
    uint2 lo[kDeltaRows];
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
        const int t = t0 + 16 * k;
        x[k] = y[k] = make_uint4(0, 0, 0, 0);
        lo[k] = make_uint2(0, 0);
        if (t < len) {
            x[k] = *reinterpret_cast<const uint4*>(row_at<const T>(p.out, b, h, t) + part * 8);
            y[k] = *reinterpret_cast<const uint4*>(row_at<const T>(p.dout, b, h, t) + part * 8);
            lo[k] = *reinterpret_cast<const uint2*>(p.low + (int64_t(bh) * p.Tp + t / kTile * kTile) * kTile +
                                                       (part / 2 * kTile + t % kTile) * 16 + part % 2 * 8);
        }
    }
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
        const uint32_t xs[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, ys[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
        float d = 0.f, rest = 0.f;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const float2 u = Elem<T>::wide(xs[z]), v = Elem<T>::wide(ys[z]);
            uint32_t f16;
            asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(f16) : "h"(uint16_t((z < 2 ? lo[k].x : lo[k].y) >> (z % 2 * 16))));
            const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&f16));
            d = fmaf(u.x, v.x, fmaf(u.y, v.y, d));
            rest = fmaf(w.x, v.x, fmaf(w.y, v.y, rest));
        }
        d = row_sum(fmaf(rest, 1.f / kLowScale, d));
        if (part == 0) p.delta[int64_t(bh) * p.Tp + t0 + 16 * k] = -d;
        if (!Elem<T>::bf16) top = fmaxf(top, row_sum(squares<T>(y[k])));
    }
    if (!Elem<T>::bf16) store_largest(top, p.peak + blockIdx.x);
}

// ------------------------------------------------------------------ backward
// One launch holds two kinds of work items: first those of the key tiles (the
// longest), then those of the query tiles, which fill the SMs that have run
// out of the first.  Warps 0-7: two per TMEM lane quarter, one 64-column half
// each.

// What a key tile's work item is: rows x of its list of (query head of the
// group, query tile), x0 <= x < x1.
struct KeyItem {
    int b, g, kt, pieces, piece;
    int nq;              // query tiles that see the key tile
    int x0, x1;
    int64_t slot;        // of its partial sums
    __device__ __forceinline__ KeyItem(const WindowAttnParams& p, int item) {
        const int bk = p.B * p.n_kv, first = p.n_long * p.p_long * bk;
        const bool lng = item < first;
        pieces = lng ? p.p_long : p.p_short;
        const int x = lng ? item : item - first;
        kt = x / (pieces * bk) + (lng ? 0 : p.n_long);
        piece = x / bk % pieces;
        b = x % bk / p.n_kv;
        g = x % p.n_kv;
        slot = lng || p.p_long == 1 ? x : int64_t(first) + x;      // a class of one piece has no slots
        const int len = length_of(p, b);
        int hi = (len - 1) / kTile;                      // -1 / 128 is 0: an empty sequence has no rows below
        if (!p.full && kt * kTile >= p.S) hi = min(hi, (kt * kTile + kTile - 1 + p.W - 1) / kTile);
        nq = len > kt * kTile ? hi - kt + 1 : 0;
        const int64_t all = int64_t(nq) * p.G;
        x0 = int(all * piece / pieces);
        x1 = int(all * (piece + 1) / pieces);
    }
};

// fp16: h with M in 2^h .. 2^(h + 1) for a sequence's key head; ds is held times f = 2^(kWeightShift - h), by
// warps 0 .. 7 together.  Without a gradient, or with one that is not finite, f = 1.  bf16: ds as it is.
template <typename T>
__device__ __forceinline__ int ds_exponent(const WindowAttnParams& p, Bars& sh, int b, int g) {
    if (Elem<T>::bf16) return 0;
    const int blocks = p.Tp / (16 * kDeltaRows);
    const float *pg = p.peak + (int64_t(b) * p.hq + g * p.G) * blocks,
                *pv = p.peak + (int64_t(p.B) * p.hq + int64_t(b) * p.n_kv + g) * blocks;
    float x = 0.f, y = 0.f;
    for (int i = threadIdx.x; i < p.G * blocks; i += 256) x = fmaxf(x, pg[i]);
    for (int i = threadIdx.x; i < blocks; i += 256) y = fmaxf(y, pv[i]);
    x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
    y = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(y)));
    if (threadIdx.x % 32 == 0) {
        sh.peak[0][threadIdx.x / 32] = x;
        sh.peak[1][threadIdx.x / 32] = y;
    }
    named_bar_sync(1, 256);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x = fmaxf(x, sh.peak[0][i]);
        y = fmaxf(y, sh.peak[1][i]);
    }
    const float m2 = x * y;             // M^2: below 2^79, and above 2^-97 where it is not zero
    return m2 > 0.f && m2 < CUDART_INF_F ? (int(__float_as_uint(m2) >> 23) - 127) >> 1 : kWeightShift;
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Key tile: K, V stay; Q (a ring of three) and g (of two) pass.  With keys
// along the TMEM lanes,
//   S^T = K Q^T, P^T = exp2(..),  dP^T = V g^T, dS^T = P^T (dP^T - D),
//   dV += P^T g,  dK += dS^T Q,
// P^T and dS^T being A operands straight from TMEM.  S^T and dP^T take turns
// in one TMEM region: as soon as one is in registers the other's product
// starts, so that dP_x is worked out under the exponentials of S_x and S_{x+1}
// under dS_x; dK_{x-1} and dV_x fill the rest.
template <typename T>
__device__ __forceinline__ void key_tile(const WindowAttnParams& p, Bars& sh, uint32_t smem, const Waiter& wait) {
    constexpr uint32_t kDims = idesc_f16(kTile, kTile, Elem<T>::bf16, false, false);
    constexpr uint32_t kRows = idesc_f16(kTile, kTile, Elem<T>::bf16, false, true);
    constexpr uint32_t kA = 0, kP = 128, kDS = 192, kDV = 256, kDK = 384;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KeyItem it(p, int(blockIdx.x));
    const uint32_t sK = smem, sV = sK + kTileBytes, sQ = sV + kTileBytes, sG = sQ + kRing3 * kTileBytes;
    // D comes with Q and goes with it after dK, the statistics with g and after dV:
    // this step's D is read while its dV runs
    const uint32_t sDelta = smem + kStatsAt, sStat = sDelta + kRing3 * kTile * 4;
    const int len = length_of(p, it.b), k0 = it.kt * kTile, n = it.x1 - it.x0;
    const uint32_t tmem = sh.tmem;

    if (warp == 8) {
        if (lane == 0 && n > 0) {
            mbar_arrive_expect_tx(smem_addr(&sh.once), 2 * kTileBytes);
            tma_tile(sK, &p.tm_k, k0, it.g, it.b, smem_addr(&sh.once));
            tma_tile(sV, &p.tm_v, k0, it.g, it.b, smem_addr(&sh.once));
            int qs = 0, gs = 0;
            for (int x = 0; x < n; ++x) {
                const int at = it.x0 + x, h = it.g * p.G + at / it.nq, i0 = (it.kt + at % it.nq) * kTile;
                const int64_t row = (int64_t(it.b) * p.hq + h) * p.Tp + i0;
                const int q3 = x % kRing3, g2 = x % kRing2;
                uint32_t bar = smem_addr(&sh.full3[q3]);
                if (!wait.thread(smem_addr(&sh.empty3[q3]), ((x / kRing3) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(bar, kTileBytes + kTile * 4);
                tma_tile(sQ + q3 * kTileBytes, &p.tm_q, i0, h, it.b, bar);
                bulk_row(sDelta + q3 * kTile * 4, p.delta + row, bar);
                ++qs;
                bar = smem_addr(&sh.full2[g2]);
                if (!wait.thread(smem_addr(&sh.empty2[g2]), ((x / kRing2) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(bar, kTileBytes + kTile * 4);
                tma_tile(sG + g2 * kTileBytes, &p.tm_do, i0, h, it.b, bar);
                bulk_row(sStat + g2 * kTile * 4, p.stats + row, bar);
                ++gs;
            }
            mbar_wait(smem_addr(&sh.once), 0, p.timeout_ns);
            drain<kRing3>(sh.full3, qs, p.timeout_ns);
            drain<kRing2>(sh.full2, gs, p.timeout_ns);
        }
    } else if (warp == 9) {
        // S and dP; warps wait as a whole and lane 0 issues
        bool ok = n > 0 && wait.warp(smem_addr(&sh.once), 0);
        for (int x = 0; ok && x < n; ++x) {
            const int q3 = x % kRing3, g2 = x % kRing2;
            ok = wait.warp(smem_addr(&sh.full3[q3]), (x / kRing3) & 1) && wait.warp(smem_addr(&sh.dp_read), x & 1);
            if (!ok) break;                                                 // dP_{x-1} is in registers
            tc_fence_after();
            if (lane == 0) {
                mma_dims(tmem + kA, sK, sQ + q3 * kTileBytes, kDims);
                umma_commit(smem_addr(&sh.s_full[0]));
            }
            __syncwarp();
            ok = wait.warp(smem_addr(&sh.full2[g2]), (x / kRing2) & 1) && wait.warp(smem_addr(&sh.s_read), x & 1);
            if (!ok) break;                                                 // S_x is in registers
            tc_fence_after();
            if (lane == 0) {
                mma_dims(tmem + kA, sV, sG + g2 * kTileBytes, kDims);
                umma_commit(smem_addr(&sh.dp_full));
                umma_commit(smem_addr(&sh.empty2[g2]));      // dV lets g go too: it may be the earlier of the two
            }
            __syncwarp();
        }
        finish_products(&sh.fin, p.timeout_ns);
    } else if (warp == 10) {
        // dV and dK: a warp of their own, so that neither pair waits for the other's operands
        bool ok = n > 0;
        for (int x = 0; ok && x < n; ++x) {
            ok = wait.warp(smem_addr(&sh.p_full[0]), x & 1);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                mma_rows(tmem + kDV, tmem + kP, 0, 8, sG + x % kRing2 * kTileBytes, kRows, x > 0);
                umma_commit(smem_addr(&sh.empty2[x % kRing2]));
            }
            __syncwarp();
            ok = wait.warp(smem_addr(&sh.ds_full[0]), x & 1);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                mma_rows(tmem + kDK, tmem + kDS, 0, 8, sQ + x % kRing3 * kTileBytes, kRows, x > 0);
                umma_commit(smem_addr(&sh.empty3[x % kRing3]));
            }
            __syncwarp();
        }
        finish_products(&sh.done[0], p.timeout_ns);
    } else {
        const int quarter = warp & 3, half = warp >> 2, r = quarter * 32 + lane, key = k0 + r, cb = half * 64;
        const uint32_t at = tmem + (uint32_t(quarter * 32) << 16);
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        // where the sequence ends inside query tile x of the list, what lies behind
        // becomes zeros before any product
        const auto trim = [&](uint64_t* full, uint32_t tile, int x, int phase) {
            const int i0 = (it.kt + (it.x0 + x) % it.nq) * kTile;
            if (!wait.warp(smem_addr(full), phase & 1)) return false;
            zero_rows(tile, len - i0, warp, 8);
            return true;
        };
        const int end_tile = len < p.T ? len / kTile : -1;     // the one that is cut (or none)
        bool ok = true;
        uint32_t ph[32];               // P of a step, then its dS: stored while dP of the next step is worked out
        int qt = it.kt + (n > 0 ? it.x0 % it.nq : 0);
        if (n > 0) {
            if (qt == end_tile) ok = trim(&sh.full3[0], sQ, 0, 0);
            if (ok) arrive_warp(&sh.dp_read);
        }
        const int h = ds_exponent<T>(p, sh, it.b, it.g);
        const float2 f2 = make_float2(power_of_two(-h), power_of_two(-h));     // the weights carry 2^kWeightShift
        // dS of step x, once that of the step before has been used
        const auto put_ds = [&](int x) {
            if (x > 0 && !wait.warp(smem_addr(&sh.empty3[(x - 1) % kRing3]), ((x - 1) / kRing3) & 1)) return false;
            tc_fence_after();
            tmem_stn<32>(at + kDS + half * 32, ph);
            tmem_wait_st();
            arrive_warp(&sh.ds_full[0]);
            return true;
        };
        for (int x = 0; ok && x < n; ++x) {
            const int i0 = qt * kTile;
            const uint32_t stat = sStat + x % kRing2 * kTile * 4 + cb * 4, delta = sDelta + x % kRing3 * kTile * 4 + cb * 4;
            // this warp's own waits for the statistics and D, while S_x is worked out
            ok = wait.warp(smem_addr(&sh.full2[x % kRing2]), (x / kRing2) & 1) &&
                 wait.warp(smem_addr(&sh.full3[x % kRing3]), (x / kRing3) & 1);
            if (!ok) break;
            if (qt == end_tile) zero_rows(sG + x % kRing2 * kTileBytes, len - i0, warp, 8);
            ok = wait.warp(smem_addr(&sh.s_full[0]), x & 1);
            if (!ok) break;
            tc_fence_after();
            float s[64];
            uint32_t* u = reinterpret_cast<uint32_t*>(s);
            tmem_ld32p(at + kA + cb, u);
            tmem_ld32p(at + kA + cb + 32, u + 32);
            tmem_wait_ld();
            arrive_warp(&sh.s_read);
            if (x > 0 && !put_ds(x - 1)) {
                ok = false;
                break;
            }
            if (qt == it.kt || !whole(p, qt, it.kt) || i0 + kTile > len) {
                // rows i0 + c with key <= row < len, within the window unless the key is a sink
                int hi = len - 1 - i0;
                if (!p.full && key >= p.S) hi = min(hi, key + p.W - 1 - i0);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int o = cb + q * 32;
                    const uint32_t keep = range_bits(key - i0 - o, hi - o);
#pragma unroll
                    for (int c = 0; c < 32; ++c) s[q * 32 + c] = (keep >> c) & 1u ? s[q * 32 + c] : -CUDART_INF_F;
                }
            }
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const uint4 nl = lds128(stat + c * 4);
                float* e = s + c;
                const float2 y = ffma2(make_float2(e[0], e[1]), sc2,
                                       make_float2(__uint_as_float(nl.x), __uint_as_float(nl.y)));
                const float2 z = ffma2(make_float2(e[2], e[3]), sc2,
                                       make_float2(__uint_as_float(nl.z), __uint_as_float(nl.w)));
                e[0] = fast_exp2(y.x);
                e[1] = fast_exp2(y.y);
                e[2] = fast_exp2(z.x);
                e[3] = fast_exp2(z.y);
                ph[c / 2] = Elem<T>::pack(e[0], e[1]);
                ph[c / 2 + 1] = Elem<T>::pack(e[2], e[3]);
            }
            // P_{x-1} has been used (and g_{x-1})
            if (x > 0) ok = wait.warp(smem_addr(&sh.empty2[(x - 1) % kRing2]), ((x - 1) / kRing2) & 1);
            if (!ok) break;
            tc_fence_after();
            tmem_stn<32>(at + kP + half * 32, ph);
            tmem_wait_st();
            arrive_warp(&sh.p_full[0]);
            ok = wait.warp(smem_addr(&sh.dp_full), x & 1);
            if (!ok) break;
            tc_fence_after();
            uint32_t d[64];
            tmem_ld32p(at + kA + cb, d);
            tmem_ld32p(at + kA + cb + 32, d + 32);
            if (++qt == it.kt + it.nq) qt = it.kt;
            if (x + 1 < n && qt == end_tile)
                ok = trim(&sh.full3[(x + 1) % kRing3], sQ + (x + 1) % kRing3 * kTileBytes, x + 1, (x + 1) / kRing3);
            if (!ok) break;
            tmem_wait_ld();
            arrive_warp(&sh.dp_read);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const uint4 dl = lds128(delta + c * 4);
                float* e = s + c;
                if (!Elem<T>::bf16) {
                    *reinterpret_cast<float2*>(e) = fmul2(make_float2(e[0], e[1]), f2);
                    *reinterpret_cast<float2*>(e + 2) = fmul2(make_float2(e[2], e[3]), f2);
                }
                const float2 y = fmul2(make_float2(e[0], e[1]),
                                       fadd2(make_float2(__uint_as_float(d[c]), __uint_as_float(d[c + 1])),
                                             make_float2(__uint_as_float(dl.x), __uint_as_float(dl.y))));
                const float2 z = fmul2(make_float2(e[2], e[3]),
                                       fadd2(make_float2(__uint_as_float(d[c + 2]), __uint_as_float(d[c + 3])),
                                             make_float2(__uint_as_float(dl.z), __uint_as_float(dl.w))));
                ph[c / 2] = Elem<T>::pack(y.x, y.y);
                ph[c / 2 + 1] = Elem<T>::pack(z.x, z.y);
            }
        }
        if (ok && n > 0) ok = put_ds(n - 1);
        if (all_agree(1, 256, ok && wait.warp(smem_addr(&sh.done[0]), 0))) {
            tc_fence_after();
            const bool row = key < len && n > 0;
            // what the sums were held times, taken out
            const float held[2] = {Elem<T>::bf16 ? 1.f : power_of_two(h - kWeightShift),
                                   Elem<T>::bf16 ? 1.f : power_of_two(-kWeightShift)};
            // through the ring: all products that read it are done
            const uint32_t tile[2] = {sQ, sQ + kTileBytes};
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[32];
                    tmem_ld32(at + (w ? kDV : kDK) + cb + c * 32, o);
                    tmem_wait_ld();
                    if (it.pieces > 1) {        // four columns of 128 rows together: whole lines
                        float4* y = reinterpret_cast<float4*>(p.part + it.slot * (2 * kTile * kTile) + w * kTile * kTile) +
                                    (cb + c * 32) / 4 * kTile + r;
#pragma unroll
                        for (int z = 0; z < 32; z += 4)
                            y[z / 4 * kTile] = row ? make_float4(__uint_as_float(o[z]) * held[w],
                                                                 __uint_as_float(o[z + 1]) * held[w],
                                                                 __uint_as_float(o[z + 2]) * held[w],
                                                                 __uint_as_float(o[z + 3]) * held[w])
                                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                    } else {
                        uint4 v[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            v[z] = row ? pack8<T>(o + 8 * z, (w ? 1.f : p.scale) * held[w]) : make_uint4(0, 0, 0, 0);
                        put_row(tile[w], r, cb + c * 32, v);
                    }
                }
            if (it.pieces == 1) {
                fence_proxy_async_smem();
                named_bar_sync(1, 256);
                if (warp == 0 && lane == 0) {
                    store_tile(&p.tm_dk, tile[0], k0, it.g, it.b);
                    store_tile(&p.tm_dv, tile[1], k0, it.g, it.b);
                    stores_read();
                }
            }
        }
    }
}

// Query tile: Q, g stay; K (a ring of three) and V (of two) pass.  With rows
// along the TMEM lanes,
//   S = Q K^T (two regions), dP = g V^T, dS over S, dQ += dS K.
// S_{j+1} is worked out under the exponentials of S_j, dP_{j+1} as soon as
// dP_j is in registers.
template <typename T>
__device__ __forceinline__ void query_tile(const WindowAttnParams& p, Bars& sh, uint32_t smem, const Waiter& wait) {
    constexpr uint32_t kDims = idesc_f16(kTile, kTile, Elem<T>::bf16, false, false);
    constexpr uint32_t kRows = idesc_f16(kTile, kTile, Elem<T>::bf16, false, true);
    constexpr uint32_t kS = 0, kDP = 256, kDQ = 384;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int item = int(blockIdx.x) - p.items_kv, heads = p.B * p.hq;
    const int qt = p.n_t - 1 - item / heads, b = item % heads / p.hq, h = item % p.hq, g = h / p.G;
    const uint32_t sQ = smem, sG = sQ + kTileBytes, sK = sG + kTileBytes, sV = sK + kRing3 * kTileBytes;
    const int len = length_of(p, b), i0 = qt * kTile;
    const KeyTiles tiles(p, qt);
    const int n = i0 < len ? tiles.n : 0;
    const bool cut = i0 + kTile > len && len < p.T;
    const uint32_t tmem = sh.tmem;

    if (warp == 8) {
        if (lane == 0 && n > 0) {
            mbar_arrive_expect_tx(smem_addr(&sh.once), 2 * kTileBytes);
            tma_tile(sQ, &p.tm_q, i0, h, b, smem_addr(&sh.once));
            tma_tile(sG, &p.tm_do, i0, h, b, smem_addr(&sh.once));
            int ks = 0, vs = 0;
            for (int j = 0; j < n; ++j) {
                const int k3 = j % kRing3, v2 = j % kRing2, t = tiles.at(j) * kTile;
                if (!wait.thread(smem_addr(&sh.empty3[k3]), ((j / kRing3) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(smem_addr(&sh.full3[k3]), kTileBytes);
                tma_tile(sK + k3 * kTileBytes, &p.tm_k, t, g, b, smem_addr(&sh.full3[k3]));
                ++ks;
                if (!wait.thread(smem_addr(&sh.empty2[v2]), ((j / kRing2) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(smem_addr(&sh.full2[v2]), kTileBytes);
                tma_tile(sV + v2 * kTileBytes, &p.tm_v, t, g, b, smem_addr(&sh.full2[v2]));
                ++vs;
            }
            mbar_wait(smem_addr(&sh.once), 0, p.timeout_ns);
            drain<kRing3>(sh.full3, ks, p.timeout_ns);
            drain<kRing2>(sh.full2, vs, p.timeout_ns);
        }
    } else if (warp == 9) {
        bool ok = n > 0 && wait.warp(smem_addr(&sh.once), 0);
        for (int j = 0; ok && j < n; ++j) {
            const int k3 = j % kRing3, v2 = j % kRing2;
            ok = wait.warp(smem_addr(&sh.full3[k3]), (j / kRing3) & 1);
            if (ok && cut && j == n - 1) ok = wait.warp(smem_addr(&sh.trimmed), 0);
            // dS_{j-2}, which lies in this S, has been used
            if (ok && j > 1) ok = wait.warp(smem_addr(&sh.empty3[(j - 2) % kRing3]), ((j - 2) / kRing3) & 1);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                mma_dims(tmem + kS + (j & 1) * 128, sQ, sK + k3 * kTileBytes, kDims);
                umma_commit(smem_addr(&sh.s_full[j & 1]));
            }
            __syncwarp();
            ok = wait.warp(smem_addr(&sh.full2[v2]), (j / kRing2) & 1);
            if (ok && j > 0) ok = wait.warp(smem_addr(&sh.dp_read), (j - 1) & 1);       // dP_{j-1} is in registers
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                mma_dims(tmem + kDP, sG, sV + v2 * kTileBytes, kDims);
                umma_commit(smem_addr(&sh.dp_full));
                umma_commit(smem_addr(&sh.empty2[v2]));
            }
            __syncwarp();
        }
        finish_products(&sh.fin, p.timeout_ns);
    } else if (warp == 10) {
        bool ok = n > 0;
        for (int j = 0; ok && j < n; ++j) {
            ok = wait.warp(smem_addr(&sh.ds_full[j & 1]), (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                const uint32_t ds = tmem + kS + (j & 1) * 128, k = sK + j % kRing3 * kTileBytes;
                mma_rows(tmem + kDQ, ds, 0, 4, k, kRows, j > 0);
                mma_rows(tmem + kDQ, ds + 32, 4, 8, k, kRows, true);
                umma_commit(smem_addr(&sh.empty3[j % kRing3]));
            }
            __syncwarp();
        }
        finish_products(&sh.done[0], p.timeout_ns);
    } else {
        const int quarter = warp & 3, half = warp >> 2, r = quarter * 32 + lane, i = i0 + r, cb = half * 64;
        const uint32_t at = tmem + (uint32_t(quarter * 32) << 16) + cb;
        const int64_t row = (int64_t(b) * p.hq + h) * p.Tp + i;
        const int e = ds_exponent<T>(p, sh, b, g);      // p_ij f = 2^(s + nl): the factor costs nothing here
        const float nl = p.stats[row] - (Elem<T>::bf16 ? 0.f : float(e)), dl = p.delta[row];
        const float scale = Elem<T>::bf16 ? p.scale : p.scale * power_of_two(e - kWeightShift);
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nl2 = make_float2(nl, nl), dl2 = make_float2(dl, dl);
        // where the sequence ends inside the last key tile, what lies behind becomes
        // zeros before any product, a step ahead
        const auto trim = [&](int j) {
            if (!wait.warp(smem_addr(&sh.full3[j % kRing3]), (j / kRing3) & 1) ||
                !wait.warp(smem_addr(&sh.full2[j % kRing2]), (j / kRing2) & 1))
                return false;
            zero_rows(sK + j % kRing3 * kTileBytes, len - i0, warp, 8);
            zero_rows(sV + j % kRing2 * kTileBytes, len - i0, warp, 8);
            arrive_warp(&sh.trimmed);
            return true;
        };
        bool ok = true;
        if (cut && n == 1) ok = trim(0);
        for (int j = 0; ok && j < n; ++j) {
            const int kt = tiles.at(j);
            const uint32_t sb = kS + (j & 1) * 128;
            if (cut && j + 2 == n) ok = trim(j + 1);
            ok = ok && wait.warp(smem_addr(&sh.s_full[j & 1]), (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            float s[64];
            uint32_t* u = reinterpret_cast<uint32_t*>(s);
            tmem_ld32p(at + sb, u);
            tmem_ld32p(at + sb + 32, u + 32);
            tmem_wait_ld();
            if (kt == qt || !whole(p, qt, kt)) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t keep = row_sees(p, i, kt * kTile + cb + q * 32);
#pragma unroll
                    for (int c = 0; c < 32; ++c) s[q * 32 + c] = (keep >> c) & 1u ? s[q * 32 + c] : -CUDART_INF_F;
                }
            }
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                const float2 y = ffma2(make_float2(s[c], s[c + 1]), sc2, nl2);
                s[c] = fast_exp2(y.x);
                s[c + 1] = fast_exp2(y.y);
            }
            ok = wait.warp(smem_addr(&sh.dp_full), j & 1);
            if (!ok) break;
            tc_fence_after();
            uint32_t d[64], ph[32];
            tmem_ld32p(at + kDP, d);
            tmem_ld32p(at + kDP + 32, d + 32);
            tmem_wait_ld();
            arrive_warp(&sh.dp_read);
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                const float2 y = fmul2(make_float2(s[c], s[c + 1]),
                                       fadd2(make_float2(__uint_as_float(d[c]), __uint_as_float(d[c + 1])), dl2));
                ph[c / 2] = Elem<T>::pack(y.x, y.y);
            }
            tmem_stn<32>(at + sb, ph);     // over this thread's own columns of S
            tmem_wait_st();
            // S_{j+1} and dP_{j+1} may be here already: these warps can be a step
            // ahead of the one that waits for this, so two barriers take turns
            arrive_warp(&sh.ds_full[j & 1]);
        }
        if (all_agree(1, 256, ok && wait.warp(smem_addr(&sh.done[0]), 0))) {
            tc_fence_after();
            // through the ring: all products that read it are done
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t o[32];
                uint4 v[4];
                tmem_ld32(at + kDQ + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int z = 0; z < 4; ++z) v[z] = i < len ? pack8<T>(o + 8 * z, scale) : make_uint4(0, 0, 0, 0);
                put_row(sK, r, cb + c * 32, v);
            }
            fence_proxy_async_smem();
            named_bar_sync(1, 256);
            if (warp == 0 && lane == 0) {
                store_tile(&p.tm_dq, sK, i0, h, b);
                stores_read();
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) window_bwd_kernel(const __grid_constant__ WindowAttnParams p) {
    extern __shared__ __align__(1024) unsigned char raw[];
    Bars& sh = bars_of(raw);
    const uint32_t smem = smem_addr(raw);
    if (smem & 1023u) {
        if (p.status && threadIdx.x == 0) set_status(p.status, DUO_STATUS_WAIT_TIMEOUT);
        return;
    }
    if (threadIdx.x < 7)
        fetch_map(threadIdx.x < 4 ? (threadIdx.x < 2 ? (threadIdx.x ? &p.tm_k : &p.tm_q) : (threadIdx.x == 2 ? &p.tm_v : &p.tm_do))
                                  : (threadIdx.x == 4 ? &p.tm_dq : threadIdx.x == 5 ? &p.tm_dk : &p.tm_dv));
    set_up(sh, 8, 1, int(blockIdx.x) < p.items_kv ? 2 : 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const Waiter wait{p.status, p.timeout_ns, &sh.abort_flag};
    if (int(blockIdx.x) < p.items_kv)
        key_tile<T>(p, sh, smem, wait);
    else
        query_tile<T>(p, sh, smem, wait);
    tear_down(sh);
}

// dK, dV of the key tiles whose rows were shared out: the pieces' sums, in
// order.  Bound by HBM.  Sixteen blocks per key tile: 16 columns each of dK
// (first 8), then of dV.
template <typename T>
__global__ void __launch_bounds__(256) window_join_kernel(const __grid_constant__ WindowAttnParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int bk = p.B * p.n_kv;
    const int n_first = p.p_long > 1 ? p.n_long * bk : 0;
    const int tile = int(blockIdx.x) / 16;
    const bool lng = tile < n_first;
    const int y = lng ? tile : tile - n_first, pieces = lng ? p.p_long : p.p_short;
    const int kt = y / bk + (lng ? 0 : p.n_long), b = y % bk / p.n_kv, g = y % p.n_kv;
    // a warp: 8 columns of 32 rows
    const int w = blockIdx.x / 8 % 2, c = (blockIdx.x % 8 * 2 + threadIdx.x / 128) * 8, r = threadIdx.x % 128;
    const int key = kt * kTile + r;
    if (key >= p.T) return;
    const int64_t first = (lng || p.p_long == 1 ? 0 : int64_t(p.n_long) * p.p_long * bk) +
                          int64_t(y / bk) * pieces * bk + y % bk;
    uint32_t o[8] = {};
    for (int k = 0; k < pieces; ++k) {
        const float4* src = reinterpret_cast<const float4*>(p.part + (first + int64_t(k) * bk) * (2 * kTile * kTile) +
                                                            w * kTile * kTile) + c / 4 * kTile + r;
        const float4 u = src[0], v = src[kTile];
        const float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int z = 0; z < 8; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) + f[z]);
    }
    *reinterpret_cast<uint4*>(row_at<T>(w ? p.dv : p.dk, b, g, key) + c) = pack8<T>(o, w ? 1.f : p.scale);
}

// ------------------------------------------------------------------ host side
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int padded(int tokens) { return (tokens + kTile - 1) / kTile * kTile; }

// [batch][heads][tokens][128] by strides; box 64 x 128 tokens, 128-byte swizzle.
bool make_map(CUtensorMap* m, const duo_heads& x, const duo_window_attn_desc& d, int heads) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t n[3] = {cuuint64_t(d.tokens), cuuint64_t(heads), cuuint64_t(d.batch)};
    const int64_t s[3] = {x.token_stride, x.head_stride, x.batch_stride};
    cuuint64_t dims[4] = {cuuint64_t(kTile), n[0], n[1], n[2]}, strides[3];
    // a dimension of one entry has no stride that matters
    for (int i = 0; i < 3; ++i) strides[i] = n[i] > 1 ? cuuint64_t(s[i]) * 2 : kTile * 2;
    cuuint32_t box[4] = {64, 128, 1, 1}, one[4] = {1, 1, 1, 1};
    return enc(m, d.dtype == DUO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, x.data,
               dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_desc(const duo_window_attn_desc* d) {
    if (!d) return DUO_ERR_INVALID_ARG;
    if (d->dtype != DUO_BF16 && d->dtype != DUO_FP16) return DUO_ERR_UNSUPPORTED;
    if (d->head_dim != kTile) return DUO_ERR_UNSUPPORTED;
    if (d->batch < 0 || d->tokens < 0 || d->num_q_heads < 1 || d->num_kv_heads < 1 ||
        d->num_q_heads % d->num_kv_heads != 0)
        return DUO_ERR_INVALID_ARG;
    if (d->sink < 0 || d->window < 0) return DUO_ERR_INVALID_ARG;
    if (!(d->scale > 0.f) || !(d->scale < 1e30f)) return DUO_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d->lengths) & 3) return DUO_ERR_ALIGNMENT;
    if (d->tokens > (1 << 26)) return DUO_ERR_UNSUPPORTED;
    // work items are counted in 31 bits, with room for the pieces
    if (int64_t(d->batch) * d->num_q_heads * (padded(d->tokens) / kTile) > (1 << 26)) return DUO_ERR_UNSUPPORTED;
    return DUO_OK;
}

int check_heads(const duo_heads* x, const duo_window_attn_desc& d, int heads) {
    if (!x || !x->data) return DUO_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(x->data) & 15) return DUO_ERR_ALIGNMENT;
    const int64_t n[3] = {d.batch, heads, d.tokens}, s[3] = {x->batch_stride, x->head_stride, x->token_stride};
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] % 8 != 0) return DUO_ERR_ALIGNMENT;
        if (s[i] < kTile || s[i] >= (int64_t(1) << 39)) return DUO_ERR_INVALID_ARG;
    }
    return DUO_OK;
}

HeadTensor head_tensor(const duo_heads& x) { return HeadTensor{x.data, x.batch_stride, x.head_stride, x.token_stride}; }

void fill_params(WindowAttnParams& p, const duo_window_attn_desc& d, float* stats, int32_t* status) {
    p.stats = stats;
    p.low = reinterpret_cast<uint8_t*>(stats + int64_t(d.batch) * d.num_q_heads * padded(d.tokens));
    p.B = d.batch;
    p.hq = d.num_q_heads;
    p.n_kv = d.num_kv_heads;
    p.G = p.hq / p.n_kv;
    p.T = d.tokens;
    p.Tp = padded(d.tokens);
    p.n_t = p.Tp / kTile;
    p.full = d.window == 0 || d.window >= d.tokens;
    p.W = std::min(p.full ? d.tokens : d.window, d.tokens);
    p.S = p.full ? 0 : std::min(d.sink, d.tokens);
    p.scale = d.scale;
    p.scale_log2 = d.scale * 1.4426950408889634f;
    p.lengths = d.lengths;
    p.status = status;
    p.timeout_ns = kWaitLimitNs;
}

// How the key tiles' work is shared out.  A key tile's list has (query tiles
// that see it) x (query heads of the group) entries; those that hold sinks
// are seen by every later row.  A class of tiles whose longest list is about
// k times an SM's share of the whole is cut in k pieces, but in none shorter
// than kPiece entries, which cost more to join than they gain.
constexpr int kPiece = 8;

void plan_pieces(WindowAttnParams& p, int num_sms) {
    const auto list = [&](int kt) {
        int hi = p.n_t - 1;
        if (!p.full && kt * kTile >= p.S) hi = std::min(hi, int((int64_t(kt) * kTile + kTile - 1 + p.W - 1) / kTile));
        return int64_t(hi - kt + 1) * p.G;
    };
    p.n_long = p.full ? 0 : std::min(p.n_t, (p.S + kTile - 1) / kTile);
    int64_t all = 0, top_long = 0, top_short = 0;
    for (int kt = 0; kt < p.n_t; ++kt) {
        all += list(kt);
        int64_t& top = kt < p.n_long ? top_long : top_short;
        top = std::max(top, list(kt));
    }
    const int64_t share = std::max<int64_t>(all * p.B * p.n_kv / num_sms, kPiece);
    const auto pieces = [&](int64_t top) { return int(std::min<int64_t>(std::max<int64_t>((top + share / 2) / share, 1), 64)); };
    p.p_long = pieces(top_long);
    p.p_short = pieces(top_short);
    p.items_kv = (p.n_long * p.p_long + (p.n_t - p.n_long) * p.p_short) * p.B * p.n_kv;
}

// Pairs of query tiles that the forward's CTAs take; those behind them go one
// tile to a CTA, which takes about 0.8 of a pair's time.  Worth it where pairs
// would leave half of the SMs or more idle: all of them where there are few
// (one head of 8192 tokens: 110 us instead of 136; 2 x 8 heads of 1024: 19.5
// instead of 23.2), and a last wave of equal ones (16 heads of 8192 tokens,
// window 1024, 3.46 waves: 113 instead of 118).  Without a window the last
// pairs are short and fill the gaps as they are (32 heads of 4096 tokens: 151.5,
// and 153 with single tiles at the end).
void plan_pairs(WindowAttnParams& p, int num_sms) {
    const int all = (p.n_t + 1) / 2 * p.B * p.hq, rest = p.full ? all : all % num_sms;
    p.pairs = 2 * rest <= num_sms ? all - rest : all;
}

// Floats of `peak`.
int64_t peaks(const WindowAttnParams& p, int dtype) {
    return dtype == DUO_BF16 ? 0 : int64_t(p.B) * (p.hq + p.n_kv) * (p.Tp / (16 * kDeltaRows));
}

int64_t partial_slots(const WindowAttnParams& p) {
    const int64_t bk = int64_t(p.B) * p.n_kv;
    return (p.p_long > 1 ? int64_t(p.n_long) * p.p_long * bk : 0) +
           (p.p_short > 1 ? int64_t(p.n_t - p.n_long) * p.p_short * bk : 0);
}

// The current device's SMs.  A thread that has made no call on the device yet
// (autograd's) has no context for the tensor maps: cudaSetDevice binds it.
int device_sms(int* sms) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess &&
                   cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess
               ? DUO_OK
               : DUO_ERR_CUDA;
}

template <typename K>
cudaError_t launch(K kernel, const WindowAttnParams& p, dim3 grid, int threads, uint32_t smem, cudaStream_t s) {
    if (smem > 0) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
int run_forward(const WindowAttnParams& p, cudaStream_t s) {
    const unsigned items = unsigned(p.pairs + 2 * ((p.n_t + 1) / 2 * p.B * p.hq - p.pairs));
    return launch(window_fwd_kernel<T>, p, dim3(items), kThreads, kSmem, s) == cudaSuccess
               ? DUO_OK
               : DUO_ERR_CUDA;
}

template <typename T>
int run_backward(const WindowAttnParams& p, cudaStream_t s) {
    const unsigned rows = unsigned(p.B) * (p.hq + (Elem<T>::bf16 ? 0 : p.n_kv)) * (p.Tp / (16 * kDeltaRows));
    if (launch(window_delta_kernel<T>, p, dim3(rows), 256, 0, s) != cudaSuccess) return DUO_ERR_CUDA;
    const unsigned items = unsigned(p.items_kv + p.n_t * p.B * p.hq);
    if (launch(window_bwd_kernel<T>, p, dim3(items), kThreads, kSmem, s) != cudaSuccess) return DUO_ERR_CUDA;
    const unsigned joins = unsigned(((p.p_long > 1 ? p.n_long : 0) + (p.p_short > 1 ? p.n_t - p.n_long : 0)) * p.B * p.n_kv);
    if (joins > 0 && launch(window_join_kernel<T>, p, dim3(16 * joins), 256, 0, s) != cudaSuccess) return DUO_ERR_CUDA;
    return DUO_OK;
}

}  // namespace

}  // namespace duo

extern "C" {

int duo_window_attn_stats_bytes(const duo_window_attn_desc* d, size_t* bytes) {
    const int rc = duo::check_desc(d);
    if (rc) return rc;
    if (!bytes) return DUO_ERR_INVALID_ARG;
    // a number and 128 bytes per row
    *bytes = size_t(d->batch) * d->num_q_heads * duo::padded(d->tokens) * (4 + duo::kTile);
    return DUO_OK;
}

int duo_window_attn_workspace_bytes(const duo_window_attn_desc* d, size_t* bytes) {
    const int rc = duo::check_desc(d);
    if (rc) return rc;
    if (!bytes) return DUO_ERR_INVALID_ARG;
    int sms = 0;
    if (duo::device_sms(&sms)) return DUO_ERR_CUDA;
    duo::WindowAttnParams p{};
    duo::fill_params(p, *d, nullptr, nullptr);
    duo::plan_pieces(p, sms);
    *bytes = duo::align256(size_t(d->batch) * d->num_q_heads * p.Tp * 4) +
             duo::align256(size_t(duo::peaks(p, d->dtype)) * 4) + size_t(duo::partial_slots(p)) * 2 * duo::kTile * duo::kTile * 4;
    return DUO_OK;
}

int duo_window_attn(const duo_window_attn_desc* d, const duo_heads* q, const duo_heads* k, const duo_heads* v,
                    const duo_heads* out, float* stats, int32_t* status, duo_stream_t stream) {
    int rc = duo::check_desc(d);
    if (rc) return rc;
    if (d->batch == 0 || d->tokens == 0) return DUO_OK;
    if (!stats) return DUO_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(stats) & 15) || (reinterpret_cast<uintptr_t>(status) & 3)) return DUO_ERR_ALIGNMENT;
    for (const duo_heads* x : {q, k, v, out})
        if ((rc = duo::check_heads(x, *d, x == k || x == v ? d->num_kv_heads : d->num_q_heads))) return rc;
    int sms = 0;
    if (duo::device_sms(&sms)) return DUO_ERR_CUDA;
    duo::WindowAttnParams p{};
    duo::fill_params(p, *d, stats, status);
    duo::plan_pairs(p, sms);
    if (!duo::make_map(&p.tm_q, *q, *d, p.hq) || !duo::make_map(&p.tm_k, *k, *d, p.n_kv) ||
        !duo::make_map(&p.tm_v, *v, *d, p.n_kv) || !duo::make_map(&p.tm_out, *out, *d, p.hq))
        return DUO_ERR_CUDA;
    p.out = duo::head_tensor(*out);
    return d->dtype == DUO_BF16 ? duo::run_forward<__nv_bfloat16>(p, stream) : duo::run_forward<__half>(p, stream);
}

int duo_window_attn_grad(const duo_window_attn_desc* d, const duo_heads* q, const duo_heads* k, const duo_heads* v,
                         const duo_heads* out, const duo_heads* dout, const float* stats, const duo_heads* dq,
                         const duo_heads* dk, const duo_heads* dv, void* workspace, size_t workspace_bytes,
                         int32_t* status, duo_stream_t stream) {
    int rc = duo::check_desc(d);
    if (rc) return rc;
    if (d->batch == 0 || d->tokens == 0) return DUO_OK;
    if (!stats || !workspace) return DUO_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(stats) & 15) || (reinterpret_cast<uintptr_t>(status) & 3) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255))
        return DUO_ERR_ALIGNMENT;
    for (const duo_heads* x : {q, out, dout, dq})
        if ((rc = duo::check_heads(x, *d, d->num_q_heads))) return rc;
    for (const duo_heads* x : {k, v, dk, dv})
        if ((rc = duo::check_heads(x, *d, d->num_kv_heads))) return rc;
    size_t need = 0;
    if ((rc = duo_window_attn_workspace_bytes(d, &need))) return rc;
    if (workspace_bytes < need) return DUO_ERR_BUFFER_TOO_SMALL;
    int sms = 0;
    if (duo::device_sms(&sms)) return DUO_ERR_CUDA;
    duo::WindowAttnParams p{};
    duo::fill_params(p, *d, const_cast<float*>(stats), status);
    duo::plan_pieces(p, sms);
    if (!duo::make_map(&p.tm_q, *q, *d, p.hq) || !duo::make_map(&p.tm_k, *k, *d, p.n_kv) ||
        !duo::make_map(&p.tm_v, *v, *d, p.n_kv) || !duo::make_map(&p.tm_do, *dout, *d, p.hq) ||
        !duo::make_map(&p.tm_dq, *dq, *d, p.hq) || !duo::make_map(&p.tm_dk, *dk, *d, p.n_kv) ||
        !duo::make_map(&p.tm_dv, *dv, *d, p.n_kv))
        return DUO_ERR_CUDA;
    p.v = duo::head_tensor(*v);
    p.out = duo::head_tensor(*out);
    p.dout = duo::head_tensor(*dout);
    p.dk = duo::head_tensor(*dk);
    p.dv = duo::head_tensor(*dv);
    p.delta = static_cast<float*>(workspace);
    p.peak = reinterpret_cast<float*>(static_cast<char*>(workspace) + duo::align256(size_t(p.B) * p.hq * p.Tp * 4));
    p.part = reinterpret_cast<float*>(reinterpret_cast<char*>(p.peak) +
                                      duo::align256(size_t(duo::peaks(p, d->dtype)) * 4));
    return d->dtype == DUO_BF16 ? duo::run_backward<__nv_bfloat16>(p, stream) : duo::run_backward<__half>(p, stream);
}

}  // extern "C"
