// Block tables and slot maps built on the GPU from the requests' lengths.
//
// State: for each sequence the pages that it holds (table, held), for each
// page how many sequences hold it (refs) and one bit while none does
// (free_bits).  A step (reserve_kernel) gives back the pages behind each
// sequence's len_before tokens, finds what each sequence lacks for its new
// tokens, and hands out free pages: the r-th page handed out is the r-th
// lowest free one, and sequence b's are numbers P(b) .. P(b) + need_b - 1,
// P the exclusive prefix sum of the needs.  "The lowest free page" and prefix
// sums depend on no order of execution, so the table is the same whenever
// the calls are.
//
// Bound by latency: a decode step touches a few hundred bytes.  One block of
// 1024 threads does the whole step (a grid would need a barrier between
// giving back, counting and handing out); the bitmap keeps the search for
// free pages at one bit per page (a pool of 32,768 pages: one word per
// thread).  The map of a long ragged batch (16 bytes per token) is written by
// a second launch over the whole GPU.
// Measured: a decode step of 8 sequences 5.7 us, 256 sequences with 8 prompts
// 11.8 us, 1024 sequences on a pool that runs out 15.2 us.  In one run, 1024
// threads took 5.8, 12.3 and 16.1 us, 512 6.0, 12.5 and 22.0, 256 5.4, 13.8 and
// 31.7.  In another, with loads moved ahead and pairs of sums in one scan, it
// took 5.7, 11.6 and 15.5 us against 5.4, 11.0 and 14.9 as it stands.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pages.cuh"

namespace duo {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSmall = 2048;         // sequences / handed-out pages kept in shared memory
constexpr int kMapInBlock = 4096;    // longer maps are written by map_kernel
constexpr int kMapThreads = 256;

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) { return __shfl_up_sync(0xffffffffu, v, d); }

// Exclusive prefix sum over the block and the block's total.  `part` is
// shared scratch of kWarps + 1 values; synchronises before it returns.
__device__ int64_t block_scan(int64_t v, int64_t* part, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = shfl_up64(x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int64_t own = part[lane];
        int64_t w = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = shfl_up64(w, d);
            if (lane >= d) w += y;
        }
        part[lane] = w - own;
        if (lane == 31) part[kWarps] = w;
    }
    __syncthreads();
    const int64_t before = part[warp] + x - v;
    total = part[kWarps];
    __syncthreads();
    return before;
}

// The last i in [0, n) with start[i] <= x (start[0] <= x).
template <typename T>
__device__ __forceinline__ int last_at_most(const T* start, int n, T x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int pages_for(int64_t tokens, int page_tokens) {
    return int(uint32_t(tokens + page_tokens - 1) / uint32_t(page_tokens));
}

// One sequence's request.
struct Request {
    int64_t lb, n;       // tokens held and to come
    int held, keep;      // pages held, and those that stay
    int total;           // pages needed after the step
    bool sane;           // lengths are usable
    bool fits;           // within capacity and the table
};

__device__ __forceinline__ Request request_of(const ReserveParams& p, int b) {
    Request r;
    r.lb = p.len_before[b];
    r.n = p.n_new ? p.n_new[b] : 1;
    r.sane = r.lb >= 0 && r.n >= 0 && r.lb <= p.cap;
    r.fits = r.sane && r.lb + r.n <= p.cap;
    r.held = r.keep = r.total = 0;
    if (p.page_tokens > 0) {
        r.held = p.st.held[b];
        r.keep = r.sane ? min(r.held, pages_for(r.lb, p.page_tokens)) : r.held;
        r.total = r.fits ? pages_for(r.lb + r.n, p.page_tokens) : r.keep;
        r.fits = r.fits && r.total <= p.max_pages;
    }
    return r;
}

// Entry t of the map, a token of sequence b, whose entries are cu[b] .. cu[b + 1] - 1.  Its position comes
// from what the step wrote and not from len_before: len_after may be the same array.
__device__ __forceinline__ void write_map(const ReserveParams& p, const int32_t* cu, int t, int b) {
    const int pos = p.len_after[b] - (cu[b + 1] - t);
    p.seq[t] = b;
    p.pos[t] = pos;
    int64_t slot;
    if (p.page_tokens > 0) {
        const uint32_t j = uint32_t(pos) / uint32_t(p.page_tokens);
        slot = int64_t(__ldcg(p.st.table + size_t(b) * p.max_pages + j)) * p.page_tokens +
               (uint32_t(pos) - j * uint32_t(p.page_tokens));
    } else {
        slot = int64_t(b) * p.cap + pos;
    }
    p.slot[t] = slot;
}

__device__ __forceinline__ void write_no_token(const ReserveParams& p, int t) {
    p.seq[t] = -1;
    p.pos[t] = -1;
    p.slot[t] = -1;
}

__global__ void __launch_bounds__(kThreads) reserve_kernel(const __grid_constant__ ReserveParams p) {
    __shared__ int64_t part[kWarps + 1];
    __shared__ int64_t tail_start[kThreads];
    __shared__ int tail_page[kThreads];
    __shared__ int32_t small_start[kSmall + 1];   // pages handed out before each sequence
    __shared__ int32_t small_cu[kSmall + 1];      // tokens served before each sequence
    __shared__ int32_t small_list[kSmall];        // pages handed out
    const int tid = threadIdx.x;
    const PageState& st = p.st;
    const bool paged = p.page_tokens > 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    // ---- give back the pages that hold no token
    if (paged) {
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int b = b0 + tid;
            int keep = 0, tail = 0;
            if (b < p.B) {
                const Request r = request_of(p, b);
                keep = r.keep;
                tail = r.held - r.keep;
            }
            if (!__syncthreads_or(tail > 0)) continue;
            int64_t all;
            tail_start[tid] = block_scan(tail, part, all);
            tail_page[tid] = keep;
            __syncthreads();
            for (int64_t x = tid; x < all; x += kThreads) {
                const int i = last_at_most<int64_t>(tail_start, kThreads, x);
                int32_t* entry = st.table + size_t(b0 + i) * p.max_pages + tail_page[i] + (x - tail_start[i]);
                const int page = *entry;
                *entry = -1;
                if (uint32_t(page) < uint32_t(p.num_pages) && atomicSub(st.refs + page, 1) == 1)
                    atomicOr(st.free_bits + page / 32, 1u << (page % 32));
            }
            __syncthreads();
        }
    }

    // ---- the free pages: each thread counts those of its run of words
    int64_t free_total = 0, free_before = 0;
    const int run = (st.words + kThreads - 1) / kThreads;
    const int w0 = min(tid * run, st.words), w1 = min(w0 + run, st.words);
    if (paged) {
        int count = 0;
        for (int w = w0; w < w1; ++w) count += __popc(__ldcg(st.free_bits + w));
        free_before = block_scan(count, part, free_total);
    }

    // ---- who is served, and the prefix sums of pages and tokens
    int32_t* start = p.B <= kSmall ? small_start : st.page_start;
    int32_t* cu = p.B <= kSmall ? small_cu : p.cu;
    int64_t asked_pages = 0, asked_tokens = 0;    // by the sequences of earlier chunks
    int64_t pages = 0, tokens = 0;                // granted to them
    int flags = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        Request r{};
        bool valid = false;
        int64_t need = 0, n = 0;
        if (b < p.B) {
            r = request_of(p, b);
            valid = r.fits;
            if (!r.sane) flags |= DUO_STATUS_BAD_LENGTH;
            else if (!r.fits) flags |= DUO_STATUS_OVER_CAPACITY;
            // the last page that stays is written by the new tokens: it must be this sequence's alone
            if (valid && paged && r.n > 0 && r.lb % p.page_tokens != 0 && r.keep == pages_for(r.lb, p.page_tokens)) {
                const int page = __ldcg(st.table + size_t(b) * p.max_pages + r.keep - 1);
                if (uint32_t(page) < uint32_t(p.num_pages) && __ldcg(st.refs + page) > 1) {
                    valid = false;
                    flags |= DUO_STATUS_SHARED_PAGE;
                }
            }
            if (valid) {
                need = max(r.total - r.keep, 0);
                n = r.n;
            }
        }
        int64_t all_pages = 0, all_tokens = 0;
        int64_t pages_at = paged ? block_scan(need, part, all_pages) : 0;
        int64_t tokens_at = block_scan(n, part, all_tokens);
        const bool short_pool = need > 0 && asked_pages + pages_at + need > free_total;
        const bool short_map = p.cu && asked_tokens + tokens_at + n > p.T;
        if (short_pool) flags |= DUO_STATUS_NO_PAGE;
        if (short_map) flags |= DUO_STATUS_OVER_CAPACITY;
        const bool served = valid && !short_pool && !short_map;
        asked_pages += all_pages;
        asked_tokens += all_tokens;
        if (__syncthreads_or(valid && !served)) {
            if (!served) need = n = 0;
            pages_at = paged ? block_scan(need, part, all_pages) : 0;
            tokens_at = block_scan(n, part, all_tokens);
        }
        if (b < p.B) {
            p.len_after[b] = int32_t(r.lb + (served ? r.n : 0));
            if (paged) {
                st.held[b] = r.keep + int(need);
                start[b] = int32_t(pages + pages_at);
            }
            if (p.cu) {
                p.cu[b] = int32_t(tokens + tokens_at);
                if (cu != p.cu) cu[b] = int32_t(tokens + tokens_at);
            }
        }
        pages += all_pages;
        tokens += all_tokens;
    }
    if (tid == 0) {
        if (paged) start[p.B] = int32_t(pages);
        if (p.cu) {
            p.cu[p.B] = int32_t(tokens);
            cu[p.B] = int32_t(tokens);
        }
    }
    if (flags) set_status(p.status, flags);

    // ---- hand out the lowest free pages
    if (paged && pages > 0) {
        int32_t* list = pages <= kSmall ? small_list : st.list;
        for (int w = w0; w < w1 && free_before < pages; ++w) {
            uint32_t bits = __ldcg(st.free_bits + w), left = bits;
            while (left && free_before < pages) {
                list[free_before++] = w * 32 + __ffs(left) - 1;
                left &= left - 1;
            }
            if (left != bits) st.free_bits[w] = left;
        }
        __syncthreads();
        for (int64_t x = tid; x < pages; x += kThreads) {
            const int b = last_at_most<int32_t>(start, p.B, int32_t(x));
            const int page = list[x];
            // sequence b's new pages follow those that it keeps
            const int first = st.held[b] - (start[b + 1] - start[b]);
            st.table[size_t(b) * p.max_pages + first + (int32_t(x) - start[b])] = page;
            st.refs[page] = 1;
        }
    }

    // ---- the map of a short batch
    if (p.cu && p.T <= kMapInBlock) {
        __syncthreads();
        for (int t = tid; t < p.T; t += kThreads) {
            if (t >= tokens) {
                write_no_token(p, t);
                continue;
            }
            write_map(p, cu, t, last_at_most<int32_t>(cu, p.B, t));
        }
    }
}

// The map of a long batch.  last_at_most finds the last sequence that starts
// at or before the token: one without tokens starts where the next one does
// and is passed over.
__global__ void __launch_bounds__(kMapThreads) map_kernel(const __grid_constant__ ReserveParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int t = int(blockIdx.x) * kMapThreads + threadIdx.x;
    if (t >= p.T) return;
    if (t >= p.cu[p.B]) {
        write_no_token(p, t);
        return;
    }
    write_map(p, p.cu, t, last_at_most<int32_t>(p.cu, p.B, t));
}

__global__ void pages_init_kernel(PageState st, int64_t entries, int64_t B, int64_t num_pages) {
    const int64_t stride = int64_t(gridDim.x) * blockDim.x, first = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    for (int64_t i = first; i < entries; i += stride) st.table[i] = -1;
    for (int64_t i = first; i < B; i += stride) st.held[i] = 0;
    for (int64_t i = first; i < num_pages; i += stride) st.refs[i] = 0;
    for (int64_t i = first; i < st.words; i += stride) {
        const int64_t left = num_pages - i * 32;
        st.free_bits[i] = left >= 32 ? 0xffffffffu : (1u << left) - 1;
    }
}

// A fork's pages: dst gives back what it holds, shares src's full pages and
// gets the lowest free page for a partly filled last one.  Where src holds
// fewer pages than the prefix has, dst ends without any (and the copy that
// follows writes nothing).
__global__ void __launch_bounds__(kThreads) share_kernel(const __grid_constant__ ShareParams p) {
    __shared__ int lowest;
    const int tid = threadIdx.x;
    const PageState& st = p.st;
    int32_t* from = st.table + size_t(p.src) * p.max_pages;
    int32_t* to = st.table + size_t(p.dst) * p.max_pages;
    const int prefix_full = p.len / p.page_tokens, prefix_partly = p.len % p.page_tokens != 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int held = st.held[p.dst];
    const bool enough = st.held[p.src] >= prefix_full + prefix_partly;
    const int full = enough ? prefix_full : 0, partly = enough ? prefix_partly : 0;
    if (!enough && tid == 0) set_status(p.status, DUO_STATUS_NO_PAGE);
    if (tid == 0) lowest = 0x7fffffff;
    __syncthreads();
    for (int j = tid; j < held; j += kThreads) {
        const int page = to[j];
        if (uint32_t(page) < uint32_t(p.num_pages) && atomicSub(st.refs + page, 1) == 1)
            atomicOr(st.free_bits + page / 32, 1u << (page % 32));
    }
    __syncthreads();
    for (int j = tid; j < max(held, full); j += kThreads) {
        const int page = j < full ? from[j] : -1;
        if (uint32_t(page) < uint32_t(p.num_pages)) atomicAdd(st.refs + page, 1);
        to[j] = page;
    }
    if (partly) {
        for (int w = tid; w < st.words; w += kThreads) {
            const uint32_t bits = __ldcg(st.free_bits + w);
            if (bits) {
                atomicMin(&lowest, w * 32 + __ffs(bits) - 1);
                break;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        const bool found = partly && lowest != 0x7fffffff;
        if (found) {
            st.free_bits[lowest / 32] = __ldcg(st.free_bits + lowest / 32) & ~(1u << (lowest % 32));
            st.refs[lowest] = 1;
            to[full] = lowest;
        } else if (partly) {
            set_status(p.status, DUO_STATUS_NO_PAGE);
        }
        st.held[p.dst] = full + found;
    }
}

template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, int blocks, int threads, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Offsets of the state's arrays, each 256-byte aligned; returns the bytes.
size_t pages_layout(int64_t B, int64_t max_pages, int64_t num_pages, char* base, PageState* st) {
    size_t off = 0;
    const auto take = [&](int64_t n) {
        char* at = base + off;
        off = (off + size_t(n) * 4 + 255) & ~size_t(255);
        return at;
    };
    PageState s{};
    s.words = int32_t((num_pages + 31) / 32);
    s.table = reinterpret_cast<int32_t*>(take(B * max_pages));
    s.held = reinterpret_cast<int32_t*>(take(B));
    s.refs = reinterpret_cast<int32_t*>(take(num_pages));
    s.free_bits = reinterpret_cast<uint32_t*>(take(s.words));
    s.list = reinterpret_cast<int32_t*>(take(num_pages));
    s.page_start = reinterpret_cast<int32_t*>(take(B + 1));
    if (st) *st = s;
    return off;
}

cudaError_t launch_pages_init(const PageState& st, int64_t B, int64_t max_pages, int64_t num_pages, cudaStream_t s) {
    const int64_t most = std::max(B * max_pages, num_pages);
    const int blocks = int(std::min<int64_t>((most + 255) / 256, 2048));
    pages_init_kernel<<<blocks, 256, 0, s>>>(st, B * max_pages, B, num_pages);
    return cudaGetLastError();
}

cudaError_t launch_reserve(const ReserveParams& p, cudaStream_t s) {
    const cudaError_t e = launch(reserve_kernel, p, 1, kThreads, s);
    if (e != cudaSuccess || !p.cu || p.T <= kMapInBlock) return e;
    return launch(map_kernel, p, (p.T - 1) / kMapThreads + 1, kMapThreads, s);     // no sum that passes 31 bits
}

cudaError_t launch_share(const ShareParams& p, cudaStream_t s) { return launch(share_kernel, p, 1, kThreads, s); }

}  // namespace duo
