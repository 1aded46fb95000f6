// Launch parameters of the page state's kernels (pages.cu).
#pragma once

#include "duo_internal.cuh"

namespace duo {

// The state's device arrays (duo_kv_pages_init), in the caller's buffer.
struct PageState {
    int32_t* table;          // [B][max_pages]
    int32_t* held;           // [B]
    int32_t* refs;           // [num_pages]
    uint32_t* free_bits;     // [words]
    int32_t* list;           // [num_pages]  scratch: the pages that a call hands out, in order
    int32_t* page_start;     // [B + 1]      scratch: pages handed out before each sequence
    int32_t words;
};

struct ReserveParams {
    PageState st;
    const int32_t* len_before;
    const int32_t* n_new;        // may be null: 1 each
    int32_t* len_after;
    int32_t* cu;                 // null: no map
    int32_t* seq;
    int32_t* pos;
    int64_t* slot;
    int32_t* status;
    int64_t cap;
    int32_t num_pages;
    int32_t page_tokens;         // 0: contiguous caches
    int32_t max_pages;
    int32_t B;
    int32_t T;                   // entries of the map
};

struct ShareParams {
    PageState st;
    int32_t* status;
    int32_t num_pages, max_pages, page_tokens;
    int32_t src, dst, len;
};

size_t pages_layout(int64_t B, int64_t max_pages, int64_t num_pages, char* base, PageState* st);
cudaError_t launch_pages_init(const PageState& st, int64_t B, int64_t max_pages, int64_t num_pages, cudaStream_t s);
cudaError_t launch_reserve(const ReserveParams& p, cudaStream_t s);
cudaError_t launch_share(const ShareParams& p, cudaStream_t s);

}  // namespace duo
