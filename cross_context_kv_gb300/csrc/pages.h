// pages.h -- the arguments of the kvfix_pages_* calls, as the kernels take them.
#pragma once

#include "pool.cuh"

namespace kvfix {

// The pool and its books: how many lists hold each page, the lists' pages and their lengths.
struct PagesArgs {
    PoolView pool;
    int page, page_log, total;  // tokens per page (2^page_log), pages of the pool
    int32_t* refs;    // [total]
    int32_t* pages;   // [lists][wide]
    int32_t* len;     // [lists]
    int lists, wide;
};

size_t extend_workspace_bytes(long long total, long long lists);
cudaError_t launch_pages_extend(const PagesArgs& a, const int32_t* parent, const int32_t* extra, void* workspace,
                                cudaStream_t s);
cudaError_t launch_pages_cut(const PagesArgs& a, const int32_t* base, const int32_t* path, int max_path,
                             const int32_t* kept, cudaStream_t s);
size_t compact_workspace_bytes(long long total);
cudaError_t launch_pages_compact(const PagesArgs& a, int32_t* live, void* workspace, cudaStream_t s);

}  // namespace kvfix
