// pages.cu -- kvfix_pages_extend, kvfix_pages_cut, kvfix_pages_compact: the pages that lists of a
// paged pool take, share, give back and leave behind, all decided on the device, so that a captured
// graph follows the lists as they change.
//
// The books.  refs[p] counts the lists that hold page p, and a page is free where there are none:
// there is no list of free pages to keep in order, and the same books always give the same pages
// (the lowest free ones, in the order of lists).  Counts change by whole numbers, whose order of
// addition does not matter.
//
// Extend and compact are a small kernel that decides (one CTA: a scan over the lists, and one over
// refs whose spans belong to a warp each, so it takes one block-wide step, not one per thousand
// pages), and one that moves: page tables and counts, and rows in all layers, both planes, codes
// and scales.  Cut is one kernel, a cluster of CTAs per list.  (A call's last kernel triggers
// nothing early: what follows on the stream may read the books before it waits.)  Moving is bound
// by HBM (a row is read and written once), deciding by latency; measured figures at the launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "pages.h"

namespace kvfix {

static __device__ unsigned int g_status_pages;

unsigned read_status_pages(cudaStream_t stream) {
    unsigned h = 0, zero = 0;
    cudaMemcpyFromSymbolAsync(&h, g_status_pages, sizeof h, 0, cudaMemcpyDeviceToHost, stream);
    cudaMemcpyToSymbolAsync(g_status_pages, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    cudaStreamSynchronize(stream);
    return h;
}

constexpr int kPlanThreads = 1024;  // of a deciding CTA
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = 152 * 6;  // persistent: what there is to move is known on the device

// Inclusive sum over the block; `warp_sums` is free again after the next block barrier.
__device__ __forceinline__ int block_sum(int x, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        const int n = warp_sums[w];
        if (w < warp) before += n;
        all += n;
    }
    *total = all;
    return x + before;
}

// The pages of a warp's span, 32 at a time and eight loads ahead: f(page, refs, there), until
// done() says that the rest is of no interest.
template <typename F, typename Done>
__device__ __forceinline__ void for_pages(const int32_t* refs, int lo, int hi, F f, Done done) {
    const int lane = threadIdx.x & 31;
    for (int p0 = lo; p0 < hi && !done(); p0 += 8 * 32) {
        int r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = p0 + 32 * i + lane;
            r[i] = p < hi ? refs[p] : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = p0 + 32 * i + lane;
            if (p0 + 32 * i < hi) f(p, r[i], p < hi);
        }
    }
}

// Pages in use of a warp's span.  (Lanes add for themselves: with a vote for every 32 pages one
// SM's issue was the bound, 31 us of an extend over 131072 pages instead of 15.)
__device__ __forceinline__ int used_pages(const int32_t* refs, int lo, int hi) {
    int n = 0;
    for_pages(refs, lo, hi, [&](int, int r, bool) { n += r > 0; }, [] { return false; });
    return __reduce_add_sync(0xffffffffu, n);
}

__device__ __forceinline__ int span_of(int total) { return ((total + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32; }

// Pages of a number of tokens (below 2^30 + 2^7).
__device__ __forceinline__ int pages_of(int tokens, const PagesArgs& a) { return (tokens + a.page - 1) >> a.page_log; }

// `n` 16-byte vectors by `threads` threads, four in flight each.
__device__ __forceinline__ void copy_vectors(const unsigned char* src, unsigned char* dst, int n, int tid, int threads) {
    constexpr int U = 4;
    const uint4* from = reinterpret_cast<const uint4*>(src);
    uint4* to = reinterpret_cast<uint4*>(dst);
    int i = tid;
    for (; i + (U - 1) * threads < n; i += U * threads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_stream(from + i + u * threads);
#pragma unroll
        for (int u = 0; u < U; ++u) st_stream(to + i + u * threads, v[u]);
    }
    for (; i < n; i += threads) st_stream(to + i, ld_stream(from + i));
}

// The first `rows` rows of a page to another page, one layer and plane.
__device__ __forceinline__ void copy_page_rows(const PagesArgs& a, int layer, int p, int src, int dst, int rows) {
    const PoolView& v = a.pool;
    const PoolPlane& pl = v.plane[p];
    const int row = v.heads * pool_head_bytes(v.format, v.dim);
    const unsigned char* from = pl.codes + layer * v.sl + (long long)src * a.page * v.ss;
    unsigned char* to = pl.codes + layer * v.sl + (long long)dst * a.page * v.ss;
    if (v.ss == row) {
        copy_vectors(from, to, rows * (row / 16), threadIdx.x, kMoveThreads);
    } else {
        // rows apart (another plane's between them): a few rows at a time
        const int per = row / 16, some = max(1, kMoveThreads / per), mine = threadIdx.x / per;
        for (int r = mine; r < rows && mine < some; r += some)
            copy_vectors(from + r * v.ss, to + r * v.ss, per, threadIdx.x - mine * per, per < kMoveThreads ? per : kMoveThreads);
    }
    if (v.format == KVFIX_POOL_BF16) return;
    const long long at = (long long)layer * v.heads * v.slots;
    if (v.format == KVFIX_POOL_E4M3) {
        for (int i = threadIdx.x; i < rows * v.heads; i += kMoveThreads) {
            const int h = i / rows, r = i - h * rows;
            unsigned char* s = pl.scales + at + (long long)h * v.slots + r;
            s[(long long)dst * a.page] = s[(long long)src * a.page];
        }
    } else {
        const int per = v.dim / kQGroup, words = rows * per;
        for (int i = threadIdx.x; i < words * v.heads; i += kMoveThreads) {
            const int h = i / words, r = i - h * words;
            uint32_t* s = reinterpret_cast<uint32_t*>(pl.scales) + (at + (long long)h * v.slots) * per + r;
            s[(long long)dst * a.page * per] = s[(long long)src * a.page * per];
        }
    }
}

// ------------------------------------------------------------------ extend
struct __align__(16) ExtendList {
    int from;         // the list whose pages it takes over (itself: it grows)
    int have, want;   // pages, on entry and after
    int first;        // its first new page's place in Extend::fresh
    int last;         // the last page on entry
    int tokens;       // length after; -1: nothing happens to this list
    int copy, rows;   // whether the last page is copied, and the tokens on it
};
struct Extend {
    ExtendList* lists;
    int32_t* copies;  // lists whose last page is copied
    int32_t* fresh;   // the free pages that the call takes, ascending
    int32_t* count;   // copies
};

static Extend extend_at(void* ws, long long total, long long lists, size_t* bytes) {
    unsigned char* base = (unsigned char*)ws;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    Extend e;
    e.lists = (ExtendList*)(base + take(sizeof(ExtendList) * (size_t)lists));
    e.copies = (int32_t*)(base + take(4 * (size_t)lists));
    e.fresh = (int32_t*)(base + take(4 * (size_t)total));
    e.count = (int32_t*)(base + take(4));
    if (bytes) *bytes = at;
    return e;
}
size_t extend_workspace_bytes(long long total, long long lists) {
    size_t n;
    extend_at(nullptr, total, lists, &n);
    return n;
}

__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const __grid_constant__ PagesArgs a,
                                                                   const __grid_constant__ Extend e, const int32_t* parent,
                                                                   const int32_t* extra) {
    __shared__ int sums[2][kPlanWarps], free_of[kPlanWarps];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int span = span_of(a.total), lo = min(a.total, warp * span), hi = min(a.total, lo + span);
    const int mine = hi - lo - used_pages(a.refs, lo, hi);
    if (lane == 0) free_of[warp] = mine;
    __syncthreads();
    int free_pages = 0, before = 0;  // free pages, those of the warps before
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) before += free_of[w];
        free_pages += free_of[w];
    }
    bool bad = false, full = false;
    int taken = 0, copies = 0;  // of the lists before
    long long asked = 0;        // pages that they asked for
    for (int i0 = 0; i0 < a.lists; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        ExtendList x = {0, 0, 0, 0, -1, -1, 0, 0};
        int need = 0;
        if (i < a.lists) {
            x.from = parent ? parent[i] : i;
            const int add = extra[i], own = a.len[i];
            if (x.from >= 0) {
                const bool fork = x.from != i;
                const long long most = (long long)a.wide * a.page;
                const int n = x.from < a.lists ? a.len[x.from] : -1;
                bool fine = n >= 0 && n <= most && add >= 0 && n + (long long)add <= most && (!fork || own == 0);
                if (fine) {
                    x.have = pages_of(n, a);
                    x.want = pages_of(n + add, a);
                    x.rows = n & (a.page - 1);
                    if (x.have > 0) {
                        x.last = a.pages[(long long)x.from * a.wide + x.have - 1];
                        fine = x.last >= 0 && x.last < a.total;
                        if (fine) x.copy = add > 0 && x.rows > 0 && (fork || a.refs[x.last] > 1);
                    }
                }
                if (fine) {
                    x.tokens = n + add;
                    need = x.want - x.have + x.copy;
                } else {
                    bad = true;
                }
            }
        }
        int all, all_copies;
        const long long upto = asked + block_sum(need, sums[0], &all);
        const bool fits = need == 0 || upto <= free_pages;
        if (!fits) {
            full = true;
            x.tokens = -1;
            x.copy = 0;
        }
        x.first = (int)min(upto - need, (long long)a.total);
        const int place = copies + block_sum(x.copy, sums[1], &all_copies) - x.copy;
        if (i < a.lists) {
            e.lists[i] = x;
            if (x.copy) e.copies[place] = i;
        }
        asked += all;
        copies += all_copies;
        __syncthreads();
    }
    // (an upper bound where some did not fit: more entries of fresh than are read)
    taken = (int)min(asked, (long long)free_pages);
    if (threadIdx.x == 0) *e.count = copies;
    if (mine > 0 && before < taken)
        for_pages(a.refs, lo, hi, [&](int p, int r, bool there) {
            const unsigned m = __ballot_sync(0xffffffffu, there && r <= 0);
            const int place = before + __popc(m & ((1u << lane) - 1u));
            if (there && r <= 0 && place < taken) e.fresh[place] = p;
            before += __popc(m);
        }, [&] { return before >= taken; });
    if (bad) atomicOr(&g_status_pages, FLAG_BOUNDS);
    if (full) atomicOr(&g_status_pages, FLAG_NOSPACE);
}

constexpr int kTablePart = 1024;  // entries of a table a CTA takes at a time

// CTAs of a moving kernel: no more than the most that `pages` moved pages and the tables can use.
static unsigned move_ctas(const PagesArgs& a, long long pages) {
    const long long items = pages * 2 * a.pool.layers + (long long)a.lists * (a.wide / kTablePart + 1);
    return (unsigned)(items < 1 ? 1 : items < kMoveCtas ? items : kMoveCtas);
}

__global__ void __launch_bounds__(kMoveThreads) extend_move_kernel(const __grid_constant__ PagesArgs a,
                                                                   const __grid_constant__ Extend e) {
    pdl_wait();
    bool bad = false;
    // page tables, lengths and counts
    const int parts = max(1, (a.wide + kTablePart - 1) / kTablePart);
    for (long long k = blockIdx.x; k < (long long)a.lists * parts; k += gridDim.x) {
        const int i = (int)(k / parts), part = (int)(k - (long long)i * parts);
        const ExtendList x = e.lists[i];
        if (x.tokens < 0) continue;
        const bool fork = x.from != i;
        const int kept = x.have - x.copy;  // entries taken over; then the copy and new pages
        int32_t* const table = a.pages + (long long)i * a.wide;
        const int32_t* const theirs = a.pages + (long long)x.from * a.wide;
        const int c1 = min(x.want, (part + 1) * kTablePart);
        for (int c = max(part * kTablePart, fork ? 0 : kept) + (int)threadIdx.x; c < c1; c += kMoveThreads) {
            int p;
            if (c < kept) {
                // (the parent's last page as it was on entry: it may be putting a copy there)
                p = c == x.have - 1 ? x.last : theirs[c];
                if (p >= 0 && p < a.total) atomicAdd(a.refs + p, 1);
                else bad = true;
            } else {
                p = e.fresh[x.first + c - kept];
                a.refs[p] = 1;
            }
            table[c] = p;
        }
        if (part == 0 && threadIdx.x == 0) {
            a.len[i] = x.tokens;
            if (x.copy && !fork) atomicSub(a.refs + x.last, 1);
        }
    }
    // rows of copied pages
    const int per = 2 * a.pool.layers;
    const long long items = (long long)*e.count * per;
    for (long long k = blockIdx.x; k < items; k += gridDim.x) {
        const int n = (int)(k / per), lp = (int)(k - (long long)n * per);
        const ExtendList x = e.lists[e.copies[n]];
        copy_page_rows(a, lp >> 1, lp & 1, x.last, e.fresh[x.first], x.rows);
    }
    if (bad) atomicOr(&g_status_pages, FLAG_BOUNDS);
}

// 40 lists (4 roots, 4 clones, 32 forks) with up to 24 rows of a page to copy in 32 layers of 8 x 128
// bf16, 155 MB read and written: 24 us, 18 of them the copies (their sources are few lists' pages and come
// from L2, so that is not what HBM moves); 64 lists that need 24 new pages and no copy: 8 us, two launches
// and the plan's four dependent loads.
cudaError_t launch_pages_extend(const PagesArgs& a, const int32_t* parent, const int32_t* extra, void* workspace,
                                cudaStream_t s) {
    if (a.lists == 0) return cudaSuccess;
    const Extend e = extend_at(workspace, a.total, a.lists, nullptr);
    const cudaError_t err = launch_chained(extend_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, e, parent, extra);
    if (err != cudaSuccess) return err;
    return launch_chained(extend_move_kernel, dim3(move_ctas(a, a.lists)), dim3(kMoveThreads), 0, s, a, e);
}

// ------------------------------------------------------------------ cut
// One cluster of CTAs per list: all of them read what the list keeps and move its rows, and the
// first gives its pages back once no other has the list's pages or length left to read (a cluster
// barrier in the place of a second kernel: 32 lists of up to 6 rows in 32 layers of 8 x 128 bf16,
// 38 MB read and written, 8.6 us, 4.4 TB/s, against 11.0; 48 int4 lists of 9 layers 6.9 against 8.3).
constexpr int kCutThreads = 384;
constexpr int kCutCtas = 8;    // of a cluster at most
constexpr int kCutRows = 128;  // rows whose places are in shared memory at a time

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A thread owns a column of a list's rows (16 bytes of a layer and plane, or a scale) and moves
// it row after row: row j comes from path[j] >= j, paths ascend, so no row is overwritten before
// it has been read, and no other thread touches the column.  Eight rows are in flight.
template <typename T>
__device__ __forceinline__ void cut_column(unsigned char* col, long long stride, const int* src, const int* dst, int rows) {
    constexpr int U = 8;
    for (int j = 0; j < rows; j += U) {
        T v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u < rows && src[j + u] >= 0) v[u] = *reinterpret_cast<const T*>(col + src[j + u] * stride);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u < rows && src[j + u] >= 0) *reinterpret_cast<T*>(col + dst[j + u] * stride) = v[u];
    }
}

__global__ void __launch_bounds__(kCutThreads, 2) cut_kernel(const __grid_constant__ PagesArgs a, const int32_t* base,
                                                             const int32_t* path, int max_path, const int32_t* kept, int ctas) {
    __shared__ int src[kCutRows], dst[kCutRows];
    pdl_wait();
    const int i = blockIdx.x / ctas, tid = threadIdx.x;
    const bool first = cluster_rank() == 0;
    const int keep = base[i], len = a.len[i], rows = kept ? kept[i] : 0;
    if (keep < 0 || (rows == 0 && !first)) return;
    bool fine = len >= 0 && len <= (long long)a.wide * a.page && keep <= len && rows >= 0 && rows <= max_path;
    if (fine)
        for (int j = tid; j < rows; j += kCutThreads) {
            const int32_t* p = path + (long long)i * max_path + j;
            fine = fine && *p > (j > 0 ? p[-1] : -1) && *p < len - keep;
        }
    // (every CTA of the cluster comes to the same answer)
    if (!__syncthreads_and(fine)) {
        if (first && tid == 0) atomicOr(&g_status_pages, FLAG_BOUNDS);
        return;
    }
    const PoolView& v = a.pool;
    const int row = v.heads * pool_head_bytes(v.format, v.dim) / 16;  // columns of codes, then of scales
    const int marks = v.format == KVFIX_POOL_BF16 ? 0 : v.format == KVFIX_POOL_E4M3 ? v.heads : v.heads * (v.dim / kQGroup);
    const long long columns = 2ll * v.layers * (row + marks);
    int32_t* const table = a.pages + (long long)i * a.wide;
    bool bad = false;
    for (int j0 = 0; j0 < rows; j0 += kCutRows) {
        const int n = min(kCutRows, rows - j0);
        __syncthreads();
        for (int j = tid; j < n; j += kCutThreads) {
            const int to = keep + j0 + j, from = keep + path[(long long)i * max_path + j0 + j];
            const int pf = table[from >> a.page_log], pt = table[to >> a.page_log], in = a.page - 1;
            const bool there = pf >= 0 && pf < a.total && pt >= 0 && pt < a.total;
            bad |= !there;
            src[j] = there && from != to ? pf * a.page + (from & in) : -1;
            dst[j] = there ? pt * a.page + (to & in) : -1;
        }
        __syncthreads();
        // the last places are known: nothing of the list's books is read any more
        if (j0 + n == rows) cluster_sync();
        for (long long col = (long long)(blockIdx.x - i * ctas) * kCutThreads + tid; col < columns; col += (long long)ctas * kCutThreads) {
            const int lp = (int)(col / (row + marks)), at = (int)(col - (long long)lp * (row + marks));
            const PoolPlane& pl = v.plane[lp & 1];
            const int layer = lp >> 1;
            if (at < row) {
                cut_column<uint4>(pl.codes + layer * v.sl + 16 * at, v.ss, src, dst, n);
            } else if (v.format == KVFIX_POOL_E4M3) {
                cut_column<unsigned char>(pl.scales + ((long long)layer * v.heads + at - row) * v.slots, 1, src, dst, n);
            } else {
                const int per = v.dim / kQGroup, h = (at - row) / per, q = at - row - h * per;
                cut_column<uint32_t>(pl.scales + 4 * (((long long)layer * v.heads + h) * v.slots * per + q), 4 * per, src, dst, n);
            }
        }
    }
    if (first) {
        const int end = keep + rows;
        for (int k = pages_of(end, a) + tid; k < pages_of(len, a); k += kCutThreads) {
            const int p = table[k];
            if (p < 0 || p >= a.total) {
                bad = true;
            } else if (atomicSub(a.refs + p, 1) <= 0) {
                atomicAdd(a.refs + p, 1);  // (nobody held it)
                bad = true;
            }
            table[k] = -1;
        }
        if (tid == 0) a.len[i] = end;
    }
    if (bad) atomicOr(&g_status_pages, FLAG_BOUNDS);
}

cudaError_t launch_pages_cut(const PagesArgs& a, const int32_t* base, const int32_t* path, int max_path,
                             const int32_t* kept, cudaStream_t s) {
    if (a.lists == 0) return cudaSuccess;
    // as many CTAs a list as give every thread a column, eight at most
    int ctas = 1;
    if (max_path > 0) {
        const PoolView& v = a.pool;
        const int per = v.format == KVFIX_POOL_BF16 ? 0 : v.format == KVFIX_POOL_E4M3 ? 1 : v.dim / kQGroup;
        const long long columns = 2ll * v.layers * v.heads * (pool_head_bytes(v.format, v.dim) / 16 + per);
        while (ctas < kCutCtas && (long long)ctas * kCutThreads < columns) ctas *= 2;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.lists * ctas));
    cfg.blockDim = dim3(kCutThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, cut_kernel, a, base, path, max_path, kept, ctas);
}

// ------------------------------------------------------------------ compact
struct Compact {
    int32_t* hole;   // [moves]: the free pages below the number of pages in use, ascending
    int32_t* mover;  // [moves]: the pages in use from there on, ascending
    int32_t* to;     // [total]: from there on, where a page goes (a free one: itself)
    int32_t* count;  // moves, pages in use
};
static Compact compact_at(void* ws, long long total, size_t* bytes) {
    unsigned char* base = (unsigned char*)ws;
    const size_t n = (4 * (size_t)total + 255) / 256 * 256;
    if (bytes) *bytes = 3 * n + 256;
    return {(int32_t*)base, (int32_t*)(base + n), (int32_t*)(base + 2 * n), (int32_t*)(base + 3 * n)};
}
size_t compact_workspace_bytes(long long total) {
    size_t n;
    compact_at(nullptr, total, &n);
    return n;
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ PagesArgs a,
                                                                    const __grid_constant__ Compact c, int32_t* live_out) {
    __shared__ int used_of[kPlanWarps], holes_of[kPlanWarps], movers_of[kPlanWarps];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int span = span_of(a.total), lo = min(a.total, warp * span), hi = min(a.total, lo + span);
    const int used = used_pages(a.refs, lo, hi);
    if (lane == 0) used_of[warp] = used;
    __syncthreads();
    int live = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) live += used_of[w];
    // pages in use below the border at `live`: all of a span before it, none of one behind
    const int border = min(max(live, lo), hi);
    const int below = border == hi ? used : border == lo ? 0 : used_pages(a.refs, lo, border);
    const int holes = border - lo - below, movers = used - below;
    if (lane == 0) {
        holes_of[warp] = holes;
        movers_of[warp] = movers;
    }
    __syncthreads();
    int at_hole = 0, at_mover = 0, moves = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) {
            at_hole += holes_of[w];
            at_mover += movers_of[w];
        }
        moves += movers_of[w];
    }
    for (int p = live + (int)threadIdx.x; p < a.total; p += kPlanThreads) c.to[p] = p;
    const unsigned lanes_below = (1u << lane) - 1u;
    const int holes_end = at_hole + holes, movers_end = at_mover + movers;
    for_pages(a.refs, lo, border, [&](int p, int r, bool there) {
        const unsigned m = __ballot_sync(0xffffffffu, there && r <= 0);
        if (there && r <= 0) c.hole[at_hole + __popc(m & lanes_below)] = p;
        at_hole += __popc(m);
    }, [&] { return at_hole >= holes_end; });
    for_pages(a.refs, border, hi, [&](int p, int r, bool) {
        const unsigned m = __ballot_sync(0xffffffffu, r > 0);
        if (r > 0) c.mover[at_mover + __popc(m & lanes_below)] = p;
        at_mover += __popc(m);
    }, [&] { return at_mover >= movers_end; });
    __syncthreads();
    for (int j = threadIdx.x; j < moves; j += kPlanThreads) c.to[c.mover[j]] = c.hole[j];
    if (threadIdx.x == 0) {
        c.count[0] = moves;
        c.count[1] = live;
        *live_out = live;
    }
}

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const __grid_constant__ PagesArgs a,
                                                                    const __grid_constant__ Compact c) {
    pdl_wait();
    const int moves = c.count[0], live = c.count[1];
    bool bad = false;
    const int parts = max(1, (a.wide + kTablePart - 1) / kTablePart);
    // (also where nothing moves: lists and entries out of range are flagged)
    for (long long k = blockIdx.x; k < (long long)a.lists * parts; k += gridDim.x) {
        const int i = (int)(k / parts), part = (int)(k - (long long)i * parts);
        const int n = a.len[i];
        if (n < 0 || n > (long long)a.wide * a.page) {
            bad = true;
            continue;
        }
        int32_t* const table = a.pages + (long long)i * a.wide;
        const int c1 = min(pages_of(n, a), (part + 1) * kTablePart);
        for (int x = part * kTablePart + threadIdx.x; x < c1; x += kMoveThreads) {
            const int p = table[x];
            if (p < 0 || p >= a.total) bad = true;
            else if (p >= live) table[x] = c.to[p];
        }
    }
    for (int j = blockIdx.x * kMoveThreads + threadIdx.x; j < moves; j += gridDim.x * kMoveThreads) {
        const int from = c.mover[j];
        a.refs[c.hole[j]] = a.refs[from];
        a.refs[from] = 0;
    }
    const int per = 2 * a.pool.layers;
    const long long items = (long long)moves * per;
    for (long long k = blockIdx.x; k < items; k += gridDim.x) {
        const int j = (int)(k / per), lp = (int)(k - (long long)j * per);
        copy_page_rows(a, lp >> 1, lp & 1, c.mover[j], c.hole[j], a.page);
    }
    if (bad) atomicOr(&g_status_pages, FLAG_BOUNDS);
}

// 245 pages of 32 tokens in 32 layers of 8 x 128 e4m3 (1.04 GB read and written): 168 to 175 us from run
// to run, 5.9 to 6.2 TB/s.
cudaError_t launch_pages_compact(const PagesArgs& a, int32_t* live, void* workspace, cudaStream_t s) {
    const Compact c = compact_at(workspace, a.total, nullptr);
    const cudaError_t e = launch_chained(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, c, live);
    if (e != cudaSuccess) return e;
    return launch_chained(compact_move_kernel, dim3(move_ctas(a, a.total)), dim3(kMoveThreads), 0, s, a, c);
}

}  // namespace kvfix
