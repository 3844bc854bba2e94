// attend.cu -- kvfix_shared_attend: attention of a round's agents over a shared prefix and
// their own tokens, straight from a paged pool.
//
// Mathematics.  The keys of a query lie in two segments, its group's prefix and its agent's
// suffix.  Softmax over their union is joined from parts: a part (any set of keys) keeps per
// query row m = max z, l = sum exp(z - m) and O = sum exp(z - m) v; parts join as
// M = max m, L = sum l exp(m - M), out = sum O exp(m - M) / L, lse = M + log L.  So a
// segment's keys can be read once for all the query rows that see it (rows of all agents of
// the group, all new tokens, all query heads of a KV head), and a long segment can be cut
// anywhere.
//
// Work.  An entry is a block of up to 256 rows of a segment; a unit is an entry and a KV
// head; its work is ceil(keys / 128) tiles of 128 keys (causally trimmed), plus one for its
// fixed cost.  One plan kernel lays all units on a line; CTA i of the persistent grid takes
// the i-th equal piece of it, whole units and parts of units alike, and writes one part per
// unit it touches; the join kernel finds a row's parts from the same line.  Everything
// depends on lengths that lie on the device, so a captured graph follows them.
//
// The attention kernel is bound by HBM for decode (a group's rows fill up to 256 lanes of the
// MMA per key read) and by the tensor pipe and the exponentials for many new tokens:
//   warps 0-3, 4-7  softmax: each group owns one 128-row accumulator.  Blocks of more than
//                   128 rows give each group its half of the rows and both use every tile;
//                   smaller blocks give both groups the same rows and alternate tiles.  A
//                   thread owns a row (a TMEM lane): no cross-lane reduction.
//   warp 8          TMA producer: pages of K and V tiles (128 keys x D) into a ring.
//   warps 12-15     (stored forms) converters: code tiles and their scales, loaded as they lie,
//                   to bf16 tiles for the MMA.
//   warp 9          one thread issues tcgen05.mma: S = Q K^T (both K-major in shared memory)
//                   and O += P V with P from tensor memory and V read N-major as it lies.
// S occupies 128 TMEM columns per group, P (bf16) overwrites the first half of S, O takes D.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attend.h"
#include "pool.cuh"
#include "tc.cuh"

namespace kvfix {

static __device__ unsigned int g_status_attend;

unsigned read_status_attend(cudaStream_t stream) {
    unsigned h = 0, zero = 0;
    cudaMemcpyFromSymbolAsync(&h, g_status_attend, sizeof h, 0, cudaMemcpyDeviceToHost, stream);
    cudaMemcpyToSymbolAsync(g_status_attend, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    cudaStreamSynchronize(stream);
    return h;
}

constexpr int kAtKeys = 128;      // keys per tile
constexpr int kAtRows = 128;      // rows per accumulator (MMA M)
constexpr int kAtBlock = 256;     // rows per entry
constexpr int kAtMaxCtas = 256;   // bound of the persistent grid

// ------------------------------------------------------------------ plan
// The line of units.  Entries of a segment are its 256-row blocks in order; segments are the
// groups' prefixes, then the agents' suffixes.  Unit (entry e, head h) begins at
// begin + h * (tiles + 1).
struct __align__(16) AtEntry {
    long long begin;  // position of head 0 on the line
    long long prow;   // part rows of head 0
    int tiles, rows, row0, seg;
    int keys;         // keys of the segment that some row of the block may see
    int agent0;       // the segment's first agent
    int prefix;       // 1: a group's prefix
    int pad;
};

struct AtPlan {
    long long total;  // length of the line
    int entries, pad;
    int start[kAtMaxCtas];  // the entry in which a CTA's piece begins
};

struct AtLayout {
    size_t plan, first, bounds, entries, ml, o, bytes;
    long long own_rows;
};

// Part rows: each unit's first part has its own rows (two sets where both softmax groups hold
// the same rows), a part that continues a unit from an earlier CTA has its CTA's 256 rows.
static AtLayout at_layout(int agents, int T, int q_heads, int kv_heads, int head_dim, int groups) {
    const long long tg = (long long)T * (q_heads / kv_heads), all = (long long)agents * tg;
    const long long small = tg < kAtRows ? tg : kAtRows;
    const long long entries = groups + all / kAtBlock + (long long)agents * ((tg + kAtBlock - 1) / kAtBlock) + 1;
    long long extra = (long long)kAtRows * groups;
    if (extra > all) extra = all;
    AtLayout l;
    l.own_rows = kv_heads * (all + extra + agents * (tg + small));
    const long long rows = l.own_rows + (long long)kAtMaxCtas * kAtBlock;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    l.plan = take(sizeof(AtPlan));
    l.first = take(4 * ((size_t)groups + agents));
    l.bounds = take(4 * ((size_t)groups + 1));
    l.entries = take(sizeof(AtEntry) * (size_t)entries);
    l.ml = take(8 * (size_t)rows);
    l.o = take(4 * (size_t)rows * head_dim);
    l.bytes = at;
    return l;
}

size_t attend_workspace_bytes(int agents, int T, int q_heads, int kv_heads, int head_dim, int groups) {
    return at_layout(agents, T, q_heads, kv_heads, head_dim, groups).bytes;
}

struct AtWork {
    AtPlan* plan;
    int* first;   // [groups + agents]: a segment's first entry
    int* bounds;  // [groups + 1]: the groups' agents, clamped and ascending
    AtEntry* entries;
    float2* ml;   // part rows: (max in base-2 units, sum)
    float* o;     // part rows x D
    long long own_rows;
    int ctas;
};

// The piece of the line that CTA i of n takes.
__host__ __device__ __forceinline__ long long piece(long long total, int i, int n) {
    return total / n * i + total % n * i / n;
}

__device__ __forceinline__ int clamp_len(int n, long long most, bool& bad) {
    if (n < 0 || n > most) bad = true;
    return (int)min(max((long long)n, 0ll), most);
}

constexpr int kPlanThreads = 512;

// Exclusive scan over the block of three sums and an (inclusive) running maximum.
struct PlanSums {
    long long entries, line, rows;
};
__device__ __forceinline__ PlanSums plan_scan(PlanSums x, PlanSums* warp_sums, PlanSums* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PlanSums inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, inc.entries, o);
        const long long b = __shfl_up_sync(0xffffffffu, inc.line, o);
        const long long c = __shfl_up_sync(0xffffffffu, inc.rows, o);
        if (lane >= o) {
            inc.entries += a;
            inc.line += b;
            inc.rows += c;
        }
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    PlanSums before = {0, 0, 0}, all = {0, 0, 0};
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const PlanSums s = warp_sums[w];
        if (w < warp) {
            before.entries += s.entries;
            before.line += s.line;
            before.rows += s.rows;
        }
        all.entries += s.entries;
        all.line += s.line;
        all.rows += s.rows;
    }
    *total = all;
    PlanSums ex;
    ex.entries = before.entries + inc.entries - x.entries;
    ex.line = before.line + inc.line - x.line;
    ex.rows = before.rows + inc.rows - x.rows;
    return ex;
}

__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const __grid_constant__ AttendArgs a, AtWork w) {
    __shared__ PlanSums warp_sums[kPlanThreads / 32];
    __shared__ int warp_max[kPlanThreads / 32];
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G, H = a.pool.heads;
    const int segs = a.groups + a.agents;
    const int per = (segs + kPlanThreads - 1) / kPlanThreads;
    const int s0 = min(segs, tid * per), s1 = min(segs, s0 + per);
    const long long most_p = (long long)a.max_prefix_pages * a.page, most_s = (long long)a.max_suffix_pages * a.page;
    bool bad = false;
    // group bounds: the running maximum of the given ones, kept within 0..agents
    if (a.groups > 0) {
        const int n = a.groups + 1, each = (n + kPlanThreads - 1) / kPlanThreads;
        const int g0 = min(n, tid * each), g1 = min(n, g0 + each);
        int mine = 0;
        for (int g = g0; g < g1; ++g) mine = max(mine, min(max(a.group_begin[g], 0), a.agents));
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc = max(inc, y);
        }
        if (lane == 31) warp_max[warp] = inc;
        __syncthreads();
        int run = 0;
        for (int x = 0; x < warp; ++x) run = max(run, warp_max[x]);
        const int left = __shfl_up_sync(0xffffffffu, inc, 1);
        if (lane > 0) run = max(run, left);
        for (int g = g0; g < g1; ++g) {
            const int b = a.group_begin[g];
            if (b < run || b > a.agents) bad = true;
            run = max(run, min(max(b, 0), a.agents));
            w.bounds[g] = run;
        }
        __syncthreads();
    }
    // one segment: rows, keys; its blocks in turn
    auto each_block = [&](int s, auto&& f) {
        const bool prefix = s < a.groups;
        const int agent0 = prefix ? w.bounds[s] : s - a.groups;
        const int count = prefix ? w.bounds[s + 1] - agent0 : 1;
        const int n = prefix ? clamp_len(a.prefix_len[s], most_p, bad) : clamp_len(a.suffix_len[agent0], most_s, bad);
        const int rows = count * TG;
        for (int r0 = 0; r0 < rows; r0 += kAtBlock) {
            AtEntry e;
            e.rows = min(kAtBlock, rows - r0);
            e.row0 = r0;
            e.seg = s;
            e.agent0 = agent0;
            e.prefix = prefix;
            // own keys are seen up to the place of the block's last row
            e.keys = prefix ? n : max(0, n - T + 1 + (r0 + e.rows - 1) / G);
            e.tiles = (e.keys + kAtKeys - 1) / kAtKeys;
            e.pad = 0;
            f(e);
        }
    };
    auto set_rows = [](const AtEntry& e) { return e.rows > kAtRows ? e.rows : 2 * e.rows; };
    auto cost = [&](const AtEntry& e) { return e.tiles > 0 ? (long long)H * (e.tiles + 1) : 0ll; };
    PlanSums mine = {0, 0, 0};
    for (int s = s0; s < s1; ++s)
        each_block(s, [&](const AtEntry& e) {
            mine.entries += 1;
            mine.line += cost(e);
            mine.rows += (long long)H * set_rows(e);
        });
    PlanSums total;
    PlanSums at = plan_scan(mine, warp_sums, &total);
    for (int s = s0; s < s1; ++s) {
        w.first[s] = (int)at.entries;
        each_block(s, [&](AtEntry e) {
            e.begin = at.line;
            e.prow = at.rows;
            const long long c = cost(e);
            w.entries[at.entries] = e;
            // the CTAs whose pieces begin inside this entry
            if (c > 0) {
                long long i = total.line ? at.line * w.ctas / total.line : 0;
                while (i > 0 && piece(total.line, (int)i, w.ctas) >= at.line) --i;
                while (i < w.ctas && piece(total.line, (int)i, w.ctas) < at.line) ++i;
                for (; i < w.ctas && piece(total.line, (int)i, w.ctas) < at.line + c; ++i) w.plan->start[i] = (int)at.entries;
            }
            at.entries += 1;
            at.line += c;
            at.rows += (long long)H * set_rows(e);
        });
    }
    if (tid == 0) {
        w.plan->total = total.line;
        w.plan->entries = (int)total.entries;
    }
    if (bad) atomicOr(&g_status_attend, FLAG_BOUNDS);
}

// A CTA's units in order.
struct AtUnit {
    int e, head, t0, nt, rows, row0, seg, keys, agent0, prefix;
    long long part;  // first part row
};

struct AtWalk {
    const AtEntry* ent;
    const AtEntry* end;
    long long lo, hi, cta_part, own;
    int H, e, h;
    AtEntry rec;
    bool have;

    __device__ __forceinline__ void open(const AtWork& w, int heads, int cta) {
        const long long total = w.plan->total;
        lo = piece(total, cta, w.ctas);
        hi = piece(total, cta + 1, w.ctas);
        ent = w.entries;
        H = heads;
        e = lo < hi ? w.plan->start[cta] : 0;
        have = lo < hi;
        if (have) {
            rec = ent[e];
            h = (int)((lo - rec.begin) / (rec.tiles + 1));
        }
        end = ent + w.plan->entries;
        cta_part = w.own_rows + (long long)cta * kAtBlock;
    }

    __device__ __forceinline__ bool next(AtUnit& u) {
        while (have) {
            const long long c = rec.tiles + 1, base = rec.begin + (long long)h * c;
            if (rec.tiles == 0 || h >= H) {
                ++e;
                h = 0;
                if (ent + e >= end) have = false;
                else {
                    rec = ent[e];
                    if (rec.tiles > 0 && rec.begin >= hi) have = false;
                }
                continue;
            }
            if (base >= hi) {
                have = false;
                continue;
            }
            const int t0 = (int)max(0ll, lo - base), t1 = (int)min((long long)rec.tiles, hi - base);
            const int head = h++;
            if (t0 >= t1) continue;
            u.e = e;
            u.head = head;
            u.t0 = t0;
            u.nt = t1 - t0;
            u.rows = rec.rows;
            u.row0 = rec.row0;
            u.seg = rec.seg;
            u.keys = rec.keys;
            u.agent0 = rec.agent0;
            u.prefix = rec.prefix;
            u.part = t0 == 0 ? rec.prow + (long long)head * (rec.rows > kAtRows ? rec.rows : 2 * rec.rows) : cta_part;
            return true;
        }
        return false;
    }
};

// ------------------------------------------------------------------ attention
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D[tmem] (+)= A[tmem] * B[smem], bf16, B as the instruction descriptor says.
__device__ __forceinline__ void tc_mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// B N-major (bit 16): keys are the contraction, a value row is contiguous along N.
__host__ __device__ constexpr uint32_t at_idesc_pv(int N) { return tc_idesc_bf16(kAtRows, N) | (1u << 16); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Registers move from the issuing and converting warpgroups to the softmax ones, whose threads
// hold a row of logits (setmaxnreg: the shares add up to what the block launches with).
template <int F, int D>
struct AtCfg {
    static constexpr bool kQuant = F != KVFIX_POOL_BF16;
    static constexpr int kThreads = kQuant ? 512 : 384;
    static constexpr int kRegsSoftmax = kQuant ? 168 : 208;
    static constexpr int kRegsOther = 88;
    static constexpr int kTile = kAtKeys * D * 2;   // a K or V tile as bf16
    static constexpr int kQ = kAtRows * D * 2;
    static constexpr int kStages = kQuant ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
    // stored tiles before conversion: codes, then scales
    static constexpr int kCodeRow = pool_head_bytes(F, D);
    static constexpr int kScaleRow = F == KVFIX_POOL_E4M3 ? 1 : F == KVFIX_POOL_INT4 ? D / 8 : 0;
    static constexpr int kRaw = kQuant ? kAtKeys * (kCodeRow + kScaleRow) : 0;
    static constexpr int kRawStages = kQuant ? (F == KVFIX_POOL_E4M3 ? 4 : 6) : 1;
    static constexpr int kSmem = 1024 + kStages * kTile + 2 * kQ + (kQuant ? kRawStages * kRaw : 0);
    static_assert(kSmem <= 231 * 1024, "shared memory");
};
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One stored tile (codes [128][kCodeRow], scales [128][kScaleRow]) to the bf16 tile the MMA
// reads: rows of 128 bytes per 64-column half, 128-byte swizzle.  Rows that hold no key
// (`gone`) become zero.  A thread takes 16 code bytes at a time; the order in which it writes
// their 16-byte chunks puts the eight threads of a store phase on different banks.
template <int F, int D, int N>
__device__ __forceinline__ void convert_tile(const unsigned char* raw, unsigned char* tile, int tid, int in_tile,
                                             unsigned absent, int page_shift) {
    using C = AtCfg<F, D>;
    constexpr int V = C::kCodeRow / 16;  // vectors per row
    const unsigned char* scales = raw + kAtKeys * C::kCodeRow;
#pragma unroll 4
    for (int i = tid; i < kAtKeys * V; i += N) {
        const int r = i / V, v = i % V;
        const bool gone = r >= in_tile || ((absent >> (r >> (4 + page_shift))) & 1u);
        const uint4 x = *reinterpret_cast<const uint4*>(raw + 16 * i);
        const unsigned c[4] = {x.x, x.y, x.z, x.w};
        if (F == KVFIX_POOL_E4M3) {
            const E4m3Scale sc = e4m3_scale(min(max((int)scales[r] - 127, kE4m3MinExp), kE4m3MaxExp));
            uint2 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = e4m3x4_to_bf16(c[k], sc);
            unsigned nan = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) nan |= ((c[k] & 0x7f7f7f7fu) + 0x01010101u);
            if (nan & 0x80808080u)
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = e4m3x4_nan(c[k], w[k]);
            uint4 o[2] = {make_uint4(w[0].x, w[0].y, w[1].x, w[1].y), make_uint4(w[2].x, w[2].y, w[3].x, w[3].y)};
            if (gone) o[0] = o[1] = make_uint4(0u, 0u, 0u, 0u);
            unsigned char* dst = tile + (v / 4) * (kAtKeys * 128) + r * 128;
            const int first = (v / 4) & 1;
            const int c0 = 2 * (v % 4);
            *reinterpret_cast<uint4*>(dst + (((c0 + first) ^ (r & 7)) << 4)) = first ? o[1] : o[0];
            *reinterpret_cast<uint4*>(dst + (((c0 + 1 - first) ^ (r & 7)) << 4)) = first ? o[0] : o[1];
        } else {
            const unsigned sz = *reinterpret_cast<const unsigned*>(scales + r * C::kScaleRow + 4 * v);
            const unsigned ss = __byte_perm(sz, 0u, 0x1010), zz = __byte_perm(sz, 0u, 0x3232);
            unsigned char* dst = tile + (v / 2) * (kAtKeys * 128) + r * 128;
            uint4 o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o[k] = int4x8_to_bf16(c[k], *reinterpret_cast<const __nv_bfloat162*>(&ss),
                                      *reinterpret_cast<const __nv_bfloat162*>(&zz));
                if (gone) o[k] = make_uint4(0u, 0u, 0u, 0u);
            }
            const bool swap = (v / 2) & 1;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(dst + (((4 * (v % 2) + (swap ? k ^ 2 : k)) ^ (r & 7)) << 4)) = swap ? o[k ^ 2] : o[k];
        }
    }
}

// A row's maximum is raised (and its accumulator rescaled) once a logit passes it by more
// than this many powers of two: weights stay below 2^8, and bf16 keeps 8 bits of any of them.
constexpr float kAtSlack = 8.f;

template <int F, int D>
__global__ void __launch_bounds__(AtCfg<F, D>::kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ AttendArgs a, const __grid_constant__ AtWork w) {
    using C = AtCfg<F, D>;
    constexpr int S = C::kStages, R = C::kRawStages;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[S], empty[S], q_ready[2], s_full[2], p_ready[2], o_full[2];
    __shared__ __align__(8) uint64_t raw_full[R], raw_empty[R];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* qsm = smem + S * C::kTile;
    unsigned char* rawsm = qsm + 2 * C::kQ;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], C::kQuant ? 128 : 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < R; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_ready[i], 128);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 128);
            mbar_init(&o_full[i], 1);
        }
        fence_mbar_init();
        abort_flag = 0;
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (warp == 9) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    pdl_trigger();
    const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G;
    AtWalk walk;
    walk.open(w, a.pool.heads, blockIdx.x);
    AtUnit u;
    const int ppt = kAtKeys / a.page;  // pages per tile
    const int pool_pages = a.pool.slots / a.page;
    const int page_shift = 31 - __clz(a.page / 16);

    auto page_list = [&](const AtUnit& x) {
        return x.prefix ? a.prefix_pages + (long long)x.seg * a.max_prefix_pages
                        : a.suffix_pages + (long long)x.agent0 * a.max_suffix_pages;
    };
    // lanes of a warp look at a tile's pages: which of those that hold keys are not there
    auto page_ok = [&](const AtUnit& x, const int32_t* pages, int tile) {
        const int i = tile * ppt + lane;
        if (lane >= ppt || i >= (x.keys + a.page - 1) / a.page) return true;
        const int p = __ldg(pages + i);
        return p >= 0 && p < pool_pages;
    };

    if (warp >= 8) {
    regs_dec<C::kRegsOther>();
    if (warp == 8) {
        // ---------------------------------------------------------------- producer
        // a lane per copy: its page of the tile, and its 64-column half (bf16), or codes and
        // scales (stored forms)
        uint64_t* const ring_full = C::kQuant ? raw_full : full;
        uint64_t* const ring_empty = C::kQuant ? raw_empty : empty;
        constexpr int N = C::kQuant ? R : S;
        const int my = lane % ppt, part = lane / ppt;
        const bool live = part < (C::kQuant ? 2 : D / 64);
        const unsigned page_bytes = (unsigned)a.page * (C::kQuant ? C::kCodeRow + C::kScaleRow : 2 * D);
        bool ok = true, bad = false;
        unsigned item = 0;  // tiles issued (K and V of a tile are two)
        while (ok && walk.next(u)) {
            const int32_t* pages = page_list(u);
            const int used = (u.keys + a.page - 1) / a.page;  // page entries that hold keys
            auto page_of = [&](int tile) {
                const int i = tile * ppt + my;
                return live && i < used ? __ldg(pages + i) : -2;
            };
            int page = page_of(u.t0);
            for (int t = 0; t < u.nt && ok; ++t) {
                const int ahead = t + 1 < u.nt ? page_of(u.t0 + t + 1) : -2;
                const bool good = page >= 0 && page < pool_pages;
                if (page != -2 && !good) bad = true;
                const int boxes = __popc(__ballot_sync(0xffffffffu, good && part == 0));
#pragma unroll
                for (int p = 0; p < 2 && ok; ++p, ++item) {
                    const int st = item % N;
                    if (item >= N) ok = mbar_wait(&ring_empty[st], (item / N - 1) & 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&ring_full[st], (unsigned)boxes * page_bytes);
                    __syncwarp();
                    if (good) {
                        if (!C::kQuant) {
                            tma_load_2d(smem + st * C::kTile + part * (kAtKeys * 128) + my * a.page * 128,
                                        p ? &tm_v : &tm_k, u.head * D + 64 * part, page * a.page, &ring_full[st]);
                        } else if (part == 0) {
                            tma_load_2d(rawsm + st * C::kRaw + my * a.page * C::kCodeRow, p ? &tm_v : &tm_k,
                                        u.head * C::kCodeRow, page * a.page, &ring_full[st]);
                        } else {
                            bulk_g2s(rawsm + st * C::kRaw + kAtKeys * C::kCodeRow + my * a.page * C::kScaleRow,
                                     a.pool.plane[p].scales +
                                         ((long long)u.head * a.pool.slots + (long long)page * a.page) * C::kScaleRow,
                                     (unsigned)a.page * C::kScaleRow, &ring_full[st]);
                        }
                    }
                }
                page = ahead;
            }
        }
        if (!ok) {
            // the copies in flight land before this block gives up its shared memory
            for (unsigned i = item > N ? item - N : 0; i < item; ++i) mbar_wait(&ring_full[i % N], (i / N) & 1u);
            if (lane == 0) atomicOr(&abort_flag, 1);
        }
        if (bad) atomicOr(&g_status_attend, FLAG_BOUNDS);
    } else if (C::kQuant && warp >= 12) {
        // ---------------------------------------------------------------- conversion
        bool ok = true;
        unsigned item = 0;
        while (ok && walk.next(u)) {
            const int32_t* pages = page_list(u);
            bool pg = page_ok(u, pages, u.t0);
            for (int t = 0; t < u.nt && ok; ++t) {
                const unsigned absent = ~__ballot_sync(0xffffffffu, pg);
                if (t + 1 < u.nt) pg = page_ok(u, pages, u.t0 + t + 1);
                const int in_tile = min(kAtKeys, u.keys - (u.t0 + t) * kAtKeys);
                for (int p = 0; p < 2; ++p, ++item) {
                    const int rs = item % R, st = item % S;
                    ok = mbar_wait(&raw_full[rs], (item / R) & 1u);
                    if (ok && item >= S) ok = mbar_wait(&empty[st], (item / S - 1) & 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    convert_tile<F, D, 128>(rawsm + rs * C::kRaw, smem + st * C::kTile, threadIdx.x - 384, in_tile, absent,
                                            page_shift);
                    mbar_arrive(&raw_empty[rs]);
                    fence_proxy_async_smem();
                    mbar_arrive(&full[st]);
                }
            }
        }
        if (!ok && lane == 0) atomicOr(&abort_flag, 1);
    } else if (warp == 9) {
        // ---------------------------------------------------------------- MMA issue
        if (lane == 0) {
            constexpr uint32_t id_qk = tc_idesc_bf16(kAtRows, kAtKeys), id_pv = at_idesc_pv(D);
            // descriptors of the first query block and the first stage (as keys, K-major, and as
            // values, N-major: 64-column halves 16 KB apart, 8-key groups 1 KB apart); an offset
            // adds to the address field, which all of shared memory fits
            const uint64_t q_desc = tc_smem_desc(qsm, 16, 1024, 2), t_desc = tc_smem_desc(smem, 16, 1024, 2);
            const uint64_t v_desc = tc_smem_desc(smem, kAtKeys * 128, 1024, 2);
            bool ok = true;
            unsigned item = 0, nq = 0, np = 0;  // phase bits by group
            while (ok && walk.next(u)) {
                const bool two = u.rows > kAtRows;
                const int jobs = two ? 2 * u.nt : u.nt;
                for (int j = 0; j <= jobs && ok; ++j) {
                    if (j < jobs) {
                        const int g = j & 1, tile = two ? j >> 1 : j;
                        const unsigned it = item + 2 * tile, st = it % S;
                        if (j < 2) {
                            ok = mbar_wait(&q_ready[g], (nq >> g) & 1u);
                            nq ^= 1u << g;
                        }
                        if (ok && (!two || g == 0)) ok = mbar_wait(&full[st], (it / S) & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = q_desc + (uint32_t)(g * C::kQ >> 4), bd = t_desc + st * (uint32_t)(C::kTile >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t at = ((kk / 4) * (kAtKeys * 128) + 32 * (kk % 4)) >> 4;
                            tc_mma_bf16(tmem + 128 * g, ad + at, bd + at, id_qk, kk > 0 ? 1u : 0u);
                        }
                        if (!two || g == 1) tc_commit(&empty[st]);
                        tc_commit(&s_full[g]);
                    }
                    if (j > 0) {
                        const int i = j - 1, g = i & 1, tile = two ? i >> 1 : i;
                        const unsigned it = item + 2 * tile + 1, st = it % S;
                        ok = mbar_wait(&p_ready[g], (np >> g) & 1u);
                        np ^= 1u << g;
                        if (ok && (!two || g == 0)) ok = mbar_wait(&full[st], (it / S) & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t bd = v_desc + st * (uint32_t)(C::kTile >> 4);
#pragma unroll
                        for (int kk = 0; kk < kAtKeys / 16; ++kk)
                            tc_mma_bf16_ta(tmem + 256 + 128 * g, tmem + 128 * g + 8 * kk, bd + (uint32_t)(2048 * kk >> 4),
                                           id_pv, (i > 1 || kk > 0) ? 1u : 0u);
                        if (!two || g == 1) tc_commit(&empty[st]);
                        if (i + 2 >= jobs) tc_commit(&o_full[g]);
                    }
                }
                item += 2 * u.nt;
            }
            if (!ok) atomicOr(&abort_flag, 1);
        }
    }
    } else {
        regs_inc<C::kRegsSoftmax>();
        // ---------------------------------------------------------------- softmax
        const int g = warp >> 2, wq = warp & 3, row = 32 * wq + lane;  // group, TMEM lane quarter, row
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t s_at = tmem + lanes + 128 * g, o_at = tmem + lanes + 256 + 128 * g;
        unsigned char* qt = qsm + g * C::kQ;
        const float c = a.scale_log2;
        bool ok = true;
        unsigned item = 0, ns = 0, no = 0;
        while (ok && walk.next(u)) {
            const bool two = u.rows > kAtRows;
            const int r0 = two ? kAtRows * g : 0;                    // the group's rows of the block
            const int rows = min(kAtRows, u.rows - r0);
            const int jobs = two ? u.nt : (u.nt + 1 - g) / 2;        // tiles of this group
            const long long part = u.part + (two ? r0 : g * u.rows);
            if (jobs == 0) {
                if (row < rows) w.ml[part + row] = make_float2(-INFINITY, 0.f);
                item += 2 * u.nt;
                continue;
            }
            // the group's queries, K-major with the 128-byte swizzle
            {
                constexpr int V = D / 8;  // 16-byte vectors per row
                const int tg = threadIdx.x & 127, cv = tg % V;
#pragma unroll 8
                for (int i = 0; i < V; ++i) {
                    const int r = tg / V + i * (128 / V);
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (r < rows) {
                        const int at = u.row0 + r0 + r, ag = at / TG, in = at - ag * TG, t = in / G;
                        x = __ldg(reinterpret_cast<const uint4*>(
                            a.q + a.qp.row(u.agent0 + ag, 0, t) + (long long)(u.head * G + in - t * G) * D + 8 * cv));
                    }
                    *reinterpret_cast<uint4*>(qt + (cv / 8) * (kAtRows * 128) + r * 128 + (((cv % 8) ^ (r & 7)) << 4)) = x;
                }
                fence_proxy_async_smem();
                mbar_arrive(&q_ready[g]);
            }
            // keys this thread's row sees, from the segment's first
            int sees = 0;
            if (row < rows) {
                const int at = u.row0 + r0 + row, ag = at / TG, t = (at - ag * TG) / G;
                const int place = t + 1 - T;
                if (u.prefix) {
                    bool ignore = false;
                    const int own = clamp_len(a.suffix_len[u.agent0 + ag], (long long)a.max_suffix_pages * a.page, ignore);
                    sees = max(0, min(u.keys, u.keys + own + place));
                } else {
                    // u.keys holds the places seen by the block's last row
                    sees = max(0, u.keys + t - (u.row0 + u.rows - 1) / G);
                }
            }
            const bool warp_live = 32 * wq < rows;
            const int32_t* pages = page_list(u);
            const int step = two ? 1 : 2;
            bool pg = page_ok(u, pages, u.t0 + (two ? 0 : g));
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < jobs; ++j) {
                const int tl = two ? j : 2 * j + g, tile = u.t0 + tl;
                const unsigned absent = ~__ballot_sync(0xffffffffu, pg);  // pages of the tile that are not there
                if (j + 1 < jobs) pg = page_ok(u, pages, tile + step);
                const int in_tile = min(kAtKeys, u.keys - tile * kAtKeys);  // keys of the segment in the tile
                const bool whole = absent == 0u && in_tile == kAtKeys;
                ok = mbar_wait(&s_full[g], ns++ & 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (!C::kQuant && !whole) {
                    // value rows that hold no key read as zero: a weight of 0 times what lies
                    // there (anything, NaN too) would not be 0
                    const unsigned it = item + 2 * tl + 1, st = it % S;
                    ok = mbar_wait(&full[st], (it / S) & 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (row >= in_tile || ((absent >> (row / a.page)) & 1u)) {
                        unsigned char* vt = smem + st * C::kTile + row * 128;
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4*>(vt + h * (kAtKeys * 128) + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                if (warp_live) {
                    uint32_t sv[128];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, sv + 32 * i);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_wait_ld32(sv + 32 * i);
                    const int nv = sees - tile * kAtKeys;  // columns this row sees
                    if (!whole || __any_sync(0xffffffffu, nv < kAtKeys)) {
#pragma unroll
                        for (int b = 0; b < 8; ++b) {  // 16 columns: part of one page
                            const int n = (absent >> (b >> page_shift)) & 1u ? 0 : nv - 16 * b;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (i >= n) sv[16 * b + i] = 0xff800000u;  // -inf
                        }
                    }
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(sv[i]);
#pragma unroll
                    for (int i = 4; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(sv[i]));
                    const float z = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                    const bool raise = z > m + kAtSlack || (m == -INFINITY && z > m);
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? ex2(m - z) : 1.f;  // m = -inf: 0
                        if (raise) {
                            m = z;
                            l *= f;
                        }
                        if (j > 0) {
#pragma unroll
                            for (int i = 0; i < D / 32; ++i) {
                                uint32_t o[32];
                                tmem_ld32(o_at + 32 * i, o);
                                tmem_wait_ld32(o);
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st32(o_at + 32 * i, o);
                            }
                        }
                    }
                    const float off = m == -INFINITY ? 0.f : -m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t pk[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float x = ex2(__fmaf_rn(__uint_as_float(sv[64 * i + 2 * k]), c, off));
                            const float y = ex2(__fmaf_rn(__uint_as_float(sv[64 * i + 2 * k + 1]), c, off));
                            sum[(2 * k) & 3] += x;
                            sum[(2 * k + 1) & 3] += y;
                            pk[k] = pack_bf16(x, y);
                        }
                        tmem_st32(s_at + 32 * i, pk);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&p_ready[g]);
            }
            if (!ok) break;
            ok = mbar_wait(&o_full[g], no++ & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (warp_live) {
                float* out = w.o + (part + row) * D;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t o[32];
                    tmem_ld32(o_at + 32 * i, o);
                    tmem_wait_ld32(o);
                    if (row < rows)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<uint4*>(out + 32 * i + 4 * k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
                if (row < rows) w.ml[part + row] = make_float2(m, l);
                tc_fence_before();
            }
            item += 2 * u.nt;
        }
        if (!ok && lane == 0) atomicOr(&abort_flag, 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (abort_flag && threadIdx.x == 0) atomicOr(&g_status_attend, FLAG_TIMEOUT);
    if (warp == 9) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join
// One warp per query row: its prefix's parts, then its suffix's, in the order of the line.
template <int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendArgs a,
                                                          const __grid_constant__ AtWork w) {
    constexpr int V = D / 32;  // values per lane
    const int lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * 4 + threadIdx.x / 32;
    pdl_wait();
    if (id >= (long long)a.agents * a.new_tokens * a.q_heads) return;
    const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G;
    const int qh = (int)(id % a.q_heads), t = (int)(id / a.q_heads % T);
    const int agent = (int)(id / ((long long)a.q_heads * T));
    const int head = qh / G, in = t * G + qh % G;
    const long long total = w.plan->total;
    int group = -1;
    if (a.groups > 0 && agent >= w.bounds[0] && agent < w.bounds[a.groups]) {
        int lo = 0, hi = a.groups;  // bounds[lo] <= agent < bounds[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (w.bounds[mid] <= agent) lo = mid;
            else hi = mid;
        }
        group = lo;
    }
    float M = -INFINITY, L = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int s = 0; s < 2; ++s) {
        if (s == 0 && group < 0) continue;
        const int seg = s == 0 ? group : a.groups + agent;
        const int r = s == 0 ? (agent - w.bounds[group]) * TG + in : in;
        const AtEntry e = w.entries[w.first[seg] + r / kAtBlock];
        if (e.tiles == 0) continue;
        const long long base = e.begin + (long long)head * (e.tiles + 1), stop = base + e.tiles;
        const bool two = e.rows > kAtRows;
        const int sets = two ? 1 : 2, rr = r - e.row0;
        const long long own = e.prow + (long long)head * (two ? e.rows : 2 * e.rows);
        // the first CTA whose piece reaches past base
        long long i0 = base * w.ctas / total;
        while (i0 > 0 && piece(total, (int)i0, w.ctas) > base) --i0;
        while (piece(total, (int)i0 + 1, w.ctas) <= base) ++i0;
        for (long long first = i0 * sets;; first += 32) {
            // lane k: part first + k (CTA, set)
            const long long k = first + lane;
            const int cta = (int)(k / sets), set = (int)(k % sets);
            const long long lo = cta < w.ctas ? piece(total, cta, w.ctas) : total;
            const long long hi = cta < w.ctas ? piece(total, cta + 1, w.ctas) : total;
            const bool in_unit = cta < w.ctas && lo < stop && hi > lo && max(lo, base) < min(hi, stop);
            const long long part = (lo <= base ? own : w.own_rows + (long long)cta * kAtBlock) + set * e.rows + rr;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (in_unit) ml = w.ml[part];
            float top = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float N = fmaxf(M, top);
            const float f = M == -INFINITY ? 0.f : ex2(M - N);
            const float wt = ml.x == -INFINITY ? 0.f : ex2(ml.x - N);
            // a part with NaN logits keeps m but has l = NaN: it must reach the result
            const bool counts = !(ml.y == 0.f);
            float sum = counts ? (ml.x == -INFINITY ? ml.y : ml.y * wt) : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            L = L * f + sum;
            M = N;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] *= f;
            unsigned live = __ballot_sync(0xffffffffu, in_unit && counts);
            while (live) {
                const int b = __ffs(live) - 1;
                live &= live - 1;
                const long long p = __shfl_sync(0xffffffffu, part, b);
                const float x = __shfl_sync(0xffffffffu, wt, b);
                const float* o = w.o + p * D + V * lane;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(o[i], x, acc[i]);
            }
            if (__all_sync(0xffffffffu, true) && __shfl_sync(0xffffffffu, (int)(cta + 1 >= w.ctas || hi >= stop), 31)) break;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const long long oo = a.op.row(agent, 0, t) + (long long)qh * D + V * lane;
    if (V == 4)
        *reinterpret_cast<uint2*>(a.out + oo) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv),
                                                           pack_bf16(acc[V - 2] * inv, acc[V - 1] * inv));
    else
        *reinterpret_cast<uint32_t*>(a.out + oo) = pack_bf16(acc[0] * inv, acc[1] * inv);
    if (a.lse && lane == 0) a.lse[id] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host
template <int F, int D>
static bool pool_map(CUtensorMap* m, const PoolView& p, int plane, int page) {
    using C = AtCfg<F, D>;
    const cuuint64_t dims[2] = {(cuuint64_t)p.heads * (C::kQuant ? C::kCodeRow : D), (cuuint64_t)p.slots};
    const cuuint64_t strides[1] = {(cuuint64_t)(p.slots > 1 ? p.ss : (long long)p.heads * C::kCodeRow)};
    const cuuint32_t box[2] = {(cuuint32_t)(C::kQuant ? C::kCodeRow : 64), (cuuint32_t)page}, one[2] = {1, 1};
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    return enc && enc(m, C::kQuant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                      p.plane[plane].codes, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      C::kQuant ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int F, int D>
static cudaError_t launch_attend_form(const AttendArgs& a, const AtWork& w, cudaStream_t s) {
    using C = AtCfg<F, D>;
    CUtensorMap mk, mv;
    if (!pool_map<F, D>(&mk, a.pool, 0, a.page) || !pool_map<F, D>(&mv, a.pool, 1, a.page)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<F, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attend_plan_kernel<<<1, kPlanThreads, 0, s>>>(a, w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_chained(attend_kernel<F, D>, dim3(w.ctas), dim3(C::kThreads), C::kSmem, s, mk, mv, a, w)) != cudaSuccess)
        return e;
    const long long rows = (long long)a.agents * a.new_tokens * a.q_heads;
    return launch_chained(attend_join_kernel<D>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, a, w);
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
    if ((long long)a.agents * a.new_tokens == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const AtLayout l = at_layout(a.agents, a.new_tokens, a.q_heads, a.pool.heads, a.pool.dim, a.groups);
    unsigned char* base = (unsigned char*)a.workspace;
    AtWork w;
    w.plan = (AtPlan*)(base + l.plan);
    w.first = (int*)(base + l.first);
    w.bounds = (int*)(base + l.bounds);
    w.entries = (AtEntry*)(base + l.entries);
    w.ml = (float2*)(base + l.ml);
    w.o = (float*)(base + l.o);
    w.own_rows = l.own_rows;
    w.ctas = sms < kAtMaxCtas ? sms : kAtMaxCtas;
    switch (a.pool.format * 2 + (a.pool.dim == 128)) {
        case KVFIX_POOL_BF16 * 2: return launch_attend_form<KVFIX_POOL_BF16, 64>(a, w, s);
        case KVFIX_POOL_BF16 * 2 + 1: return launch_attend_form<KVFIX_POOL_BF16, 128>(a, w, s);
        case KVFIX_POOL_E4M3 * 2: return launch_attend_form<KVFIX_POOL_E4M3, 64>(a, w, s);
        case KVFIX_POOL_E4M3 * 2 + 1: return launch_attend_form<KVFIX_POOL_E4M3, 128>(a, w, s);
        case KVFIX_POOL_INT4 * 2: return launch_attend_form<KVFIX_POOL_INT4, 64>(a, w, s);
        default: return launch_attend_form<KVFIX_POOL_INT4, 128>(a, w, s);
    }
}

}  // namespace kvfix
