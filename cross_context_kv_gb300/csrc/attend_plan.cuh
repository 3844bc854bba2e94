// attend_plan.cuh -- how kvfix_shared_attend cuts its work: entries, lines, pieces, and where the
// parts of a row lie; the kernel that lays them out, and the walk of a piece.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attend.h"
#include "pool.cuh"

namespace kvfix {

static __device__ unsigned int g_status_attend;

constexpr int kAtKeys = 128;      // keys per tile
constexpr int kAtRows = 128;      // rows per accumulator (MMA M)
constexpr int kAtBlock = 256;     // rows per entry
constexpr int kAtMaxCtas = 256;   // bound of the persistent grid
constexpr int kFewWarps = 8;      // warps of a few-row CTA (12 or 16 are no faster)

// A row's maximum is raised (and its accumulator rescaled) once a logit passes it by more
// than this many powers of two: weights stay below 2^8, and bf16 keeps 8 bits of any of them.
constexpr float kAtSlack = 8.f;

// ------------------------------------------------------------------ plan
// A segment's rows are cut into blocks of 256; the last block may be smaller.  By its rows a
// block is a pair (more than 128: both softmax groups of a CTA share its tiles), a single (one
// group's) or, up to AtWork::few rows, the few-row kernel's.  Each kind lies on a line of its own:
// unit (entry e, head h) begins at begin + h * (tiles + at_pad), in tiles of 128 keys, or of 16
// for the few-row kernel.  The pairs' line is cut into one piece per CTA, the singles' into two
// (one per softmax group), the few-row kernel's into one per warp.
enum : int { kPairs = 0, kSingles = 1, kFew = 2 };
__host__ __device__ constexpr int at_keys(int kind) { return kind == kFew ? 16 : kAtKeys; }
// What a unit costs beside its tiles (queries in, masks, its part out), in tiles: measured on
// pairs of short own segments at head_dim 128, 17000 cycles a unit against 4000 a tile; with 1
// there, the CTAs that had those units ran 1.7 times as long as the others.
__host__ __device__ constexpr int at_pad(int kind) { return kind == kPairs ? 4 : kind == kSingles ? 1 : 2; }

struct __align__(16) AtEntry {
    long long begin;  // position of head 0 on the line
    int tiles, rows;
    int row0, seg, keys, agent0;  // keys: those that some row of the block may see
};

// Where a piece of a line begins, all that its walk needs in one round of loads.
struct __align__(16) AtStart {
    AtEntry rec;        // the entry
    long long lo, hi;   // the piece
    int e, h, n, have;  // the entry's index, the head, the line's entries; whether there is a piece
};

struct AtPlan {
    long long chunk[3];            // by kind: length of a piece of the line
    int many_ctas;                 // CTAs that pairs and singles are cut for; the few-row blocks have the others
    AtStart start[4][kAtMaxCtas];  // pairs, singles of group 0, of group 1, few-row blocks
};

struct AtLayout {
    size_t plan, first, bounds, entries[3], ml, o, bytes;
    long long own_rows, few_rows;
    int few;    // largest block of the few-row kernel; 0: it is not launched
    bool many;  // some block may have more rows
};

// Part rows.  The first part of a unit has its rows' own places (prefix rows, then suffix
// rows: [head][agent][token, query head]); a part that continues a unit from an earlier piece
// has its CTA's (256 rows for a pair, 2 x 128 for singles) or its warp's.
static AtLayout at_layout(int agents, int T, int q_heads, int kv_heads, int head_dim, int groups) {
    const long long tg = (long long)T * (q_heads / kv_heads), all = (long long)agents * tg;
    AtLayout l;
    // An agent's rows decide: an own segment has tg, a prefix between tg and all.  Blocks of up to
    // 16 rows where that leaves nothing for the other kernel, else the suffixes' 8 or 16; with more
    // rows an agent the other kernel has all blocks, small last ones too.
    const long long most = groups > 0 ? all : tg;
    l.few = most <= 8 ? 8 : most <= 16 ? 16 : tg <= 8 ? 8 : tg <= 16 ? 16 : 0;
    l.many = most > l.few;
    l.own_rows = 2 * kv_heads * all;
    l.few_rows = l.own_rows + (l.many ? (long long)kAtMaxCtas * 2 * kAtBlock : 0);
    const long long rows = l.few_rows + (long long)kAtMaxCtas * kFewWarps * l.few;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    l.plan = take(sizeof(AtPlan));
    l.first = take(8 * ((size_t)groups + agents));
    l.bounds = take(4 * ((size_t)groups + 1));
    l.entries[kPairs] = take(sizeof(AtEntry) * (size_t)(2 * all / kAtRows + 2));
    l.entries[kSingles] = take(sizeof(AtEntry) * ((size_t)groups + agents + 1));
    l.entries[kFew] = take(sizeof(AtEntry) * ((size_t)groups + agents + 1));
    l.ml = take(8 * (size_t)rows);
    l.o = take(4 * (size_t)rows * head_dim);
    l.bytes = at;
    return l;
}

struct AtWork {
    AtPlan* plan;
    int2* first;          // [groups + agents]: a segment's first pair, and its last block if that is not one
    int* bounds;          // [groups + 1]: the groups' agents, clamped and ascending
    AtEntry* entries[3];  // by kind
    float2* ml;           // part rows: (max in base-2 units, sum)
    float* o;             // part rows x D
    long long own_rows, few_rows;
    int ctas, few;
    bool many;            // the kernel for larger blocks runs too
};

__device__ __forceinline__ int at_kind(int rows, int few) { return rows > kAtRows ? kPairs : rows > few ? kSingles : kFew; }

__device__ __forceinline__ int clamp_len(int n, long long most, bool& bad) {
    if (n < 0 || n > most) bad = true;
    return (int)min(max((long long)n, 0ll), most);
}

// Trees: an agent's number of nodes, with `keys` own keys.
__device__ __forceinline__ int tree_nodes(const AttendArgs& a, int agent, int keys, bool& bad) {
    const int given = a.nodes ? __ldg(a.nodes + agent) : a.new_tokens;
    return clamp_len(given, min(a.new_tokens, keys), bad);
}

// Trees: 32 keys of node t's view as bits, the first of them node d of its tree (below 0: before
// the tree, and seen).  Bits past t mean nothing.
__device__ __forceinline__ uint32_t tree_view(const AttendArgs& a, const uint32_t* mask, int d) {
    if (d <= -32) return 0xffffffffu;
    if (d < 0) return (__ldg(mask) << -d) | ((1u << -d) - 1u);
    const int w = d >> 5;
    const uint32_t lo = w < a.tree_words ? __ldg(mask + w) : 0u, hi = w + 1 < a.tree_words ? __ldg(mask + w + 1) : 0u;
    return __funnelshift_r(lo, hi, d & 31);
}

// A quotient of non-negative numbers, in 32 bits where they fit (a 64-bit division takes
// about a hundred instructions).
__device__ __forceinline__ long long quotient(long long x, long long y) {
    return (x | y) >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
}

// The plan is one CTA whose code runs once, so its time is latency: trips to memory and fetches of
// instructions.  Scans are loops, and what a segment's thread worked out for the scan it keeps for
// what comes after.  (640 threads, one for each piece's beginning: 0.6 us less for a round of 8
// trees, but 0.6 more for one small tree.)
constexpr int kPlanThreads = 256;

struct PlanSums {
    int n[3];
    long long line[3];
};
// Exclusive scan over the block, and the totals.
__device__ __forceinline__ PlanSums plan_scan(const PlanSums& x, PlanSums* warp_sums, PlanSums* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PlanSums inc = x;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int a = __shfl_up_sync(0xffffffffu, inc.n[k], o);
            const long long b = __shfl_up_sync(0xffffffffu, inc.line[k], o);
            if (lane >= o) {
                inc.n[k] += a;
                inc.line[k] += b;
            }
        }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    PlanSums ex, all = {};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        ex.n[k] = inc.n[k] - x.n[k];
        ex.line[k] = inc.line[k] - x.line[k];
    }
#pragma unroll 2
    for (int w = 0; w < kPlanThreads / 32; ++w)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int a = warp_sums[w].n[k];
            const long long b = warp_sums[w].line[k];
            if (w < warp) {
                ex.n[k] += a;
                ex.line[k] += b;
            }
            all.n[k] += a;
            all.line[k] += b;
        }
    *total = all;
    return ex;
}

constexpr int kPlanKept = 256;  // entries of a line that stay in shared memory

// TREE: kvfix_tree_attend's, whose agents have numbers of new tokens of their own.
template <bool TREE>
__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const __grid_constant__ AttendArgs a,
                                                                   const __grid_constant__ AtWork w) {
    __shared__ PlanSums warp_sums[kPlanThreads / 32];
    __shared__ int warp_max[kPlanThreads / 32];
    __shared__ AtEntry kept[3][kPlanKept];
    struct Seg {
        int agent0, rows, keys;
        int nodes;  // trees: of a suffix
        bool prefix;
    };
    // Few enough segments for one a thread: what they are, where their pairs begin on their line
    // and among the entries, and the group bounds (read again at once, and a trip to memory is a
    // microsecond).
    __shared__ Seg near_seg[kPlanThreads];
    __shared__ long long pair_line[kPlanThreads];
    __shared__ int pair_first[kPlanThreads], near_bounds[kPlanThreads + 1];
    pdl_wait();  // the lengths may be the work of the kernel before
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G, H = a.pool.heads;
    const int segs = a.groups + a.agents;
    const int per = (segs + kPlanThreads - 1) / kPlanThreads;
    const int s0 = min(segs, tid * per), s1 = min(segs, s0 + per);
    const long long most_p = (long long)a.max_prefix_pages * a.page, most_s = (long long)a.max_suffix_pages * a.page;
    bool bad = false;
    // the first segment's length is on its way while the bounds are worked out
    int len0 = 0, nodes0 = T;
    if (s0 < s1) {
        len0 = s0 < a.groups ? __ldg(a.prefix_len + s0) : __ldg(a.suffix_len + s0 - a.groups);
        if (TREE && a.nodes && s0 >= a.groups) nodes0 = __ldg(a.nodes + s0 - a.groups);
    }
    const bool near = segs <= kPlanThreads;
    auto bound = [&](int g) { return near ? near_bounds[g] : w.bounds[g]; };
    // group bounds: the running maximum of the given ones, kept within 0..agents
    if (a.groups > 0) {
        const int n = a.groups + 1, each = (n + kPlanThreads - 1) / kPlanThreads;
        const int g0 = min(n, tid * each), g1 = min(n, g0 + each);
        int mine = 0;
        for (int g = g0; g < g1; ++g) mine = max(mine, min(max(__ldg(a.group_begin + g), 0), a.agents));
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
            const int b = __ldg(a.group_begin + g);
            if (b < run || b > a.agents) bad = true;
            run = max(run, min(max(b, 0), a.agents));
            w.bounds[g] = run;
            if (near) near_bounds[g] = run;
        }
        __syncthreads();
    }
    auto segment = [&](int s) {
        Seg g;
        g.prefix = s < a.groups;
        g.agent0 = g.prefix ? bound(s) : s - a.groups;
        const int given = s == s0 ? len0 : g.prefix ? __ldg(a.prefix_len + s) : __ldg(a.suffix_len + g.agent0);
        g.keys = clamp_len(given, g.prefix ? most_p : most_s, bad);
        g.rows = (g.prefix ? bound(s + 1) - g.agent0 : 1) * TG;
        g.nodes = T;
        if (TREE && !g.prefix)
            g.nodes = s == s0 ? clamp_len(nodes0, min(T, g.keys), bad) : tree_nodes(a, g.agent0, g.keys, bad);
        return g;
    };
    auto block = [&](const Seg& g, int s, int r0, int& kind) {
        AtEntry e;
        e.rows = min(kAtBlock, g.rows - r0);
        e.row0 = r0;
        e.seg = s;
        e.agent0 = g.agent0;
        // own keys are seen up to the place of the block's last row
        if constexpr (TREE)
            e.keys = g.prefix ? g.keys : r0 / G >= g.nodes ? 0 : g.keys - g.nodes + 1 + min(g.nodes - 1, (r0 + e.rows - 1) / G);
        else
            e.keys = g.prefix ? g.keys : max(0, g.keys - T + 1 + (r0 + e.rows - 1) / G);
        kind = at_kind(e.rows, w.few);
        e.tiles = (e.keys + at_keys(kind) - 1) / at_keys(kind);
        return e;
    };
    auto cost = [&](const AtEntry& e, int kind) { return e.tiles > 0 ? (long long)H * (e.tiles + at_pad(kind)) : 0ll; };
    // what a segment's first n blocks, pairs all, take: a prefix's are alike
    auto pairs_cost = [&](const Seg& g, int s, int n) {
        int k;
        if (g.prefix) return n > 0 ? n * cost(block(g, s, 0, k), kPairs) : 0ll;
        long long sum = 0;
        for (int b = 0; b < n; ++b) sum += cost(block(g, s, b * kAtBlock, k), kPairs);
        return sum;
    };
    auto full_pairs = [&](const Seg& g) { return g.rows / kAtBlock; };
    auto keep = [&](AtEntry e, int k, int i, long long begin) {
        e.begin = begin;
        w.entries[k][i] = e;
        if (i < kPlanKept) kept[k][i] = e;
    };
    // a segment, its full blocks and what they take, its last block and what that takes
    struct Look {
        Seg g;
        int full, kind;
        long long pairs, cost;
        AtEntry last;  // no rows: there is none
    };
    auto look = [&](int s) {
        Look l;
        l.g = segment(s);
        l.full = full_pairs(l.g);
        l.pairs = pairs_cost(l.g, s, l.full);
        l.last.rows = 0;
        if (l.g.rows > l.full * kAtBlock) {
            l.last = block(l.g, s, l.full * kAtBlock, l.kind);
            l.cost = cost(l.last, l.kind);
        }
        return l;
    };
    PlanSums mine = {};
    Look now;
    for (int s = s0; s < s1; ++s) {
        now = look(s);
        if (near) near_seg[s] = now.g;
        mine.n[kPairs] += now.full;
        mine.line[kPairs] += now.pairs;
        if (now.last.rows > 0) {
#pragma unroll
            for (int x = 0; x < 3; ++x)
                if (x == now.kind) {
                    mine.n[x] += 1;
                    mine.line[x] += now.cost;
                }
        }
    }
    PlanSums total;
    PlanSums at = plan_scan(mine, warp_sums, &total);
    for (int s = s0; s < s1; ++s) {
        if (!near) now = look(s);
        const Seg& g = now.g;
        const int full = now.full;
        int2 first = make_int2(at.n[kPairs], 0);
        // full blocks: by all threads below, where each has one segment at most
        if (!near)
            for (int b = 0; b < full; ++b) {
                int k;
                const AtEntry e = block(g, s, b * kAtBlock, k);
                keep(e, kPairs, at.n[kPairs] + b, at.line[kPairs] + pairs_cost(g, s, b));
            }
        else {
            pair_line[s] = at.line[kPairs];
            pair_first[s] = at.n[kPairs];
        }
        at.n[kPairs] += full;
        at.line[kPairs] += now.pairs;
        if (now.last.rows > 0) {
#pragma unroll
            for (int x = 0; x < 3; ++x)
                if (x == now.kind) {
                    keep(now.last, x, at.n[x], at.line[x]);
                    if (x != kPairs) first.y = at.n[x];
                    at.n[x] += 1;
                    at.line[x] += now.cost;
                }
        }
        w.first[s] = first;
    }
    __syncthreads();
    if (near)
        for (int i = tid; i < total.n[kPairs]; i += kPlanThreads) {
            int x = 0, y = segs;  // the last segment whose pairs begin at or before i
            while (y - x > 1) {
                const int m = (x + y) / 2;
                if (pair_first[m] <= i) x = m;
                else y = m;
            }
            const Seg g = near_seg[x];
            const int b = i - pair_first[x];
            if (b >= full_pairs(g)) continue;  // (the last block's, written above)
            int k;
            keep(block(g, x, b * kAtBlock, k), kPairs, i, pair_line[x] + pairs_cost(g, x, b));
        }
    __syncthreads();
    // The two kernels share the GPU: CTAs of the first that have no piece end at once, and the
    // second's take their places.  The split has both end together, from what 128 keys cost a CTA
    // of each and what the first takes before and after its tiles, in microseconds as measured at
    // head_dim 128: F + X / n = Y / (ctas - n), solved for n.  (Only the split depends on them.)
    int nm = w.ctas, nf = w.ctas;
    if (total.line[kPairs] + total.line[kSingles] > 0 && total.line[kFew] > 0) {
        const bool stored = a.pool.format != KVFIX_POOL_BF16;
        const float F = 4.f, S = (float)w.ctas;
        const float X = (stored ? 2.5f : 1.6f) * (float)(total.line[kPairs] + total.line[kSingles]);
        const float Y = (stored ? 1.1f : 1.5f) * (float)total.line[kFew] / (float)(kAtKeys / at_keys(kFew));
        const float B = F * S - X - Y;
        nm = (int)((B + sqrtf(B * B + 4.f * F * X * S)) / (2.f * F) + 0.5f);
        nm = min(max(nm, 1), w.ctas - 1);
        nf = w.ctas - nm;
    }
    const int few_pieces = nf * kFewWarps;
    const long long chunk[3] = {max(1ll, quotient(total.line[0] + nm - 1, nm)),
                                max(1ll, quotient(total.line[1] + 2 * nm - 1, 2 * nm)),
                                max(1ll, quotient(total.line[2] + few_pieces - 1, few_pieces))};
    // (a few-row CTA has its warps' pieces as one)
    for (int i = tid; i < 4 * w.ctas; i += kPlanThreads) {
        const int cta = i % w.ctas, set = i / w.ctas, k = set == 0 ? kPairs : set == 3 ? kFew : kSingles;
        AtStart* st = &w.plan->start[set][cta];
        const long long size = k == kFew ? chunk[kFew] * kFewWarps : k == kSingles ? chunk[kSingles] : chunk[kPairs];
        const long long lo = k != kFew && cta >= nm ? total.line[k] : size * (set == 2 ? cta + nm : cta);
        if (lo >= total.line[k]) {
            st->have = 0;
            continue;
        }
        // The last entry that begins at or before the piece does: entries without tiles take no
        // room, and of several at one place the last has it.
        int x = 0, y = total.n[k];  // begin[x] <= lo < begin[y]
        const bool here = total.n[k] <= kPlanKept;
        while (y - x > 1) {
            const int m = (x + y) / 2;
            const long long b = here ? kept[k][m].begin : w.entries[k][m].begin;
            if (b <= lo) x = m;
            else y = m;
        }
        AtStart r;
        r.rec = here ? kept[k][x] : w.entries[k][x];
        r.lo = lo;
        r.hi = min(total.line[k], lo + size);
        r.e = x;
        r.h = (int)quotient(lo - r.rec.begin, r.rec.tiles + at_pad(k));
        r.n = total.n[k];
        r.have = 1;
        *st = r;
    }
    if (tid < 3) w.plan->chunk[tid] = tid == 0 ? chunk[0] : tid == 1 ? chunk[1] : chunk[2];
    if (tid == 0) w.plan->many_ctas = nm;
    if (bad) atomicOr(&g_status_attend, FLAG_BOUNDS);
}

// Pieces of a line in order of units.
struct AtWalk {
    const AtEntry* ent;
    long long lo, hi;
    int e, n, h, H, pad;
    AtEntry rec;
    bool have;

    __device__ __forceinline__ void open(const AtStart& s, const AtEntry* entries, int heads, int kind) {
        rec = s.rec;
        lo = s.lo;
        hi = s.hi;
        e = s.e;
        h = s.h;
        n = s.n;
        have = s.have != 0;
        ent = entries;
        H = heads;
        pad = at_pad(kind);
    }

    // The next unit's tiles [t0, t1) of head `head` in this piece.
    __device__ __forceinline__ bool next(int& head, int& t0, int& t1) {
        while (have) {
            if (rec.tiles == 0 || h >= H) {
                ++e;
                h = 0;
                have = e < n;
                if (have) rec = ent[e];
                continue;
            }
            const long long base = rec.begin + (long long)h * (rec.tiles + pad);
            if (base >= hi) {
                have = false;
                break;
            }
            t0 = (int)max(0ll, lo - base);
            t1 = (int)min((long long)rec.tiles, hi - base);
            head = h++;
            if (t0 < t1) return true;
        }
        return false;
    }
};

// ------------------------------------------------------------------ small parts
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace kvfix
