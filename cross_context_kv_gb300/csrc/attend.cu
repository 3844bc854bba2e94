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
// head; its work is its keys in tiles (causally trimmed), plus a few tiles for its fixed cost.
// One plan kernel lays all units on lines and cuts the lines into equal pieces
// (attend_plan.cuh); a worker writes one part per unit that its piece touches, and the join
// kernel finds a row's parts from the same lines.  Small blocks go to a kernel without tensor
// memory (attend_few.cuh), the others to the one below; a call's rows decide how many are few
// (at_layout: 8, 16, or none).  Everything depends on lengths that lie on the device, so a
// captured graph follows them.
//
// What bounds the kernel below: HBM for bf16 prefixes of a decoding round (131072 keys and
// 128 rows of 8 heads: 537 MB in 95 us, 5.6 TB/s), the conversion of stored tiles and the chain
// from logits to weights for e4m3 and int4 (138 us for the same keys as e4m3), the
// exponentials and the tensor pipe for many new tokens (288 GFLOP in 256 us, 1.12 PFLOP/s):
//   warps 0-3, 4-7  softmax: each group owns one 128-row accumulator.  Blocks of more than
//                   128 rows (pairs) give each group its half of the rows, and both use every
//                   tile; smaller ones (singles) are one group's alone, and the two groups
//                   walk pieces of their own.  A thread owns a row (a TMEM lane): no
//                   cross-lane reduction.
//   warp 10         scheduler: walks the CTA's pieces of the lines, reads the page lists and
//                   hands each tile of either group to the other roles.
//   warp 8          TMA producer: pages of K and V tiles (128 keys x D) into their rings.
//   warps 9, 11     one per softmax group: loads a unit's queries and issues tcgen05.mma,
//                   S = Q K^T (both K-major in shared memory), and O += P V with P from tensor
//                   memory and V read N-major as it lies.
//   warps 12-19     (stored forms) converters: code tiles and their scales, loaded as they lie,
//                   to bf16 tiles for the MMA; four warps for keys, four for values.
// S occupies 128 TMEM columns per group, P (bf16) overwrites the first half of S, O takes D.
// (e4m3 codes as operands of 8-bit products, with queries in two pieces and the scales on the
// logits, are right too and were slower: 186 us against 169 for the e4m3 case above, as the
// softmax warps, which are the bound, get the factors' work.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "attend_few.cuh"
#include "attend_plan.cuh"
#include "tc.cuh"

namespace kvfix {

unsigned read_status_attend(cudaStream_t stream) {
    unsigned h = 0, zero = 0;
    cudaMemcpyFromSymbolAsync(&h, g_status_attend, sizeof h, 0, cudaMemcpyDeviceToHost, stream);
    cudaMemcpyToSymbolAsync(g_status_attend, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    cudaStreamSynchronize(stream);
    return h;
}

// ------------------------------------------------------------------ a CTA's work
// One tile of a softmax group's work, as the scheduling warp hands it to the others.
struct __align__(16) AtItem {
    int head, tile, flags, keys;        // tile: running number of the CTA's tiles (ring places); keys in the tile
    int key0, rows, row0, agent0;       // first key of the tile in its segment; the group's rows
    int sees0, absent;                  // see the softmax; 16-key parts of the tile that are not there
    long long part;                     // first part row
    int page[8];                        // pool pages, -1: not read
};
enum : int { kFirst = 1, kLast = 2, kPair = 4, kPrefix = 8, kEnd = 16, kKeyTurn = 32, kValueTurn = 64 };
constexpr int kItems = 4;  // items ahead per group

// ------------------------------------------------------------------ attention
// One lane of a converged warp, by elect.sync: in a branch on it the compiler knows that one
// lane runs, and keeps the operands of tensor instructions in uniform registers.  (Behind
// `lane == 0` every operand of every product moves through a vector register: 95 cycles a
// product with four busy warps beside it, against the tensor pipe's 64.)
__device__ __forceinline__ bool elect_lane() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
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

// 16 consecutive 32-bit columns of this warp's 32 TMEM lanes from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// 16 TMEM lanes x 64 32-bit columns: v[4k], v[4k+1] are columns 8k + 2 (lane % 4) + {0, 1} of
// row lane / 4, v[4k+2], v[4k+3] those of the row 8 below.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// Registers move from the other warpgroups to the softmax ones (setmaxnreg: the shares add up
// to no more than what the block launches with).
template <int F, int D>
struct AtCfg {
    static constexpr bool kQuant = F != KVFIX_POOL_BF16;
    static constexpr int kConvWarps = 4;  // per converting team: one for keys, one for values
    static constexpr int kThreads = kQuant ? 384 + 64 * kConvWarps : 384;
    static constexpr int kRegsSoftmax = kQuant ? 120 : 208;
    static constexpr int kRegsOther = kQuant ? 80 : 88;
    static constexpr int kTile = kAtKeys * D * 2;   // a K or V tile as bf16
    static constexpr int kQ = kAtRows * D * 2;
    // rings of bf16 tiles: keys are free once their product is done, values wait for the weights
    static constexpr int kKeyStages = D == 128 ? 2 : 4;
    static constexpr int kValueStages = D == 128 ? (kQuant ? 2 : 3) : 4;
    static constexpr int kStages = kKeyStages + kValueStages;
    // stored tiles before conversion: codes, then scales
    static constexpr int kCodeRow = pool_head_bytes(F, D);
    static constexpr int kScaleRow = F == KVFIX_POOL_E4M3 ? 1 : F == KVFIX_POOL_INT4 ? D / 8 : 0;
    static constexpr int kRaw = kQuant ? kAtKeys * (kCodeRow + kScaleRow) : 0;
    static constexpr int kRawStages = kQuant && D == 64 ? 4 : 2;  // half for keys
    static constexpr int kSmem = 1024 + kStages * kTile + 2 * kQ + (kQuant ? kRawStages * kRaw : 0);
    static_assert(kSmem <= 227 * 1024 - 1536, "shared memory, with the barriers and items");
    static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * (65536 / kThreads / 8 * 8), "registers");
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
// reads: rows of 128 bytes per 64-column half, 128-byte swizzle.  Rows that hold no key become
// zero.  A team of N threads first takes the whole stored tile into registers, so that the
// next one can be on its way while this one is converted; a thread has 16 code bytes of a row
// at a time, and the order in which it writes their 16-byte chunks puts the eight threads of a
// store phase on different banks.
template <int F, int D, int N>
struct StoredTile {
    using C = AtCfg<F, D>;
    static constexpr int V = C::kCodeRow / 16;  // vectors per row
    static constexpr int P = kAtKeys * V / N;   // vectors per thread
    uint4 x[P];
    unsigned sc[P];

    __device__ __forceinline__ void take(const unsigned char* raw, int tid) {
        const unsigned char* scales = raw + kAtKeys * C::kCodeRow;
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const int r = tid / V + k * (N / V);
            x[k] = *reinterpret_cast<const uint4*>(raw + 16 * (tid + k * N));
            if (F == KVFIX_POOL_E4M3) sc[k] = scales[r];
            else sc[k] = *reinterpret_cast<const unsigned*>(scales + r * C::kScaleRow + 4 * (tid % V));
        }
    }

    // In rounds of two vectors, the rest moving down between them: with all eight unrolled the
    // roles' code outgrows the instruction caches (a quarter of the stalls were for
    // instructions).
    __device__ __forceinline__ void put(unsigned char* tile, int tid, int in_tile, unsigned absent) {
        constexpr int B = P < 2 ? P : 2;
        int r0 = tid / V;
        const int v = tid % V;
        const bool partial = in_tile < kAtKeys || absent != 0u;
#pragma unroll 1
        for (int k0 = 0; k0 < P; k0 += B, r0 += B * (N / V)) {
            put_some<B>(tile, r0, v, partial, in_tile, absent);
#pragma unroll
            for (int k = 0; k + B < P; ++k) {
                x[k] = x[k + B];
                sc[k] = sc[k + B];
            }
        }
    }

    template <int B>
    __device__ __forceinline__ void put_some(unsigned char* tile, int r0, int v, bool partial, int in_tile,
                                             unsigned absent) const {
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int r = r0 + k * (N / V);
            const bool gone = partial && (r >= in_tile || ((absent >> (r >> 4)) & 1u));
            const unsigned c[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            if (F == KVFIX_POOL_E4M3) {
                E4m3Scale es = e4m3_scale_byte(sc[k]);
                if (gone) es.a = __nv_bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
                uint4 o0, o1;
                e4m3x16_to_bf16(x[k], es, o0, o1);
                unsigned char* dst = tile + (v / 4) * (kAtKeys * 128) + r * 128;
                const int c0 = 2 * (v % 4), sw = (v / 4) & 1;  // the upper half's odd chunk first
                const int a0 = ((c0 ^ (r & 7)) << 4), a1 = (((c0 + 1) ^ (r & 7)) << 4);
                *reinterpret_cast<uint4*>(dst + (sw ? a1 : a0)) = sw ? o1 : o0;
                *reinterpret_cast<uint4*>(dst + (sw ? a0 : a1)) = sw ? o0 : o1;
            } else {
                const unsigned sz = gone ? 0u : sc[k];
                const unsigned ss = __byte_perm(sz, 0u, 0x1010), zz = __byte_perm(sz, 0u, 0x3232);
                unsigned char* dst = tile + (v / 2) * (kAtKeys * 128) + r * 128;
                const int sw = ((v / 2) & 1) ? 2 : 0;  // the upper half's chunks in the order 2 3 0 1
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 o = int4x8_to_bf16(sw ? c[q ^ 2] : c[q], *reinterpret_cast<const __nv_bfloat162*>(&ss),
                                                   *reinterpret_cast<const __nv_bfloat162*>(&zz));
                    *reinterpret_cast<uint4*>(dst + (((4 * (v % 2) + (q ^ sw)) ^ (r & 7)) << 4)) = o;
                }
            }
        }
    }
};


// Two floats at once (packed 32-bit arithmetic).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<unsigned long long*>(&d))
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long*>(&d))
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return d;
}

template <int F, int D>
__global__ void __launch_bounds__(AtCfg<F, D>::kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ AttendArgs a, const __grid_constant__ AtWork w) {
    using C = AtCfg<F, D>;
    constexpr int SK = C::kKeyStages, SV = C::kValueStages, R = C::kRawStages / 2;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[3][SK + SV], empty[SK + SV], raw_full[2 * R], raw_empty[2 * R];
    __shared__ __align__(8) uint64_t q_free[2], s_full[2], p_ready[2], o_full[2];
    __shared__ __align__(8) uint64_t item_full[2][kItems], item_free[2][kItems];
    __shared__ AtItem items[2][kItems];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, mma_lock;
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* qsm = smem + (SK + SV) * C::kTile;
    unsigned char* rawsm = qsm + 2 * C::kQ;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < SK + SV; ++i) {
            for (int f = 0; f < 3; ++f) mbar_init(&full[f][i], C::kQuant ? 32 * C::kConvWarps : 1);
            mbar_init(&empty[i], 2);  // one release per softmax group (a group alone releases twice)
        }
        for (int i = 0; i < 2 * R; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], C::kQuant ? 32 * C::kConvWarps : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_free[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 128);
            mbar_init(&o_full[i], 1);
            for (int k = 0; k < kItems; ++k) {
                mbar_init(&item_full[i][k], 1);
                // readers: producer, MMA, four softmax warps, converters
                mbar_init(&item_free[i][k], 6 + (C::kQuant ? 2 * C::kConvWarps : 0));
            }
        }
        fence_mbar_init();
        abort_flag = 0;
        mma_lock = 0;
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    // Ring place of tile n's keys (p = 0) or values (1).  Who fills a place waits for each of its
    // releases in turn; who reads it sees only its own tiles, and a parity tells a barrier's
    // last phase from the one before, no more: so a place has a full barrier per reader (group
    // 0, group 1, both), whose phases that reader sees one by one, and the item says which
    // parity its tile's phase has.
    auto place = [](int p, int n) { return p ? SK + n % SV : n % SK; };
    auto reader = [](int flags, int g) { return flags & kPair ? 2 : g; };
    auto released = [](int p, int n) { return (unsigned)((p ? n / SV : n / SK) - 1) & 1u; };  // its use before n's
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
    const int page_log = 31 - __clz(a.page);

    // Items of group g in order.  The roles that serve both groups take them in turn, group 0
    // then 1, an ended group left out; `at` counts a group's items.
    auto item_wait = [&](int g, unsigned at) {
        return __all_sync(0xffffffffu, mbar_wait(&item_full[g][at % kItems], (at / kItems) & 1u));
    };
    auto item_done = [&](int g, unsigned at) { mbar_arrive(&item_free[g][at % kItems]); };

    if (warp >= 8) {
        regs_dec<C::kRegsOther>();
        if (warp == 10) {
            // ------------------------------------------------------------ schedule
            bool ok = true, bad = false;
            unsigned put[2] = {0, 0};
            unsigned turns[3] = {0, 0, 0};  // by reader: the parities of the places' next phases
            int tile_no = 0;
            const int ppt = kAtKeys >> page_log, pool_pages = a.pool.slots >> page_log;
            const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G;
            const long long all = (long long)a.agents * TG;
            struct Feed {
                AtWalk walk;
                int head, t, t1;   // the unit's tiles left
                int page;          // this lane's page of tile t
                bool first, live;
            };
            auto fetch = [&](Feed& f) {
                const bool prefix = f.walk.rec.seg < a.groups;
                const int32_t* pages = prefix ? a.prefix_pages + (long long)f.walk.rec.seg * a.max_prefix_pages
                                              : a.suffix_pages + (long long)f.walk.rec.agent0 * a.max_suffix_pages;
                const int i = f.t * ppt + lane;
                const bool used = lane < ppt && i < (f.walk.rec.keys + a.page - 1) >> page_log;
                f.page = used ? __ldg(pages + i) : -2;
            };
            auto advance = [&](Feed& f) {
                f.live = f.walk.next(f.head, f.t, f.t1);
                f.first = true;
                if (f.live) fetch(f);
            };
            // hands tile f.t, or the end, to group g
            auto push = [&](const Feed& f, int g, bool pair) {
                const int slot = put[g] % kItems;
                if (put[g] >= kItems) ok = mbar_wait(&item_free[g][slot], (put[g] / kItems - 1) & 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                AtItem* it = &items[g][slot];
                if (!f.live) {
                    if (lane == 0) {
                        it->flags = kEnd;
                        mbar_arrive(&item_full[g][slot]);
                    }
                    ++put[g];
                    return;
                }
                const AtEntry& e = f.walk.rec;
                const bool there = f.page >= 0 && f.page < pool_pages;
                const unsigned gone = __ballot_sync(0xffffffffu, f.page != -2 && !there);
                if (gone) bad = true;
                if (lane < 8) it->page[lane] = there ? f.page : -1;
                if (lane == 0) {
                    unsigned absent = 0;  // by 16 keys
                    for (int b = 0; b < 8; ++b) absent |= ((gone >> (b >> (page_log - 4))) & 1u) << b;
                    const bool prefix = e.seg < a.groups;
                    const int r0 = pair ? kAtRows * g : 0;
                    it->head = f.head;
                    it->tile = tile_no;
                    const unsigned bits = pair ? turns[2] : g ? turns[1] : turns[0];
                    it->flags = (f.first ? kFirst : 0) | (f.t + 1 == f.t1 ? kLast : 0) | (pair ? kPair : 0) |
                                (prefix ? kPrefix : 0) | ((bits >> place(0, tile_no)) & 1u ? kKeyTurn : 0) |
                                ((bits >> place(1, tile_no)) & 1u ? kValueTurn : 0);
                    it->keys = min(kAtKeys, e.keys - f.t * kAtKeys);
                    it->key0 = f.t * kAtKeys;
                    it->rows = min(kAtRows, e.rows - r0);
                    it->row0 = e.row0 + r0;
                    it->agent0 = e.agent0;
                    // prefix: its keys; suffix: a row of new token t sees sees0 + t keys
                    it->sees0 = prefix ? e.keys : e.keys - (e.row0 + e.rows - 1) / G;
                    it->absent = (int)absent;
                    // a unit's first part lies in its rows' own places, a continued one in the CTA's
                    const bool own = e.begin + (long long)f.head * (e.tiles + at_pad(pair ? kPairs : kSingles)) >= f.walk.lo;
                    it->part = own ? ((prefix ? 0 : a.pool.heads) + (long long)f.head) * all + (long long)e.agent0 * TG + e.row0 + r0
                                   : w.own_rows + (long long)blockIdx.x * (2 * kAtBlock) + (pair ? 0 : kAtBlock) + kAtRows * g;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_full[g][slot]);
                ++put[g];
            };
            auto step = [&](Feed& f, unsigned& reader_turns) {
                reader_turns ^= (1u << place(0, tile_no)) | (1u << place(1, tile_no));
                ++tile_no;
                f.first = false;
                if (++f.t < f.t1) fetch(f);
                else advance(f);
            };
            Feed f0, f1;
            const AtStart s0 = w.plan->start[0][blockIdx.x], s1 = w.plan->start[1][blockIdx.x],
                          s2 = w.plan->start[2][blockIdx.x];
            f0.walk.open(s0, w.entries[kPairs], a.pool.heads, kPairs);
            advance(f0);
            while (ok && f0.live) {
                push(f0, 0, true);
                if (ok) push(f0, 1, true);
                step(f0, turns[2]);
            }
            f0.walk.open(s1, w.entries[kSingles], a.pool.heads, kSingles);
            f1.walk.open(s2, w.entries[kSingles], a.pool.heads, kSingles);
            advance(f0);
            advance(f1);
            // a group that is done says so at its next turn: the other roles wait for that turn
            bool open0 = true, open1 = true;
            while (ok && (open0 || open1)) {
                if (open0) {
                    open0 = f0.live;
                    push(f0, 0, false);
                    if (open0) step(f0, turns[0]);
                }
                if (ok && open1) {
                    open1 = f1.live;
                    push(f1, 1, false);
                    if (open1) step(f1, turns[1]);
                }
            }
            if (!ok && lane == 0) atomicOr(&abort_flag, 1);
            if (bad && lane == 0) atomicOr(&g_status_attend, FLAG_BOUNDS);
        } else if (warp == 8) {
            // ------------------------------------------------------------ producer
            // a lane per copy: its page of the tile, and its 64-column half (bf16), or codes
            // and scales (stored forms)
            const int ppt = kAtKeys >> page_log, my = lane & (ppt - 1), part = lane >> (7 - page_log);
            const bool mine = part < (C::kQuant ? 2 : D / 64);
            const unsigned page_bytes = (unsigned)a.page * (C::kQuant ? C::kCodeRow + C::kScaleRow : 2 * D);
            bool ok = true, live[2] = {true, true};
            unsigned at[2] = {0, 0};
            int n = 0;
            uint64_t* last_bar[C::kQuant ? 2 * R : SK + SV] = {};  // of each place's last copy, with its parity
            unsigned last_turn = 0;
            while (ok && (live[0] || live[1])) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (!ok || !live[g]) continue;
                    ok = item_wait(g, at[g]);
                    if (!ok) break;
                    const AtItem& it = items[g][at[g] % kItems];
                    const int flags = it.flags, head = it.head;
                    const int page = mine ? it.page[my] : -1;
                    __syncwarp();
                    if (lane == 0) item_done(g, at[g]);
                    ++at[g];
                    if (flags & kEnd) {
                        live[g] = false;
                        continue;
                    }
                    if ((flags & kPair) && g == 1) continue;  // the tile is loaded already
                    const int boxes = __popc(__ballot_sync(0xffffffffu, page >= 0 && part == 0));
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int st = C::kQuant ? p * R + n % R : place(p, n);
                        uint64_t* const bar = C::kQuant ? &raw_full[st] : &full[reader(flags, g)][st];
                        if (C::kQuant) {
                            if (n >= R) ok = mbar_wait(&raw_empty[st], (unsigned)(n / R - 1) & 1u);
                        } else if (n >= (p ? SV : SK)) {
                            ok = mbar_wait(&empty[st], released(p, n));
                        }
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(bar, (unsigned)boxes * page_bytes);
                        __syncwarp();
                        if (page >= 0) {
                            if (!C::kQuant) {
                                tma_load_2d(smem + st * C::kTile + part * (kAtKeys * 128) + (my << page_log) * 128,
                                            p ? &tm_v : &tm_k, head * D + 64 * part, page << page_log, bar);
                            } else if (part == 0) {
                                tma_load_2d(rawsm + st * C::kRaw + (my << page_log) * C::kCodeRow, p ? &tm_v : &tm_k,
                                            head * C::kCodeRow, page << page_log, bar);
                            } else {
                                bulk_g2s(rawsm + st * C::kRaw + kAtKeys * C::kCodeRow + (my << page_log) * C::kScaleRow,
                                         a.pool.plane[p].scales +
                                             ((long long)head * a.pool.slots + (page << page_log)) * C::kScaleRow,
                                         (unsigned)a.page * C::kScaleRow, bar);
                            }
                        }
                        const unsigned t = C::kQuant ? (unsigned)(n / R) & 1u : flags & (p ? kValueTurn : kKeyTurn) ? 1u : 0u;
#pragma unroll
                        for (int i = 0; i < (C::kQuant ? 2 * R : SK + SV); ++i)
                            if (i == st) last_bar[i] = bar;
                        last_turn = (last_turn & ~(1u << st)) | (t << st);
                    }
                    ++n;
                }
            }
            if (!ok) {
                // the copies in flight land before this block gives up its shared memory: each
                // place's last one
                for (int st = 0; st < (C::kQuant ? 2 * R : SK + SV); ++st)
                    if (last_bar[st]) mbar_wait(last_bar[st], last_turn >> st & 1u);
                if (lane == 0) atomicOr(&abort_flag, 1);
            }
        } else if (warp == 9 || warp == 11) {
            // ------------------------------------------------------------ queries and MMA issue
            // One warp per softmax group: S = Q K^T, then, once the weights are in tensor
            // memory, O += P V.  While the group works on a tile's weights the warp looks at its
            // next tile and, where that begins a unit, brings the unit's queries.
            const int g = warp == 9 ? 0 : 1;
            constexpr uint32_t id_qk = tc_idesc_bf16(kAtRows, kAtKeys), id_pv = at_idesc_pv(D);
            // descriptors of the group's queries and of the first stage (as keys, K-major, and as
            // values, N-major: 64-column halves 16 KB apart, 8-key groups 1 KB apart); an offset
            // adds to the address field, which all of shared memory fits
            unsigned char* const qt = qsm + g * C::kQ;
            const uint64_t q_desc = tc_smem_desc(qt, 16, 1024, 2), t_desc = tc_smem_desc(smem, 16, 1024, 2);
            const uint64_t v_desc = tc_smem_desc(smem, kAtKeys * 128, 1024, 2);
            const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G;
            bool ok = true;
            unsigned at = 0, units = 0, p_phase = 0;
            int flags = 0, tile = 0;
            // Reads the next item; begins to load its queries where it opens a unit, K-major
            // with the 128-byte swizzle, once the last product with the rows before them is
            // done.  Rows past the unit's keep what they hold (a row of a product depends on its
            // own operand row alone).
            auto open_item = [&]() {
                ok = item_wait(g, at);
                if (!ok) return;
                const AtItem& it = items[g][at % kItems];
                flags = __shfl_sync(0xffffffffu, it.flags, 0);
                tile = __shfl_sync(0xffffffffu, it.tile, 0);
                const int head = it.head, rows = it.rows, row0 = it.row0, agent0 = it.agent0;
                __syncwarp();
                if (lane == 0) item_done(g, at);
                ++at;
                if ((flags & kEnd) || !(flags & kFirst)) return;
                if (units > 0) ok = __all_sync(0xffffffffu, mbar_wait(&q_free[g], (units - 1) & 1u));
                ++units;
                if (!ok) return;
                constexpr int V = D / 8, P = 32 / V;  // 16-byte vectors per row, rows per step
                const int cv = lane % V;
                unsigned char* const dst = qt + (cv / 8) * (kAtRows * 128);
#pragma unroll 1
                for (int r32 = 0; r32 < rows; r32 += 32) {
                    // a lane finds one row's place; then P rows a step
                    const int x = row0 + min(r32 + lane, rows - 1), ag = x / TG, t = (x - ag * TG) / G, m = x - ag * TG - t * G;
                    const long long off = a.qp.row(agent0 + ag, 0, t) + (long long)(head * G + m) * D;
#pragma unroll 4
                    for (int i = 0; i < 32; i += P) {
                        const int k = i + lane / V, r = r32 + k;
                        const long long o = __shfl_sync(0xffffffffu, off, k);
                        if (r < rows) cp_async16(dst + r * 128 + (((cv % 8) ^ (r & 7)) << 4), a.q + o + 8 * cv);
                    }
                }
                cp_async_commit();
            };
            auto queries_here = [&]() {
                cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
            };
            // The tensor pipe takes products in the order of issue.  A group's O += P V and next
            // S = Q K^T go in one piece, so that its softmax waits for those alone and the other
            // group's follow while it works: the two groups settle half a turn apart.  (Pairs: the
            // tensor pipe is what they wait for; 329 against 377 us on 8 x 256 new tokens over
            // 8192 keys.  Units alone wait for memory, and save the lock.)
            auto take_pipe = [&]() {
                if (lane == 0) {
                    const long long t0 = clock64();
                    while (ok && atomicCAS_block(&mma_lock, 0, 1) != 0) ok = clock64() - t0 < kWaitCycles;
                }
                ok = __all_sync(0xffffffffu, ok);
            };
            auto leave_pipe = [&]() {
                if (lane == 0) atomicExch_block(&mma_lock, 0);
                __syncwarp();
            };
            auto keys_here = [&]() {
                ok = __all_sync(0xffffffffu, mbar_wait(&full[reader(flags, g)][place(0, tile)], flags & kKeyTurn ? 1u : 0u));
            };
            // S of the open item (one lane)
            auto logits = [&]() {
                const int ks = place(0, tile);
                const uint64_t bd = t_desc + (uint32_t)ks * (uint32_t)(C::kTile >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk / 4) * (kAtKeys * 128) + 32 * (kk % 4)) >> 4;
                    tc_mma_bf16(tmem + 128 * g, q_desc + off, bd + off, id_qk, kk > 0 ? 1u : 0u);
                }
                tc_commit(&s_full[g]);
                tc_commit(&empty[ks]);
                if (!(flags & kPair)) tc_commit(&empty[ks]);
                if (flags & kLast) tc_commit(&q_free[g]);
            };
            open_item();
            if (ok && !(flags & kEnd)) {
                queries_here();
                keys_here();
                if (ok) {
                    tc_fence_after();
                    if (elect_lane()) logits();
                    __syncwarp();
                }
            }
            while (ok && !(flags & kEnd)) {
                const int now = flags, vs = place(1, tile);
                open_item();
                if (!ok) break;
                const bool more = !(flags & kEnd);
                // all that the two products read, the weights last
                if (more) {
                    if (flags & kFirst) queries_here();
                    keys_here();
                    if (!ok) break;
                }
                ok = mbar_wait(&full[reader(now, g)][vs], now & kValueTurn ? 1u : 0u);
                if (ok) ok = mbar_wait(&p_ready[g], p_phase & 1u);
                p_phase ^= 1u;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (now & kPair) take_pipe();
                if (!ok) break;
                tc_fence_after();
                if (elect_lane()) {
                    const uint64_t bd = v_desc + (uint32_t)vs * (uint32_t)(C::kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < kAtKeys / 16; ++kk)
                        tc_mma_bf16_ta(tmem + 256 + 128 * g, tmem + 128 * g + 8 * kk, bd + (uint32_t)(2048 * kk >> 4), id_pv,
                                       kk > 0 || !(now & kFirst) ? 1u : 0u);
                    tc_commit(&empty[vs]);
                    if (!(now & kPair)) tc_commit(&empty[vs]);
                    if (now & kLast) tc_commit(&o_full[g]);
                    if (more) logits();
                }
                __syncwarp();
                if (now & kPair) leave_pipe();
            }
            if (!ok && lane == 0) atomicOr(&abort_flag, 1);
        } else if (C::kQuant) {
            // ------------------------------------------------------------ conversion
            // one team of warps converts the key tiles, another the value tiles
            constexpr int N = 32 * C::kConvWarps;
            const int p = (int)(threadIdx.x - 384) / N, tid = (int)(threadIdx.x - 384) % N;
            bool ok = true, live[2] = {true, true};
            unsigned at[2] = {0, 0};
            int n = 0;
            while (ok && (live[0] || live[1])) {
#pragma unroll 1
                for (int g = 0; g < 2; ++g) {
                    if (!ok || !live[g]) continue;
                    ok = item_wait(g, at[g]);
                    if (!ok) break;
                    const AtItem& it = items[g][at[g] % kItems];
                    const int flags = it.flags, keys = it.keys;
                    const unsigned absent = it.absent;
                    __syncwarp();
                    if (lane == 0) item_done(g, at[g]);
                    ++at[g];
                    if (flags & kEnd) {
                        live[g] = false;
                        continue;
                    }
                    if ((flags & kPair) && g == 1) continue;
                    const int rs = p * R + n % R, st = place(p, n);
                    ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[rs], (unsigned)(n / R) & 1u));
                    if (!ok) break;
                    StoredTile<F, D, N> stored;
                    stored.take(rawsm + rs * C::kRaw, tid);
                    mbar_arrive(&raw_empty[rs]);
                    if (n >= (p ? SV : SK)) ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], released(p, n)));
                    if (!ok) break;
                    stored.put(smem + st * C::kTile, tid, keys, absent);
                    fence_proxy_async_smem();
                    mbar_arrive(&full[reader(flags, g)][st]);
                    ++n;
                }
            }
            if (!ok && lane == 0) atomicOr(&abort_flag, 1);
        }
    } else {
        regs_inc<C::kRegsSoftmax>();
        // ---------------------------------------------------------------- softmax
        const int g = warp >> 2, wq = warp & 3, row = 32 * wq + lane;  // group, TMEM lane quarter, row
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t s_at = tmem + lanes + 128 * g, o_at = tmem + lanes + 256 + 128 * g;
        const float c = a.scale_log2;
        const float2 c2 = make_float2(c, c);
        bool ok = true;
        unsigned at = 0, units = 0;
        int rows = 0, sees = 0;   // of the unit: the group's rows; keys this row sees
        float m = -INFINITY, l = 0.f;
        while (true) {
            ok = item_wait(g, at);
            if (!ok) break;
            const AtItem& it = items[g][at % kItems];
            const int flags = it.flags;
            if (flags & kEnd) break;
            const int keys = it.keys, key0 = it.key0, tile = it.tile;
            const unsigned absent = it.absent;
            if (flags & kFirst) {
                rows = it.rows;
                m = -INFINITY;
                l = 0.f;
                sees = 0;
                if (row < rows) {
                    const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G;
                    const int x = it.row0 + row, ag = x / TG, t = (x - ag * TG) / G;
                    if (flags & kPrefix) {
                        // the new tokens stand at the end of the sequence: with fewer own keys
                        // than new tokens the first ones miss part of the prefix
                        bool ignore = false;
                        const int own = clamp_len(__ldg(a.suffix_len + it.agent0 + ag), (long long)a.max_suffix_pages * a.page, ignore);
                        sees = max(0, min(it.sees0, it.sees0 + own - T + 1 + t));
                    } else {
                        sees = max(0, it.sees0 + t);
                    }
                }
            }
            const bool warp_live = 32 * wq < rows;
            const int nv = sees - key0;  // columns this row sees
            const bool whole = absent == 0u && keys == kAtKeys;
            ok = __all_sync(0xffffffffu, mbar_wait(&s_full[g], at & 1u));
            if (!ok) break;
            tc_fence_after();
            if (!C::kQuant && !whole) {
                // value rows that hold no key read as zero: a weight of 0 times what lies there
                // (anything, NaN too) would not be 0
                const int st = place(1, tile);
                ok = __all_sync(0xffffffffu, mbar_wait(&full[reader(flags, g)][st], flags & kValueTurn ? 1u : 0u));
                if (!ok) break;
                if (row >= keys || ((absent >> (row >> 4)) & 1u)) {
                    unsigned char* vt = smem + st * C::kTile + row * 128;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<uint4*>(vt + h * (kAtKeys * 128) + 16 * k) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            if (warp_live) {
                // two sweeps over the row in 32-column pieces, the next piece on its way while
                // one is worked on: the maximum, then the weights
                uint32_t x[2][32];
                float mx = -INFINITY;
                if (__any_sync(0xffffffffu, absent != 0u || nv < kAtKeys)) {
                    // columns that hold no key, or none that this row sees: -inf (on the side, so
                    // that the sweeps' code stays small)
#pragma unroll 1
                    for (int c0 = 0; c0 < kAtKeys; c0 += 32) {
                        tmem_ld32(s_at + c0, x[0]);
                        tmem_wait_ld32(x[0]);
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int n = (absent >> (c0 / 16 + b)) & 1u ? 0 : nv - c0 - 16 * b;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (i >= n) x[0][16 * b + i] = 0xff800000u;
                        }
                        tmem_st32(s_at + c0, x[0]);
                    }
                    tmem_wait_st();
                }
                tmem_ld32(s_at, x[0]);
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        tmem_wait_ld32(x[k]);
                        const int at32 = 64 * h + 32 * k;
                        if (at32 < 96) tmem_ld32(s_at + at32 + 32, x[1 - k]);
                        float m4[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) m4[i] = fmaxf(__uint_as_float(x[k][i]), __uint_as_float(x[k][i + 4]));
#pragma unroll
                        for (int i = 8; i < 32; i += 8)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                m4[q] = fmaxf(fmaxf(__uint_as_float(x[k][i + q]), __uint_as_float(x[k][i + 4 + q])), m4[q]);
                        mx = fmaxf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), mx);
                    }
                }
                tmem_ld32(s_at, x[0]);
                const float z = mx * c;
                const bool raise = z > m + kAtSlack || (m == -INFINITY && z > m);
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise ? ex2(m - z) : 1.f;  // m = -inf: 0
                    if (raise) {
                        m = z;
                        l *= f;
                    }
                    if (!(flags & kFirst)) {
#pragma unroll 1
                        for (int i = 0; i < D; i += 32) {
                            tmem_ld32(o_at + i, x[1]);
                            tmem_wait_ld32(x[1]);
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[1][k] = __float_as_uint(__uint_as_float(x[1][k]) * f);
                            tmem_st32(o_at + i, x[1]);
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.f : -m;
                const float2 off2 = make_float2(off, off);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        tmem_wait_ld32(x[k]);
                        const int at32 = 64 * h + 32 * k;
                        if (at32 < 96) tmem_ld32(s_at + at32 + 32, x[1 - k]);
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 y = fma2(make_float2(__uint_as_float(x[k][2 * i]), __uint_as_float(x[k][2 * i + 1])), c2, off2);
                            y.x = ex2(y.x);
                            y.y = ex2(y.y);
                            sum[i & 1] = add2(sum[i & 1], y);
                            pk[i] = pack_bf16(y.x, y.y);
                        }
                        // over logits of this piece or an earlier one
                        tmem_st16(s_at + at32 / 2, pk);
                    }
                }
                l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                tmem_wait_st();
            }
            tc_fence_before();
            mbar_arrive(&p_ready[g]);
            if (flags & kLast) {
                const long long part = it.part;
                ok = __all_sync(0xffffffffu, mbar_wait(&o_full[g], units & 1u));
                if (!ok) break;
                ++units;
                tc_fence_after();
                if (warp_live) {
                    // 16 rows x 64 columns a load, 8 bytes of a row per lane: a store writes eight
                    // rows' 32-byte sectors (a lane per row would write 32 rows' 16 bytes: 15000
                    // cycles for the 128 rows against 3000)
                    const int pair_col = 2 * (lane & 3);
#pragma unroll 1
                    for (int i = 0; i < 2 * (D / 64); ++i) {
                        const int r = 32 * wq + 16 * (i & 1) + lane / 4, c0 = 64 * (i / 2) + pair_col;
                        uint32_t o[32];
                        tmem_ld_16x64(o_at + ((uint32_t)(16 * (i & 1)) << 16) + 64 * (i / 2), o);
                        tmem_wait_ld32(o);
                        float* out = w.o + (part + r) * D + c0;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            if (r < rows) *reinterpret_cast<uint2*>(out + 8 * k) = make_uint2(o[4 * k], o[4 * k + 1]);
                            if (r + 8 < rows) *reinterpret_cast<uint2*>(out + 8 * D + 8 * k) = make_uint2(o[4 * k + 2], o[4 * k + 3]);
                        }
                    }
                    if (row < rows) w.ml[part + row] = make_float2(m, l);
                    tc_fence_before();
                }
            }
            __syncwarp();
            if (lane == 0) item_done(g, at);
            ++at;
        }
        if (!ok && lane == 0) atomicOr(&abort_flag, 1);
    }
    // The roles end in their own ways: a barrier that counts threads, not warps, for the one that
    // stands before the tensor memory goes (a warp that reached an aligned barrier in two parts
    // would count twice, and the memory would go under a group still reading it).
    tc_fence_before();
    __syncwarp();
    asm volatile("barrier.sync 0;" ::: "memory");
    __syncwarp();
    tc_fence_after();
    if (abort_flag && threadIdx.x == 0) atomicOr(&g_status_attend, FLAG_TIMEOUT);
    if (warp == 9) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join
// A warp takes RPW consecutive rows (new token, query head) of an agent's KV head, whose parts
// lie side by side: their prefix's parts, then their suffix's; its lanes first read up to 32
// parts' (max, sum), then each part's O rows.  With few rows WPR warps share the parts of one
// row (a long prefix has as many as there are pieces in its head's share of the line); with
// many rows each has few parts, and several rows per warp share the look-ups.
template <int D, int WPR, int RPW>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendArgs a,
                                                          const __grid_constant__ AtWork w) {
    static_assert(WPR == 1 || RPW == 1, "shared parts or shared rows");
    constexpr int V = D / 32;  // values per lane
    __shared__ float sh_m[4], sh_l[4], sh_acc[4][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
    const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G, H = a.pool.heads;
    const int chunks = (TG + RPW - 1) / RPW;
    const long long id = (long long)blockIdx.x * (4 / WPR) + warp / WPR;
    const bool live = id < (long long)a.agents * H * chunks;
    const long long ah = live ? quotient(id, chunks) : 0;
    const int in0 = live ? (int)(id - ah * chunks) * RPW : 0, rows = min(RPW, TG - in0);
    const int agent = (int)quotient(ah, H), head = (int)(ah - (long long)agent * H);
    const long long all = (long long)a.agents * TG;
    // The plan lies ready before this kernel can start (the attention kernel lets it start only
    // after its own wait for the plan); only the parts need the wait below.
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
    const int many_ctas = w.plan->many_ctas;
    // where the parts of row r of a segment (block-wise the same for its neighbours) lie
    struct Place {
        long long own;  // part row of the segment's row 0, first part
        long long i0;   // first piece
        int n, kind, row0;
    };
    auto find = [&](int s, int r, int seg, int agent0, int seg_rows) {
        Place p = {0, 0, 0, 0, 0};
        const int block = r / kAtBlock;
        const int k = at_kind(seg_rows - block * kAtBlock, w.few);
        p.kind = k;
        const int2 first = w.first[seg];
        const AtEntry e = w.entries[k][k == kPairs ? first.x + block : first.y];
        if (e.tiles == 0) return p;
        const long long chunk = w.plan->chunk[k];
        const long long base = e.begin + (long long)head * (e.tiles + at_pad(k));
        p.own = (s * H + (long long)head) * all + (long long)agent0 * TG;
        p.i0 = quotient(base, chunk);
        p.n = (int)(quotient(base + e.tiles - 1, chunk) - p.i0) + 1;  // pieces that hold tiles
        p.row0 = e.row0;
        return p;
    };
    int seg[2] = {group, a.groups + agent}, agent0[2] = {agent, agent}, seg_rows[2] = {0, TG};
    Place at[2] = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (!live || (s == 0 && group < 0)) continue;
        if (s == 0) {
            agent0[0] = w.bounds[group];
            seg_rows[0] = (w.bounds[group + 1] - agent0[0]) * TG;
        }
        at[s] = find(s, (agent - agent0[s]) * TG + in0, seg[s], agent0[s], seg_rows[s]);
    }
    pdl_wait();
    float M[RPW], L[RPW], acc[RPW][V];
#pragma unroll
    for (int q = 0; q < RPW; ++q) {
        M[q] = -INFINITY;
        L[q] = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[q][i] = 0.f;
    }
    // first part row of the segment's rows from r0 on, in the j-th piece that holds them
    auto part_of = [&](const Place& p, int j, int r0) {
        if (j == 0) return p.own + r0;
        const long long i = p.i0 + j;
        if (p.kind == kFew) return w.few_rows + i * w.few + (r0 - p.row0);
        const int half = p.kind == kSingles && i >= many_ctas ? 1 : 0, cta = (int)i - half * many_ctas;
        return w.own_rows + (long long)cta * (2 * kAtBlock) + (p.kind == kPairs ? 0 : kAtBlock + kAtRows * half) + (r0 - p.row0);
    };
    if constexpr (RPW > 1) {
        // few parts per row: one after another, the next one's rows on their way
        struct Part {
            float2 ml[RPW];
            float x[RPW][V];
        };
        int s = -1, q0 = rows, q1 = rows, j = 0;  // the segment, its rows in one block, their part
        Place p = {0, 0, 0, 0, 0};
        auto fetch = [&](Part& d) {
            for (++j; j >= p.n || q0 >= rows;) {
                q0 = q1;
                if (q0 >= rows) {
                    if (++s > 1) return false;
                    q0 = 0;
                    if (!live || (s == 0 && group < 0)) {
                        q0 = q1 = rows;
                        continue;
                    }
                }
                const int r0 = (agent - agent0[s]) * TG + in0;
                q1 = min(rows, (r0 + q0) / kAtBlock * kAtBlock + kAtBlock - r0);
                p = q0 == 0 ? at[s] : find(s, r0 + q0, seg[s], agent0[s], seg_rows[s]);
                j = 0;
            }
            const long long part = part_of(p, j, (agent - agent0[s]) * TG + in0);
#pragma unroll
            for (int q = 0; q < RPW; ++q) {
                const bool in = q >= q0 && q < q1;
                d.ml[q] = in ? __ldcg(w.ml + part + q) : make_float2(-INFINITY, 0.f);
                const float* src = w.o + (part + q) * D + V * lane;
                if (V == 4) {
                    const float4 v = in ? __ldcg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    d.x[q][0] = v.x;
                    d.x[q][1] = v.y;
                    d.x[q][V - 2] = v.z;
                    d.x[q][V - 1] = v.w;
                } else {
                    const float2 v = in ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
                    d.x[q][0] = v.x;
                    d.x[q][1] = v.y;
                }
            }
            return true;
        };
        Part now;
        bool have = fetch(now);
        while (have) {
            Part next;
            const bool more = fetch(next);
#pragma unroll
            for (int q = 0; q < RPW; ++q) {
                const float2 ml = now.ml[q];
                if (ml.y == 0.f) continue;  // (a row with a NaN logit has l = NaN and must keep it)
                const float N = fmaxf(M[q], ml.x);
                const float f = M[q] == -INFINITY ? 1.f : exp2f(M[q] - N);  // (nothing there yet, or NaN)
                const float wt = ml.x == -INFINITY ? 1.f : exp2f(ml.x - N);
                M[q] = N;
                L[q] = L[q] * f + ml.y * wt;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[q][i] = fmaf(now.x[q][i], wt, acc[q][i] * f);
            }
            now = next;
            have = more;
        }
    } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (!live || (s == 0 && group < 0)) continue;
        const int r0 = (agent - agent0[s]) * TG + in0;
        for (int q0 = 0; q0 < rows;) {  // once, or twice where the rows straddle two blocks
            const int q1 = min(rows, (r0 + q0) / kAtBlock * kAtBlock + kAtBlock - r0);
            Place p = at[s];
            if (q0 > 0) p = find(s, r0 + q0, seg[s], agent0[s], seg_rows[s]);
            for (int j0 = sub; j0 < p.n; j0 += 32 * WPR) {
                const int j = j0 + lane * WPR;
                const bool in_unit = j < p.n;
                const long long part = in_unit ? part_of(p, j, r0) : 0;
                float wt[RPW];
                unsigned has[RPW], any = 0;
#pragma unroll
                for (int q = 0; q < RPW; ++q) {
                    float2 ml = make_float2(-INFINITY, 0.f);
                    if (in_unit && q >= q0 && q < q1) ml = __ldcg(w.ml + part + q);
                    float top = ml.x;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const float N = fmaxf(M[q], top);
                    const float f = M[q] == -INFINITY ? 0.f : exp2f(M[q] - N);
                    wt[q] = ml.x == -INFINITY ? 0.f : exp2f(ml.x - N);
                    // (a row with a NaN logit has l = NaN and must keep it)
                    float sum = ml.y == 0.f ? 0.f : ml.y * (ml.x == -INFINITY ? 1.f : wt[q]);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (top != -INFINITY || !(sum == 0.f)) {
                        L[q] = L[q] * (M[q] == -INFINITY ? (L[q] == 0.f ? 0.f : 1.f) : f) + sum;
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[q][i] *= f;
                        M[q] = N;
                    }
                    has[q] = __ballot_sync(0xffffffffu, !(ml.y == 0.f));
                    any |= has[q];
                }
                const int count = 32 - __clz(any);
                constexpr int B = 8;  // parts whose rows are on their way at once
#pragma unroll 1
                for (int b0 = 0; b0 < count; b0 += B) {
                    float x[B][RPW][V], wb[B][RPW];
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        const long long row = __shfl_sync(0xffffffffu, part, (b0 + b) & 31);
#pragma unroll
                        for (int q = 0; q < RPW; ++q) {
                            const bool there = b0 + b < count && ((has[q] >> ((b0 + b) & 31)) & 1u);
                            wb[b][q] = __shfl_sync(0xffffffffu, wt[q], (b0 + b) & 31);
                            if (!there) wb[b][q] = 0.f;
                            const float* src = w.o + (row + q) * D + V * lane;
                            if (V == 4) {
                                const float4 v = there ? __ldcg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
                                x[b][q][0] = v.x;
                                x[b][q][1] = v.y;
                                x[b][q][V - 2] = v.z;
                                x[b][q][V - 1] = v.w;
                            } else {
                                const float2 v = there ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
                                x[b][q][0] = v.x;
                                x[b][q][1] = v.y;
                            }
                        }
                    }
#pragma unroll
                    for (int b = 0; b < B; ++b)
#pragma unroll
                        for (int q = 0; q < RPW; ++q)
#pragma unroll
                            for (int i = 0; i < V; ++i) acc[q][i] = fmaf(x[b][q][i], wb[b][q], acc[q][i]);
                }
            }
            q0 = q1;
        }
    }
    }
    if (WPR > 1) {
        if (lane == 0) {
            sh_m[warp] = M[0];
            sh_l[warp] = L[0];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sh_acc[warp][V * lane + i] = acc[0][i];
        __syncthreads();
        if (sub != 0) return;
        float N = M[0];
#pragma unroll
        for (int x = 1; x < WPR; ++x) N = fmaxf(N, sh_m[warp + x]);
        const float f = M[0] == -INFINITY ? 1.f : exp2f(M[0] - N);  // (M = -inf: L is 0, or NaN)
        L[0] *= f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[0][i] *= f;
#pragma unroll
        for (int x = 1; x < WPR; ++x) {
            const float mx = sh_m[warp + x], fx = mx == -INFINITY ? 1.f : exp2f(mx - N);
            L[0] += sh_l[warp + x] * fx;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[0][i] = fmaf(sh_acc[warp + x][V * lane + i], fx, acc[0][i]);
        }
        M[0] = N;
    }
    if (!live) return;
#pragma unroll
    for (int q = 0; q < RPW; ++q) {
        if (q >= rows) continue;
        const int in = in0 + q, t = in / G, qh = head * G + in - t * G;
        const float inv = L[q] == 0.f ? 0.f : 1.f / L[q];
        const long long oo = a.op.row(agent, 0, t) + (long long)qh * D + V * lane;
        if (V == 4)
            *reinterpret_cast<uint2*>(a.out + oo) = make_uint2(pack_bf16(acc[q][0] * inv, acc[q][1] * inv),
                                                               pack_bf16(acc[q][V - 2] * inv, acc[q][V - 1] * inv));
        else
            *reinterpret_cast<uint32_t*>(a.out + oo) = pack_bf16(acc[q][0] * inv, acc[q][1] * inv);
        if (a.lse && lane == 0)
            a.lse[((long long)agent * T + t) * a.q_heads + qh] = L[q] == 0.f ? -INFINITY : (M[q] + log2f(L[q])) * 0.69314718055994531f;
    }
}

// ------------------------------------------------------------------ host
size_t attend_workspace_bytes(int agents, int T, int q_heads, int kv_heads, int head_dim, int groups) {
    return at_layout(agents, T, q_heads, kv_heads, head_dim, groups).bytes;
}

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

// A kernel's dynamic shared memory, once per device (a form has one kernel of each K).
template <int F, int D, int K, typename Kernel>
static cudaError_t allow_smem(Kernel* kernel, int bytes, int device) {
    static std::atomic<unsigned long long> ready{0};
    const unsigned long long bit = 1ull << (device & 63);
    if ((ready.load(std::memory_order_acquire) & bit) && device <= 63) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
    return e;
}

template <int F, int D, int NT>
static cudaError_t launch_few(const AttendArgs& a, const AtWork& w, int device, cudaStream_t s) {
    using C = FewCfg<F, D>;
    const cudaError_t e = allow_smem<F, D, NT>(attend_few_kernel<F, D, NT>, C::kSmem, device);
    if (e != cudaSuccess) return e;
    return launch_chained(attend_few_kernel<F, D, NT>, dim3(w.ctas), dim3(32 * kFewWarps), C::kSmem, s, a, w);
}

template <int F, int D>
static cudaError_t launch_attend_form(const AttendArgs& a, const AtWork& w, int device, cudaStream_t s) {
    using C = AtCfg<F, D>;
    cudaError_t e;
    if ((e = launch_chained(attend_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, w)) != cudaSuccess) return e;
    if (w.many) {
        CUtensorMap mk, mv;
        if (!pool_map<F, D>(&mk, a.pool, 0, a.page) || !pool_map<F, D>(&mv, a.pool, 1, a.page)) return cudaErrorInvalidValue;
        if ((e = allow_smem<F, D, 0>(attend_kernel<F, D>, C::kSmem, device)) != cudaSuccess) return e;
        e = launch_chained(attend_kernel<F, D>, dim3(w.ctas), dim3(C::kThreads), C::kSmem, s, mk, mv, a, w);
        if (e != cudaSuccess) return e;
    }
    if (w.few > 0) {
        e = w.few == 8 ? launch_few<F, D, 1>(a, w, device, s) : launch_few<F, D, 2>(a, w, device, s);
        if (e != cudaSuccess) return e;
    }
    const long long rows = (long long)a.agents * a.new_tokens * a.q_heads;
    // four warps per row while that leaves them all resident (48 rows of 32 heads, 1536, join in
    // 7 us less by one), one while rows are few
    if (rows <= (long long)w.ctas * 8) return launch_chained(attend_join_kernel<D, 4, 1>, dim3((unsigned)rows), dim3(128), 0, s, a, w);
    const int tg = a.new_tokens * (a.q_heads / a.pool.heads);
    if (tg >= 4 && rows > (long long)w.ctas * 128) {
        const long long warps = (long long)a.agents * a.pool.heads * ((tg + 3) / 4);
        return launch_chained(attend_join_kernel<D, 1, 4>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, s, a, w);
    }
    return launch_chained(attend_join_kernel<D, 1, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, a, w);
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
    w.first = (int2*)(base + l.first);
    w.bounds = (int*)(base + l.bounds);
    for (int k = 0; k < 3; ++k) w.entries[k] = (AtEntry*)(base + l.entries[k]);
    w.ml = (float2*)(base + l.ml);
    w.o = (float*)(base + l.o);
    w.own_rows = l.own_rows;
    w.few_rows = l.few_rows;
    w.few = l.few;
    w.many = l.many;
    w.ctas = sms < kAtMaxCtas ? sms : kAtMaxCtas;
    switch (a.pool.format * 2 + (a.pool.dim == 128)) {
        case KVFIX_POOL_BF16 * 2: return launch_attend_form<KVFIX_POOL_BF16, 64>(a, w, dev, s);
        case KVFIX_POOL_BF16 * 2 + 1: return launch_attend_form<KVFIX_POOL_BF16, 128>(a, w, dev, s);
        case KVFIX_POOL_E4M3 * 2: return launch_attend_form<KVFIX_POOL_E4M3, 64>(a, w, dev, s);
        case KVFIX_POOL_E4M3 * 2 + 1: return launch_attend_form<KVFIX_POOL_E4M3, 128>(a, w, dev, s);
        case KVFIX_POOL_INT4 * 2: return launch_attend_form<KVFIX_POOL_INT4, 64>(a, w, dev, s);
        default: return launch_attend_form<KVFIX_POOL_INT4, 128>(a, w, dev, s);
    }
}

}  // namespace kvfix
