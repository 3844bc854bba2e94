// attend_few.cuh -- kvfix_shared_attend for small blocks of query rows, up to AtWork::few (8 or
// 16) of them: an agent's own tokens while it decodes, and a short round's prefix.
//
// Mathematics.  The products are turned around: logits are S^T = K Q^T (keys along the rows of the
// matrix instruction, queries along its 8 columns) and the output O^T = V^T P^T, so few queries
// leave nothing of an instruction empty that costs more than the keys' own loading.
//
// Layout.  A warp takes 16 keys at a time, alone, without barriers.  The order of a
// contraction's terms is free, so lane (g = lane / 4, t = lane % 4) takes up to 16 contiguous
// bytes of key rows g and g + 8 as its own terms of consecutive instructions, and of value rows
// 2t, 2t+1, 2t+8, 2t+9 the same D/8 values, which are its rows of consecutive instructions:
// copies are as wide as the rows allow, a lane reads from shared memory only what it copied
// there itself (scales excepted), and stored codes become operands in the registers that feed
// the tensor cores: int4 as bf16, e4m3 as f16, which holds every code.  A logit's key belongs
// to one lane, so an e4m3 row's scales are one multiplication of the logit and one exponent
// added in the weight; maxima are lanes' own until a row's has to be raised.  Weights go from
// the logits' layout to the operand's by movmatrix.
//
// What bounds it: latency and the issue of its instructions, about 350 for 16 keys of an e4m3
// head of 128 (IPC 1.6 of 4, HBM at half its rate).  48 agents' own keys (200 MB of e4m3, 4 rows
// each): 45 us beside a prefix's kernel, 66 us for the call, 136 when 128-row tiles held these
// rows.  The next tiles' loads in registers instead of a ring in shared memory cost 2 us more,
// e4m3 as bf16 operands 7.
#pragma once

#include "attend_plan.cuh"

namespace kvfix {

// C += A B, bf16 or f16 operands.
template <bool HALF>
__device__ __forceinline__ void mma_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    if constexpr (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes to two f16 pairs: every code is an f16 value.
__device__ __forceinline__ uint2 e4m3x4_to_f16(uint32_t codes) {
    uint2 y;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}"
        : "=r"(y.x), "=r"(y.y)
        : "r"(codes));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int F, int D>
struct FewCfg {
    static constexpr int kRow = F == KVFIX_POOL_BF16 ? 2 * D : F == KVFIX_POOL_E4M3 ? D : D / 2;  // bytes
    static constexpr int kKeyBytes = kRow / 4 < 16 ? kRow / 4 : 16;   // of one load of a key row
    static constexpr int kKeyLoads = kRow / 4 / kKeyBytes;
    static constexpr int kKeyVals = kKeyBytes * D / kRow;             // values in it
    static constexpr int kValBytes = kRow / 8 < 16 ? kRow / 8 : 16;
    static constexpr int kValLoads = kRow / 8 / kValBytes;
    static constexpr int kValVals = kValBytes * D / kRow;
    static constexpr int kScaleBytes = F == KVFIX_POOL_E4M3 ? 1 : F == KVFIX_POOL_INT4 ? D / 8 : 0;  // of a row
    // A warp's ring of tiles on their way: codes as the lanes copied them, then scales by key.
    static constexpr int kKeyPart = 16 * kRow, kScalePart = 16 * kScaleBytes;
    static constexpr int kStage = 2 * kKeyPart + 2 * kScalePart;
    static constexpr int kStages = F == KVFIX_POOL_BF16 && D == 128 ? 3 : 4;
    static constexpr int kSmem = kFewWarps * kStages * kStage;
};

// N (4, 8, 16) bytes from global to shared memory; nothing is read, and zeros come, where `there`
// is false.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const unsigned char* src, bool there) {
    const int n = there ? N : 0;
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}

template <int N>
__device__ __forceinline__ void read_words(uint32_t* w, const unsigned char* p) {
    if constexpr (N == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// NT: groups of 8 queries.
template <int F, int D, int NT>
__global__ void __launch_bounds__(32 * kFewWarps, 1)
    attend_few_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ AtWork w) {
    using C = FewCfg<F, D>;
    constexpr bool kE4m3 = F == KVFIX_POOL_E4M3, kInt4 = F == KVFIX_POOL_INT4;
    constexpr int KW = C::kKeyBytes / 4, VW = C::kValBytes / 4;
    constexpr int kScaleBytes = C::kScaleBytes;
    extern __shared__ __align__(128) unsigned char few_smem[];
    unsigned char* const ring = few_smem + (threadIdx.x >> 5) * (C::kStages * C::kStage);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    constexpr int kSteps = D / 16;  // products of 16 along D; blocks of 16 values of the output
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int G = a.q_heads / a.pool.heads, T = a.new_tokens, TG = T * G;
    const long long all = (long long)a.agents * TG;
    const int page_log = 31 - __clz(a.page), pool_pages = a.pool.slots >> page_log;
    const float c = a.scale_log2;
    bool bad = false;
    // (the plan lies ready: the kernel before waited for it before it let this one start)
    if (!w.many) pdl_wait();
    pdl_trigger();
    AtWalk walk;
    walk.open(w.plan->start[3][blockIdx.x], w.entries[kFew], a.pool.heads, kFew);
    const long long piece = w.plan->chunk[kFew];
    const long long slot_row = w.few_rows + ((long long)blockIdx.x * kFewWarps + warp) * w.few;
    walk.lo += piece * warp;
    walk.hi = min(walk.hi, walk.lo + piece);
    int head, t0, t1;
    while (walk.next(head, t0, t1)) {
        const AtEntry e = walk.rec;
        const bool prefix = e.seg < a.groups;
        const int32_t* pages = prefix ? a.prefix_pages + (long long)e.seg * a.max_prefix_pages
                                      : a.suffix_pages + (long long)e.agent0 * a.max_suffix_pages;
        // pages of 32 tiles, one a lane, and of the next 32
        auto fetch_pages = [&](int tile) {
            const int i = tile + lane;
            return i < t1 ? __ldg(pages + (i >> (page_log - 4))) : 0;
        };
        int page_now = fetch_pages(t0), page_next = fetch_pages(t0 + 32);

        // this lane's places in a tile's first rows
        const unsigned char* const k0 = a.pool.plane[0].codes + (long long)head * C::kRow + g * a.pool.ss + t * C::kKeyBytes;
        const unsigned char* const v0 = a.pool.plane[1].codes + (long long)head * C::kRow + 2 * t * a.pool.ss + g * C::kValBytes;
        // its 16 bytes of a tile's scales: keys' then values' (lanes beyond have none)
        constexpr int kScaleCopies = C::kScalePart / 16;
        const unsigned char* const s0 = a.pool.plane[lane >= kScaleCopies].scales + (long long)head * a.pool.slots * kScaleBytes +
                                        (lane >= kScaleCopies ? lane - kScaleCopies : lane) * 16;
        unsigned gone = 0;  // by tile mod 32: a tile on its way whose page is not there
        auto load = [&](int tile) {
            const int at = tile - t0;
            if (tile < t1) {
                if ((at & 31) == 0 && at > 0) {
                    page_now = page_next;
                    page_next = fetch_pages(tile + 32);
                }
                const int page = __shfl_sync(0xffffffffu, page_now, at & 31);
                const bool stray = page < 0 || page >= pool_pages;
                bad |= stray;
                gone = (gone & ~(1u << (tile & 31))) | ((stray ? 1u : 0u) << (tile & 31));
                const int keys = stray ? 0 : min(16, e.keys - tile * 16);
                const long long slot = stray ? 0 : (long long)page * a.page + ((tile * 16) & (a.page - 1));
                const uint32_t dst = ring_at + at % C::kStages * C::kStage;
                const unsigned char* const pk = k0 + slot * a.pool.ss;
                const unsigned char* const pv = v0 + slot * a.pool.ss;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < C::kKeyLoads; ++i)
                        copy_async<C::kKeyBytes>(dst + (r * C::kKeyLoads + i) * 32 * C::kKeyBytes + lane * C::kKeyBytes,
                                                 pk + 8 * r * a.pool.ss + i * 4 * C::kKeyBytes, g + 8 * r < keys);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = (r & 1) + 8 * (r >> 1);
#pragma unroll
                    for (int i = 0; i < C::kValLoads; ++i)
                        copy_async<C::kValBytes>(dst + C::kKeyPart + (r * C::kValLoads + i) * 32 * C::kValBytes + lane * C::kValBytes,
                                                 pv + row * a.pool.ss + i * 8 * C::kValBytes, 2 * t + row < keys);
                }
                if (kScaleCopies > 0 && lane < 2 * kScaleCopies)
                    copy_async<16>(dst + 2 * C::kKeyPart + lane * 16, s0 + slot * kScaleBytes, true);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        __syncwarp();
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) load(t0 + i);

        // queries, and how many keys each of this lane's columns sees
        uint32_t qf[NT][kSteps][2];
        int sees[NT][2];
        // running maxima of the logits, and of the logits with the values' exponents (e4m3); sums
        float m[NT][2], my[NT][2], l[NT][2], o[kSteps][NT][4];
        float unit[NT][2];  // what a product of a query and a key's codes counts, in base-2 logits
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            const bool there = r < e.rows;
            const int row = e.row0 + (there ? r : 0), ag = row / TG, in = row - ag * TG, tok = in / G;
            const uint16_t* src = a.q + a.qp.row(e.agent0 + ag, 0, tok) + (long long)(head * G + in - tok * G) * D;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                constexpr int kPer = C::kKeyVals / 4;  // steps of one load
                const int d = (s / kPer) * 4 * C::kKeyVals + t * C::kKeyVals + (s % kPer) * 4;
                const uint2 v = there ? __ldg(reinterpret_cast<const uint2*>(src + d)) : make_uint2(0, 0);
                qf[n][s][0] = v.x;
                qf[n][s][1] = v.y;
            }
            if (kE4m3) {
                // f16 has the codes exactly, and a query after division by its row's power of two:
                // 2^12 at its largest, so all 8 bits down to 2^-26 of that, and never infinite
                uint32_t top = 0;
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int x = 0; x < 2; ++x) top = max(top, max(qf[n][s][x] & 0x7fffu, (qf[n][s][x] >> 16) & 0x7fffu));
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                // exponent field of the largest; an infinity or NaN stays one
                const int ex = min(max((int)(top >> 7), 16), 254) - 127;
                const float down0 = pow2f((12 - ex) / 2), down1 = pow2f((12 - ex) - (12 - ex) / 2);
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        qf[n][s][x] = pack_f16(__uint_as_float(qf[n][s][x] << 16) * down0 * down1,
                                               __uint_as_float(qf[n][s][x] & 0xffff0000u) * down0 * down1);
                // (a column's lanes: its query's power lies in lanes 4 (2t + x) ...)
#pragma unroll
                for (int x = 0; x < 2; ++x) unit[n][x] = c * pow2f(__shfl_sync(0xffffffffu, ex - 12, 4 * (2 * t + x)));
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // The new tokens stand at the end of the sequence: new token i sees the own keys up
                // to its own, and with fewer own keys than new tokens the first ones miss part of
                // the prefix.
                const int col = 8 * n + 2 * t + x, rc = e.row0 + col, ag = rc / TG, tok = (rc - ag * TG) / G;
                if (col >= e.rows) {
                    sees[n][x] = 0;
                } else if (prefix) {
                    bool ignore = false;
                    const int mine = clamp_len(__ldg(a.suffix_len + e.agent0 + ag), (long long)a.max_suffix_pages * a.page, ignore);
                    sees[n][x] = min(e.keys, e.keys + mine - T + 1 + tok);
                } else {
                    sees[n][x] = e.keys - (e.row0 + e.rows - 1) / G + rc / G;
                }
                m[n][x] = my[n][x] = -INFINITY;
                if (!kE4m3) unit[n][x] = c;
                l[n][x] = 0.f;
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[s][n][x] = 0.f;
        }

#pragma unroll 1
        for (int tile = t0; tile < t1; ++tile) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
            __syncwarp();  // the scales come from several lanes; and the tile before is read by all
            load(tile + C::kStages - 1);
            const unsigned char* const st_k = ring + (tile - t0) % C::kStages * C::kStage;
            const unsigned char* const st_v = st_k + C::kKeyPart;
            const unsigned char* const st_s = st_k + 2 * C::kKeyPart;
            const int keys_here = (gone >> (tile & 31)) & 1u ? 0 : min(16, e.keys - tile * 16);
            uint32_t ksz[2], vsz[4];
            if (kInt4) {
                // (rows that are not there are zeros, whatever their scales hold)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    read_words<4>(&ksz[r], st_s + (g + 8 * r) * kScaleBytes + t * C::kKeyVals / 32 * 4);
                    if (g + 8 * r >= keys_here) ksz[r] = 0;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = 2 * t + (r & 1) + 8 * (r >> 1);
                    read_words<4>(&vsz[r], st_s + C::kScalePart + key * kScaleBytes + g * C::kValVals / 32 * 4);
                    if (key >= keys_here) vsz[r] = 0;
                }
            }

            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
            // ---- logits
#pragma unroll
            for (int i = 0; i < C::kKeyLoads; ++i) {
                uint32_t kx[2][KW];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    read_words<C::kKeyBytes>(kx[r], st_k + (r * C::kKeyLoads + i) * 32 * C::kKeyBytes + lane * C::kKeyBytes);
#pragma unroll
                for (int x = 0; x < KW; ++x) {
                    constexpr int kSub = F == KVFIX_POOL_BF16 ? 1 : kE4m3 ? 2 : 4;  // pairs in a word
                    uint32_t p[2][kSub];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t word = kx[r][x];
                        if constexpr (kE4m3) {
                            const uint2 y = e4m3x4_to_f16(word);  // (the row's scale comes with the logit)
                            p[r][0] = y.x;
                            p[r][1] = y.y;
                        } else if constexpr (kInt4) {
                            const unsigned ss = __byte_perm(ksz[r], 0u, 0x1010), zz = __byte_perm(ksz[r], 0u, 0x3232);
                            const uint4 y = int4x8_to_bf16(word, *reinterpret_cast<const __nv_bfloat162*>(&ss),
                                                           *reinterpret_cast<const __nv_bfloat162*>(&zz));
                            p[r][0] = y.x;
                            p[r][1] = y.y;
                            p[r][2] = y.z;
                            p[r][3] = y.w;
                        } else {
                            p[r][0] = word;
                        }
                    }
                    if constexpr (kSub == 1) {
                        if (x & 1) {
                            const int st = (i * KW + x) / 2;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_16816<kE4m3>(s[n], kx[0][x - 1], kx[1][x - 1], p[0][0], p[1][0], qf[n][st][0], qf[n][st][1]);
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < kSub; y += 2) {
                            const int st = ((i * KW + x) * kSub + y) / 2;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_16816<kE4m3>(s[n], p[0][y], p[1][y], p[0][y + 1], p[1][y + 1], qf[n][st][0], qf[n][st][1]);
                        }
                    }
                }
            }
            float ke[2], ve[2];  // e4m3: the key's factor, the value's exponent
            if (kE4m3) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const unsigned kb = st_s[g + 8 * r], vb = st_s[C::kScalePart + g + 8 * r];
                    ke[r] = kb == kE4m3NanByte ? __int_as_float(0x7fffffff) : pow2f((int)e4m3_scale_within(kb) - 127);
                    ve[r] = vb == kE4m3NanByte ? __int_as_float(0x7fffffff) : (float)((int)e4m3_scale_within(vb) - 127);
                }
            }
            // ---- softmax: key g + 8 (x / 2), column 2t + x % 2
            // e4m3: weights come with their value row's power of two, against a maximum of their own,
            // so that the largest summand has f16's full precision whatever the rows' scales are
            bool raise = false;
            float top[NT][2], y[NT][4], top_y[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = x >> 1, key = g + 8 * r;
                    const bool seen = key < keys_here && tile * 16 + key < sees[n][x & 1];
                    float z = s[n][x] * unit[n][x & 1];
                    if (kE4m3) z *= ke[r];
                    s[n][x] = seen ? z : -INFINITY;
                    if (kE4m3) y[n][x] = seen ? z + ve[r] : -INFINITY;
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    top[n][x] = fmaxf(s[n][x], s[n][x + 2]);
                    raise |= top[n][x] > m[n][x] + kAtSlack;
                    if (kE4m3) {
                        top_y[n][x] = fmaxf(y[n][x], y[n][x + 2]);
                        raise |= top_y[n][x] > my[n][x] + kAtSlack;
                    }
                }
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float f = 1.f, hi = top[n][x], hi_y = kE4m3 ? top_y[n][x] : 0.f;
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
                            if (kE4m3) hi_y = fmaxf(hi_y, __shfl_xor_sync(0xffffffffu, hi_y, d));
                        }
                        if (hi > m[n][x]) {
                            f = ex2(m[n][x] - hi);  // (0 from -infinity)
                            m[n][x] = hi;
                            l[n][x] *= f;
                        }
                        if (kE4m3) {
                            f = 1.f;
                            if (hi_y > my[n][x]) {
                                f = ex2(my[n][x] - hi_y);
                                my[n][x] = hi_y;
                            }
                        }
#pragma unroll
                        for (int st = 0; st < kSteps; ++st) {
                            o[st][n][x] *= f;
                            o[st][n][x + 2] *= f;
                        }
                    }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float base = m[n][x & 1] == -INFINITY ? 0.f : m[n][x & 1];
                    p[x] = ex2(s[n][x] - base);
                    l[n][x & 1] += p[x];
                    // (weights up to 2^8 before a maximum is raised: 2^15 here, of f16's 2^16)
                    if (kE4m3) p[x] = ex2(y[n][x] - (my[n][x & 1] == -INFINITY ? 0.f : my[n][x & 1] - 7.f));
                }
                // weights rounded to the operand's type, by half a step: up to 2^-8 of each for bf16, 2^-11
                // for f16.  An f16 below 2^-14, 2^-21 of what the largest is or exceeds, has fewer bits and is
                // off by up to 2^-25: 2^-32 of the largest, where a row's codes are off by 2^-10 of its scale.
                pf[n][0] = transpose_8x8(kE4m3 ? pack_f16(p[0], p[1]) : pack_bf16(p[0], p[1]));
                pf[n][1] = transpose_8x8(kE4m3 ? pack_f16(p[2], p[3]) : pack_bf16(p[2], p[3]));
            }
            // ---- values: blocks st of 16 rows, this lane's values 2 st and 2 st + 1
#pragma unroll
            for (int i = 0; i < C::kValLoads; ++i) {
                uint32_t vx[4][VW];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    read_words<C::kValBytes>(vx[r], st_v + (r * C::kValLoads + i) * 32 * C::kValBytes + lane * C::kValBytes);
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    const uint32_t w0 = vx[0][x], w1 = vx[1][x], w2 = vx[2][x], w3 = vx[3][x];
                    if constexpr (kE4m3) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int st = 2 * (i * VW + x) + y;
                            const uint2 u = e4m3x4_to_f16(__byte_perm(w0, w1, y ? 0x7362 : 0x5140));
                            const uint2 v = e4m3x4_to_f16(__byte_perm(w2, w3, y ? 0x7362 : 0x5140));
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_16816<kE4m3>(o[st][n], u.x, u.y, v.x, v.y, pf[n][0], pf[n][1]);
                        }
                    } else if constexpr (kInt4) {
                        uint4 y[4];
                        const uint32_t ww[4] = {w0, w1, w2, w3};
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const unsigned ss = __byte_perm(vsz[r], 0u, 0x1010), zz = __byte_perm(vsz[r], 0u, 0x3232);
                            y[r] = int4x8_to_bf16(ww[r], *reinterpret_cast<const __nv_bfloat162*>(&ss),
                                                  *reinterpret_cast<const __nv_bfloat162*>(&zz));
                        }
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int st = 4 * (i * VW + x) + z;
                            const uint32_t p0 = z == 0 ? y[0].x : z == 1 ? y[0].y : z == 2 ? y[0].z : y[0].w;
                            const uint32_t p1 = z == 0 ? y[1].x : z == 1 ? y[1].y : z == 2 ? y[1].z : y[1].w;
                            const uint32_t p2 = z == 0 ? y[2].x : z == 1 ? y[2].y : z == 2 ? y[2].z : y[2].w;
                            const uint32_t p3 = z == 0 ? y[3].x : z == 1 ? y[3].y : z == 2 ? y[3].z : y[3].w;
                            const uint32_t a0 = __byte_perm(p0, p1, 0x5410), a1 = __byte_perm(p0, p1, 0x7632);
                            const uint32_t a2 = __byte_perm(p2, p3, 0x5410), a3 = __byte_perm(p2, p3, 0x7632);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_16816<kE4m3>(o[st][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                        }
                    } else {
                        const int st = i * VW + x;
                        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
                        const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_16816<kE4m3>(o[st][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                    }
                }
            }
        }

        // ---- the part: the sums over the lanes of a column, then values as the lanes hold them
        const bool own = e.begin + (long long)head * (e.tiles + at_pad(kFew)) >= walk.lo;
        const long long part = own ? ((prefix ? 0 : a.pool.heads) + (long long)head) * all + (long long)e.agent0 * TG + e.row0
                                   : slot_row;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int col = 8 * n + 2 * t + x;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], d);
                if (col >= e.rows) continue;
                if (g == 0) w.ml[part + col] = make_float2(m[n][x], l[n][x]);
                const float f = !kE4m3 ? 1.f : my[n][x] == -INFINITY ? 1.f : ex2(my[n][x] - 7.f - m[n][x]);
                float* dst = w.o + (part + col) * D + g * C::kValVals;
#pragma unroll
                for (int i = 0; i < C::kValLoads; ++i)
#pragma unroll
                    for (int v = 0; v < C::kValVals; v += 4) {
                        const int st = (i * C::kValVals + v) / 2;
                        *reinterpret_cast<float4*>(dst + i * 8 * C::kValVals + v) =
                            make_float4(o[st][n][x] * f, o[st][n][x + 2] * f, o[st + 1][n][x] * f, o[st + 1][n][x + 2] * f);
                    }
            }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&g_status_attend, FLAG_BOUNDS);
    // (what follows waits for this kernel alone: it ends after the one before it)
    if (w.many) pdl_wait();
}

}  // namespace kvfix
