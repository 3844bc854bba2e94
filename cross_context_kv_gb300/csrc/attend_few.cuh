// attend_few.cuh -- kvfix_shared_attend for blocks of up to 16 query rows: an agent's own tokens
// while it decodes, and a short round's prefix.
//
// Mathematics.  The products are turned around: logits are S^T = K Q^T (keys along the rows of the
// matrix instruction, queries along its 8 columns) and the output O^T = V^T P^T, so few queries
// leave nothing of an instruction empty that costs more than the keys' own loading.
//
// Layout.  A warp takes 16 keys at a time, alone: no shared memory, no barrier.  The order of a
// contraction's terms is free, so lane (g = lane / 4, t = lane % 4) loads 16 contiguous bytes of
// key rows g and g + 8 and takes them as its own terms of consecutive instructions, and of value
// rows 2t, 2t+1, 2t+8, 2t+9 the same D/8 values, which are its rows of consecutive instructions:
// every load is as wide as the rows allow, and stored codes become operands in the registers that
// feed the tensor cores: int4 as bf16, e4m3 as f16, which holds every code.  A logit's key belongs
// to one lane, so an e4m3 row's scales are one multiplication of the logit and one exponent added
// in the weight; maxima are lanes' own until a row's has to be raised.  Weights go from the logits' layout to the operand's by movmatrix.
//
// What bounds it: HBM (the next 16 keys' rows are on their way while these are worked on:
// 4 to 8 KB per warp, 8 or 12 warps per SM), then the conversions of the stored forms.
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
    // Rows on their way take 64 registers a lane of bf16, at most 32 of the stored forms, and 16
    // queries' output and operands twice those of 8: 8 warps where 12 do not fit the registers.
    static constexpr int warps(int nt) { return F == KVFIX_POOL_BF16 || (nt == 2 && D == 128) ? 8 : kFewWarps; }
};

// N (4, 8, 16) bytes as 32-bit words; nothing is read, and zeros come, where `there` is false.
template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const unsigned char* p, bool there) {
    if constexpr (N == 16) {
        const uint4 v = there ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 8) {
        const uint2 v = there ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = there ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
    }
}

// NT: groups of 8 queries.
template <int F, int D, int NT>
__global__ void __launch_bounds__(32 * FewCfg<F, D>::warps(NT), 1)
    attend_few_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ AtWork w) {
    using C = FewCfg<F, D>;
    constexpr bool kE4m3 = F == KVFIX_POOL_E4M3, kInt4 = F == KVFIX_POOL_INT4;
    constexpr int KW = C::kKeyBytes / 4, VW = C::kValBytes / 4;
    constexpr int kScaleBytes = kInt4 ? D / 8 : 1;  // of a row
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
    const long long slot_row = w.few_rows + ((long long)blockIdx.x * C::warps(NT) + warp) * w.few;
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

        struct Keys {
            uint32_t x[2][C::kKeyLoads][KW];
            uint32_t s[2];
        } kr;
        struct Values {
            uint32_t x[4][C::kValLoads][VW];
            uint32_t s[kInt4 ? 4 : 2];
        } vr;
        int keys_k = 0, keys_v = 0;  // keys there are in the tiles that kr and vr hold
        // this lane's places in a tile's first rows
        const unsigned char* const k0 = a.pool.plane[0].codes + (long long)head * C::kRow + g * a.pool.ss + t * C::kKeyBytes;
        const unsigned char* const v0 = a.pool.plane[1].codes + (long long)head * C::kRow + 2 * t * a.pool.ss + g * C::kValBytes;
        const unsigned char* const ks0 = a.pool.plane[0].scales + ((long long)head * a.pool.slots + g) * kScaleBytes;
        const unsigned char* const vs0 =
            a.pool.plane[1].scales + ((long long)head * a.pool.slots + (kInt4 ? 2 * t : g)) * kScaleBytes;
        auto slot_of = [&](int tile, int page) { return (long long)page * a.page + ((tile * 16) & (a.page - 1)); };
        auto load_keys = [&](int tile, int page) {
            keys_k = page >= 0 && page < pool_pages ? min(16, e.keys - tile * 16) : 0;
            const long long slot = slot_of(tile, page);
            const unsigned char* const p = k0 + slot * a.pool.ss;
            const unsigned char* const ps = ks0 + slot * kScaleBytes;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool there = g + 8 * r < keys_k;
#pragma unroll
                for (int i = 0; i < C::kKeyLoads; ++i)
                    load_words<C::kKeyBytes>(kr.x[r][i], p + 8 * r * a.pool.ss + i * 4 * C::kKeyBytes, there);
                if (kE4m3) kr.s[r] = there ? __ldg(ps + 8 * r) : 127u;
                if (kInt4) load_words<4>(&kr.s[r], ps + 8 * r * kScaleBytes + t * C::kKeyVals / 32 * 4, there);
            }
        };
        auto load_values = [&](int tile, int page) {
            keys_v = page >= 0 && page < pool_pages ? min(16, e.keys - tile * 16) : 0;
            const long long slot = slot_of(tile, page);
            const unsigned char* const p = v0 + slot * a.pool.ss;
            const unsigned char* const ps = vs0 + slot * kScaleBytes;
            if (kE4m3) {
#pragma unroll
                for (int r = 0; r < 2; ++r) vr.s[r] = g + 8 * r < keys_v ? __ldg(ps + 8 * r) : 127u;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = (r & 1) + 8 * (r >> 1);
                const bool there = 2 * t + row < keys_v;
#pragma unroll
                for (int i = 0; i < C::kValLoads; ++i)
                    load_words<C::kValBytes>(vr.x[r][i], p + row * a.pool.ss + i * 8 * C::kValBytes, there);
                if (kInt4) load_words<4>(&vr.s[r], ps + row * kScaleBytes + g * C::kValVals / 32 * 4, there);
            }
        };
        int page = __shfl_sync(0xffffffffu, page_now, 0);
        bad |= page < 0 || page >= pool_pages;
        load_keys(t0, page);
        load_values(t0, page);

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
                const int col = 8 * n + 2 * t + x, rc = e.row0 + col;
                // a prefix is seen whole; new token i sees the keys up to its own
                const int unseen = prefix ? 0 : (e.row0 + e.rows - 1) / G - rc / G;
                sees[n][x] = col < e.rows ? e.keys - unseen : 0;
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
            // the next tile's page
            const int next = tile + 1 - t0;
            if ((next & 31) == 0) {
                page_now = page_next;
                page_next = fetch_pages(tile + 1 + 32);
            }
            page = __shfl_sync(0xffffffffu, page_now, next & 31);
            const bool more = tile + 1 < t1;
            if (more) bad |= page < 0 || page >= pool_pages;

            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
            // ---- logits
#pragma unroll
            for (int i = 0; i < C::kKeyLoads; ++i)
#pragma unroll
                for (int x = 0; x < KW; ++x) {
                    constexpr int kSub = F == KVFIX_POOL_BF16 ? 1 : kE4m3 ? 2 : 4;  // pairs in a word
                    uint32_t p[2][kSub];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t word = kr.x[r][i][x];
                        if constexpr (kE4m3) {
                            const uint2 y = e4m3x4_to_f16(word);  // (the row's scale comes with the logit)
                            p[r][0] = y.x;
                            p[r][1] = y.y;
                        } else if constexpr (kInt4) {
                            const unsigned ss = __byte_perm(kr.s[r], 0u, 0x1010), zz = __byte_perm(kr.s[r], 0u, 0x3232);
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
                                mma_16816<kE4m3>(s[n], kr.x[0][i][x - 1], kr.x[1][i][x - 1], p[0][0], p[1][0], qf[n][st][0], qf[n][st][1]);
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
            const int keys_here = keys_k;
            float ke[2], ve[2];  // e4m3: the key's factor, the value's exponent
            if (kE4m3) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    ke[r] = kr.s[r] == kE4m3NanByte ? __int_as_float(0x7fffffff) : pow2f((int)kr.s[r] - 127);
                    ve[r] = vr.s[r] == kE4m3NanByte ? __int_as_float(0x7fffffff) : (float)((int)vr.s[r] - 127);
                }
            }
            if (more) load_keys(tile + 1, page);
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
                // weights rounded to the operand's type: half a step, 2^-9 of each for bf16, 2^-12 for f16
                pf[n][0] = transpose_8x8(kE4m3 ? pack_f16(p[0], p[1]) : pack_bf16(p[0], p[1]));
                pf[n][1] = transpose_8x8(kE4m3 ? pack_f16(p[2], p[3]) : pack_bf16(p[2], p[3]));
            }
            // ---- values: blocks st of 16 rows, this lane's values 2 st and 2 st + 1
#pragma unroll
            for (int i = 0; i < C::kValLoads; ++i)
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    uint32_t w0 = vr.x[0][i][x], w1 = vr.x[1][i][x], w2 = vr.x[2][i][x], w3 = vr.x[3][i][x];
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
                            const unsigned ss = __byte_perm(vr.s[r], 0u, 0x1010), zz = __byte_perm(vr.s[r], 0u, 0x3232);
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
            if (more) load_values(tile + 1, page);
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
