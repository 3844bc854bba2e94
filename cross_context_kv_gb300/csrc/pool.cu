// pool.cu -- kvfix_pool_write and kvfix_pool_read: rows of a KV cache into a paged pool in
// one of its stored forms (bf16, e4m3, int4; pool.cuh) and back, keys re-aligned on the way.
//
// Both are one pass over the rows, bound by HBM: a (token, head) of both planes moves
// 4 D bytes on the bf16 side and 2 pool_head_bytes (+ scales) on the pool's.  A lane owns the
// two 8-wide vectors that rotate-half RoPE mixes, [8j, 8j+8) and [D/2 + 8j, D/2 + 8j + 8), so
// a rotation needs no exchange; D/16 lanes share a (token, head), and the row's largest
// magnitude (e4m3) or a group's smallest and largest value (int4) take two or three shuffles
// among them.  A CTA keeps one (chunk, layer) and a run of tokens: the rotation's
// (cos, sin) of a lane's eight pairs stay in registers for all of them.
//
// Measured: 4096 tokens x 32 layers x 8 heads of 128 written rotated as e4m3 in 146 us, 5.5 TB/s
// (a copy's bytes take 119); 512 tokens x 8 chunks x 48 layers read back rotated in 203 us,
// 6.0 TB/s.  int4 is bound by issue: 3 x 1237 tokens x 9 layers x 5 heads of 64 in 18.7 us,
// 2.7 TB/s, 68 % of the issue slots.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pool.cuh"

namespace kvfix {

static __device__ unsigned int g_status_pool;

unsigned read_status_pool(cudaStream_t stream) {
    unsigned h = 0, zero = 0;
    cudaMemcpyFromSymbolAsync(&h, g_status_pool, sizeof h, 0, cudaMemcpyDeviceToHost, stream);
    cudaMemcpyToSymbolAsync(g_status_pool, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    cudaStreamSynchronize(stream);
    return h;
}

constexpr int kPoolThreads = 256;
// (token, head) rows in flight per lane, both planes each.  Writing int4 takes one: its
// arithmetic (20 instructions a value) wants warps more than loads in flight.
constexpr int pool_unroll(int format, bool write) { return format == KVFIX_POOL_INT4 && write ? 1 : 2; }

struct PoolArgs {
    const uint16_t* in[2];  // write: the source planes
    uint16_t* out[2];       // read: the destination planes
    Plane p;                // their layout
    PoolView pool;
    const int32_t* delta;   // per chunk, or null
    const int32_t* slots;   // [chunks][tokens]
    int blocks;             // token runs per (chunk, layer)
    int run;                // tokens per run
};

// Largest |value| bits of 16 bf16 (as two vectors), infinities and NaN included.
__device__ __forceinline__ unsigned abs_max16(const uint4& a, const uint4& b) {
    const unsigned m = 0x7fff7fffu;
    unsigned x = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
    unsigned y = __vmaxu2(__vmaxu2(b.x & m, b.y & m), __vmaxu2(b.z & m, b.w & m));
    x = __vmaxu2(x, y);
    return max(x & 0xffffu, x >> 16);
}

__device__ __forceinline__ unsigned finite_abs_max8(const uint4& v) {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
    unsigned r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        r = max(r, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
    return r;
}

// The e4m3 scale exponent of a row whose largest finite magnitude has bf16 bits `a`: the
// least k with magnitude <= 448 2^k = 1.75 2^(k+8), within the format's limits.
__device__ __forceinline__ int e4m3_exponent(unsigned a) {
    const int k = (int)(a >> 7) - 127 - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0);
    return min(max(k, kE4m3MinExp), kE4m3MaxExp);
}

constexpr unsigned kNanRow = 0xffffu;

__device__ __forceinline__ uint2 to_e4m3(const uint4& v, float inv) {
    float f[8];
    unpack8(v, f);
    unsigned r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * inv, f[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Eight codes (as 2^23 + code in float, whose low byte is the code) to their word: value 2i in
// nibble i, value 2i+1 in nibble i + 4.
__device__ __forceinline__ unsigned int4_word(const float* t) {
    unsigned w = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i)
        w = w * 16u + __byte_perm(__float_as_uint(t[2 * i]), __float_as_uint(t[2 * i + 1]), 0x5410);
    return w;
}

// Eight values against their group's zero and 1/scale -> one word of codes.  Adding 2^23
// rounds to the nearest integer, ties to even.  Values below 2^127 lie within their group's
// range, and the rounded scale takes its end to at most 15 (1 + 2^-8), so they need no bounds;
// infinities and clipped ranges do, and the maximum with 0 takes a NaN to code 0.
template <bool kTame>
__device__ __forceinline__ unsigned to_int4(const uint4& v, float zero, float inv) {
    float f[8];
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float t = __fmul_rn(__fsub_rn(f[i], zero), inv);
        if (!kTame) t = fminf(fmaxf(t, 0.f), 15.f);
        f[i] = __fadd_rn(t, 8388608.f);
    }
    return int4_word(f);
}

struct Int4Group {
    float zero, inv;
    unsigned word;  // bf16 scale, bf16 zero
};

// Scale and zero of the group of 32 values whose 4 lanes each hold 8 of them.
// Smallest and largest values go through the lanes as one pair of bf16, (min, -max).
template <bool kTame>
__device__ __forceinline__ Int4Group int4_group(const uint4& v) {
    __nv_bfloat162 ends;
    if (kTame) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
        const __nv_bfloat162 lo = __hmin2(__hmin2(h[0], h[1]), __hmin2(h[2], h[3]));
        const __nv_bfloat162 hi = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        ends = __halves2bfloat162(__hmin(__low2bfloat16(lo), __high2bfloat16(lo)),
                                  __hneg(__hmax(__low2bfloat16(hi), __high2bfloat16(hi))));
    } else {
        float f[8], lo = INFINITY, hi = -INFINITY;
        unpack8(v, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool fine = fabsf(f[i]) < INFINITY;  // false for NaN too
            lo = fine ? fminf(lo, f[i]) : lo;
            hi = fine ? fmaxf(hi, f[i]) : hi;
        }
        ends = __floats2bfloat162_rn(lo, -hi);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const unsigned other = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const unsigned*>(&ends), o);
        ends = __hmin2(ends, *reinterpret_cast<const __nv_bfloat162*>(&other));
    }
    float lo = __low2float(ends), hi = -__high2float(ends);
    if (!kTame && lo > hi) lo = hi = 0.f;  // no finite value
    const float range = fminf(__fsub_rn(hi, lo), 3.402823466e38f);
    float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(range, 15.f)));
    if (s < pow2f(-120)) s = 0.f;
    Int4Group g;
    // (-0 and +0 compare equal: which of them a group that has both keeps as its zero decides
    // no value)
    g.zero = lo;
    g.inv = s > 0.f ? __frcp_rn(s) : 0.f;
    const __nv_bfloat162 w = __floats2bfloat162_rn(s, lo);
    g.word = *reinterpret_cast<const unsigned*>(&w);
    return g;
}

// Both halves of a lane's row: codes and their groups' words.
template <bool kTame>
__device__ __forceinline__ void int4_rows(const uint4& x, const uint4& y, unsigned& cx, unsigned& cy, unsigned& wx,
                                          unsigned& wy) {
    const Int4Group gx = int4_group<kTame>(x), gy = int4_group<kTame>(y);
    cx = to_int4<kTame>(x, gx.zero, gx.inv);
    cy = to_int4<kTame>(y, gy.zero, gy.inv);
    wx = gx.word;
    wy = gy.word;
}

struct PairAngles {
    float c[8], s[8];
};

__device__ __forceinline__ void turn(uint4& lo, uint4& hi, const PairAngles& a) {
    float x[8], y[8];
    unpack8(lo, x);
    unpack8(hi, y);
    rotate_pair(x, y, a.c, a.s);
    lo = pack8(x);
    hi = pack8(y);
}

// The lane's eight (cos, sin), from a per-CTA table.
template <int D>
__device__ __forceinline__ void lane_angles(PairAngles& a, int d, const RopeTheta& th, int j) {
    __shared__ float2 tab[D / 2];
    for (int i = threadIdx.x; i < D / 2; i += kPoolThreads) {
        float c, s;
        rope_cos_sin(d, th.theta[i], &c, &s);
        tab[i] = make_float2(c, s);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 t = tab[8 * j + i];
        a.c[i] = t.x;
        a.s[i] = t.y;
    }
}

// The run of tokens and (chunk, layer) of this CTA.
struct Run {
    int c, l, t0, t1;
};
__device__ __forceinline__ Run run_of(const PoolArgs& a) {
    Run r;
    const int b = (int)(blockIdx.x % (unsigned)a.blocks);
    const unsigned cl = blockIdx.x / (unsigned)a.blocks;
    r.l = (int)(cl % (unsigned)a.p.layers);
    r.c = (int)(cl / (unsigned)a.p.layers);
    r.t0 = b * a.run;
    r.t1 = min(a.p.tokens, r.t0 + a.run);
    return r;
}

template <int F, int D>
__global__ void __launch_bounds__(kPoolThreads, F == KVFIX_POOL_INT4 ? 4 : 3)
pool_write_kernel(const __grid_constant__ PoolArgs a, const __grid_constant__ RopeTheta th) {
    constexpr int kLanes = D / 16;                 // lanes per (token, head)
    constexpr int kRows = kPoolThreads / kLanes;   // (token, head) rows per step of the CTA
    constexpr int HB = pool_head_bytes(F, D), kU = pool_unroll(F, true);
    const Run r = run_of(a);
    const int j = threadIdx.x % kLanes;
    const int d = a.delta ? __ldg(a.delta + r.c) : 0;
    PairAngles ang;
    if (d != 0) lane_angles<D>(ang, d, th, j);
    const int H = a.p.heads;
    const long long base = a.p.row(r.c, r.l, r.t0);
    const int32_t* slots = a.slots + (long long)r.c * a.p.tokens + r.t0;
    const int items = (r.t1 - r.t0) * H;
    bool bad = false;
    // every lane of a warp runs the same number of steps (the reductions are warp-wide)
    for (int i0 = 0; i0 < items; i0 += kU * kRows) {
        uint4 lo[kU][2], hi[kU][2];
        int slot[kU], head[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * kRows + (int)threadIdx.x / kLanes;
            slot[u] = -1;
            head[u] = 0;
#pragma unroll
            for (int p = 0; p < 2; ++p) lo[u][p] = hi[u][p] = make_uint4(0u, 0u, 0u, 0u);
            if (i < items) {
                const int t = i / H;
                head[u] = i - t * H;
                slot[u] = __ldg(slots + t);
                const long long off = base + (long long)t * a.p.st + head[u] * D + 8 * j;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    lo[u][p] = ld_stream(reinterpret_cast<const uint4*>(a.in[p] + off));
                    hi[u][p] = ld_stream(reinterpret_cast<const uint4*>(a.in[p] + off + D / 2));
                }
                if (slot[u] >= a.pool.slots) {
                    bad = true;
                    slot[u] = -1;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (d != 0) turn(lo[u][0], hi[u][0], ang);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint4 x = lo[u][p], y = hi[u][p];
                const long long at = (long long)r.l * a.pool.sl + (long long)slot[u] * a.pool.ss + (long long)head[u] * HB;
                const long long row = ((long long)r.l * H + head[u]) * a.pool.slots + slot[u];
                unsigned char* codes = a.pool.plane[p].codes;
                if (F == KVFIX_POOL_BF16) {
                    if (slot[u] >= 0) {
                        *reinterpret_cast<uint4*>(codes + at + 16 * j) = x;
                        *reinterpret_cast<uint4*>(codes + at + D + 16 * j) = y;
                    }
                } else if (F == KVFIX_POOL_E4M3) {
                    // the largest finite magnitude; above them all, a mark that the row has a NaN
                    unsigned m = abs_max16(x, y);
                    if (m > 0x7f80u) m = kNanRow;
                    else if (m == 0x7f80u) m = max(finite_abs_max8(x), finite_abs_max8(y));
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const int k = m == kNanRow ? (int)kE4m3NanByte - 127 : e4m3_exponent(m);
                    const float inv = pow2f(-min(k, kE4m3MaxExp));
                    uint2 cx = to_e4m3(x, inv), cy = to_e4m3(y, inv);
                    if (m == kNanRow) cx = cy = make_uint2(0u, 0u);
                    if (slot[u] >= 0) {
                        *reinterpret_cast<uint2*>(codes + at + 8 * j) = cx;
                        *reinterpret_cast<uint2*>(codes + at + D / 2 + 8 * j) = cy;
                        if (j == 0) a.pool.plane[p].scales[row] = (unsigned char)(k + 127);
                    }
                } else {
                    unsigned cx, cy, wx, wy;
                    // (2^127 and above: infinities, NaN, and ranges past the largest float)
                    if (__any_sync(0xffffffffu, abs_max16(x, y) >= 0x7f00u)) int4_rows<false>(x, y, cx, cy, wx, wy);
                    else int4_rows<true>(x, y, cx, cy, wx, wy);
                    if (slot[u] >= 0) {
                        *reinterpret_cast<unsigned*>(codes + at + 4 * j) = cx;
                        *reinterpret_cast<unsigned*>(codes + at + D / 4 + 4 * j) = cy;
                        if (j % 4 == 0) {
                            unsigned* sc = reinterpret_cast<unsigned*>(a.pool.plane[p].scales) + row * (D / kQGroup);
                            sc[j / 4] = wx;
                            sc[j / 4 + D / (2 * kQGroup)] = wy;
                        }
                    }
                }
            }
        }
    }
    if (bad && j == 0) atomicOr(&g_status_pool, FLAG_BOUNDS);
}

template <int F, int D>
__global__ void __launch_bounds__(kPoolThreads)
pool_read_kernel(const __grid_constant__ PoolArgs a, const __grid_constant__ RopeTheta th) {
    constexpr int kLanes = D / 16;
    constexpr int kRows = kPoolThreads / kLanes;
    constexpr int HB = pool_head_bytes(F, D), kU = pool_unroll(F, false);
    const Run r = run_of(a);
    const int j = threadIdx.x % kLanes;
    const int d = a.delta ? __ldg(a.delta + r.c) : 0;
    PairAngles ang;
    if (d != 0) lane_angles<D>(ang, d, th, j);
    const int H = a.p.heads;
    const long long base = a.p.row(r.c, r.l, r.t0);
    const int32_t* slots = a.slots + (long long)r.c * a.p.tokens + r.t0;
    const int items = (r.t1 - r.t0) * H;
    bool bad = false;
    for (int i0 = threadIdx.x / kLanes; i0 < items; i0 += kU * kRows) {
        uint4 x[kU][2], y[kU][2];  // codes (in part), then values
        unsigned sx[kU][2], sy[kU][2];
        long long off[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * kRows;
            off[u] = -1;
            if (i >= items) continue;
            const int t = i / H, head = i - t * H;
            const int slot = __ldg(slots + t);
            if (slot >= a.pool.slots) bad = true;
            if (slot < 0 || slot >= a.pool.slots) continue;
            off[u] = base + (long long)t * a.p.st + head * D + 8 * j;
            const long long at = (long long)r.l * a.pool.sl + (long long)slot * a.pool.ss + (long long)head * HB;
            const long long row = ((long long)r.l * H + head) * a.pool.slots + slot;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const unsigned char* codes = a.pool.plane[p].codes + at;
                if (F == KVFIX_POOL_BF16) {
                    x[u][p] = ld_stream(reinterpret_cast<const uint4*>(codes + 16 * j));
                    y[u][p] = ld_stream(reinterpret_cast<const uint4*>(codes + D + 16 * j));
                } else if (F == KVFIX_POOL_E4M3) {
                    const uint2 cx = __ldg(reinterpret_cast<const uint2*>(codes + 8 * j));
                    const uint2 cy = __ldg(reinterpret_cast<const uint2*>(codes + D / 2 + 8 * j));
                    x[u][p].x = cx.x;
                    x[u][p].y = cx.y;
                    y[u][p].x = cy.x;
                    y[u][p].y = cy.y;
                    sx[u][p] = __ldg(a.pool.plane[p].scales + row);
                } else {
                    x[u][p].x = __ldg(reinterpret_cast<const unsigned*>(codes + 4 * j));
                    y[u][p].x = __ldg(reinterpret_cast<const unsigned*>(codes + D / 4 + 4 * j));
                    const unsigned* sc = reinterpret_cast<const unsigned*>(a.pool.plane[p].scales) + row * (D / kQGroup);
                    sx[u][p] = __ldg(sc + j / 4);
                    sy[u][p] = __ldg(sc + j / 4 + D / (2 * kQGroup));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (off[u] < 0) continue;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint4 vx = x[u][p], vy = y[u][p];
                if (F == KVFIX_POOL_E4M3) {
                    const E4m3Scale s = e4m3_scale_byte(sx[u][p]);
                    e4m3x16_to_bf16(make_uint4(vx.x, vx.y, vy.x, vy.y), s, vx, vy);
                } else if (F == KVFIX_POOL_INT4) {
                    const unsigned a0 = __byte_perm(sx[u][p], 0u, 0x1010), z0 = __byte_perm(sx[u][p], 0u, 0x3232);
                    const unsigned a1 = __byte_perm(sy[u][p], 0u, 0x1010), z1 = __byte_perm(sy[u][p], 0u, 0x3232);
                    vx = int4x8_to_bf16(vx.x, *reinterpret_cast<const __nv_bfloat162*>(&a0),
                                        *reinterpret_cast<const __nv_bfloat162*>(&z0));
                    vy = int4x8_to_bf16(vy.x, *reinterpret_cast<const __nv_bfloat162*>(&a1),
                                        *reinterpret_cast<const __nv_bfloat162*>(&z1));
                }
                if (p == 0 && d != 0) turn(vx, vy, ang);
                st_stream(reinterpret_cast<uint4*>(a.out[p] + off[u]), vx);
                st_stream(reinterpret_cast<uint4*>(a.out[p] + off[u] + D / 2), vy);
            }
        }
    }
    if (bad && j == 0) atomicOr(&g_status_pool, FLAG_BOUNDS);
}

// Token runs: about eight CTAs per SM over all (chunk, layer), each run long enough that the
// rotation table (one double-precision angle per pair) is a small part of its work.
constexpr int kPoolCtas = 152 * 8;

static void plan_runs(PoolArgs& a, bool write) {
    const long long cl = (long long)a.p.chunks * a.p.layers;
    const int rows = kPoolThreads / (a.p.dim / 16);
    const long long per = (cl * a.p.tokens + kPoolCtas - 1) / kPoolCtas;  // tokens per CTA
    // whole steps of the CTA: a step more for a few rows would cost as much as a full one
    const int step = pool_unroll(a.pool.format, write) * rows;
    const long long steps = (per * a.p.heads + step / 2) / step;
    long long run = (steps > 1 ? steps : 1) * step / a.p.heads;
    if (run < 1) run = 1;
    if (run > a.p.tokens) run = a.p.tokens;
    while ((a.p.tokens + run - 1) / run * cl > 0x7fffffffll) run *= 2;  // grid.x limit
    a.run = (int)run;
    a.blocks = (int)((a.p.tokens + run - 1) / run);
}

template <int F, int D>
static cudaError_t launch_pool_form(const PoolArgs& a, const RopeTheta& th, bool write, cudaStream_t s) {
    const unsigned grid = (unsigned)((long long)a.blocks * a.p.chunks * a.p.layers);
    if (write)
        pool_write_kernel<F, D><<<grid, kPoolThreads, 0, s>>>(a, th);
    else
        pool_read_kernel<F, D><<<grid, kPoolThreads, 0, s>>>(a, th);
    return cudaGetLastError();
}

static cudaError_t launch_pool(PoolArgs& a, const RopeTheta& th, bool write, cudaStream_t s) {
    if (a.p.chunks == 0 || a.p.layers == 0 || a.p.tokens == 0) return cudaSuccess;
    plan_runs(a, write);
    switch (a.pool.format * 2 + (a.p.dim == 128)) {
        case KVFIX_POOL_BF16 * 2: return launch_pool_form<KVFIX_POOL_BF16, 64>(a, th, write, s);
        case KVFIX_POOL_BF16 * 2 + 1: return launch_pool_form<KVFIX_POOL_BF16, 128>(a, th, write, s);
        case KVFIX_POOL_E4M3 * 2: return launch_pool_form<KVFIX_POOL_E4M3, 64>(a, th, write, s);
        case KVFIX_POOL_E4M3 * 2 + 1: return launch_pool_form<KVFIX_POOL_E4M3, 128>(a, th, write, s);
        case KVFIX_POOL_INT4 * 2: return launch_pool_form<KVFIX_POOL_INT4, 64>(a, th, write, s);
        default: return launch_pool_form<KVFIX_POOL_INT4, 128>(a, th, write, s);
    }
}

cudaError_t launch_pool_write(const uint16_t* k, const uint16_t* v, const kvfix_kv_desc& d, const int32_t* delta,
                              const RopeTheta& th, const int32_t* slots, const kvfix_pool& pool, cudaStream_t s) {
    PoolArgs a = {};
    a.in[0] = k;
    a.in[1] = v;
    a.p = plane_of(d);
    a.pool = view_of(pool);
    a.delta = delta;
    a.slots = slots;
    return launch_pool(a, th, true, s);
}

cudaError_t launch_pool_read(const kvfix_pool& pool, const int32_t* slots, const int32_t* delta, const RopeTheta& th,
                             uint16_t* k, uint16_t* v, const kvfix_kv_desc& d, cudaStream_t s) {
    PoolArgs a = {};
    a.out[0] = k;
    a.out[1] = v;
    a.p = plane_of(d);
    a.pool = view_of(pool);
    a.delta = delta;
    a.slots = slots;
    return launch_pool(a, th, false, s);
}

}  // namespace kvfix
