// rotary.cu -- kvfix_rotary: rotary positions of queries and keys, one position per token.
//
// Mathematics.  A pair (a, b) of a head turns by the angle p theta_i: (a c - b s, b c + a s) with
// c, s = m cos, m sin.  Positions reach 2^31 and theta_i is a double, so the angle is kept in
// turns as a 64-bit fraction: p (theta_i / 2 pi) 2^64 modulo 2^64 is one integer product, exact
// but for the rounding of theta_i / 2 pi itself (2^-52 of it), where a product of doubles would
// lose what lies beyond 53 bits and this part has few double units.  One conversion to float
// and sincospi follow: both are off by 2^-23 or less of their value.
//
// Layout.  A thread owns a column of its token's heads: two 8-wide vectors, the ones that turn into each
// other (half layout) or neighbours (interleaved), so it computes eight (cos, sin) once and uses
// them for every head of queries and keys, and for the layers of its block; four heads' loads
// are in flight together.  Where little work is left for each, the heads of a token are spread over
// threads, then every thread has its own head.  Values beyond rotary_dim are columns that are
// copied, or left out when the call works in place.  In the half layout a rotary_dim that is no
// multiple of 16 has halves that vectors do not meet: its columns are runs of 4, 2 or 1 values of
// either half, and vectors of what does not turn.
//
// Bound by HBM: see the measured figures at launch_rotary.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "rotary.h"
#include "rotary_split.h"

namespace kvfix {

constexpr int kRotaryHeads = 4;  // heads whose loads are in flight together

// What a thread has of a head.  Vectors: two 8-wide ones.
struct RotaryVectors {
    static constexpr int kPairs = 8;
    uint4 lo, hi;
    __device__ __forceinline__ void load(const uint16_t* p, int a, int b, bool) {
        lo = *reinterpret_cast<const uint4*>(p + a);
        hi = *reinterpret_cast<const uint4*>(p + b);
    }
    __device__ __forceinline__ void store(uint16_t* p, int a, int b, bool) const {
        *reinterpret_cast<uint4*>(p + a) = lo;
        *reinterpret_cast<uint4*>(p + b) = hi;
    }
    // `pairs`: the first of them turn (half layout: all)
    template <int LAYOUT>
    __device__ __forceinline__ void turn(const float* c, const float* s, int pairs) {
        if (LAYOUT == KVFIX_ROPE_HALF) {
            float x[8], y[8];
            unpack8(lo, x);
            unpack8(hi, y);
            rotate_pair(x, y, c, s);
            lo = pack8(x);
            hi = pack8(y);
        } else {
            unsigned w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};  // a pair each
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float x = __uint_as_float(w[k] << 16), y = __uint_as_float(w[k] & 0xffff0000u);
                const __nv_bfloat162 r = __floats2bfloat162_rn(__fmaf_rn(x, c[k], __fmul_rn(y, -s[k])),
                                                               __fmaf_rn(y, c[k], __fmul_rn(x, s[k])));
                if (k < pairs) w[k] = *reinterpret_cast<const unsigned*>(&r);
            }
            lo = make_uint4(w[0], w[1], w[2], w[3]);
            hi = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
};
// Half layout with halves that no vector border meets: P pairs whose parts are two runs of P 16-bit
// values (4, 2 or 1 of them, as the halves' length is a multiple of that), or a vector of those that do
// not turn.
template <int P>
struct RotaryMixed {
    static constexpr int kPairs = P;
    uint4 x;  // the runs in x, y and z, w
    static __device__ __forceinline__ void get(const uint16_t* p, unsigned& a, unsigned& b) {
        if (P == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            a = v.x;
            b = v.y;
        } else {
            a = P == 2 ? *reinterpret_cast<const unsigned*>(p) : (unsigned)*p;
        }
    }
    static __device__ __forceinline__ void put(uint16_t* p, unsigned a, unsigned b) {
        if (P == 4) *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
        else if (P == 2) *reinterpret_cast<unsigned*>(p) = a;
        else *p = (uint16_t)a;
    }
    __device__ __forceinline__ void load(const uint16_t* p, int a, int b, bool wide) {
        if (wide) {
            x = *reinterpret_cast<const uint4*>(p + a);
        } else {
            get(p + a, x.x, x.y);
            get(p + b, x.z, x.w);
        }
    }
    __device__ __forceinline__ void store(uint16_t* p, int a, int b, bool wide) const {
        if (wide) {
            *reinterpret_cast<uint4*>(p + a) = x;
        } else {
            put(p + a, x.x, x.y);
            put(p + b, x.z, x.w);
        }
    }
    template <int LAYOUT>
    __device__ __forceinline__ void turn(const float* c, const float* s, int) {
        const unsigned lo[2] = {x.x, x.y}, hi[2] = {x.z, x.w};
        unsigned u[2] = {0, 0}, v[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const int w = k >> 1, at = 16 * (k & 1);
            const float a = __uint_as_float(lo[w] >> at << 16), b = __uint_as_float(hi[w] >> at << 16);
            u[w] |= (unsigned)__bfloat16_as_ushort(__float2bfloat16_rn(__fmaf_rn(a, c[k], __fmul_rn(b, -s[k])))) << at;
            v[w] |= (unsigned)__bfloat16_as_ushort(__float2bfloat16_rn(__fmaf_rn(b, c[k], __fmul_rn(a, s[k])))) << at;
        }
        x = make_uint4(u[0], u[1], v[0], v[1]);
    }
};

template <int LAYOUT, typename V>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryArgs a,
                                                                const __grid_constant__ RotarySplit w) {
    constexpr int N = V::kPairs;
    constexpr bool kMixed = N < 8;
    RotaryPlace at;
    if (!rotary_place(w, a.tokens, blockIdx.x, threadIdx.x, at)) return;
    const int t = (int)at.token, chunk = at.chunk, col = at.column, run = at.run;
    const int turning = (a.rotary_dim + 2 * N - 1) / (2 * N);  // columns that turn
    const int pairs = a.rotary_dim / 2 - col * N;              // (of this one)
    // places of the column's two parts in a head
    int pa, pb;
    bool wide = false;
    if (LAYOUT == KVFIX_ROPE_HALF && col < turning) {
        pa = col * N;
        pb = pa + a.rotary_dim / 2;
    } else if (!kMixed) {
        pa = col * 2 * N;
        pb = pa + N;
    } else {
        // behind those that turn: runs up to a border of vectors, then vectors
        const int behind = col - turning, border = (a.rotary_dim + 7) / 8 * 8, odd = (border - a.rotary_dim) / (2 * N);
        wide = behind >= odd;
        pa = wide ? border + 8 * (behind - odd) : a.rotary_dim + 2 * N * behind;
        pb = pa + N;
    }
    const int p = __ldg(a.positions + (long long)chunk * a.tokens + t);
    const int heads0 = a.ip[0].heads, heads = heads0 + a.ip[1].heads;
    const int l0 = at.layer0, l1 = l0 + rotary_layers(w, a.layers, l0);
    V v[kRotaryHeads];
    auto load = [&](int l, int h0) {
        const uint16_t* in0 = a.in[0] + a.ip[0].row(chunk, l, t);
        const uint16_t* in1 = a.in[1] + a.ip[1].row(chunk, l, t);
#pragma unroll
        for (int i = 0; i < kRotaryHeads; ++i) {
            const int h = h0 + i * w.runs;
            if (h < heads) v[i].load(h < heads0 ? in0 + h * a.dim : in1 + (h - heads0) * a.dim, pa, pb, wide);
        }
    };
    load(l0, run);  // (on their way while the angles are worked out)
    // (position 0 and no factor: the values as they are, infinities and signs of zeros too)
    const bool turns = col < turning && (p != 0 || a.attention != 1.f);
    float c[N], s[N];
    if (turns) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            // (turns is 0 behind the last pair)
            const long long phase = (long long)((unsigned long long)(long long)p * a.turns[col * N + k]);
            sincospif(__ll2float_rn(phase) * 1.0842021724855044e-19f, &s[k], &c[k]);  // 2^-63: half turns
            c[k] *= a.attention;
            s[k] *= a.attention;
        }
    }
    for (int l = l0; l < l1; ++l) {
        uint16_t* out0 = a.out[0] + a.op[0].row(chunk, l, t);
        uint16_t* out1 = a.out[1] + a.op[1].row(chunk, l, t);
        for (int h0 = run; h0 < heads; h0 += kRotaryHeads * w.runs) {
            if (l > l0 || h0 > run) load(l, h0);
#pragma unroll
            for (int i = 0; i < kRotaryHeads; ++i) {
                const int h = h0 + i * w.runs;
                if (h >= heads) continue;
                if (turns) v[i].template turn<LAYOUT>(c, s, pairs);
                v[i].store(h < heads0 ? out0 + h * a.dim : out1 + (h - heads0) * a.dim, pa, pb, wide);
            }
        }
    }
}

void rotary_angles(const kvfix_rope& r, RotaryArgs* a) {
    const int n = r.rotary_dim;
    const double kTwoPi = 6.283185307179586;
    double lo = 0.0, width = 1.0;  // yarn: the pair from which frequencies change, and over how many
    if (r.scaling == KVFIX_ROPE_YARN) {
        auto pair = [&](double turns) { return n * log(r.original_tokens / (kTwoPi * turns)) / (2.0 * log(r.base)); };
        const double hi = fmin(ceil(pair(r.low)), (double)(n - 1));
        lo = fmax(floor(pair(r.high)), 0.0);
        width = fmax(hi - lo, 1e-3);
    }
    memset(a->turns, 0, sizeof a->turns);
    for (int i = 0; i < n / 2; ++i) {
        double theta = pow(r.base, -2.0 * (double)i / (double)n);
        double keep = 1.0;  // the share that keeps its frequency
        if (r.scaling == KVFIX_ROPE_LINEAR) keep = 0.0;
        if (r.scaling == KVFIX_ROPE_BANDS) keep = (r.original_tokens * theta / kTwoPi - r.low) / (r.high - r.low);
        if (r.scaling == KVFIX_ROPE_YARN) keep = 1.0 - (i - lo) / width;
        keep = fmin(fmax(keep, 0.0), 1.0);
        if (r.scaling != KVFIX_ROPE_PLAIN) theta *= keep + (1.0 - keep) / r.factor;
        const double turn = theta / kTwoPi;
        a->turns[i] = (unsigned long long)ldexp(turn - floor(turn), 64);
    }
    a->rotary_dim = n;
    a->layout = r.layout;
    a->attention = (float)r.attention;
}

// Measured: 4096 tokens x 32 layers x 8 heads of 128, half of each head turned: 87 us, 6.2 TB/s (a
// copy's bytes take 79); 8192 tokens x 40 heads of 128 in place: 29 us, 5.7 TB/s (32 with the first
// loads behind the angles); 16 x 8 tokens x 40 heads: 3.4 us, one launch and two trips to memory.
// Halves that vectors do not meet: 24 of 96 turned 4.5 TB/s (3.6 by single pairs), 60 of 64 3.4 (2.5),
// 20 of 128 4.2 (4.4); all of a head by pairs: 2.1.  In 4096 tokens x 32 layers x 8 heads: 81 us (5.0 TB/s),
// 64 (4.2) and 102 (5.3).
// Two or eight heads in flight, streaming loads or stores: even, or up to 10 % slower.
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
    const int heads = a.ip[0].heads + a.ip[1].heads;
    if (a.chunks == 0 || a.layers == 0 || a.tokens == 0 || heads == 0) return cudaSuccess;
    const bool half = a.layout == KVFIX_ROPE_HALF, mixed = half && a.rotary_dim % 16 != 0;
    const int P = mixed_pairs(a.rotary_dim);
    const RotarySplit w = rotary_split(a.chunks, a.layers, a.tokens, heads, a.dim, a.rotary_dim, half, a.in_place);
    const double blocks = (double)a.chunks * w.tiles * w.layer_blocks;
    if (blocks > 2147483647.0) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)((long long)a.chunks * w.tiles * w.layer_blocks)), threads(kRotaryThreads);
    if (mixed && P == 4) rotary_kernel<KVFIX_ROPE_HALF, RotaryMixed<4>><<<grid, threads, 0, s>>>(a, w);
    else if (mixed && P == 2) rotary_kernel<KVFIX_ROPE_HALF, RotaryMixed<2>><<<grid, threads, 0, s>>>(a, w);
    else if (mixed) rotary_kernel<KVFIX_ROPE_HALF, RotaryMixed<1>><<<grid, threads, 0, s>>>(a, w);
    else if (half) rotary_kernel<KVFIX_ROPE_HALF, RotaryVectors><<<grid, threads, 0, s>>>(a, w);
    else rotary_kernel<KVFIX_ROPE_INTERLEAVED, RotaryVectors><<<grid, threads, 0, s>>>(a, w);
    return cudaGetLastError();
}

}  // namespace kvfix
