// pool.cuh -- the stored forms of a paged pool's rows (kvfix_pool), shared by the kernels
// that write, read and attend over a pool.
//
//   bf16  the values.
//   e4m3  one byte per value and one byte b per (slot, head): value = e4m3(code) 2^(b-127),
//         or NaN throughout for b = 255 (a row that held a NaN).
//         The scale is a power of two, so scaling a value to its code's range is exact, and
//         every stored value is exactly a bf16 value (4 significant bits, an exponent within
//         [-110-9, 119+8]): nothing is lost when rows are read back or become bf16
//         tensor-core operands.
//   int4  groups of 32 values share a scale and a zero, both bf16: value =
//         bf16(scale code + zero), code in 0..15.  A 32-bit word holds 8 codes, value 2i in
//         nibble i and value 2i+1 in nibble i+4, so that (word >> 4i) & 0x000f000f is the
//         pair (2i, 2i+1) as two 16-bit lanes.
#pragma once

#include "common.cuh"

namespace kvfix {

constexpr int kQGroup = 32;         // values per int4 group
constexpr int kE4m3MinExp = -110;   // smallest and largest power-of-two scale of a row
constexpr int kE4m3MaxExp = 119;

// One layer-major code plane and its scales.
struct PoolPlane {
    unsigned char* codes;
    unsigned char* scales;  // e4m3: [layers][heads][slots] bytes; int4: [layers][heads][slots][dim/32] words
};

struct PoolView {
    int format, layers, slots, heads, dim;
    long long sl, ss;  // byte strides of layer and slot
    PoolPlane plane[2];
};

inline PoolView view_of(const kvfix_pool& p) {
    PoolView v;
    v.format = p.format;
    v.layers = p.layers;
    v.slots = p.slots;
    v.heads = p.kv_heads;
    v.dim = p.head_dim;
    v.sl = p.stride_layer;
    v.ss = p.stride_slot;
    v.plane[0] = {(unsigned char*)p.k, (unsigned char*)p.k_scales};
    v.plane[1] = {(unsigned char*)p.v, (unsigned char*)p.v_scales};
    return v;
}

// Code bytes of one (slot, head).
__host__ __device__ constexpr int pool_head_bytes(int format, int dim) {
    return format == KVFIX_POOL_BF16 ? 2 * dim : format == KVFIX_POOL_E4M3 ? dim : dim / 2;
}

// 2^k, k in [-126, 127].
__device__ __forceinline__ float pow2f(int k) { return __uint_as_float((unsigned)(k + 127) << 23); }

// ------------------------------------------------------------- e4m3 -> bf16, exactly
// A code s eeee mmm moved to the bf16 fields s 0000eeee mmm0000 is the value times 2^-120
// (subnormal codes included, as bf16 subnormals), so one or two exact multiplications by
// powers of two give the stored value: pairs of 2^(120+min(k,7)) and 2^max(k-7,0), k = b - 127.
struct E4m3Scale {
    __nv_bfloat162 a, b;
    bool two;
};

constexpr unsigned kE4m3NanByte = 255;  // the scale byte of a row that holds a NaN: all of it reads NaN

// A stored scale byte (not the NaN one) kept within the format's limits.
__device__ __forceinline__ unsigned e4m3_scale_within(unsigned byte) {
    return min(max(byte, (unsigned)(kE4m3MinExp + 127)), (unsigned)(kE4m3MaxExp + 127));
}

__device__ __forceinline__ E4m3Scale e4m3_scale_byte(unsigned byte) {
    E4m3Scale s;
    const unsigned b = e4m3_scale_within(byte);
    // a bf16 power of two in both halves: (exponent field) * (2^7 + 2^23)
    unsigned aa = (min(b, 134u) + 120u) * 0x00800080u;
    const unsigned bb = (max(b, 134u) - 134u + 127u) * 0x00800080u;
    if (byte == kE4m3NanByte) aa = 0x7fff7fffu;
    s.a = *reinterpret_cast<const __nv_bfloat162*>(&aa);
    s.b = *reinterpret_cast<const __nv_bfloat162*>(&bb);
    s.two = b > 134u;
    return s;
}

// Four codes (bytes in order) to two bf16 pairs: the nibbles of every code at their places in
// the high and the low bytes of the results, then the bytes side by side.
__device__ __forceinline__ uint2 e4m3x4_to_bf16(unsigned codes, __nv_bfloat162 a) {
    const unsigned hi = ((codes >> 4) & 0x07070707u) | (codes & 0x80808080u);
    const unsigned lo = (codes << 4) & 0xf0f0f0f0u;
    unsigned r0 = __byte_perm(lo, hi, 0x5140), r1 = __byte_perm(lo, hi, 0x7362);
    const __nv_bfloat162 p0 = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&r0), a);
    const __nv_bfloat162 p1 = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&r1), a);
    return make_uint2(*reinterpret_cast<const unsigned*>(&p0), *reinterpret_cast<const unsigned*>(&p1));
}

// Sixteen codes to eight pairs.  Scales above 2^7 (values beyond 57344) are rare.
__device__ __forceinline__ void e4m3x16_to_bf16(const uint4& codes, const E4m3Scale& s, uint4& o0, uint4& o1) {
    const uint2 w0 = e4m3x4_to_bf16(codes.x, s.a), w1 = e4m3x4_to_bf16(codes.y, s.a);
    const uint2 w2 = e4m3x4_to_bf16(codes.z, s.a), w3 = e4m3x4_to_bf16(codes.w, s.a);
    unsigned w[8] = {w0.x, w0.y, w1.x, w1.y, w2.x, w2.y, w3.x, w3.y};
    if (s.two) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), s.b);
            w[k] = *reinterpret_cast<const unsigned*>(&p);
        }
    }
    o0 = make_uint4(w[0], w[1], w[2], w[3]);
    o1 = make_uint4(w[4], w[5], w[6], w[7]);
}

// ------------------------------------------------------------- int4 -> bf16
// Eight codes to four bf16 pairs: 128 + code is exact in bf16, so is the difference, and one
// fused multiply-add rounds once.
__device__ __forceinline__ uint4 int4x8_to_bf16(unsigned word, __nv_bfloat162 scale, __nv_bfloat162 zero) {
    unsigned r[4];
    const unsigned k128 = 0x43004300u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unsigned c = ((word >> (4 * i)) & 0x000f000fu) | k128;
        const __nv_bfloat162 n =
            __hsub2(*reinterpret_cast<__nv_bfloat162*>(&c), *reinterpret_cast<const __nv_bfloat162*>(&k128));
        const __nv_bfloat162 v = __hfma2(n, scale, zero);
        r[i] = *reinterpret_cast<const unsigned*>(&v);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace kvfix
