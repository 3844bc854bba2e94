// attend.cu -- kvfix_shared_attend: attention of a round's agents over a shared prefix and
// their own tokens, straight from a paged pool.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attend.h"
#include "pool.cuh"
#include "softmax.cuh"

namespace kvfix {

static __device__ unsigned int g_status_attend;

unsigned read_status_attend(cudaStream_t stream) {
    unsigned h = 0, zero = 0;
    cudaMemcpyFromSymbolAsync(&h, g_status_attend, sizeof h, 0, cudaMemcpyDeviceToHost, stream);
    cudaMemcpyToSymbolAsync(g_status_attend, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    cudaStreamSynchronize(stream);
    return h;
}

// One stored value in float.
template <int F>
__device__ __forceinline__ float stored_value(const PoolView& p, int plane, int slot, int head, int e) {
    const unsigned char* row = p.plane[plane].codes + (long long)slot * p.ss +
                               (long long)head * pool_head_bytes(F, p.dim);
    const long long r = (long long)head * p.slots + slot;
    if (F == KVFIX_POOL_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[e]);
    if (F == KVFIX_POOL_E4M3) {
        const E4m3Scale s = e4m3_scale(min(max((int)p.plane[plane].scales[r] - 127, kE4m3MinExp), kE4m3MaxExp));
        const unsigned c = row[e];
        uint2 v = e4m3x4_to_bf16(c, s);
        if (e4m3x4_has_nan(c)) v = e4m3x4_nan(c, v);
        return __uint_as_float(v.x << 16);
    }
    const unsigned sz = reinterpret_cast<const unsigned*>(p.plane[plane].scales)[r * (p.dim / kQGroup) + e / kQGroup];
    const unsigned w = reinterpret_cast<const unsigned*>(row)[e / 8];
    const int at = 4 * ((e % 8) / 2) + 16 * (e & 1);
    const float v = fmaf((float)((w >> at) & 15u), __uint_as_float(sz << 16), __uint_as_float(sz & 0xffff0000u));
    return __bfloat162float(__float2bfloat16_rn(v));
}

// One warp per (agent, token, query head): the definition, key by key.
template <int F>
__global__ void __launch_bounds__(128) attend_rows_kernel(const __grid_constant__ AttendArgs a) {
    const long long w = (long long)blockIdx.x * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (w >= (long long)a.agents * a.new_tokens * a.q_heads) return;
    const int qh = (int)(w % a.q_heads), t = (int)(w / a.q_heads % a.new_tokens);
    const int agent = (int)(w / ((long long)a.q_heads * a.new_tokens));
    const int D = a.pool.dim, per = D / 32, head = qh / (a.q_heads / a.pool.heads);
    bool bad = false;
    int group = -1, reached = 0;
    for (int g = 0; g < a.groups; ++g) {
        const int b = a.group_begin[g], e = a.group_begin[g + 1];
        if (b < reached || e < b || e > a.agents) bad = true;
        const int bb = min(max(b, reached), a.agents), ee = min(max(e, bb), a.agents);
        reached = ee;
        if (agent >= bb && agent < ee) group = g;
    }
    const int pages = a.pool.slots / a.page;
    int n0 = group >= 0 ? a.prefix_len[group] : 0, n1 = a.suffix_len[agent];
    if (n0 < 0 || n0 > a.max_prefix_pages * a.page || n1 < 0 || n1 > a.max_suffix_pages * a.page) bad = true;
    n0 = min(max(n0, 0), a.max_prefix_pages * a.page);
    n1 = min(max(n1, 0), a.max_suffix_pages * a.page);
    const int sees = min(n0 + n1, n0 + n1 - a.new_tokens + 1 + t);
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, s = 0.f;
    const long long qo = a.qp.row(agent, 0, t) + (long long)qh * D + lane * per;
    for (int i = 0; i < per; ++i) q[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[qo + i]);
    for (int key = 0; key < sees; ++key) {
        const bool own = key >= n0;
        const int at = own ? key - n0 : key;
        const int page = own ? a.suffix_pages[(long long)agent * a.max_suffix_pages + at / a.page]
                             : a.prefix_pages[(long long)group * a.max_prefix_pages + at / a.page];
        if (page < 0 || page >= pages) {
            bad = true;
            continue;
        }
        const int slot = page * a.page + at % a.page;
        float z = 0.f;
        for (int i = 0; i < per; ++i) z += q[i] * stored_value<F>(a.pool, 0, slot, head, lane * per + i);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
        z *= a.scale_log2;
        const float M = fmaxf(m, z), c = exp2f(m - M), p = exp2f(z - M);
        s = s * c + p;
        for (int i = 0; i < per; ++i) o[i] = o[i] * c + p * stored_value<F>(a.pool, 1, slot, head, lane * per + i);
        m = M;
    }
    const float inv = s > 0.f ? 1.f / s : 0.f;
    const long long oo = a.op.row(agent, 0, t) + (long long)qh * D + lane * per;
    for (int i = 0; i < per; ++i)
        reinterpret_cast<__nv_bfloat16*>(a.out)[oo + i] = __float2bfloat16_rn(o[i] * inv);
    if (a.lse && lane == 0) a.lse[w] = s > 0.f ? (m + log2f(s)) * 0.69314718055994531f : -INFINITY;
    if (bad && lane == 0) atomicOr(&g_status_attend, FLAG_BOUNDS);
}

size_t attend_workspace_bytes(int, int, int, int, int, int) { return 16; }

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
    const long long rows = (long long)a.agents * a.new_tokens * a.q_heads;
    if (rows == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (a.pool.format == KVFIX_POOL_BF16) attend_rows_kernel<KVFIX_POOL_BF16><<<grid, 128, 0, s>>>(a);
    else if (a.pool.format == KVFIX_POOL_E4M3) attend_rows_kernel<KVFIX_POOL_E4M3><<<grid, 128, 0, s>>>(a);
    else attend_rows_kernel<KVFIX_POOL_INT4><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kvfix
