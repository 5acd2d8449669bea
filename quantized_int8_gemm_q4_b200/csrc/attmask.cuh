// Attention under key intervals: query i attends to the keys [kv_begin[i], kv_end[i]), with
// an optional tanh cap on the scores and an optional bias that falls with distance.
#pragma once
#include "attention.cuh"
#include "rope.cuh"

namespace dllm {

struct MaskArgs {
    const __half *q, *k, *v;
    int64_t ldq, ldk, ldv;
    int32_t Lq, Lk, H, group;
    const int32_t *kv_begin, *kv_end, *q_pos;
    float cap;
    const float* slopes;
    void* o;
    int32_t o_f16;
};

// One warp per (query, head), one online softmax over its interval; lane l holds the
// head-dim values 4l .. 4l + 3.
__global__ void __launch_bounds__(256) attention_masked_kernel(const __grid_constant__ MaskArgs a) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t g = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (g >= (int64_t)a.Lq * a.H) return;
    const int i = (int)(g / a.H), h = (int)(g % a.H), hk = h / a.group;
    const int lo = a.kv_begin ? max(0, a.kv_begin[i]) : 0, hi = a.kv_end ? min(a.Lk, a.kv_end[i]) : a.Lk;
    const int qp = a.q_pos ? a.q_pos[i] : i + a.Lk - a.Lq;
    auto load4 = [&](const __half* p, float (&x)[4]) {
        const uint2 u = *reinterpret_cast<const uint2*>(p + 4 * lane);
        const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&u.x)),
                     t = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
        x[0] = s.x, x[1] = s.y, x[2] = t.x, x[3] = t.y;
    };
    float q[4], acc[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
    load4(a.q + i * a.ldq + h * 128, q);
    const float slope = a.slopes ? a.slopes[h] : 0.0f;
    for (int j = lo; j < hi; j++) {
        float x[4];
        load4(a.k + j * a.ldk + hk * 128, x);
        float s = q[0] * x[0] + q[1] * x[1] + q[2] * x[2] + q[3] * x[3];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        s *= 0.08838834764831845f;
        if (a.cap > 0.0f) s = a.cap * tanhf(s / a.cap);
        if (a.slopes) s -= slope * fabsf((float)qp - (float)j);
        const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn);
        load4(a.v + j * a.ldv + hk * 128, x);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] = acc[e] * c + p * x[e];
        m = mn;
    }
    const float inv = lo < hi ? 1.0f / l : 0.0f;
    const int64_t at = g * 128 + 4 * lane;
    if (a.o_f16)
        *reinterpret_cast<uint2*>(static_cast<__half*>(a.o) + at) =
            make_uint2(pack_h2(acc[0] * inv, acc[1] * inv), pack_h2(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at) =
            make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
}

}  // namespace dllm
