// Rotary positions of queries and keys between the Q/K/V projections and attention
// (mojo-dllm Architecture page, "A forward pass", step 2; "Source map", kernels/ops.mojo:
// RoPE in its NORM and NEOX variants), with an optional RMSNorm of each query and key
// head in the same pass, and the rounding of q, k and v to f16.
//
//   y = x gamma / sqrt(mean(x^2) + eps)                      (only with a gamma)
//   (y1, y2) -> ms (y1 cos a - y2 sin a, y2 cos a + y1 sin a),  a = 2 pi pos turns[i]
//
// over the pairs i of the head's first n_rot elements: (2i, 2i + 1) in the NORM layout,
// (i, i + n_rot / 2) in the NEOX layout; the other elements pass through.
//
// Bound by HBM: 4 bytes read and 2 written per element, ~10 operations.  A head is
// dealt with by G lanes (G = dh / 8 rounded up to a power of two) of 8 elements each: two
// 16-byte loads, one 16-byte store (NORM, or past n_rot) or two 8-byte ones.  Lane l of
// every head rotates the pairs 4l .. 4l + 3, so a thread forms its four angles once and
// uses them for all the heads it visits.  The angle's turns are formed in f64 (position
// times turns, minus the nearest whole number): exact to 2^-24 of a turn for every int32
// position, where an f32 product is off by whole turns.  Norm sums, rotation: f32; one
// rounding to f16.
//
// Measured (one B200, launches replayed from a graph): 4096 positions of 32 + 32 + 32 heads of 128
// with both norms 52.5 us, 5.75 TB/s, 0.89 of the measured copy rate; 1021 positions of 28 + 4 + 4
// 7.6 us (0.57; 36 heads leave the last of three per thread mostly idle, and a quarter of the
// instructions are the angles); 128 positions 3.4 us, one position 1.7 us (a launch).  Three heads
// in flight per thread at 64 registers beat two (1021 positions: 8.8 us) and one (9.4).
#pragma once

#include "layout.cuh"

namespace dllm {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_BATCH = 3;  // heads in flight per thread

struct RopeArgs {
    const float *q, *k, *v;
    int64_t ldq, ldk, ldv;
    int64_t L;
    int32_t H, Hkv, T;   // query heads, key heads, all heads with v's
    int32_t dh, n_rot;
    int32_t chunk;       // heads per CTA
    const int32_t* pos;
    const double* turns;
    float ms, eps;
    const float *gq, *gk;
    __half *oq, *ok, *ov;
};

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Grid (tokens, head chunks).  G lanes per head.
template <int G, bool NEOX>
__global__ void __launch_bounds__(ROPE_THREADS) qk_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int SLOTS = ROPE_THREADS / G;
    pdl_trigger();
    pdl_wait();
    const int l = threadIdx.x % G, slot = threadIdx.x / G;
    const int64_t tok = blockIdx.x;
    const bool on = 8 * l < a.dh;  // lanes past the head (dh / 8 not a power of two) idle along
    const bool rot = 8 * l < a.n_rot;
    // element offsets of this lane's two float4
    const int e0 = NEOX && rot ? 4 * l : 8 * l;
    const int e1 = NEOX && rot ? 4 * l + a.n_rot / 2 : 8 * l + 4;

    const int h_end = min(a.T, ((int)blockIdx.y + 1) * a.chunk);
    const int h_begin = (int)blockIdx.y * a.chunk;

    float cs[4], sn[4];
    bool have = false;
    for (int hb = h_begin; hb < h_end; hb += ROPE_BATCH * SLOTS) {
        float x[ROPE_BATCH][8];
#pragma unroll
        for (int j = 0; j < ROPE_BATCH; j++) {
            const int h = hb + j * SLOTS + slot;
            if (on && h < h_end) {
                const float* src = h < a.H ? a.q + tok * a.ldq + (int64_t)h * a.dh
                                   : h < a.H + a.Hkv ? a.k + tok * a.ldk + (int64_t)(h - a.H) * a.dh
                                                     : a.v + tok * a.ldv + (int64_t)(h - a.H - a.Hkv) * a.dh;
                const float4 u = __ldg(reinterpret_cast<const float4*>(src + e0));
                const float4 w = __ldg(reinterpret_cast<const float4*>(src + e1));
                x[j][0] = u.x; x[j][1] = u.y; x[j][2] = u.z; x[j][3] = u.w;
                x[j][4] = w.x; x[j][5] = w.y; x[j][6] = w.z; x[j][7] = w.w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) x[j][e] = 0.0f;
            }
        }
        if (!have && rot && hb < a.H + a.Hkv) {
            have = true;
            const double p = a.pos ? (double)__ldg(a.pos + tok) : (double)tok;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const double t = p * __ldg(a.turns + 4 * l + e);
                const float r = (float)(t - rint(t));  // -0.5 .. 0.5 of a turn
                sincospif(2.0f * r, &sn[e], &cs[e]);
                sn[e] *= a.ms;
                cs[e] *= a.ms;
            }
        }
#pragma unroll
        for (int j = 0; j < ROPE_BATCH; j++) {
            const int h = hb + j * SLOTS + slot;
            const bool is_q = h < a.H, is_v = h >= a.H + a.Hkv;
            const float* gamma = is_q ? a.gq : is_v ? nullptr : a.gk;
            if (a.gq != nullptr || a.gk != nullptr) {  // uniform: every lane takes part in the sum
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++) ss = fmaf(x[j][e], x[j][e], ss);
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (gamma != nullptr && on) {
                    const float rn = 1.0f / sqrtf(ss / (float)a.dh + a.eps);
                    const float4 u = __ldg(reinterpret_cast<const float4*>(gamma + e0));
                    const float4 w = __ldg(reinterpret_cast<const float4*>(gamma + e1));
                    x[j][0] *= rn * u.x; x[j][1] *= rn * u.y; x[j][2] *= rn * u.z; x[j][3] *= rn * u.w;
                    x[j][4] *= rn * w.x; x[j][5] *= rn * w.y; x[j][6] *= rn * w.z; x[j][7] *= rn * w.w;
                }
            }
            if (!on || h >= h_end) continue;
            if (rot && !is_v) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float& y1 = x[j][NEOX ? e : 2 * e];
                    float& y2 = x[j][NEOX ? e + 4 : 2 * e + 1];
                    const float t1 = y1 * cs[e] - y2 * sn[e], t2 = y2 * cs[e] + y1 * sn[e];
                    y1 = t1;
                    y2 = t2;
                }
            }
            __half* dst = is_q ? a.oq + (tok * a.H + h) * (int64_t)a.dh
                          : is_v ? a.ov + (tok * a.Hkv + (h - a.H - a.Hkv)) * (int64_t)a.dh
                                 : a.ok + (tok * a.Hkv + (h - a.H)) * (int64_t)a.dh;
            const uint2 lo = make_uint2(pack_h2(x[j][0], x[j][1]), pack_h2(x[j][2], x[j][3]));
            const uint2 hi = make_uint2(pack_h2(x[j][4], x[j][5]), pack_h2(x[j][6], x[j][7]));
            if (NEOX && rot) {
                *reinterpret_cast<uint2*>(dst + e0) = lo;
                *reinterpret_cast<uint2*>(dst + e1) = hi;
            } else {
                *reinterpret_cast<uint4*>(dst + e0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
    }
}

}  // namespace dllm
