// Sampling one token per row of logits (mojo-dllm Architecture page, "Source map",
// diffusion/sampler.mojo; "A forward pass", step 4: the logits of the requested rows),
// with the two figures that order the rows of a denoising step: the chosen token's
// probability and the entropy, both of the plain softmax.
//
//   w_i = exp((l_i - max) / T);  candidates in the order (l descending, i ascending);
//   kept: the first k, of these the ones with w_i >= min_p, of these (mass S) the ones
//   whose preceding mass is < p S, and always the first;
//   token = the first kept i, in index order, whose running mass exceeds u * kept mass.
//
// Every limit keeps a prefix of the one order, so no sort is needed: a limit is a cut
// (value, index), found by a histogram over the values and an exact ranking of the one
// bin it falls into.  Weights are 64-bit fixed point (at least 2^-45 of the largest at
// 2^17 candidates) from an f64 exponential: integer sums do not depend on their order, so
// atomics and any split over threads and CTAs give one result, and a border between two
// tokens is off by less than 2^-36 of the mass (f32 sums put 1 row in ~400 on the wrong
// side of one).
//
// One cluster of C CTAs per row.  Each CTA keeps its slice of the row in shared memory (read
// from HBM once); every step is one pass over the slices and one cluster barrier:
//   load and largest logit | plain softmax sums and histogram | gathering of the crossing
//   bin (one per limit) | kept mass of each warp's range.
// What a step exchanges is written into every CTA of the cluster and evaluated by all of them
// alike, so that no step waits for an answer.  A histogram is exchanged as 64 coarse sums;
// the 32 bins behind the crossing one are then read from the other CTAs.
// Bound: the logits' bytes; in practice the passes' arithmetic (the f64 exponentials) and the
// cluster barriers between them.
#pragma once
#include <cooperative_groups.h>

#include "layout.cuh"

namespace dllm {

constexpr int SMP_THREADS = 512;
constexpr int SMP_WARPS = SMP_THREADS / 32;
constexpr int SMP_BINS = 2048;
constexpr int SMP_COARSE = SMP_BINS / 32;
constexpr int SMP_LIST = SMP_THREADS;  // elements ranked exactly, one per thread
constexpr int SMP_MAX_CLUSTER = 16;
constexpr int SMP_TABLE = 256;
constexpr int ERR_LOGITS = -10;
typedef unsigned long long u64;

struct SampleArgs {
    const float* logits;
    int64_t V, ldl;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* token;
    float *conf, *entropy;
    int32_t slice;   // elements per CTA (a multiple of 128)
    int32_t cached;  // of them, held in shared memory (a multiple of 4)
    int32_t fix;     // weights are multiples of 2^-fix
};

struct alignas(16) SampleShared {  // the slice follows it, read in 16-byte vectors
    uint32_t cnt[SMP_BINS], lo[SMP_BINS], hi[SMP_BINS];  // this CTA's histogram: count, mass
    uint32_t ccnt[SMP_MAX_CLUSTER][SMP_COARSE];          // every CTA's coarse sums
    u64 cmass[SMP_MAX_CLUSTER][SMP_COARSE];
    u64 before_c[SMP_COARSE + 1], before_m[SMP_COARSE + 1];  // the cluster's, before each coarse bin
    u64 lcode[SMP_LIST], lw[SMP_LIST];                   // the gathered bin: order code, weight
    u64 box[2][4][SMP_MAX_CLUSTER];                      // one exchange: words of every CTA
    u64 red[4][SMP_WARPS];
    u64 found[3], kept_mass;  // crossing bin: count before, mass before, its count; mass up to the cut
    double table[SMP_TABLE];  // 2^(i / 256)
    uint32_t found_bin, n_list, best;
    u64 cut;                  // order code
};

static_assert(sizeof(SampleShared) % 16 == 0, "the slice behind it is read as float4");

// Order-preserving code of a float (which is not -0): larger value, larger code.
__device__ __forceinline__ uint32_t smp_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float smp_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ u64 smp_warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ u64 smp_warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}
__device__ __forceinline__ double smp_warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One row, as one CTA of its cluster sees it.
struct SampleRow {
    cooperative_groups::cluster_group cl;
    SampleShared& sm;
    const float* src;   // row in global memory
    float* cache;
    int64_t V;
    int C, r, w, lane;  // CTAs, this one's rank; warp, lane
    int n, cached;      // elements of the slice (a multiple of 4), and of them in shared memory
    int64_t first;      // row index of the slice's first element (before the row: filled with -inf)
    float top;          // largest logit
    double scale;       // log2(e) / T
    double least;       // base-2 exponents below it round to weight 0
    double min_w;       // 2^fix * min_p
    int fix;
    float cut_val;      // kept: above, or equal and not behind cut_idx
    uint32_t cut_idx;
    int phase;
    // the present histogram: values [vmin, vmax], spread evenly by value or by code
    float vmin, vmax, vhi, inv;
    int shift;
    bool linear;

    // Four elements; outside the row -inf.  -0 becomes +0.
    __device__ __forceinline__ float4 load4(int i) const {
        const int64_t g = first + i;
        float4 x;
        if (g >= 0 && g + 4 <= V) {
            x = __ldg(reinterpret_cast<const float4*>(src + g));
        } else {
            x.x = g >= 0 && g < V ? __ldg(src + g) : -INFINITY;
            x.y = g + 1 >= 0 && g + 1 < V ? __ldg(src + g + 1) : -INFINITY;
            x.z = g + 2 >= 0 && g + 2 < V ? __ldg(src + g + 2) : -INFINITY;
            x.w = g + 3 >= 0 && g + 3 < V ? __ldg(src + g + 3) : -INFINITY;
        }
        return make_float4(x.x + 0.0f, x.y + 0.0f, x.z + 0.0f, x.w + 0.0f);
    }
    __device__ __forceinline__ float4 at4(int i) const {
        return i < cached ? *reinterpret_cast<const float4*>(cache + i) : load4(i);
    }
    __device__ __forceinline__ uint32_t index(int i) const { return (uint32_t)(first + i); }

    // Fixed-point weight of a logit, 0 below min_p: 2^t by table and polynomial (Tang 1989),
    // t = k + j / 256 + f, |f| <= 2^-9, the polynomial's next term below 2^-54.  Adding
    // 1.5 2^44 rounds t to a multiple of 1/256 and leaves 256 k + j in the low word; adding
    // 2^52 to the weight times 2^fix rounds it to a whole number, held by the low mantissa.
    __device__ __forceinline__ u64 weight(float l) const {
        const double t = ((double)l - (double)top) * scale;
        if (!(t > least)) return 0;
        const double tm = t + 26388279066624.0;
        const int kj = __double2loint(tm);
        const double f = t - (tm - 26388279066624.0);
        const double b = sm.table[kj & 255];
        double q = fma(f, 0.009618129107628477, 0.05550410866482158);
        q = fma(f, q, 0.2402265069591007);
        q = fma(f, q, 0.6931471805599453);
        double e = fma(b * f, q, b);
        e = __hiloint2double(__double2hiint(e) + (((kj >> 8) + fix) << 20), __double2loint(e));
        return e < min_w ? 0 : __double_as_longlong(e + 4503599627370496.0) & 0xfffffffffffffull;
    }
    __device__ __forceinline__ bool kept(float l, int i) const {
        return l > cut_val || (l == cut_val && index(i) <= cut_idx);
    }
    __device__ __forceinline__ bool in_range(float l, int i) const { return l >= vmin && l <= vmax && kept(l, i); }
    __device__ __forceinline__ int bin_of(float l) const {
        return linear ? min(SMP_BINS - 1, (int)(fmaf(-0.25f, l, vhi) * inv)) : (int)((smp_key(vmax) - smp_key(l)) >> shift);
    }
    // The slice's elements, four at a time per thread.
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
        for (int i = 4 * threadIdx.x; i < n; i += 4 * SMP_THREADS) {
            const float4 x = at4(i);
            f(x.x, i);
            f(x.y, i + 1);
            f(x.z, i + 2);
            f(x.w, i + 3);
        }
    }

    // Exchange of four words per CTA (thread 0's); after it every CTA holds all of them in
    // the returned box.  Boxes alternate: a CTA may write the next exchange while another
    // still reads this one.
    __device__ __forceinline__ const u64 (*exchange(u64 a, u64 b, u64 c, u64 d))[SMP_MAX_CLUSTER] {
        u64(*box)[SMP_MAX_CLUSTER] = sm.box[phase++ & 1];
        if ((int)threadIdx.x < C) {
            u64* dst = cl.map_shared_rank(&box[0][0], threadIdx.x);
            dst[r] = a;
            dst[SMP_MAX_CLUSTER + r] = b;
            dst[2 * SMP_MAX_CLUSTER + r] = c;
            dst[3 * SMP_MAX_CLUSTER + r] = d;
        }
        cl.sync();
        return box;
    }

    // Counts (and masses) of the candidates with values in [lo, hi] over the bins, and their
    // sums before each coarse bin, starting from c0, m0.  by_value spreads the values evenly
    // over the bins (both sides scaled by 1/4, so that no difference overflows; monotone, as
    // each operation rounds monotonically); else the codes, which always splits the range.
    __device__ void histogram(float lo, float hi, bool by_value, bool mass, u64 c0, u64 m0) {
        vmin = lo;
        vmax = hi;
        vhi = 0.25f * hi;
        const float span = vhi - 0.25f * lo;
        inv = (float)SMP_BINS / span;
        shift = max(0, 32 - __clz(smp_key(hi) - smp_key(lo)) - 11);
        linear = by_value && span > 0.0f && inv < 1e30f;
        for (int i = threadIdx.x; i < SMP_BINS; i += SMP_THREADS) sm.cnt[i] = sm.lo[i] = sm.hi[i] = 0;
        __syncthreads();
        each([&](float l, int i) {
            if (!in_range(l, i)) return;
            const int b = bin_of(l);
            if (mass) {
                const u64 wt = weight(l);
                if (wt == 0) return;  // no candidate, or one that no mass limit can tell apart
                const uint32_t wl = (uint32_t)wt, old = atomicAdd(&sm.lo[b], wl);
                const uint32_t wh = (uint32_t)(wt >> 32) + (old + wl < old ? 1u : 0u);
                if (wh) atomicAdd(&sm.hi[b], wh);
            }
            atomicAdd(&sm.cnt[b], 1u);
        });
        __syncthreads();
        for (int cb = w; cb < SMP_COARSE; cb += SMP_WARPS) {
            const int b = 32 * cb + lane;
            const uint32_t c = __reduce_add_sync(0xffffffffu, sm.cnt[b]);
            u64 m = 0;
            if (mass) {
                const uint32_t x = sm.lo[b];
                m = ((u64)__reduce_add_sync(0xffffffffu, sm.hi[b]) << 32) +
                    ((u64)__reduce_add_sync(0xffffffffu, x >> 16) << 16) + __reduce_add_sync(0xffffffffu, x & 0xffffu);
            }
            if (lane < C) {
                *cl.map_shared_rank(&sm.ccnt[r][cb], lane) = c;
                *cl.map_shared_rank(&sm.cmass[r][cb], lane) = m;
            }
        }
        cl.sync();
        if (w == 0) {
            u64 c[2] = {0, 0}, m[2] = {0, 0};
            for (int t = 0; t < C; t++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    c[h] += sm.ccnt[t][2 * lane + h];
                    m[h] += sm.cmass[t][2 * lane + h];
                }
            const u64 ic = smp_warp_scan(c[0] + c[1], lane) + c0, im = smp_warp_scan(m[0] + m[1], lane) + m0;
            sm.before_c[2 * lane + 1] = ic - c[1];
            sm.before_c[2 * lane + 2] = ic;
            sm.before_m[2 * lane + 1] = im - m[1];
            sm.before_m[2 * lane + 2] = im;
            if (lane == 0) sm.before_c[0] = c0, sm.before_m[0] = m0;
        }
        __syncthreads();
    }

    // The cut at the first `limit` candidates (by_count), or at the candidates whose preceding
    // mass is < limit; the present histogram holds the border.  Its bins are lost (false) where
    // the crossing one had to be spread again.  mass: the histogram has masses.
    __device__ bool narrow(bool by_count, bool mass, u64 limit) {
        bool whole = true;
        for (;;) {
            // the crossing bin: the first with count (mass) up to its end >= limit
            if (w == 0) {
                const u64* before = by_count ? sm.before_c : sm.before_m;
                const bool x0 = before[lane] < limit && before[lane + 1] >= limit;
                const bool x1 = before[lane + 32] < limit && before[lane + 33] >= limit;
                const uint32_t y0 = __ballot_sync(0xffffffffu, x0), y1 = __ballot_sync(0xffffffffu, x1);
                const int cb = y0 ? __ffs(y0) - 1 : 31 + __ffs(y1);
                const int b = 32 * cb + lane;
                u64 c = 0, m = 0;
#pragma unroll 8
                for (int t = 0; t < C; t++) {
                    const SampleShared* o = cl.map_shared_rank(&sm, t);
                    c += o->cnt[b];
                    m += ((u64)o->hi[b] << 32) + o->lo[b];
                }
                const u64 ec = sm.before_c[cb] + smp_warp_scan(c, lane) - c, em = sm.before_m[cb] + smp_warp_scan(m, lane) - m;
                const u64 x = by_count ? ec : em, y = x + (by_count ? c : m);
                if (x < limit && y >= limit) {
                    sm.found_bin = b;
                    sm.found[0] = ec;
                    sm.found[1] = em;
                    sm.found[2] = c;
                }
                if (lane == 0) sm.best = 0;
            }
            if (r == 0 && threadIdx.x == 32) sm.n_list = 0;
            // CTA 0's counter is zero, and every CTA has read the bins, before any goes on
            cl.sync();
            const int bin = (int)sm.found_bin;
            const u64 c0 = sm.found[0], m0 = sm.found[1];
            // What lies below this is behind the bin: its lower edge, less a hundredth of a bin
            // for the rounding of bin_of and a few units in the last place for its own.
            const float under = linear ? 4.0f * (vhi - ((float)bin + 1.01f) / inv) - 4e-6f * fabsf(vhi) : vmin;
            if (sm.found[2] <= SMP_LIST) {
                each([&](float l, int i) {
                    if (l < under || !in_range(l, i) || bin_of(l) != bin) return;
                    const u64 wt = mass ? weight(l) : 0;
                    if (mass && wt == 0) return;
                    const uint32_t slot = atomicAdd(cl.map_shared_rank(&sm.n_list, 0), 1u);
                    if (slot >= SMP_LIST) return;
                    const u64 code = ((u64)smp_key(l) << 32) | (uint32_t)~index(i);
                    for (int t = 0; t < C; t++) {
                        SampleShared* o = cl.map_shared_rank(&sm, t);
                        o->lcode[slot] = code;
                        o->lw[slot] = wt;
                    }
                });
                cl.sync();
                // each gathered element's rank: the last one kept is the cut
                const int m = (int)sm.found[2], e = (int)threadIdx.x;
                const u64 code = e < m ? sm.lcode[e] : 0;
                uint32_t rank = 0;
                u64 pre = m0;
                bool in = false;
                if (e < m) {
#pragma unroll 4
                    for (int j = 0; j < m; j++) {
                        const bool is_before = sm.lcode[j] > code;
                        rank += is_before;
                        pre += is_before ? sm.lw[j] : 0;
                    }
                    in = (by_count ? c0 + rank : pre) < limit;
                }
                const uint32_t last = __reduce_max_sync(0xffffffffu, in ? rank + 1 : 0);
                if (lane == 0 && last) atomicMax(&sm.best, last);
                __syncthreads();
                if (in && rank + 1 == sm.best) sm.cut = code, sm.kept_mass = pre + sm.lw[e];
                __syncthreads();
                break;
            }
            // too many to rank: the bin's own range of codes
            whole = false;
            uint32_t a = 0, b = 0;  // largest code, largest complement
            if (linear) {
                each([&](float l, int i) {
                    if (l < under || !in_range(l, i) || bin_of(l) != bin) return;
                    a = max(a, smp_key(l));
                    b = max(b, ~smp_key(l));
                });
                a = __reduce_max_sync(0xffffffffu, a);
                b = __reduce_max_sync(0xffffffffu, b);
                if (lane == 0) sm.red[0][w] = a, sm.red[1][w] = b;
                __syncthreads();
                for (int j = 0; j < SMP_WARPS; j++) a = max(a, (uint32_t)sm.red[0][j]), b = max(b, (uint32_t)sm.red[1][j]);
                const u64(*box)[SMP_MAX_CLUSTER] = exchange(a, b, 0, 0);
                for (int t = 0; t < C; t++) a = max(a, (uint32_t)box[0][t]), b = max(b, (uint32_t)box[1][t]);
                b = ~b;
            } else {
                a = smp_key(vmax) - ((uint32_t)bin << shift);
                b = max(smp_key(vmin), shift ? a - ((1u << shift) - 1u) : a);
            }
            if (a != b) {
                histogram(smp_value(b), smp_value(a), false, mass, c0, m0);
                continue;
            }
            // all equal: the first q of them in index order
            const float tie = smp_value(a);
            const u64 wt = mass ? weight(tie) : 0;
            const u64 q = by_count ? limit - c0 : (limit - m0 + wt - 1) / wt;  // before = m0 + j wt < limit
            locate([&](float l, int i) -> u64 { return l == tie && kept(l, i) ? 1 : 0; }, tie, q - 1, -1.0, 0.0, 0.0, 0.0,
                   [&](float, uint32_t at) {
                       for (int t = 0; t < C; t++) *cl.map_shared_rank(&sm.cut, t) = ((u64)a << 32) | (uint32_t)~at;
                   });
            if (threadIdx.x == 0) sm.kept_mass = m0 + q * wt;
            cl.sync();
            break;
        }
        cut_val = smp_value((uint32_t)(sm.cut >> 32));
        cut_idx = ~(uint32_t)sm.cut;
        return whole;
    }

    // The first element, in index order, whose running sum of weight_of exceeds `target`
    // (below the row's total); with u >= 0 the target is min(floor(u * total), total - 1).
    // Elements below `under` weigh nothing.  Calls hit(value, index) on the one thread that
    // finds it.  s1, s2, s3: this warp's sums, which the same exchange adds up over the row
    // (into sums[]).
    template <typename W, typename H>
    __device__ void locate(W weight_of, float under, u64 target, double u, double s1, double s2, double s3, H hit) {
        const int per = ((n + SMP_WARPS - 1) / SMP_WARPS + 3) & ~3;  // a warp's contiguous share
        const int lo = min(n, w * per), hi = min(n, lo + per);
        u64 s = 0;
        auto four = [&](const float4& x, int i, u64 (&v)[4]) {
            v[0] = x.x >= under ? weight_of(x.x, i) : 0;
            v[1] = x.y >= under ? weight_of(x.y, i + 1) : 0;
            v[2] = x.z >= under ? weight_of(x.z, i + 2) : 0;
            v[3] = x.w >= under ? weight_of(x.w, i + 3) : 0;
        };
#pragma unroll 2
        for (int i = lo + 4 * lane; i < hi; i += 128) {
            u64 v[4];
            four(at4(i), i, v);
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        s = smp_warp_sum(s);
        __syncthreads();
        if (lane == 0) {
            sm.red[0][w] = s;
            sm.red[1][w] = __double_as_longlong(s1);
            sm.red[2][w] = __double_as_longlong(s2);
            sm.red[3][w] = __double_as_longlong(s3);
        }
        __syncthreads();
        u64 mine = 0;
        s1 = s2 = s3 = 0.0;
        for (int j = 0; j < SMP_WARPS; j++) {
            mine += sm.red[0][j];
            s1 += __longlong_as_double(sm.red[1][j]);
            s2 += __longlong_as_double(sm.red[2][j]);
            s3 += __longlong_as_double(sm.red[3][j]);
        }
        const u64(*box)[SMP_MAX_CLUSTER] =
            exchange(mine, __double_as_longlong(s1), __double_as_longlong(s2), __double_as_longlong(s3));
        u64 before = 0, total = 0;
        s1 = s2 = s3 = 0.0;
        for (int t = 0; t < C; t++) {
            if (t < r) before += box[0][t];
            total += box[0][t];
            s1 += __longlong_as_double(box[1][t]);
            s2 += __longlong_as_double(box[2][t]);
            s3 += __longlong_as_double(box[3][t]);
        }
        sums[0] = s1;
        sums[1] = s2;
        sums[2] = s3;
        if (u >= 0.0) {
            target = (u64)(u * (double)total);
            if (target >= total) target = total - 1;
        }
        if (target < before || target - before >= mine) return;  // another CTA's (uniform)
        u64 run = before;
        int wi = 0;
        while (run + sm.red[0][wi] <= target) run += sm.red[0][wi++];
        const int a = min(n, wi * per), b = min(n, a + per);
        for (int i0 = a; i0 < b; i0 += 4 * SMP_THREADS) {
            const int i = i0 + 4 * (int)threadIdx.x;
            u64 v[4] = {0, 0, 0, 0};
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < b) {
                x = at4(i);
                four(x, i, v);
            }
            const u64 sum = (v[0] + v[1]) + (v[2] + v[3]);
            const u64 inc = smp_warp_scan(sum, lane);
            __syncthreads();
            if (lane == 31) sm.red[1][w] = inc;
            __syncthreads();
            u64 upto = run + inc - sum;
            for (int j = 0; j < SMP_WARPS; j++) {
                const u64 y = sm.red[1][j];
                upto += j < w ? y : 0;
                run += y;
            }
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (v[e] != 0 && upto <= target && upto + v[e] > target) hit(xs[e], index(i + e));
                upto += v[e];
            }
        }
    }
    double sums[3];
};

// Grid (C * rows), clusters of C.
__global__ void __launch_bounds__(SMP_THREADS, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    SampleShared& sm = *reinterpret_cast<SampleShared*>(smem);
    SampleRow row{cooperative_groups::this_cluster(), sm};
    const int C = row.C = (int)row.cl.num_blocks(), r = row.r = (int)row.cl.block_rank();
    const int64_t i_row = blockIdx.x / C;
    row.w = threadIdx.x >> 5;
    row.lane = threadIdx.x & 31;
    row.phase = 0;
    row.cl.barrier_arrive();  // every CTA has started before another writes into it (waited for below)
    if (threadIdx.x < SMP_TABLE) sm.table[threadIdx.x] = exp2((double)threadIdx.x / SMP_TABLE);
    pdl_trigger();
    pdl_wait();

    // Slices start on 16-byte boundaries of global memory, whatever the row's address: the
    // first one begins up to three elements before the row.
    row.src = a.logits + i_row * a.ldl;
    row.V = a.V;
    row.cache = reinterpret_cast<float*>(smem + sizeof(SampleShared));
    const int64_t before = (int64_t)(reinterpret_cast<uintptr_t>(row.src) >> 2 & 3);
    row.first = (int64_t)r * a.slice - before;
    const int64_t left = a.V - row.first;
    const int n = row.n = (int)(left < a.slice ? max((int64_t)0, (left + 3) & ~(int64_t)3) : a.slice);
    row.cached = min(n, a.cached);

    const float T = a.temperature ? __ldg(a.temperature + i_row) : 1.0f;
    const bool greedy = !(T > 0.0f);
    const float mp = a.min_p ? __ldg(a.min_p + i_row) : 0.0f;
    const float p = a.top_p ? __ldg(a.top_p + i_row) : 1.0f;
    const int32_t k = greedy ? 1 : a.top_k ? __ldg(a.top_k + i_row) : 0;
    float u = a.u ? __ldg(a.u + i_row) : 0.0f;
    u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;  // NaN counts as 0

    // the slice into shared memory; the row's largest and smallest finite logit
    float hi = -INFINITY, lo = INFINITY;
    bool bad = false;
#pragma unroll 4
    for (int i = 4 * threadIdx.x; i < n; i += 4 * SMP_THREADS) {
        const float4 x = row.load4(i);
        if (i < row.cached) *reinterpret_cast<float4*>(row.cache + i) = x;
        const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
            bad |= !(xs[e] < INFINITY);  // +inf or NaN
            hi = fmaxf(hi, xs[e]);
            lo = fminf(lo, xs[e] > -INFINITY ? xs[e] : INFINITY);
        }
    }
    uint32_t m1 = __reduce_max_sync(0xffffffffu, smp_key(hi)), m2 = __reduce_max_sync(0xffffffffu, ~smp_key(lo));
    uint32_t m3 = __any_sync(0xffffffffu, bad);
    if (row.lane == 0) sm.red[0][row.w] = m1, sm.red[1][row.w] = m2, sm.red[2][row.w] = m3;
    __syncthreads();
    for (int j = 0; j < SMP_WARPS; j++)
        m1 = max(m1, (uint32_t)sm.red[0][j]), m2 = max(m2, (uint32_t)sm.red[1][j]), m3 |= (uint32_t)sm.red[2][j];
    row.cl.barrier_wait();
    {
        const u64(*box)[SMP_MAX_CLUSTER] = row.exchange(m1, m2, m3, 0);
        for (int t = 0; t < C; t++)
            m1 = max(m1, (uint32_t)box[0][t]), m2 = max(m2, (uint32_t)box[1][t]), m3 |= (uint32_t)box[2][t];
    }
    const float top = row.top = smp_value(m1), bottom = smp_value(~m2);
    if (m3 || top == -INFINITY) {  // uniform over the cluster
        if (r == 0 && threadIdx.x == 0) {
            a.token[i_row] = -1;
            if (a.conf) a.conf[i_row] = 0.0f;
            if (a.entropy) a.entropy[i_row] = 0.0f;
            set_err(ERR_LOGITS);
        }
        return;
    }
    const double Td = greedy ? 1.0 : (double)T;
    const double min_p = mp > 0.0f ? fmin((double)mp, 1.0) : 0.0;
    row.scale = 1.4426950408889634 / Td;
    row.fix = a.fix;
    row.least = -(double)(a.fix + 2);
    row.min_w = min_p * (double)(1ull << a.fix);
    row.cut_val = -INFINITY;
    row.cut_idx = 0xffffffffu;

    // plain softmax: mass and first moment of the elements below the largest, and the
    // number equal to it (kept apart, so that a peaked row's small entropy stays exact)
    double s1 = 0.0, s2 = 0.0, s3 = 0.0;
    if (a.conf || a.entropy) {
        float e1 = 0.0f, e2 = 0.0f;
        uint32_t eq = 0;
        row.each([&](float l, int) {
            const float z = fmaxf(l - top, -200.0f);  // e^-200 is 0 in f32
            const float e = z < 0.0f ? exp2f(z * 1.4426950408889634f) : 0.0f;
            eq += z == 0.0f;
            e1 += e;
            e2 = fmaf(e, z, e2);
        });
        s1 = smp_warp_sum((double)e1);
        s2 = smp_warp_sum((double)e2);
        s3 = (double)__reduce_add_sync(0xffffffffu, eq);
    }

    // Limits.  min_p is part of the weight; a count limit needs masses only where a mass
    // limit follows it.
    const bool by_p = !(p >= 1.0f) && k != 1;
    const bool mass = by_p || min_p > 0.0;
    if (k > 0 || by_p) {
        // The bins need not reach below the values whose weight is 0 (with some room for the
        // rounding of either side).
        float floor_v = bottom;
        if (mass) {
            const double deep = fmin(-row.least * 0.6931471805599453, min_p > 0.0 ? -log(min_p) : INFINITY);
            floor_v = fmaxf(bottom, __double2float_rd((double)top - (deep * 1.000001 + 1e-12) * Td - fabs((double)top) * 1e-12));
        }
        row.histogram(floor_v, top, true, mass, 0, 0);
        u64 total = sm.before_m[SMP_COARSE];
        bool whole = true;
        if (k > 0 && (u64)k < sm.before_c[SMP_COARSE]) {
            whole = row.narrow(true, mass, (u64)k);
            total = sm.kept_mass;
        }
        if (by_p) {
            if (!whole) row.histogram(fmaxf(floor_v, row.cut_val), top, true, mass, 0, 0);
            // preceding mass < p S of whole numbers: preceding mass < ceil(p S); at least 1
            // keeps the first candidate
            const u64 limit = (u64)ceil((p > 0.0f ? (double)p : 0.0) * (double)total);
            row.narrow(false, mass, limit < 1 ? 1 : limit);
        }
    }

    // After this exchange no CTA reads or writes another's memory: they leave one by one.
    row.locate([&](float l, int i) -> u64 { return row.kept(l, i) ? row.weight(l) : 0; }, row.cut_val, 0, (double)u, s1, s2,
               s3, [&](float l, uint32_t at) {
                   a.token[i_row] = (int32_t)at;
                   if (a.conf) a.conf[i_row] = (float)(exp((double)l - (double)top) / (row.sums[0] + row.sums[2]));
               });
    if (a.entropy && r == 0 && threadIdx.x == 0)
        a.entropy[i_row] = (float)(log1p(row.sums[0] + (row.sums[2] - 1.0)) - row.sums[1] / (row.sums[0] + row.sums[2]));
}

}  // namespace dllm
