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
// bin it falls into.  Weights are fixed point, multiples of 2^-fix of the largest with fix =
// min(51, 62 - ceil(log2 V)) (45 at 2^17 words), from an f64 exponential: integer sums do not depend
// on their order, so atomics and any split over threads and CTAs give one result.  A border
// between two tokens is off by at most V 2^-(fix + 1) of the largest weight (2^-29 at 2^17 words, if a whole
// flat tail lies just below half a unit; ~2^-38 where the roundings fall to either side; f32 sums put
// 1 row in ~400 on the wrong side of one).  A word below half a unit weighs 0 and is not drawn.  Only
// u at its ends, which asks for the first or the last kept word, would show that, and only without
// top_p and min_p, which keep no such word: there every kept word weighs the same.
//
// One cluster of C CTAs per row.  Each CTA keeps its slice of the row in shared memory (read
// from HBM once); every step is one pass over the slices and one cluster barrier:
//   load and largest logit | plain softmax sums and histogram | gathering of the crossing
//   bin (one per limit) | kept mass of each warp's range.
// What a step exchanges is written into every CTA of the cluster and evaluated by all of them
// alike, so that no step waits for an answer.  A histogram is exchanged as 64 coarse sums;
// the 32 bins behind the crossing one are then read from the other CTAs.
// Few candidates (up to 256 up to the end of a limit's bin, as min_p, top_k and peaked rows leave)
// are gathered in one CTA, which ranks them and takes the token from them.
// Bound: the logits' bytes; in practice the chain of passes and barriers (~26,000 cycles per
// CTA where few candidates are left, two CTAs per SM) and, for flat rows, the weights: ~40
// instructions an element, a third of them f64, on pipes that take one every other cycle, and two
// to three shared-memory atomics of 4-5 cycles each.
//
// Measured (one B200): 1 row of 152064 words with all limits 11.3-12.3 us; 32 rows of 126464 with
// top_p 51 us; 256 rows with all limits 124-127 us (1.03 TB/s).  Steps on the way: f64 exponentials of the math
// library, a histogram per limit, 1024 threads 60 / 139 / 934 us; one histogram for both limits,
// two CTAs per SM 39 / 79 / 385; weights by table 22 / 52 / 221; bulk copies and the list of few
// candidates 15.5 / 62 / 177; 256 threads at 128 registers 14.4 / 60 / 158; coarse sums by vector
// loads, lists gathered per CTA 12.0 / 55 / 137; vectors passed over whole 11.1 / 57 / 124; bins of
// top_p alone no lower than its cut can be 11.3 / 51 / 126.
#pragma once
#include <cooperative_groups.h>

#include <cfloat>

#include "attention.cuh"

namespace dllm {

constexpr int SMP_THREADS = 256;
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
    // All CTAs' elements of a gathered bin, order code and weight.  This CTA alone writes it, and may still
    // rank one limit's bin in it while another CTA has gone on to the next limit.
    ulonglong2 list[SMP_LIST];
    // CTA 0's: the order codes of few candidates, written once per row by every CTA that has some, and read
    // behind the cluster barrier that follows.  Not `list`: no barrier lies between the ranking of top_k's
    // bin and these writes.
    u64 sent[SMP_LIST];
    uint32_t cnt[SMP_BINS], lo[SMP_BINS], hi[SMP_BINS];  // this CTA's histogram: count, mass
    uint32_t ccnt[SMP_MAX_CLUSTER][SMP_COARSE];          // every CTA's coarse sums
    u64 cmass[SMP_MAX_CLUSTER][SMP_COARSE];
    u64 before_c[SMP_COARSE + 1], before_m[SMP_COARSE + 1];  // the cluster's, before each coarse bin
    u64 mine[2][SMP_LIST];                               // this CTA's elements of a gathered bin: order codes
    u64 box[2][4][SMP_MAX_CLUSTER];                      // one exchange: words of every CTA
    u64 plain[3][SMP_MAX_CLUSTER];                       // every CTA's sums of the plain softmax
    u64 red[4][SMP_WARPS];
    u64 found[2], kept_mass;  // crossing bin: count before, mass before; mass up to the cut
    double table[SMP_TABLE];  // 2^(fix + i / 256)
    uint32_t found_bin, found_upto, n_mine[2], n_list, best;
    u64 cut;                  // order code
    uint64_t landed;          // mbarrier: the slice is in shared memory
    double scale, ln_min_p;   // log2(e) / T (or 0: all weigh alike), ln(min_p)
};

static_assert(sizeof(SampleShared) % 16 == 0, "the slice behind it is read as float4");

// Order-preserving code of a float (-0 counts as +0): larger value, larger code.
__device__ __forceinline__ uint32_t smp_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float smp_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The largest of three; NaN if one is.
__device__ __forceinline__ float smp_max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
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

__device__ __forceinline__ SampleShared& smp_shared() {
    extern __shared__ __align__(1024) uint8_t smem[];
    return *reinterpret_cast<SampleShared*>(smem);
}
__device__ __forceinline__ float* smp_cache() {
    extern __shared__ __align__(1024) uint8_t smem[];
    return reinterpret_cast<float*>(smem + sizeof(SampleShared));
}

// One row, as one CTA of its cluster sees it.
struct SampleRow {
    cooperative_groups::cluster_group cl;
    const float* src;   // row in global memory
    int64_t V;
    int C, r, w, lane;  // CTAs, this one's rank; warp, lane
    int n, cached;      // elements of the slice (a multiple of 4), and of them in shared memory
    int64_t first;      // row index of the slice's first element (before the row: filled with -inf)
    float top;          // largest logit
    double topd, scale; // it widened; log2(e) / T
    float lowest;       // weighs less than half a unit, or is the lowest float
    bool coarse;
    double floor_t;     // base-2 exponent that rounds to weight 0
    u64 min_w;          // min_p in fixed point
    float cut_val;      // kept: above, or equal and not behind cut_i
    int cut_i;
    int phase;          // which box comes next
    // the present histogram: values [vmin, vmax], spread evenly by value or by code
    float vmin, vmax, vhi, inv;
    float low_val;      // the higher of vmin and the cut
    int low_i;
    int shift;
    bool linear;

    // Four elements; outside the row -inf.
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
        return x;
    }
    // f(x, i) for the elements lo + 4 k .. lo + 4 k + 3 of [lo, hi), k = first thread, + step ...;
    // two loads are in flight.
    template <typename F>
    __device__ __forceinline__ void each(int lo, int hi, int thread, int threads, F f) const {
        const float* const cache = smp_cache();
        const int step = 4 * threads, end = min(hi, cached);
        int i = lo + 4 * thread;
        for (; i + step < end; i += 2 * step) {
            const float4 x = *reinterpret_cast<const float4*>(cache + i);
            const float4 y = *reinterpret_cast<const float4*>(cache + i + step);
            f(x, i);
            f(y, i + step);
        }
        for (; i < end; i += step) f(*reinterpret_cast<const float4*>(cache + i), i);
        for (; i < hi; i += step) f(load4(i), i);
    }
    __device__ __forceinline__ uint32_t index(int i) const { return (uint32_t)first + (uint32_t)i; }

    // Fixed-point weight of a logit: 2^t by table and polynomial (Tang 1989), t = k + j / 256 + f,
    // |f| <= 2^-9, the polynomial's next term below 2^-54.  Adding 1.5 2^44 rounds t to a
    // multiple of 1/256 and leaves 256 k + j in the low word; adding 2^52 to the weight (the
    // table holds 2^(fix + j / 256)) rounds it to a whole number, held by the low mantissa.
    __device__ __forceinline__ u64 weight_of(double t) const {
        const double tm = t + 26388279066624.0;
        const int kj = __double2loint(tm);
        const double f = t - (tm - 26388279066624.0);
        const double b = smp_shared().table[kj & 255];
        double q = fma(f, 0.009618129107628477, 0.05550410866482158);
        q = fma(f, q, 0.2402265069591007);
        q = fma(f, q, 0.6931471805599453);
        const double e = fma(b * f, q, b);
        const double g = __hiloint2double(__double2hiint(e) + ((kj & ~255) << 12), __double2loint(e));
        return __double_as_longlong(g + 4503599627370496.0) & 0xfffffffffffffull;
    }
    // f32 -> f64 with integer operations, as the conversion unit has an eighth of their rate: a
    // zero or denormal value comes out up to 2^-126 off.
    __device__ static __forceinline__ double widen(float x) {
        const int b = __float_as_int(x);
        return __hiloint2double(((b >> 3) & 0x8fffffff) + 0x38000000, b << 29);
    }
    // The weights of four elements together, so that their chains overlap; 0 below min_p and
    // where not ok (-inf never is).  What lies below `lowest` has weight 0 and is raised to
    // it.  A row whose T could tell widen's error, or is so small that nothing lies between the
    // top and weight 0, goes the plain way (coarse).
    __device__ __forceinline__ void weight4(const float (&l)[4], const bool (&ok)[4], u64 (&v)[4]) const {
        double t[4];
        if (!coarse) {  // uniform
#pragma unroll
            for (int e = 0; e < 4; e++) t[e] = (widen(fmaxf(l[e], lowest)) - topd) * scale;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                t[e] = ((double)l[e] - (double)top) * scale;
                t[e] = t[e] > floor_t ? t[e] : floor_t;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = weight_of(t[e]);
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = ok[e] ? v[e] : 0;
        if (min_w != 0) {  // uniform
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = v[e] >= min_w ? v[e] : 0;
        }
    }
    __device__ __forceinline__ u64 weight1(float l) const {
        const double t = coarse ? fmax(((double)l - (double)top) * scale, floor_t)
                                : (widen(fmaxf(l, lowest)) - topd) * scale;
        const u64 v = weight_of(t);
        return v >= min_w ? v : 0;
    }
    // Above the cut; i counts from the slice's first element.
    __device__ __forceinline__ bool kept(float l, int i) const { return l > cut_val || (l == cut_val && i <= cut_i); }
    __device__ __forceinline__ bool in_range(float l, int i) const {
        return (l > low_val || (l == low_val && i <= low_i)) && l <= vmax;
    }
    // (a value below 2^23 plus 2^23 holds the nearest whole number in its low bits)
    __device__ __forceinline__ int bin_of(float l) const {
        return linear ? min(SMP_BINS - 1, __float_as_int(fmaf(fmaf(-0.25f, l, vhi), inv, 8388608.0f)) - 0x4b000000)
                      : (int)((smp_key(vmax) - smp_key(l)) >> shift);
    }
    // Moves the cut to the element of an order code.
    __device__ __forceinline__ void cut_at(u64 code) {
        cut_val = smp_value((uint32_t)(code >> 32));
        const int64_t i = (int64_t)(uint32_t)~(uint32_t)code - first;
        cut_i = i > INT_MAX ? INT_MAX : i < 0 ? -1 : (int)i;
    }

    // Exchange of four words per CTA (those of thread t < C, alike in all of them); after it
    // every CTA holds all of them in the returned box.  Boxes alternate: a CTA may write the
    // next exchange while another still reads this one.
    __device__ __forceinline__ const u64 (*exchange(u64 a, u64 b, u64 c, u64 d))[SMP_MAX_CLUSTER] {
        u64(*box)[SMP_MAX_CLUSTER] = smp_shared().box[phase++ & 1];
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
    // By value and with masses the bins may begin at `bins`, above lo: the last has all from lo to there.
    __device__ __forceinline__ void histogram(float lo, float hi, float bins, bool by_value, bool clear, bool mass, u64 c0, u64 m0) {
        SampleShared& sm = smp_shared();
        vmin = lo;
        vmax = hi;
        low_val = fmaxf(lo, cut_val);
        low_i = lo > cut_val ? INT_MAX : cut_i;
        vhi = 0.25f * hi;
        const float span = vhi - 0.25f * bins;
        inv = (float)SMP_BINS / span;
        shift = max(0, 32 - __clz(smp_key(hi) - smp_key(lo)) - 11);
        linear = by_value && span > 0.0f && inv < 1e30f;
        if (!linear) bins = lo;
        const bool uncut = by_value && low_i == INT_MAX;  // every value from lo up is a candidate
        if (clear) {
            for (int i = threadIdx.x; i < SMP_BINS; i += SMP_THREADS) sm.cnt[i] = sm.lo[i] = sm.hi[i] = 0;
            __syncthreads();
        }
        u64 below = 0;  // mass and number of what lies below the bins: summed here, not by atomics on one bin
        uint32_t n_below = 0;
        each(0, n, threadIdx.x, SMP_THREADS, [&](const float4& x, int i) {
            const float l[4] = {x.x, x.y, x.z, x.w};
            if (!(fmaxf(max3f(l[0], l[1], l[2]), l[3]) >= low_val)) return;
            bool ok[4];
#pragma unroll
            for (int e = 0; e < 4; e++) ok[e] = uncut ? l[e] >= lo : in_range(l[e], i + e);
            u64 v[4];
            const bool any4[4] = {true, true, true, true};  // what is not ok is left out below
            if (mass) weight4(l, any4, v);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                // a weight of 0: no candidate, or one that no mass limit can tell apart
                if (!ok[e] || (mass && v[e] == 0)) continue;
                if (l[e] < bins) {
                    below += v[e];
                    n_below++;
                    continue;
                }
                const int b = bin_of(l[e]);
                if (mass) {  // two 32-bit adds: a 64-bit one is a compare-and-swap loop
                    const uint32_t wl = (uint32_t)v[e], old = atomicAdd(&sm.lo[b], wl);
                    const uint32_t wh = (uint32_t)(v[e] >> 32) + (old + wl < old ? 1u : 0u);
                    if (wh) atomicAdd(&sm.hi[b], wh);
                }
                atomicAdd(&sm.cnt[b], 1u);
            }
        });
        if (bins > lo) {  // uniform
            below = smp_warp_sum(below);
            n_below = __reduce_add_sync(0xffffffffu, n_below);
            if (lane == 0 && n_below) {
                const uint32_t bl = (uint32_t)below, old = atomicAdd(&sm.lo[SMP_BINS - 1], bl);
                atomicAdd(&sm.hi[SMP_BINS - 1], (uint32_t)(below >> 32) + (old + bl < old ? 1u : 0u));
                atomicAdd(&sm.cnt[SMP_BINS - 1], n_below);
            }
        }
        __syncthreads();
        // Coarse sums: eight bins per thread, four threads' together, written by those into every CTA.
        static_assert(SMP_BINS == 8 * SMP_THREADS, "bins per thread");
        uint32_t c = 0;
        u64 m = 0;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int b = 8 * (int)threadIdx.x + 4 * h;
            const uint4 y = *reinterpret_cast<const uint4*>(&sm.cnt[b]);
            c += (y.x + y.y) + (y.z + y.w);
            if (mass) {
                const uint4 a = *reinterpret_cast<const uint4*>(&sm.lo[b]), d = *reinterpret_cast<const uint4*>(&sm.hi[b]);
                m += ((u64)((d.x + d.y) + (d.z + d.w)) << 32) + (((u64)a.x + a.y) + ((u64)a.z + a.w));
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            c += __shfl_xor_sync(0xffffffffu, c, o);
            m += __shfl_xor_sync(0xffffffffu, m, o);
        }
        for (int t = lane & 3; t < C; t += 4) {
            const int cb = (int)threadIdx.x >> 2;
            *cl.map_shared_rank(&sm.ccnt[r][cb], t) = c;
            *cl.map_shared_rank(&sm.cmass[r][cb], t) = m;
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

    // The crossing bin of the present histogram, the first with count (mass) up to its end
    // >= limit: into sm.found.  Warp 0 of every CTA.
    __device__ __forceinline__ void cross(bool by_count, u64 limit) {
        SampleShared& sm = smp_shared();
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
            sm.found_upto = (uint32_t)min(ec + c, (u64)0xffffffffu);
            sm.found[0] = ec;
            sm.found[1] = em;
        }
    }
};

// Grid (C * rows), clusters of C.
__global__ void __launch_bounds__(SMP_THREADS, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    SampleShared& sm = smp_shared();
    SampleRow row{cooperative_groups::this_cluster()};
    cooperative_groups::cluster_group& cl = row.cl;
    const int C = row.C = (int)cl.num_blocks(), r = row.r = (int)cl.block_rank();
    const int64_t i_row = blockIdx.x / C;
    const int w = row.w = threadIdx.x >> 5, lane = row.lane = threadIdx.x & 31;
    row.phase = 0;
    cl.barrier_arrive();  // every CTA has started before another writes into it (waited for below)
    if (threadIdx.x == 0) {
        mbar_init(&sm.landed, 1);
        fence_mbar_init();
        sm.n_list = 0;
    }
    pdl_trigger();
    pdl_wait();

    // Slices start on 16-byte boundaries of global memory, whatever the row's address: the
    // first one begins up to three elements before the row.
    row.src = a.logits + i_row * a.ldl;
    row.V = a.V;
    row.first = (int64_t)r * a.slice - (int64_t)(reinterpret_cast<uintptr_t>(row.src) >> 2 & 3);
    const int64_t left = a.V - row.first;
    const int n = row.n = (int)(left < a.slice ? max((int64_t)0, (left + 3) & ~(int64_t)3) : a.slice);
    row.cached = min(n, a.cached);

    const float T = a.temperature ? __ldg(a.temperature + i_row) : 1.0f;
    const bool greedy = !(T > 0.0f);
    const double Td = greedy ? 1.0 : (double)T;
    const float mp = a.min_p ? __ldg(a.min_p + i_row) : 0.0f;
    const double min_p = mp > 0.0f ? fmin((double)mp, 1.0) : 0.0;
    const float p = a.top_p ? __ldg(a.top_p + i_row) : 1.0f;
    const int32_t k = greedy ? 1 : a.top_k ? __ldg(a.top_k + i_row) : 0;
    float u = a.u ? __ldg(a.u + i_row) : 0.0f;
    u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;  // NaN counts as 0

    // The slice into shared memory: what the row fills of its 16-byte vectors by bulk copies of
    // eight lanes, the vectors at the row's ends by two threads; meanwhile the table, the
    // cleared histogram and what depends on the row's parameters.
    if (w == 0) {
        const int i0 = row.first < 0 ? 4 : 0;
        const int i1 = max(i0, min(row.cached, (int)min((int64_t)n, left & ~(int64_t)3)));
        const int part = ((i1 - i0) / 8 + 3) & ~3;
        const int from = min(i1, i0 + lane * part), to = lane == 7 ? i1 : min(i1, from + part);
        if (lane == 0) mbar_arrive_expect_tx(&sm.landed, (uint32_t)(i1 - i0) * 4);
        __syncwarp();
        if (lane < 8 && to > from)
            bulk_g2s_hint(smp_cache() + from, row.src + row.first + from, (uint32_t)(to - from) * 4, &sm.landed,
                          policy_evict_first());
        const int edge = lane == 8 && i0 > 0 ? 0 : lane == 9 && i1 < row.cached && i1 >= i0 ? i1 : -1;
        if (edge >= 0 && edge < row.cached) *reinterpret_cast<float4*>(smp_cache() + edge) = row.load4(edge);
    } else if (w == 1 && lane == 0) {
        // The first or the last kept word without a mass limit: all weigh alike, however unlikely.
        const bool ends = (u == 0.0f || u == 1.0f) && (p >= 1.0f || k == 1) && min_p == 0.0;
        sm.scale = ends ? 0.0 : 1.4426950408889634 / Td;
        sm.ln_min_p = min_p > 0.0 ? log(min_p) : 0.0;
    }
    static_assert(SMP_TABLE == SMP_THREADS, "one entry per thread");
    sm.table[threadIdx.x] = exp2((double)threadIdx.x / SMP_TABLE + a.fix);
    for (int i = threadIdx.x; i < SMP_BINS; i += SMP_THREADS) sm.cnt[i] = sm.lo[i] = sm.hi[i] = 0;
    __syncthreads();  // the barrier and the edges are there
    bool bad = false;
    {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&sm.landed, 0))
            if (globaltimer_ns() - t0 > 2000000000ull) {
                set_err(ERR_TIMEOUT);
                bad = true;  // the whole cluster leaves: nothing is sampled from a slice that may still change
                break;
            }
    }

    // the row's largest and smallest finite logit
    float hi = -INFINITY, lo = INFINITY;
    row.each(0, n, threadIdx.x, SMP_THREADS, [&](const float4& x, int) {
        const float xs[4] = {x.x, x.y, x.z, x.w};
        hi = smp_max3(smp_max3(hi, x.x, x.y), x.z, x.w);
#pragma unroll
        for (int e = 0; e < 4; e++) lo = fminf(lo, xs[e] > -INFINITY ? xs[e] : INFINITY);
    });
    bad |= !(hi < INFINITY);  // +inf or NaN
    uint32_t m1 = __reduce_max_sync(0xffffffffu, smp_key(hi)), m2 = __reduce_max_sync(0xffffffffu, ~smp_key(lo));
    uint32_t m3 = __any_sync(0xffffffffu, bad);
    if (lane == 0) sm.red[0][w] = m1, sm.red[1][w] = m2, sm.red[2][w] = m3;
    __syncthreads();
    auto max_of = [&](const u64* v, int count) {
        return __reduce_max_sync(0xffffffffu, lane < count ? (uint32_t)v[lane] : 0u);
    };
    if (w == 0) m1 = max_of(sm.red[0], SMP_WARPS), m2 = max_of(sm.red[1], SMP_WARPS), m3 = max_of(sm.red[2], SMP_WARPS);
    cl.barrier_wait();
    {
        const u64(*box)[SMP_MAX_CLUSTER] = row.exchange(m1, m2, m3, 0);
        m1 = max_of(box[0], C), m2 = max_of(box[1], C), m3 = max_of(box[2], C);
    }
    const float top = row.top = smp_value(m1);
    const float bottom = smp_value(~m2);
    if (m3 || top == -INFINITY) {  // uniform over the cluster
        if (r == 0 && threadIdx.x == 0) {
            a.token[i_row] = -1;
            if (a.conf) a.conf[i_row] = 0.0f;
            if (a.entropy) a.entropy[i_row] = 0.0f;
            set_err(ERR_LOGITS);
        }
        if (threadIdx.x == 0) drain_wait(&sm.landed, 0);  // no copy may land after the CTA's exit
        return;
    }
    row.scale = sm.scale;
    row.min_w = __double2ull_rn(min_p * (double)(1ull << a.fix));
    row.floor_t = -(double)(a.fix + 2);
    // 2^-(fix + 1.5) of the top, rounded down (and by a hair more than its own rounding)
    const double deep = (a.fix + 1.5) * 0.6931471805599453, hair = fabs((double)top) * 1e-12;
    row.lowest = fmaxf(-FLT_MAX, __double2float_rd((double)top - deep * 1.000001 * Td - hair));
    row.coarse = Td < 1e-18 || ((double)top - (double)row.lowest) * row.scale > 1000.0;
    row.topd = SampleRow::widen(top);
    row.cut_val = bottom;  // everything finite
    row.cut_i = INT_MAX;

    // plain softmax: mass and first moment of the elements below the largest, and the
    // number equal to it (kept apart, so that a peaked row's small entropy stays exact).  f32 within a thread
    // (V / (256 C) terms, off by 5e-8 of conf and entropy in all at 2^17 words), f64 from there on: f64
    // sums here would add two of the slow operations per element for figures that are rounded to f32.
    double s1 = 0.0, s2 = 0.0, s3 = 0.0;
    if (a.conf || a.entropy) {
        float e1 = 0.0f, e2 = 0.0f;
        uint32_t eq = 0;
        row.each(0, n, threadIdx.x, SMP_THREADS, [&](const float4& x, int) {
            const float l[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float z = fmaxf(l[j] - top, -200.0f);  // e^-200 is 0 in f32
                const float e = z < 0.0f ? att_ex2(z * 1.4426950408889634f) : 0.0f;
                eq += z == 0.0f;
                e1 += e;
                e2 = fmaf(e, z, e2);
            }
        });
        s1 = smp_warp_sum((double)e1);
        s2 = smp_warp_sum((double)e2);
        s3 = (double)__reduce_add_sync(0xffffffffu, eq);
    }

    // Every CTA has all of them after the next cluster barrier.
    {
        if (lane == 0) {
            sm.red[1][w] = __double_as_longlong(s1);
            sm.red[2][w] = __double_as_longlong(s2);
            sm.red[3][w] = __double_as_longlong(s3);
        }
        __syncthreads();
        if (w < 3) {
            const u64 sum =
                __double_as_longlong(smp_warp_sum(lane < SMP_WARPS ? __longlong_as_double(sm.red[1 + w][lane]) : 0.0));
            if (lane < C) *cl.map_shared_rank(&sm.plain[w][r], lane) = sum;
        }
    }
    auto plain_sum = [&](int which) {
        double x = 0.0;
        for (int t = 0; t < C; t++) x += __longlong_as_double(sm.plain[which][t]);
        return x;
    };
    // The token (one thread of the row), and the row's entropy with it.
    auto report = [&](float l, uint32_t at) {
        const double below = plain_sum(0), others = plain_sum(2) - 1.0, all = (1.0 + others) + below;
        a.token[i_row] = (int32_t)at;
        if (a.conf) a.conf[i_row] = (float)(exp((double)l - (double)top) / all);
        if (a.entropy) a.entropy[i_row] = (float)(log1p(others + below) - plain_sum(1) / all);
    };

    // Stage 0: top_k; stage 1: top_p; stage 2: the token.  min_p is part of the weight; a count
    // limit needs masses only where min_p or a mass limit follows it, or the list below ends it.
    const bool by_p = !(p >= 1.0f) && k != 1;
    const bool mass = by_p || min_p > 0.0;
    // Where all weigh alike, nothing is kept that has no weight in 64 bits either (2^-1075).
    if (!mass && sm.scale == 0.0) row.cut_val = fmaxf(bottom, __double2float_rd((double)top - 745.1332191019412 * Td));
    bool have = false, clear = false;  // the histogram over all candidates is there; must be cleared first
    bool cut_mass = false;
    int half = 0;       // which list comes next
#pragma unroll 1
    for (int stage = 0; stage < 3; stage++) {
        const bool by_count = stage == 0;
        bool tie = false;
        float tie_val = 0.0f;
        u64 target = 0, tie_mass = 0;
        if (stage < 2) {
            if (!(by_count ? k > 0 : by_p)) continue;
            float from = row.cut_val, to = top;
            if (mass) {
                // no bins for values whose weight is 0 (with some room for either side's rounding)
                from = fmaxf(from, row.lowest);
                if (min_p > 0.0)
                    from = fmaxf(from, __double2float_rd((double)top - (-sm.ln_min_p * 1.000001 + 1e-12) * Td - hair));
            }
            // The cut and what follows it hold more than (1 - p) of the mass, which is at least the
            // largest weight, 1, and none of them weighs more than the cut: it weighs more than
            // (1 - p) / V, so the bins need not reach below that (with some room for rounding).
            float bins = from;
            if (!by_count && k <= 0 && p > 0.0f)
                bins = fmaxf(from, __double2float_rd((double)top + (log((1.0 - (double)p) / (double)a.V) - 0.01) * Td - hair));
            u64 c0 = 0, m0 = 0, limit = 0;
            bool whole = true, done = false;
#pragma unroll 1
            while (!done) {
                if (!have) row.histogram(from, to, whole ? bins : from, whole, clear, mass, c0, m0);
                have = clear = true;
                int bin = SMP_BINS - 1;
                uint32_t upto = 0;
                bool all = false;  // no limit is reached
                if (whole) {
                    const u64 candidates = sm.before_c[SMP_COARSE];
                    if (by_count) {
                        limit = (u64)k;
                        all = limit >= candidates;
                    } else {
                        // preceding mass < p S of whole numbers: preceding mass < ceil(p S); at
                        // least 1 keeps the first candidate
                        const u64 S = cut_mass ? sm.kept_mass : sm.before_m[SMP_COARSE];
                        limit = (u64)ceil((p > 0.0f ? (double)p : 0.0) * (double)S);
                        if (limit < 1) limit = 1;
                    }
                    upto = (uint32_t)min(candidates, (u64)0xffffffffu);
                    if (all && upto > SMP_LIST) break;
                }
                if (w == 0) {
                    if (!all) row.cross(by_count, limit);
                    if (lane == 0) sm.best = 0, sm.n_mine[half] = 0;
                }
                __syncthreads();
                if (!all) {
                    bin = (int)sm.found_bin;
                    upto = sm.found_upto;
                    c0 = sm.found[0];
                    m0 = sm.found[1];
                }
                // The bin's edges, with a hundredth of a bin for the rounding of bin_of and a
                // few units in the last place for their own; the last bin reaches down.
                const float slack = 4e-6f * fabsf(row.vhi);
                const float under = !row.linear               ? row.vmin
                                    : bin == SMP_BINS - 1 ? -INFINITY
                                                          : 4.0f * (row.vhi - ((float)bin + 0.51f) / row.inv) - slack;
                if (whole && upto <= SMP_LIST) {
                    // Few candidates up to the end of the crossing bin (any cut of an earlier
                    // stage included): CTA 0 ranks them all and takes the token from them.  They
                    // are gathered here first, so that each CTA asks for its place once.
                    const float least = fmaxf(row.low_val, under);
                    row.each(0, n, threadIdx.x, SMP_THREADS, [&](const float4& x, int i) {
                        const float l[4] = {x.x, x.y, x.z, x.w};
                        if (!(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= least)) return;
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (l[e] >= least && row.in_range(l[e], i + e) && row.kept(l[e], i + e) && row.bin_of(l[e]) <= bin) {
                                if (mass && row.weight1(l[e]) == 0) continue;
                                const uint32_t slot = atomicAdd(&sm.n_mine[half], 1u);
                                if (slot < SMP_LIST)
                                    sm.mine[half][slot] = ((u64)smp_key(l[e]) << 32) | (uint32_t)~row.index(i + e);
                            }
                    });
                    __syncthreads();
                    const uint32_t count = min(sm.n_mine[half], (uint32_t)SMP_LIST);
                    if (w * 32 < (int)count) {
                        SampleShared* o = cl.map_shared_rank(&sm, 0);
                        const uint32_t of_warp = min(count - 32 * w, 32u);
                        uint32_t slot = 0;
                        if (lane == 0) slot = atomicAdd(&o->n_list, of_warp);
                        slot = __shfl_sync(0xffffffffu, slot, 0) + lane;
                        if (lane < (int)of_warp && slot < SMP_LIST) o->sent[slot] = sm.mine[half][threadIdx.x];
                    }
                    cl.sync();
                    if (r != 0) return;  // nothing of this CTA's memory is read from here on
                    const int m = (int)min(sm.n_list, (uint32_t)SMP_LIST), e = (int)threadIdx.x;
                    const u64 code = e < m ? sm.sent[e] : 0;
                    const float l = smp_value((uint32_t)(code >> 32));
                    u64 weight = e < m ? row.weight1(l) : 0;
                    if (e < m) sm.list[e].x = code, sm.list[e].y = weight;
                    __syncthreads();
                    uint32_t rank = 0;
                    u64 pre = 0;
                    if (e < m) {
#pragma unroll 4
                        for (int j = 0; j < m; j++) {
                            const ulonglong2 y = sm.list[j];
                            rank += y.x > code;
                            pre += y.x > code ? y.y : 0;
                        }
                    }
                    auto block_sum = [&](u64 y) {
                        y = smp_warp_sum(y);
                        __syncthreads();
                        if (lane == 0) sm.red[0][w] = y;
                        __syncthreads();
                        return smp_warp_sum(lane < SMP_WARPS ? sm.red[0][lane] : 0ull);
                    };
                    bool in = e < m && (!by_count || rank < (uint32_t)k);
                    if (by_count && by_p) {
                        const u64 S = block_sum(in ? weight : 0);
                        limit = (u64)ceil((p > 0.0f ? (double)p : 0.0) * (double)S);
                        if (limit < 1) limit = 1;
                    }
                    in = in && (!by_p || pre < limit);
                    if (!in) weight = 0;
                    __syncthreads();
                    if (e < m) sm.list[e].y = weight;
                    const u64 total = block_sum(weight);
                    target = (u64)((double)u * (double)total);
                    if (target >= total) target = total - 1;
                    if (in) {
                        u64 run = 0;
                        const uint32_t at = (uint32_t)code;  // complement of the index
#pragma unroll 4
                        for (int j = 0; j < m; j++) {
                            const ulonglong2 y = sm.list[j];
                            run += (uint32_t)y.x > at ? y.y : 0;
                        }
                        if (run <= target && target - run < weight) report(l, ~at);
                    }
                    return;
                }
                const float over = row.linear ? 4.0f * (row.vhi - ((float)bin - 0.51f) / row.inv) + slack : row.vmax;
                uint32_t k_hi = 0, k_lo = 0;  // largest code of the bin, largest complement
                row.each(0, n, threadIdx.x, SMP_THREADS, [&](const float4& x, int i) {
                    const float l[4] = {x.x, x.y, x.z, x.w};
                    bool ok[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) ok[e] = l[e] <= over && l[e] >= under;
                    if (!(ok[0] | ok[1] | ok[2] | ok[3])) return;
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (ok[e] && row.in_range(l[e], i + e) && row.bin_of(l[e]) == bin) {
                            const uint32_t key = smp_key(l[e]), slot = atomicAdd(&sm.n_mine[half], 1u);
                            k_hi = max(k_hi, key);
                            k_lo = max(k_lo, ~key);
                            if (slot < SMP_LIST) sm.mine[half][slot] = ((u64)key << 32) | (uint32_t)~row.index(i + e);
                        }
                });
                cl.sync();  // also: every CTA has read the bins
                const int n_of = lane < C ? (int)*cl.map_shared_rank(&sm.n_mine[half], lane) : 0;
                const int e = (int)threadIdx.x;
                int m = 0, source = 0, slot = 0;
#pragma unroll 1
                for (int t = 0; t < C; t++) {
                    const int c = __shfl_sync(0xffffffffu, n_of, t);
                    if (e >= m && e < m + c) source = t, slot = e - m;
                    m += c;
                }
                done = m <= SMP_LIST;
                if (done) {
                    // each gathered element's rank: the last one kept is the cut
                    u64 code = 0;
                    if ((int)threadIdx.x < m) {
                        code = cl.map_shared_rank(&sm, source)->mine[half][slot];
                        sm.list[e].x = code;
                        sm.list[e].y = mass ? row.weight1(smp_value((uint32_t)(code >> 32))) : 0;
                    }
                    __syncthreads();
                    uint32_t rank = 0;
                    u64 pre = m0;
                    bool in = false;
                    if ((int)threadIdx.x < m) {
#pragma unroll 4
                        for (int j = 0; j < m; j++) {
                            const ulonglong2 y = sm.list[j];
                            rank += y.x > code;
                            pre += y.x > code ? y.y : 0;
                        }
                        // what weighs nothing is no candidate where masses count
                        in = (by_count ? c0 + rank : pre) < limit && (!mass || sm.list[e].y != 0);
                    }
                    const uint32_t last = __reduce_max_sync(0xffffffffu, in ? rank + 1 : 0);
                    if (lane == 0 && last) atomicMax(&sm.best, last);
                    __syncthreads();
                    if (in && rank + 1 == sm.best) sm.cut = code, sm.kept_mass = pre + sm.list[e].y;
                    __syncthreads();
                    row.cut_at(sm.cut);
                    cut_mass = true;
                } else {
                    // too many to rank: the range of codes the bin really spans, or its ties
                    k_hi = __reduce_max_sync(0xffffffffu, k_hi);
                    k_lo = __reduce_max_sync(0xffffffffu, k_lo);
                    if (lane == 0) sm.red[0][w] = k_hi, sm.red[1][w] = k_lo;
                    __syncthreads();
                    if (w == 0) k_hi = max_of(sm.red[0], SMP_WARPS), k_lo = max_of(sm.red[1], SMP_WARPS);
                    const u64(*box)[SMP_MAX_CLUSTER] = row.exchange(k_hi, k_lo, 0, 0);
                    k_hi = max_of(box[0], C), k_lo = ~max_of(box[1], C);
                    from = smp_value(k_lo);
                    to = smp_value(k_hi);
                    whole = have = false;
                    if (k_hi == k_lo) {  // all equal: the first ones in index order
                        const u64 wt = mass ? row.weight1(to) : 0;
                        target = by_count ? limit - c0 : (limit - m0 + wt - 1) / wt;  // before = m0 + j wt < limit
                        tie_mass = m0 + target * wt;
                        target -= 1;
                        tie_val = to;
                        tie = done = true;
                    }
                }
                half ^= 1;  // another CTA may still read this list
            }
            if (!whole) have = false;
            if (!tie) continue;
        }

        // The first element, in index order, whose running sum of weights (ties: of ones) exceeds
        // the target; for the token, min(floor(u * sum), sum - 1).
        const float under = tie ? tie_val : row.cut_val;
        auto weigh = [&](const float4& x, int i, u64 (&v)[4]) {
            const float l[4] = {x.x, x.y, x.z, x.w};
            bool ok[4];
#pragma unroll
            for (int e = 0; e < 4; e++) ok[e] = row.kept(l[e], i + e);
            if (tie) {
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = ok[e] && l[e] == tie_val ? 1 : 0;
            } else {
                row.weight4(l, ok, v);
            }
        };
        const int per = ((n + SMP_WARPS - 1) / SMP_WARPS + 3) & ~3;  // a warp's contiguous share
        u64 s = 0;
        row.each(min(n, w * per), min(n, w * per + per), lane, 32, [&](const float4& x, int i) {
            if (!(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) >= under)) return;
            u64 v[4];
            weigh(x, i, v);
            s += (v[0] + v[1]) + (v[2] + v[3]);
        });
        s = smp_warp_sum(s);
        __syncthreads();
        if (lane == 0) sm.red[0][w] = s;
        __syncthreads();
        const u64 mine = smp_warp_sum(lane < SMP_WARPS ? sm.red[0][lane] : 0ull);
        const u64(*box)[SMP_MAX_CLUSTER] = row.exchange(mine, 0, 0, 0);
        const u64 of = lane < C ? box[0][lane] : 0;
        const u64 total = smp_warp_sum(of), before = smp_warp_sum(lane < r ? of : 0);
        if (!tie) {
            target = (u64)((double)u * (double)total);
            if (target >= total) target = total - 1;
        }
        if (target >= before && target - before < mine) {  // in this CTA's slice (uniform)
            u64 run = before;
            int wi = 0;
            while (wi < SMP_WARPS - 1 && run + sm.red[0][wi] <= target) run += sm.red[0][wi++];
            const int from = min(n, wi * per), to = min(n, from + per);
            for (int i0 = from; i0 < to; i0 += 4 * SMP_THREADS) {
                const int i = i0 + 4 * (int)threadIdx.x;
                u64 v[4] = {0, 0, 0, 0};
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i < to) {
                    x = i < row.cached ? *reinterpret_cast<const float4*>(smp_cache() + i) : row.load4(i);
                    weigh(x, i, v);
                }
                const u64 sum = (v[0] + v[1]) + (v[2] + v[3]);
                const u64 inc = smp_warp_scan(sum, lane);
                __syncthreads();
                if (lane == 31) sm.red[1][w] = inc;
                __syncthreads();
                const u64 y = lane < SMP_WARPS ? sm.red[1][lane] : 0;
                u64 upto = run + inc - sum + smp_warp_sum(lane < w ? y : 0);
                run += smp_warp_sum(y);
                const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if (v[e] != 0 && upto <= target && upto + v[e] > target) {  // one thread of the row
                        const uint32_t at = row.index(i + e);
                        if (tie) {
                            const u64 code = ((u64)smp_key(tie_val) << 32) | (uint32_t)~at;
                            for (int t = 0; t < C; t++) *cl.map_shared_rank(&sm.cut, t) = code;
                        } else {
                            report(xs[e], at);
                        }
                    }
                    upto += v[e];
                }
            }
        }
        if (!tie) return;  // after the exchange no CTA reads or writes another's memory
        if (threadIdx.x == 0) sm.kept_mass = tie_mass;
        cl.sync();
        row.cut_at(sm.cut);
        cut_mass = true;
    }
}

}  // namespace dllm
