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
// One cluster of C CTAs per row; the row's slice of each CTA stays in shared memory (read
// from HBM once), and every step is one pass over it and one exchange of a few words
// through distributed shared memory.  Bound: the logits' bytes; in practice the passes'
// arithmetic and the cluster barriers between them.
#pragma once
#include <cooperative_groups.h>

#include "layout.cuh"

namespace dllm {

constexpr int SMP_THREADS = 1024;
constexpr int SMP_WARPS = SMP_THREADS / 32;
constexpr int SMP_BINS = 2048;
constexpr int SMP_LIST = 512;  // elements ranked exactly
constexpr int SMP_MAX_CLUSTER = 8;
constexpr int ERR_LOGITS = -10;

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
    int32_t slice;   // elements per CTA (a multiple of 32)
    int32_t cached;  // of them, held in shared memory
    int32_t fix;     // weights are multiples of 2^-fix
};

struct SampleBox {  // one exchange: word r comes from CTA r of the cluster
    unsigned long long a[SMP_MAX_CLUSTER], b[SMP_MAX_CLUSTER], c[SMP_MAX_CLUSTER];
};

struct SampleShared {
    uint32_t cnt[SMP_BINS], lo[SMP_BINS], hi[SMP_BINS];  // this CTA's histogram
    uint32_t lkey[SMP_LIST], lidx[SMP_LIST];             // the ranked bin (CTA 0)
    unsigned long long lw[SMP_LIST];
    SampleBox box[2];
    unsigned long long wsum[SMP_WARPS];
    unsigned long long red[3][SMP_WARPS];
    unsigned long long found[5];  // crossing bin: bin, count before, mass before, count, mass
    uint32_t cut[2];              // key, index
    uint32_t n_list, best;
};

// Order-preserving code of a float (-0 counts as +0): larger value, larger code.
__device__ __forceinline__ uint32_t smp_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float smp_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

struct SampleRow {
    const float* src;   // the CTA's slice in global memory
    const float* cache;
    int n, cached;      // elements of the slice, and of them in shared memory
    uint32_t first;     // row index of the slice's first element
    float top;          // largest logit
    double inv_t, unit; // 1 / T, 2^fix
    double min_p;
    uint32_t cut_key, cut_idx;

    __device__ __forceinline__ float at(int i) const { return i < cached ? cache[i] : __ldg(src + i) + 0.0f; }
    // Fixed-point weight of a logit; 0 below min_p.  The sum with 2^52 rounds to a whole
    // number, which the low mantissa bits then hold.
    __device__ __forceinline__ unsigned long long weight(float l) const {
        if (l == -INFINITY) return 0;
        const double w = exp(((double)l - (double)top) * inv_t);
        if (w < min_p) return 0;
        return __double_as_longlong(fma(w, unit, 4503599627370496.0)) & 0xfffffffffffffull;
    }
    __device__ __forceinline__ bool kept(uint32_t key, int i) const {
        return key > cut_key || (key == cut_key && first + i <= cut_idx);
    }
};

// Exchange of three words per CTA through the cluster (thread 0's values); all threads
// return after every CTA's words are in this CTA's box.  Boxes alternate: a CTA may
// write the next exchange while another still reads this one.
__device__ __forceinline__ const SampleBox& smp_exchange(cooperative_groups::cluster_group& cl, SampleShared& sm,
                                                         int& phase, unsigned long long a, unsigned long long b,
                                                         unsigned long long c) {
    SampleBox& box = sm.box[phase & 1];
    phase++;
    const int C = (int)cl.num_blocks(), r = (int)cl.block_rank();
    if (threadIdx.x == 0)
        for (int t = 0; t < C; t++) {
            SampleBox* dst = cl.map_shared_rank(&box, t);
            dst->a[r] = a;
            dst->b[r] = b;
            dst->c[r] = c;
        }
    cl.sync();
    return box;
}

template <typename F>
__device__ __forceinline__ unsigned long long smp_warp_reduce(unsigned long long v, F f) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The CTA's reduction of one word per thread, in thread 0 (slot: 0..2).
template <typename F>
__device__ __forceinline__ unsigned long long smp_block_reduce(SampleShared& sm, int slot, unsigned long long v, F f) {
    v = smp_warp_reduce(v, f);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sm.red[slot][w] = v;
    __syncthreads();
    if (w == 0) v = smp_warp_reduce(sm.red[slot][lane], f);
    return v;
}

__device__ __forceinline__ unsigned long long smp_add(unsigned long long a, unsigned long long b) { return a + b; }

// The first element, in index order, whose running sum of weight_of(i) exceeds `target`
// (below the row's total); with u >= 0 the target is min(floor(u * total), total - 1).
// Calls hit(i) on the one thread that finds it.
template <typename W, typename H>
__device__ void smp_locate(cooperative_groups::cluster_group& cl, SampleShared& sm, int& phase, const SampleRow& row,
                           W weight_of, unsigned long long target, double u, H hit) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (row.n + SMP_WARPS - 1) / SMP_WARPS;  // a warp's contiguous share
    const int lo = min(row.n, w * per), hi = min(row.n, lo + per);
    unsigned long long s = 0;
    for (int i = lo + lane; i < hi; i += 32) s += weight_of(i);
    s = smp_warp_reduce(s, smp_add);
    __syncthreads();
    if (lane == 0) sm.wsum[w] = s;
    __syncthreads();
    unsigned long long mine = 0;
    for (int j = 0; j < SMP_WARPS; j++) mine += sm.wsum[j];
    const SampleBox& box = smp_exchange(cl, sm, phase, mine, 0, 0);
    unsigned long long before = 0, total = 0;
    for (int r = 0; r < (int)cl.num_blocks(); r++) {
        if (r < (int)cl.block_rank()) before += box.a[r];
        total += box.a[r];
    }
    if (u >= 0.0) {
        target = (unsigned long long)(u * (double)total);
        if (target >= total) target = total - 1;
    }
    if (target < before || target - before >= mine) return;  // another CTA's (uniform)
    unsigned long long run = before;
    int wi = 0;
    while (run + sm.wsum[wi] <= target) run += sm.wsum[wi++];
    const int a = min(row.n, wi * per), b = min(row.n, a + per);
    for (int i0 = a; i0 < b; i0 += SMP_THREADS) {
        const int i = i0 + (int)threadIdx.x;
        const unsigned long long v = i < b ? weight_of(i) : 0;
        unsigned long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        __syncthreads();
        if (lane == 31) sm.red[0][w] = inc;
        __syncthreads();
        unsigned long long base = run;
        for (int j = 0; j < w; j++) base += sm.red[0][j];
        const unsigned long long upto = base + inc;
        if (v != 0 && upto > target && upto - v <= target) hit(i);
        for (int j = w; j < SMP_WARPS; j++) base += sm.red[0][j];
        run = base;
    }
}

// Tightens the row's cut: by_count, to the first `want` candidates in order; else to the
// candidates whose preceding mass is < p * (their whole mass), and always the first.
// Candidates are the finite elements the present cut keeps.
__device__ void smp_narrow(cooperative_groups::cluster_group& cl, SampleShared& sm, int& phase, SampleRow& row,
                           float vmin, bool by_count, unsigned long long want, double p) {
    const int C = (int)cl.num_blocks(), r = (int)cl.block_rank();
    const int per = SMP_BINS / C;  // bins this CTA merges
    uint32_t kmax = smp_key(row.top), kmin = max(smp_key(vmin), row.cut_key);
    unsigned long long cnt0 = 0, mass0 = 0, limit = want;
    for (int level = 0;; level++) {
        // Level 0 spreads the values evenly over the bins (both sides scaled by 1/4, so that
        // no difference overflows; monotone, as each operation rounds monotonically); a bin
        // that is still too full is spread by codes, which always splits it.
        const float vhi = 0.25f * smp_value(kmax), span = vhi - 0.25f * smp_value(kmin);
        const float inv = (float)SMP_BINS / span;
        const int shift = max(0, 32 - __clz(kmax - kmin) - 11);
        const bool linear = level == 0 && span > 0.0f && inv < 1e30f;
        auto bin_of = [&](float l, uint32_t key) -> int {
            return linear ? min(SMP_BINS - 1, (int)(fmaf(-0.25f, l, vhi) * inv)) : (int)((kmax - key) >> shift);
        };
        for (int i = threadIdx.x; i < SMP_BINS; i += SMP_THREADS) sm.cnt[i] = sm.lo[i] = sm.hi[i] = 0;
        if (threadIdx.x == 0) sm.n_list = sm.best = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < row.n; i += SMP_THREADS) {
            const float l = row.at(i);
            const uint32_t key = smp_key(l);
            if (l == -INFINITY || key > kmax || key < kmin || !row.kept(key, i)) continue;
            const int b = bin_of(l, key);
            if (!by_count) {
                const unsigned long long wt = row.weight(l);
                const uint32_t wl = (uint32_t)wt, old = atomicAdd(&sm.lo[b], wl);
                const uint32_t wh = (uint32_t)(wt >> 32) + (old + wl < old ? 1u : 0u);
                if (wh) atomicAdd(&sm.hi[b], wh);
            }
            atomicAdd(&sm.cnt[b], 1u);
        }
        cl.sync();
        // merge this CTA's share of the bins: thread t takes bins r * per + t, + 1024
        unsigned long long mc[2] = {0, 0}, mm[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int t = 2 * (int)threadIdx.x + h;  // adjacent bins, in order
            if (t < per)
                for (int s = 0; s < C; s++) {
                    const SampleShared* o = cl.map_shared_rank(&sm, s);
                    const int b = r * per + t;
                    mc[h] += o->cnt[b];
                    mm[h] += ((unsigned long long)o->hi[b] << 32) + o->lo[b];
                }
        }
        const unsigned long long cs = mc[0] + mc[1], ms = mm[0] + mm[1];
        const unsigned long long tc = smp_block_reduce(sm, 0, cs, smp_add), tm = smp_block_reduce(sm, 1, ms, smp_add);
        const SampleBox& box = smp_exchange(cl, sm, phase, tc, tm, 0);
        unsigned long long bc = cnt0, bm = mass0, allc = 0, allm = 0, myc = 0, mym = 0;
        for (int s = 0; s < C; s++) {
            if (s < r) bc += box.a[s], bm += box.b[s];
            if (s == r) myc = box.a[s], mym = box.b[s];
            allc += box.a[s];
            allm += box.b[s];
        }
        if (level == 0) {
            if (by_count) {
                if (allc <= want) return;  // nothing to cut (uniform over the cluster)
            } else {
                // preceding mass < p S of whole numbers: preceding mass < ceil(p S); at least 1
                // keeps the first candidate
                limit = (unsigned long long)ceil(p * (double)allm);
                if (limit < 1) limit = 1;
            }
        }
        // The crossing bin: the first with count (mass) up to its end >= limit.
        const unsigned long long b0 = by_count ? bc : bm, mine = by_count ? myc : mym;
        if (b0 < limit && b0 + mine >= limit) {  // this CTA's bins hold it (uniform)
            const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
            unsigned long long ic = cs, im = ms;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long x = __shfl_up_sync(0xffffffffu, ic, o), y = __shfl_up_sync(0xffffffffu, im, o);
                if (lane >= o) ic += x, im += y;
            }
            __syncthreads();
            if (lane == 31) sm.red[0][w] = ic, sm.red[1][w] = im;
            __syncthreads();
            unsigned long long xc = bc + ic - cs, xm = bm + im - ms;  // before this thread's bins
            for (int j = 0; j < w; j++) xc += sm.red[0][j], xm += sm.red[1][j];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const unsigned long long x = by_count ? xc : xm, y = by_count ? mc[h] : mm[h];
                if (x < limit && x + y >= limit)
                    for (int s = 0; s < C; s++) {
                        unsigned long long* f = cl.map_shared_rank(sm.found, s);
                        f[0] = r * per + 2 * threadIdx.x + h;
                        f[1] = xc;
                        f[2] = xm;
                        f[3] = mc[h];
                    }
                xc += mc[h];
                xm += mm[h];
            }
        }
        cl.sync();
        const int bin = (int)sm.found[0];
        cnt0 = sm.found[1];
        mass0 = sm.found[2];
        const unsigned long long n_bin = sm.found[3];
        if (n_bin > SMP_LIST) {
            // too many to rank: the bin's own range of codes, or its ties by index
            if (linear) {
                unsigned long long a = 0, b = 0;  // largest code, largest complement
                for (int i = threadIdx.x; i < row.n; i += SMP_THREADS) {
                    const float l = row.at(i);
                    const uint32_t key = smp_key(l);
                    if (l == -INFINITY || key > kmax || key < kmin || !row.kept(key, i) || bin_of(l, key) != bin) continue;
                    a = max(a, (unsigned long long)key);
                    b = max(b, (unsigned long long)(uint32_t)~key);
                }
                auto mx = [](unsigned long long x, unsigned long long y) { return x > y ? x : y; };
                const unsigned long long a1 = smp_block_reduce(sm, 0, a, mx), b1 = smp_block_reduce(sm, 1, b, mx);
                const SampleBox& rng = smp_exchange(cl, sm, phase, a1, b1, 0);
                for (int s = 0; s < C; s++) a = s ? mx(a, rng.a[s]) : rng.a[s], b = s ? mx(b, rng.b[s]) : rng.b[s];
                kmax = (uint32_t)a;
                kmin = ~(uint32_t)b;
            } else {
                const uint32_t top = kmax - ((uint32_t)bin << shift);
                kmin = max(kmin, shift ? top - ((1u << shift) - 1u) : top);
                kmax = top;
            }
            if (kmin != kmax) continue;
            // all equal: the first q of them in index order
            unsigned long long q = limit - cnt0;
            if (!by_count) {
                const unsigned long long wt = row.weight(smp_value(kmax));
                q = (limit - mass0 + wt - 1) / wt;  // before = mass0 + j wt < limit
            }
            const uint32_t tie = kmax;
            smp_locate(cl, sm, phase, row,
                       [&](int i) -> unsigned long long {
                           const uint32_t key = smp_key(row.at(i));
                           return key == tie && row.kept(key, i) ? 1 : 0;
                       },
                       q - 1, -1.0, [&](int i) {
                           for (int s = 0; s < C; s++) {
                               uint32_t* c = cl.map_shared_rank(sm.cut, s);
                               c[0] = tie;
                               c[1] = row.first + i;
                           }
                       });
            break;
        }
        // rank the crossing bin in CTA 0
        for (int i = threadIdx.x; i < row.n; i += SMP_THREADS) {
            const float l = row.at(i);
            const uint32_t key = smp_key(l);
            if (l == -INFINITY || key > kmax || key < kmin || !row.kept(key, i) || bin_of(l, key) != bin) continue;
            SampleShared* o = cl.map_shared_rank(&sm, 0);
            const uint32_t at = atomicAdd(&o->n_list, 1u);
            if (at < SMP_LIST) {
                o->lkey[at] = key;
                o->lidx[at] = row.first + i;
                o->lw[at] = by_count ? 0 : row.weight(l);
            }
        }
        cl.sync();
        if (r == 0) {
            const int n = (int)min(sm.n_list, (uint32_t)SMP_LIST), t = threadIdx.x;
            uint32_t rank = 0;
            bool in = false;
            if (t < n) {
                const uint32_t key = sm.lkey[t], idx = sm.lidx[t];
                unsigned long long m = mass0;
                for (int j = 0; j < n; j++)
                    if (sm.lkey[j] > key || (sm.lkey[j] == key && sm.lidx[j] < idx)) rank++, m += sm.lw[j];
                in = by_count ? cnt0 + rank < limit : m < limit;
                if (in) atomicMax(&sm.best, rank);
            }
            __syncthreads();
            if (in && rank == sm.best)  // the last one kept
                for (int s = 0; s < C; s++) {
                    uint32_t* c = cl.map_shared_rank(sm.cut, s);
                    c[0] = sm.lkey[t];
                    c[1] = sm.lidx[t];
                }
        }
        break;
    }
    cl.sync();
    row.cut_key = sm.cut[0];
    row.cut_idx = sm.cut[1];
}

// Grid (C * rows), clusters of C.
__global__ void __launch_bounds__(SMP_THREADS) sample_kernel(const __grid_constant__ SampleArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    SampleShared& sm = *reinterpret_cast<SampleShared*>(smem);
    float* cache = reinterpret_cast<float*>(smem + sizeof(SampleShared));
    cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
    const int C = (int)cl.num_blocks(), r = (int)cl.block_rank();
    const int64_t i_row = blockIdx.x / C;
    int phase = 0;
    pdl_trigger();
    pdl_wait();

    SampleRow row;
    const int64_t first = min(a.V, (int64_t)r * a.slice);
    row.first = (uint32_t)first;
    row.n = (int)min((int64_t)a.slice, a.V - first);
    row.cached = min(row.n, a.cached);
    row.src = a.logits + i_row * a.ldl + first;
    row.cache = cache;

    // the slice into shared memory; the row's largest and smallest finite logit
    float hi = -INFINITY, lo = INFINITY;
    bool bad = false;
#pragma unroll 8
    for (int i = threadIdx.x; i < row.n; i += SMP_THREADS) {
        const float l = __ldg(row.src + i) + 0.0f;
        if (i < row.cached) cache[i] = l;
        bad |= !(l < INFINITY);  // +inf or NaN
        hi = fmaxf(hi, l);
        if (l > -INFINITY) lo = fminf(lo, l);
    }
    auto mx = [](unsigned long long x, unsigned long long y) { return x > y ? x : y; };
    const unsigned long long k1 = smp_block_reduce(sm, 0, smp_key(hi), mx);
    const unsigned long long k2 = smp_block_reduce(sm, 1, (uint32_t)~smp_key(lo), mx);
    const unsigned long long k3 = smp_block_reduce(sm, 2, bad ? 1ull : 0ull, mx);
    unsigned long long m1 = 0, m2 = 0, m3 = 0;
    {
        const SampleBox& box = smp_exchange(cl, sm, phase, k1, k2, k3);
        for (int s = 0; s < C; s++) m1 = mx(m1, box.a[s]), m2 = mx(m2, box.b[s]), m3 = mx(m3, box.c[s]);
    }
    row.top = smp_value((uint32_t)m1);
    const float vmin = smp_value(~(uint32_t)m2);
    if (m3 || row.top == -INFINITY) {  // uniform over the cluster
        if (r == 0 && threadIdx.x == 0) {
            a.token[i_row] = -1;
            if (a.conf) a.conf[i_row] = 0.0f;
            if (a.entropy) a.entropy[i_row] = 0.0f;
            set_err(ERR_LOGITS);
        }
        cl.sync();  // no CTA leaves while another may still write its box
        return;
    }

    const float T = a.temperature ? a.temperature[i_row] : 1.0f;
    const bool greedy = !(T > 0.0f);
    const float mp = a.min_p ? a.min_p[i_row] : 0.0f;
    const float p = a.top_p ? a.top_p[i_row] : 1.0f;
    const int32_t k = greedy ? 1 : a.top_k ? a.top_k[i_row] : 0;
    float u = a.u ? a.u[i_row] : 0.0f;
    u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;  // NaN counts as 0
    row.inv_t = greedy ? 1.0 : 1.0 / (double)T;
    row.unit = (double)(1ull << a.fix);
    row.min_p = mp > 0.0f ? fmin((double)mp, 1.0) : 0.0;
    row.cut_key = 0;
    row.cut_idx = 0xffffffffu;

    // plain softmax: mass and first moment of the elements below the largest, and the
    // number equal to it (kept apart, so that a peaked row's small entropy stays exact)
    double s1 = 0.0, s2 = 0.0, n_top = 0.0;
    if (a.conf || a.entropy) {
        float e1 = 0.0f, e2 = 0.0f;
        uint32_t eq = 0;
        for (int i = threadIdx.x; i < row.n; i += SMP_THREADS) {
            const float l = row.at(i), z = l - row.top;
            if (z == 0.0f) {
                eq++;
            } else if (z > -INFINITY) {
                const float e = expf(z);
                e1 += e;
                e2 = fmaf(e, z, e2);
            }
        }
        auto dadd = [](unsigned long long x, unsigned long long y) -> unsigned long long {
            return __double_as_longlong(__longlong_as_double(x) + __longlong_as_double(y));
        };
        const unsigned long long b1 = smp_block_reduce(sm, 0, __double_as_longlong((double)e1), dadd);
        const unsigned long long b2 = smp_block_reduce(sm, 1, __double_as_longlong((double)e2), dadd);
        const unsigned long long b3 = smp_block_reduce(sm, 2, eq, smp_add);
        const SampleBox& box = smp_exchange(cl, sm, phase, b1, b2, b3);
        for (int s = 0; s < C; s++) {
            s1 += __longlong_as_double(box.a[s]);
            s2 += __longlong_as_double(box.b[s]);
            n_top += (double)box.c[s];
        }
        if (a.entropy && r == 0 && threadIdx.x == 0) {
            const double total = n_top + s1;
            a.entropy[i_row] = (float)(log1p(s1 + (n_top - 1.0)) - s2 / total);
        }
    }

    if (k > 0) smp_narrow(cl, sm, phase, row, vmin, true, (unsigned long long)k, 0.0);
    if (!(p >= 1.0f) && k != 1) smp_narrow(cl, sm, phase, row, vmin, false, 0, p > 0.0f ? (double)p : 0.0);

    smp_locate(cl, sm, phase, row,
               [&](int i) -> unsigned long long {
                   const float l = row.at(i);
                   return row.kept(smp_key(l), i) ? row.weight(l) : 0;
               },
               0, (double)u, [&](int i) {
                   a.token[i_row] = (int32_t)(row.first + i);
                   if (a.conf) a.conf[i_row] = (float)(exp((double)row.at(i) - (double)row.top) / (n_top + s1));
               });
    cl.sync();
}

}  // namespace dllm
