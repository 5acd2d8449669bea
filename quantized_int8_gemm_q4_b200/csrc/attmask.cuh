// Attention under key intervals on the sm_100a tensor cores: query i attends to the keys
// [kv_begin[i], kv_end[i]), with an optional tanh cap on the scores and an optional bias
// that falls with distance (packed documents, prefixes, blocks of a canvas over the kept
// ones before it, windows, padding).
//
//   s_ij = q_i . k_j / sqrt(dh);  s = cap tanh(s / cap);  s -= slope_h |q_pos_i - j|
//   o_i = sum over the interval of softmax(s_i)_j v_j;  an empty interval gives zeros
//
// A tile is 128 rows (tensor-memory lanes) of one key head: gp query heads of its group
// (the largest divisor of the group up to 128) x 128 / gp queries, row = query * gp + head,
// which is the order in which one TMA box of gp heads x 128 / gp rows lands in shared memory.  So
// grouped heads read their keys once, and one query of 8 heads fills 8 rows.  A CTA has one tile
// and the key blocks of 64 that any of its rows sees, or one of `splits` equal parts of them.
// Two chains of blocks run on each SM, in one of two ways:
//   two CTAs      of 8 warps each share the SM (more tiles than SMs): one's start, masks and
//                 output run beside the other's blocks
//   halves        a CTA of 12 warps with two chains: the first takes the first half of the
//                 blocks, the second the others, and their results are joined from tensor
//                 memory at the end
// Warps (of halves; the others' in brackets):
//   0-3, 4-7 [0-3]  softmax of chain 0, chain 1; thread = row, all 64 scores of a block in
//                   registers; the running maximum is raised by more than 2^8 at a time
//   8, 9 [4]        issue the MMAs of a chain (S = Q K^T, O += P V; kind::f16, f32 in
//                   tensor memory); the first owns tensor memory.  The whole warp runs the
//                   issue loop and an elected lane's predicate guards each instruction, so
//                   that its operands stay in uniform registers: 75-97 cycles per MMA from
//                   one warp against 141 inside a one-lane branch; two warps together issue
//                   one per 64, the tensor core's rate.  [5 has nothing to do]
//   10 [6]          TMA producer of Q, K and V (4 and 8 [2 and 3] slots of 64 keys x dh)
//   11 [7]          V's gate: in a block that some row does not see whole, it replaces what
//                   is not finite by zeros and marks those keys (a weight of zero times NaN is
//                   NaN, and the hidden key of one row is another's).  A row that attends a
//                   marked key loses, at the end, the columns where a value of its keys from
//                   there on is not finite, as it would where all rows see the block whole
// Tensor memory: O of chain t at columns 256 t, two S slots of 64 columns behind it, block kb in slot
// kb & 1; P lies over the first half of its S (f16 pairs).  Issue order per chain: S(0), S(1), then
// P V(kb), S(kb + 2): the scores of the next block are there when a softmax ends, and the
// tensor core works while the softmax of either chain runs.
//
// Bounds per SM, for two tiles and 128 keys: 2048 cycles of MMA at 8192 operations per cycle (2600
// as issued: a 128 x 64 x 16 MMA takes 49 cycles for its 6 KB of shared memory), and 2048 of the
// special-function unit (32768 exponentials at 16 per cycle).  A softmax thread's own chain (wait,
// load, maximum, exponentials, store, hand-over) takes ~1900 cycles per block, and the two chains of
// an SM run side by side: ~2000 cycles per block of both.
//
// Measured (one B200): 4096 positions under a 1000-position prefix, 32 heads: 154 us at 1965 MHz, 177 us
// once the power cap holds the clock at 1680 MHz (820 TFLOP/s of attended pairs); six packed
// documents over 1024 positions 16.7 us; one query over 20011 keys of 32 heads 58-59 us (5.6 TB/s);
// 32 queries over 8200 keys, 28 heads on 4, 19.7 us; capped and biased, 1531 positions in three
// documents, 39 us.
// Measured and not kept: two tiles per CTA that share their key blocks (1200 positions of 32 heads,
// all keys, 53 us against 42 for two CTAs; in eight documents 24.5 against 19.3; with the long
// prefix the same); 128-key blocks with one score slot (prefix 182 us against 157: S waits for P);
// two threads per row, or the two slots' softmax on two warpgroups that hand the maximum over
// (both 3-10% slower: the special-function unit is shared, the chains are longer); one
// exponential in four by polynomial (no gain) or in two (10% slower); all commits after the MMAs
// (slots return later: one over 20011 66 -> 72 us).
#pragma once
#include <cfloat>

#include "attention.cuh"
#include "qgemm.cuh"
#include "rope.cuh"

namespace dllm {

constexpr int msk_threads(bool halves) { return halves ? 384 : 256; }
constexpr int MSK_BK = 64;    // keys per block
// Slots: with halves, the scores of four blocks ahead leave four V blocks waiting for their
// weights, and as many are on their way.  Two CTAs per SM have the space of five slots each: K is
// read two blocks ahead of its V.
constexpr int MSK_K_SLOTS = 4, MSK_V_SLOTS = 8;  // at most
constexpr int msk_k_slots(bool halves) { return halves ? 4 : 2; }
constexpr int msk_v_slots(bool halves) { return halves ? 8 : 3; }
constexpr int MSK_KV = MSK_BK * ATT_DH * 2;
// Registers per thread after setmaxnreg (softmax warpgroups; the others), out of the
// launch's 384 x 168.
constexpr int MSK_REG_SOFTMAX = 200;
constexpr int msk_reg_other(bool halves) { return halves ? 96 : 56; }
constexpr int msk_reg_launch(bool halves) { return halves ? 168 : 128; }
static_assert(256 * MSK_REG_SOFTMAX + 128 * msk_reg_other(true) <= 384 * msk_reg_launch(true), "setmaxnreg split");
static_assert(128 * MSK_REG_SOFTMAX + 128 * msk_reg_other(false) <= 256 * msk_reg_launch(false), "setmaxnreg split");

struct MaskShared {
    uint64_t q_full, k_full[MSK_K_SLOTS], k_empty[MSK_K_SLOTS];
    uint64_t v_full[MSK_V_SLOTS], v_ready[MSK_V_SLOTS], v_empty[MSK_V_SLOTS];
    uint64_t s_full[2][2], p_full[2][2], o_done[2][2], fin;  // [chain][S slot]
    uint32_t tmem, flags[MSK_V_SLOTS][2];  // per V slot, bit j: key j's value is not finite
    int32_t lo_min[8], hi_max[8], lo_max[8], hi_min[8];  // per softmax warp, over rows with keys
    float2 ml[2][128];  // halves only (the last field: without them it is not there)
};
constexpr size_t msk_smem(bool halves) {
    return ATT_TILE + (size_t)(msk_k_slots(halves) + msk_v_slots(halves)) * MSK_KV +
           (halves ? sizeof(MaskShared) : offsetof(MaskShared, ml));
}
static_assert(msk_smem(true) <= 227 * 1024, "shared memory of a CTA");
static_assert(2 * (msk_smem(false) + 1024) <= 228 * 1024, "shared memory of two CTAs");

struct MaskArgs {
    int32_t Lq, Lk, H, group;
    int32_t gp, tq;   // heads and queries per tile
    int32_t splits;   // parts of the key range (grid y)
    const int32_t *kv_begin, *kv_end, *q_pos;
    const __half* v;  // as in the tensor map, for the columns of values that are not finite
    int64_t ldv;
    float cap_in, cap_out;  // base-2 exponents: cap_out tanh(cap_in q.k)
    const float* slopes;
    void* o;
    int32_t o_f16;
    float* part;      // splits > 1: unnormalised O [splits][Lq][H][128]
    float2* part_ml;  // and (m, l) [splits][Lq][H]; m = -inf: no key of the row in this part
};

__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
          "l"(*reinterpret_cast<uint64_t*>(&c)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}

__device__ __forceinline__ void prefetch_tensormap(const void* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// One lane of a converged warp, as a predicate.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}
// mma_f16_ss and mma_f16_ts where `issue` is not 0.
__device__ __forceinline__ void mma_f16_ss_if(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue)
        : "memory");
}
__device__ __forceinline__ void mma_f16_ts_if(uint32_t issue, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue)
        : "memory");
}

// An f16 with all exponent bits set (infinity or NaN) carries into its sign bit, for two at a time.
__device__ __forceinline__ uint32_t att_not_finite(uint32_t y) { return (y & 0x7fff7fffu) + 0x04000400u; }

// tanh(y) = 1 - 2 / (1 + 2^(2 log2(e) y)), good to a few 2^-24 absolute.
__device__ __forceinline__ float att_tanh(float y) {
    const float e = att_ex2(y * 2.885390081777927f);
    return 1.0f - __fdividef(2.0f, 1.0f + e);
}

// tanh of two values on the multiply-add pipe: odd polynomials fitted to it, of degree 7 up to
// 0.35 (off by less than 2^-24) and of degree 13 up to 1 (2^-23).
__device__ __forceinline__ float2 att_tanh_small(float2 y) {
    auto k = [](float c) { return make_float2(c, c); };
    const float2 q = fmul2(y, y);
    float2 p = ffma2(q, k(-0.04837692156434059f), k(0.13283324241638184f));
    p = ffma2(p, q, k(-0.3333165645599365f));
    p = ffma2(p, q, k(0.9999998211860657f));
    return fmul2(p, y);
}
__device__ __forceinline__ float2 att_tanh_poly(float2 y) {
    auto k = [](float c) { return make_float2(c, c); };
    const float2 q = fmul2(y, y);
    float2 p = ffma2(q, k(0.0009637725888751447f), k(-0.005951281636953354f));
    p = ffma2(p, q, k(0.019973283633589745f));
    p = ffma2(p, q, k(-0.05326583608984947f));
    p = ffma2(p, q, k(0.13319583237171173f));
    p = ffma2(p, q, k(-0.33332130312919617f));
    p = ffma2(p, q, k(0.9999997019767761f));
    return fmul2(p, y);
}

// Turns into NaN, in the warp's rows of O (tensor memory), the columns where a value of the row's keys
// [first, end) is not finite; first >= end leaves a row as it is.  All lanes take part: 8 bytes each
// of a key's value, row by row.  Not inlined: rare, and its registers are the hot loop's.
__device__ __noinline__ void msk_lose_columns(uint32_t tO, int first, int end, const __half* v, int64_t ldv) {
    const int lane = threadIdx.x & 31;
    uint32_t lost[4] = {0, 0, 0, 0};  // bit i of word j: column 4 i + j
#pragma unroll 1
    for (uint32_t rows = __ballot_sync(~0u, first < end); rows; rows &= rows - 1) {
        const int r = __ffs(rows) - 1, k1 = __shfl_sync(~0u, end, r);
        uint32_t x = 0, y = 0;
#pragma unroll 4
        for (int k = __shfl_sync(~0u, first, r); k < k1; k++) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(v + k * ldv) + lane);
            x |= att_not_finite(u.x);
            y |= att_not_finite(u.y);
        }
        const uint32_t w[4] = {x & 0x8000u, x & 0x80000000u, y & 0x8000u, y & 0x80000000u};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t b = __ballot_sync(~0u, w[j] != 0);
            if (lane == r) lost[j] = b;
        }
    }
#pragma unroll 1
    for (int c = 0; c < 8; c++) {
        uint32_t o[16];
        tmem_ld16(tO + 16 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e++) o[e] = lost[e & 3] >> (4 * c + (e >> 2)) & 1 ? 0x7fffffffu : o[e];
        tmem_st16(tO + 16 * c, o);
    }
    tmem_wait_st();
}

// MODE bit 0: cap, bit 1: distance bias, bit 2: halves.
template <int MODE>
__global__ void __launch_bounds__(msk_threads(MODE & 4), MODE & 4 ? 1 : 2)
    attention_masked_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                            const __grid_constant__ CUtensorMap tv, const __grid_constant__ MaskArgs a) {
    constexpr bool CAP = MODE & 1, BIAS = MODE & 2, halves = MODE & 4;
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int CHAINS = halves ? 2 : 1;
    constexpr int MMA_WARP = 4 * CHAINS, TMA_WARP = MMA_WARP + 2, GATE_WARP = MMA_WARP + 3;
    constexpr int k_slots = msk_k_slots(halves), v_slots = msk_v_slots(halves);
    uint8_t* const sQ = smem;
    uint8_t* const sK = smem + ATT_TILE;
    uint8_t* const sV = sK + k_slots * MSK_KV;
    MaskShared& sh = *reinterpret_cast<MaskShared*>(sV + v_slots * MSK_KV);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The last queries first (under causal intervals theirs are the longest), all heads of them.
    const int n_heads = a.H / a.gp, h0 = (int)(blockIdx.x % n_heads) * a.gp, hk = h0 / a.group;
    const int q0 = (int)((gridDim.x - 1 - blockIdx.x) / n_heads) * a.tq;

    if (warp == MMA_WARP) {
        tmem_alloc(&sh.tmem, 256 * CHAINS);
        tmem_relinquish();
    }
    if (threadIdx.x == 32 * TMA_WARP) {
        prefetch_tensormap(&tq);
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
        mbar_init(&sh.q_full, 1);
        for (int b = 0; b < 2; b++)
            for (int x = 0; x < CHAINS; x++) {
                mbar_init(&sh.s_full[x][b], 1);
                mbar_init(&sh.p_full[x][b], 4);
                mbar_init(&sh.o_done[x][b], 1);
            }
        for (int b = 0; b < k_slots; b++) {
            mbar_init(&sh.k_full[b], 1);
            mbar_init(&sh.k_empty[b], CHAINS);
        }
        for (int b = 0; b < v_slots; b++) {
            mbar_init(&sh.v_full[b], 1);
            mbar_init(&sh.v_ready[b], 1);
            mbar_init(&sh.v_empty[b], CHAINS);
        }
        mbar_init(&sh.fin, CHAINS);
        fence_mbar_init();
    }
    pdl_trigger();
    pdl_wait();  // q, k, v and the intervals may come from the previous kernel on the stream
    if (warp == TMA_WARP) {
        // the queries at once, while the intervals are read
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(a.gp * a.tq) * ATT_DH * 2);
        __syncwarp();
        att_tma_tile(sQ, &tq, h0, q0, &sh.q_full, lane);
    }

    // This thread's row (softmax warps): query, head, interval.
    const int t = halves ? warp >> 2 : 0, quad = warp & 3, row = threadIdx.x & 127;
    int qi = 0, head = 0, lo = 0, hi = 0;
    bool live = false;
    if (warp < MMA_WARP) {
        qi = q0 + row / a.gp;
        head = h0 + row % a.gp;
        live = row < a.tq * a.gp && qi < a.Lq;
        if (live) {
            lo = a.kv_begin ? max(0, __ldg(a.kv_begin + qi)) : 0;
            hi = a.kv_end ? min(a.Lk, __ldg(a.kv_end + qi)) : a.Lk;
        }
        const bool some = live && lo < hi;
        const int l0 = __reduce_min_sync(~0u, some ? lo : INT_MAX), h1 = __reduce_max_sync(~0u, some ? hi : 0);
        const int l1 = __reduce_max_sync(~0u, some ? lo : 0), h2 = __reduce_min_sync(~0u, some ? hi : INT_MAX);
        if (lane == 0) sh.lo_min[warp] = l0, sh.hi_max[warp] = h1, sh.lo_max[warp] = l1, sh.hi_min[warp] = h2;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh.tmem;

    // Key blocks that any row of the CTA sees, and the CTA's part of them: [B0, B1).
    int l0 = INT_MAX, h1 = 0, b_full0 = 0, b_full1 = INT_MAX;  // keys that every row sees
#pragma unroll
    for (int w = 0; w < 4; w++) {  // (halves: both chains have the same rows)
        l0 = min(l0, sh.lo_min[w]);
        h1 = max(h1, sh.hi_max[w]);
        b_full0 = max(b_full0, sh.lo_max[w]);
        b_full1 = min(b_full1, sh.hi_min[w]);
    }
    int B0 = l0 < h1 ? l0 / MSK_BK : 0, B1 = l0 < h1 ? (h1 + MSK_BK - 1) / MSK_BK : 0;
    if (a.splits > 1) {
        const int n = (B1 - B0 + a.splits - 1) / a.splits;
        B0 = min(B1, B0 + (int)blockIdx.y * n);
        B1 = min(B1, B0 + n);
    }
    const int N = B1 - B0, mid = B0 + (N + 1) / 2;
    // The blocks of each chain; the n-th block that is loaded: in order, or from the halves in
    // turn; and whether chain x works on it, as its block number i.
    const int t0[2] = {B0, halves ? mid : B1}, t1[2] = {halves ? mid : B1, B1};
    auto block = [&](int n) { return halves ? ((n & 1) ? mid : B0) + (n >> 1) : B0 + n; };
    auto owns = [&](int x, int n) { return !halves || (n & 1) == x; };
    auto local = [&](int x, int n) { return halves ? n >> 1 : n; };
    // A block that every row sees whole needs no gate.
    auto whole = [&](int kb) { return kb * MSK_BK >= b_full0 && (kb + 1) * MSK_BK <= b_full1; };

    if (warp >= MMA_WARP) {
        setmaxnreg_dec<msk_reg_other(halves)>();
        if (warp == TMA_WARP) {
            // ------------------------------------------------------------ TMA producer
            int nk = 0, nv = 0;
            auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* full, int kb) {
                if (lane == 0) mbar_arrive_expect_tx(full, MSK_KV);
                __syncwarp();
                if (lane < 2) tma_load_3d(dst + lane * (MSK_KV / 2), map, 64 * lane, hk, kb * MSK_BK, full);
            };
            // (slots as counters: three of them make no mask)
            int b = 0, c = 0;
            uint32_t kp = 1, vp = 1;  // parity of the slot's last release (first round: passes at once)
            for (int n = 0; n < N; n++) {
                if (!__all_sync(~0u, att_wait(&sh.k_empty[b], kp))) break;
                load(sK + b * MSK_KV, &tk, &sh.k_full[b], block(n));
                nk = n + 1;
                if (++b == k_slots) b = 0, kp ^= 1;
                if (!__all_sync(~0u, att_wait(&sh.v_empty[c], vp))) break;
                load(sV + c * MSK_KV, &tv, &sh.v_full[c], block(n));
                nv = n + 1;
                if (++c == v_slots) c = 0, vp ^= 1;
            }
            // No copy may still be landing when the CTA exits, also when a wait ran out.
            if (lane == 0) {
                for (int m = max(0, nk - k_slots); m < nk; m++) drain_wait(&sh.k_full[m % k_slots], (m / k_slots) & 1);
                for (int m = max(0, nv - v_slots); m < nv; m++) drain_wait(&sh.v_full[m % v_slots], (m / v_slots) & 1);
                drain_wait(&sh.q_full, 0);
            }
            __syncwarp();
        } else if (warp == GATE_WARP) {
            // ------------------------------------------------------------ V's gate
            int b = 0;
            uint32_t vp = 0;
            for (int n = 0; n < N; n++) {
                if (!__all_sync(~0u, att_wait(&sh.v_full[b], vp))) break;
                if (!whole(block(n))) {
                    if (lane < 2) sh.flags[b][lane] = 0;
                    __syncwarp();
                    uint4* const v = reinterpret_cast<uint4*>(sV + b * MSK_KV);
                    auto c = att_not_finite;
#pragma unroll 1
                    for (int i0 = lane; i0 < MSK_KV / 16; i0 += 8 * 32) {
                        uint4 x[8];
#pragma unroll
                        for (int e = 0; e < 8; e++) x[e] = v[i0 + 32 * e];
                        uint32_t any = 0;
#pragma unroll
                        for (int e = 0; e < 8; e++) any |= c(x[e].x) | c(x[e].y) | c(x[e].z) | c(x[e].w);
                        if (!(any & 0x80008000u)) continue;
                        for (int i = i0; i < i0 + 8 * 32; i += 32) {
                            const uint4 y = v[i];
                            auto z = [&](uint32_t u) {
                                const uint32_t m = (c(u) & 0x80008000u) >> 15;  // 1 per half to clear
                                return u & ~(m * 0xffffu);
                            };
                            if (!((c(y.x) | c(y.y) | c(y.z) | c(y.w)) & 0x80008000u)) continue;
                            v[i] = make_uint4(z(y.x), z(y.y), z(y.z), z(y.w));
                            const int key = (i >> 3) & (MSK_BK - 1);  // 128-byte rows of 64 head-dim values
                            atomicOr(&sh.flags[b][key >> 5], 1u << (key & 31));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&sh.v_ready[b]);
                if (++b == v_slots) b = 0, vp ^= 1;
            }
        } else if (warp < MMA_WARP + CHAINS) {
            // ------------------------------------------------------------ MMA issue, chain x
            constexpr uint32_t ID_S = idesc_f16(128, MSK_BK);
            constexpr uint32_t ID_O = idesc_f16(128, ATT_DH) | (1u << 16);  // B (V) MN-major
            const int x = __shfl_sync(~0u, warp - MMA_WARP, 0);
            const uint32_t el = elect_one();
            const uint32_t tO = tm + 256 * x, tS = tO + 128;
            const uint64_t dq = att_qk_desc(sQ), dk = att_qk_desc(sK);
            const uint64_t dv = sdesc_sw128(smem_u32(sV), MSK_KV / 2, 1024);
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && __all_sync(~0u, att_wait(bar, parity)); };
            // S of the n-th block.  A block that is not the tile's is waited for all the same
            // before its slot is given back.
            int kb = 0, vb = 0;
            uint32_t kp = 0, vp = 0;
            auto scores = [&](int n) {
                const int b = kb;
                if (n >= N) return;
                wait(&sh.k_full[b], kp);
                if (!ok) return;
                if (++kb == k_slots) kb = 0, kp ^= 1;
                if (owns(x, n)) {
                    tc_fence_after();
                    const int sl = local(x, n) & 1;
                    const uint64_t d = dk + (uint64_t)(b * (MSK_KV >> 4));
                    const uint32_t ts = tS + 64 * sl;
                    mma_f16_ss_if(el, ts, dq, d, ID_S, 0);
#pragma unroll
                    for (int kk = 1; kk < ATT_DH / 16; kk++)
                        mma_f16_ss_if(el, ts, dq + att_qk_step(kk), d + att_k64_step(kk), ID_S, 1);
                    if (el) tc_commit(&sh.s_full[x][sl]);
                }
                if (el) tc_commit(&sh.k_empty[b]);
            };
            if (N > 0) wait(&sh.q_full, 0);
            const int ahead = halves ? 4 : 2;  // two of the tile's own blocks
#pragma unroll 1
            for (int n = -ahead; ok && n < N; n++) {
                if (n >= 0) {
                    const int b = vb;
                    wait(&sh.v_ready[b], vp);
                    if (++vb == v_slots) vb = 0, vp ^= 1;
                    if (owns(x, n)) {
                        const int i = local(x, n), sl = i & 1;
                        wait(&sh.p_full[x][sl], (i >> 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t d = dv + (uint64_t)(b * (MSK_KV >> 4));
                        const uint32_t tp = tS + 64 * sl;
                        mma_f16_ts_if(el, tO, tp, d, ID_O, i > 0);
#pragma unroll
                        for (int kk = 1; kk < MSK_BK / 16; kk++)
                            mma_f16_ts_if(el, tO, tp + 8 * kk, d + att_v_step(kk), ID_O, 1);
                        if (el) tc_commit(&sh.o_done[x][sl]);
                    }
                    if (!ok) break;
                    if (el) tc_commit(&sh.v_empty[b]);
                }
                scores(n + ahead);
            }
            // Every MMA issued above completes before tensor memory is released.
            if (el) {
                tc_commit(&sh.fin);
                drain_wait(&sh.fin, 0);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax, output
        setmaxnreg_inc<MSK_REG_SOFTMAX>();
        const uint32_t tO = tm + ((uint32_t)(32 * quad) << 16) + 256 * t;
        const int kb0 = t ? t0[1] : t0[0], kb1 = t ? t1[1] : t1[0];
        int vs = t, vp = 0;  // V slot of the present block and its parity
        const int w_lo0 = sh.lo_min[warp], w_hi1 = sh.hi_max[warp], w_lo1 = sh.lo_max[warp], w_hi0 = sh.hi_min[warp];
        const bool some = lo < hi;
        if (!some) lo = hi = 0;  // a row without keys runs along; it stores zeros
        float slope = 0.0f;
        int qp = 0;
        if (BIAS && live) {
            slope = __ldg(a.slopes + head) * 1.4426950408889634f;
            qp = a.q_pos ? __ldg(a.q_pos + qi) : qi + a.Lk - a.Lq;
        }
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        int first = INT_MAX;  // the first attended key that the gate marked
        for (int kb = kb0; kb < kb1; kb++) {
            const int sl = (kb - kb0) & 1, use = (kb - kb0) >> 1, k0 = kb * MSK_BK;
            const uint32_t tS = tO + 128 + 64 * sl;
            ok = __all_sync(~0u, att_wait(&sh.s_full[t][sl], use & 1));
            if (!ok) break;
            tc_fence_after();
            const bool unseen = k0 >= w_hi1 || k0 + MSK_BK <= w_lo0;  // by any row of the warp
            if (unseen) {
                uint32_t z[16];
#pragma unroll
                for (int e = 0; e < 16; e++) z[e] = 0u;
                tmem_st16(tS, z);
                tmem_st16(tS + 16, z);
            } else {
                float s[MSK_BK];
#pragma unroll
                for (int c = 0; c < 4; c++) tmem_ld16(tS + 16 * c, reinterpret_cast<uint32_t*>(s) + 16 * c);
                tmem_wait_ld();
                const bool partial = k0 < w_lo1 || k0 + MSK_BK > w_hi0;  // warp-uniform: some row hides some key
                const int from = lo - k0, shown = hi - lo;
                if constexpr (CAP) {
                    // s = tanh(cap_in s); where every score that the row sees is below the cap,
                    // as scores mostly are, without the special-function unit, which the
                    // exponentials need (three of its operations per score otherwise).  The
                    // two ways round differently, so each row chooses by its own keys alone.
                    if (partial)
#pragma unroll
                        for (int j = 0; j < MSK_BK; j++)
                            if ((uint32_t)(j - from) >= (uint32_t)shown) s[j] = 0.0f;
                    float big[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < MSK_BK; j++) big[j & 3] = fmaxf(big[j & 3], fabsf(s[j]));
                    const float most = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3])) * a.cap_in;
                    const float2 c2 = make_float2(a.cap_in, a.cap_in);
                    if (most <= 0.35f || !live) {
#pragma unroll
                        for (int j = 0; j < MSK_BK; j += 2) {
                            const float2 y = att_tanh_small(fmul2(make_float2(s[j], s[j + 1]), c2));
                            s[j] = y.x;
                            s[j + 1] = y.y;
                        }
                    } else if (most <= 1.0f) {
#pragma unroll
                        for (int j = 0; j < MSK_BK; j += 2) {
                            const float2 y = att_tanh_poly(fmul2(make_float2(s[j], s[j + 1]), c2));
                            s[j] = y.x;
                            s[j + 1] = y.y;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < MSK_BK; j++) s[j] = att_tanh(s[j] * a.cap_in);
                    }
                }
                if constexpr (BIAS) {
                    const float d = (float)((int64_t)qp - k0), c = CAP ? a.cap_out : ATT_C;
#pragma unroll
                    for (int j = 0; j < MSK_BK; j++) s[j] = fmaf(-slope, fabsf(d - (float)j), s[j] * c);
                }
                if (partial)
#pragma unroll
                    for (int j = 0; j < MSK_BK; j++)
                        if ((uint32_t)(j - from) >= (uint32_t)shown) s[j] = -INFINITY;
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; e++) mx[e] = fmaxf(s[e], s[4 + e]);
#pragma unroll
                for (int j = 8; j < MSK_BK; j += 8)
#pragma unroll
                    for (int e = 0; e < 4; e++) mx[e] = max3f(mx[e], s[j + e], s[j + 4 + e]);
                const float C = BIAS ? 1.0f : CAP ? a.cap_out : ATT_C;
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * C;
                const bool raise = top > m + ATT_RESCALE_LOG2;  // also from -inf; not where all is hidden
                if (__any_sync(~0u, raise)) {
                    const float alpha = raise ? att_ex2(m - top) : 1.0f;  // 0 from -inf
                    const bool had = __any_sync(~0u, raise && m != -INFINITY);  // else those rows of O are zeros
                    if (raise) m = top;
                    l *= alpha;
                    if (had) {
                        // O must hold the blocks before this one
                        ok = __all_sync(~0u, att_wait(&sh.o_done[t][sl ^ 1], ((kb - 1 - kb0) >> 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 8; c++) {
                            uint32_t r[16];
                            tmem_ld16(tO + 16 * c, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; e++) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                            tmem_st16(tO + 16 * c, r);
                        }
                    }
                }
                // P is rounded to f16, the type of V in the same MMA (the rest would double the products); l sums
                // it unrounded.  Over the output this is ~1.1-1.8 2^-13 relative, beside 1.7 2^-13 of an f16 output.
                const float neg = m == -INFINITY ? 0.0f : -m;
                const float2 c2 = make_float2(C, C), n2 = make_float2(neg, neg);
                float2 sum[2];
                sum[0] = sum[1] = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        float2 x = make_float2(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]);
                        x = BIAS ? fadd2(x, n2) : ffma2(x, c2, n2);
                        x.x = att_ex2(x.x);
                        x.y = att_ex2(x.y);
                        sum[e & 1] = fadd2(sum[e & 1], x);
                        pk[e] = pack_h2(x.x, x.y);
                    }
                    tmem_st16(tS + 16 * c, pk);
                }
                const float2 u = fadd2(sum[0], sum[1]);
                l += u.x + u.y;
            }
            if (!unseen && !whole(kb)) {  // V's gate: a marked key of the row's own?
                // (before P is handed over: after that the slot may be refilled)
                if (!__all_sync(~0u, att_wait(&sh.v_ready[vs], vp))) l = NAN;
#pragma unroll 1
                for (int w = 0; w < 2; w++)
                    for (uint32_t f = sh.flags[vs][w]; f; f &= f - 1) {
                        const int key = k0 + 32 * w + __ffs(f) - 1;
                        if ((uint32_t)(key - lo) < (uint32_t)(hi - lo)) first = min(first, key);
                    }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[t][sl]);
            vs += CHAINS;
            if (vs >= v_slots) vs -= v_slots, vp ^= 1;
        }
        // The last P V of this chain.
        auto last = [&](int x) {
            const int i = (x ? t1[1] - t0[1] : t1[0] - t0[0]) - 1;
            return i < 0 || __all_sync(~0u, att_wait(&sh.o_done[x][i & 1], (i >> 1) & 1));
        };
        if (ok) ok = last(t);
        if (ok && __any_sync(~0u, first != INT_MAX)) {
            tc_fence_after();
            msk_lose_columns(tO, first, min(hi, kb1 * MSK_BK), a.v + hk * ATT_DH, a.ldv);
        }
        // O = f O_t (+ fx O_other): halves join their results, in the scale of the larger maximum.
        const bool ran = kb0 < kb1, ran_x = halves && t0[t ^ 1] < t1[t ^ 1];
        float f = 1.0f, fx = 0.0f;
        if (halves) {
            // Each of the two warps that share these rows has waited for its own chain's last P V; what hands
            // the other's O over (and the space of Q and K, which both chains read) is this barrier.  A
            // wait for the other's o_done here could pass early: its phases were not followed.
            sh.ml[t][row] = ran ? make_float2(m, l) : make_float2(-INFINITY, 0.0f);
            tc_fence_after();
            tc_fence_before();
            ok = named_barrier_and(1 + quad, 64, ok);
            tc_fence_after();
            const float2 o = sh.ml[t ^ 1][row];
            if (!ran) m = -INFINITY, l = 0.0f;
            const float top = fmaxf(m, o.x), zero = top == -INFINITY ? 0.0f : top;
            f = att_ex2(m - zero);
            fx = att_ex2(o.x - zero);
            l = l * f + o.y * fx;
            m = top;
        }
        const bool any = some && (ran || ran_x);
        // Without a block: the queries' copy must have landed before their space is used again.
        if (!ran && !ran_x) ok = ok && __all_sync(~0u, att_wait(&sh.q_full, 0));
        if (ok) {
            tc_fence_after();
            const int64_t at = (int64_t)qi * a.H + head;
            const bool split = a.splits > 1;
            const int64_t pat = (int64_t)blockIdx.y * a.Lq * a.H + at;
            const float inv = split ? 1.0f : 1.0f / l;
            f *= inv;
            fx *= inv;
            if (split && live && !(halves && t)) {
                // m = -inf says that the row has no key here.  With keys whose scores are all NaN or -inf the
                // lowest float stands for it: the join then takes the part's l and O, whose NaN the row gets.
                const bool keys = any && lo < B1 * MSK_BK && hi > B0 * MSK_BK;
                a.part_ml[pat] = keys ? make_float2(fmaxf(m, -FLT_MAX), l) : make_float2(-INFINITY, 0.0f);
            }
            // 64 columns at a time (halves: one each) through shared memory (8 KB a warp of the
            // queries' and, with halves, the keys' space, which nothing reads any more), so that a store covers whole
            // lines: 32 rows of 16 bytes keep the store unit busy for 32 cycles.  Rows of 256
            // bytes, 16-byte chunk c of row i at c ^ (i & 15).  Small loops: this code runs once.
            const bool f32 = split || !a.o_f16;
            uint8_t* const buf = sQ + t * ATT_TILE + quad * 8192;
            uint8_t* const out = static_cast<uint8_t*>(split ? static_cast<void*>(a.part) : a.o);
            const int64_t mine = live && !(split && !ran && !ran_x) ? (split ? pat : at) : -1;
            const uint32_t tX = tm + ((uint32_t)(32 * quad) << 16) + 256 * (t ^ 1);
#pragma unroll 1
            for (int g = halves ? t : 0; g < (halves ? t + 1 : 2); g++) {
#pragma unroll 1
                for (int d = 0; d < 4; d++) {
                    float r[16];
                    if (ran) {
                        tmem_ld16(tO + 64 * g + 16 * d, reinterpret_cast<uint32_t*>(r));
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int e = 0; e < 16; e++) r[e] = any && ran ? r[e] * f : 0.0f;
                    if (ran_x) {
                        float y[16];
                        tmem_ld16(tX + 64 * g + 16 * d, reinterpret_cast<uint32_t*>(y));
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e++) r[e] = any ? fmaf(y[e], fx, r[e]) : 0.0f;
                    }
                    auto put = [&](int chunk, uint4 x) {
                        *reinterpret_cast<uint4*>(buf + lane * 256 + ((chunk ^ (lane & 15)) * 16)) = x;
                    };
                    if (f32) {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            put(4 * d + e, make_uint4(__float_as_uint(r[4 * e]), __float_as_uint(r[4 * e + 1]),
                                                      __float_as_uint(r[4 * e + 2]), __float_as_uint(r[4 * e + 3])));
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; e++)
                            put(2 * d + e, make_uint4(pack_h2(r[8 * e], r[8 * e + 1]), pack_h2(r[8 * e + 2], r[8 * e + 3]),
                                                      pack_h2(r[8 * e + 4], r[8 * e + 5]), pack_h2(r[8 * e + 6], r[8 * e + 7])));
                    }
                }
                __syncwarp();
                const int per = f32 ? 16 : 8;  // chunks of a row
#pragma unroll 2
                for (int i = 0; i < per; i++) {
                    const int c = i * 32 + lane, rw = c / per, chunk = c % per;
                    const int64_t to = __shfl_sync(~0u, mine, rw);
                    if (to < 0) continue;
                    *reinterpret_cast<uint4*>(out + (to * 2 + g) * (16 * per) + chunk * 16) =
                        *reinterpret_cast<const uint4*>(buf + rw * 256 + ((chunk ^ (rw & 15)) * 16));
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tm, 256 * CHAINS);
    }
}

// Joins the parts of the key range: o = sum_z 2^(m_z - M) O_z / sum_z 2^(m_z - M) l_z, one
// warp per (query, head); no key at all (every m -inf) gives zeros, keys without a finite score NaN
// (a part with keys has a finite m or +inf, see MaskArgs).
__global__ void __launch_bounds__(128) attention_masked_join_kernel(const float* __restrict__ part,
                                                                    const float2* __restrict__ ml, int64_t rows,
                                                                    int splits, void* __restrict__ o, int o_f16) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (at >= rows) return;
    float M = -INFINITY;
    for (int z = lane; z < splits; z += 32) M = fmaxf(M, ml[z * rows + at].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, d));
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    for (int z0 = 0; z0 < splits; z0 += 32) {
        // lane z: the part's weight, -1 where it has no key of the row (a weight that underflows
        // still takes its O: a NaN or an infinity there makes the row one)
        const int z = z0 + lane;
        const float2 x = z < splits ? ml[z * rows + at] : make_float2(-INFINITY, 0.0f);
        const float w = x.x == -INFINITY ? -1.0f : att_ex2(x.x - M);
        l = fmaf(fmaxf(w, 0.0f), x.y, l);
        for (int j = 0; j < min(32, splits - z0); j += 8) {  // eight loads in flight
            float4 p[8];
            float wj[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                wj[e] = __shfl_sync(~0u, w, j + e);
                p[e] = !(wj[e] < 0.0f) ? reinterpret_cast<const float4*>(part + ((z0 + j + e) * rows + at) * ATT_DH)[lane]
                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int e = 0; e < 8; e++) {
                acc.x = fmaf(wj[e], p[e].x, acc.x);
                acc.y = fmaf(wj[e], p[e].y, acc.y);
                acc.z = fmaf(wj[e], p[e].z, acc.z);
                acc.w = fmaf(wj[e], p[e].w, acc.w);
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
    const float inv = M == -INFINITY ? 0.0f : 1.0f / l;
    if (o_f16)
        reinterpret_cast<uint2*>(static_cast<__half*>(o) + at * ATT_DH)[lane] =
            make_uint2(pack_h2(acc.x * inv, acc.y * inv), pack_h2(acc.z * inv, acc.w * inv));
    else
        reinterpret_cast<float4*>(static_cast<float*>(o) + at * ATT_DH)[lane] =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
}

}  // namespace dllm
