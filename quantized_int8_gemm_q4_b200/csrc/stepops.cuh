// Entry points of the operators between the projections of a step: dllm_rope_turns,
// dllm_qk_rope, dllm_attention_masked and dllm_sample.  Part of dllm.cu (it uses its launch
// and device helpers).
#pragma once
#include <cmath>

#include "attmask.cuh"
#include "rope.cuh"
#include "sample.cuh"

namespace {

template <int G>
cudaError_t launch_rope(const RopeArgs& a, dim3 grid, bool neox, cudaStream_t s) {
    return neox ? launch_pdl(qk_rope_kernel<G, true>, grid, dim3(ROPE_THREADS), 0, s, a)
                : launch_pdl(qk_rope_kernel<G, false>, grid, dim3(ROPE_THREADS), 0, s, a);
}

bool g_sample_attr_done[MAX_DEV], g_sample_cluster16[MAX_DEV];

int status_of(cudaError_t e) {
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return DLLM_ERR_CUDA;
    }
    return launch_status();
}

// A [rows][heads][128] f16 tensor with rows `ld` values apart as the 3-D tensor (head dim,
// head, row), 128-byte swizzled boxes of 64 head-dim values.  Encoded on every call: a map
// kept by address would outlive the buffer it describes.
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t heads, int64_t ld, int box_heads,
                 int box_rows) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)ATT_DH, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)ATT_DH * 2, (cuuint64_t)(ld * 2)};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct MaskPlan {
    int gp, tq, splits;
    bool halves;
    int64_t grid;
    size_t ml_off, bytes;
};

// CTAs and key parts of a masked attention call.  Two CTAs share an SM once there are more tiles
// than SMs; else each has an SM and two chains of blocks; with at most half a wave of those the
// keys are cut into parts, up to one wave in all.  The intervals lie on the device, so the plan goes
// by Lk: what a tile does see is dealt out over as many parts (one query of 32 heads with a window of
// 1401 in 20011 keys 12.3 us; over a cache cut to the window fewer parts would do).
MaskPlan mask_plan(int64_t Lq, int64_t Lk, int64_t H, int64_t Hkv, int sms) {
    MaskPlan p;
    const int group = (int)(H / Hkv);
    p.gp = group < 128 ? group : 128;
    while (group % p.gp) p.gp--;
    p.tq = 128 / p.gp;
    const int64_t n_heads = H / p.gp, n_tiles = (Lq + p.tq - 1) / p.tq, blocks = (Lk + MSK_BK - 1) / MSK_BK;
    p.grid = n_tiles * n_heads;
    p.halves = p.grid <= sms;
    p.splits = 1;
    if (2 * p.grid <= sms && blocks >= 12) {
        // n parts take ~0.45 us blocks / n for their chains and 0.18 us n for the join, least at
        // n^2 = 2.5 blocks (one query of 28 heads on 4: 1000 keys 2 parts 11.9 us, 5 10.1; 8200 keys
        // 16 parts 16.9, 32 18.0)
        const int64_t most = sms / p.grid;
        int64_t n = most < blocks / 3 ? most : blocks / 3;
        while (2 * n * n > 5 * blocks) n--;
        p.splits = (int)n;
        // One part per SM can leave SMs without work (32 tiles on 148 SMs: 20), two CTAs per SM in parts of
        // half the length fewer.  That saves each SM 0.75 us per block, its share of HBM, and costs 0.45 us
        // per further part, up to 1.1 us where a part has all 128 rows to write and join.  One query, one against
        // two per SM: 32 heads, 4000 keys 19.6 and 21.3 us, 10000 34.6 and 34.9, 14500 45.8 and 44.9, 60000 163.8
        // and 147.6; 22 heads, 20011 keys 43.9 and 44.4, 30000 60.8 and 60.1; 40 heads, 2500 keys 18.6 and
        // 19.0, 4000 23.6 and 23.4, 10000 43.3 and 39.7; 50 heads, 2500 keys 24.1 and 21.3.  128 queries of 32
        // heads, 14000 keys 48.0 and 50.7, 20011 68.7 and 66.9.  (8 tiles, which leave 4 SMs idle, 60000 keys
        // 49.4 and 54.6.)
        const int64_t more = 2 * sms / p.grid;
        const double saved = (double)blocks / most - 2.0 * blocks / more;
        const double rows = (double)(Lq < p.tq ? Lq : p.tq) * p.gp;
        if (n == most && saved > (0.6 + rows / 140) * (double)(more - most))
            p.halves = false, p.splits = (int)more;
    }
    p.ml_off = p.bytes = 0;
    if (p.splits > 1) {
        p.ml_off = align256((size_t)p.splits * Lq * H * ATT_DH * 4);
        p.bytes = p.ml_off + align256((size_t)p.splits * Lq * H * 8);
    }
    return p;
}

bool g_mask_attr_done[MAX_DEV];

typedef void (*MaskKernel)(CUtensorMap, CUtensorMap, CUtensorMap, MaskArgs);

template <int MODE>
bool mask_attribute() {
    cudaFuncAttributes fa;
    return cudaFuncSetAttribute(attention_masked_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)msk_smem(MODE & 4)) == cudaSuccess &&
           cudaFuncGetAttributes(&fa, attention_masked_kernel<MODE>) == cudaSuccess &&
           fa.numRegs >= msk_reg_launch(MODE & 4);  // the warpgroups' setmaxnreg split must fit in the launch's registers
}

bool mask_attributes(int dev) {
    if (!g_mask_attr_done[dev])
        g_mask_attr_done[dev] = mask_attribute<0>() && mask_attribute<1>() && mask_attribute<2>() && mask_attribute<3>() &&
                                mask_attribute<4>() && mask_attribute<5>() && mask_attribute<6>() && mask_attribute<7>();
    return g_mask_attr_done[dev];
}

}  // namespace

extern "C" {

int dllm_rope_turns(int64_t n_rot, double base, dllm_rope_scaling kind, double factor, double trained_len,
                    double beta_fast, double beta_slow, double* turns, float* mscale) {
    if (n_rot < 0 || n_rot % 2 || n_rot > 65536 || !(base > 1.0) || !(base < INFINITY) || !mscale) return DLLM_ERR_ARG;
    if (n_rot > 0 && !turns) return DLLM_ERR_ARG;
    if (kind != DLLM_ROPE_PLAIN && (!(factor > 0.0) || !(factor < INFINITY))) return DLLM_ERR_ARG;
    const double two_pi = 6.283185307179586476925;
    double lo = 0.0, span = 1.0;
    *mscale = 1.0f;
    switch (kind) {
        case DLLM_ROPE_PLAIN:
        case DLLM_ROPE_LINEAR: break;
        case DLLM_ROPE_NTK:
            if (n_rot == 2) return DLLM_ERR_ARG;  // n / (n - 2)
            if (n_rot > 2) base *= std::pow(factor, (double)n_rot / (double)(n_rot - 2));
            if (!(base > 0.0) || !(base < INFINITY)) return DLLM_ERR_ARG;
            break;
        case DLLM_ROPE_YARN: {
            if (!(trained_len > 0.0) || !(trained_len < INFINITY) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
                !(beta_fast < INFINITY))
                return DLLM_ERR_ARG;
            auto dim = [&](double beta) { return 0.5 * n_rot * std::log(trained_len / (beta * two_pi)) / std::log(base); };
            lo = std::fmax(std::floor(dim(beta_fast)), 0.0);
            const double hi = std::fmin(std::ceil(dim(beta_slow)), (double)n_rot - 1.0);
            span = std::fmax(hi - lo, 0.001);
            if (factor > 1.0) *mscale = (float)(0.1 * std::log(factor) + 1.0);
            break;
        }
        default: return DLLM_ERR_ARG;
    }
    for (int64_t i = 0; i < n_rot / 2; i++) {
        double f = std::pow(base, -2.0 * (double)i / (double)n_rot);
        if (kind == DLLM_ROPE_LINEAR) f /= factor;
        if (kind == DLLM_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax(((double)i - lo) / span, 0.0), 1.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        turns[i] = f / two_pi;
    }
    return DLLM_OK;
}

int dllm_qk_rope(const float* q, int64_t ldq, const float* k, int64_t ldk, const float* v, int64_t ldv, int64_t L,
                 int64_t H, int64_t Hkv, int64_t dh, const int32_t* pos, const double* turns, int64_t n_rot,
                 dllm_rope_layout layout, float mscale, const float* gamma_q, const float* gamma_k, float eps,
                 void* oq, void* ok, void* ov, dllm_stream_t stream) {
    if (L < 0 || H <= 0 || Hkv <= 0 || dh <= 0 || dh > 256 || dh % 8 || n_rot < 0 || n_rot > dh || n_rot % 8)
        return DLLM_ERR_ARG;
    if (layout != DLLM_ROPE_NORM && layout != DLLM_ROPE_NEOX) return DLLM_ERR_ARG;
    if (H > 65535 || Hkv > 65535 || L > (1LL << 31) - 1) return DLLM_ERR_ARG;
    if (ldq < H * dh || ldk < Hkv * dh || (v && ldv < Hkv * dh)) return DLLM_ERR_ARG;
    if (!(std::fabs(mscale) < INFINITY)) return DLLM_ERR_ARG;
    if ((gamma_q || gamma_k) && (!(eps > 0.0f) || !(eps < INFINITY))) return DLLM_ERR_ARG;
    if (L == 0) return DLLM_OK;
    if (!q || !k || !oq || !ok || (v && !ov) || (n_rot > 0 && !turns)) return DLLM_ERR_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(oq) || !aligned16(ok) || (v && !aligned16(ov)) ||
        !aligned16(pos) || !aligned16(turns) || !aligned16(gamma_q) || !aligned16(gamma_k) || ldq % 4 || ldk % 4 ||
        (v && ldv % 4))
        return DLLM_ERR_ALIGN;
    int dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    RopeArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q, a.k = k, a.v = v;
    a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
    a.L = L;
    a.H = (int32_t)H, a.Hkv = (int32_t)Hkv, a.T = (int32_t)(H + Hkv * (v ? 2 : 1));
    a.dh = (int32_t)dh, a.n_rot = (int32_t)n_rot;
    a.pos = pos, a.turns = turns;
    a.ms = mscale, a.eps = eps;
    a.gq = gamma_q, a.gk = gamma_k;
    a.oq = static_cast<__half*>(oq), a.ok = static_cast<__half*>(ok), a.ov = static_cast<__half*>(ov);
    const int G = dh <= 64 ? 8 : dh <= 128 ? 16 : 32;
    // Heads per CTA: one per lane group while the CTAs of all tokens fit one wave of full
    // SMs (8 of 256 threads each), else all of a token's, whose angles are then formed once.
    const int slots = ROPE_THREADS / G;
    const int64_t parts = (a.T + slots - 1) / slots;
    a.chunk = L * parts <= 8LL * g_num_sms[dev] ? slots : a.T;
    const dim3 grid((unsigned)L, (unsigned)((a.T + a.chunk - 1) / a.chunk));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool neox = layout == DLLM_ROPE_NEOX;
    return status_of(G == 8 ? launch_rope<8>(a, grid, neox, s) : G == 16 ? launch_rope<16>(a, grid, neox, s)
                                                                          : launch_rope<32>(a, grid, neox, s));
}

int dllm_attention_masked_workspace_bytes(int64_t Lq, int64_t Lk, int64_t H, int64_t Hkv, size_t* bytes) {
    if (Lq < 0 || Lk < 0 || Lq > (1LL << 30) || Lk > (1LL << 30) || H <= 0 || H > 65535 || Hkv <= 0 || H % Hkv || !bytes)
        return DLLM_ERR_ARG;
    int dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    *bytes = mask_plan(Lq, Lk, H, Hkv, g_num_sms[dev]).bytes;
    return DLLM_OK;
}

int dllm_attention_masked(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                          int64_t Lq, int64_t Lk, int64_t H, int64_t Hkv, int64_t dh, const int32_t* kv_begin,
                          const int32_t* kv_end, const int32_t* q_pos, float softcap, const float* slopes, void* o,
                          dllm_ftype o_type, void* workspace, size_t workspace_bytes, dllm_stream_t stream) {
    if (Lq < 0 || Lk < 0 || H <= 0 || Hkv <= 0 || H % Hkv || dh != ATT_DH) return DLLM_ERR_ARG;
    if (o_type != DLLM_F32 && o_type != DLLM_F16) return DLLM_ERR_ARG;
    // a cap whose reciprocal or base-2 form leaves f32 is refused
    if (softcap != 0.0f && !(softcap >= 0x1p-100f && softcap <= 0x1p100f)) return DLLM_ERR_ARG;
    if (Lq > (1LL << 30) || Lk > (1LL << 30) || H > 65535) return DLLM_ERR_ARG;
    if (ldq < H * dh || ldk < Hkv * dh || ldv < Hkv * dh) return DLLM_ERR_ARG;
    if (ldq >= (1LL << 39) || ldk >= (1LL << 39) || ldv >= (1LL << 39)) return DLLM_ERR_ARG;  // tensor-map strides
    if (Lq == 0) return DLLM_OK;
    if (!q || !o || (Lk > 0 && (!k || !v))) return DLLM_ERR_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(kv_begin) ||
        !aligned16(kv_end) || !aligned16(q_pos) || !aligned16(slopes) || !aligned16(workspace) || ldq % 8 || ldk % 8 ||
        ldv % 8)
        return DLLM_ERR_ALIGN;
    int dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (Lk == 0)
        return status_of(cudaMemsetAsync(o, 0, (size_t)(Lq * H * dh) * (o_type == DLLM_F16 ? 2 : 4), s));
    const MaskPlan p = mask_plan(Lq, Lk, H, Hkv, g_num_sms[dev]);
    if (p.grid > (1LL << 31) - 1) return DLLM_ERR_ARG;
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return DLLM_ERR_WORKSPACE;
    if (!mask_attributes(dev)) return DLLM_ERR_CUDA;
    CUtensorMap tq, tk, tv;
    if (!encode_rows(&tq, q, Lq, H, ldq, p.gp, p.tq) || !encode_rows(&tk, k, Lk, Hkv, ldk, 1, MSK_BK) ||
        !encode_rows(&tv, v, Lk, Hkv, ldv, 1, MSK_BK))
        return DLLM_ERR_CUDA;
    MaskArgs a;
    memset(&a, 0, sizeof(a));
    a.Lq = (int32_t)Lq, a.Lk = (int32_t)Lk, a.H = (int32_t)H, a.group = (int32_t)(H / Hkv);
    a.gp = p.gp, a.tq = p.tq, a.splits = p.splits;
    a.kv_begin = kv_begin, a.kv_end = kv_end, a.q_pos = q_pos;
    a.v = static_cast<const __half*>(v), a.ldv = ldv;
    const double scale = 0.08838834764831844, log2e = 1.4426950408889634;  // 1 / sqrt(128)
    a.cap_in = softcap > 0.0f ? (float)(scale / softcap) : 0.0f;
    a.cap_out = (float)(softcap * log2e);
    a.slopes = slopes;
    a.o = o;
    a.o_f16 = o_type == DLLM_F16;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.ml_off);
    const dim3 grid((unsigned)p.grid, (unsigned)p.splits);
    static const MaskKernel kernels[8] = {attention_masked_kernel<0>, attention_masked_kernel<1>, attention_masked_kernel<2>,
                                          attention_masked_kernel<3>, attention_masked_kernel<4>, attention_masked_kernel<5>,
                                          attention_masked_kernel<6>, attention_masked_kernel<7>};
    const MaskKernel kernel = kernels[(softcap > 0.0f ? 1 : 0) + (slopes ? 2 : 0) + (p.halves ? 4 : 0)];
    rc = status_of(launch_pdl(kernel, grid, dim3(msk_threads(p.halves)), msk_smem(p.halves), s, tq, tk, tv, a));
    if (rc || p.splits == 1) return rc;
    return status_of(launch_pdl(attention_masked_join_kernel, dim3((unsigned)((Lq * H + 3) / 4)), dim3(128), 0, s, a.part,
                                a.part_ml, Lq * H, p.splits, o, a.o_f16));
}

int dllm_sample(const float* logits, int64_t R, int64_t V, int64_t ldl, const float* temperature, const int32_t* top_k,
                const float* top_p, const float* min_p, const float* u, int32_t* token, float* conf, float* entropy,
                dllm_stream_t stream) {
    if (R < 0 || V <= 0 || V > (1LL << 31) - 64 || ldl < V || R > (1LL << 27)) return DLLM_ERR_ARG;
    if (R == 0) return DLLM_OK;
    if (!logits || !token) return DLLM_ERR_ARG;
    const void* ptrs[] = {logits, temperature, top_k, top_p, min_p, u, token, conf, entropy};
    for (const void* p : ptrs)
        if (!aligned16(p)) return DLLM_ERR_ALIGN;
    int dev;
    int rc = current_device(&dev);
    if (rc) return rc;
    const size_t most = 227 * 1024;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.blockDim = dim3(SMP_THREADS);
    if (!g_sample_attr_done[dev]) {
        if (cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess ||
            cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return DLLM_ERR_CUDA;
        // clusters of 16 are not portable: asked for only where the device can hold one
        cfg.gridDim = dim3(SMP_MAX_CLUSTER);
        cfg.dynamicSmemBytes = most;
        cfg.numAttrs = 1;
        attr[0].val.clusterDim.x = SMP_MAX_CLUSTER;
        int n = 0;
        g_sample_cluster16[dev] = cudaOccupancyMaxActiveClusters(&n, sample_kernel, &cfg) == cudaSuccess && n > 0;
        (void)cudaGetLastError();
        g_sample_attr_done[dev] = true;
    }
    SampleArgs a;
    memset(&a, 0, sizeof(a));
    a.logits = logits;
    a.V = V, a.ldl = ldl;
    a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p, a.u = u;
    a.token = token, a.conf = conf, a.entropy = entropy;
    // CTAs per row: about 8192 elements each, up to 8 (up to 16 for a few rows of a large
    // vocabulary, 22 -> 15 us for one of 152064 words).
    int C = 1;
    while (C < 8 && (int64_t)C * 8192 < V) C *= 2;
    if (C == 8 && 16 * R <= g_num_sms[dev] && g_sample_cluster16[dev]) C = 16;
    a.slice = (int32_t)round_up((V + 3 + C - 1) / C, 128);
    // Two CTAs per SM where at least 3/4 of a slice then fits in shared memory (the rest is
    // read again from L2), else one.  113 KB and the system's 1 KB per CTA twice are an SM's 228 KB.
    const int64_t pair = (int64_t)((113 * 1024 - sizeof(SampleShared)) / 16 * 4);
    const int64_t room = 4 * pair >= 3 * (int64_t)a.slice ? pair : (int64_t)((most - sizeof(SampleShared)) / 16 * 4);
    a.cached = (int32_t)(a.slice < room ? a.slice : room);
    int bits = 0;
    while ((1LL << bits) < V) bits++;
    a.fix = 62 - bits < 51 ? 62 - bits : 51;
    cfg.gridDim = dim3((unsigned)(C * R));
    cfg.dynamicSmemBytes = sizeof(SampleShared) + (size_t)a.cached * 4;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.numAttrs = 2;
    attr[0].val.clusterDim.x = (unsigned)C;
    return status_of(cudaLaunchKernelEx(&cfg, sample_kernel, a));
}

}  // extern "C"
