// tw_postnorm.cu -- the fused step of a layer with sandwich norms: a norm of
// the block's output, its gate and scales between the reduce and the residual
// add.  Per token, in fp32:
//   s = sum_r partials[r]              ranks in order
//   u = s / sqrt(mean s^2 + post_eps) * post_weight
//   x = residual_scale * residual + block_scale * gate * u
//   residual_out = x,  out[k] = x / sqrt(mean x^2 + eps) * weight
// Two reductions over the row, the second on what the first gives: the row
// stays in registers for both.  (One pass over sums of s^2, r^2, r v and v^2
// would give mean x^2 too, but loses it to cancellation where the block's output
// and the residual nearly cancel.)  Bound by HBM: n_parts + 1 rows (and a gate's) in,
// n_out + 1 out.  These kernels serve few tokens (a cluster of eight CTAs to a token)
// and short rows (a CTA or less to a row); many tokens with long rows stream through
// a ring (tw_postnorm_rows.cu).  Few tokens are bound by their chain of latencies: the
// launch, one load, two exchanges (8 x 1 x 8192 bf16 2.8 us, 64 tokens 4.7; the step
// with one norm 2.5 and 4.1).
#include "tw_tcgen05.cuh"

namespace tw {
namespace {

constexpr int kThreads = 256;         // per CTA where a row has CTAs to itself
constexpr int kClusterCta = 128;      // per CTA where a row has a cluster

__device__ __forceinline__ uint32_t cluster_cta_count() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The start-up barrier of a cluster in two halves: every CTA must be running
// before any writes into its shared memory.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// Write a float into CTA `rank`'s shared memory, at `local`'s place in this one's.
__device__ __forceinline__ void st_peer_f32(float* local, uint32_t rank, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_rank(smem_addr(local), rank)),
                 "f"(v)
                 : "memory");
}

// MANY: three or four CTAs share an SM: fewer partials in flight a thread, the weights read
// when they are needed (2 x 4096 x 1024 11.9 -> 9.4 us, 8 x 2048 x 1024 10.7 -> 8.9, 2 x
// 16000 x 256 11.0 -> 9.6; but where two on an SM are enough 2 x 1000 x 1024 3.6 -> 4.2).
__host__ __device__ constexpr int many_ctas(int vpt) { return vpt == 3 ? 3 : 4; }

// VPT: 16-byte vectors of the row per thread; W: warps per row (of a CTA, where a
// cluster of CTAs shares the row: CL).
template <typename T, int VPT, int W, bool CL, bool Q8, bool MANY = false>
__global__ void __launch_bounds__(CL ? kClusterCta : kThreads, MANY ? many_ctas(VPT) : 0)
    postnorm_kernel(const __grid_constant__ PostParams pp) {
    using V = Vec<T>;
    constexpr int E = V::kElems;
    constexpr int kWarps = (CL ? kClusterCta : kThreads) / 32;
    constexpr int kRows = kWarps / W;
    // Rows of partials whose loads are in flight at once.
    constexpr int kAhead = MANY && VPT < 3 ? 4 / VPT : 8 / VPT;
    constexpr bool kEarly = VPT <= 2 && !MANY;
    constexpr bool kLate = MANY && VPT < 3;
    const Params& p = pp.p;
    // Warp totals: [second reduction][buffer][warp], of sums and of maxima.
    __shared__ float warp_part[2][2][kWarps];
    __shared__ float warp_max[Q8 ? 2 : 1][kWarps];
    // The CTAs' totals, written into every CTA of the cluster.
    __shared__ float cta_part[CL ? 2 : 1][2][kClusterMaxSize];
    __shared__ float cta_max[CL && Q8 ? 2 : 1][kClusterMaxSize];

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int slot = warp / W;                     // row of the CTA
    const int rtid = threadIdx.x - slot * W * 32;  // thread of the row
    uint32_t crank = 0, csize = 1;
    if constexpr (CL) {
        crank = cluster_cta_rank();
        csize = cluster_cta_count();
    }
    const int nvec = static_cast<int>(p.row_bytes / 16);
    const int per_cta = CL ? (nvec + static_cast<int>(csize) - 1) / static_cast<int>(csize) : nvec;
    const int v_begin = static_cast<int>(crank) * per_cta;
    const int v_end = v_begin + per_cta < nvec ? v_begin + per_cta : nvec;
    const int64_t step = CL ? static_cast<int64_t>(gridDim.x / csize)
                            : static_cast<int64_t>(gridDim.x) * kRows;
    int64_t t = p.t0 + (CL ? static_cast<int64_t>(blockIdx.x / csize)
                           : static_cast<int64_t>(blockIdx.x) * kRows + slot);
    // The first token on its way into L2 while the launch before this one ends (a hint
    // that reads nothing: what that launch writes is seen all the same).
    if (p.prefetch && rtid == 0 && t < p.t1 && v_begin < v_end) {
        const int64_t off = t * p.row_bytes + static_cast<int64_t>(v_begin) * 16;
        const auto bytes = static_cast<uint32_t>((v_end - v_begin) * 16);
        for (int r = 0; r < p.n_parts; ++r)
            bulk_prefetch_l2(static_cast<const char*>(p.partials[r]) + off, bytes);
        bulk_prefetch_l2(static_cast<const char*>(p.residual) + off, bytes);
    }
    if constexpr (CL) cluster_arrive_relaxed();
    grid_dependency_wait();
    grid_launch_dependents();
    bool peers_started = false;
    int buf = 0;

    // Sum (and maximum) of the row over its threads; `which`: 0 the block's
    // norm, 1 the layer's.  Buffers alternate by row, so that a row's totals are
    // read before any thread can be two rows on.
    auto reduce = [&](int which, float v, float m, float* most) {
        v = warp_sum(v);
        if (Q8 && which) m = warp_max_abs(m);
        if constexpr (W > 1 || CL) {
            if (lane == 0) {
                warp_part[which][buf][warp] = v;
                if (Q8 && which) warp_max[Q8 ? buf : 0][warp] = m;
            }
            if constexpr (CL || W == kWarps)
                __syncthreads();
            else
                named_barrier(1 + slot, W * 32);
            v = 0.f;
            m = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                v += warp_part[which][buf][slot * W + w];
                if (Q8 && which) m = max_abs(m, warp_max[Q8 ? buf : 0][slot * W + w]);
            }
        }
        if constexpr (CL) {
            if (!peers_started) {
                cluster_wait();
                peers_started = true;
            }
            // Every CTA gets every total and adds them in rank order.
            if (threadIdx.x < csize) {
                st_peer_f32(&cta_part[which][buf][crank], threadIdx.x, v);
                if (Q8 && which) st_peer_f32(&cta_max[Q8 ? buf : 0][crank], threadIdx.x, m);
            }
            cluster_barrier();
            v = 0.f;
            m = 0.f;
            for (uint32_t r = 0; r < csize; ++r) {
                v += cta_part[which][buf][r];
                if (Q8 && which) m = max_abs(m, cta_max[Q8 ? buf : 0][r]);
            }
        }
        *most = m;
        return v;
    };

    // A group of warps takes its rows on its own; a CTA's groups that share a
    // barrier (W == kWarps) are one.
    for (; t < p.t1; t += step, buf ^= 1) {
        const int64_t row_off = t * p.row_bytes;
        // What the sum does not need is on its way beside it, the weights too where there
        // are registers for them; where other CTAs hide its latency, only behind it (2 x
        // 4096 x 1024 9.4 -> 9.0 us, 4 x 2000 x 1504 10.8 -> 9.6; 10 KB rows 9.8 -> 10.7).
        uint4 res[VPT], gate[VPT], pw[VPT], wv[VPT];
        const char* gate_row =
            pp.gate ? static_cast<const char*>(pp.gate) + t / pp.gate_tokens * p.row_bytes
                    : nullptr;
        auto load = [&](const void* row, int k) {
            const int v = v_begin + rtid + k * W * 32;
            return row && v < v_end ? ld_global(static_cast<const char*>(row) +
                                                static_cast<int64_t>(v) * 16)
                                    : make_uint4(0, 0, 0, 0);
        };
        auto load_beside = [&]() {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                res[k] = load(static_cast<const char*>(p.residual) + row_off, k);
                gate[k] = load(gate_row, k);
            }
        };
        if constexpr (!kLate) load_beside();
        if constexpr (kEarly) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                pw[k] = load(pp.post_weight, k);
                wv[k] = load(p.weight, k);
            }
        }
        float s[VPT][E];
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) s[k][e] = 0.f;
        for (int r0 = 0; r0 < p.n_parts; r0 += kAhead) {
            uint4 raw[kAhead][VPT];
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int v = v_begin + rtid + k * W * 32;
                    if (r0 + a < p.n_parts && v < v_end)
                        raw[a][k] = ld_global_nc(static_cast<const char*>(p.partials[r0 + a]) +
                                                 row_off + static_cast<int64_t>(v) * 16);
                }
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (r0 + a < p.n_parts && v_begin + rtid + k * W * 32 < v_end)
                        add_vec(s[k], raw[a][k], static_cast<T*>(nullptr));
        }
        if constexpr (kLate) load_beside();
        float c = 1.f, most = 0.f;
        if (pp.post_weight) {
            float ss2[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < VPT; ++k) sum_squares<E>(ss2, s[k]);
            const float total = reduce(0, ss2[0] + ss2[1], 0.f, &most);
            c = rsqrtf(total * p.inv_H + pp.post_eps);
        }
        float ss2[2] = {0.f, 0.f}, m = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float f[E];
            if (pp.post_weight) {
                V::to_float(kEarly ? pw[k] : load(pp.post_weight, k), f);
#pragma unroll
                for (int e = 0; e < E; ++e) s[k][e] = s[k][e] * c * f[e];
            }
            if (gate_row) {
                V::to_float(gate[k], f);
#pragma unroll
                for (int e = 0; e < E; ++e) s[k][e] *= f[e];
            }
            V::to_float(res[k], f);
#pragma unroll
            for (int e = 0; e < E; ++e)
                s[k][e] = fmaf(pp.block_scale, s[k][e], pp.residual_scale * f[e]);
            sum_squares<E>(ss2, s[k]);
            if constexpr (!kEarly) wv[k] = load(p.weight, k);
            if constexpr (Q8) m = max_abs_product<T>(m, s[k], wv[k]);
        }
        const float total = reduce(1, ss2[0] + ss2[1], m, &most);
        const float inv = rsqrtf(total * p.inv_H + p.eps);
        [[maybe_unused]] RowQuant rq;
        if constexpr (Q8) {
            rq = RowQuant(most, inv, quant_top(p.qtype));
            if (crank == 0 && rtid < p.n_out)
                p.out_scale[rtid][t] = row_scale(rq.y, quant_top(p.qtype), rq.zero);
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = v_begin + rtid + k * W * 32;
            if (v >= v_end) continue;
            const int64_t off = row_off + static_cast<int64_t>(v) * 16;
            st_global_cs(static_cast<char*>(p.residual_out) + off, V::from_float(s[k]));
            float w[E], y[E];
            V::to_float(wv[k], w);
            if constexpr (Q8) {
#pragma unroll
                for (int e = 0; e < E; e += 2) mul2(y + e, s[k] + e, w + e);
                store_q8<E>(p.out, p.n_out, t * p.H + static_cast<int64_t>(v) * E, y, rq, p.qtype);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = (s[k][e] * inv) * w[e];
                const uint4 packed = V::from_float(y);
                for (int o = 0; o < p.n_out; ++o)
                    st_global_cs(static_cast<char*>(p.out[o]) + off, packed);
            }
        }
    }
    // A CTA with no token still completes the start-up barrier.
    if constexpr (CL)
        if (!peers_started) cluster_wait();
}

template <typename T, bool Q8>
void* postnorm_rows_entry(int vpt, int w, bool many) {
    if (many)
        return vpt == 3   ? reinterpret_cast<void*>(&postnorm_kernel<T, 3, 8, false, Q8, true>)
               : w == 8   ? reinterpret_cast<void*>(&postnorm_kernel<T, 2, 8, false, Q8, true>)
               : w == 4   ? reinterpret_cast<void*>(&postnorm_kernel<T, 2, 4, false, Q8, true>)
               : w == 2   ? reinterpret_cast<void*>(&postnorm_kernel<T, 2, 2, false, Q8, true>)
               : vpt == 2 ? reinterpret_cast<void*>(&postnorm_kernel<T, 2, 1, false, Q8, true>)
                          : reinterpret_cast<void*>(&postnorm_kernel<T, 1, 1, false, Q8, true>);
    switch (w * 16 + vpt) {
        case 1 * 16 + 1: return reinterpret_cast<void*>(&postnorm_kernel<T, 1, 1, false, Q8>);
        case 1 * 16 + 2: return reinterpret_cast<void*>(&postnorm_kernel<T, 2, 1, false, Q8>);
        case 2 * 16 + 2: return reinterpret_cast<void*>(&postnorm_kernel<T, 2, 2, false, Q8>);
        case 4 * 16 + 2: return reinterpret_cast<void*>(&postnorm_kernel<T, 2, 4, false, Q8>);
        case 8 * 16 + 2: return reinterpret_cast<void*>(&postnorm_kernel<T, 2, 8, false, Q8>);
        default: return nullptr;
    }
}

template <typename T, bool Q8>
void* postnorm_cluster_entry(int vpt) {
    switch (vpt) {
        case 1: return reinterpret_cast<void*>(&postnorm_kernel<T, 1, 4, true, Q8>);
        case 2: return reinterpret_cast<void*>(&postnorm_kernel<T, 2, 4, true, Q8>);
        case 4: return reinterpret_cast<void*>(&postnorm_kernel<T, 4, 4, true, Q8>);
        default: return nullptr;
    }
}

// The instantiation for vpt vectors per thread and w warps per row (0: a cluster), many
// rows or few.
void* postnorm_kernel_for(int dtype, int vpt, int w, bool q8, bool many = false) {
    if (dtype == TW_BF16) {
        using T = __nv_bfloat16;
        if (w == 0) return q8 ? postnorm_cluster_entry<T, true>(vpt)
                              : postnorm_cluster_entry<T, false>(vpt);
        return q8 ? postnorm_rows_entry<T, true>(vpt, w, many)
                  : postnorm_rows_entry<T, false>(vpt, w, many);
    }
    if (w == 0) return q8 ? postnorm_cluster_entry<float, true>(vpt)
                          : postnorm_cluster_entry<float, false>(vpt);
    return q8 ? postnorm_rows_entry<float, true>(vpt, w, many)
              : postnorm_rows_entry<float, false>(vpt, w, many);
}

// Warps per row and vectors per thread for rows of nvec <= 768 vectors.
void rows_shape(int64_t nvec, int* vpt, int* w) {
    *w = 1;
    *vpt = nvec <= 32 ? 1 : 2;
    while (*w < 8 && nvec > static_cast<int64_t>(*w) * 32 * *vpt) *w *= 2;
    if (nvec > static_cast<int64_t>(*w) * 32 * *vpt) *vpt = 3;
}

// Which kernel (us, 8 partials bf16: cluster / this file's rows / ring):
//   rows above 8 KB  a cluster per token while all of them run at once (1 x 8192 2.8 / 4.6
//                    / 5.5, 100 x 8192 5.4 / 7.3 / 6.6, 128 x 8192 8.6 / - / 7.1)
//   rows to 12 KB    this file's, a CTA or less per row, while all CTAs run at once: four
//                    on an SM (1 x 4096 - / 2.8 / -, 500 x 4096 - / 8.7 / 10.4, 2 x 1000 x
//                    2048 - / 4.8 / 6.1), above 8 KB three (400 x 5120 - / 9.8 / 11.1; with
//                    16 KB it would be two, 256 x 8192 - / 10.4 / 10.1); rows
//                    below 4 KB always (1000 x 256 - / 2.5 / 7.5, 2 x 4096 x 1024 - / 9.0 / 10.7)
//   everything else  the ring kernel's bulk copies (1024 x 8192 - / 38.3 / 28.9, 1000 x 4096 - /
//                    18.4 / 15.8)
// Under a budget each CTA is alone on its SM: few rows to each, to 8 KB, go without the ring.
constexpr int64_t kShortRowBytes = 4096, kRowsRowBytes = 8192, kLongestRowBytes = 12288;

cudaLaunchConfig_t cluster_config(int cluster, int64_t tokens, size_t smem, bool pdl, void* stream,
                                  cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster * tokens));
    cfg.blockDim = dim3(kClusterCta);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cfg;
}

}  // namespace

int postnorm_prepare(int smem_optin, int (*clusters)[3][2]) {
    if (smem_optin < kExclusiveSmemBytes + 2048) return static_cast<int>(cudaErrorInvalidValue);
    // (Which also loads them, those for many rows too, whose launches ask for no shared memory.)
    for (int dt = 0; dt < 2; ++dt)
        for (int w = 0; w <= 8; w = w ? 2 * w : 1)
            for (int vpt = 1; vpt <= 4; ++vpt)
                for (bool q8 : {false, true})
                    for (bool many : {false, true}) {
                        void* fn = postnorm_kernel_for(dt, vpt, w, q8, many);
                        if (!fn) continue;
                        cudaError_t e = cudaFuncSetAttribute(
                            fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kExclusiveSmemBytes);
                        if (e != cudaSuccess) return static_cast<int>(e);
                    }
    // Clusters of 8 CTAs that run at once, by vectors per thread (1, 2, 4).
    for (int v = 0; v < 3; ++v) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = cluster_config(8, 1, 0, false, nullptr, attr);
        for (int dt = 0; dt < 2; ++dt)
            for (bool q8 : {false, true}) {
                int n = 0;
                cudaError_t e = cudaOccupancyMaxActiveClusters(
                    &n, postnorm_kernel_for(dt, 1 << v, 0, q8), &cfg);
                if (e != cudaSuccess) return static_cast<int>(e);
                clusters[dt][v][q8] = n;
            }
    }
    return 0;
}

int launch_postnorm(const PostParams& pp, int dtype, int max_sms, const PostDevice& d,
                    void* stream) {
    const Params& p = pp.p;
    const int64_t tokens = p.t1 - p.t0, nvec = p.row_bytes / 16;
    const int64_t sms = max_sms < d.sm_count ? max_sms : d.sm_count;
    // Under a budget each CTA is alone on its SM.
    const bool whole = max_sms >= d.sm_count;
    const size_t smem = whole ? 0 : kExclusiveSmemBytes;
    if (p.row_bytes > kRowsRowBytes) {
        int cluster = 1;
        while (cluster * 2 <= 8 && cluster * 2 <= sms) cluster *= 2;
        const int vc = cluster_vectors_per_thread(p.row_bytes, cluster);
        const int64_t at_once =
            whole ? vc ? d.clusters[dtype][vc == 4 ? 2 : vc - 1][p.q8] : 0 : sms / cluster;
        if (vc != 0 && tokens <= at_once) {
            cudaLaunchAttribute attr[2];
            const cudaLaunchConfig_t cfg =
                cluster_config(cluster, tokens, smem, whole, stream, attr);
            void* args[] = {const_cast<PostParams*>(&pp)};
            return static_cast<int>(
                cudaLaunchKernelExC(&cfg, postnorm_kernel_for(dtype, vc, 0, p.q8 != 0), args));
        }
    }
    int vpt = 0, w = 0;
    rows_shape(nvec, &vpt, &w);
    const int64_t rows = kThreads / 32 / w;
    const int64_t ctas = (tokens + rows - 1) / rows;
    const int64_t at_once = (whole ? many_ctas(vpt) : vpt == 3 ? 0 : 2) * sms;
    if (p.row_bytes >= kShortRowBytes && (p.row_bytes > kLongestRowBytes || ctas > at_once))
        return launch_postnorm_rows(pp, dtype, static_cast<int>(sms), whole, d.smem_optin, stream);
    // Two CTAs on an SM need not spare registers.
    const bool many = (whole && ctas > 2 * sms) || vpt == 3;
    const int64_t most = whole ? (int64_t{1} << 31) - 1 : sms;
    return launch_with_pdl(postnorm_kernel_for(dtype, vpt, w, p.q8 != 0, many), pp,
                           static_cast<int>(ctas < most ? ctas : most), kThreads, smem, whole,
                           stream);
}

}  // namespace tw
