// tw_postnorm_rows.cu -- the step with two norms for many tokens with long
// rows: persistent CTAs, rows streamed through a ring of bulk copies.
//
// Per token (fp32): s = sum_r partials[r]; u = s / rms(s) * post_weight;
// x = residual_scale * residual + block_scale * gate * u; residual_out = x;
// out[k] = x / rms(x) * weight.
//
// A CTA, alone on its SM, is one to eight pipelines that share sixteen warps, each with a
// producer warp and its part of the ring (pipelines_for, below).  A ring slot holds one
// row: a token's partials come first and are added up and handed back one by one, its
// residual and gate last;
// those stay in their slots while the sum's square is reduced, so that registers
// hold one row in fp32 only; the two weights lie in shared memory (in registers they
// spilled: 8 x 1024 x 8192 36.8 us against 28.9).  Each of the two reductions is a
// warp sum and one barrier of the pipeline; while one pipeline waits there the others
// stream.  A gate that tokens share is copied for each of them: out of L2.
// Bound by HBM: n_parts + 1 rows (and a gate's) in, n_out + 1 out (8 x 1024 x 8192 bf16
// 29.0 us, 6.4 TB/s; 4 x 1111 x 5120 fp32 with a gate and two outputs 28.4; 2 x 2048 x
// 4096 with a gate per token 17.4, 5.8 TB/s: 13 rows a CTA, the last of them alone).
#include "tw_device.cuh"

namespace tw {
namespace {

constexpr int kWarps = 16;     // of all pipelines, without the producers
constexpr int kMaxSlots = 16;  // of a pipeline
constexpr int kMaxPipes = 8;
__host__ __device__ constexpr int block_of(int pipes) { return 32 * (kWarps + pipes); }

struct Header {
    uint64_t full[kMaxPipes][kMaxSlots], empty[kMaxPipes][kMaxSlots];  // of each pipeline
    // Warp totals: [reduction][buffer][warp].
    float sums[2][2][kWarps];
    float most[2][kWarps];
    int abort;
};
constexpr int kHeaderBytes = 2560;
static_assert(sizeof(Header) <= kHeaderBytes, "header too large");

struct RingPos {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ void gave_up(const Params& p, volatile int* abort) {
    *abort = 1;
    atomicOr(p.status, 1u);
}

// NV: 16-byte vectors of a row per thread.
template <typename T, int NV, int kPipes, bool Q8>
__global__ void __launch_bounds__(block_of(kPipes), 1)
    postnorm_rows_kernel(const __grid_constant__ PostParams pp, int slots) {
    using V = Vec<T>;
    constexpr int E = V::kElems;
    constexpr int kPipeWarps = kWarps / kPipes, kPipeThreads = 32 * kPipeWarps;
    extern __shared__ __align__(128) unsigned char smem[];
    Header& h = *reinterpret_cast<Header*>(smem);
    volatile int* abort = &h.abort;
    const Params& p = pp.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool producer = warp >= kPipes * kPipeWarps;
    const int pipe = producer ? warp - kPipes * kPipeWarps : warp / kPipeWarps;
    const int64_t rb = p.row_bytes;
    const uint32_t row_bytes = static_cast<uint32_t>(rb);
    const uint32_t n_slots = static_cast<uint32_t>(slots);
    unsigned char* rows_at = smem + kHeaderBytes + 2 * row_bytes;
    const uint32_t ring = smem_addr(rows_at) + pipe * n_slots * row_bytes;
    const uint32_t full = smem_addr(&h.full[pipe][0]), empty = smem_addr(&h.empty[pipe][0]);
    const int rows = p.n_parts + 1 + (pp.gate ? 1 : 0);  // of a token
    // Row r of token t: the partials, the residual, the gate's.
    auto row_of = [&](int64_t t, int r) {
        const void* base = r < p.n_parts ? p.partials[r] : r == p.n_parts ? p.residual : pp.gate;
        return static_cast<const char*>(base) + (r <= p.n_parts ? t : t / pp.gate_tokens) * rb;
    };

    if (threadIdx.x == 0) {
        for (int g = 0; g < kPipes; ++g)
            for (int s = 0; s < slots; ++s) {
                mbar_init(smem_addr(&h.full[g][s]), 1);
                mbar_init(smem_addr(&h.empty[g][s]), kPipeWarps);
            }
        h.abort = 0;
        mbar_init_fence();
    }
    __syncthreads();
    // Pipeline g's tokens: t0 + block + (kPipes i + g) * grid.
    const int64_t first = p.t0 + blockIdx.x + static_cast<int64_t>(pipe) * gridDim.x;
    const int64_t step = static_cast<int64_t>(kPipes) * gridDim.x;
    // The first token's rows on their way into L2 while the launch before this one ends
    // (a hint that reads nothing: what that launch writes is seen all the same).
    if (producer && lane == 0 && p.prefetch && first < p.t1)
        for (int r = 0; r < rows; ++r) bulk_prefetch_l2(row_of(first, r), row_bytes);
    grid_dependency_wait();
    grid_launch_dependents();

    if (producer) {
        if (lane != 0) return;
        const uint64_t policy = policy_evict_first();
        RingPos pos;
        uint64_t issued = 0;
        bool stop = false;
        for (int64_t t = first; t < p.t1 && !stop; t += step)
            for (int r = 0; r < rows; ++r, ++issued, pos.next(n_slots)) {
                const uint32_t s = pos.slot;
                if (*abort ||
                    (issued >= n_slots && !mbar_wait(empty + 8 * s, pos.phase ^ 1u, abort))) {
                    gave_up(p, abort);
                    stop = true;
                    break;
                }
                mbar_arrive_expect_tx(full + 8 * s, row_bytes);
                const char* from = row_of(t, r);
                if (r <= p.n_parts)
                    bulk_g2s(ring + s * row_bytes, from, row_bytes, full + 8 * s, policy);
                else  // a gate's row may serve other tokens
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
                        "[%0], [%1], %2, [%3];" ::"r"(ring + s * row_bytes),
                        "l"(from), "r"(row_bytes), "r"(full + 8 * s)
                        : "memory");
            }
        // This pipeline's copies must have landed before the CTA leaves.
        for (uint32_t k = 0; k < n_slots && k < issued; ++k) {
            if (pos.slot == 0) {
                pos.slot = n_slots - 1;
                pos.phase ^= 1u;
            } else {
                --pos.slot;
            }
            if (!mbar_wait(full + 8 * pos.slot, pos.phase, nullptr)) atomicOr(p.status, 2u);
        }
        return;
    }

    // Consumers.  Bounded waits; one that gave up keeps walking (no waits, no stores), so
    // that the barriers stay whole.
    const int gtid = static_cast<int>(threadIdx.x) - pipe * kPipeThreads;
    const int nvec = static_cast<int>(rb / 16);
    // Both weights in shared memory (in registers those of a 16 KB row spilled: 8 x 1024 x
    // 8192 36.8 us, 29.2).  Vector k of post_weight (which 0) or weight (1):
    unsigned char* weights = smem + kHeaderBytes;
    auto weight_at = [&](int which, int k) {
        return *reinterpret_cast<const uint4*>(weights + which * row_bytes +
                                               (gtid + k * kPipeThreads) * 16);
    };
    for (int v = threadIdx.x; v < 2 * nvec; v += 32 * kWarps) {
        const void* from = v < nvec ? pp.post_weight : p.weight;
        if (from)
            *reinterpret_cast<uint4*>(weights + v * 16) =
                ld_global_nc(static_cast<const char*>(from) + (v < nvec ? v : v - nvec) * 16);
    }
    named_barrier(1 + kMaxPipes, 32 * kWarps);
    RingPos pos;
    bool alive = true;
    int buf = 0;
    auto wait_full = [&](const RingPos& at) {
        if (alive && !mbar_wait(full + 8 * at.slot, at.phase, abort)) {
            gave_up(p, abort);
            alive = false;
        }
    };
    auto release = [&](const RingPos& at) {
        __syncwarp();
        if (alive && lane == 0) mbar_arrive(empty + 8 * at.slot);
    };
    auto total_of = [&](int which, float v) {
        v = warp_sum(v);
        if (lane == 0) h.sums[which][buf][warp] = v;
        named_barrier(1 + pipe, kPipeThreads);
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kPipeWarps; ++w) total += h.sums[which][buf][pipe * kPipeWarps + w];
        return total;
    };
    for (int64_t t = first; t < p.t1; t += step, buf ^= 1) {
        float x[NV][E];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) x[k][e] = 0.f;
        for (int r = 0; r < p.n_parts; ++r, pos.next(n_slots)) {
            wait_full(pos);
            const unsigned char* row =
                rows_at + (pipe * n_slots + pos.slot) * row_bytes + gtid * 16;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (gtid + k * kPipeThreads < nvec)
                    add_vec(x[k], *reinterpret_cast<const uint4*>(row + k * kPipeThreads * 16),
                            static_cast<T*>(nullptr));
            release(pos);
        }
        float c = 1.f;
        if (pp.post_weight) {
            float ss2[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < NV; ++k) sum_squares<E>(ss2, x[k]);
            c = rsqrtf(total_of(0, ss2[0] + ss2[1]) * p.inv_H + pp.post_eps);
        }
        const RingPos at = pos;
        RingPos gate_at = pos;
        wait_full(at);
        pos.next(n_slots);
        if (pp.gate) {
            gate_at = pos;
            wait_full(gate_at);
            pos.next(n_slots);
        }
        const unsigned char* base = rows_at + pipe * n_slots * row_bytes + gtid * 16;
        const unsigned char* residual = base + at.slot * row_bytes;
        const unsigned char* gate = base + gate_at.slot * row_bytes;
        float ss2[2] = {0.f, 0.f}, m = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (gtid + k * kPipeThreads >= nvec) continue;
            float f[E];
            if (pp.post_weight) {
                V::to_float(weight_at(0, k), f);
#pragma unroll
                for (int e = 0; e < E; ++e) x[k][e] = x[k][e] * c * f[e];
            }
            if (pp.gate) {
                V::to_float(*reinterpret_cast<const uint4*>(gate + k * kPipeThreads * 16), f);
#pragma unroll
                for (int e = 0; e < E; ++e) x[k][e] *= f[e];
            }
            V::to_float(*reinterpret_cast<const uint4*>(residual + k * kPipeThreads * 16), f);
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[k][e] = fmaf(pp.block_scale, x[k][e], pp.residual_scale * f[e]);
            sum_squares<E>(ss2, x[k]);
            if constexpr (Q8)
                m = max_abs_product<T>(m, x[k], weight_at(1, k));
        }
        release(at);
        if (pp.gate) release(gate_at);
        if constexpr (Q8) {
            m = warp_max_abs(m);
            if (lane == 0) h.most[buf][warp] = m;
        }
        const float inv = rsqrtf(total_of(1, ss2[0] + ss2[1]) * p.inv_H + p.eps);
        [[maybe_unused]] RowQuant rq;
        if constexpr (Q8) {
            m = 0.f;
#pragma unroll
            for (int w = 0; w < kPipeWarps; ++w) m = max_abs(m, h.most[buf][pipe * kPipeWarps + w]);
            rq = RowQuant(m, inv, quant_top(p.qtype));
            if (gtid < p.n_out && alive)
                p.out_scale[gtid][t] = row_scale(rq.y, quant_top(p.qtype), rq.zero);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = gtid + k * kPipeThreads;
            if (v >= nvec || !alive) continue;
            const int64_t off = t * rb + static_cast<int64_t>(v) * 16;
            st_global_cs(static_cast<char*>(p.residual_out) + off, V::from_float(x[k]));
            float w[E], y[E];
            V::to_float(weight_at(1, k), w);
            if constexpr (Q8) {
#pragma unroll
                for (int e = 0; e < E; e += 2) mul2(y + e, x[k] + e, w + e);
                store_q8<E>(p.out, p.n_out, t * p.H + static_cast<int64_t>(v) * E, y, rq, p.qtype);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = (x[k][e] * inv) * w[e];
                const uint4 packed = V::from_float(y);
                for (int o = 0; o < p.n_out; ++o)
                    st_global_cs(static_cast<char*>(p.out[o]) + off, packed);
            }
        }
    }
}

// Pipelines for rows of this size.  More of them hide each other's barriers, where the
// ring still holds rows enough for each and there are tokens for all:
//   rows above 24 KB   one, whose ring holds more of them
//   rows to 5 KB       eight, unless four's rounds are fewer tokens (8 x 2048 x 2048 bf16 with
//                      two, four and eight 25.0, 16.9 and 16.2 us; 5 x 600 x 1024 fp32 7.3,
//                      5.5 and 5.9, 6 x 1500 x 2048 bf16 16.0, 11.6 and 13.1)
//   rows to 8 KB       four, unless their last round is emptier than two's by more than
//                      they gain, the more the shorter the row (8 x 700 x 3000 12.4 -> 11.0,
//                      2 x 4096 x 4096 30.0 -> 27.3, but 2 x 2048 x 4096 16.0 -> 16.3)
//   others             two (fp32 rows of 10 KB, four: 15.0 -> 16.0)
int pipelines_for(int64_t row_bytes, int64_t tokens, int64_t sms) {
    auto rounds = [&](int pipes) { return (tokens + pipes * sms - 1) / (pipes * sms) * pipes; };
    if (row_bytes > 24 * 1024) return 1;
    if (row_bytes <= 5 * 1024 && rounds(8) <= rounds(4)) return 8;
    return row_bytes <= 8 * 1024 && rounds(4) * row_bytes < rounds(2) * 9 * 1024 ? 4 : 2;
}

template <typename T, bool Q8>
void* entry(int nv, int pipes) {
    if (pipes == 1) return reinterpret_cast<void*>(&postnorm_rows_kernel<T, 4, 1, Q8>);
    // (Rows of 4 KB at least: two vectors a thread and more.)
    if (pipes == 8)
        return nv <= 4 ? reinterpret_cast<void*>(&postnorm_rows_kernel<T, 4, 8, Q8>)
                       : reinterpret_cast<void*>(&postnorm_rows_kernel<T, 5, 8, Q8>);
    if (pipes == 4)
        return nv <= 2   ? reinterpret_cast<void*>(&postnorm_rows_kernel<T, 2, 4, Q8>)
               : nv == 3 ? reinterpret_cast<void*>(&postnorm_rows_kernel<T, 3, 4, Q8>)
                         : reinterpret_cast<void*>(&postnorm_rows_kernel<T, 4, 4, Q8>);
    switch (nv) {
        case 1:
        case 2: return reinterpret_cast<void*>(&postnorm_rows_kernel<T, 2, 2, Q8>);
        case 3: return reinterpret_cast<void*>(&postnorm_rows_kernel<T, 3, 2, Q8>);
        case 4: return reinterpret_cast<void*>(&postnorm_rows_kernel<T, 4, 2, Q8>);
        case 5: return reinterpret_cast<void*>(&postnorm_rows_kernel<T, 5, 2, Q8>);
        default: return reinterpret_cast<void*>(&postnorm_rows_kernel<T, 6, 2, Q8>);
    }
}
void* kernel_for(int dtype, int nv, int pipes, bool q8) {
    if (dtype == TW_BF16)
        return q8 ? entry<__nv_bfloat16, true>(nv, pipes) : entry<__nv_bfloat16, false>(nv, pipes);
    return q8 ? entry<float, true>(nv, pipes) : entry<float, false>(nv, pipes);
}

}  // namespace

int postnorm_rows_prepare(int smem_optin) {
    for (int dt = 0; dt < 2; ++dt)
        for (int nv = 1; nv <= 6; ++nv)
            for (int pipes = 1; pipes <= 8; pipes *= 2)
                for (bool q8 : {false, true}) {
                    cudaError_t e = cudaFuncSetAttribute(
                        kernel_for(dt, nv, pipes, q8), cudaFuncAttributeMaxDynamicSharedMemorySize,
                        smem_optin);
                    if (e != cudaSuccess) return static_cast<int>(e);
                }
    return 0;
}

int launch_postnorm_rows(const PostParams& pp, int dtype, int sms, bool whole, int smem_optin,
                         void* stream) {
    const Params& p = pp.p;
    const int64_t tokens = p.t1 - p.t0;
    const int pipes = pipelines_for(p.row_bytes, tokens, sms);
    const int threads = 32 * kWarps / pipes;
    const int nv = static_cast<int>((p.row_bytes / 16 + threads - 1) / threads);
    const int64_t held = kHeaderBytes + 2 * p.row_bytes;
    int slots = static_cast<int>((smem_optin - held) / (pipes * p.row_bytes));
    if (slots > kMaxSlots) slots = kMaxSlots;
    if (slots < 2) return static_cast<int>(cudaErrorInvalidConfiguration);
    size_t smem = static_cast<size_t>(held + pipes * slots * p.row_bytes);
    if (smem < kExclusiveSmemBytes) smem = kExclusiveSmemBytes;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tokens < sms ? tokens : sms));
    cfg.blockDim = dim3(static_cast<unsigned>(block_of(pipes)));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = whole ? 1 : 0;
    void* args[] = {const_cast<PostParams*>(&pp), &slots};
    return static_cast<int>(
        cudaLaunchKernelExC(&cfg, kernel_for(dtype, nv, pipes, p.q8 != 0), args));
}

}  // namespace tw
