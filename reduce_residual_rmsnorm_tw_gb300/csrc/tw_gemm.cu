// tw_gemm.cu -- matrix product of 8-bit operands with scales per token and
// channel: out[t,n] = xs[t] ws[n] sum_k x[t,k] w[n,k].
//
// The channels are the tensor cores' M side (128 rows of W per CTA), the
// tokens their N side (a tile of BN, sized to the call), so that a few tokens
// cost a narrow MMA and the weights stream through once.  A unit of CG CTAs
// (1, or a pair sharing each token tile: CG = 2) walks the tiles persistently;
// its accumulators are double-buffered in TMEM, so that a tile's epilogue
// runs beside the next tile's products.
//
//   e4m3  both operands go from TMA's 128-byte-swizzled boxes straight into
//         tcgen05.mma.kind::f8f6f4.
//   int8  sm_103a has no integer tcgen05.  Integers to 2^11 are exact in f16
//         and the products accumulate in fp32, so the operands are widened to
//         f16 on the way: W into TMEM (the MMA's A operand may live there, and
//         shared memory, which bounds this kernel, sees W once in 8 bits
//         instead of three times), x into a second ring in shared memory.
//         f16 rather than bf16, whose 8 bits of mantissa hold -128..127 as
//         well, because one byte permute and one packed subtract make an
//         f16: 0x6400 | (v + 128) is 1024 + 128 + v.
//
// With few tokens there are fewer tiles than SMs: a cluster of S CTAs then
// splits K, and each adds up its share of the token columns from all S
// accumulators, pushed into its shared memory by the others (in rank order:
// the same bits every time).
#include <cuda.h>

#include <mutex>

#include "tw_tcgen05.cuh"

namespace tw {
namespace {

constexpr int kBlockK = 128;     // bytes (= 8-bit elements) of K per ring stage
constexpr int kUnitK = 64;       // int8: K elements per widened slot
constexpr int kRows = 128;       // channels per CTA
constexpr int kSlots = 4;        // int8: widened slots (TMEM and shared memory)
constexpr int kSlotColumns = kUnitK / 2;
constexpr int kMaxStages = 8;
constexpr int kTmemColumns = 512;
constexpr int kMaxSplit = 8;

// Warp roles: 0 TMA, 1 MMA, 4-7 epilogue, from 8 on kGroups of four widen
// (int8).
constexpr int kGroups = 4;
constexpr int kEpilogueWarp = 4, kWidenWarp = 8;

// Largest token tile: one unit's two accumulators (and, for int8, the widened
// W) share 512 TMEM columns; a single CTA takes short tiles only.
__host__ __device__ constexpr int max_tokens(int cg, bool int8) { return cg == 1 ? 64 : (int8 ? 192 : 256); }
// Bytes of the ring, per CTA.
__host__ __device__ constexpr int x_bytes(int cg, bool int8) { return max_tokens(cg, int8) / cg * kBlockK; }
__host__ __device__ constexpr int stage_bytes(int cg, bool int8) { return kRows * kBlockK + x_bytes(cg, int8); }
__host__ __device__ constexpr int slot_bytes(int cg, bool int8) {
    return int8 ? max_tokens(cg, int8) / cg * kUnitK * 2 : 0;
}
__host__ __device__ constexpr int stages(int cg, bool int8) {
    return cg == 1 ? (int8 ? 6 : 7) : (int8 ? 5 : 6);
}
// Staging of the output: two chunks of 32 tokens (bf16) or 16 (fp32) x 128
// channels for TMA to store; or, with split K, the accumulators of every CTA
// of the cluster for this CTA's columns.
constexpr int kChunkBytes = 8192;
__host__ __device__ constexpr int out_bytes(int cg, bool int8) {
    return cg == 1 ? max_tokens(cg, int8) * kRows * 4 : 2 * kChunkBytes;
}

struct Header {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t wide_full[kSlots], wide_empty[kSlots];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t joined, drained;
    uint32_t tmem;
    int abort;
    alignas(16) float x_scale[4][256];  // each epilogue warp's copy of its tile's
};
constexpr int kHeaderBytes = 5120;
static_assert(sizeof(Header) <= kHeaderBytes, "header too large");

__host__ __device__ constexpr int smem_bytes(int cg, bool int8) {
    return 1024 + kHeaderBytes + stages(cg, int8) * stage_bytes(cg, int8) +
           kSlots * slot_bytes(cg, int8) + out_bytes(cg, int8);
}
static_assert(smem_bytes(1, true) <= 232448 && smem_bytes(1, false) <= 232448 &&
                  smem_bytes(2, true) <= 232448 && smem_bytes(2, false) <= 232448,
              "over the shared memory of an SM");

struct GemmParams {
    const float* x_scale;
    const float* w_scale;
    void* out;
    unsigned int* status;
    int64_t N;
    int M;
    int k_blocks;      // ring stages of the whole K
    int channel_tiles; // of kRows * CG
    int tiles;         // channel tiles * token tiles
    int bn;            // tokens per tile
    int split;         // CTAs that share K (CG 1)
    int tma_out;       // rows of out are whole 16-byte units: stored by TMA
    int f32;           // output type
};

struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++at == n) {
            at = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ void gave_up(const GemmParams& p, volatile int* abort) {
    *abort = 1;
    atomicOr(p.status, 1u);
}

// A whole warp's wait: all lanes go on or all give up, so that the warp stays
// whole for the .aligned instructions that follow.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(const GemmParams& p, uint64_t* bar, uint32_t parity,
                                          volatile int* abort) {
    const bool ok = mbar_wait_slice<CLUSTER>(smem_addr(bar), parity, abort);
    if (__all_sync(0xffffffffu, ok)) return true;
    gave_up(p, abort);
    return false;
}

// Four int8 as two pairs of f16.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = v ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 ha = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 hb = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&ha);
    hi = *reinterpret_cast<const uint32_t*>(&hb);
}

__device__ __forceinline__ void widen16(const uint4& v, uint32_t* f) {
    widen4(v.x, f[0], f[1]);
    widen4(v.y, f[2], f[3]);
    widen4(v.z, f[4], f[5]);
    widen4(v.w, f[6], f[7]);
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint32_t* v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}

__device__ __forceinline__ void store_out(const GemmParams& p, int64_t at, float v) {
    if (p.f32)
        static_cast<float*>(p.out)[at] = v;
    else
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
}

// y[j] = v[j] * x_scale[j] * ws for sixteen tokens (in this order: the product
// of two small scales alone could lose its bits as a subnormal).
__device__ __forceinline__ void scale16(float (&y)[16], const uint32_t (&v)[16],
                                        const float (&xs)[16], float ws) {
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(v[j]) * xs[j] * ws;
}
__device__ __forceinline__ void load16(float (&y)[16], const float* x) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const float4 q = *reinterpret_cast<const float4*>(x + j);
        y[j] = q.x;
        y[j + 1] = q.y;
        y[j + 2] = q.z;
        y[j + 3] = q.w;
    }
}

// This warp has read its part of an accumulator: hand it back to the leader.
__device__ __forceinline__ void release_acc(uint64_t& bar, int cg, uint32_t rank, int lane) {
    tcgen05_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(map_to_rank(smem_addr(&bar), cg == 2 ? 0u : rank));
}

template <int CG, bool INT8>
__global__ void __launch_bounds__(INT8 ? 256 + 128 * kGroups : 256, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap x_map,
                const __grid_constant__ CUtensorMap w_map,
                const __grid_constant__ CUtensorMap out_map,
                const __grid_constant__ GemmParams p) {
    constexpr uint32_t S = stages(CG, INT8);
    constexpr int kStage = stage_bytes(CG, INT8), kSlot = slot_bytes(CG, INT8);
    constexpr uint32_t kAcc = max_tokens(CG, INT8);         // TMEM columns between accumulators
    constexpr uint32_t kWide = 2 * kAcc;                    // first widened slot's column
    extern __shared__ unsigned char raw_smem[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t{1023});
    Header& h = *reinterpret_cast<Header*>(smem);
    const uint32_t ring = smem_addr(smem) + kHeaderBytes;
    const uint32_t slots = ring + S * kStage;
    unsigned char* staging = smem + kHeaderBytes + S * kStage + kSlots * kSlot;
    volatile int* abort = &h.abort;

    // A warp index the compiler knows to be the same in all lanes: the MMA
    // warp's operands then live in uniform registers.
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = threadIdx.x % 32;
    // With CG 2 the cluster is the pair; the even CTA issues its MMAs.  With
    // CG 1 the cluster's CTAs split K.
    const uint32_t rank = cluster_cta_rank();
    const uint32_t unit = cluster_id_x(), units = cluster_count_x();
    const bool leader = CG == 1 || rank == 0;
    const int split = CG == 1 ? p.split : 1;
    const int kb0 = CG == 1 ? static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / split) : 0;
    const int kb1 = CG == 1 ? static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / split)
                            : p.k_blocks;
    const int bn_cta = p.bn / CG;  // token rows this CTA loads

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < S; ++s) {
            mbar_init(smem_addr(&h.full[s]), 1);
            mbar_init(smem_addr(&h.empty[s]), INT8 ? 8 : 1);
        }
        for (int c = 0; c < kSlots; ++c) {
            mbar_init(smem_addr(&h.wide_full[c]), 4 * CG);
            mbar_init(smem_addr(&h.wide_empty[c]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&h.acc_full[b]), 1);
            mbar_init(smem_addr(&h.acc_empty[b]), 4 * CG);
        }
        mbar_init(smem_addr(&h.joined), 1);
        mbar_init(smem_addr(&h.drained), 1);
        h.abort = 0;
        mbar_init_fence();
        if (split > 1)
            mbar_arrive_expect_tx(smem_addr(&h.joined), static_cast<uint32_t>(p.bn) * kRows * 4);
        tensormap_prefetch(&x_map);
        tensormap_prefetch(&w_map);
    }
    if (warp == 1) tmem_alloc<CG>(smem_addr(&h.tmem), kTmemColumns);
    tcgen05_fence_before();
    __syncthreads();
    // The peers' barriers must be initialised before anything arrives there.
    if (CG == 2 || split > 1) cluster_barrier();
    tcgen05_fence_after();
    const uint32_t tmem = h.tmem;
    grid_dependency_wait();
    grid_launch_dependents();

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------- TMA -----
        Ring r;
        uint32_t issued = 0;
        bool ok = true;
        const uint32_t bytes = static_cast<uint32_t>((kRows + bn_cta) * kBlockK);
        for (uint32_t tile = unit; ok && tile < static_cast<uint32_t>(p.tiles); tile += units) {
            const int channel = static_cast<int>(tile % p.channel_tiles) * (kRows * CG) +
                                (CG == 2 ? static_cast<int>(rank) * kRows : 0);
            const int token = static_cast<int>(tile / p.channel_tiles) * p.bn +
                              (CG == 2 ? static_cast<int>(rank) * bn_cta : 0);
            for (int kb = kb0; kb < kb1; ++kb, ++issued, r.next(S)) {
                if (!mbar_wait_slice(smem_addr(&h.empty[r.at]), r.phase ^ 1u, abort)) {
                    gave_up(p, abort);
                    ok = false;
                    break;
                }
                // e4m3 pairs: both CTAs' copies count on the leader's barrier,
                // which alone issues the products; int8: on this CTA's, whose
                // warps widen them.
                const uint32_t local = smem_addr(&h.full[r.at]);
                const uint32_t bar = CG == 2 && !INT8 ? map_to_rank(local, 0) : local;
                if (INT8 || leader) mbar_arrive_expect_tx(local, INT8 ? bytes : bytes * CG);
                const uint32_t dst = ring + r.at * kStage;
                tma_load_2d<INT8 ? 1 : CG>(dst, &w_map, kb * kBlockK, channel, bar);
                tma_load_2d<INT8 ? 1 : CG>(dst + kRows * kBlockK, &x_map, kb * kBlockK, token,
                                           bar);
            }
        }
        if (*abort && (INT8 || leader)) {
            // The copies in flight must land before the CTA may leave.
            for (uint32_t k = 0; k < S && k < issued; ++k) {
                if (r.at == 0) {
                    r.at = S - 1;
                    r.phase ^= 1u;
                } else {
                    --r.at;
                }
                if (!mbar_wait(smem_addr(&h.full[r.at]), r.phase, nullptr))
                    atomicOr(p.status, 2u);
            }
        }
    } else if (warp == 1 && leader) {
        // ------------------------------------------------------- MMA -----
        // The whole warp walks the slices and one elected lane issues: with
        // the operands in warp-uniform code a slice's four MMAs issue in a
        // fraction of the time a lone lane takes.
        Ring r, acc;
        bool ok = true;
        const uint32_t shape = mma_shape(kRows * CG, static_cast<uint32_t>(p.bn));
        [[maybe_unused]] const uint64_t slot_operand = smem_operand(slots);
        [[maybe_unused]] const uint64_t ring_operand = smem_operand(ring);
        for (uint32_t tile = unit; ok && tile < static_cast<uint32_t>(p.tiles);
             tile += units, acc.next(2)) {
            ok = warp_wait(p, &h.acc_empty[acc.at], acc.phase ^ 1u, abort);
            if (!ok) break;
            tcgen05_fence_after();
            const uint32_t d = tmem + acc.at * kAcc;
            // Whether the next slice is there is asked while this one's products
            // issue: an answer takes about 100 clocks, a slice's products 300.
            bool there = false;
            if constexpr (INT8) {
                const int n = 2 * (kb1 - kb0);
                for (int k = 0; k < n; ++k) {
                    if (!there) ok = warp_wait(p, &h.wide_full[r.at], r.phase, abort);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t at = r.at;
                    r.next(kSlots);
                    there = k + 1 < n && mbar_test(smem_addr(&h.wide_full[r.at]), r.phase);
                    if (elect_one()) {
                        const uint64_t b = slot_operand + at * (kSlot >> 4);
                        const uint32_t a = tmem + kWide + at * kSlotColumns;
#pragma unroll
                        for (int i = 0; i < kUnitK / 16; ++i)
                            mma_f16_tmem<CG>(d, a + 8 * i, b + 2 * i, shape, k > 0 || i > 0);
                        mma_commit<CG>(smem_addr(&h.wide_empty[at]));
                    }
                    __syncwarp();
                    there = __all_sync(0xffffffffu, there);
                }
            } else {
                const int n = kb1 - kb0;
                for (int k = 0; k < n; ++k) {
                    if (!there) ok = warp_wait(p, &h.full[r.at], r.phase, abort);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t at = r.at;
                    r.next(S);
                    there = k + 1 < n && mbar_test(smem_addr(&h.full[r.at]), r.phase);
                    if (elect_one()) {
                        const uint64_t a = ring_operand + at * (kStage >> 4);
                        const uint64_t b = a + (kRows * kBlockK >> 4);
#pragma unroll
                        for (int i = 0; i < kBlockK / 32; ++i)
                            mma_e4m3<CG>(d, a + 2 * i, b + 2 * i, shape, k > 0 || i > 0);
                        mma_commit<CG>(smem_addr(&h.empty[at]));
                    }
                    __syncwarp();
                    there = __all_sync(0xffffffffu, there);
                }
            }
            if (ok && elect_one()) mma_commit<CG>(smem_addr(&h.acc_full[acc.at]));
            __syncwarp();
        }
        if (!ok) {
            // Products in flight still read shared memory and write TMEM.
            if (elect_one()) mma_commit<CG>(smem_addr(&h.drained));
            if (!mbar_wait_slice(smem_addr(&h.drained), 0, nullptr)) atomicOr(p.status, 2u);
        }
    } else if (warp >= kEpilogueWarp && warp < kEpilogueWarp + 4) {
        // -------------------------------------------------- epilogue -----
        // Thread = channel (TMEM lane), registers = tokens.
        const int quarter = warp - kEpilogueWarp;
        const int etid = quarter * 32 + lane;
        float* x_scale = h.x_scale[quarter];
        int chunk = 0;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        Ring acc;
        for (uint32_t tile = unit; tile < static_cast<uint32_t>(p.tiles);
             tile += units, acc.next(2)) {
            const int64_t n = static_cast<int64_t>(tile % p.channel_tiles) * (kRows * CG) +
                              (CG == 2 ? rank * kRows : 0) + etid;
            const int t0 = static_cast<int>(tile / p.channel_tiles) * p.bn;
            // Every load of the tile's scales in flight at once.
            const float ws = n < p.N ? p.w_scale[n] : 0.f;
            float xs[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = i * 32 + lane;
                xs[i] = j < p.bn && t0 + j < p.M ? p.x_scale[t0 + j] : 0.f;
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) x_scale[i * 32 + lane] = xs[i];
            __syncwarp();
            // The four warps go on or give up together (they meet at barriers
            // below).
            const bool ok = warp_wait(p, &h.acc_full[acc.at], acc.phase, abort);
            if (named_barrier_or(1, 128, !ok)) break;
            tcgen05_fence_after();
            const uint32_t d = tmem + acc.at * kAcc + lanes;
            const int n_tok = p.M - t0 < p.bn ? p.M - t0 : p.bn;
            if (CG == 1 && split > 1) {
                // Push every CTA's columns to it, then add up this CTA's: four
                // columns of a channel travel as 16 bytes, [source][column /
                // 4][channel].
                const int own = p.bn / split;  // a multiple of 4
                const uint32_t local = smem_addr(staging) +
                                       (static_cast<uint32_t>(rank) * (own / 4) * kRows + etid) * 16;
                const uint32_t bar = smem_addr(&h.joined);
                int to = 0, at = 0;
                for (int c = 0; c < p.bn; c += 16) {
                    uint32_t v[16];
                    tmem_load16(v, d + c);
                    tmem_wait_loads();
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        st_async4(map_to_rank(local + at * (kRows * 4), to), v + j,
                                  map_to_rank(bar, to));
                        at += 4;
                        if (at == own) {
                            at = 0;
                            ++to;
                        }
                    }
                }
                if (!warp_wait<true>(p, &h.joined, 0, abort)) break;
                const float4* part = reinterpret_cast<const float4*>(staging) + etid;
                for (int j = 0; j < own; j += 4) {
                    float4 sum = part[j / 4 * kRows];
                    for (int s = 1; s < split; ++s) {
                        const float4 q = part[(s * own + j) / 4 * kRows];
                        sum.x += q.x;
                        sum.y += q.y;
                        sum.z += q.z;
                        sum.w += q.w;
                    }
                    const int c = static_cast<int>(rank) * own + j;
                    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < n_tok && n < p.N)
                            store_out(p, (static_cast<int64_t>(t0) + c + i) * p.N + n,
                                      v[i] * x_scale[c + i] * ws);
                }
                break;  // one tile per cluster
            }
            if (p.tma_out) {
                // Through shared memory, [token][channel], and out by TMA: the
                // rows of a chunk leave as whole 256- or 512-byte lines beside
                // the next chunk's loads.
                const int per_chunk = p.f32 ? 16 : 32;
                for (int c = 0; c < p.bn; c += per_chunk, chunk ^= 1) {
                    unsigned char* to = staging + chunk * kChunkBytes;
                    if (etid == 0) bulk_wait_read<1>();
                    named_barrier(1, 128);
                    for (int k = 0; k < per_chunk; k += 16) {
                        uint32_t v[16];
                        tmem_load16(v, d + c + k);
                        float xs16[16], y[16];
                        load16(xs16, x_scale + c + k);
                        tmem_wait_loads();
                        scale16(y, v, xs16, ws);
                        if (p.f32) {
                            float* row = reinterpret_cast<float*>(to) + etid;
#pragma unroll
                            for (int j = 0; j < 16; ++j) row[j * kRows] = y[j];
                        } else {
                            __nv_bfloat16* row =
                                reinterpret_cast<__nv_bfloat16*>(to) + k * kRows + etid;
#pragma unroll
                            for (int j = 0; j < 16; ++j) row[j * kRows] = __float2bfloat16_rn(y[j]);
                        }
                    }
                    if (c + per_chunk >= p.bn) release_acc(h.acc_empty[acc.at], CG, rank, lane);
                    fence_async_shared();
                    named_barrier(1, 128);
                    if (etid == 0) {
                        if (c < n_tok && n < p.N)
                            tma_store_2d(&out_map, static_cast<int>(n), t0 + c, smem_addr(to));
                        bulk_commit();
                    }
                }
                continue;
            }
            for (int c = 0; c < p.bn; c += 16) {
                uint32_t v[16];
                tmem_load16(v, d + c);
                float xs16[16], y[16];
                load16(xs16, x_scale + c);
                tmem_wait_loads();
                scale16(y, v, xs16, ws);
                if (c + 16 >= p.bn) release_acc(h.acc_empty[acc.at], CG, rank, lane);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < n_tok && n < p.N)
                        store_out(p, (static_cast<int64_t>(t0) + c + j) * p.N + n, y[j]);
                __syncwarp();
            }
        }
        if (etid == 0) bulk_wait_read<0>();
    } else if (INT8 && warp >= kWidenWarp) {
        // ------------------------------------------------- widening ------
        // Groups of four warps take the 64-element halves of the stages in
        // turn: row `row` of W into TMEM lane `row`, and the token rows.
        const int group = (warp - kWidenWarp) / 4;
        const int row = threadIdx.x % 128;
        // 16-byte chunks of the token rows per thread: 32 rows x 4 chunks at
        // a time, this warp's first row x_row0.
        constexpr int kTokenChunks = max_tokens(CG, true) / CG / 32;
        const int x_row0 = row / 32 * 8, x_row = x_row0 + (row & 7), x_chunk = row / 8 % 4;
        const uint32_t lanes = static_cast<uint32_t>(row / 32 * 32) << 16;
        Ring r, c;
        const int tile_units = 2 * (kb1 - kb0);
        const int my_tiles = static_cast<int>(unit) < p.tiles
                                 ? (p.tiles - 1 - static_cast<int>(unit)) / static_cast<int>(units) + 1
                                 : 0;
        const int64_t n_units = static_cast<int64_t>(my_tiles) * tile_units;
        for (int i = 0; i < group; ++i) c.next(kSlots);
        for (int i = 0; i < group / 2; ++i) r.next(S);
        for (int64_t u = group; u < n_units; u += kGroups) {
            const int half = static_cast<int>(u) & 1;
            if (!warp_wait(p, &h.full[r.at], r.phase, abort)) break;
            const uint32_t stage = ring + r.at * kStage;
            // 16-byte chunk i of row R lies at chunk i ^ (R & 7).  Eight
            // neighbouring threads take one chunk of eight rows (eight
            // different bank groups, read and written).
            uint4 raw[4 + kTokenChunks];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                raw[i] = lds16(stage + row * kBlockK + (((half * 4 + i) ^ (row & 7)) << 4));
#pragma unroll
            for (int i = 0; i < kTokenChunks; ++i)
                if (i * 32 + x_row0 < bn_cta)
                    raw[4 + i] = lds16(stage + kRows * kBlockK + (i * 32 + x_row) * kBlockK +
                                       (((half * 4 + x_chunk) ^ (x_row & 7)) << 4));
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) widen16(raw[i], w + 8 * i);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&h.empty[r.at]));
            if (!warp_wait(p, &h.wide_empty[c.at], c.phase ^ 1u, abort)) break;
            tcgen05_fence_after();
            tmem_store32(tmem + lanes + kWide + c.at * kSlotColumns, w);
            const uint32_t slot = slots + c.at * kSlot + x_row * 128;
#pragma unroll
            for (int i = 0; i < kTokenChunks; ++i)
                if (i * 32 + x_row0 < bn_cta) {
                    uint32_t x[8];
                    widen16(raw[4 + i], x);
                    const uint32_t to = slot + i * 32 * 128;
                    sts16(to + (((2 * x_chunk) ^ (x_row & 7)) << 4), x);
                    sts16(to + (((2 * x_chunk + 1) ^ (x_row & 7)) << 4), x + 4);
                }
            fence_async_shared();
            tmem_wait_stores();
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_pair(map_to_rank(smem_addr(&h.wide_full[c.at]), CG == 2 ? 0u : rank));
            const int step = (half + kGroups) / 2;  // stages on to unit u + kGroups
            for (int i = 0; i < step; ++i) r.next(S);
            for (int i = 0; i < kGroups; ++i) c.next(kSlots);
        }
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    // After a wait that ran out, the other CTAs' pushes may still be on their
    // way here.
    if (split > 1 && *abort && threadIdx.x == 0 &&
        !mbar_wait_slice<true>(smem_addr(&h.joined), 0, nullptr))
        atomicOr(p.status, 2u);
    __syncwarp();
    // No CTA leaves while another may still write into it or read its rows.
    if (CG == 2 || split > 1) cluster_barrier();
    tcgen05_fence_after();
    if (warp == 1) tmem_free<CG>(tmem, kTmemColumns);
}

// ------------------------------------------------------------ host side ---
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

// A dense [rows, columns] tensor moved in boxes of box_columns x box_rows; what
// lies outside reads as zeros (0 in every type).
bool encode(CUtensorMap* m, CUtensorMapDataType type, int64_t elem, const void* base, int64_t rows,
            int64_t columns, int box_columns, int box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t size[2] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(rows)};
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(columns * elem)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_columns),
                               static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t step[2] = {1, 1};
    return g_encode(m, type, 2, const_cast<void*>(base), size, stride, box, step,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An 8-bit operand [rows, K], in boxes one swizzle row (128 bytes) wide.
bool encode_operand(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int box_rows) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, rows, K, kBlockK, box_rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

void* gemm_kernel_for(int cg, bool int8) {
    if (cg == 1)
        return int8 ? reinterpret_cast<void*>(&gemm_kernel<1, true>)
                    : reinterpret_cast<void*>(&gemm_kernel<1, false>);
    return int8 ? reinterpret_cast<void*>(&gemm_kernel<2, true>)
                : reinterpret_cast<void*>(&gemm_kernel<2, false>);
}

}  // namespace

int gemm_prepare(int smem_optin) {
    for (int cg = 1; cg <= 2; ++cg)
        for (bool int8 : {false, true}) {
            if (smem_bytes(cg, int8) > smem_optin) return static_cast<int>(cudaErrorInvalidValue);
            cudaError_t e = cudaFuncSetAttribute(gemm_kernel_for(cg, int8),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 smem_bytes(cg, int8));
            if (e != cudaSuccess) return static_cast<int>(e);
        }
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                     cudaEnableDefault, &found);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (found != cudaDriverEntryPointSuccess || !fn)
        return static_cast<int>(cudaErrorSymbolNotFound);
    g_encode = reinterpret_cast<EncodeTiled>(fn);
    return 0;
}

int launch_gemm(const GemmArgs& g, int max_sms, const DeviceInfo& d, void* stream) {
    const bool int8 = g.qtype == TW_INT8;
    const int64_t sms = max_sms < d.sm_count ? max_sms : d.sm_count;
    const int cg = g.M <= max_tokens(1, int8) || sms < 2 ? 1 : 2;
    const int64_t token_tiles = (g.M + max_tokens(cg, int8) - 1) / max_tokens(cg, int8);
    const int64_t per_tile = (g.M + token_tiles - 1) / token_tiles;
    GemmParams p{};
    p.x_scale = g.x_scale;
    p.w_scale = g.w_scale;
    p.out = g.out;
    p.status = d.status;
    p.N = g.N;
    p.M = static_cast<int>(g.M);
    p.k_blocks = static_cast<int>((g.K + kBlockK - 1) / kBlockK);
    p.f32 = g.dtype == TW_F32;
    const int64_t channel_tiles = (g.N + kRows * cg - 1) / (kRows * cg);
    const int64_t tiles = channel_tiles * token_tiles;
    if (tiles > (int64_t{1} << 31) - 1 - sms) return static_cast<int>(cudaErrorInvalidValue);
    p.channel_tiles = static_cast<int>(channel_tiles);
    p.tiles = static_cast<int>(tiles);
    p.split = 1;
    if (cg == 1)
        while (p.split < kMaxSplit && tiles * p.split * 2 <= sms && p.split * 2 <= p.k_blocks)
            p.split *= 2;
    // Whole chunks of the output's staging, or of each CTA's share of the
    // columns (never above max_tokens, a multiple of both).
    const int align = p.split > 1 ? (p.split > 4 ? 4 * p.split : 16) : 32;
    p.bn = static_cast<int>((per_tile + align - 1) / align * align);
    const int64_t es = p.f32 ? 4 : 2;
    p.tma_out = p.split == 1 && g.N * es % 16 == 0;
    CUtensorMap x_map, w_map, out_map{};
    if (!encode_operand(&x_map, g.x, g.M, g.K, p.bn / cg) ||
        !encode_operand(&w_map, g.w, g.N, g.K, kRows) ||
        (p.tma_out && !encode(&out_map,
                              p.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              es, g.out, g.M, g.N, kRows, p.f32 ? 16 : 32,
                              CU_TENSOR_MAP_SWIZZLE_NONE)))
        return static_cast<int>(cudaErrorInvalidValue);

    const int cluster = cg == 1 ? p.split : 2;
    const int64_t most = sms / cluster;
    const int64_t units = tiles < most ? tiles : most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * cluster));
    cfg.blockDim = dim3(int8 ? 256 + 128 * kGroups : 256);
    cfg.dynamicSmemBytes = smem_bytes(cg, int8);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = max_sms >= d.sm_count ? 2 : 1;
    void* args[] = {&x_map, &w_map, &out_map, &p};
    return static_cast<int>(cudaLaunchKernelExC(&cfg, gemm_kernel_for(cg, int8), args));
}

}  // namespace tw
