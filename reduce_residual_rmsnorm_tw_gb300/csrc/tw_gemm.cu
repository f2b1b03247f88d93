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
//         shared memory sees W once, in 8 bits: its write and two reads by
//         the MMAs of a pair in 16 bits fall away), x into a second ring in
//         shared memory.
//         f16 rather than bf16, whose 8 bits of mantissa hold -128..127 as
//         well, because one byte permute and one packed subtract make an
//         f16: 0x6400 | (v + 128) is 1024 + 128 + v.
//
// With fewer tiles than SMs a cluster of S units splits K, and each adds up its
// share of the token columns from all S accumulators, copied into its shared
// memory by the others (and added in rank order: the same bits every time).
//
// Measured (N = K = 8192, bf16 out, inputs larger than L2 in turn):
//   tokens       16     64    256    512   1024   4096
//   int8       16.5   17.4   25.9     47     87    325  us
//   e4m3       13.6   14.3   17.3     25     45    178  us
// What bounds it: at 16 and 64 tokens the 67 MB of weights (4.7 TB/s in e4m3 with
// launch, ramp and join in the time).  From 512 tokens on the board's power: back
// to back the SM clock falls to 1.5 to 1.9 GHz; with pauses between calls it
// stays at 2.07 and 1024 tokens take 82 us (int8) and 43 (e4m3), 4096 tokens 300
// (1.83 PFLOP/s) and 151 (3.63).  e4m3 at 1024: 1.7 waves of tiles on 76 pairs,
// run as two.  int8 below 512 tokens: issue slots, for which the MMA warp (its wait,
// eight MMAs and commit of a stage take about 680 clocks at 96 tokens to a tile, the
// products 384) and sixteen widening warps compete (when 256 tokens took 28.3 us, half the MMAs took it to 25.6, leaving
// out the widening's arithmetic to 24.2).
#include <cuda.h>

#include "tw_tcgen05.cuh"

namespace tw {
namespace {

constexpr int kBlockK = 128;     // bytes (= 8-bit elements) of K per ring stage
constexpr int kRows = 128;       // channels per CTA
constexpr int kWideSlots = 4;    // int8: widened stages (TMEM and shared memory)
constexpr int kSlotColumns = kBlockK / 2;
constexpr int kRingStages = 12;
constexpr int kTmemColumns = 512;

// Warp roles: 0 loads W, 1 MMA, 3 loads x, 4-7 epilogue, from 8 on kGroups of
// four widen (int8).
constexpr int kGroups = 4;
// Groups two apart work on neighbouring stages and slots (Ring::skip).
static_assert((kTmemColumns - 2 * 192) / kSlotColumns >= kGroups / 2, "too few slots");
constexpr int kWeightWarp = 0, kTokenWarp = 3, kEpilogueWarp = 4, kWidenWarp = 8;

// Largest token tile: a unit's two accumulators (and, for int8, two slots of
// widened W) share 512 TMEM columns; a single CTA takes short tiles only.
__host__ __device__ constexpr int max_tokens(int cg, bool int8) {
    return cg == 1 ? 64 : (int8 ? 192 : 256);
}
// Largest token tile whose K is split: what a join receives takes its room from the
// ring (32 to 56 KB at 128 columns).  256 columns over two pairs, not measured, would
// cost 256 x 8192 x 8192 in e4m3 32.1 thousand clocks by the model below, the cut taken
// (128 columns, K whole) 34.0.
constexpr int kJoinTokens = 128;
// Staging of the output: two chunks of 32 tokens (bf16) or 16 (fp32) x 128
// channels for TMA to store.
constexpr int kChunkBytes = 8192;

// W that a launch warms L2 with before the one before it has ended: 24 x 8192 x
// 1024 in e4m3 4.84 -> 3.55 us, 64 x 8192 x 8192 in int8 19.3 -> 18.2 (4 MB:
// 4.06 and 18.6; 16 MB, which stands in the way of the other launch's reads:
// 3.55 and 18.9).
constexpr int64_t kWarmBytes = int64_t{8} << 20;

struct Header {
    uint64_t full[kRingStages], empty[kRingStages];
    uint64_t wide_full[kWideSlots], wide_empty[kWideSlots];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t joined, drained;
    uint32_t tmem;
    int abort;
    alignas(16) float x_scale[4][256];  // each epilogue warp's copy of its tile's
};
constexpr int kHeaderBytes = 5120;
static_assert(sizeof(Header) <= kHeaderBytes, "header too large");

// All of an SM's shared memory: alignment, header, the pool that the ring and
// the slots are cut from, the output's staging.
constexpr int kSmemBytes = 232448;
constexpr int kPoolBytes = kSmemBytes - 1024 - kHeaderBytes - 2 * kChunkBytes;
static_assert(kPoolBytes % 1024 == 0, "the staging must stay aligned");

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
    int split;         // CTAs or pairs that share K
    int tma_out;       // rows of out are whole 16-byte units: stored by TMA
    int f32;           // output type
    int warm;          // stages of W each CTA warms L2 with
    // Shared memory and TMEM, cut to the tile: a stage holds 128 rows of W and
    // bn / CG of x, a slot the latter in f16 (two halves of K); accumulators
    // are acc_columns apart, the slots' W behind them.
    int stages, stage_bytes;
    int slots, slot_bytes;
    int acc_columns;
};

struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++at == n) {
            at = 0;
            phase ^= 1u;
        }
    }
    // On by k places, k <= n.
    __device__ __forceinline__ void skip(uint32_t k, uint32_t n) {
        at += k;
        if (at >= n) {
            at -= n;
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
__device__ __noinline__ bool warp_wait_slow(const GemmParams& p, uint32_t bar, uint32_t parity,
                                            volatile int* abort) {
    const bool ok = mbar_wait_slice<CLUSTER>(bar, parity, abort);
    if (__all_sync(0xffffffffu, ok)) return true;
    gave_up(p, abort);
    return false;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(const GemmParams& p, uint64_t* bar, uint32_t parity,
                                          volatile int* abort) {
    const uint32_t at = smem_addr(bar);
    // Mostly there already: a try and a vote.
    if (!CLUSTER && __all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
    return warp_wait_slow<CLUSTER>(p, at, parity, abort);
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

// This warp has read its part of an accumulator: hand it back to the leader.
__device__ __forceinline__ void release_acc(uint64_t& bar, uint32_t lead, int lane) {
    tcgen05_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(map_to_rank(smem_addr(&bar), lead));
}

// ------------------------------------------------------------- epilogue ---
// W columns (tokens) of a thread's share of an accumulator, as W registers:
//   lanes      column c + j of the thread's channel (TMEM lane)
//   fragments  (W = 16) 8x8 fragments of the warp's 32 channels x 16 columns:
//              registers 8 q + 4 i + 2 r + e of lane l hold channel
//              16 q + 8 r + l / 4, column c + 8 i + 2 (l % 4) + e
template <int W, bool FRAGMENTS>
__device__ __forceinline__ void read_acc(uint32_t (&v)[W], uint32_t d, int c) {
    if constexpr (FRAGMENTS) {
        tmem_load_fragments(reinterpret_cast<uint32_t(&)[8]>(v[0]), d + c);
        tmem_load_fragments(reinterpret_cast<uint32_t(&)[8]>(v[8]), d + (16u << 16) + c);
    } else if constexpr (W == 16) {
        tmem_load16(v, d + c);
    } else {
        tmem_load8(v, d + c);
    }
    tmem_wait_loads();
}

// Split K: unit q of the cluster adds up columns [q own, (q + 1) own).  The
// others' registers for them go to shared memory as they are (16 bytes of each
// of the 128 threads in turn; the ring, which their own products have left), and
// from there as one bulk copy each to a place that the unit they belong to keeps
// for them (in its ring they would have to ask first whether its products are
// done, with a release at cluster scope of about 1000 clocks).
struct Join {
    uint32_t outgoing, incoming, block;  // shared memory; bytes of one share
    int part, split, own;
    // Where sender q's share lies among the split - 1 of receiver r.
    __device__ __forceinline__ uint32_t place(int q, int r) const {
        return incoming + static_cast<uint32_t>(q < r ? q : q - 1) * block;
    }
};

template <int W, bool FRAGMENTS>
__device__ __forceinline__ void send_columns(const Join& g, uint32_t d, int etid) {
    for (int q = 0; q < g.split; ++q) {
        if (q == g.part) continue;
        uint32_t to = g.outgoing + q * g.block + etid * 16;
        for (int c = q * g.own; c < (q + 1) * g.own; c += W, to += W * kRows * 4) {
            uint32_t v[W];
            read_acc<W, FRAGMENTS>(v, d, c);
#pragma unroll
            for (int i = 0; i < W / 4; ++i) sts16(to + i * kRows * 16, v + 4 * i);
        }
    }
}

// The sum over the cluster (in rank order) of columns c to c + W - 1.
template <int W, bool FRAGMENTS, bool SPLIT>
__device__ __forceinline__ void read_columns(float (&y)[W], const Join& g, uint32_t d, int c,
                                             int etid) {
    uint32_t v[W];
    read_acc<W, FRAGMENTS>(v, d, c);
    if constexpr (SPLIT) {
        const uint32_t from = (c - g.part * g.own) * (kRows * 4) + etid * 16;
#pragma unroll
        for (int j = 0; j < W; ++j) y[j] = 0.f;
        for (int q = 0; q < g.split; ++q) {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint4 w = q == g.part
                                    ? make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3])
                                    : lds16(g.place(q, g.part) + from + i * kRows * 16);
                y[4 * i] += __uint_as_float(w.x);
                y[4 * i + 1] += __uint_as_float(w.y);
                y[4 * i + 2] += __uint_as_float(w.z);
                y[4 * i + 3] += __uint_as_float(w.w);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) y[j] = __uint_as_float(v[j]);
    }
}

// What an epilogue thread knows of its tile: its channel, the tile's first
// token and its tokens inside the call, the token scales (shared memory).
struct Tile {
    int64_t n;
    int t0, n_tok, etid;
    const float* x_scale;
};

// The output's way out where its rows allow: through shared memory as
// [token][channel] and out by TMA, so that the rows of a chunk leave as whole
// lines beside the next chunk's reads (stored straight from registers, a
// column costs each warp about 50 clocks).  Two chunks are in turn; the 128
// threads of the epilogue fill one and call flush together, which sends it and
// returns with the other free.
//   fp32  16 tokens x 128 channels, rows of 512 bytes
//   bf16  32 tokens x 64 channels twice, rows of 128 bytes in the 128-byte
//         swizzle (16-byte piece i of token t at piece i ^ (t & 7)), which
//         keeps the transposing stores below free of bank conflicts
__device__ __forceinline__ void flush(const GemmParams& p, const CUtensorMap* out_map,
                                      uint32_t staging, int& chunk, const Tile& t, int c) {
    fence_async_shared();
    if (t.etid == 0) bulk_wait_read<0>();  // the other chunk's store, a chunk ago
    __syncwarp();
    named_barrier(1, 128);
    if (t.etid == 0) {
        const uint32_t from = staging + chunk * kChunkBytes;
        if (c < t.n_tok && t.n < p.N) {
            tma_store_2d(out_map, static_cast<int>(t.n), t.t0 + c, from);
            if (!p.f32 && t.n + 64 < p.N)
                tma_store_2d(out_map, static_cast<int>(t.n) + 64, t.t0 + c, from + kChunkBytes / 2);
        }
        bulk_commit();
    }
    __syncwarp();
    chunk ^= 1;
}

// Every value is scaled first by its token's scale, then by its channel's (the
// product of two small scales alone could lose bits as a subnormal).
//
// bf16: a warp's fragments are scaled, packed (a register pair holds
// neighbouring tokens of a channel) and stored transposed: 2 stores per 16
// tokens instead of 16 narrow ones, in shared memory that the running products
// keep busy.  ws: the scales of the warp's channels lane / 4 + 8 i.
template <bool SPLIT, class Done>
__device__ __forceinline__ void emit_bf16(const GemmParams& p, const CUtensorMap* out_map,
                                          uint32_t staging, int& chunk, const Tile& t,
                                          const float (&ws)[4], const Join& g, uint32_t d, int c0,
                                          int c1, Done done) {
    const int lane = t.etid % 32;
    for (int c = c0; c < c1; c += 32) {
        const uint32_t to = staging + chunk * kChunkBytes;
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
            float y[16];
            read_columns<16, true, SPLIT>(y, g, d, c + k, t.etid);
            const float2 xs[2] = {
                *reinterpret_cast<const float2*>(t.x_scale + c + k + lane % 4 * 2),
                *reinterpret_cast<const float2*>(t.x_scale + c + k + 8 + lane % 4 * 2)};
            if (k == 16 && c + 32 >= c1) done();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // Matrix i: channels 16 q + 8 (i % 2) on, tokens 8 (i / 2) on.
                    const float w = ws[2 * q + i % 2];
                    const __nv_bfloat162 two =
                        __floats2bfloat162_rn(y[8 * q + 2 * i] * xs[i / 2].x * w,
                                              y[8 * q + 2 * i + 1] * xs[i / 2].y * w);
                    m[i] = *reinterpret_cast<const uint32_t*>(&two);
                }
                // Lane 8 m + j gives the place of matrix m's token j.
                const int row = k + lane / 16 * 8 + lane % 8;
                const int piece = t.etid / 32 * 4 + 2 * q + lane / 8 % 2;
                store_matrices_transposed(to + (piece >> 3) * (kChunkBytes / 2) + row * 128 +
                                              (((piece & 7) ^ (row & 7)) << 4),
                                          m[0], m[1], m[2], m[3]);
            }
        }
        flush(p, out_map, staging, chunk, t, c);
    }
}

// y[j] = v[j] * token scale * channel scale for this thread's channel.
template <int W>
__device__ __forceinline__ void scale_columns(float (&y)[W], const float* x_scale, float ws) {
#pragma unroll
    for (int j = 0; j < W; j += 4) {
        const float4 xs = *reinterpret_cast<const float4*>(x_scale + j);
        y[j] = y[j] * xs.x * ws;
        y[j + 1] = y[j + 1] * xs.y * ws;
        y[j + 2] = y[j + 2] * xs.z * ws;
        y[j + 3] = y[j + 3] * xs.w * ws;
    }
}

template <bool SPLIT, class Done>
__device__ __forceinline__ void emit_f32(const GemmParams& p, const CUtensorMap* out_map,
                                         uint32_t staging, int& chunk, const Tile& t, float ws,
                                         const Join& g, uint32_t d, int c0, int c1, Done done) {
    for (int c = c0; c < c1; c += 16) {
        float y[16];
        read_columns<16, false, SPLIT>(y, g, d, c, t.etid);
        if (c + 16 >= c1) done();
        scale_columns(y, t.x_scale + c, ws);
        const uint32_t to = staging + chunk * kChunkBytes + t.etid * 4;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + j * kRows * 4), "f"(y[j]) : "memory");
        flush(p, out_map, staging, chunk, t, c);
    }
}

// Rows of out that are not whole 16-byte units, or shares too short for a
// chunk: straight from registers.
template <int W, bool SPLIT, class Done>
__device__ __forceinline__ void emit_direct(const GemmParams& p, const Tile& t, float ws,
                                            const Join& g, uint32_t d, int c0, int c1, Done done) {
    for (int c = c0; c < c1; c += W) {
        float y[W];
        read_columns<W, false, SPLIT>(y, g, d, c, t.etid);
        if (c + W >= c1) done();
        scale_columns(y, t.x_scale + c, ws);
        const int64_t at = (static_cast<int64_t>(t.t0) + c) * p.N + t.n;
        if (p.f32) {
            float* out = static_cast<float*>(p.out) + at;
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (c + j < t.n_tok && t.n < p.N) out[j * p.N] = y[j];
        } else {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (c + j < t.n_tok && t.n < p.N) out[j * p.N] = __float2bfloat16_rn(y[j]);
        }
        __syncwarp();
    }
}

// SPLIT: the cluster's units share K (without it the compiler knows the pair's
// ranks, worth 3 to 7 % of the int8 kernel's time).
template <int CG, bool INT8, bool SPLIT>
__global__ void __launch_bounds__(INT8 ? 256 + 128 * kGroups : 256, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap x_map,
                const __grid_constant__ CUtensorMap w_map,
                const __grid_constant__ CUtensorMap out_map,
                const __grid_constant__ GemmParams p) {
    const uint32_t n_stages = p.stages, stage_bytes = p.stage_bytes;
    [[maybe_unused]] const uint32_t n_slots = p.slots, slot_bytes = p.slot_bytes;
    const uint32_t acc_columns = p.acc_columns;
    extern __shared__ unsigned char raw_smem[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t{1023});
    Header& h = *reinterpret_cast<Header*>(smem);
    const uint32_t ring = smem_addr(smem) + kHeaderBytes;
    [[maybe_unused]] const uint32_t slots = ring + n_stages * stage_bytes;
    const uint32_t staging = ring + kPoolBytes;
    volatile int* abort = &h.abort;

    // A warp index the compiler knows to be the same in all lanes: the MMA
    // warp's operands then live in uniform registers.
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = threadIdx.x % 32;
    // The cluster's CTAs (CG 1) or pairs (CG 2) split K: `part` is this one's
    // share, `half` the CTA of a pair, `lead` the rank that issues its MMAs.
    const uint32_t rank = __shfl_sync(0xffffffffu, cluster_cta_rank(), 0);
    const uint32_t unit = __shfl_sync(0xffffffffu, cluster_id_x(), 0);
    const uint32_t units = __shfl_sync(0xffffffffu, cluster_count_x(), 0);
    const int half = CG == 2 ? static_cast<int>(rank & 1) : 0;
    const int part = SPLIT ? static_cast<int>(rank) / CG : 0;
    const uint32_t lead = SPLIT || CG == 1 ? rank - half : 0;
    const bool leader = half == 0;
    const uint16_t pair = static_cast<uint16_t>(3u << lead);
    const int split = SPLIT ? p.split : 1;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * part / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (part + 1) / split);
    const int bn_cta = p.bn / CG;  // token rows this CTA loads

    if (warp == kTokenWarp && unit < static_cast<uint32_t>(p.channel_tiles)) {
        // The first stages of W on their way into L2 while the CTA sets up and
        // the launch before this one ends (a hint that reads nothing: what that
        // launch writes is seen all the same).
        const uint32_t one = elect_one();
        const int row = static_cast<int>(unit) * (kRows * CG) + half * kRows;
        for (int kb = kb0; kb < kb1 && kb - kb0 < p.warm; ++kb)
            tma_warm_2d(&w_map, kb * kBlockK, row, one);
    }
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < n_stages; ++s) {
            mbar_init(smem_addr(&h.full[s]), 2);  // W, x
            mbar_init(smem_addr(&h.empty[s]), INT8 ? 8 : 1);
        }
        for (int c = 0; c < kWideSlots; ++c) {
            mbar_init(smem_addr(&h.wide_full[c]), 8 * CG);
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
            mbar_arrive_expect_tx(smem_addr(&h.joined),
                                  static_cast<uint32_t>((p.bn - p.bn / split) * kRows * 4));
        tensormap_prefetch(&x_map);
        tensormap_prefetch(&w_map);
    }
    if (warp == 1) tmem_alloc<CG>(smem_addr(&h.tmem), kTmemColumns);
    tcgen05_fence_before();
    __syncthreads();
    // The peers' barriers must be initialised before anything arrives there.
    if (CG == 2 || split > 1) cluster_barrier();
    tcgen05_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, h.tmem, 0);
    [[maybe_unused]] const uint32_t wide = tmem + 2 * acc_columns;
    grid_dependency_wait();
    grid_launch_dependents();

    if (warp == kWeightWarp || warp == kTokenWarp) {
        // ------------------------------------------------------- TMA -----
        // One warp loads W, one x.  As in the MMA warp, the whole warp walks
        // and one lane issues.
        const bool weights = warp == kWeightWarp;
        const CUtensorMap* map = weights ? &w_map : &x_map;
        const uint32_t place = ring + (weights ? 0 : kRows * kBlockK);
        const uint32_t bytes = static_cast<uint32_t>((weights ? kRows : bn_cta) * kBlockK);
        const uint32_t one = elect_one();
        Ring r;
        uint32_t issued = 0;
        bool ok = true;
        for (uint32_t tile = unit; ok && tile < static_cast<uint32_t>(p.tiles); tile += units) {
            const int row = weights ? static_cast<int>(tile % p.channel_tiles) * (kRows * CG) +
                                          half * kRows
                                    : static_cast<int>(tile / p.channel_tiles) * p.bn +
                                          half * bn_cta;
            for (int kb = kb0; kb < kb1; ++kb, ++issued, r.next(n_stages)) {
                ok = warp_wait(p, &h.empty[r.at], r.phase ^ 1u, abort);
                if (!ok) break;
                // e4m3 pairs: both CTAs' copies count on the leader's barrier,
                // which alone issues the products; int8: on this CTA's, whose
                // warps widen them.
                const uint32_t local = smem_addr(&h.full[r.at]);
                const uint32_t bar = CG == 2 && !INT8 ? map_to_rank(local, lead) : local;
                if (INT8 || leader) mbar_arrive_expect_tx(local, INT8 ? bytes : bytes * CG, one);
                tma_load_2d<INT8 ? 1 : CG>(place + r.at * stage_bytes, map, kb * kBlockK, row,
                                           bar, one);
            }
        }
        if (lane == 0 && *abort && (INT8 || leader)) {
            // The copies in flight must land before the CTA may leave.
            for (uint32_t k = 0; k < n_stages && k < issued; ++k) {
                if (r.at == 0) {
                    r.at = n_stages - 1;
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
        // The whole warp walks the stages and one elected lane issues: with
        // the operands in warp-uniform code a stage's MMAs issue in a fraction
        // of the time a lone lane takes.
        // int8: beside sixteen widening warps every instruction of this one
        // counts.  One hand-over per 128 elements of K instead of 64 took 512 x
        // 8192 x 8192 from 62.6 to 57.1 us; issuing in a branch of its own, not
        // under a predicate of each MMA, took it from 49 to 46.5 (e4m3, whose
        // warp has no such neighbours, was 5 % slower so).
        Ring r, acc;
        bool ok = true;
        const uint32_t shape = mma_shape(kRows * CG, static_cast<uint32_t>(p.bn));
        const uint32_t one = elect_one();
        [[maybe_unused]] const uint32_t slot_operand = smem_operand(slots);
        [[maybe_unused]] const uint32_t ring_operand = smem_operand(ring);
        for (uint32_t tile = unit; ok && tile < static_cast<uint32_t>(p.tiles);
             tile += units, acc.next(2)) {
            ok = warp_wait(p, &h.acc_empty[acc.at], acc.phase ^ 1u, abort);
            if (!ok) break;
            tcgen05_fence_after();
            const uint32_t d = tmem + acc.at * acc_columns;
            if constexpr (INT8) {
                const int n = kb1 - kb0;
                for (int k = 0; k < n; ++k, r.next(n_slots)) {
                    ok = warp_wait(p, &h.wide_full[r.at], r.phase, abort);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t b = slot_operand + r.at * (slot_bytes >> 4);
                    const uint32_t a = wide + r.at * kSlotColumns;
                    if (one) {
#pragma unroll
                        for (int i = 0; i < kBlockK / 16; ++i)
                            mma_f16_tmem<CG>(d, a + 8 * i,
                                             b + (i / 4) * (slot_bytes >> 5) + 2 * (i % 4), shape,
                                             k > 0 || i > 0, 1u);
                        mma_commit<CG>(smem_addr(&h.wide_empty[r.at]), pair, 1u);
                    }
                }
            } else {
                const int n = kb1 - kb0;
                for (int k = 0; k < n; ++k, r.next(n_stages)) {
                    ok = warp_wait(p, &h.full[r.at], r.phase, abort);
                    if (!ok) break;
                    tcgen05_fence_after();
                    // (The maximum of equal numbers: a warp-uniform one.)
                    const uint32_t at = __reduce_max_sync(0xffffffffu, r.at);
                    const uint32_t a = ring_operand + at * (stage_bytes >> 4);
                    const uint32_t b = a + (kRows * kBlockK >> 4);
#pragma unroll
                    for (int i = 0; i < kBlockK / 32; ++i)
                        mma_e4m3<CG>(d, a + 2 * i, b + 2 * i, shape, k > 0 || i > 0, one);
                    mma_commit<CG>(smem_addr(&h.empty[r.at]), pair, one);
                }
            }
            if (ok) mma_commit<CG>(smem_addr(&h.acc_full[acc.at]), pair, one);
        }
        if (!ok) {
            // Products in flight still read shared memory and write TMEM.
            mma_commit<CG>(smem_addr(&h.drained), pair, one);
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
                              half * kRows + etid;
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
            const uint32_t d = tmem + acc.at * acc_columns + lanes;
            const Tile t{n, t0, p.M - t0 < p.bn ? p.M - t0 : p.bn, etid, x_scale};
            // Fragments for the transposing stores, lanes otherwise.
            const bool fragments = p.tma_out && !p.f32;
            Join g{};
            if constexpr (SPLIT) {
                const int own = p.bn / split;  // a multiple of 8 (tma_out: of a chunk)
                const uint32_t block = static_cast<uint32_t>(own * kRows * 4);
                g = Join{ring, staging - (split - 1) * block, block, part, split, own};
                if (fragments)
                    send_columns<16, true>(g, d, etid);
                else
                    send_columns<8, false>(g, d, etid);
                fence_async_shared();
                named_barrier(1, 128);
                if (etid == 0) {
                    for (int q = 0; q < split; ++q) {
                        if (q == part) continue;
                        const uint32_t dest = static_cast<uint32_t>(q * CG + half);
                        bulk_push(map_to_rank(g.place(part, q), dest), g.outgoing + q * block,
                                  block, map_to_rank(smem_addr(&h.joined), dest));
                    }
                }
                __syncwarp();
                const bool in = warp_wait<true>(p, &h.joined, 0, abort);
                if (named_barrier_or(1, 128, !in)) break;
            }
            const int c0 = SPLIT ? part * g.own : 0, c1 = SPLIT ? c0 + g.own : p.bn;
            const auto done = [&]() {
                if constexpr (!SPLIT) release_acc(h.acc_empty[acc.at], lead, lane);
            };
            if (fragments) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __shfl_sync(0xffffffffu, ws, lane / 4 + 8 * i);
                emit_bf16<SPLIT>(p, &out_map, staging, chunk, t, w, g, d, c0, c1, done);
            } else if (p.tma_out) {
                if constexpr (SPLIT)
                    emit_direct<8, SPLIT>(p, t, ws, g, d, c0, c1, done);
                else
                    emit_f32<SPLIT>(p, &out_map, staging, chunk, t, ws, g, d, c0, c1, done);
            } else {
                emit_direct<SPLIT ? 8 : 16, SPLIT>(p, t, ws, g, d, c0, c1, done);
            }
            if (SPLIT) break;  // one tile per cluster
        }
        if (etid == 0) bulk_wait_read<0>();
    } else if (INT8 && warp >= kWidenWarp) {
        // ------------------------------------------------- widening ------
        // Two groups of four warps widen a stage, a 64-element half of K each
        // (row `row` of W into TMEM lane `row`, and the token rows), the other
        // two the next one.
        const int group = (warp - kWidenWarp) / 4;
        const int upper = group % 2;
        const int row = threadIdx.x % 128;
        // 16-byte chunks of the token rows per thread: 32 rows x 4 chunks at
        // a time, this warp's first row x_row0.
        constexpr int kTokenChunks = max_tokens(CG, true) / CG / 32;
        const int x_row0 = row / 32 * 8, x_row = x_row0 + (row & 7), x_chunk = row / 8 % 4;
        const uint32_t lanes = static_cast<uint32_t>(row / 32 * 32) << 16;
        // Where this thread reads in a stage (16-byte chunk i of row R lies at
        // chunk i ^ (R & 7): neighbouring chunks are an exclusive or of 16
        // apart) and writes in a slot.  Eight neighbouring threads take one
        // chunk of eight rows: eight different bank groups, read and written.
        const uint32_t w_at = row * kBlockK + (((upper * 4) ^ (row & 7)) << 4);
        const uint32_t x_at = kRows * kBlockK + x_row * kBlockK +
                              (((upper * 4 + x_chunk) ^ (x_row & 7)) << 4);
        const uint32_t slot_at = slots + upper * (slot_bytes / 2) + x_row * 128 +
                                 (((2 * x_chunk) ^ (x_row & 7)) << 4);
        const uint32_t wide_at = wide + lanes + upper * (kSlotColumns / 2);
        const uint32_t full_to = map_to_rank(smem_addr(&h.wide_full[0]), lead);
        Ring r, c;  // of stages, of slots
        const int first = static_cast<int>(unit);
        const int my_tiles =
            first < p.tiles ? (p.tiles - 1 - first) / static_cast<int>(units) + 1 : 0;
        const int64_t n = static_cast<int64_t>(my_tiles) * (kb1 - kb0);
        r.skip(group / 2, n_stages);
        c.skip(group / 2, n_slots);
        for (int64_t k = group / 2; k < n; k += kGroups / 2) {
            if (!warp_wait(p, &h.full[r.at], r.phase, abort)) break;
            const uint32_t stage = ring + r.at * stage_bytes;
            uint4 raw[4 + kTokenChunks];
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i] = lds16((stage + w_at) ^ (i << 4));
#pragma unroll
            for (int i = 0; i < kTokenChunks; ++i)
                if (i * 32 + x_row0 < bn_cta)
                    raw[4 + i] = lds16(stage + x_at + i * 32 * kBlockK);
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) widen16(raw[i], w + 8 * i);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&h.empty[r.at]));
            if (!warp_wait(p, &h.wide_empty[c.at], c.phase ^ 1u, abort)) break;
            tcgen05_fence_after();
            tmem_store32(wide_at + c.at * kSlotColumns, w);
            const uint32_t slot = slot_at + c.at * slot_bytes;
#pragma unroll
            for (int i = 0; i < kTokenChunks; ++i)
                if (i * 32 + x_row0 < bn_cta) {
                    uint32_t x[8];
                    widen16(raw[4 + i], x);
                    sts16(slot + i * 32 * 128, x);
                    sts16((slot + i * 32 * 128) ^ 16, x + 4);
                }
            fence_async_shared();
            tmem_wait_stores();
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(full_to + c.at * 8);
            r.skip(kGroups / 2, n_stages);
            c.skip(kGroups / 2, n_slots);
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

template <int CG, bool INT8>
void* gemm_entry(bool split) {
    return split ? reinterpret_cast<void*>(&gemm_kernel<CG, INT8, true>)
                 : reinterpret_cast<void*>(&gemm_kernel<CG, INT8, false>);
}

void* gemm_kernel_for(int cg, bool int8, bool split) {
    if (cg == 1) return int8 ? gemm_entry<1, true>(split) : gemm_entry<1, false>(split);
    return int8 ? gemm_entry<2, true>(split) : gemm_entry<2, false>(split);
}

// Launch configuration of `grid` CTAs in clusters; attr[0] is the cluster's.
void cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int cluster, int grid,
                    int cg, bool int8) {
    cfg->gridDim = dim3(static_cast<unsigned>(grid));
    cfg->blockDim = dim3(int8 ? 256 + 128 * kGroups : 256);
    cfg->dynamicSmemBytes = kSmemBytes;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg->attrs = attr;
}

// How a call is cut up.
struct Plan {
    int cg = 0, split = 1, bn = 0;
    int64_t token_tiles = 0, tiles = 0;
    double cost = 0;
};

// The cheapest of the cuts a call allows, by the clocks its busiest unit takes
// (fitted to sweeps of every cut over 13 shapes from 16 x 8192 x 1024 to
// 1024 x 8192 x 8192; over these and four more the cut taken was the best or
// within 4 % of it, but for e4m3 200 x 2048 x 5120, 8 % behind).
//   A ring stage costs what a unit's hand-overs of it do, plus its products
//   (Costs: lone CTA, pair); together never less than reading W and x once.
//   The last tile's way out adds a cost per column, a split the join of its
//   shares.
struct Costs {
    double stage[2], stage_column[2], out_column, join, join_part, join_column;
};
constexpr Costs kCosts[2] = {
    {{350, 340}, {0.88, 1.26}, 15, 860, 520, 20},   // e4m3; lone CTA, pair
    {{580, 570}, {0.8, 1.1}, 70, 4600, 390, 11}};   // int8
Plan plan(int64_t M, int64_t N, int k_blocks, bool int8, int64_t sms, const DeviceInfo& d) {
    Plan best;
    const Costs& k = kCosts[int8];
    // 6.3 TB/s at 1.9 GHz: 3300 bytes a clock.
    const double once = static_cast<double>(M + N) * k_blocks * kBlockK / 3300.0;
    for (int cg = 1; cg <= 2; ++cg) {
        const int most_bn = max_tokens(cg, int8);
        const int64_t channel_tiles = (N + kRows * cg - 1) / (kRows * cg);
        for (int bn = cg == 1 ? 16 : 32; bn <= most_bn; bn += bn < 32 ? 16 : 32) {
            if (bn >= M + 32 && bn > 32) break;
            Plan c;
            c.cg = cg;
            c.bn = bn;
            c.token_tiles = (M + bn - 1) / bn;
            c.tiles = channel_tiles * c.token_tiles;
            const double stage = k.stage[cg - 1] + k.stage_column[cg - 1] * bn;
            for (int split = 1, log2 = cg - 1; log2 < 4 && split <= k_blocks; split *= 2, ++log2) {
                int64_t units = sms >> log2;
                const int at_once = d.gemm_clusters[cg - 1][int8][log2];
                if (units > at_once) units = at_once;
                if (units < 1 || (split > 1 && c.tiles > units)) break;
                // Whole chunks of the output's staging, or eights of a share.
                if (bn % (split == 1 ? 32 : 8 * split) != 0) continue;
                if (split > 1 && bn > kJoinTokens) break;
                const int64_t waves = (c.tiles + units - 1) / units;
                c.split = split;
                const double main =
                    static_cast<double>(waves * ((k_blocks + split - 1) / split)) * stage;
                c.cost = (main > once ? main : once) + k.out_column * bn;
                if (split > 1)
                    c.cost += k.join + k.join_part * split + k.join_column * bn;
                if (best.cg == 0 || c.cost < best.cost) best = c;
            }
        }
    }
    return best;
}

}  // namespace

int gemm_prepare(int smem_optin, int (*clusters)[2][4]) {
    if (kSmemBytes > smem_optin) return static_cast<int>(cudaErrorInvalidValue);
    for (int cg = 1; cg <= 2; ++cg)
        for (bool int8 : {false, true}) {
            cudaError_t e;
            for (bool split : {false, true})
                if ((e = cudaFuncSetAttribute(gemm_kernel_for(cg, int8, split),
                                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              kSmemBytes)) != cudaSuccess)
                    return static_cast<int>(e);
            // Clusters of 1, 2, 4 and 8 CTAs that run at once (they do not
            // cross a GPC, so a few SMs can be out of reach).
            for (int i = 0; i < 4; ++i) {
                cudaLaunchConfig_t cfg = {};
                cudaLaunchAttribute attr[1];
                cluster_config(&cfg, attr, 1 << i, 1 << i, cg, int8);
                cfg.numAttrs = 1;
                int n = 0;
                void* fn = gemm_kernel_for(cg, int8, (1 << i) > cg);
                e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
                if (e != cudaSuccess) return static_cast<int>(e);
                clusters[cg - 1][int8][i] = n;
            }
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
    GemmParams p{};
    p.x_scale = g.x_scale;
    p.w_scale = g.w_scale;
    p.out = g.out;
    p.status = d.status;
    p.N = g.N;
    p.M = static_cast<int>(g.M);
    p.k_blocks = static_cast<int>((g.K + kBlockK - 1) / kBlockK);
    p.f32 = g.dtype == TW_F32;
    const Plan c = plan(g.M, g.N, p.k_blocks, int8, sms, d);
    if (c.cg == 0 || c.tiles > (int64_t{1} << 31) - 1 - sms)
        return static_cast<int>(cudaErrorInvalidValue);
    const int cg = c.cg;
    p.tiles = static_cast<int>(c.tiles);
    p.channel_tiles = static_cast<int>(c.tiles / c.token_tiles);
    p.split = c.split;
    p.bn = c.bn;
    // As many slots as TMEM has room for behind the accumulators, then as many
    // stages as fit (two slots and five stages at bn = 192).
    p.acc_columns = c.bn < 32 ? 32 : c.bn;
    p.stage_bytes = (kRows + c.bn / cg) * kBlockK;
    p.slot_bytes = c.bn / cg * kBlockK * 2;
    p.slots = int8 ? (kTmemColumns - 2 * p.acc_columns) / kSlotColumns : 0;
    if (p.slots > kWideSlots) p.slots = kWideSlots;
    const int pool = kPoolBytes - (c.bn - c.bn / c.split) * kRows * 4;  // less the join's
    for (;; --p.slots) {
        p.stages = (pool - p.slots * p.slot_bytes) / p.stage_bytes;
        if (p.stages > kRingStages) p.stages = kRingStages;
        // An odd number of stages hands a place of the ring from one pair of
        // widening groups to the other, and a wait by parity must not look at
        // it before the other's load k has landed.  Who is about to widen
        // stage k + stages has seen the products of k + stages - 2 - slots
        // done, which must not lie before k.
        // (An even number is fine if it is more than the slots: 4 and 4 were 5 %
        // slower than 6 and 3.)
        if (!int8 || p.stages >= p.slots + 2 || (p.stages % 2 == 0 && p.stages > p.slots)) break;
    }
    const int64_t es = p.f32 ? 4 : 2;
    p.tma_out = g.N * es % 16 == 0 && p.bn / p.split % (p.f32 ? 16 : 32) == 0;
    CUtensorMap x_map, w_map, out_map{};
    if (!encode_operand(&x_map, g.x, g.M, g.K, p.bn / cg) ||
        !encode_operand(&w_map, g.w, g.N, g.K, kRows) ||
        (p.tma_out && !encode(&out_map,
                              p.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              es, g.out, g.M, g.N, p.f32 ? kRows : kRows / 2, p.f32 ? 16 : 32,
                              p.f32 ? CU_TENSOR_MAP_SWIZZLE_NONE
                                    : CU_TENSOR_MAP_SWIZZLE_128B)))
        return static_cast<int>(cudaErrorInvalidValue);

    const int cluster = cg * p.split;
    const int64_t most = sms / cluster;
    const int64_t units = c.tiles < most ? c.tiles : most;
    const int64_t reading = units < p.channel_tiles ? units : p.channel_tiles;
    p.warm = static_cast<int>(kWarmBytes / (reading * cluster * kRows * kBlockK));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cluster_config(&cfg, attr, cluster, static_cast<int>(units * cluster), cg, int8);
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = max_sms >= d.sm_count ? 2 : 1;
    void* args[] = {&x_map, &w_map, &out_map, &p};
    void* fn = gemm_kernel_for(cg, int8, p.split > 1);
    return static_cast<int>(cudaLaunchKernelExC(&cfg, fn, args));
}

}  // namespace tw
