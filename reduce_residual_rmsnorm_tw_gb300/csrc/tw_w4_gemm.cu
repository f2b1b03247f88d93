// tw_w4_gemm.cu -- the product on 4-bit weights with group scales, for few
// tokens: out[t,n] = xs[t] sum_g s[n,g] sum_{k in g} x[t,k] q[n,k].
//
// Bound by reading W once from HBM, half a byte per weight.  The weights become
// bf16 in registers (exact for both types) and feed m16n8k16 with fp32 sums; a
// group's sum is scaled and added to the row's in fp32.  x becomes bf16 without
// loss on its way into shared memory: 8-bit values as they are, fp32 as three
// terms of eight bits each, which count as three tokens.
//
// A tile of W lies in HBM as the lanes read it (tw.h): lane (g, q) takes 16 bytes
// of row g and 16 of row g + 8; word j holds k = 32 j + 8 q .. + 7, so that a word's
// two MMAs stay within 32 k and a group of 32 can be scaled on its own.  A stripe of
// 16 channels is contiguous, so a tile is one bulk copy into the warp's own ring in
// shared memory, a few tiles ahead, with no barrier but the copy's.
//
// Two CTAs of eight warps share an SM, so that one streams while the other starts,
// joins or stores.  A CTA holds x of its K in shared memory and takes an even share
// of the stripes, `at_once` of them at a time: as many warps share a stripe, each a
// contiguous piece of its K, and their sums are joined through shared memory in warp
// order.  A cluster of CTAs may split K as well (where x would not fit, or its copies
// into every SM would outweigh W), and joins through distributed shared memory in
// rank order.
#include <cuda_fp16.h>

#include "tw_tcgen05.cuh"

namespace tw {
namespace {

// Tiles of a bulk copy, and copies that a warp's ring holds: few and long where one
// block of columns leaves the room (8 x 8192 x 8192 15.1 -> 13.2 us, 1 10.8 -> 10.5;
// with more columns short ones, so that three or four of them fit beside x).
__host__ __device__ constexpr int chunk_of(int nt) { return nt == 1 ? 4 : 2; }
__host__ __device__ constexpr int max_slots(int nt) { return nt == 1 ? 2 : 4; }
constexpr int kMinSlots = 2, kMaxSlots = 4;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kXPad = 32;  // bf16: rows of x 64 bytes off each other in the banks
constexpr int kXAhead = 4;
constexpr int kColumnsMax = 32;  // tokens at a time (fp32 x: three for one)

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}
// `bytes` of global memory to shared memory, counted on `bar` (multiples of 16).
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A word's eight values as four pairs of bf16, (k, k + 1) for k = 0, 2, 4, 6: the
// values themselves (e2m1) or times 2^-7 (int4; the factor comes back in at the
// end, so results below 2^-119 in magnitude may lose bits).  bf16 numbers below
// 2^-125 are their last eight bits times 2^-133, so that two nibbles in eight need no
// shift.
constexpr float kInt4Factor = 128.f;
template <bool INT4>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&h)[4]) {
    if constexpr (INT4) {
        // u 2^-133 2^126 - 8 2^-7 and 16 u 2^-133 2^122 - 8 2^-7.
        const uint32_t w8 = w >> 8;
        const uint32_t u[4] = {w & 0x000f000fu, w & 0x00f000f0u, w8 & 0x000f000fu,
                               w8 & 0x00f000f0u};
#pragma unroll
        for (int v = 0; v < 4; ++v)
            asm("fma.rn.bf16x2 %0, %1, %2, %3;"
                : "=r"(h[v])
                : "r"(u[v]), "r"(v % 2 ? 0x7c807c80u : 0x7e807e80u), "r"(0xbd80bd80u));
    } else {
        // Sign and exponent bits in bf16's places are the value times 2^-126.
        h[0] = w & 0x81c081c0u;
        h[1] = w << 3 & 0x81c081c0u;
        h[2] = (w >> 3 & 0x01c001c0u) | (w << 1 & 0x80008000u);
        h[3] = (w << 6 & 0x01c001c0u) | (w << 2 & 0x80008000u);
#pragma unroll
        for (int v = 0; v < 4; ++v)
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(h[v]) : "r"(0x7e807e80u));
    }
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight values of x as they lie in memory: 16 bytes of bf16, 32 of fp32, 8 of
// 8-bit values.
struct XEight {
    uint4 v[2];
    __device__ __forceinline__ void load(const char* from, int xtype) {
        if (xtype >= TW_X_INT8) {
            const uint2 b = *reinterpret_cast<const uint2*>(from);
            v[0].x = b.x;
            v[0].y = b.y;
            return;
        }
        v[0] = ld_global(from);
        if (xtype == TW_X_F32) v[1] = ld_global(from + 16);
    }
};

// They as bf16 in terms[0] (8-bit and bf16) or as three terms that add up to them
// (fp32: the leading eight bits, cut off, then the next eight, then the rest; an
// infinity or a NaN as its own first term).
__device__ __forceinline__ void x_terms(const XEight& x, int xtype, uint4 (&terms)[3]) {
    if (xtype == TW_X_BF16) {
        terms[0] = x.v[0];
    } else if (xtype == TW_X_F32) {
        float f[8];
        Vec<float>::to_float(x.v[0], f);
        Vec<float>::to_float(x.v[1], f + 4);
        uint32_t w[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t[3][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float v = f[2 * i + h];
                const bool finite = fabsf(v) <= 3.402823466e38f;
                t[0][h] = finite ? __uint_as_float(__float_as_uint(v) & 0xffff0000u) : v;
                const float rest = finite ? v - t[0][h] : 0.f;
                t[1][h] = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
                t[2][h] = rest - t[1][h];
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) w[p][i] = pack_bf16(t[p][0], t[p][1]);
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) terms[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = (i < 2 ? x.v[0].x : x.v[0].y) >> (i % 2 * 16) & 0xffffu;
            if (xtype == TW_X_INT8) {
                w[i] = pack_bf16(static_cast<float>(static_cast<int8_t>(two & 0xffu)),
                                 static_cast<float>(static_cast<int8_t>(two >> 8)));
            } else {
                uint32_t h;
                asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\t"
                    "cvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
                    : "=r"(h)
                    : "r"(two));
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                w[i] = pack_bf16(f.x, f.y);
            }
        }
        terms[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Floats between the columns of a warp's sums.
constexpr int kRowStride = kW4Channels + 1;
// Tiles that a warp warms L2 with before the launch before this one has ended.
constexpr int kWarm = 16;
// Tiles of x that a CTA holds at a time.
__host__ __device__ constexpr int x_tiles(int tiles, int split, int slices) {
    return ((tiles + split - 1) / split + slices - 1) / slices;
}

struct W4Plan {
    W4GemmArgs a;
    int tokens;       // at a time
    int log_at_once;  // stripes of a CTA at a time
    int log_split;    // CTAs of a cluster, which split K
    int slots;        // of a warp's ring
    int slices;       // of a CTA's K, whose x is in shared memory one after the other
    unsigned int* status;
};

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) {
    return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}
// The scales of rows g and g + 8 for a tile's groups.
template <int G>
__device__ __forceinline__ void lds_scales(uint32_t (&s)[128 / G], uint32_t addr) {
    if constexpr (G == 128)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(s[0]) : "r"(addr));
    else if constexpr (G == 64)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(s[0]), "=r"(s[1]) : "r"(addr));
    else
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3])
                     : "r"(addr));
}

// A warp's way through its CTA's stripes: rounds of up to 2^log_at_once stripes (fewer
// in the last), each round in slices of K, in each a contiguous piece of a stripe's
// tiles.
struct Way {
    int at, end;    // the round's first stripe and the CTA's last
    int log_n;      // stripes of the round
    int stripe;     // this warp's
    __device__ __forceinline__ void round(int log_at_once, int warp) {
        log_n = log_at_once;
        while (log_n > 0 && (1 << (log_n - 1)) >= end - at) --log_n;
        stripe = at + (warp << log_n) / kWarps;
    }
    // This warp's first tile and tiles of [lo, hi).
    __device__ __forceinline__ void piece(int warp, int lo, int hi, int* first, int* n) const {
        const int shares = kWarps >> log_n, share = warp & (shares - 1);
        *first = lo + (hi - lo) * share / shares;
        *n = stripe < end ? lo + (hi - lo) * (share + 1) / shares - *first : 0;
    }
};

// INT4: the weights' type; NT: blocks of eight columns of x (fp32: three per token);
// G: the group.
template <bool INT4, int NT, int G>
__global__ void __launch_bounds__(kThreads, 2)
    w4_gemm_kernel(const __grid_constant__ W4Plan plan) {
    constexpr int kTile = w4_tile_bytes(G);
    constexpr int kChunk = chunk_of(NT), kSlot = kChunk * kTile;
    constexpr int kColumns = NT * 8;
    const W4GemmArgs& a = plan.a;
    extern __shared__ __align__(128) unsigned char smem[];
    float* part = reinterpret_cast<float*>(smem);  // [warp][column][kRowStride]
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = threadIdx.x % 32;
    const int row = lane / 4, quad = lane % 4;
    const int parts = a.xtype == TW_X_F32 ? 3 : 1;
    const int K = static_cast<int>(a.K);
    const int tiles_k = (K + kW4Inner - 1) / kW4Inner;
    const int stripes = static_cast<int>((a.N + kW4Channels - 1) / kW4Channels);
    // This CTA's share of K (of the cluster), cut into slices, and of the stripes.
    const int split = 1 << plan.log_split, slices = plan.slices;
    const int rank = split > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
    const int lo = tiles_k * rank / split, hi = tiles_k * (rank + 1) / split;
    auto slice_at = [&](int s) { return lo + (hi - lo) * s / slices; };
    const int64_t sets = gridDim.x / split, set = blockIdx.x / split;
    const int first = static_cast<int>(stripes * set / sets);
    const int end = static_cast<int>(stripes * (set + 1) / sets);
    const int x_stride = (x_tiles(tiles_k, split, slices) * kW4Inner + kXPad) * 2;
    // Sums that the cluster's CTAs write here: [buffer][rank][column][channel of this
    // rank's]; the rings; their barriers; x.
    float* joined = part + kWarps * kColumns * kRowStride;
    const int own = (kW4Channels << plan.log_at_once) / split;
    const uint32_t rings = smem_addr(joined) + (split > 1 ? 2 * split * kColumns * own * 4 : 0);
    const uint32_t ring = rings + warp * plan.slots * kSlot;
    const uint32_t bars = rings + kWarps * plan.slots * kSlot;
    const uint32_t bar = bars + warp * kMaxSlots * 8;
    const uint32_t xs = bars + kWarps * kMaxSlots * 8;

    if (lane == 0) {
        for (int i = 0; i < plan.slots; ++i) mbar_init(bar + i * 8, 1);
        mbar_init_fence();
    }
    __syncwarp();
    const char* packed = static_cast<const char*>(a.packed);
    Way ld{first, end, 0, 0};
    int ld_slice = 0, ld_first = 0, left = 0;
    const char* from = packed;
    auto begin = [&]() {
        ld.piece(warp, slice_at(ld_slice), slice_at(ld_slice + 1), &ld_first, &left);
        from = packed + (static_cast<int64_t>(ld.stripe) * tiles_k + ld_first) * kTile;
    };
    ld.round(plan.log_at_once, warp);
    begin();
    // The first W on its way into L2 while the launch before this one ends (a hint that
    // reads nothing: what that launch writes is seen all the same).
    if (lane == 0 && left > 0)
        bulk_prefetch_l2(from, static_cast<uint32_t>((left < kWarm ? left : kWarm) * kTile));
    if (split > 1) cluster_barrier();  // every CTA runs before any writes into it
    grid_dependency_wait();
    grid_launch_dependents();

    const uint32_t one = elect_one();
    uint32_t slot_ld = 0, slot = 0, phase = 0;
    int buf = 0;
    for (int64_t m0 = 0; m0 < a.M; m0 += plan.tokens) {
        const int tokens = static_cast<int>(a.M - m0 < plan.tokens ? a.M - m0 : plan.tokens);
        const int cols = tokens * parts;
        auto load = [&]() {
            while (left == 0) {  // a warp may be without tiles for whole rounds
                if (ld.at >= end) return;
                if (++ld_slice >= slices) {
                    ld_slice = 0;
                    ld.at += 1 << ld.log_n;
                    if (ld.at >= end) return;
                    ld.round(plan.log_at_once, warp);
                }
                begin();
            }
            const int n = left < kChunk ? left : kChunk;
            if (one) {
                mbar_arrive_expect_tx(bar + slot_ld * 8, n * kTile);
                bulk_copy(ring + slot_ld * kSlot, from, n * kTile, bar + slot_ld * 8);
            }
            from += kSlot;
            left -= n;
            if (++slot_ld == static_cast<uint32_t>(plan.slots)) slot_ld = 0;
        };
        ld = Way{first, end, 0, 0};
        ld.round(plan.log_at_once, warp);
        ld_slice = 0;
        begin();
        for (int d = 0; d < plan.slots; ++d) load();

        // x of a slice of this CTA's K, zero up to the end of its last tile; kXAhead
        // loads of a thread in flight.
        auto stage_x = [&](int slice) {
            const int x_size = a.xtype == TW_X_BF16 ? 2 : a.xtype == TW_X_F32 ? 4 : 1;
            const int k0 = slice_at(slice) * kW4Inner;
            const uint32_t row_pieces =
                static_cast<uint32_t>(slice_at(slice + 1) - slice_at(slice)) * (kW4Inner / 8);
            // The thread's next piece: the at-th of token t.
            uint32_t t = 0, at = threadIdx.x;
            const auto count = static_cast<uint32_t>(tokens);
            while (t < count) {
                XEight x[kXAhead] = {};
                uint32_t to[kXAhead];
                bool in[kXAhead];
#pragma unroll
                for (int i = 0; i < kXAhead; ++i, at += kThreads) {
                    while (at >= row_pieces && t < count) {
                        at -= row_pieces;
                        ++t;
                    }
                    in[i] = t < count;
                    to[i] = xs + t * parts * x_stride + at * 16;
                    const int64_t k = k0 + static_cast<int64_t>(at) * 8;
                    if (in[i] && k < K)
                        x[i].load(static_cast<const char*>(a.x) + ((m0 + t) * a.K + k) * x_size,
                                  a.xtype);
                }
#pragma unroll
                for (int i = 0; i < kXAhead; ++i) {
                    if (!in[i]) break;
                    uint4 terms[3];
                    x_terms(x[i], a.xtype, terms);
                    for (int p = 0; p < parts; ++p) sts128(to[i] + p * x_stride, terms[p]);
                }
            }
            __syncthreads();
        };
        if (slices == 1) stage_x(0);
        // Where the lane's rows of x begin.  Columns beyond the last repeat the first:
        // one read for all of them, and nothing of theirs is stored.
        uint32_t x_row[NT];
#pragma unroll
        for (int b = 0; b < NT; ++b)
            x_row[b] = xs + (b * 8 + row < cols ? b * 8 + row : 0) * x_stride + quad * 16;

        Way at{first, end, 0, 0};
        for (; at.at < end; at.at += 1 << at.log_n) {
            at.round(plan.log_at_once, warp);
            float total[NT][4] = {};
            for (int slice = 0; slice < slices; ++slice) {
                if (slices > 1) {
                    __syncthreads();  // the x before has been read
                    stage_x(slice);
                }
                int tile = 0, tiles = 0;
                at.piece(warp, slice_at(slice), slice_at(slice + 1), &tile, &tiles);
                uint32_t x_at = (tile - slice_at(slice)) * (kW4Inner * 2);
                for (int i = 0; i < tiles; i += kChunk) {
                    // (A copy that does not arrive: the device status says so.)
                    if (!mbar_wait_slice(bar + slot * 8, phase, nullptr))
                        atomicOr(plan.status, 1u);
                    const uint32_t t = ring + slot * kSlot + lane * 16;
                    const uint32_t ts = ring + slot * kSlot + 1024 + row * (512 / G);
#pragma unroll
                    for (int c = 0; c < kChunk; ++c, x_at += kW4Inner * 2) {
                        if (c > 0 && i + c >= tiles) break;
                        const uint4 w[2] = {lds128(t + c * kTile), lds128(t + c * kTile + 512)};
                        uint32_t s[128 / G];
                        lds_scales<G>(s, ts + c * kTile);
                        // Two chains of MMAs a group, so that one hides the other's latency.
                        float sum[2][NT][4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint4 xv[NT];
#pragma unroll
                            for (int b = 0; b < NT; ++b) xv[b] = lds128(x_row[b] + x_at + j * 64);
                            uint32_t u[4], v[4];
                            widen<INT4>(word_of(w[0], j), u);
                            widen<INT4>(word_of(w[1], j), v);
#pragma unroll
                            for (int b = 0; b < NT; ++b) {
                                if (j * 32 % G == 0) {
                                    mma_first(sum[0][b], u[0], v[0], u[1], v[1], xv[b].x, xv[b].y);
                                    mma_first(sum[1][b], u[2], v[2], u[3], v[3], xv[b].z, xv[b].w);
                                } else {
                                    mma(sum[0][b], u[0], v[0], u[1], v[1], xv[b].x, xv[b].y);
                                    mma(sum[1][b], u[2], v[2], u[3], v[3], xv[b].z, xv[b].w);
                                }
                            }
                            if ((j + 1) * 32 % G == 0) {
                                // The group is whole.
                                const float s0 = __uint_as_float(s[j * 32 / G] << 16);
                                const float s1 = __uint_as_float(s[j * 32 / G] & 0xffff0000u);
#pragma unroll
                                for (int b = 0; b < NT; ++b)
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        total[b][e] = fmaf(sum[0][b][e] + sum[1][b][e],
                                                           e < 2 ? s0 : s1, total[b][e]);
                            }
                        }
                    }
                    if (++slot == static_cast<uint32_t>(plan.slots)) {
                        slot = 0;
                        phase ^= 1u;
                    }
                    __syncwarp();  // every lane has read the slot
                    load();
                }
            }
            // The warps' sums, joined in warp order.
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    part[(warp * kColumns + b * 8 + quad * 2 + e % 2) * kRowStride + row +
                         e / 2 * 8] = total[b][e];
            __syncthreads();
            const int shares = kWarps >> at.log_n, log_channels = 4 + at.log_n;
            const int64_t n0 = static_cast<int64_t>(at.at) * kW4Channels;
            // Of column c, channel i of the round.
            auto sum_of = [&](int c, int i) {
                const float* from = part + ((i / 16 * shares) * kColumns + c) * kRowStride + i % 16;
                float sum = 0.f;
                for (int w = 0; w < shares; ++w) sum += from[w * kColumns * kRowStride];
                return sum;
            };
            auto store = [&](int t, int i, float sum) {
                if (n0 + i >= a.N || at.at + i / kW4Channels >= end) return;
                if (INT4) sum *= kInt4Factor;
                if (a.x_scale) sum *= a.x_scale[m0 + t];
                const int64_t to = (m0 + t) * a.N + n0 + i;
                if (a.dtype == TW_BF16)
                    static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(sum);
                else
                    static_cast<float*>(a.out)[to] = sum;
            };
            if (split == 1) {
                for (int e = threadIdx.x; e < tokens << log_channels; e += kThreads) {
                    const int t = e >> log_channels, i = e & ((1 << log_channels) - 1);
                    float sum = 0.f;
                    // fp32 x: the smaller terms first.
                    for (int p = parts - 1; p >= 0; --p) sum += sum_of(t * parts + p, i);
                    store(t, i, sum);
                }
                __syncthreads();  // the sums are read
            } else {
                // Rank q finishes channels [q, q + 1) * channels / split of the round.  A
                // buffer is written again two rounds later, behind the barrier that its
                // readers reach when done.
                const int log_own = log_channels - plan.log_split;
                float* sums = joined + buf * split * kColumns * own;
                for (int e = threadIdx.x; e < cols << log_channels; e += kThreads) {
                    const int c = e >> log_channels, i = e & ((1 << log_channels) - 1);
                    float* to = sums + (rank * kColumns + c) * own + (i & ((1 << log_own) - 1));
                    st_cluster_f32(map_to_rank(smem_addr(to), static_cast<uint32_t>(i >> log_own)),
                                   sum_of(c, i));
                }
                cluster_barrier();
                for (int e = threadIdx.x; e < tokens << log_own; e += kThreads) {
                    const int t = e >> log_own, i = e & ((1 << log_own) - 1);
                    float sum = 0.f;
                    for (int p = parts - 1; p >= 0; --p)
                        for (int r = 0; r < split; ++r)
                            sum += sums[(r * kColumns + t * parts + p) * own + i];
                    store(t, (rank << log_own) + i, sum);
                }
                buf ^= 1;
            }
        }
        __syncthreads();  // x is read
    }
}

template <bool INT4, int G>
void* entry(int nt) {
    return nt == 1   ? reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 1, G>)
           : nt == 2 ? reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 2, G>)
                     : reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 4, G>);
}
void* kernel_for(int wtype, int nt, int group) {
    if (wtype == TW_INT4)
        return group == 32 ? entry<true, 32>(nt) : group == 64 ? entry<true, 64>(nt)
                                                               : entry<true, 128>(nt);
    return group == 32 ? entry<false, 32>(nt) : group == 64 ? entry<false, 64>(nt)
                                                            : entry<false, 128>(nt);
}

// Shared memory of a CTA for `columns` columns of x in `nt` blocks.
int64_t smem_bytes(int nt, int columns, int64_t K, int group, const W4Plan& p) {
    const int64_t part = static_cast<int64_t>(kWarps) * nt * 8 * kRowStride * 4;
    const int64_t joined =
        p.log_split > 0 ? int64_t{2} * nt * 8 * (kW4Channels << p.log_at_once) * 4 : 0;
    const int64_t rings = kWarps * (p.slots * chunk_of(nt) * w4_tile_bytes(group) + kMaxSlots * 8);
    const int tiles = static_cast<int>((K + kW4Inner - 1) / kW4Inner);
    return part + joined + rings +
           static_cast<int64_t>(columns) *
               (x_tiles(tiles, 1 << p.log_split, p.slices) * kW4Inner + kXPad) * 2;
}
// What a CTA may use where two share an SM.
int64_t half_smem(int smem_optin) { return (smem_optin - 1024) / 2; }

cudaLaunchConfig_t config(int grid, int split, size_t smem, bool pdl, void* stream,
                          cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cfg;
}

}  // namespace

int w4_gemm_prepare(int smem_optin, int (*clusters)[4]) {
    for (int wtype : {TW_INT4, TW_E2M1})
        for (int nt = 1; nt <= 4; nt *= 2)
            for (int group = 32; group <= 128; group *= 2) {
                cudaError_t e =
                    cudaFuncSetAttribute(kernel_for(wtype, nt, group),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem_optin);
                if (e != cudaSuccess) return static_cast<int>(e);
            }
    // Clusters of 1, 2, 4, 8 CTAs that run at once, with a CTA and with two on an SM.
    for (int ctas = 1; ctas <= 2; ++ctas)
        for (int i = 0; i < 4; ++i) {
            cudaLaunchAttribute attr[2];
            const cudaLaunchConfig_t cfg =
                config(1 << i, 1 << i, static_cast<size_t>(ctas == 1 ? smem_optin : half_smem(smem_optin)),
                       false, nullptr, attr);
            cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters[ctas - 1][i],
                                                           kernel_for(TW_INT4, 1, 128), &cfg);
            if (e != cudaSuccess) return static_cast<int>(e);
        }
    return 0;
}

int launch_w4_gemm(const W4GemmArgs& a, int max_sms, const DeviceInfo& d, void* stream) {
    const int64_t sms = max_sms < d.sm_count ? max_sms : d.sm_count;
    const bool whole = max_sms >= d.sm_count;
    const int parts = a.xtype == TW_X_F32 ? 3 : 1;
    const int64_t stripes = (a.N + kW4Channels - 1) / kW4Channels;
    const int64_t tiles = (a.K + kW4Inner - 1) / kW4Inner;
    W4Plan plan{a, 0, 0, 0, 0, 1, d.status};
    int64_t smem = 0, sets = 0;
    int nt = 0;
    // The most tokens at a time whose x fits, K over the fewest CTAs, two of them on an
    // SM if they fit so (under a budget each is alone there).  One token that does not
    // fit the SMs of a budget: in slices, staged again for each round.
    auto choose = [&](int64_t tokens, int slices) {
        const int columns = static_cast<int>(tokens) * parts;
        const int blocks = columns <= 8 ? 1 : columns <= 16 ? 2 : 4;
        for (int ctas = whole ? 2 : 1; ctas > 0; --ctas)
            for (int i = 0; i < 4 && (1 << i) <= tiles; ++i) {
                int64_t at_once = sms * ctas >> i;
                const int64_t clusters = d.w4_clusters[ctas - 1][i];
                if (i > 0 && at_once > clusters) at_once = clusters;
                if (at_once < 1) break;
                sets = at_once < stripes ? at_once : stripes;
                // Stripes at a time: a warp for each if there are that many, but some
                // warps for one while they have two tiles each.
                const int64_t share = (stripes + sets - 1) / sets;
                plan.log_split = i;
                plan.log_at_once = 0;
                while ((1 << plan.log_at_once) < kWarps && (1 << plan.log_at_once) < share &&
                       (i > 0 || plan.log_at_once < 1 ||
                        2 * kWarps >> plan.log_at_once > tiles >> i))
                    ++plan.log_at_once;
                plan.slices = slices;
                const int64_t room = ctas == 1 ? d.smem_optin : half_smem(d.smem_optin);
                for (plan.slots = max_slots(blocks); plan.slots >= kMinSlots; --plan.slots) {
                    smem = smem_bytes(blocks, columns, a.K, a.group, plan);
                    if (smem > room) continue;
                    if (ctas == 1 && smem < kExclusiveSmemBytes) smem = kExclusiveSmemBytes;
                    plan.tokens = static_cast<int>(tokens);
                    nt = blocks;
                    return true;
                }
            }
        return false;
    };
    bool found = false;
    for (int64_t tokens = a.M < kColumnsMax / parts ? a.M : kColumnsMax / parts;
         tokens > 0 && !found; --tokens)
        found = choose(tokens, 1);
    for (int slices = 2; !found && slices <= tiles; slices *= 2) found = choose(1, slices);
    if (!found) return static_cast<int>(cudaErrorInvalidConfiguration);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(static_cast<int>(sets << plan.log_split),
                                          1 << plan.log_split, static_cast<size_t>(smem), whole,
                                          stream, attr);
    void* args[] = {&plan};
    return static_cast<int>(cudaLaunchKernelExC(&cfg, kernel_for(a.wtype, nt, a.group), args));
}

}  // namespace tw
