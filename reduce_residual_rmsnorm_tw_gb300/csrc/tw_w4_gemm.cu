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
// Two CTAs of eight warps share an SM, so that one streams while the other starts or
// joins.  A CTA holds x of its K in shared memory and takes an even share of the
// stripes; a cluster of CTAs may split K (where x would not fit, or its copies into
// every SM would outweigh W).  A warp's piece of work is a share of a stripe's K; the
// warps take pieces in turn and never wait for each other, but leave their sums where
// the stripe's CTA of the cluster adds them up, in their order, when all are done.
//
// Measured: 1 x 8192 x 8192 int4 10.5 us, of which 4 are the launch, x and the join (a K
// of 256 takes 4.0), the rest 5.4 TB/s; 8 x 8192 x 32768 32.7, 4.3 TB/s; 16 x 8192 x
// 8192 14.5, 32 22.5, where the matrix instructions set the pace: one takes 6 to 8
// clocks of an SM's quarter, and four blocks of columns need four for each piece of W.
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
// A barrier of the cluster in two halves.  At the start the first half says only that the
// CTA runs, and orders nothing; between passes that it has read the sums it held, which the
// others' next ones, behind the second half, must not overtake: a release.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_release() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A word's eight values as four pairs of bf16, (k, k + 1) for k = 0, 2, 4, 6: the
// values themselves (e2m1) or times 2^-7 (int4; the factor comes back in at the
// end, so a group's contribution below 2^-119 in magnitude, fp32's 2^-126 times 2^7, may
// lose bits).  bf16 numbers below
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

// int8 x is held times 2^-7: a byte in a bf16's last bits is v 2^-133 (as in widen).  No
// bits are lost for it: a group's sum is a multiple of 2^-14 (e2m1: 2^-8), times a bf16
// scale's last bit one of 2^-147, which fp32 holds below its normal range too.
constexpr float kInt8Factor = 128.f;

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Sixteen bytes of x (4 fp32 or 16 8-bit values) as bf16 to `to` and, fp32, as three terms
// that add up to them to three rows `stride` apart: the leading eight bits, cut off, then
// the next eight, then the rest; an infinity or a NaN as its own first term.
template <int XTYPE>
__device__ __forceinline__ void store_x(const uint4& x, uint32_t to, int stride) {
    const uint32_t word[4] = {x.x, x.y, x.z, x.w};
    if constexpr (XTYPE == TW_X_F32) {
        float t[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = __uint_as_float(word[i]);
            const bool finite = fabsf(v) <= 3.402823466e38f;
            t[0][i] = finite ? __uint_as_float(word[i] & 0xffff0000u) : v;
            const float rest = finite ? v - t[0][i] : 0.f;
            t[1][i] = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
            t[2][i] = rest - t[1][i];
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
            sts64(to + p * stride, pack_bf16(t[p][0], t[p][1]), pack_bf16(t[p][2], t[p][3]));
    } else {
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (XTYPE == TW_X_INT8) {
                const uint32_t u = __byte_perm(word[i / 2] ^ 0x80808080u, 0,
                                               i % 2 ? 0x4342 : 0x4140);  // v + 128
                asm("fma.rn.bf16x2 %0, %1, %2, %3;"
                    : "=r"(h[i])
                    : "r"(u), "r"(0x7e807e80u), "r"(0xbf80bf80u));  // 2^126, -1
            } else {
                uint32_t f;
                asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\t"
                    "cvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
                    : "=r"(f)
                    : "r"(word[i / 2] >> (i % 2 * 16)));
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
                h[i] = pack_bf16(v.x, v.y);
            }
        }
        sts128(to, make_uint4(h[0], h[1], h[2], h[3]));
        sts128(to + 16, make_uint4(h[4], h[5], h[6], h[7]));
    }
}

// Where row t of `tokens` rows of x lands, `bytes` each, before it becomes `token` bytes of
// bf16 at t * token: packed towards the end of those and one row more, so that no
// row's bf16 comes to lie on a later row, or on itself, before it has been read.
__device__ __forceinline__ int landing(int t, int tokens, int token, int bytes) {
    return tokens * token - (tokens - 1 - t) * bytes;
}
// The rows that landed there as bf16: `inner` values of a row, zero from `own` on.  (One
// piece of a thread at a time; with eight, longer code: 1 x 256 x 32768 fp32 4.3 -> 5.0 us.)
template <int XTYPE>
__device__ __forceinline__ void widen_x(uint32_t xs, int x_stride, int tokens, int inner,
                                        int own) {
    constexpr int kValues = XTYPE == TW_X_F32 ? 4 : 16;  // of a piece
    const int token = x_stride * (XTYPE == TW_X_F32 ? 3 : 1);
    const int pieces = inner / kValues, from_x = own / kValues;
    int t = 0, at = threadIdx.x;  // the thread's piece: the at-th of token t
#pragma unroll 1
    for (int n = 0; n < tokens * pieces; n += kThreads, at += kThreads) {
        while (at >= pieces && t < tokens) {
            at -= pieces;
            ++t;
        }
        uint4 x = make_uint4(0, 0, 0, 0);
        if (t < tokens && at < from_x)
            x = lds128(xs + landing(t, tokens, token, pieces * 16) + at * 16);
        __syncthreads();  // all of these are read
        if (t < tokens) store_x<XTYPE>(x, xs + t * token + at * kValues * 2, x_stride);
    }
}

// Floats between the columns of a piece's sums (a fragment's stores meet no bank twice).
constexpr int kRowStride = kW4Channels + 4;
// Bytes of shared memory before the sums (the word that says that a wait gave up).
constexpr int kHeader = 16;
// Tiles that a warp warms L2 with before the launch before this one has ended.
constexpr int kWarm = 16;
// Tiles of x that a CTA holds at a time.
__host__ __device__ constexpr int x_tiles(int tiles, int split, int slices) {
    return ((tiles + split - 1) / split + slices - 1) / slices;
}

struct W4Plan {
    W4GemmArgs a;
    int tokens;       // at a time
    int log_split;    // CTAs of a cluster, which split K
    int slots;        // of a warp's ring
    int slices;       // of a CTA's K, whose x is in shared memory one after the other
    int log_shares;   // pieces of a stripe's K in a slice
    int pass;         // stripes whose sums are held at a time
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

// A warp's way through its CTA's pieces: passes of up to `pass` stripes, in each the
// slices of K one after the other, in each the pieces warp, warp + kWarps, ...
struct Way {
    int at, end;    // the pass's first stripe and the CTA's last
    int slice, item;
    int stripe, first, tiles;  // the piece: its stripe, first tile and tiles
};

// INT4: the weights' type; NT: blocks of eight columns of x (fp32: three per token);
// G: the group.
template <bool INT4, int NT, int G>
__global__ void __launch_bounds__(kThreads, 2)
    w4_gemm_kernel(const __grid_constant__ W4Plan plan) {
    constexpr int kTile = w4_tile_bytes(G);
    constexpr int kChunk = chunk_of(NT), kSlot = kChunk * kTile;
    const W4GemmArgs& a = plan.a;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = threadIdx.x % 32;
    const int row = lane / 4, quad = lane % 4;
    const int parts = a.xtype == TW_X_F32 ? 3 : 1;
    const int K = static_cast<int>(a.K);
    const int tiles_k = (K + kW4Inner - 1) / kW4Inner;
    const int stripes = static_cast<int>((a.N + kW4Channels - 1) / kW4Channels);
    // This CTA's share of K (of the cluster), cut into slices, and of the stripes.
    const int log_split = plan.log_split, split = 1 << log_split;
    const int log_shares = plan.log_shares, shares = 1 << log_shares, slices = plan.slices;
    const int rank = split > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
    const int lo = tiles_k * rank >> log_split, hi = tiles_k * (rank + 1) >> log_split;
    auto slice_at = [&](int s) {
        return slices == 1 ? (s ? hi : lo) : lo + (hi - lo) * s / slices;
    };
    const int64_t sets = gridDim.x >> log_split, set = blockIdx.x >> log_split;
    const int first = static_cast<int>(stripes * set / sets);
    const int end = static_cast<int>(stripes * (set + 1) / sets);
    const int x_stride = (x_tiles(tiles_k, split, slices) * kW4Inner + kXPad) * 2;
    // Stripe i of a pass belongs to rank i % split, which holds its pieces' sums:
    // [piece][i / split][column][kRowStride].  Then the rings, their barriers, x.
    const int columns = plan.tokens * parts;
    const int owned = (plan.pass + split - 1) >> log_split;
    // Before them, not 0 where a copy did not arrive in time (the device status says so).
    volatile int* const gave_up = reinterpret_cast<volatile int*>(smem);
    float* sums = reinterpret_cast<float*>(smem + kHeader);
    const uint32_t rings =
        smem_addr(sums) + ((split * slices) << log_shares) * owned * columns * kRowStride * 4;
    const uint32_t ring = rings + warp * plan.slots * kSlot;
    const uint32_t bars = rings + kWarps * plan.slots * kSlot;
    const uint32_t bar = bars + warp * kMaxSlots * 8;
    const uint32_t x_bar = bars + kWarps * kMaxSlots * 8;
    const uint32_t xs = x_bar + 16;

    if (lane == 0) {
        for (int i = 0; i < plan.slots; ++i) mbar_init(bar + i * 8, 1);
        if (warp == 0) {
            mbar_init(x_bar, 1);
            *gave_up = 0;
        }
        mbar_init_fence();
    }
    __syncthreads();
    auto items_of = [&](const Way& w) {
        return (end - w.at < plan.pass ? end - w.at : plan.pass) << log_shares;
    };
    auto piece = [&](Way& w) {
        const int share = w.item & (shares - 1);
        const int from = slice_at(w.slice), to = slice_at(w.slice + 1);
        w.stripe = w.at + (w.item >> log_shares);
        w.first = from + ((to - from) * share >> log_shares);
        w.tiles = from + ((to - from) * (share + 1) >> log_shares) - w.first;
    };
    const char* packed = static_cast<const char*>(a.packed);
    auto place = [&](const Way& w) {
        return packed + (static_cast<int64_t>(w.stripe) * tiles_k + w.first) * kTile;
    };
    Way ld{first, end, 0, warp, 0, 0, 0};
    // The first W on its way into L2 while the launch before this one ends (a hint that
    // reads nothing: what that launch writes is seen all the same).
    if (ld.item < items_of(ld)) {
        piece(ld);
        if (lane == 0 && ld.tiles > 0)
            bulk_prefetch_l2(place(ld), static_cast<uint32_t>(
                                            (ld.tiles < kWarm ? ld.tiles : kWarm) * kTile));
    }
    // A CTA may write into the others' sums: waited for before the first of a pass.
    bool may_write = split == 1;
    auto wait_to_write = [&]() {
        if (may_write) return;
        cluster_wait();
        may_write = true;
    };
    if (split > 1) cluster_arrive_relaxed();
    grid_dependency_wait();
    grid_launch_dependents();

    // Waits for a copy.  Where one gives up the CTA's others wait no longer than a copy in
    // flight takes to land; nothing more is stored, and behind the pass and its block of
    // tokens the CTA, with the others of its cluster, leaves.
    auto await = [&](uint32_t on, uint32_t parity) {
        uint64_t start = 0;
        for (uint32_t tries = 1; !mbar_try_wait(on, parity); ++tries) {
            if (tries % 64 != 0) continue;
            const uint64_t now = global_timer_ns();
            if (start == 0) start = now;
            if (now - start <= kWaitLimitNs / 1000 ||
                (now - start <= kWaitLimitNs && !*gave_up))
                continue;
            *gave_up = 1;
            atomicOr(plan.status, 1u);
            break;
        }
    };
    const uint32_t one = elect_one();
    uint32_t slot_ld = 0, slot = 0, phase = 0, x_phase = 0;
    int64_t m0 = 0;
    for (; m0 < a.M && !*gave_up; m0 += plan.tokens) {
        const int tokens = static_cast<int>(a.M - m0 < plan.tokens ? a.M - m0 : plan.tokens);
        const int cols = tokens * parts;
        // The next chunk to load.
        const char* from = packed;
        int left = 0;
        ld = Way{first, end, 0, warp - kWarps, 0, 0, 0};
        auto load = [&]() {
            while (left == 0) {  // on to the warp's next piece (which may be without tiles)
                if (ld.at >= end) return;
                ld.item += kWarps;
                if (ld.item >= items_of(ld)) {
                    ld.item = warp - kWarps;
                    if (++ld.slice == slices) {
                        ld.slice = 0;
                        ld.at += plan.pass;
                    }
                    continue;
                }
                piece(ld);
                left = ld.tiles;
                from = place(ld);
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
        for (int d = 0; d < plan.slots; ++d) load();

        // x of a slice of this CTA's K, zero up to the end of its last tile: a bulk copy a
        // row (16 x 8192 x 8192 17.2 -> 14.7 us against loads through registers).  Other
        // types become bf16 from there.
        auto stage_x = [&](int slice) {
            const int log_size = a.xtype == TW_X_BF16 ? 1 : a.xtype == TW_X_F32 ? 2 : 0;
            const int k0 = slice_at(slice) * kW4Inner, k1 = slice_at(slice + 1) * kW4Inner;
            const int own = (k1 < K ? k1 : K) - k0;
            if (warp == 0) {
                if (lane == 0) mbar_arrive_expect_tx(x_bar, tokens * own << log_size);
                __syncwarp();
                if (lane < tokens)
                    bulk_copy(xs + (a.xtype == TW_X_BF16
                                        ? lane * x_stride
                                        : landing(lane, tokens, parts * x_stride,
                                                  (k1 - k0) << log_size)),
                              static_cast<const char*>(a.x) +
                                  (((m0 + lane) * a.K + k0) << log_size),
                              own << log_size, x_bar);
            }
            await(x_bar, x_phase);
            x_phase ^= 1u;
            if (a.xtype == TW_X_BF16) {
                for (int e = threadIdx.x; k1 > K && e < tokens * 16; e += kThreads)
                    if (e % 16 * 8 < k1 - K)
                        sts128(xs + e / 16 * x_stride + own * 2 + e % 16 * 16,
                               make_uint4(0, 0, 0, 0));
            } else if (a.xtype == TW_X_F32) {
                widen_x<TW_X_F32>(xs, x_stride, tokens, k1 - k0, own);
            } else if (a.xtype == TW_X_INT8) {
                widen_x<TW_X_INT8>(xs, x_stride, tokens, k1 - k0, own);
            } else {
                widen_x<TW_X_E4M3>(xs, x_stride, tokens, k1 - k0, own);
            }
            // (Ordered before bulk copies of other tokens to the same place.)
            fence_async_shared();
            __syncthreads();
        };
        if (slices == 1) stage_x(0);
        // Where the lane's rows of x begin.  Columns beyond the last repeat the first:
        // one read for all of them, and nothing of theirs is stored.
        uint32_t x_row[NT];
#pragma unroll
        for (int b = 0; b < NT; ++b)
            x_row[b] = xs + (b * 8 + row < cols ? b * 8 + row : 0) * x_stride + quad * 16;

        Way at{first, end, 0, 0, 0, 0, 0};
        for (; at.at < end; at.at += plan.pass) {
            const int items = items_of(at);
            for (at.slice = 0; at.slice < slices; ++at.slice) {
                if (slices > 1) {
                    __syncthreads();  // the x before has been read
                    stage_x(at.slice);
                }
                for (at.item = warp; at.item < items; at.item += kWarps) {
                    piece(at);
                    const int tiles = at.tiles;
                    float total[NT][4] = {};
                    uint32_t x_at = (at.first - slice_at(at.slice)) * (kW4Inner * 2);
                    for (int i = 0; i < tiles; i += kChunk) {
                        await(bar + slot * 8, phase);
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
                                for (int b = 0; b < NT; ++b)
                                    xv[b] = lds128(x_row[b] + x_at + j * 64);
                                uint32_t u[4], v[4];
                                widen<INT4>(word_of(w[0], j), u);
                                widen<INT4>(word_of(w[1], j), v);
#pragma unroll
                                for (int b = 0; b < NT; ++b) {
                                    if (j * 32 % G == 0) {
                                        mma_first(sum[0][b], u[0], v[0], u[1], v[1], xv[b].x,
                                                  xv[b].y);
                                        mma_first(sum[1][b], u[2], v[2], u[3], v[3], xv[b].z,
                                                  xv[b].w);
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
                    // The piece's sums, to where its stripe's rank adds them up.
                    wait_to_write();
                    const int i = at.stripe - at.at;
                    const int which = ((rank * slices + at.slice) << log_shares) +
                                      (at.item & (shares - 1));
                    uint32_t to =
                        smem_addr(sums) +
                        ((which * owned + (i >> log_split)) * columns * kRowStride + row) * 4;
                    if (split > 1) to = map_to_rank(to, static_cast<uint32_t>(i & (split - 1)));
#pragma unroll
                    for (int b = 0; b < NT; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = b * 8 + quad * 2 + e % 2;
                            const uint32_t place_of = to + (c * kRowStride + e / 2 * 8) * 4;
                            if (c < cols && split > 1)
                                st_cluster_f32(place_of, total[b][e]);
                            else if (c < cols)
                                asm volatile("st.shared.f32 [%0], %1;" ::"r"(place_of),
                                             "f"(total[b][e])
                                             : "memory");
                        }
                }
            }
            __syncwarp();
            wait_to_write();
            // (The others would add up what this CTA has left them.)
            if (split > 1 && *gave_up && lane < split)
                st_cluster_f32(map_to_rank(smem_addr(smem), static_cast<uint32_t>(lane)), 1.f);
            if (split > 1)
                cluster_barrier();
            else
                __syncthreads();
            // Every piece of the pass is there: this rank's stripes, added up in order.
            const int pieces = (split * slices) << log_shares;
            const int mine =  // stripes
                *gave_up ? 0 : ((items >> log_shares) - rank + split - 1) >> log_split;
            const int apart = owned * columns * kRowStride;
            const float factor =
                (INT4 ? kInt4Factor : 1.f) * (a.xtype == TW_X_INT8 ? kInt8Factor : 1.f);
            for (int e = threadIdx.x; e < mine * tokens * kW4Channels; e += kThreads) {
                const int ch = e % kW4Channels, rest = e / kW4Channels;
                const int i = tokens == 1 ? rest : rest / tokens, t = rest - i * tokens;
                const int64_t n =
                    static_cast<int64_t>(at.at + (i << log_split) + rank) * kW4Channels + ch;
                if (n >= a.N) continue;
                float sum = 0.f;
                // fp32 x: the smaller terms first.
                for (int p = parts - 1; p >= 0; --p) {
                    const float* of = sums + (i * columns + t * parts + p) * kRowStride + ch;
                    for (int q = 0; q < pieces; ++q, of += apart) sum += *of;
                }
                sum *= factor;
                if (a.x_scale) sum *= a.x_scale[m0 + t];
                const int64_t to = (m0 + t) * a.N + n;
                if (a.dtype == TW_BF16)
                    static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(sum);
                else
                    static_cast<float*>(a.out)[to] = sum;
            }
            // The sums are read before another pass (and x before other tokens') comes.
            __syncwarp();
            const bool last = at.at + plan.pass >= end;
            if (!last || m0 + plan.tokens < a.M) {
                if (split > 1) {
                    cluster_arrive_release();
                    may_write = false;
                }
                if (split == 1 || last) __syncthreads();
            }
        }
    }
    // Given up: copies in flight have time to land before their shared memory is another CTA's.
    if (m0 < a.M) {
        wait_to_write();
        const uint64_t start = global_timer_ns();
        while (global_timer_ns() - start < kWaitLimitNs / 100) {
        }
    }
}

template <bool INT4, int G>
void* entry(int nt) {
    return nt == 1   ? reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 1, G>)
           : nt == 2 ? reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 2, G>)
           : nt == 3 ? reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 3, G>)
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
    const int split = 1 << p.log_split;
    const int64_t sums = (static_cast<int64_t>(split) * p.slices << p.log_shares) *
                         ((p.pass + split - 1) / split) * columns * kRowStride * 4;
    const int64_t rings =
        kWarps * (p.slots * chunk_of(nt) * w4_tile_bytes(group) + kMaxSlots * 8) + 16;
    const int tiles = static_cast<int>((K + kW4Inner - 1) / kW4Inner);
    const int64_t inner = x_tiles(tiles, split, p.slices) * kW4Inner;
    const int64_t landing = p.a.xtype == TW_X_BF16 ? 0 : inner * (p.a.xtype == TW_X_F32 ? 4 : 1);
    return kHeader + sums + rings + columns * (inner + kXPad) * 2 + landing;
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
        for (int nt = 1; nt <= 4; ++nt)
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
            const int64_t smem = ctas == 1 ? smem_optin : half_smem(smem_optin);
            const cudaLaunchConfig_t cfg =
                config(1 << i, 1 << i, static_cast<size_t>(smem), false, nullptr, attr);
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
    // Every cut that fits, by the time it takes in ns: a warp's tiles (more of them with
    // two CTAs on an SM than with one) and pieces, each pass's barrier, x on its way into
    // shared memory, and what a second CTA and a cluster cost once.  Fitted to 976 times
    // of 36 sizes (1 to 32 tokens, 300 to 32768 channels, K 256 to 8192): the cut taken
    // is 2 % slower than the best of them on average, 12 % at most.  The most tokens at a
    // time that fit, even shares of them; one token that does not fit the SMs of a budget
    // goes in slices, staged for each pass.
    constexpr int64_t kTile2 = 382, kBlock2 = 223, kTile1 = 221, kBlock1 = 80;
    constexpr int64_t kPiece = 1030, kPass = 595, kClusterPass = 860;
    constexpr int64_t kSecondCta = 541, kCluster = 370, kClusterOf8 = 3350;
    const int64_t stage_of = a.xtype == TW_X_BF16 ? 63 : 160;
    W4Plan best{}, plan{a, 0, 0, 0, 1, 0, 0, d.status};
    int64_t best_cost = -1, best_smem = 0, best_sets = 0;
    int nt = 0;
    auto choose = [&](int64_t tokens, int slices) {
        const int columns = static_cast<int>(tokens) * parts;
        const int blocks = (columns + 7) / 8;
        plan.tokens = static_cast<int>(tokens);
        plan.slices = slices;
        for (int ctas = whole ? 2 : 1; ctas > 0; --ctas)
            for (int i = 0; i < 4 && slices << i <= tiles; ++i) {  // a tile for each slice
                int64_t sets = sms * ctas >> i;
                const int64_t clusters = d.w4_clusters[ctas - 1][i];
                if (i > 0 && sets > clusters) sets = clusters;
                if (sets < 1) break;
                if (sets > stripes) sets = stripes;
                const int64_t own = (stripes + sets - 1) / sets;  // stripes of a set
                const int64_t room = ctas == 1 ? d.smem_optin : half_smem(d.smem_optin);
                const int64_t inner = x_tiles(static_cast<int>(tiles), 1 << i, slices);
                plan.log_split = i;
                for (plan.log_shares = 0;
                     plan.log_shares < 4 && (1 << plan.log_shares) <= inner; ++plan.log_shares) {
                    const int64_t shares = 1 << plan.log_shares;
                    // As many stripes a pass as their sums find room, few slots if need be.
                    plan.pass = static_cast<int>(own < 1024 ? own : 1024);
                    int64_t smem = 0;
                    for (;;) {
                        for (plan.slots = max_slots(blocks); plan.slots >= kMinSlots; --plan.slots)
                            if ((smem = smem_bytes(blocks, columns, a.K, a.group, plan)) <= room)
                                break;
                        if (plan.slots >= kMinSlots || plan.pass == 1) break;
                        plan.pass = (plan.pass + 1) / 2;
                    }
                    if (plan.slots < kMinSlots) continue;
                    const int64_t passes = (own + plan.pass - 1) / plan.pass;
                    const int64_t rounds =
                        ((own < plan.pass ? own : plan.pass) * shares + kWarps - 1) / kWarps;
                    const int64_t each = (inner + shares - 1) / shares;
                    const int64_t tile = ctas == 2 ? kTile2 + kBlock2 * (blocks - 1)
                                                   : kTile1 + kBlock1 * (blocks - 1);
                    const int64_t stage = columns * inner * stage_of / 16;
                    const int64_t cost =
                        passes * (slices * rounds * (each * tile + kPiece) + kPass +
                                  (i > 0 ? kClusterPass : 0)) +
                        (slices == 1 ? stage : stage * slices * passes) +
                        (ctas == 2 ? kSecondCta : 0) + (i > 0 ? kCluster : 0) +
                        (i == 3 ? kClusterOf8 : 0);
                    if (best_cost >= 0 && cost >= best_cost) continue;
                    best_cost = cost;
                    best = plan;
                    best_smem = smem;
                    if (ctas == 1 && smem < kExclusiveSmemBytes) best_smem = kExclusiveSmemBytes;
                    best_sets = sets;
                    nt = blocks;
                }
            }
        return best_cost >= 0;
    };
    bool found = false;
    const int64_t most = kColumnsMax / parts, turns = (a.M + most - 1) / most;
    for (int64_t tokens = (a.M + turns - 1) / turns; tokens > 0 && !found; --tokens)
        found = choose(tokens, 1);
    for (int slices = 2; !found && slices <= tiles; slices *= 2) found = choose(1, slices);
    if (!found) return static_cast<int>(cudaErrorInvalidConfiguration);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        config(static_cast<int>(best_sets << best.log_split), 1 << best.log_split,
               static_cast<size_t>(best_smem), whole, stream, attr);
    void* args[] = {&best};
    return static_cast<int>(cudaLaunchKernelExC(&cfg, kernel_for(a.wtype, nt, a.group), args));
}

}  // namespace tw
