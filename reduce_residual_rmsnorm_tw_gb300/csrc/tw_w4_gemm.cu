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
// of row g and 16 of row g + 8 straight into registers, kDepth tiles ahead; word j
// holds k = 32 j + 8 q .. + 7, so that a word's two MMAs stay within 32 k and a
// group of 32 can be scaled on its own.
//
// One CTA of 16 warps per SM.  It holds x of its K in shared memory and takes an even
// share of the 16-channel stripes, `at_once` of them (times R) at a time: as many
// warps share a stripe, each a contiguous piece of its K, and their sums are joined
// through shared memory in warp order.  Where x does not fit, a cluster of CTAs
// splits K, and joins through distributed shared memory in rank order.
#include <cuda_fp16.h>

#include "tw_tcgen05.cuh"

namespace tw {
namespace {

constexpr int kWarps = 16;
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
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A word's eight values as four pairs of bf16, (k, k + 1) for k = 0, 2, 4, 6: the
// values themselves (e2m1) or times 2^-7 (int4).  bf16 numbers below 2^-125 are their
// last eight bits times 2^-133, so that two nibbles in eight need no shift.
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

struct W4Plan {
    W4GemmArgs a;
    int tokens;   // at a time
    int at_once;  // stripe groups (of R stripes) of a CTA at a time, a power of two
    int split;    // CTAs of a cluster, which split K
};

// A tile's words for one lane, and its scales (rows g and g + 8 of each group).
template <int R, int G>
struct Tile {
    uint4 w[R][2];
    uint32_t s[R][128 / G];
};
template <int G>
__device__ __forceinline__ void load_scales(uint32_t (&s)[128 / G], const char* p) {
    if constexpr (G == 128)
        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(s[0]) : "l"(p));
    else if constexpr (G == 64)
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                     : "=r"(s[0]), "=r"(s[1])
                     : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3])
                     : "l"(p));
}

// A warp's way through its CTA's stripe groups: rounds of at_once groups (fewer in
// the last), in each a contiguous piece of a group's tiles.
struct Way {
    int at, end;      // the round's first group and the CTA's last
    int groups;       // of the round
    int group, tile;  // this warp's group and first tile
    int tiles;        // this warp's tiles
    __device__ __forceinline__ void round(int at_once, int warp, int lo, int hi) {
        const int rest = end - at;
        groups = at_once;
        while (groups / 2 >= rest && groups > 1) groups /= 2;
        const int shares = kWarps / groups;  // warps of a group
        const int share = warp % shares;
        group = at + warp / shares;
        tile = lo + (hi - lo) * share / shares;
        tiles = group < end ? lo + (hi - lo) * (share + 1) / shares - tile : 0;
    }
};

// INT4: the weights' type; NT: blocks of eight tokens (fp32 x: three per token);
// R: stripes per warp; G: the group; kDepth: tiles in flight per warp.
template <bool INT4, int NT, int R, int G, int kDepth>
__global__ void __launch_bounds__(kThreads, 1)
    w4_gemm_kernel(const __grid_constant__ W4Plan plan) {
    constexpr int kTile = w4_tile_bytes(G);
    constexpr int kColumns = NT * 8, kRowStride = 16 * R + 1;
    const W4GemmArgs& a = plan.a;
    extern __shared__ __align__(128) unsigned char smem[];
    float* part = reinterpret_cast<float*>(smem);  // [warp][column][kRowStride]
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = lane / 4, quad = lane % 4;
    const int parts = a.xtype == TW_X_F32 ? 3 : 1;
    const int K = static_cast<int>(a.K);
    const int tiles_k = (K + kW4Inner - 1) / kW4Inner;
    const int stripes = static_cast<int>((a.N + 15) / 16);
    const int groups = (stripes + R - 1) / R;
    // This CTA's share of K (of the cluster) and of the groups.
    const int split = plan.split;
    const int rank = split > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
    const int lo = tiles_k * rank / split, hi = tiles_k * (rank + 1) / split;
    const int64_t sets = gridDim.x / split, set = blockIdx.x / split;
    const int first = static_cast<int>(groups * set / sets);
    const int end = static_cast<int>(groups * (set + 1) / sets);
    const int x_tiles = (tiles_k + split - 1) / split;  // at most, of any rank
    const int x_stride = (x_tiles * kW4Inner + kXPad) * 2;
    // Sums that the cluster's CTAs write here: [buffer][rank][output / split].
    float* joined = part + kWarps * kColumns * kRowStride;
    const int outputs = plan.at_once * 16 * R * plan.tokens;
    const int per_rank = (outputs + split - 1) / split;
    const uint32_t xs =
        smem_addr(joined) + (split > 1 ? (2 * split * per_rank * 4 + 15) / 16 * 16 : 0);

    const char* packed = static_cast<const char*>(a.packed);
    Way ld{first, end, 0, 0, 0, 0};
    ld.round(plan.at_once, warp, lo, hi);
    // The first round's W on its way into L2 while the launch before this one ends (a
    // hint that reads nothing: what that launch writes is seen all the same).
    if (lane == 0 && ld.tiles > 0)
        for (int r = 0; r < R; ++r)
            if (ld.group * R + r < stripes)
                bulk_prefetch_l2(packed + (static_cast<int64_t>(ld.group * R + r) * tiles_k +
                                           ld.tile) * kTile,
                                 static_cast<uint32_t>((ld.tiles < 16 ? ld.tiles : 16) * kTile));
    if (split > 1) cluster_barrier();  // every CTA runs before any writes into it
    grid_dependency_wait();
    grid_launch_dependents();

    int buf = 0;
    for (int64_t m0 = 0; m0 < a.M; m0 += plan.tokens) {
        const int tokens = static_cast<int>(a.M - m0 < plan.tokens ? a.M - m0 : plan.tokens);
        const int cols = tokens * parts;
        // The next tile to load: its place in the round, whose tiles count up to a
        // multiple of kDepth so that registers are named at compile time.
        int ld_i = 0;
        ld = Way{first, end, 0, 0, 0, 0};
        ld.round(plan.at_once, warp, lo, hi);
        Tile<R, G> ahead[kDepth];
        auto load = [&](Tile<R, G>& t) {
            // (A warp may be without tiles for whole rounds.)
            while (ld_i == (ld.tiles + kDepth - 1) / kDepth * kDepth && ld.at < end) {
                ld_i = 0;
                ld.at += ld.groups;
                if (ld.at < end)
                    ld.round(plan.at_once, warp, lo, hi);
                else
                    ld.tiles = 0;
            }
            if (ld_i < ld.tiles) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    // A stripe beyond the last: the last once more, not stored.
                    const int stripe = R == 1 || ld.group * R + r < stripes ? ld.group * R + r
                                                                           : stripes - 1;
                    const char* from =
                        packed + (static_cast<int64_t>(stripe) * tiles_k + ld.tile + ld_i) * kTile;
                    t.w[r][0] = ld_global_nc(from + lane * 16);
                    t.w[r][1] = ld_global_nc(from + 512 + lane * 16);
                    load_scales<G>(t.s[r], from + 1024 + row * (512 / G));
                }
            }
            ++ld_i;
        };
#pragma unroll
        for (int d = 0; d < kDepth; ++d) load(ahead[d]);

        // x of this CTA's K, zero up to the end of its last tile; kXAhead loads of a
        // thread in flight.
        const int x_size = a.xtype == TW_X_BF16 ? 2 : a.xtype == TW_X_F32 ? 4 : 1;
        const uint32_t row_pieces = static_cast<uint32_t>(hi - lo) * (kW4Inner / 8);
        const uint32_t pieces = row_pieces * tokens;
        for (uint32_t e0 = threadIdx.x; e0 < pieces; e0 += kThreads * kXAhead) {
            XEight x[kXAhead] = {};
#pragma unroll
            for (int i = 0; i < kXAhead; ++i) {
                const uint32_t e = e0 + i * kThreads, t = e / row_pieces;
                const int64_t k = lo * kW4Inner + static_cast<int64_t>(e % row_pieces) * 8;
                if (e < pieces && k < K)
                    x[i].load(static_cast<const char*>(a.x) + ((m0 + t) * a.K + k) * x_size,
                              a.xtype);
            }
#pragma unroll
            for (int i = 0; i < kXAhead; ++i) {
                const uint32_t e = e0 + i * kThreads, t = e / row_pieces;
                if (e >= pieces) break;
                uint4 terms[3];
                x_terms(x[i], a.xtype, terms);
                for (int p = 0; p < parts; ++p)
                    sts128(xs + (p * tokens + t) * x_stride + e % row_pieces * 16, terms[p]);
            }
        }
        __syncthreads();

        Way at{first, end, 0, 0, 0, 0};
        for (; at.at < end; at.at += at.groups) {
            at.round(plan.at_once, warp, lo, hi);
            float total[R][NT][4] = {};
            for (int i0 = 0; i0 < at.tiles; i0 += kDepth) {
#pragma unroll
                for (int d = 0; d < kDepth; ++d) {
                    if (i0 + d < at.tiles) {
                        const Tile<R, G>& t = ahead[d];
                        const uint32_t x_at =
                            xs + (at.tile + i0 + d - lo) * (kW4Inner * 2) + quad * 16;
                        float sum[R][NT][4] = {};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint4 xv[NT];
#pragma unroll
                            for (int b = 0; b < NT; ++b)
                                xv[b] = b * 8 + row < cols
                                            ? lds128(x_at + (b * 8 + row) * x_stride + j * 64)
                                            : make_uint4(0, 0, 0, 0);
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                uint32_t u[4], v[4];
                                widen<INT4>(j == 0   ? t.w[r][0].x
                                            : j == 1 ? t.w[r][0].y
                                            : j == 2 ? t.w[r][0].z
                                                     : t.w[r][0].w, u);
                                widen<INT4>(j == 0   ? t.w[r][1].x
                                            : j == 1 ? t.w[r][1].y
                                            : j == 2 ? t.w[r][1].z
                                                     : t.w[r][1].w, v);
#pragma unroll
                                for (int b = 0; b < NT; ++b) {
                                    mma(sum[r][b], u[0], v[0], u[1], v[1], xv[b].x, xv[b].y);
                                    mma(sum[r][b], u[2], v[2], u[3], v[3], xv[b].z, xv[b].w);
                                }
                                if ((j + 1) * 32 % G == 0) {
                                    // The group is whole.
                                    const uint32_t s = t.s[r][j * 32 / G];
                                    const float s0 = __uint_as_float(s << 16);
                                    const float s1 = __uint_as_float(s & 0xffff0000u);
#pragma unroll
                                    for (int b = 0; b < NT; ++b)
#pragma unroll
                                        for (int e = 0; e < 4; ++e) {
                                            if (INT4) sum[r][b][e] *= kInt4Factor;
                                            total[r][b][e] = fmaf(sum[r][b][e], e < 2 ? s0 : s1,
                                                                  total[r][b][e]);
                                            sum[r][b][e] = 0.f;
                                        }
                                }
                            }
                        }
                    }
                    load(ahead[d]);
                }
            }
            // The warps' sums, joined in warp order.
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        part[(warp * kColumns + b * 8 + quad * 2 + e % 2) * kRowStride + r * 16 +
                             row + e / 2 * 8] = total[r][b][e];
            __syncthreads();
            const int shares = kWarps / at.groups;
            const int channels = at.groups * 16 * R;
            const int64_t n0 = static_cast<int64_t>(at.at) * 16 * R;
            auto store = [&](int t, int c, float sum) {
                if (n0 + c >= a.N || at.at + c / (16 * R) >= end) return;
                if (a.x_scale) sum *= a.x_scale[m0 + t];
                const int64_t to = (m0 + t) * a.N + n0 + c;
                if (a.dtype == TW_BF16)
                    static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(sum);
                else
                    static_cast<float*>(a.out)[to] = sum;
            };
            for (int e = threadIdx.x; e < tokens * channels; e += kThreads) {
                const int t = e / channels, c = e % channels;
                const float* from = part +
                                    (c / (16 * R) * shares * kColumns + t) * kRowStride +
                                    c % (16 * R);
                float sum = 0.f;
                // fp32 x: the smaller terms first.
                for (int p = parts - 1; p >= 0; --p)
                    for (int w = 0; w < shares; ++w)
                        sum += from[(w * kColumns + p * tokens) * kRowStride];
                if (split == 1)
                    store(t, c, sum);
                else
                    st_cluster_f32(map_to_rank(smem_addr(joined + (buf * split + rank) * per_rank +
                                                         e / split),
                                               static_cast<uint32_t>(e % split)),
                                   sum);
            }
            if (split > 1) {
                // Output e is rank e % split's.  A buffer is written again two rounds
                // later, behind the barrier that its readers reach when done.
                cluster_barrier();
                for (int e = threadIdx.x * split + rank; e < tokens * channels;
                     e += kThreads * split) {
                    float sum = 0.f;
                    for (int r = 0; r < split; ++r)
                        sum += joined[(buf * split + r) * per_rank + e / split];
                    store(e / channels, e % channels, sum);
                }
                buf ^= 1;
            }
            __syncthreads();  // the sums are read
        }
    }
}

// R and depth by the tokens' blocks: x is read from shared memory once per R stripes.
template <bool INT4, int G>
void* entry(int nt) {
    switch (nt) {
        case 1: return reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 1, 1, G, 4>);
        case 2: return reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 2, 2, G, 2>);
        default: return reinterpret_cast<void*>(&w4_gemm_kernel<INT4, 4, 1, G, 2>);
    }
}
constexpr int stripes_per_warp(int nt) { return nt == 2 ? 2 : 1; }
void* kernel_for(int wtype, int nt, int group) {
    if (wtype == TW_INT4)
        return group == 32 ? entry<true, 32>(nt) : group == 64 ? entry<true, 64>(nt)
                                                               : entry<true, 128>(nt);
    return group == 32 ? entry<false, 32>(nt) : group == 64 ? entry<false, 64>(nt)
                                                            : entry<false, 128>(nt);
}

// Shared memory for `columns` columns of x in `nt` blocks, K over `split` CTAs and
// at_once groups at a time of `tokens` tokens.
int64_t smem_bytes(int nt, int columns, int tokens, int64_t K, int split, int at_once) {
    const int r = stripes_per_warp(nt);
    const int64_t part = static_cast<int64_t>(kWarps) * nt * 8 * (16 * r + 1) * 4;
    const int64_t per_rank = (static_cast<int64_t>(at_once) * 16 * r * tokens + split - 1) / split;
    const int64_t joined = split > 1 ? (2 * split * per_rank * 4 + 15) / 16 * 16 : 0;
    const int64_t tiles_k = (K + kW4Inner - 1) / kW4Inner;
    return part + joined + columns * ((tiles_k + split - 1) / split * kW4Inner + kXPad) * 2;
}
// Groups at a time of a CTA that shares them with a cluster (its sums take room).
constexpr int kSplitAtOnce = 4;

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

int w4_gemm_prepare(int smem_optin, int* clusters) {
    for (int wtype : {TW_INT4, TW_E2M1})
        for (int nt = 1; nt <= 4; nt *= 2)
            for (int group = 32; group <= 128; group *= 2) {
                cudaError_t e =
                    cudaFuncSetAttribute(kernel_for(wtype, nt, group),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem_optin);
                if (e != cudaSuccess) return static_cast<int>(e);
            }
    // Clusters of 1, 2, 4, 8 CTAs that run at once (a CTA takes an SM's registers, so
    // the instantiations do not differ).
    for (int i = 0; i < 4; ++i) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = config(1 << i, 1 << i, smem_optin, false, nullptr, attr);
        cudaError_t e =
            cudaOccupancyMaxActiveClusters(clusters + i, kernel_for(TW_INT4, 1, 128), &cfg);
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    return 0;
}

int launch_w4_gemm(const W4GemmArgs& a, int max_sms, const DeviceInfo& d, void* stream) {
    const int64_t sms = max_sms < d.sm_count ? max_sms : d.sm_count;
    const bool whole = max_sms >= d.sm_count;
    const int parts = a.xtype == TW_X_F32 ? 3 : 1;
    // The most tokens at a time whose x fits, K over the fewest CTAs.
    W4Plan plan{a, 0, 1, 1};
    int nt = 0;
    int64_t smem = 0;
    for (int64_t tokens = a.M < kColumnsMax / parts ? a.M : kColumnsMax / parts;
         tokens > 0 && nt == 0; --tokens) {
        const int columns = static_cast<int>(tokens) * parts;
        const int blocks = columns <= 8 ? 1 : columns <= 16 ? 2 : 4;
        for (int split = 1, i = 0; split <= 8 && split <= sms; split *= 2, ++i) {
            if (d.w4_clusters[i] < 1) break;
            const int64_t need = smem_bytes(blocks, columns, static_cast<int>(tokens), a.K, split,
                                            kSplitAtOnce);
            if (need > d.smem_optin) continue;
            plan.tokens = static_cast<int>(tokens);
            plan.split = split;
            nt = blocks;
            smem = need;
            break;
        }
    }
    if (nt == 0) return static_cast<int>(cudaErrorInvalidConfiguration);
    int log2_split = 0;
    while ((1 << log2_split) < plan.split) ++log2_split;
    const int r = stripes_per_warp(nt);
    const int64_t groups = (a.N + 16 * r - 1) / (16 * r);
    int64_t sets = sms / plan.split;
    if (plan.split > 1 && sets > d.w4_clusters[log2_split]) sets = d.w4_clusters[log2_split];
    if (sets > groups) sets = groups;
    // Groups at a time: what a CTA has, at most one per warp; a group's warps have
    // two tiles each where there are that many.
    const int64_t share = (groups + sets - 1) / sets;
    const int64_t tiles = ((a.K + kW4Inner - 1) / kW4Inner + plan.split - 1) / plan.split;
    const int most = plan.split > 1 ? kSplitAtOnce : kWarps;
    while (plan.at_once < most && plan.at_once < share &&
           (plan.at_once < 4 || 2 * kWarps / plan.at_once > tiles))
        plan.at_once *= 2;
    if (!whole && smem < kExclusiveSmemBytes) smem = kExclusiveSmemBytes;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(static_cast<int>(sets * plan.split), plan.split,
                                          static_cast<size_t>(smem), whole, stream, attr);
    void* args[] = {&plan};
    return static_cast<int>(cudaLaunchKernelExC(&cfg, kernel_for(a.wtype, nt, a.group), args));
}

}  // namespace tw
