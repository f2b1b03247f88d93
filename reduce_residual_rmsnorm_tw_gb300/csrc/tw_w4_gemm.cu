// tw_w4_gemm.cu -- the product on 4-bit weights with group scales, for few
// tokens: out[t,n] = xs[t] sum_g s[n,g] sum_{k in g} x[t,k] q[n,k].
//
// Bound by reading W once from HBM, half a byte per weight.  The weights become
// bf16 in registers (exact for both types) and feed m16n8k16 with fp32 sums; a
// group's sum is scaled and added to the row's in fp32.  x becomes bf16 without
// loss on its way into shared memory: 8-bit values as they are, fp32 as three
// terms of eight bits each, which count as three tokens.
//
// A CTA owns 16 R channels; its warps take the tiles of K (128 each) in turn and
// add their sums up through shared memory in warp order.  A tile lies in HBM as
// the lanes read it (tw.h): lane (g, q) takes 16 bytes of row g and 16 of row
// g + 8, word j of which holds k = 32 j + 8 q .. + 7, so that a word's two MMAs
// stay within 32 k and a group of 32 can be scaled on its own.
#include <cuda_fp16.h>

#include "tw_device.cuh"

namespace tw {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// k of x in shared memory at a time: whole turns of the warps.
constexpr int kTurn = kWarps * kW4Inner;
constexpr int kXPad = 32;  // bf16: rows of x 64 bytes off each other in the banks
constexpr int kColumnsMax = 32;  // tokens at a time (fp32 x: three for one)
constexpr int kXBytes = kColumnsMax * (kTurn + kXPad) * 2;  // one turn fits for any x

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 16u : 0u)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// A word's eight values as four pairs of bf16: (k, k + 1) for k = 0, 2, 4, 6.
template <bool INT4>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&h)[4]) {
    if constexpr (INT4) {
        // 0x4300 | u is the bf16 128 + u; less 136 it is q = u - 8, exactly.
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t u = (w >> 4 * v & 0x000f000fu) | 0x43004300u;
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(h[v]) : "r"(u), "r"(0x43084308u));
        }
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

// Eight values of x at `from` as bf16 into terms[0] (8-bit and bf16) or as three
// terms that add up to them (fp32: the leading eight bits, cut off, then the next
// eight, then the rest; an infinity or a NaN as its own first term).
__device__ __forceinline__ void x_terms(const char* from, int xtype, uint4 (&terms)[3]) {
    if (xtype == TW_X_BF16) {
        terms[0] = ld_global(from);
    } else if (xtype == TW_X_F32) {
        const uint4 v[2] = {ld_global(from), ld_global(from + 16)};
        float f[8];
        Vec<float>::to_float(v[0], f);
        Vec<float>::to_float(v[1], f + 4);
        uint32_t w[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t[3][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float x = f[2 * i + h];
                const bool finite = fabsf(x) <= 3.402823466e38f;
                t[0][h] = finite ? __uint_as_float(__float_as_uint(x) & 0xffff0000u) : x;
                const float rest = finite ? x - t[0][h] : 0.f;
                t[1][h] = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
                t[2][h] = rest - t[1][h];
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) w[p][i] = pack_bf16(t[p][0], t[p][1]);
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) terms[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(from);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = (i < 2 ? v.x : v.y) >> (i % 2 * 16) & 0xffffu;
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

// Tiles of a warp's FIFO: one is being read.
constexpr int kSlots = 5;

struct W4Plan {
    W4GemmArgs a;
    int tokens;   // per block of tokens
    int x_inner;  // k of x in shared memory at a time, a multiple of kTurn
};

__host__ __device__ constexpr int slot_bytes(int r, int group) {
    return r * (1024 + 4096 / group);
}

// INT4: the weights' type; NT: blocks of eight tokens (fp32 x: three per token);
// R: 16-channel tiles per warp; G: the group.
template <bool INT4, int NT, int R, int G>
__global__ void __launch_bounds__(kThreads)
    w4_gemm_kernel(const __grid_constant__ W4Plan plan) {
    constexpr int kTile = 1024 + 4096 / G, kPieces = kTile / 16;
    const W4GemmArgs& a = plan.a;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = lane / 4, quad = lane % 4;
    const int parts = a.xtype == TW_X_F32 ? 3 : 1;
    const int K = static_cast<int>(a.K);
    const int tiles_k = (K + kW4Inner - 1) / kW4Inner;
    const int64_t stripes = (a.N + 15) / 16;
    const int64_t groups = (stripes + R - 1) / R;
    const int64_t units = groups * ((a.M + plan.tokens - 1) / plan.tokens);
    const uint32_t fifo = smem_addr(smem) + warp * kSlots * slot_bytes(R, G);
    const uint32_t xs = smem_addr(smem) + kWarps * kSlots * slot_bytes(R, G);
    const int x_stride = (plan.x_inner + kXPad) * 2;

    grid_dependency_wait();
    grid_launch_dependents();

    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t m0 = unit / groups * plan.tokens;
        const int tokens = static_cast<int>(a.M - m0 < plan.tokens ? a.M - m0 : plan.tokens);
        const int cols = tokens * parts;
        const int64_t stripe0 = unit % groups * R;
        // This warp's tiles: warp, warp + kWarps, ...
        const int mine = (tiles_k - warp + kWarps - 1) / kWarps;
        auto load = [&](int i) {
            if (i < mine) {
                const int tile = warp + i * kWarps;
                const uint32_t to = fifo + i % kSlots * slot_bytes(R, G);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const bool in = stripe0 + r < stripes;
                    const char* from = static_cast<const char*>(a.packed) +
                                       ((in ? stripe0 + r : 0) * tiles_k + tile) * kTile;
#pragma unroll
                    for (int p = 0; p < kPieces; p += 32)
                        if (p + 32 <= kPieces || p + lane < kPieces)
                            copy_async16(to + r * kTile + (p + lane) * 16, from + (p + lane) * 16, in);
                }
            }
            copy_commit();
        };
#pragma unroll
        for (int i = 0; i < kSlots - 1; ++i) load(i);

        float total[R][NT][4] = {};
        int i = 0;
        for (int k0 = 0; k0 < K; k0 += plan.x_inner) {
            // x of this stretch of K, zero up to the end of its last tile.
            const int k_end = tiles_k * kW4Inner;
            const int inner = k_end - k0 < plan.x_inner ? k_end - k0 : plan.x_inner;
            if (k0 > 0) __syncthreads();
            const int x_size = a.xtype == TW_X_BF16 ? 2 : a.xtype == TW_X_F32 ? 4 : 1;
            for (int e = threadIdx.x; e < tokens * (inner / 8); e += kThreads) {
                const int t = e / (inner / 8), k = e % (inner / 8) * 8;
                uint4 terms[3] = {};
                if (k0 + k < K)
                    x_terms(static_cast<const char*>(a.x) + ((m0 + t) * a.K + k0 + k) * x_size,
                            a.xtype, terms);
                for (int p = 0; p < parts; ++p)
                    sts128(xs + (p * tokens + t) * x_stride + k * 2, terms[p]);
            }
            __syncthreads();
            for (; i < mine && (warp + i * kWarps) * kW4Inner < k0 + inner; ++i) {
                copy_wait<kSlots - 2>();
                __syncwarp();  // pieces that other lanes copied; all have read the last slot
                load(i + kSlots - 1);
                const uint32_t from = fifo + i % kSlots * slot_bytes(R, G);
                const uint32_t x_at = xs + ((warp + i * kWarps) * kW4Inner - k0) * 2 + quad * 16;
                uint4 w[R][2];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    w[r][0] = lds128(from + r * kTile + lane * 16);
                    w[r][1] = lds128(from + r * kTile + 512 + lane * 16);
                }
                float sum[R][NT][4] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 xv[NT];
#pragma unroll
                    for (int b = 0; b < NT; ++b)
                        xv[b] = b * 8 + row < cols ? lds128(x_at + (b * 8 + row) * x_stride + j * 64)
                                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        uint32_t lo[4], hi[4];
                        widen<INT4>(reinterpret_cast<const uint32_t*>(&w[r][0])[j], lo);
                        widen<INT4>(reinterpret_cast<const uint32_t*>(&w[r][1])[j], hi);
#pragma unroll
                        for (int b = 0; b < NT; ++b) {
                            mma(sum[r][b], lo[0], hi[0], lo[1], hi[1], xv[b].x, xv[b].y);
                            mma(sum[r][b], lo[2], hi[2], lo[3], hi[3], xv[b].z, xv[b].w);
                        }
                        if ((j + 1) * 32 % G == 0) {
                            // The group is whole: its scales for rows `row` and + 8.
                            const uint32_t s =
                                lds32(from + r * kTile + 1024 + j * 32 / G * 32 + row * 4);
                            const float s0 = __uint_as_float(s << 16);
                            const float s1 = __uint_as_float(s & 0xffff0000u);
#pragma unroll
                            for (int b = 0; b < NT; ++b) {
                                total[r][b][0] = fmaf(sum[r][b][0], s0, total[r][b][0]);
                                total[r][b][1] = fmaf(sum[r][b][1], s0, total[r][b][1]);
                                total[r][b][2] = fmaf(sum[r][b][2], s1, total[r][b][2]);
                                total[r][b][3] = fmaf(sum[r][b][3], s1, total[r][b][3]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) sum[r][b][e] = 0.f;
                            }
                        }
                    }
                }
            }
        }
        copy_wait<0>();
        // The warps' sums, joined in warp order where x was.
        __syncthreads();
        float* part = reinterpret_cast<float*>(smem + kWarps * kSlots * slot_bytes(R, G));
        constexpr int kColumns = NT * 8, kRowStride = 16 * R + 1;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    part[(warp * kColumns + b * 8 + quad * 2 + e % 2) * kRowStride + r * 16 + row +
                         e / 2 * 8] = total[r][b][e];
        __syncthreads();
        for (int e = threadIdx.x; e < tokens * 16 * R; e += kThreads) {
            const int t = e / (16 * R), c = e % (16 * R);
            const int64_t n = stripe0 * 16 + c;
            if (n >= a.N) continue;
            float sum = 0.f;
            // fp32 x: the smaller terms first.
            for (int p = parts - 1; p >= 0; --p)
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    sum += part[(w * kColumns + p * tokens + t) * kRowStride + c];
            if (a.x_scale) sum *= a.x_scale[m0 + t];
            const int64_t at = (m0 + t) * a.N + n;
            if (a.dtype == TW_BF16)
                static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(sum);
            else
                static_cast<float*>(a.out)[at] = sum;
        }
        __syncthreads();  // the sums are read before x comes again
    }
}

constexpr int kR = 2;

template <bool INT4, int NT>
void* entry(int group) {
    switch (group) {
        case 32: return reinterpret_cast<void*>(&w4_gemm_kernel<INT4, NT, kR, 32>);
        case 64: return reinterpret_cast<void*>(&w4_gemm_kernel<INT4, NT, kR, 64>);
        default: return reinterpret_cast<void*>(&w4_gemm_kernel<INT4, NT, kR, 128>);
    }
}
void* kernel_for(int wtype, int nt, int group) {
    if (wtype == TW_INT4)
        return nt == 1 ? entry<true, 1>(group) : nt == 2 ? entry<true, 2>(group)
                                                         : entry<true, 4>(group);
    return nt == 1 ? entry<false, 1>(group) : nt == 2 ? entry<false, 2>(group)
                                                      : entry<false, 4>(group);
}

// The FIFOs, and x or the warps' sums.
int smem_bytes(int nt, int group, int x_bytes) {
    const int join = kWarps * nt * 8 * (16 * kR + 1) * 4;
    return kWarps * kSlots * slot_bytes(kR, group) + (join > x_bytes ? join : x_bytes);
}

}  // namespace

int w4_gemm_prepare(int smem_optin) {
    for (int wtype : {TW_INT4, TW_E2M1})
        for (int nt = 1; nt <= 4; nt *= 2)
            for (int group = 32; group <= 128; group *= 2) {
                if (smem_bytes(nt, group, kXBytes) > smem_optin)
                    return static_cast<int>(cudaErrorInvalidValue);
                cudaError_t e = cudaFuncSetAttribute(kernel_for(wtype, nt, group),
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     smem_bytes(nt, group, kXBytes));
                if (e != cudaSuccess) return static_cast<int>(e);
            }
    return 0;
}

int launch_w4_gemm(const W4GemmArgs& a, int max_sms, int sm_count, void* stream) {
    const int parts = a.xtype == TW_X_F32 ? 3 : 1;
    W4Plan plan{a, 0, 0};
    plan.tokens = static_cast<int>(a.M < kColumnsMax / parts ? a.M : kColumnsMax / parts);
    const int columns = plan.tokens * parts;
    const int nt = columns <= 8 ? 1 : columns <= 16 ? 2 : 4;
    plan.x_inner = (kXBytes / (columns * 2) - kXPad) / kTurn * kTurn;  // >= kTurn
    const int64_t all = (a.K + kTurn - 1) / kTurn * kTurn;
    if (plan.x_inner > all) plan.x_inner = static_cast<int>(all);
    const int64_t units =
        (a.N + 16 * kR - 1) / (16 * kR) * ((a.M + plan.tokens - 1) / plan.tokens);
    const bool whole = max_sms >= sm_count;
    int smem = smem_bytes(nt, a.group, columns * (plan.x_inner + kXPad) * 2);
    if (!whole && smem < kExclusiveSmemBytes) smem = kExclusiveSmemBytes;
    const int64_t most = whole ? int64_t{1} << 30 : max_sms;
    return launch_with_pdl(kernel_for(a.wtype, nt, a.group), plan,
                           static_cast<int>(units < most ? units : most), kThreads, smem, whole,
                           stream);
}

}  // namespace tw
