// tw_gemv.cu -- the 8-bit matrix product for up to 8 tokens:
// out[t,n] = xs[t] ws[n] sum_k x[t,k] w[n,k].
//
// Every weight is used for so few products that the kernel is bound by reading
// W once from HBM; what counts is that the loads of the whole GPU are in
// flight at once and that little stands between them and the sums.  So there
// is no TMA and no TMEM here: each lane copies 16-byte pieces of W into a FIFO
// of its own in shared memory and multiplies them as they arrive.
//
// Two ways to multiply:
//   DOT   int8, up to 4 tokens: integer dot products of four (dp4a) into
//         32-bit sums, 4 instructions per 16 weights and token.
//   MMA   e4m3, and int8 from 5 tokens on: widened to f16 in registers (exact
//         for both), then m16n8k16 with fp32 sums; the same work for 1 to 8
//         tokens.  The order of K inside a sum is free, so a lane's fragment is
//         simply the 16 bytes it loaded: lane (g, q) holds bytes 16 q ..
//         16 q + 15 of a 64-byte block of rows g and g + 8 of W and of token g,
//         and the four MMAs of the block use four K elements of them each.
// x 8192 x 8192 in int8: one token 12.05 us (5.6 TB/s, 82 % of the measured copy
// rate; 32768 channels 42.4 us, 6.3 TB/s) by DOT against 15.6 by MMA, eight
// tokens 14.7 by MMA against 18.1 by DOT (both before the warming below: 15.7).
//
// A CTA owns 16 R channels; its warps take the 64-byte blocks of K in turn
// (so that the CTA reads long contiguous pieces of a row) and add their sums up
// through shared memory in warp order.
#include <cuda_fp16.h>

#include <type_traits>

#include "tw_device.cuh"

namespace tw {
namespace {

constexpr int kBlock = 64;  // bytes of K per block

// Sixteen 8-bit values as f16 (exact), in an order that is the same for W and
// x.  int8: 0x6400 | (v + 128) is the f16 1024 + 128 + v; one three-input logic
// operation makes two of them from bytes 0 and 2 (and, shifted, 1 and 3).
template <bool INT8>
__device__ __forceinline__ void widen(const uint4& v, uint32_t (&h)[8]) {
    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (INT8) {
            const uint32_t two[2] = {(word[i] & 0x00ff00ffu) ^ 0x64806480u,
                                     ((word[i] >> 8) & 0x00ff00ffu) ^ 0x64806480u};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&two[k]),
                                          __half2half2(__ushort_as_half(0x6480)));
                h[2 * i + k] = *reinterpret_cast<const uint32_t*>(&q);
            }
        } else {
            asm("{\n\t.reg .b16 lo, hi;\n\t"
                "mov.b32 {lo, hi}, %2;\n\t"
                "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
                "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
                : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
                : "r"(word[i]));
        }
    }
}
// d += the products of one block: two rows' pieces of W with x's (n8 tokens).
template <bool INT8>
__device__ __forceinline__ void block_mma(float (&d)[4], const uint4& w0, const uint4& w8,
                                          const uint4& x) {
    uint32_t a[8], c[8], b[8];
    widen<INT8>(w0, a);
    widen<INT8>(w8, c);
    widen<INT8>(x, b);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[2 * i]), "r"(c[2 * i]), "r"(a[2 * i + 1]), "r"(c[2 * i + 1]), "r"(b[2 * i]),
              "r"(b[2 * i + 1]));
}

// 16 bytes of global memory to shared memory behind this thread's back, zeros
// where `in` is false (src is then not read).  CACHED: keep the line in L1.
template <bool CACHED>
__device__ __forceinline__ void copy_async16(uint32_t dst, const char* src, bool in) {
    const uint32_t bytes = in ? 16u : 0u;
    if constexpr (CACHED)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                     "r"(bytes)
                     : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                     "r"(bytes)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
    c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
    c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
    c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

// Bytes of each of its first channels a CTA warms L2 with before the launch
// before it has ended (8 tokens int8, 8192 x 8192: 15.6 -> 14.7 us; one token,
// 8192 x 1024: 3.64 -> 3.05; 1024 bytes 15.2, 8192 bytes 17.5 and 3.05).
constexpr int kWarm = 2048;

// Slots of a warp's FIFO, by what a step costs in shared memory: 2 R pieces of W
// per lane and one of x.  One slot is being read, so one step fewer is in flight.
__host__ __device__ constexpr int ahead(int r) { return r == 2 ? 4 : 7; }
__host__ __device__ constexpr int step_bytes(int r) { return (2 * r + 1) * 32 * 16; }
__host__ __device__ constexpr int fifo_bytes(int warps, int r) {
    return warps * ahead(r) * step_bytes(r);
}
__host__ __device__ constexpr int gemv_smem(int warps, int r) {
    return fifo_bytes(warps, r) + warps * 8 * (16 * r + 1) * 4;
}

// MT: at most this many tokens (1, 2, 4: DOT; 8: MMA); R: 16-channel tiles per
// CTA; kWarps: 8, two CTAs to an SM, or 16, one.  Two smaller CTAs keep the SM
// reading while one reduces a group, and the next launch's start beside the
// last groups (one token int8, 8192 x 1024: 5.1 -> 4.1 us, 5120 x 5120:
// 8.2 -> 6.9 us); one of 16 where there are not enough channel groups for two
// (4096 x 4096: 5.0 us against 5.4), and under an SM budget.
//
// The bytes in flight are what the HBM rate follows, so the loads go through a
// FIFO in shared memory instead of registers, with ahead(R) - 1 steps in flight: 96
// KB of W per SM.  Each lane reads back the pieces of W it copied itself.  The steps
// run on across the CTA's channel groups, so that a group's reduction does not
// drain the FIFO.
template <bool INT8, int MT, int R, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps)
    gemv_kernel(const __grid_constant__ GemmArgs g) {
    constexpr bool DOT = INT8 && MT < 8;
    static_assert(DOT || MT == 8, "the MMA's tokens come in eights");
    using Sum = std::conditional_t<DOT, int, float>;
    constexpr int kChannels = 16 * R, D = ahead(R);
    extern __shared__ __align__(16) unsigned char smem[];
    Sum(*part)[MT][kChannels + 1] =
        reinterpret_cast<Sum(*)[MT][kChannels + 1]>(smem + fifo_bytes(kWarps, R));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = lane / 4, piece = warp * kBlock + lane % 4 * 16;
    const int M = static_cast<int>(g.M), K = static_cast<int>(g.K);
    const uint32_t warp_fifo = smem_addr(smem) + static_cast<uint32_t>(warp * D * step_bytes(R));
    const uint32_t fifo = warp_fifo + lane * 16;
    // The first steps' W on its way into L2 while the launch before this one
    // ends (a hint that reads nothing: what that launch writes is seen all the
    // same): the CTA's first channels, a row per thread.
    if (threadIdx.x < kChannels) {
        const int64_t n = static_cast<int64_t>(blockIdx.x) * kChannels + threadIdx.x;
        const int bytes = K < kWarm ? K : kWarm;
        if (n < g.N) bulk_prefetch_l2(static_cast<const char*>(g.w) + n * g.K, bytes);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t groups = (g.N + kChannels - 1) / kChannels;
    const int per_group = (K + kWarps * kBlock - 1) / (kWarps * kBlock);  // steps
    const int64_t my_groups = (groups - blockIdx.x + gridDim.x - 1) / gridDim.x;
    const int64_t steps = my_groups * per_group;

    // The step to load next: its channel group's first row (of this lane) and
    // its place in K.
    int64_t n_load = static_cast<int64_t>(blockIdx.x) * kChannels + row;
    int at_load = 0, slot_load = 0;
    const char* w0 = static_cast<const char*>(g.w);
    const char* w = w0 + n_load * g.K;
    const char* x = static_cast<const char*>(g.x) + static_cast<int64_t>(row) * g.K;
    const int64_t next_group = static_cast<int64_t>(gridDim.x) * kChannels;
    auto load = [&]() {
        const int k = at_load * kWarps * kBlock + piece;
        const uint32_t to = fifo + slot_load * step_bytes(R);
#pragma unroll
        for (int r = 0; r < 2 * R; ++r) {
            const bool in = k < K && n_load + r * 8 < g.N;
            copy_async16<false>(to + r * 512, in ? w + static_cast<int64_t>(r) * 8 * g.K + k : w0,
                                in);
        }
        const bool in = k < K && row < M;
        if (MT == 8 || row < MT) copy_async16<true>(to + 2 * R * 512, in ? x + k : w0, in);
        if (++at_load == per_group) {
            at_load = 0;
            n_load += next_group;
            w += next_group * g.K;
        }
        if (++slot_load == D) slot_load = 0;
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) {
        if (i < steps) load();
        copy_commit();
    }

    // DOT: [row of W][token]; MMA: the accumulators of each tile.
    Sum d[DOT ? 2 * R : R][DOT ? MT : 4] = {};
    int at = 0, slot = 0;
    int64_t n0 = static_cast<int64_t>(blockIdx.x) * kChannels;
    for (int64_t s = 0; s < steps; ++s) {
        copy_wait<D - 2>();
        __syncwarp();  // DOT lanes read the x that other lanes copied
        const uint32_t from = fifo + slot * step_bytes(R);
        uint4 wv[2 * R];
#pragma unroll
        for (int r = 0; r < 2 * R; ++r) wv[r] = lds(from + r * 512);
        if constexpr (DOT) {
            const uint32_t xs = warp_fifo + slot * step_bytes(R) + 2 * R * 512 + lane % 4 * 16;
            uint4 xv[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) xv[t] = lds(xs + t * 64);
            // Into the slot read a step ago (by every lane: the __syncwarp).
            if (s + D - 1 < steps) load();
            copy_commit();
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int r = 0; r < 2 * R; ++r) d[r][t] = dot16(wv[r], xv[t], d[r][t]);
        } else {
            const uint4 xv = lds(from + 2 * R * 512);
            if (s + D - 1 < steps) load();
            copy_commit();
#pragma unroll
            for (int r = 0; r < R; ++r) block_mma<INT8>(d[r], wv[2 * r], wv[2 * r + 1], xv);
        }
        if (++slot == D) slot = 0;
        if (++at < per_group) continue;
        // The group is done.
        at = 0;
        if constexpr (DOT) {
#pragma unroll
            for (int r = 0; r < 2 * R; ++r)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    int v = d[r][t];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    if (lane % 4 == 0) part[warp][t][r * 8 + row] = v;
                    d[r][t] = 0;
                }
        } else {
            // d[r]: channels row and row + 8, tokens 2 (lane % 4) and the next.
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    part[warp][lane % 4 * 2 + (e & 1)][r * 16 + row + (e >> 1) * 8] = d[r][e];
                    d[r][e] = 0;
                }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < MT * kChannels; i += 32 * kWarps) {
            const int t = i / kChannels, c = i % kChannels;
            const int64_t n = n0 + c;
            if (t >= M || n >= g.N) continue;
            Sum total = 0;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) total += part[k][t][c];
            const float sum = static_cast<float>(total) * g.x_scale[t] * g.w_scale[n];
            if (g.dtype == TW_BF16)
                static_cast<__nv_bfloat16*>(g.out)[t * g.N + n] = __float2bfloat16_rn(sum);
            else
                static_cast<float*>(g.out)[t * g.N + n] = sum;
        }
        __syncthreads();
        n0 += next_group;
    }
}

template <int R, int WARPS>
void* gemv_entry(bool int8, int mt) {
    if (!int8) return reinterpret_cast<void*>(&gemv_kernel<false, 8, R, WARPS>);
    switch (mt) {
        case 1: return reinterpret_cast<void*>(&gemv_kernel<true, 1, R, WARPS>);
        case 2: return reinterpret_cast<void*>(&gemv_kernel<true, 2, R, WARPS>);
        case 4: return reinterpret_cast<void*>(&gemv_kernel<true, 4, R, WARPS>);
        default: return reinterpret_cast<void*>(&gemv_kernel<true, 8, R, WARPS>);
    }
}

// The instantiation for mt = 1, 2, 4, 8 tokens, r = 1, 2 tiles and 8 or 16
// warps.
void* gemv_kernel_for(bool int8, int mt, int r, int warps) {
    if (warps == 8) return r == 1 ? gemv_entry<1, 8>(int8, mt) : gemv_entry<2, 8>(int8, mt);
    return r == 1 ? gemv_entry<1, 16>(int8, mt) : gemv_entry<2, 16>(int8, mt);
}

}  // namespace

int gemv_prepare(int smem_optin) {
    for (bool int8 : {false, true})
        for (int mt = 1; mt <= 8; mt *= 2)
            for (int r = 1; r <= 2; ++r)
                for (int warps = 8; warps <= 16; warps *= 2) {
                    if (gemv_smem(warps, r) > smem_optin)
                        return static_cast<int>(cudaErrorInvalidValue);
                    cudaError_t e = cudaFuncSetAttribute(
                        gemv_kernel_for(int8, mt, r, warps),
                        cudaFuncAttributeMaxDynamicSharedMemorySize, gemv_smem(warps, r));
                    if (e != cudaSuccess) return static_cast<int>(e);
                }
    return 0;
}

int launch_gemv(const GemmArgs& g, int max_sms, const DeviceInfo& d, void* stream) {
    const int64_t sms = max_sms < d.sm_count ? max_sms : d.sm_count;
    const bool whole = max_sms >= d.sm_count;
    int mt = 1;
    while (mt < g.M) mt *= 2;
    // Two channel tiles per CTA halve what each channel pays for x; one where
    // that leaves SMs without work.
    const int r = g.N > 16 * sms ? 2 : 1;
    const int warps = whole && g.N > 32 * sms ? 8 : 16;
    const int64_t groups = (g.N + 16 * r - 1) / (16 * r);
    const int64_t most = warps == 8 ? 2 * sms : sms;
    const int grid = static_cast<int>(groups < most ? groups : most);
    return launch_with_pdl(gemv_kernel_for(g.qtype == TW_INT8, mt, r, warps), g, grid, 32 * warps,
                           gemv_smem(warps, r), whole, stream);
}

}  // namespace tw
