// tw_gemm.cu -- matrix product of 8-bit operands with scales per token and
// channel: out[t,n] = xs[t] ws[n] sum_k x[t,k] w[n,k].
//
// Plain tiles: a CTA computes 64 tokens x 64 channels, each thread 4 x 4 of
// them, from 32-deep slices of both operands widened to fp32 in shared memory.
#include <cuda_fp8.h>

#include "tw_device.cuh"

namespace tw {
namespace {

constexpr int kTile = 64, kDeep = 32;

__device__ __forceinline__ float widen(uint8_t b, int qtype) {
    if (qtype == TW_INT8) return static_cast<float>(static_cast<int8_t>(b));
    __nv_fp8_e4m3 v;
    v.__x = b;
    return static_cast<float>(v);
}

__global__ void __launch_bounds__(256) gemm_kernel(const __grid_constant__ GemmArgs g) {
    __shared__ float xs[kDeep][kTile + 1], ws[kDeep][kTile + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int64_t nt = (g.N + kTile - 1) / kTile, mt = (g.M + kTile - 1) / kTile;
    for (int64_t tile = blockIdx.x; tile < nt * mt; tile += gridDim.x) {
        const int64_t n0 = tile % nt * kTile, m0 = tile / nt * kTile;
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < g.K; k0 += kDeep) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTile * kDeep; i += 256) {
                const int r = i / kDeep, k = i % kDeep;
                const bool in = k0 + k < g.K;
                xs[k][r] = in && m0 + r < g.M
                               ? widen(static_cast<const uint8_t*>(g.x)[(m0 + r) * g.K + k0 + k], g.qtype)
                               : 0.f;
                ws[k][r] = in && n0 + r < g.N
                               ? widen(static_cast<const uint8_t*>(g.w)[(n0 + r) * g.K + k0 + k], g.qtype)
                               : 0.f;
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < kDeep; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], acc[i][j]);
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m >= g.M || n >= g.N) continue;
                const float v = acc[i][j] * g.x_scale[m] * g.w_scale[n];
                if (g.dtype == TW_BF16)
                    static_cast<__nv_bfloat16*>(g.out)[m * g.N + n] = __float2bfloat16_rn(v);
                else
                    static_cast<float*>(g.out)[m * g.N + n] = v;
            }
    }
}

}  // namespace

int gemm_prepare(int) {
    return static_cast<int>(cudaFuncSetAttribute(
        gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExclusiveSmemBytes));
}

int launch_gemm(const GemmArgs& g, int max_sms, const DeviceInfo& d, void* stream) {
    const int64_t tiles = ((g.N + kTile - 1) / kTile) * ((g.M + kTile - 1) / kTile);
    const bool whole = max_sms >= d.sm_count;
    const int64_t most = whole ? int64_t{4} * d.sm_count : max_sms;
    const int grid = static_cast<int>(tiles < most ? tiles : most);
    return launch_with_pdl(reinterpret_cast<void*>(&gemm_kernel), g, grid, 256,
                           whole ? 0 : kExclusiveSmemBytes, whole, stream);
}

}  // namespace tw
