// tw_quant.cu -- rows quantised to 8 bits with one scale per token.
//
// s_t = max_h |x[t,h]| / top, q[t,h] = rne(x[t,h] * top / max): a row must be
// seen whole before its first value is written, and is read only once: its
// 16-byte vectors stay in registers between the two.  A row belongs to W
// warps (W * 32 threads holding VPT vectors each), so short rows share a CTA
// and long ones spread over it; one shuffle-free warp maximum, and for W > 1
// one exchange through shared memory.  Bound by HBM: row_bytes in, H + 4 out
// (4096 x 8192 bf16: 16.1 us, 6.2 TB/s).
#include "tw_device.cuh"

namespace tw {
namespace {

constexpr int kQuantThreads = 256;

// CTAs per SM: enough to keep rows' loads in flight while others reduce (bf16 4096 x
// 8192 with three instead of four 19.1 us, 16.1; fp32 4096 x 4096 with four instead
// of five 13.5, 12.8).
__host__ __device__ constexpr int quantize_ctas(int vpt, int elems, bool ahead) {
    return ahead ? 1 : vpt <= 2 ? 8 : vpt == 4 ? (elems == 8 ? 4 : 5) : 1;
}

// AHEAD: a CTA keeps the next row's loads in flight while it reduces and
// stores one (launches held to few SMs, whose CTAs are alone there: 512 x 8192
// on 8 SMs 67 -> 42 us; with eight CTAs on an SM the others do that already,
// and the registers cost 3 %).
template <typename T, int VPT, int W, bool AHEAD>
__global__ void __launch_bounds__(kQuantThreads, quantize_ctas(VPT, Vec<T>::kElems, AHEAD))
    quantize_kernel(const __grid_constant__ QuantParams p) {
    constexpr int E = Vec<T>::kElems;
    constexpr int kRows = kQuantThreads / 32 / W;  // rows per CTA at a time
    __shared__ float warp_max[2][kQuantThreads / 32];
    const int warp = threadIdx.x / 32;
    const int slot = warp / W;                      // row of the CTA
    const int rtid = threadIdx.x - slot * W * 32;   // thread of the row
    const int nvec = static_cast<int>(p.row_bytes / 16);
    const float top = quant_top(p.qtype);
    // The CTA's rows step together, so that every thread meets the barrier.
    int64_t t = p.t0 + static_cast<int64_t>(blockIdx.x) * kRows + slot;
    // The first row on its way into L2 while the launch before this one ends (a
    // hint that reads nothing: what that launch writes is seen all the same;
    // 4096 x 8192 16.8 -> 15.9 us, 1024 x 8192 fp32 7.95 -> 7.2).
    if (!AHEAD && rtid == 0 && t < p.t1)
        bulk_prefetch_l2(static_cast<const char*>(p.x) + t * p.row_bytes,
                         static_cast<uint32_t>(p.row_bytes));
    grid_dependency_wait();
    grid_launch_dependents();
    int buf = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    auto load = [&](uint4 (&raw)[VPT], int64_t t) {
        const char* row = static_cast<const char*>(p.x) + t * p.row_bytes;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = rtid + k * W * 32;
            raw[k] = t < p.t1 && v < nvec ? ld_global_nc(row + static_cast<int64_t>(v) * 16)
                                          : make_uint4(0, 0, 0, 0);
        }
    };
    uint4 next[VPT];
    if constexpr (AHEAD) load(next, t);
    for (; t - slot < p.t1; t += step) {
        const bool live = t < p.t1;
        uint4 raw[VPT];
        if constexpr (AHEAD) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) raw[k] = next[k];
            load(next, t + step);
        } else {
            load(raw, t);
        }
        uint32_t most = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) max_abs_vec(most, raw[k], static_cast<T*>(nullptr));
        float m = warp_max_abs(max_abs_of(most, static_cast<T*>(nullptr)));
        if constexpr (W > 1) {
            if ((threadIdx.x & 31) == 0) warp_max[buf][warp] = m;
            __syncthreads();
            m = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) m = max_abs(m, warp_max[buf][slot * W + w]);
            buf ^= 1;
        }
        const RowExact row(m, top);
        // By every thread: computed in the branch, it holds up the loads ahead (512 x
        // 8192 on 8 SMs 50.6 us against 42.0).
        const float scale = row_scale(m, top, row.zero);
        if (live && rtid == 0) p.out_scale[t] = scale;
        void* out[1] = {p.out};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = rtid + k * W * 32;
            if (live && v < nvec) {
                float f[E];
                Vec<T>::to_float(raw[k], f);
                store_q8<E>(out, 1, t * p.H + static_cast<int64_t>(v) * E, f, row, p.qtype);
            }
        }
    }
}

template <typename T, bool AHEAD>
void* quantize_entry(int vpt, int w) {
    switch (w * 16 + vpt) {
        case 1 * 16 + 1: return reinterpret_cast<void*>(&quantize_kernel<T, 1, 1, AHEAD>);
        case 1 * 16 + 2: return reinterpret_cast<void*>(&quantize_kernel<T, 2, 1, AHEAD>);
        case 2 * 16 + 2: return reinterpret_cast<void*>(&quantize_kernel<T, 2, 2, AHEAD>);
        case 4 * 16 + 2: return reinterpret_cast<void*>(&quantize_kernel<T, 2, 4, AHEAD>);
        case 8 * 16 + 2: return reinterpret_cast<void*>(&quantize_kernel<T, 2, 8, AHEAD>);
        case 8 * 16 + 4: return reinterpret_cast<void*>(&quantize_kernel<T, 4, 8, AHEAD>);
        case 8 * 16 + 8: return reinterpret_cast<void*>(&quantize_kernel<T, 8, 8, AHEAD>);
        default: return nullptr;
    }
}

void* quantize_kernel_for(int dtype, int vpt, int w, bool ahead) {
    if (dtype == TW_BF16)
        return ahead ? quantize_entry<__nv_bfloat16, true>(vpt, w)
                     : quantize_entry<__nv_bfloat16, false>(vpt, w);
    return ahead ? quantize_entry<float, true>(vpt, w) : quantize_entry<float, false>(vpt, w);
}

// Warps per row and vectors per thread for rows of nvec vectors: two vectors
// per thread (32 bytes in flight) until a row takes the whole CTA, more from
// there on.
void quantize_shape(int64_t nvec, int* vpt, int* w) {
    *w = 1;
    *vpt = nvec <= 32 ? 1 : 2;
    while (*w < 8 && nvec > static_cast<int64_t>(*w) * 32 * *vpt) *w *= 2;
    while (nvec > static_cast<int64_t>(*w) * 32 * *vpt) *vpt *= 2;
}

}  // namespace

int quantize_prepare(int smem_optin) {
    if (smem_optin < kExclusiveSmemBytes + 1024) return static_cast<int>(cudaErrorInvalidValue);
    for (int dt = 0; dt < 2; ++dt)
        for (int w = 1; w <= 8; w *= 2)
            for (int vpt = 1; vpt <= 8; vpt *= 2)
                for (bool ahead : {false, true}) {
                    void* fn = quantize_kernel_for(dt, vpt, w, ahead);
                    if (!fn) continue;
                    cudaError_t e = cudaFuncSetAttribute(
                        fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kExclusiveSmemBytes);
                    if (e != cudaSuccess) return static_cast<int>(e);
                }
    return 0;
}

int launch_quantize(const QuantParams& p, int dtype, int max_sms, int sm_count, void* stream) {
    int vpt = 0, w = 0;
    quantize_shape(p.row_bytes / 16, &vpt, &w);
    // Under a budget each CTA is alone on its SM.  Without one, a CTA per row
    // where rows take whole CTAs (the hardware keeps the SMs evenly loaded:
    // 4096 x 8192 17.1 -> 16.8 us), else eight CTAs per SM that loop.
    const bool whole = max_sms >= sm_count;
    void* fn = quantize_kernel_for(dtype, vpt, w, !whole);
    if (!fn) return static_cast<int>(cudaErrorInvalidValue);
    const int64_t rows = kQuantThreads / 32 / w;
    const int64_t ctas = (p.t1 - p.t0 + rows - 1) / rows;
    const int64_t most = !whole ? max_sms : w == 8 ? int64_t{1} << 30 : int64_t{8} * sm_count;
    const int grid = static_cast<int>(ctas < most ? ctas : most);
    return launch_with_pdl(fn, p, grid, kQuantThreads, whole ? 0 : kExclusiveSmemBytes, whole,
                           stream);
}

}  // namespace tw
