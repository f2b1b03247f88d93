// tw_w4_rows.cu -- weights into 4-bit packed form (tw.h) and back.
//
// A group's scale is bf16(max |w| / top), a value's code the nearest to w / s: each
// weight is read once and stays in registers between the two.  A warp takes a
// tile of 16 channels x 128 k: lane l of step i holds the eight k from 8 (l % 16)
// of channel 2 i + l / 16 -- exactly one 32-bit word of the tile -- so a group's
// maximum is a few shuffles and a channel's words are 64 contiguous bytes.
// Bound by HBM: the rows in and half a byte per weight out, or the other way
// round.
#include "tw_device.cuh"

namespace tw {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float top4(int wtype) { return wtype == TW_INT4 ? 7.f : 6.f; }

// The eight values of a lane, loaded and as floats.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const void* row, int64_t k) {
        v = ld_global_nc(static_cast<const __nv_bfloat16*>(row) + k);
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void to_float(float* f) const {
        Vec<__nv_bfloat16>::to_float(v, f);
    }
    __device__ __forceinline__ float max_abs8() const {
        uint32_t m = 0;
        max_abs_vec(m, v, static_cast<__nv_bfloat16*>(nullptr));
        return max_abs_of(m, static_cast<__nv_bfloat16*>(nullptr));
    }
};
template <>
struct Eight<float> {
    uint4 v[2];
    __device__ __forceinline__ void load(const void* row, int64_t k) {
        v[0] = ld_global_nc(static_cast<const float*>(row) + k);
        v[1] = ld_global_nc(static_cast<const float*>(row) + k + 4);
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void to_float(float* f) const {
        Vec<float>::to_float(v[0], f);
        Vec<float>::to_float(v[1], f + 4);
    }
    __device__ __forceinline__ float max_abs8() const {
        uint32_t m = 0;
        max_abs_vec(m, v[0], static_cast<float*>(nullptr));
        max_abs_vec(m, v[1], static_cast<float*>(nullptr));
        return __uint_as_float(m);
    }
};

// bf16(m / top), rounded to nearest even once: the quotient in fp32 by Markstein's
// correction (row_scale), then, where it is the very middle of two bf16 values,
// moved an ulp to the side on which the real quotient lies (the remainder is exact).
__device__ __forceinline__ float group_scale(float m, float top) {
    const float c = top == 7.f ? 1.f / 7.f : 1.f / 6.f;
    float s = m * c;
    s = fmaf(fmaf(-s, top, m), c, s);
    const float rest = fmaf(-s, top, m);
    uint32_t bits = __float_as_uint(s);
    if ((bits & 0xffffu) == 0x8000u && rest != 0.f) bits += rest > 0.f ? 1u : ~0u;
    return __bfloat162float(__float2bfloat16_rn(__uint_as_float(bits)));
}

// An fp32 quotient p of v / s that may be the very middle of two codes though the
// real one is not: an ulp towards the real one.  Middles have at most four
// significant bits, so p times s is exact and so is the sign of the remainder.
// (bf16 v: never needed, a real quotient is the middle or a 2^-12th of it away.)
__device__ __forceinline__ float off_middle(float p, float v, float s) {
    uint32_t bits = __float_as_uint(p);
    if ((bits & 0xffffu) == 0) {
        const float rest = fmaf(-p, s, v);
        if (rest != 0.f) bits += (rest > 0.f) == (p > 0.f) ? 1u : ~0u;
    }
    return __uint_as_float(bits);
}

// The word that holds eight codes (tw.h): q[0..7] quotients.  int4: adding 1.5 *
// 2^23 rounds to the nearest even integer; the codes of one half add up, 16 times
// each other, in fp32 without rounding (16 bits).
__device__ __forceinline__ uint32_t word_int4(const float* q) {
    constexpr float kMagic = 12582912.f;
    float half[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 3; v >= 0; --v)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            half[h] = fmaf(half[h], 16.f, (q[2 * v + h] + kMagic) - kMagic);
    // + 8 for each code; 2^23 + x holds x in its low bits.
    const uint32_t lo = __float_as_uint(half[0] + (8388608.f + 0x8888));
    const uint32_t hi = __float_as_uint(half[1] + (8388608.f + 0x8888));
    return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ uint32_t word_e2m1(const float* q) {
    uint32_t w;  // nibbles: values 0, 2, 4, 6 in the low half, 1, 3, 5, 7 in the high
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %3, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %7, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %4, %2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %6;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]),
          "f"(q[7]));
    return (w & 0x00080008u) << 12 | (w & 0x00070007u) << 6 |    // 15, 8..6
           (w & 0x00800080u) << 5 | (w & 0x00700070u) >> 1 |     // 12, 5..3
           (w & 0x08000800u) << 3 | (w & 0x07000700u) << 1 |     // 14, 11..9
           (w & 0x80008000u) >> 2 | (w & 0x70007000u) >> 12;     // 13, 2..0
}

// The eight values of a word.
__device__ __forceinline__ void values_int4(uint32_t w, float* f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t nibble = w >> (i / 2 * 4 + i % 2 * 16) & 15u;
        f[i] = __uint_as_float(0x4b000000u | nibble) - 8388616.f;  // 2^23 + u - (2^23 + 8)
    }
}
// Sign and exponent bits in bf16's places are the value times 2^-126.
__device__ __forceinline__ void values_e2m1(uint32_t w, float* f) {
    const uint32_t p[4] = {w & 0x81c081c0u, w << 3 & 0x81c081c0u,
                           (w >> 3 & 0x01c001c0u) | (w << 1 & 0x80008000u),
                           (w << 6 & 0x01c001c0u) | (w << 2 & 0x80008000u)};
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        f[2 * v] = __uint_as_float(p[v] << 16) * 0x1p126f;
        f[2 * v + 1] = __uint_as_float(p[v] & 0xffff0000u) * 0x1p126f;
    }
}

// Where the lane's word of step i and a group's scale lie in a tile.
__device__ __forceinline__ int word_at(int row, int kk) {
    return row / 8 * 512 + (row % 8 * 4 + kk % 4) * 16 + kk / 4 * 4;
}
__device__ __forceinline__ int scale_at(int row, int kk, int group) {
    return 1024 + row % 8 * (512 / group) + kk * 8 / group * 4 + row / 8 * 2;
}

// kDepth: steps (of two channels) whose loads are in flight at once.
template <typename T, int kDepth>
__global__ void __launch_bounds__(kThreads) quantize_w4_kernel(const __grid_constant__ W4RowsArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, kk = lane % 16;
    const int64_t tiles_k = (a.K + kW4Inner - 1) / kW4Inner;
    const int64_t tiles = (a.N + kW4Channels - 1) / kW4Channels * tiles_k;
    const int tile_bytes = w4_tile_bytes(a.group);
    const float top = top4(a.wtype);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t tile = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
         tile < tiles; tile += warps) {
        const int64_t n0 = tile / tiles_k * kW4Channels;
        const int64_t k = tile % tiles_k * kW4Inner + kk * 8;
        char* to = static_cast<char*>(a.to) + tile * tile_bytes;
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += kDepth) {
            Eight<T> raw[kDepth];
#pragma unroll
            for (int i = 0; i < kDepth; ++i) {
                const int64_t n = n0 + 2 * (i0 + i) + lane / 16;
                if (n < a.N && k < a.K)
                    raw[i].load(static_cast<const T*>(a.from) + n * a.K, k);
                else
                    raw[i].zero();
            }
#pragma unroll
            for (int i = 0; i < kDepth; ++i) {
                const int row = 2 * (i0 + i) + lane / 16;
                float m = raw[i].max_abs8();
                // NaN above everything: the bits of non-negative floats are in order.
                uint32_t most = __float_as_uint(m);
                for (int o = 1; o < a.group / 8; o *= 2)
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                m = __uint_as_float(most);
                const bool finite = quant_finite(m);
                const bool zero = !finite || m < kQuantTiny;
                const float s = group_scale(zero ? 1.f : m, top);
                const RowExact by(s, 1.f);
                float f[8], q[8];
                raw[i].to_float(f);
#pragma unroll
                for (int e = 0; e < 8; e += 2) by.quotients(q + e, f + e);
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[e] = off_middle(q[e], f[e], s);
                }
                uint32_t word = a.wtype == TW_INT4 ? word_int4(q) : word_e2m1(q);
                if (zero) word = a.wtype == TW_INT4 ? 0x88888888u : 0u;
                *reinterpret_cast<uint32_t*>(to + word_at(row, kk)) = word;
                if (kk % (a.group / 8) == 0) {
                    const float held = !finite ? __uint_as_float(0x7fff0000u) : zero ? 0.f : s;
                    *reinterpret_cast<uint16_t*>(to + scale_at(row, kk, a.group)) =
                        static_cast<uint16_t>(__float_as_uint(held) >> 16);
                }
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_w4_kernel(const __grid_constant__ W4RowsArgs a) {
    constexpr int E = Vec<T>::kElems;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, kk = lane % 16;
    const int64_t tiles_k = (a.K + kW4Inner - 1) / kW4Inner;
    const int64_t tiles = (a.N + kW4Channels - 1) / kW4Channels * tiles_k;
    const int tile_bytes = w4_tile_bytes(a.group);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t tile = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
         tile < tiles; tile += warps) {
        const int64_t n0 = tile / tiles_k * kW4Channels;
        const int64_t k = tile % tiles_k * kW4Inner + kk * 8;
        const char* from = static_cast<const char*>(a.from) + tile * tile_bytes;
        uint32_t word[8];
        uint16_t scale[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 2 * i + lane / 16;
            word[i] = *reinterpret_cast<const uint32_t*>(from + word_at(row, kk));
            scale[i] = *reinterpret_cast<const uint16_t*>(from + scale_at(row, kk, a.group));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t n = n0 + 2 * i + lane / 16;
            if (n >= a.N || k >= a.K) continue;
            const float s = __uint_as_float(static_cast<uint32_t>(scale[i]) << 16);
            float f[8];
            if (a.wtype == TW_INT4)
                values_int4(word[i], f);
            else
                values_e2m1(word[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= s;
            T* to = static_cast<T*>(a.to) + n * a.K + k;
#pragma unroll
            for (int e = 0; e < 8; e += E) st_global_cs(to + e, Vec<T>::from_float(f + e));
        }
    }
}

int launch(void* fn, const W4RowsArgs& a, int max_sms, int sm_count, void* stream) {
    const int64_t tiles =
        (a.N + kW4Channels - 1) / kW4Channels * ((a.K + kW4Inner - 1) / kW4Inner);
    const bool whole = max_sms >= sm_count;
    const int64_t ctas = (tiles + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t most = whole ? int64_t{8} * sm_count : max_sms;
    return launch_with_pdl(fn, a, static_cast<int>(ctas < most ? ctas : most), kThreads,
                           whole ? 0 : kExclusiveSmemBytes, whole, stream);
}

void* quantize_for(int dtype) {
    return dtype == TW_BF16 ? reinterpret_cast<void*>(&quantize_w4_kernel<__nv_bfloat16, 4>)
                            : reinterpret_cast<void*>(&quantize_w4_kernel<float, 2>);
}
void* dequantize_for(int dtype) {
    return dtype == TW_BF16 ? reinterpret_cast<void*>(&dequantize_w4_kernel<__nv_bfloat16>)
                            : reinterpret_cast<void*>(&dequantize_w4_kernel<float>);
}

}  // namespace

int w4_rows_prepare(int smem_optin) {
    if (smem_optin < kExclusiveSmemBytes) return static_cast<int>(cudaErrorInvalidValue);
    for (int dt = 0; dt < 2; ++dt)
        for (void* fn : {quantize_for(dt), dequantize_for(dt)}) {
            cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kExclusiveSmemBytes);
            if (e != cudaSuccess) return static_cast<int>(e);
        }
    return 0;
}

int launch_w4_quantize(const W4RowsArgs& a, int max_sms, int sm_count, void* stream) {
    return launch(quantize_for(a.dtype), a, max_sms, sm_count, stream);
}

int launch_w4_dequantize(const W4RowsArgs& a, int max_sms, int sm_count, void* stream) {
    return launch(dequantize_for(a.dtype), a, max_sms, sm_count, stream);
}

}  // namespace tw
