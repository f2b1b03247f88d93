// tw_w4_rows.cu -- weights into 4-bit packed form (tw.h) and back.
//
// A group's scale is bf16(max |w| / top), a value's code the nearest to w / s: each
// weight is read once and stays in registers between the two.  A warp takes a
// tile of 16 channels x 128 k: lane l of step i holds the eight k from 8 (l % 16)
// of channel 2 i + l / 16 -- exactly one 32-bit word of the tile -- so a group's
// maximum is a few shuffles and a channel's words are 64 contiguous bytes.
// Bound by HBM: the rows in and half a byte per weight out, or the other way
// round (8192 x 8192 bf16 to int4 27.2 us, 6.2 TB/s, to e2m1 30.7; back 25.6, 6.6 TB/s;
// 4090 x 5120 fp32 to e2m1 with groups of 32 17.0 and 15.1).  Quantising takes some ten
// instructions a weight, for which loads in flight have to cover.
#include "tw_device.cuh"

namespace tw {
namespace {

constexpr int kThreads = 256, kTilesPerUnit = kThreads / 32;

// The eight values of a lane, loaded and as floats.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p, bool) { v = ld_global_nc(p); }
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
    __device__ __forceinline__ void load(const float* p, bool sectors) {
        if (!sectors) {  // p is 16-byte aligned only
            v[0] = ld_global_nc(p);
            v[1] = ld_global_nc(p + 4);
            return;
        }
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x),
                       "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                     : "l"(p));
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
// correction (row_scale), then, where that is the very middle of two bf16 values,
// moved an ulp to the side on which the real quotient lies (the remainder is exact).
// bf16 maxima need no look: thirds and sevenths of eight bits stay away from middles.
template <typename T, bool INT4>
__device__ __forceinline__ float group_scale(float m) {
    constexpr float top = INT4 ? 7.f : 6.f;
    constexpr float c = 1.f / top;
    float s = m * c;
    s = fmaf(fmaf(-s, top, m), c, s);
    if constexpr (sizeof(T) == 4) {
        const float rest = fmaf(-s, top, m);
        uint32_t bits = __float_as_uint(s);
        if ((bits & 0xffffu) == 0x8000u && rest != 0.f) bits += rest > 0.f ? 1u : ~0u;
        s = __uint_as_float(bits);
    }
    return __bfloat162float(__float2bfloat16_rn(s));
}

// An fp32 quotient p of v / s that may be the very middle of two codes though the
// real one is not: an ulp towards the real one.  Middles have at most four
// significant bits, so p times s is exact and so is the sign of the remainder.  A zero
// (v = 0, or a quotient that underflowed) is no middle and has no ulp below it.
// (bf16 v: never needed, a real quotient is the middle or a 2^-12th of it away.)
__device__ __forceinline__ float off_middle(float p, float v, float s) {
    uint32_t bits = __float_as_uint(p);
    if ((bits & 0xffffu) == 0 && p != 0.f) {
        const float rest = fmaf(-p, s, v);
        if (rest != 0.f) bits += (rest > 0.f) == (p > 0.f) ? 1u : ~0u;
    }
    return __uint_as_float(bits);
}

// Whether any of eight floats has zeros only in its last 16 bits, as middles have.
__device__ __forceinline__ bool any_round(const float* q) {
    uint32_t least = 0xffffffffu;  // two halves side by side
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        asm("min.u16x2 %0, %0, %1;"
            : "+r"(least)
            : "r"(__byte_perm(__float_as_uint(q[e]), __float_as_uint(q[e + 1]), 0x5410)));
    return (least & 0xffffu) == 0 || least >> 16 == 0;
}

// Quotients of bf16 v, plus kGridBase: v times an approximate reciprocal, off by 2^-20 at
// most, rounded to multiples of 2^-15.  A real quotient is a middle, which that gives
// exactly, or 2^-14 of one away at least, which stays on its side.
constexpr float kGridBase = 384.f;
template <bool PLUS_BASE>
__device__ __forceinline__ void grid_quotients(float* q, const float* v, float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        asm("{\n\t.reg .b64 a, h, c;\n\t"
            "mov.b64 a, {%2, %3};\n\t"
            "mov.b64 h, {%4, %4};\n\t"
            "mov.b64 c, {%5, %5};\n\t"
            "fma.rn.f32x2 a, a, h, c;\n\t"
            "mov.b64 {%0, %1}, a;\n\t}"
            : "=f"(q[e]), "=f"(q[e + 1])
            : "f"(v[e]), "f"(v[e + 1]), "f"(r), "f"(kGridBase));
        if constexpr (!PLUS_BASE)
            asm("{\n\t.reg .b64 a, c;\n\t"
                "mov.b64 a, {%0, %1};\n\t"
                "mov.b64 c, {%2, %2};\n\t"
                "add.rn.f32x2 a, a, c;\n\t"
                "mov.b64 {%0, %1}, a;\n\t}"
                : "+f"(q[e]), "+f"(q[e + 1])
                : "f"(-kGridBase));
    }
}

// Quotients of fp32 v: p = v r with an approximate reciprocal r, then p + (v - p s) r,
// the remainder being exact but for what is below fp32's range (Markstein's correction:
// right to 2^-45 before the one rounding, under every scale; a reciprocal in two parts is
// not from 2^125 up, where its low part is a subnormal).
__device__ __forceinline__ void quotients(float* q, const float* v, float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        asm("{\n\t.reg .b64 a, p, h, s;\n\t"
            "mov.b64 a, {%2, %3};\n\t"
            "mov.b64 h, {%4, %4};\n\t"
            "mov.b64 s, {%5, %5};\n\t"
            "mul.rn.f32x2 p, a, h;\n\t"
            "fma.rn.f32x2 a, p, s, a;\n\t"
            "fma.rn.f32x2 p, a, h, p;\n\t"
            "mov.b64 {%0, %1}, p;\n\t}"
            : "=f"(q[e]), "=f"(q[e + 1])
            : "f"(v[e]), "f"(v[e + 1]), "f"(r), "f"(-s));
}

// The word that holds eight codes (tw.h): q[0..7] quotients.  int4: 2^23 + 8 + q is
// rounded to the nearest even integer and holds q + 8 in its last bits; a half's four
// are put together by multiplying by 16 and adding, modulo 2^32 (of the rest, 0x4b000000,
// nothing reaches the last 24 bits).
__device__ __forceinline__ uint32_t word_int4(const float* q, float base) {
    uint32_t half[2] = {0, 0};
#pragma unroll
    for (int v = 3; v >= 0; --v) {
        uint32_t b[2];
        asm("{\n\t.reg .b64 a, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 c, {%4, %4};\n\t"
            "add.rn.f32x2 a, a, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
            : "=r"(b[0]), "=r"(b[1])
            : "f"(q[2 * v]), "f"(q[2 * v + 1]), "f"(8388616.f - base));
#pragma unroll
        for (int h = 0; h < 2; ++h) half[h] = half[h] * 16u + b[h];
    }
    return __byte_perm(half[0], half[1], 0x5410);
}
__device__ __forceinline__ uint32_t word_e2m1(const float* q) {
    uint32_t w;  // nibbles: values 6, 2, 4, 0 in the low half, 7, 3, 5, 1 in the high: the
                 // order whose fields take the fewest shifts
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %3, %7;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %1, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %4, %8;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %2, %6;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]),
          "f"(q[7]));
    return (w & 0x80078007u) |                                   // 15; 2..0
           (w >> 6 & 0x01c001c0u) |                              // 8..6
           (w >> 1 & 0x00380038u) | (w << 5 & 0x10001000u) |     // 5..3, 12
           (w << 1 & 0x0e000e00u) | (w << 3 & 0x40004000u) |     // 11..9, 14
           (w << 10 & 0x20002000u);                              // 13
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
template <int G>
__device__ __forceinline__ int scale_at(int row, int kk) {
    return 1024 + row % 8 * (512 / G) + kk / (G / 8) * 4 + row / 8 * 2;
}

// A unit of work: eight tiles (a warp each) of one stripe of channels.
struct Unit {
    int64_t stripe;
    int tile;  // of the stripe, this warp's
    __device__ __forceinline__ Unit(int64_t unit, int units_k) {
        int64_t rest;
        if (unit >> 31 == 0) {  // 64-bit division: tens of instructions more
            stripe = static_cast<uint32_t>(unit) / static_cast<uint32_t>(units_k);
            rest = static_cast<uint32_t>(unit) % static_cast<uint32_t>(units_k);
        } else {
            stripe = unit / units_k;
            rest = unit % units_k;
        }
        tile = static_cast<int>(rest) * kTilesPerUnit + static_cast<int>(threadIdx.x / 32);
    }
};

// Steps (of two channels) of a warp, whose loads are in flight at once, and CTAs on an SM
// that find registers: bf16 a whole tile and four (three CTAs 31.2 us, 28.9; half a tile
// 33), fp32 half a tile, the next CTA the other half, and five (a whole tile in two steps
// 18.4, 17.0; four CTAs 17.0, 16.7).
template <typename T>
__host__ __device__ constexpr int depth_of() { return sizeof(T) == 2 ? 8 : 4; }

template <typename T, bool INT4, int G>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 5)
    quantize_w4_kernel(const __grid_constant__ W4RowsArgs a) {
    constexpr int kTile = w4_tile_bytes(G);
    constexpr int kDepth = depth_of<T>(), kParts = kW4Channels / 2 / kDepth;
    const int lane = threadIdx.x % 32, kk = lane % 16;
    const int K = static_cast<int>(a.K);
    const int tiles_k = (K + kW4Inner - 1) / kW4Inner;
    const int units_k = (tiles_k + kTilesPerUnit - 1) / kTilesPerUnit;
    const int64_t units = (a.N + kW4Channels - 1) / kW4Channels * units_k * kParts;
    const bool sectors = (reinterpret_cast<uintptr_t>(a.from) & 31) == 0;
    // The first rows on their way into L2 while the launch before this one ends (a hint
    // that reads nothing: what that launch writes is seen all the same).  By the CTAs that
    // may start before it has ended only (8192 x 8192 there and back, in turn, 53.1 us with
    // all of them, 48.2).
    if (threadIdx.x < 2 * kDepth && blockIdx.x < a.warm) {
        const Unit at(blockIdx.x / kParts, units_k);
        const int64_t n =
            at.stripe * kW4Channels + blockIdx.x % kParts * (2 * kDepth) + threadIdx.x;
        const int k = at.tile * kW4Inner;
        const int left = K - k < kTilesPerUnit * kW4Inner ? K - k : kTilesPerUnit * kW4Inner;
        if (n < a.N)
            bulk_prefetch_l2(static_cast<const T*>(a.from) + n * a.K + k,
                             static_cast<uint32_t>(left * sizeof(T)));
    }
    grid_dependency_wait();
    grid_launch_dependents();
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const Unit at(unit / kParts, units_k);
        if (at.tile >= tiles_k) continue;
        const int i0 = static_cast<int>(unit % kParts) * kDepth;
        const int64_t n0 = at.stripe * kW4Channels;
        const int rows = a.N - n0 < kW4Channels ? static_cast<int>(a.N - n0) : kW4Channels;
        const int k = at.tile * kW4Inner + kk * 8;
        const T* from = static_cast<const T*>(a.from) + (n0 + lane / 16) * a.K + k;
        char* to = static_cast<char*>(a.to) + (at.stripe * tiles_k + at.tile) * kTile;
        Eight<T> raw[kDepth];
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            if (2 * (i0 + i) + lane / 16 < rows && k < K)
                raw[i].load(from + 2 * (i0 + i) * a.K, sectors);
            else
                raw[i].zero();
        }
        uint32_t most[kDepth];
#pragma unroll
        for (int i = 0; i < kDepth; ++i) most[i] = __float_as_uint(raw[i].max_abs8());
        // NaN above everything: the bits of non-negative floats are in order.
#pragma unroll
        for (int o = 1; o < G / 8; o *= 2)
#pragma unroll
            for (int i = 0; i < kDepth; ++i)
                most[i] = max(most[i], __shfl_xor_sync(0xffffffffu, most[i], o));
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            const int row = 2 * (i0 + i) + lane / 16;
            const float m = __uint_as_float(most[i]);
            const bool finite = quant_finite(m);
            const bool zero = !finite || m < kQuantTiny;
            const float s = group_scale<T, INT4>(zero ? 1.f : m);
            float f[8], q[8];
            raw[i].to_float(f);
            constexpr bool kGrid = sizeof(T) == 2;
            if constexpr (kGrid) {
                grid_quotients<INT4>(q, f, s);
            } else {
                quotients(q, f, s);
                if (any_round(q)) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[e] = off_middle(q[e], f[e], s);
                }
            }
            uint32_t word = INT4 ? word_int4(q, kGrid ? kGridBase : 0.f) : word_e2m1(q);
            if (zero) word = INT4 ? 0x88888888u : 0u;
            *reinterpret_cast<uint32_t*>(to + word_at(row, kk)) = word;
            if (kk % (G / 8) == 0) {
                const float held = !finite ? __uint_as_float(0x7fff0000u) : zero ? 0.f : s;
                *reinterpret_cast<uint16_t*>(to + scale_at<G>(row, kk)) =
                    static_cast<uint16_t>(__float_as_uint(held) >> 16);
            }
        }
    }
}

template <typename T, bool INT4, int G>
__global__ void __launch_bounds__(kThreads)
    dequantize_w4_kernel(const __grid_constant__ W4RowsArgs a) {
    constexpr int kTile = w4_tile_bytes(G), kSteps = kW4Channels / 2;
    const int lane = threadIdx.x % 32, kk = lane % 16;
    const int K = static_cast<int>(a.K);
    const int tiles_k = (K + kW4Inner - 1) / kW4Inner;
    const int units_k = (tiles_k + kTilesPerUnit - 1) / kTilesPerUnit;
    const int64_t units = (a.N + kW4Channels - 1) / kW4Channels * units_k;
    const bool sectors = (reinterpret_cast<uintptr_t>(a.to) & 31) == 0;
    // As above, by every CTA (8192 x 8192 27.0 -> 25.6 us; by the first ones only 26.7).
    if (threadIdx.x == 0) {
        const Unit at(blockIdx.x, units_k);
        const int left = tiles_k - at.tile < kTilesPerUnit ? tiles_k - at.tile : kTilesPerUnit;
        bulk_prefetch_l2(static_cast<const char*>(a.from) + (at.stripe * tiles_k + at.tile) * kTile,
                         static_cast<uint32_t>(left * kTile));
    }
    grid_dependency_wait();
    grid_launch_dependents();
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const Unit at(unit, units_k);
        if (at.tile >= tiles_k) continue;
        const int64_t n0 = at.stripe * kW4Channels;
        const int rows = a.N - n0 < kW4Channels ? static_cast<int>(a.N - n0) : kW4Channels;
        const int k = at.tile * kW4Inner + kk * 8;
        const char* from =
            static_cast<const char*>(a.from) + (at.stripe * tiles_k + at.tile) * kTile;
        T* to = static_cast<T*>(a.to) + (n0 + lane / 16) * a.K + k;
        uint32_t word[kSteps];
        uint16_t scale[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int row = 2 * i + lane / 16;
            word[i] = *reinterpret_cast<const uint32_t*>(from + word_at(row, kk));
            scale[i] = *reinterpret_cast<const uint16_t*>(from + scale_at<G>(row, kk));
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i, to += 2 * a.K) {
            if (2 * i + lane / 16 >= rows || k >= K) continue;
            const float s = __uint_as_float(static_cast<uint32_t>(scale[i]) << 16);
            float f[8];
            if (INT4)
                values_int4(word[i], f);
            else
                values_e2m1(word[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= s;
            if constexpr (sizeof(T) == 2) {
                st_global_cs(to, Vec<T>::from_float(f));
            } else if (sectors) {
                asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to),
                             "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]),
                             "f"(f[6]), "f"(f[7])
                             : "memory");
            } else {
                st_global_cs(to, Vec<T>::from_float(f));
                st_global_cs(to + 4, Vec<T>::from_float(f + 4));
            }
        }
    }
}

template <typename T, bool INT4, int G>
void* entry(bool quantize) {
    return quantize
               ? reinterpret_cast<void*>(&quantize_w4_kernel<T, INT4, G>)
               : reinterpret_cast<void*>(&dequantize_w4_kernel<T, INT4, G>);
}
template <typename T, bool INT4>
void* entry_for(int group, bool quantize) {
    return group == 32   ? entry<T, INT4, 32>(quantize)
           : group == 64 ? entry<T, INT4, 64>(quantize)
                         : entry<T, INT4, 128>(quantize);
}
void* kernel_for(const W4RowsArgs& a, bool quantize) {
    const bool int4 = a.wtype == TW_INT4;
    if (a.dtype == TW_BF16)
        return int4 ? entry_for<__nv_bfloat16, true>(a.group, quantize)
                    : entry_for<__nv_bfloat16, false>(a.group, quantize);
    return int4 ? entry_for<float, true>(a.group, quantize)
                : entry_for<float, false>(a.group, quantize);
}

// A CTA for eight tiles (a whole GPU's persistent ones were slower: 8192 x 8192 bf16 54.4
// us against 51.1), fewer that loop, each alone on its SM, under a budget.
int launch(W4RowsArgs a, bool quantize, int max_sms, int sm_count, void* stream) {
    const int64_t tiles_k = (a.K + kW4Inner - 1) / kW4Inner;
    const int parts = !quantize ? 1 : kW4Channels / 2 /
                                          (a.dtype == TW_BF16 ? depth_of<__nv_bfloat16>()
                                                              : depth_of<float>());
    const int64_t units = (a.N + kW4Channels - 1) / kW4Channels *
                          ((tiles_k + kTilesPerUnit - 1) / kTilesPerUnit) * parts;
    const bool whole = max_sms >= sm_count;
    a.warm = whole ? 4 * static_cast<unsigned>(sm_count) : 0;
    const int64_t most = whole ? (int64_t{1} << 31) - 1 : max_sms;
    return launch_with_pdl(kernel_for(a, quantize), a,
                           static_cast<int>(units < most ? units : most), kThreads,
                           whole ? 0 : kExclusiveSmemBytes, whole, stream);
}

}  // namespace

int w4_rows_prepare(int smem_optin) {
    if (smem_optin < kExclusiveSmemBytes) return static_cast<int>(cudaErrorInvalidValue);
    W4RowsArgs a{};
    for (a.dtype = 0; a.dtype < 2; ++a.dtype)
        for (a.wtype = 0; a.wtype < 2; ++a.wtype)
            for (a.group = 32; a.group <= 128; a.group *= 2)
                for (bool quantize : {false, true}) {
                    cudaError_t e = cudaFuncSetAttribute(
                        kernel_for(a, quantize), cudaFuncAttributeMaxDynamicSharedMemorySize,
                        kExclusiveSmemBytes);
                    if (e != cudaSuccess) return static_cast<int>(e);
                }
    return 0;
}

int launch_w4_quantize(const W4RowsArgs& a, int max_sms, int sm_count, void* stream) {
    return launch(a, true, max_sms, sm_count, stream);
}

int launch_w4_dequantize(const W4RowsArgs& a, int max_sms, int sm_count, void* stream) {
    return launch(a, false, max_sms, sm_count, stream);
}

}  // namespace tw
