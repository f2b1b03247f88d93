// tw_device.cuh -- device helpers for the sm_103a kernels: mbarrier and
// bulk-async-copy PTX, L2 cache policies, bounded waits, bf16/fp32 vector
// packing.  Everything here is written from the public PTX ISA description.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tw_internal.h"

namespace tw {

// ---------------------------------------------------------------- timers ---
__device__ __forceinline__ uint64_t global_timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t sm_id() {
    uint32_t id;
    asm volatile("mov.u32 %0, %%smid;" : "=r"(id));
    return id;
}

// Every wait on an mbarrier gives up after this long; a healthy pipeline
// stage completes in microseconds.
constexpr uint64_t kWaitLimitNs = 1000ull * 1000ull * 1000ull;  // 1 s

// ------------------------------------------------------------- mbarrier ---
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count)
                 : "memory");
}

// Make barrier initialisation visible to the async (bulk copy) proxy.
__device__ __forceinline__ void mbar_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Wait for the phase with the given parity to complete.  Returns false when
// the CTA is aborting (abort non-NULL and set by another thread) or after
// kWaitLimitNs.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity,
                                          const volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t start = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (abort && *abort) return false;
        if (global_timer_ns() - start > kWaitLimitNs) return false;
    }
}

// One acquire read of a readiness flag: has *flag reached `epoch` (compared
// wrap-safe as a signed difference)?
__device__ __forceinline__ bool flag_is_ready(const unsigned int* flag, unsigned int epoch) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    return static_cast<int>(v - epoch) >= 0;
}

// Wait until *flag has reached `epoch` (compared wrap-safe as a signed
// difference), reading with acquire semantics at GPU scope, then order the
// async proxy (bulk copies) after it.  Returns false after kWaitLimitNs or
// when the CTA is aborting.
__device__ __forceinline__ bool flag_wait(const unsigned int* flag, unsigned int epoch,
                                          const volatile int* abort) {
    const uint64_t start = global_timer_ns();
    while (true) {
        unsigned int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (static_cast<int>(v - epoch) >= 0) {
            asm volatile("fence.proxy.async.global;" ::: "memory");
            return true;
        }
        if (abort && *abort) return false;
        if (global_timer_ns() - start > kWaitLimitNs) return false;
        __nanosleep(256);
    }
}

// ------------------------------------------------------ bulk async copy ---
__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// 1-D bulk copy global -> this CTA's shared memory, completion counted on
// `bar` as transaction bytes.  dst, src and bytes must be multiples of 16.
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes,
                                         uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// Programmatic dependent launch.  wait: block until the grids this launch
// depends on have completed and their memory is visible (a no-op when the
// launch had no programmatic dependency).  launch_dependents: allow the next
// grid of the stream to begin launching.
__device__ __forceinline__ void grid_dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Warm L2 with `bytes` bytes at `src` (a bulk prefetch: no data returns to
// the SM, nothing waits on it).  src and bytes must be multiples of 16.
__device__ __forceinline__ void bulk_prefetch_l2(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// Named barrier over `threads` threads (a multiple of 32), id != 0.
__device__ __forceinline__ void named_barrier(uint32_t id, uint32_t threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Named barrier that also returns the OR of `pred` over the `threads`
// participating threads (the same value in all of them).
__device__ __forceinline__ bool named_barrier_or(uint32_t id, uint32_t threads, bool pred) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(threads)
        : "memory");
    return any != 0;
}

// ---------------------------------------------------- 16-byte vectors ---
// A 16-byte vector holds 8 bf16 or 4 fp32 elements.
template <typename T>
struct Vec;

template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kElems = 8;
    __device__ __forceinline__ static void to_float(const uint4& v, float* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static uint4 from_float(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Vec<float> {
    static constexpr int kElems = 4;
    __device__ __forceinline__ static void to_float(const uint4& v, float* f) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ static uint4 from_float(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                          __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// acc[e] += element e of the 16-byte vector v, in fp32 with one rounding per
// add (the same bits as widening the element and adding).  bf16 elements go
// through the mixed-precision add (the bf16 operand is widened exactly);
// fp32 pairs through the packed two-lane add.
__device__ __forceinline__ void add_vec(float (&acc)[8], const uint4& v, __nv_bfloat16*) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "add.rn.f32.bf16 %0, lo, %0;\n\t"
            "add.rn.f32.bf16 %1, hi, %1;\n\t}"
            : "+f"(acc[2 * i]), "+f"(acc[2 * i + 1])
            : "r"(w[i]));
}
__device__ __forceinline__ void add_vec(float (&acc)[4], const uint4& v, float*) {
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%6, %7};\n\t"
        "add.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%2, %3}, a;\n\t}"
        : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
        : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
}

// ss2 += x * x on two lanes at a time (packed fp32 FMA); the caller adds the
// two lanes at the end.
template <int E>
__device__ __forceinline__ void sum_squares(float (&ss2)[2], const float (&x)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 2)
        asm("{\n\t.reg .b64 a, s;\n\t"
            "mov.b64 a, {%2, %3};\n\t"
            "mov.b64 s, {%0, %1};\n\t"
            "fma.rn.f32x2 s, a, a, s;\n\t"
            "mov.b64 {%0, %1}, s;\n\t}"
            : "+f"(ss2[0]), "+f"(ss2[1])
            : "f"(x[e]), "f"(x[e + 1]));
}

// ------------------------------------------------------ 8-bit outputs ---
// A row v quantised to 8 bits with one scale: scale = max|v| / top and
// q = rne(v * top / max|v|), top = 127 (int8) or 448 (e4m3).  The norm multiplies
// by a rounded top / max|v| (RowQuant), row quantisation by one of 44 bits (RowExact).
// Rows whose largest magnitude is below kQuantTiny (their scale would be a
// subnormal and lose bits) count as zero rows: scale 0, values 0.  A row that holds
// a NaN or an infinity has no scale: scale NaN, values 0.
constexpr float kQuantTiny = 0x1p-117f;

__device__ __forceinline__ float quant_top(int qtype) { return qtype == TW_INT8 ? 127.f : 448.f; }

// max(m, |v|), NaN if either is.
__device__ __forceinline__ float max_abs(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

// max(|m|, |a|, |b|), NaN if any is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

// Largest of the warp's non-negative floats (NaN if any is): the bits of
// non-negative floats order as unsigned integers, NaN above infinity.
__device__ __forceinline__ float warp_max_abs(float m) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

__device__ __forceinline__ bool quant_finite(float m) {
    return m <= 3.402823466e38f;  // false for NaN too
}

// Four values times mul, rounded to nearest even, as four int8 (|v * mul| is
// at most 127 and a few ulps).  Adding 1.5 * 2^23 leaves the rounded integer
// in the low bits of the sum's mantissa, its low byte being the int8.
__device__ __forceinline__ uint32_t pack_int8(const float* v, float mul) {
    uint32_t b[4];
    asm("{\n\t.reg .b64 a, s, c;\n\t"
        "mov.b64 s, {%8, %8};\n\t"
        "mov.b64 c, {%9, %9};\n\t"
        "mov.b64 a, {%4, %5};\n\t"
        "fma.rn.f32x2 a, a, s, c;\n\t"
        "mov.b64 {%0, %1}, a;\n\t"
        "mov.b64 a, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, s, c;\n\t"
        "mov.b64 {%2, %3}, a;\n\t}"
        : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(mul), "f"(12582912.f));
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// Four values as four e4m3 (nearest even, saturating at 448).
__device__ __forceinline__ uint32_t pack_e4m3(float v0, float v1, float v2, float v3) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
    return r;
}

// The scale of a row whose largest magnitude is m: m / top, the division's result
// by Markstein's quotient (IBM J. Res. Dev. 34, 1990): p = rn(m c) with c = rn(1 /
// top), then rn(p + (m - p top) c), the remainder being exact in a fused multiply-add
// (equal to m / top for every fp32 m from kQuantTiny up).
__device__ __forceinline__ float row_scale(float m, float top, bool zero) {
    const float c = top == 127.f ? 1.f / 127.f : 1.f / 448.f;
    const float p = m * c;
    const float s = fmaf(fmaf(-p, top, m), c, p);
    return !quant_finite(m) ? __uint_as_float(0x7fffffffu) : zero ? 0.f : s;
}

// How the norm quantises a row y = gain * v, m = max|v| (NaN or infinite where the
// row holds one), gain = 1 / rms: the gain cancels out of q = rne(v * mul), mul = top
// / m, and no element pays a division.  Whether the row is a zero row or holds an
// infinity goes by max|y| = m * gain (a sum of squares that leaves fp32 makes the
// gain 0 or infinite); by m as well where the row is that small before the gain.  A
// quotient within two ulp of the middle of two codes may go to either.  The
// reciprocal is an approximate one, off by at most an ulp; of m / 4, so that it is a
// normal number for every m from kQuantTiny up (2 x 2048 x 4096 13.1 us, with a
// division in every thread 2 % more).  The norm's fp32 values seldom lie in the very
// middle of two 8-bit ones.
struct RowQuant {
    float mul;  // top / max|v|
    float y;    // max|y|
    bool zero;  // every value of the row is 0, whatever mul makes of it

    RowQuant() = default;
    __device__ __forceinline__ RowQuant(float m, float gain, float top) {
        y = m * gain;
        zero = !(fminf(m, y) >= kQuantTiny && quant_finite(y));
        float inverse;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inverse) : "f"(m * 0.25f));
        mul = (top * 0.25f) * inverse;
    }
    __device__ __forceinline__ uint32_t codes(const float* v, int qtype) const {
        return qtype == TW_INT8
                   ? pack_int8(v, mul)
                   : pack_e4m3(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul);
    }
};

// How row quantisation does it: q = rne(rn(v * top / m)), the quotient as good as
// exact before it is rounded to fp32.  bf16 rows hold many values in the very middle
// of two codes: multiplied by a rounded top / m, or divided by a rounded scale, they go
// to the side that its rounding points to, a whole row's to the same (of the codes of
// 1024 x 8192 normal values 0.055 % in int8 and 0.08 % in e4m3 are then off the
// definition's, by a division 0.003 % and 0.016 %).
//   top / m is kept to 44 bits as hi + lo: hi = rn(top r) with r an approximate
// reciprocal of m, lo the rest, rn((top - m hi) r), all of m / 4 and top / 4, so that r
// is a normal number for every m from kQuantTiny up.  rn(v hi + rn(v lo)) is right
// wherever v * top / m is an fp32 number, the middle of two codes in particular, and
// elsewhere rounds what is off by 2^-44 (rows above 2^100, whose lo is a subnormal:
// 2^-28).  So every code of bf16 rows is the definition's (checked for all mantissas and
// exponents), and of fp32 rows where the quotient is not within half an ulp of a
// middle.  Two packed operations for two elements: 4096 x 8192 16.15 us, as with one
// multiplication.
struct RowExact {
    float hi, lo;
    bool zero;  // every value of the row is 0

    __device__ __forceinline__ RowExact(float m, float top) {
        zero = !quant_finite(m) || m < kQuantTiny;
        m *= 0.25f;
        top *= 0.25f;
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(m));
        hi = top * r;
        lo = fmaf(-m, hi, top) * r;
    }
    // q[0..1] = v[0..1] * top / m.
    __device__ __forceinline__ void quotients(float* q, const float* v) const {
        asm("{\n\t.reg .b64 a, p, h, l;\n\t"
            "mov.b64 a, {%2, %3};\n\t"
            "mov.b64 h, {%4, %4};\n\t"
            "mov.b64 l, {%5, %5};\n\t"
            "mul.rn.f32x2 p, a, l;\n\t"
            "fma.rn.f32x2 p, a, h, p;\n\t"
            "mov.b64 {%0, %1}, p;\n\t}"
            : "=f"(q[0]), "=f"(q[1])
            : "f"(v[0]), "f"(v[1]), "f"(hi), "f"(lo));
    }
    __device__ __forceinline__ uint32_t codes(const float* v, int qtype) const {
        float q[4];
        quotients(q, v);
        quotients(q + 2, v + 2);
        return qtype == TW_INT8 ? pack_int8(q, 1.f) : pack_e4m3(q[0], q[1], q[2], q[3]);
    }
};

// max(|m|, |v|) over one vector's elements, NaN if any is.  bf16: two maxima side by
// side in the halves of m (signs are of no meaning), without widening; max_abs_of
// joins them.
__device__ __forceinline__ void max_abs_vec(uint32_t& m, const uint4& v, __nv_bfloat16*) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
}
__device__ __forceinline__ void max_abs_vec(uint32_t& m, const uint4& v, float*) {
    const float a = max_abs(__uint_as_float(m), __uint_as_float(v.x), __uint_as_float(v.y));
    m = __float_as_uint(max_abs(a, __uint_as_float(v.z), __uint_as_float(v.w)));
}
__device__ __forceinline__ float max_abs_of(uint32_t m, __nv_bfloat16*) {
    return max_abs(0.f, __uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}
__device__ __forceinline__ float max_abs_of(uint32_t m, float*) { return __uint_as_float(m); }

// The E elements (8 or 4) of one 16-byte vector's worth of a row, quantised
// and stored at p (E bytes, E-byte aligned) in each of n destinations.
template <int E, class Row>
__device__ __forceinline__ void store_q8(void* const* out, int n, int64_t off, const float* v,
                                         const Row& q, int qtype) {
    uint32_t b[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        b[i] = q.codes(v + 4 * i, qtype);
        if (q.zero) b[i] = 0;
    }
    for (int k = 0; k < n; ++k) {
        char* p = static_cast<char*>(out[k]) + off;
        if constexpr (E == 8)
            __stcs(reinterpret_cast<uint2*>(p), make_uint2(b[0], b[1]));
        else
            __stcs(reinterpret_cast<unsigned int*>(p), b[0]);
    }
}

// y[0..1] = a[0..1] * b[0..1], two lanes per instruction.
__device__ __forceinline__ void mul2(float* y, const float* a, const float* b) {
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(y[0]), "=f"(y[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}

// max(m, |x * w|) over one vector's elements (NaN if any product is).
template <typename T>
__device__ __forceinline__ float max_abs_product(float m, const float* x, const uint4& wv) {
    constexpr int E = Vec<T>::kElems;
    float w[E], v[E];
    Vec<T>::to_float(wv, w);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        mul2(v + e, x + e, w + e);
        m = max_abs(m, v[e], v[e + 1]);
    }
    return m;
}

// Streaming 16-byte global store (written once, not re-read by this kernel).
__device__ __forceinline__ void st_global_cs(void* p, const uint4& v) {
    __stcs(reinterpret_cast<uint4*>(p), v);
}

// Read-only 16-byte global load that does not allocate in L1.  Volatile so
// the compiler never hoists it out of the bounds check that guards it.
__device__ __forceinline__ uint4 ld_global_nc(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Coherent 16-byte global load (used where the buffer may also be written by
// this kernel, e.g. a residual updated in place).
__device__ __forceinline__ uint4 ld_global(const void* p) {
    return *reinterpret_cast<const uint4*>(p);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Host side: launch fn(p) with the given shape, optionally with programmatic
// stream serialization (see grid_dependency_wait).  Returns a cudaError_t.
template <typename P>
inline int launch_with_pdl(void* fn, const P& p, int grid, int block, size_t smem_bytes,
                           bool pdl, void* stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem_bytes;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    void* args[] = {const_cast<P*>(&p)};
    return static_cast<int>(cudaLaunchKernelExC(&cfg, fn, args));
}

}  // namespace tw
