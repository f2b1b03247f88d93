// tw_q8.cu -- entry points of the 8-bit operators beside the fused step: row
// quantisation and the matrix product.  Every rule stated in tw.h is checked
// here on the host before the first CUDA call.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "tw.h"
#include "tw_internal.h"

namespace tw {
namespace {

int refuse(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_last_error(code, buf);
}

int launch_status(int err, const char* what) {
    if (err == cudaSuccess) return TW_OK;
    const cudaError_t e = static_cast<cudaError_t>(err);
    return refuse(TW_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// An operator whose kernels could not be set up on this device.
int check_set_up(int err, const char* what) {
    if (err == cudaSuccess) return TW_OK;
    return refuse(TW_ERR_UNSUPPORTED, "%s unavailable on this device (%s)", what,
                  cudaGetErrorName(static_cast<cudaError_t>(err)));
}

bool misaligned(const void* p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return na != 0 && nb != 0 && a0 < b0 + nb && b0 < a0 + na;
}

// The rules common to both entry points.
int check_common(int64_t T, int64_t t0, int64_t t1, int max_sms, int dtype, int qtype) {
    if (dtype != TW_BF16 && dtype != TW_F32)
        return refuse(TW_ERR_INVALID_ARG, "dtype %d is not TW_BF16 or TW_F32", dtype);
    if (qtype != TW_INT8 && qtype != TW_E4M3)
        return refuse(TW_ERR_INVALID_ARG, "qtype %d is not TW_INT8 or TW_E4M3", qtype);
    if (T < 0) return refuse(TW_ERR_INVALID_ARG, "T %lld < 0", (long long)T);
    if (t0 < 0 || t0 > t1 || t1 > T)
        return refuse(TW_ERR_INVALID_ARG, "token range [%lld, %lld) not within [0, %lld]",
                      (long long)t0, (long long)t1, (long long)T);
    if (max_sms < 1) return refuse(TW_ERR_INVALID_ARG, "max_sms %d < 1", max_sms);
    return TW_OK;
}

}  // namespace
}  // namespace tw

using tw::refuse;

extern "C" int tw_quantize_rows_q8(const void* x, void* out, float* out_scale, int64_t T,
                                   int64_t H, int64_t t0, int64_t t1, int max_sms, void* stream,
                                   int dtype, int qtype) {
    int rc = tw::check_common(T, t0, t1, max_sms, dtype, qtype);
    if (rc != TW_OK) return rc;
    if (!x || !out || !out_scale) return refuse(TW_ERR_INVALID_ARG, "NULL pointer argument");
    if (H < 1) return refuse(TW_ERR_INVALID_ARG, "H %lld < 1", (long long)H);
    const int64_t max_h = dtype == TW_BF16 ? TW_MAX_H_BF16 : TW_MAX_H_F32;
    if (H > max_h)
        return refuse(TW_ERR_UNSUPPORTED, "H %lld above the limit %lld for this dtype",
                      (long long)H, (long long)max_h);
    const int64_t es = dtype == TW_BF16 ? 2 : 4;
    if (T > (int64_t{1} << 48) / (H * es))
        return refuse(TW_ERR_INVALID_ARG, "T %lld x H %lld buffers exceed 2^48 bytes",
                      (long long)T, (long long)H);
    if ((H * es) % 16 != 0)
        return refuse(TW_ERR_ALIGNMENT, "H * element size (%lld bytes) is not a multiple of 16",
                      (long long)(H * es));
    if (tw::misaligned(x, 16) || tw::misaligned(out, 16))
        return refuse(TW_ERR_ALIGNMENT, "x and out must be 16-byte aligned");
    if (tw::misaligned(out_scale, 4))
        return refuse(TW_ERR_ALIGNMENT, "out_scale must be 4-byte aligned");
    const uint64_t n = static_cast<uint64_t>(T) * H, sb = static_cast<uint64_t>(T) * 4;
    if (tw::overlaps(x, n * es, out, n) || tw::overlaps(x, n * es, out_scale, sb) ||
        tw::overlaps(out, n, out_scale, sb))
        return refuse(TW_ERR_ALIAS, "x, out and out_scale overlap");
    if (t0 == t1) return TW_OK;
    tw::DeviceInfo d;
    if ((rc = tw::device_info(&d)) != TW_OK ||
        (rc = tw::check_set_up(d.quantize_error, "row quantisation")) != TW_OK)
        return rc;
    const tw::QuantParams p{x, out, out_scale, t0, t1, H, H * es, qtype};
    return tw::launch_status(tw::launch_quantize(p, dtype, max_sms, d.sm_count, stream),
                             "quantize_rows launch");
}

extern "C" int tw_gemm_q8(const void* x, const float* x_scale, const void* w,
                          const float* w_scale, void* out, int64_t T, int64_t N, int64_t K,
                          int64_t t0, int64_t t1, int max_sms, void* stream, int dtype,
                          int qtype) {
    int rc = tw::check_common(T, t0, t1, max_sms, dtype, qtype);
    if (rc != TW_OK) return rc;
    if (!x || !x_scale || !w || !w_scale || !out)
        return refuse(TW_ERR_INVALID_ARG, "NULL pointer argument");
    constexpr int64_t kMax = (int64_t{1} << 31) - 512;  // a tile beyond fits 32 bits
    if (T > kMax || N < 1 || N > kMax)
        return refuse(TW_ERR_INVALID_ARG, "T %lld and N %lld must be at most 2^31 - 512, N >= 1",
                      (long long)T, (long long)N);
    if (K < 1) return refuse(TW_ERR_INVALID_ARG, "K %lld < 1", (long long)K);
    if (K > TW_MAX_K_Q8)
        return refuse(TW_ERR_UNSUPPORTED, "K %lld above the limit %d", (long long)K, TW_MAX_K_Q8);
    if (K % 16 != 0)
        return refuse(TW_ERR_ALIGNMENT, "K %lld is not a multiple of 16", (long long)K);
    const int64_t es = dtype == TW_BF16 ? 2 : 4;
    if (T > (int64_t{1} << 48) / (N * es))
        return refuse(TW_ERR_INVALID_ARG, "T %lld x N %lld buffers exceed 2^48 bytes",
                      (long long)T, (long long)N);
    if (tw::misaligned(x, 16) || tw::misaligned(w, 16) || tw::misaligned(out, 16))
        return refuse(TW_ERR_ALIGNMENT, "x, w and out must be 16-byte aligned");
    if (tw::misaligned(x_scale, 4) || tw::misaligned(w_scale, 4))
        return refuse(TW_ERR_ALIGNMENT, "x_scale and w_scale must be 4-byte aligned");
    const uint64_t ob = static_cast<uint64_t>(T) * N * es;
    if (tw::overlaps(out, ob, x, static_cast<uint64_t>(T) * K) ||
        tw::overlaps(out, ob, w, static_cast<uint64_t>(N) * K) ||
        tw::overlaps(out, ob, x_scale, static_cast<uint64_t>(T) * 4) ||
        tw::overlaps(out, ob, w_scale, static_cast<uint64_t>(N) * 4))
        return refuse(TW_ERR_ALIAS, "out overlaps an input");
    if (t0 == t1) return TW_OK;
    tw::DeviceInfo d;
    const bool few = t1 - t0 <= tw::kGemvTokens;
    if ((rc = tw::device_info(&d)) != TW_OK ||
        (rc = tw::check_set_up(few ? d.gemv_error : d.gemm_error, "8-bit product")) != TW_OK)
        return rc;
    const tw::GemmArgs g{static_cast<const char*>(x) + t0 * K,
                         x_scale + t0,
                         w,
                         w_scale,
                         static_cast<char*>(out) + t0 * N * es,
                         t1 - t0,
                         N,
                         K,
                         dtype,
                         qtype};
    const int err = few ? tw::launch_gemv(g, max_sms, d, stream)
                        : tw::launch_gemm(g, max_sms, d, stream);
    return tw::launch_status(err, "gemm_q8 launch");
}
