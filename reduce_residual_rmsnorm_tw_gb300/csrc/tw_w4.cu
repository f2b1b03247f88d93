// tw_w4.cu -- entry points of the operators on 4-bit weights.  Every rule
// stated in tw.h is checked here on the host before the first CUDA call.
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

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 512;  // a tile beyond fits 32 bits

// The weights' shape, and their packed bytes (at most 2^47: no overflow).
int check_shape(int64_t N, int64_t K, int group, uint64_t* bytes) {
    if (N < 1 || N > kMaxRows)
        return refuse(TW_ERR_INVALID_ARG, "N %lld outside [1, 2^31 - 512]", (long long)N);
    if (K < 1) return refuse(TW_ERR_INVALID_ARG, "K %lld < 1", (long long)K);
    if (K > TW_MAX_K_Q8)
        return refuse(TW_ERR_UNSUPPORTED, "K %lld above the limit %d", (long long)K, TW_MAX_K_Q8);
    if (K % 16 != 0)
        return refuse(TW_ERR_ALIGNMENT, "K %lld is not a multiple of 16", (long long)K);
    if (group != 32 && group != 64 && group != 128)
        return refuse(TW_ERR_INVALID_ARG, "group %d is not 32, 64 or 128", group);
    *bytes = static_cast<uint64_t>((N + kW4Channels - 1) / kW4Channels) *
             ((K + kW4Inner - 1) / kW4Inner) * w4_tile_bytes(group);
    return TW_OK;
}

int check_types(int max_sms, int dtype, int wtype) {
    if (dtype != TW_BF16 && dtype != TW_F32)
        return refuse(TW_ERR_INVALID_ARG, "dtype %d is not TW_BF16 or TW_F32", dtype);
    if (wtype != TW_INT4 && wtype != TW_E2M1)
        return refuse(TW_ERR_INVALID_ARG, "wtype %d is not TW_INT4 or TW_E2M1", wtype);
    if (max_sms < 1) return refuse(TW_ERR_INVALID_ARG, "max_sms %d < 1", max_sms);
    return TW_OK;
}

// tw_quantize_w4 and tw_dequantize_w4: the same rules for the two tensors.
int rows_call(const void* from, void* to, const void* rows, const void* packed, int64_t N,
              int64_t K, int group, int max_sms, void* stream, int dtype, int wtype,
              bool quantize) {
    uint64_t bytes = 0;
    int rc = check_types(max_sms, dtype, wtype);
    if (rc != TW_OK || (rc = check_shape(N, K, group, &bytes)) != TW_OK) return rc;
    if (!rows || !packed) return refuse(TW_ERR_INVALID_ARG, "NULL pointer argument");
    if (misaligned(rows, 16) || misaligned(packed, 16))
        return refuse(TW_ERR_ALIGNMENT, "w and packed must be 16-byte aligned");
    if (overlaps(rows, static_cast<uint64_t>(N) * K * (dtype == TW_BF16 ? 2 : 4), packed, bytes))
        return refuse(TW_ERR_ALIAS, "w and packed overlap");
    DeviceInfo d;
    if ((rc = device_info(&d)) != TW_OK ||
        (rc = check_set_up(d.w4_rows_error, "4-bit weights")) != TW_OK)
        return rc;
    const W4RowsArgs a{from, to, N, K, group, dtype, wtype};
    return launch_status(quantize ? launch_w4_quantize(a, max_sms, d.sm_count, stream)
                                  : launch_w4_dequantize(a, max_sms, d.sm_count, stream),
                         quantize ? "quantize_w4 launch" : "dequantize_w4 launch");
}

}  // namespace
}  // namespace tw

using tw::refuse;

extern "C" int tw_w4_bytes(int64_t N, int64_t K, int group, size_t* bytes) {
    if (!bytes) return refuse(TW_ERR_INVALID_ARG, "NULL pointer argument");
    uint64_t n = 0;
    const int rc = tw::check_shape(N, K, group, &n);
    if (rc == TW_OK) *bytes = n;
    return rc;
}

extern "C" int tw_quantize_w4(const void* w, void* packed, int64_t N, int64_t K, int group,
                              int max_sms, void* stream, int dtype, int wtype) {
    return tw::rows_call(w, packed, w, packed, N, K, group, max_sms, stream, dtype, wtype, true);
}

extern "C" int tw_dequantize_w4(const void* packed, void* w, int64_t N, int64_t K, int group,
                                int max_sms, void* stream, int dtype, int wtype) {
    return tw::rows_call(packed, w, w, packed, N, K, group, max_sms, stream, dtype, wtype, false);
}

extern "C" int tw_gemm_w4(const void* x, const float* x_scale, const void* packed, void* out,
                          int64_t T, int64_t N, int64_t K, int group, int64_t t0, int64_t t1,
                          int max_sms, void* stream, int xtype, int dtype, int wtype) {
    uint64_t bytes = 0;
    int rc = tw::check_types(max_sms, dtype, wtype);
    if (rc != TW_OK || (rc = tw::check_shape(N, K, group, &bytes)) != TW_OK) return rc;
    if (xtype < TW_X_BF16 || xtype > TW_X_E4M3)
        return refuse(TW_ERR_INVALID_ARG, "xtype %d is not a tw_xtype", xtype);
    const bool scaled = xtype == TW_X_INT8 || xtype == TW_X_E4M3;
    if (!x || !packed || !out || (scaled && !x_scale))
        return refuse(TW_ERR_INVALID_ARG, "NULL pointer argument");
    if (!scaled && x_scale)
        return refuse(TW_ERR_INVALID_ARG, "x_scale goes with 8-bit x only");
    if (T < 0 || T > tw::kMaxRows)
        return refuse(TW_ERR_INVALID_ARG, "T %lld outside [0, 2^31 - 512]", (long long)T);
    if (t0 < 0 || t0 > t1 || t1 > T)
        return refuse(TW_ERR_INVALID_ARG, "token range [%lld, %lld) not within [0, %lld]",
                      (long long)t0, (long long)t1, (long long)T);
    const int64_t es = dtype == TW_BF16 ? 2 : 4;
    if (T > (int64_t{1} << 48) / (N * es))
        return refuse(TW_ERR_INVALID_ARG, "T %lld x N %lld buffers exceed 2^48 bytes",
                      (long long)T, (long long)N);
    if (tw::misaligned(x, 16) || tw::misaligned(packed, 16) || tw::misaligned(out, 16))
        return refuse(TW_ERR_ALIGNMENT, "x, packed and out must be 16-byte aligned");
    if (tw::misaligned(x_scale, 4))
        return refuse(TW_ERR_ALIGNMENT, "x_scale must be 4-byte aligned");
    const int64_t xs = xtype == TW_X_BF16 ? 2 : xtype == TW_X_F32 ? 4 : 1;
    const uint64_t ob = static_cast<uint64_t>(T) * N * es;
    if (tw::overlaps(out, ob, x, static_cast<uint64_t>(T) * K * xs) ||
        tw::overlaps(out, ob, packed, bytes) ||
        (x_scale && tw::overlaps(out, ob, x_scale, static_cast<uint64_t>(T) * 4)))
        return refuse(TW_ERR_ALIAS, "out overlaps an input");
    if (t0 == t1) return TW_OK;
    tw::DeviceInfo d;
    if ((rc = tw::device_info(&d)) != TW_OK ||
        (rc = tw::check_set_up(d.w4_gemm_error, "4-bit product")) != TW_OK)
        return rc;
    const tw::W4GemmArgs a{static_cast<const char*>(x) + t0 * K * xs,
                           scaled ? x_scale + t0 : nullptr,
                           packed,
                           static_cast<char*>(out) + t0 * N * es,
                           t1 - t0,
                           N,
                           K,
                           group,
                           xtype,
                           dtype,
                           wtype};
    return tw::launch_status(tw::launch_w4_gemm(a, max_sms, d, stream),
                             "gemm_w4 launch");
}
