/* A stand-in for the CUDA runtime calls of libtw.so, for tests without a GPU:
 * preloaded into a child process, it reports a device, notes which kernels are
 * launched and lets the set-up of those named in FAKE_FAIL fail. */
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

enum { kMaxKernels = 4096, kInvalidValue = 1, kSymbolNotFound = 500 };
static const void* kernel[kMaxKernels];
static const char* kernel_name[kMaxKernels];
static int n_kernels;
static char word[1 << 20];

/* Every kernel's host handle and mangled name pass through here at load. */
void __cudaRegisterFunction(void** handle, const char* host, char* device, const char* name,
                            int threads, void* tid, void* bid, void* block, void* grid, int* w) {
    (void)handle, (void)device, (void)threads, (void)tid, (void)bid, (void)block, (void)grid, (void)w;
    if (n_kernels < kMaxKernels) {
        kernel[n_kernels] = host;
        kernel_name[n_kernels++] = name;
    }
}
static const char* name_of(const void* fn) {
    for (int i = 0; i < n_kernels; ++i)
        if (kernel[i] == fn) return kernel_name[i];
    return "unknown";
}
static int fails(const char* name) {
    const char* f = getenv("FAKE_FAIL");
    return f && *f && strstr(name, f) != NULL;
}

int cudaGetDevice(int* d) { return *d = 0; }
int cudaDeviceGetAttribute(int* v, int attr, int device) {
    (void)device;
    switch (attr) {
        case 75: *v = 10; break;      /* compute capability, major */
        case 16: *v = 152; break;     /* multiprocessors */
        case 97: *v = 232448; break;  /* shared memory per block, opt-in */
        default: return kInvalidValue;
    }
    return 0;
}
int cudaFuncSetAttribute(const void* fn, int attr, int value) {
    (void)attr, (void)value;
    return fails(name_of(fn)) ? kInvalidValue : 0;
}
int cudaFuncGetAttributes(void* attr, const void* fn) {
    (void)attr, (void)fn;
    return 0;
}
int cudaOccupancyMaxActiveClusters(int* n, const void* fn, const void* config) {
    (void)fn, (void)config;
    *n = 16;
    return 0;
}
int cudaGetSymbolAddress(void** p, const void* symbol) {
    (void)symbol;
    *p = word;
    return 0;
}
int cudaEventCreateWithFlags(void** e, unsigned flags) {
    (void)flags;
    *e = word;
    return 0;
}
int cudaEventRecord(void* e, void* stream) {
    (void)e, (void)stream;
    return 0;
}
int cudaEventQuery(void* e) {
    (void)e;
    return 0;
}
int cudaStreamIsCapturing(void* stream, int* status) {
    (void)stream;
    return *status = 0;
}
static int encode(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char* symbol, void** fn, unsigned version,
                                     unsigned long long flags, int* found) {
    (void)version, (void)flags;
    *found = fails(symbol);
    *fn = *found ? NULL : (void*)encode;
    return 0;
}
int cudaLaunchKernelExC(const void* config, const void* fn, void** args) {
    (void)config, (void)args;
    printf("launch %s\n", name_of(fn));
    fflush(stdout);
    return 0;
}
int cudaGetLastError(void) { return 0; }
