/* The stand-in of fake_cudart.c that also notes which kernels set-up asks the runtime
 * for, and so loads: in full, a line each. */
#define cudaFuncSetAttribute quiet_cudaFuncSetAttribute
#define cudaFuncGetAttributes quiet_cudaFuncGetAttributes
#include "fake_cudart.c"
#undef cudaFuncSetAttribute
#undef cudaFuncGetAttributes

static void note(const void* fn) {
    printf("load %s\n", name_of(fn));
    fflush(stdout);
}
int cudaFuncSetAttribute(const void* fn, int attr, int value) {
    note(fn);
    return quiet_cudaFuncSetAttribute(fn, attr, value);
}
int cudaFuncGetAttributes(void* attr, const void* fn) {
    note(fn);
    return quiet_cudaFuncGetAttributes(attr, fn);
}
