/* Which kernel does a call launch? This program stands in for the runtime's
 * launch (its definitions come before those of the libraries it loads), so that
 * calls on pointers that nobody reads end in a line of output: the kernel's
 * name, its workgroups and its threads. It needs no GPU.
 *
 * launch_probe LIBRARY < lines of numbers:
 *   M N K act out_dtype ldx ldw                          pw_linear_fp8
 *   M N K act out_dtype ldx ldw experts in_dtype gather  pw_grouped_linear */
#define _GNU_SOURCE
#include <dlfcn.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "pagedweight.h"

typedef struct {
    uint32_t x, y, z;
} dim3_t;

static const void* stubs[4096];
static const char* names[4096];
static int known;

void** __hipRegisterFatBinary(const void* data) {
    static void* handle;
    (void)data;
    return &handle;
}
void __hipUnregisterFatBinary(void** handle) { (void)handle; }
void __hipRegisterFunction(void** handle, const void* stub, char* device, const char* name, unsigned limit, void* a, void* b, void* c,
                           void* d, int* e) {
    (void)handle, (void)device, (void)limit, (void)a, (void)b, (void)c, (void)d, (void)e;
    if (known < 4096) {
        stubs[known] = stub;
        names[known++] = name;
    }
}

static dim3_t grid, block;
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t lds, void* stream) {
    (void)lds, (void)stream;
    grid = g;
    block = b;
    return 0;
}
int __hipPopCallConfiguration(dim3_t* g, dim3_t* b, size_t* lds, void** stream) {
    *g = grid;
    *b = block;
    *lds = 0;
    *stream = NULL;
    return 0;
}
int hipLaunchKernel(const void* stub, dim3_t g, dim3_t b, void** args, size_t lds, void* stream) {
    (void)args, (void)lds, (void)stream;
    for (int i = 0; i < known; ++i)
        if (stubs[i] == stub) printf("%s %ux%u %u\n", names[i], g.x, g.y, b.x);
    return 0;
}
int hipGetLastError(void) { return 0; }

int main(int argc, char** argv) {
    void* lib = argc == 2 ? dlopen(argv[1], RTLD_NOW) : NULL;
    if (!lib) {
        fprintf(stderr, "%s\n", argc == 2 ? dlerror() : "one library");
        return 2;
    }
    __typeof__(&pw_linear_fp8) dense = (__typeof__(&pw_linear_fp8))dlsym(lib, "pw_linear_fp8");
    __typeof__(&pw_grouped_linear) grouped = (__typeof__(&pw_grouped_linear))dlsym(lib, "pw_grouped_linear");
    for (int i = 0; i < known; ++i) printf("has %s\n", names[i]);
    char line[256];
    void* at = (void*)(uintptr_t)(1 << 20);
    while (fgets(line, sizeof line, stdin)) {
        int M, N, K, act, out, E, in, gather;
        long long ldx, ldw;
        const int n = sscanf(line, "%d %d %d %d %d %lld %lld %d %d %d", &M, &N, &K, &act, &out, &ldx, &ldw, &E, &in, &gather);
        const int64_t halves = act == PW_ACT_SWIGLU ? 2 : 1, blocks = (K + 127) / 128, tiles = halves * (((int64_t)N + 127) / 128);
        int status;
        if (n == 7) {
            const pw_linear_fp8_desc d = {M, N, K, out, act, ldx, ldw, N, N, 1, M, blocks, 1};
            status = dense(&d, at, at, at, at, NULL, NULL, at, NULL);
        } else {
            const int eight = in == PW_E4M3;
            const pw_grouped_desc d = {M, N, K, E, M, in, out, act, ldx, ldw, halves * N * ldw, N, N, 1, M, blocks, 1, tiles * blocks};
            status = grouped(&d, at, eight ? at : NULL, at, eight ? at : NULL, at, gather ? at : NULL, NULL, NULL, at, NULL);
        }
        if (status != 0) printf("refused %d\n", status);
    }
    return 0;
}
