/*
 * Says which kernels calls of the experts' products would launch: this program has its own
 * launch functions, which libep.so's calls reach, so nothing runs and no device is needed.
 * Built and run by tests/test_launched_kernels.py.
 *
 * Reads lines `op tokens topk experts token_rows k n gated fp32` (op 0: int8 product of k to n
 * channels; 1: the gated block of k channels and n between them, and its gradients) and prints
 * for every line the status, 0 if all is well, and the place of each launched kernel's symbol in
 * the library.
 */
#define _GNU_SOURCE
#include <dlfcn.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "ep_expert.h"

static struct {
    dim3 grid, block;
    size_t lds;
    hipStream_t stream;
} at;
static uintptr_t base;

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
    at.grid = grid, at.block = block, at.lds = lds, at.stream = stream;
    return hipSuccess;
}

hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, hipStream_t *stream) {
    *grid = at.grid, *block = at.block, *lds = at.lds, *stream = at.stream;
    return hipSuccess;
}

hipError_t hipLaunchKernel(const void *kernel, dim3 grid, dim3 block, void **args, size_t lds,
                           hipStream_t stream) {
    (void)args, (void)lds, (void)stream;
    if ((uint64_t)grid.x * grid.y * grid.z * block.x * block.y * block.z >> 32)
        return hipErrorInvalidConfiguration;
    printf(" %llx", (unsigned long long)((uintptr_t)kernel - base));
    return hipSuccess;
}

hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipFuncSetAttribute(const void *f, hipFuncAttribute a, int v) {
    (void)f, (void)a, (void)v;
    return hipSuccess;
}
hipError_t hipGetDevice(int *d) { return *d = 0, hipSuccess; }
hipError_t hipDeviceGetAttribute(int *v, hipDeviceAttribute_t a, int d) {
    (void)a, (void)d;
    return *v = 256, hipSuccess;
}

/* Places further apart than any of the sizes reach; never read or written. */
static void *place(int i) { return (void *)((uintptr_t)(i + 1) << 42); }

int main(void) {
    static int32_t some[16];
    static uint64_t status[1];
    Dl_info info;
    int op, tokens, topk, experts, own, k, n, gated, fp32;
    if (!dladdr((void *)ep_expert_ffn_backward, &info)) return 1;
    base = (uintptr_t)info.dli_fbase;
    while (scanf("%d %d %d %d %d %d %d %d %d", &op, &tokens, &topk, &experts, &own, &k, &n,
                 &gated, &fp32) == 9) {
        ep_handle h;
        ep_status s;
        memset(&h, 0, sizeof(h));
        h.max_tokens = h.num_tokens = tokens;
        h.num_topk = topk;
        h.num_experts = experts;
        h.expert_alignment = h.laid_out = h.status_tiles = 1;
        h.capacity = (int64_t)tokens * topk;
        h.counts = h.psum = h.dst_slot = h.src_meta = h.scalars = some;
        h.recv_row = h.recv_src = some;
        h.tile_status = status;
        if (op == 0) {
            s = ep_expert_i8(&h, place(0), place(1), own, k, place(2), place(3), n, gated, NULL,
                             place(4), NULL);
        } else {
            s = ep_expert_ffn(&h, place(0), own, k, place(1), place(2), n, NULL, place(3), place(4),
                              place(5), NULL);
            if (s == EP_OK)
                s = ep_expert_ffn_backward(&h, place(6), place(0), own, k, place(1), place(2), n,
                                           NULL, place(4), place(3), 0, place(7), place(8),
                                           fp32 ? EP_F32 : EP_BF16, place(9), place(10), place(11),
                                           place(12), (size_t)1 << 41, NULL);
        }
        printf(" %d\n", s);
    }
    return 0;
}
