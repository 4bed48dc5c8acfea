/*
 * Records the launches of the quantiser's entry points: this program has its own
 * launch functions, which libep.so's calls reach, so nothing runs and no device is
 * needed.  Built and run by tests/test_launch_sizes.py.
 *
 * launch_sizes rows ROWS CHANNELS
 * launch_sizes slots TOKENS TOPK CHANNELS
 *   prints the entry's status, then of every launch: blocks, threads of a block, first
 *   row (the kernel's second argument).
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "ep_expert.h"

/* Where <<< >>> leaves a launch's sizes for the kernel's host function. */
static struct {
    dim3 grid, block;
    size_t lds;
    hipStream_t stream;
} at;

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
    (void)kernel, (void)lds, (void)stream;
    int64_t first;
    memcpy(&first, args[1], sizeof(first));
    printf("%llu %llu %lld\n", (unsigned long long)grid.x * grid.y * grid.z,
           (unsigned long long)block.x * block.y * block.z, (long long)first);
    return hipSuccess;
}

hipError_t hipGetLastError(void) { return hipSuccess; }

int main(int argc, char **argv) {
    /* places further apart than any of the sizes reach; never read or written */
    void *x = (void *)((uintptr_t)1 << 44), *q = (void *)((uintptr_t)1 << 45);
    float *scale = (float *)((uintptr_t)1 << 46);
    if (argc == 4 && !strcmp(argv[1], "rows")) {
        printf("%d\n", ep_quantize_i8(x, atoi(argv[2]), atoi(argv[3]), q, scale, NULL));
        return 0;
    }
    if (argc == 5 && !strcmp(argv[1], "slots")) {
        static int32_t some[16];
        static uint64_t status[1];
        ep_handle h;
        memset(&h, 0, sizeof(h));
        h.max_tokens = h.num_tokens = atoi(argv[2]);
        h.num_topk = atoi(argv[3]);
        h.num_experts = 4;
        h.expert_alignment = h.laid_out = h.status_tiles = 1;
        h.capacity = 64;
        h.counts = h.psum = h.dst_slot = h.src_meta = h.scalars = some;
        h.recv_row = h.recv_src = some;
        h.tile_status = status;
        printf("%d\n", ep_quantize_i8_rows(&h, x, atoi(argv[4]), q, scale, NULL));
        return 0;
    }
    fprintf(stderr, "usage: launch_sizes rows ROWS CHANNELS | slots TOKENS TOPK CHANNELS\n");
    return 2;
}
