/* Stands in for the HIP runtime's launch calls, so that the launches of libengram.so can be looked at where there is no
 * GPU: loaded ahead of the runtime, it notes every launch's grid and block and runs nothing.  Like the runtime it refuses
 * 2^32 threads or more along an axis; `fail_at` makes one launch (counted from 0) fail as well. */
#include <stddef.h>
#include <stdint.h>

typedef struct {
    uint32_t x, y, z;
} dim3_t;

enum { kMost = 4096, kInvalidConfiguration = 9, kLaunchFailure = 719 };

static dim3_t grids[kMost], blocks[kMost], next_grid, next_block;
static size_t next_shared;
static void* next_stream;
static int count, fail_at = -1, last_error;

void recorder_reset(int fail) {
    count = 0;
    fail_at = fail;
    last_error = 0;
}
int recorder_count(void) { return count; }
void recorder_get(int i, uint32_t* out) {
    const dim3_t g = grids[i], b = blocks[i];
    out[0] = g.x, out[1] = g.y, out[2] = g.z, out[3] = b.x, out[4] = b.y, out[5] = b.z;
}

int __hipPushCallConfiguration(dim3_t grid, dim3_t block, size_t shared, void* stream) {
    next_grid = grid, next_block = block, next_shared = shared, next_stream = stream;
    return 0;
}
int __hipPopCallConfiguration(dim3_t* grid, dim3_t* block, size_t* shared, void** stream) {
    *grid = next_grid, *block = next_block, *shared = next_shared, *stream = next_stream;
    return 0;
}
int hipLaunchKernel(const void* function, dim3_t grid, dim3_t block, void** args, size_t shared, void* stream) {
    (void)function, (void)args, (void)shared, (void)stream;
    const int at = count;
    if (at < kMost) {
        grids[at] = grid;
        blocks[at] = block;
        count = at + 1;
    }
    const uint64_t most = 1ull << 32;
    int error = 0;
    if (!grid.x || !grid.y || !grid.z || (uint64_t)grid.x * block.x >= most || (uint64_t)grid.y * block.y >= most ||
        (uint64_t)grid.z * block.z >= most)
        error = kInvalidConfiguration;
    if (at == fail_at) error = kLaunchFailure;
    if (error) last_error = error;
    return error;
}
int hipGetLastError(void) {
    const int e = last_error;
    last_error = 0;
    return e;
}
