/* One compaction after another, as a host thread of a C program would call them: no
 * interpreter between the calls.  `call` is pa_device_compact_blocks.  Returns the first
 * error, or PA_OK after n calls. */
#include "pagedattn.h"

typedef int (*compact_fn)(pa_pool*, const void*, const int*, const int*, int, const int*, int, void*, int*,
                          int*, int*, void*, size_t, pa_stream_t);

int compact_loop(compact_fn call, int n, pa_pool* pool, const void* stack, const int* tables, const int* lens,
                 void* out_stack, int* out_tables, int* remap, void* ws, size_t ws_bytes, pa_stream_t stream) {
    for (int i = 0; i < n; ++i) {
        const int rc = call(pool, stack, 0, tables, 1, lens, 1, out_stack, 0, out_tables, remap, ws, ws_bytes,
                            stream);
        if (rc != PA_OK) return rc;
    }
    return PA_OK;
}
