// tkv8_plan_driver.cpp -- how the host half of libtkv (tkv_host.cpp, linked in
// directly) splits attention on a gfx950 of 256 compute units.  Reads lines of
// sizes and prints what the launcher is given.  The HIP calls and the launchers
// are the ones below.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstring>

#include "../tiled_tensor_bulk_amd/csrc/tkv_internal.h"

#undef hipGetDeviceProperties
extern "C" {
hipError_t hipGetDevice(int *dev) {
    *dev = 0;
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600 *p, int) {
    std::memset(p, 0, sizeof *p);
    std::strcpy(p->gcnArchName, "gfx950");
    p->multiProcessorCount = 256;
    return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "an error"; }
}

namespace tkv {
int launch_append(const MoveArgs &, void *) { return 0; }
int launch_read(const MoveArgs &, void *) { return 0; }
static int attended(const AttendArgs &a, int row_tile) {
    std::printf("%d %d %d %d %d %d\n", row_tile, a.row_blocks, a.n_split, 1 << a.chunk_shift, a.even, a.window);
    return 0;
}
int launch_attend_d64(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d96(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d128(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d256(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_weigh(const AttendArgs &, void *) { return 0; }
int launch_evict(const EvictArgs &, void *) { return 0; }
}  // namespace tkv

int main() {
    int bits, dim, heads, page, n_seq, q_heads, max_new, width, max_len, window, sinks;
    void *const at = (void *)(uintptr_t)(1 << 20);  // never read
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d", &bits, &dim, &heads, &page, &n_seq, &q_heads, &max_new, &width, &max_len,
                      &window, &sinks) == 11) {
        tkv_cache c;
        const tmap_status st = bits == 8 ? tkv_encode8(&c, at, 1 << 20, heads, dim, page) : tkv_encode(&c, at, 1 << 20, heads, dim, page, 32);
        tkv_batch b;
        std::memset(&b, 0, sizeof b);
        b.table = b.lens = b.starts = (const int32_t *)at;
        b.table_stride = b.table_width = width;
        b.n_seq = n_seq;
        b.max_new = max_new;
        b.n_tokens = (int64_t)n_seq * max_new;
        tkv_attend_args a;
        std::memset(&a, 0, sizeof a);
        a.q = a.out = {at, (int64_t)q_heads * dim, dim, TMAP_F16};
        a.lse = (float *)at;
        a.q_heads = q_heads;
        a.max_len = max_len;
        a.scale = 1.0f;
        a.causal = 1;
        a.workspace = at;
        a.workspace_bytes = ~0ull;
        const tkv_window w = {window, sinks};
        if (st != TMAP_SUCCESS || tkv_attend_window(&c, &a, window ? &w : nullptr, &b, nullptr) != TMAP_SUCCESS) {
            std::printf("refused: %s\n", tkv_last_error_detail());
            return 1;
        }
    }
    return 0;
}
