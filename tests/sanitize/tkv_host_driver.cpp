// tkv_host_driver.cpp -- drives the host half of libtkv (tkv_host.cpp, linked
// in directly) under AddressSanitizer and UndefinedBehaviorSanitizer: the HIP
// calls that it makes and the kernel launchers are the ones below, which
// pretend a gfx950 device and look at what they would launch.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../tiled_tensor_bulk_amd/csrc/tkv_internal.h"

static int g_cus = 256;

#undef hipGetDeviceProperties
extern "C" {
hipError_t hipGetDevice(int *dev) {
    *dev = g_cus == 256 ? 0 : 1;  // what the library remembers of a device is its number of compute units
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600 *p, int) {
    std::memset(p, 0, sizeof *p);
    std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
    p->multiProcessorCount = g_cus;
    return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "an error"; }
}

static int bad = 0, accepted = 0, launches = 0;
static void expect(bool ok, const char *what) {
    if (!ok && bad++ < 20) std::fprintf(stderr, "unexpected: %s (%s)\n", what, tkv_last_error_detail());
}

// A kernel of so many threads for each of so many units of work, some of which a workgroup takes.
static void launch(const char *what, double units, int of_a_workgroup, int threads = 256) {
    ++launches;
    const double blocks = std::ceil(units / of_a_workgroup);
    expect(blocks >= 1 && blocks * threads < 4294967296.0, what);
}

namespace tkv {
static int moved(const MoveArgs &a, bool append) {
    launch("records of a move", (double)a.tiles * a.b.n_seq * a.c.heads, append && a.b.max_new <= 4 ? 4 : 2);
    expect(a.tiles > 0 && a.tiles >= a.b.max_new / kTile, "positions of a move");
    return 0;
}
int launch_append(const MoveArgs &a, void *) { return moved(a, true); }
int launch_read(const MoveArgs &a, void *) { return moved(a, false); }
static int attended(const AttendArgs &a, int row_tile) {
    const double heads = (double)a.b.n_seq * a.c.heads;
    expect((int64_t)a.row_blocks * row_tile >= a.rows && (1 << a.row_shift) == row_tile, "rows of attention");
    expect(a.even || ((int64_t)a.n_split << a.chunk_shift) >= a.max_len, "positions of attention");
    if (!a.even) launch("attention", heads * a.n_split * a.row_blocks, 1);
    if (a.n_split > 1 && (a.even || a.n_split <= 16)) launch("joining few parts", heads * a.rows, 1024 / a.c.dim);
    if (a.n_split > 16 && !a.even) launch("joining", heads * a.rows * (a.c.dim / 32), 1);
    if (a.scores_out && a.max_len) launch("scores", heads * std::ceil(a.max_len / (a.rows <= 8 ? 1024.0 : 128.0)), 1);
    return 0;
}
int launch_attend_d64(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d96(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d128(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d256(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_weigh(const AttendArgs &a, void *) {
    launch("scores alone", (double)a.b.n_seq * a.c.heads * std::ceil(a.max_len / 1024.0), 1);
    return 0;
}
int launch_evict(const EvictArgs &a, void *) {
    const double heads = (double)a.b.n_seq * a.c.heads, most = a.budget < a.max_len ? a.budget : a.max_len;
    launch("choosing", heads, 1, 1024);
    if (most) launch("moving", heads * std::ceil(most / 32), 4);
    return 0;
}
}  // namespace tkv

static uint64_t g_state = 0x9E3779B97F4A7C15ull;
static uint64_t rnd() {
    g_state ^= g_state >> 12;
    g_state ^= g_state << 25;
    g_state ^= g_state >> 27;
    return g_state * 0x2545F4914F6CDD1Dull;
}
// Of every size up to hi, its last few among them.
static int64_t any(int64_t hi) {
    if (rnd() % 8 == 0) return hi - (int64_t)(rnd() % 200) % (hi + 1);
    const int64_t n = (int64_t)(rnd() >> (1 + rnd() % 62));
    return n <= hi ? n : n % (hi + 1);
}

static void *const kAt = (void *)(uintptr_t)(1 << 20);  // never read

static tkv_cache random_cache() {
    static const uint32_t dims[] = {64, 96, 128, 256};
    tkv_cache c;
    uint32_t dim, group;
    do {
        dim = dims[rnd() % 4];
        group = 32u << (rnd() % 3);
    } while (dim % group);
    expect(tkv_encode(&c, kAt, 1 + any(0x7FFFFFFD), 1 + (uint32_t)any(rnd() % 2 ? 15 : 65534), dim, 32u << (rnd() % 6),
                      group) == TMAP_SUCCESS, "encode");
    return c;
}

static tkv_batch random_batch(bool few) {
    tkv_batch b;
    std::memset(&b, 0, sizeof b);
    b.table = (const int32_t *)kAt;
    b.lens = (const int32_t *)kAt;
    b.n_seq = (int32_t)any(few ? 300 : 0x7FFFFFFF);
    b.table_width = (int32_t)any(few ? 5000 : 0x7FFFFFFF);
    b.table_stride = b.table_width + any(1000);
    b.n_tokens = any(0x7FFFFFFF);
    b.max_new = (int32_t)any(few ? 2000 : 0x7FFFFFFF);
    if (rnd() % 2)
        b.starts = (const int32_t *)kAt;
    else if (b.n_seq)
        b.n_tokens -= b.n_tokens % b.n_seq;
    return b;
}

static bool documented(tmap_status st) {
    accepted += st == TMAP_SUCCESS;
    return st == TMAP_SUCCESS || (st == TMAP_ERROR_INVALID_VALUE && tkv_last_error_detail()[0]);
}

int main() {
    const int32_t types[] = {TMAP_F16, TMAP_BF16, TMAP_F32};
    for (int round = 0; round < 200000; ++round) {
        g_cus = rnd() % 2 ? 256 : 32;
        const tkv_cache c = random_cache();
        const bool few = rnd() % 4 != 0;
        const tkv_batch b = random_batch(few);
        const tkv_tokens t = {kAt, any(1 << 20), any(1 << 20), types[rnd() % 2]};
        expect(documented(tkv_append(&c, &t, &t, &b, nullptr)), "append");
        expect(documented(tkv_read(&c, &t, &t, &b, nullptr)), "read");
        tkv_attend_args a;
        std::memset(&a, 0, sizeof a);
        a.q = a.out = t;
        a.lse = (float *)kAt;
        a.q_heads = (int32_t)any(few ? 1000 : 0x7FFFFFFF);
        if (rnd() % 8) a.q_heads = (int32_t)((1 + any(16)) * ((const tkv::Cache *)&c)->heads);
        a.max_len = (int32_t)any(rnd() % 2 ? 100000 : 0x7FFFFFFF);
        a.scale = 0.1f;
        a.causal = (int32_t)(rnd() % 2);
        if (rnd() % 2) {
            a.scores_out = (float *)kAt;
            a.score_stride = (int64_t)a.max_len + any(1000);
        }
        uint64_t need = 0;
        const tmap_status st = tkv_attend_workspace(&c, &a, &b, &need);
        expect(documented(st), "attend's workspace");
        if (st == TMAP_SUCCESS) {
            a.workspace = kAt;
            a.workspace_bytes = need;
            expect(documented(tkv_attend(&c, &a, &b, nullptr)), "attend");
            if (need) {
                a.workspace_bytes = need - 1;
                expect(tkv_attend(&c, &a, &b, nullptr) == TMAP_ERROR_INVALID_VALUE, "attend with less workspace");
            }
        }
        uint64_t bound = 0;
        if (st == TMAP_SUCCESS) {
            expect(documented(tkv_attend_workspace_bound(&c, &a, &b, &bound)) && bound >= need, "the bound of a workspace");
            for (int i = 0; i < 4; ++i) {  // smaller calls
                tkv_attend_args less = a;
                tkv_batch fewer = b;
                if (rnd() % 2) less.max_len = (int32_t)any(a.max_len);
                if (rnd() % 2) fewer.table_width = (int32_t)any(b.table_width);
                if (rnd() % 2) fewer.max_new = (int32_t)any(b.max_new);
                if (rnd() % 2) fewer.n_seq = (int32_t)any(b.n_seq);
                if (rnd() % 2) fewer.n_tokens = any(b.n_tokens);
                if (rnd() % 2) less.scores_out = nullptr;
                fewer.starts = (const int32_t *)kAt;
                uint64_t some = 0;
                expect(tkv_attend_workspace(&c, &less, &fewer, &some) == TMAP_SUCCESS && some <= bound,
                       "the workspace of a smaller call");
            }
        }
        tkv_evict_args e;
        std::memset(&e, 0, sizeof e);
        e.scores = (const float *)kAt;
        e.scores_out = (float *)kAt;
        e.kept = e.lens_out = (int32_t *)kAt;
        e.dst_table = (const int32_t *)kAt;
        e.dst_width = (int32_t)any(0x7FFFFFFF);
        e.dst_stride = e.dst_width + any(1000);
        e.budget = (int32_t)any(few ? 100000 : 0x7FFFFFFF);
        e.recent = (int32_t)any(0x7FFFFFFF);
        e.max_len = (int32_t)any(0x7FFFFFFF);
        e.score_stride = e.max_len + any(1000);
        expect(documented(tkv_evict(&c, &e, &b, nullptr)), "evict");
    }
    std::printf("%d calls accepted, %d launches, %d unexpected results\n", accepted, launches, bad);
    return bad != 0;
}
