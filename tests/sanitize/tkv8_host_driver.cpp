// tkv8_host_driver.cpp -- drives the host half of libtkv (tkv_host.cpp, linked
// in directly) under AddressSanitizer and UndefinedBehaviorSanitizer, with what
// it does for the 8-bit cache, rotations and windows: random calls up to the
// largest sizes.  The HIP calls and the launchers are the ones below.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../tiled_tensor_bulk_amd/csrc/tkv_internal.h"

#undef hipGetDeviceProperties
extern "C" {
hipError_t hipGetDevice(int *dev) {
    *dev = 0;
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600 *p, int) {
    std::memset(p, 0, sizeof *p);
    std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
    p->multiProcessorCount = 256;
    return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "an error"; }
}

static int bad = 0, accepted = 0, launches = 0;
static void expect(bool ok, const char *what) {
    if (!ok && bad++ < 20) std::fprintf(stderr, "unexpected: %s (%s)\n", what, tkv_last_error_detail());
}

static void launch(const char *what, double blocks, int threads = 256) {
    ++launches;
    expect(blocks >= 1 && std::ceil(blocks) * threads < 4294967296.0, what);
}

namespace tkv {
static int moved(const MoveArgs &a, bool append) {
    const bool few = append && a.b.max_new <= kFewTokens;
    double blocks = std::ceil((double)a.tiles * a.b.n_seq * a.c.heads / (few && a.c.group ? 4 : 2));
    const double tokens = a.rot.dim && a.rot.q_heads ? (double)a.b.n_seq * a.b.max_new : 0;
    const int waves = tokens > (double)kQueryTokens ? 1 : kQueryWaves;  // at most
    if (few && a.rot.dim)
        blocks += std::ceil(tokens * waves / 4);
    else if (tokens)
        launch("queries", std::ceil(tokens / 4));
    launch("records of a move", blocks);
    return 0;
}
int launch_append(const MoveArgs &a, void *) { return moved(a, true); }
int launch_read(const MoveArgs &a, void *) { return moved(a, false); }
static int attended(const AttendArgs &a, int row_tile) {
    const double heads = (double)a.b.n_seq * a.c.heads;
    expect(!a.window || (a.sinks >= 0 && a.sinks < 0x7FFFFFFF && a.window > 0), "a window");
    expect((int64_t)a.row_blocks * row_tile >= a.rows && (1 << a.row_shift) == row_tile, "rows of attention");
    expect(row_tile == 16 || (row_tile == 32 && a.c.dim <= 128) || row_tile == (a.c.group ? 64 : 128) ||
               (row_tile == 128 && a.c.dim <= 128), "a kernel");
    // the places that a block of rows may see: the sinks and a window before each of its tokens, in whole records
    double span = a.max_len;
    if (a.window) {
        const int64_t block = ((int64_t)row_tile + 2 * a.group_heads - 2) / a.group_heads;
        const int64_t tokens = row_tile <= 32 || a.b.max_new < block ? a.b.max_new : block;
        const double most = std::ceil(a.sinks / 32.0) * 32 + (double)a.window + (double)tokens - 1 + 31;
        span = most < span ? most : span;
    }
    expect(a.even || (double)((int64_t)a.n_split << a.chunk_shift) >= span, "positions of attention");
    if (!a.even) launch("attention", heads * a.n_split * a.row_blocks);
    if (a.n_split > 1 && (a.even || a.n_split <= 16)) launch("joining few parts", std::ceil(heads * a.rows / (1024 / a.c.dim)));
    if (a.n_split > 16 && !a.even) launch("joining", heads * a.rows * (a.c.dim / 32));
    return 0;
}
int launch_attend_d64(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d96(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d128(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_attend_d256(const AttendArgs &a, int row_tile, void *) { return attended(a, row_tile); }
int launch_weigh(const AttendArgs &, void *) { return 0; }
int launch_evict(const EvictArgs &a, void *) {
    expect(a.c.group, "eviction of the 8-bit cache");
    return 0;
}
}  // namespace tkv

static uint64_t g_state = 0x243F6A8885A308D3ull;
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
static void *const kElse = (void *)(uintptr_t)(1 << 30);

static bool documented(tmap_status st) {
    accepted += st == TMAP_SUCCESS;
    return st == TMAP_SUCCESS || (st == TMAP_ERROR_INVALID_VALUE && tkv_last_error_detail()[0]);
}

int main() {
    static const uint32_t dims[] = {64, 96, 128, 256};
    for (int round = 0; round < 200000; ++round) {
        tkv_cache c;
        const uint32_t dim = dims[rnd() % 4], heads = 1 + (uint32_t)any(rnd() % 2 ? 15 : 65534), page = 32u << (rnd() % 6);
        const int64_t pages = 1 + any(0x7FFFFFFD);
        expect((rnd() % 4 ? tkv_encode8(&c, kAt, pages, heads, dim, page) : tkv_encode(&c, kAt, pages, heads, dim, page, 32)) ==
                   TMAP_SUCCESS, "encode");
        const bool few = rnd() % 4 != 0;
        tkv_batch b;
        std::memset(&b, 0, sizeof b);
        b.table = b.lens = (const int32_t *)kAt;
        b.n_seq = (int32_t)any(few ? 300 : 0x7FFFFFFF);
        b.table_width = (int32_t)any(few ? 5000 : 0x7FFFFFFF);
        b.table_stride = b.table_width + any(1000);
        b.n_tokens = any(0x7FFFFFFF);
        b.max_new = (int32_t)any(rnd() % 2 ? 8 : few ? 2000 : 0x7FFFFFFF);
        if (rnd() % 2)
            b.starts = (const int32_t *)kAt;
        else if (b.n_seq)
            b.n_tokens -= b.n_tokens % b.n_seq;
        const tkv_tokens t = {kAt, any(1 << 20), any(1 << 20), rnd() % 2 ? TMAP_F16 : TMAP_BF16};
        expect(documented(tkv_append(&c, &t, &t, &b, nullptr)), "append");
        expect(documented(tkv_read(&c, &t, &t, &b, nullptr)), "read");
        tkv_rotation r;
        std::memset(&r, 0, sizeof r);
        r.cos_sin = (const float *)kAt;
        r.rot_dim = rnd() % 8 ? 16 * (int32_t)(1 + any(dim / 16 - 1)) : (int32_t)any(300);
        r.stride = r.rot_dim + any(rnd() % 2 ? 100 : (int64_t)1 << 40);
        r.n_positions = any(0x80000000ll);
        r.neighbours = (int32_t)(rnd() % 2);
        r.positions = rnd() % 2 ? (const int32_t *)kAt : nullptr;
        r.q = r.q_out = t;
        if (rnd() % 2) r.q_out.data = kElse;
        r.q_heads = (int32_t)any(few ? 300 : 0x7FFFFFFF);
        expect(documented(tkv_append_rotated(&c, &t, &t, &r, &b, nullptr)), "rotated append");
        tkv_attend_args a;
        std::memset(&a, 0, sizeof a);
        a.q = a.out = t;
        a.lse = (float *)kAt;
        a.q_heads = (int32_t)any(few ? 1000 : 0x7FFFFFFF);
        if (rnd() % 8) a.q_heads = (int32_t)((1 + any(16)) * (int64_t)heads);
        a.max_len = (int32_t)any(rnd() % 2 ? 100000 : 0x7FFFFFFF);
        a.scale = 0.1f;
        a.causal = (int32_t)(rnd() % 2);
        tkv_window w = {(int32_t)any(rnd() % 2 ? 5000 : 0x7FFFFFFF), (int32_t)any(rnd() % 2 ? 100 : 0x7FFFFFFF)};
        const tkv_window *const which = rnd() % 4 ? &w : nullptr;
        uint64_t need = 0, bound = 0;
        const tmap_status st = tkv_attend_window_workspace(&c, &a, which, &b, &need);
        expect(documented(st), "attend's workspace");
        if (st != TMAP_SUCCESS) continue;
        expect(documented(tkv_attend_workspace_bound(&c, &a, &b, &bound)) && bound >= need, "the bound of a workspace");
        a.workspace = kAt;
        a.workspace_bytes = need;
        expect(documented(tkv_attend_window(&c, &a, which, &b, nullptr)), "attend");
        if (need) {
            a.workspace_bytes = need - 1;
            expect(tkv_attend_window(&c, &a, which, &b, nullptr) == TMAP_ERROR_INVALID_VALUE, "attend with less workspace");
        }
        for (int i = 0; i < 4; ++i) {  // smaller calls, other windows
            tkv_attend_args less = a;
            tkv_batch fewer = b;
            tkv_window other = {1 + (int32_t)any(0x7FFFFFFE), (int32_t)any(0x7FFFFFFF)};
            if (rnd() % 2) less.max_len = (int32_t)any(a.max_len);
            if (rnd() % 2) fewer.max_new = (int32_t)any(b.max_new);
            if (rnd() % 2) fewer.n_seq = (int32_t)any(b.n_seq);
            fewer.starts = (const int32_t *)kAt;
            uint64_t some = 0;
            expect(tkv_attend_window_workspace(&c, &less, rnd() % 2 ? &other : nullptr, &fewer, &some) == TMAP_SUCCESS &&
                       some <= bound, "the workspace of a smaller call");
        }
        tkv_evict_args e;
        std::memset(&e, 0, sizeof e);
        expect(documented(tkv_evict(&c, &e, &b, nullptr)), "evict");
    }
    std::printf("%d calls accepted, %d launches, %d unexpected results\n", accepted, launches, bad);
    return bad != 0;
}
