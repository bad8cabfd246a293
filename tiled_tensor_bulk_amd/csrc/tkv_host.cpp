// tkv_host.cpp -- host half of libtkv: the cache descriptor, the checks of
// every call's arguments, the gfx950 gate and the split of attention's work.
// Nothing here throws: details of a failure go into a fixed buffer.

#include <hip/hip_runtime_api.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "tkv_internal.h"

namespace {

using tkv::Cache;

thread_local char g_detail[256];

tmap_status fail(tmap_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
tmap_status fail(tmap_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_detail, sizeof g_detail, fmt, ap);
    va_end(ap);
    return st;
}

tmap_status ok() {
    g_detail[0] = 0;
    return TMAP_SUCCESS;
}

#define TKV_REQUIRE(cond, ...) \
    do {                       \
        if (!(cond)) return fail(TMAP_ERROR_INVALID_VALUE, __VA_ARGS__); \
    } while (0)
#define TKV_TRY(call)                              \
    do {                                           \
        const tmap_status st_ = (call);            \
        if (st_ != TMAP_SUCCESS) return st_;       \
    } while (0)

bool decode(const tkv_cache *cache, Cache &c) {
    if (!cache) return false;
    std::memcpy(&c, cache, sizeof c);
    return c.magic == tkv::kMagic;
}

bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Compute units of the current device, which has to be a gfx950 one.
tmap_status device(int &cus) {
    static std::atomic<int> seen[64];  // 0: not looked at, -1: another device, else its compute units
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) {
        (void)hipGetLastError();
        return fail(TMAP_ERROR_UNSUPPORTED_DEVICE, "no HIP device is available");
    }
    int v = seen[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        hipDeviceProp_t p;
        if (hipGetDeviceProperties(&p, dev) != hipSuccess) {
            (void)hipGetLastError();
            return fail(TMAP_ERROR_UNSUPPORTED_DEVICE, "cannot query HIP device %d", dev);
        }
        v = std::strncmp(p.gcnArchName, "gfx950", 6) == 0 && p.multiProcessorCount > 0 ? p.multiProcessorCount : -1;
        seen[dev].store(v, std::memory_order_relaxed);
    }
    if (v < 0) return fail(TMAP_ERROR_UNSUPPORTED_DEVICE, "device %d is not gfx950", dev);
    (void)hipGetLastError();  // one that an earlier call on this thread left is not this call's
    cus = v;
    return TMAP_SUCCESS;
}

tmap_status launched(int rc) {
    if (rc != 0) return fail(TMAP_ERROR_LAUNCH, "launch failed: %s", hipGetErrorString((hipError_t)rc));
    return ok();
}

constexpr int64_t kMostBlocks = 0x7FFFFFFF;

// Whether a product of sizes is less than kMostBlocks; of numbers that the
// arguments' types allow it may take more than 64 bits.
template <class... Sizes>
bool launchable(Sizes... sizes) {
    return ((__int128)1 * ... * (int64_t)sizes) < kMostBlocks;
}

// A launch has fewer than 2^32 threads.
bool fits(int64_t blocks, int threads = tkv::kBlockThreads) { return blocks <= 0xFFFFFFFF / threads; }
int64_t over(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Positions of a sequence: what kernels add to one before they compare it, a
// chunk at most, stays within 31 bits.
constexpr int64_t kMostPositions = 0x7FFFFFFF - 2 * (1 << 16);

tmap_status check_batch(const Cache &c, const tkv_batch *in, tkv::Batch &b, bool tokens) {
    TKV_REQUIRE(in, "batch is NULL");
    TKV_REQUIRE(in->n_seq >= 0, "n_seq is negative");
    TKV_REQUIRE(in->table_width >= 0 && in->table_stride >= in->table_width,
                "table_width must be >= 0 and at most table_stride");
    TKV_REQUIRE(((int64_t)in->table_width << c.page_shift) <= kMostPositions, "a row of the table holds 2^31 positions");
    TKV_REQUIRE(in->n_seq == 0 || (in->lens && aligned(in->lens, 4)), "lens is NULL or not 4-byte aligned");
    TKV_REQUIRE(in->n_seq == 0 || in->table_width == 0 || (in->table && aligned(in->table, 4)),
                "table is NULL or not 4-byte aligned");
    b.table = in->table;
    b.table_stride = in->table_stride;
    b.lens = in->lens;
    b.starts = nullptr;
    b.n_tokens = 0;
    b.n_seq = in->n_seq;
    b.table_width = in->table_width;
    b.max_new = b.uniform = 0;
    if (!tokens) return TMAP_SUCCESS;
    TKV_REQUIRE(in->n_tokens >= 0 && in->n_tokens <= 0x7FFFFFFF, "n_tokens must be in [0, 2^31)");
    TKV_REQUIRE(in->max_new >= 0, "max_new is negative");
    TKV_REQUIRE(!in->starts || aligned(in->starts, 4), "starts is not 4-byte aligned");
    if (!in->starts && in->n_seq > 0) {
        TKV_REQUIRE(in->n_tokens % in->n_seq == 0, "without starts, n_tokens must be a multiple of n_seq");
        b.uniform = (int32_t)(in->n_tokens / in->n_seq);
    }
    b.starts = in->starts;
    b.n_tokens = in->n_tokens;
    b.max_new = in->max_new;
    if (b.max_new > in->n_tokens) b.max_new = (int32_t)in->n_tokens;
    return TMAP_SUCCESS;
}

tmap_status check_tokens(const tkv_tokens &in, const char *name, bool fp32_too, bool empty, tkv::Tokens &t) {
    int size = 2;
    switch (in.dtype) {
        case TMAP_F16: t.type = tkv::kF16; break;
        case TMAP_BF16: t.type = tkv::kBf16; break;
        case TMAP_F32:
            if (fp32_too) {
                t.type = tkv::kF32;
                size = 4;
                break;
            }
            [[fallthrough]];
        default: return fail(TMAP_ERROR_INVALID_VALUE, "%s must be fp16 or bf16%s", name, fp32_too ? " or fp32" : "");
    }
    TKV_REQUIRE(empty || (in.data && aligned(in.data, (uintptr_t)size)), "%s is NULL or not aligned to its elements", name);
    TKV_REQUIRE(in.token_stride >= 0 && in.head_stride >= 0, "%s has a negative stride", name);
    t.data = in.data;
    t.token_stride = in.token_stride;
    t.head_stride = in.head_stride;
    t.wide = aligned(in.data, 16) && in.token_stride % 8 == 0 && in.head_stride % 8 == 0;
    return TMAP_SUCCESS;
}

// Rows that a call writes may not lie in one another.
tmap_status check_written(const tkv_tokens &out, const char *name, int64_t n_tokens, int64_t heads, uint32_t dim) {
    TKV_REQUIRE((n_tokens < 2 || out.token_stride >= dim) && (heads < 2 || out.head_stride >= dim),
                "%s's rows overlap: a stride is less than head_dim", name);
    return TMAP_SUCCESS;
}

tmap_status move_args(const tkv_cache *cache, const tkv_tokens *k, const tkv_tokens *v, const tkv_batch *batch,
                      bool append, tkv::MoveArgs &a) {
    TKV_REQUIRE(decode(cache, a.c), "cache was never encoded");
    TKV_REQUIRE(k && v, "k or v is NULL");
    TKV_TRY(check_batch(a.c, batch, a.b, true));
    TKV_TRY(check_tokens(*k, "k", !append, a.b.n_tokens == 0, a.k));
    TKV_TRY(check_tokens(*v, "v", !append, a.b.n_tokens == 0, a.v));
    TKV_REQUIRE(k->dtype == v->dtype, "k and v must have one type");
    if (!append) {
        TKV_TRY(check_written(*k, "k", a.b.n_tokens, a.c.heads, a.c.dim));
        TKV_TRY(check_written(*v, "v", a.b.n_tokens, a.c.heads, a.c.dim));
    }
    // a run of n positions that starts anywhere touches at most this many records
    a.tiles = a.b.max_new == 0 ? 0 : (int32_t)(((int64_t)a.b.max_new + 2 * (tkv::kTile - 1)) / tkv::kTile);
    // a wave for each record, or two
    constexpr int kWaves = tkv::kBlockThreads / 64;
    TKV_REQUIRE(launchable(a.tiles, a.b.n_seq, a.c.heads) &&
                    fits(over((int64_t)a.tiles * a.b.n_seq * a.c.heads,
                              append && a.b.max_new <= tkv::kFewTokens && a.c.group ? kWaves : kWaves / 2)),
                "too many sequences, heads and new tokens");
    return TMAP_SUCCESS;
}

// How attention is split: see plan().
struct Split {
    int row_tile, row_blocks, n_split, chunk, row_tiles;
    bool even;
    uint64_t part_o, part_ml, dealt, frag_q, row_info, total;  // offsets, and bytes in all
};

tkv::Divisor divisor(uint32_t d) {
    tkv::Divisor r{0, 0};
    while ((1u << r.shift) < d) ++r.shift;
    r.mul = (uint32_t)(((1ull << (31 + r.shift)) + d - 1) / d);
    return r;
}

uint64_t up(uint64_t v, uint64_t to) { return (v + to - 1) / to * to; }

// Rows of a workgroup: 16 or 32 whose positions its waves share, or 64 or 128
// that its waves share.  With 256 channels the registers hold 16 in the first
// manner, and that reads each record for every 16 rows, which pays up to 48 of
// them: 8 sequences of up to 1500 positions, 34 rows, 22 us, with 64 rows of the
// second manner 31; 4 of up to 8192, 32 rows 38 us, 48 rows 46 and 42, 64 rows
// 60 and 44.  The 8-bit format's many rows come in blocks of 128 only, and it
// takes tiles of 16 or 32 up to 64 rows: 128 channels, 8 heads, 48 rows, 8
// sequences of up to 1500 positions 20 us, in a block of 64 that was 25; 4 of up
// to 8192 34 and 33; 256 channels, 4 heads, 64 rows, 31 and 46, 60 and 49.
//
// Chunks: as long as they leave 8 workgroups of few rows for a compute unit, 2
// of many (512 new tokens over 8192 positions, 2 sequences: 217 us with 2, 307
// with 1, 243 with 4), and at least 512 positions, as each costs a partial sum:
// 16 sequences of up to 4099 positions, 22.7 us, at least 256 22.1, 1024 24.8;
// 12 of up to 8191, 18.2, 20.5 and 17.0.  Few rows have chunks of 256 as long
// as that is no more than 2 workgroups for a compute unit: 8 heads, 1 sequence of
// 2000 positions 10.7 us, 512 at least 12.3; 16 of 1000 12.1 and 12.8; but 16 of
// 2000 17.0 and 15.8.  Powers of two, so that another bound
// on the lengths mostly leaves the order of sums as it is.
//
// The host does not know the lengths, though, and where chunks are long a block
// is a whole sequence or a good part of one.  Then few rows go by an even split,
// the lengths in device memory deciding.  128 channels, 8 heads of 4 rows,
// microseconds, even and in chunks: 64 sequences of 4096 to 32768 positions 269
// and 290; 120 of 100 to 8000 122 and 133; one of 131072 and 63 of 1000 67 and
// 227; 64 of 1000 in tables for 32768 29 and 47; but 64 of 8192 128 and 121, for
// finding its share costs a workgroup some 3 us.  It does not pay where row
// blocks alone fill the card, 200 sequences of 100 to 4000 109 and 98, or 256 of
// 1000 62 and 54, unless one may be so long that the others wait for it: one of
// 131072 and 199 of 1000 102 and 453.
constexpr int kLeastChunk = 512;
constexpr int kMostChunk = 1 << 16;  // kMostPositions leaves room for two
constexpr int kLongForOne = 1 << 14;
constexpr int kBlocksPerCu = 8;
constexpr int kRowBlocksPerCu = 2;

// With a window the same of what a block of rows may see of a sequence.
int64_t seen_at_most(const tkv::AttendArgs &a, int row_tile) {
    if (!a.window) return a.max_len;
    int64_t tokens = a.b.max_new;
    if (row_tile > 32) {
        const int64_t block = (row_tile + 2 * (int64_t)a.group_heads - 2) / a.group_heads;
        tokens = block < tokens ? block : tokens;
    }
    const int64_t n = (int64_t)a.sinks + a.window + tokens + 2 * tkv::kTile;  // both ends in whole records
    return n < a.max_len ? n : a.max_len;
}

// Rows up to which the waves of a workgroup share the positions.
int64_t most_few_rows(const Cache &c) { return c.group == 0 ? 64 : c.dim > 128 ? 48 : 32; }

Split plan(const tkv::AttendArgs &a, int cus) {
    const Cache &c = a.c;
    const int64_t n_seq = a.b.n_seq, rows = a.rows;
    const bool scores = a.scores_out;
    Split s{};
    const bool few = rows <= most_few_rows(c);
    s.row_tile = rows <= 16 || (few && c.dim > 128) ? 16 : few ? 32 : c.group && (rows <= 64 || c.dim > 128) ? 64 : 128;
    s.row_blocks = (int)((rows + s.row_tile - 1) / s.row_tile);
    s.row_tiles = (int)((rows + 15) / 16);
    const int64_t max_len = seen_at_most(a, s.row_tile);
    const int64_t units = n_seq * c.heads * s.row_blocks;
    s.chunk = kLeastChunk;
    const int64_t most = (int64_t)cus * (s.row_tile <= 32 ? kBlocksPerCu : kRowBlocksPerCu);
    if (s.row_tile <= 32 && max_len > kLeastChunk && units * ((max_len + 255) / 256) <= (int64_t)cus * 2) s.chunk = 256;
    while (s.chunk < kMostChunk && units * ((max_len + s.chunk - 1) / s.chunk) > most) s.chunk *= 2;
    s.n_split = (int)((max_len + s.chunk - 1) / s.chunk);
    if (s.n_split < 1) s.n_split = 1;
    const uint64_t heads = (uint64_t)n_seq * c.heads;
    const int64_t groups = (int64_t)cus * tkv::kMostResident;
    s.even = s.row_tile <= 32 && s.chunk > kLeastChunk && n_seq <= tkv::kEvenSeqs &&
             (units < groups || max_len > kLongForOne) && units * (max_len / kLeastChunk + 1) < (1 << 28);
    if (s.even) {
        s.n_split = (int)(groups / units + 2);
        const uint64_t parts = (uint64_t)(units + groups) * (rows < s.row_tile ? rows : s.row_tile);
        s.part_o = s.total;
        s.total = up(s.total + parts * c.dim * 4, 256);
        s.part_ml = s.total;
        s.total = up(s.total + parts * 8, 256);
        s.dealt = s.total;
        s.total = up(s.total + (tkv::kEvenSeqs + 1) * 4, 256);
    } else if (s.n_split > 1) {
        s.part_o = s.total;
        s.total = up(s.total + heads * s.n_split * rows * c.dim * 4, 256);
        s.part_ml = s.total;
        s.total = up(s.total + heads * s.n_split * rows * 8, 256);
    }
    if (scores) {
        s.frag_q = s.total;
        if (rows <= tkv::kLogitRows)
            s.total = up(s.total + heads * up((uint64_t)max_len, tkv::kTile) * rows * 4, 256);
        else
            s.total = up(s.total + heads * s.row_tiles * (32 * c.dim + 1024), 256);
        s.row_info = s.total;
        s.total = up(s.total + heads * s.row_tiles * 16 * 8, 256);
    }
    return s;
}

// What plan() takes at most of a workspace for no more sequences, rows and
// positions than these.  Fewer of them may need more: chunks get shorter when
// there are fewer workgroups to fill the card with.
uint64_t most_workspace(const Cache &c, int64_t n_seq, int64_t rows, int64_t max_len, bool scores, int cus) {
    const auto least = [](uint64_t a, uint64_t b) { return a < b ? a : b; };
    const auto most = [](uint64_t a, uint64_t b) { return a > b ? a : b; };
    const uint64_t heads = (uint64_t)n_seq * c.heads, few = least(rows, c.group ? 48 : 64);
    const auto chunks = [&](int64_t chunk) { return (uint64_t)((max_len + chunk - 1) / chunk); };
    // rows of partial sums.  In chunks shorter than kMostChunk: the workgroups, kBlocksPerCu for a
    // compute unit of 32 rows or kRowBlocksPerCu of 128, and no more than chunks of 256 make
    uint64_t parts = least((uint64_t)cus * most(kBlocksPerCu * 32, kRowBlocksPerCu * 128), heads * rows * chunks(256));
    if (chunks(kMostChunk) > 1) parts = most(parts, heads * rows * chunks(kMostChunk));
    if (max_len > kLeastChunk)  // an even split: tiles of 16 rows up to 48 of them, or one of 32; in 8 bits several
        parts = most(parts, least(n_seq, tkv::kEvenSeqs) * c.heads * (few + (c.group ? 15 : 31)) +
                                (uint64_t)cus * tkv::kMostResident * least(rows, 32));
    uint64_t total = 0;
    if (max_len > 256) total = up(parts * c.dim * 4, 256) + up(parts * 8, 256) + up((tkv::kEvenSeqs + 1) * 4, 256);
    if (scores) {
        const uint64_t tiles = (uint64_t)(rows + 15) / 16;
        const uint64_t logits = heads * up((uint64_t)max_len, tkv::kTile) * least(rows, tkv::kLogitRows) * 4;
        total += up(most(logits, heads * tiles * (32 * c.dim + 1024)), 256) + up(heads * tiles * 16 * 8, 256);
    }
    return total;
}

tmap_status attend_args(const tkv_cache *cache, const tkv_attend_args *in, const tkv_window *window,
                        const tkv_batch *batch, bool pointers, tkv::AttendArgs &a) {
    TKV_REQUIRE(decode(cache, a.c), "cache was never encoded");
    TKV_REQUIRE(in, "args is NULL");
    TKV_TRY(check_batch(a.c, batch, a.b, true));
    const bool empty = !pointers || a.b.n_tokens == 0;
    TKV_TRY(check_tokens(in->q, "q", false, empty, a.q));
    TKV_TRY(check_tokens(in->out, "out", false, empty, a.out));
    TKV_REQUIRE(in->q.dtype == in->out.dtype, "q and out must have one type");
    TKV_REQUIRE(empty || (in->lse && aligned(in->lse, 4)), "lse is NULL or not 4-byte aligned");
    TKV_REQUIRE(in->q_heads > 0 && in->q_heads % (int64_t)a.c.heads == 0, "q_heads must be a multiple of n_heads");
    if (pointers) TKV_TRY(check_written(in->out, "out", a.b.n_tokens, in->q_heads, a.c.dim));
    TKV_REQUIRE(in->max_len >= 0, "max_len is negative");
    TKV_REQUIRE(std::isfinite(in->scale), "scale is not finite");
    TKV_REQUIRE(in->causal == 0 || in->causal == 1, "causal must be 0 or 1");
    if (in->scores_out) {
        TKV_REQUIRE(aligned(in->scores_out, 4) && aligned(in->scores_in, 4), "scores are not 4-byte aligned");
        TKV_REQUIRE(in->score_stride >= in->max_len, "score_stride is less than max_len");
        TKV_REQUIRE(a.c.group, "scores are kept of a cache in 4 bits, and this one has 8");
        TKV_REQUIRE(!window, "scores are not kept with a window");
    } else {
        TKV_REQUIRE(!in->scores_in, "scores_in without scores_out");
    }
    if (window) {
        TKV_REQUIRE(window->window >= 1, "window is less than 1");
        TKV_REQUIRE(window->sinks >= 0, "sinks is negative");
        a.window = window->window;
        a.sinks = window->sinks < kMostPositions ? window->sinks : (int32_t)kMostPositions;
    }
    a.lse = in->lse;
    a.scale_log2 = in->scale * 1.44269504089f;
    a.causal = in->causal;
    a.group_heads = in->q_heads / (int32_t)a.c.heads;
    const int64_t rows = (int64_t)a.b.max_new * a.group_heads;
    TKV_REQUIRE(rows < (1 << 30), "too many new tokens and query heads");
    a.rows = (int32_t)rows;
    a.max_len = in->max_len;
    // no position lies past the table
    const int64_t width = (int64_t)a.b.table_width << a.c.page_shift;
    if (a.max_len > width) a.max_len = (int32_t)width;
    TKV_REQUIRE(launchable(a.b.n_seq, a.c.heads, a.max_len / 128 + 1) &&
                    launchable(a.b.n_seq, a.c.heads, a.rows, a.c.dim / 32), "too many sequences, heads and rows");
    a.scores_in = in->scores_in;
    a.scores_out = in->scores_out;
    a.score_stride = in->score_stride;
    return TMAP_SUCCESS;
}

tmap_status check_pool(const tkv_cache *cache, const void *pool, int64_t n_pages, uint32_t n_heads, uint32_t head_dim,
                       uint32_t page_tokens) {
    TKV_REQUIRE(cache, "cache is NULL");
    TKV_REQUIRE(pool && aligned(pool, 16), "pool is NULL or not 16-byte aligned");
    TKV_REQUIRE(n_pages >= 1 && n_pages < 0x7FFFFFFF, "n_pages must be in [1, 2^31 - 1)");
    TKV_REQUIRE(n_heads >= 1 && n_heads <= 65535, "n_heads must be in [1, 65535]");
    TKV_REQUIRE(head_dim == 64 || head_dim == 96 || head_dim == 128 || head_dim == 256,
                "head_dim must be 64, 96, 128 or 256");
    TKV_REQUIRE(page_tokens >= 32 && page_tokens <= 1024 && (page_tokens & (page_tokens - 1)) == 0,
                "page_tokens must be a power of two in [32, 1024]");
    return TMAP_SUCCESS;
}

void describe(tkv_cache *cache, void *pool, int64_t n_pages, uint32_t n_heads, uint32_t head_dim, uint32_t page_tokens,
              uint32_t group, uint32_t record) {
    Cache c{};
    c.pool = (uint64_t)(uintptr_t)pool;
    c.n_pages = (uint32_t)n_pages;
    c.heads = n_heads;
    c.dim = head_dim;
    c.group = group;
    while ((1u << c.page_shift) < page_tokens) ++c.page_shift;
    c.record = record;
    c.head_bytes = c.record * (page_tokens / tkv::kTile);
    c.page_bytes = (uint64_t)c.head_bytes * n_heads;
    c.magic = tkv::kMagic;
    std::memcpy(cache, &c, sizeof c);
}

tmap_status rotation_args(const tkv_rotation *in, tkv::MoveArgs &a) {
    TKV_REQUIRE(in, "rotation is NULL");
    const bool empty = a.b.n_tokens == 0;
    tkv::Rotation &r = a.rot;
    TKV_REQUIRE(in->rot_dim >= 16 && in->rot_dim % 16 == 0 && (uint32_t)in->rot_dim <= a.c.dim,
                "rot_dim must be a multiple of 16 and at most head_dim");
    TKV_REQUIRE(in->neighbours == 0 || in->neighbours == 1, "neighbours must be 0 or 1");
    TKV_REQUIRE(in->n_positions >= 0 && in->n_positions <= 0x7FFFFFFF, "n_positions must be in [0, 2^31)");
    TKV_REQUIRE(in->stride >= in->rot_dim, "the table's stride is less than rot_dim");
    TKV_REQUIRE(empty || in->n_positions == 0 || (in->cos_sin && aligned(in->cos_sin, 4)),
                "cos_sin is NULL or not 4-byte aligned");
    TKV_REQUIRE(aligned(in->positions, 4), "positions is not 4-byte aligned");
    TKV_REQUIRE(in->q_heads >= 0, "q_heads is negative");
    TKV_REQUIRE(in->q_heads <= 1 << 30, "q_heads is more than 2^30");  // heads are counted in 31 bits, some past the last one
    r.table = in->cos_sin;
    r.stride = in->stride;
    r.positions = in->positions;
    r.n_positions = (int32_t)in->n_positions;
    r.dim = in->rot_dim;
    r.neighbours = in->neighbours;
    r.wide = aligned(in->cos_sin, 16) && in->stride % 4 == 0 && in->rot_dim % 8 == 0;
    r.q_heads = in->q_heads;
    if (!r.q_heads) return TMAP_SUCCESS;
    TKV_TRY(check_tokens(in->q, "q", false, empty, r.q));
    TKV_TRY(check_tokens(in->q_out, "q_out", false, empty, r.q_out));
    TKV_REQUIRE(in->q.dtype == in->q_out.dtype, "q and q_out must have one type");
    TKV_TRY(check_written(in->q_out, "q_out", a.b.n_tokens, in->q_heads, a.c.dim));
    r.same = in->q.data == in->q_out.data && in->q.token_stride == in->q_out.token_stride &&
             in->q.head_stride == in->q_out.head_stride;
    TKV_REQUIRE(r.same || in->q.data != in->q_out.data || empty, "q_out is q with other strides");
    // a wave for each token, or more of them for few
    const int64_t tokens = (int64_t)a.b.n_seq * a.b.max_new;
    const int64_t blocks = over(tokens > tkv::kQueryTokens ? tokens : tkv::kQueryTokens * tkv::kQueryWaves, tkv::kBlockThreads / 64);
    const int64_t records = a.b.max_new <= tkv::kFewTokens ? over((int64_t)a.tiles * a.b.n_seq * a.c.heads, 2) : 0;
    TKV_REQUIRE(launchable(a.b.n_seq, a.b.max_new) && fits(blocks + records), "too many sequences and new tokens");
    return TMAP_SUCCESS;
}

tmap_status append(tkv::MoveArgs &a, void *hip_stream) {
    int cus = 0;
    TKV_TRY(device(cus));
    if (a.tiles == 0 || a.b.n_seq == 0) return ok();
    return launched(tkv::launch_append(a, hip_stream));
}

}  // namespace

extern "C" {

tmap_status tkv_encode(tkv_cache *cache, void *pool, int64_t n_pages, uint32_t n_heads, uint32_t head_dim,
                       uint32_t page_tokens, uint32_t group) {
    TKV_TRY(check_pool(cache, pool, n_pages, n_heads, head_dim, page_tokens));
    TKV_REQUIRE((group == 32 || group == 64 || group == 128) && head_dim % group == 0,
                "group must be 32, 64 or 128 and divide head_dim");
    describe(cache, pool, n_pages, n_heads, head_dim, page_tokens, group,
             32 * head_dim + 256 * (head_dim / group));
    return ok();
}

tmap_status tkv_encode8(tkv_cache *cache, void *pool, int64_t n_pages, uint32_t n_heads, uint32_t head_dim,
                        uint32_t page_tokens) {
    TKV_TRY(check_pool(cache, pool, n_pages, n_heads, head_dim, page_tokens));
    describe(cache, pool, n_pages, n_heads, head_dim, page_tokens, 0, 64 * head_dim + 128);
    return ok();
}

uint64_t tkv_page_bytes(const tkv_cache *cache) {
    Cache c;
    return decode(cache, c) ? c.page_bytes : 0;
}

tmap_status tkv_append(const tkv_cache *cache, const tkv_tokens *k, const tkv_tokens *v, const tkv_batch *batch,
                       void *hip_stream) {
    tkv::MoveArgs a{};
    TKV_TRY(move_args(cache, k, v, batch, true, a));
    return append(a, hip_stream);
}

tmap_status tkv_append_rotated(const tkv_cache *cache, const tkv_tokens *k, const tkv_tokens *v,
                               const tkv_rotation *rotation, const tkv_batch *batch, void *hip_stream) {
    tkv::MoveArgs a{};
    TKV_TRY(move_args(cache, k, v, batch, true, a));
    TKV_TRY(rotation_args(rotation, a));
    return append(a, hip_stream);
}

tmap_status tkv_read(const tkv_cache *cache, const tkv_tokens *k, const tkv_tokens *v, const tkv_batch *batch,
                     void *hip_stream) {
    tkv::MoveArgs a{};
    TKV_TRY(move_args(cache, k, v, batch, false, a));
    int cus = 0;
    TKV_TRY(device(cus));
    if (a.tiles == 0 || a.b.n_seq == 0) return ok();
    return launched(tkv::launch_read(a, hip_stream));
}

tmap_status tkv_attend_window_workspace(const tkv_cache *cache, const tkv_attend_args *args, const tkv_window *window,
                                        const tkv_batch *batch, uint64_t *bytes) {
    tkv::AttendArgs a{};
    TKV_REQUIRE(bytes, "bytes is NULL");
    TKV_TRY(attend_args(cache, args, window, batch, false, a));
    int cus = 0;
    TKV_TRY(device(cus));
    *bytes = a.rows > 0 && a.b.n_seq > 0 ? plan(a, cus).total : 0;
    return ok();
}

tmap_status tkv_attend_workspace(const tkv_cache *cache, const tkv_attend_args *args, const tkv_batch *batch,
                                 uint64_t *bytes) {
    return tkv_attend_window_workspace(cache, args, nullptr, batch, bytes);
}

tmap_status tkv_attend_workspace_bound(const tkv_cache *cache, const tkv_attend_args *args, const tkv_batch *batch,
                                       uint64_t *bytes) {
    tkv::AttendArgs a{};
    TKV_REQUIRE(bytes, "bytes is NULL");
    TKV_TRY(attend_args(cache, args, nullptr, batch, false, a));
    int cus = 0;
    TKV_TRY(device(cus));
    *bytes = a.rows > 0 && a.b.n_seq > 0 ? most_workspace(a.c, a.b.n_seq, a.rows, a.max_len, a.scores_out, cus) : 0;
    return ok();
}

tmap_status tkv_attend(const tkv_cache *cache, const tkv_attend_args *args, const tkv_batch *batch, void *hip_stream) {
    return tkv_attend_window(cache, args, nullptr, batch, hip_stream);
}

tmap_status tkv_attend_window(const tkv_cache *cache, const tkv_attend_args *args, const tkv_window *window,
                              const tkv_batch *batch, void *hip_stream) {
    tkv::AttendArgs a{};
    TKV_TRY(attend_args(cache, args, window, batch, true, a));
    int cus = 0;
    TKV_TRY(device(cus));
    if (a.b.n_seq == 0) return ok();
    if (a.rows == 0) {  // no row to answer; scores_out is still to be scores_in, or 0
        if (!a.scores_out || a.scores_out == a.scores_in || a.max_len == 0) return ok();
        TKV_REQUIRE(fits((int64_t)a.b.n_seq * a.c.heads * over(a.max_len, tkv::kWeighPositions)),
                    "too many sequences, heads and positions");
        a.by_heads = divisor(a.c.heads);
        return launched(tkv::launch_weigh(a, hip_stream));
    }
    const Split s = plan(a, cus);
    // every launch of the call, so that none is refused after another has begun
    const int64_t heads = (int64_t)a.b.n_seq * a.c.heads;
    int64_t joining = 0, weighing = 0;
    if (s.n_split > 1)
        joining = s.even || s.n_split <= tkv::kFewParts ? over(heads * a.rows, tkv::kBlockThreads / (a.c.dim / 4))
                                                        : heads * a.rows * (a.c.dim / 32);
    if (a.scores_out) weighing = heads * over(a.max_len, a.rows <= tkv::kLogitRows ? tkv::kWeighPositions : 128);
    TKV_REQUIRE((s.even || (launchable(heads, s.n_split, s.row_blocks) && fits(heads * s.n_split * s.row_blocks))) &&
                    fits(joining + weighing), "too many sequences, heads, rows and positions");
    if (s.total) {
        TKV_REQUIRE(args->workspace && aligned(args->workspace, 16), "workspace is NULL or not 16-byte aligned");
        TKV_REQUIRE(args->workspace_bytes >= s.total, "workspace holds %llu bytes, %llu are needed",
                    (unsigned long long)args->workspace_bytes, (unsigned long long)s.total);
    }
    char *ws = (char *)args->workspace;
    a.row_blocks = s.row_blocks;
    a.row_tiles = s.row_tiles;
    a.n_split = s.n_split;
    a.even = s.even;
    a.cus = cus;
    while ((1 << a.row_shift) < s.row_tile) ++a.row_shift;
    while ((1 << a.chunk_shift) < s.chunk) ++a.chunk_shift;
    a.by_heads = divisor(a.c.heads);
    a.by_group_heads = divisor(a.group_heads);
    a.by_row_blocks = divisor(a.row_blocks);
    a.by_split = divisor(a.n_split);
    a.by_rows = divisor(a.rows);
    if (s.n_split > 1) {
        a.part_o = (float *)(ws + s.part_o);
        a.part_ml = (float *)(ws + s.part_ml);
        a.dealt = (int32_t *)(ws + s.dealt);
    }
    if (a.scores_out) {
        if (a.rows <= tkv::kLogitRows)
            a.logits = (float *)(ws + s.frag_q);
        else
            a.frag_q = ws + s.frag_q;
        a.row_info = (float *)(ws + s.row_info);
    }
    switch (a.c.dim) {
        case 64: return launched(tkv::launch_attend_d64(a, s.row_tile, hip_stream));
        case 96: return launched(tkv::launch_attend_d96(a, s.row_tile, hip_stream));
        case 128: return launched(tkv::launch_attend_d128(a, s.row_tile, hip_stream));
        default: return launched(tkv::launch_attend_d256(a, s.row_tile, hip_stream));
    }
}

tmap_status tkv_evict(const tkv_cache *cache, const tkv_evict_args *args, const tkv_batch *batch, void *hip_stream) {
    tkv::EvictArgs a{};
    TKV_REQUIRE(decode(cache, a.c), "cache was never encoded");
    TKV_REQUIRE(args, "args is NULL");
    TKV_REQUIRE(a.c.group, "eviction is of a cache in 4 bits, and this one has 8");
    TKV_TRY(check_batch(a.c, batch, a.b, false));
    TKV_REQUIRE(args->budget >= 0 && args->recent >= 0, "budget or recent is negative");
    TKV_REQUIRE(args->max_len >= 0 && args->score_stride >= args->max_len, "score_stride is less than max_len");
    TKV_REQUIRE(args->dst_width >= 0 && args->dst_stride >= args->dst_width,
                "dst_width must be >= 0 and at most dst_stride");
    const bool any = a.b.n_seq > 0;
    TKV_REQUIRE(!any || (args->lens_out && aligned(args->lens_out, 4)), "lens_out is NULL or not 4-byte aligned");
    // one sequence's new length may not take another's place before that is read
    const uintptr_t lens_in = (uintptr_t)a.b.lens, lens_out = (uintptr_t)args->lens_out, size = 4 * (uintptr_t)a.b.n_seq;
    TKV_REQUIRE(lens_out == lens_in || lens_out >= lens_in + size || lens_in >= lens_out + size,
                "lens_out overlaps lens and is not lens itself");
    if (any && args->budget > 0) {
        TKV_REQUIRE(args->kept && args->scores_out && aligned(args->kept, 4) && aligned(args->scores_out, 4),
                    "kept or scores_out is NULL or not 4-byte aligned");
        TKV_REQUIRE(args->max_len == 0 || (args->scores && aligned(args->scores, 4)),
                    "scores is NULL or not 4-byte aligned");
        TKV_REQUIRE(args->dst_width == 0 || (args->dst_table && aligned(args->dst_table, 4)),
                    "dst_table is NULL or not 4-byte aligned");
    }
    TKV_REQUIRE(launchable(a.b.n_seq, a.c.heads, args->budget / tkv::kTile + 1),
                "too many sequences, heads and positions");
    a.scores = args->scores;
    a.scores_out = args->scores_out;
    a.score_stride = args->score_stride;
    a.kept = args->kept;
    a.lens_out = args->lens_out;
    a.dst_table = args->dst_table;
    a.dst_stride = args->dst_stride;
    a.dst_width = args->dst_width;
    a.budget = args->budget;
    a.recent = args->recent;
    a.max_len = args->max_len;
    const int64_t width = (int64_t)a.b.table_width << a.c.page_shift;
    if (a.max_len > width) a.max_len = (int32_t)width;
    const int64_t heads = (int64_t)a.b.n_seq * a.c.heads;
    TKV_REQUIRE(fits(heads, tkv::kSelectThreads) &&
                    fits(over(heads * over(a.budget < a.max_len ? a.budget : a.max_len, tkv::kTile), tkv::kBlockThreads / 64)),
                "too many sequences, heads and positions");
    int cus = 0;
    TKV_TRY(device(cus));
    if (!any) return ok();
    return launched(tkv::launch_evict(a, hip_stream));
}

const char *tkv_last_error_detail(void) { return g_detail; }

}  // extern "C"
