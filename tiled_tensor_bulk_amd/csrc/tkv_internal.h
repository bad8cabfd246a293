// tkv_internal.h -- private layout of the 128-byte cache descriptor and the
// kernels' argument blocks.  Shared by the host half (tkv_host.cpp) and the
// device halves of libtkv only.
#pragma once

#include <stdint.h>

#include "../../include/tkv.h"

namespace tkv {

constexpr uint32_t kMagic = 0x544B5634u;  // "TKV4"
constexpr int kTile = 32;                 // positions of a record
constexpr int kBlockThreads = 256;        // of a workgroup of every kernel but the next
constexpr int kSelectThreads = 1024;      // ... of the one that chooses what eviction keeps
constexpr int kFewTokens = 4;             // up to so many new ones append takes one by one
constexpr int kFewParts = 16;             // up to so many partial sums of a row are joined by its own lanes
constexpr int kWeighPositions = 4 * kBlockThreads;  // of a workgroup that turns logarithms into weights
constexpr int kMostResident = 4;           // workgroups that an even split deals to a compute unit
constexpr int kEvenSeqs = 256;            // most sequences of an even split
// Scores of up to so many rows go by logarithms kept in memory, 8 bytes a row
// and position written and read, against half of a record read again (72 bytes
// of 128 channels): 16 sequences of up to 16384 positions, 4 rows, 95 us with
// the second, 69 with the first.
constexpr int kLogitRows = 8;
constexpr float kLimit = 32000.0f;        // largest magnitude quantised: 15 * scale stays inside fp16

// The decoded form of tkv_cache.
struct Cache {
    uint64_t pool;
    uint64_t page_bytes;
    uint32_t n_pages;
    uint32_t heads;
    uint32_t dim, group;
    uint32_t page_shift;   // log2(page_tokens)
    uint32_t record;       // bytes of 32 positions of one head
    uint32_t head_bytes;   // bytes of one head's positions of a page
    uint32_t magic;
    uint32_t reserved[20];
};
static_assert(sizeof(Cache) == 128, "cache descriptor must be 128 bytes");
static_assert(sizeof(tkv_cache) == 128, "tkv_cache must be 128 bytes");

enum Type : int32_t { kF16 = 0, kBf16 = 1, kF32 = 2 };

struct Tokens {
    void *data;
    int64_t token_stride, head_stride;  // elements
    int32_t type;
    int32_t wide;  // every 8 elements of a row can be read at once: 16-byte aligned
};

struct Batch {
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens;
    const int32_t *starts;  // nullptr: uniform new tokens each
    int64_t n_tokens;
    int32_t n_seq, table_width, max_new, uniform;
};

// Division by a number that the host knows: n / d = n * mul >> (31 + shift),
// exact for 0 <= n < 2^31.
struct Divisor {
    uint32_t mul;
    int32_t shift;
};

struct MoveArgs {  // append and read
    Cache c;
    Tokens k, v;
    Batch b;
    int32_t tiles;  // records that a sequence's new tokens can touch
};

struct AttendArgs {
    Cache c;
    Batch b;
    Tokens q, out;
    float *lse;
    float scale_log2;      // scale * log2(e)
    int32_t causal;
    int32_t group_heads;   // query heads of a key/value head
    int32_t rows;          // max_new * group_heads
    int32_t row_blocks;
    int32_t max_len;
    int32_t chunk_shift;   // a workgroup has at most 1 << chunk_shift positions
    int32_t n_split;
    int32_t even;          // the steps of all sequences are dealt evenly (Even), not in chunks
    int32_t groups;        // ... to so many workgroups
    int32_t cus;
    int32_t *dealt;        // [kEvenSeqs + 1]: the line's steps before each sequence, and a share's
    int32_t row_shift;     // log2 of a workgroup's rows
    float *part_o;         // [parts][rows][dim], parts [n_seq][heads][n_split], or as Even numbers them
    float *part_ml;        // [parts][rows][2]
    // with scores: what turns products into weights, and either the logarithms
    // of a few rows' products or the queries as the matrix unit takes them
    float *logits;         // [n_seq][heads][records of max_len][rows][32], or nullptr
    void *frag_q;          // fp16 [n_seq][heads][row tiles][dim/32 + 1][64 lanes][8]: q, and its sums over groups
    float *row_info;       // [n_seq][heads][row tiles][16][2]: factor, lse2
    int32_t row_tiles;
    Divisor by_heads, by_group_heads, by_row_blocks, by_split, by_rows;
    const float *scores_in;
    float *scores_out;
    int64_t score_stride;
};

struct EvictArgs {
    Cache c;
    Batch b;
    const float *scores;
    float *scores_out;
    int64_t score_stride;
    int32_t *kept;
    int32_t *lens_out;
    const int32_t *dst_table;
    int64_t dst_stride;
    int32_t dst_width, budget, recent, max_len;
};

// Launchers, one translation unit each; they return a hipError_t as int.
int launch_append(const MoveArgs &a, void *stream);
int launch_read(const MoveArgs &a, void *stream);
// row_tile: rows of a workgroup, 16 or 32 (its waves share the positions), 64
// or 128 (its waves share the rows)
int launch_attend_d64(const AttendArgs &a, int row_tile, void *stream);
int launch_attend_d96(const AttendArgs &a, int row_tile, void *stream);
int launch_attend_d128(const AttendArgs &a, int row_tile, void *stream);
int launch_attend_d256(const AttendArgs &a, int row_tile, void *stream);
int launch_combine(const AttendArgs &a, void *stream);
int launch_weigh(const AttendArgs &a, void *stream);  // of sequences without rows: the scores as they are
int launch_evict(const EvictArgs &a, void *stream);

}  // namespace tkv
