/*
 * tkv.h -- C ABI of libtkv: a paged key/value cache held in 4 bits, and the
 * operators of a language model's decoding loop on it, on AMD Instinct
 * MI355X (gfx950).
 *
 * A pool holds pages; a page holds `page_tokens` positions of every key/value
 * head.  32 positions of one head are one contiguous record, a multiple of
 * 128 bytes, so a page is a run of bytes that the tile copies of tmap.h move
 * like any other tensor (a u8 tensor of pages, one box per piece of a page).
 * A table names the pages of each sequence: position p of sequence b lies in
 * page table[b][p / page_tokens].
 *
 * Numbers.  A key or value element is scale * code + zero: code in 0..15,
 * scale and zero fp16, one pair for each position and each group of `group`
 * neighbouring channels.
 *
 * Record of 32 positions (dim = head_dim, W = dim / 32 words, groups =
 * dim / group; S = 2 where W > 4, else 1, and w = W / S):
 *   byte 0                    K codes, uint32 [2 halves][S][64 lanes][w]
 *   16 * dim                  V codes, the same shape
 *   32 * dim                  K pairs, fp16 [groups][32 positions][scale, zero]
 *   32 * dim + 128 * groups   V pairs, fp16 [groups][scale, zero][32 slots]
 * A word holds 8 codes; code j (0..7) is its nibble (j >> 1) + 4 * (j & 1).
 * With lane = 16 * g + m, word i of the half (i = S-index * w + last index):
 *   K: position 16 * half + m, channel 32 * i + 8 * g + j
 *   V: channel 16 * (half * W + i) + m, position 4 * g + (j & 3) + 16 * (j >> 2)
 * and slot 8 * g + j of the V pairs is that same position.  This is the order
 * in which v_mfma_f32_16x16x32_f16 takes its operands: attention reads words in
 * whole wave-wide runs, and a lane's words are its part of the operand.
 *
 * Conventions for every call:
 *   - Pointers are HIP device pointers, unless they are `tkv_cache *`.  The
 *     library takes no ownership and keeps nothing from one call to the next.
 *   - Calls enqueue on `hip_stream` (NULL: the default stream) and return
 *     without waiting.  They allocate no memory and can be captured into a
 *     HIP graph.  Argument errors are reported before anything is launched.
 *   - Statuses are tmap.h's; tkv_last_error_detail() says what was wrong.
 *   - `n_seq` sequences.  `table` is int32 [n_seq][table_stride], of which
 *     `table_width` entries of each row are read; `lens` is int32 [n_seq].
 *     New tokens are packed: sequence b's are rows starts[b] .. starts[b+1]-1
 *     of the token tensors (`starts` int32 [n_seq + 1], 0 first and n_tokens
 *     last), at most max_new of them; with starts == NULL every sequence has
 *     n_tokens / n_seq.  Rows past max_new are left alone.
 *   - A row of the table holds fewer than 2^31 - 2^17 positions.  A call is
 *     refused whose sequences and heads have together more records, rows or
 *     positions than launches of 2^32 threads hold.
 *   - A length below 0 counts as 0 to attention and eviction; append and read
 *     leave such a sequence alone.
 *   - Positions whose page is outside the pool (< 0 or >= n_pages), or past
 *     the table's width, do not exist: they are never read or written.
 *   - No two sequences may name the same page where a call writes to it.
 */
#ifndef TKV_H
#define TKV_H

#include "tmap.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 128 opaque bytes, filled by tkv_encode. */
typedef struct __attribute__((aligned(64))) tkv_cache {
    uint64_t opaque[16];
} tkv_cache;

/*
 * tkv_encode -- describe a pool.  Host-only: needs no GPU.
 *   pool         device, n_pages * tkv_page_bytes bytes, 16-byte aligned
 *   n_pages      1 .. 2^31 - 2
 *   n_heads      key/value heads, 1 .. 65535
 *   head_dim     64, 96, 128 or 256
 *   page_tokens  a power of two, 32 .. 1024
 *   group        32, 64 or 128, a divisor of head_dim
 */
tmap_status tkv_encode(tkv_cache *cache, void *pool, int64_t n_pages, uint32_t n_heads, uint32_t head_dim,
                       uint32_t page_tokens, uint32_t group);

/* Bytes of one page (all heads): n_heads * page_tokens / 32 *
 * (32 * head_dim + 256 * head_dim / group).  0 for a cache never encoded. */
uint64_t tkv_page_bytes(const tkv_cache *cache);

/* A strided tensor of 16- or 32-bit elements [tokens][heads][head_dim], the
 * last dimension contiguous; strides in elements.  Rows that a call writes lie
 * apart, and apart from what it reads, but that out may be q itself. */
typedef struct tkv_tokens {
    void *data;
    int64_t token_stride, head_stride;
    int32_t dtype; /* TMAP_F16, TMAP_BF16; TMAP_F32 too where tkv_read writes */
} tkv_tokens;

typedef struct tkv_batch {
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens;
    const int32_t *starts; /* NULL: n_tokens / n_seq each */
    int64_t n_tokens;
    int32_t n_seq, table_width, max_new;
} tkv_batch;

/*
 * tkv_append -- quantise new keys and values and put them at positions
 * lens[b], lens[b] + 1, .. of each sequence.  In each group of channels
 *   x      = 0 for NaN, else clamped to +-32000
 *   zero   = fp16(min x),  scale = fp16((max x - min x) / 15)   (the
 *            difference and the quotient in fp32)
 *   code   = (x - zero) / scale to the nearest whole number, ties to even,
 *            within 0..15 (decided exactly); 0 where scale is 0
 * k and v are fp16 or bf16, of the same type.  What is cached is finite.
 */
tmap_status tkv_append(const tkv_cache *cache, const tkv_tokens *k, const tkv_tokens *v, const tkv_batch *batch,
                       void *hip_stream);

/*
 * tkv_read -- the reverse: positions lens[b], lens[b] + 1, .. of each
 * sequence as numbers (computed in fp32, rounded once), in rows starts[b],
 * starts[b] + 1, ..  Positions that do not exist read as 0.
 */
tmap_status tkv_read(const tkv_cache *cache, const tkv_tokens *k, const tkv_tokens *v, const tkv_batch *batch,
                     void *hip_stream);

/*
 * tkv_attend -- attention of the new tokens' queries over the cache:
 *   out[t][a] = sum_p softmax_p(scale * q[t][a] . K[p]) V[p],  query head a
 * on key/value head a / (q_heads / n_heads), lse the logarithm of the
 * softmax's denominator.  lens[b] counts every cached position, the new
 * tokens' own included.  With causal, the i-th of n new tokens sees positions
 * below lens[b] - n + 1 + i, else all lens[b]; lens[b] itself counts there,
 * also where it is more than the table holds.  A row that sees no position
 * gives 0 and lse -inf.
 *
 * With scores_out, also scores_out[b][h][p] = scores_in[b][h][p] + the sum
 * over the sequence's new tokens and the query heads of h of position p's
 * attention weight, for p < lens[b] (other places are left alone).
 * scores_in may be scores_out, or NULL for 0.
 *
 * Products of q with codes are exact up to their fp32 sum; softmax, sums and
 * K's scales are fp32; a weight, and a V element's scale * (code - 8), are
 * rounded to fp16 once each on their way into the matrix unit.  A row whose
 * logarithms to base 2 all lie below -10^30 counts as one that sees nothing.
 */
typedef struct tkv_attend_args {
    tkv_tokens q, out;        /* [n_tokens][q_heads][head_dim], fp16 or bf16, one type  */
    float *lse;               /* [n_tokens][q_heads]                                    */
    const float *scores_in;   /* [n_seq][n_heads][score_stride], or NULL                */
    float *scores_out;        /* the same shape, or NULL                                */
    int64_t score_stride;     /* at least max_len where scores are used                 */
    int32_t q_heads;          /* a multiple of n_heads                                  */
    int32_t max_len;          /* no lens[b] is larger; positions past it are not seen   */
    float scale;
    int32_t causal;
    void *workspace;          /* tkv_attend_workspace bytes, 16-byte aligned            */
    uint64_t workspace_bytes;
} tkv_attend_args;
tmap_status tkv_attend(const tkv_cache *cache, const tkv_attend_args *args, const tkv_batch *batch,
                       void *hip_stream);

/* Workspace that tkv_attend needs for these arguments (pointers are not
 * read; a gfx950 device must be current, as the split of the work goes by
 * its number of compute units).  Smaller sizes may need more, since fewer
 * workgroups are given shorter pieces. */
tmap_status tkv_attend_workspace(const tkv_cache *cache, const tkv_attend_args *args, const tkv_batch *batch,
                                 uint64_t *bytes);

/* Enough for these arguments and for every call with no more sequences, new
 * tokens (n_tokens and max_new) and positions (max_len and what the table
 * holds), with scores if these have them: to allocate once. */
tmap_status tkv_attend_workspace_bound(const tkv_cache *cache, const tkv_attend_args *args, const tkv_batch *batch,
                                       uint64_t *bytes);

/*
 * tkv_evict -- shrink sequences to `budget` positions for each head: the
 * last min(recent, budget) positions stay, and of those before them the
 * budget - recent with the largest scores (NaN counts as lowest, the lowest
 * position first among equals).  A sequence of at most budget positions
 * keeps all.  What stays keeps its order and is written, with its scores, to
 * positions 0, 1, .. of the pages that dst_table names; the source pages are
 * not changed, and may not be among those.
 *   scores      [n_seq][n_heads][score_stride]
 *   scores_out  [n_seq][n_heads][budget]: the kept positions', then 0
 *   kept        int32 [n_seq][n_heads][budget]: kept positions, then -1
 *   lens_out    int32 [n_seq]: min(lens[b], budget); may be lens, and else
 *               may not overlap it
 * scores_out and scores may not overlap.  batch: table, lens and n_seq are
 * used.
 */
typedef struct tkv_evict_args {
    const float *scores;
    float *scores_out;
    int64_t score_stride;
    int32_t *kept;
    int32_t *lens_out;
    const int32_t *dst_table;  /* [n_seq][dst_stride], dst_width entries of each row */
    int64_t dst_stride;
    int32_t dst_width;
    int32_t budget, recent;
    int32_t max_len;           /* no lens[b] is larger; at most score_stride */
} tkv_evict_args;
tmap_status tkv_evict(const tkv_cache *cache, const tkv_evict_args *args, const tkv_batch *batch, void *hip_stream);

/* Thread-local text on the last failure of a call on this thread, "" after
 * success. */
const char *tkv_last_error_detail(void);

#ifdef __cplusplus
}
#endif
#endif /* TKV_H */
