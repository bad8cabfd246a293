// tkv_rotate.h -- the rotation by positions on the way into the cache, and of
// the queries beside it.
//
// A pair (a, b) of channels becomes (a c - b s, b c + a s), c and s from the
// table's row of the token's position.  Each product and sum is rounded to fp32
// by itself, so that what is cached is what the formula says, bit for bit.
//
// Rows of 16-bit numbers go by units of 16 channels, 8 whole pairs: of pairs
// (i, i + dim / 2) two runs of 8 channels, else one of 16.  A lane has one unit
// of several heads' rows, so that it reads a token's cosines and sines once.
#pragma once

#include "tkv_format.h"

namespace tkv {

constexpr int kMoveWaves = kBlockThreads / 64;

// What of a number is cached.
__device__ __forceinline__ float limited(float y) { return y != y ? 0.0f : fminf(fmaxf(y, -kLimit), kLimit); }

// What a wave, or two, of append and read has: one record.
struct Unit {
    int seq, head, tile;   // record: positions 32 * tile ..
    int first, n;          // the sequence's first new position and their number
    int64_t start;         // row of the first
    char *rec;             // nullptr where the position's page does not exist
};

__device__ __forceinline__ bool unit_of(const MoveArgs &a, int unit, Unit &u) {
    u.head = unit % (int)a.c.heads;
    const int rest = unit / (int)a.c.heads;
    u.seq = rest / a.tiles;
    if (u.seq >= a.b.n_seq) return false;
    new_tokens(a.b, u.seq, u.start, u.n);
    u.first = a.b.lens[u.seq];
    if (u.first < 0 || u.n <= 0) return false;
    u.tile = u.first / kTile + rest % a.tiles;
    if ((int64_t)u.tile * kTile >= (int64_t)u.first + u.n) return false;
    const int page = page_at(a.b.table + u.seq * a.b.table_stride, a.b.table_width, a.c.n_pages,
                             u.tile >> (a.c.page_shift - 5));
    u.rec = page < 0 ? nullptr : record_at(a.c, page, u.head, u.tile);
    return true;
}

// Channels of the first and the second 8 of a unit.
__device__ __forceinline__ void unit_channels(const Rotation &r, int unit, int &c0, int &c1) {
    const bool halves = r.dim && !r.neighbours && unit < r.dim / 16;
    c0 = halves ? 8 * unit : 16 * unit;
    c1 = halves ? 8 * unit + r.dim / 2 : 16 * unit + 8;
}

// Where the table's row for a token begins, -1 where the table has none.  row: of
// the token tensors.
__device__ __forceinline__ int64_t turn_of(const Rotation &r, int64_t row, int64_t position) {
    if (r.positions) position = r.positions[row];
    return position >= 0 && position < r.n_positions ? position * r.stride : -1;
}

template <int N>
__device__ __forceinline__ void load_floats(const float *p, bool wide, float *out) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(p)[i];
            out[4 * i] = v.x, out[4 * i + 1] = v.y, out[4 * i + 2] = v.z, out[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = p[i];
    }
}

// The numbers of both members of a pair after the turn.
__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s) {
#pragma clang fp contract(off)
    const float x = a, y = b;
    a = x * c - y * s;
    b = y * c + x * s;
}

// E neighbouring channels of a key row, from channel ch, turned; row_at: where the row begins.
template <int E>
__device__ __forceinline__ void turn_few(const MoveArgs &a, int64_t turn_at, int64_t row_at, int ch, float (&x)[E]) {
    const Rotation &r = a.rot;
    const int half = r.dim / 2;
    const float *turn = r.table + turn_at;
    if (ch >= r.dim) return;
    if (r.neighbours) {
#pragma unroll
        for (int e = 0; e < E; e += 2) turn_pair(x[e], x[e + 1], turn[(ch + e) / 2], turn[half + (ch + e) / 2]);
        return;
    }
    const bool second = ch >= half;
    const int pair = second ? ch - half : ch, other = second ? ch - half : ch + half;
    float y[E], c[E], s[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        y[e] = elem_to_float(((const uint16_t *)a.k.data)[row_at + other + e], a.k.type);
        c[e] = turn[pair + e];
        s[e] = turn[half + pair + e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float first = second ? y[e] : x[e], last = second ? x[e] : y[e];
        turn_pair(first, last, c[e], s[e]);
        x[e] = second ? last : first;
    }
}

struct Turn {  // of a unit's 8 pairs
    float c[8], s[8];
    __device__ __forceinline__ void load(const Rotation &r, int64_t turn, int unit) {
        const float *row = r.table + turn;
        load_floats<8>(row + 8 * unit, r.wide, c);
        load_floats<8>(row + r.dim / 2 + 8 * unit, r.wide, s);
    }
    __device__ __forceinline__ void apply(bool neighbours, float (&x)[16]) const {
        if (neighbours) {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn_pair(x[i], x[8 + i], c[i], s[i]);
        }
    }
};

__device__ __forceinline__ void unit_floats(uint4 lo, uint4 hi, int type, float (&x)[16]) {
    if (type == kBf16) {
        raw_to_float<true>(lo, x);
        raw_to_float<true>(hi, x + 8);
    } else {
        raw_to_float<false>(lo, x);
        raw_to_float<false>(hi, x + 8);
    }
}

template <int D>
constexpr int kQueryHeads = 64 / (D / 16);  // rows that a wave has at once

// Waves of a token's queries in a launch of few tokens.
inline int query_waves(const MoveArgs &a, int64_t tokens, int heads_at_once) {
    if (tokens > kQueryTokens) return 1;
    const int waves = (a.rot.q_heads + heads_at_once - 1) / heads_at_once;
    return waves < kQueryWaves ? waves : kQueryWaves;
}

// The queries of one token by `waves` waves, of which this is one, AHEAD rows at a
// time.  `token` counts max_new for each sequence.  One row at a time in a step of
// few tokens, and as many waves as that takes: 32 sequences with 32 query heads
// of 128 channels 4.3 us, keys and values included, where a wave that had four
// rows at a time took 7.6; four where there are thousands of tokens, whose rows
// move at 5.0 TB/s (8 sequences of up to 4001, 410 MB).
template <int D, int AHEAD>
__device__ __forceinline__ void rotate_queries(const MoveArgs &a, int token, int wave, int waves, int lane) {
    constexpr int U = D / 16, HEADS = kQueryHeads<D>;  // units of a row
    const Rotation &r = a.rot;
    const int seq = token / a.b.max_new, i = token % a.b.max_new;
    if (seq >= a.b.n_seq) return;
    int64_t start;
    int n;
    new_tokens(a.b, seq, start, n);
    const int first = a.b.lens[seq];
    if (first < 0 || i >= n) return;
    const int64_t at_turn = turn_of(r, start + i, (int64_t)first + i);
    const int unit = lane % U, sub = lane / U;
    const bool turned = unit < r.dim / 16;
    if (at_turn < 0 || sub >= HEADS || (!turned && r.same)) return;
    Turn turn;
    if (turned) turn.load(r, at_turn, unit);
    int c0, c1;
    unit_channels(r, unit, c0, c1);
    const int64_t from = (start + i) * r.q.token_stride, to = (start + i) * r.q_out.token_stride;
    for (int h0 = sub + wave * HEADS * AHEAD; h0 < r.q_heads; h0 += waves * HEADS * AHEAD) {
        uint4 lo[AHEAD], hi[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t at = from + (int64_t)(h0 + k * HEADS) * r.q.head_stride;
            if (h0 + k * HEADS < r.q_heads) lo[k] = load8_raw(r.q, at + c0), hi[k] = load8_raw(r.q, at + c1);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (h0 + k * HEADS >= r.q_heads) break;
            float x[16];
            unit_floats(lo[k], hi[k], r.q.type, x);
            if (turned) turn.apply(r.neighbours, x);
            const int64_t at = to + (int64_t)(h0 + k * HEADS) * r.q_out.head_stride;
            store8(r.q_out, at + c0, x);
            store8(r.q_out, at + c1, x + 8);
        }
    }
}

}  // namespace tkv
