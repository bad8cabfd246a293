// tkv_attend.h -- attention over the cache, and the attention weights summed over
// query rows.
//
// Rows.  A sequence's new tokens times the query heads of one key/value head
// are that head's rows (row = token * group_heads + head in its group); a
// wave holds NT tiles of 16 of them.
//
// Products.  v_mfma_f32_16x16x32_f16 with the cache as the left operand:
// S^T = K Q^T, so a lane holds 4 positions of one row of each 16, and
// O^T = V^T P^T, whose right operand wants 8 positions of one row in a lane:
// the same ones, in the order in which the record holds V's words.  So weights
// go from one product to the next without a move between lanes.
//
// Numbers.  With code c, scale s and zero z of a position and channel group,
//   q . k = sum over groups of s * (q . c) + z * (sum of q)
//   p . v = sum over positions of p * (s * c), plus p * z
// q . c is a product of fp16 numbers, exact up to its fp32 sum (a bf16 row of
// q is first scaled by a power of two to a largest magnitude in [2^14, 2^15),
// so what fp16 drops is below 2^-38 of that largest); s and z come in at fp32.
// Where a record is unpacked for few rows, its codes are 64 too large, and the
// sum starts at -64 * (sum of q).  For V, s * (c - 8) is
// rounded to fp16 (half a step is 2^-11 of it, relative; with c itself, whose
// numbers lie on one side of zero, the error of the sum was 3 times as
// large), and so is p.  The sums of p * (z + 8 s) are two more rows of the
// product: the groups' scales and zeros, as they lie, are rows of an operand,
// and a row of ones gives the sum of the rounded p, by which the output is
// divided: what rounding adds to a weight it then adds to both.  (256
// channels in groups of 32 fill all 16 rows, and are divided by the sum of the
// p before rounding.)  lse goes by the p before rounding.
//
// Softmax in one pass: each row keeps a reference m and sums exp2(y - m + 7)
// of its scaled products y.  m moves only when a y passes m + 8, which keeps
// the weights below 2^15 in fp16 and, fp16's smallest step being 2^-24, drops
// only what is below 2^-31 of the largest; the four lanes of a row compare
// notes only then.
//
// Split.  A workgroup takes a chunk of positions of one (sequence, head, block
// of rows), or an even share of all positions (Even; the host's plan says when);
// a second kernel joins the partial sums.  (To
// have the last workgroup of a row block join them instead took 55 us where the
// two kernels take 22: a release and an acquire at the agent's scope write the
// L2 back, in every workgroup.)
//
// Few rows, attend_kernel: all four waves hold the same rows, up to 32, take
// every fourth record, each with its own m, and are joined through LDS at the
// end.  What bounds it is the cache, read once.  A wave's records land in a
// ring of two in LDS, asked for two ahead by loads that name no register: a
// compute unit holds 16 waves, 32 records on their way, and with 128 channels
// 128 registers a wave are enough for that.  All loads of the loop go by that
// ring, as one load of another kind (a spilled register, a table entry) waits
// for all before it: 325 us against 295 in the first of these, in chunks.
// Measured, 128 channels in groups of 64, 8 heads of 4 rows: 64 sequences of
// 4096 to 32768 positions 266 us, 5.2 TB/s, where a loop that only reads
// records has 6.0; 16 of up to 4099 positions 17 us, 2.6 TB/s, of which 5.5 are
// a block's start, its rows' way into operands and its end; a single one of 57
// positions 5.7 us.
// More rows: tkv_rows.h, and tkv_rows8.h for 8 bits.
//
// 8 bits (GROUP 0).  A code becomes an fp16 number exactly (448 and the smallest
// subnormal are within fp16), so q . k is summed in units of the record's power
// of two, a factor of its logarithms, and only a row's weights are rounded.  The
// values are multiplied in units of the largest power that the wave has met: one
// that is larger shrinks the sums so far, by a power of two; codes of a smaller
// one are multiplied with the quotient, exactly where it is 2^-15 or more, and
// else an error of 2^-25 of a unit at most remains, 2^-32 of the largest value
// in that record.  128 channels, 8 heads of 4
// rows: 64 sequences of up to 32768 positions 434 us, 5.6 TB/s; 16 of up to 4099
// 21 us and the joining 4; one of 57 6.2 us.
//
// Window.  Rows see the last positions before their border and a few first ones.
// A sequence's seen positions are numbered through without the gap between (View:
// places), in whole records, so that chunks and even shares split what is seen
// and nothing else; the mask is asked for where a record holds a row's border,
// first or last.  64 sequences of up to 32768, a window of 4096: 102 us and the
// joining 5, 5.3 TB/s.  In 4 bits the window has kernels of its own (WIN), with
// 24 registers more: without a window they keep the registers that they had.
#pragma once

#include "tkv_format.h"

namespace tkv {

constexpr int kAttendWaves = kBlockThreads / 64;
constexpr float kFar = -1e30f;  // reference of a row that has seen nothing
constexpr float kLift = 7.0f;   // weights are held times 2^7
constexpr float kSlack = 8.0f;

// Rows 0, 1, 2, .. of the operand of scales and zeros are scale and zero of
// each group as they lie in the record; then comes a row of ones, if there is
// room, then zeros.
template <int D, int GROUP>
constexpr bool kOnes = 2 * Format<D, GROUP>::NG < 16;

template <int D, int GROUP>
__device__ __forceinline__ h8 one_row(int lane) {
    const _Float16 x = (lane & 15) == 2 * Format<D, GROUP>::NG ? (_Float16)1.0f : (_Float16)0.0f;
    return (h8){x, x, x, x, x, x, x, x};
}

// A sequence's extent and the rows of one block.
struct Extent {
    int64_t start;  // first row of its tokens
    int n, len, rows;
    int sees;  // causal: the first new token sees positions below this, by the length before it is cut to what exists
    __device__ __forceinline__ Extent(const AttendArgs &a, int seq) {
        const int given = a.b.lens[seq], l = given < 0 ? 0 : given;
        new_tokens(a.b, seq, start, n);
        len = l < a.max_len ? l : a.max_len;  // max_len is at most what the table holds
        sees = l - n + 1;
        rows = n * a.group_heads;
    }
    // positions below this are seen by the i-th new token
    __device__ __forceinline__ int limit(const AttendArgs &a, int i) const {
        return a.causal && sees + i < len ? sees + i : len;
    }
    // the same by the length before it is cut: a window counts from here
    __device__ __forceinline__ int border(const AttendArgs &a, int i) const { return sees + (a.causal ? i : n - 1); }
};

// What of a sequence some rows see, and in which order it is gone over.  With a
// window, rows of the tokens i0 .. i1 see positions below gap_at, the first ones
// that stay visible, and from gap_at + gap on: places 0, 1, .. below `span` count
// these.  gap and gap_at are whole records.  Without a window a place is a
// position.
template <bool WIN>
struct View : Extent {
    __device__ __forceinline__ View(const AttendArgs &a, int seq) : Extent(a, seq) {}
    __device__ __forceinline__ int span() const { return len; }
    __device__ __forceinline__ int position(int place) const { return place; }
    __device__ __forceinline__ int place(int position) const { return position; }
    __device__ __forceinline__ void narrow_to_block(const AttendArgs &, int) {}
    __device__ __forceinline__ bool windowed(const AttendArgs &, int, int) const { return false; }
};

constexpr int kManyRowShift = 6;  // of a workgroup whose waves have rows of their own

template <>
struct View<true> : Extent {
    int gap_at, gap, all;
    __device__ __forceinline__ View(const AttendArgs &a, int seq) : Extent(a, seq) {
        gap_at = gap = 0;
        all = len;
        if (a.window) narrow(a, 0, n - 1);
    }
    __device__ __forceinline__ int span() const { return all; }
    __device__ __forceinline__ void narrow(const AttendArgs &a, int i0, int i1) {
        const int64_t from = (int64_t)border(a, i0) - a.window;
        const int low = from > 0 ? (int)from & -kTile : 0, high = limit(a, i1), first = (a.sinks + kTile - 1) & -kTile;
        gap_at = gap = 0;
        all = high;
        if (low > first) {
            gap_at = first;
            gap = low - first;
            all = place(high);
        }
    }
    __device__ __forceinline__ int position(int place) const { return place + (place < gap_at ? 0 : gap); }
    // of the first position from `position` on that has one
    __device__ __forceinline__ int place(int position) const {
        return position < gap_at ? position : position - gap > gap_at ? position - gap : gap_at;
    }
    // to the tokens of a block of rows, where a workgroup has many rows: few stay with all of the sequence's tokens
    __device__ __forceinline__ void narrow_to_block(const AttendArgs &a, int block) {
        if (!a.window || a.row_shift < kManyRowShift) return;
        const int first = block << a.row_shift, last = first + (1 << a.row_shift) < rows ? first + (1 << a.row_shift) : rows;
        narrow(a, divided(first, a.by_group_heads), divided(last - 1, a.by_group_heads));
    }
    // whether one of some rows, the last of which is of token i1, does not see a record for its window
    __device__ __forceinline__ bool windowed(const AttendArgs &a, int i1, int record) const {
        return a.window && border(a, i1) - record > a.window && record + kTile > a.sinks;
    }
};

// What a row sees: positions below its limit, and with a window only the last of
// those below its border and the first ones.
template <bool WIN>
struct Sight {
    int until;  // the limit, or with a window the border
    __device__ __forceinline__ void load(const AttendArgs &a, const Extent &e, int row) {
        const int i = divided(row, a.by_group_heads);
        until = row >= e.rows ? 0 : WIN ? e.border(a, i) : e.limit(a, i);
    }
    // The products of a record that the row does not see become -inf: of a lane's 16 positions 4 h + 0..3 of each 8.  Of a
    // record that is gone no row sees anything.
    template <class X>
    __device__ __forceinline__ void mask(const AttendArgs &a, const Extent &e, int at, bool gone, int h, X &x) const {
        static_assert(WIN, "of a border");
        const int first = at + 4 * h, limit = until < e.len ? until : e.len;
        uint32_t seen = gone ? 0 : below(limit - first);
        if (a.window) {
            const int64_t low = (int64_t)until - a.window - first;
            seen &= ~below(low < 0 ? 0 : low > kTile ? kTile : (int)low) | below(a.sinks - first);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t all = (uint32_t)((int32_t)(seen << (31 - j)) >> 31);  // of bit j
            const float y = x[j];  // a bit cast of a vector's element would be one of its first
            x[j] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, y) & all) | (0xFF800000u & ~all));
        }
    }
    // which of the 16 are less than n from the first one
    static __device__ __forceinline__ uint32_t below(int n) {
        n = n < 0 ? 0 : n > kTile ? kTile : n;
        const int part = n & 7;
        return (1u << (4 * (n >> 3) + (part < 4 ? part : 4))) - 1;
    }
    // (the difference counts where the border is above the position)
    __device__ __forceinline__ bool sees(const AttendArgs &a, const Extent &e, int position) const {
        if (!WIN) return position < until;
        const bool out = a.window && (int)((uint32_t)until - (uint32_t)position) > a.window && position >= a.sinks;
        return position < until && position < e.len && !out;
    }
};

// The chunks of so many places: as few as the launch's chunk allows, of equal
// length up to whole steps of the workgroup.
constexpr int kStep = kTile * kAttendWaves;
struct Chunks {
    int size, n;
    __device__ __forceinline__ Chunks(const AttendArgs &a, int len) {
        const int steps = (len + kStep - 1) / kStep;
        int each = (1 << a.chunk_shift) / kStep, parts = (len + (1 << a.chunk_shift) - 1) >> a.chunk_shift;
        if (parts > 1) {
            each = over(steps, parts);
            parts = over(steps, each);
        }
        size = each * kStep;
        n = parts > 1 ? parts : 1;
    }
    // p / q rounded up, of numbers below 2^24: the quotient in fp32 is one off at most
    static __device__ __forceinline__ int over(int p, int q) {
        int r = (int)((float)p * __builtin_amdgcn_rcpf((float)q));
        r -= (r - 1) * q >= p ? 1 : 0;
        return r + (r * q < p ? 1 : 0);
    }
};

// An even split: the steps (kTile * kAttendWaves positions) of all row blocks
// of all sequences in a line, cut into equal shares, one for each workgroup.  A
// share may span several row blocks, and a row block several shares: such a
// piece's partial sums are part (row block's number + share's number), which no
// two pieces have in common.  What a piece costs beside its steps stands in the
// line as kLead steps before each row block's own.
struct Even {
    static constexpr int kSeqs = kEvenSeqs / 64;  // of a lane
    static constexpr int kLead = 1;
    int first[kSeqs];  // steps of the sequences before each
    int total, share;
    template <bool WIN>
    static __device__ __forceinline__ int steps(const View<WIN> &e) {
        return e.span() > kStep ? (e.span() + kStep - 1) / kStep : 1;
    }
    static __device__ __forceinline__ int blocks(const AttendArgs &a, const Extent &e) {
        return (e.rows + (1 << a.row_shift) - 1) >> a.row_shift;
    }
    template <bool WIN>
    static __device__ __forceinline__ int all(const AttendArgs &a, const View<WIN> &e) {
        return (int)a.c.heads * blocks(a, e) * (steps(e) + kLead);
    }
    template <bool WIN>
    __device__ __forceinline__ void load(const AttendArgs &a, int lane) {
        int sum = 0, most = 0, mine[kSeqs];
#pragma unroll
        for (int k = 0; k < kSeqs; ++k) {
            const int seq = kSeqs * lane + k;
            const View<WIN> e(a, seq < a.b.n_seq ? seq : a.b.n_seq - 1);
            mine[k] = seq < a.b.n_seq ? all(a, e) : 0;
            most = most > steps(e) ? most : steps(e);
        }
#pragma unroll
        for (int k = 0; k < kSeqs; ++k) {
            first[k] = sum;
            sum += mine[k];
        }
        int upto = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int x = __shfl_up(upto, d);
            upto += lane >= d ? x : 0;
        }
#pragma unroll
        for (int k = 0; k < kSeqs; ++k) first[k] += upto - sum;
        total = __builtin_amdgcn_readlane(upto, 63);
        // at least 512 positions, if any row block has so many
        const int least = (__any(most >= 4) ? 4 : __any(most >= 2) ? 2 : 1) + kLead;
        share = (int)(((uint32_t)total + (uint32_t)a.groups - 1) / (uint32_t)a.groups);
        share = share < least ? least : share;
    }
    // for the joining kernel
    __device__ __forceinline__ void store(const AttendArgs &a, int lane) const {
#pragma unroll
        for (int k = 0; k < kSeqs; ++k) a.dealt[kSeqs * lane + k] = first[k];
        if (lane == 0) a.dealt[kEvenSeqs] = share;
    }
    __device__ __forceinline__ int first_of(int seq) const {
        int r = 0;
#pragma unroll
        for (int k = 0; k < kSeqs; ++k) {
            const int x = __shfl(first[k], seq / kSeqs);
            r = seq % kSeqs == k ? x : r;
        }
        return r;
    }
    // the sequence that a step is in: the last one that begins at or before it
    __device__ __forceinline__ int seq_of(int step) const {
        int n = 0;
#pragma unroll
        for (int k = 0; k < kSeqs; ++k) n += __popcll(__ballot(first[k] <= step));
        return n - 1;
    }
};

// Table entries of up to 64 neighbouring pages, one in each lane.
struct Pages {
    int mine, base;
    __device__ __forceinline__ void load(const AttendArgs &a, const int32_t *row, int first, int lane) {
        base = first;
        mine = page_at(row, a.b.table_width, a.c.n_pages, first + lane);
    }
    __device__ __forceinline__ int get(const AttendArgs &a, const int32_t *row, int index, int lane) {
        if (index - base >= 64) load(a, row, index, lane);
        return __builtin_amdgcn_readlane(mine, index - base);
    }
};

// The 8-bit format's: of codes alone.
template <int D, int NT>
__device__ __forceinline__ void products8(const char *rec, int lane, const h8 (&q)[NT][D / 32], float (&x)[NT][8]) {
    using F = Format<D, 0>;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        f4 acc[NT];
#pragma unroll
        for (int c = 0; c < F::W; ++c) {
            const h8 key = codes8(*reinterpret_cast<const uint2 *>(rec + codes8_at(half * F::W + c, lane)), 1.0f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[nt][c], c ? acc[nt] : (f4){0, 0, 0, 0}, 0, 0, 0);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][4 * half + i] = acc[nt][i];
    }
}

// Products of a record's 32 positions with the wave's rows, in fp32:
// x[nt][4 * half + i] for position 16 half + 4 g + i.  first: -kPlus * qsum, four times.
template <int D, int GROUP, int NT>
__device__ __forceinline__ void products(const char *rec, int lane, const h8 (&q)[NT][D / 32],
                                         const float (&qsum)[NT][D / GROUP], const f4 (&first)[NT][D / GROUP],
                                         float (&x)[NT][8]) {
    using F = Format<D, GROUP>;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t w[F::W];
#pragma unroll
        for (int s = 0; s < F::S; ++s)
            load_words<F::WV>(rec + ((half * F::S + s) * 64 + lane) * (F::WV * 4), &w[s * F::WV]);
        f4 acc[NT][F::NG];
#pragma unroll
        for (int c = 0; c < F::W; ++c) {
            const h8 key = codes_plus(w[c]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                acc[nt][c / F::KG] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    key, q[nt][c], c % F::KG ? acc[nt][c / F::KG] : first[nt][c / F::KG], 0, 0, 0);
        }
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) {
            // (scale, zero) of positions 16 half + 4 g + 0..3
            const h8 pair = *reinterpret_cast<const h8 *>(rec + F::KP + (grp * kTile + 16 * half + 4 * (lane >> 4)) * 4);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y = fmaf((float)pair[2 * i + 1], qsum[nt][grp], grp ? x[nt][4 * half + i] : 0.0f);
                    x[nt][4 * half + i] = fmaf((float)pair[2 * i], acc[nt][grp][i], y);
                }
        }
    }
}

// Sum and maximum over the four lanes of a row: each swap of lanes leaves a
// lane with its own number and that of the one 16, or 32, away.
// (From assembly: given one number twice, the compiler takes the builtin's two
// results for one.  The swap waits for what a VALU has just written.)
template <class Op>
__device__ __forceinline__ float over_groups(float v, Op op) {
    float a = v, b = v;
    asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(a), "+v"(b));
    a = b = op(a, b);
    asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(b));
    return op(a, b);
}
__device__ __forceinline__ float over_groups_sum(float v) {
    return over_groups(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float over_groups_max(float v) {
    return over_groups(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float over_rows_sum(float v) {  // over 16 neighbouring lanes, by rotations
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 15, 15, true));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x124, 15, 15, true));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x122, 15, 15, true));
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x121, 15, 15, true));
}
// Four channels of an output row, and with the first ones its lse.
__device__ __forceinline__ void write_row(const AttendArgs &a, const Extent &e, int seq, int head, int row, int channel,
                                          f4 y, float best, float sum) {
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    int rest = row;
    const int i = divide(rest, a.group_heads, a.by_group_heads), hq = head * a.group_heads + rest;
    store4(a.out, (e.start + i) * a.out.token_stride + hq * a.out.head_stride + channel, y * inv);
    if (channel == 0) {
        const float log_sum = best - kLift + log2f(sum);  // log2(0) = -inf: nothing seen
        a.lse[(e.start + i) * (a.c.heads * a.group_heads) + hq] = log_sum * 0.69314718056f;
        if (a.row_info && (sum > 0.0f || sum != sum)) {
            const int64_t tile = ((int64_t)seq * a.c.heads + head) * a.row_tiles + row / 16;
            a.row_info[(tile * 16 + row % 16) * 2 + 1] = log_sum;
        }
    }
}

// Rows of one (sequence, head) as the right operand: lane (g, n) of a tile
// holds channels 32 c + 8 g .. of row r.
template <int D, int GROUP>
struct Row {
    uint4 raw[D / 32];
    __device__ __forceinline__ void load(const AttendArgs &a, const Extent &e, int head, int r, int g, bool live) {
        r = live ? r : 0;  // the first row is read for one that is not there, and dropped
        const int i = divide(r, a.group_heads, a.by_group_heads), hq = head * a.group_heads + r;
        const int64_t row = (e.start + i) * a.q.token_stride + hq * a.q.head_stride + 8 * g;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) raw[c] = load8_raw(a.q, row + 32 * c);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            raw[c] = live ? raw[c] : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void wait() {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) asm volatile("" : "+v"(raw[c].x), "+v"(raw[c].y), "+v"(raw[c].z), "+v"(raw[c].w));
    }
    // q, its sums over the groups of channels, and what turns products into
    // logarithms to base 2: at least the smallest normal number, as masked
    // products are -inf.
    template <bool BF16>
    __device__ __forceinline__ void operand(const AttendArgs &a, h8 (&q)[D / 32], float (&qsum)[Format<D, GROUP>::NG],
                                            float &factor) const {
        using F = Format<D, GROUP>;
        const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0;  // moves into q
        float x[F::W][8], top = 0.0f;
#pragma unroll
        for (int c = 0; c < F::W; ++c) {
            raw_to_float<BF16>(make_uint4(raw[c].x ^ sign, raw[c].y ^ sign, raw[c].z ^ sign, raw[c].w ^ sign), x[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (BF16) top = fmaxf(top, fabsf(x[c][j]));
        }
        int power = 0;
        if constexpr (BF16) {
            top = over_groups_max(top);
            if (top > 0.0f && top < __builtin_inff()) power = 15 - __builtin_amdgcn_frexp_expf(top);
        }
        const float f = fabsf(ldexpf(a.scale_log2, -power));
        factor = fminf(fmaxf(f, 0x1p-126f), 0x1.fffffep127f);
#pragma unroll
        for (int c = 0; c < F::W; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) q[c][j] = (_Float16)(BF16 ? ldexpf(x[c][j], power) : x[c][j]);
        if constexpr (GROUP != 0) {
            const h8 ones = {1, 1, 1, 1, 1, 1, 1, 1};
#pragma unroll
            for (int grp = 0; grp < F::NG; ++grp) {
                f4 sum = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < F::KG; ++c)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, q[grp * F::KG + c], sum, 0, 0, 0);
                qsum[grp] = sum[0];
            }
        }
    }
};

// The sums of a row's q over the groups of channels as an operand: three fp16
// numbers that add up to a sum, in units of 2^kSumBits, in the lanes of g = 0, 1
// and 2, group j in place j.  Its left operand is the zeros of a position.
constexpr int kSumBits = 8;

template <int D, int GROUP>
__device__ __forceinline__ h8 sum_parts(const float (&qsum)[D / GROUP], int g) {
    h8 r = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int grp = 0; grp < D / GROUP; ++grp) {
        float y = qsum[grp] * (1.0f / (1 << kSumBits));
        const _Float16 a = (_Float16)y;
        y -= (float)a;
        const _Float16 b = (_Float16)y;
        const _Float16 c = (_Float16)(y - (float)b);
        r[grp] = g == 0 ? a : g == 1 ? b : g == 2 ? c : (_Float16)0.0f;
    }
    return r;
}
// what turns products in those units into logarithms
__device__ __forceinline__ float sums_factor(float factor) {
    return fminf(factor * (float)(1 << kSumBits), 0x1.fffffep127f);
}

// Where the scores kernels find a tile of 16 rows and what belongs to it.
template <int D, int GROUP>
__device__ __forceinline__ void keep_rows(const AttendArgs &a, int64_t tile, int lane, const h8 (&q)[D / 32], h8 sums,
                                          float factor) {
    using F = Format<D, GROUP>;
    if (a.frag_q) {
        h8 *to = (h8 *)a.frag_q + tile * ((F::W + 1) * 64);
#pragma unroll
        for (int c = 0; c < F::W; ++c) to[c * 64 + lane] = q[c];
        to[F::W * 64 + lane] = sums;
    }
    // a row without positions weighs nothing: its logarithm stays at inf
    if (lane < 16) *reinterpret_cast<float2 *>(a.row_info + (tile * 16 + lane) * 2) = make_float2(factor, __builtin_inff());
}

// What a row's running softmax holds, and one step of it: x (32 positions'
// products) become weights p; o and z are scaled where the reference moves.
template <int D, int GROUP>
struct Softmax {
    float m, l;
    f4 o[D / 16], z;
    __device__ __forceinline__ void clear() {
        m = kFar;
        l = 0.0f;
        z = (f4){0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[c] = (f4){0, 0, 0, 0};
    }
    template <int N>
    static __device__ __forceinline__ float top(const float (&x)[N]) {
        float t[2] = {x[0], x[1]};  // maxima of three
#pragma unroll
        for (int j = 2; j < N; j += 4) {
            t[0] = fmaxf(fmaxf(t[0], x[j]), x[j + 1]);
            if (j + 2 < N) t[1] = fmaxf(fmaxf(t[1], x[j + 2]), x[j + 3]);
        }
        return fmaxf(t[0], t[1]);
    }
    __device__ __forceinline__ void grow(float y) {  // y: the largest logarithm of the lane's positions
        const float t = over_groups_max(y);
        const float m1 = t > m + kSlack ? t : m;
        const float f = __builtin_amdgcn_exp2f(m - m1);
        m = m1;
        l *= f;
        z *= f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[c] *= f;
    }
    template <int RECS>
    __device__ __forceinline__ void weights(const float (&x)[8 * RECS], float factor, h8 (&p)[RECS]) {
        const float lift = kLift - m;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8 * RECS; ++j) {
            const float w = __builtin_amdgcn_exp2f(fmaf(x[j], factor, lift));
            sum += w;
            p[j >> 3][j & 7] = (_Float16)w;
        }
        l += sum;
    }
    // after the last position: l whole in every lane, o what a division by l makes the output.  power: the 8-bit
    // format's o are in units of it
    __device__ __forceinline__ void finish(int lane, float power = 1.0f) {
        using F = Format<D, GROUP>;
        l = over_groups_sum(l);
        if constexpr (GROUP == 0) {
            const float ratio = z[0] > 0.0f ? l / z[0] * power : power;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[c] *= ratio;
        } else {
            float ratio = 1.0f;
            if constexpr (kOnes<D, GROUP>) {
                const float rounded = __shfl(z[(2 * F::NG) & 3], 16 * (2 * F::NG / 4) + (lane & 15));
                ratio = rounded > 0.0f ? l / rounded : 1.0f;
            }
#pragma unroll
            for (int grp = 0; grp < F::NG; ++grp) {
                const int from = 16 * (grp / 2) + (lane & 15);
                const float zero = fmaf(8.0f, __shfl(z[(2 * grp) & 3], from), __shfl(z[(2 * grp + 1) & 3], from));
#pragma unroll
                for (int c = grp * F::VG; c < (grp + 1) * F::VG; ++c) o[c] = (o[c] + zero) * ratio;
            }
        }
    }
    // o in units of a power of two of its own
    __device__ __forceinline__ void rescale(float f) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[c] *= f;
    }
};

// What a workgroup of the attention kernels has to do.
__device__ __forceinline__ void place(const AttendArgs &a, int &block, int &split, int &head, int &seq) {
    block = blockIdx.x;
    split = divide(block, a.row_blocks, a.by_row_blocks);
    head = divide(split, a.n_split, a.by_split);
    seq = divide(head, (int)a.c.heads, a.by_heads);
}

// Few rows: the four waves share them and take every fourth record.  A wave
// has a ring of two records in LDS, which its loads fill without passing
// through registers: while it works on one, the other is on its way, and the
// registers leave room for four waves on a SIMD.
template <int D, int GROUP, int NT, bool WIN>
struct FewRows {
    using F = Format<D, GROUP>;
    static constexpr int kLoads = (F::REC + 1023) / 1024;  // of a record
    static constexpr int kSlot = kLoads * 1024;
    static constexpr int kDepth = 2;
    static constexpr int kRing = kDepth * kSlot;  // a wave's; later CH words of its sums, and its references and sums
    static constexpr int kJoinM = kRing - 32 * 4 * NT, kJoinL = kRing - 16 * 4 * NT;
    static constexpr int kRounds = 2 * F::W * NT * 1024 <= kJoinM ? 1 : 2;
    static constexpr int CH = 2 * F::W / kRounds;
    static_assert(CH * kRounds == 2 * F::W && CH * NT * 1024 <= kJoinM, "rounds cover the channels, and fit");
    static constexpr int kRegs = NT * (12 * F::W + 4 * F::NG + 20) + (GROUP ? 8 * F::NG + 2 * F::W : 4 * F::W) + 28 +
                                 (WIN ? 24 : 0);
    static constexpr int kWaves = kRegs <= 128 ? 4 : kRegs <= 168 ? 3 : kRegs <= 256 ? 2 : 1;
    static constexpr int kFit = 163840 / (kAttendWaves * kRing);
    static constexpr int kResident = kFit < kWaves ? kFit : kWaves;  // workgroups of a compute unit
    static_assert(kResident >= 1 && kResident <= kMostResident, "the workspace has room for no more parts");
};

// The 8-bit format's sums of weights times values, and of weights.  power: of
// the values in the units of the sums.  live: positions of the record that the
// sequence has; what lies past its end may be anything.
template <int D, int NT>
__device__ __forceinline__ void values8(const char *rec, int lane, float power, int live, const h8 (&p)[NT][1],
                                        Softmax<D, 0> (&s)[NT]) {
    using F = Format<D, 0>;
    const h8 ones = {1, 1, 1, 1, 1, 1, 1, 1};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt].z = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p[nt][0], s[nt].z, 0, 0, 0);
    const auto add = [&](uint2 mask, bool whole) {
#pragma unroll
        for (int c = 0; c < 2 * F::W; ++c) {
            uint2 w = *reinterpret_cast<const uint2 *>(rec + F::VC + codes8_at(c, lane));
            if (!whole) w.x &= mask.x, w.y &= mask.y;
            const h8 value = codes8(w, power);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                s[nt].o[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, p[nt][0], s[nt].o[c], 0, 0, 0);
        }
    };
    if (live >= kTile)
        add(make_uint2(0, 0), true);
    else
        add(live_codes(live, lane), false);
}

// Rows block * R .. of one (sequence, head) at places t0 .. t1 - 1.  part:
// where the partial sums go, or -1 where these are all of the rows' positions.
template <int D, int GROUP, int NT, bool BF16, bool EVEN, bool WIN>
__device__ __forceinline__ void attend_piece(const AttendArgs &a, char *ring, int wave, int tid, const View<WIN> &e, int seq,
                                             int head, int block, int t0, int t1, int64_t part) {
    using F = Format<D, GROUP>;
    using K = FewRows<D, GROUP, NT, WIN>;
    constexpr int R = 16 * NT;
    constexpr bool k8 = GROUP == 0;
    const int lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int shift = a.c.page_shift;
    const int32_t *table = a.b.table + seq * a.b.table_stride;
    const int r0 = block * R;
    Pages pages;
    pages.load(a, table, e.position(t0) >> shift, lane);

    const int rows_here = e.rows - r0 < R ? e.rows - r0 : R;
    const int i1 = divided(r0 + rows_here - 1, a.by_group_heads);
    const int all_see = e.limit(a, divided(r0, a.by_group_heads));  // below this no row is masked, but for a window
    int end = e.place(e.limit(a, i1));                              // at this and above every row is
    end = end < t1 ? end : t1;

    Row<D, GROUP> raw[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        raw[nt].load(a, e, head, r0 + 16 * nt + n, g, r0 + 16 * nt + n < e.rows);
        raw[nt].wait();  // no wait for them later, which would be one for the records too
    }
    char *const mine = ring + wave * K::kRing;
    const uint32_t mine_at = lds_address(mine);
    int missing = 0;  // bit s: the record in slot s has no page
    const auto fetch = [&](int place, int slot) {
        const int pos = e.position(place);
        const int page = pages.get(a, table, pos >> shift, lane);
        const char *rec = record_at(a.c, page < 0 ? 0 : page, head, pos / kTile);
        missing = (missing & ~(1 << slot)) | ((page < 0 ? 1 : 0) << slot);
        load_run_to_lds<K::kLoads>(rec, page < 0 ? 0 : F::REC, mine_at + slot * K::kSlot, lane * 16);
    };
    int p0 = t0 + kTile * wave;
#pragma unroll
    for (int i = 0; i < K::kDepth; ++i)
        if (p0 + i * kStep < end) fetch(p0 + i * kStep, i);

    h8 q[NT][F::W];
    float qsum[NT][F::NG], factor[NT];
    f4 first[NT][F::NG];
    Sight<WIN> sight[NT];
    Softmax<D, GROUP> s[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        sight[nt].load(a, e, r0 + 16 * nt + n);
        raw[nt].template operand<BF16>(a, q[nt], qsum[nt], factor[nt]);
        if constexpr (!k8) {
#pragma unroll
            for (int grp = 0; grp < F::NG; ++grp) {
                const float f = -kPlus * qsum[nt][grp];
                first[nt][grp] = (f4){f, f, f, f};
            }
        }
        s[nt].clear();
        if constexpr (!k8)
            if (a.row_info && t0 == 0 && wave == 0 && r0 / 16 + nt < a.row_tiles)
                keep_rows<D, GROUP>(a, ((int64_t)seq * a.c.heads + head) * a.row_tiles + r0 / 16 + nt, lane, q[nt],
                                    sum_parts<D, GROUP>(qsum[nt], g), sums_factor(factor[nt]));
    }

    int units = 0;  // of o: 2^(units - 127); 0: nothing but zeros has been summed
    for (int slot = 0; p0 < end; p0 += kStep, slot ^= 1) {
        static_assert(K::kDepth == 2, "slots alternate");
        if (p0 + kStep < end)
            wait_loads<K::kLoads>();
        else
            wait_loads<0>();
        const char *rec = mine + slot * K::kSlot;
        const bool gone = (missing >> slot) & 1;
        const int at = e.position(p0);
        float x[NT][8], scaled[NT];
        const float(&f)[NT] = k8 ? scaled : factor;
        int power = 0;  // E of the values
        if constexpr (k8) {
            const uint32_t ex = (uint32_t)__builtin_amdgcn_readfirstlane(*reinterpret_cast<const int *>(rec + F::EX));
            products8<D, NT>(rec, lane, q, x);
            power = (ex >> 8) & 255;
            const float of_keys = power_of(ex & 255);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) scaled[nt] = fminf(fmaxf(factor[nt] * of_keys, 0x1p-126f), 0x1.fffffep127f);
            if (power > units) {
                const float shrunk = units ? __builtin_amdgcn_ldexpf(1.0f, units - power) : 1.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[nt].rescale(shrunk);
                units = power;
            }
        } else {
            products<D, GROUP, NT>(rec, lane, q, qsum, first, x);
        }
        const bool masked = at + kTile > all_see || gone || e.windowed(a, i1, at);  // some position is not seen by some row
        if (masked) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int pos = at + 16 * (j >> 2) + 4 * g + (j & 3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (!sight[nt].sees(a, e, pos) || gone) x[nt][j] = -__builtin_inff();
            }
        }
        if (!k8 && NT == 1 && a.logits && n < a.rows) {
            float *to = a.logits + (((int64_t)(seq * (int)a.c.heads + head) * ((a.max_len + kTile - 1) / kTile) + p0 / kTile) *
                                        a.rows + n) * kTile + 4 * g;
#pragma unroll
            for (int half = 0; half < 2; ++half)
                *reinterpret_cast<f4 *>(to + 16 * half) = (f4){x[0][4 * half], x[0][4 * half + 1], x[0][4 * half + 2],
                                                              x[0][4 * half + 3]} * factor[0];
        }
        bool grown = false;
        float top[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            top[nt] = Softmax<D, GROUP>::top(x[nt]) * f[nt];
            grown |= top[nt] > s[nt].m + kSlack;
        }
        if (__any(grown)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt].grow(top[nt]);
        }
        h8 p[NT][1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt].weights(x[nt], f[nt], p[nt]);
        if constexpr (k8) {
            values8<D, NT>(rec, lane, power_in(power, units), masked ? e.len - at : kTile, p, s);
        } else {
        h8 scale[F::NG];  // of the lane's 8 positions
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp)
            scale[grp] = *reinterpret_cast<const h8 *>(rec + F::VP + grp * 128 + g * 16);
        h8 row = one_row<D, GROUP>(lane);
        if (n < 2 * F::NG) row = *reinterpret_cast<const h8 *>(rec + F::VP + n * 64 + g * 16);
        if (masked) {  // what lies past the sequence's end may be anything
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at + 16 * (j >> 2) + 4 * g + (j & 3) >= e.len) {
#pragma unroll
                    for (int grp = 0; grp < F::NG; ++grp) scale[grp][j] = (_Float16)0.0f;
                    row[j] = (_Float16)0.0f;
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            s[nt].z = __builtin_amdgcn_mfma_f32_16x16x32_f16(row, p[nt][0], s[nt].z, 0, 0, 0);
#pragma unroll
        for (int hs = 0; hs < 2 * F::S; ++hs) {
            uint32_t w[F::WV];
            load_words<F::WV>(rec + F::VC + (hs * 64 + lane) * (F::WV * 4), w);
#pragma unroll
            for (int i = 0; i < F::WV; ++i) {
                const int c = hs * F::WV + i;
                const h8 value = codes_minus<8>(w[i]) * scale[c / F::VG];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[nt].o[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, p[nt][0], s[nt].o[c], 0, 0, 0);
            }
        }
        }
        if (p0 + K::kDepth * kStep < end) {
            wait_lds();  // the slot has been read
            fetch(p0 + K::kDepth * kStep, slot);
        }
    }

    // ---- join the waves
    wait_lds();
    const auto m_of = [&](int w, int r) -> float & { return reinterpret_cast<float *>(ring + w * K::kRing + K::kJoinM)[r]; };
    const auto l_of = [&](int w, int r) -> float & { return reinterpret_cast<float *>(ring + w * K::kRing + K::kJoinL)[r]; };
    const int row_bits = rows_here > 1 ? 32 - __builtin_clz(rows_here - 1) : 0;  // room for the rows that are there
    const auto o_of = [&](int w, int item) -> f4 & { return reinterpret_cast<f4 *>(ring + w * K::kRing)[item]; };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        s[nt].finish(lane, k8 ? power_of(units) : 1.0f);
        if (g == 0) m_of(wave, 16 * nt + n) = s[nt].m, l_of(wave, 16 * nt + n) = s[nt].l;
    }
    const int part_rows = EVEN && a.rows > R ? R : a.rows;
#pragma unroll
    for (int round = 0; round < K::kRounds; ++round) {
        if (round) __syncthreads();
#pragma unroll
        for (int c = 0; c < K::CH; ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) o_of(wave, (c * NT + nt) * 64 + lane) = s[nt].o[round * K::CH + c];
        __syncthreads();
        // four channels of a row that is there for each thread
        for (int item = tid; item < (K::CH * 4) << row_bits; item += 64 * kAttendWaves) {
            const int rl = item & ((1 << row_bits) - 1), quad = item >> row_bits, row = r0 + rl;
            if (rl >= rows_here) continue;
            float best = m_of(0, rl);
#pragma unroll
            for (int w = 1; w < kAttendWaves; ++w) best = fmaxf(best, m_of(w, rl));
            float sum = 0.0f;
            f4 y = (f4){0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kAttendWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(m_of(w, rl) - best);
                sum += l_of(w, rl) * f;
                y += o_of(w, ((quad >> 2) * NT + (rl >> 4)) * 64 + 16 * (quad & 3) + (rl & 15)) * f;
            }
            const int channel = 16 * K::CH * round + 4 * quad;
            if (part >= 0) {
                const int64_t to = part * part_rows + (EVEN ? rl : row);
                *reinterpret_cast<f4 *>(a.part_o + to * D + channel) = y;
                if (channel == 0) a.part_ml[2 * to] = best, a.part_ml[2 * to + 1] = sum;
            } else {
                write_row(a, e, seq, head, row, channel, y, best, sum);
            }
        }
    }
}

template <int D, int GROUP, int NT, bool BF16, bool EVEN, bool WIN>
__global__ void __launch_bounds__(64 * kAttendWaves, (FewRows<D, GROUP, NT, WIN>::kWaves)) attend_kernel(const AttendArgs a) {
    __shared__ __attribute__((aligned(1024))) char ring[kAttendWaves * FewRows<D, GROUP, NT, WIN>::kRing];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (EVEN) {
        int seq, at, left;  // a step of the sequence's line, and how many are to do
        {
            const int lane = threadIdx.x & 63;
            Even even;
            even.load<WIN>(a, lane);
            if (blockIdx.x == 0 && wave == 0) even.store(a, lane);
            at = (int)blockIdx.x * even.share;
            left = even.total - at < even.share ? even.total - at : even.share;
            if (left <= 0) return;
            seq = __builtin_amdgcn_readfirstlane(even.seq_of(at));
            at -= __builtin_amdgcn_readfirstlane(even.first_of(seq));
        }
        for (;;) {
            int tid = threadIdx.x;
            asm volatile("" : "+v"(tid));  // or what comes of it would be kept from one piece for the next
            const View<WIN> e(a, seq);
            const int steps = Even::steps(e), line = steps + Even::kLead, blocks = Even::blocks(a, e);
            const int unit = (int)((uint32_t)at / (uint32_t)line);
            int from = at - unit * line, to = from + left < line ? from + left : line;
            at += to - from;
            left -= to - from;
            from = from > Even::kLead ? from - Even::kLead : 0;
            to -= Even::kLead;
            if (to <= from) break;  // no more than a row block's lead was left
            const int head = (int)((uint32_t)unit / (uint32_t)blocks), block = unit - head * blocks;
            const int64_t part = ((int64_t)seq * a.c.heads + head) * a.row_blocks + block + blockIdx.x;
            attend_piece<D, GROUP, NT, BF16, EVEN, WIN>(a, ring, wave, tid, e, seq, head, block, from * kStep, to * kStep,
                                                   to - from < steps ? part : -1);
            if (left <= 0) break;
            for (int all = Even::all(a, e); at >= all; all = Even::all(a, View<WIN>(a, seq))) at -= all, ++seq;
            __syncthreads();  // the ring is read no longer
        }
    } else {
        int block, split, head, seq;
        place(a, block, split, head, seq);
        const View<WIN> e(a, seq);
        const Chunks chunks(a, e.span());
        if (block * 16 * NT >= e.rows || split >= chunks.n) return;
        attend_piece<D, GROUP, NT, BF16, EVEN, WIN>(
            a, ring, wave, threadIdx.x, e, seq, head, block, split * chunks.size, (split + 1) * chunks.size,
            a.n_split > 1 ? ((int64_t)seq * a.c.heads + head) * a.n_split + split : -1);
    }
}

}  // namespace tkv
