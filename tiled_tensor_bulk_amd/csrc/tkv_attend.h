// tkv_attend.h -- attention over the 4-bit cache, and the attention weights
// summed over query rows.
//
// Rows.  A sequence's new tokens times the query heads of one key/value head
// are that head's rows (row = token * group_heads + head in its group); a
// wave holds NT tiles of 16 of them.
//
// Products.  v_mfma_f32_16x16x32_f16 with the cache as the left operand:
// S^T = K Q^T, so a lane holds 4 positions of one row of each 16, and
// O^T = V^T P^T, whose right operand wants 8 positions of one row in a lane:
// the same ones, in the order in which the record holds V's words.  Nothing
// moves between lanes or through LDS in the loop over positions.
//
// Numbers.  With code c, scale s and zero z of a position and channel group,
//   q . k = sum over groups of s * (q . c) + z * (sum of q)
//   p . v = sum over positions of p * (s * c), plus p * z
// q . c is a product of fp16 numbers, exact up to its fp32 sum (a row of q is
// first scaled by a power of two to a largest magnitude in [2^14, 2^15), and
// its elements that meet an upper nibble by 2^-4 more, so what fp16 drops is
// below 2^-35 of that largest); s and z come in at fp32.  For V, s * (c - 8) is
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
// Split.  A workgroup takes `chunk` positions of one (sequence, head, block
// of rows); its four waves take every fourth record, each with its own m,
// and are joined through LDS at the end; with several chunks a second kernel
// joins their partial sums.
#pragma once

#include "tkv_format.h"

namespace tkv {

constexpr int kAttendWaves = 4;
template <int D>
constexpr int kScoreRecords = D <= 128 ? 2 : 1;  // records of a wave of the scores kernel
constexpr float kFar = -1e30f;  // reference of a row that has seen nothing
constexpr float kLift = 7.0f;   // weights are held times 2^7
constexpr float kSlack = 8.0f;

template <int D, int GROUP>
struct KTile {
    uint32_t w[2][Format<D, GROUP>::W];
    h8 pair[2][Format<D, GROUP>::NG];  // (scale, zero) of positions 16 half + 4 g + 0..3
};

template <int D, int GROUP>
struct VTile {
    uint32_t w[2 * Format<D, GROUP>::W];
    h8 scale[Format<D, GROUP>::NG];  // of the lane's 8 positions
    h8 row;                          // row n of the operand of scales and zeros
};

template <int D, int GROUP>
__device__ __forceinline__ void load_k(const char *rec, int lane, KTile<D, GROUP> &k) {
    using F = Format<D, GROUP>;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int s = 0; s < F::S; ++s)
            load_words<F::WV>(rec + (((half * F::S + s) * 64 + lane) * F::WV) * 4, &k.w[half][s * F::WV]);
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp)
            k.pair[half][grp] =
                *reinterpret_cast<const h8 *>(rec + F::KP + (grp * kTile + 16 * half + 4 * (lane >> 4)) * 4);
    }
}

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

template <int D, int GROUP>
__device__ __forceinline__ void load_v(const char *rec, int lane, VTile<D, GROUP> &v) {
    using F = Format<D, GROUP>;
#pragma unroll
    for (int hs = 0; hs < 2 * F::S; ++hs)
        load_words<F::WV>(rec + F::VC + ((hs * 64 + lane) * F::WV) * 4, &v.w[hs * F::WV]);
#pragma unroll
    for (int grp = 0; grp < F::NG; ++grp)
        v.scale[grp] = *reinterpret_cast<const h8 *>(rec + F::VP + grp * 128 + (lane >> 4) * 16);
    v.row = one_row<D, GROUP>(lane);
    if ((lane & 15) < 2 * F::NG)
        v.row = *reinterpret_cast<const h8 *>(rec + F::VP + (lane & 15) * 64 + (lane >> 4) * 16);
}

// A sequence's extent and the rows of one block.
struct Extent {
    int64_t start;  // first row of its tokens
    int n, len, rows;
    __device__ __forceinline__ Extent(const AttendArgs &a, int seq) {
        new_tokens(a.b, seq, start, n);
        const int64_t width = (int64_t)a.b.table_width << a.c.page_shift;
        int l = a.b.lens[seq];
        l = l < 0 ? 0 : l;
        l = l < a.max_len ? l : a.max_len;
        len = (int64_t)l < width ? l : (int)width;
        rows = n * a.group_heads;
    }
    // positions below this are seen by the i-th new token
    __device__ __forceinline__ int limit(const AttendArgs &a, int i) const { return a.causal ? len - n + 1 + i : len; }
};

// A sequence's chunks: as few as the launch's chunk allows, of equal length up
// to whole steps of the workgroup.
struct Chunks {
    int size, n;
    __device__ __forceinline__ Chunks(const AttendArgs &a, int len) {
        constexpr int kStep = kTile * kAttendWaves;
        const int parts = (len + a.chunk - 1) / a.chunk;
        size = parts > 1 ? ((len + parts - 1) / parts + kStep - 1) / kStep * kStep : a.chunk;
        n = len > 0 ? (len + size - 1) / size : 1;
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

// Products of a record's 32 positions with the wave's rows, in fp32:
// x[nt][4 * half + i] for position 16 half + 4 g + i, times 2^-kCodeBits as qsum is.
template <int D, int GROUP, int NT>
__device__ __forceinline__ void products(const KTile<D, GROUP> &k, const h8 (&q)[NT][D / 32],
                                         const float (&qsum)[NT][D / GROUP], float (&x)[NT][8]) {
    using F = Format<D, GROUP>;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) {
            f4 acc[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt] = (f4){0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < F::KG; ++c) {
                const h8 key = codes_as_bits(k.w[half][grp * F::KG + c]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[nt][grp * F::KG + c], acc[nt], 0, 0, 0);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = (float)k.pair[half][grp][2 * i], z = (float)k.pair[half][grp][2 * i + 1];
                    const float y = grp == 0 ? z * qsum[nt][grp] : fmaf(z, qsum[nt][grp], x[nt][4 * half + i]);
                    x[nt][4 * half + i] = fmaf(s, acc[nt][i], y);
                }
        }
}

__device__ __forceinline__ float over_groups_sum(float v) {  // over the four lanes of a row
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float over_rows_sum(float v) {  // over 16 neighbouring lanes, by rotations
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 15, 15, true));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x124, 15, 15, true));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x122, 15, 15, true));
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x121, 15, 15, true));
}
__device__ __forceinline__ float over_groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

// Four channels of an output row, and with the first ones its lse.
__device__ __forceinline__ void write_row(const AttendArgs &a, const Extent &e, int seq, int head, int row, int channel,
                                          f4 y, float best, float sum) {
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const int i = row / a.group_heads, hq = head * a.group_heads + row % a.group_heads;
    store4(a.out, (e.start + i) * a.out.token_stride + hq * a.out.head_stride + channel, y * inv);
    if (channel == 0) {
        const float log_sum = best - kLift + log2f(sum);  // log2(0) = -inf: nothing seen
        a.lse[(e.start + i) * (a.c.heads * a.group_heads) + hq] = log_sum * 0.69314718056f;
        if (a.frag_q && (sum > 0.0f || sum != sum)) {
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
        const int i = live ? r / a.group_heads : 0, hq = head * a.group_heads + (live ? r - i * a.group_heads : 0);
        const int64_t row = (e.start + i) * a.q.token_stride + hq * a.q.head_stride + 8 * g;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) raw[c] = live ? load8_raw(a.q, row + 32 * c) : make_uint4(0, 0, 0, 0);
    }
    // q, its sums over the groups of channels (times 2^-kCodeBits), and what
    // turns products into logarithms to base 2: at least the smallest normal
    // number, as masked products are -inf.
    __device__ __forceinline__ void operand(const AttendArgs &a, h8 (&q)[D / 32], float (&qsum)[D / GROUP],
                                            float &factor) const {
        using F = Format<D, GROUP>;
        float x[F::W][8], top = 0.0f;
#pragma unroll
        for (int c = 0; c < F::W; ++c) {
            raw_to_float(raw[c], a.q.type, x[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[c][j]));
        }
        top = over_groups_max(top);
        int power = 0;
        if (top > 0.0f && top < __builtin_inff()) {
            (void)frexpf(top, &power);  // top = m * 2^power, m in [0.5, 1)
            power = 15 - power;
        }
        const float f = fabsf(ldexpf(a.scale_log2, kCodeBits - power));
        factor = fminf(fmaxf(f, 0x1p-126f), 0x1.fffffep127f);
        const float sign = a.scale_log2 < 0.0f ? -1.0f : 1.0f;
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) qsum[grp] = 0.0f;
#pragma unroll
        for (int c = 0; c < F::W; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const _Float16 v = (_Float16)ldexpf(sign * x[c][j], power - code_shift(j));
                q[c][j] = v;
                qsum[c / F::KG] = fmaf((float)v, (float)(1 << code_shift(j)), qsum[c / F::KG]);
            }
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) qsum[grp] = over_groups_sum(qsum[grp]) * (1.0f / (1 << kCodeBits));
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
        float y = qsum[grp] * (float)(1 << (kCodeBits - kSumBits));
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
    return fmaxf(factor * (1.0f / (1 << (kCodeBits - kSumBits))), 0x1p-126f);
}

// Where the scores kernel finds a tile of 16 rows and what belongs to it.
template <int D, int GROUP>
__device__ __forceinline__ void keep_rows(const AttendArgs &a, int64_t tile, int lane, const h8 (&q)[D / 32], h8 sums,
                                          float factor) {
    using F = Format<D, GROUP>;
    h8 *to = (h8 *)a.frag_q + tile * ((F::W + 1) * 64);
#pragma unroll
    for (int c = 0; c < F::W; ++c) to[c * 64 + lane] = q[c];
    to[F::W * 64 + lane] = sums;
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
        const float f = exp2f(m - m1);
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
    // after the last position: l whole in every lane, o what a division by l makes the output
    __device__ __forceinline__ void finish(int lane) {
        using F = Format<D, GROUP>;
        l = over_groups_sum(l);
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
};

// Waves of a SIMD that the registers of a wave leave room for: queries, sums
// and logits of its rows, a record on its way, and what is being worked on.
template <int D, int GROUP, int NT>
struct FewRows {
    using F = Format<D, GROUP>;
    static constexpr int kRegs = NT * (4 * F::W + 8 * F::W + 4 + 8 + 8) + 4 * F::W + 4 + 12 * F::NG + 32;
    static constexpr int kWaves = kRegs <= 128 ? 4 : kRegs <= 168 ? 3 : kRegs <= 256 ? 2 : 1;
};

// Few rows: the four waves share them and take every fourth record.
template <int D, int GROUP, int NT>
__global__ void __launch_bounds__(64 * kAttendWaves, (FewRows<D, GROUP, NT>::kWaves)) attend_kernel(const AttendArgs a) {
    using F = Format<D, GROUP>;
    constexpr int R = 16 * NT;
    constexpr int CH = NT == 2 ? (D == 96 ? 3 : 4) : (D / 16 < 8 ? D / 16 : 8);  // V words joined in a round
    constexpr int ROUNDS = (2 * F::W) / CH;
    static_assert(ROUNDS * CH == 2 * F::W, "rounds cover the channels");
    __shared__ float join[kAttendWaves][CH * NT][64][4];
    __shared__ float join_m[kAttendWaves][R], join_l[kAttendWaves][R];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    int at = blockIdx.x;
    const int block = at % a.row_blocks;
    at /= a.row_blocks;
    const int split = at % a.n_split;
    at /= a.n_split;
    const int head = at % (int)a.c.heads, seq = at / (int)a.c.heads;
    const int shift = a.c.page_shift;
    const int32_t *table = a.b.table + seq * a.b.table_stride;
    const Extent e(a, seq);
    const Chunks chunks(a, e.len);
    const int r0 = block * R;
    if (r0 >= e.rows || split >= chunks.n) return;
    const int t0 = split * chunks.size;
    Pages pages;
    pages.load(a, table, t0 >> shift, lane);

    const int rows_here = e.rows - r0 < R ? e.rows - r0 : R;
    const int all_see = e.limit(a, r0 / a.group_heads);                  // below this no row is masked
    int end = e.limit(a, (r0 + rows_here - 1) / a.group_heads);          // at this and above every row is
    end = end < t0 + chunks.size ? end : t0 + chunks.size;

    Row<D, GROUP> raw[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) raw[nt].load(a, e, head, r0 + 16 * nt + n, g, r0 + 16 * nt + n < e.rows);
    KTile<D, GROUP> k;
    VTile<D, GROUP> v;
    int p0 = t0 + kTile * wave;
    int page = -1;
    if (p0 < end) {
        page = pages.get(a, table, p0 >> shift, lane);
        const char *rec = record_at(a.c, page < 0 ? 0 : page, head, p0 / kTile);
        load_k<D, GROUP>(rec, lane, k);
        load_v<D, GROUP>(rec, lane, v);
    }

    h8 q[NT][F::W];
    float qsum[NT][F::NG], factor[NT];
    int limit[NT];
    Softmax<D, GROUP> s[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + 16 * nt + n;
        limit[nt] = r < e.rows ? e.limit(a, r / a.group_heads) : 0;
        raw[nt].operand(a, q[nt], qsum[nt], factor[nt]);
        s[nt].clear();
        if (a.frag_q && split == 0 && wave == 0 && r0 / 16 + nt < a.row_tiles)
            keep_rows<D, GROUP>(a, ((int64_t)seq * a.c.heads + head) * a.row_tiles + r0 / 16 + nt, lane, q[nt],
                                sum_parts<D, GROUP>(qsum[nt], g), sums_factor(factor[nt]));
    }

    while (p0 < end) {
        const int next = p0 + kTile * kAttendWaves;
        const int page_now = page;
        const char *rec = nullptr;
        if (next < end) {
            page = pages.get(a, table, next >> shift, lane);
            rec = record_at(a.c, page < 0 ? 0 : page, head, next / kTile);
        }
        float x[NT][8];
        products<D, GROUP, NT>(k, q, qsum, x);
        if (rec) load_k<D, GROUP>(rec, lane, k);

        if (p0 + kTile > all_see || page_now < 0) {  // some position is not seen by some row
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int pos = p0 + 16 * (j >> 2) + 4 * g + (j & 3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (pos >= limit[nt] || page_now < 0) x[nt][j] = -__builtin_inff();
                if (pos >= e.len || page_now < 0) {  // what lies past the sequence's end may be anything
#pragma unroll
                    for (int grp = 0; grp < F::NG; ++grp) v.scale[grp][j] = (_Float16)0.0f;
                    v.row[j] = (_Float16)0.0f;
                }
            }
        }
        bool grown = false;
        float top[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            top[nt] = Softmax<D, GROUP>::top(x[nt]) * factor[nt];
            grown |= top[nt] > s[nt].m + kSlack;
        }
        if (__any(grown)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt].grow(top[nt]);
        }
        h8 p[NT][1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            s[nt].weights(x[nt], factor[nt], p[nt]);
            s[nt].z = __builtin_amdgcn_mfma_f32_16x16x32_f16(v.row, p[nt][0], s[nt].z, 0, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < 2 * F::W; ++c) {
            const h8 value = codes_minus_8(v.w[c]) * v.scale[c / F::VG];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                s[nt].o[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, p[nt][0], s[nt].o[c], 0, 0, 0);
        }
        if (rec) load_v<D, GROUP>(rec, lane, v);
        p0 = next;
    }

    // ---- join the waves
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        s[nt].finish(lane);
        if (g == 0) join_m[wave][16 * nt + n] = s[nt].m, join_l[wave][16 * nt + n] = s[nt].l;
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float best = join_m[0][16 * nt + n];
#pragma unroll
        for (int w = 1; w < kAttendWaves; ++w) best = fmaxf(best, join_m[w][16 * nt + n]);
        const float f = exp2f(s[nt].m - best);
#pragma unroll
        for (int c = 0; c < 2 * F::W; ++c) s[nt].o[c] *= f;
    }
    const int64_t unit = ((int64_t)seq * a.c.heads + head) * a.n_split + split;
#pragma unroll
    for (int round = 0; round < ROUNDS; ++round) {
        if (round) __syncthreads();
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                *reinterpret_cast<f4 *>(join[wave][c * NT + nt][lane]) = s[nt].o[round * CH + c];
        __syncthreads();
        for (int item = threadIdx.x; item < CH * NT * 64; item += 64 * kAttendWaves) {
            const int cn = item >> 6, ln = item & 63;
            const int row = r0 + 16 * (cn % NT) + (ln & 15);
            if (row >= e.rows) continue;
            const int rl = 16 * (cn % NT) + (ln & 15);
            float best = join_m[0][rl];
#pragma unroll
            for (int w = 1; w < kAttendWaves; ++w) best = fmaxf(best, join_m[w][rl]);
            float sum = 0.0f;
            f4 y = (f4){0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kAttendWaves; ++w) {
                sum += join_l[w][rl] * exp2f(join_m[w][rl] - best);
                y += *reinterpret_cast<const f4 *>(join[w][cn][ln]);
            }
            const int channel = 16 * (round * CH + cn / NT) + 4 * (ln >> 4);
            if (a.n_split > 1) {
                const int64_t to = unit * a.rows + row;
                *reinterpret_cast<f4 *>(a.part_o + to * D + channel) = y;
                if (channel == 0) a.part_ml[2 * to] = best, a.part_ml[2 * to + 1] = sum;
            } else {
                write_row(a, e, seq, head, row, channel, y, best, sum);
            }
        }
    }
}

}  // namespace tkv
