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
// q . c is a product of fp16 numbers, exact up to its fp32 sum (a bf16 row of
// q is first scaled by a power of two to a largest magnitude in [2^14, 2^15),
// so what fp16 drops is below 2^-38 of that); s and z come in at fp32.  For V, s * c is
// rounded to fp16 (half a step is 2^-11 of it, relative), and so is p.
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
    h8 scale[Format<D, GROUP>::NG], zero[Format<D, GROUP>::NG];  // of the lane's 8 positions
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

template <int D, int GROUP>
__device__ __forceinline__ void load_v(const char *rec, int lane, VTile<D, GROUP> &v) {
    using F = Format<D, GROUP>;
#pragma unroll
    for (int hs = 0; hs < 2 * F::S; ++hs)
        load_words<F::WV>(rec + F::VC + ((hs * 64 + lane) * F::WV) * 4, &v.w[hs * F::WV]);
#pragma unroll
    for (int grp = 0; grp < F::NG; ++grp) {
        const char *p = rec + F::VP + grp * 128 + (lane >> 4) * 16;
        v.scale[grp] = *reinterpret_cast<const h8 *>(p);
        v.zero[grp] = *reinterpret_cast<const h8 *>(p + 64);
    }
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
// x[nt][4 * half + i] for position 16 half + 4 g + i.
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
                const h8 key = codes_to_half(k.w[half][grp * F::KG + c]);
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
__device__ __forceinline__ float over_groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

template <int D, int GROUP, int NT>
__global__ void __launch_bounds__(64 * kAttendWaves) attend_kernel(const AttendArgs a) {
    using F = Format<D, GROUP>;
    constexpr int R = 16 * NT;
    constexpr int CH = NT >= 4 ? 2 : NT == 2 ? (D == 96 ? 3 : 4) : (D / 16 < 8 ? D / 16 : 8);  // V words joined in a round
    constexpr int ROUNDS = (2 * F::W) / CH;
    static_assert(ROUNDS * CH == 2 * F::W, "rounds cover the channels");
    __shared__ float join[kAttendWaves][CH * NT][64][4];
    __shared__ float join_m[kAttendWaves][R], join_l[kAttendWaves][R];

    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    int at = blockIdx.x;
    const int block = at % a.row_blocks;
    at /= a.row_blocks;
    const int split = at % a.n_split;
    at /= a.n_split;
    const int head = at % (int)a.c.heads, seq = at / (int)a.c.heads;
    const Extent e(a, seq);
    const int r0 = block * R;
    if (r0 >= e.rows) return;
    const int t0 = split * a.chunk;
    if (split > 0 && t0 >= e.len) return;

    // ---- the queries
    h8 q[NT][F::W];
    float qsum[NT][F::NG], factor[NT];
    int limit[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + 16 * nt + n;
        const bool live = r < e.rows;
        const int i = r / a.group_heads, hq = head * a.group_heads + r % a.group_heads;
        limit[nt] = live ? e.limit(a, i) : 0;
        float x[F::W][8], top = 0.0f;
        const int64_t row = (e.start + i) * a.q.token_stride + hq * a.q.head_stride + 8 * g;
#pragma unroll
        for (int c = 0; c < F::W; ++c) {
            if (live) {
                load8(a.q, row + 32 * c, x[c]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[c][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[c][j]));
        }
        int power = 0;
        if (a.q.type == kBf16) {
            top = over_groups_max(top);
            int ex;
            (void)frexpf(top, &ex);  // top = m * 2^ex, m in [0.5, 1)
            if (top > 0.0f && top < __builtin_inff()) power = 15 - ex;
        }
        factor[nt] = ldexpf(a.scale_log2, -power);
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) qsum[nt][grp] = 0.0f;
#pragma unroll
        for (int c = 0; c < F::W; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const _Float16 v = (_Float16)ldexpf(x[c][j], power);
                q[nt][c][j] = v;
                qsum[nt][c / F::KG] += (float)v;
            }
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) qsum[nt][grp] = over_groups_sum(qsum[nt][grp]);
        if (a.frag_q && split == 0 && wave == 0) {
            const int64_t tile = ((int64_t)seq * a.c.heads + head) * a.row_tiles + r0 / 16 + nt;
            if (r0 / 16 + nt < a.row_tiles) {
                h8 *to = (h8 *)a.frag_q + tile * (F::W * 64);
#pragma unroll
                for (int c = 0; c < F::W; ++c) to[c * 64 + lane] = q[nt][c];
                if (g == 0) {
                    float *info = a.row_info + (tile * 16 + n) * (2 + F::NG);
                    info[0] = factor[nt];
                    info[1] = __builtin_inff();  // a row without positions weighs nothing
#pragma unroll
                    for (int grp = 0; grp < F::NG; ++grp) info[2 + grp] = qsum[nt][grp];
                }
            }
        }
    }

    // ---- the positions
    const int rows_here = e.rows - r0 < R ? e.rows - r0 : R;
    const int all_see = e.limit(a, r0 / a.group_heads);                  // below this no row is masked
    int end = e.limit(a, (r0 + rows_here - 1) / a.group_heads);          // at this and above every row is
    end = end < t0 + a.chunk ? end : t0 + a.chunk;

    f4 o[NT][2 * F::W];
    float m[NT], l[NT], zsum[NT][F::NG];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt] = kFar;
        l[nt] = 0.0f;
#pragma unroll
        for (int c = 0; c < 2 * F::W; ++c) o[nt][c] = (f4){0, 0, 0, 0};
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) zsum[nt][grp] = 0.0f;
    }

    const int32_t *table = a.b.table + seq * a.b.table_stride;
    const int shift = a.c.page_shift;
    const int page_first = t0 >> shift;
    Pages pages;
    pages.load(a, table, page_first, lane);
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
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int pos = p0 + 16 * (j >> 2) + 4 * g + (j & 3);
                    if (pos >= limit[nt] || page_now < 0) x[nt][j] = -__builtin_inff();
                }
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // what lies past the sequence's end may be anything
                const int pos = p0 + 16 * (j >> 2) + 4 * g + (j & 3);
                if (pos >= e.len || page_now < 0) {
#pragma unroll
                    for (int grp = 0; grp < F::NG; ++grp) v.scale[grp][j] = (_Float16)0.0f, v.zero[grp][j] = (_Float16)0.0f;
                }
            }
        }
        bool grown = false;
        float top[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[nt][j] *= factor[nt];
            top[nt] = fmaxf(fmaxf(fmaxf(x[nt][0], x[nt][1]), fmaxf(x[nt][2], x[nt][3])),
                            fmaxf(fmaxf(x[nt][4], x[nt][5]), fmaxf(x[nt][6], x[nt][7])));
            grown |= top[nt] > m[nt] + kSlack;
        }
        if (__any(grown)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float t = over_groups_max(top[nt]);
                const float m1 = t > m[nt] + kSlack ? t : m[nt];
                const float f = exp2f(m[nt] - m1);
                m[nt] = m1;
                l[nt] *= f;
#pragma unroll
                for (int grp = 0; grp < F::NG; ++grp) zsum[nt][grp] *= f;
#pragma unroll
                for (int c = 0; c < 2 * F::W; ++c) o[nt][c] *= f;
            }
        }
        h8 p[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float lift = kLift - m[nt];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = __builtin_amdgcn_exp2f(x[nt][j] + lift);
                l[nt] += w;
                p[nt][j] = (_Float16)w;
#pragma unroll
                for (int grp = 0; grp < F::NG; ++grp) zsum[nt][grp] = fmaf(w, (float)v.zero[grp][j], zsum[nt][grp]);
            }
        }
#pragma unroll
        for (int c = 0; c < 2 * F::W; ++c) {
            const h8 value = codes_to_half(v.w[c]) * v.scale[c / F::VG];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                o[nt][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, p[nt], o[nt][c], 0, 0, 0);
        }
        if (rec) load_v<D, GROUP>(rec, lane, v);
        p0 = next;
    }

    // ---- join the waves
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        l[nt] = over_groups_sum(l[nt]);
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) {
            const float z = over_groups_sum(zsum[nt][grp]);
#pragma unroll
            for (int c = 0; c < F::VG; ++c) o[nt][grp * F::VG + c] += z;
        }
        if (g == 0) join_m[wave][16 * nt + n] = m[nt], join_l[wave][16 * nt + n] = l[nt];
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float best = join_m[0][16 * nt + n];
#pragma unroll
        for (int w = 1; w < kAttendWaves; ++w) best = fmaxf(best, join_m[w][16 * nt + n]);
        const float f = exp2f(m[nt] - best);
#pragma unroll
        for (int c = 0; c < 2 * F::W; ++c) o[nt][c] *= f;
    }
    const int64_t unit = ((int64_t)seq * a.c.heads + head) * a.n_split + split;
#pragma unroll
    for (int round = 0; round < ROUNDS; ++round) {
        if (round) __syncthreads();
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                *reinterpret_cast<f4 *>(join[wave][c * NT + nt][lane]) = o[nt][round * CH + c];
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
                const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
                const int i = row / a.group_heads, hq = head * a.group_heads + row % a.group_heads;
                uint16_t *to = (uint16_t *)a.out.data + (e.start + i) * a.out.token_stride + hq * a.out.head_stride + channel;
#pragma unroll
                for (int j = 0; j < 4; ++j) to[j] = float_to_elem(y[j] * inv, a.out.type);
                if (channel == 0) {
                    const float log_sum = best - kLift + log2f(sum);  // log2(0) = -inf: nothing seen
                    a.lse[(e.start + i) * (a.c.heads * a.group_heads) + hq] = log_sum * 0.69314718056f;
                    if (a.frag_q) {
                        const int64_t tile = ((int64_t)seq * a.c.heads + head) * a.row_tiles + row / 16;
                        if (sum > 0.0f || sum != sum)
                            a.row_info[(tile * 16 + row % 16) * (2 + F::NG) + 1] = log_sum;
                    }
                }
            }
        }
    }
}

// scores_out = scores_in + the weights of each position, summed over rows:
// exp2(y - lse2), with y computed again from the K codes (half of a record)
// rather than kept in memory by the first kernel, which would be 4 bytes for
// each position and row.  One wave owns a record, so sums have one order.
template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kAttendWaves) scores_kernel(const AttendArgs a) {
    using F = Format<D, GROUP>;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int splits = (a.max_len + a.score_chunk - 1) / a.score_chunk;
    int at = blockIdx.x;
    const int split = at % splits;
    at /= splits;
    const int head = at % (int)a.c.heads, seq = at / (int)a.c.heads;
    const Extent e(a, seq);
    const int t0 = split * a.score_chunk;
    if (t0 >= e.len) return;
    const int end = e.len < t0 + a.score_chunk ? e.len : t0 + a.score_chunk;
    const int32_t *table = a.b.table + seq * a.b.table_stride;
    const int64_t first_tile = ((int64_t)seq * a.c.heads + head) * a.row_tiles;
    const h8 *frags = (const h8 *)a.frag_q + first_tile * (F::W * 64);
    const float *infos = a.row_info + first_tile * 16 * (2 + F::NG);
    const int tiles = (e.rows + 15) / 16;
    h8 q[1][F::W];
    float qsum[1][F::NG], factor = 0.0f, lse2 = 0.0f;
    int limit = 0;
    auto load_rows = [&](int t) {
#pragma unroll
        for (int c = 0; c < F::W; ++c) q[0][c] = frags[(t * F::W + c) * 64 + lane];
        const float *info = infos + (t * 16 + n) * (2 + F::NG);
        factor = info[0];
        lse2 = info[1];
#pragma unroll
        for (int grp = 0; grp < F::NG; ++grp) qsum[0][grp] = info[2 + grp];
        const int r = t * 16 + n;
        limit = r < e.rows ? e.limit(a, r / a.group_heads) : 0;
    };
    if (tiles == 1) load_rows(0);
    for (int p0 = t0 + kTile * wave; p0 < end; p0 += kTile * kAttendWaves) {
        const int page = page_at(table, a.b.table_width, a.c.n_pages, p0 >> a.c.page_shift);
        KTile<D, GROUP> k;
        load_k<D, GROUP>(record_at(a.c, page < 0 ? 0 : page, head, p0 / kTile), lane, k);
        float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        // the first row that sees the record
        int t = 0;
        if (a.causal) {
            const int i = p0 - (e.len - e.n);
            if (i > 0) t = i * a.group_heads / 16;
        }
        for (; t < tiles; ++t) {
            if (tiles > 1) load_rows(t);
            float x[1][8];
            products<D, GROUP, 1>(k, q, qsum, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int pos = p0 + 16 * (j >> 2) + 4 * g + (j & 3);
                const float w = __builtin_amdgcn_exp2f(fmaf(x[0][j], factor, -lse2));
                sum[j] += pos < limit && page >= 0 ? w : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int mask = 1; mask < 16; mask <<= 1) sum[j] += __shfl_xor(sum[j], mask);
        if (n == 0) {
            const int64_t row = ((int64_t)seq * a.c.heads + head) * a.score_stride;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int pos = p0 + 16 * (j >> 2) + 4 * g + (j & 3);
                if (pos < e.len) a.scores_out[row + pos] = (a.scores_in ? a.scores_in[row + pos] : 0.0f) + sum[j];
            }
        }
    }
}

template <int D, int GROUP>
static int launch_group(const AttendArgs &a, int row_tile, void *stream) {
    const dim3 block(64 * kAttendWaves);
    const dim3 grid((uint32_t)((int64_t)a.b.n_seq * a.c.heads * a.n_split * a.row_blocks));
    hipStream_t s = (hipStream_t)stream;
    if (row_tile == 16)
        attend_kernel<D, GROUP, 1><<<grid, block, 0, s>>>(a);
    else if (row_tile == 32)
        attend_kernel<D, GROUP, 2><<<grid, block, 0, s>>>(a);
    else if constexpr (D <= 128)
        attend_kernel<D, GROUP, 4><<<grid, block, 0, s>>>(a);
    else
        return (int)hipErrorInvalidValue;
    int rc = (int)hipGetLastError();
    if (rc == 0 && a.n_split > 1) rc = launch_combine(a, stream);
    if (rc == 0 && a.scores_out && a.max_len > 0) {
        const int64_t splits = (a.max_len + a.score_chunk - 1) / a.score_chunk;
        scores_kernel<D, GROUP><<<dim3((uint32_t)(splits * a.c.heads * a.b.n_seq)), block, 0, s>>>(a);
        rc = (int)hipGetLastError();
    }
    return rc;
}

}  // namespace tkv
