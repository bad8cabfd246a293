// tkv_scores.h -- attention weights summed over rows:
//   scores_out = scores_in + sum over rows of exp2(y - lse2)
// with the logarithms y computed again from the K codes (half of a record)
// rather than kept in memory by the first kernel, which would be 4 bytes for
// each position and row: less only for up to 8 rows, which weigh_kernel takes.
//
// A wave owns a record, unpacked in registers with its scales and zeros, and
// goes over the tiles of 16 rows that see it (two records for each wave come out
// the same: half the reads of tiles, but half the waves).  A workgroup's waves go over
// the same tiles, four at a time from LDS, each of which one wave loads there
// while the four before are worked on.  One wave adds up a position, in the
// order of the rows.
//
// Bound by the vector units, which take an exponential for each row and
// position: 2 sequences of up to 8192 positions, 512 tokens of 32 heads on 8, 78
// us, 610 TFLOP/s of products.
#pragma once

#include "tkv_attend.h"

namespace tkv {

template <int D>
struct ScoreRows {  // a tile of 16 rows
    h8 q[D / 32], sums;
    float factor, lse2;
    __device__ __forceinline__ void load(const char *from, float2 info, int lane) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) q[c] = reinterpret_cast<const h8 *>(from)[c * 64 + lane];
        sums = reinterpret_cast<const h8 *>(from)[D / 32 * 64 + lane];
        factor = info.x;
        lse2 = info.y;
    }
};

template <int D, int GROUP>
struct ScoreKeys {  // 32 positions
    using F = Format<D, GROUP>;
    h8 k[2][F::W], zero[2];
    float scale[F::NG][8], sum[8];
    __device__ __forceinline__ void load(const char *rec, int lane) {
        const int g = lane >> 4, m = lane & 15;
        uint32_t w[2][F::W];
#pragma unroll
        for (int hs = 0; hs < 2 * F::S; ++hs)
            load_words<F::WV>(rec + (hs * 64 + lane) * F::WV * 4, &w[hs / F::S][(hs % F::S) * F::WV]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            zero[half] = (h8){0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int grp = 0; grp < F::NG; ++grp) {
                const _Float16 *pairs = reinterpret_cast<const _Float16 *>(rec + F::KP) + (grp * kTile + 16 * half) * 2;
                zero[half][grp] = pairs[2 * m + 1];
                const h8 mine = *reinterpret_cast<const h8 *>(pairs + 8 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    scale[grp][4 * half + i] = (float)mine[2 * i] * (1.0f / (1 << kSumBits));
            }
#pragma unroll
            for (int c = 0; c < F::W; ++c) k[half][c] = codes_minus<0>(w[half][c]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    }
    // add the rows' weights; MASKED: some row does not see some position
    template <bool MASKED>
    __device__ __forceinline__ void add(const ScoreRows<D> &r, int p0, int limit, int lane) {
        const int g = lane >> 4;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f4 y = __builtin_amdgcn_mfma_f32_16x16x32_f16(zero[half], r.sums, (f4){0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int grp = 0; grp < F::NG; ++grp) {
                f4 acc = {0, 0, 0, 0};
#pragma unroll
                for (int c = grp * F::KG; c < (grp + 1) * F::KG; ++c)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[half][c], r.q[c], acc, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = fmaf(scale[grp][4 * half + i], acc[i], y[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float w = __builtin_amdgcn_exp2f(fmaf(y[i], r.factor, -r.lse2));
                if (MASKED) w = p0 + 16 * half + 4 * g + i < limit ? w : 0.0f;
                sum[4 * half + i] += w;
            }
        }
    }
};

template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kAttendWaves, (D > 128 ? 2 : D / GROUP > 3 ? 3 : 4)) scores_kernel(const AttendArgs a) {
    constexpr int TILE = (D / 32 + 1) * 1024;  // bytes of a tile of rows
    __shared__ __attribute__((aligned(1024))) char stage[2][kAttendWaves][TILE];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int splits = (a.max_len + kTile * kAttendWaves - 1) / (kTile * kAttendWaves);
    int at = blockIdx.x;
    const int split = at % splits;
    int head = at / splits;
    const int seq = divide(head, (int)a.c.heads, a.by_heads);
    const Extent e(a, seq);
    const int first_pos = split * kAttendWaves * kTile, p0 = first_pos + wave * kTile;
    if (first_pos >= e.len) return;
    const int32_t *table = a.b.table + seq * a.b.table_stride;
    const int64_t first_tile = ((int64_t)seq * a.c.heads + head) * a.row_tiles;
    const int tiles = (e.rows + 15) / 16;
    ScoreKeys<D, GROUP> keys;
    const int page = page_at(table, a.b.table_width, a.c.n_pages, p0 >> a.c.page_shift);
    // of a page that does not exist another one's are read, and dropped
    keys.load(record_at(a.c, page < 0 ? 0 : page, head, p0 / kTile), lane);
    int t0 = 0;  // the first tile with a row that sees the workgroup's first position
    if (a.causal) {
        const int i = first_pos + 1 - e.sees;
        if (i > 0) t0 = (int)((int64_t)i * a.group_heads / 16);
    }
    // tiles whose every row sees all of the wave's positions, and, before and after, others
    int full = tiles, last_full = e.rows / 16;
    if (!a.causal) {
        if (p0 + kTile <= e.len) full = 0;
    } else {
        const int i = p0 + kTile - e.sees;  // the first new token that does
        const int64_t r = i > 0 ? (int64_t)i * a.group_heads : 0;
        if (p0 + kTile <= e.len && r <= e.rows) full = (int)((r + 15) / 16);
    }
    float2 info[kAttendWaves];
    const auto fetch = [&](int t, int slot) {  // the wave's tile of four, and what all of them need of each row
        if (t + wave < tiles)
            load_run_to_lds<TILE / 1024>((const char *)a.frag_q + (first_tile + t + wave) * TILE, TILE,
                                         lds_address(stage[slot][wave]), lane * 16);
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w)
            if (t + w < tiles)
                info[w] = *reinterpret_cast<const float2 *>(a.row_info + ((first_tile + t + w) * 16 + n) * 2);
    };
    if (t0 < tiles) fetch(t0, 0);
    int slot = 0;
    for (int t = t0; t < tiles; t += kAttendWaves, slot ^= 1) {
        float2 now[kAttendWaves];
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) now[w] = info[w];
        wait_loads<0>();
        __syncthreads();  // the stage is full, and the other one has been read
        if (t + kAttendWaves < tiles) fetch(t + kAttendWaves, slot ^ 1);
        if (p0 >= e.len) continue;
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) {
            if (t + w >= tiles) break;
            ScoreRows<D> rows;
            rows.load(stage[slot][w], now[w], lane);
            if (t + w >= full && t + w < last_full) {
                keys.template add<false>(rows, 0, 0, lane);
            } else {
                const int r = (t + w) * 16 + n, limit = r < e.rows ? e.limit(a, divided(r, a.by_group_heads)) : 0;
                keys.template add<true>(rows, p0, limit, lane);
            }
        }
    }
    if (p0 >= e.len) return;
    const int64_t row = ((int64_t)seq * a.c.heads + head) * a.score_stride;
#pragma unroll
    for (int j = 0; j < 8; ++j) keys.sum[j] = over_rows_sum(keys.sum[j]);
    if (n < 8) {  // lane n of a group has position n of its 8
        float mine = keys.sum[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) mine = n == j ? keys.sum[j] : mine;
        const int pos = p0 + 16 * (n >> 2) + 4 * g + (n & 3);
        if (pos < e.len)
            a.scores_out[row + pos] = (a.scores_in ? a.scores_in[row + pos] : 0.0f) + (page < 0 ? 0.0f : mine);
    }
}

}  // namespace tkv
