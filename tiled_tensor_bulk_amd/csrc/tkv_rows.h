// tkv_rows.h -- attention of many rows over the 4-bit cache: a chunk of a
// prompt, or all of a decoder's tokens over an encoder's states.
//
// Each of a workgroup's four waves holds NT tiles of 16 rows of its own and
// goes over all positions of the chunk, so what a record costs to unpack is
// shared: the waves unpack a quarter each of a step's records into LDS, as the
// matrix unit takes them, and read all of it back.  There are two stages: while
// one is read, the next one's words, which were loaded a step ahead, are
// unpacked into the other; one barrier a step.
//
// What is left for each row and position is fp32 work: with 128 channels in 2
// groups, for 16 rows and 32 positions, 16 fmas of scales, 8 fmas, 8
// exponentials (of 4 times an fma's time) and 8 additions of the softmax, 4
// maxima and 4 conversions, some 72 instruction slots of 4 cycles next to 19
// matrix instructions of 16.  So z * (sum of q) is one more matrix product: the
// sum of a row's q over a group is held as three fp16 numbers, 33 bits in all.
//
// Measured: 2 sequences of up to 8192 positions, the last 512 of them new, 8
// heads of 4 rows of 128 channels: 150 us, 640 TFLOP/s of products, where a
// large matrix product reaches 1160.  128 rows a workgroup (NT = 2) share an
// unpacked record: 177 us with 8 waves of 16, which read LDS twice as much, and
// 422 with 4 tiles a wave, which are out of registers.  A step of the softmax
// for each record, with V in registers, took 180.
#pragma once

#include "tkv_attend.h"

namespace tkv {

// z * (sum of q) is in units of 2^kSumBits, and so scales are held divided by that.
template <int D, int GROUP, int RECS>
struct Stage {
    using F = Format<D, GROUP>;
    h8 k[RECS][2][F::W][64];
    h8 v[RECS][2 * F::W][64];
    float ks[RECS][F::NG][kTile];
    h8 kz[RECS][kTile];          // a position's zeros, and 0 where there is no group
    uint32_t zs[RECS][2 * F::NG][kTile / 2];
};

// What a wave brings of a step's records: a quarter of the words, and of the
// pairs one each in a lane.
template <int D, int GROUP>
struct Share {
    using F = Format<D, GROUP>;
    uint32_t k[F::WV], v[F::WV];
    h8 scale[F::WV];
    uint32_t kpair, vpair;
    int p0;       // of its record
    bool there;   // the record's page exists, and some row sees it
    __device__ __forceinline__ void load(const AttendArgs &a, int page, int head, int pos, int hs, int lane) {
        p0 = pos;
        there = page >= 0;
        if (!there) return;
        const char *rec = record_at(a.c, page, head, pos / kTile);
        load_words<F::WV>(rec + (hs * 64 + lane) * F::WV * 4, k);
        load_words<F::WV>(rec + F::VC + (hs * 64 + lane) * F::WV * 4, v);
#pragma unroll
        for (int i = 0; i < F::WV; ++i)
            scale[i] = *reinterpret_cast<const h8 *>(rec + F::VP + ((hs * F::WV + i) / F::VG) * 128 + (lane >> 4) * 16);
        const int at = hs * 64 + lane;
        if (at < 32 * F::NG) {
            kpair = *reinterpret_cast<const uint32_t *>(rec + F::KP + 4 * at);
            vpair = *reinterpret_cast<const uint32_t *>(rec + F::VP + 4 * at);
        }
    }
    template <int RECS>
    __device__ __forceinline__ void unpack(Stage<D, GROUP, RECS> &to, int rec, int hs, int lane, int len) const {
        const int g = lane >> 4;
        if (there) {
#pragma unroll
            for (int i = 0; i < F::WV; ++i) to.k[rec][hs / F::S][(hs % F::S) * F::WV + i][lane] = codes_minus<0>(k[i]);
        }
        const int live = there ? len - p0 : 0;  // what lies past the sequence's end may be anything
        if (live >= kTile) {
#pragma unroll
            for (int i = 0; i < F::WV; ++i) to.v[rec][hs * F::WV + i][lane] = codes_minus<8>(v[i]) * scale[i];
        } else {
#pragma unroll
            for (int i = 0; i < F::WV; ++i) {
                h8 s = scale[i];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (4 * g + (j & 3) + 16 * (j >> 2) >= live) s[j] = (_Float16)0.0f;
                to.v[rec][hs * F::WV + i][lane] = codes_minus<8>(there ? v[i] : 0) * s;
            }
        }
        const int at = hs * 64 + lane;
        if (at < 32 * F::NG) {
            const int grp = at >> 5, pos = at & 31, slot = 2 * (at & 15);
            if (there) {
                const h2 pair = __builtin_bit_cast(h2, kpair);
                to.ks[rec][grp][pos] = (float)pair[0] * (1.0f / (1 << kSumBits));
                reinterpret_cast<_Float16 *>(&to.kz[rec][pos])[grp] = pair[1];
            }
            const int first = 4 * (slot >> 3) + (slot & 3) + 16 * ((slot >> 2) & 1);  // position of that slot
            uint32_t w = there ? vpair : 0;
            if (first >= live) w = 0;
            else if (first + 1 >= live) w &= 0xFFFFu;
            to.zs[rec][at >> 4][at & 15] = w;
        }
    }
};

// Pages of a step's records, -1 where there is none or past `end`.
template <int RECS>
struct StepPages {
    int page[RECS];
    __device__ __forceinline__ void load(const AttendArgs &a, const int32_t *table, Pages &pages, int pos, int end,
                                         int lane) {
#pragma unroll
        for (int i = 0; i < RECS; ++i)
            page[i] = pos + kTile * i < end ? pages.get(a, table, (pos + kTile * i) >> a.c.page_shift, lane) : -1;
    }
    __device__ __forceinline__ int of(int rec) const { return RECS == 1 || rec == 0 ? page[0] : page[RECS - 1]; }
};

template <int D, int GROUP, int NT, bool BF16>
__global__ void __launch_bounds__(64 * kAttendWaves, 2) rows_kernel(const AttendArgs a) {
    using F = Format<D, GROUP>;
    constexpr int R = 16 * NT * kAttendWaves;
    constexpr int RECS = 2 / F::S;  // with four runs of words, one for each wave
    constexpr int STEP = RECS * kTile;
    __shared__ Stage<D, GROUP, RECS> stage[2];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    int block, split, head, seq;
    place(a, block, split, head, seq);
    const int32_t *table = a.b.table + seq * a.b.table_stride;
    const Extent e(a, seq);
    const Chunks chunks(a, e.len);
    if (block * R >= e.rows || split >= chunks.n) return;
    const int t0 = split * chunks.size;
    Pages pages;
    pages.load(a, table, t0 >> a.c.page_shift, lane);
    const int r0 = block * R + wave * 16 * NT;

    // positions that some row of the workgroup sees, and of the wave
    const int last = block * R + R < e.rows ? block * R + R - 1 : e.rows - 1;
    int end = e.limit(a, divided(last, a.by_group_heads));
    end = end < t0 + chunks.size ? end : t0 + chunks.size;
    const int wave_last = r0 + 16 * NT < e.rows ? r0 + 16 * NT - 1 : e.rows - 1;
    const int wave_end = r0 < e.rows ? e.limit(a, divided(wave_last, a.by_group_heads)) : 0;
    const int all_see = r0 < e.rows ? e.limit(a, divided(r0, a.by_group_heads)) : 0;

    Row<D, GROUP> raw[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) raw[nt].load(a, e, head, r0 + 16 * nt + n, g, r0 + 16 * nt + n < e.rows);
    const int rec = wave / (2 * F::S), hs = wave % (2 * F::S);
    Share<D, GROUP> share;
    StepPages<RECS> step_now, step_next;
    step_now.load(a, table, pages, t0, end, lane);
    share.load(a, step_now.of(rec), head, t0 + rec * kTile, hs, lane);

    h8 q[NT][F::W], sums[NT];
    float factor[NT];
    int limit[NT];
    Softmax<D, GROUP> s[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + 16 * nt + n;
        limit[nt] = r < e.rows ? e.limit(a, divided(r, a.by_group_heads)) : 0;
        float qsum[F::NG], f;
        raw[nt].template operand<BF16>(a, q[nt], qsum, f);
        sums[nt] = sum_parts<D, GROUP>(qsum, g);
        factor[nt] = sums_factor(f);
        s[nt].clear();
        if (a.row_info && split == 0 && r0 / 16 + nt < a.row_tiles)
            keep_rows<D, GROUP>(a, ((int64_t)seq * a.c.heads + head) * a.row_tiles + r0 / 16 + nt, lane, q[nt],
                                sums[nt], factor[nt]);
    }
    for (int i = threadIdx.x; i < 2 * RECS * kTile; i += 64 * kAttendWaves)
        stage[i / (RECS * kTile)].kz[i / kTile % RECS][i % kTile] = (h8){0, 0, 0, 0, 0, 0, 0, 0};
    __syncthreads();
    share.unpack(stage[0], rec, hs, lane, e.len);
    step_next.load(a, table, pages, t0 + STEP, end, lane);
    share.load(a, step_next.of(rec), head, t0 + STEP + rec * kTile, hs, lane);
    __syncthreads();

    int now = 0;
    for (int p0 = t0; p0 < end; p0 += STEP, now ^= 1) {
        const Stage<D, GROUP, RECS> &from = stage[now];
        if (p0 < wave_end) {
            float x[NT][8 * RECS];
#pragma unroll
            for (int i = 0; i < RECS; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    f4 acc[NT][F::NG], y[NT];
                    const h8 kz = from.kz[i][16 * half + n];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        y[nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kz, sums[nt], (f4){0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < F::W; ++c) {
                        const h8 key = from.k[i][half][c][lane];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            acc[nt][c / F::KG] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                key, q[nt][c], c % F::KG ? acc[nt][c / F::KG] : (f4){0, 0, 0, 0}, 0, 0, 0);
                    }
#pragma unroll
                    for (int grp = 0; grp < F::NG; ++grp) {
                        const f4 ks = *reinterpret_cast<const f4 *>(&from.ks[i][grp][16 * half + 4 * g]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) y[nt][j] = fmaf(ks[j], acc[nt][grp][j], y[nt][j]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[nt][8 * i + 4 * half + j] = y[nt][j];
                }
            bool missing = false;
#pragma unroll
            for (int i = 0; i < RECS; ++i) missing |= step_now.page[i] < 0;
            if (p0 + STEP > all_see || missing) {  // some position is not seen by some row
#pragma unroll
                for (int j = 0; j < 8 * RECS; ++j) {
                    const int pos = p0 + kTile * (j >> 3) + 16 * ((j >> 2) & 1) + 4 * g + (j & 3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        if (pos >= limit[nt] || step_now.page[j >> 3] < 0) x[nt][j] = -__builtin_inff();
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
            h8 p[NT][RECS];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt].weights(x[nt], factor[nt], p[nt]);
#pragma unroll
            for (int i = 0; i < RECS; ++i) {
                h8 row = one_row<D, GROUP>(lane);
                if (n < 2 * F::NG) row = *reinterpret_cast<const h8 *>(&from.zs[i][n][4 * g]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[nt].z = __builtin_amdgcn_mfma_f32_16x16x32_f16(row, p[nt][i], s[nt].z, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 2 * F::W; ++c) {
                    const h8 value = from.v[i][c][lane];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        s[nt].o[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, p[nt][i], s[nt].o[c], 0, 0, 0);
                }
            }
        }
        share.unpack(stage[now ^ 1], rec, hs, lane, e.len);
        step_now = step_next;
        step_next.load(a, table, pages, p0 + 2 * STEP, end, lane);
        share.load(a, step_next.of(rec), head, p0 + 2 * STEP + rec * kTile, hs, lane);
        __syncthreads();
    }

    const int64_t unit = ((int64_t)seq * a.c.heads + head) * a.n_split + split;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        s[nt].finish(lane);
        const int row = r0 + 16 * nt + n;
        if (row >= e.rows) continue;
#pragma unroll
        for (int c = 0; c < 2 * F::W; ++c) {
            const int channel = 16 * c + 4 * g;
            if (a.n_split > 1) {
                const int64_t to = unit * a.rows + row;
                *reinterpret_cast<f4 *>(a.part_o + to * D + channel) = s[nt].o[c];
                if (channel == 0) a.part_ml[2 * to] = s[nt].m, a.part_ml[2 * to + 1] = s[nt].l;
            } else {
                write_row(a, e, seq, head, row, channel, s[nt].o[c], s[nt].m, s[nt].l);
            }
        }
    }
}

}  // namespace tkv
