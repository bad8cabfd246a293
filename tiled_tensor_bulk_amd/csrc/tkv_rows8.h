// tkv_rows8.h -- attention of many rows over the 8-bit cache: a chunk of a
// prompt, or all of a decoder's tokens over an encoder's states.
//
// As with 4 bits (tkv_rows.h) each of a workgroup's four waves holds NT tiles of
// 16 rows of its own and goes over all positions of the chunk; the waves convert
// a quarter each of a step's records into LDS, as fp16 numbers in the order in
// which the matrix unit takes them, and read all of it back; while one stage is
// read, the next one is filled.
//
// A record's one scale of the keys is a factor of its logarithms.  The values
// are held in units of a power of two that all waves raise alike when a record
// with a larger one comes; a wave's sums follow when it takes that step.
#pragma once

#include "tkv_rows.h"

namespace tkv {

template <int D, int RECS>
struct Stage8 {
    h8 k[RECS][2 * (D / 32)][64];
    h8 v[RECS][2 * (D / 32)][64];
};

// What a wave brings of a step's records: half of one's words, or a quarter.
template <int D, int PARTS>
struct Share8 {
    using F = Format<D, 0>;
    static constexpr int N = 2 * F::W / PARTS;
    uint2 k[N], v[N];
    int at;      // of its record
    bool there;  // the record's page exists, and some row sees it
    __device__ __forceinline__ void load(const AttendArgs &a, int page, int head, int position, int part, int lane) {
        at = position;
        there = page >= 0;
        if (!there) return;
        const char *rec = record_at(a.c, page, head, position / kTile);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            k[i] = *reinterpret_cast<const uint2 *>(rec + codes8_at(part * N + i, lane));
            v[i] = *reinterpret_cast<const uint2 *>(rec + F::VC + codes8_at(part * N + i, lane));
        }
    }
    // power: of the values in the units of the sums
    template <int RECS>
    __device__ __forceinline__ void unpack(Stage8<D, RECS> &to, int rec, int part, int lane, int len, float power) const {
        const int live = there ? len - at : 0;  // what lies past the sequence's end may be anything
        const uint2 mask = live_codes(live, lane);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (there) to.k[rec][part * N + i][lane] = codes8(k[i], 1.0f);
            const uint2 w = there ? v[i] : make_uint2(0, 0);
            to.v[rec][part * N + i][lane] = codes8(make_uint2(w.x & mask.x, w.y & mask.y), power);
        }
    }
};

// The powers of a step's records: the same in every wave.
template <int RECS>
struct Powers {
    uint32_t ex[RECS];
    template <int D>
    __device__ __forceinline__ void load(const AttendArgs &a, const View<true> &e, const StepPages<RECS> &pages, int head,
                                         int place) {
#pragma unroll
        for (int i = 0; i < RECS; ++i) {
            ex[i] = 0;
            if (pages.page[i] >= 0)
                ex[i] = *reinterpret_cast<const uint32_t *>(
                    record_at(a.c, pages.page[i], head, e.position(place + kTile * i) / kTile) + Format<D, 0>::EX);
        }
    }
    __device__ __forceinline__ int keys(int i) const { return __builtin_amdgcn_readfirstlane((int)(ex[i] & 255)); }
    __device__ __forceinline__ int values(int i) const { return __builtin_amdgcn_readfirstlane((int)((ex[i] >> 8) & 255)); }
};

template <int D, int NT, bool BF16>
__global__ void __launch_bounds__(64 * kAttendWaves, 2) rows8_kernel(const AttendArgs a) {
    using F = Format<D, 0>;
    constexpr int R = 16 * NT * kAttendWaves;
    constexpr int RECS = D > 128 ? 1 : 2, PARTS = kAttendWaves / RECS;
    constexpr int STEP = RECS * kTile;
    __shared__ Stage8<D, RECS> stage[2];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    int block, split, head, seq;
    place(a, block, split, head, seq);
    const int32_t *table = a.b.table + seq * a.b.table_stride;
    View<true> e(a, seq);
    if (block * R >= e.rows) return;
    e.narrow_to_block(a, block);
    const Chunks chunks(a, e.span());
    if (split >= chunks.n) return;
    const int t0 = split * chunks.size;
    Pages pages;
    pages.load(a, table, e.position(t0) >> a.c.page_shift, lane);
    const int r0 = block * R + wave * 16 * NT;

    // places that some row of the workgroup sees, and of the wave
    const int last = block * R + R < e.rows ? block * R + R - 1 : e.rows - 1;
    int end = e.place(e.limit(a, divided(last, a.by_group_heads)));
    end = end < t0 + chunks.size ? end : t0 + chunks.size;
    const int wave_last = r0 + 16 * NT < e.rows ? r0 + 16 * NT - 1 : e.rows - 1;
    const int wave_i1 = divided(wave_last, a.by_group_heads);
    const int wave_end = r0 < e.rows ? e.place(e.limit(a, wave_i1)) : 0;
    const int all_see = r0 < e.rows ? e.limit(a, divided(r0, a.by_group_heads)) : 0;

    Row<D, 0> raw[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) raw[nt].load(a, e, head, r0 + 16 * nt + n, g, r0 + 16 * nt + n < e.rows);
    const int rec = wave / PARTS, part = wave % PARTS;
    Share8<D, PARTS> share;
    Powers<RECS> powers;
    StepPages<RECS> step_now, step_next;
    step_now.load(a, e, table, pages, t0, end, lane);
    share.load(a, step_now.of(rec), head, e.position(t0 + rec * kTile), part, lane);
    powers.template load<D>(a, e, step_now, head, t0);

    h8 q[NT][F::W];
    float factor[NT];
    Sight<true> sight[NT];
    Softmax<D, 0> s[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        sight[nt].load(a, e, r0 + 16 * nt + n);
        float none[1];
        raw[nt].template operand<BF16>(a, q[nt], none, factor[nt]);
        s[nt].clear();
    }
    int units = 0;                        // of the wave's sums: 2^(units - 127)
    int stage_units = 0, next_units = 0;  // of the stage that is read, and of the one that is filled
    float of_keys[RECS], next_keys[RECS];
    const auto fill = [&](Stage8<D, RECS> &to) {
        int own = 0;
#pragma unroll
        for (int i = 0; i < RECS; ++i) {
            const int v = powers.values(i);
            next_units = v > next_units ? v : next_units;
            own = i == rec ? v : own;
            next_keys[i] = power_of(powers.keys(i));
        }
        share.unpack(to, rec, part, lane, e.len, power_of(own - next_units + 127));
    };
    fill(stage[0]);
    step_next.load(a, e, table, pages, t0 + STEP, end, lane);
    share.load(a, step_next.of(rec), head, e.position(t0 + STEP + rec * kTile), part, lane);
    powers.template load<D>(a, e, step_next, head, t0 + STEP);
    __syncthreads();

    int now = 0;
    for (int p0 = t0; p0 < end; p0 += STEP, now ^= 1) {
        const Stage8<D, RECS> &from = stage[now];
        stage_units = next_units;
        int at[RECS];  // positions of the step's records
        bool windowed = false;
#pragma unroll
        for (int i = 0; i < RECS; ++i) {
            of_keys[i] = next_keys[i];
            at[i] = e.position(p0 + kTile * i);
            windowed |= e.windowed(a, wave_i1, at[i]);
        }
        if (p0 < wave_end) {
            if (stage_units > units) {
                const float shrunk = units ? __builtin_amdgcn_ldexpf(1.0f, units - stage_units) : 1.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[nt].rescale(shrunk);
                units = stage_units;
            }
            float x[NT][8 * RECS];
#pragma unroll
            for (int i = 0; i < RECS; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    f4 acc[NT];
#pragma unroll
                    for (int c = 0; c < F::W; ++c) {
                        const h8 key = from.k[i][half * F::W + c][lane];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[nt][c],
                                                                             c ? acc[nt] : (f4){0, 0, 0, 0}, 0, 0, 0);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[nt][8 * i + 4 * half + j] = acc[nt][j] * of_keys[i];
                }
            bool missing = false;
#pragma unroll
            for (int i = 0; i < RECS; ++i) missing |= step_now.page[i] < 0;
            if (at[RECS - 1] + kTile > all_see || missing || windowed) {  // some position is not seen by some row
#pragma unroll
                for (int j = 0; j < 8 * RECS; ++j) {
                    const int pos = at[j >> 3] + 16 * ((j >> 2) & 1) + 4 * g + (j & 3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        if (step_now.page[j >> 3] < 0 || !sight[nt].sees(a, e, pos)) x[nt][j] = -__builtin_inff();
                }
            }
            bool grown = false;
            float top[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                top[nt] = Softmax<D, 0>::top(x[nt]) * factor[nt];
                grown |= top[nt] > s[nt].m + kSlack;
            }
            if (__any(grown)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[nt].grow(top[nt]);
            }
            h8 p[NT][RECS];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt].weights(x[nt], factor[nt], p[nt]);
            const h8 ones = {1, 1, 1, 1, 1, 1, 1, 1};
#pragma unroll
            for (int i = 0; i < RECS; ++i) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[nt].z = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p[nt][i], s[nt].z, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 2 * F::W; ++c) {
                    const h8 value = from.v[i][c][lane];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        s[nt].o[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, p[nt][i], s[nt].o[c], 0, 0, 0);
                }
            }
        }
        fill(stage[now ^ 1]);
        step_now = step_next;
        step_next.load(a, e, table, pages, p0 + 2 * STEP, end, lane);
        share.load(a, step_next.of(rec), head, e.position(p0 + 2 * STEP + rec * kTile), part, lane);
        powers.template load<D>(a, e, step_next, head, p0 + 2 * STEP);
        __syncthreads();
    }

    const int64_t unit = ((int64_t)seq * a.c.heads + head) * a.n_split + split;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        s[nt].finish(lane, power_of(units));
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
