// tkv_rows8.h -- attention of many rows over the 8-bit cache: a chunk of a
// prompt, or all of a decoder's tokens over an encoder's states.
//
// A workgroup's four waves hold 32 rows each and go over all positions of the
// chunk, a record at a time.  Each wave converts its part of the next
// record's words into LDS, as fp16 numbers in the order in which the matrix unit
// takes them, and all read all of it back; there are two stages and one barrier
// a record, and a word is asked for a record before it is converted.
//
// Products.  v_mfma_f32_32x32x16_f16 with the cache as the left operand: S^T = K
// Q^T leaves in a lane 16 positions of one row, which are its part of the right
// operand of O^T = V^T P^T where V's positions are put into that order.  Tiles
// of 32 rows take half as many matrix instructions as tiles of 16, and a row's
// maximum, factor and sum are one number a lane.
//
// A record's one scale of the keys is a factor of its logarithms.  The values
// are held in units of a power of two that all waves raise alike when a record
// with a larger one comes; a wave's sums follow when they take that record.
//
// What bounds it: by its counters a record takes a wave 124 vector instructions,
// 630 cycles of issue (16 exponentials, at four times an fma's, are 256 of them),
// and 512 cycles of matrix instructions, of 1500 that a SIMD has for them.  Of
// what neither fills, a record's barrier and its branches are the cause, which
// three waves on a SIMD (168 registers) hide better than two that make one
// record's products beside another's softmax (137 us against 160).  128 channels,
// 8 heads of 4 rows, with the joining: 512 new tokens each over 2 sequences of up
// to 8192 positions 141 us, 675 TFLOP/s, where the longer one's workgroups are the
// last ones; 6000 tokens through a window of 1024 138 us, 680 TFLOP/s.  Tiles of
// 16 rows, as with 4 bits, took 143 and 171.
//
// 256 channels (304 TFLOP/s, 4 heads of 2 rows, the first of these) leave one wave
// on a SIMD, and the products' sums in accumulation registers.
#pragma once

#include "tkv_rows.h"

namespace tkv {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));

// Two records.  Keys lie as the record's words do; of values 32 channels (v[..][b])
// by 16 positions (s): lane 32 h + c has channel c, positions 16 s + 4 h + 0..3
// and 8 more.
template <int D>
struct Stage8 {
    h8 k[2][2][D / 32][64];
    h8 v[2][D / 32][2][64];
};

// A record: where it lies, and its powers.  The same in every lane.  Of one that
// is not there (past `end`, or without a page) page 0's is read, and dropped.
template <int D>
struct Record8 {
    const char *at;
    int position;
    bool there;
    uint32_t ex;
    __device__ __forceinline__ void find(const AttendArgs &a, const View<true> &e, const int32_t *table, Pages &pages, int head,
                                         int place, int end, int lane) {
        position = e.position(place);
        const int page = place < end ? pages.get(a, table, position >> a.c.page_shift, lane) : -1;
        there = page >= 0;
        at = record_at(a.c, there ? page : 0, head, (int)((uint32_t)position / kTile));
        ex = *reinterpret_cast<const uint16_t *>(at + Format<D, 0>::EX);
    }
    __device__ __forceinline__ void settle() { ex = (uint32_t)__builtin_amdgcn_readfirstlane((int)ex); }
    __device__ __forceinline__ int keys() const { return (int)(ex & 255); }
    __device__ __forceinline__ int values() const { return there ? (int)(ex >> 8) : 0; }
};

// What a wave brings of a record's keys, or values: words wave, wave + 4, ..
// of the record's 2 * (D / 32); past the last one, that again.
template <int D>
struct Share8 {
    static constexpr int WORDS = 2 * (D / 32), COUNT = (WORDS + kAttendWaves - 1) / kAttendWaves;
    uint2 w[COUNT];
    static __device__ __forceinline__ int which(int i, int wave) {
        const int word = wave + i * kAttendWaves;
        return WORDS % kAttendWaves && word >= WORDS ? WORDS - 1 : word;
    }
    __device__ __forceinline__ void load(const char *codes, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) load_one(i, codes, wave, lane);
    }
    __device__ __forceinline__ void load_one(int i, const char *codes, int wave, int lane) {
        w[i] = *reinterpret_cast<const uint2 *>(codes + codes8_at(which(i, wave), lane));
    }
    __device__ __forceinline__ void unpack_keys(int i, h8 (&to)[2][D / 32][64], int wave, int lane) {
        asm volatile("" : "+v"(w[i].x), "+v"(w[i].y));  // here, not where it has come
        (&to[0][0])[which(i, wave)][lane] = codes8(w[i], 1.0f);
    }
    // power: what the codes are multiplied with
    __device__ __forceinline__ void unpack_values(int i, h8 (&to)[D / 32][2][64], int wave, int lane, float power) {
        asm volatile("" : "+v"(w[i].x), "+v"(w[i].y));
        const int word = which(i, wave), g = lane >> 4, m = lane & 15;
        const h8 x = codes8(w[i], power);
        h8 *at = to[word >> 1][0] + 32 * (g & 1) + 16 * (word & 1) + m;
        reinterpret_cast<h4 *>(at)[g >> 1] = (h4){x[0], x[1], x[2], x[3]};
        reinterpret_cast<h4 *>(at + 64)[g >> 1] = (h4){x[4], x[5], x[6], x[7]};
    }
    __device__ __forceinline__ void keep(uint2 mask) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) w[i].x &= mask.x, w[i].y &= mask.y;
    }
};

// Sum and maximum over the two lanes of a row.
template <class Op>
__device__ __forceinline__ float over_halves(float v, Op op) {
    float a = v, b = v;
    asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(b));
    return op(a, b);
}
__device__ __forceinline__ float over_halves_sum(float v) {
    return over_halves(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float over_halves_max(float v) {
    return over_halves(v, [](float a, float b) { return fmaxf(a, b); });
}

// A row as the right operand: lane 32 h + n has channels 16 c + 8 h .. of row n;
// and what turns products into logarithms to base 2 (Row::operand of 16 rows).
template <int D, bool BF16>
__device__ __forceinline__ float wide_operand(const AttendArgs &a, const uint4 (&raw)[D / 16], h8 (&q)[D / 16]) {
    const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0;  // moves into q
    float x[D / 16][8], top = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        raw_to_float<BF16>(make_uint4(raw[c].x ^ sign, raw[c].y ^ sign, raw[c].z ^ sign, raw[c].w ^ sign), x[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (BF16) top = fmaxf(top, fabsf(x[c][j]));
    }
    int power = 0;
    if constexpr (BF16) {
        top = over_halves_max(top);
        if (top > 0.0f && top < __builtin_inff()) power = 15 - __builtin_amdgcn_frexp_expf(top);
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) q[c][j] = (_Float16)(BF16 ? ldexpf(x[c][j], power) : x[c][j]);
    return fminf(fmaxf(fabsf(ldexpf(a.scale_log2, -power)), 0x1p-126f), 0x1.fffffep127f);
}

// Waves of a SIMD that the registers are to suffice for.
constexpr int rows8_waves(int d) { return d > 128 ? 1 : d > 64 ? 3 : 4; }

// Sums that are made by here, and not later.  A kernel of more than 256
// registers has products in the accumulation registers.
template <int D>
__device__ __forceinline__ void here(f16v &x) {
    if constexpr (rows8_waves(D) == 1)
        asm volatile("" : "+a"(x));
    else
        asm volatile("" : "+v"(x));
}

// 4 numbers rounded to 16 bits.
template <bool BF16>
__device__ __forceinline__ uint2 packed(f4 x) {
    if constexpr (BF16) {
        typedef __bf16 b4 __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(uint2, __builtin_convertvector(x, b4));
    } else {
        return __builtin_bit_cast(uint2, __builtin_convertvector(x, h4));
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(64 * kAttendWaves, rows8_waves(D)) rows8_kernel(const AttendArgs a) {
    using F = Format<D, 0>;
    using Share = Share8<D>;
    constexpr int R = 32 * kAttendWaves, W = F::W;
    constexpr int FRAGS = 2 * W;  // operands of a record's keys, of 16 channels, and of its values
    __shared__ Stage8<D> stage;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, h = lane >> 5, n = lane & 31;
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
    const int r0 = block * R + wave * 32, row = r0 + n;

    // places that some row of the workgroup sees
    const int last = block * R + R < e.rows ? block * R + R - 1 : e.rows - 1;
    int end = e.place(e.limit(a, divided(last, a.by_group_heads)));
    end = end < t0 + chunks.size ? end : t0 + chunks.size;
    const int wave_last = r0 + 32 < e.rows ? r0 + 31 : e.rows - 1;
    const int wave_i1 = divided(wave_last, a.by_group_heads);
    const int all_see = r0 < e.rows ? e.limit(a, divided(r0, a.by_group_heads)) : 0;

    int token = row < e.rows ? row : 0, query = token;  // the first row is read for one that is not there, and dropped
    token = divide(query, a.group_heads, a.by_group_heads);
    query += head * a.group_heads;
    uint4 raw[FRAGS];
    {
        const int64_t at = (e.start + token) * a.q.token_stride + query * a.q.head_stride + 8 * h;
#pragma unroll
        for (int c = 0; c < FRAGS; ++c) raw[c] = load8_raw(a.q, at + 16 * c);
    }

    Record8<D> now, next1, next2;
    Share keys, values;  // of record i + 1
    const auto find = [&](Record8<D> &r, int at) { r.find(a, e, table, pages, head, at, end, lane); };
    const auto drop_end = [&](const Record8<D> &r) {  // of values: what lies past the sequence's end may be anything
        const int live = r.there ? e.len - r.position : 0;
        if (live < kTile) values.keep(live_codes(live, lane));
    };
    find(now, t0);
    find(next1, t0 + kTile);
    keys.load(now.at, wave, lane);
    values.load(now.at + F::VC, wave, lane);
    now.settle(), next1.settle();
    // sums are in units of 2^(units - 127), 0 while nothing but zeros has been summed, and values in those of the
    // largest power up to them
    int units = 0, units_now = now.values();
    drop_end(now);
#pragma unroll
    for (int i = 0; i < Share::COUNT; ++i) {
        keys.unpack_keys(i, stage.k[0], wave, lane);
        values.unpack_values(i, stage.v[0], wave, lane, power_in(units_now, units_now));
    }
    keys.load(next1.at, wave, lane);
    values.load(next1.at + F::VC, wave, lane);

    h8 q[FRAGS];
    if (row >= e.rows) {
#pragma unroll
        for (int c = 0; c < FRAGS; ++c) raw[c] = make_uint4(0, 0, 0, 0);
    }
    const float factor = wide_operand<D, BF16>(a, raw, q);
    Sight<true> sight;
    sight.load(a, e, row);
    float m = kFar, l = 0.0f, z = 0.0f;
    f16v o[W];
#pragma unroll
    for (int b = 0; b < W; ++b) o[b] = (f16v)0.0f;
    __syncthreads();

    // Operands come from LDS some products before they are multiplied with, and between the products stands what the
    // vector unit can do beside them: all written down in that order, and held to it by empty assembly, as the compiler
    // puts reads next to their products, and all of a softmax behind them.
    constexpr int AHEAD = 2;
    h8 frag[2 * FRAGS];  // operands of keys, then of values
    const int key_lane = ((n >> 4) * W) * 64 + 16 * h + (n & 15);  // of keys' operand c: position n, channels 16 c + 8 h ..
    const auto ask = [&](int c, int from) {
        if (c < FRAGS)
            frag[c] = (&stage.k[from][0][0][0])[key_lane + (c >> 1) * 64 + (c & 1) * 32];
        else if (c < 2 * FRAGS)
            frag[c] = stage.v[from][(c - FRAGS) % W][(c - FRAGS) / W][lane];
    };
    const auto scale_sums = [&](float f) {
#pragma unroll
        for (int b = 0; b < W; ++b) o[b] *= f;
    };
    int odd = 0;
    for (int p0 = t0; p0 < end; p0 += kTile, odd ^= 1) {
#pragma unroll
        for (int c = 0; c < AHEAD; ++c) ask(c, odd);
        find(next2, p0 + 2 * kTile);
        drop_end(next1);
        const int units_next = next1.values() > units_now ? next1.values() : units_now;
        const float power = power_in(next1.values(), units_next);
        if (units_now > units) {
            if (units) scale_sums(__builtin_amdgcn_ldexpf(1.0f, units - units_now));
            units = units_now;
        }
        const float f = fminf(fmaxf(factor * power_of(now.keys()), 0x1p-126f), 0x1.fffffep127f);
        __builtin_amdgcn_sched_barrier(0);
        f16v x = (f16v)0.0f;
#pragma unroll
        for (int c = 0; c < FRAGS; ++c) {
            x = __builtin_amdgcn_mfma_f32_32x32x16_f16(frag[c], q[c], x, 0, 0, 0);
            here<D>(x);
            ask(c + AHEAD, odd);
            // a word is asked for again where it has been unpacked: it has a step to come
#pragma unroll
            for (int i = 2 * Share::COUNT * c / FRAGS; i < 2 * Share::COUNT * (c + 1) / FRAGS; ++i) {
                if (i < Share::COUNT) {
                    keys.unpack_keys(i, stage.k[odd ^ 1], wave, lane);
                    keys.load_one(i, next2.at, wave, lane);
                } else {
                    values.unpack_values(i - Share::COUNT, stage.v[odd ^ 1], wave, lane, power);
                    values.load_one(i - Share::COUNT, next2.at + F::VC, wave, lane);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if ((now.position + kTile > all_see) | !now.there | e.windowed(a, wave_i1, now.position))
            sight.mask(a, e, now.position, !now.there, h, x);  // some position is not seen by some row
        float peak = fmaxf(x[0], x[1]);
#pragma unroll
        for (int j = 2; j < 16; j += 2) peak = fmaxf(fmaxf(peak, x[j]), x[j + 1]);
        if (__any(peak * f > m + kSlack)) {
            const float t = over_halves_max(peak * f), m1 = t > m + kSlack ? t : m;
            const float shrunk = __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= shrunk;
            z *= shrunk;
            scale_sums(shrunk);
        }
        __builtin_amdgcn_sched_barrier(0);
        const float lift = kLift - m;
        float sum = 0.0f;
        const h2 ones = {(_Float16)1.0f, (_Float16)1.0f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            h2 weight[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w0 = __builtin_amdgcn_exp2f(fmaf(x[8 * s + 2 * j], f, lift));
                const float w1 = __builtin_amdgcn_exp2f(fmaf(x[8 * s + 2 * j + 1], f, lift));
                sum += w0;
                sum += w1;
                weight[j] = (h2){(_Float16)w0, (_Float16)w1};
                z = __builtin_amdgcn_fdot2(weight[j], ones, z, false);
            }
            const h8 p = {weight[0][0], weight[0][1], weight[1][0], weight[1][1],
                          weight[2][0], weight[2][1], weight[3][0], weight[3][1]};
#pragma unroll
            for (int b = 0; b < W; ++b) {
                const int c = FRAGS + s * W + b;
                o[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(frag[c], p, o[b], 0, 0, 0);
                here<D>(o[b]);
                ask(c + AHEAD, odd);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        l += sum;
        asm volatile("" : "+v"(z), "+v"(l));  // here, not where they are looked at
        now = next1, next1 = next2;
        next1.settle();
        units_now = units_next;
        __syncthreads();
    }

    // what a division by l makes the output: so by the sum of the rounded weights
    l = over_halves_sum(l);
    z = over_halves_sum(z);
    scale_sums(z > 0.0f ? l / z * power_of(units) : power_of(units));
    if (row >= e.rows) return;
    const auto quad = [&](int c) {  // channels 8 c + 4 h ..
        return (f4){o[c >> 2][4 * (c & 3)], o[c >> 2][4 * (c & 3) + 1], o[c >> 2][4 * (c & 3) + 2], o[c >> 2][4 * (c & 3) + 3]};
    };
    if (a.n_split > 1) {
        const int64_t to = (((int64_t)seq * a.c.heads + head) * a.n_split + split) * a.rows + row;
        float *out = a.part_o + to * D + 4 * h;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) *reinterpret_cast<f4 *>(out + 8 * c) = quad(c);
        if (h == 0) *reinterpret_cast<float2 *>(a.part_ml + 2 * to) = make_float2(m, l);
    } else {
        scale_sums(l > 0.0f || l != l ? 1.0f / l : 0.0f);
        uint16_t *out = (uint16_t *)a.out.data + (e.start + token) * a.out.token_stride + query * a.out.head_stride + 4 * h;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint2 w = packed<BF16>(quad(c));
            if (a.out.wide) {
                *reinterpret_cast<uint2 *>(out + 8 * c) = w;
            } else {
                out[8 * c] = (uint16_t)w.x, out[8 * c + 1] = (uint16_t)(w.x >> 16);
                out[8 * c + 2] = (uint16_t)w.y, out[8 * c + 3] = (uint16_t)(w.y >> 16);
            }
        }
        if (h == 0)  // log2(0) = -inf: nothing seen
            a.lse[(e.start + token) * (a.c.heads * a.group_heads) + query] = (m - kLift + log2f(l)) * 0.69314718056f;
    }
}

}  // namespace tkv
