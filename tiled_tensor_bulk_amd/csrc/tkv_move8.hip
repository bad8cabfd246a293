// tkv_move8.hip -- new tokens into the 8-bit cache (append) and positions out of
// it (read).
//
// The keys and the values of a record, 32 positions of one head of one
// sequence, have a wave each.  Append: a lane takes units of 16 channels of a
// position as they lie in the rows (turned by the position, if asked for),
// the wave finds the largest magnitude of all, and with it the record's power of
// two; the codes change from rows to the record's order through LDS, as
// bytes, four channels' words of values by a transposition of 4 by 4 bytes.
// Where a record has earlier positions, its power is at least theirs, and
// where it grows their codes are rounded once more to it: exactly, but for
// those that become subnormal.  Read goes the other way.
//
// Memory bounds both: 8 sequences of up to 4001 positions, 8 heads of 128
// channels in fp16, 196 MB that move: append, turned, 47 us, 4.2 TB/s, read 36 us,
// 5.4 TB/s, beside 4.9 TB/s of a large copy.  Two waves a record, as the keys'
// and the values' powers and orders have nothing in common, leave a lane 64
// numbers of 16 bits, 32 registers, at a time (of 128 channels; of 64 half as
// many, of 256 twice).  A few tokens (append8_few_kernel:
// 32 sequences, one token each, 4.3 us) are a launch and four dependent loads:
// lengths, table, power and rows, of which none can be left out.
#include "tkv_rotate.h"

namespace tkv {

typedef float f2 __attribute__((ext_vector_type(2)));

// 4 numbers, already in units of the record's power, as codes: to nearest, ties
// to even.
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}

__device__ __forceinline__ void numbers_of(uint32_t w, float *x) {
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
}

// 4 codes in units 1 / f as large.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float f) {
    float x[4];
    numbers_of(w, x);
    return codes_of(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}

// The smallest E with top <= 448 * 2^(E - 127): 448 has a fraction of 1.75.
__device__ __forceinline__ int power_for(float top) {
    const int e = (int)((__builtin_bit_cast(uint32_t, top) + 0x1FFFFFu) >> 23) - 8;
    return e > kLeastPower ? e : kLeastPower;
}

__device__ __forceinline__ float largest(float v) {  // over the wave
#pragma unroll
    for (int mask = 1; mask < 64; mask <<= 1) v = fmaxf(v, __shfl_xor(v, mask));
    return v;
}

// Bytes of four words turned: byte j of word i becomes byte i of word j.
__device__ __forceinline__ void transpose(uint32_t (&w)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602);
    const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
    w[0] = __builtin_amdgcn_perm(c, a, 0x05040100);
    w[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
    w[2] = __builtin_amdgcn_perm(d, b, 0x05040100);
    w[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

__device__ __forceinline__ void wave_sync() {  // of what a wave's lanes have put into LDS
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int D>
struct Rows8 {  // how a record's rows lie on the lanes
    static constexpr int U = D / 16;                            // units of a row
    static constexpr int AT_ONCE = U <= 4 ? 16 : U <= 8 ? 8 : 4;  // rows: 48 lanes of 96 channels
    static constexpr int STEPS = kTile / AT_ONCE;
    static constexpr int PITCH = D + 8;                         // bytes of a row in LDS
};

// Which of a record's positions are there, as bits.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }

// A mask of bytes from 4 bits.
__device__ __forceinline__ uint32_t byte_mask(uint32_t bits) {
    return ((bits & 1) | (bits & 2) << 7 | (bits & 4) << 14 | (bits & 8) << 21) * 255u;
}

// Of a record that has no earlier positions and gets none, as the rotation's
// table turns none of its new ones: later ones may count them, and would take
// for its power what the byte was before.
__device__ __forceinline__ void no_power_yet(char *ex) { *reinterpret_cast<uint8_t *>(ex) = 0; }

template <int D, bool ROT>
__global__ void __launch_bounds__(64 * kMoveWaves) append8_kernel(const MoveArgs a) {
    using F = Format<D, 0>;
    using L = Rows8<D>;
    __shared__ __attribute__((aligned(16))) uint8_t bytes[kMoveWaves][kTile * L::PITCH];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const bool keys = __builtin_amdgcn_readfirstlane(wave & 1) == 0;
    Unit u;
    if (!unit_of(a, blockIdx.x * (kMoveWaves / 2) + (wave >> 1), u) || !u.rec) return;  // waves share nothing
    uint8_t *mine = bytes[wave];
    const int p0 = u.tile * kTile;
    const Tokens &from = keys ? a.k : a.v;
    const int unit = lane % L::U, sub = lane / L::U;
    const bool turned = ROT && keys && unit < a.rot.dim / 16;
    int c0 = 16 * unit, c1 = 16 * unit + 8;
    if (ROT && keys) unit_channels(a.rot, unit, c0, c1);

    uint4 lo[L::STEPS], hi[L::STEPS];
    int64_t turn[L::STEPS];
    bool live[L::STEPS];
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s) {
        const int i = p0 + s * L::AT_ONCE + sub - u.first;
        live[s] = sub < L::AT_ONCE && i >= 0 && i < u.n;
        const int64_t row = u.start + (live[s] ? i : 0);
        if (ROT) {
            turn[s] = turn_of(a.rot, row, (int64_t)u.first + i);
            live[s] = live[s] && turn[s] >= 0;
        }
        const int64_t at = row * from.token_stride + u.head * from.head_stride;
        lo[s] = load8_raw(from, at + c0), hi[s] = load8_raw(from, at + c1);
    }
    // earlier positions of the record, if there are any, and their power
    const uint32_t old = below(u.first - p0);
    char *const ex = u.rec + F::EX + (keys ? 0 : 1);
    const int had = old ? *reinterpret_cast<const uint8_t *>(ex) : 0;

    float x[L::STEPS][16], top = 0.0f;
    uint32_t mine_live = 0;
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s) {
        unit_floats(lo[s], hi[s], from.type, x[s]);
        if (turned && live[s]) {
            Turn t;
            t.load(a.rot, turn[s], unit);
            t.apply(a.rot.neighbours, x[s]);
        }
        if (live[s]) mine_live |= 1u << (s * L::AT_ONCE + sub);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            x[s][j] = limited(x[s][j]);
            if (live[s]) top = fmaxf(top, fabsf(x[s][j]));
        }
    }
    uint32_t fresh = mine_live;  // new positions, over the wave
#pragma unroll
    for (int mask = 1; mask < 64; mask <<= 1) fresh |= __shfl_xor(fresh, mask);
    if (!fresh) {  // all of them are left alone
        if (!old && lane == 0) no_power_yet(ex);
        return;
    }
    int e = power_for(largest(top));
    e = e > had ? e : had;
    const float inverse = power_of(254 - e), shrunk = power_of(had - e + 127);
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = codes_of(x[s][4 * j] * inverse, x[s][4 * j + 1] * inverse, x[s][4 * j + 2] * inverse,
                            x[s][4 * j + 3] * inverse);
        if (sub < L::AT_ONCE) {
            uint8_t *row = mine + (s * L::AT_ONCE + sub) * L::PITCH;
            *reinterpret_cast<uint2 *>(row + c0) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(row + c1) = make_uint2(w[2], w[3]);
        }
    }
    if (lane == 0) *reinterpret_cast<uint8_t *>(ex) = (uint8_t)e;
    wave_sync();
    const bool grown = old && had < e;
    if (keys) {
        // 16 bytes: 8 channels of two positions
#pragma unroll
        for (int i = 0; i < F::W; ++i) {
            const int item = i * 64 + lane, pair = item >> 5, at = (2 * item) & 63;  // of lanes at, at + 1
            const int t = 16 * (pair / F::W) + (at & 15), ch = 32 * (pair % F::W) + 8 * (at >> 4);
            const uint2 first = *reinterpret_cast<const uint2 *>(mine + t * L::PITCH + ch);
            const uint2 second = *reinterpret_cast<const uint2 *>(mine + (t + 1) * L::PITCH + ch);
            uint4 *to = reinterpret_cast<uint4 *>(u.rec + codes8_at(pair, at));
            const uint32_t both = 3u << t;
            if ((fresh & both) == both) {
                *to = make_uint4(first.x, first.y, second.x, second.y);
            } else if ((fresh | (grown ? old : 0)) & both) {
                uint4 w = *to;
                if (grown && (old >> t & 1)) w.x = rescaled(w.x, shrunk), w.y = rescaled(w.y, shrunk);
                if (grown && (old >> t & 2)) w.z = rescaled(w.z, shrunk), w.w = rescaled(w.w, shrunk);
                if (fresh >> t & 1) w.x = first.x, w.y = first.y;
                if (fresh >> t & 2) w.z = second.x, w.w = second.y;
                *to = w;
            }
        }
    } else {
        // 32 bytes: 8 positions of four channels
#pragma unroll
        for (int i = 0; i < (D + 63) / 64; ++i) {
            const int item = i * 64 + lane, g = (item >> 2) & 3, t = 4 * g;
            if (item >= D) break;
            const int ch = 16 * (item >> 4) + 4 * (item & 3);
            uint32_t w[2][4];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[half][j] = *reinterpret_cast<const uint32_t *>(mine + (16 * half + t + j) * L::PITCH + ch);
                transpose(w[half]);
            }
            uint4 *to = reinterpret_cast<uint4 *>(u.rec + F::VC + item * 32);
            const uint32_t m0 = byte_mask(fresh >> t & 15), m1 = byte_mask(fresh >> (t + 16) & 15);
            const uint32_t o0 = grown ? byte_mask(old >> t & 15) : 0, o1 = grown ? byte_mask(old >> (t + 16) & 15) : 0;
            if ((m0 & m1) != ~0u) {
                if (!(m0 | m1 | o0 | o1)) continue;
                const uint4 b0 = to[0], b1 = to[1];
                const uint32_t before[2][4] = {{b0.x, b0.z, b1.x, b1.z}, {b0.y, b0.w, b1.y, b1.w}};
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t o = half ? o1 : o0, m = half ? m1 : m0;
                        uint32_t b = before[half][j];
                        if (grown) b = (b & ~o) | (rescaled(b, shrunk) & o);
                        w[half][j] = (b & ~m) | (w[half][j] & m);
                    }
            }
            to[0] = make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]);
            to[1] = make_uint4(w[0][2], w[1][2], w[0][3], w[1][3]);
        }
    }
}

// Positions out of the cache.
template <int D>
__global__ void __launch_bounds__(64 * kMoveWaves) read8_kernel(const MoveArgs a) {
    using F = Format<D, 0>;
    using L = Rows8<D>;
    __shared__ __attribute__((aligned(16))) uint8_t bytes[kMoveWaves][kTile * L::PITCH];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const bool keys = __builtin_amdgcn_readfirstlane(wave & 1) == 0;
    Unit u;
    if (!unit_of(a, blockIdx.x * (kMoveWaves / 2) + (wave >> 1), u)) return;
    uint8_t *mine = bytes[wave];
    const int p0 = u.tile * kTile;
    const Tokens &to = keys ? a.k : a.v;
    float power = 0.0f;
    if (u.rec) {
        power = power_of(*reinterpret_cast<const uint8_t *>(u.rec + F::EX + (keys ? 0 : 1)));
        if (keys) {
            uint4 w[F::W];
#pragma unroll
            for (int i = 0; i < F::W; ++i) w[i] = reinterpret_cast<const uint4 *>(u.rec)[i * 64 + lane];
#pragma unroll
            for (int i = 0; i < F::W; ++i) {
                const int item = i * 64 + lane, pair = item >> 5, at = (2 * item) & 63;
                const int t = 16 * (pair / F::W) + (at & 15), ch = 32 * (pair % F::W) + 8 * (at >> 4);
                *reinterpret_cast<uint2 *>(mine + t * L::PITCH + ch) = make_uint2(w[i].x, w[i].y);
                *reinterpret_cast<uint2 *>(mine + (t + 1) * L::PITCH + ch) = make_uint2(w[i].z, w[i].w);
            }
        } else {
            constexpr int N = (D + 63) / 64;
            uint4 b[N][2];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint4 *at = reinterpret_cast<const uint4 *>(u.rec + F::VC + (i * 64 + lane) * 32);
                if (i * 64 + lane < D) b[i][0] = at[0], b[i][1] = at[1];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int item = i * 64 + lane, t = 4 * ((item >> 2) & 3), ch = 16 * (item >> 4) + 4 * (item & 3);
                if (item >= D) break;
                uint32_t w[2][4] = {{b[i][0].x, b[i][0].z, b[i][1].x, b[i][1].z}, {b[i][0].y, b[i][0].w, b[i][1].y, b[i][1].w}};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    transpose(w[half]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint32_t *>(mine + (16 * half + t + j) * L::PITCH + ch) = w[half][j];
                }
            }
        }
        wave_sync();
    }
    const int unit = lane % L::U, sub = lane / L::U;
    if (sub >= L::AT_ONCE) return;
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s) {
        const int t = s * L::AT_ONCE + sub, i = p0 + t - u.first;
        if (i < 0 || i >= u.n) continue;
        float x[16];
        if (u.rec) {
            const uint2 *w = reinterpret_cast<const uint2 *>(mine + t * L::PITCH + 16 * unit);
            numbers_of(w[0].x, x);
            numbers_of(w[0].y, x + 4);
            numbers_of(w[1].x, x + 8);
            numbers_of(w[1].y, x + 12);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= power;
        const int64_t at = (u.start + i) * to.token_stride + u.head * to.head_stride + 16 * unit;
        store8(to, at, x);
        store8(to, at + 8, x + 8);
    }
}

// A few new tokens: a wave has the keys or the values of a record's new
// positions, E channels of each in a lane, and stores their bytes where they
// belong; what a rescaling of the earlier positions costs is rare.
template <int D, bool ROT>
__global__ void __launch_bounds__(64 * kMoveWaves) append8_few_kernel(const MoveArgs a) {
    using F = Format<D, 0>;
    constexpr int E = D <= 128 ? 2 : 4;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if constexpr (ROT)
        if ((int)blockIdx.x >= a.move_blocks) {
            const int w = (blockIdx.x - a.move_blocks) * kMoveWaves + wave;
            rotate_queries<D, 1>(a, w / a.query_waves, w % a.query_waves, a.query_waves, lane);
            return;
        }
    const bool keys = __builtin_amdgcn_readfirstlane(wave & 1) == 0;
    Unit u;
    if (!unit_of(a, blockIdx.x * (kMoveWaves / 2) + (wave >> 1), u) || !u.rec) return;
    const int p0 = u.tile * kTile, ch = E * lane;
    const Tokens &from = keys ? a.k : a.v;
    const bool there = ch < D;
    const int first = u.first > p0 ? u.first : p0;
    const int n = (u.first + u.n < p0 + kTile ? u.first + u.n : p0 + kTile) - first;  // 1 .. kFewTokens
    const bool old = u.first > p0;
    char *const ex = u.rec + F::EX + (keys ? 0 : 1);
    const int had = old ? *reinterpret_cast<const uint8_t *>(ex) : 0;
    float x[kFewTokens][E], top = 0.0f;
    uint32_t live = 0;
#pragma unroll
    for (int k = 0; k < kFewTokens; ++k) {
        if (k >= n) break;
        const int64_t row = u.start + (first - u.first) + k;
        const int64_t at = row * from.token_stride + u.head * from.head_stride;
        const int64_t turn = ROT ? turn_of(a.rot, row, (int64_t)first + k) : 0;
        if (turn < 0) continue;
        live |= 1u << k;
#pragma unroll
        for (int j = 0; j < E; ++j)
            x[k][j] = there ? elem_to_float(((const uint16_t *)from.data)[at + ch + j], from.type) : 0.0f;
        if (ROT && keys && there) turn_few<E>(a, turn, at, ch, x[k]);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            x[k][j] = limited(x[k][j]);
            top = fmaxf(top, fabsf(x[k][j]));
        }
    }
    if (!live) {
        if (!old && lane == 0) no_power_yet(ex);
        return;
    }
    int e = power_for(largest(top));
    e = e > had ? e : had;
    if (old && had < e) {
        const float shrunk = power_of(had - e + 127);
        const uint32_t bits = below(u.first - p0);  // the earlier positions; others' codes stay
        uint4 *codes = reinterpret_cast<uint4 *>(u.rec + (keys ? 0 : F::VC));
        uint4 w[F::W];
#pragma unroll
        for (int i = 0; i < F::W; ++i) w[i] = codes[i * 64 + lane];
#pragma unroll
        for (int i = 0; i < F::W; ++i) {
            const int pair = i * 2 + (lane >> 5), at = (2 * lane) & 63;  // 8 codes each of lanes at, at + 1 of a run
            const uint32_t x = rescaled(w[i].x, shrunk), y = rescaled(w[i].y, shrunk);
            const uint32_t z = rescaled(w[i].z, shrunk), v = rescaled(w[i].w, shrunk);
            if (keys) {  // 8 channels of two positions
                const int t = 16 * (pair / F::W) + (at & 15);
                if (bits >> t & 1) w[i].x = x, w[i].y = y;
                if (bits >> t & 2) w[i].z = z, w[i].w = v;
            } else {  // 8 positions of two channels
                const uint32_t lo = byte_mask(bits >> 4 * (at >> 4) & 15), hi = byte_mask(bits >> (4 * (at >> 4) + 16) & 15);
                w[i].x = (w[i].x & ~lo) | (x & lo), w[i].y = (w[i].y & ~hi) | (y & hi);
                w[i].z = (w[i].z & ~lo) | (z & lo), w[i].w = (w[i].w & ~hi) | (v & hi);
            }
            codes[i * 64 + lane] = w[i];
        }
        // other lanes' stores to what is stored below have to be there first
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        wait_loads<0>();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    }
    if (lane == 0) *reinterpret_cast<uint8_t *>(ex) = (uint8_t)e;
    if (!there) return;
    const float inverse = power_of(254 - e);
#pragma unroll
    for (int k = 0; k < kFewTokens; ++k) {
        if (!(live >> k & 1)) continue;
        const int t = (first + k) & (kTile - 1);
        const uint32_t w = codes_of(x[k][0] * inverse, x[k][1] * inverse, E > 2 ? x[k][E - 2] * inverse : 0.0f,
                                    E > 2 ? x[k][E - 1] * inverse : 0.0f);
        if (keys) {
            char *to = u.rec + codes8_at(t / 16 * F::W + ch / 32, ch % 32 / 8 * 16 + t % 16) + ch % 8;
            if constexpr (E == 2)
                *reinterpret_cast<uint16_t *>(to) = (uint16_t)w;
            else
                *reinterpret_cast<uint32_t *>(to) = w;
        } else {
            char *to = u.rec + F::VC + codes8_at(ch / 16, t % 16 / 4 * 16 + ch % 16) + t % 4 + t / 16 * 4;
#pragma unroll
            for (int j = 0; j < E; ++j) reinterpret_cast<uint8_t *>(to)[8 * j] = (uint8_t)(w >> (8 * j));
        }
    }
}

template <int D>
static int launch_move8(const MoveArgs &a, bool append, void *stream) {
    const int64_t units = (int64_t)a.b.n_seq * a.tiles * a.c.heads;
    const dim3 block(64 * kMoveWaves), two_waves((uint32_t)((units * 2 + kMoveWaves - 1) / kMoveWaves));  // for a record
    hipStream_t s = (hipStream_t)stream;
    if (!append) {
        read8_kernel<D><<<two_waves, block, 0, s>>>(a);
    } else if (a.b.max_new <= kFewTokens && a.rot.dim) {
        MoveArgs both = a;  // and the queries
        both.move_blocks = (int)two_waves.x;
        const int64_t tokens = a.rot.q_heads ? (int64_t)a.b.n_seq * a.b.max_new : 0;
        both.query_waves = query_waves(a, tokens, kQueryHeads<D>);
        const dim3 all((uint32_t)(two_waves.x + (tokens * both.query_waves + kMoveWaves - 1) / kMoveWaves));
        append8_few_kernel<D, true><<<all, block, 0, s>>>(both);
    } else if (a.b.max_new <= kFewTokens) {
        append8_few_kernel<D, false><<<two_waves, block, 0, s>>>(a);
    } else if (a.rot.dim) {
        append8_kernel<D, true><<<two_waves, block, 0, s>>>(a);
    } else {
        append8_kernel<D, false><<<two_waves, block, 0, s>>>(a);
    }
    return (int)hipGetLastError();
}

static int move8(const MoveArgs &a, bool append, void *stream) {
    switch (a.c.dim) {
        case 64: return launch_move8<64>(a, append, stream);
        case 96: return launch_move8<96>(a, append, stream);
        case 128: return launch_move8<128>(a, append, stream);
        default: return launch_move8<256>(a, append, stream);
    }
}

int launch_append8(const MoveArgs &a, void *stream) { return move8(a, true, stream); }
int launch_read8(const MoveArgs &a, void *stream) { return move8(a, false, stream); }

}  // namespace tkv
