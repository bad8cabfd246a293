// tkv_move.hip -- new tokens into the cache (append) and positions out of it
// (read).
//
// A record, 32 positions of one head of one sequence, has two waves, one for
// its keys and one for its values; of a few new tokens one wave takes both.  A K
// word belongs to one position, but a V word holds 8 positions of a channel,
// so one wave owns a record's V words: where some of a word's positions are not
// new, it reads the word, replaces the new nibbles and writes it back, with no
// atomics.  Rows are read as the K operand lies (lane 16 g + m: position m,
// channels 32 i + 8 g ..); V codes change places through LDS, as bytes.
//
// What bounds them: memory, at two bytes of input (or four of output) for each
// half byte of cache, and in append next to it the vector units, which take some
// 17 instructions to quantise an element, and the code's size: the exact
// comparison is there for every word, 39 KB in all with 128 channels, and 75 with
// 256, where the instruction cache holds 64 for two compute units.  8 prompts of up to 4001 tokens, 25
// thousand in all, 8 heads of 128 channels: append 47 us for 131 MB, 2.8 TB/s, of
// which the instructions alone are 29; read into fp32 42 us for 234 MB, 5.5 TB/s.
// 4 heads of 256 channels, as many bytes: append 56 us (242 registers, two
// waves a SIMD), read 49; 8 heads of 96: 33 and 31.
#include "tkv_format.h"

namespace tkv {

constexpr int kMoveWaves = kBlockThreads / 64;

// Nearest whole numbers to (x - z) / s within 0..15, ties to even.  The
// quotient in fp32 is within 1e-5 of the true one, so only one that close to a
// border needs the exact comparison, in fp64, where products of an fp16 number
// and a small integer, and differences of fp16 and bf16 numbers, are exact; a
// lane goes there when one of its N is.
template <int N>
__device__ __forceinline__ void codes_of(const float *x, float z, float s, float *c) {
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    float off = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float t = (x[i] - z) * inv;
        c[i] = rintf(t);
        off = fmaxf(off, fabsf(t - c[i]));
    }
    if (off > 0.4999f) {
        for (int i = 0; i < N; ++i) {
            const float t = (x[i] - z) * inv, low = floorf(t);
            if (fabsf(t - low - 0.5f) < 1e-4f && t > 0.0f && t < 15.0f) {
                const double twice = 2.0 * ((double)x[i] - (double)z);
                const double border = (2.0 * (double)low + 1.0) * (double)s;
                const int k = (int)low;
                c[i] = (float)(twice > border ? k + 1 : twice < border ? k : k + (k & 1));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = fminf(fmaxf(c[i], 0.0f), 15.0f);
}
// 8 codes as a word: two sums of 16 bits, exact in fp32.
__device__ __forceinline__ uint32_t word_of(const float *c) {
    const float lo = fmaf(fmaf(fmaf(c[6], 16.0f, c[4]), 16.0f, c[2]), 16.0f, c[0]);
    const float hi = fmaf(fmaf(fmaf(c[7], 16.0f, c[5]), 16.0f, c[3]), 16.0f, c[1]);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
static_assert(nibble_of(0) == 0 && nibble_of(2) == 1 && nibble_of(4) == 2 && nibble_of(6) == 3 && nibble_of(1) == 4 &&
                  nibble_of(3) == 5 && nibble_of(5) == 6 && nibble_of(7) == 7, "even codes, then odd ones");

__device__ __forceinline__ void scale_of(float lo, float hi, _Float16 &scale, _Float16 &zero) {
    scale = (_Float16)((hi - lo) / 15.0f);
    zero = (_Float16)lo;
}

// Quantise one position's channels: lane group g holds channels 32 i + 8 g + j
// in x[8 i + j]; the four lanes of a position share its scales.
template <int D, int GROUP>
__device__ __forceinline__ void quantise(const float *x, _Float16 *scale, _Float16 *zero, float *code) {
    using F = Format<D, GROUP>;
#pragma unroll
    for (int grp = 0; grp < F::NG; ++grp) {
        const float *y = x + grp * F::KG * 8;
        float lo = y[0], hi = y[0];
#pragma unroll
        for (int i = 1; i < F::KG * 8; ++i) lo = fminf(lo, y[i]), hi = fmaxf(hi, y[i]);
#pragma unroll
        for (int mask = 16; mask <= 32; mask <<= 1) {
            lo = fminf(lo, __shfl_xor(lo, mask));
            hi = fmaxf(hi, __shfl_xor(hi, mask));
        }
        scale_of(lo, hi, scale[grp], zero[grp]);
#pragma unroll
        for (int i = 0; i < F::KG; ++i)
            codes_of<8>(y + 8 * i, (float)zero[grp], (float)scale[grp], code + (grp * F::KG + i) * 8);
    }
}

__device__ __forceinline__ float limited(float y) { return y != y ? 0.0f : fminf(fmaxf(y, -kLimit), kLimit); }

// A row's channels 32 i + 8 g .. as they lie.
template <int D>
__device__ __forceinline__ void load_row(const Tokens &t, int64_t row, int head, int g, uint4 (&raw)[D / 32]) {
    const int64_t at = row * t.token_stride + head * t.head_stride + 8 * g;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) raw[i] = load8_raw(t, at + 32 * i);
}

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

// Codes, scales and zeros of one position's channels, from its row.
template <int D, int GROUP>
__device__ __forceinline__ void quantise_row(const uint4 (&raw)[D / 32], int type, _Float16 *scale, _Float16 *zero,
                                             float *code) {
    float x[D / 4];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        if (type == kBf16)
            raw_to_float<true>(raw[i], x + 8 * i);
        else
            raw_to_float<false>(raw[i], x + 8 * i);
    }
#pragma unroll
    for (int j = 0; j < D / 4; ++j) x[j] = limited(x[j]);
    quantise<D, GROUP>(x, scale, zero, code);
}

// Many new tokens: of two waves on a record one takes the keys and one the
// values.  Each asks for all its rows before it works on the first: with both
// in one wave and one row at a time a prompt waited for memory four times over.
template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kMoveWaves) append_kernel(const MoveArgs a) {
    using F = Format<D, GROUP>;
    constexpr int PITCH = D + 4;  // bytes of a row in LDS, off a multiple of the banks
    __shared__ uint8_t codes[kMoveWaves / 2][16 * PITCH];  // V codes of positions m and m + 16 in a byte
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const bool keys = __builtin_amdgcn_readfirstlane(wave & 1) == 0;
    Unit u;
    if (!unit_of(a, blockIdx.x * (kMoveWaves / 2) + (wave >> 1), u) || !u.rec) return;  // waves share nothing
    uint8_t *mine = codes[wave >> 1];
    const int p0 = u.tile * kTile;
    const Tokens &from = keys ? a.k : a.v;
    uint4 raw[2][F::W];
    bool live[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = p0 + 16 * half + m - u.first;
        live[half] = i >= 0 && i < u.n;  // the four lanes of a position are live together
        load_row<D>(from, u.start + (live[half] ? i : 0), u.head, g, raw[half]);
    }
    _Float16 scale[F::NG], zero[F::NG];
    if (keys) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float code[D / 4];
            quantise_row<D, GROUP>(raw[half], from.type, scale, zero, code);
            if (!live[half]) continue;
            uint32_t word[F::W];
#pragma unroll
            for (int w = 0; w < F::W; ++w) word[w] = word_of(code + 8 * w);
#pragma unroll
            for (int s = 0; s < F::S; ++s)
                store_words<F::WV>(u.rec + (((half * F::S + s) * 64 + lane) * F::WV) * 4, word + s * F::WV);
            if (g == 0) {
#pragma unroll
                for (int grp = 0; grp < F::NG; ++grp)
                    *reinterpret_cast<h2 *>(u.rec + F::KP + (grp * kTile + 16 * half + m) * 4) =
                        (h2){scale[grp], zero[grp]};
            }
        }
        return;
    }
    uint32_t low[2 * F::W];  // four channels' codes in a word's bytes, of the first half
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float code[D / 4];
        quantise_row<D, GROUP>(raw[half], from.type, scale, zero, code);
        if (live[half] && g == 0) {
            const int slot = 8 * (m >> 2) + 4 * half + (m & 3);
#pragma unroll
            for (int grp = 0; grp < F::NG; ++grp) {
                _Float16 *to = reinterpret_cast<_Float16 *>(u.rec + F::VP) + grp * 64 + slot;
                to[0] = scale[grp], to[32] = zero[grp];
            }
        }
#pragma unroll
        for (int w = 0; w < 2 * F::W; ++w) {  // sums of 16 bits, exact in fp32; those of positions not new are masked below
            const float *c = code + 4 * w;
            const uint32_t bytes = (uint32_t)fmaf(c[1], 256.0f, c[0]) | (uint32_t)fmaf(c[3], 256.0f, c[2]) << 16;
            if (half == 0)
                low[w] = bytes;
            else
                *reinterpret_cast<uint32_t *>(mine + m * PITCH + 32 * (w >> 1) + 8 * g + 4 * (w & 1)) = low[w] | bytes << 4;
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    // V words: 8 positions of one channel
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = p0 + 4 * g + (j & 3) + 16 * (j >> 2) - u.first;
        if (i >= 0 && i < u.n) mask |= 0xFu << (4 * nibble_of(j));
    }
    if (mask == 0) return;
#pragma unroll
    for (int hs = 0; hs < 2 * F::S; ++hs) {
        char *at = u.rec + F::VC + ((hs * 64 + lane) * F::WV) * 4;
        uint32_t word[F::WV];
        if (mask != 0xFFFFFFFFu) load_words<F::WV>(at, word);
#pragma unroll
        for (int w = 0; w < F::WV; ++w) {
            // byte j: position 4 g + j below, 16 more above; the places of codes j and j + 4
            const uint8_t *b = mine + 4 * g * PITCH + 16 * (hs * F::WV + w) + m;
            const uint32_t even = b[0] | ((uint32_t)b[PITCH] << 16), odd = b[2 * PITCH] | ((uint32_t)b[3 * PITCH] << 16);
            const uint32_t x = (even & 0x000F000Fu) | (even & 0x00F000F0u) << 4 | (odd & 0x000F000Fu) << 4 |
                               (odd & 0x00F000F0u) << 8;
            word[w] = mask == 0xFFFFFFFFu ? x : (word[w] & ~mask) | (x & mask);
        }
        store_words<F::WV>(at, word);
    }
}

// A few new tokens: a wave takes their positions in its record one by one, with
// all lanes on one position, E channels each, as a step of decoding has a
// token or so for each sequence and latency is what counts.  32 sequences of 8
// heads: 3.6 us for one token each, 6.6 for 4 and 8.6 for 6, where the kernel
// above takes 7.1, 7.2 and 7.4; so it is used up to kFewTokens.
template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kMoveWaves) append_few_kernel(const MoveArgs a) {
    using F = Format<D, GROUP>;
    constexpr int E = D <= 128 ? 2 : 4;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    Unit u;
    if (!unit_of(a, blockIdx.x * kMoveWaves + wave, u) || !u.rec) return;
    const int ch = E * lane;
    if (ch >= D) return;
    const int p0 = u.tile * kTile;
    const int from = u.first > p0 ? u.first : p0;
    const int to = u.first + u.n < p0 + kTile ? u.first + u.n : p0 + kTile;
    const int grp = ch / GROUP;
    // this lane's part of a K word, whose first lane stores it
    const int i = ch / 32, kg = ch % 32 / 8, j = ch % 8;
    for (int pos = from; pos < to; ++pos) {
        const int t = pos & (kTile - 1), half = t >> 4, m = t & 15;
        const int64_t row = u.start + (pos - u.first);
        const int64_t ka = row * a.k.token_stride + u.head * a.k.head_stride + ch;
        const int64_t va = row * a.v.token_stride + u.head * a.v.head_stride + ch;
        float x[2][E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[0][e] = limited(elem_to_float(((const uint16_t *)a.k.data)[ka + e], a.k.type));
            x[1][e] = limited(elem_to_float(((const uint16_t *)a.v.data)[va + e], a.v.type));
        }
        // a V code is half a byte of its word; the other half may be another position's
        const int nibble = nibble_of((t & 3) + 4 * half);
        uint8_t *byte[E], old[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int chunk = (ch + e) / 16;
            byte[e] = (uint8_t *)u.rec + F::VC + nibble / 2 +
                      (((chunk / F::WV) * 64 + 16 * (m >> 2) + (ch + e) % 16) * F::WV + chunk % F::WV) * 4;
            old[e] = *byte[e];
        }
        float lo[2], hi[2];
        _Float16 scale[2], zero[2];
        float code[2][E];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            lo[s] = hi[s] = x[s][0];
#pragma unroll
            for (int e = 1; e < E; ++e) lo[s] = fminf(lo[s], x[s][e]), hi[s] = fmaxf(hi[s], x[s][e]);
        }
#pragma unroll
        for (int mask = 1; mask < GROUP / E; mask <<= 1)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                lo[s] = fminf(lo[s], __shfl_xor(lo[s], mask));
                hi[s] = fmaxf(hi[s], __shfl_xor(hi[s], mask));
            }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            scale_of(lo[s], hi[s], scale[s], zero[s]);
            codes_of<E>(x[s], (float)zero[s], (float)scale[s], code[s]);
        }
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) word |= (uint32_t)code[0][e] << (4 * nibble_of(j + e));
#pragma unroll
        for (int mask = 1; mask < 8 / E; mask <<= 1) word |= __shfl_xor(word, mask);
        if (j == 0)
            *reinterpret_cast<uint32_t *>(u.rec + (((half * F::S + i / F::WV) * 64 + 16 * kg + m) * F::WV + i % F::WV) * 4) = word;
        const int shift = 4 * (nibble & 1);
#pragma unroll
        for (int e = 0; e < E; ++e) *byte[e] = (uint8_t)((old[e] & (0xF0 >> shift)) | ((uint32_t)code[1][e] << shift));
        if (ch % GROUP == 0) {
            *reinterpret_cast<h2 *>(u.rec + F::KP + (grp * kTile + t) * 4) = (h2){scale[0], zero[0]};
            _Float16 *v = reinterpret_cast<_Float16 *>(u.rec + F::VP) + grp * 64 + 8 * (m >> 2) + 4 * half + (m & 3);
            v[0] = scale[1], v[32] = zero[1];
        }
    }
}

// Positions out of the cache, keys and values by a wave each: V codes go through
// LDS as above; then a lane takes 8
// channels of a position, neighbouring lanes the next 8, so that a position's
// row is written in one run.
template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kMoveWaves) read_kernel(const MoveArgs a) {
    using F = Format<D, GROUP>;
    constexpr int PITCH = D + 8;
    constexpr int LANES = D / 8, AT_ONCE = 64 / LANES;  // of a position, and positions
    __shared__ __attribute__((aligned(8))) uint8_t codes[kMoveWaves / 2][kTile * PITCH];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const bool values = wave & 1;
    Unit u;
    if (!unit_of(a, blockIdx.x * (kMoveWaves / 2) + (wave >> 1), u)) return;
    uint8_t *mine = codes[wave >> 1];  // of the wave with the values alone
    const int p0 = u.tile * kTile;
    const int which = lane / LANES, ch = 8 * (lane % LANES), grp = ch / GROUP, i = ch / 32, kg = ch % 32 / 8;
    // all that is read first: no step waits for another's
    constexpr int STEPS = (kTile + AT_ONCE - 1) / AT_ONCE;
    uint32_t word[STEPS];
    h2 pair[STEPS];
    if (u.rec && values) {
        uint32_t own[2 * F::W];
#pragma unroll
        for (int hs = 0; hs < 2 * F::S; ++hs)
            load_words<F::WV>(u.rec + F::VC + ((hs * 64 + lane) * F::WV) * 4, own + hs * F::WV);
#pragma unroll
        for (int step = 0; step < STEPS; ++step) {
            const int t = (step * AT_ONCE + which) & (kTile - 1), half = t >> 4, mt = t & 15;
            const _Float16 *v = reinterpret_cast<const _Float16 *>(u.rec + F::VP) + grp * 64 + 8 * (mt >> 2) + 4 * half;
            pair[step] = (h2){v[mt & 3], v[32 + (mt & 3)]};
        }
#pragma unroll
        for (int w = 0; w < 2 * F::W; ++w)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                mine[(4 * g + (j & 3) + 16 * (j >> 2)) * PITCH + 16 * w + m] =
                    (uint8_t)((own[w] >> (4 * nibble_of(j))) & 15);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    } else if (u.rec) {
#pragma unroll
        for (int step = 0; step < STEPS; ++step) {
            const int t = (step * AT_ONCE + which) & (kTile - 1), half = t >> 4, mt = t & 15;
            word[step] = *reinterpret_cast<const uint32_t *>(
                u.rec + (((half * F::S + i / F::WV) * 64 + 16 * kg + mt) * F::WV + i % F::WV) * 4);
            pair[step] = *reinterpret_cast<const h2 *>(u.rec + F::KP + (grp * kTile + t) * 4);
        }
    }
    if (which >= AT_ONCE) return;
    const Tokens &to = values ? a.v : a.k;
#pragma unroll
    for (int step = 0; step < STEPS; ++step) {
        const int t = step * AT_ONCE + which, n = p0 + t - u.first;
        if (t >= kTile || n < 0 || n >= u.n) continue;
        float x[8];
        if (u.rec) {
            const float scale = (float)pair[step][0], zero = (float)pair[step][1];
            if (values) {
                const uint2 c = *reinterpret_cast<const uint2 *>(mine + t * PITCH + ch);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = fmaf(scale, (float)(((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 255), zero);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = fmaf(scale, (float)((word[step] >> (4 * nibble_of(j))) & 15), zero);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
        }
        store8(to, (u.start + n) * to.token_stride + u.head * to.head_stride + ch, x);
    }
}

template <int D, int GROUP>
static int launch_move(const MoveArgs &a, bool append, void *stream) {
    const int64_t units = (int64_t)a.b.n_seq * a.tiles * a.c.heads;
    const dim3 grid((uint32_t)((units + kMoveWaves - 1) / kMoveWaves)), block(64 * kMoveWaves);
    const dim3 two_waves((uint32_t)((units * 2 + kMoveWaves - 1) / kMoveWaves));  // for a record
    if (append && a.b.max_new <= kFewTokens)
        append_few_kernel<D, GROUP><<<grid, block, 0, (hipStream_t)stream>>>(a);
    else if (append)
        append_kernel<D, GROUP><<<two_waves, block, 0, (hipStream_t)stream>>>(a);
    else
        read_kernel<D, GROUP><<<two_waves, block, 0, (hipStream_t)stream>>>(a);
    return (int)hipGetLastError();
}

static int move(const MoveArgs &a, bool append, void *stream) {
    switch (a.c.dim * 1000 + a.c.group) {
        case 64032: return launch_move<64, 32>(a, append, stream);
        case 64064: return launch_move<64, 64>(a, append, stream);
        case 96032: return launch_move<96, 32>(a, append, stream);
        case 128032: return launch_move<128, 32>(a, append, stream);
        case 128064: return launch_move<128, 64>(a, append, stream);
        case 128128: return launch_move<128, 128>(a, append, stream);
        case 256032: return launch_move<256, 32>(a, append, stream);
        case 256064: return launch_move<256, 64>(a, append, stream);
        case 256128: return launch_move<256, 128>(a, append, stream);
    }
    return (int)hipErrorInvalidValue;
}

int launch_append(const MoveArgs &a, void *stream) { return move(a, true, stream); }
int launch_read(const MoveArgs &a, void *stream) { return move(a, false, stream); }

}  // namespace tkv
