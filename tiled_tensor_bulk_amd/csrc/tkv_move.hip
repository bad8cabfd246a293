// tkv_move.hip -- new tokens into the cache (append) and positions out of it
// (read).
//
// One wave takes one record: 32 positions of one head of one sequence.  A K
// word belongs to one position, but a V word holds 8 positions of a channel,
// so the wave that owns the record also owns its V words: where some of a
// word's positions are not new, it reads the word, replaces the new nibbles
// and writes it back, with no atomics.  Rows are read as the K operand lies
// (lane 16 g + m: position m, channels 32 i + 8 g ..); V codes change places
// through LDS, as bytes.
//
// What bounds both is memory: two bytes of input (or four of output) for each
// half byte of cache.
#include "tkv_format.h"

namespace tkv {

constexpr int kMoveWaves = 4;

// Nearest whole number to (x - z) / s, ties to even.  The quotient in fp32 is
// within 1e-5 of the true one, so only one that close to a border needs the
// exact comparison, in fp64, where products of an fp16 number and a small
// integer, and differences of fp16 and bf16 numbers, are exact.
__device__ __forceinline__ int code_of(float x, float z, float s, float inv) {
    const float t = (x - z) * inv;
    float c = rintf(t);
    const float low = floorf(t);
    if (fabsf(t - low - 0.5f) < 1e-4f && t > 0.0f && t < 15.0f) {
        const double twice = 2.0 * ((double)x - (double)z);
        const double border = (2.0 * (double)low + 1.0) * (double)s;
        const int k = (int)low;
        c = (float)(twice > border ? k + 1 : twice < border ? k : k + (k & 1));
    }
    return (int)fminf(fmaxf(c, 0.0f), 15.0f);
}

// Quantise one position's channels: lane group g holds channels 32 i + 8 g + j
// in x[8 i + j]; the four lanes of a position share its scales.
template <int D, int GROUP>
__device__ __forceinline__ void quantise(const float *x, _Float16 *scale, _Float16 *zero, uint8_t *code) {
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
        const _Float16 s16 = (_Float16)((hi - lo) / 15.0f), z16 = (_Float16)lo;
        const float s = (float)s16, z = (float)z16, inv = s > 0.0f ? 1.0f / s : 0.0f;
        scale[grp] = s16;
        zero[grp] = z16;
#pragma unroll
        for (int i = 0; i < F::KG * 8; ++i) code[grp * F::KG * 8 + i] = (uint8_t)code_of(y[i], z, s, inv);
    }
}

template <int D>
__device__ __forceinline__ void load_row(const Tokens &t, int64_t row, int head, int g, float *x) {
    const int64_t at = row * t.token_stride + head * t.head_stride + 8 * g;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        load8(t, at + 32 * i, x + 8 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = x[8 * i + j];
            x[8 * i + j] = y != y ? 0.0f : fminf(fmaxf(y, -kLimit), kLimit);
        }
    }
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

template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kMoveWaves) append_kernel(const MoveArgs a) {
    using F = Format<D, GROUP>;
    constexpr int PITCH = D + 4;  // bytes of a position's codes in LDS, off a multiple of the banks
    __shared__ uint8_t codes[kMoveWaves][kTile * PITCH];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    Unit u;
    if (!unit_of(a, blockIdx.x * kMoveWaves + wave, u) || !u.rec) return;  // waves share nothing
    uint8_t *mine = codes[wave];
    const int p0 = u.tile * kTile;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int pos = p0 + 16 * half + m, i = pos - u.first;
        const bool live = i >= 0 && i < u.n;
        float x[D / 4];
        _Float16 scale[F::NG], zero[F::NG];
        uint8_t code[D / 4];
        if (live) {
            load_row<D>(a.k, u.start + i, u.head, g, x);
            quantise<D, GROUP>(x, scale, zero, code);  // the four lanes of a position are live together
            uint32_t word[F::W];
#pragma unroll
            for (int w = 0; w < F::W; ++w) {
                word[w] = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) word[w] |= (uint32_t)code[8 * w + j] << (4 * nibble_of(j));
            }
#pragma unroll
            for (int s = 0; s < F::S; ++s)
                store_words<F::WV>(u.rec + (((half * F::S + s) * 64 + lane) * F::WV) * 4, word + s * F::WV);
            if (g == 0) {
#pragma unroll
                for (int grp = 0; grp < F::NG; ++grp)
                    *reinterpret_cast<h2 *>(u.rec + F::KP + (grp * kTile + 16 * half + m) * 4) =
                        (h2){scale[grp], zero[grp]};
            }
            load_row<D>(a.v, u.start + i, u.head, g, x);
            quantise<D, GROUP>(x, scale, zero, code);
#pragma unroll
            for (int w = 0; w < F::W; ++w) {
                uint32_t c[2] = {0, 0};
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j >> 2] |= (uint32_t)code[8 * w + j] << (8 * (j & 3));
                uint32_t *to = reinterpret_cast<uint32_t *>(mine + (16 * half + m) * PITCH + 32 * w + 8 * g);
                to[0] = c[0], to[1] = c[1];
            }
            if (g == 0) {
                const int slot = 8 * (m >> 2) + 4 * half + (m & 3);
#pragma unroll
                for (int grp = 0; grp < F::NG; ++grp) {
                    _Float16 *to = reinterpret_cast<_Float16 *>(u.rec + F::VP) + grp * 64 + slot;
                    to[0] = scale[grp], to[32] = zero[grp];
                }
            }
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
            const int channel = 16 * (hs * F::WV + w) + m;
            uint32_t x = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x |= (uint32_t)(mine[(4 * g + (j & 3) + 16 * (j >> 2)) * PITCH + channel] & 15) << (4 * nibble_of(j));
            word[w] = mask == 0xFFFFFFFFu ? x : (word[w] & ~mask) | (x & mask);
        }
        store_words<F::WV>(at, word);
    }
}

template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kMoveWaves) read_kernel(const MoveArgs a) {
    using F = Format<D, GROUP>;
    constexpr int PITCH = D + 4;
    __shared__ uint8_t codes[kMoveWaves][kTile * PITCH];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    Unit u;
    if (!unit_of(a, blockIdx.x * kMoveWaves + wave, u)) return;
    uint8_t *mine = codes[wave];
    const int p0 = u.tile * kTile;
    if (u.rec) {
#pragma unroll
        for (int hs = 0; hs < 2 * F::S; ++hs) {
            uint32_t word[F::WV];
            load_words<F::WV>(u.rec + F::VC + ((hs * 64 + lane) * F::WV) * 4, word);
#pragma unroll
            for (int w = 0; w < F::WV; ++w)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mine[(4 * g + (j & 3) + 16 * (j >> 2)) * PITCH + 16 * (hs * F::WV + w) + m] =
                        (uint8_t)((word[w] >> (4 * nibble_of(j))) & 15);
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = p0 + 16 * half + m - u.first;
        if (i < 0 || i >= u.n) continue;
        uint32_t word[F::W];
        if (u.rec) {
#pragma unroll
            for (int s = 0; s < F::S; ++s)
                load_words<F::WV>(u.rec + (((half * F::S + s) * 64 + lane) * F::WV) * 4, word + s * F::WV);
        }
        const int slot = 8 * (m >> 2) + 4 * half + (m & 3);
#pragma unroll
        for (int w = 0; w < F::W; ++w) {
            const int grp = w / F::KG;
            float x[8], y[8];
            if (u.rec) {
                const h2 kp = *reinterpret_cast<const h2 *>(u.rec + F::KP + (grp * kTile + 16 * half + m) * 4);
                const _Float16 *vp = reinterpret_cast<const _Float16 *>(u.rec + F::VP) + grp * 64 + slot;
                const float ks = (float)kp[0], kz = (float)kp[1], vs = (float)vp[0], vz = (float)vp[32];
                const uint32_t *from =
                    reinterpret_cast<const uint32_t *>(mine + (16 * half + m) * PITCH + 32 * w + 8 * g);
                const uint32_t c[2] = {from[0], from[1]};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = ks * (float)((word[w] >> (4 * nibble_of(j))) & 15) + kz;
                    y[j] = vs * (float)((c[j >> 2] >> (8 * (j & 3))) & 255) + vz;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.0f;
            }
            const int64_t row = u.start + i;
            store8(a.k, row * a.k.token_stride + u.head * a.k.head_stride + 32 * w + 8 * g, x);
            store8(a.v, row * a.v.token_stride + u.head * a.v.head_stride + 32 * w + 8 * g, y);
        }
    }
}

template <int D, int GROUP>
static int launch_move(const MoveArgs &a, bool append, void *stream) {
    const int64_t units = (int64_t)a.b.n_seq * a.tiles * a.c.heads;
    const dim3 grid((uint32_t)((units + kMoveWaves - 1) / kMoveWaves)), block(64 * kMoveWaves);
    if (append)
        append_kernel<D, GROUP><<<grid, block, 0, (hipStream_t)stream>>>(a);
    else
        read_kernel<D, GROUP><<<grid, block, 0, (hipStream_t)stream>>>(a);
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
