// tkv_evict.hip -- keep a sequence's last positions and those of the largest
// scores, and move them to other pages.
//
// Choosing.  One workgroup takes one (sequence, head).  A score becomes a
// 32-bit key that orders like it (NaN lowest, -0 equal to +0); the key of the
// last one kept is found digit by digit from the top, 11 + 11 + 10 bits, each
// with a histogram in LDS.  A last pass writes the kept positions in order:
// each wave owns a run of positions, counts its keys above and equal to that
// key, and takes its places from the other waves' counts; of the equal keys
// the lowest positions stay.  The scores are read once, 16 bytes a lane, and
// stay in registers as far as kHeld for a lane go (32768 positions); only a
// longer row is read anew in each pass.
//
// Moving.  One wave takes one record of the destination.  K words and pairs
// move as they are, 16 bytes a lane; a V word is put together from 8 nibbles
// of 8 source words.  What stays is known from `kept`, and a sequence's new
// length is written here, by the only wave that still reads the old one: lens
// may be shrunk in place.
//
// 8 sequences of up to 32768 positions to 8192, 8 heads of 128 channels:
// choosing 25 us, a pass over LDS for each of three digits by the one workgroup
// that a row has; moving 70 us for 74 MB written and, as kept positions share
// 128-byte lines of source words with others, the source read nearly whole (77
// with each load under its own test of the page, and so a wait for each).
#include "tkv_format.h"

namespace tkv {

constexpr int kSelectWaves = kSelectThreads / 64;
constexpr int kBins = 2048;
constexpr int kHeld = 8;  // rows of 4 scores that a lane holds
constexpr int kEvictWaves = kBlockThreads / 64;

__device__ __forceinline__ uint32_t key_of(float f) {
    uint32_t u = __builtin_bit_cast(uint32_t, f);
    if (f != f) return 0;
    if (u == 0x80000000u) u = 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive count of set lanes below this one.
__device__ __forceinline__ int below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

__device__ __forceinline__ int evict_len(const EvictArgs &a, int seq) {
    const int64_t width = (int64_t)a.b.table_width << a.c.page_shift;
    int l = a.b.lens[seq];
    l = l < 0 ? 0 : l < a.max_len ? l : a.max_len;
    return (int64_t)l < width ? l : (int)width;
}

// The candidates as the waves own them: wave w has positions w * run .., row r
// of its run is 256 of them, 4 in a lane.  HELD rows stay in registers; with
// HELD 0 every pass reads them.
template <int HELD>
struct Scores {
    const float *from;
    int run, count, base, lane;
    bool wide;
    float held[HELD ? HELD : 1][4];
    __device__ __forceinline__ Scores(const float *scores, int n, int wave, int lane_) {
        from = scores;
        count = n;
        lane = lane_;
        run = ((n + kSelectWaves - 1) / kSelectWaves + 255) & ~255;
        base = wave * run;
        wide = ((uintptr_t)scores & 15) == 0;
#pragma unroll
        for (int r = 0; r < HELD; ++r)
            if (r * 256 < run) read(r, held[r]);
    }
    __device__ __forceinline__ int at(int r) const { return base + 256 * r + 4 * lane; }
    __device__ __forceinline__ void read(int r, float (&x)[4]) const {
        const int i = at(r);
        if (wide && i + 4 <= count) {
            const float4 v = *reinterpret_cast<const float4 *>(from + i);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = i + e < count ? from[i + e] : 0.0f;
        }
    }
    // f(position of x[0], x, how many of the 4 are there), in order
    template <class Fn>
    __device__ __forceinline__ void each(Fn f) const {
        if constexpr (HELD > 0) {
#pragma unroll
            for (int r = 0; r < HELD; ++r)
                if (r * 256 < run) f(at(r), held[r], count - at(r));
        } else {
            for (int r = 0; r * 256 < run; ++r) {
                float x[4];
                read(r, x);
                f(at(r), x, count - at(r));
            }
        }
    }
};

// only: no moves follow, and then nothing that is left to do goes by the length.
template <int HELD>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictArgs a, const bool only) {
    __shared__ uint32_t bins[kBins];
    __shared__ uint32_t found[2];  // digit, and how many are still wanted below it
    __shared__ int count_above[kSelectWaves], count_equal[kSelectWaves];
    const int head = blockIdx.x % a.c.heads, seq = blockIdx.x / a.c.heads;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int len = evict_len(a, seq);
    const int n = len < a.budget ? len : a.budget;
    const int64_t unit = (int64_t)seq * a.c.heads + head;
    const float *scores = a.scores + unit * a.score_stride;
    float *scores_out = a.scores_out + unit * a.budget;
    int32_t *kept = a.kept + unit * a.budget;
    if (only && head == 0 && tid == 0) a.lens_out[seq] = n;
    for (int i = n + tid; i < a.budget; i += kSelectThreads) kept[i] = -1, scores_out[i] = 0.0f;
    if (len <= a.budget) {
        for (int i = tid; i < n; i += kSelectThreads) kept[i] = i, scores_out[i] = scores[i];
        return;
    }
    const int recent = a.recent < a.budget ? a.recent : a.budget;
    const int old = len - recent;                   // candidates
    uint32_t want = (uint32_t)(a.budget - recent);  // of which so many stay; want < old
    for (int i = tid; i < recent; i += kSelectThreads) {
        kept[a.budget - recent + i] = old + i;
        scores_out[a.budget - recent + i] = scores[old + i];
    }
    if (want == 0) return;
    const Scores<HELD> mine(scores, old, wave, lane);
    uint32_t prefix = 0, prefix_mask = 0;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
        __syncthreads();
        mine.each([&](int, const float (&x)[4], int there) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t key = key_of(x[e]);
                if (e < there && (key & prefix_mask) == prefix) atomicAdd(&bins[(key >> shift) & digit_mask], 1u);
            }
        });
        __syncthreads();
        if (wave == 0) {
            // lane i owns bins 32 i .. 32 i + 31; from the top
            uint32_t own = 0;
#pragma unroll
            for (int j = 0; j < kBins / 64; ++j) own += bins[lane * (kBins / 64) + ((j + lane) & 31)];
            uint32_t above = own;  // inclusive sum from this lane up
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t y = __shfl_down(above, d);
                if (lane + d < 64) above += y;
            }
            above -= own;
            // the lane whose bins hold the last one wanted, and then its bin, again by sums from the top
            const bool here = above < want && above + own >= want;
            const int who = __ffsll((long long)__ballot(here)) - 1;
            const uint32_t left = want - __shfl(above, who);
            const uint32_t bin = lane < 32 ? bins[who * 32 + lane] : 0;
            uint32_t sum = bin;
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_down(sum, d);
                if (lane + d < 32) sum += y;
            }
            if (lane < 32 && sum - bin < left && sum >= left) {
                found[0] = who * 32 + lane;
                found[1] = left - (sum - bin);
            }
        }
        __syncthreads();
        prefix |= found[0] << shift;
        prefix_mask |= digit_mask << shift;
        want = found[1];
    }
    // keys above `prefix` stay, and the first `want` of those equal to it
    int above = 0, equal = 0;
    mine.each([&](int, const float (&x)[4], int there) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t key = key_of(x[e]);
            above += __popcll(__ballot(e < there && key > prefix));
            equal += __popcll(__ballot(e < there && key == prefix));
        }
    });
    if (lane == 0) count_above[wave] = above, count_equal[wave] = equal;
    __syncthreads();
    int out = 0, equal_before = 0;
    for (int w = 0; w < wave; ++w) {
        const int left = (int)want - equal_before;
        out += count_above[w] + (count_equal[w] < left ? count_equal[w] : left > 0 ? left : 0);
        equal_before += count_equal[w];
    }
    mine.each([&](int i, const float (&x)[4], int there) {
        uint32_t key[4];
        int before = equal_before, all_equal = 0;
        uint64_t same[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            key[e] = key_of(x[e]);
            same[e] = __ballot(e < there && key[e] == prefix);
            before += below(same[e]);  // equal ones of lower lanes
            all_equal += __popcll(same[e]);
        }
        bool stay[4];
        int at = out;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool equal_here = e < there && key[e] == prefix;
            stay[e] = (e < there && key[e] > prefix) || (equal_here && before < (int)want);
            before += equal_here;
            const uint64_t staying = __ballot(stay[e]);
            at += below(staying);
            out += __popcll(staying);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (stay[e]) {
                kept[at] = i + e;
                scores_out[at] = x[e];
                ++at;
            }
        equal_before += all_equal;
    });
}

template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kEvictWaves) move_kernel(const EvictArgs a, const int tiles) {
    using F = Format<D, GROUP>;
    constexpr int PAIRS = (F::NG + 3) / 4, JS = F::W > 4 ? 4 : 8;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int64_t unit = (int64_t)blockIdx.x * kEvictWaves + wave;
    const int tile = (int)(unit % tiles);
    const int64_t row = unit / tiles;
    const int head = (int)(row % a.c.heads);
    if (row / a.c.heads >= a.b.n_seq) return;
    const int seq = (int)(row / a.c.heads);
    // lane i < 32: where the record of the i-th kept position is, and its place there
    int pos = -1;
    if (lane < kTile && tile * kTile + lane < a.budget) pos = a.kept[row * a.budget + tile * kTile + lane];
    if (tile == 0 && head == 0 && lane == 0) {
        const int len = evict_len(a, seq);
        a.lens_out[seq] = len < a.budget ? len : a.budget;
    }
    if (!__any(pos >= 0)) return;
    const int dst_page = page_at(a.dst_table + seq * a.dst_stride, a.dst_width, a.c.n_pages, tile >> (a.c.page_shift - 5));
    if (dst_page < 0) return;
    char *dst = record_at(a.c, dst_page, head, tile);
    const int32_t *table = a.b.table + seq * a.b.table_stride;
    const int page = pos < 0 ? -1 : page_at(table, a.b.table_width, a.c.n_pages, pos >> a.c.page_shift);
    if (page < 0) pos = -1;
    // what has no source reads the destination's record, and drops it
    const char *src = page < 0 ? dst : record_at(a.c, page, head, pos / kTile);
    const uint32_t src_lo = (uint32_t)(uint64_t)src, src_hi = (uint32_t)((uint64_t)src >> 32);
    const auto record_of = [&](int i) {
        return (const char *)(global_char *)(((uint64_t)(uint32_t)__shfl((int)src_hi, i) << 32) |
                                             (uint32_t)__shfl((int)src_lo, i));
    };
    // All loads of K and the pairs, then of V's words for JS codes at a time: no
    // load waits for another's.
    uint32_t key[2][F::W], kp[2][PAIRS];
    uint16_t vs[2][PAIRS], vz[2][PAIRS];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const char *rec = record_of(16 * half + m);
        const int place = __shfl(pos, 16 * half + m) & 31;
        const int from_half = place >> 4, from_lane = 16 * g + (place & 15);
#pragma unroll
        for (int s = 0; s < F::S; ++s)
            load_words<F::WV>(rec + (((from_half * F::S + s) * 64 + from_lane) * F::WV) * 4, key[half] + s * F::WV);
        // lane g takes every fourth group's pairs of position m
        const int from_slot = 8 * ((place & 15) >> 2) + 4 * from_half + (place & 3);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const int grp = 4 * i + g < F::NG ? 4 * i + g : 0;
            const uint16_t *vp = reinterpret_cast<const uint16_t *>(rec + F::VP) + grp * 64 + from_slot;
            kp[half][i] = *reinterpret_cast<const uint32_t *>(rec + F::KP + (grp * kTile + place) * 4);
            vs[half][i] = vp[0], vz[half][i] = vp[32];
        }
    }
    uint32_t word[2 * F::W];
#pragma unroll
    for (int w = 0; w < 2 * F::W; ++w) word[w] = 0;
#pragma unroll
    for (int js = 0; js < 8; js += JS) {
        uint32_t x[JS][2 * F::W];
        int at[JS];
#pragma unroll
        for (int j = 0; j < JS; ++j) {
            const int i = 4 * g + ((js + j) & 3) + 16 * ((js + j) >> 2);
            const char *rec = record_of(i);
            at[j] = __shfl(pos, i);
            const int from_lane = 16 * ((at[j] & 15) >> 2) + m;
#pragma unroll
            for (int hs = 0; hs < 2 * F::S; ++hs)
                load_words<F::WV>(rec + F::VC + ((hs * 64 + from_lane) * F::WV) * 4, x[j] + hs * F::WV);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < JS; ++j) {
            const int from_shift = 4 * nibble_of((at[j] & 3) + ((at[j] & 16) >> 2));
            const uint32_t mask = at[j] < 0 ? 0u : 15u;
#pragma unroll
            for (int w = 0; w < 2 * F::W; ++w) word[w] |= ((x[j][w] >> from_shift) & mask) << (4 * nibble_of(js + j));
        }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const bool there = __shfl(pos, 16 * half + m) >= 0;
#pragma unroll
        for (int w = 0; w < F::W; ++w) key[half][w] = there ? key[half][w] : 0;
#pragma unroll
        for (int s = 0; s < F::S; ++s)
            store_words<F::WV>(dst + (((half * F::S + s) * 64 + lane) * F::WV) * 4, key[half] + s * F::WV);
        const int to_slot = 8 * (m >> 2) + 4 * half + (m & 3);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const int grp = 4 * i + g;
            if (grp < F::NG) {
                uint16_t *vp = reinterpret_cast<uint16_t *>(dst + F::VP) + grp * 64 + to_slot;
                *reinterpret_cast<uint32_t *>(dst + F::KP + (grp * kTile + 16 * half + m) * 4) = there ? kp[half][i] : 0;
                vp[0] = there ? vs[half][i] : 0, vp[32] = there ? vz[half][i] : 0;
            }
        }
    }
#pragma unroll
    for (int hs = 0; hs < 2 * F::S; ++hs)
        store_words<F::WV>(dst + F::VC + ((hs * 64 + lane) * F::WV) * 4, word + hs * F::WV);
}

template <int D, int GROUP>
static int launch_moves(const EvictArgs &a, int tiles, void *stream) {
    const int64_t units = (int64_t)a.b.n_seq * a.c.heads * tiles;
    move_kernel<D, GROUP><<<dim3((uint32_t)((units + kEvictWaves - 1) / kEvictWaves)), dim3(64 * kEvictWaves), 0,
                            (hipStream_t)stream>>>(a, tiles);
    return (int)hipGetLastError();
}

int launch_evict(const EvictArgs &a, void *stream) {
    const dim3 grid((uint32_t)(a.b.n_seq * (int64_t)a.c.heads)), block(kSelectThreads);
    hipStream_t s = (hipStream_t)stream;
    constexpr int kRow = 256 * kSelectWaves;  // positions of a row of every wave
    const int most = a.budget < a.max_len ? a.budget : a.max_len;
    const int tiles = (most + kTile - 1) / kTile;
    if (a.max_len <= kRow)
        select_kernel<1><<<grid, block, 0, s>>>(a, tiles == 0);
    else if (a.max_len <= kHeld * kRow)
        select_kernel<kHeld><<<grid, block, 0, s>>>(a, tiles == 0);
    else
        select_kernel<0><<<grid, block, 0, s>>>(a, tiles == 0);
    const int rc = (int)hipGetLastError();
    if (rc || tiles == 0) return rc;
    switch (a.c.dim * 1000 + a.c.group) {
        case 64032: return launch_moves<64, 32>(a, tiles, stream);
        case 64064: return launch_moves<64, 64>(a, tiles, stream);
        case 96032: return launch_moves<96, 32>(a, tiles, stream);
        case 128032: return launch_moves<128, 32>(a, tiles, stream);
        case 128064: return launch_moves<128, 64>(a, tiles, stream);
        case 128128: return launch_moves<128, 128>(a, tiles, stream);
        case 256032: return launch_moves<256, 32>(a, tiles, stream);
        case 256064: return launch_moves<256, 64>(a, tiles, stream);
        case 256128: return launch_moves<256, 128>(a, tiles, stream);
    }
    return (int)hipErrorInvalidValue;
}

}  // namespace tkv
