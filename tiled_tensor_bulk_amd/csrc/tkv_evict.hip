// tkv_evict.hip -- keep a sequence's last positions and those of the largest
// scores, and move them to other pages.
//
// Choosing.  One workgroup takes one (sequence, head).  A score becomes a
// 32-bit key that orders like it (NaN lowest, -0 equal to +0); the key of the
// last one kept is found digit by digit from the top, 11 + 11 + 10 bits, each
// with a histogram in LDS.  A last pass writes the kept positions in order:
// each wave owns a run of positions, counts its keys above and equal to that
// key, and takes its places from the other waves' counts; of the equal keys
// the lowest positions stay.
//
// Moving.  One wave takes one record of the destination.  K words and pairs
// move as they are, 16 bytes a lane; a V word is put together from 8 nibbles
// of 8 source words.
#include "tkv_format.h"

namespace tkv {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / 64;
constexpr int kBins = 2048;
constexpr int kEvictWaves = 4;

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

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictArgs a) {
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
    if (head == 0 && tid == 0) a.lens_out[seq] = n;
    for (int i = n + tid; i < a.budget; i += kSelectThreads) kept[i] = -1, scores_out[i] = 0.0f;
    if (len <= a.budget) {
        for (int i = tid; i < n; i += kSelectThreads) kept[i] = i, scores_out[i] = scores[i];
        return;
    }
    const int recent = a.recent < a.budget ? a.recent : a.budget;
    const int old = len - recent;               // candidates
    uint32_t want = (uint32_t)(a.budget - recent);  // of which so many stay; want < old
    uint32_t prefix = 0, prefix_mask = 0;
    if (want > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
            for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
            __syncthreads();
            for (int i = tid; i < old; i += kSelectThreads) {
                const uint32_t key = key_of(scores[i]);
                if ((key & prefix_mask) == prefix) atomicAdd(&bins[(key >> shift) & digit_mask], 1u);
            }
            __syncthreads();
            if (wave == 0) {
                // lane i owns bins 32 i .. 32 i + 31; from the top
                uint32_t mine = 0;
                for (int j = 0; j < kBins / 64; ++j) mine += bins[lane * (kBins / 64) + ((j + lane) & 31)];
                uint32_t above = mine;  // inclusive sum from this lane up
                for (int d = 1; d < 64; d <<= 1) {
                    const uint32_t y = __shfl_down(above, d);
                    if (lane + d < 64) above += y;
                }
                above -= mine;
                if (above < want && above + mine >= want) {
                    uint32_t left = want - above;
                    int j = kBins / 64 - 1;
                    while (j > 0 && bins[lane * (kBins / 64) + j] < left) left -= bins[lane * (kBins / 64) + j], --j;
                    found[0] = lane * (kBins / 64) + j;
                    found[1] = left;
                }
            }
            __syncthreads();
            prefix |= found[0] << shift;
            prefix_mask |= digit_mask << shift;
            want = found[1];
        }
    }
    // keys above `prefix` stay, and the first `want` of those equal to it
    const bool any = a.budget > recent;
    const int run = ((old + kSelectWaves - 1) / kSelectWaves + 63) & ~63;
    const int from = wave * run, to = from + run < old ? from + run : old;
    int above = 0, equal = 0;
    if (any)
        for (int i = from; i < to; i += 64) {
            const uint32_t key = i + lane < to ? key_of(scores[i + lane]) : 0;
            above += __popcll(__ballot(i + lane < to && key > prefix));
            equal += __popcll(__ballot(i + lane < to && key == prefix));
        }
    if (lane == 0) count_above[wave] = above, count_equal[wave] = equal;
    __syncthreads();
    int out = 0, equal_before = 0;
    for (int w = 0; w < wave; ++w) {
        const int left = (int)want - equal_before;
        out += count_above[w] + (count_equal[w] < left ? count_equal[w] : left > 0 ? left : 0);
        equal_before += count_equal[w];
    }
    if (any)
        for (int i = from; i < to; i += 64) {
            const bool in = i + lane < to;
            const float s = in ? scores[i + lane] : 0.0f;
            const uint32_t key = key_of(s);
            const uint64_t same = __ballot(in && key == prefix);
            const bool stay = in && (key > prefix || (key == prefix && equal_before + below(same) < (int)want));
            const uint64_t all = __ballot(stay);
            if (stay) {
                const int at = out + below(all);
                kept[at] = i + lane;
                scores_out[at] = s;
            }
            out += __popcll(all);
            equal_before += __popcll(same);
        }
    for (int i = tid; i < recent; i += kSelectThreads) {
        kept[a.budget - recent + i] = old + i;
        scores_out[a.budget - recent + i] = scores[old + i];
    }
}

template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kEvictWaves) move_kernel(const EvictArgs a, const int tiles) {
    using F = Format<D, GROUP>;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int64_t unit = (int64_t)blockIdx.x * kEvictWaves + wave;
    const int tile = (int)(unit % tiles);
    const int64_t row = unit / tiles;
    const int head = (int)(row % a.c.heads);
    if (row / a.c.heads >= a.b.n_seq) return;
    const int seq = (int)(row / a.c.heads);
    const int len = evict_len(a, seq), n = len < a.budget ? len : a.budget;
    if (tile * kTile >= n) return;
    const int dst_page = page_at(a.dst_table + seq * a.dst_stride, a.dst_width, a.c.n_pages, tile >> (a.c.page_shift - 5));
    if (dst_page < 0) return;
    char *dst = record_at(a.c, dst_page, head, tile);
    const int32_t *table = a.b.table + seq * a.b.table_stride;
    // lane i < 32: where the record of the i-th kept position is, and its place there
    int pos = -1;
    if (lane < kTile && tile * kTile + lane < n) pos = a.kept[row * a.budget + tile * kTile + lane];
    const int page = pos < 0 ? -1 : page_at(table, a.b.table_width, a.c.n_pages, pos >> a.c.page_shift);
    const char *src = page < 0 ? nullptr : record_at(a.c, page, head, pos / kTile);
    const uint32_t src_lo = (uint32_t)(uint64_t)src, src_hi = (uint32_t)((uint64_t)src >> 32);
    const auto record_of = [&](int i) {
        return (const char *)(((uint64_t)(uint32_t)__shfl((int)src_hi, i) << 32) | (uint32_t)__shfl((int)src_lo, i));
    };
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const char *rec = record_of(16 * half + m);
        const int place = __shfl(pos, 16 * half + m) & 31;
        const int from_half = place >> 4, from_lane = 16 * g + (place & 15);
#pragma unroll
        for (int s = 0; s < F::S; ++s) {
            uint32_t word[F::WV];
#pragma unroll
            for (int w = 0; w < F::WV; ++w) word[w] = 0;
            if (rec) load_words<F::WV>(rec + (((from_half * F::S + s) * 64 + from_lane) * F::WV) * 4, word);
            store_words<F::WV>(dst + (((half * F::S + s) * 64 + lane) * F::WV) * 4, word);
        }
        // lane g takes every fourth group's pairs of position m
        const int from_slot = 8 * ((place & 15) >> 2) + 4 * from_half + (place & 3);
        const int to_slot = 8 * (m >> 2) + 4 * half + (m & 3);
#pragma unroll
        for (int base = 0; base < F::NG; base += 4) {
            const int grp = base + g;
            if (grp < F::NG) {
                uint32_t kp = 0;
                uint16_t vs = 0, vz = 0;
                if (rec) {
                    kp = *reinterpret_cast<const uint32_t *>(rec + F::KP + (grp * kTile + place) * 4);
                    const uint16_t *vp = reinterpret_cast<const uint16_t *>(rec + F::VP) + grp * 64 + from_slot;
                    vs = vp[0], vz = vp[32];
                }
                *reinterpret_cast<uint32_t *>(dst + F::KP + (grp * kTile + 16 * half + m) * 4) = kp;
                uint16_t *vp = reinterpret_cast<uint16_t *>(dst + F::VP) + grp * 64 + to_slot;
                vp[0] = vs, vp[32] = vz;
            }
        }
    }
    uint32_t word[2 * F::W];
#pragma unroll
    for (int w = 0; w < 2 * F::W; ++w) word[w] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = 4 * g + (j & 3) + 16 * (j >> 2);
        const char *rec = record_of(i);
        const int place = __shfl(pos, i) & 31;
        const int from_lane = 16 * ((place & 15) >> 2) + m, from_j = (place & 3) + 4 * (place >> 4);
        const int from_shift = 4 * nibble_of(from_j);
        if (rec) {
#pragma unroll
            for (int hs = 0; hs < 2 * F::S; ++hs) {
                uint32_t x[F::WV];
                load_words<F::WV>(rec + F::VC + ((hs * 64 + from_lane) * F::WV) * 4, x);
#pragma unroll
                for (int w = 0; w < F::WV; ++w)
                    word[hs * F::WV + w] |= ((x[w] >> from_shift) & 15u) << (4 * nibble_of(j));
            }
        }
    }
#pragma unroll
    for (int hs = 0; hs < 2 * F::S; ++hs)
        store_words<F::WV>(dst + F::VC + ((hs * 64 + lane) * F::WV) * 4, word + hs * F::WV);
}

template <int D, int GROUP>
static int launch_moves(const EvictArgs &a, void *stream) {
    const int most = a.budget < a.max_len ? a.budget : a.max_len;
    const int tiles = (most + kTile - 1) / kTile;
    if (tiles == 0) return 0;
    const int64_t units = (int64_t)a.b.n_seq * a.c.heads * tiles;
    move_kernel<D, GROUP><<<dim3((uint32_t)((units + kEvictWaves - 1) / kEvictWaves)), dim3(64 * kEvictWaves), 0,
                            (hipStream_t)stream>>>(a, tiles);
    return (int)hipGetLastError();
}

int launch_evict(const EvictArgs &a, void *stream) {
    select_kernel<<<dim3((uint32_t)(a.b.n_seq * (int64_t)a.c.heads)), dim3(kSelectThreads), 0, (hipStream_t)stream>>>(a);
    const int rc = (int)hipGetLastError();
    if (rc) return rc;
    switch (a.c.dim * 1000 + a.c.group) {
        case 64032: return launch_moves<64, 32>(a, stream);
        case 64064: return launch_moves<64, 64>(a, stream);
        case 96032: return launch_moves<96, 32>(a, stream);
        case 128032: return launch_moves<128, 32>(a, stream);
        case 128064: return launch_moves<128, 64>(a, stream);
        case 128128: return launch_moves<128, 128>(a, stream);
        case 256032: return launch_moves<256, 32>(a, stream);
        case 256064: return launch_moves<256, 64>(a, stream);
        case 256128: return launch_moves<256, 128>(a, stream);
    }
    return (int)hipErrorInvalidValue;
}

}  // namespace tkv
