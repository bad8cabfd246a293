// tkv_combine.hip -- join the partial sums of attention's chunks.
//
// A row's chunks each bring a reference m, a sum l and a vector o, all scaled
// by exp2(-m): with M the largest m, l = sum l_i exp2(m_i - M), and the same
// for o.  A lane holds 4 channels of a row.  Where a row has many chunks, as a
// few rows of a long context have, a workgroup takes 32 channels of one row and
// reads 32 chunks at a time; else a row's lanes go over its chunks alone, up to
// 16 of them on their way at once.
//
// What bounds it is the way there and back, as the partial sums are few: 512
// rows of 5 to 9 chunks 4.1 us, 32 rows of 256 chunks 5.2; 16384 rows of 4
// chunks of 128 channels, 34 MB, 10.5 us.
#include "tkv_attend.h"

namespace tkv {

constexpr int kCombineThreads = kBlockThreads;

// Where a row's partial sums are: part s at first + s * stride.
struct Parts {
    int n, stride;  // n 0: the row has been written where it was computed
    int64_t first;
    __device__ __forceinline__ Parts(const AttendArgs &a, const Extent &e, int unit, int seq, int head, int row) {
        if (a.even) {
            const int rows = 1 << a.row_shift, steps = Even::steps(e), block = row >> a.row_shift;
            const uint32_t share = (uint32_t)a.dealt[kEvenSeqs];
            const uint32_t from = (uint32_t)(a.dealt[seq] + Even::kLead +
                                             (head * Even::blocks(a, e) + block) * (steps + Even::kLead));
            const uint32_t part = from / share;
            n = (int)((from + steps - 1) / share - part) + 1;
            n = n == 1 ? 0 : n;
            stride = a.rows < rows ? a.rows : rows;
            first = ((int64_t)unit * a.row_blocks + block + part) * stride + (row & (rows - 1));
        } else {
            n = Chunks(a, e.len).n;
            stride = a.rows;
            first = (int64_t)unit * a.n_split * a.rows + row;
        }
    }
};

template <int D, int PARTS>
__device__ __forceinline__ void combine_few(const AttendArgs &a, int workgroup) {
    constexpr int LANES = D / 4, AT_ONCE = kCombineThreads / LANES;
    const int which = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    int row = workgroup * AT_ONCE + which;
    const int unit = divide(row, a.rows, a.by_rows);
    int head = unit;
    const int seq = divide(head, (int)a.c.heads, a.by_heads);
    if (which >= AT_ONCE || seq >= a.b.n_seq) return;
    const Extent e(a, seq);
    if (row >= e.rows) return;
    const Parts parts(a, e, unit, seq, head, row);
    if (parts.n == 0) return;
    float best = kFar, sum = 0.0f;
    f4 y = (f4){0, 0, 0, 0};
    for (int base = 0; base < parts.n; base += PARTS) {
        float2 ml[PARTS];
        f4 o[PARTS];
#pragma unroll
        for (int s = 0; s < PARTS; ++s) {  // past the last one: it again, without weight
            const int64_t from = parts.first + (int64_t)(base + s < parts.n ? base + s : parts.n - 1) * parts.stride;
            ml[s] = *reinterpret_cast<const float2 *>(a.part_ml + 2 * from);
            o[s] = *reinterpret_cast<const f4 *>(a.part_o + from * D + 4 * lane);
        }
        float m = best;
#pragma unroll
        for (int s = 0; s < PARTS; ++s) m = fmaxf(m, ml[s].x);
        const float f = exp2f(best - m);
        best = m, sum *= f, y *= f;
#pragma unroll
        for (int s = 0; s < PARTS; ++s)
            if (base + s < parts.n) {
                const float f = exp2f(ml[s].x - best);
                sum += f * ml[s].y;
                y += f * o[s];
            }
    }
    write_row(a, e, seq, head, row, 4 * lane, y, best, sum);
}

template <int D, int PARTS>
__global__ void __launch_bounds__(kCombineThreads) combine_few_kernel(const AttendArgs a) {
    combine_few<D, PARTS>(a, blockIdx.x);
}

template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const AttendArgs a) {
    constexpr int LANES = 8, AT_ONCE = kCombineThreads / LANES, PIECES = D / 32;
    __shared__ float4 join[AT_ONCE][LANES];
    __shared__ float join_m[kCombineThreads / 64], join_l[AT_ONCE];
    const int tid = threadIdx.x, which = tid / LANES, lane = tid % LANES;
    int row = blockIdx.x / PIECES;
    const int channel = blockIdx.x % PIECES * 32 + 4 * lane;
    const int unit = divide(row, a.rows, a.by_rows);
    int head = unit;
    const int seq = divide(head, (int)a.c.heads, a.by_heads);
    const Extent e(a, seq);
    if (row >= e.rows) return;
    const int parts = Chunks(a, e.len).n;
    const int64_t first = ((int64_t)unit * a.n_split) * a.rows + row;
    float best = kFar, sum = 0.0f;
    f4 y = (f4){0, 0, 0, 0};
    for (int s = tid; s < parts; s += kCombineThreads) best = fmaxf(best, a.part_ml[2 * (first + (int64_t)s * a.rows)]);
#pragma unroll
    for (int mask = 32; mask; mask >>= 1) best = fmaxf(best, __shfl_xor(best, mask));
    if ((tid & 63) == 0) join_m[tid >> 6] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kCombineThreads / 64; ++w) best = fmaxf(best, join_m[w]);
#pragma unroll 4
    for (int s = which; s < parts; s += AT_ONCE) {
        const int64_t from = first + (int64_t)s * a.rows;
        const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + 2 * from);
        const float f = exp2f(ml.x - best);
        sum += f * ml.y;
        y += f * *reinterpret_cast<const f4 *>(a.part_o + from * D + channel);
    }
    *reinterpret_cast<f4 *>(&join[which][lane]) = y;
    if (lane == 0) join_l[which] = sum;
    __syncthreads();
    if (which) return;
#pragma unroll
    for (int w = 1; w < AT_ONCE; ++w) {
        sum += join_l[w];
        y += *reinterpret_cast<const f4 *>(&join[w][lane]);
    }
    write_row(a, e, seq, head, row, channel, y, best, sum);
}

// scores_out = scores_in + the weights of a few rows, exp2(y - lse2), summed,
// from the logarithms that the first kernel has kept: masked ones are -inf.
// A lane takes 4 positions.  JOIN: lse2 comes of the partial sums, so that this
// need not wait for them to be joined.
template <bool JOIN>
__device__ __forceinline__ void weigh(const AttendArgs &a, int workgroup, int blocks) {
    __shared__ float joined[kLogitRows];
    const int unit = workgroup / blocks, block = workgroup % blocks;
    int head = unit;
    const int seq = divide(head, (int)a.c.heads, a.by_heads);
    const Extent e(a, seq);
    if (block * kWeighPositions >= e.len) return;
    const int pos = block * kWeighPositions + (int)threadIdx.x * 4;
    const int64_t records = (a.max_len + kTile - 1) / kTile;
    const float *y = a.logits + (unit * records + pos / kTile) * a.rows * kTile + (pos & (kTile - 1));
    const float *info = a.row_info + (int64_t)unit * 16 * 2;
    f4 x[kLogitRows];
#pragma unroll
    for (int r = 0; r < kLogitRows; ++r)
        if (r < e.rows && pos < e.len) x[r] = *reinterpret_cast<const f4 *>(y + r * kTile);
    if (JOIN) {
        const int r = threadIdx.x / 32, lane = threadIdx.x % 32;
        static_assert(kLogitRows * 32 == kCombineThreads, "32 lanes for each row");
        if (r < e.rows) {
            const Parts parts(a, e, unit, seq, head, r);
            float best = kFar, sum = 0.0f;
            for (int s = lane; s < parts.n; s += 32) {
                const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + 2 * (parts.first + (int64_t)s * parts.stride));
                const float m = fmaxf(best, ml.x);
                sum = sum * exp2f(best - m) + ml.y * exp2f(ml.x - m);
                best = m;
            }
#pragma unroll
            for (int mask = 16; mask; mask >>= 1) {
                const float other = __shfl_xor(best, mask), m = fmaxf(best, other);
                sum = sum * exp2f(best - m) + __shfl_xor(sum, mask) * exp2f(other - m);
                best = m;
            }
            const float lse2 = sum > 0.0f || sum != sum ? best - kLift + log2f(sum) : __builtin_inff();
            if (lane == 0) joined[r] = parts.n ? lse2 : info[2 * r + 1];
        }
        __syncthreads();
    }
    if (pos >= e.len) return;
    f4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < kLogitRows; ++r)
        if (r < e.rows) {
            const float lse2 = JOIN ? joined[r] : info[2 * r + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] += __builtin_amdgcn_exp2f(x[r][i] - lse2);
        }
    const int64_t at = unit * a.score_stride + pos;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (pos + i < e.len) a.scores_out[at + i] = (a.scores_in ? a.scores_in[at + i] : 0.0f) + sum[i];
}

__global__ void __launch_bounds__(kCombineThreads) weigh_kernel(const AttendArgs a, const int blocks) {
    weigh<false>(a, blockIdx.x, blocks);
}

// Joining and weighing in one launch, where a row has few parts: 16 sequences of
// up to 16384 positions, 8 heads of 4 rows, 11.5 us, where two take 5.1 and 9.0.
// The logarithms, 20 MB mostly in the caches yet, are less of it than the way to
// the partial sums by lengths and shares.
template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_weigh_kernel(const AttendArgs a, const int combining,
                                                                        const int blocks) {
    if ((int)blockIdx.x < combining)
        combine_few<D, 4>(a, blockIdx.x);
    else
        weigh<true>(a, blockIdx.x - combining, blocks);
}

static int weighing_blocks(const AttendArgs &a) { return (a.max_len + kWeighPositions - 1) / kWeighPositions; }

int launch_weigh(const AttendArgs &a, void *stream) {
    const int blocks = weighing_blocks(a);
    weigh_kernel<<<dim3((uint32_t)((int64_t)a.b.n_seq * a.c.heads * blocks)), dim3(kCombineThreads), 0,
                   (hipStream_t)stream>>>(a, blocks);
    return (int)hipGetLastError();
}

template <int D>
static int launch(const AttendArgs &a, hipStream_t s) {
    const int64_t rows = (int64_t)a.b.n_seq * a.c.heads * a.rows;
    constexpr int AT_ONCE = kCombineThreads / (D / 4);
    const int combining = (int)((rows + AT_ONCE - 1) / AT_ONCE);
    const int blocks = weighing_blocks(a);
    const int64_t weighing = a.logits ? (int64_t)a.b.n_seq * a.c.heads * blocks : 0;
    const dim3 block(kCombineThreads);
    const bool few = a.even || a.n_split <= kFewParts;
    if (a.n_split > 1) {
        if (few && weighing) {
            combine_weigh_kernel<D><<<dim3((uint32_t)(combining + weighing)), block, 0, s>>>(a, combining, blocks);
            return (int)hipGetLastError();
        }
        if (a.n_split <= 4)  // an even split: its usual number
            combine_few_kernel<D, 4><<<dim3((uint32_t)combining), block, 0, s>>>(a);
        else if (few)
            combine_few_kernel<D, kFewParts><<<dim3((uint32_t)combining), block, 0, s>>>(a);
        else
            combine_kernel<D><<<dim3((uint32_t)(rows * (D / 32))), block, 0, s>>>(a);
    }
    if (weighing) weigh_kernel<<<dim3((uint32_t)weighing), block, 0, s>>>(a, blocks);
    return (int)hipGetLastError();
}

int launch_combine(const AttendArgs &a, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    switch (a.c.dim) {
        case 64: return launch<64>(a, s);
        case 96: return launch<96>(a, s);
        case 128: return launch<128>(a, s);
        case 256: return launch<256>(a, s);
    }
    return (int)hipErrorInvalidValue;
}

}  // namespace tkv
