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

constexpr int kCombineThreads = 256;
constexpr int kFewParts = 16;

template <int D, int PARTS>
__global__ void __launch_bounds__(kCombineThreads) combine_few_kernel(const AttendArgs a) {
    constexpr int LANES = D / 4, AT_ONCE = kCombineThreads / LANES;
    const int which = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    int row = blockIdx.x * AT_ONCE + which;
    const int unit = divide(row, a.rows, a.by_rows);
    int head = unit;
    const int seq = divide(head, (int)a.c.heads, a.by_heads);
    if (which >= AT_ONCE || seq >= a.b.n_seq) return;
    const Extent e(a, seq);
    if (row >= e.rows) return;
    int parts, part_rows = a.rows;
    int64_t first;
    if (a.even) {
        const int rows = 1 << a.row_shift, steps = Even::steps(e), block = row >> a.row_shift;
        const uint32_t share = (uint32_t)a.dealt[kEvenSeqs];
        const uint32_t from = (uint32_t)(a.dealt[seq] + (head * Even::blocks(a, e) + block) * (steps + Even::kLead) + Even::kLead);
        const uint32_t part = from / share;
        parts = (int)((from + steps - 1) / share - part) + 1;
        if (parts == 1) return;  // written where it was computed
        part_rows = part_rows < rows ? part_rows : rows;
        first = ((int64_t)unit * a.row_blocks + block + part) * part_rows + (row & (rows - 1));
    } else {
        parts = Chunks(a, e.len).n;
        first = ((int64_t)unit * a.n_split) * a.rows + row;
    }
    float best = kFar, sum = 0.0f;
    f4 y = (f4){0, 0, 0, 0};
    for (int base = 0; base < parts; base += PARTS) {  // once, but for an even split's longest
        float2 ml[PARTS];
        f4 o[PARTS];
#pragma unroll
        for (int s = 0; s < PARTS; ++s) {  // past the last one: it again, without weight
            const int64_t from = first + (int64_t)(base + s < parts ? base + s : parts - 1) * part_rows;
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
            if (base + s < parts) {
                const float f = exp2f(ml[s].x - best);
                sum += f * ml[s].y;
                y += f * o[s];
            }
    }
    write_row(a, e, seq, head, row, 4 * lane, y, best, sum);
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

template <int D>
static int launch(const AttendArgs &a, hipStream_t s) {
    const int64_t rows = (int64_t)a.b.n_seq * a.c.heads * a.rows;
    constexpr int AT_ONCE = kCombineThreads / (D / 4);
    if (a.n_split <= 4)  // an even split: its usual number
        combine_few_kernel<D, 4><<<dim3((uint32_t)((rows + AT_ONCE - 1) / AT_ONCE)), dim3(kCombineThreads), 0, s>>>(a);
    else if (a.even || a.n_split <= kFewParts)
        combine_few_kernel<D, kFewParts><<<dim3((uint32_t)((rows + AT_ONCE - 1) / AT_ONCE)), dim3(kCombineThreads), 0, s>>>(a);
    else
        combine_kernel<D><<<dim3((uint32_t)(rows * (D / 32))), dim3(kCombineThreads), 0, s>>>(a);
    return (int)hipGetLastError();
}

// scores_out = scores_in + the weights of a few rows, exp2(y - lse2), summed,
// from the logarithms that the first kernel has kept: masked ones are -inf.
// A lane takes 4 positions.  Memory bounds it: 16 sequences of up to 16384
// positions, 8 heads of 4 rows, 9 us for 32 MB, some of it still in the caches.
__global__ void __launch_bounds__(256) weigh_kernel(const AttendArgs a, const int blocks) {
    const int64_t unit = blockIdx.x / (uint32_t)blocks;
    const int block = blockIdx.x % (uint32_t)blocks;
    int head = (int)unit;
    const int seq = divide(head, (int)a.c.heads, a.by_heads);
    const Extent e(a, seq);
    const int pos = (block * 256 + (int)threadIdx.x) * 4;
    if (pos >= e.len) return;
    const int64_t records = (a.max_len + kTile - 1) / kTile;
    const float *y = a.logits + (unit * records + pos / kTile) * a.rows * kTile + (pos & (kTile - 1));
    const float *info = a.row_info + unit * 16 * 2;
    f4 sum = {0, 0, 0, 0};
    for (int r = 0; r < e.rows; ++r) {
        const f4 x = *reinterpret_cast<const f4 *>(y + r * kTile);
        const float lse2 = info[2 * r + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += __builtin_amdgcn_exp2f(x[i] - lse2);
    }
    const int64_t at = unit * a.score_stride + pos;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (pos + i < e.len) a.scores_out[at + i] = (a.scores_in ? a.scores_in[at + i] : 0.0f) + sum[i];
}

int launch_weigh(const AttendArgs &a, void *stream) {
    const int blocks = (a.max_len + 1023) / 1024;
    const int64_t grid = (int64_t)a.b.n_seq * a.c.heads * blocks;
    if (grid == 0) return 0;
    weigh_kernel<<<dim3((uint32_t)grid), dim3(256), 0, (hipStream_t)stream>>>(a, blocks);
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
