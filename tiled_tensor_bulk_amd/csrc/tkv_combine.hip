// tkv_combine.hip -- join the partial sums of attention's chunks.
//
// A row's chunks each bring a reference m, a sum l and a vector o, all scaled
// by exp2(-m): with M the largest m, l = sum l_i exp2(m_i - M), and the same
// for o.  dim / 4 lanes hold 4 channels each of a row; where a row has many
// chunks, as a few rows of a long context have, a workgroup takes one row and
// reads 256 / (dim / 4) chunks at a time, else it takes as many rows.
#include "tkv_attend.h"

namespace tkv {

constexpr int kCombineThreads = 256;
constexpr int kFewParts = 4;

template <int D, bool FEW>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const AttendArgs a) {
    constexpr int LANES = D / 4, AT_ONCE = kCombineThreads / LANES;
    const int tid = threadIdx.x, which = tid / LANES, lane = tid % LANES;
    const int64_t id = FEW ? (int64_t)blockIdx.x * AT_ONCE + which : blockIdx.x;
    const int row = (int)(id % a.rows);
    const int64_t unit = id / a.rows;
    const int head = (int)(unit % a.c.heads);
    if (FEW && (which >= AT_ONCE || unit / a.c.heads >= a.b.n_seq)) return;
    const int seq = (int)(unit / a.c.heads);
    const Extent e(a, seq);
    if (row >= e.rows) return;
    const int parts = Chunks(a, e.len).n;
    const int64_t first = (unit * a.n_split) * a.rows + row;
    float best = kFar, sum = 0.0f;
    f4 y = (f4){0, 0, 0, 0};
    if constexpr (FEW) {
        float2 ml[kFewParts];
        f4 o[kFewParts];
#pragma unroll
        for (int s = 0; s < kFewParts; ++s)
            if (s < parts) {
                const int64_t from = first + (int64_t)s * a.rows;
                ml[s] = *reinterpret_cast<const float2 *>(a.part_ml + 2 * from);
                o[s] = *reinterpret_cast<const f4 *>(a.part_o + from * D + 4 * lane);
                best = fmaxf(best, ml[s].x);
            }
#pragma unroll
        for (int s = 0; s < kFewParts; ++s)
            if (s < parts) {
                const float f = exp2f(ml[s].x - best);
                sum += f * ml[s].y;
                y += f * o[s];
            }
    } else {
        __shared__ float4 join[AT_ONCE][LANES];
        __shared__ float join_m[kCombineThreads / 64], join_l[AT_ONCE];
        for (int s = tid; s < parts; s += kCombineThreads)
            best = fmaxf(best, a.part_ml[2 * (first + (int64_t)s * a.rows)]);
#pragma unroll
        for (int mask = 32; mask; mask >>= 1) best = fmaxf(best, __shfl_xor(best, mask));
        if ((tid & 63) == 0) join_m[tid >> 6] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kCombineThreads / 64; ++w) best = fmaxf(best, join_m[w]);
        if (which < AT_ONCE) {
#pragma unroll 4
            for (int s = which; s < parts; s += AT_ONCE) {
                const int64_t from = first + (int64_t)s * a.rows;
                const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + 2 * from);
                const float f = exp2f(ml.x - best);
                sum += f * ml.y;
                y += f * *reinterpret_cast<const f4 *>(a.part_o + from * D + 4 * lane);
            }
            *reinterpret_cast<f4 *>(&join[which][lane]) = y;
            if (lane == 0) join_l[which] = sum;
        }
        __syncthreads();
        if (which) return;
#pragma unroll
        for (int w = 1; w < AT_ONCE; ++w) {
            sum += join_l[w];
            y += *reinterpret_cast<const f4 *>(&join[w][lane]);
        }
    }
    write_row(a, e, seq, head, row, 4 * lane, y, best, sum);
}

template <int D>
static int launch(const AttendArgs &a, hipStream_t s) {
    const int64_t rows = (int64_t)a.b.n_seq * a.c.heads * a.rows;
    constexpr int AT_ONCE = kCombineThreads / (D / 4);
    if (a.n_split <= kFewParts)
        combine_kernel<D, true><<<dim3((uint32_t)((rows + AT_ONCE - 1) / AT_ONCE)), dim3(kCombineThreads), 0, s>>>(a);
    else
        combine_kernel<D, false><<<dim3((uint32_t)rows), dim3(kCombineThreads), 0, s>>>(a);
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
