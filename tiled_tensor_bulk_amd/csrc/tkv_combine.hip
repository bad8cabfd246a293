// tkv_combine.hip -- join the partial sums of attention's chunks.
//
// A row's chunks each bring a reference m, a sum l and a vector o, all scaled
// by exp2(-m): with M the largest m, l = sum l_i exp2(m_i - M), and the same
// for o.  A workgroup takes a row: dim / 4 lanes hold 4 channels each of one
// chunk, and 256 / (dim / 4) chunks are read at a time, as a long context has
// few rows and many chunks.
#include "tkv_attend.h"

namespace tkv {

constexpr int kCombineThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const AttendArgs a) {
    constexpr int LANES = D / 4, AT_ONCE = kCombineThreads / LANES;
    __shared__ float4 join[AT_ONCE][LANES];
    __shared__ float join_m[kCombineThreads / 64], join_l[AT_ONCE];
    const int row = (int)(blockIdx.x % (uint32_t)a.rows);
    const int64_t unit = blockIdx.x / (uint32_t)a.rows;
    const int head = (int)(unit % a.c.heads), seq = (int)(unit / a.c.heads);
    const Extent e(a, seq);
    if (row >= e.rows) return;
    int parts = (e.len + a.chunk - 1) / a.chunk;
    parts = parts < 1 ? 1 : parts;
    const int64_t first = (unit * a.n_split) * a.rows + row;
    const int tid = threadIdx.x, which = tid / LANES, lane = tid % LANES;
    float best = kFar;
    for (int s = tid; s < parts; s += kCombineThreads) best = fmaxf(best, a.part_ml[2 * (first + (int64_t)s * a.rows)]);
#pragma unroll
    for (int mask = 32; mask; mask >>= 1) best = fmaxf(best, __shfl_xor(best, mask));
    if ((tid & 63) == 0) join_m[tid >> 6] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kCombineThreads / 64; ++w) best = fmaxf(best, join_m[w]);
    float sum = 0.0f;
    f4 y = (f4){0, 0, 0, 0};
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
    write_row(a, e, seq, head, row, 4 * lane, y, best, sum);
}

int launch_combine(const AttendArgs &a, void *stream) {
    const dim3 grid((uint32_t)((int64_t)a.b.n_seq * a.c.heads * a.rows)), block(kCombineThreads);
    hipStream_t s = (hipStream_t)stream;
    switch (a.c.dim) {
        case 64: combine_kernel<64><<<grid, block, 0, s>>>(a); break;
        case 96: combine_kernel<96><<<grid, block, 0, s>>>(a); break;
        case 128: combine_kernel<128><<<grid, block, 0, s>>>(a); break;
        case 256: combine_kernel<256><<<grid, block, 0, s>>>(a); break;
        default: return (int)hipErrorInvalidValue;
    }
    return (int)hipGetLastError();
}

}  // namespace tkv
