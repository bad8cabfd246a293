// tkv_combine.hip -- join the partial sums of attention's chunks.
//
// A row's chunks each bring a reference m, a sum l and a vector o, all scaled
// by exp2(-m): with M the largest m, l = sum l_i exp2(m_i - M), and the same
// for o.  dim / 4 lanes take a row, 4 channels each.
#include "tkv_attend.h"

namespace tkv {

__global__ void __launch_bounds__(256) combine_kernel(const AttendArgs a) {
    const int lanes = (int)a.c.dim / 4, per_block = 256 / lanes;
    const int which = threadIdx.x / lanes, channel = 4 * (threadIdx.x % lanes);
    if (which >= per_block) return;
    const int64_t id = (int64_t)blockIdx.x * per_block + which;
    const int row = (int)(id % a.rows);
    const int64_t rest = id / a.rows;
    const int head = (int)(rest % a.c.heads);
    if (rest / a.c.heads >= a.b.n_seq) return;
    const int seq = (int)(rest / a.c.heads);
    const Extent e(a, seq);
    if (row >= e.rows) return;
    int parts = (e.len + a.chunk - 1) / a.chunk;
    parts = parts < 1 ? 1 : parts;
    const int64_t first = (rest * a.n_split) * a.rows + row;
    float best = kFar;
    for (int s = 0; s < parts; ++s) best = fmaxf(best, a.part_ml[2 * (first + (int64_t)s * a.rows)]);
    float sum = 0.0f;
    f4 y = (f4){0, 0, 0, 0};
    for (int s = 0; s < parts; ++s) {
        const int64_t from = first + (int64_t)s * a.rows;
        const float f = exp2f(a.part_ml[2 * from] - best);
        sum += f * a.part_ml[2 * from + 1];
        y += f * *reinterpret_cast<const f4 *>(a.part_o + from * a.c.dim + channel);
    }
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const int i = row / a.group_heads, hq = head * a.group_heads + row % a.group_heads;
    uint16_t *to = (uint16_t *)a.out.data + (e.start + i) * a.out.token_stride + hq * a.out.head_stride + channel;
#pragma unroll
    for (int j = 0; j < 4; ++j) to[j] = float_to_elem(y[j] * inv, a.out.type);
    if (channel == 0) {
        const float log_sum = best - kLift + log2f(sum);
        a.lse[(e.start + i) * (a.c.heads * a.group_heads) + hq] = log_sum * 0.69314718056f;
        if (a.frag_q) {
            const int64_t tile = rest * a.row_tiles + row / 16;
            if (sum > 0.0f || sum != sum)
                a.row_info[(tile * 16 + row % 16) * (2 + a.c.dim / a.c.group) + 1] = log_sum;
        }
    }
}

int launch_combine(const AttendArgs &a, void *stream) {
    const int per_block = 256 / ((int)a.c.dim / 4);
    const int64_t rows = (int64_t)a.b.n_seq * a.c.heads * a.rows;
    combine_kernel<<<dim3((uint32_t)((rows + per_block - 1) / per_block)), dim3(256), 0, (hipStream_t)stream>>>(a);
    return (int)hipGetLastError();
}

}  // namespace tkv
