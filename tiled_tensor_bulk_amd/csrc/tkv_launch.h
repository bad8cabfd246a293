// tkv_launch.h -- the launches of one attention call, for one head_dim.
#pragma once

#include "tkv_rows8.h"
#include "tkv_scores.h"

namespace tkv {

template <int D, int GROUP, bool BF16, bool WIN>
static int launch_type(const AttendArgs &a, int row_tile, void *stream) {
    const dim3 block(64 * kAttendWaves);
    const dim3 grid((uint32_t)(a.even ? a.groups : (int64_t)a.b.n_seq * a.c.heads * a.n_split * a.row_blocks));
    hipStream_t s = (hipStream_t)stream;
    if (row_tile == 16) {
        if (a.even)
            attend_kernel<D, GROUP, 1, BF16, true, WIN><<<grid, block, 0, s>>>(a);
        else
            attend_kernel<D, GROUP, 1, BF16, false, WIN><<<grid, block, 0, s>>>(a);
    } else if (row_tile == 32) {
        if constexpr (D > 128)
            return (int)hipErrorInvalidValue;
        else if (a.even)
            attend_kernel<D, GROUP, 2, BF16, true, WIN><<<grid, block, 0, s>>>(a);
        else
            attend_kernel<D, GROUP, 2, BF16, false, WIN><<<grid, block, 0, s>>>(a);
    } else if (row_tile == 64) {
        if constexpr (GROUP == 0)
            return (int)hipErrorInvalidValue;
        else
            rows_kernel<D, GROUP, 1, BF16, WIN><<<grid, block, 0, s>>>(a);
    } else {
        if constexpr (D > 128 && GROUP != 0)
            return (int)hipErrorInvalidValue;
        else if constexpr (GROUP == 0)
            rows8_kernel<D, BF16><<<grid, block, 0, s>>>(a);
        else
            rows_kernel<D, GROUP, 2, BF16, WIN><<<grid, block, 0, s>>>(a);
    }
    return (int)hipGetLastError();
}

// The 8-bit format's kernels have registers left for a window, which then may be
// none; those of 4 bits are there without one too.
template <int D, int GROUP>
static int launch_types(const AttendArgs &a, int row_tile, void *stream) {
    const bool bf16 = a.q.type == kBf16;
    if (GROUP == 0 || a.window)
        return bf16 ? launch_type<D, GROUP, true, true>(a, row_tile, stream)
                    : launch_type<D, GROUP, false, true>(a, row_tile, stream);
    if constexpr (GROUP == 0)
        return (int)hipErrorInvalidValue;
    else
        return bf16 ? launch_type<D, GROUP, true, false>(a, row_tile, stream)
                    : launch_type<D, GROUP, false, false>(a, row_tile, stream);
}

template <int D, int GROUP, bool WIN>
static int resident(int row_tile) {
    if constexpr (D <= 128)
        if (row_tile == 32) return FewRows<D, GROUP, 2, WIN>::kResident;
    return FewRows<D, GROUP, 1, WIN>::kResident;
}

template <int D, int GROUP>
static int launch_group(AttendArgs a, int row_tile, void *stream) {
    const dim3 block(64 * kAttendWaves);
    a.groups = a.cus * (GROUP == 0 || a.window ? resident<D, GROUP, true>(row_tile) : resident<D, GROUP, false>(row_tile));
    hipStream_t s = (hipStream_t)stream;
    int rc = launch_types<D, GROUP>(a, row_tile, stream);
    if (rc == 0 && (a.n_split > 1 || a.logits)) rc = launch_combine(a, stream);
    if constexpr (GROUP != 0) {
        if (rc == 0 && a.scores_out && !a.logits && a.max_len > 0) {
            constexpr int kPositions = kTile * kAttendWaves;
            const int64_t splits = (a.max_len + kPositions - 1) / kPositions;
            scores_kernel<D, GROUP><<<dim3((uint32_t)(splits * a.c.heads * a.b.n_seq)), block, 0, s>>>(a);
            rc = (int)hipGetLastError();
        }
    }
    return rc;
}

}  // namespace tkv
