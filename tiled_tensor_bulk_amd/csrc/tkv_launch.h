// tkv_launch.h -- the launches of one attention call, for one head_dim.
#pragma once

#include "tkv_rows.h"
#include "tkv_scores.h"

namespace tkv {

template <int D, int GROUP, bool BF16>
static int launch_type(const AttendArgs &a, int row_tile, void *stream) {
    const dim3 block(64 * kAttendWaves);
    const dim3 grid((uint32_t)(a.even ? a.groups : (int64_t)a.b.n_seq * a.c.heads * a.n_split * a.row_blocks));
    hipStream_t s = (hipStream_t)stream;
    if (row_tile == 16) {
        if (a.even)
            attend_kernel<D, GROUP, 1, BF16, true><<<grid, block, 0, s>>>(a);
        else
            attend_kernel<D, GROUP, 1, BF16, false><<<grid, block, 0, s>>>(a);
    } else if (row_tile == 32) {
        if constexpr (D > 128)
            return (int)hipErrorInvalidValue;
        else if (a.even)
            attend_kernel<D, GROUP, 2, BF16, true><<<grid, block, 0, s>>>(a);
        else
            attend_kernel<D, GROUP, 2, BF16, false><<<grid, block, 0, s>>>(a);
    } else if (row_tile == 64) {
        rows_kernel<D, GROUP, 1, BF16><<<grid, block, 0, s>>>(a);
    } else {
        if constexpr (D > 128)
            return (int)hipErrorInvalidValue;
        else
            rows_kernel<D, GROUP, 2, BF16><<<grid, block, 0, s>>>(a);
    }
    return (int)hipGetLastError();
}

template <int D, int GROUP>
static int launch_group(AttendArgs a, int row_tile, void *stream) {
    const dim3 block(64 * kAttendWaves);
    int resident = FewRows<D, GROUP, 1>::kResident;
    if constexpr (D <= 128)
        if (row_tile == 32) resident = FewRows<D, GROUP, 2>::kResident;
    a.groups = a.cus * resident;
    hipStream_t s = (hipStream_t)stream;
    int rc = a.q.type == kBf16 ? launch_type<D, GROUP, true>(a, row_tile, stream)
                               : launch_type<D, GROUP, false>(a, row_tile, stream);
    if (rc == 0 && (a.n_split > 1 || a.logits)) rc = launch_combine(a, stream);
    if (rc == 0 && a.scores_out && !a.logits && a.max_len > 0) {
        constexpr int kPositions = kTile * kAttendWaves;
        const int64_t splits = (a.max_len + kPositions - 1) / kPositions;
        scores_kernel<D, GROUP><<<dim3((uint32_t)(splits * a.c.heads * a.b.n_seq)), block, 0, s>>>(a);
        rc = (int)hipGetLastError();
    }
    return rc;
}

}  // namespace tkv
