// pn_launch.h -- how many workgroups one launch takes.
#pragma once

#include "pn_common.h"

namespace pn {

// Workgroups of `threads` threads that one launch takes. HIP counts a grid's threads in 32 bits: of more it runs what is left
// modulo 2^32, without an error.
constexpr int64_t launch_most(int threads) { return (((int64_t)1 << 32) - 1) / threads; }

// launch(first row, rows, workgroups of 256 threads) for N rows of `threads` threads each, in as many launches as it takes.
template <typename F>
inline int launch_rows(int64_t N, int64_t threads, F launch)
{
    const int64_t most = launch_most(256) * 256 / threads;
    if (most == 0)
        return PN_ERR_SHAPE;
    int st = PN_OK;
    for (int64_t first = 0; first < N && st == PN_OK; first += most) {
        const int64_t rows = N - first < most ? N - first : most;
        launch(first, rows, dim3((unsigned)((rows * threads + 255) / 256)));
        st = launch_status();
    }
    return st;
}

}  // namespace pn
