// Grids larger than one launch holds (host code only).
#pragma once

#include <cstdint>

namespace zs {

// Calls launch(first, count) for the workgroups first .. first + count - 1 of `grid`,
// in order, each with fewer than 2^32 threads, which is what HIP takes at a time.
// `first` is a multiple of 8, so that a workgroup's number says the same XCD in every
// launch.  Stops at the first error.
template <typename Launch>
auto launch_ranges(int64_t grid, int threads, Launch launch) {
    const int64_t most = 0xffffffffll / threads / 8 * 8;
    decltype(launch(int64_t(0), int64_t(0))) err{};
    for (int64_t first = 0; first < grid && err == decltype(err){}; first += most)
        err = launch(first, grid - first < most ? grid - first : most);
    return err;
}

}  // namespace zs
