// norm_plan.h - launches of the gradients' norm (adamw.cu) and the room that their sums take; plain C++ as well, so that
// the room is checked on the host against every launch's blocks (tests/test_norm_plan.py).
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace moe {

constexpr int kListMost = 384;       // tensors of a launch
constexpr int kListUnit = 256;       // values of a warp at a time
constexpr int kListWarps = 8;        // of a block
constexpr int kNormMostSms = 1024;   // that there is room for

inline long long list_units(long long n) { return (n + kListUnit - 1) / kListUnit; }

// Blocks of a launch over so many units, one at least (a list without values has a norm too).  Four units a warp at
// least: blocks come to one ticket at the end, a few nanoseconds each (1.2 M values in 586 blocks took 8.6 us).
inline int norm_blocks_of(long long units, int num_sms) {
    return (int)std::max<long long>(1, std::min<long long>((units + 4 * kListWarps - 1) / (4 * kListWarps), 4 * num_sms));
}

// The status word's line, the ticket's, a partial sum for each block of each launch: at most four blocks an SM and launch, and
// not more than one for each unit and launch.
inline size_t norm_room(int64_t elements, int64_t count) {
    const int64_t launches = std::max<int64_t>(1, (count + kListMost - 1) / kListMost);
    return 512 + 8 * (size_t)std::min<int64_t>(launches * 4 * kNormMostSms, elements / kListUnit + count + launches);
}

// What state[0] of a workspace's handle says about the buffer.
enum : uint64_t { kWorkspaceZero = 0, kWorkspaceData = 1, kWorkspaceSums = 2 };

// A norm's launches, of the tensors from `first` on, until one fails (not 0).  The sums' ticket is zero again after the
// last of them only, so until then, and after a failure, the buffer counts as one that holds data: it is to be set
// to zero again, its handle with it.
template <typename Launch>
auto norm_launches(int64_t count, uint64_t* state, Launch launch) -> decltype(launch(count)) {
    *state = kWorkspaceData;
    for (int64_t first = 0; first == 0 || first < count; first += kListMost)
        if (const auto failed = launch(first)) return failed;
    *state = kWorkspaceSums;   // which moe_balance_fwd refuses
    return decltype(launch(count))(0);
}

}  // namespace moe
