// Answers to "how many clusters of this width run at once", kept for the process: one per device, since devices differ
// in how their SMs are grouped, and per width.  They choose how a product's K is split and with that the order of its
// sums, so a query that failed leaves nothing behind.  Plain C++.
#pragma once

#include <atomic>

namespace ttm {

class KnownClusters {
    static constexpr int kDevices = 64, kWidths = 9;
    std::atomic<int> kept_[kDevices][kWidths] = {};     // an answer and one; 0: not asked

public:
    // `ask(&n)` returns 0 and sets n, or an error code, which is passed on.
    template <typename Ask>
    auto get(int device, int width, int& n, Ask ask) -> decltype(ask(&n)) {
        std::atomic<int>* at = device >= 0 && device < kDevices && width > 0 && width < kWidths ? &kept_[device][width] : nullptr;
        const int kept = at ? at->load(std::memory_order_relaxed) : 0;
        n = kept - 1;
        if (kept) return {};
        n = 0;
        const auto error = ask(&n);
        if (error == decltype(error){} && at) at->store(n + 1, std::memory_order_relaxed);
        return error;
    }
};

}  // namespace ttm
