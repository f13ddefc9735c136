// cluster_counts.h -- how many clusters of a kernel run at once, asked once for
// each device, kernel and launch shape.  Host code without CUDA, so that a test
// can put a fake in the place of the query.
#pragma once

#include <map>
#include <mutex>
#include <tuple>

namespace zs {

class ClusterCounts {
public:
    // query() is called where the count is not known yet.  An answer below 1 (the
    // query failed) is passed on and not kept: the next call asks again.
    template <typename Query>
    int get(int device, const void* kernel, int ctas, int smem, Query query) {
        const auto key = std::make_tuple(device, kernel, ctas, smem);
        {
            std::lock_guard<std::mutex> lock(mu_);
            const auto it = known_.find(key);
            if (it != known_.end()) return it->second;
        }
        const int n = query();
        if (n < 1) return n;
        try {
            std::lock_guard<std::mutex> lock(mu_);
            known_[key] = n;
        } catch (...) {  // no memory to remember it: asked again at the next call
        }
        return n;
    }

private:
    std::mutex mu_;
    std::map<std::tuple<int, const void*, int, int>, int> known_;
};

}  // namespace zs
