// rmsq_ops_plan.h -- host rules of the layer-norm and int8 operators that need nothing of CUDA, in plain
// C++ so that tests run them without a device.
#pragma once

#include <cstdint>
#include <map>
#include <set>
#include <tuple>
#include <utility>

namespace rmsq {

// How many clusters of a launch a device runs at a time, as CUDA was asked once: it goes by the
// kernel, the device and the whole shape of the launch. Not synchronised.
class ResidentClusters {
public:
    using Key = std::tuple<const void*, int, unsigned, int, int>;     // kernel, device, threads, smem, cluster

    // query() gives the number, or less than 1 where it cannot be had; that is not kept.
    template <class Query> int get(const Key& key, Query query)
    {
        const auto it = known_.find(key);
        if (it != known_.end()) return it->second;
        const int n = query();
        if (n >= 1) {
            try {
                known_.emplace(key, n);
            } catch (...) {}                                          // no memory: asked again next time
        }
        return n;
    }

private:
    std::map<Key, int> known_;
};

// Kernels whose attributes are set on a device. Not synchronised.
class PreparedKernels {
public:
    bool has(const void* fn, int dev) const { return set_.count({fn, dev}) != 0; }
    void add(const void* fn, int dev)
    {
        try {
            set_.insert({fn, dev});
        } catch (...) {}                                              // no memory: set again next time
    }

private:
    std::set<std::pair<const void*, int>> set_;
};

// Device-side waits count in units of 1024 ns: 32 bits of those last 73 minutes (registers are scarce
// where the kernels wait, and a bound in nanoseconds would be 4 s at most). At least one unit, so that a
// bound is never cut to none, and at most 2^30 (18 minutes).
constexpr uint32_t kWaitMost = 1u << 30;

inline uint32_t wait_units(uint64_t timeout_ns)
{
    const uint64_t units = timeout_ns / 1024 + 1;
    return units < kWaitMost ? static_cast<uint32_t>(units) : kWaitMost;
}

// The bound for copies and products that a stopping CTA still has in flight: four times the wait's, and
// a second at least, because they land within microseconds and nobody may stop waiting for them because
// of a bound set short.
inline uint32_t drain_units(uint64_t timeout_ns)
{
    const uint32_t units = wait_units(timeout_ns);
    constexpr uint32_t second = 1000000000u / 1024;
    if (units > kWaitMost / 2) return 2 * kWaitMost;
    return 4 * units < second ? second : 4 * units;
}

// Clusters (CTAs where a cluster is one) that walk the rows of layer norm's backward pass, each with
// `groups` row groups and one partial row of the column sums: group g of cluster c takes row
// g * clusters + c and every (clusters * groups)-th from there. At most `most`, and otherwise as many as
// run at a time (`resident`), but a CTA's rows have to start at the same place against a 16-byte boundary,
// which rows do that are a multiple of `period` apart (1 to 8). So the clusters are a multiple of the period,
// unless nobody has more than one row; more than are resident run one after another, which they may, as
// clusters do not wait for each other. most >= min(rows, period).
inline int64_t bwd_clusters(int64_t rows, int groups, int period, int64_t resident, int64_t most)
{
    if (rows < period) return rows;
    int64_t n = (rows + groups - 1) / groups;
    if (n > resident) n = resident;
    if (n > most) n = most;
    if (groups == 1 && n == rows) return n;
    return n < period ? period : n / period * period;
}

}  // namespace rmsq
