// rmsq_ops_plan.h -- host rules of the layer-norm and int8 operators that need nothing of CUDA, in plain
// C++ so that tests run them without a device.
#pragma once

#include <cstdint>

namespace rmsq {

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

}  // namespace rmsq
