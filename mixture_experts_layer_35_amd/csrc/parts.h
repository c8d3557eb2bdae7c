// parts.h -- arithmetic that kernels and host code share, without HIP, so that it can be tried at any size without a GPU.
#pragma once

namespace moe {

// Pieces of `unit` that hold n things, none for n <= 0.  n + unit - 1 would leave 32 bits for the last `unit` counts
// below 2^31, which an expert's rows may reach.
constexpr int parts_of(int n, int unit) { return n > 0 ? (n - 1) / unit + 1 : 0; }

}  // namespace moe
