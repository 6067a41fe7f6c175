// The sum behind the prompt kernel's line of work, for the kernel and for a test on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define LORA_HOST_DEVICE __host__ __device__
#else
#define LORA_HOST_DEVICE
#endif

namespace lora {

// Sum of floor((2 i + b) / m) over 0 <= i < n, m >= 1.
// With b = m q + r the i-th term is q and the number of k >= 1 with k m <= 2 i + r,
// so the sum is n q and, for each k up to the last that occurs, K =
// floor((2 (n - 1) + r) / m), the count of the i from ceil((k m - r) / 2) to n - 1:
//     n q + n K - sum_k (k m - r + [k m - r odd]) / 2.
// k m - r is odd for every k or none where m is even (as r is odd or not), and
// for every other k where m is odd: the even ones if r is odd, else the odd ones.
LORA_HOST_DEVICE inline long long sum_of_floors(uint32_t n, uint32_t m, uint32_t b) {
    if (n == 0) return 0;
    const uint32_t q = b / m, r = b % m;
    const uint32_t K = (2 * (n - 1) + r) / m;
    const uint32_t odd = m % 2 == 0 ? (r % 2 ? K : 0) : r % 2 ? K / 2 : (K + 1) / 2;
    const long long k_sum = static_cast<long long>(K) * (K + 1) / 2;
    return static_cast<long long>(n) * q + static_cast<long long>(n) * K -
           (m * k_sum - static_cast<long long>(r) * K + odd) / 2;
}

}  // namespace lora
