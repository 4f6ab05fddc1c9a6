// ccc_waits.h -- what a kernel with bounded waits is given (ccc_waits.cu).
#pragma once

#include <cstdint>

namespace ccc {

struct Waits {
    unsigned int *given_up;  // the device's counter of CTAs that gave a wait up; null where it cannot be found
    int64_t limit;           // clocks that a wait lasts at most
};

Waits current_waits();

}  // namespace ccc
