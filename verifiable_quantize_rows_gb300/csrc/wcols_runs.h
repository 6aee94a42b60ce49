// wcols_runs.h -- how the list of blocks of a product of few tokens is dealt out.
#pragma once

#include <stdint.h>

namespace bsg {

// Equal runs of the list (`all` blocks) for each of `blocks` groups of tokens: one CTA takes an SM,
// so no more of them than there are SMs.  (Rounded up, 51 for each of three groups on 152 SMs, the
// 153rd ran by itself after the others: 192 x 4096 x 4096 38 us in place of 32, 192 x
// 8192 x 8192 99 in place of 60.)
constexpr int64_t wcols_runs(int64_t all, int64_t blocks, int64_t sms) {
    const int64_t runs = sms > blocks ? sms / blocks : 1;
    return all < runs ? all : runs;
}

}  // namespace bsg
