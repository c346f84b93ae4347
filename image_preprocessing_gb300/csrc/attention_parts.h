// Device parts shared by the attention kernels: where sequences lie.
#pragma once

#include <cuda_runtime.h>

#include "attention_plan.h"
#include "token_ops.h"

namespace trfn {

// Rows of one sequence in a matrix, whatever the arrays hold: within 0 .. rows.
struct Range {
    int start, length;
};
__device__ __forceinline__ Range range_of(const int32_t* starts, const int32_t* lengths, int s, int rows) {
    const int at = min(max(starts[s], 0), rows);
    const long long end = lengths != nullptr ? (long long)at + max(lengths[s], 0) : (long long)starts[s + 1];
    return Range{at, (int)min(max(end, (long long)at), (long long)rows) - at};
}

struct Sequences {
    const int32_t* q_starts;
    const int32_t* k_starts;
    const int32_t* q_lengths;
    const int32_t* k_lengths;
    int q_rows, k_rows, count;
};

// tcgen05 attention (attention_tc.cu), where it applies.
bool attention_tc_supported(const AttentionArgs& a);
int launch_attention_tc(const AttentionArgs& a);
size_t attention_tc_workspace(long long q_rows, long long heads, long long kv_heads, long long dim);

}  // namespace trfn
