// What the kernels on drafted trees share (gpt.h, "drafted trees").
#pragma once

#include "common.cuh"

namespace gpt {

constexpr int kMaxNodes = GPT_TREE_MAX_NODES;

// The set A(i) (node i and its ancestors) as a bit mask, 0 for no node.  par: the sequence's parents
// in shared memory.  A parent lies below its child, so the walk ends after at most i steps.
GPT_DEVINL unsigned long long ancestors(const int* par, int i) {
    unsigned long long m = 0;
    for (int j = i;;) {
        m |= 1ull << j;
        const int p = par[j];
        if (p == -1) return m;
        if (p < 0 || p >= j) return 0;
        j = p;
    }
}

GPT_DEVINL int clamp_length(int len, int block_size, int32_t* status) {
    if (len >= 0 && len <= block_size) return len;
    set_status(status, GPT_ERR_BAD_SHAPE);
    return len < 0 ? 0 : block_size;
}

}  // namespace gpt
