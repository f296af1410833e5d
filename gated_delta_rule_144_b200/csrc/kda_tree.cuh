// Read-outs of a tree of drafted tokens against a state, and the state advanced along a path.
#pragma once

#include "kda_internal.cuh"

namespace kda {

constexpr int kMaxTreeNodes = 64;

struct TreeParams {
    const void* q;          // [N, T, H, 128] (tree only)
    const void* k;
    const void* v;
    const float* log_g;     // [N, T, H, 128]
    const void* beta;       // [N, T, H]
    const int32_t* nodes;   // tree: parents [N, T]; path: rows [N, A]
    float* S;               // [N, H, 128, 128] (read only for the tree)
    void* o;                // [N, T, H, 128] (tree only)
    int N, H, T, A;
    bool bf16;
    unsigned* err;
    bool clear;             // tree: zeros to the rows of o without a node
};

cudaError_t launch_decode_tree(const TreeParams& p, cudaStream_t stream);
cudaError_t launch_commit_path(const TreeParams& p, cudaStream_t stream);

}  // namespace kda
