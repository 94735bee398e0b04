// prompt.cuh -- causal attention of packed prompts with grouped heads: what its kernels (prompt_simt.cu, prompt_fwd.cu,
// prompt_dq.cu, prompt_dkv.cu) share.
//
//     O[i, h] = softmax_k(scale q_i . K[k]) V,  the keys k <= Lk - Lq + j seen by query j of a sequence's Lq,
// query head h on key head h / G.  The G heads of a group read the same keys, so their queries are rows of one matrix:
// row r of (sequence, key head) is token r / G, head r % G of the group, and only which keys a row sees depends on r.
// Grouped heads are thus plain attention with G times as many rows, and the gradients of K and V, summed over the
// group, are the sums over the rows that they are without groups.
#pragma once

#include "internal.h"
#include "prompt_order.h"
#include "rotary.cuh"

namespace triattn {
namespace prompt {

// A sequence that breaks the contract counts as holding nothing.
__device__ __forceinline__ Seq load_seq(const PromptParams& p, int s, bool tell) {
    Seq q;
    q.q0 = p.cu_q[s];
    q.k0 = p.cu_k[s];
    const int q1 = p.cu_q[s + 1], k1 = p.cu_k[s + 1];
    q.lq = q1 - q.q0;
    q.lk = k1 - q.k0;
    if (q.q0 < 0 || q.k0 < 0 || q1 < q.q0 || k1 < q.k0 || q1 > p.total_q || k1 > p.total_k || q.lq > p.max_q ||
        q.lk > p.max_k) {
        if (tell) atomicCAS(p.status, 0, kStatusDevice);
        q.lq = q.lk = 0;
        q.q0 = q.k0 = 0;
    }
    q.shift = q.lk - q.lq;
    return q;
}

constexpr float kToLog2 = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

}  // namespace prompt
}  // namespace triattn
