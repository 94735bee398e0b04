// bwd_layout.h -- shared memory of the backward's per-key-tile kernel (tc_bwd.cu), and what is given up where
// it is short.  Plain integer arithmetic, for host and device (and for a host program that checks it
// without the CUDA headers).
#pragma once

#include <stdint.h>

#include "sink_window.h"

namespace triattn {
namespace tc {

constexpr uint32_t kBwdBox = 128 * 128;        // one [128 rows][128 B] box
constexpr uint32_t kBwdMaxSmem = 232448;       // 227 KB, what a block may have (kMaxDynamicSmem)
constexpr uint32_t kBwdAlign = 1024;           // of the first box

// What the layout depends on.
struct BwdShape {
    int qs;               // stages of (Q, dO, the rows' sums): 2 or 1
    int lo;               // 1: dS in two 16-bit pieces
    int lse_row;          // 1: the rows' lse lie beside them; 0: they are read from global memory where they are needed
    int bias_alias;       // 1: the two bias halves share one slot (an fp32 bias with D > 64)
    uint32_t bias_bytes;  // 0: no bias
    int qcap;             // entries of the q-block list (0: triangle form)
};

// Offsets from a 1024-byte aligned base.
// Stage s of the query-tile ring: Q at q + s * 2 tile, dO after it; the rows' -lse log2e, -delta and lse
// (128 floats each) at lse + s * bwd_row_bytes
// (tile = nsub boxes of 128 rows x 128 bytes).
struct BwdLayout {
    uint32_t k, v, q, ds, bias, dqst, lse, qlist, bars, tmem_slot, abort_flag, qn, total;
};
// kv_full, q_full[2], q_empty[2], lse_full[2], bias_full[2], bias_empty[2], s_full[2], p_full[2],
// dq_full, dq_empty, ds_free, fin, drain
constexpr int kBwdBars = 20;
TRIATTN_HD uint32_t bwd_row_bytes(bool lse_row) { return (lse_row ? 3u : 2u) * 128 * 4; }
// nsub: the kernel passes its compile-time box count, so that the offsets fold into constants.
TRIATTN_HD BwdLayout bwd_layout(const BwdShape& P, int nsub) {
    BwdLayout L;
    const uint32_t tile = (uint32_t)nsub * kBwdBox;  // one 128-row tile of D columns
    L.k = 0;
    L.v = L.k + tile;
    L.q = L.v + tile;
    L.ds = L.q + (uint32_t)P.qs * 2 * tile;  // dS as [key][query]: two 64-query boxes (its second pieces after them)
    L.bias = L.ds + (P.lo ? 4 : 2) * kBwdBox;
    L.dqst = L.bias + (P.bias_alias ? P.bias_bytes / 2u : P.bias_bytes);  // dQ staging: 16 warps x 32 rows x 16 fp32
    L.lse = L.dqst + 16u * 2048u;
    L.qlist = L.lse + (uint32_t)P.qs * bwd_row_bytes(P.lse_row != 0);  // packed form: the q blocks the key tile visits
    L.bars = L.qlist + (((uint32_t)P.qcap * 4u + 15u) & ~15u);
    L.tmem_slot = L.bars + 8 * kBwdBars;
    L.abort_flag = L.tmem_slot + 4;
    L.qn = L.abort_flag + 4;                   // packed form: entries of the q-block list
    L.total = L.qn + 4;
    return L;
}
TRIATTN_HD bool bwd_fits(const BwdShape& P, int nsub) { return bwd_layout(P, nsub).total + kBwdAlign <= kBwdMaxSmem; }

// The shape of a problem; false: it does not fit.  bias: 0 none, 2 or 4 bytes an element; max_q: of packed sequences
// (-1: triangle form); two_pieces: dS in two pieces where they fit.
TRIATTN_HD bool bwd_shape(BwdShape& P, int D, int bias, int max_q, bool two_pieces) {
    const int nsub = (D + 63) / 64;
    P.lo = 0;
    P.bias_alias = D > 64 && bias == 4;
    P.bias_bytes = bias ? (bias == 4 ? 4u : 2u) * kBwdBox : 0u;  // 128 keys x 128 rows
    P.qcap = max_q < 0 ? 0 : (max_q + 127) / 128;
    // Two stages where they fit (D > 64: one, taken per query half).  The q-block list of a long sequence may push the lse
    // row out, as an fp32 bias with D > 64 does: only rows of blocks on the mask's edges, or with queries past the
    // end, then go to global memory for it.  (Heads of 65 to 128 with a 16-bit bias: from 10753 rows of a sequence.)
    const bool row = !P.bias_alias;
    for (P.qs = D > 64 ? 1 : 2; P.qs > 0; --P.qs) {
        P.lse_row = row;
        if (!bwd_fits(P, nsub) && max_q >= 0) P.lse_row = 0;
        if (bwd_fits(P, nsub)) break;
    }
    if (P.qs == 0) return false;
    if (two_pieces) {
        P.lo = 1;
        if (!bwd_fits(P, nsub)) P.lo = 0;
    }
    return true;
}

}  // namespace tc
}  // namespace triattn
