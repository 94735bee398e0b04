// prompt_dkv.cu -- the gradients of keys and values in the causal attention of packed prompts with grouped heads on tcgen05
// tensor cores: 16-bit inputs, D <= 128.  (dQ: prompt_dq.cu; delta = dO . O: prompt_simt.cu, before both.)
//
// Rows are tokens x heads of a group (prompt.cuh), in tiles as in the forward.  With P = 2^(s - lse) recomputed, one CTA for
// each (sequence, key head, 128 keys) walks the row tiles that see a key of its own:
//     S^T = K Q^T, dP^T = V dO^T         keys on the tensor-memory lanes, rows of the tile in the columns
//     dV += P^T dO                       P^T as 16-bit pairs over S^T
//     dS = P (dP - delta),  dK += dS^T Q dS^T as 16-bit pairs over dP^T (as two in rows that see few keys: prompt_dq.cu)
// (fp16: P and dS times powers of two, prompt_tc.cuh).
// Tensor memory: S^T, dP^T, dV, dK: 4 x 128 columns at D = 128.  The sums over the group's heads are sums over rows.
//
// 12 warps: 0-7 softmax and dS (key = lane, 64 rows each half), 8 MMA, 9 TMA, 10 the rows' lse and delta.  The tensor core's
// order is dV(i), S(i+1), dK(i), dP(i+1): while dS(i) is formed it has dV(i) and S(i+1) to do, and dK(i) and dP(i+1) while
// P(i+1) is.
//
// Bound: the tensor core and shared memory alike, 2048 clocks a tile at D = 128 (192 KB of operands and 64 KB of loads at 128
// bytes a clock; a tile takes some 2650), then the softmax warps, two phases of about a thousand clocks a tile, which is what
// counts at D = 64.  bf16, four sequences of 8192 tokens, 16 heads over 4 of 128: 1.26 ms of the backward's 2.45.  (16 softmax
// warps of 32 rows: a twentieth less at D = 64, the same at 128, and short sequences pay for the threads.)
// Where there are too few (sequence, head, key tile) for the GPU, the row tiles of one are dealt to several CTAs, whose fp32
// parts are added in their order.
#include "prompt_tc.cuh"

namespace triattn {
namespace prompt {

namespace {

struct DkvParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;
    PromptParams p;
    Tiles t;
    int splits;                // CTAs of a key tile
    uint32_t idesc_s, idesc_g;
    int ksteps;                // D / 16, rounded up
    float scale_log2e;
};

constexpr int kWarps = 12;
constexpr int kQStages = 3;    // (a tile of Q stays until dK: with two stages the next but one came too late)

template <int NB>
struct Smem {
    static constexpr uint32_t kTile = NB * kBox;
    static constexpr uint32_t kK = 0, kV = kTile, kQ = 2 * kTile, kDO = kQ + kQStages * kTile;
    static constexpr uint32_t kRows = kDO + 2 * kTile;                 // [2 stages][-lse log2 e, delta][128]
    static constexpr uint32_t kBars = kRows + 2 * 2 * 128 * 4;
    static constexpr int kNumBars = 1 + 2 * kQStages + 2 * 2 + 2 * 2 + 5;
    static constexpr uint32_t kSlot = kBars + 8 * kNumBars, kAbort = kSlot + 4, kTotal = kAbort + 4;
};
static_assert(Smem<2>::kTotal <= kMaxDynamicSmem, "shared memory");

// Where a CTA's part of dK (0) or dV (1) begins: keys from row `key` on of split `split`.
__device__ __forceinline__ float* part(const PromptParams& p, int split, int which, long long key, int h) {
    return p.parts + (((long long)split * 2 + which) * p.total_k + key) * p.Hk * p.D + (long long)h * p.D;
}

template <bool BF16, int NB>
__global__ void __launch_bounds__(kWarps * 32, 1) prompt_dkv_kernel(const __grid_constant__ DkvParams P) {
    using M = Smem<NB>;
    constexpr uint32_t kTile = M::kTile;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* g0 = smem_raw;
    const uint32_t base = smem_u32(smem_raw);
    const PromptParams& p = P.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    // ---- The CTA's work: key tile slowest, as the first of a sequence is seen by most rows.
    const unsigned per = (unsigned)p.num_seqs * (unsigned)p.Hk * (unsigned)P.splits;
    const int kt = (int)(blockIdx.x / per);
    unsigned rest = blockIdx.x % per;
    const int split = (int)(rest % (unsigned)P.splits);
    rest /= (unsigned)P.splits;
    const int h = (int)(rest % (unsigned)p.Hk), seq = (int)(rest / (unsigned)p.Hk);
    const Seq q = load_seq(p, seq, threadIdx.x == 0 && kt == 0 && h == 0 && split == 0);
    const int k0 = 128 * kt;
    if (k0 >= q.lk) return;
    const int keys = min(128, q.lk - k0);                               // that exist
    const int blocks = (q.lq + P.t.tq - 1) / P.t.tq;
    const int first = max(0, k0 - q.shift) / P.t.tq * P.t.ng + split;       // the first tile with a row that sees the key k0
    const int n = first < blocks * P.t.ng ? (blocks * P.t.ng - first + P.splits - 1) / P.splits : 0;
    uint16_t* dk = static_cast<uint16_t*>(p.dk) + ((long long)(q.k0 + k0) * p.Hk + h) * p.D;
    uint16_t* dv = static_cast<uint16_t*>(p.dv) + ((long long)(q.k0 + k0) * p.Hk + h) * p.D;
    if (n == 0) {  // no row for this CTA: zeros
        const int pieces = p.D / 8;
        for (int e = threadIdx.x; e < keys * pieces; e += kWarps * 32) {
            const int k = e / pieces, d = (e % pieces) * 8;
            if (P.splits == 1) {
                *reinterpret_cast<uint4*>(dk + (long long)k * p.Hk * p.D + d) = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(dv + (long long)k * p.Hk * p.D + d) = make_uint4(0u, 0u, 0u, 0u);
            } else {
                for (int w = 0; w < 2; ++w) {
                    float4* to = reinterpret_cast<float4*>(part(p, split, w, q.k0 + k0 + k, h) + d);
                    to[0] = to[1] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
        }
        return;
    }
    // fp16: the exponents by which P and dS are held (prompt_tc.cuh).
    constexpr int kP = BF16 ? 0 : kHalfP;
    int ds_exp = 0;
    if constexpr (!BF16) {
        const float* most = p.most + ((long long)seq * p.Hk + h) * 3;
        ds_exp = half_exponent(fmaf(most[0], most[1], most[2]));
    }
    // The tiles of the walk whose rows see up to kFineKeys keys.
    const int fine_blocks = min(blocks, max(0, kFineKeys - q.shift) / P.t.tq) * P.t.ng;
    const int fine = max(0, (fine_blocks - first + P.splits - 1) / P.splits);
    // Tile j of the walk: its first token, first query head and rows.
    auto tile = [&](int j, int& tok, int& head, int& rows) {
        const int t = first + j * P.splits, b = P.t.ng == 1 ? t : t / P.t.ng;
        tok = b * P.t.tq;
        head = h * p.G + (t - b * P.t.ng) * P.t.hp;
        rows = min(P.t.tq, q.lq - tok) * P.t.hp;
    };

    volatile int* abort_flag = reinterpret_cast<volatile int*>(g0 + M::kAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(g0 + M::kSlot);
    float* row_s = reinterpret_cast<float*>(g0 + M::kRows);
    auto bar = [&](int i) { return base + M::kBars + 8u * (uint32_t)i; };
    const uint32_t kv_full = bar(0);
    auto q_full = [&](int s) { return bar(1 + s); };
    auto q_empty = [&](int s) { return bar(1 + kQStages + s); };
    constexpr int b0 = 1 + 2 * kQStages;
    auto do_full = [&](int s) { return bar(b0 + s); };
    auto do_empty = [&](int s) { return bar(b0 + 2 + s); };
    auto row_full = [&](int s) { return bar(b0 + 4 + s); };
    auto row_empty = [&](int s) { return bar(b0 + 6 + s); };
    const uint32_t s_full = bar(b0 + 8), p_full = bar(b0 + 9), dp_full = bar(b0 + 10), ds_full = bar(b0 + 11), fin = bar(b0 + 12);
    static_assert(b0 + 13 == M::kNumBars, "barriers");
    auto q_smem = [&](int s) { return base + M::kQ + (uint32_t)s * kTile; };
    auto do_smem = [&](int s) { return base + M::kDO + (uint32_t)s * kTile; };
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(kv_full, 1);
#pragma unroll 1
        for (int s = 0; s < kQStages; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
        }
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
            mbar_init(do_full(s), 1);
            mbar_init(do_empty(s), 1);
            mbar_init(row_full(s), 1);
            mbar_init(row_empty(s), 8);
        }
        mbar_init(s_full, 1);
        mbar_init(p_full, 8);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tDP = tmem + 128, tDV = tmem + 256, tDK = tmem + 256 + NB * 64;
    bool ok = true;

    if (warp == 9) {
        // -------------------------------------------------------- TMA
        if (lane == 0) {
            mbar_expect_tx(kv_full, 2 * kTile);
            for (int b = 0; b < NB; ++b) {
                tma_load_3d(base + M::kK + b * kBox, &P.tm_k, 64 * b, h, q.k0 + k0, kv_full);
                tma_load_3d(base + M::kV + b * kBox, &P.tm_v, 64 * b, h, q.k0 + k0, kv_full);
            }
        }
        StageRing qr = {0, 0u, false};
        for (int j = 0; j < n && ok; ++j) {
            int tok, head, rows;
            tile(j, tok, head, rows);
            const int s = j & 1;
            const uint32_t before = (uint32_t)(j / 2 - 1) & 1u;
            if (qr.wrapped) ok = __all_sync(0xffffffffu, wait(q_empty(qr.idx), qr.ph ^ 1u, abort_flag, p.status));
            if (ok && lane == 0) {
                mbar_expect_tx(q_full(qr.idx), kTile);
                for (int b = 0; b < NB; ++b)
                    tma_load_3d(q_smem(qr.idx) + b * kBox, &P.tm_q, 64 * b, head, q.q0 + tok, q_full(qr.idx));
            }
            qr.next(kQStages);
            if (j >= 2 && ok) ok = __all_sync(0xffffffffu, wait(do_empty(s), before, abort_flag, p.status));
            if (ok && lane == 0) {
                mbar_expect_tx(do_full(s), kTile);
                for (int b = 0; b < NB; ++b) tma_load_3d(do_smem(s) + b * kBox, &P.tm_do, 64 * b, head, q.q0 + tok, do_full(s));
            }
        }
        if (!ok) *abort_flag = 1;
    } else if (warp == 10) {
        // -------------------------------------------------------- the rows' factors
        for (int j = 0; j < n && ok; ++j) {
            int tok, head, rows;
            tile(j, tok, head, rows);
            const int s = j & 1;
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 32 * i + lane, t = (int)P.t.fd_hp.div((uint32_t)r);
                const long long at = (long long)(head + r - t * P.t.hp) * p.total_q + q.q0 + tok + t;
                a[i] = r < rows ? p.lse[at] : 0.f;
                b[i] = r < rows ? p.delta[at] : 0.f;
            }
            if (j >= 2) ok = __all_sync(0xffffffffu, wait(row_empty(s), (uint32_t)(j / 2 - 1) & 1u, abort_flag, p.status));
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                row_s[s * 256 + 32 * i + lane] = fmaf(-a[i], tc::kLog2e, (float)kP);
                row_s[s * 256 + 128 + 32 * i + lane] = BF16 ? -b[i] : -b[i] * pow2(ds_exp - kP);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(row_full(s));
        }
        if (!ok) *abort_flag = 1;
    } else if (warp == 8) {
        // ------------------------------------------------------------ MMA
        // One thread runs the loop; the others help where a tile ends with rows that are not the sequence's: they are
        // another's, or nobody's, and are zeroed up to the next 16, which dV and dK multiply with zeros.
        const bool leader = elect_one();
        const int lead = __ffs((int)__ballot_sync(0xffffffffu, leader)) - 1;
        const int last_from = (blocks - 1) * P.t.ng, last_rows = min(P.t.tq, q.lq - (blocks - 1) * P.t.tq) * P.t.hp;
        auto rows_of = [&](int j) { return first + j * P.splits < last_from ? 128 : last_rows; };
        auto await = [&](uint32_t b, uint32_t parity) {
            if (ok) ok = wait(b, parity, abort_flag, p.status);
            tc_fence_after();
        };
        const int whole = max(0, (last_from - first + P.splits - 1) / P.splits);  // tiles before the last block's
        StageRing qs = {0, 0u, false}, qk = {0, 0u, false};  // Q for S, Q for dK
        // Whole tiles, without a question (a few dozen instructions of one thread are a product's time; by all sixteens of
        // columns, or by as many as there are).
        auto straight = [&](auto all, int& u) {
            constexpr bool kAll = decltype(all)::value == 1;
            for (; u > 0 && (u & 3) == 0 && u / 4 + 1 < whole; u += 4) {
                const uint32_t ph = (uint32_t)(u >> 2) & 1u, to = (uint32_t)(u >> 3);  // (tile j = u / 4's parity; dO(j + 1)'s below)
                const int s = (int)ph;
                await(p_full, ph);
                if (!ok) break;
                issue_cols<64>(tDV, tS, desc_lo(do_smem(s), kBox), P.idesc_g, 0, 8, 8, false);
                mma_commit(do_empty(s));
                await(q_full(qs.idx), qs.ph);
                if (!ok) break;
                issue_rows<NB>(tS, desc_lo(base + M::kK, 16), desc_lo(q_smem(qs.idx), 16), P.idesc_s, kAll ? 4 * NB : P.ksteps);
                mma_commit(s_full);
                qs.next(kQStages);
                await(ds_full, ph);
                if (!ok) break;
                issue_cols<64>(tDK, tDP, desc_lo(q_smem(qk.idx), kBox), P.idesc_g, 0, 8, 8, false);
                if (u / 4 < fine) issue_cols<64>(tDK, tDP + 32u, desc_lo(q_smem(qk.idx), kBox), P.idesc_g, 0, 8, 8, false);
                mma_commit(q_empty(qk.idx));
                qk.next(kQStages);
                await(do_full(s ^ 1), (to + ph) & 1u);
                if (!ok) break;
                issue_rows<NB>(tDP, desc_lo(base + M::kV, 16), desc_lo(do_smem(s ^ 1), 16), P.idesc_s, kAll ? 4 * NB : P.ksteps);
                mma_commit(dp_full);
            }
        };
        bool clean = false;
        for (int u = -2;;) {  // S(0), dP(0); then for each j: dV(j), S(j + 1), dK(j), dP(j + 1)
            int tail = 0;
            uint32_t tail_at = 0;
            if (leader) {
                if (u == -2 && !clean) await(kv_full, 0);
                while (ok && u < 4 * n) {
                    if (P.ksteps == 4 * NB) straight(Count<1>(), u);
                    else straight(Count<0>(), u);
                    if (!ok || u >= 4 * n) break;
                    const bool odd = u & 1, second = u < 0 ? odd : (u & 2) != 0;   // S or dP; and dP or dK
                    const int j = u < 0 ? 0 : u / 4 + (odd ? 1 : 0), s = j & 1;
                    if (u < 0 || odd) {
                        if (j < n) {
                            const uint32_t at = second ? do_smem(s) : q_smem(qs.idx);
                            if (!clean) {
                                await(second ? do_full(s) : q_full(qs.idx), second ? (uint32_t)(j / 2) & 1u : qs.ph);
                                const int rows = rows_of(j);
                                if (ok && rows < 128 && rows % 16) {
                                    tail = rows;
                                    tail_at = at;
                                    clean = true;
                                    break;
                                }
                            }
                            clean = false;
                            if (!ok) break;
                            issue_rows<NB>(second ? tDP : tS, desc_lo(base + (second ? M::kV : M::kK), 16), desc_lo(at, 16), P.idesc_s,
                                           P.ksteps);
                            mma_commit(second ? dp_full : s_full);
                            if (!second) qs.next(kQStages);
                        }
                    } else {
                        await(second ? ds_full : p_full, (uint32_t)j & 1u);
                        if (!ok) break;
                        // (the rows of the second half: 64 columns on)
                        const uint32_t b = desc_lo(second ? q_smem(qk.idx) : do_smem(s), kBox);
                        const int sixteens = (rows_of(j) + 15) / 16;
                        issue_cols<64>(second ? tDK : tDV, second ? tDP : tS, b, P.idesc_g, 0, 8, sixteens, j == 0);
                        if (second && j < fine) issue_cols<64>(tDK, tDP + 32u, b, P.idesc_g, 0, 8, sixteens, false);
                        mma_commit(second ? q_empty(qk.idx) : do_empty(s));
                        if (second) qk.next(kQStages);
                    }
                    ++u;
                }
            }
            tail = __shfl_sync(0xffffffffu, tail, lead);
            if (tail == 0) break;
            clear_rows<NB>(__shfl_sync(0xffffffffu, tail_at, lead), tail, (tail + 15) & ~15);
        }
        if (!ok && leader) *abort_flag = 1;
        if (leader) mma_commit(fin);
        wait_bar_drain(fin, 0);
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ P and dS
        const int half = warp / 4, kr = warp % 4 * 32 + lane;          // rows [64 half, + 64) of a tile; key
        const uint32_t lane_off = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t sA = tS + lane_off + 64u * half, dpA = tDP + lane_off + 64u * half;
        const float f = P.scale_log2e;
        [[maybe_unused]] const float2 ds2 = make_float2(pow2(ds_exp - kP), pow2(ds_exp - kP));
        auto less_delta = [&](uint32_t x, uint32_t y, float2 d) {  // (d: -delta as it is held)
            const float2 v = make_float2(__uint_as_float(x), __uint_as_float(y));
            return BF16 ? __fadd2_rn(v, d) : __ffma2_rn(v, ds2, d);
        };
        for (int j = 0; j < n && ok; ++j) {
            const uint32_t ph = (uint32_t)j & 1u;
            const int s = j & 1;
            int tok, head, rows;
            tile(j, tok, head, rows);
            const bool edge = rows < 128 || keys < 128 || k0 + 127 > tok + q.shift;
            uint32_t see[2] = {0xffffffffu, 0xffffffffu};
            if (edge) {
                // the rows that see this key: from `from` on, of those that exist
                const long long from = (long long)(k0 + kr - q.shift - tok) * P.t.hp;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c0 = 64 * half + 32 * i;
                    const int lo = from <= c0 ? 0 : from >= c0 + 32 ? 32 : (int)from - c0;
                    see[i] = kr < keys ? low_bits(rows - c0) & ~low_bits(lo) : 0u;
                }
            }
            const float4* nl = reinterpret_cast<const float4*>(row_s + s * 256 + 64 * half);
            const float4* nd = nl + 32;
            ok = __all_sync(0xffffffffu, wait(row_full(s), (uint32_t)(j / 2) & 1u, abort_flag, p.status) &&
                                             wait(s_full, ph, abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
            float pr[64];
            {
                uint32_t sr[64];
                tmem_ld_x64(sA, sr);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float4 l = nl[c];
                    const float2 a = __ffma2_rn(make_float2(__uint_as_float(sr[4 * c]), __uint_as_float(sr[4 * c + 1])),
                                                make_float2(f, f), make_float2(l.x, l.y));
                    const float2 b = __ffma2_rn(make_float2(__uint_as_float(sr[4 * c + 2]), __uint_as_float(sr[4 * c + 3])),
                                                make_float2(f, f), make_float2(l.z, l.w));
                    pr[4 * c] = ex2(a.x);
                    pr[4 * c + 1] = ex2(a.y);
                    pr[4 * c + 2] = ex2(b.x);
                    pr[4 * c + 3] = ex2(b.y);
                }
            }
            if (edge) {
#pragma unroll
                for (int c = 0; c < 64; ++c) pr[c] = (see[c / 32] >> (c % 32)) & 1u ? pr[c] : 0.f;
            }
            {
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) pk[c] = pack2<BF16>(pr[2 * c], pr[2 * c + 1]);
                tmem_st_x32(sA, pk);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            ok = __all_sync(0xffffffffu, wait(dp_full, ph, abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
            auto form = [&](auto pieces) {
                constexpr bool kFine = decltype(pieces)::value == 2;
                uint32_t pk[32], low[kFine ? 32 : 1];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t dr[32];
                    tmem_ld_x32(dpA + 32 * i, dr);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 d = nd[8 * i + c / 4];
                        const int pa = 32 * i + c;
                        float2 u = less_delta(dr[c], dr[c + 1], make_float2(d.x, d.y));
                        float2 v = less_delta(dr[c + 2], dr[c + 3], make_float2(d.z, d.w));
                        u = __fmul2_rn(u, make_float2(pr[pa], pr[pa + 1]));
                        v = __fmul2_rn(v, make_float2(pr[pa + 2], pr[pa + 3]));
                        if (edge) {  // (dP and delta of a row that is not there may be anything)
                            u.x = (see[i] >> c) & 1u ? u.x : 0.f;
                            u.y = (see[i] >> (c + 1)) & 1u ? u.y : 0.f;
                            v.x = (see[i] >> (c + 2)) & 1u ? v.x : 0.f;
                            v.y = (see[i] >> (c + 3)) & 1u ? v.y : 0.f;
                        }
                        pk[pa / 2] = pack2<BF16>(u.x, u.y);
                        pk[pa / 2 + 1] = pack2<BF16>(v.x, v.y);
                        if constexpr (kFine) {
                            low[pa / 2] = rest2<BF16>(u, pk[pa / 2]);
                            low[pa / 2 + 1] = rest2<BF16>(v, pk[pa / 2 + 1]);
                        }
                    }
                }
                tmem_st_x32(dpA, pk);
                if constexpr (kFine) tmem_st_x32(dpA + 32, low);
            };
            if (__builtin_expect(j >= fine, 1)) form(Count<1>());
            else form(Count<2>());
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(ds_full);
                mbar_arrive(row_empty(s));
            }
        }
        // ---- dV (warps 0-3) and dK (4-7), when every product is done.
        if (ok) ok = __all_sync(0xffffffffu, wait(fin, 0, abort_flag, p.status));
        if (ok && !*abort_flag) {
            tc_fence_after();
            const uint32_t from = (half ? tDK : tDV) + lane_off;
            const float by = half ? p.scale * pow2(-ds_exp) : pow2(-kP);
            uint16_t* to = (half ? dk : dv) + (long long)kr * p.Hk * p.D;
            float* acc = P.splits > 1 ? part(p, split, half ? 0 : 1, q.k0 + k0 + kr, h) : nullptr;
#pragma unroll 1
            for (int c = 0; c < p.D; c += 16) {
                uint32_t o[16];
                tmem_ld_x16(from + c, o);
                if (kr >= keys) continue;
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    if (c + e >= p.D) break;
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[e + k]) * by;
                    if (acc) {
                        *reinterpret_cast<float4*>(acc + c + e) = make_float4(x[0], x[1], x[2], x[3]);
                        *reinterpret_cast<float4*>(acc + c + e + 4) = make_float4(x[4], x[5], x[6], x[7]);
                    } else {
                        *reinterpret_cast<uint4*>(to + c + e) = make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]),
                                                                           pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
                    }
                }
            }
        }
        if (!ok) *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// The CTAs' parts of a (sequence, key head, 128 keys), added in their order.  (Eight CTAs for each of them, four pieces of 32
// bytes and their parts a thread: there are few such where parts are made; 3507 tokens, 8 heads over 2 of 128:
// 32 us with one CTA for each, 7 so.)
constexpr int kJoin = 8;
template <bool BF16>
__global__ void __launch_bounds__(256) prompt_dkv_join(const PromptParams p, int splits) {
    const unsigned per = (unsigned)p.num_seqs * (unsigned)p.Hk;
    const int k0 = 128 * (int)(blockIdx.x / per), h = (int)(blockIdx.x % per % (unsigned)p.Hk);
    const Seq q = load_seq(p, (int)(blockIdx.x % per / (unsigned)p.Hk), false);
    const int keys = min(128, q.lk - k0), pieces = p.D / 8;
    for (int e = (int)blockIdx.y * 256 + threadIdx.x; e < 2 * keys * pieces; e += 256 * kJoin) {
        const int which = e >= keys * pieces, x = which ? e - keys * pieces : e, k = x / pieces, d = (x - k * pieces) * 8;
        const long long key = q.k0 + k0 + k;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
        for (int i = 0; i < splits; ++i) {
            const float4* from = reinterpret_cast<const float4*>(part(p, i, which, key, h) + d);
            const float4 u = from[0], v = from[1];
            a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
            b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
        }
        uint16_t* to = static_cast<uint16_t*>(which ? p.dv : p.dk) + (key * p.Hk + h) * p.D + d;
        *reinterpret_cast<uint4*>(to) =
            make_uint4(pack2<BF16>(a.x, a.y), pack2<BF16>(a.z, a.w), pack2<BF16>(b.x, b.y), pack2<BF16>(b.z, b.w));
    }
}

template <bool BF16, int NB>
cudaError_t start(const DkvParams& P, unsigned grid, cudaStream_t stream) {
    const cudaError_t e = allow_smem<prompt_dkv_kernel<BF16, NB>>(Smem<NB>::kTotal);
    if (e != cudaSuccess) return e;
    prompt_dkv_kernel<BF16, NB><<<grid, kWarps * 32, Smem<NB>::kTotal, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dq(const PromptParams& p, cudaStream_t stream);     // prompt_dq.cu
cudaError_t launch_delta(const PromptParams& p, cudaStream_t stream);  // prompt_simt.cu

}  // namespace prompt

// CTAs of a key tile: one, or as many as give the GPU's 152 SMs two each where there are few (sequence, head, key tile), but
// four row tiles for each at least.
int prompt_bwd_splits(int num_seqs, int total_k, int max_q, int max_k, int Hk, int G) {
    const long long a = (long long)num_seqs * ((max_k + 127) / 128), b = (long long)total_k / 128 + num_seqs;
    const long long ctas = (a < b ? a : b) * Hk, tiles = ((long long)max_q * G + 127) / 128;
    if (ctas <= 0 || ctas >= 304) return 1;
    long long s = (304 + ctas - 1) / ctas;
    if (s > tiles / 4) s = tiles / 4;
    return s < 1 ? 1 : (int)(s > 32 ? 32 : s);
}

cudaError_t launch_prompt_tc_bwd(const PromptParams& p, cudaStream_t stream) {
    using namespace prompt;
    const bool rows = p.total_q > 0 && p.max_q > 0;
    cudaError_t e = rows ? launch_delta(p, stream) : cudaSuccess;
    if (e == cudaSuccess && rows) e = launch_dq(p, stream);
    if (e != cudaSuccess || p.max_k <= 0) return e;
    DkvParams P;
    P.p = p;
    P.t = make_tiles(p);
    P.splits = p.parts ? prompt_bwd_splits(p.num_seqs, p.total_k, p.max_q, p.max_k, p.Hk, p.G) : 1;
    const bool bf16 = p.dtype == TA_BF16;
    P.idesc_s = make_idesc(bf16, 128, 0, 0);
    P.idesc_g = make_idesc(bf16, (uint32_t)(p.D + 15) / 16 * 16, 0, 1);
    P.ksteps = (p.D + 15) / 16;
    P.scale_log2e = p.scale * kToLog2;
    const long long tiles = (long long)p.num_seqs * p.Hk * ((p.max_k + 127) / 128), grid = tiles * P.splits;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (!make_rows_map(&P.tm_q, bf16, p.q, p.D, p.Hq, p.total_q, p.q_rs, P.t.hp, P.t.tq) ||
        !make_rows_map(&P.tm_do, bf16, p.d_out, p.D, p.Hq, p.total_q, (long long)p.Hq * p.D, P.t.hp, P.t.tq) ||
        !make_rows_map(&P.tm_k, bf16, p.k, p.D, p.Hk, p.total_k, p.k_rs, 1, 128) ||
        !make_rows_map(&P.tm_v, bf16, p.v, p.D, p.Hk, p.total_k, p.v_rs, 1, 128))
        return cudaErrorInvalidValue;
    if (p.D <= 64) e = bf16 ? start<true, 1>(P, (unsigned)grid, stream) : start<false, 1>(P, (unsigned)grid, stream);
    else e = bf16 ? start<true, 2>(P, (unsigned)grid, stream) : start<false, 2>(P, (unsigned)grid, stream);
    if (e != cudaSuccess || P.splits == 1) return e;
    if (bf16) prompt_dkv_join<true><<<dim3((unsigned)tiles, kJoin), 256, 0, stream>>>(p, P.splits);
    else prompt_dkv_join<false><<<dim3((unsigned)tiles, kJoin), 256, 0, stream>>>(p, P.splits);
    return cudaGetLastError();
}

}  // namespace triattn
