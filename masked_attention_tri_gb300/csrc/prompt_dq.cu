// prompt_dq.cu -- the gradient of the queries in the causal attention of packed prompts with grouped heads on tcgen05 tensor
// cores: 16-bit inputs, D <= 128.
//
// A tile of rows (prompt_tc.cuh) walks the key tiles that it sees, as in the forward, with P = 2^(s - lse) recomputed:
//     S = Q K^T, dP = dO V^T             rows on the tensor-memory lanes
//     dS = P (dP - delta)                as 16-bit pairs over dP (fp16: times a power of two, prompt_tc.cuh)
//     dQ += dS K                         dS from tensor memory
// lse and delta = dO . O (one pass of its own before: half a row a thread at the start of an item was 5 us of each) are one
// number a thread, dQ stays in tensor memory, and is rounded once: no sum in memory, no order that varies.
// dS goes to the products as one 16-bit number, which adds as much to the gradient's error as its own rounding does, but as
// two (the rounding's rest is the second, and one product more) in rows that see up to kFineKeys keys: P spreads over the
// keys, so those rows carry most of the gradients' norms.  bf16, prompts of 777 to 8192 tokens: off by 0.0018 of dQ's norm
// with two everywhere, 0.0022 so, 0.0025 with one, 0.0017 by the rounding alone; the backward takes 864, 801 and 775 us.
// (One kernel for dQ, dK and dV computes S and dP once, five products a tile where the two kernels have seven; but its dQ has
// to be added up in memory over the key tiles and stands between the tiles' products, and four 128 x 128 x D products a tile
// from shared memory are more than that gives: four sequences of 8192 tokens, 16 heads over 4 of 128, 3.86 ms, of which 0.5 ms
// were the reductions.)
//
// One CTA a SM, 12 warps: 0-7 softmax and dS (a row's two halves of 64 keys each), 8 MMA, 9 TMA, 10 the items.  Tensor
// memory: S, dP twice (dS over it), dQ: 4 x 128 columns at D = 128.  The tensor core's order is dQ(i - 2), S(i), dP(i): S(i)
// follows as soon as S(i - 1) is in registers, and both are there when dS(i - 1) is done, across items too.
//
// Bound: shared memory, 1792 clocks a tile at D = 128 (160 KB of operands, 64 KB of loads), the tensor core 1536, the softmax
// warps' two phases 1500 and more; a tile takes some 1900.  Four sequences of 8192 tokens, 16 heads over 4 of 128: 0.94 ms.
#include "prompt_tc.cuh"

namespace triattn {
namespace prompt {
namespace {

struct DqParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;
    PromptParams p;
    Tiles t;
    uint32_t idesc_s, idesc_q;
    int ksteps;                // D / 16, rounded up
    float scale_log2e;
};

constexpr int kRing = 2, kWarps = 12, kConsumers = 10;
constexpr int kKStages = 3, kVStages = 2;

template <int NB>
struct Smem {
    static constexpr uint32_t kTile = NB * kBox;
    static constexpr uint32_t kQ = 0, kDO = kTile, kK = 2 * kTile, kV = kK + kKStages * kTile;
    static constexpr uint32_t kItems = kV + kVStages * kTile, kClc = kItems + kRing * sizeof(Item<1>), kBars = kClc + 16;
    static constexpr int kNumBars = 4 + 2 * kKStages + 2 * kVStages + 8 + 2 * kRing + 2;
    static constexpr uint32_t kSlot = kBars + 8 * kNumBars, kAbort = kSlot + 4, kTotal = kAbort + 4;
};
static_assert(Smem<2>::kTotal <= kMaxDynamicSmem, "shared memory");

template <bool BF16, int NB>
__global__ void __launch_bounds__(kWarps * 32, 1) prompt_dq_kernel(const __grid_constant__ DqParams P) {
    using M = Smem<NB>;
    constexpr uint32_t kTile = M::kTile;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* g0 = smem_raw;
    const uint32_t base = smem_u32(smem_raw);
    const PromptParams& p = P.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(g0 + M::kAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(g0 + M::kSlot);
    Item<1>* items = reinterpret_cast<Item<1>*>(g0 + M::kItems);
    auto bar = [&](int i) { return base + M::kBars + 8u * (uint32_t)i; };
    const uint32_t q_full = bar(0), q_empty = bar(1), do_full = bar(2), do_empty = bar(3);
    auto k_full = [&](int s) { return bar(4 + s); };
    auto k_empty = [&](int s) { return bar(4 + kKStages + s); };
    constexpr int b0 = 4 + 2 * kKStages;
    auto v_full = [&](int s) { return bar(b0 + s); };
    auto v_empty = [&](int s) { return bar(b0 + kVStages + s); };
    constexpr int b1 = b0 + 2 * kVStages;
    const uint32_t s_full = bar(b1), s_read = bar(b1 + 1);
    auto dp_full = [&](uint32_t b) { return bar(b1 + 2 + (int)b); };
    auto ds_full = [&](uint32_t b) { return bar(b1 + 4 + (int)b); };
    const uint32_t dq_full = bar(b1 + 6), dq_empty = bar(b1 + 7);
    auto it_full = [&](int r) { return bar(b1 + 8 + r); };
    auto it_empty = [&](int r) { return bar(b1 + 8 + kRing + r); };
    const uint32_t clc = bar(b1 + 8 + 2 * kRing), drain = bar(b1 + 9 + 2 * kRing);
    static_assert(b1 + 10 + 2 * kRing == M::kNumBars, "barriers");
    auto k_smem = [&](int s) { return base + M::kK + (uint32_t)s * kTile; };
    auto v_smem = [&](int s) { return base + M::kV + (uint32_t)s * kTile; };

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(do_full, 1);
        mbar_init(do_empty, 1);
#pragma unroll 1
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(k_empty(s), 1);
        }
#pragma unroll 1
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(v_full(s), 1);
            mbar_init(v_empty(s), 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_read, 8);
#pragma unroll 1
        for (uint32_t b = 0; b < 2; ++b) {
            mbar_init(dp_full(b), 1);
            mbar_init(ds_full(b), 8);
        }
        mbar_init(dq_full, 1);
        mbar_init(dq_empty, 8);
        for (int r = 0; r < kRing; ++r) {
            mbar_init(it_full(r), 1);
            mbar_init(it_empty(r), kConsumers);
        }
        mbar_init(clc, 1);
        mbar_init(drain, 1);
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
    const uint32_t tmem = *tmem_slot, tDP = tmem + 128, tDQ = tmem + 384;  // S, dP and dS twice, dQ
    bool ok = true;
    int item_n = 0;
    auto next_item = [&](Item<1>& it) -> bool {
        const int r = item_n % kRing;
        ok = __all_sync(0xffffffffu, wait(it_full(r), (uint32_t)(item_n / kRing) & 1u, abort_flag, p.status));
        if (!ok) return false;
        it = items[r];
        __syncwarp();
        if (lane == 0) mbar_arrive(it_empty(r));
        ++item_n;
        return it.on != 0;
    };

    if (warp == 10) {
        // ------------------------------------------------------------ the items
        ok = hand_out<1, kRing>(p, P.t, items, it_full, it_empty, base + M::kClc, clc, abort_flag);
        if (!ok) *abort_flag = 1;
    } else if (warp == 9) {
        // ------------------------------------------------------------ TMA
        StageRing kr = {0, 0u, false}, vr = {0, 0u, false};
        Item<1> it;
        uint32_t q_use = 0;
        while (ok && next_item(it)) {
            const int n = (it.keys[0] + 127) / 128;
            if (n == 0) continue;
            // Q (false) or dO of the item's rows, when the last item's are read
            auto load_rows = [&](bool d_o) {
                const uint32_t full = d_o ? do_full : q_full;
                if (ok && q_use > 0) ok = __all_sync(0xffffffffu, wait(d_o ? do_empty : q_empty, (q_use - 1u) & 1u, abort_flag, p.status));
                if (ok && lane == 0) {
                    mbar_expect_tx(full, kTile);
                    for (int b = 0; b < NB; ++b)
                        tma_load_3d(base + (d_o ? M::kDO : M::kQ) + b * kBox, d_o ? &P.tm_do : &P.tm_q, 64 * b, it.head[0],
                                    it.q0 + it.tok[0], full);
                }
            };
            auto load = [&](StageRing& r, int stages, bool v, int j) {
                const uint32_t full = v ? v_full(r.idx) : k_full(r.idx);
                if (ok && r.wrapped)
                    ok = __all_sync(0xffffffffu, wait(v ? v_empty(r.idx) : k_empty(r.idx), r.ph ^ 1u, abort_flag, p.status));
                if (ok && lane == 0) {
                    mbar_expect_tx(full, kTile);
                    for (int b = 0; b < NB; ++b)
                        tma_load_3d((v ? v_smem(r.idx) : k_smem(r.idx)) + b * kBox, v ? &P.tm_v : &P.tm_k, 64 * b, it.h,
                                    it.k0 + 128 * j, full);
                }
                r.next(stages);
            };
            load(kr, kKStages, false, 0);
            load_rows(false);
            load_rows(true);
            ++q_use;
            for (int j = 0; j < n && ok; ++j) {
                if (j > 0) load(kr, kKStages, false, j);
                load(vr, kVStages, true, j);
            }
        }
        if (!ok) *abort_flag = 1;
    } else if (warp == 8) {
        // ------------------------------------------------------------ MMA
        // One thread runs the loop; the others help where a tile of K ends with rows that are not the sequence's (dQ multiplies
        // their zeros with them, sixteen keys at a time).
        const bool leader = elect_one();
        const int lead = __ffs((int)__ballot_sync(0xffffffffu, leader)) - 1;
        StageRing ks = {0, 0u, false}, kq = {0, 0u, false}, vr = {0, 0u, false};  // K for S, K for dQ, V
        auto await = [&](uint32_t b, uint32_t parity) {
            if (ok) ok = wait(b, parity, abort_flag, p.status);
            tc_fence_after();
        };
        auto fetch = [&](int& keys, int& lk) -> bool {  // the next item
            const int r = item_n % kRing;
            await(it_full(r), (uint32_t)(item_n / kRing) & 1u);
            if (!ok) return false;
            const bool on = items[r].on != 0;
            keys = items[r].keys[0];
            lk = items[r].lq + items[r].shift;
            mbar_arrive(it_empty(r));
            ++item_n;
            return on;
        };
        // dQ of tile u (of all that the CTA walks), whose dS is in buffer u % 2
        auto dq_mma = [&](uint32_t u, int steps, bool fresh, bool fine) {
            const uint32_t a = tDP + (u & 1u) * 128u, b = desc_lo(k_smem(kq.idx), kBox);
            issue_cols<64>(tDQ, a, b, P.idesc_q, 0, 8, steps, fresh);
            if (fine) issue_cols<64>(tDQ, a + 32u, b, P.idesc_q, 0, 8, steps, false);
            mma_commit(k_empty(kq.idx));
            kq.next(kKStages);
        };
        // S of tile u, K there, and dP of it
        auto s_mma = [&](uint32_t u, uint32_t idesc, int ksteps) {
            if (u > 0) await(s_read, (u - 1u) & 1u);
            if (!ok) return;
            issue_rows<NB>(tmem, desc_lo(base + M::kQ, 16), desc_lo(k_smem(ks.idx), 16), idesc, ksteps);
            mma_commit(s_full);
            ks.next(kKStages);
        };
        auto dp_mma = [&](uint32_t u, uint32_t idesc, int ksteps) {
            await(v_full(vr.idx), vr.ph);
            if (!ok) return;
            issue_rows<NB>(tDP + (u & 1u) * 128u, desc_lo(base + M::kDO, 16), desc_lo(v_smem(vr.idx), 16), idesc, ksteps);
            mma_commit(dp_full(u & 1u));
            mma_commit(v_empty(vr.idx));
            vr.next(kVStages);
        };
        // Step u: dQ of tile u - 2, S and dP of tile u, which is tile j of an item.  Of the two tiles between: sixteens of
        // keys, 16 for an item's first, 32 for its last, 64 for two pieces of dS (0: no tile).
        int keys = 0, lk = 0, j = 0, one = 0, two = 0;
        uint32_t u = 0, items_in = 0, items_out = 0;
        bool there = true, ask = true, clean = false;
        auto finish = [&](int what, uint32_t v) {  // dQ of tile v
            await(ds_full(v & 1u), (v >> 1) & 1u);
            if ((what & 16) && items_out > 0) await(dq_empty, (items_out - 1u) & 1u);  // the last item's dQ is read
            if (!ok) return;
            dq_mma(v, what & 15, what & 16, what & 64);
            if (what & 32) {
                mma_commit(dq_full);
                ++items_out;
            }
        };
        // Whole key tiles in the middle of an item, without a question (a few dozen instructions of one thread are a
        // product's time; by all sixteens of columns, or by as many as there are).
        auto straight = [&](auto all) {
            constexpr bool kAll = decltype(all)::value == 1;
            for (const int whole = there && !ask ? keys : 0; j > 2 && two && 128 * (j + 1) < whole; ++j, ++u) {
                await(ds_full(u & 1u), ((u - 2u) >> 1) & 1u);
                if (!ok) break;
                dq_mma(u, 8, false, keys <= kFineKeys);
                await(k_full(ks.idx), ks.ph);
                if (!ok) break;
                s_mma(u, P.idesc_s | (16u << 17), kAll ? 4 * NB : P.ksteps);
                if (!ok) break;
                dp_mma(u, P.idesc_s | (16u << 17), kAll ? 4 * NB : P.ksteps);
            }
        };
        for (;;) {
            int tail = 0, tail_st = 0;
            if (leader) {
                while (ok) {
                    if (P.ksteps == 4 * NB) straight(Count<1>());
                    else straight(Count<0>());
                    if (!ok) break;
                    if (two) {
                        finish(two, u - 2u);
                        two = 0;
                    }
                    if (!ok) break;
                    if (ask) {
                        // The first item that has keys.  Past one without, the last dQ of the item before may wait no longer:
                        // the ring's third item from there waits for the warps that wait for it.
                        while ((there = fetch(keys, lk)) && keys <= 0) {
                            if (one) finish(one, u - 1u);
                            one = 0;
                            if (!ok) break;
                        }
                        if (!ok) break;
                        ask = false;
                        j = 0;
                        if (there) {
                            await(q_full, items_in & 1u);
                            ++items_in;
                        }
                        if (!ok) break;
                    }
                    if (!there) {
                        if (!one) break;
                        two = one;
                        one = 0;
                        ++u;
                        continue;
                    }
                    if (!clean) {
                        await(k_full(ks.idx), ks.ph);
                        if (!ok) break;
                        const int valid = lk - 128 * j;
                        if (valid < 128 && valid % 16) {
                            tail = valid;
                            tail_st = ks.idx;
                            clean = true;
                            break;
                        }
                    }
                    clean = false;
                    const int steps = min(8, (keys - 128 * j + 15) / 16);
                    const bool last = 128 * (j + 1) >= keys;
                    s_mma(u, P.idesc_s | ((uint32_t)(2 * steps) << 17), P.ksteps);
                    if (!ok) break;
                    if (last) mma_commit(q_empty);
                    if (j == 0) {
                        if (one) {  // (the last item's dQ first: this dO may be on its way yet)
                            finish(one, u - 1u);
                            one = 0;
                        }
                        await(do_full, (items_in - 1u) & 1u);
                    }
                    dp_mma(u, P.idesc_s | ((uint32_t)(2 * steps) << 17), P.ksteps);
                    if (!ok) break;
                    if (last) mma_commit(do_empty);
                    two = one;
                    one = steps | (j == 0 ? 16 : 0) | (last ? 32 : 0) | (keys <= kFineKeys ? 64 : 0);
                    ++u;
                    ++j;
                    ask = last;
                }
            }
            tail = __shfl_sync(0xffffffffu, tail, lead);
            if (tail == 0) break;
            clear_rows<NB>(k_smem(__shfl_sync(0xffffffffu, tail_st, lead)), tail, (tail + 15) & ~15);
        }
        if (!ok && leader) *abort_flag = 1;
        if (leader) mma_commit(drain);
        wait_bar_drain(drain, 0);
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ dS, and dQ to memory
        const int half = warp / 4, r = warp % 4 * 32 + lane;
        const uint32_t lane_off = (uint32_t)(warp % 4 * 32) << 16;
        const int tok_r = (int)P.t.fd_hp.div((uint32_t)r), head_r = r - tok_r * P.t.hp;
        const bool wide = p.D % 16 == 0 && (reinterpret_cast<uintptr_t>(p.dq) & 31) == 0;
        const float f = P.scale_log2e;
        Item<1> it;
        uint32_t g = 0, dq_use = 0;  // tiles so far
        while (ok && next_item(it)) {
            const int keys = it.keys[0], n = (keys + 127) / 128;
            const bool row = r < it.rows[0];
            const long long tok = it.q0 + it.tok[0] + tok_r, head = it.head[0] + head_r;
            const long long at = head * p.total_q + tok, row0 = (tok * p.Hq + head) * p.D;
            const int limit = it.tok[0] + tok_r + it.shift, first = it.tok[0] + it.shift;
            const float nl = row ? -p.lse[at] * tc::kLog2e : 0.f;
            float nd = row ? -p.delta[at] : 0.f, by = p.scale;
            [[maybe_unused]] float ds = 1.f;
            if constexpr (!BF16) {  // dS times a power of two (prompt_tc.cuh)
                const float most = p.most[((long long)it.seq * p.Hk + it.h) * 3];
                const int e = row ? half_exponent(fmaf(p.norm[at], most, fabsf(nd))) : 0;
                ds = pow2(e);
                nd *= ds;
                by *= pow2(-e);
            }
            for (int j = 0; j < n && ok; ++j, ++g) {
                const uint32_t b = g & 1u;
                const uint32_t sA = tmem + lane_off + 64u * half, dpA = tDP + lane_off + 128u * b + 64u * half;
                const bool edge = 128 * j + 127 > first;  // some row does not see every key
                uint32_t see[2] = {0xffffffffu, 0xffffffffu};
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) see[i] = low_bits(limit - 128 * j - 64 * half - 32 * i + 1);
                }
                ok = __all_sync(0xffffffffu, wait(s_full, g & 1u, abort_flag, p.status));
                if (!ok) break;
                tc_fence_after();
                float pr[64];
                {
                    uint32_t sr[64];
                    tmem_ld_x64(sA, sr);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_read);
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), make_float2(f, f),
                                                    make_float2(nl, nl));
                        pr[c] = ex2(y.x);
                        pr[c + 1] = ex2(y.y);
                    }
                }
                ok = __all_sync(0xffffffffu, wait(dp_full(b), (g >> 1) & 1u, abort_flag, p.status));
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
                        for (int c = 0; c < 32; c += 2) {
                            float2 x = make_float2(__uint_as_float(dr[c]), __uint_as_float(dr[c + 1]));
                            x = BF16 ? __fadd2_rn(x, make_float2(nd, nd)) : __ffma2_rn(x, make_float2(ds, ds), make_float2(nd, nd));
                            x = __fmul2_rn(x, make_float2(pr[32 * i + c], pr[32 * i + c + 1]));
                            if (edge) {
                                x.x = (see[i] >> c) & 1u ? x.x : 0.f;
                                x.y = (see[i] >> (c + 1)) & 1u ? x.y : 0.f;
                            }
                            const uint32_t hi = pack2<BF16>(x.x, x.y);
                            pk[16 * i + c / 2] = hi;
                            if constexpr (kFine) low[16 * i + c / 2] = rest2<BF16>(x, hi);
                        }
                    }
                    tmem_st_x32(dpA, pk);
                    if constexpr (kFine) tmem_st_x32(dpA + 32, low);
                };
                if (__builtin_expect(keys > kFineKeys, 1)) form(Count<1>());
                else form(Count<2>());
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full(b));
            }
            if (!ok) break;
            if (n > 0) {
                ok = __all_sync(0xffffffffu, wait(dq_full, dq_use & 1u, abort_flag, p.status));
                if (!ok) break;
                ++dq_use;
                tc_fence_after();
            }
            uint16_t* to = static_cast<uint16_t*>(p.dq) + row0;
#pragma unroll 1
            for (int c = half * 32 * NB; c < (half + 1) * 32 * NB; c += 32) {
                uint32_t o[32];
                if (n > 0) tmem_ld_x32(tDQ + lane_off + c, o);
                if (n > 0 && c + 32 >= (half + 1) * 32 * NB) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(dq_empty);
                }
#pragma unroll
                for (int e = 0; e < 32; e += 16) {
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        w[k] = n > 0 ? pack2<BF16>(__uint_as_float(o[e + 2 * k]) * by, __uint_as_float(o[e + 2 * k + 1]) * by) : 0u;
                    if (row && c + e + 16 <= p.D) {
                        if (wide) {
                            store32(to + c + e, w);
                        } else {
                            *reinterpret_cast<uint4*>(to + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                            *reinterpret_cast<uint4*>(to + c + e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    } else if (row && c + e + 8 <= p.D) {
                        *reinterpret_cast<uint4*>(to + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
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

template <bool BF16, int NB>
cudaError_t start(const DqParams& P, unsigned grid, cudaStream_t stream) {
    const cudaError_t e = allow_smem<prompt_dq_kernel<BF16, NB>>(Smem<NB>::kTotal);
    if (e != cudaSuccess) return e;
    prompt_dq_kernel<BF16, NB><<<grid, kWarps * 32, Smem<NB>::kTotal, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dq(const PromptParams& p, cudaStream_t stream) {
    DqParams P;
    P.p = p;
    P.t = make_tiles(p);
    const bool bf16 = p.dtype == TA_BF16;
    P.idesc_s = make_idesc(bf16, 0, 0, 0);  // (N is set for each product)
    P.idesc_q = make_idesc(bf16, (uint32_t)(p.D + 15) / 16 * 16, 0, 1);
    P.ksteps = (p.D + 15) / 16;
    P.scale_log2e = p.scale * kToLog2;
    if (!make_rows_map(&P.tm_q, bf16, p.q, p.D, p.Hq, p.total_q, p.q_rs, P.t.hp, P.t.tq) ||
        !make_rows_map(&P.tm_do, bf16, p.d_out, p.D, p.Hq, p.total_q, (long long)p.Hq * p.D, P.t.hp, P.t.tq) ||
        !make_rows_map(&P.tm_k, bf16, p.k, p.D, p.Hk, p.total_k, p.k_rs, 1, 128) ||
        !make_rows_map(&P.tm_v, bf16, p.v, p.D, p.Hk, p.total_k, p.v_rs, 1, 128))
        return cudaErrorInvalidValue;
    const long long items = most_items(p, P.t, 1);
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (p.D <= 64) return bf16 ? start<true, 1>(P, (unsigned)items, stream) : start<false, 1>(P, (unsigned)items, stream);
    return bf16 ? start<true, 2>(P, (unsigned)items, stream) : start<false, 2>(P, (unsigned)items, stream);
}

}  // namespace prompt
}  // namespace triattn
