// prompt_fwd.cu -- causal attention of packed prompts with grouped heads on tcgen05 tensor cores: 16-bit inputs, D <= 128.
//
// The mathematics is prompt.cuh's: the heads of a group are rows.  A tile is 128 rows, tq tokens x hp heads of a group (hp the
// largest power of two in the group's heads: all of 4, one of 7), loaded by one TMA box of a (D, head, token) map, so that
// short sequences fill tiles by their heads and the keys past the causal border are few.  A work item is two neighbouring
// tiles of one (sequence, key head), which share every K and V tile (128 keys) that is loaded.
//
// One CTA a SM, 16 warps:
//   0-3, 4-7   softmax of tile 0 / 1: thread = row = tensor-memory lane, the row's 128 logits in registers
//   8-11       epilogue: O / l to memory while the next item has begun
//   12         tcgen05.mma, by one thread: S_i = Q_i K^T (shared x shared), O_i += P_i V (P from tensor memory, over S_i)
//   13         TMA of Q_0, Q_1 and the ring of K and V tiles
//   14         the items, handed to the others through a ring
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (64 or 128 each): all 512 columns at D = 128.  The tensor core works on
// one tile while the other's softmax runs.
//
// Softmax: one pass with a reference maximum that is raised only when a row's maximum passes it by 2^8 (fp16's range allows
// that), which scales O by its own threads and is rare; sums, maxima, O in fp32, P rounded to the inputs' type.  P is handed
// over in two halves.  V's rows past the sequence's end are other sequences' (or NaN that nobody wrote): their weights are 0,
// and the products stop at the sixteen keys that hold the last one, the rest of which is zeroed in shared memory.
//
// Items go by falling cost (the number of key tiles), one at a time to the CTA that has finished its own: the grid has a
// block for every item, and a running CTA takes the next block's place by clusterlaunchcontrol.try_cancel, so no
// counter in memory has to be zeroed and the tail is as short as one item.
//
// Bound: the tensor core, 2048 clocks a pair of tiles and 128 keys at D = 128, as long as its products are asked for in time.
// So one thread issues them, without votes or other lanes to wait for, straight on over whole key tiles and from one item into the
// next (bf16, 32 heads over 8 of 128, in short runs; a warp whose waits were votes, before: one chunk of 1216 tokens on a prefix
// of 30000, 152 equal items, 425 us, 1434 TFLOP/s; so 333 us, 1830; eight prompts of 512 to 4096 tokens 360 and 290, 1510
// TFLOP/s, where an item is 9 steps and its first and last are slower; back to back for seconds 315, 1390, as the clock gives
// way).  Heads of 64 are bound by the softmax (two sequences of 16384, 16 heads over 4: 1.01 ms,
// 1090 TFLOP/s). Code is time as well: a second form of the softmax for the causal border, with fewer columns, cost 3%.
#include "prompt_tc.cuh"

namespace triattn {
namespace prompt {
namespace {

struct FwdParams {
    CUtensorMap tm_q, tm_k, tm_v;
    PromptParams p;
    Tiles t;
    uint32_t idesc_qk, idesc_pv;
    int ksteps;                // D / 16, rounded up
    float scale_log2e;         // |scale| log2 e
    int negative;              // scale < 0: the logits change their sign
};

constexpr int kRing = 2;       // items known ahead
constexpr int kWarps = 16;
constexpr int kConsumers = 14; // warps that read an item: 8 softmax, 4 epilogue, MMA, TMA

template <int NB>
struct Smem {
    static constexpr uint32_t kTile = NB * kBox;                       // 128 rows
    static constexpr int kStages = NB == 1 ? 8 : 4;
    static constexpr uint32_t kQ = 0, kKV = 2 * kTile, kMl = kKV + kStages * kTile;  // (m, l) of the rows
    static constexpr uint32_t kItems = kMl + 2 * 128 * 8, kClc = kItems + kRing * sizeof(Item<2>);
    static constexpr uint32_t kBars = kClc + 16;
    static constexpr int kNumBars = 2 * 2 + 2 * kStages + 5 * 2 + 2 * 2 + 2 * kRing + 2;
    static constexpr uint32_t kSlot = kBars + 8 * kNumBars, kAbort = kSlot + 4, kTotal = kAbort + 4 + 1024;
};

// 128 columns by two loads and one wait.
__device__ __forceinline__ void tmem_ld_2x64(uint32_t ta, uint32_t (&r)[128]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%128];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, %80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, %96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%129];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
          "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
          "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
          "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
          "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
          "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
          "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
          "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
          "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(ta), "r"(ta + 64u));
}

template <bool BF16, int NB>
__global__ void __launch_bounds__(kWarps * 32, 1) prompt_fwd_kernel(const __grid_constant__ FwdParams P) {
    using M = Smem<NB>;
    constexpr int S = M::kStages;
    constexpr uint32_t kTile = M::kTile, kOCols = NB * 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* g0 = smem_raw + (base - raw);
    const PromptParams& p = P.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(g0 + M::kAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(g0 + M::kSlot);
    Item<2>* items = reinterpret_cast<Item<2>*>(g0 + M::kItems);
    float2* ml = reinterpret_cast<float2*>(g0 + M::kMl);
    auto bar = [&](int i) { return base + M::kBars + 8u * (uint32_t)i; };
    auto q_full = [&](int i) { return bar(i); };
    auto q_empty = [&](int i) { return bar(2 + i); };
    auto kv_full = [&](int s) { return bar(4 + s); };
    auto kv_empty = [&](int s) { return bar(4 + S + s); };
    constexpr int b0 = 4 + 2 * S;
    auto s_full = [&](int i) { return bar(b0 + i); };
    auto p_half = [&](int i, int h) { return bar(b0 + 2 + 2 * i + h); };
    auto o_full = [&](int i) { return bar(b0 + 6 + i); };
    auto o_empty = [&](int i) { return bar(b0 + 8 + i); };
    auto ml_full = [&](int i) { return bar(b0 + 10 + i); };
    auto ml_empty = [&](int i) { return bar(b0 + 12 + i); };
    auto it_full = [&](int r) { return bar(b0 + 14 + r); };
    auto it_empty = [&](int r) { return bar(b0 + 14 + kRing + r); };
    const uint32_t clc = bar(b0 + 14 + 2 * kRing), drain = bar(b0 + 15 + 2 * kRing);
    static_assert(4 + 2 * S + 16 + 2 * kRing <= M::kNumBars + 0, "barriers");
    auto q_smem = [&](int i) { return base + M::kQ + (uint32_t)i * kTile; };
    auto kv_smem = [&](int s) { return base + M::kKV + (uint32_t)s * kTile; };

    if (threadIdx.x == 0) {
        *abort_flag = 0;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(p_half(i, 0), 4);
            mbar_init(p_half(i, 1), 4);
            mbar_init(o_full(i), 1);
            mbar_init(o_empty(i), 4);
            mbar_init(ml_full(i), 4);
            mbar_init(ml_empty(i), 4);
        }
#pragma unroll 1
        for (int s = 0; s < S; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int r = 0; r < kRing; ++r) {
            mbar_init(it_full(r), 1);
            mbar_init(it_empty(r), kConsumers);
        }
        mbar_init(clc, 1);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    int item_n = 0;            // items so far
    // The next item, for the warps that consume them: false at the end.
    auto next_item = [&](Item<2>& it) -> bool {
        const int r = item_n % kRing;
        ok = __all_sync(0xffffffffu, wait(it_full(r), (uint32_t)(item_n / kRing) & 1u, abort_flag, p.status));
        if (!ok) return false;
        it = items[r];
        __syncwarp();
        if (lane == 0) mbar_arrive(it_empty(r));
        ++item_n;
        return it.on != 0;
    };

    // (the block has 128 registers a thread: 2 x 184 + 80 + 64 = 4 x 128)
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 14) {
            // ------------------------------------------------------------ the items
            ok = hand_out<2, kRing>(p, P.t, items, it_full, it_empty, base + M::kClc, clc, abort_flag);
            if (!ok) *abort_flag = 1;
        } else if (warp == 13) {
            // ------------------------------------------------------------ TMA
            StageRing kr = {0, 0u, false};
            Item<2> it;
            uint32_t q_use[2] = {0u, 0u};
            // (kTile, as a number of the launch: with the constant the compiler's loop of the issuing thread is 2% slower)
            const uint32_t q_bytes = (uint32_t)(P.t.tq * P.t.hp) * 128u * NB;
            while (ok && next_item(it)) {
                const int n = (max(it.keys[0], it.keys[1]) + 127) / 128;
                auto load_q = [&](int i) {
                    if (it.keys[i] <= 0 || !ok) return;
                    if (q_use[i] > 0) ok = __all_sync(0xffffffffu, wait(q_empty(i), (q_use[i] - 1u) & 1u, abort_flag, p.status));
                    ++q_use[i];
                    if (ok && lane == 0) {
                        mbar_expect_tx(q_full(i), q_bytes);
                        for (int b = 0; b < NB; ++b)
                            tma_load_3d(q_smem(i) + b * kBox, &P.tm_q, 64 * b, it.head[i], it.q0 + it.tok[i], q_full(i));
                    }
                };
                auto load_kv = [&](const CUtensorMap* tm, int j) {
                    if (!ok) return;
                    if (kr.wrapped) ok = __all_sync(0xffffffffu, wait(kv_empty(kr.idx), kr.ph ^ 1u, abort_flag, p.status));
                    if (ok && lane == 0) {
                        mbar_expect_tx(kv_full(kr.idx), kTile);
                        for (int b = 0; b < NB; ++b)
                            tma_load_3d(kv_smem(kr.idx) + b * kBox, tm, 64 * b, it.h, it.k0 + 128 * j, kv_full(kr.idx));
                    }
                    kr.next(S);
                };
                if (n > 0) load_kv(&P.tm_k, 0);
                load_q(0);
                load_q(1);
                for (int j = 0; j < n && ok; ++j) {
                    load_kv(&P.tm_v, j);
                    if (j + 1 < n) load_kv(&P.tm_k, j + 1);
                }
            }
            if (!ok) *abort_flag = 1;
        } else if (warp == 12) {
            // ------------------------------------------------------------ MMA
            // One thread runs the loop; the others help where a tile of V ends with rows that are not the sequence's.
            const bool leader = elect_one();
            const int lead = __ffs((int)__ballot_sync(0xffffffffu, leader)) - 1;
            StageRing kr = {0, 0u, false};
            uint32_t use = 0;  // parities of tile i's barriers: bit i of Q, 2 + i of P, 4 + i of O; 6 + i: O was in use
            auto await = [&](uint32_t b, uint32_t parity) {
                if (ok) ok = wait(b, parity, abort_flag, p.status);
                tc_fence_after();
            };
            // The next item: the keys of its tiles, and of its sequence.  One at a time while a product of the item before is
            // pending: the ring's third item from there waits for the epilogue, and the epilogue for that product.
            auto fetch = [&](int& k0, int& k1, int& lk) -> bool {
                const int r = item_n % kRing;
                await(it_full(r), (uint32_t)(item_n / kRing) & 1u);
                if (!ok) return false;
                const bool on = items[r].on != 0;
                k0 = items[r].keys[0];
                k1 = items[r].keys[1];
                lk = items[r].lq + items[r].shift;
                mbar_arrive(it_empty(r));
                ++item_n;
                return on;
            };
            // S_i of key tile j of a tile that sees `keys`, K in stage st
            auto qk = [&](int i, int keys, int j, int st) {
                if (j == 0) {
                    await(q_full(i), (use >> i) & 1u);
                    if (!ok) return;
                    use ^= 1u << i;
                }
                const int cols = min(128, (keys - 128 * j + 15) & ~15);
                issue_rows<NB>(tmem + i * 128, desc_lo(q_smem(i), 16), desc_lo(kv_smem(st), 16),
                               P.idesc_qk | ((uint32_t)(cols >> 3) << 17), P.ksteps);
                mma_commit(s_full(i));
                if (128 * (j + 1) >= keys) mma_commit(q_empty(i));
            };
            // The epilogue has read the last item's O_i.
            auto o_mine = [&](int i) {
                if ((use >> (6 + i)) & 1u) {
                    await(o_empty(i), (use >> (4 + i)) & 1u);
                    use ^= 16u << i;
                }
                use |= 64u << i;
            };
            // O_i += P_i V of key tile j, V in stage st
            auto pv = [&](int i, int keys, int j, int st) {
                if (j == 0) o_mine(i);
                const int steps = min(8, (keys - 128 * j + 15) / 16);
                const uint32_t b = desc_lo(kv_smem(st), kBox), d = tmem + 256u + (uint32_t)i * kOCols, a = tmem + i * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    await(p_half(i, h), (use >> (2 + i)) & 1u);
                    if (!ok) return;
                    issue_cols<32>(d, a, b, P.idesc_pv, 4 * h, 4 * h + 4, steps, j == 0);
                }
                use ^= 4u << i;
                if (128 * (j + 1) >= keys) mma_commit(o_full(i));
            };
            // Step j of an item: PV of key tile j - 1, tile 0 then tile 1, behind each QK of key tile j; after the last PV
            // the next item's first, whose K tile is the next in the ring: its softmax runs while the other tile ends.
            int k0 = 0, k1 = 0, lk = 0, n = 0, j = 0;
            bool there = true, clean = false;
            for (;;) {
                int tail = 0, tail_st = 0;
                if (leader) {
                    if (j == 0) {  // (nothing is pending)
                        do there = fetch(k0, k1, lk);
                        while (there && max(k0, k1) <= 0);
                        if (there) await(kv_full(kr.idx), kr.ph);
                        if (there && ok && k0 > 0) qk(0, k0, 0, kr.idx);
                        if (there && ok && k1 > 0) qk(1, k1, 0, kr.idx);
                        if (there && ok) mma_commit(kv_empty(kr.idx));
                        kr.next(S);
                        n = (max(k0, k1) + 127) / 128;
                        j = 1;
                    }
                    while (ok && there) {
                        // Whole key tiles in the middle of an item, without a question (a few dozen instructions of one
                        // thread are a product's time).
                        for (const int whole = min(k0, k1); 128 * (j + 1) < whole; ++j) {
                            const int vst = kr.idx;
                            const uint32_t vph = kr.ph;
                            kr.next(S);
                            const uint32_t v = desc_lo(kv_smem(vst), kBox), k = desc_lo(kv_smem(kr.idx), 16);
                            const uint32_t pp = (use >> 2) & 1u, pq = (use >> 3) & 1u;
                            ok = wait(kv_full(vst), vph, abort_flag, p.status);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t d = tmem + 256u + (uint32_t)i * kOCols, a = tmem + i * 128;
                                if (j == 1) o_mine(i);
                                if (ok) ok = wait(p_half(i, 0), i ? pq : pp, abort_flag, p.status);
                                tc_fence_after();
                                if (!ok) break;
                                issue_cols<32>(d, a, v, P.idesc_pv, 0, 4, 8, j == 1);
                                ok = wait(p_half(i, 1), i ? pq : pp, abort_flag, p.status);
                                tc_fence_after();
                                if (!ok) break;
                                issue_cols<32>(d, a, v, P.idesc_pv, 4, 8, 8, false);
                                if (i == 0) {
                                    ok = wait(kv_full(kr.idx), kr.ph, abort_flag, p.status);
                                    tc_fence_after();
                                    if (!ok) break;
                                } else {
                                    mma_commit(kv_empty(vst));
                                }
                                issue_rows<NB>(a, desc_lo(q_smem(i), 16), k, P.idesc_qk | (16u << 17), P.ksteps);
                                mma_commit(s_full(i));
                            }
                            if (!ok) break;
                            mma_commit(kv_empty(kr.idx));
                            kr.next(S);
                            use ^= 12u;
                        }
                        if (!ok) break;
                        if (!clean) {
                            await(kv_full(kr.idx), kr.ph);
                            if (!ok) break;
                            const int valid = lk - 128 * (j - 1);  // rows of V that are the sequence's
                            if (valid < 128 && valid % 16) {
                                tail = valid;
                                tail_st = kr.idx;
                                clean = true;
                                break;
                            }
                        }
                        clean = false;
                        const int vst = kr.idx;
                        kr.next(S);
                        const bool last = j == n;
                        int n0 = 0, n1 = 0, nlk = 0;
                        bool k_here = false;
                        if (last) there = fetch(n0, n1, nlk);  // (while the last P is made)
                        if (!ok) break;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int keys = i ? k1 : k0;
                            if (128 * (j - 1) < keys) pv(i, keys, j - 1, vst);
                            if (!ok) break;
                            if (i == 1) mma_commit(kv_empty(vst));
                            const int to = last ? (i ? n1 : n0) : keys, at = last ? 0 : j;
                            if (!ok || 128 * at >= to) continue;
                            if (!k_here) await(kv_full(kr.idx), kr.ph);
                            k_here = true;
                            if (ok) qk(i, to, at, kr.idx);
                        }
                        if (k_here) {
                            if (ok) mma_commit(kv_empty(kr.idx));
                            kr.next(S);
                        }
                        ++j;
                        if (last) {
                            k0 = n0;
                            k1 = n1;
                            lk = nlk;
                            n = (max(k0, k1) + 127) / 128;
                            j = 1;
                            if (there && n == 0) {  // an item without keys: its rows are the epilogue's
                                j = 0;
                                tail = -1;
                                break;
                            }
                        }
                    }
                }
                tail = __shfl_sync(0xffffffffu, tail, lead);
                if (tail == 0) break;
                if (tail > 0) clear_rows<NB>(kv_smem(__shfl_sync(0xffffffffu, tail_st, lead)), tail, (tail + 15) & ~15);
            }
            if (!ok && leader) *abort_flag = 1;
            if (leader) mma_commit(drain);
            wait_bar_drain(drain, 0);
            __syncwarp();
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int i = warp / 4, r = warp % 4 * 32 + lane;
        const uint32_t lane_off = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t st = tmem + lane_off + i * 128, ot = tmem + lane_off + 256u + (uint32_t)i * kOCols;
        const int tok_r = (int)P.t.fd_hp.div((uint32_t)r);
        const float f = P.scale_log2e, step = kRescaleLog2 / f;
        Item<2> it;
        uint32_t s_use = 0, ml_use = 0;
        while (ok && next_item(it)) {
            const int keys = i == 0 ? it.keys[0] : it.keys[1], tok = (i == 0 ? it.tok[0] : it.tok[1]) + tok_r;
            const int n = (keys + 127) / 128;
            const int limit = tok + it.shift;                            // the last key that this row sees
            const int first = (i == 0 ? it.tok[0] : it.tok[1]) + it.shift;  // ... and the tile's first row
            float m = -INFINITY, l = 0.f;                                // the reference maximum (of S), the sum
            for (int j = 0; j < n && ok; ++j) {
                ok = __all_sync(0xffffffffu, wait(s_full(i), s_use & 1u, abort_flag, p.status));
                if (!ok) break;
                ++s_use;
                tc_fence_after();
                uint32_t sr[128];
                tmem_ld_2x64(st, sr);
                float x[128];
#pragma unroll
                for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sr[c]);
                if (P.negative) {
#pragma unroll
                    for (int c = 0; c < 128; ++c) x[c] = -x[c];
                }
                if (128 * j + 127 > first) {  // some row does not see every key
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t vm = low_bits(limit - 128 * j - 32 * h + 1);
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[32 * h + c] = (vm >> c) & 1u ? x[32 * h + c] : -INFINITY;
                    }
                }
                float a0 = x[0], a1 = x[1], a2 = x[2], a3 = x[3];
#pragma unroll
                for (int c = 4; c < 124; c += 8) {
                    a0 = max3(a0, x[c], x[c + 1]);
                    a1 = max3(a1, x[c + 2], x[c + 3]);
                    a2 = max3(a2, x[c + 4], x[c + 5]);
                    a3 = max3(a3, x[c + 6], x[c + 7]);
                }
                a0 = max3(a0, x[124], x[125]);
                a1 = max3(a1, x[126], x[127]);
                const float tm = fmaxf(max3(a0, a1, a2), a3);
                // (from -inf: inf, a new reference)
                if (__any_sync(0xffffffffu, tm - m > step)) {
                    const float mn = fmaxf(m, tm);
                    const float alpha = mn == -INFINITY ? 1.f : ex2((m - mn) * f);
                    m = mn;
                    l *= alpha;
                    if (j > 0) {  // (PV of the last key tile is done: S was asked for behind it)
#pragma unroll 1
                        for (uint32_t c = 0; c < kOCols; c += 16) {
                            uint32_t o[16];
                            tmem_ld_x16(ot + c, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st_x16(ot + c, o);
                        }
                    }
                }
                const float nb = m == -INFINITY ? 0.f : -m * f;
                const float2 f2 = make_float2(f, f), nb2 = make_float2(nb, nb);
                float2 s0 = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 y = __ffma2_rn(make_float2(x[32 * h + 2 * c], x[32 * h + 2 * c + 1]), f2, nb2);
                        const float2 w = make_float2(ex2(y.x), ex2(y.y));
                        if (c & 1) s1 = __fadd2_rn(s1, w);
                        else s0 = __fadd2_rn(s0, w);
                        pk[c] = pack2<BF16>(w.x, w.y);
                    }
                    tmem_st_x16(st + 16 * h, pk);
                    if (h & 1) {
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_half(i, h / 2));
                    }
                }
                l += (s0.x + s0.y) + (s1.x + s1.y);
            }
            if (!ok) break;
            if (ml_use > 0) ok = __all_sync(0xffffffffu, wait(ml_empty(i), (ml_use - 1u) & 1u, abort_flag, p.status));
            if (!ok) break;
            ++ml_use;
            ml[i * 128 + r] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(ml_full(i));
        }
        if (!ok) *abort_flag = 1;
    } else {
        // ------------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const int wq = warp % 4, r = wq * 32 + lane;
        const int tok_r = (int)P.t.fd_hp.div((uint32_t)r), head_r = r - tok_r * P.t.hp;
        const bool wide = p.D % 16 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;  // rows in 32-byte pieces
        Item<2> it;
        uint32_t ml_use = 0, o_use[2] = {0u, 0u};
        while (ok && next_item(it)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ok = ok && __all_sync(0xffffffffu, wait(ml_full(i), ml_use & 1u, abort_flag, p.status));
                if (!ok) break;
                const float2 x = ml[i * 128 + r];
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_empty(i));
                const bool none = x.x == -INFINITY && x.y == 0.f;
                const float inv = none ? 0.f : __fdividef(1.f, x.y);
                const bool row = r < it.rows[i];
                const long long tok = it.q0 + it.tok[i] + tok_r, head = it.head[i] + head_r;
                uint16_t* out = static_cast<uint16_t*>(p.out) + (tok * p.Hq + head) * p.D;
                if (row && p.lse) p.lse[head * p.total_q + tok] = none ? -INFINITY : (x.x * P.scale_log2e + log2f(x.y)) * kLn2;
                const bool any = it.keys[i] > 0;
                if (any) {
                    ok = __all_sync(0xffffffffu, wait(o_full(i), o_use[i] & 1u, abort_flag, p.status));
                    if (!ok) break;
                    ++o_use[i];
                    tc_fence_after();
                }
                const uint32_t ot = tmem + ((uint32_t)(wq * 32) << 16) + 256u + (uint32_t)i * kOCols;
#pragma unroll 1
                for (int c = 0; c < (int)kOCols; c += 32) {
                    uint32_t o[32];
                    if (any) tmem_ld_x32(ot + c, o);
                    if (any && c + 32 >= (int)kOCols) {  // the last columns are in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_empty(i));
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            // (a row that sees no key: its columns may hold anything)
                            const float a = none ? 0.f : __uint_as_float(o[e + 2 * k]) * inv;
                            const float b = none ? 0.f : __uint_as_float(o[e + 2 * k + 1]) * inv;
                            w[k] = pack2<BF16>(a, b);
                        }
                        if (row && c + e + 16 <= p.D) {
                            if (wide) {
                                store32(out + c + e, w);
                            } else {
                                *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                                *reinterpret_cast<uint4*>(out + c + e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        } else if (row && c + e + 8 <= p.D) {
                            *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
            ++ml_use;
        }
        if (!ok) *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

template <bool BF16, int NB>
cudaError_t start(const FwdParams& P, unsigned grid, cudaStream_t stream) {
    const cudaError_t e = allow_smem<prompt_fwd_kernel<BF16, NB>>(Smem<NB>::kTotal);
    if (e != cudaSuccess) return e;
    prompt_fwd_kernel<BF16, NB><<<grid, kWarps * 32, Smem<NB>::kTotal, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

// Heads of a tile: the largest power of two that divides the group (up to 128), so that tokens fill the rest of the 128 rows.
Tiles make_tiles(const PromptParams& p) {
    Tiles t;
    t.hp = p.G & -p.G;
    if (t.hp > 128) t.hp = 128;
    t.tq = 128 / t.hp;
    t.ng = p.G / t.hp;
    t.fd_hp = make_fastdiv((uint32_t)t.hp);
    return t;
}

}  // namespace prompt

cudaError_t launch_prompt_tc_fwd(const PromptParams& p, cudaStream_t stream) {
    using namespace prompt;
    FwdParams P;
    P.p = p;
    P.t = make_tiles(p);
    const bool bf16 = p.dtype == TA_BF16;
    P.idesc_qk = make_idesc(bf16, 0, 0, 0);  // (N is set for each product)
    P.idesc_pv = make_idesc(bf16, (uint32_t)(p.D + 15) / 16 * 16, 0, 1);
    P.ksteps = (p.D + 15) / 16;
    // (a scale of 0 makes every logit 0: so does one far below the least that counts, and a hidden key's -inf stays)
    P.scale_log2e = fmaxf(fabsf(p.scale) * kToLog2, 1e-30f);
    P.negative = p.scale < 0.f;
    if (!make_rows_map(&P.tm_q, bf16, p.q, p.D, p.Hq, p.total_q, p.q_rs, P.t.hp, P.t.tq) ||
        !make_rows_map(&P.tm_k, bf16, p.k, p.D, p.Hk, p.total_k, p.k_rs, 1, 128) ||
        !make_rows_map(&P.tm_v, bf16, p.v, p.D, p.Hk, p.total_k, p.v_rs, 1, 128))
        return cudaErrorInvalidValue;
    const long long items = most_items(p, P.t, 2);
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)items;
    if (p.D <= 64) return bf16 ? start<true, 1>(P, grid, stream) : start<false, 1>(P, grid, stream);
    return bf16 ? start<true, 2>(P, grid, stream) : start<false, 2>(P, grid, stream);
}

}  // namespace triattn
