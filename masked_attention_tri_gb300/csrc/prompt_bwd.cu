// prompt_bwd.cu -- gradients of the causal attention of packed prompts with grouped heads on tcgen05 tensor cores:
// 16-bit inputs, D <= 128.
//
// Rows are tokens x heads of a group (prompt.cuh), in the forward's tiles of tq tokens x hp heads.  With P = 2^(s - lse)
// recomputed and delta = dO . O, one CTA for each (sequence, key head, 128 keys) walks the row tiles that see a key of its own:
//     S^T = K Q^T, dP^T = V dO^T         keys on the tensor-memory lanes, rows of the tile in the columns
//     dV += P^T dO                       P^T from tensor memory, over S^T
//     dS = P (dP - delta),  dK += dS^T Q dS in shared memory, which serves both products
//     dQ = dS K                          over S^T, when dV has read P^T; read out and added to an fp32 sum in memory
// Tensor memory: S^T (then P^T, then dQ), dP^T, dV, dK: 4 x 128 columns at D = 128.
//
// 16 warps: 0-7 softmax and dS (key = lane, 64 rows each half), 8-11 dQ to memory, 12 MMA, 13 TMA, 14 the rows' lse and delta.
// The tensor core's order: S(i) | dP(i), dK(i-1), dV(i), dQ(i), S(i+1) ...: dP and the last tile's dK run while P(i) is formed, dV
// while dS(i) is, and only dQ's read-out stands between dQ(i) and S(i+1).
//
// Bound: shared memory (the operands of five products of 128 x 128 x D, of which all but dV's read both from there) and the
// tensor core, which needs 2560 clocks a tile at D = 128.  dQ is summed over the key tiles by fp32 reductions in memory, whose
// order varies.  Where there are too few (sequence, head, key tile) for the GPU, the row tiles of one are dealt to several CTAs,
// and dK and dV are summed the same way.
#include "prompt.cuh"
#include "tc_kernel.cuh"

namespace triattn {
namespace prompt {

void tile_shape(int G, int& hp, int& tq);

namespace {

using namespace tc;

struct GradParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;
    PromptParams p;
    int hp, tq, ng;            // heads and tokens of a tile; tiles of the same tokens (G / hp)
    int splits;                // CTAs of a key tile
    FastDiv fd_hp;
    uint32_t idesc_s, idesc_g, idesc_k, idesc_q;
    int ksteps;                // D / 16, rounded up
    float scale_log2e;
};

constexpr int kWarps = 16;

template <int NB>
struct Smem {
    static constexpr uint32_t kTile = NB * kBox;
    static constexpr uint32_t kK = 0, kV = kTile, kQ = 2 * kTile, kDO = kQ + 2 * kTile, kDS = kDO + 2 * kTile;
    static constexpr uint32_t kRows = kDS + 2 * kBox;                  // [2 stages][-lse log2 e, delta][128]
    static constexpr uint32_t kBars = kRows + 2 * 2 * 128 * 4;
    static constexpr int kNumBars = 1 + 2 * 2 + 2 * 2 + 2 * 2 + 8;
    static constexpr uint32_t kSlot = kBars + 8 * kNumBars, kAbort = kSlot + 4, kTotal = kAbort + 4;
};
static_assert(Smem<2>::kTotal <= kMaxDynamicSmem, "shared memory");

// (inline: see prompt_fwd.cu)
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    if (mbar_test(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > kTimeoutCycles) {
                *abort_flag = 1;
                atomicCAS(status, 0, kStatusTimeout);
                return false;
            }
        }
    }
}

__device__ __forceinline__ void red_v4(float* p, float a, float b, float c, float d) {
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

template <bool BF16, int NB>
__global__ void __launch_bounds__(kWarps * 32, 1) prompt_bwd_kernel(const __grid_constant__ GradParams P) {
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
    const int blocks = (q.lq + P.tq - 1) / P.tq;
    const int first = max(0, k0 - q.shift) / P.tq * P.ng + split;       // the first tile with a row that sees the key k0
    const int n = first < blocks * P.ng ? (blocks * P.ng - first + P.splits - 1) / P.splits : 0;
    uint16_t* dk = static_cast<uint16_t*>(p.dk) + ((long long)(q.k0 + k0) * p.Hk + h) * p.D;
    uint16_t* dv = static_cast<uint16_t*>(p.dv) + ((long long)(q.k0 + k0) * p.Hk + h) * p.D;
    if (n == 0) {  // keys that no query sees
        if (P.splits == 1) {
            const int pieces = p.D / 8;
            for (int e = threadIdx.x; e < keys * pieces; e += kWarps * 32) {
                const long long at = (long long)(e / pieces) * p.Hk * p.D + (e % pieces) * 8;
                *reinterpret_cast<uint4*>(dk + at) = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(dv + at) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }
    // Tile j of the walk: its first token, first query head and rows.
    auto tile = [&](int j, int& tok, int& head, int& rows) {
        const int t = first + j * P.splits, b = t / P.ng;
        tok = b * P.tq;
        head = h * p.G + (t - b * P.ng) * P.hp;
        rows = min(P.tq, q.lq - tok) * P.hp;
    };

    volatile int* abort_flag = reinterpret_cast<volatile int*>(g0 + M::kAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(g0 + M::kSlot);
    float* row_s = reinterpret_cast<float*>(g0 + M::kRows);
    auto bar = [&](int i) { return base + M::kBars + 8u * (uint32_t)i; };
    const uint32_t kv_full = bar(0);
    auto q_full = [&](int s) { return bar(1 + s); };
    auto q_empty = [&](int s) { return bar(3 + s); };
    auto do_full = [&](int s) { return bar(5 + s); };
    auto do_empty = [&](int s) { return bar(7 + s); };
    auto row_full = [&](int s) { return bar(9 + s); };
    auto row_empty = [&](int s) { return bar(11 + s); };
    const uint32_t s_full = bar(13), p_full = bar(14), dp_full = bar(15), ds_full = bar(16), ds_free = bar(17),
                   dq_full = bar(18), dq_empty = bar(19), fin = bar(20);
    auto q_smem = [&](int s) { return base + M::kQ + (uint32_t)s * kTile; };
    auto do_smem = [&](int s) { return base + M::kDO + (uint32_t)s * kTile; };
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(kv_full, 1);
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
            mbar_init(do_full(s), 1);
            mbar_init(do_empty(s), 1);
            mbar_init(row_full(s), 1);
            mbar_init(row_empty(s), 8);
        }
        mbar_init(s_full, 1);
        mbar_init(p_full, 8);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(ds_free, 1);
        mbar_init(dq_full, 1);
        mbar_init(dq_empty, 4);
        mbar_init(fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // Rows of Q and dO that no box fills (tq hp < 128) stay zeros.
    const int full_rows = P.tq * P.hp;
    for (int e = threadIdx.x; e < 4 * NB * (128 - full_rows) * 8; e += kWarps * 32) {
        const int c = e % 8, r = e / 8 % (128 - full_rows) + full_rows, b = e / 8 / (128 - full_rows);
        st_shared_v4(base + M::kQ + (uint32_t)b * kBox + (uint32_t)r * 128u + c * 16u, 0u, 0u, 0u, 0u);
    }
    fence_async_shared();
    if (warp == 12) {
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

    // (the block has 128 registers a thread: 2 x 184 + 88 + 56 = 4 x 128)
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 13) {
            // -------------------------------------------------------- TMA
            if (lane == 0) {
                mbar_expect_tx(kv_full, 2 * kTile);
                for (int b = 0; b < NB; ++b) {
                    tma_load_3d(base + M::kK + b * kBox, &P.tm_k, 64 * b, h, q.k0 + k0, kv_full);
                    tma_load_3d(base + M::kV + b * kBox, &P.tm_v, 64 * b, h, q.k0 + k0, kv_full);
                }
            }
            const uint32_t bytes = (uint32_t)full_rows * 128u * NB;
            for (int j = 0; j < n && ok; ++j) {
                int tok, head, rows;
                tile(j, tok, head, rows);
                const int s = j & 1;
                const uint32_t before = (uint32_t)(j / 2 - 1) & 1u;
                if (j >= 2) ok = __all_sync(0xffffffffu, wait(q_empty(s), before, abort_flag, p.status));
                if (ok && lane == 0) {
                    mbar_expect_tx(q_full(s), bytes);
                    for (int b = 0; b < NB; ++b) tma_load_3d(q_smem(s) + b * kBox, &P.tm_q, 64 * b, head, q.q0 + tok, q_full(s));
                }
                if (j >= 2 && ok) ok = __all_sync(0xffffffffu, wait(do_empty(s), before, abort_flag, p.status));
                if (ok && lane == 0) {
                    mbar_expect_tx(do_full(s), bytes);
                    for (int b = 0; b < NB; ++b) tma_load_3d(do_smem(s) + b * kBox, &P.tm_do, 64 * b, head, q.q0 + tok, do_full(s));
                }
            }
            if (!ok) *abort_flag = 1;
        } else if (warp == 14) {
            // -------------------------------------------------------- the rows' factors
            for (int j = 0; j < n && ok; ++j) {
                int tok, head, rows;
                tile(j, tok, head, rows);
                const int s = j & 1;
                float a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 32 * i + lane, t = (int)P.fd_hp.div((uint32_t)r);
                    const long long at = (long long)(head + r - t * P.hp) * p.total_q + q.q0 + tok + t;
                    a[i] = r < rows ? p.lse[at] : 0.f;
                    b[i] = r < rows ? p.delta[at] : 0.f;
                }
                if (j >= 2) ok = __all_sync(0xffffffffu, wait(row_empty(s), (uint32_t)(j / 2 - 1) & 1u, abort_flag, p.status));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    row_s[s * 256 + 32 * i + lane] = -a[i] * tc::kLog2e;
                    row_s[s * 256 + 128 + 32 * i + lane] = -b[i];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(row_full(s));
            }
            if (!ok) *abort_flag = 1;
        } else if (warp == 12) {
            // -------------------------------------------------------- MMA
            const bool leader = elect_one();
            auto wait_all = [&](uint32_t b, uint32_t parity) {
                if (ok) ok = __all_sync(0xffffffffu, wait(b, parity, abort_flag, p.status));
                tc_fence_after();
                return ok;
            };
            auto kstep = [](int kk) { return (uint64_t)(((kk >> 2) * kBox + (kk & 3) * 32) >> 4); };
            // Rows of a tile past its own are another sequence's, or nobody's: zeroed up to the next 16.
            auto clear = [&](uint32_t at, int rows) {
                if (!(rows & 15)) return;
                const int zeros = 16 - (rows & 15);
                for (int e = lane; e < zeros * 8 * NB; e += 32)
                    st_shared_v4(at + (uint32_t)(e / 8 / zeros) * kBox + (uint32_t)(rows + e / 8 % zeros) * 128u + (e % 8) * 16u, 0u,
                                 0u, 0u, 0u);
                fence_async_shared();
                __syncwarp();
            };
            const uint64_t kK = sw128_desc(base + M::kK, 16, 1024), vK = sw128_desc(base + M::kV, 16, 1024);
            const uint64_t kM = sw128_desc(base + M::kK, kBox, 1024);
            const uint64_t dsK = sw128_desc(base + M::kDS, 16, 1024), dsM = sw128_desc(base + M::kDS, kBox, 1024);
            int tok, head, rows = 0, last_rows = 0;
            if (wait_all(kv_full, 0)) {
                if (keys < 128) {  // keys that are not the sequence's: dQ multiplies their zeros with K
                    for (int e = lane; e < (128 - keys) * 8 * NB; e += 32)
                        st_shared_v4(base + M::kK + (uint32_t)(e / 8 / (128 - keys)) * kBox +
                                         (uint32_t)(keys + e / 8 % (128 - keys)) * 128u + (e % 8) * 16u, 0u, 0u, 0u, 0u);
                    fence_async_shared();
                    __syncwarp();
                }
            }
            auto s_mma = [&](int j) {
                if (!wait_all(q_full(j & 1), (uint32_t)(j / 2) & 1u)) return;
                int r2;
                tile(j, tok, head, r2);
                if (r2 < full_rows) clear(q_smem(j & 1), r2);
                if (leader) {
                    const uint64_t b = sw128_desc(q_smem(j & 1), 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < 4 * NB; ++kk)
                        if (kk < P.ksteps) mma_ss(tS, kK + kstep(kk), b + kstep(kk), P.idesc_s, kk > 0 ? 1u : 0u);
                    mma_commit(s_full);
                }
            };
            auto dk_mma = [&](int j, int r2) {  // dK += dS^T Q
                if (leader) {
                    const int steps = (r2 + 15) / 16;
                    const uint64_t b = sw128_desc(q_smem(j & 1), kBox, 1024);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if (kk < steps) mma_ss(tDK, dsK + kstep(kk), b + (uint64_t)kk * 128, P.idesc_k, (j > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(q_empty(j & 1));
                    mma_commit(ds_free);
                }
            };
            if (ok) s_mma(0);
            for (int j = 0; j < n && ok; ++j) {
                const int s = j & 1;
                const uint32_t ph = (uint32_t)j & 1u;
                last_rows = rows;
                tile(j, tok, head, rows);
                // dP(j): the compute warps have read dP(j - 1), as dS(j - 1) is there
                if (!wait_all(do_full(s), (uint32_t)(j / 2) & 1u)) break;
                if (rows < full_rows) clear(do_smem(s), rows);
                if (leader) {
                    const uint64_t b = sw128_desc(do_smem(s), 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < 4 * NB; ++kk)
                        if (kk < P.ksteps) mma_ss(tDP, vK + kstep(kk), b + kstep(kk), P.idesc_s, kk > 0 ? 1u : 0u);
                    mma_commit(dp_full);
                }
                if (j > 0) dk_mma(j - 1, last_rows);
                // dV += P^T dO: 16 rows a step, those of the second half 64 columns on
                if (!wait_all(p_full, ph)) break;
                if (leader) {
                    const int steps = (rows + 15) / 16;
                    const uint64_t b = sw128_desc(do_smem(s), kBox, 1024);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if (kk < steps)
                            mma_ts(tDV, tS + (kk >> 2) * 64 + (kk & 3) * 8, b + (uint64_t)kk * 128, P.idesc_g, (j > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(do_empty(s));
                }
                // dQ = dS K over S^T and P^T
                if (!wait_all(ds_full, ph)) break;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ss(tS, dsM + (uint64_t)kk * 128, kM + (uint64_t)kk * 128, P.idesc_q, kk > 0 ? 1u : 0u);
                    mma_commit(dq_full);
                }
                if (j + 1 < n) {
                    if (!wait_all(dq_empty, ph)) break;
                    s_mma(j + 1);
                }
            }
            if (ok) dk_mma(n - 1, rows);
            if (!ok && leader) *abort_flag = 1;
            if (leader) mma_commit(fin);
            wait_bar_drain(fin, 0);
            __syncwarp();
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ P and dS
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int half = warp / 4, kr = warp % 4 * 32 + lane;          // rows [64 half, + 64) of a tile; key
        const uint32_t lane_off = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t sA = tS + lane_off + 64u * half, dpA = tDP + lane_off + 64u * half;
        const float f = P.scale_log2e;
        const uint32_t ds_row = base + M::kDS + (uint32_t)half * kBox + (uint32_t)kr * 128u, sw = (uint32_t)kr & 7u;
        for (int j = 0; j < n && ok; ++j) {
            const uint32_t ph = (uint32_t)j & 1u;
            const int s = j & 1;
            int tok, head, rows;
            tile(j, tok, head, rows);
            // the rows that see this key: from `from` on, of those that exist
            const long long from = (long long)(k0 + kr - q.shift - tok) * P.hp;
            const bool edge = rows < 128 || keys < 128 || k0 + 127 > tok + q.shift;
            uint32_t see[2] = {0xffffffffu, 0xffffffffu};
            if (edge) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c0 = 64 * half + 32 * i;
                    const int lo = from <= c0 ? 0 : from >= c0 + 32 ? 32 : (int)from - c0;
                    see[i] = kr < keys ? low_bits(rows - c0) & ~low_bits(lo) : 0u;
                }
            }
            const float4* nl = reinterpret_cast<const float4*>(row_s + s * 256 + 64 * half);
            const float4* nd = nl + 32;
            ok = __all_sync(0xffffffffu, wait(row_full(s), (uint32_t)(j / 2) & 1u, abort_flag, p.status)) &&
                 __all_sync(0xffffffffu, wait(s_full, ph, abort_flag, p.status));
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
            if (ok && j > 0) ok = __all_sync(0xffffffffu, wait(ds_free, (uint32_t)(j - 1) & 1u, abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t dr[32];
                tmem_ld_x32(dpA + 32 * i, dr);
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // eight rows: 16 bytes
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 d = nd[8 * i + 2 * c + e];
                        const int at = 8 * c + 4 * e, pa = 32 * i + at;
                        const float2 x = __fadd2_rn(make_float2(__uint_as_float(dr[at]), __uint_as_float(dr[at + 1])), make_float2(d.x, d.y));
                        const float2 y = __fadd2_rn(make_float2(__uint_as_float(dr[at + 2]), __uint_as_float(dr[at + 3])), make_float2(d.z, d.w));
                        float2 u = __fmul2_rn(x, make_float2(pr[pa], pr[pa + 1]));
                        float2 v = __fmul2_rn(y, make_float2(pr[pa + 2], pr[pa + 3]));
                        if (edge) {  // (dP and delta of a row that is not there may be anything)
                            u.x = (see[i] >> at) & 1u ? u.x : 0.f;
                            u.y = (see[i] >> (at + 1)) & 1u ? u.y : 0.f;
                            v.x = (see[i] >> (at + 2)) & 1u ? v.x : 0.f;
                            v.y = (see[i] >> (at + 3)) & 1u ? v.y : 0.f;
                        }
                        w[2 * e] = pack2<BF16>(u.x, u.y);
                        w[2 * e + 1] = pack2<BF16>(v.x, v.y);
                    }
                    st_shared_v4(ds_row + ((((uint32_t)(4 * i + c)) ^ sw) << 4), w[0], w[1], w[2], w[3]);
                }
            }
            fence_async_shared();
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
            const float by = half ? p.scale : 1.f;
            uint16_t* to = (half ? dk : dv) + (long long)kr * p.Hk * p.D;
            float* acc = P.splits > 1 ? (half ? p.dk_acc : p.dv_acc) + ((long long)(q.k0 + k0 + kr) * p.Hk + h) * p.D : nullptr;
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
                        red_v4(acc + c + e, x[0], x[1], x[2], x[3]);
                        red_v4(acc + c + e + 4, x[4], x[5], x[6], x[7]);
                    } else {
                        *reinterpret_cast<uint4*>(to + c + e) = make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]),
                                                                           pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
                    }
                }
            }
        }
        if (!ok) *abort_flag = 1;
    } else {
        // ------------------------------------------------------------ dQ to memory
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        const int r = warp % 4 * 32 + lane, tok_r = (int)P.fd_hp.div((uint32_t)r), head_r = r - tok_r * P.hp;
        const uint32_t from = tS + ((uint32_t)(warp % 4 * 32) << 16);
        for (int j = 0; j < n && ok; ++j) {
            int tok, head, rows;
            tile(j, tok, head, rows);
            ok = __all_sync(0xffffffffu, wait(dq_full, (uint32_t)j & 1u, abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
            float* to = p.dq_acc + ((long long)(q.q0 + tok + tok_r) * p.Hq + head + head_r) * p.D;
#pragma unroll 1
            for (int c = 0; c < NB * 64; c += 32) {
                uint32_t o[32];
                tmem_ld_x32(from + c, o);
                if (c + 32 >= NB * 64) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(dq_empty);
                }
                if (r < rows) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (c + e < p.D)
                            red_v4(to + c + e, __uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                   __uint_as_float(o[e + 3]));
                }
            }
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

// The fp32 sums as the outputs: dQ times the scale, and dK and dV where several CTAs summed them (their scale is in the
// sums).  Rows past the last sequence are left as they are.
template <bool BF16>
__global__ void __launch_bounds__(256) prompt_bwd_convert(const PromptParams p) {
    const long long nq = (long long)min(max(p.cu_q[p.num_seqs], 0), p.total_q) * p.Hq * (p.D / 8);
    const long long nk = p.dk_acc ? (long long)min(max(p.cu_k[p.num_seqs], 0), p.total_k) * p.Hk * (p.D / 8) : 0;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < nq + 2 * nk; e += (long long)gridDim.x * 256) {
        const float* from;
        uint16_t* to;
        float by = 1.f;
        if (e < nq) {
            from = p.dq_acc + e * 8;
            to = static_cast<uint16_t*>(p.dq) + e * 8;
            by = p.scale;
        } else {
            const long long x = e - nq;
            from = (x < nk ? p.dk_acc : p.dv_acc) + (x < nk ? x : x - nk) * 8;
            to = static_cast<uint16_t*>(x < nk ? p.dk : p.dv) + (x < nk ? x : x - nk) * 8;
        }
        const float4 a = reinterpret_cast<const float4*>(from)[0], b = reinterpret_cast<const float4*>(from)[1];
        *reinterpret_cast<uint4*>(to) = make_uint4(pack2<BF16>(a.x * by, a.y * by), pack2<BF16>(a.z * by, a.w * by),
                                                   pack2<BF16>(b.x * by, b.y * by), pack2<BF16>(b.z * by, b.w * by));
    }
}

template <bool BF16, int NB>
cudaError_t start(const GradParams& P, unsigned grid, cudaStream_t stream) {
    auto kern = prompt_bwd_kernel<BF16, NB>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<NB>::kTotal);
    if (e != cudaSuccess) return e;
    kern<<<grid, kWarps * 32, Smem<NB>::kTotal, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace
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
    GradParams P;
    P.p = p;
    cudaError_t e = p.total_q > 0 ? launch_delta(p, stream) : cudaSuccess;  // (and zeroes the sums)
    if (e != cudaSuccess) return e;
    tile_shape(p.G, P.hp, P.tq);
    P.ng = p.G / P.hp;
    P.splits = p.dk_acc ? prompt_bwd_splits(p.num_seqs, p.total_k, p.max_q, p.max_k, p.Hk, p.G) : 1;
    P.fd_hp = tc::make_fastdiv((uint32_t)P.hp);
    const bool bf16 = p.dtype == TA_BF16;
    const uint32_t ab = bf16 ? 1u : 0u, nd = (uint32_t)(p.D + 15) / 16 * 16;
    auto idesc = [&](uint32_t N, uint32_t a_mn, uint32_t b_mn) {
        return (1u << 4) | (ab << 7) | (ab << 10) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | (8u << 24);
    };
    P.idesc_s = idesc(128, 0, 0);
    P.idesc_g = idesc(nd, 0, 1);
    P.idesc_k = idesc(nd, 0, 1);
    P.idesc_q = idesc(nd, 1, 1);
    P.ksteps = (p.D + 15) / 16;
    P.scale_log2e = p.scale * kToLog2;
    const CUtensorMapDataType dt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t D = (uint64_t)p.D;
    const long long per = (long long)p.num_seqs * p.Hk * P.splits, grid = per * ((p.max_k + 127) / 128);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (grid > 0) {
        if (!tc::encode_map_3d(&P.tm_q, dt, p.q, D, p.Hq, p.total_q > 0 ? p.total_q : 1, D * 2, p.q_rs * 2, 64, P.hp, P.tq, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !tc::encode_map_3d(&P.tm_do, dt, p.d_out, D, p.Hq, p.total_q > 0 ? p.total_q : 1, D * 2, D * 2 * p.Hq, 64, P.hp, P.tq, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !tc::encode_map_3d(&P.tm_k, dt, p.k, D, p.Hk, p.total_k, D * 2, p.k_rs * 2, 64, 1, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !tc::encode_map_3d(&P.tm_v, dt, p.v, D, p.Hk, p.total_k, D * 2, p.v_rs * 2, 64, 1, 128, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
        if (p.D <= 64) e = bf16 ? start<true, 1>(P, (unsigned)grid, stream) : start<false, 1>(P, (unsigned)grid, stream);
        else e = bf16 ? start<true, 2>(P, (unsigned)grid, stream) : start<false, 2>(P, (unsigned)grid, stream);
        if (e != cudaSuccess) return e;
    }
    const long long pieces = ((long long)p.total_q * p.Hq + (p.dk_acc ? 2LL * p.total_k * p.Hk : 0)) * (p.D / 8);
    if (pieces == 0) return cudaSuccess;
    const long long blocks = (pieces + 255) / 256 < 152 * 16 ? (pieces + 255) / 256 : 152 * 16;
    if (bf16) prompt_bwd_convert<true><<<(unsigned)blocks, 256, 0, stream>>>(p);
    else prompt_bwd_convert<false><<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace triattn
