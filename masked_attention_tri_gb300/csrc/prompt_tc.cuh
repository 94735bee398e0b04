// prompt_tc.cuh -- what the tensor-core kernels of prompt attention share: tiles of rows, the order in which CTAs take them,
// bounded waits.
#pragma once

#include <atomic>

#include "prompt.cuh"
#include "tc_kernel.cuh"

namespace triattn {
namespace prompt {

using namespace tc;

// Tiles of 128 rows: tq tokens x hp heads of a group (both powers of two), ng tiles of the same tokens (G / hp).
struct Tiles {
    int hp, tq, ng;
    FastDiv fd_hp;
};
Tiles make_tiles(const PromptParams& p);

// A kernel's shared-memory limit, set once per device (an attribute call costs a part of a launch).
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    static std::atomic<unsigned long long> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev <= 63 && (set.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_release);
    return e;
}

// wait_bar inline: a call keeps the compiler from giving a kernel's warps the registers that setmaxnreg gives them.
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

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Products issued by one thread.  A descriptor is its low word (start and leading offset; the high word is the same for all
// tiles here: a stride of 1024 bytes, 128-byte swizzle), so that a step to the next 16 of K is one addition, and a thread that
// runs its loop alone waits for no other lane: the thread that feeds the tensor core has 64 clocks for a product of 128 x 128
// x 16.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | (lbo >> 4 << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ void issue_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(add ? 1u : 0u), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b), "r"(idesc), "r"(add ? 1u : 0u), "n"(kDescHi)
        : "memory");
}
// D = A B^T, A and B tiles of NB boxes of 64 columns in shared memory; `ksteps` sixteens of columns.
template <int NB>
__device__ __forceinline__ void issue_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int ksteps) {
    if (ksteps == 4 * NB) {
#pragma unroll
        for (int kk = 0; kk < 4 * NB; ++kk) {
            const uint32_t s = ((uint32_t)(kk >> 2) * kBox + (uint32_t)(kk & 3) * 32u) >> 4;
            issue_ss(d, a + s, b + s, idesc, kk > 0);
        }
    } else {
#pragma unroll 1
        for (int kk = 0; kk < ksteps; ++kk) {
            const uint32_t s = ((uint32_t)(kk >> 2) * kBox + (uint32_t)(kk & 3) * 32u) >> 4;
            issue_ss(d, a + s, b + s, idesc, kk > 0);
        }
    }
}
// D += A B, A: rows x up to 128 of K in tensor memory, the second 64 of K `HALF` columns on; B: those rows of a tile in
// shared memory. Sixteens [from, to) of K, of `steps` that there are.
template <int HALF>
__device__ __forceinline__ void issue_cols(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int from, int to, int steps, bool fresh) {
    if (steps == 8) {
#pragma unroll
        for (int kk = from; kk < to; ++kk)
            issue_ts(d, a + (uint32_t)((kk >> 2) * HALF + (kk & 3) * 8), b + (uint32_t)kk * 128u, idesc, !fresh || kk > 0);
    } else {
#pragma unroll 1
        for (int kk = from; kk < min(to, steps); ++kk)
            issue_ts(d, a + (uint32_t)((kk >> 2) * HALF + (kk & 3) * 8), b + (uint32_t)kk * 128u, idesc, !fresh || kk > 0);
    }
}

// dS of rows that see up to so many keys is two 16-bit numbers, the second the rest of the first's rounding (prompt_dq.cu).
constexpr int kFineKeys = 512;
template <int N>
struct Count {
    static constexpr int value = N;
};
// fp16 operands of the gradients are held times a power of two, which their products' fp32 sums are divided by exactly: the
// least step of fp16 is 2^-24, and with thousands of keys and the dO of a mean loss (1e-4) dS = P (dP - delta) lies below it.
// P, at most 1, is held times 2^14.  |dP - delta| <= |dO| |V| + |delta|: dS times 2^e is below 2^15 with e = 14 - floor(log2 of
// that bound), for the row itself in dQ, for the largest of the sequence's rows of a key head in dK, whose sums run over rows.
// bf16 has fp32's exponents and needs neither.
constexpr int kHalfP = 14;
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }  // -126 to 127
__device__ __forceinline__ int half_exponent(float bound) {
    const int e = 14 + 127 - (int)(__float_as_uint(bound) >> 23 & 255u);
    return min(max(e, -100), 100);
}
template <bool BF16>
__device__ __forceinline__ uint32_t rest2(float2 x, uint32_t rounded) {
    const float2 y = unpack2<BF16>(rounded);
    return pack2<BF16>(x.x - y.x, x.y - y.y);
}

// An item: PER tiles of one (sequence, key head).
template <int PER>
struct alignas(16) Item {
    int on;                    // 0: the end
    int q0, k0, lq, shift;     // the sequence: first packed rows, queries, and how many more keys than queries it has
    int seq, h;                // the sequence's number, key head
    int tok[PER], head[PER];     // of each tile: first token (of the sequence), first query head
    int keys[PER];             // keys that some row of the tile sees
    int rows[PER];             // rows that exist (0: no tile)
};

// The next block's place in the grid, or -1 (none is left): asks (one thread), and reads the answer.
__device__ __forceinline__ void clc_ask(uint32_t to, uint32_t bar) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    mbar_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to),
                 "r"(bar)
                 : "memory");
}
__device__ __forceinline__ int clc_answer(uint32_t at) {
    int x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 r, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "mov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n\t}"
        : "=r"(x)
        : "r"(at)
        : "memory");
    return x;
}

// The sequences to a warp (prompt_order.h), a lane each.
struct WarpSeqs {
    const PromptParams& p;
    __device__ __forceinline__ int n() const { return p.num_seqs; }
    __device__ __forceinline__ Seq at(int s) const { return load_seq(p, s, false); }
    template <typename F>
    __device__ __forceinline__ int of_lane(int s0, F f, int none) const {
        const int s = s0 + threadIdx.x % 32;
        return s < p.num_seqs ? f(at(s)) : none;
    }
    template <typename F>
    __device__ __forceinline__ int sum(int s0, F f) const {
        return __reduce_add_sync(0xffffffffu, of_lane(s0, f, 0));
    }
    template <typename F>
    __device__ __forceinline__ int most(int s0, F f) const {
        return __reduce_max_sync(0xffffffffu, of_lane(s0, f, -1));
    }
    template <typename F>
    __device__ __forceinline__ bool find(int s0, F f, int& place, int& s) const {
        const int c = of_lane(s0, f, 0);
        int upto = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (threadIdx.x % 32 >= d) upto += x;
        }
        const uint32_t has = __ballot_sync(0xffffffffu, place < upto);
        if (!has) {
            place -= __shfl_sync(0xffffffffu, upto, 31);
            return false;
        }
        const int l = __ffs((int)has) - 1;
        place -= __shfl_sync(0xffffffffu, upto - c, l);
        s = s0 + l;
        return true;
    }
};
// Item `at` of the order: false past the last.
template <int PER>
__device__ __forceinline__ bool order_item(const PromptParams& p, const Tiles& T, Order<PER>& o, long long at, Item<PER>& it) {
    const WarpSeqs seqs{p};
    int n = 0;
    if (!o.locate(seqs, at, it.seq, n, it.h)) return false;
    const Seq q = seqs.at(it.seq);
    it.on = 1;
    it.q0 = q.q0;
    it.k0 = q.k0;
    it.lq = q.lq;
    it.shift = q.shift;
    const int blocks = (it.lq + T.tq - 1) / T.tq;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int t = PER * n + i, b = t / T.ng;
        const bool there = b < blocks;
        it.tok[i] = b * T.tq;
        it.head[i] = it.h * p.G + (t - b * T.ng) * T.hp;
        const int tokens = there ? min(T.tq, it.lq - it.tok[i]) : 0;
        it.rows[i] = tokens * T.hp;
        it.keys[i] = there ? max(0, it.tok[i] + tokens + it.shift) : 0;
    }
    return true;
}
// The warp that hands the items to `consumers` warps through a ring of R: items in shared memory, barriers full(r) (1) and
// empty(r) (consumers), the answer's place and barrier.  False after a wait that ran out.
template <int PER, int R, typename Full, typename Empty>
__device__ __forceinline__ bool hand_out(const PromptParams& p, const Tiles& T, Item<PER>* items, Full full, Empty empty,
                                         uint32_t clc_at, uint32_t clc_bar, volatile int* abort_flag) {
    const int lane = threadIdx.x % 32;
    Order<PER> o;
    o.begin(WarpSeqs{p}, __ffs(T.tq) - 1, T.ng, p.Hk);
    int at = (int)blockIdx.x;
    uint32_t asked = 0;
    // (awaited whatever happens: the answer is written into this block's memory)
    auto next = [&]() -> bool {
        if (lane == 0) clc_ask(clc_at, clc_bar);
        if (!__all_sync(0xffffffffu, wait_bar_drain(clc_bar, asked++ & 1u))) return false;
        at = clc_answer(clc_at);
        __syncwarp();
        return true;
    };
    for (int n = 0;; ++n) {
        Item<PER> it{};
        // A place without an item is passed over and the next one asked for, so that the rest of the grid need not start to
        // learn that (up to 4096 of them, some milliseconds: the others wait for this item with a limit).
        for (int over = 0; at >= 0 && !order_item<PER>(p, T, o, at, it); ++over) {
            if (over == 4096) at = -1;
            else if (!next()) return false;
        }
        const int r = n % R;
        if (n >= R && !__all_sync(0xffffffffu, wait(empty(r), (uint32_t)(n / R - 1) & 1u, abort_flag, p.status))) return false;
        if (lane == 0) {
            items[r] = it;
            mbar_arrive(full(r));
        }
        if (!it.on) break;
        if (!next()) return false;
    }
    if (blockIdx.x == 0)
        for (int s = lane; s < p.num_seqs; s += 32) load_seq(p, s, true);  // (records a broken sequence)
    return true;
}
// Blocks of the grid: one for each item that there can be.  A sequence has ceil(ceil(lq / tq) ng / PER) items, at most
// lq ng / (PER tq) + (ng + PER - 1) / PER, and no more than the longest has.
inline long long most_items(const PromptParams& p, const Tiles& T, int PER) {
    const long long longest = (((long long)p.max_q + T.tq - 1) / T.tq * T.ng + PER - 1) / PER;
    const long long sum = (long long)p.total_q * T.ng / (PER * T.tq) + (long long)p.num_seqs * ((T.ng + PER - 1) / PER) + 1;
    return (longest * p.num_seqs < sum ? longest * p.num_seqs : sum) * p.Hk;
}

// Zeros into rows [from, to) of a tile of NB boxes (a warp), for the async proxy to read.
template <int NB>
__device__ __forceinline__ void clear_rows(uint32_t tile, int from, int to) {
    const int n = to - from;
    if (n <= 0) return;
    for (int e = threadIdx.x % 32; e < n * 8 * NB; e += 32)
        st_shared_v4(tile + (uint32_t)(e / 8 / n) * kBox + (uint32_t)(from + e / 8 % n) * 128u + (e % 8) * 16u, 0u, 0u, 0u, 0u);
    fence_async_shared();
    __syncwarp();
}

// Instruction descriptors (tc_bwd.cu has the fields); N may be left out and added later.
inline uint32_t make_idesc(bool bf16, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
    const uint32_t ab = bf16 ? 1u : 0u;
    return (1u << 4) | (ab << 7) | (ab << 10) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | (8u << 24);
}
// A map of packed rows (total, heads, D): boxes of 64 columns x heads x tokens.
inline bool make_rows_map(CUtensorMap* m, bool bf16, const void* ptr, int D, int heads, int total, long long rs, int box_heads,
                          int box_rows) {
    return encode_map_3d(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ptr, (uint64_t)D,
                         (uint64_t)heads, (uint64_t)(total > 0 ? total : 1), (uint64_t)D * 2, (uint64_t)rs * 2, 64,
                         (uint32_t)box_heads, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace prompt
}  // namespace triattn
