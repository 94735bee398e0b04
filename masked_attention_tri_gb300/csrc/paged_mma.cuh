// paged_mma.cuh -- attention over a paged cache for 16-bit queries on tensor cores:
// the kernel template (instantiated per cache type in paged_mma_*.cu, launched from
// paged_mma.cu).  The split of the work and the treatment of the scales stand in paged.cuh.
//
// Bound: memory.  Each visible byte of K and V is read once, and a new token brings
// only its few grouped heads to multiply it with: 4 G FLOPs a byte in 8 bits, 2 G in 16.
// Eight query rows are one n8 operand, so mma.sync takes K (16 slots) and V^T (16 columns) as
// its A operand with no row of padding for G = 8; a tcgen05 tile has 128 rows and would carry
// 8.  The kernel therefore aims to keep loads in flight: one producer warp fills a ring of
// stages (a tile of K and of V each, up to 190 KB) by TMA, 128-byte swizzled; the consumer
// warps take blocks of 16 slots, each with a running maximum, sum and O of its own, and
// merge once at the unit's end.  No warp waits for another within a unit.  A warp takes half
// a stage at a time where there are plenty, or a block or two where the share holds few tiles
// and the time of one tile on one warp would be what counts.  The loop over blocks is not
// unrolled further than two: that code fits the instruction cache of a cold start.  Where a
// unit ends the producer is already loading the next one's first tiles, and its queries are in registers.
//
// Measured from a cold L2, 32 heads over 8 of 128, pages of 64: 64 sequences of 1k to 16k slots in 8 bits
// 208 us (5.5 TB/s; the copies alone 198, the arithmetic alone 175), in 16 bits 355 us (6.4 TB/s); 256
// sequences of 256 to 1024 slots in 8 bits 118 us, of which 79 are waits, set-up and merges of the 14 units
// that a CTA has there.  64 query heads 216 us.
//
//   S^T = K Q^T      A: slots x d from shared memory, B: Q^T, kept in fragment order
//   O^T += V^T P^T   A: d x slots; P^T comes from S^T's accumulators by movmatrix
//
// 8-bit codes become fp16 on the way, by cvt.rn.f16x2.e4m3x2 (exact): the ALU's two operations a clock an
// SM are the kernel's second bound.  (mma.sync takes e4m3 operands itself, but on this GPU each such
// product is ten instructions more: the conversions again, for every use.)  Queries of an 8-bit
// cache are fp16 scaled by a power of two, their row's largest magnitude in [1, 2): exact down to 2^-14 of it
// and off by 2^-25 of it below.
//
// Fragments.  K (and 16-bit V, transposed) by ldmatrix, whose four matrices are an A operand's four
// registers as they stand; of 8-bit K a matrix holds 16 columns, a lane's four codes are two pairs, and
// k index 2t, 2t + 1, 2t + 8, 2t + 9 of a product stands for columns 4t to 4t + 3.  8-bit V^T: lane
// (g, t) = (lane / 4, lane % 4) reads eight columns of four slots and pairs the slots' bytes by prmt.  The 16 rows of K's operand may be any slots: row g is slot pi(g)
// (and row g + 8 slot pi(g) + 8), pi(2i) = 2i, pi(2i + 1) = (2i ^ 4) + 1, so that the lanes' slots of V
// are 0, 2, 4, 6 and 5, 7, 1, 3 in turn, whose swizzled reads meet no bank twice.
//
// Roundings: P to the products' 16-bit type (fp16 for 8-bit caches: 2^-12 of a weight),
// as everywhere in this library; S, the maxima, sums and O are fp32.  O is rescaled only
// when a logit passes the reference by 2^8 (base 2: by 8), which fp16's range allows.
#pragma once

#include <atomic>

#include "paged.cuh"
#include "tc_kernel.cuh"

namespace triattn {
namespace paged {

using tc::ex2;
using tc::mbar_arrive;
using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::pack2;
using tc::smem_u32;
using tc::wait_bar;

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};
template <int M>
struct Blocks {
    static constexpr int value = M;
};

constexpr uint32_t kMmaSmem = 232448 - 1024 - 256;  // 227 KB less the alignment of the ring and the static part

// What the producer tells of a stage; sc[i]: key scale, log2 and reciprocal of the value scale of the i-th
// page in it (written as one 16-byte store).
struct alignas(16) StageMeta {
    float4 sc[8];
    uint32_t valid;                  // bit b: slots [16 b, 16 b + 16) were loaded
    int key0;
    int use;                         // how often the stage has been given out, less one
    int pad;
};

struct MmaParams {
    CUtensorMap tm_k, tm_v;
    PagedParams p;
};

// TYPE: 0 fp16 cache, 1 bf16 cache, 2 e4m3 codes.  NDC: 64-column chunks of D.  NT: groups of eight rows.
template <int TYPE, int NDC, int NT>
struct MmaConfig {
    static constexpr bool kCodes = TYPE == 2;
    static constexpr int kBoxes = kCodes ? (NDC + 1) / 2 : NDC;         // 128-byte columns of a tile
    static constexpr int kSlots = 128 / kBoxes;                         // slots of a stage: 32 KB, K and V
    static constexpr uint32_t kBoxBytes = kSlots * 128;
    static constexpr uint32_t kStage = 2 * kBoxes * kBoxBytes;          // K boxes, then V boxes
    static constexpr int kRows = NT * 8;
    // Consumers: with the producer eight warps, so that a thread may have 255 registers (O alone takes 16 NDC
    // NT).  Measured on 64 sequences of 1k to 16k slots in 8 bits (before the warps took two blocks at once):
    // 7 warps 226 us, 11 warps 257, 15 warps 275: the more warps work on stages at a time, the fewer stages
    // are left for copies in flight.
    static constexpr int kWarps = 7;
    static constexpr int kThreads = (kWarps + 1) * 32;
    // Merge buffers: one for each warp where the ring keeps its six stages, else four taken in two turns.
    static constexpr int kBufs = NT * NDC <= 2 ? kWarps : 4;
    static constexpr int kOStride = NDC * 64 + 4;                       // floats of a merged row
    static constexpr uint32_t kQ = NDC * NT * 1024;  // Q in fragment order
    static constexpr uint32_t kO = (uint32_t)kBufs * kRows * kOStride * 4;
    static constexpr uint32_t kFixed = kQ + kO + kWarps * kRows * 8 + kRows * 8 + kRows * 4 + 16 * 16;
    static constexpr int kFit = (int)((kMmaSmem - kFixed) / (kStage + sizeof(StageMeta)));
    static constexpr int kStages = kFit > 12 ? 12 : kFit;
    static constexpr uint32_t kSmem = kStages * (kStage + (uint32_t)sizeof(StageMeta)) + kFixed + 1024;
    static_assert(kStages >= 2, "two stages at least");
};

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm_x4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Two e4m3 codes (low byte first) as fp16.
__device__ __forceinline__ uint32_t codes_f16(uint32_t two) {
    uint32_t y;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(y) : "r"(two));
    return y;
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t two) {
    uint32_t y;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(y) : "r"(two));
    return y;
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
// Slot (within eight) of row i of an A operand.
__device__ __forceinline__ int pi8(int i) { return (i & 1) ? ((i - 1) ^ 4) + 1 : i; }

// Waits until use `use` of a stage has arrived.  A parity wait alone can tell only two neighbouring
// uses apart, and warps run free: one may ask for a use while the one before it is still in
// flight.  So the producer's count is awaited first: once it says `use`, the use before it has
// arrived and been read.  Bounded like wait_bar.
static __device__ __noinline__ bool wait_use_slow(const volatile int* count, int use, volatile int* abort_flag,
                                                  int* status) {
    const long long t0 = clock64();
    for (uint32_t it = 1; *count != use; ++it) {
        if (*abort_flag) return false;
        if ((it & 63) == 0 && clock64() - t0 > tc::kTimeoutCycles) {
            *abort_flag = 1;
            atomicCAS(status, 0, kStatusTimeout);
            return false;
        }
        __nanosleep(32);
    }
    return true;
}
__device__ __forceinline__ bool wait_stage(const volatile int* count, int use, uint32_t bar, volatile int* abort_flag,
                                           int* status) {
    return (*count == use || wait_use_slow(count, use, abort_flag, status)) &&
           wait_bar(bar, (uint32_t)use & 1u, abort_flag, status);
}

template <int TYPE, int NDC, int NT>
__global__ void __launch_bounds__(MmaConfig<TYPE, NDC, NT>::kThreads, 1) paged_mma_kernel(const __grid_constant__ MmaParams P) {
    using C = MmaConfig<TYPE, NDC, NT>;
    constexpr bool kBF16 = TYPE == 1;
    constexpr bool kCodes = C::kCodes;
    constexpr int kBlocks = C::kSlots / 16;
    constexpr int kWarps = C::kWarps;
    const PagedParams& p = P.p;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* g0 = smem_raw + (base - raw);
    // ring, metadata, merge buffers, Q, (m, l) by warp, (M, L) by row, query factors, barriers
    const uint32_t ring = base;
    StageMeta* meta = reinterpret_cast<StageMeta*>(g0 + C::kStages * C::kStage);
    float* so = reinterpret_cast<float*>(meta + C::kStages);
    uint8_t* sq = reinterpret_cast<uint8_t*>(so + C::kBufs * C::kRows * C::kOStride);
    float2* sml = reinterpret_cast<float2*>(sq + C::kQ);
    float2* srow = sml + kWarps * C::kRows;
    float* sqf = reinterpret_cast<float*>(srow + C::kRows);
    const uint32_t bars = smem_u32(sqf + C::kRows);
    __shared__ long long scan[kWarps + 1], found[2];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    auto full = [&](int s) { return bars + 16u * (uint32_t)s; };
    auto empty = [&](int s) { return bars + 16u * (uint32_t)s + 8u; };
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up meanwhile

    if (threadIdx.x == 0) {
        abort_word = 0;
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kBlocks);  // one arrival a block
            meta[s].use = -1;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    const Workspace ws = workspace(p.ws, p.RT, p.D);
    const Share sh = find_share<C::kThreads>(p, C::kBoxes, scan, found);  // (not below 128 slots; synchronizes the block)
    if (threadIdx.x == 0) ws.join[blockIdx.x].parts = 0;
    Walk w = walk_begin(p, sh);
    Unit u;

    if (warp == kWarps) {
        // ------------------------------------------------------------ producer
        const int span = min(p.page, C::kSlots);      // slots of one load
        const int nb = C::kSlots / span;               // pages of a tile
        // Tiles of one batch: each has nb lanes of its own, which look its pages up, wait for its stage and
        // start its copies, all tiles of a batch at once (a loop over the tiles would cost the
        // warp some 600 clocks each, about the memory's time for one).  No more than the ring
        // has stages, so that the tiles of a batch are uses of different stages.
        const int per = min(32 / nb, C::kStages);
        constexpr int nbox = C::kBoxes;                // (a box past D is all zeros and reads nothing)
        const int mysub = lane % nb, mytile = lane / nb;
        const int blocks = span / 16;                  // blocks of 16 slots of one load
        const uint32_t bytes = (uint32_t)(2 * nbox * span * 128);
        int slot0 = 0, turn0 = 0;                      // the next stage and how often the ring has gone round
        bool ok = true;
        // The next batch: unit u, tiles from jb.  Its table entries and scales are loaded while the batch before it
        // is given out (the last of one unit while the first of the next is looked up), and not
        // looked at before they are needed.
        int jb = 0, j_end = 0, key_n = 0, page_n = -1;
        bool need_n = false;
        float ks_n = 1.f, vs_n = 1.f;
        auto next_batch = [&]() -> bool {
            jb += per;
            while (jb >= j_end) {
                if (!walk_next(p, w, u)) return false;
                jb = u.j0;
                j_end = min(u.j1, u.t.nt);
            }
            // the entry of this lane's part of tile jb + mytile (-1: not needed)
            const int j = mytile < per ? jb + mytile : j_end;
            key_n = j < j_end ? u.t.tile(j) * C::kSlots + mysub * span : 0;
            need_n = j < j_end && key_n <= u.t.p1 &&
                     (p.window <= 0 || (long long)u.t.p0 - (key_n + span - 1) < p.window || key_n < p.sinks);
            page_n = need_n ? p.table[(long long)u.seq * p.max_pages + key_n / p.page] : -1;
            return true;
        };
        auto check_and_scale = [&]() {
            if (need_n && (page_n < 0 || page_n >= p.num_pages)) {
                atomicCAS(p.status, 0, kStatusDevice);
                page_n = -1;
            }
            if (kCodes && page_n >= 0) {
                ks_n = p.k_scale[(long long)page_n * p.Hk + u.h];
                vs_n = p.v_scale[(long long)page_n * p.Hk + u.h];
            }
        };
        bool have = next_batch();
        if (have) check_and_scale();
        while (have) {
            // What each lane's tile needs, made ready for all of them at once.
            const bool v_ok = !kCodes || page_n < 0 || v_scale_ok(vs_n);  // (else its slots are not seen)
            if (!v_ok) atomicCAS(p.status, 0, kStatusDevice);
            const int page = v_ok ? page_n : -1, key = key_n, h = u.h;
            const float4 sc = kCodes ? make_float4(ks_n, log2f(vs_n), 1.f / vs_n, 0.f) : make_float4(1.f, 0.f, 1.f, 0.f);
            uint32_t valid = page >= 0 ? ((1u << blocks) - 1u) << (mysub * blocks) : 0u;
            int loads = page >= 0 ? 1 : 0;
            for (int o = 1; o < nb; o <<= 1) {  // over the lanes of the tile
                valid |= __shfl_xor_sync(0xffffffffu, valid, o);
                loads += __shfl_xor_sync(0xffffffffu, loads, o);
            }
            const int in_page = key % p.page;
            const int todo = min(per, j_end - jb);
            const int slot = slot0 + mytile < C::kStages ? slot0 + mytile : slot0 + mytile - C::kStages;
            const int turn = slot0 + mytile < C::kStages ? turn0 : turn0 + 1;
            bool wait = mytile < todo, looked = false, checked = false;
            // (bounded: after a wait that ran out every tile is given out empty and the CTA runs to its end)
            while (__any_sync(0xffffffffu, wait)) {
                // tiles whose stage has been read (the lanes of a tile go by their first)
                bool go = wait && (turn == 0 || !ok || tc::mbar_test(empty(slot), (uint32_t)(turn - 1) & 1u));
                go = __shfl_sync(0xffffffffu, go, lane - mysub);
                StageMeta& mt = meta[slot];
                if (go) {
                    if (kCodes) mt.sc[mysub] = sc;
                    if (mysub == 0)
                        tc::st_shared_v4(smem_u32(&mt.valid), ok ? valid : 0u, (uint32_t)key, (uint32_t)turn, 0u);
                }
                __syncwarp();
                if (go && mysub == 0) mbar_expect_tx(full(slot), ok ? (uint32_t)loads * bytes : 0u);
                __syncwarp();
                if (go && page >= 0 && ok) {
                    const uint32_t dst = ring + (uint32_t)slot * C::kStage + (uint32_t)(mysub * span) * 128u;
                    for (int b = 0; b < nbox; ++b) {
                        const int x = b * 64;  // (16-bit units)
                        tc::tma_load_4d(dst + b * C::kBoxBytes, &P.tm_k, x, in_page, h, page, full(slot));
                        tc::tma_load_4d(dst + (C::kBoxes + b) * C::kBoxBytes, &P.tm_v, x, in_page, h, page, full(slot));
                    }
                }
                wait = wait && !go;
                if (!looked) {
                    looked = true;
                    have = next_batch();
                } else if (!checked) {
                    checked = true;
                    if (have) check_and_scale();
                } else if (!__any_sync(0xffffffffu, go) && ok) {  // none: sleep until the first of them has been read
                    const int first = __ffs(__ballot_sync(0xffffffffu, wait)) - 1;
                    const uint32_t bar = __shfl_sync(0xffffffffu, empty(slot), first);
                    const int use = __shfl_sync(0xffffffffu, turn, first);
                    ok = __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)(use - 1) & 1u, abort_flag, p.status));
                }
            }
            if (!checked && have) check_and_scale();
            slot0 += todo;
            if (slot0 >= C::kStages) {
                slot0 -= C::kStages;
                ++turn0;
            }
        }
        if (*abort_flag && lane == 0) {  // copies in flight end before the CTA does
            for (int i = 0; i < 2000; ++i) __nanosleep(1000);
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    auto consumers_sync = [] { tc::named_barrier(1, kWarps * 32); };
    const int g = lane / 4, t = lane % 4;
    const int sub_shift = p.page >= C::kSlots ? 3 : __ffs(p.page) - 5;  // log2 of a page's blocks (in a stage)
    const uint32_t rg = (uint32_t)pi8(g);                      // slot (of eight) of this lane's rows of K
    const uint32_t r0 = 2u * t, r1 = (r0 ^ 4u) + 1u;           // slots (of eight) of this lane's columns of V^T
    // Byte offsets in a block of 16 swizzled rows: this lane's row address of K's loads (matrices: slots
    // 0-7, slots 8-15, the same 16 bytes further; the next 32 bytes at ^ 32), 8-bit V's words of
    // columns g (rows r0, r1; the upper 64 columns at ^ 64), 16-bit V's rows of the transposing load
    // (16 columns further at ^ 32).
    const uint32_t k_row = (uint32_t)pi8(lane & 7) + ((lane & 8) ? 8u : 0u);
    const uint32_t k_off = k_row * 128u + ((((uint32_t)lane >> 4) ^ (k_row & 7u)) << 4);
    const uint32_t v_off0 = r0 * 128u + (((uint32_t)(g >> 1) ^ r0) << 4) + (g & 1) * 8u;
    const uint32_t v_off1 = r1 * 128u + (((uint32_t)(g >> 1) ^ r1) << 4) + (g & 1) * 8u;
    const uint32_t v_row = (uint32_t)pi8(lane & 7) + ((lane & 16) ? 8u : 0u);
    const uint32_t v_offt = v_row * 128u + ((((uint32_t)lane >> 3 & 1u) ^ (v_row & 7u)) << 4);
    // Reference of a row that has seen no key: below the logits of any finite bf16 rows whose sums fp32 holds (far above
    // it a difference from it overflows to an infinity, which is a new maximum like any other).
    constexpr float kNone = -3e38f;
    uint32_t idx = 0;
    bool ok = true;
    long long at = sh.begin;
    // Q of a unit: warp w takes rows w, w + kWarps, ...  Loaded a unit ahead, so that its latency passes
    // behind the tiles; lane l holds elements [4 l, 4 l + 4) and, for D > 128, 128 further on.
    constexpr int kQRows = (C::kRows + kWarps - 1) / kWarps, kQPieces = (NDC + 1) / 2;
    uint2 xq[kQRows][kQPieces];
    auto fetch_q = [&](const Unit& v) {
#pragma unroll
        for (int i = 0; i < kQRows; ++i) {
            const int r = warp + i * kWarps, row = v.rt * C::kRows + r;
            const bool there = r < C::kRows && row < v.q.n * p.G;
            const uint16_t* qp = static_cast<const uint16_t*>(p.q);
            if (there) qp += (long long)(v.q.row0 + row / p.G) * p.q_rs + ((long long)v.h * p.G + row % p.G) * p.D;
#pragma unroll
            for (int c = 0; c < kQPieces; ++c) {
                const int d = c * 128 + lane * 4;
                xq[i][c] = there && d < p.D ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0u, 0u);
            }
        }
    };
    // ... and into shared memory in fragment order.
    auto put_q = [&]() {
#pragma unroll
        for (int i = 0; i < kQRows; ++i) {
            const int r = warp + i * kWarps;
            if (r >= C::kRows) break;
            float factor = p.scale_log2e;
            uint2 (&x)[kQPieces] = xq[i];
            if constexpr (kCodes) {
                const bool bf = p.dtype == TA_BF16;
                float y[kQPieces][4];
                uint32_t most = 0;
#pragma unroll
                for (int c = 0; c < kQPieces; ++c) {
                    const float2 a = bf ? tc::unpack2<true>(x[c].x) : tc::unpack2<false>(x[c].x);
                    const float2 b = bf ? tc::unpack2<true>(x[c].y) : tc::unpack2<false>(x[c].y);
                    y[c][0] = a.x, y[c][1] = a.y, y[c][2] = b.x, y[c][3] = b.y;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t e = __float_as_uint(y[c][k]) & 0x7fffffffu;
                        if (e < 0x7f800000u) most = max(most, e);
                    }
                }
                // the exponent of the largest finite element, and the factor that makes it 0
                uint32_t ex = __reduce_max_sync(0xffffffffu, most) >> 23;
                ex = ex < 1 ? 1u : (ex > 253 ? 253u : ex);
                const float up = __uint_as_float((254u - ex) << 23);
                factor *= __uint_as_float(ex << 23);
#pragma unroll
                for (int c = 0; c < kQPieces; ++c) {
                    x[c].x = pack2<false>(y[c][0] * up, y[c][1] * up);
                    x[c].y = pack2<false>(y[c][2] * up, y[c][3] * up);
                }
            }
#pragma unroll
            for (int c = 0; c < kQPieces; ++c) {
                const int d = c * 128 + lane * 4, ch = d / 64, in = d % 64;
                if (ch >= NDC) continue;
                uint8_t* dst = sq + ((ch * 4 + in / 16) * NT + r / 8) * 256 + (r % 8) * 32;
                if constexpr (kCodes) {
                    *reinterpret_cast<uint2*>(dst + (in % 16) / 4 * 8) = x[c];
                } else {
                    dst += (in % 8) / 2 * 8 + (in % 16) / 8 * 4;
                    *reinterpret_cast<uint32_t*>(dst) = x[c].x;
                    *reinterpret_cast<uint32_t*>(dst + 8) = x[c].y;
                }
            }
            if (lane == 0) sqf[r] = factor;
        }
    };
    Unit un;
    bool have = walk_next(p, w, un);
    if (have) fetch_q(un);
    while (have) {
        u = un;
        const long long head0 = (long long)u.h * p.G;
        const int total_rows = u.q.n * p.G, row_first = u.rt * C::kRows;
        put_q();
        // ---- This lane's columns of S^T and O^T: rows nt * 8 + 2 t and the next.
        int pos[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                pos[nt][e] = u.q.len - u.q.n + min(row_first + nt * 8 + 2 * t + e, total_rows - 1) / p.G;
        consumers_sync();
        float qf[NT][2], m[NT][2], l[NT][2], o[NDC * 4][NT][4];  // m: the reference maximum
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qf[nt][e] = sqf[nt * 8 + 2 * t + e];
                m[nt][e] = kNone;
                l[nt][e] = 0.f;
            }
#pragma unroll
        for (int i = 0; i < NDC * 4; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
        // Q stays in registers where it is small.
        constexpr int kSteps = NDC * 4;   // k-steps of 16 columns
        constexpr bool kKeepQ = kSteps * NT <= 8;
        uint2 qr[kKeepQ ? kSteps * NT : 1];
        if constexpr (kKeepQ) {
#pragma unroll
            for (int i = 0; i < kSteps * NT; ++i) qr[i] = *reinterpret_cast<const uint2*>(sq + i * 256 + lane * 8);
        }

        have = walk_next(p, w, un);
        if (have) fetch_q(un);

        const int tiles = max(0, min(u.j1, u.t.nt) - u.j0);
        // Blocks that a warp takes at a time: half a stage's (twelve such pieces in a ring of six), or
        // fewer where that leaves warps without work: two (whose products overlap), or one.
        constexpr int kTake = kBlocks / 2;
        const int blocks = tiles * kBlocks;
        const int take = blocks >= 2 * kWarps * kTake ? kTake : (kTake >= 2 && blocks >= 2 * kWarps ? 2 : 1);
        const int grains = tiles * kBlocks / take;
        for (int gr = warp; gr < grains; gr += kWarps) {
            const int b_first = (gr * take) % kBlocks;
            const uint32_t it = idx + (uint32_t)(gr * take / kBlocks);
            const int slot = (int)(it % C::kStages);
            if (ok)
                ok = __all_sync(0xffffffffu, wait_stage(&meta[slot].use, (int)(it / C::kStages), full(slot), abort_flag,
                                                        p.status));
            const StageMeta& mt = meta[slot];
            const uint32_t valid = mt.valid;
            const int stage_key0 = mt.key0;
            // every row sees every slot of the stage
            const bool plain_stage = valid == (1u << kBlocks) - 1u && stage_key0 + C::kSlots - 1 <= u.t.p0 &&
                                     (p.window <= 0 || u.t.p1 - stage_key0 < p.window || stage_key0 + C::kSlots <= p.sinks);
            const uint32_t stage = ring + (uint32_t)slot * C::kStage;
            // M blocks at once: S^T, the softmax step, O^T.  PLAIN: every row sees every slot of them.
            auto block = [&](auto plain_tag, auto m_tag, int blk) {
                constexpr bool PLAIN = decltype(plain_tag)::value;
                constexpr int M = decltype(m_tag)::value;
                const uint32_t kb = stage + (uint32_t)blk * 2048u, vb = kb + C::kBoxes * C::kBoxBytes;
                const int key0 = stage_key0 + blk * 16;
                if constexpr (!PLAIN) {
                    // Slots that no row sees may hold anything: their V is made 0 in the stage (their weight is 0,
                    // but 0 times NaN is not).
                    if (!unit_sees(p, u.t, key0 + lane / 2)) {
                        for (int b = 0; b < C::kBoxes; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                tc::st_shared_v4(vb + b * C::kBoxBytes + (uint32_t)(lane / 2) * 128u + (lane & 1) * 64u + i * 16u,
                                                 0u, 0u, 0u, 0u);
                    }
                    tc::fence_async_shared();  // before the stage is filled again
                    __syncwarp();
                }

                // ---- S^T
                float s[M][NT][4];
#pragma unroll
                for (int mb = 0; mb < M; ++mb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mb][nt][e] = 0.f;
                auto step = [&](int mb, int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint2 b;
                        if constexpr (kKeepQ) b = qr[i * NT + nt];
                        else b = *reinterpret_cast<const uint2*>(sq + (i * NT + nt) * 256 + lane * 8);
                        mma16816<kBF16>(s[mb][nt], a0, a1, a2, a3, b);
                    }
                };
                // (32 bytes of a row at a time: 16 columns, or 32 codes)
#pragma unroll
                for (int i = 0; i < (kCodes ? kSteps / 2 : kSteps); ++i) {
#pragma unroll
                    for (int mb = 0; mb < M; ++mb) {
                        uint32_t a[4];
                        ldsm_x4(kb + mb * 2048u + (k_off ^ (32u * (i & 3))) + (i / 4) * C::kBoxBytes, a);
                        if constexpr (kCodes) {
                            step(mb, 2 * i, codes_f16(a[0]), codes_f16(a[1]), codes_f16_hi(a[0]), codes_f16_hi(a[1]));
                            step(mb, 2 * i + 1, codes_f16(a[2]), codes_f16(a[3]), codes_f16_hi(a[2]), codes_f16_hi(a[3]));
                        } else {
                            step(mb, i, a[0], a[1], a[2], a[3]);
                        }
                    }
                }
                // ---- Logits in base 2 (with the value scale's log2) less the reference: y = x - m.
                float4 sc[M];
#pragma unroll
                for (int mb = 0; mb < M; ++mb)
                    sc[mb] = kCodes ? mt.sc[(blk + mb) >> sub_shift] : make_float4(1.f, 0.f, 1.f, 0.f);
                float y[M][NT][4];
                auto factor = [&](int mb, int nt, int e) { return kCodes ? qf[nt][e] * sc[mb].x : qf[nt][e]; };
                bool grew = false;
#pragma unroll
                for (int mb = 0; mb < M; ++mb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float f = factor(mb, nt, e), d = sc[mb].y - m[nt][e];
                            y[mb][nt][e] = fmaf(s[mb][nt][e], f, d);
                            y[mb][nt][e + 2] = fmaf(s[mb][nt][e + 2], f, d);
                        }
                if constexpr (!PLAIN) {
#pragma unroll
                    for (int mb = 0; mb < M; ++mb)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!sees(p, pos[nt][e & 1], key0 + mb * 16 + (int)rg + (e & 2) * 4))
                                    y[mb][nt][e] = -INFINITY;
                }
#pragma unroll
                for (int mb = 0; mb < M; ++mb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) grew = grew || fmaxf(y[mb][nt][e], y[mb][nt][e + 2]) > 8.f;
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float al[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // (the reference may be far off: x is formed from s again)
                            float x = -INFINITY;
#pragma unroll
                            for (int mb = 0; mb < M; ++mb)
#pragma unroll
                                for (int k = e; k < 4; k += 2) {
                                    if (y[mb][nt][k] != -INFINITY) y[mb][nt][k] = fmaf(s[mb][nt][k], factor(mb, nt, e), sc[mb].y);
                                    x = fmaxf(x, y[mb][nt][k]);
                                }
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                            x = fmaxf(m[nt][e], x);
                            al[e] = ex2(m[nt][e] - x);
                            m[nt][e] = x;
                            l[nt][e] *= al[e];
#pragma unroll
                            for (int mb = 0; mb < M; ++mb) {
                                y[mb][nt][e] -= x;
                                y[mb][nt][e + 2] -= x;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < NDC * 4; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[i][nt][e] *= al[e & 1];
                    }
                }
                // ---- P^T as the B operand, and O^T += V^T P^T.
                uint2 b[M][NT];
#pragma unroll
                for (int mb = 0; mb < M; ++mb)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float pr[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pr[e] = ex2(y[mb][nt][e]);
                            if constexpr (kCodes) l[nt][e & 1] = fmaf(pr[e], sc[mb].z, l[nt][e & 1]);
                            else l[nt][e & 1] += pr[e];
                        }
                        b[mb][nt].x = transpose8(pack2<kBF16>(pr[0], pr[1]));
                        b[mb][nt].y = transpose8(pack2<kBF16>(pr[2], pr[3]));
                    }
#pragma unroll
                for (int mb = 0; mb < M; ++mb)
#pragma unroll
                    for (int c = 0; c < NDC; ++c) {
                        const uint32_t vc = vb + mb * 2048u;
                        if constexpr (kCodes) {
                            const uint32_t a0 = vc + (v_off0 ^ (64u * (c & 1))) + (c / 2) * C::kBoxBytes;
                            const uint32_t a1 = vc + (v_off1 ^ (64u * (c & 1))) + (c / 2) * C::kBoxBytes;
                            const uint2 w0 = lds64(a0), w1 = lds64(a1), w2 = lds64(a0 + 1024u), w3 = lds64(a1 + 1024u);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const uint32_t sel = (h & 1) ? 0x7362u : 0x5140u;
                                const uint32_t x = __byte_perm(h < 2 ? w0.x : w0.y, h < 2 ? w1.x : w1.y, sel);
                                const uint32_t z = __byte_perm(h < 2 ? w2.x : w2.y, h < 2 ? w3.x : w3.y, sel);
                                const uint32_t f0 = codes_f16(x), f1 = codes_f16_hi(x), f2 = codes_f16(z),
                                               f3 = codes_f16_hi(z);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816<false>(o[c * 4 + h][nt], f0, f1, f2, f3, b[mb][nt]);
                            }
                        } else {
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                uint32_t a[4];
                                ldsm_x4_t(vc + (v_offt ^ (32u * h)) + c * C::kBoxBytes, a);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816<kBF16>(o[c * 4 + h][nt], a[0], a[1], a[2], a[3], b[mb][nt]);
                            }
                        }
                    }
            };
            if (plain_stage) {
                // (two at a time where a warp has several: the one's products fill the other's waits)
                constexpr int M = kTake >= 2 && NT <= 2 ? 2 : 1;
                if (M == 1 || take == 1) {
#pragma unroll 1
                    for (int blk = b_first; blk < b_first + take; ++blk) block(Yes{}, Blocks<1>{}, blk);
                } else {
#pragma unroll 1
                    for (int blk = b_first; blk < b_first + take; blk += M) block(Yes{}, Blocks<M>{}, blk);
                }
            } else {
#pragma unroll 1
                for (int blk = b_first; blk < b_first + take; ++blk) {
                    const int key0 = stage_key0 + blk * 16;
                    // (a block that was not loaded, or that no row sees, is passed over)
                    if (((valid >> blk) & 1u) && key0 <= u.t.p1 &&
                        (p.window <= 0 || (long long)u.t.p0 - (key0 + 15) < p.window || key0 < p.sinks))
                        block(No{}, Blocks<1>{}, blk);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_n(empty(slot), (uint32_t)take);
        }
        idx += (uint32_t)tiles;

        // ---- Merge: (m, l) of the warps, then their O over the buffers (the last warps first, the others on top).
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0)
                    sml[warp * C::kRows + nt * 8 + 2 * t + e] = make_float2(m[nt][e] == kNone ? -INFINITY : m[nt][e], x);
            }
        consumers_sync();
        float f[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * t + e;
                float M = -INFINITY;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sml[i * C::kRows + r].x);
                const float2 mine = sml[warp * C::kRows + r];
                f[nt][e] = no_key(mine.x, mine.y) ? 0.f : ex2(mine.x - M);
            }
        if (threadIdx.x < C::kRows) {
            const int r = threadIdx.x;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sml[i * C::kRows + r].x);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 ml = sml[i * C::kRows + r];
                if (!no_key(ml.x, ml.y)) L = fmaf(ml.y, ex2(ml.x - M), L);
            }
            srow[r] = make_float2(M, L);
        }
        // element e of accumulator i2, nt: row nt * 8 + 2 t + (e & 1), column 64 c + 8 g + 2 h + (e >> 1) of 8-bit V,
        // 64 c + 16 h + g + 8 (e >> 1) of 16-bit V (c = i2 / 4, h = i2 % 4)
#pragma unroll 1
        for (int turn = (kWarps - 1) / C::kBufs; turn >= 0; --turn) {
            if (warp / C::kBufs == turn) {
                float* dst = so + (warp % C::kBufs) * C::kRows * C::kOStride;
                const bool first = warp + C::kBufs >= kWarps;  // of the warps that share the buffer
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float* row = dst + (nt * 8 + 2 * t + e) * C::kOStride;
                        const float ff = f[nt][e];
                        if constexpr (kCodes) {  // eight neighbouring columns a chunk
#pragma unroll
                            for (int i2 = 0; i2 < NDC * 4; i2 += 2) {
                                float4* q = reinterpret_cast<float4*>(row + (i2 / 4) * 64 + g * 8 + (i2 % 4) * 2);
                                float4 v = make_float4(o[i2][nt][e] * ff, o[i2][nt][e + 2] * ff, o[i2 + 1][nt][e] * ff,
                                                       o[i2 + 1][nt][e + 2] * ff);
                                if (!first) {
                                    const float4 x = *q;
                                    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                                }
                                *q = v;
                            }
                        } else {
#pragma unroll
                            for (int i2 = 0; i2 < NDC * 4; ++i2)
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    float* q = row + (i2 / 4) * 64 + 16 * (i2 % 4) + g + 8 * k;
                                    const float v = o[i2][nt][e + 2 * k] * ff;
                                    *q = first ? v : *q + v;
                                }
                        }
                    }
            }
            consumers_sync();
        }
        const bool whole = u.starts && u.ends;
        const int slot = u.starts ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
        const int D4 = p.D / 4;
        for (int e = threadIdx.x; e < u.rows * D4; e += kWarps * 32) {
            const int r = e / D4, d = (e - r * D4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < C::kBufs; ++i) {
                const float4 y = *reinterpret_cast<const float4*>(so + (i * C::kRows + r) * C::kOStride + d);
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
            }
            const float2 ML = srow[r];
            if (whole) {
                const int row = row_first + r;
                const long long tok = u.q.row0 + row / p.G, head = head0 + row % p.G;
                const float inv = no_key(ML.x, ML.y) ? 0.f : 1.f / ML.y;
                const bool bf = p.dtype == TA_BF16;
                uint2 v;
                v.x = bf ? pack2<true>(x.x * inv, x.y * inv) : pack2<false>(x.x * inv, x.y * inv);
                v.y = bf ? pack2<true>(x.z * inv, x.w * inv) : pack2<false>(x.z * inv, x.w * inv);
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (tok * p.Hq + head) * p.D + d) = v;
                if (d == 0 && p.lse) p.lse[head * p.total_q + tok] = row_lse(ML.x, ML.y);
            } else {
                *reinterpret_cast<float4*>(ws.o + ((long long)slot * p.RT + r) * p.D + d) = x;
                if (d == 0) ws.ml[slot * p.RT + r] = ML;
            }
        }
        if (u.starts && !u.ends && threadIdx.x == 0) {
            Join& jn = ws.join[blockIdx.x];
            jn.seq_row0 = u.q.row0;
            jn.h = u.h;
            jn.row0 = row_first;
            jn.rows = u.rows;
            jn.parts = unit_parts(sh, u, at);
        }
        at += u.j1 - u.j0;
    }
}

template <int TYPE, int NDC, int NT>
cudaError_t launch_mma_variant(const MmaParams& P, cudaStream_t stream) {
    using C = MmaConfig<TYPE, NDC, NT>;
    auto kern = paged_mma_kernel<TYPE, NDC, NT>;
    // The shared-memory limit is set once per device (an attribute call costs as much as a launch).
    static std::atomic<unsigned long long> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev > 63 || !(set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    kern<<<kGrid, C::kThreads, C::kSmem, stream>>>(P);
    return cudaGetLastError();
}

#define TRIATTN_PAGED_VARIANTS(X, T) X(T, 1, 1) X(T, 1, 2) X(T, 1, 4) X(T, 2, 1) X(T, 2, 2) X(T, 4, 1) X(T, 4, 2)
#define TRIATTN_PAGED_EXTERN(t, d, n) \
    extern template cudaError_t launch_mma_variant<t, d, n>(const MmaParams&, cudaStream_t);
#define TRIATTN_PAGED_INSTANTIATE(t, d, n) \
    template cudaError_t launch_mma_variant<t, d, n>(const MmaParams&, cudaStream_t);

}  // namespace paged
}  // namespace triattn
