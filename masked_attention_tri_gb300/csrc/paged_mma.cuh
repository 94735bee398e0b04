// paged_mma.cuh -- attention over a paged cache for 16-bit queries on tensor cores:
// the kernel template (instantiated per cache type in paged_mma_*.cu, launched from
// paged_mma.cu).  The split of the work and the treatment of the scales stand in paged.cuh.
//
// Bound: memory.  Each visible byte of K and V is read once, and a new token brings
// only its few grouped heads to multiply it with: 4 G FLOPs a byte in 8 bits, 2 G in 16.
// Eight query rows are one n8 operand, so mma.sync m16n8k16 takes K (16 slots) and V^T
// (16 columns) as its A operand with no row of padding for G = 8; a tcgen05 tile has 128
// rows and would carry 8.  The kernel therefore aims to keep loads in flight:
// one producer warp fills a ring of stages (a tile of K and of V each, up to 190 KB) by TMA,
// 128-byte swizzled; seven consumer warps take the stages in turn, each with a running
// maximum, sum and O of its own, and merge once at the unit's end.  No warp waits for
// another within a unit.
//
//   S^T = K Q^T   A: slots x d from shared memory, B: Q^T, kept in fragment order
//   O^T += V^T P^T   A: d x slots; P^T comes from S^T's accumulators by movmatrix
//
// Fragments straight from the swizzled rows.  A product's k index may be permuted if both
// operands agree, and the 16 rows of A may be any slots (or columns of V).  So lane (g, t)
// = (lane / 4, lane % 4) reads whole 16-byte pieces: row g of K's A operand is slot pi(g),
// pi(2i) = 2i, pi(2i + 1) = (2i ^ 4) + 1, which makes every shared-memory read below
// free of bank conflicts: 8 lanes of K's reads meet rows whose bit 2 differs, and
// V's reads four rows 0, 2, 4, 6 or 5, 7, 1, 3.  8-bit codes go to fp16 by
// cvt.rn.f16x2.e4m3x2 (exact); pairs of slots of V^T are put together by prmt first.
//
// Roundings: P to the products' 16-bit type (fp16 for 8-bit caches: 2^-12 of a weight),
// as everywhere in this library; S, the maxima, sums and O are fp32.  bf16 queries of an
// 8-bit cache become fp16 scaled by a power of two to [1, 2) at their row's largest magnitude: exact
// down to 2^-14 of it, off by 2^-25 of it below.
#pragma once

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

// Consumers: with the producer eight warps, two on each of the SM's four register files, so that a
// thread may have 255 registers (a ninth warp would leave it 168: the wider variants would spill).
constexpr int kMmaWarps = 7;
constexpr int kMmaThreads = (kMmaWarps + 1) * 32;   // and the producer
constexpr int kMmaMinTiles = 4;
constexpr uint32_t kMmaSmem = 232448 - 1024 - 256;  // 227 KB less the alignment of the ring and the static part

struct StageMeta {
    float ks[4], vlog2[4], vinv[4];  // by 16 slots: key scale, log2 and reciprocal of the value scale
    uint32_t valid;                  // bit b: slots [16 b, 16 b + 16) were loaded
    int key0;
    int pad[2];
};

struct MmaParams {
    CUtensorMap tm_k, tm_v;
    PagedParams p;
};

// TYPE: 0 fp16 cache, 1 bf16 cache, 2 e4m3 codes.  NDC: 64-column chunks of D.  NT: groups of eight rows.
template <int TYPE, int NDC, int NT>
struct MmaConfig {
    static constexpr int kSlots = TYPE != 2 && NDC == 4 ? 32 : 64;      // slots of a stage
    static constexpr int kBoxes = TYPE == 2 ? (NDC + 1) / 2 : NDC;      // 128-byte columns of a tile
    static constexpr uint32_t kBoxBytes = kSlots * 128;
    static constexpr uint32_t kStage = 2 * kBoxes * kBoxBytes;          // K boxes, then V boxes
    static constexpr int kRows = NT * 8;
    static constexpr int kOStride = NDC * 64 + 4;                       // floats of a merged row
    static constexpr uint32_t kQ = NDC * 4 * NT * 32 * 8;               // Q in fragment order
    static constexpr uint32_t kO = 4u * kRows * kOStride * 4;           // merge buffers
    static constexpr uint32_t kFixed = kQ + kO + kMmaWarps * kRows * 8 + kRows * 8 + kRows * 4 + 16 * 16;
    static constexpr int kFit = (int)((kMmaSmem - kFixed) / (kStage + sizeof(StageMeta)));
    static constexpr int kStages = kFit > 12 ? 12 : kFit;
    static constexpr uint32_t kSmem = kStages * (kStage + (uint32_t)sizeof(StageMeta)) + kFixed + 1024;
    static_assert(kStages >= 2, "two stages at least");
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
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

__device__ __forceinline__ void consumers_sync() { tc::named_barrier(1, kMmaWarps * 32); }

template <int TYPE, int NDC, int NT>
__global__ void __launch_bounds__(kMmaThreads, 1) paged_mma_kernel(const __grid_constant__ MmaParams P) {
    using C = MmaConfig<TYPE, NDC, NT>;
    constexpr bool kBF16 = TYPE == 1;
    constexpr int kMT = C::kSlots / 16;
    const PagedParams& p = P.p;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* g0 = smem_raw + (base - raw);
    // ring, metadata, merge buffers, Q, (m, l) by warp, (M, L) by row, query factors, barriers
    const uint32_t ring = base;
    StageMeta* meta = reinterpret_cast<StageMeta*>(g0 + C::kStages * C::kStage);
    float* so = reinterpret_cast<float*>(meta + C::kStages);
    uint2* sq = reinterpret_cast<uint2*>(so + 4 * C::kRows * C::kOStride);
    float2* sml = reinterpret_cast<float2*>(sq + NDC * 4 * NT * 32);
    float2* srow = sml + kMmaWarps * C::kRows;
    float* sqf = reinterpret_cast<float*>(srow + C::kRows);
    const uint32_t bars = smem_u32(sqf + C::kRows);
    __shared__ long long scan[kMmaThreads / 32], found[2];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    auto full = [&](int s) { return bars + 16u * (uint32_t)s; };
    auto empty = [&](int s) { return bars + 16u * (uint32_t)s + 8u; };
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        abort_word = 0;
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    const Workspace ws = workspace(p.ws, p.RT, p.D);
    const Share sh = find_share<kMmaThreads>(p, kMmaMinTiles, scan, found);  // (synchronizes the block)
    if (threadIdx.x == 0) ws.join[blockIdx.x].parts = 0;
    Walk w = walk_begin(p, sh);
    Unit u;

    if (warp == kMmaWarps) {
        // ------------------------------------------------------------ producer
        const int span = min(p.page, C::kSlots);      // slots of one load
        const int nb = C::kSlots / span;               // pages of a tile
        const int per = 32 / nb;                       // tiles whose pages the lanes look up at once
        const int nbox = TYPE == 2 ? (p.D + 127) / 128 : (p.D + 63) / 64;
        const int mysub = lane % nb, mytile = lane / nb;
        uint32_t idx = 0;                              // stages filled so far
        bool ok = true;
        while (walk_next(p, w, u)) {
            const int j_end = min(u.j1, u.t.nt);
            const int32_t* row = p.table + (long long)u.seq * p.max_pages;
            // the page of this lane's part of tile jb + mytile: -1 not needed, -2 out of range
            auto look = [&](int jb, int& key) -> int {
                const int j = jb + mytile;
                key = 0;
                if (j >= j_end) return -1;
                key = u.t.tile(j) * C::kSlots + mysub * span;
                const bool need = key <= u.t.p1 && (p.window <= 0 || (long long)u.t.p0 - (key + span - 1) < p.window ||
                                                    key < p.sinks);
                if (!need) return -1;
                const int page = row[key / p.page];
                return page >= 0 && page < p.num_pages ? page : -2;
            };
            int key_n, page_n = look(u.j0, key_n);
            float ks_n = 1.f, vs_n = 1.f;
            auto look_scales = [&]() {
                if (TYPE == 2 && page_n >= 0) {
                    ks_n = p.k_scale[(long long)page_n * p.Hk + u.h];
                    vs_n = p.v_scale[(long long)page_n * p.Hk + u.h];
                }
            };
            look_scales();
            for (int jb = u.j0; jb < j_end; jb += per) {
                const int page = page_n, key = key_n;
                const float ks = ks_n, vs = vs_n;
                if (page == -2) atomicCAS(p.status, 0, kStatusDevice);
                page_n = look(jb + per, key_n);
                const int todo = min(per, j_end - jb);
                for (int i = 0; i < todo; ++i) {
                    if (i == todo / 2) look_scales();
                    const int slot = idx % C::kStages;
                    const uint32_t turn = idx / C::kStages;
                    if (turn > 0 && ok)
                        ok = __all_sync(0xffffffffu, wait_bar(empty(slot), (turn - 1) & 1u, abort_flag, p.status));
                    const bool load = ok && mytile == i && page >= 0;
                    const int blocks = span / 16;
                    const uint32_t bits = load ? ((1u << blocks) - 1u) << (mysub * blocks) : 0u;
                    const uint32_t valid = __reduce_or_sync(0xffffffffu, bits);
                    const int loads = __popc(__ballot_sync(0xffffffffu, load));
                    if (TYPE == 2 && load) {
                        for (int b = 0; b < blocks; ++b) {
                            meta[slot].ks[mysub * blocks + b] = ks;
                            meta[slot].vlog2[mysub * blocks + b] = log2f(vs);
                            meta[slot].vinv[mysub * blocks + b] = 1.f / vs;
                        }
                    }
                    if (lane == 0) {
                        meta[slot].valid = valid;
                        meta[slot].key0 = u.t.tile(jb + i) * C::kSlots;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_expect_tx(full(slot), (uint32_t)(loads * 2 * nbox * span * 128));
                    __syncwarp();
                    if (load) {
                        const uint32_t dst = ring + (uint32_t)slot * C::kStage + (uint32_t)(mysub * span) * 128u;
                        for (int b = 0; b < nbox; ++b) {
                            const int x = b * (TYPE == 2 ? 128 : 64);
                            tc::tma_load_4d(dst + b * C::kBoxBytes, &P.tm_k, x, key % p.page, u.h, page, full(slot));
                            tc::tma_load_4d(dst + (C::kBoxes + b) * C::kBoxBytes, &P.tm_v, x, key % p.page, u.h, page,
                                            full(slot));
                        }
                    }
                    ++idx;
                }
            }
        }
        if (*abort_flag && lane == 0) {  // copies in flight end before the CTA does
            for (int i = 0; i < 2000; ++i) __nanosleep(1000);
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int g = lane / 4, t = lane % 4;
    const int nch = (p.D + 63) / 64;
    const uint32_t rg = (uint32_t)pi8(g);                      // slot (of eight) of this lane's rows of K
    const uint32_t k_row = rg * 128u;
    const uint32_t r0 = 2u * t, r1 = (r0 ^ 4u) + 1u;           // slots (of eight) of this lane's columns of V^T
    // 16-bit V: this lane's row address of the transposing load
    const uint32_t vrow = (uint32_t)pi8(lane & 7) + ((lane & 16) ? 8u : 0u);
    uint32_t idx = 0;
    bool ok = true;
    long long at = sh.begin;
    while (walk_next(p, w, u)) {
        const long long head0 = (long long)u.h * p.G;
        const int total_rows = u.q.n * p.G, row_first = u.rt * C::kRows;
        // ---- Q of the unit, in fragment order: warp w takes rows w, w + kMmaWarps, ...
        for (int r = warp; r < C::kRows; r += kMmaWarps) {
            const int row = row_first + r;
            const bool there = row < total_rows;
            const uint16_t* qp = static_cast<const uint16_t*>(p.q);
            if (there) qp += (long long)(u.q.row0 + row / p.G) * p.q_rs + (head0 + row % p.G) * p.D;
            float factor = p.scale_log2e;
            // lane l holds elements [4 l, 4 l + 4) and, for D > 128, 128 further on
            uint2 x[(NDC + 1) / 2];
#pragma unroll
            for (int c = 0; c < (NDC + 1) / 2; ++c) {
                const int d = c * 128 + lane * 4;
                x[c] = there && d < p.D ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0u, 0u);
            }
            if (TYPE == 2 && p.dtype == TA_BF16) {
                uint32_t most = 0;
#pragma unroll
                for (int c = 0; c < (NDC + 1) / 2; ++c) {
                    const uint32_t e[4] = {x[c].x & 0x7fffu, (x[c].x >> 16) & 0x7fffu, x[c].y & 0x7fffu,
                                           (x[c].y >> 16) & 0x7fffu};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e[i] < 0x7f80u) most = max(most, e[i]);
                }
                most = __reduce_max_sync(0xffffffffu, most) >> 7;  // the exponent of the largest finite element
                const uint32_t ex = most < 2 ? 2u : (most > 252 ? 252u : most);
                const float down = __uint_as_float((254u - ex) << 23);  // 2^(127 - ex)
                factor *= __uint_as_float(ex << 23);
#pragma unroll
                for (int c = 0; c < (NDC + 1) / 2; ++c) {
                    const float2 a = tc::unpack2<true>(x[c].x), b = tc::unpack2<true>(x[c].y);
                    x[c].x = pack2<false>(a.x * down, a.y * down);
                    x[c].y = pack2<false>(b.x * down, b.y * down);
                }
            }
#pragma unroll
            for (int c = 0; c < (NDC + 1) / 2; ++c) {
                const int d = c * 128 + lane * 4, ch = d / 64, in = d % 64;
                // four consecutive elements are one k-step's share of lane (row, t)
                const int ks = TYPE == 2 ? (in % 16) / 4 : (in / 32) * 2 + (in % 8) / 4;
                const int tt = TYPE == 2 ? in / 16 : (in % 32) / 8;
                if (ch < NDC) sq[((ch * 4 + ks) * NT + r / 8) * 32 + (r % 8) * 4 + tt] = x[c];
            }
            if (lane == 0) sqf[r] = factor;
        }
        // ---- This lane's columns of S^T and O^T: rows nt * 8 + 2 t and the next.
        int pos[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                pos[nt][e] = u.q.len - u.q.n + min(row_first + nt * 8 + 2 * t + e, total_rows - 1) / p.G;
        consumers_sync();
        float qf[NT][2], m[NT][2], l[NT][2], o[NDC * 4][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qf[nt][e] = sqf[nt * 8 + 2 * t + e];
                m[nt][e] = -INFINITY;
                l[nt][e] = 0.f;
            }
#pragma unroll
        for (int i = 0; i < NDC * 4; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;

        const int tiles = max(0, min(u.j1, u.t.nt) - u.j0);
        // stage idx + i goes to warp (idx + i) % kMmaWarps
        for (int i = (int)((uint32_t)(warp + kMmaWarps - (idx % kMmaWarps)) % kMmaWarps); i < tiles; i += kMmaWarps) {
            const uint32_t it = idx + (uint32_t)i;
            const int slot = (int)(it % C::kStages);
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(full(slot), (it / C::kStages) & 1u, abort_flag, p.status));
            const StageMeta& mt_ = meta[slot];
            const int key0 = mt_.key0;
            const uint32_t valid = mt_.valid;
            const uint32_t kb = ring + (uint32_t)slot * C::kStage, vb = kb + C::kBoxes * C::kBoxBytes;

            // ---- S^T
            float s[kMT][NT][4];
#pragma unroll
            for (int i2 = 0; i2 < kMT; ++i2)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i2][nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < NDC; ++c) {
                if (c >= nch) break;
                uint2 b[4][NT];
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) b[ks][nt] = sq[((c * 4 + ks) * NT + nt) * 32 + lane];
#pragma unroll
                for (int i2 = 0; i2 < kMT; ++i2) {
                    if constexpr (TYPE == 2) {
                        const uint32_t a = kb + (c / 2) * C::kBoxBytes + i2 * 2048u + k_row +
                                           (((uint32_t)t + 4u * (c & 1)) ^ rg) * 16u;
                        const uint4 x = lds128(a), y = lds128(a + 1024u);
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint32_t a0 = codes_f16(xw[ks]), a2 = codes_f16_hi(xw[ks]);
                            const uint32_t a1 = codes_f16(yw[ks]), a3 = codes_f16_hi(yw[ks]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816<false>(s[i2][nt], a0, a1, a2, a3, b[ks][nt]);
                        }
                    } else {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t a = kb + c * C::kBoxBytes + i2 * 2048u + k_row +
                                               (((uint32_t)t + 4u * hf) ^ rg) * 16u;
                            const uint4 x = lds128(a), y = lds128(a + 1024u);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816<kBF16>(s[i2][nt], x.x, y.x, x.y, y.y, b[2 * hf][nt]);
                                mma16816<kBF16>(s[i2][nt], x.z, y.z, x.w, y.w, b[2 * hf + 1][nt]);
                            }
                        }
                    }
                }
            }
            // ---- Logits in base 2 (with the value scale's log2), masks, the tile's maxima.
            const bool plain = valid == (1u << kMT) - 1u && key0 + C::kSlots - 1 <= u.t.p0 &&
                               (p.window <= 0 || u.t.p1 - key0 < p.window || key0 + C::kSlots <= p.sinks);
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
            for (int i2 = 0; i2 < kMT; ++i2) {
                const float ks = TYPE == 2 ? mt_.ks[i2] : 1.f, vl = TYPE == 2 ? mt_.vlog2[i2] : 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[i2][nt][e];
                        if constexpr (TYPE == 2) x = fmaf(x, qf[nt][e & 1] * ks, vl);
                        else x *= qf[nt][e & 1];
                        if (!plain) {
                            const int key = key0 + i2 * 16 + (int)rg + (e & 2) * 4;
                            if (!((valid >> i2) & 1u) || !sees(p, pos[nt][e & 1], key)) x = -INFINITY;
                        }
                        s[i2][nt][e] = x;
                        mx[nt][e & 1] = fmaxf(mx[nt][e & 1], x);
                    }
            }
            bool grew = false;
            float mn[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = mx[nt][e];
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    mn[nt][e] = fmaxf(m[nt][e], x);
                    grew = grew || mn[nt][e] > m[nt][e];
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float al[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        al[e] = mn[nt][e] == -INFINITY ? 1.f : ex2(m[nt][e] - mn[nt][e]);
                        m[nt][e] = mn[nt][e];
                        l[nt][e] *= al[e];
                    }
#pragma unroll
                    for (int i2 = 0; i2 < NDC * 4; ++i2)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[i2][nt][e] *= al[e & 1];
                }
            }
            // ---- P^T as the B operand, and O^T += V^T P^T, 16 slots at a time.
#pragma unroll
            for (int i2 = 0; i2 < kMT; ++i2) {
                uint2 b[NT];
                // (the scales of slots that were not loaded are whatever an earlier stage left)
                const float vi = TYPE != 2 ? 1.f : ((valid >> i2) & 1u) ? mt_.vinv[i2] : 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float pr[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float ref = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
                        pr[e] = ex2(s[i2][nt][e] - ref);
                        l[nt][e & 1] = fmaf(pr[e], vi, l[nt][e & 1]);
                    }
                    b[nt].x = transpose8(pack2<kBF16>(pr[0], pr[1]));
                    b[nt].y = transpose8(pack2<kBF16>(pr[2], pr[3]));
                }
                // Slots that no row sees may hold anything: their V is taken as 0.
                uint32_t k01 = 0xffffffffu, k23 = 0xffffffffu;  // halves: slots r0, r1; r0 + 8, r1 + 8
                if (!plain) {
                    const int k = key0 + i2 * 16;
                    const bool in = (valid >> i2) & 1u;
                    k01 = (in && unit_sees(p, u.t, k + (int)r0) ? 0xffffu : 0u) |
                          (in && unit_sees(p, u.t, k + (int)r1) ? 0xffff0000u : 0u);
                    k23 = (in && unit_sees(p, u.t, k + (int)r0 + 8) ? 0xffffu : 0u) |
                          (in && unit_sees(p, u.t, k + (int)r1 + 8) ? 0xffff0000u : 0u);
                }
#pragma unroll
                for (int c = 0; c < NDC; ++c) {
                    if (c >= nch) break;
                    if constexpr (TYPE == 2) {
                        const uint32_t vbox = vb + (c / 2) * C::kBoxBytes + i2 * 2048u + (g & 1) * 8u;
                        const uint32_t col = (uint32_t)(c & 1) * 4u + (uint32_t)(g >> 1);
                        const uint32_t a0 = vbox + r0 * 128u + (col ^ r0) * 16u, a1 = vbox + r1 * 128u + (col ^ r1) * 16u;
                        const uint2 w0 = lds64(a0), w1 = lds64(a1), w2 = lds64(a0 + 1024u), w3 = lds64(a1 + 1024u);
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const uint32_t sel = (h & 1) ? 0x7362u : 0x5140u;
                            const uint32_t x = __byte_perm(h < 2 ? w0.x : w0.y, h < 2 ? w1.x : w1.y, sel);
                            const uint32_t y = __byte_perm(h < 2 ? w2.x : w2.y, h < 2 ? w3.x : w3.y, sel);
                            uint32_t f0 = codes_f16(x), f1 = codes_f16_hi(x), f2 = codes_f16(y), f3 = codes_f16_hi(y);
                            if (!plain) {
                                f0 &= k01;
                                f1 &= k01;
                                f2 &= k23;
                                f3 &= k23;
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[c * 4 + h][nt], f0, f1, f2, f3, b[nt]);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            uint32_t f[4];
                            const uint32_t col = 2u * h + ((lane >> 3) & 1);
                            ldsm_x4_t(vb + c * C::kBoxBytes + i2 * 2048u + vrow * 128u + ((col ^ (vrow & 7u)) * 16u), f);
                            if (!plain) {
                                f[0] &= k01;
                                f[1] &= k01;
                                f[2] &= k23;
                                f[3] &= k23;
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<kBF16>(o[c * 4 + h][nt], f[0], f[1], f[2], f[3], b[nt]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(slot));
        }
        idx += (uint32_t)tiles;

        // ---- Merge: (m, l) of the warps, then their O over four buffers (warps 4.. first, warps 0..3 on top).
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) sml[warp * C::kRows + nt * 8 + 2 * t + e] = make_float2(m[nt][e], x);
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
                for (int i = 0; i < kMmaWarps; ++i) M = fmaxf(M, sml[i * C::kRows + r].x);
                const float2 mine = sml[warp * C::kRows + r];
                f[nt][e] = no_key(mine.x, mine.y) ? 0.f : ex2(mine.x - M);
            }
        if (threadIdx.x < C::kRows) {
            const int r = threadIdx.x;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int i = 0; i < kMmaWarps; ++i) M = fmaxf(M, sml[i * C::kRows + r].x);
#pragma unroll
            for (int i = 0; i < kMmaWarps; ++i) {
                const float2 ml = sml[i * C::kRows + r];
                if (!no_key(ml.x, ml.y)) L = fmaf(ml.y, ex2(ml.x - M), L);
            }
            srow[r] = make_float2(M, L);
        }
        // element (d, row) of accumulator i2, nt: 8-bit d = 64 c + 8 g + 2 h (+ 1), 16-bit d = 64 c + 16 h + g (+ 8)
        auto place = [&](int i2, int e) {
            const int c = i2 / 4, h = i2 % 4;
            return TYPE == 2 ? c * 64 + g * 8 + 2 * h + (e >> 1) : c * 64 + 16 * h + g + 8 * (e >> 1);
        };
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
            if (warp / 4 == half) {
                float* dst = so + (warp % 4) * C::kRows * C::kOStride;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i2 = 0; i2 < NDC * 4; ++i2)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float* q = dst + (nt * 8 + 2 * t + (e & 1)) * C::kOStride + place(i2, e);
                            const float v = o[i2][nt][e] * f[nt][e & 1];
                            *q = half || warp + 4 >= kMmaWarps ? v : *q + v;
                        }
            }
            consumers_sync();
        }
        const bool whole = u.starts && u.ends;
        const int slot = u.starts ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
        const int D4 = p.D / 4;
        for (int e = threadIdx.x; e < u.rows * D4; e += kMmaWarps * 32) {
            const int r = e / D4, d = (e - r * D4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<kGrid, kMmaThreads, C::kSmem, stream>>>(P);
    return cudaGetLastError();
}

#define TRIATTN_PAGED_VARIANTS(X, T) X(T, 1, 1) X(T, 1, 2) X(T, 1, 4) X(T, 2, 1) X(T, 2, 2) X(T, 2, 4) X(T, 4, 1) X(T, 4, 2)
#define TRIATTN_PAGED_EXTERN(t, d, n) \
    extern template cudaError_t launch_mma_variant<t, d, n>(const MmaParams&, cudaStream_t);
#define TRIATTN_PAGED_INSTANTIATE(t, d, n) \
    template cudaError_t launch_mma_variant<t, d, n>(const MmaParams&, cudaStream_t);

}  // namespace paged
}  // namespace triattn
