// paged_simt.cu -- attention over a paged cache on CUDA cores in exact fp32: fp32
// queries, with an fp32, an 8-bit or a 4-bit cache; and the kernel that joins split rows.
//
// One CTA of eight warps per share of the tile axis (paged.cuh); the warps of a CTA
// take the tiles of a unit in turn, each with its own running maximum, sum and O,
// and merge at the unit's end.  A warp reads one slot's row of K (and V) with
// coalesced vectors, four elements a lane, for eight query rows at once: the 32 dot
// products of four slots are summed over the lanes by a transposing reduction (31 shuffles),
// after which each lane holds one (slot, row) logit.  Bound: the FMAs
// (8 rows x 2 an element) and shuffles, at about half the memory rate for fp32.

#include <type_traits>

#include "cache4.cuh"
#include "paged.cuh"

namespace triattn {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 8;
constexpr int kMinTiles = 8;   // shares are not cut finer than one tile a warp

template <typename C>
__device__ __forceinline__ float4 load4(const C* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<uint8_t>(const uint8_t* p) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3)));
    const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3)));
    return make_float4(a.x, a.y, b.x, b.y);
}

// One slot's row of a 4-bit cache, elements [d, d + 4).
__device__ __forceinline__ float4 load4_codes(const uint8_t* codes, const uint8_t* scale, int d) {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(codes + d / 2);
    const float s = cache4::scale_value(scale[d / 16]);
    auto value = [&](int i) { return (float)((int)((w >> (4 * i)) & 15u) - 8) * s; };
    return make_float4(value(0), value(1), value(2), value(3));
}

// C: the cache's elements: fp32, uint8_t (e4m3) or cache4::Code.  NC: vectors of 4 elements a lane (D up to 128 NC).
template <typename C, int NC>
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(const PagedParams p) {
    constexpr bool kFour = std::is_same<C, cache4::Code>::value, kCodes = std::is_same<C, uint8_t>::value;
    extern __shared__ float smem[];  // O [kWarps][kRows][D], (m, l) [kWarps][kRows]
    __shared__ long long scan[kWarps], found[2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int D = p.D;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up meanwhile
    float* so = smem;
    float2* sml = reinterpret_cast<float2*>(smem + kWarps * kRows * D);
    const Workspace ws = workspace(p.ws, p.RT, D);
    const Share sh = find_share<kThreads>(p, kMinTiles, scan, found);
    Walk w = walk_begin(p, sh);
    if (threadIdx.x == 0) ws.join[blockIdx.x].parts = 0;
    long long at = sh.begin;  // axis position of the unit's first tile in this share
    Unit u;
    while (walk_next(p, w, u)) {
        const long long head0 = (long long)u.h * p.G;
        // this lane's logits belong to row lane % 8
        const int myrow = u.rt * kRows + lane % kRows;
        const int mypos = u.q.len - u.q.n + min(myrow, u.q.n * p.G - 1) / p.G;
        float4 qf[kRows][NC];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int row = u.rt * kRows + r;
            const long long tok = u.q.row0 + row / p.G, head = head0 + row % p.G;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = (c * 32 + lane) * 4;
                qf[r][c] = row < u.q.n * p.G && d < D
                               ? load4<float>(static_cast<const float*>(p.q) + tok * p.q_rs + head * D + d)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float4 acc[kRows][NC];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -INFINITY, l = 0.f;  // m of row lane % 8; l: this lane's share of the sum

        for (int j = u.j0 + warp; j < u.j1 && j < u.t.nt; j += kWarps) {
            const int key_t = u.t.tile(j) * p.tile;
            for (int k0 = key_t; k0 < key_t + p.tile; k0 += 4) {
                // (pages hold at least 16 slots: four slots lie in one)
                if (!unit_sees(p, u.t, k0) && !unit_sees(p, u.t, k0 + 1) && !unit_sees(p, u.t, k0 + 2) &&
                    !unit_sees(p, u.t, k0 + 3))
                    continue;
                const long long page = p.table[(long long)u.seq * p.max_pages + k0 / p.page];
                if (page < 0 || page >= p.num_pages) {
                    if (lane == 0) atomicCAS(p.status, 0, kStatusDevice);
                    continue;
                }
                const int slot = k0 % p.page;
                // row kk of four slots, elements [d, d + 4)
                auto row = [&](int kind, int kk, int d) {
                    if constexpr (kFour) {
                        const Cache4& c = p.c4;
                        return load4_codes(c.codes[kind] + page * c.cs[kind][0] + u.h * c.cs[kind][1] + (long long)(slot + kk) * (D / 2),
                                           c.scale[kind] + page * c.ss[kind][0] + u.h * c.ss[kind][1] + (long long)(slot + kk) * (D / 16), d);
                    } else {
                        const long long* st = kind == 0 ? p.ks : p.vs;
                        return load4<C>(static_cast<const C*>(kind == 0 ? p.k_cache : p.v_cache) + page * st[0] + u.h * st[1] +
                                        (slot + kk) * st[2] + d);
                    }
                };
                float kscale = p.scale_log2e, vs_inv = 1.f, vs_log2 = 0.f;
                if constexpr (kFour) {
                    if (p.c4.factor[0]) kscale *= p.c4.factor[0][u.h];
                }
                if constexpr (kCodes) {
                    kscale *= p.k_scale[page * p.Hk + u.h];
                    const float v = p.v_scale[page * p.Hk + u.h];
                    if (!v_scale_ok(v)) {
                        if (lane == 0) atomicCAS(p.status, 0, kStatusDevice);
                        continue;
                    }
                    vs_inv = 1.f / v;
                    vs_log2 = log2f(v);
                }
                float dot[32];
                bool on[4];
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    on[kk] = unit_sees(p, u.t, k0 + kk);
                    float4 kv[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int d = (c * 32 + lane) * 4;
                        kv[c] = on[kk] && d < D ? row(0, kk, d) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        float s = 0.f;
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            s = fmaf(qf[r][c].x, kv[c].x, s);
                            s = fmaf(qf[r][c].y, kv[c].y, s);
                            s = fmaf(qf[r][c].z, kv[c].z, s);
                            s = fmaf(qf[r][c].w, kv[c].w, s);
                        }
                        dot[kk * kRows + r] = s;
                    }
                }
                // lane L ends with the sum of dot[L] over the lanes
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    const bool up = lane & o;
#pragma unroll
                    for (int i = 0; i < o; ++i) {
                        const float keep = up ? dot[i + o] : dot[i], send = up ? dot[i] : dot[i + o];
                        dot[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                }
                const int mykey = k0 + lane / kRows;
                const float x = sees(p, mypos, mykey) ? fmaf(dot[0], kscale, vs_log2) : -INFINITY;
                float mt = x;
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                if (__any_sync(0xffffffffu, mt > m)) {
                    const float mn = fmaxf(m, mt);
                    const float alpha = mn == -INFINITY ? 1.f : exp2f(m - mn);
                    m = mn;
                    l *= alpha;
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const float al = __shfl_sync(0xffffffffu, alpha, r);
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            acc[r][c].x *= al;
                            acc[r][c].y *= al;
                            acc[r][c].z *= al;
                            acc[r][c].w *= al;
                        }
                    }
                }
                const float pr = x == -INFINITY ? 0.f : exp2f(x - m);
                l = fmaf(pr, vs_inv, l);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (!on[kk]) continue;  // (a slot that no row sees is not read: it may hold anything)
                    float4 vv[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int d = (c * 32 + lane) * 4;
                        vv[c] = d < D ? row(1, kk, d) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const float pk = __shfl_sync(0xffffffffu, pr, kk * kRows + r);
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            acc[r][c].x = fmaf(pk, vv[c].x, acc[r][c].x);
                            acc[r][c].y = fmaf(pk, vv[c].y, acc[r][c].y);
                            acc[r][c].z = fmaf(pk, vv[c].z, acc[r][c].z);
                            acc[r][c].w = fmaf(pk, vv[c].w, acc[r][c].w);
                        }
                    }
                }
            }
        }
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);

        // ---- Merge of the warps.
        __syncthreads();
        if (lane < kRows) sml[warp * kRows + lane] = make_float2(m, l);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = (c * 32 + lane) * 4;
                if (d < D) *reinterpret_cast<float4*>(so + (warp * kRows + r) * D + d) = acc[r][c];
            }
        __syncthreads();
        const bool whole = u.starts && u.ends;
        const int slot = u.starts ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
        const float v_factor = kFour && p.c4.factor[1] ? p.c4.factor[1][u.h] : 1.f;
        for (int e = threadIdx.x; e < u.rows * D; e += kThreads) {
            const int r = e / D, d = e - r * D;
            float M = -INFINITY, L = 0.f, o = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sml[i * kRows + r].x);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 ml = sml[i * kRows + r];
                if (no_key(ml.x, ml.y)) continue;
                const float f = exp2f(ml.x - M);
                L = fmaf(ml.y, f, L);
                o = fmaf(so[(i * kRows + r) * D + d], f, o);
            }
            if constexpr (kFour) o *= v_factor;
            if (whole) {
                const int row = u.rt * kRows + r;
                const long long tok = u.q.row0 + row / p.G, head = head0 + row % p.G;
                store_out(p, (tok * p.Hq + head) * D + d, no_key(M, L) ? 0.f : o / L);
                if (d == 0 && p.lse) p.lse[head * p.total_q + tok] = row_lse(M, L);
            } else {
                ws.o[((long long)slot * p.RT + r) * D + d] = o;
                if (d == 0) ws.ml[slot * p.RT + r] = make_float2(M, L);
            }
        }
        if (u.starts && !u.ends && threadIdx.x == 0) {
            Join& jn = ws.join[blockIdx.x];
            jn.seq_row0 = u.q.row0;
            jn.h = u.h;
            jn.row0 = u.rt * kRows;
            jn.rows = u.rows;
            jn.parts = unit_parts(p, sh, u, at);
        }
        at += u.j1 - u.j0;
    }
}

// Share c's split unit, if one starts there: its parts in the order of the shares.
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p) {
    // Launched while the first kernel runs (programmatic dependent launch): wait for its end.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Workspace ws = workspace(p.ws, p.RT, p.D);
    const Join jn = ws.join[blockIdx.x];
    if (jn.parts <= 1) return;
    // (m, l) of all parts at once, then each row's maximum and sum over the lanes of a warp: a loop over the
    // parts from memory would cost a latency for each (a long sequence alone has up to 152 of them).
    __shared__ float2 sml[kGrid * kMaxRT];  // part i, row r at i * rows + r; then the part's weight (-1: no key) in x
    __shared__ float2 srow[kMaxRT];
    const int D4 = p.D / 4, c = blockIdx.x, rows = jn.rows;
    // part 0 in slot 2c + 1, part i in slot 2 (c + i)
    auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
    for (int e = threadIdx.x; e < jn.parts * rows; e += blockDim.x) {
        const int i = e / rows;
        sml[e] = ws.ml[slot(i) * p.RT + (e - i * rows)];
    }
    __syncthreads();
    for (int r = threadIdx.x / 32; r < rows; r += blockDim.x / 32) {
        const int lane = threadIdx.x % 32;
        float M = -INFINITY, L = 0.f;
        for (int i = lane; i < jn.parts; i += 32) M = fmaxf(M, sml[i * rows + r].x);
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        for (int i = lane; i < jn.parts; i += 32) {
            const float2 ml = sml[i * rows + r];
            const bool none = no_key(ml.x, ml.y);
            const float f = none ? -1.f : exp2f(ml.x - M);
            if (!none) L = fmaf(ml.y, f, L);
            sml[i * rows + r].x = f;
        }
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0) srow[r] = make_float2(M, L);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * D4; e += blockDim.x) {
        const int r = e / D4, d = (e - r * D4) * 4;
        const float M = srow[r].x, L = srow[r].y;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const float* at = ws.o + (long long)r * p.D + d;
#pragma unroll 8
        for (int i = 0; i < jn.parts; ++i) {
            const float f = sml[i * rows + r].x;
            const float4 x = *reinterpret_cast<const float4*>(at + (long long)slot(i) * p.RT * p.D);
            if (!(f < 0.f)) {  // (after the load, so that eight are in flight)
                o.x = fmaf(x.x, f, o.x);
                o.y = fmaf(x.y, f, o.y);
                o.z = fmaf(x.z, f, o.z);
                o.w = fmaf(x.w, f, o.w);
            }
        }
        const float inv = no_key(M, L) ? 0.f : 1.f / L;
        const int row = jn.row0 + r;
        const long long tok = jn.seq_row0 + row / p.G, head = (long long)jn.h * p.G + row % p.G;
        const long long i0 = (tok * p.Hq + head) * p.D + d;
        store_out(p, i0, o.x * inv);
        store_out(p, i0 + 1, o.y * inv);
        store_out(p, i0 + 2, o.z * inv);
        store_out(p, i0 + 3, o.w * inv);
        if (d == 0 && p.lse) p.lse[head * p.total_q + tok] = row_lse(M, L);
    }
}

template <typename C>
cudaError_t launch(const PagedParams& p, cudaStream_t stream) {
    const size_t smem = (size_t)kWarps * kRows * (p.D + 2) * 4;
    auto kern = p.D <= 128 ? paged_simt_kernel<C, 1> : paged_simt_kernel<C, 2>;
    // (the limit of the kernel's widest heads, whatever this call's: two threads' calls may come between one another)
    const int most = kWarps * kRows * ((p.D <= 128 ? 128 : 256) + 2) * 4;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    kern<<<kGrid, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_simt(const PagedParams& p, cudaStream_t stream) {
    if (p.cache_dtype == TA_INT4) return launch<cache4::Code>(p, stream);
    return p.cache_dtype == TA_E4M3 ? launch<uint8_t>(p, stream) : launch<float>(p, stream);
}

cudaError_t launch_join(const PagedParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kGrid);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel, p);
}

}  // namespace paged

// Rows of a unit: eight on CUDA cores; on tensor cores one to four groups of eight (two for D > 128, where
// four would not leave registers for the accumulators), as few as hold a sequence's rows.
int paged_rows(int dtype, int max_q, int G, int D) {
    const long long rows = (long long)max_q * G;
    if (dtype == TA_F32 || rows <= 8) return 8;
    // 32 rows a unit where the registers hold their O (D <= 64); else 16, and K and V are read again for the
    // next 16.  (16 sequences, 32 heads over 8, eight tokens each: heads of 64 in 16 bits 98 us by 32 and
    // 117 by 16; heads of 128 in 16 bits 272 and 206, in 8 bits 175 and 168.)
    return rows <= 16 || D > 64 ? 16 : 32;
}
// Slots of a tile: on tensor cores 32 KB of K and V with columns padded to whole 128 bytes.
int paged_tile(int dtype, int cache_dtype, int D) {
    if (dtype == TA_F32) return 64;
    if (cache_dtype == TA_INT4) return D <= 64 ? 256 : 128;  // (16 KB with up to 128 columns, 32 KB above)
    if (cache_dtype == TA_E4M3) return D <= 128 ? 128 : 64;
    return D <= 64 ? 128 : (D <= 128 ? 64 : 32);
}
// A unit's set-up and merge in tiles: four-bit pages on tensor cores, whose tiles take little time, 6.  (64 sequences of 1k to
// 16k slots in one batch, 32 heads over 8: 0 took 218 us, since the CTAs that got the short sequences took half as long again
// as the others; 3 180 us; 6 to 8 163 us.  One sequence of 1000 slots, 8 tiles a head, weighs 14 so: 6 of 14 shares a head hold no
// tile, and the join reads empty parts, which cost little beside a call of 14.5 us but give nothing.)
int paged_unit_tiles(int dtype, int cache_dtype) { return dtype != TA_F32 && cache_dtype == TA_INT4 ? 6 : 0; }
size_t paged_workspace_bytes(int RT, int D) { return paged::workspace_bytes(RT, D); }

cudaError_t launch_paged(const PagedParams& p, cudaStream_t stream) {
    const cudaError_t e = p.dtype == TA_F32 ? paged::launch_simt(p, stream) : paged::launch_mma(p, stream);
    return e == cudaSuccess ? paged::launch_join(p, stream) : e;
}

}  // namespace triattn
