// host_cache.cu -- the C entry points of rotary positions, of the paged cache and of prompts:
// argument checks and launches (include/triattn.h).

#include <cuda_runtime.h>

#include "host_checks.h"

using namespace triattn;

namespace {

// The row stride of a packed (total, H, D) buffer: 0 = H * D, at least H * D, whole 16-byte
// vectors.
ta_status row_stride(long long& rs, int H, int D, int esz) {
    const long long hd = (long long)H * D;
    if (rs == 0) rs = hd;
    if (rs < hd) return TA_ERR_INVALID_ARG;
    if ((rs * esz) % 16 != 0 || rs * esz >= (1LL << 40)) return TA_ERR_UNSUPPORTED;
    return TA_OK;
}

// The element strides {page, head, slot} of a cache whose D elements are contiguous: the given
// ones (checked), or the contiguous layout.
ta_status cache_strides(const long long* given, int num_pages, int Hk, int page, int D, int esz, long long (&st)[3]) {
    if (!given) {
        st[2] = D;
        st[1] = (long long)page * D;
        st[0] = st[1] * Hk;
    } else {
        const long long ext[3] = {num_pages, Hk, page};
        for (int i = 0; i < 3; ++i) {
            st[i] = given[i];
            if (st[i] < D) return TA_ERR_INVALID_ARG;  // no two rows overlap
            if (st[i] > ((1LL << 60) / ext[i])) return TA_ERR_UNSUPPORTED;
        }
    }
    for (int i = 0; i < 3; ++i)  // tensor-map strides: 16-byte multiples below 2^40 bytes
        if ((st[i] * esz) % 16 != 0 || st[i] * esz >= (1LL << 40)) return TA_ERR_UNSUPPORTED;
    return TA_OK;
}

// A launch whose grid would pass the hardware's limits (odd head counts in the ten thousands) is refused.
ta_status launched(cudaError_t e) {
    return e == cudaSuccess ? TA_OK : e == cudaErrorInvalidConfiguration ? TA_ERR_UNSUPPORTED : TA_ERR_CUDA;
}

// What the two operators on a paged cache check alike.
ta_status check_cache(const void* k_cache, const void* v_cache, int dtype, int cache_dtype, const float* k_scale,
                      const float* v_scale, int num_pages, int page_size, int max_pages, int Hk, int D,
                      const long long* k_strides, const long long* v_strides, long long (&ks)[3], long long (&vs)[3]) {
    if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return TA_ERR_INVALID_ARG;
    if (num_pages <= 0 || page_size <= 0 || max_pages <= 0) return TA_ERR_INVALID_ARG;
    if (!valid_dtype(cache_dtype) && cache_dtype != TA_E4M3) return TA_ERR_INVALID_ARG;
    const bool codes = cache_dtype == TA_E4M3;
    if (codes ? (!k_scale || !v_scale) : (k_scale || v_scale)) return TA_ERR_INVALID_ARG;
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return TA_ERR_INVALID_ARG;
    if (!codes && cache_dtype != dtype) return TA_ERR_UNSUPPORTED;
    if (codes && D % 16 != 0) return TA_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return TA_ERR_UNSUPPORTED;
    const int esz = dtype_bytes(cache_dtype);
    const ta_status st = cache_strides(k_strides, num_pages, Hk, page_size, D, esz, ks);
    return st != TA_OK ? st : cache_strides(v_strides, num_pages, Hk, page_size, D, esz, vs);
}

}  // namespace

namespace {

// tri_attn_rotary (pair_axes NULL, num_axes 1) and tri_attn_rotary_axes.
ta_status rotary(const void* q, const void* k, ta_dtype dtype, const int32_t* positions, int num_axes,
                 const int32_t* pair_axes, const uint64_t* turns, int rotary_dim, int interleaved, float mscale,
                 int inverse, int total, int Hq, int Hk, int D, long long q_row_stride, long long k_row_stride,
                 long long q_out_row_stride, long long k_out_row_stride, void* q_out, void* k_out, void* stream) {
    if (!q || !q_out || !positions || !turns) return TA_ERR_INVALID_ARG;
    if (total < 0 || Hq <= 0 || Hk < 0 || D <= 0) return TA_ERR_INVALID_ARG;
    if (Hk > 0 ? (!k || !k_out) : (k || k_out)) return TA_ERR_INVALID_ARG;
    if (!valid_dtype(dtype)) return TA_ERR_INVALID_ARG;
    if (rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0) return TA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(positions, 4) ||
        !aligned(turns, 8))
        return TA_ERR_INVALID_ARG;
    if (!supported_d(dtype, D)) return TA_ERR_UNSUPPORTED;
    const int esz = dtype_bytes(dtype);
    ta_status st;
    if ((st = row_stride(q_row_stride, Hq, D, esz)) != TA_OK) return st;
    if ((st = row_stride(q_out_row_stride, Hq, D, esz)) != TA_OK) return st;
    if (Hk > 0) {
        if ((st = row_stride(k_row_stride, Hk, D, esz)) != TA_OK) return st;
        if ((st = row_stride(k_out_row_stride, Hk, D, esz)) != TA_OK) return st;
    }
    if ((q == q_out && q_row_stride != q_out_row_stride) || (k && k == k_out && k_row_stride != k_out_row_stride))
        return TA_ERR_INVALID_ARG;
    if (total == 0) return TA_OK;
    RotaryParams p{};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.positions = positions;
    p.axes = pair_axes;
    p.num_axes = num_axes;
    p.turns = reinterpret_cast<const unsigned long long*>(turns);
    p.dtype = dtype;
    p.dim = rotary_dim;
    p.interleaved = interleaved != 0;
    p.inverse = inverse != 0;
    p.mscale = mscale;
    p.total = total;
    p.Hq = Hq;
    p.Hk = Hk;
    p.D = D;
    p.q_rs = q_row_stride;
    p.k_rs = k_row_stride;
    p.qo_rs = q_out_row_stride;
    p.ko_rs = k_out_row_stride;
    return launched(launch_rotary(p, static_cast<cudaStream_t>(stream)));
}

// The axes of a rotation: one, or several with an axis for each pair.
ta_status check_axes(const int32_t* pair_axes, int num_axes) {
    return num_axes < 1 || !pair_axes || !aligned(pair_axes, 4) ? TA_ERR_INVALID_ARG : TA_OK;
}

// A 4-bit cache, checked, for heads of D.
ta_status check_cache4(const ta_cache4* c, int Hk, int D, int max_pages, Cache4& out) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return TA_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
        !aligned(c->k_factor, 4) || !aligned(c->v_factor, 4))
        return TA_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->page_size <= 0 || max_pages <= 0) return TA_ERR_INVALID_ARG;
    if (D % 32 != 0 || c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
        return TA_ERR_UNSUPPORTED;
    bool given = false;
    for (long long s : c->strides) given = given || s != 0;
    for (int i = 0; i < 4; ++i) {
        const long long head = (long long)c->page_size * (i < 2 ? D / 2 : D / 16);  // bytes of a page's head
        long long st[2] = {head * Hk, head};
        if (given) {
            for (int j = 0; j < 2; ++j) {
                st[j] = c->strides[2 * i + j];
                if (st[j] < head) return TA_ERR_INVALID_ARG;  // no two heads overlap
                if (st[j] % 16 != 0 || st[j] >= (1LL << 40)) return TA_ERR_UNSUPPORTED;
            }
        }
        if (st[0] > (1LL << 60) / c->num_pages || st[1] > (1LL << 60) / Hk || st[0] >= (1LL << 40)) return TA_ERR_UNSUPPORTED;
        for (int j = 0; j < 2; ++j) (i < 2 ? out.cs : out.ss)[i % 2][j] = st[j];
    }
    out.codes[0] = static_cast<uint8_t*>(c->k);
    out.codes[1] = static_cast<uint8_t*>(c->v);
    out.scale[0] = c->k_scale;
    out.scale[1] = c->v_scale;
    out.factor[0] = c->k_factor;
    out.factor[1] = c->v_factor;
    return TA_OK;
}

// All forms of tri_attn_kv_append (one axis: pair_axes NULL, num_axes 1; a 4-bit cache: c4, cache_dtype TA_INT4).
ta_status kv_append(const void* q, const void* k, const void* v, ta_dtype dtype, const int32_t* cu_seqlens,
                    const int32_t* kv_lengths, const int32_t* page_table, int num_seqs, int total, int max_seqlen,
                    int Hq, int Hk, int D, long long q_row_stride, long long k_row_stride, long long v_row_stride,
                    long long q_out_row_stride, const int32_t* positions, int num_axes, const int32_t* pair_axes,
                    const uint64_t* turns, int rotary_dim, int interleaved, float mscale, void* k_cache, void* v_cache,
                    ta_dtype cache_dtype, float* k_scale, float* v_scale, const ta_cache4* c4, int num_pages,
                    int page_size, int max_pages, const long long* k_strides, const long long* v_strides, void* q_out,
                    void* stream) {
    if (!k || !v || !kv_lengths || !page_table) return TA_ERR_INVALID_ARG;
    if (num_seqs <= 0 || total < 0 || max_seqlen < 0 || Hk <= 0 || D <= 0) return TA_ERR_INVALID_ARG;
    if (Hq > 0 ? (!q || !q_out || !turns) : (q || q_out || Hq < 0)) return TA_ERR_INVALID_ARG;
    if (!cu_seqlens && (total != num_seqs || max_seqlen != 1)) return TA_ERR_INVALID_ARG;
    if (!valid_dtype(dtype)) return TA_ERR_INVALID_ARG;
    if (turns ? (rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0) : (rotary_dim != 0 || positions))
        return TA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(cu_seqlens, 4) ||
        !aligned(kv_lengths, 4) || !aligned(page_table, 4) || !aligned(positions, 4) || !aligned(turns, 8))
        return TA_ERR_INVALID_ARG;
    if (!supported_d(dtype, D)) return TA_ERR_UNSUPPORTED;
    KvAppendParams p{};
    ta_status st = c4 ? check_cache4(c4, Hk, D, max_pages, p.c4)
                      : check_cache(k_cache, v_cache, dtype, cache_dtype, k_scale, v_scale, num_pages, page_size,
                                    max_pages, Hk, D, k_strides, v_strides, p.ks, p.vs);
    if (st != TA_OK) return st;
    if (c4 && rotary_dim % 32 != 0) return TA_ERR_UNSUPPORTED;
    const int esz = dtype_bytes(dtype);
    if ((st = row_stride(k_row_stride, Hk, D, esz)) != TA_OK) return st;
    if ((st = row_stride(v_row_stride, Hk, D, esz)) != TA_OK) return st;
    if (Hq > 0) {
        if ((st = row_stride(q_row_stride, Hq, D, esz)) != TA_OK) return st;
        if ((st = row_stride(q_out_row_stride, Hq, D, esz)) != TA_OK) return st;
        if (q == q_out && q_row_stride != q_out_row_stride) return TA_ERR_INVALID_ARG;
    }
    if ((long long)num_seqs * (max_seqlen / page_size + 2) > 0x7fffffffLL || Hk > 16384 || Hq > 65536)
        return TA_ERR_UNSUPPORTED;
    if (total == 0 || max_seqlen == 0) return TA_OK;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.cu = cu_seqlens;
    p.kv_len = kv_lengths;
    p.table = page_table;
    p.positions = positions;
    p.axes = pair_axes;
    p.num_axes = num_axes;
    p.turns = reinterpret_cast<const unsigned long long*>(turns);
    p.dtype = dtype;
    p.cache_dtype = cache_dtype;
    p.dim = rotary_dim;
    p.interleaved = interleaved != 0;
    p.mscale = mscale;
    p.num_seqs = num_seqs;
    p.total = total;
    p.max_n = max_seqlen;
    p.Hq = Hq;
    p.Hk = Hk;
    p.D = D;
    p.num_pages = num_pages;
    p.page = page_size;
    p.max_pages = max_pages;
    p.q_rs = q_row_stride;
    p.k_rs = k_row_stride;
    p.v_rs = v_row_stride;
    p.qo_rs = q_out_row_stride;
    p.status = status_word();
    if (!p.status) return TA_ERR_CUDA;
    return launched(launch_kv_append(p, static_cast<cudaStream_t>(stream)));
}

// tri_attn_paged_fwd, and over a 4-bit cache (c4, cache_dtype TA_INT4).
ta_status paged_fwd(const void* q, ta_dtype dtype, const int32_t* cu_seqlens_q, const int32_t* kv_lengths,
                    const int32_t* page_table, int num_seqs, int total_q, int max_seqlen_q, int Hq, int Hk, int D,
                    long long q_row_stride, float scale, int window, int sinks, const void* k_cache,
                    const void* v_cache, ta_dtype cache_dtype, const float* k_scale, const float* v_scale,
                    const ta_cache4* c4, int num_pages, int page_size, int max_pages, const long long* k_strides,
                    const long long* v_strides, void* out, float* lse, void* workspace, size_t workspace_bytes,
                    void* stream) {
    if (!q || !out || !kv_lengths || !page_table) return TA_ERR_INVALID_ARG;
    if (num_seqs <= 0 || total_q < 0 || max_seqlen_q < 0 || Hq <= 0 || Hk <= 0 || D <= 0 || Hq % Hk != 0)
        return TA_ERR_INVALID_ARG;
    if (!cu_seqlens_q && (total_q != num_seqs || max_seqlen_q != 1)) return TA_ERR_INVALID_ARG;
    if (window < 0 || sinks < 0) return TA_ERR_INVALID_ARG;
    if (!valid_dtype(dtype)) return TA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(cu_seqlens_q, 4) ||
        !aligned(kv_lengths, 4) || !aligned(page_table, 4) || !aligned(lse, 4))
        return TA_ERR_INVALID_ARG;
    if (!supported_d(dtype, D)) return TA_ERR_UNSUPPORTED;
    PagedParams p{};
    ta_status st = c4 ? check_cache4(c4, Hk, D, max_pages, p.c4)
                      : check_cache(k_cache, v_cache, dtype, cache_dtype, k_scale, v_scale, num_pages, page_size,
                                    max_pages, Hk, D, k_strides, v_strides, p.ks, p.vs);
    if (st != TA_OK) return st;
    if ((st = row_stride(q_row_stride, Hq, D, dtype_bytes(dtype))) != TA_OK) return st;
    if ((long long)total_q * Hq > 0x7fffffffLL || (long long)max_seqlen_q * Hq > 0x7fffffffLL)
        return TA_ERR_UNSUPPORTED;
    if (total_q == 0 || max_seqlen_q == 0) return TA_OK;
    if (!workspace || workspace_bytes < paged_workspace_bytes(paged_rows(dtype, max_seqlen_q, Hq / Hk, D), D))
        return TA_ERR_INVALID_ARG;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.cu = cu_seqlens_q;
    p.kv_len = kv_lengths;
    p.table = page_table;
    p.out = out;
    p.lse = lse;
    p.ws = workspace;
    p.dtype = dtype;
    p.cache_dtype = cache_dtype;
    p.num_seqs = num_seqs;
    p.total_q = total_q;
    p.max_q = max_seqlen_q;
    p.Hq = Hq;
    p.Hk = Hk;
    p.G = Hq / Hk;
    p.D = D;
    p.num_pages = num_pages;
    p.page = page_size;
    p.max_pages = max_pages;
    p.window = window;
    p.sinks = sinks;
    p.RT = paged_rows(dtype, max_seqlen_q, p.G, D);
    p.tile = paged_tile(dtype, cache_dtype, D);
    p.unit_tiles = paged_unit_tiles(dtype, cache_dtype);
    p.scale_log2e = scale * 1.4426950408889634f;
    p.q_rs = q_row_stride;
    p.status = status_word();
    if (!p.status) return TA_ERR_CUDA;
    return launch_paged(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TA_OK : TA_ERR_CUDA;
}

// tri_attn_kv_read, and from a 4-bit cache (c4, cache_dtype TA_INT4).
ta_status kv_read(const int32_t* cu_seqlens, const int32_t* kv_lengths, const int32_t* page_table, int num_seqs,
                  int total, int max_seqlen, int Hk, int D, const void* k_cache, const void* v_cache,
                  ta_dtype cache_dtype, const float* k_scale, const float* v_scale, const ta_cache4* c4, int num_pages,
                  int page_size, int max_pages, const long long* k_strides, const long long* v_strides, void* k_out,
                  void* v_out, ta_dtype dtype, long long k_row_stride, long long v_row_stride, void* stream) {
    if (!k_out || !v_out || !kv_lengths || !page_table) return TA_ERR_INVALID_ARG;
    if (num_seqs <= 0 || total < 0 || max_seqlen < 0 || Hk <= 0 || D <= 0) return TA_ERR_INVALID_ARG;
    if (!cu_seqlens && (total != num_seqs || max_seqlen != 1)) return TA_ERR_INVALID_ARG;
    if (!valid_dtype(dtype)) return TA_ERR_INVALID_ARG;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(cu_seqlens, 4) || !aligned(kv_lengths, 4) ||
        !aligned(page_table, 4))
        return TA_ERR_INVALID_ARG;
    if (!supported_d(dtype, D)) return TA_ERR_UNSUPPORTED;
    KvReadParams p{};
    ta_status st = c4 ? check_cache4(c4, Hk, D, max_pages, p.c4)
                      : check_cache(k_cache, v_cache, dtype, cache_dtype, k_scale, v_scale, num_pages, page_size,
                                    max_pages, Hk, D, k_strides, v_strides, p.st[0], p.st[1]);
    if (st != TA_OK) return st;
    const int esz = dtype_bytes(dtype);
    if ((st = row_stride(k_row_stride, Hk, D, esz)) != TA_OK) return st;
    if ((st = row_stride(v_row_stride, Hk, D, esz)) != TA_OK) return st;
    if ((long long)num_seqs * (max_seqlen / page_size + 2) > 0x7fffffffLL || Hk > 16384) return TA_ERR_UNSUPPORTED;
    if (total == 0 || max_seqlen == 0) return TA_OK;
    p.cache[0] = k_cache;
    p.cache[1] = v_cache;
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.cu = cu_seqlens;
    p.kv_len = kv_lengths;
    p.table = page_table;
    p.dtype = dtype;
    p.cache_dtype = cache_dtype;
    p.num_seqs = num_seqs;
    p.total = total;
    p.max_n = max_seqlen;
    p.Hk = Hk;
    p.D = D;
    p.num_pages = num_pages;
    p.page = page_size;
    p.max_pages = max_pages;
    p.rs[0] = k_row_stride;
    p.rs[1] = v_row_stride;
    p.status = status_word();
    if (!p.status) return TA_ERR_CUDA;
    return launched(launch_kv_read(p, static_cast<cudaStream_t>(stream)));
}

// What the forward and the backward of prompts check alike.
ta_status prompt_params(const void* q, const void* k, const void* v, ta_dtype dtype, const int32_t* cu_q,
                        const int32_t* cu_k, int num_seqs, int total_q, int total_k, int max_q, int max_k, int Hq,
                        int Hk, int D, float scale, long long q_rs, long long k_rs, long long v_rs, void* out,
                        float* lse, PromptParams& p) {
    if (!q || !k || !v || !out || !cu_q || !cu_k) return TA_ERR_INVALID_ARG;
    if (num_seqs <= 0 || total_q < 0 || total_k < 0 || max_q < 0 || max_k < 0 || Hq <= 0 || Hk <= 0 || D <= 0 ||
        Hq % Hk != 0)
        return TA_ERR_INVALID_ARG;
    if (!valid_dtype(dtype)) return TA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
        !aligned(cu_k, 4) || !aligned(lse, 4))
        return TA_ERR_INVALID_ARG;
    if (!supported_d(dtype, D)) return TA_ERR_UNSUPPORTED;
    const int esz = dtype_bytes(dtype);
    ta_status st;
    if ((st = row_stride(q_rs, Hq, D, esz)) != TA_OK) return st;
    if ((st = row_stride(k_rs, Hk, D, esz)) != TA_OK) return st;
    if ((st = row_stride(v_rs, Hk, D, esz)) != TA_OK) return st;
    if ((long long)total_q * Hq > 0x7fffffffLL || (long long)total_k * Hk > 0x7fffffffLL ||
        (long long)max_q * Hq > 0x3fffffffLL || max_k > 0x3fffffff || Hk > 65535 || num_seqs > 65535)
        return TA_ERR_UNSUPPORTED;
    p.q = q;
    p.k = k;
    p.v = v;
    p.out = out;
    p.lse = lse;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.dtype = dtype;
    p.num_seqs = num_seqs;
    p.total_q = total_q;
    p.total_k = total_k;
    p.max_q = max_q < total_q ? max_q : total_q;
    p.max_k = max_k < total_k ? max_k : total_k;
    p.Hq = Hq;
    p.Hk = Hk;
    p.G = Hq / Hk;
    p.D = D;
    p.scale = scale;
    p.q_rs = q_rs;
    p.k_rs = k_rs;
    p.v_rs = v_rs;
    return TA_OK;
}

// The backward's workspace: dO . O, in fp16 what scales dS (prompt_tc.cuh), and fp32 parts of dK and dV where several CTAs share them (tensor cores); its size, and
// with p its parts.
size_t prompt_workspace(int dtype, int num_seqs, int total_q, int total_k, int max_q, int max_k, int Hq, int Hk, int D,
                        char* ws, PromptParams* p) {
    if (max_q > total_q) max_q = total_q;
    if (max_k > total_k) max_k = total_k;
    const size_t rows = ((size_t)total_q * Hq + 63) / 64 * 64 * sizeof(float);
    const int splits = prompt_on_tc(dtype, D) ? prompt_bwd_splits(num_seqs, total_k, max_q, max_k, Hk, Hq / Hk) : 1;
    const bool scaled = dtype == TA_F16 && prompt_on_tc(dtype, D);
    const size_t most = scaled ? ((size_t)num_seqs * Hk * 3 + 63) / 64 * 64 * sizeof(float) : 0, sums = rows + (scaled ? rows + most : 0);
    if (p) {
        p->delta = reinterpret_cast<float*>(ws);
        p->norm = scaled ? reinterpret_cast<float*>(ws + rows) : nullptr;
        p->most = scaled ? reinterpret_cast<float*>(ws + 2 * rows) : nullptr;
        p->parts = splits > 1 ? reinterpret_cast<float*>(ws + sums) : nullptr;
    }
    return sums + (splits > 1 ? (size_t)splits * 2 * total_k * Hk * D * sizeof(float) : 0);
}

}  // namespace

TA_EXPORT ta_status tri_attn_rotary(const void* q, const void* k, ta_dtype dtype, const int32_t* positions,
                                    const uint64_t* turns, int rotary_dim, int interleaved, float mscale,
                                    int inverse, int total, int Hq, int Hk, int D, long long q_row_stride,
                                    long long k_row_stride, long long q_out_row_stride,
                                    long long k_out_row_stride, void* q_out, void* k_out, void* stream) {
    return rotary(q, k, dtype, positions, 1, nullptr, turns, rotary_dim, interleaved, mscale, inverse, total, Hq, Hk, D,
                  q_row_stride, k_row_stride, q_out_row_stride, k_out_row_stride, q_out, k_out, stream);
}

TA_EXPORT ta_status tri_attn_rotary_axes(const void* q, const void* k, ta_dtype dtype, const int32_t* positions,
                                         int num_axes, const int32_t* pair_axes, const uint64_t* turns,
                                         int rotary_dim, int interleaved, float mscale, int inverse, int total, int Hq,
                                         int Hk, int D, long long q_row_stride, long long k_row_stride,
                                         long long q_out_row_stride, long long k_out_row_stride, void* q_out,
                                         void* k_out, void* stream) {
    const ta_status st = check_axes(pair_axes, num_axes);
    return st != TA_OK ? st
                       : rotary(q, k, dtype, positions, num_axes, pair_axes, turns, rotary_dim, interleaved, mscale,
                                inverse, total, Hq, Hk, D, q_row_stride, k_row_stride, q_out_row_stride,
                                k_out_row_stride, q_out, k_out, stream);
}

TA_EXPORT ta_status tri_attn_kv_append(const void* q, const void* k, const void* v, ta_dtype dtype,
                                       const int32_t* cu_seqlens, const int32_t* kv_lengths,
                                       const int32_t* page_table, int num_seqs, int total, int max_seqlen, int Hq,
                                       int Hk, int D, long long q_row_stride, long long k_row_stride,
                                       long long v_row_stride, long long q_out_row_stride, const int32_t* positions,
                                       const uint64_t* turns, int rotary_dim, int interleaved, float mscale,
                                       void* k_cache, void* v_cache, ta_dtype cache_dtype, float* k_scale,
                                       float* v_scale, int num_pages, int page_size, int max_pages,
                                       const long long* k_strides, const long long* v_strides, void* q_out,
                                       void* stream) {
    return kv_append(q, k, v, dtype, cu_seqlens, kv_lengths, page_table, num_seqs, total, max_seqlen, Hq, Hk, D,
                     q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, positions, 1, nullptr, turns,
                     rotary_dim, interleaved, mscale, k_cache, v_cache, cache_dtype, k_scale, v_scale, nullptr,
                     num_pages, page_size, max_pages, k_strides, v_strides, q_out, stream);
}

TA_EXPORT ta_status tri_attn_kv_append_axes(const void* q, const void* k, const void* v, ta_dtype dtype,
                                            const int32_t* cu_seqlens, const int32_t* kv_lengths,
                                            const int32_t* page_table, int num_seqs, int total, int max_seqlen, int Hq,
                                            int Hk, int D, long long q_row_stride, long long k_row_stride,
                                            long long v_row_stride, long long q_out_row_stride,
                                            const int32_t* positions, int num_axes, const int32_t* pair_axes,
                                            const uint64_t* turns, int rotary_dim, int interleaved, float mscale,
                                            void* k_cache, void* v_cache, ta_dtype cache_dtype, float* k_scale,
                                            float* v_scale, int num_pages, int page_size, int max_pages,
                                            const long long* k_strides, const long long* v_strides, void* q_out,
                                            void* stream) {
    const ta_status st = check_axes(pair_axes, num_axes);
    if (st != TA_OK || !turns) return TA_ERR_INVALID_ARG;
    return kv_append(q, k, v, dtype, cu_seqlens, kv_lengths, page_table, num_seqs, total, max_seqlen, Hq, Hk, D,
                     q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, positions, num_axes, pair_axes, turns,
                     rotary_dim, interleaved, mscale, k_cache, v_cache, cache_dtype, k_scale, v_scale, nullptr,
                     num_pages, page_size, max_pages, k_strides, v_strides, q_out, stream);
}

TA_EXPORT ta_status tri_attn_kv_append4(const void* q, const void* k, const void* v, ta_dtype dtype,
                                        const int32_t* cu_seqlens, const int32_t* kv_lengths,
                                        const int32_t* page_table, int num_seqs, int total, int max_seqlen, int Hq,
                                        int Hk, int D, long long q_row_stride, long long k_row_stride,
                                        long long v_row_stride, long long q_out_row_stride, const int32_t* positions,
                                        int num_axes, const int32_t* pair_axes, const uint64_t* turns, int rotary_dim,
                                        int interleaved, float mscale, const ta_cache4* cache, int max_pages,
                                        void* q_out, void* stream) {
    if (!cache) return TA_ERR_INVALID_ARG;
    if (pair_axes ? check_axes(pair_axes, num_axes) != TA_OK || !turns : num_axes != 1) return TA_ERR_INVALID_ARG;
    return kv_append(q, k, v, dtype, cu_seqlens, kv_lengths, page_table, num_seqs, total, max_seqlen, Hq, Hk, D,
                     q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, positions, num_axes, pair_axes, turns,
                     rotary_dim, interleaved, mscale, nullptr, nullptr, TA_INT4, nullptr, nullptr, cache,
                     cache->num_pages, cache->page_size, max_pages, nullptr, nullptr, q_out, stream);
}

TA_EXPORT size_t tri_attn_paged_workspace_size(ta_dtype dtype, int max_seqlen_q, int Hq, int Hk, int D) {
    if (max_seqlen_q <= 0 || Hq <= 0 || Hk <= 0 || D <= 0 || Hq % Hk != 0) return 0;
    return paged_workspace_bytes(paged_rows(dtype, max_seqlen_q, Hq / Hk, D), D);
}


TA_EXPORT ta_status tri_attn_paged_fwd(const void* q, ta_dtype dtype, const int32_t* cu_seqlens_q,
                                       const int32_t* kv_lengths, const int32_t* page_table, int num_seqs, int total_q,
                                       int max_seqlen_q, int Hq, int Hk, int D, long long q_row_stride, float scale,
                                       int window, int sinks, const void* k_cache, const void* v_cache,
                                       ta_dtype cache_dtype, const float* k_scale, const float* v_scale,
                                       int num_pages, int page_size, int max_pages, const long long* k_strides,
                                       const long long* v_strides, void* out, float* lse, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    return paged_fwd(q, dtype, cu_seqlens_q, kv_lengths, page_table, num_seqs, total_q, max_seqlen_q, Hq, Hk, D,
                     q_row_stride, scale, window, sinks, k_cache, v_cache, cache_dtype, k_scale, v_scale, nullptr,
                     num_pages, page_size, max_pages, k_strides, v_strides, out, lse, workspace, workspace_bytes,
                     stream);
}

TA_EXPORT ta_status tri_attn_paged4_fwd(const void* q, ta_dtype dtype, const int32_t* cu_seqlens_q,
                                        const int32_t* kv_lengths, const int32_t* page_table, int num_seqs,
                                        int total_q, int max_seqlen_q, int Hq, int Hk, int D, long long q_row_stride,
                                        float scale, int window, int sinks, const ta_cache4* cache, int max_pages,
                                        void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (!cache) return TA_ERR_INVALID_ARG;
    return paged_fwd(q, dtype, cu_seqlens_q, kv_lengths, page_table, num_seqs, total_q, max_seqlen_q, Hq, Hk, D,
                     q_row_stride, scale, window, sinks, nullptr, nullptr, TA_INT4, nullptr, nullptr, cache,
                     cache->num_pages, cache->page_size, max_pages, nullptr, nullptr, out, lse, workspace,
                     workspace_bytes, stream);
}

TA_EXPORT ta_status tri_attn_kv_read(const int32_t* cu_seqlens, const int32_t* kv_lengths, const int32_t* page_table,
                                     int num_seqs, int total, int max_seqlen, int Hk, int D, const void* k_cache,
                                     const void* v_cache, ta_dtype cache_dtype, const float* k_scale,
                                     const float* v_scale, int num_pages, int page_size, int max_pages,
                                     const long long* k_strides, const long long* v_strides, void* k_out, void* v_out,
                                     ta_dtype dtype, long long k_row_stride, long long v_row_stride, void* stream) {
    return kv_read(cu_seqlens, kv_lengths, page_table, num_seqs, total, max_seqlen, Hk, D, k_cache, v_cache,
                   cache_dtype, k_scale, v_scale, nullptr, num_pages, page_size, max_pages, k_strides, v_strides, k_out,
                   v_out, dtype, k_row_stride, v_row_stride, stream);
}

TA_EXPORT ta_status tri_attn_kv_read4(const int32_t* cu_seqlens, const int32_t* kv_lengths, const int32_t* page_table,
                                      int num_seqs, int total, int max_seqlen, int Hk, int D, const ta_cache4* cache,
                                      int max_pages, void* k_out, void* v_out, ta_dtype dtype, long long k_row_stride,
                                      long long v_row_stride, void* stream) {
    if (!cache) return TA_ERR_INVALID_ARG;
    return kv_read(cu_seqlens, kv_lengths, page_table, num_seqs, total, max_seqlen, Hk, D, nullptr, nullptr, TA_INT4,
                   nullptr, nullptr, cache, cache->num_pages, cache->page_size, max_pages, nullptr, nullptr, k_out,
                   v_out, dtype, k_row_stride, v_row_stride, stream);
}

TA_EXPORT ta_status tri_attn_prompt_fwd(const void* q, const void* k, const void* v, ta_dtype dtype,
                                        const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs,
                                        int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int Hq, int Hk,
                                        int D, float scale, long long q_row_stride, long long k_row_stride,
                                        long long v_row_stride, void* out, float* lse, void* stream) {
    PromptParams p{};
    const ta_status st = prompt_params(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                       max_seqlen_q, max_seqlen_k, Hq, Hk, D, scale, q_row_stride, k_row_stride,
                                       v_row_stride, out, lse, p);
    if (st != TA_OK) return st;
    if (total_q == 0 || max_seqlen_q == 0) return TA_OK;
    p.status = status_word();
    if (!p.status) return TA_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(prompt_on_tc(dtype, D) ? launch_prompt_tc_fwd(p, s) : launch_prompt_simt_fwd(p, s));
}

TA_EXPORT size_t tri_attn_prompt_bwd_workspace_size(ta_dtype dtype, int num_seqs, int total_q, int total_k,
                                                    int max_seqlen_q, int max_seqlen_k, int Hq, int Hk, int D) {
    if (num_seqs <= 0 || total_q <= 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || Hq <= 0 || Hk <= 0 ||
        D <= 0 || Hq % Hk != 0)
        return 0;
    return prompt_workspace(dtype, num_seqs, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hk, D, nullptr, nullptr);
}

TA_EXPORT ta_status tri_attn_prompt_bwd(const void* q, const void* k, const void* v, ta_dtype dtype,
                                        const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs,
                                        int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int Hq, int Hk,
                                        int D, float scale, long long q_row_stride, long long k_row_stride,
                                        long long v_row_stride, const float* lse, const void* out, const void* d_out,
                                        void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    if (!lse || !d_out || !dq || !dk || !dv) return TA_ERR_INVALID_ARG;
    if (!aligned(d_out, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(workspace, 256))
        return TA_ERR_INVALID_ARG;
    PromptParams p{};
    const ta_status st = prompt_params(q, k, v, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                       max_seqlen_q, max_seqlen_k, Hq, Hk, D, scale, q_row_stride, k_row_stride,
                                       v_row_stride, const_cast<void*>(out), const_cast<float*>(lse), p);
    if (st != TA_OK) return st;
    if ((total_q == 0 || max_seqlen_q == 0) && (total_k == 0 || max_seqlen_k == 0)) return TA_OK;
    const size_t need = tri_attn_prompt_bwd_workspace_size(dtype, num_seqs, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq,
                                                           Hk, D);
    if (need && (!workspace || workspace_bytes < need)) return TA_ERR_INVALID_ARG;
    p.d_out = d_out;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    if (total_q > 0)
        prompt_workspace(dtype, num_seqs, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hk, D,
                         static_cast<char*>(workspace), &p);
    p.status = status_word();
    if (!p.status) return TA_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(prompt_on_tc(dtype, D) ? launch_prompt_tc_bwd(p, s) : launch_prompt_simt_bwd(p, s));
}

TA_EXPORT ta_status tri_attn_zero_rest(void* x, ta_dtype dtype, const int32_t* cu_seqlens, int num_seqs, int total, int H, int D,
                                       void* stream) {
    if (!x || !cu_seqlens || num_seqs < 0 || total < 0 || H <= 0 || D <= 0) return TA_ERR_INVALID_ARG;
    if (!valid_dtype(dtype) || !aligned(x, 16) || !aligned(cu_seqlens, 4)) return TA_ERR_INVALID_ARG;
    if (!supported_d(dtype, D)) return TA_ERR_UNSUPPORTED;
    if (total == 0) return TA_OK;
    return launched(launch_zero_rest(x, (long long)H * D * dtype_bytes(dtype), cu_seqlens, num_seqs, total,
                                     static_cast<cudaStream_t>(stream)));
}
