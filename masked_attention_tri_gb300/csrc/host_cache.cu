// host_cache.cu -- the C entry points of rotary positions and of the paged cache:
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

TA_EXPORT ta_status tri_attn_rotary(const void* q, const void* k, ta_dtype dtype, const int32_t* positions,
                                    const uint64_t* turns, int rotary_dim, int interleaved, float mscale,
                                    int inverse, int total, int Hq, int Hk, int D, long long q_row_stride,
                                    long long k_row_stride, long long q_out_row_stride,
                                    long long k_out_row_stride, void* q_out, void* k_out, void* stream) {
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
    ta_status st = check_cache(k_cache, v_cache, dtype, cache_dtype, k_scale, v_scale, num_pages, page_size, max_pages,
                               Hk, D, k_strides, v_strides, p.ks, p.vs);
    if (st != TA_OK) return st;
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
    ta_status st = check_cache(k_cache, v_cache, dtype, cache_dtype, k_scale, v_scale, num_pages, page_size, max_pages,
                               Hk, D, k_strides, v_strides, p.ks, p.vs);
    if (st != TA_OK) return st;
    if ((st = row_stride(q_row_stride, Hq, D, dtype_bytes(dtype))) != TA_OK) return st;
    if ((long long)total_q * Hq > 0x7fffffffLL || (long long)max_seqlen_q * Hq > 0x7fffffffLL)
        return TA_ERR_UNSUPPORTED;
    if (total_q == 0 || max_seqlen_q == 0) return TA_OK;
    if (!workspace || workspace_bytes < tri_attn_paged_workspace_size(dtype, max_seqlen_q, Hq, Hk, D))
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
    p.scale_log2e = scale * 1.4426950408889634f;
    p.q_rs = q_row_stride;
    p.status = status_word();
    if (!p.status) return TA_ERR_CUDA;
    return launch_paged(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TA_OK : TA_ERR_CUDA;
}
