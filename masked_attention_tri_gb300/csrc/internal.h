// internal.h -- parameter blocks and launchers shared by the host entry points
// and the kernels of the triangle-attention library.  Not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/triattn.h"
#include "sink_window.h"

namespace triattn {

// Device-side status codes (match ta_status).  A kernel that gives up writes
// one with atomicCAS(status, 0, code) so the first fault is kept.
enum : int { kStatusOk = 0, kStatusTimeout = TA_ERR_TIMEOUT, kStatusDevice = TA_ERR_DEVICE };

// Dynamic shared memory that a block may have (227 KB).  A kernel without static shared memory raises its limit to
// this and not to a call's size: two host threads' calls may come between one another, and a smaller call's limit would
// make the larger one's launch fail.
constexpr int kMaxDynamicSmem = 232448;

// One attention problem as the kernels see it.  Triangle form: units are
// (b, n, h) slabs with Q query rows and K keys.  Varlen form: units are
// (sequence, h) with lengths read from cu_seqlens.
struct AttnParams {
    const void* q;
    const void* k;
    const void* v;
    const void* bias;       // triangle only, may be NULL in varlen
    const uint8_t* mask;    // triangle dense key mask (B,N,K) or NULL
    const int32_t* kv_len;  // triangle kv_lengths (B,N) or NULL
    void* out;
    float* lse;
    float* mx;
    int* status;            // device status word

    int dtype;              // ta_dtype of q/k/v/out
    int bias_f32;           // 1: bias is fp32, 0: bias has the q/k/v dtype
    float scale;

    // triangle sizes
    int B, N, H, Q, K, D;
    // triangle q, k, v: element strides of the b, n, h and row (q / key) indices; the D elements of
    // a row are contiguous.  Contiguous tensors: {N*H*rows*D, H*rows*D, rows*D, D}.
    long long qs[4], ks[4], vs[4];

    // varlen
    int varlen;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int num_seqs, max_q, max_k;
    const int32_t* kv_num;
    const int32_t* kv_idx;
    const int32_t* full_num;
    const int32_t* full_idx;
    int mask_heads, MQ, MK, mask_mod;
    int window;             // TA_MASK_SLIDING_WINDOW / SINK_WINDOW: keys q - window < k <= q
    const int32_t* prefix_len;  // TA_MASK_PREFIX_LM: per-sequence prefix lengths (SINK_WINDOW: sinks), or NULL:
    int prefix_all;         //   then prefix_all for every sequence
    int total_q;            // rows of q/out (lse/max stride in varlen)
    int total_k;            // rows of k/v
    long long q_rs, k_rs, v_rs;  // varlen: elements between packed rows of q, k, v (out: H * D)
};

// Backward of the triangle form (CUDA cores, exact fp32 arithmetic).
struct BwdParams {
    const void* q;
    const void* k;
    const void* v;
    const void* bias;
    const void* d_out;
    const uint8_t* mask;
    const int32_t* kv_len;
    const float* lse;       // (B, N, H, Q) from the forward
    const void* out;        // the forward's O (q dtype) or NULL: delta = rowsum(dO * O) if given
    void* dq;
    void* dk;
    void* dv;
    void* dbias;            // (B, 1, H, Q, K) or NULL
    float* dq_acc;          // workspace: fp32 dQ (B, N, H, Q, D)
    float* dbias_acc;       // workspace: fp32 dBias (B, H, Q, K), NULL with dbias
    float* delta;           // workspace: sum_k P dP per query row (B, N, H, Q)
    int dtype, bias_f32;
    float scale;
    int B, N, H, Q, K, D;
    int tc_main;            // 1: the per-key-tile gradients on tensor cores (tc_bwd.cu)
    // Element counts of dQ and dBias and the number of per-row sums (either form).
    long long dq_elems, dbias_elems, delta_rows;
    // Packed sequences (varlen = 1): q / k / v / O / dO (total, H, D), lse / delta (H, total_q),
    // the optional bias and dBias (H, max_seqlen_q, max_seqlen_k), the BlockMask lists.
    int varlen;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int num_seqs, total_q, total_k, max_q, max_k;
    const int32_t* kv_num;
    const int32_t* kv_idx;
    const int32_t* full_num;
    const int32_t* full_idx;
    int mask_heads, MQ, MK, mask_mod, window;
    const int32_t* prefix_len;
    int prefix_all;
    int* status;
    // Sink window without lists on tensor cores: the first nb key blocks of every sequence are shared by
    // several CTAs, which sum dK and dV in acc: (num_seqs, H, nb, {dK, dV}, 128, D) fp32.
    struct {
        float* acc;
        int nb, chunk, chunks;  // key blocks; q blocks of a far CTA; far CTAs of a key block (0 nb: off)
        long long elems;        // of acc
    } sink;
};
// The sharing of a problem (sink.acc left NULL): nb = 0 where it is not worth it.
void bwd_sink_share(BwdParams& p);
// Workspace of the backward in floats: dQ, dBias and the per-row sums, each rounded up
// to a multiple of 64 floats.
size_t bwd_workspace_floats(int B, int N, int H, int Q, int K, int D);
size_t bwd_workspace_floats_n(long long dq_elems, long long dbias_elems, long long delta_rows);
cudaError_t launch_simt_bwd(const BwdParams& p, cudaStream_t stream);
// The tensor-core form of the backward's per-key-tile kernel (16-bit, D % 16 == 0,
// D <= 64, K % 8 == 0); the caller runs the per-row sums before and the conversion after.
cudaError_t launch_tc_bwd_main(const BwdParams& p, cudaStream_t stream);
bool tc_bwd_supported(const BwdParams& p);

// CUDA-core path: exact fp32 arithmetic, any dtype, both forms.
cudaError_t launch_simt_fwd(const AttnParams& p, cudaStream_t stream);

// tcgen05 / TMA path for fp16 / bf16 (both forms).
cudaError_t launch_tc_fwd(const AttnParams& p, cudaStream_t stream);

// mask -> prefix lengths.
cudaError_t launch_mask_to_kv_lengths(const uint8_t* mask, long long rows, int K, int32_t* kv_len,
                                      int32_t* nonprefix, cudaStream_t stream);

// Rotary positions of packed q (total, Hq, D) and, optionally, k (total, Hk, D).
struct RotaryParams {
    const void* q;
    const void* k;              // NULL with Hk = 0
    void* q_out;
    void* k_out;
    const int32_t* positions;   // (total), or with axes (num_axes, total)
    const int32_t* axes;        // (dim / 2): the axis of each pair, or NULL (one axis)
    const unsigned long long* turns;  // (dim / 2): turns per position, 2^-64 units
    int dtype, dim, interleaved, inverse, num_axes;
    float mscale;
    int total, Hq, Hk, D;
    long long q_rs, k_rs, qo_rs, ko_rs;  // elements between rows
};
cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream);

// The parts of a 4-bit cache: codes two a byte (the even element in the low half), 16 of them to an e4m3 scale, a
// factor a head; byte strides {page, head} (a head's slots lie one after the other).
struct Cache4 {
    uint8_t* codes[2];          // k, v: (num_pages, Hk, page, D / 2)
    uint8_t* scale[2];          // (num_pages, Hk, page, D / 16)
    const float* factor[2];     // (Hk) or NULL: 1
    long long cs[2][2], ss[2][2];
};

// New k / v rows (and the rotation of q) into a paged cache.  C of the caches: dtype, e4m3 or 4-bit codes.
struct KvAppendParams {
    const void* q;              // (total, Hq, D) or NULL
    const void* k;              // (total, Hk, D)
    const void* v;
    void* q_out;
    void* k_cache;
    void* v_cache;
    float* k_scale;             // (num_pages, Hk), e4m3 only
    float* v_scale;
    const int32_t* cu;          // (num_seqs + 1), or NULL: one row a sequence
    const int32_t* kv_len;      // (num_seqs): rows held after the call
    const int32_t* table;       // (num_seqs, max_pages)
    const int32_t* positions;   // (total), or with axes (num_axes, total), or NULL: the row's slot
    const int32_t* axes;        // (dim / 2): the axis of each pair, or NULL
    const unsigned long long* turns;
    int dtype, cache_dtype, dim, interleaved, num_axes;  // dim 0: no rotation
    float mscale;
    int num_seqs, total, max_n, Hq, Hk, D, num_pages, page, max_pages;
    long long q_rs, k_rs, v_rs, qo_rs;
    long long ks[3], vs[3];     // element strides {page, head, slot} of the caches
    Cache4 c4;                  // 4-bit caches
    int* status;
};
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream);

// Attention over a paged cache.
struct PagedParams {
    const void* q;              // (total_q, Hq, D)
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;       // (num_pages, Hk), e4m3 only
    const float* v_scale;
    const int32_t* cu;          // (num_seqs + 1), or NULL: one row a sequence
    const int32_t* kv_len;      // (num_seqs)
    const int32_t* table;       // (num_seqs, max_pages)
    void* out;                  // (total_q, Hq, D)
    float* lse;                 // (Hq, total_q) or NULL
    void* ws;
    int* status;
    int dtype, cache_dtype;
    int num_seqs, total_q, max_q, Hq, Hk, G, D, num_pages, page, max_pages;
    int window, sinks;          // window 0: every earlier slot
    int RT;                     // rows of a unit
    int tile;                   // slots of a tile
    int unit_tiles;             // what a unit's set-up and merge weigh, in tiles
    float scale_log2e;
    long long q_rs;
    long long ks[3], vs[3];     // element strides {page, head, slot} of the caches
    Cache4 c4;                  // 4-bit caches
};
int paged_rows(int dtype, int max_q, int G, int D);  // RT of a problem
int paged_tile(int dtype, int cache_dtype, int D);   // and its tile
int paged_unit_tiles(int dtype, int cache_dtype);    // and what a unit weighs beside its tiles
size_t paged_workspace_bytes(int RT, int D);
cudaError_t launch_paged(const PagedParams& p, cudaStream_t stream);

// Rows of a paged cache into packed k / v rows.
struct KvReadParams {
    const void* cache[2];       // k, v: as in KvAppendParams, or c4
    const float* scale[2];      // (num_pages, Hk), e4m3 only
    void* out[2];               // (total, Hk, D) of dtype
    const int32_t* cu;          // (num_seqs + 1), or NULL: one row a sequence
    const int32_t* kv_len;      // (num_seqs): the rows read are the last of these slots
    const int32_t* table;
    int dtype, cache_dtype;
    int num_seqs, total, max_n, Hk, D, num_pages, page, max_pages;
    long long rs[2];            // elements between rows of out
    long long st[2][3];         // element strides {page, head, slot} of the caches
    Cache4 c4;
    int* status;
};
cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream);

// Causal attention of packed prompts with grouped heads, and its gradients.
struct PromptParams {
    const void* q;              // (total_q, Hq, D)
    const void* k;              // (total_k, Hk, D)
    const void* v;
    const int32_t* cu_q;        // (num_seqs + 1)
    const int32_t* cu_k;
    void* out;                  // (total_q, Hq, D): written by the forward, read by the backward
    float* lse;                 // (Hq, total_q), or NULL in the forward
    int* status;
    int dtype, num_seqs, total_q, total_k, max_q, max_k, Hq, Hk, G, D;
    float scale;
    long long q_rs, k_rs, v_rs; // elements between rows
    // backward
    const void* d_out;          // (total_q, Hq, D)
    void* dq;
    void* dk;
    void* dv;
    float* delta;               // workspace: dO . O (Hq, total_q)
    float* norm;                // workspace, fp16 on tensor cores (else NULL): |dO| of the rows (Hq, total_q)
    float* most;                // workspace, with norm: the largest |V|, |dO| and |delta| of each (sequence, key head) (num_seqs, Hk, 3)
    float* parts;               // workspace: fp32 parts of dK and dV (splits, 2, total_k, Hk, D) where several CTAs share them, else NULL
};
// 16-bit inputs with D <= 128 run on tensor cores.
inline bool prompt_on_tc(int dtype, int D) { return dtype != TA_F32 && D <= 128; }
cudaError_t launch_prompt_simt_fwd(const PromptParams& p, cudaStream_t stream);
cudaError_t launch_prompt_simt_bwd(const PromptParams& p, cudaStream_t stream);
cudaError_t launch_prompt_tc_fwd(const PromptParams& p, cudaStream_t stream);
cudaError_t launch_prompt_tc_bwd(const PromptParams& p, cudaStream_t stream);
int prompt_bwd_splits(int num_seqs, int total_k, int max_q, int max_k, int Hk, int G);  // CTAs of a key tile there

// Zeros into the rows [0, cu[0]) and [cu[num_seqs], total) of x, row_bytes (a multiple of 16) each.
cudaError_t launch_zero_rest(void* x, long long row_bytes, const int32_t* cu, int num_seqs, int total, cudaStream_t stream);

// Device address of the status word on the current device (set up once per device).
int* status_word();

}  // namespace triattn
