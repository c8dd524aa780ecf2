// C ABI of the rotary positions, the rotating appends and the fp4 cache:
// argument validation, planning and launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "api_common.h"
#include "rope_fp4.h"

namespace kvd {

const ChunkKernel* fp4_table_d64(int nt, bool f32);
const ChunkKernel* fp4_table_d128(int nt, bool f32);
const ChunkKernel* fp4_table_d256(int nt, bool f32);

// The query rows of a pair are the columns of the kernel's MMAs, 8 to a tile; a
// CTA takes up to 6 tiles (48 rows), so that a cached row is converted once for
// all of them. More rows are dealt evenly to blocks of at most 48, a CTA each.
const ChunkKernel* fp4_chunk_kernel(int head_dim, bool f32_out, int rows) {
    const int blocks = (rows + 47) / 48;
    const int nt = ((rows + blocks - 1) / blocks + 7) / 8;  // 5 tiles run as 6 (64 x 2,048 tokens, 40 heads on one: 27.4 us, 25.0 as 5)
    switch (head_dim) {
        case 64: return fp4_table_d64(nt, f32_out);
        case 128: return fp4_table_d128(nt, f32_out);
        case 256: return fp4_table_d256(nt, f32_out);
        default: return nullptr;
    }
}

namespace {

std::atomic<uint64_t> g_fp4_ready[kMaxDevices];  // bit 10 * (head_dim index) + kernel index: shared memory allowed

kvd_status check_rope(const kvd_rope* rope, int head_dim, RopeTable* out) {
    if (!rope || !rope->turns || !aligned(rope->turns, 8)) return KVD_ERR_INVALID_ARG;
    if (rope->rotary_dim < 16 || rope->rotary_dim > 256 || rope->rotary_dim % 16 != 0 || rope->rotary_dim > head_dim)
        return KVD_ERR_INVALID_ARG;
    if (!std::isfinite(rope->factor)) return KVD_ERR_INVALID_ARG;
    *out = RopeTable{rope->turns, rope->factor, rope->rotary_dim, rope->interleaved != 0};
    return KVD_OK;
}

// Token numbers of the fp4 calls stay this far below 2^31, so that the tile after the last has one too.
constexpr int kMaxTokens4 = 0x7ffffc00;

// The checks the two rotating appends share, and the launch.
kvd_status append_rope(AppendTarget to, size_t cache_bytes, size_t scale_bytes, const kvd_rope* rope, const void* q,
                       long long q_stride, void* q_out, long long q_out_stride, const void* k_new, long long k_stride,
                       const void* v_new, long long v_stride, const int32_t* pos, const int32_t* row_offsets, int batch,
                       long long n_rows, int Hq, int Hkv, int D, int32_t* status, kvd_stream_t stream) {
    kvd_status st = check_append(to.k, to.v, k_new, v_new, pos, batch, to.S_max, Hkv, D, status);
    if (st != KVD_OK) return st;
    if (n_rows < 0 || n_rows > 0x7fffffffLL || (q != nullptr) != (q_out != nullptr)) return KVD_ERR_INVALID_ARG;
    if (row_offsets && !aligned(row_offsets, 4)) return KVD_ERR_INVALID_ARG;
    if (!row_offsets && (batch > 0 ? n_rows % batch != 0 : n_rows != 0)) return KVD_ERR_INVALID_ARG;
    if (D > 1024) return KVD_ERR_UNSUPPORTED;
    if (Hkv > (1 << 20) || (q && (Hq < 1 || Hq > (1 << 20)))) return KVD_ERR_INVALID_ARG;
    RopeTable table{nullptr, 1.f, 0, 0};
    if (rope) {
        st = check_rope(rope, D, &table);
        if (st != KVD_OK) return st;
    } else if (q) {
        return KVD_ERR_INVALID_ARG;
    }
    const long long kw = (long long)Hkv * D, qw = q ? (long long)Hq * D : 0;
    if ((st = check_strided(k_new, k_stride, kw, 2)) != KVD_OK) return st;
    if ((st = check_strided(v_new, v_stride, kw, 2)) != KVD_OK) return st;
    if (q) {
        if ((st = check_strided(q, q_stride, qw, 2)) != KVD_OK) return st;
        if ((st = check_strided(q_out, q_out_stride, qw, 2)) != KVD_OK) return st;
    }
    if (batch == 0 || n_rows == 0) return KVD_OK;
    // What is written overlaps nothing that is read, or written otherwise: q_out against the new rows (it may be q
    // itself), the caches and their scales against all of those and each other.
    const Rows rk{k_new, k_stride, kw, n_rows, 2}, rv{v_new, v_stride, kw, n_rows, 2}, rq{q, q_stride, qw, n_rows, 2},
        ro{q_out, q_out_stride, qw, n_rows, 2};
    const ByteRange ck{to.k, cache_bytes}, cv{to.v, cache_bytes}, sk{to.k_scale, scale_bytes}, sv{to.v_scale, scale_bytes};
    const bool in_place = q && q == q_out;
    if (in_place && q_stride != q_out_stride) return KVD_ERR_INVALID_ARG;
    const ByteRange rp{pos, (size_t)batch * 4}, rf{row_offsets, row_offsets ? ((size_t)batch + 1) * 4 : 0};
    if (q && ((!in_place && rows_meet(ro, rq)) || rows_meet(ro, rk) || rows_meet(ro, rv) || ro.range().overlaps(rp) ||
              ro.range().overlaps(rf)))
        return KVD_ERR_INVALID_ARG;
    const ByteRange none{nullptr, 0}, written[4] = {ck, cv, sk, sv},
                    other[6] = {rk.range(), rv.range(), q ? rq.range() : none, q ? ro.range() : none, rp, rf};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < i; ++j)
            if (written[i].overlaps(written[j])) return KVD_ERR_INVALID_ARG;
        for (const ByteRange& o : other)
            if (written[i].overlaps(o)) return KVD_ERR_INVALID_ARG;
    }
    int sms = 0;
    if ((st = device_sms(&sms)) != KVD_OK) return st;
    const NewRows in{q, q_out, k_new, v_new, q_stride, q_out_stride, k_stride, v_stride, pos, row_offsets,
                     batch, row_offsets ? 0 : (int)(n_rows / batch), q ? Hq : 0, Hkv, D, n_rows};
    return launch_append_rope(to, table, in, status, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVD_OK
                                                                                                            : KVD_ERR_CUDA;
}

// An fp4 cache's description, checked; *rows: token rows of the whole cache per KV head.
kvd_status check_fp4(const kvd_cache_fp4* c, int batch, int head_dim, PagedCache* pg, int* s_max, long long* rows) {
    if (!c) return KVD_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return head_dim <= 0 ? KVD_ERR_INVALID_ARG : KVD_ERR_UNSUPPORTED;
    *pg = PagedCache{nullptr, 0, 0, 0};
    *s_max = c->s_max;
    if (c->block_table) {
        const kvd_status st = check_paged(c->block_table, c->max_blocks, c->page_size, c->num_pages, pg, s_max);
        if (st != KVD_OK) return st;
        *rows = (long long)c->num_pages * c->page_size;
    } else {
        if (c->s_max <= 0 || c->s_max % 16 != 0 || batch < 0) return KVD_ERR_INVALID_ARG;
        *rows = (long long)batch * c->s_max;
    }
    return KVD_OK;
}

// Split count: one CTA per resident slot, shared among the row blocks of a
// token run, but no fewer than a pair or 256 tokens of one (2 blocks for each of a CTA's 8 warps): 41 sequences of one token,
// 64 and 8 heads of 256, take 12 us, and 18 where a CTA gets 256 tokens of any pairs; 108 of up to 31, 2 heads of 128, 7 and 26.
kvd_status plan_fp4(int batch, int T, int Hq, int Hkv, int D, int max_len, int num_sms, int request, int* n_split,
                    size_t* ws) {
    kvd_status st = check_shape(batch, Hq, Hkv, D, KVD_OUT_BF16);
    if (st != KVD_OK) return st;
    if (T < 1 || max_len < 0 || request < 0 || num_sms < 0) return KVD_ERR_INVALID_ARG;
    if (T > KVD_MAX_TOKENS || max_len > kMaxTokens4) return KVD_ERR_UNSUPPORTED;
    const int rows = T * (Hq / Hkv);
    const ChunkKernel* k = fp4_chunk_kernel(D, false, rows);
    if (!k) return KVD_ERR_UNSUPPORTED;
    int n = request;
    if (n == 0) {
        int sms = num_sms;
        if (sms == 0 && (st = device_sms(&sms)) != KVD_OK) return st;
        const long long blocks = (rows + k->mma_rows - 1) / k->mma_rows;
        const long long slots = std::max(1LL, (long long)sms * k->ctas_per_sm / blocks);
        const long long work = (long long)batch * Hkv * ((max_len + 255LL) / 256);
        n = (int)std::max(1LL, std::min(slots, work));
    }
    *n_split = n;
    *ws = workspace_for(n, batch, Hq * T, Hkv, D);
    return KVD_OK;
}

}  // namespace

// The frequencies of pairs that share a table of 2 * pairs columns.
kvd_status rope_turns(int pairs, double base, kvd_rope_scaling scaling, double scale, double original_len, double slow, double fast,
                      double attn_factor, uint64_t* turns_host, float* factor_out) {
    if (!turns_host || !factor_out || pairs < 8 || pairs > 128) return KVD_ERR_INVALID_ARG;
    if (!std::isfinite(base) || base <= 1.0 || !std::isfinite(attn_factor) || attn_factor < 0) return KVD_ERR_INVALID_ARG;
    const bool ramp = scaling == KVD_ROPE_PARTS || scaling == KVD_ROPE_WAVELENGTH;
    if (scaling < KVD_ROPE_NONE || scaling > KVD_ROPE_WAVELENGTH) return KVD_ERR_INVALID_ARG;
    if (scaling != KVD_ROPE_NONE && !(std::isfinite(scale) && scale >= 1.0)) return KVD_ERR_INVALID_ARG;
    if (ramp && !(std::isfinite(original_len) && original_len > 0 && slow > 0 && std::isfinite(fast) && fast > slow))
        return KVD_ERR_INVALID_ARG;
    const double R = 2.0 * pairs, two_pi = 6.283185307179586476925;
    if (scaling == KVD_ROPE_BASE) base *= std::pow(scale, R / (R - 2.0));
    if (!std::isfinite(base)) return KVD_ERR_INVALID_ARG;
    double lo = 0, hi = 0;
    if (scaling == KVD_ROPE_PARTS) {
        auto index = [&](double turns) { return R * std::log(original_len / (two_pi * turns)) / (2.0 * std::log(base)); };
        lo = std::max(std::floor(index(fast)), 0.0);
        hi = std::min(std::ceil(index(slow)), R - 1.0);
        if (hi <= lo) hi = lo + 0.001;  // a step
    }
    for (int i = 0; i < pairs; ++i) {
        double w = std::pow(base, -2.0 * i / R);
        double keep = 1.0;
        if (scaling == KVD_ROPE_LINEAR) keep = 0.0;
        if (scaling == KVD_ROPE_WAVELENGTH) keep = (original_len * w / two_pi - slow) / (fast - slow);
        if (scaling == KVD_ROPE_PARTS) keep = 1.0 - (i - lo) / (hi - lo);
        keep = std::min(1.0, std::max(0.0, keep));
        if (keep < 1.0) w = w * keep + w / scale * (1.0 - keep);
        turns_host[i] = (uint64_t)std::nearbyint(std::ldexp(w / two_pi, 64));  // w <= 1: below 2^62
    }
    *factor_out = (float)(attn_factor > 0 ? attn_factor : scaling == KVD_ROPE_PARTS ? 0.1 * std::log(scale) + 1.0 : 1.0);
    return KVD_OK;
}

}  // namespace kvd

using namespace kvd;

extern "C" {

kvd_status kvd_rope_table(int rotary_dim, double base, kvd_rope_scaling scaling, double scale, double original_len,
                          double slow, double fast, double attn_factor, uint64_t* turns_host, float* factor_out) {
    if (rotary_dim % 16 != 0) return KVD_ERR_INVALID_ARG;
    return rope_turns(rotary_dim / 2, base, scaling, scale, original_len, slow, fast, attn_factor, turns_host, factor_out);
}

kvd_status kvd_rope_apply(const kvd_rope* rope, const void* x, long long x_stride, kvd_out_dtype in_dtype, void* y,
                          long long y_stride, kvd_out_dtype out_dtype, const int32_t* positions, long long rows,
                          int n_heads, int head_dim, kvd_stream_t stream) {
    if (rows < 0 || rows > 0x7fffffffLL || n_heads < 1 || n_heads > (1 << 20) || head_dim < 8 || head_dim % 8 != 0)
        return KVD_ERR_INVALID_ARG;
    if (head_dim > 1024) return KVD_ERR_UNSUPPORTED;
    if ((in_dtype != KVD_OUT_BF16 && in_dtype != KVD_OUT_F32) || (out_dtype != KVD_OUT_BF16 && out_dtype != KVD_OUT_F32))
        return KVD_ERR_INVALID_ARG;
    RopeTable table;
    kvd_status st = check_rope(rope, head_dim, &table);
    if (st != KVD_OK) return st;
    const size_t ies = in_dtype == KVD_OUT_F32 ? 4 : 2, oes = out_dtype == KVD_OUT_F32 ? 4 : 2;
    const long long width = (long long)n_heads * head_dim;
    if (!positions || !aligned(positions, 4)) return KVD_ERR_INVALID_ARG;
    if ((st = check_strided(x, x_stride, width, ies)) != KVD_OK) return st;
    if ((st = check_strided(y, y_stride, width, oes)) != KVD_OK) return st;
    const Rows rx{x, x_stride, width, rows, ies}, ry{y, y_stride, width, rows, oes};
    const bool in_place = x == y && x_stride == y_stride && in_dtype == out_dtype;
    if ((!in_place && rows_meet(rx, ry)) || ry.range().overlaps(ByteRange{positions, (size_t)rows * 4}))
        return KVD_ERR_INVALID_ARG;
    if (rows == 0) return KVD_OK;
    int sms = 0;
    if ((st = device_sms(&sms)) != KVD_OK) return st;
    return launch_rope(table, x, x_stride, in_dtype == KVD_OUT_F32, y, y_stride, out_dtype == KVD_OUT_F32, positions, rows,
                       n_heads, head_dim, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KVD_OK
               : KVD_ERR_CUDA;
}

kvd_status kvd_kv_append_rope(const kvd_cache* cache, const kvd_rope* rope, const void* q, long long q_stride,
                              void* q_out, long long q_out_stride, const void* k_new, long long k_stride,
                              const void* v_new, long long v_stride, const int32_t* pos, const int32_t* row_offsets,
                              int batch, long long n_rows, int n_heads_q, int n_heads_kv, int head_dim,
                              int32_t* status_word, kvd_stream_t stream) {
    if (!cache || !rope || batch < 0 || n_heads_kv <= 0 || head_dim <= 0) return KVD_ERR_INVALID_ARG;
    const bool quant = cache->k_scales || cache->v_scales;
    if (quant && (!cache->k_scales || !cache->v_scales || !aligned(cache->k_scales, 4) || !aligned(cache->v_scales, 4)))
        return KVD_ERR_INVALID_ARG;
    if (cache->fp8 && !quant) return KVD_ERR_INVALID_ARG;
    if (quant && head_dim != 64 && head_dim != 128 && head_dim != 256) return KVD_ERR_UNSUPPORTED;
    AppendTarget to{cache->k, cache->v, cache->k_scales, cache->v_scales,
                    quant ? (cache->fp8 ? CacheForm::kFp8 : CacheForm::kInt8) : CacheForm::kBf16, cache->s_max,
                    PagedCache{nullptr, 0, 0, 0}};
    size_t rows = (size_t)batch * (size_t)std::max(cache->s_max, 0);
    if (cache->block_table) {
        const kvd_status st = check_paged(cache->block_table, cache->max_blocks, cache->page_size, cache->num_pages, &to.pg,
                                          &to.S_max);
        if (st != KVD_OK) return st;
        rows = (size_t)cache->num_pages * cache->page_size;
    }
    return append_rope(to, rows * n_heads_kv * head_dim * (quant ? 1 : 2), quant ? rows * n_heads_kv * 4 : 0, rope, q,
                       q_stride, q_out, q_out_stride, k_new, k_stride, v_new, v_stride, pos, row_offsets, batch, n_rows,
                       n_heads_q, n_heads_kv, head_dim, status_word, stream);
}

kvd_status kvd_kv_append_fp4(const kvd_cache_fp4* cache, const kvd_rope* rope, const void* q, long long q_stride,
                             void* q_out, long long q_out_stride, const void* k_new, long long k_stride,
                             const void* v_new, long long v_stride, const int32_t* pos, const int32_t* row_offsets,
                             int batch, long long n_rows, int n_heads_q, int n_heads_kv, int head_dim,
                             int32_t* status_word, kvd_stream_t stream) {
    if (batch < 0 || n_heads_kv <= 0) return KVD_ERR_INVALID_ARG;
    PagedCache pg;
    int s_max = 0;
    long long rows = 0;
    const kvd_status st = check_fp4(cache, batch, head_dim, &pg, &s_max, &rows);
    if (st != KVD_OK) return st;
    const AppendTarget to{cache->k, cache->v, nullptr, nullptr, CacheForm::kFp4, s_max, pg};
    return append_rope(to, (size_t)(rows / 16) * n_heads_kv * kvd_fp4_block_bytes(head_dim), 0, rope, q, q_stride, q_out,
                       q_out_stride, k_new, k_stride, v_new, v_stride, pos, row_offsets, batch, n_rows, n_heads_q,
                       n_heads_kv, head_dim, status_word, stream);
}

size_t kvd_fp4_block_bytes(int head_dim) {
    return head_dim == 64 || head_dim == 128 || head_dim == 256 ? (size_t)(9 * head_dim + 16) : 0;
}

kvd_status kvd_kv_quantize_fp4(const void* cache, void* blocks, const int32_t* seq_lens, int batch, int s_max,
                               int s_max_blocks, int max_seq_len, int n_heads_kv, int head_dim, kvd_stream_t stream) {
    if (max_seq_len > kMaxTokens4) return KVD_ERR_UNSUPPORTED;
    if (batch < 0 || s_max <= 0 || s_max_blocks <= 0 || s_max_blocks % 16 != 0 || max_seq_len < 0 || max_seq_len > s_max ||
        max_seq_len > s_max_blocks || n_heads_kv <= 0)
        return KVD_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVD_ERR_UNSUPPORTED;
    if (!cache || !blocks || !seq_lens || !aligned(cache, 16) || !aligned(blocks, 16) || !aligned(seq_lens, 4))
        return KVD_ERR_INVALID_ARG;
    const ByteRange rc{cache, (size_t)batch * s_max * n_heads_kv * head_dim * 2},
        rb{blocks, (size_t)batch * n_heads_kv * (s_max_blocks / 16) * kvd_fp4_block_bytes(head_dim)},
        rl{seq_lens, (size_t)batch * 4};
    if (rb.overlaps(rc) || rb.overlaps(rl)) return KVD_ERR_INVALID_ARG;
    if (batch == 0 || max_seq_len == 0) return KVD_OK;
    if ((long long)batch * ((max_seq_len + 15) / 16) > 0x7fffffffLL) return KVD_ERR_INVALID_ARG;
    int sms = 0;
    const kvd_status st = device_sms(&sms);
    if (st != KVD_OK) return st;
    return launch_quantize_fp4(cache, blocks, seq_lens, batch, s_max, s_max_blocks, max_seq_len, n_heads_kv, head_dim, sms,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KVD_OK
               : KVD_ERR_CUDA;
}

kvd_status kvd_kv_read_fp4(const void* blocks, const int32_t* block_table, int s_max_blocks, int max_blocks,
                           int page_size, int num_pages, void* out, int s_out, const int32_t* seq_lens, int batch,
                           int max_seq_len, int n_heads_kv, int head_dim, int32_t* status_word, kvd_stream_t stream) {
    if (max_seq_len > kMaxTokens4) return KVD_ERR_UNSUPPORTED;
    if (batch < 0 || s_out <= 0 || max_seq_len < 0 || max_seq_len > s_out || n_heads_kv <= 0) return KVD_ERR_INVALID_ARG;
    const kvd_cache_fp4 c{const_cast<void*>(blocks), nullptr, block_table, s_max_blocks, max_blocks, page_size, num_pages};
    PagedCache pg;
    int s_max = 0;
    long long rows = 0;
    kvd_status st = check_fp4(&c, batch, head_dim, &pg, &s_max, &rows);
    if (st != KVD_OK) return st;
    if (max_seq_len > s_max) return KVD_ERR_INVALID_ARG;
    if (!blocks || !out || !seq_lens || !aligned(blocks, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) ||
        (status_word && !aligned(status_word, 4)))
        return KVD_ERR_INVALID_ARG;
    const ByteRange ro{out, (size_t)batch * s_out * n_heads_kv * head_dim * 2},
        rb{blocks, (size_t)(rows / 16) * n_heads_kv * kvd_fp4_block_bytes(head_dim)}, rl{seq_lens, (size_t)batch * 4};
    if (ro.overlaps(rb) || ro.overlaps(rl)) return KVD_ERR_INVALID_ARG;
    if (batch == 0 || max_seq_len == 0) return KVD_OK;
    if ((long long)batch * ((max_seq_len + 15) / 16) > 0x7fffffffLL) return KVD_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != KVD_OK) return st;
    return launch_read_fp4(blocks, pg, s_max, out, s_out, seq_lens, batch, max_seq_len, n_heads_kv, head_dim, status_word,
                           sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KVD_OK
               : KVD_ERR_CUDA;
}

kvd_status kvd_decode_plan_fp4(int batch, int n_tokens, int n_heads_q, int n_heads_kv, int head_dim, int max_seq_len,
                               int num_sms, int n_split_request, int* n_split_out, size_t* workspace_bytes_out) {
    if (!n_split_out || !workspace_bytes_out) return KVD_ERR_INVALID_ARG;
    return plan_fp4(batch, n_tokens, n_heads_q, n_heads_kv, head_dim, max_seq_len, num_sms, n_split_request, n_split_out,
                    workspace_bytes_out);
}

kvd_status kvd_decode_fp4(const kvd_cache_fp4* cache, const void* q, const int32_t* seq_lens, int batch, int n_tokens,
                          int max_seq_len, int n_heads_q, int n_heads_kv, int head_dim, float scale, int n_split,
                          void* workspace, size_t workspace_bytes, void* out, kvd_out_dtype out_dtype,
                          float* lse_out, const void* k_new, const void* v_new, const int32_t* pos,
                          int32_t* status_word, kvd_stream_t stream) {
    kvd_status st = check_shape(batch, n_heads_q, n_heads_kv, head_dim, out_dtype);
    if (st != KVD_OK) return st;
    PagedCache pg;
    int s_max = 0;
    long long rows = 0;
    st = check_fp4(cache, batch, head_dim, &pg, &s_max, &rows);
    if (st != KVD_OK) return st;
    if (max_seq_len < 0 || max_seq_len > s_max || !std::isfinite(scale)) return KVD_ERR_INVALID_ARG;
    if (!cache->k || !cache->v || !q || !seq_lens || !out) return KVD_ERR_INVALID_ARG;
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) ||
        (lse_out && !aligned(lse_out, 4)) || (status_word && !aligned(status_word, 4)))
        return KVD_ERR_INVALID_ARG;
    const bool append = k_new || v_new || pos;
    if (append && !(k_new && v_new && pos)) return KVD_ERR_INVALID_ARG;
    int n = 0;
    size_t need = 0;
    st = plan_fp4(batch, n_tokens, n_heads_q, n_heads_kv, head_dim, max_seq_len, 0, n_split, &n, &need);
    if (st != KVD_OK) return st;
    const int G = n_heads_q / n_heads_kv, pair_rows = n_tokens * G;
    const bool f32 = out_dtype == KVD_OUT_F32;
    const ChunkKernel* k = fp4_chunk_kernel(head_dim, f32, pair_rows);
    const int row_blocks = (pair_rows + k->mma_rows - 1) / k->mma_rows;
    if ((long long)n * row_blocks > 0x7fffffffLL) return KVD_ERR_INVALID_ARG;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return KVD_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 256)) return KVD_ERR_INVALID_ARG;
    }
    const long long kv_row = (long long)n_heads_kv * head_dim;
    if (append) {
        const AppendTarget to{cache->k, cache->v, nullptr, nullptr, CacheForm::kFp4, s_max, pg};
        st = append_rope(to, (size_t)(rows / 16) * n_heads_kv * kvd_fp4_block_bytes(head_dim), 0, nullptr, nullptr, 0, nullptr,
                         0, k_new, kv_row, v_new, kv_row, pos, nullptr, batch, (long long)batch * n_tokens, 0, n_heads_kv,
                         head_dim, status_word, stream);
        if (st != KVD_OK) return st;
    }
    if (batch == 0) return KVD_OK;

    DecodeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = q;
    p.k = cache->k;
    p.v = cache->v;
    p.seq_lens = seq_lens;
    p.B = batch;
    p.S_max = s_max;
    p.len_cap = std::min(s_max, max_seq_len);
    p.Hq = n_heads_q;
    p.Hkv = n_heads_kv;
    p.G = G;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.n_split = n;
    p.tile_tokens = k->tile_tokens;
    p.seg_unit = k->seg_unit;
    p.seg_cost = k->seg_cost;
    p.early = append ? 1 : 0;
    p.pos = pos;
    p.out = out;
    p.lse = lse_out;
    p.status = status_word;
    p.T = n_tokens;
    p.vT = 1;
    p.row_blocks = row_blocks;
    if (pg.block_table) {
        p.block_table = pg.block_table;
        p.max_blocks = pg.max_blocks;
        p.page_shift = pg.page_shift;
        p.num_pages = pg.num_pages;
    }
    if (need > 0) {
        const size_t slots = (size_t)n + (size_t)batch * n_heads_kv - 1;
        uint8_t* w = static_cast<uint8_t*>(workspace);
        p.ws_o = reinterpret_cast<float*>(w);
        w += align256(slots * pair_rows * head_dim * sizeof(float));
        p.ws_ml = reinterpret_cast<float2*>(w);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return KVD_ERR_CUDA;
    const uint64_t bit = 1ull << (k->index + (head_dim == 64 ? 0 : head_dim == 128 ? 10 : 20));
    if (!(g_fp4_ready[dev].load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(k->fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k->smem_bytes) != cudaSuccess)
            return KVD_ERR_CUDA;
        g_fp4_ready[dev].fetch_or(bit, std::memory_order_acq_rel);
    }
    if (k->launch(*k, p, s) != cudaSuccess) return KVD_ERR_CUDA;
    if (n > 1) {
        if ((st = device_sms(&sms)) != KVD_OK) return st;
        if (launch_merge(p, head_dim, f32, sms, s) != cudaSuccess) return KVD_ERR_CUDA;
    }
    return KVD_OK;
}

}  // extern "C"
