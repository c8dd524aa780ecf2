// C ABI of the page tables, the rotary positions of several axes and the
// attention over selected blocks: argument validation, planning and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "api_common.h"
#include "blocks.h"

namespace kvd {

cudaError_t allow_clusters(const void* kernel, int smem_bytes, std::atomic<uint64_t>* ready) {
    int dev = 0;
    const cudaError_t got = cudaGetDevice(&dev);
    if (got != cudaSuccess) return got;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const uint64_t bit = 1ull << dev;
    if (ready->load(std::memory_order_acquire) & bit) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) ready->fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

cudaError_t clusters_at_once(const void* kernel, int threads, int smem_bytes, std::atomic<uint64_t>* ready, std::atomic<uint64_t>* known,
                             int (&n)[5]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    uint64_t all = known[dev].load(std::memory_order_acquire);  // 12 bits a size, and a bit that says so
    if (!all) {
        if ((e = allow_clusters(kernel, smem_bytes, ready)) != cudaSuccess) return e;
        all = 1ull << 63;
        for (int i = 0; i < 5; ++i) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(16, 1, 1);
            cfg.blockDim = dim3((unsigned)threads, 1, 1);
            cfg.dynamicSmemBytes = (size_t)smem_bytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << i;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int count = 0;
            if (cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                count = 0;  // none of this size
            }
            all |= (uint64_t)std::min(std::max(count, i == 0 ? 1 : 0), 0xfff) << (12 * i);
        }
        known[dev].store(all, std::memory_order_release);
    }
    for (int i = 0; i < 5; ++i) n[i] = (int)(all >> (12 * i)) & 0xfff;
    return cudaSuccess;
}

namespace {

constexpr int kMaxKept = 1 << 20;  // entries of a list

bool power_of_two(int x, int lo, int hi) { return x >= lo && x <= hi && (x & (x - 1)) == 0; }
int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// No range that is written overlaps another of the call; the first n_written of them are.
bool apart(const ByteRange* r, int n_written, int n) {
    for (int i = 0; i < n_written; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && r[i].overlaps(r[j])) return false;
    return true;
}

kvd_status check_axes(const kvd_rope_axes* rope, const int32_t* positions, long long axis_stride, long long rows, int head_dim,
                      RopeAxes* out) {
    if (!rope || !rope->turns || !aligned(rope->turns, 8) || !rope->axes || !aligned(rope->axes, 8)) return KVD_ERR_INVALID_ARG;
    if (rope->rotary_dim < 16 || rope->rotary_dim > 256 || rope->rotary_dim % 16 != 0 || rope->rotary_dim > head_dim)
        return KVD_ERR_INVALID_ARG;
    if (!std::isfinite(rope->factor) || rope->n_axes < 1 || rope->n_axes > KVD_MAX_AXES) return KVD_ERR_INVALID_ARG;
    if (!positions || !aligned(positions, 4) || (rope->n_axes > 1 && axis_stride < rows) || axis_stride < 0 || axis_stride > (1LL << 40))
        return KVD_ERR_INVALID_ARG;
    *out = RopeAxes{RopeTable{rope->turns, rope->factor, rope->rotary_dim, rope->interleaved != 0}, rope->axes, positions, axis_stride,
                    rope->n_axes};
    return KVD_OK;
}

size_t positions_bytes(const RopeAxes& r, long long rows) {
    return rows > 0 ? ((size_t)(r.n_axes - 1) * (size_t)r.axis_stride + (size_t)rows) * 4 : 0;
}

// A description of a cache or its bounds: paged or contiguous; *rows: token rows of the whole cache.
kvd_status check_place(const int32_t* block_table, int s_max, int max_blocks, int page_size, int num_pages, int batch,
                       PagedCache* pg, int* cap, long long* rows) {
    *pg = PagedCache{nullptr, 0, 0, 0};
    *cap = s_max;
    if (block_table) {
        const kvd_status st = check_paged(block_table, max_blocks, page_size, num_pages, pg, cap);
        if (st != KVD_OK) return st;
        *rows = (long long)num_pages * page_size;
    } else {
        if (s_max <= 0 || batch < 0) return KVD_ERR_INVALID_ARG;
        *rows = (long long)batch * s_max;
    }
    return KVD_OK;
}

// CTAs of a pair (a cluster of n) and clusters of a pair. Clusters run in waves, as many at once as the
// multiprocessors' groups hold (at_once, by log2 n; 0: none of that size). A CTA costs about what 18 stages
// cost one CTA (start, list, join), so that n is the one with the least waves * (18 + stages / n). 16 pairs of
// 4,096 tokens, 8 heads: clusters of 4 / 8 / 16 take 17.6 / 11.8 / 17.7 us (two waves of 16); 360 pairs of
// 2,048: one CTA 64, two 58, four 67. Pairs of which clusters of 16 leave places free get several clusters of
// 128 stages and more, joined by a second launch (4 us; one pair of 16,384 tokens: 17.4 -> 12).
void split_blocks(long long pairs, long long stages, const int (&at_once)[5], int* parts, int* shards) {
    long long best = 0, room = 0;
    *parts = *shards = 1;
    for (int i = 0; i < 5 && (i == 0 || stages >= 1 << i); ++i) {
        if (at_once[i] == 0) continue;
        const long long cost = (pairs + at_once[i] - 1) / at_once[i] * (18 * 16 + (stages * 16 >> i));
        if (best == 0 || cost < best) best = cost, *parts = 1 << i, room = at_once[i] / pairs;
    }
    if (*parts == 16) *shards = (int)std::max(1LL, std::min(room, stages / 128));
}

// Of 152 multiprocessors with room for one CTA or two, as the device has it: for plans made for a number of
// multiprocessors.
constexpr int kAtOnce[2][5] = {{152, 76, 36, 15, 7}, {304, 152, 74, 36, 14}};

kvd_status plan_blocks(int batch, int T, int Hq, int Hkv, int D, int K, int block_tokens, int num_sms, BlocksParams* p, size_t* ws) {
    kvd_status st = check_shape(batch, Hq, Hkv, D, KVD_OUT_BF16);
    if (st != KVD_OK) return st;
    if (T < 1 || K < 1 || num_sms < 0 || !power_of_two(block_tokens, 16, 4096)) return KVD_ERR_INVALID_ARG;
    if (T > KVD_MAX_TOKENS || K > kMaxKept || (long long)K * block_tokens > 0x3fffffffLL) return KVD_ERR_UNSUPPORTED;
    int at_once[5];
    for (int i = 0; i < 5; ++i) at_once[i] = (int)((long long)kAtOnce[D != 256][i] * num_sms / 152);
    at_once[0] = std::max(at_once[0], 1);
    if (num_sms == 0) {
        const cudaError_t e = D == 64    ? blocks_at_once_d64(at_once)
                              : D == 128 ? blocks_at_once_d128(at_once)
                                         : blocks_at_once_d256(at_once);
        if (e != cudaSuccess) return KVD_ERR_CUDA;
    }
    p->B = batch;
    p->T = T;
    p->Hq = Hq;
    p->Hkv = Hkv;
    p->G = Hq / Hkv;
    p->K = K;
    p->block_log2 = log2_of(block_tokens);
    const long long pairs = (long long)batch * T * Hkv;
    // Query rows to warps: 16 each (two column tiles), at head_dim 256, whose accumulators take the registers
    // of one, 8. As many teams as the warps give, with three stages each at least.
    p->head_rows = p->G <= 8 || D == 256 ? 8 : 16;
    p->head_warps = (p->G + p->head_rows - 1) / p->head_rows;
    p->teams = std::max(1, std::min(blocks_warps(D) / p->head_warps, blocks_slots(D) / 3));
    if (pairs > (1 << 26)) return KVD_ERR_UNSUPPORTED;
    p->pairs = (int)pairs;
    *ws = 0;
    p->parts = p->shards = 1;
    if (pairs == 0) return KVD_OK;
    split_blocks(pairs, std::max(1LL, (long long)K * block_tokens / kBlocksStage), at_once, &p->parts, &p->shards);
    if (p->shards > 1) {
        const size_t rows = (size_t)pairs * p->G;
        *ws = align256(p->shards * rows * D * sizeof(float)) + align256(p->shards * rows * sizeof(float));
    }
    return KVD_OK;
}

// Keys of a query token in the workspace: whole 16-byte vectors.
int select_key_stride(int max_seq_len, int block_tokens) { return (max_seq_len / block_tokens + 3) & ~3; }

kvd_status check_bounds(const kvd_block_bounds* b, int batch, int Hkv, int D, PagedCache* pg, int* cap, size_t* blocks) {
    if (!b || !power_of_two(b->block_tokens, 16, 4096) || batch < 0 || Hkv <= 0 || D <= 0) return KVD_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return KVD_ERR_UNSUPPORTED;
    long long rows = 0;
    const kvd_status st = check_place(b->block_table, b->s_max, b->max_blocks, b->page_size, b->num_pages, batch, pg, cap, &rows);
    if (st != KVD_OK) return st;
    if (b->block_table && b->block_tokens > b->page_size) return KVD_ERR_INVALID_ARG;
    *blocks = b->block_table ? (size_t)(rows / b->block_tokens) : (size_t)batch * (size_t)(b->s_max / b->block_tokens);
    if ((*blocks > 0 && (!b->codes || !b->scales)) || !aligned(b->codes, 16) || !aligned(b->scales, 4)) return KVD_ERR_INVALID_ARG;
    return KVD_OK;
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" {

kvd_status kvd_pages_update(int32_t* block_table, int32_t* free_pages, int32_t* free_count, int32_t* seq_lens,
                            const int32_t* new_lens, int batch, int max_blocks, int page_size, int num_pages, int32_t* pos,
                            int32_t* row_offsets, int32_t* slots, int32_t* positions, long long n_rows, int32_t* status_word,
                            kvd_stream_t stream) {
    if (batch < 0 || n_rows < 0 || n_rows > 0x7fffffffLL) return KVD_ERR_INVALID_ARG;
    PagedCache pg;
    int cap = 0;
    // (Without sequences there may be no table and no lengths; slots and positions are filled all the same.)
    const kvd_status st = check_paged(batch > 0 ? block_table : free_pages, max_blocks, page_size, num_pages, &pg, &cap);
    if (st != KVD_OK) return st;
    if ((long long)batch * max_blocks > 0x7fffffffLL) return KVD_ERR_INVALID_ARG;
    if (batch > kPagesMaxBatch) return KVD_ERR_UNSUPPORTED;
    const void* all[10] = {free_pages, free_count, block_table, seq_lens, new_lens, pos, row_offsets, slots, positions, status_word};
    for (int i = 0; i < 10; ++i)
        if ((i < (batch > 0 ? 5 : 2) && !all[i]) || (all[i] && !aligned(all[i], 4))) return KVD_ERR_INVALID_ARG;
    const size_t b4 = (size_t)batch * 4;
    const ByteRange r[9] = {{block_table, b4 * max_blocks}, {free_pages, (size_t)num_pages * 4}, {free_count, 4}, {seq_lens, b4},
                            {pos, pos ? b4 : 0}, {row_offsets, row_offsets ? b4 + 4 : 0}, {slots, slots ? (size_t)n_rows * 4 : 0},
                            {positions, positions ? (size_t)n_rows * 4 : 0}, {new_lens, b4}};
    if (!apart(r, 8, 9)) return KVD_ERR_INVALID_ARG;
    if (batch == 0 && n_rows == 0 && !row_offsets) return KVD_OK;
    const PagesParams p{block_table, free_pages, free_count, seq_lens, new_lens, pos, row_offsets, slots, positions, status_word,
                        batch, max_blocks, pg.page_shift, num_pages, n_rows};
    return launch_pages(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

kvd_status kvd_rope_axes_table(const int* sections, int n_axes, int dealt, int per_axis, double base, kvd_rope_scaling scaling,
                               double scale, double original_len, double slow, double fast, double attn_factor,
                               uint64_t* turns_host, uint8_t* axes_host, float* factor_out) {
    if (!sections || !turns_host || !axes_host || !factor_out || n_axes < 1 || n_axes > KVD_MAX_AXES) return KVD_ERR_INVALID_ARG;
    int half = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < (per_axis ? 8 : 1) || sections[a] > 128) return KVD_ERR_INVALID_ARG;
        half += sections[a];
    }
    if (half > 128 || half % 8 != 0) return KVD_ERR_INVALID_ARG;
    uint8_t axis[128];
    int number[128], seen[KVD_MAX_AXES] = {};  // a pair's axis, and its number among that axis' pairs
    for (int i = 0, a = 0; i < half; ++i) {
        while (seen[a] == sections[a]) a = dealt ? (a + 1) % n_axes : a + 1;
        axis[i] = (uint8_t)a;
        number[i] = seen[a]++;
        if (dealt) a = (a + 1) % n_axes;
    }
    uint64_t turns[128];
    float factor = 1.f;
    for (int a = 0; a < (per_axis ? n_axes : 1); ++a) {
        uint64_t own[128];
        const kvd_status st = rope_turns(per_axis ? sections[a] : half, base, scaling, scale, original_len, slow, fast, attn_factor,
                                         own, &factor);
        if (st != KVD_OK) return st;
        for (int i = 0; i < half; ++i)
            if (!per_axis || axis[i] == a) turns[i] = own[per_axis ? number[i] : i];
    }
    std::memcpy(turns_host, turns, (size_t)half * sizeof(uint64_t));
    std::memcpy(axes_host, axis, (size_t)half);
    *factor_out = factor;
    return KVD_OK;
}

kvd_status kvd_rope_apply_axes(const kvd_rope_axes* rope, const void* x, long long x_stride, kvd_out_dtype in_dtype, void* y,
                               long long y_stride, kvd_out_dtype out_dtype, const int32_t* positions, long long axis_stride,
                               long long rows, int n_heads, int head_dim, kvd_stream_t stream) {
    if (rows < 0 || rows > 0x7fffffffLL || n_heads < 1 || n_heads > (1 << 20) || head_dim < 8 || head_dim % 8 != 0)
        return KVD_ERR_INVALID_ARG;
    if (head_dim > 1024) return KVD_ERR_UNSUPPORTED;
    if ((in_dtype != KVD_OUT_BF16 && in_dtype != KVD_OUT_F32) || (out_dtype != KVD_OUT_BF16 && out_dtype != KVD_OUT_F32))
        return KVD_ERR_INVALID_ARG;
    RopeAxes r;
    kvd_status st = check_axes(rope, positions, axis_stride, rows, head_dim, &r);
    if (st != KVD_OK) return st;
    const size_t ies = in_dtype == KVD_OUT_F32 ? 4 : 2, oes = out_dtype == KVD_OUT_F32 ? 4 : 2;
    const long long width = (long long)n_heads * head_dim;
    if ((st = check_strided(x, x_stride, width, ies)) != KVD_OK) return st;
    if ((st = check_strided(y, y_stride, width, oes)) != KVD_OK) return st;
    const Rows rx{x, x_stride, width, rows, ies}, ry{y, y_stride, width, rows, oes};
    const bool in_place = x == y && x_stride == y_stride && in_dtype == out_dtype;
    if ((!in_place && rows_meet(rx, ry)) || ry.range().overlaps(ByteRange{positions, positions_bytes(r, rows)}))
        return KVD_ERR_INVALID_ARG;
    if (rows == 0) return KVD_OK;
    int sms = 0;
    if ((st = device_sms(&sms)) != KVD_OK) return st;
    return launch_rope_axes(r, x, x_stride, in_dtype == KVD_OUT_F32, y, y_stride, out_dtype == KVD_OUT_F32, rows, n_heads, head_dim, sms,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KVD_OK
               : KVD_ERR_CUDA;
}

kvd_status kvd_kv_append_axes(const kvd_cache* cache, const kvd_rope_axes* rope, const void* q, long long q_stride, void* q_out,
                              long long q_out_stride, const void* k_new, long long k_stride, const void* v_new, long long v_stride,
                              const int32_t* slots, const int32_t* positions, long long axis_stride, int batch, long long n_rows,
                              int n_heads_q, int n_heads_kv, int head_dim, int32_t* status_word, kvd_stream_t stream) {
    if (!cache || batch < 0 || n_rows < 0 || n_rows > 0x7fffffffLL || n_heads_kv <= 0 || head_dim < 8 || head_dim % 8 != 0)
        return KVD_ERR_INVALID_ARG;
    const bool quant = cache->k_scales || cache->v_scales;
    if (quant && (!cache->k_scales || !cache->v_scales || !aligned(cache->k_scales, 4) || !aligned(cache->v_scales, 4)))
        return KVD_ERR_INVALID_ARG;
    if (cache->fp8 && !quant) return KVD_ERR_INVALID_ARG;
    if (quant ? (head_dim != 64 && head_dim != 128 && head_dim != 256) : head_dim > 1024) return KVD_ERR_UNSUPPORTED;
    if (!cache->k || !cache->v || !aligned(cache->k, 16) || !aligned(cache->v, 16) || (status_word && !aligned(status_word, 4)))
        return KVD_ERR_INVALID_ARG;
    // The slots name rows of the cache; a paged cache's table has no part in this call.
    long long rows = (long long)batch * cache->s_max;
    if (cache->page_size != 0 || cache->num_pages != 0) {
        if (!power_of_two(cache->page_size, 16, 4096) || cache->num_pages < 1) return KVD_ERR_INVALID_ARG;
        rows = (long long)cache->num_pages * cache->page_size;
    } else if (cache->s_max <= 0) {
        return KVD_ERR_INVALID_ARG;
    }
    if (rows > 0x7fffffffLL || (rows == 0 && n_rows > 0)) return KVD_ERR_INVALID_ARG;
    if ((q != nullptr) != (q_out != nullptr) || n_heads_kv > (1 << 20) || (q && (n_heads_q < 1 || n_heads_q > (1 << 20))))
        return KVD_ERR_INVALID_ARG;
    if (!slots || !aligned(slots, 4)) return KVD_ERR_INVALID_ARG;
    RopeAxes r;
    kvd_status st = check_axes(rope, positions, axis_stride, n_rows, head_dim, &r);
    if (st != KVD_OK) return st;
    const long long kw = (long long)n_heads_kv * head_dim, qw = q ? (long long)n_heads_q * head_dim : 0;
    if ((st = check_strided(k_new, k_stride, kw, 2)) != KVD_OK) return st;
    if ((st = check_strided(v_new, v_stride, kw, 2)) != KVD_OK) return st;
    if (q) {
        if ((st = check_strided(q, q_stride, qw, 2)) != KVD_OK) return st;
        if ((st = check_strided(q_out, q_out_stride, qw, 2)) != KVD_OK) return st;
    }
    if (n_rows == 0) return KVD_OK;
    const Rows rk{k_new, k_stride, kw, n_rows, 2}, rv{v_new, v_stride, kw, n_rows, 2}, rq{q, q_stride, qw, n_rows, 2},
        ro{q_out, q_out_stride, qw, n_rows, 2};
    const ByteRange none{nullptr, 0}, rp{positions, positions_bytes(r, n_rows)}, rs{slots, (size_t)n_rows * 4};
    const bool in_place = q && q == q_out;
    if (in_place && q_stride != q_out_stride) return KVD_ERR_INVALID_ARG;
    if (q && ((!in_place && rows_meet(ro, rq)) || rows_meet(ro, rk) || rows_meet(ro, rv) || ro.range().overlaps(rp) ||
              ro.range().overlaps(rs)))
        return KVD_ERR_INVALID_ARG;
    const size_t cbytes = (size_t)rows * kw * (quant ? 1 : 2), sbytes = quant ? (size_t)rows * n_heads_kv * 4 : 0;
    const ByteRange ranges[10] = {{cache->k, cbytes}, {cache->v, cbytes}, {cache->k_scales, sbytes}, {cache->v_scales, sbytes},
                                  rk.range(), rv.range(), q ? rq.range() : none, q ? ro.range() : none, rp, rs};
    if (!apart(ranges, 4, 10)) return KVD_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != KVD_OK) return st;
    const AppendTarget to{cache->k, cache->v, cache->k_scales, cache->v_scales,
                          quant ? (cache->fp8 ? CacheForm::kFp8 : CacheForm::kInt8) : CacheForm::kBf16, 0,
                          PagedCache{nullptr, 0, 0, 0}};
    const NewRows in{q, q_out, k_new, v_new, q_stride, q_out_stride, k_stride, v_stride, nullptr, nullptr, 0, 0, q ? n_heads_q : 0,
                     n_heads_kv, head_dim, n_rows};
    return launch_append_axes(to, r, in, slots, rows, status_word, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KVD_OK
               : KVD_ERR_CUDA;
}

kvd_status kvd_kv_block_bounds(const void* k_cache, const kvd_block_bounds* bounds, const int32_t* from_lens, const int32_t* seq_lens,
                               int batch, int max_new, int n_heads_kv, int head_dim, int32_t* status_word, kvd_stream_t stream) {
    PagedCache pg;
    int cap = 0;
    size_t blocks = 0;
    const kvd_status st = check_bounds(bounds, batch, n_heads_kv, head_dim, &pg, &cap, &blocks);
    if (st != KVD_OK) return st;
    if (max_new < 0 || !k_cache || !seq_lens || !aligned(k_cache, 16) || !aligned(seq_lens, 4) ||
        (from_lens && !aligned(from_lens, 4)) || (status_word && !aligned(status_word, 4)))
        return KVD_ERR_INVALID_ARG;
    const long long rows =
        bounds->block_table ? (long long)bounds->num_pages * bounds->page_size : (long long)batch * bounds->s_max;
    const size_t heads = blocks * n_heads_kv;
    const ByteRange r[5] = {{bounds->codes, heads * 2 * head_dim}, {bounds->scales, heads * 4},
                            {k_cache, (size_t)rows * n_heads_kv * head_dim * 2}, {seq_lens, (size_t)batch * 4},
                            {from_lens, from_lens ? (size_t)batch * 4 : 0}};
    if (!apart(r, 2, 5)) return KVD_ERR_INVALID_ARG;
    if (batch == 0 || max_new == 0) return KVD_OK;
    const int span = std::min(max_new, cap);
    const long long per = ((long long)span + bounds->block_tokens - 1) / bounds->block_tokens;
    if (per * batch * n_heads_kv > 0x7fffffffLL) return KVD_ERR_UNSUPPORTED;
    const BoundsParams p{k_cache, bounds->codes, bounds->scales, from_lens, seq_lens, status_word, batch, n_heads_kv, head_dim, cap,
                         log2_of(bounds->block_tokens), span, pg};
    return launch_block_bounds(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

kvd_status kvd_block_select_plan(int batch, int n_tokens, int n_heads_kv, int max_seq_len, int block_tokens,
                                 size_t* workspace_bytes_out) {
    if (!workspace_bytes_out || batch < 0 || n_tokens < 1 || n_heads_kv <= 0 || max_seq_len < 0 ||
        !power_of_two(block_tokens, 16, 4096))
        return KVD_ERR_INVALID_ARG;
    if (n_tokens > KVD_MAX_TOKENS) return KVD_ERR_UNSUPPORTED;
    *workspace_bytes_out = align256((size_t)batch * n_tokens * n_heads_kv * select_key_stride(max_seq_len, block_tokens) * 4);
    return KVD_OK;
}

kvd_status kvd_block_select(const kvd_block_bounds* bounds, const void* q, const int32_t* seq_lens, int batch, int n_tokens,
                            int max_seq_len, int n_keep, int n_first, int n_last, int n_heads_q, int n_heads_kv, int head_dim,
                            void* workspace, size_t workspace_bytes, int32_t* blocks_out, int32_t* status_word, kvd_stream_t stream) {
    kvd_status st = check_shape(batch, n_heads_q, n_heads_kv, head_dim, KVD_OUT_BF16);
    if (st != KVD_OK) return st;
    PagedCache pg;
    int cap = 0;
    size_t blocks = 0, need = 0;
    st = check_bounds(bounds, batch, n_heads_kv, head_dim, &pg, &cap, &blocks);
    if (st != KVD_OK) return st;
    st = kvd_block_select_plan(batch, n_tokens, n_heads_kv, max_seq_len, bounds->block_tokens, &need);
    if (st != KVD_OK) return st;
    if (max_seq_len / bounds->block_tokens > cap / bounds->block_tokens || n_keep < 1 || n_first < 0 || n_last < 1 ||
        (long long)n_first + n_last > n_keep)
        return KVD_ERR_INVALID_ARG;
    if (n_keep > kMaxKept) return KVD_ERR_UNSUPPORTED;
    if (!q || !seq_lens || !blocks_out || !aligned(q, 16) || !aligned(seq_lens, 4) || !aligned(blocks_out, 4) ||
        (status_word && !aligned(status_word, 4)))
        return KVD_ERR_INVALID_ARG;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return KVD_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 256)) return KVD_ERR_INVALID_ARG;
    }
    const size_t heads = blocks * n_heads_kv;
    const ByteRange r[6] = {{blocks_out, (size_t)batch * n_tokens * n_heads_kv * n_keep * 4}, {workspace, need},
                            {q, (size_t)batch * n_tokens * n_heads_q * head_dim * 2}, {seq_lens, (size_t)batch * 4},
                            {bounds->codes, heads * 2 * head_dim}, {bounds->scales, heads * 4}};
    if (!apart(r, 2, 6)) return KVD_ERR_INVALID_ARG;
    const long long pairs = (long long)batch * n_heads_kv;
    if (pairs * n_tokens > 0x7fffffffLL) return KVD_ERR_UNSUPPORTED;
    if (batch == 0) return KVD_OK;
    int sms = 0;
    if ((st = device_sms(&sms)) != KVD_OK) return st;
    SelectParams p;
    std::memset(&p, 0, sizeof p);
    p.q = q;
    p.codes = bounds->codes;
    p.scales = bounds->scales;
    p.seq_lens = seq_lens;
    p.blocks = blocks_out;
    p.status = status_word;
    p.keys = static_cast<uint32_t*>(workspace);
    p.B = batch;
    p.T = n_tokens;
    p.Hq = n_heads_q;
    p.Hkv = n_heads_kv;
    p.G = n_heads_q / n_heads_kv;
    p.D = head_dim;
    p.K = n_keep;
    p.S_max = cap;
    p.len_cap = max_seq_len;
    p.block_shift = log2_of(bounds->block_tokens);
    p.n_first = n_first;
    p.n_last = n_last;
    p.key_stride = select_key_stride(max_seq_len, bounds->block_tokens);
    p.pg = pg;
    // CTAs of a pair: for about three rounds of those that are resident, as far as every warp has a tile of 16
    // blocks. One / two / three / four / six rounds, us: 32 sequences of 16,384 to 131,072 tokens in blocks of
    // 32, 32 heads on 8 of 128, 46.5 / 42.2 / 41.3 / 42.1 / 43.4; of 64 columns 40.6 / 36.3 / 35.6 / 36.4 / 37.6;
    // 4 query tokens 71 / 67.2 / 66.8 / 67.2 / 70.4; 64 sequences, 48 heads on one of 256, 60.2 / 57.1 / 56.5 /
    // 58.8 / 56.9. One sequence of 65,536 blocks alone would have one round: 70 against 74.
    const int tiles_cta = head_dim == 256 ? 16 : 8;
    const long long tiles = (p.key_stride + 15LL) / 16;
    const long long three = (3LL * select_ctas(head_dim, p.G, n_tokens) * sms + pairs - 1) / pairs;
    const int parts = (int)std::max(1LL, std::min(three, (tiles + tiles_cta - 1) / tiles_cta));
    if (pairs * parts > 0x7fffffffLL) return KVD_ERR_UNSUPPORTED;
    p.parts = parts;
    return launch_block_select(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

kvd_status kvd_decode_blocks_plan(int batch, int n_tokens, int n_heads_q, int n_heads_kv, int head_dim, int n_blocks,
                                  int block_tokens, int num_sms, size_t* workspace_bytes_out) {
    if (!workspace_bytes_out) return KVD_ERR_INVALID_ARG;
    BlocksParams p;
    return plan_blocks(batch, n_tokens, n_heads_q, n_heads_kv, head_dim, n_blocks, block_tokens, num_sms, &p, workspace_bytes_out);
}

kvd_status kvd_decode_blocks(const kvd_cache* cache, const void* q, const int32_t* blocks, const int32_t* seq_lens, int batch,
                             int n_tokens, int n_blocks, int block_tokens, int n_heads_q, int n_heads_kv, int head_dim, float scale,
                             void* workspace, size_t workspace_bytes, void* out, kvd_out_dtype out_dtype, float* lse_out,
                             int32_t* status_word, kvd_stream_t stream) {
    if (!cache) return KVD_ERR_INVALID_ARG;
    kvd_status st = check_shape(batch, n_heads_q, n_heads_kv, head_dim, out_dtype);
    if (st != KVD_OK) return st;
    if (cache->k_scales || cache->v_scales || cache->fp8) return KVD_ERR_UNSUPPORTED;  // bf16 caches
    BlocksParams p;
    std::memset(&p, 0, sizeof p);
    int cap = 0;
    long long rows = 0;
    st = check_place(cache->block_table, cache->s_max, cache->max_blocks, cache->page_size, cache->num_pages, batch, &p.pg, &cap,
                     &rows);
    if (st != KVD_OK) return st;
    if (rows > 0x7fffffffLL - 16) return KVD_ERR_UNSUPPORTED;  // TMA coordinates are 32-bit
    if (!std::isfinite(scale)) return KVD_ERR_INVALID_ARG;
    if (!cache->k || !cache->v || !q || !blocks || !seq_lens || !out || !aligned(cache->k, 16) || !aligned(cache->v, 16) ||
        !aligned(q, 16) || !aligned(blocks, 4) || !aligned(seq_lens, 4) || !aligned(out, 16) || (lse_out && !aligned(lse_out, 4)) ||
        (status_word && !aligned(status_word, 4)))
        return KVD_ERR_INVALID_ARG;
    size_t need = 0;
    st = plan_blocks(batch, n_tokens, n_heads_q, n_heads_kv, head_dim, n_blocks, block_tokens, 0, &p, &need);
    if (st != KVD_OK) return st;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return KVD_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 256)) return KVD_ERR_INVALID_ARG;
    }
    if (batch == 0) return KVD_OK;
    p.unit_log2 = block_tokens >= 32 && (!p.pg.block_table || p.pg.page_shift >= 5) ? 5 : 4;
    const bool f32 = out_dtype == KVD_OUT_F32;
    const size_t out_rows = (size_t)p.pairs * p.G;
    p.q = q;
    p.k = cache->k;
    p.v = cache->v;
    p.blocks = blocks;
    p.seq_lens = seq_lens;
    p.status = status_word;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.S_max = cap;
    p.out = out;
    p.lse = lse_out;
    if (p.shards > 1) {
        uint8_t* w = static_cast<uint8_t*>(workspace);
        p.out = w;
        p.lse = reinterpret_cast<float*>(w + align256(p.shards * out_rows * head_dim * sizeof(float)));
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool run_f32 = f32 || p.shards > 1;
    const cudaError_t e = head_dim == 64    ? launch_decode_blocks_d64(p, run_f32, s)
                          : head_dim == 128 ? launch_decode_blocks_d128(p, run_f32, s)
                                            : launch_decode_blocks_d256(p, run_f32, s);
    if (e != cudaSuccess) return KVD_ERR_CUDA;
    if (p.shards > 1 &&
        launch_merge_shards(p.out, p.lse, p.shards, (long long)out_rows, head_dim, true, out, f32, lse_out, s) != cudaSuccess)
        return KVD_ERR_CUDA;
    return KVD_OK;
}

}  // extern "C"
