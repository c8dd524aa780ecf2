// Argument checks and planning shared by the C entry points (defined in api.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/kvdecode.h"
#include "params.h"

namespace kvd {

constexpr int kMaxDevices = 64;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// A byte range [p, p + n) of device memory; empty when n == 0.
struct ByteRange {
    const void* p;
    size_t n;
    bool overlaps(const ByteRange& o) const {
        if (n == 0 || o.n == 0) return false;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return a < b + o.n && b < a + n;
    }
};

// Bytes from the first to the last element of `rows` rows of `width` elements `stride` apart.
inline size_t span_bytes(long long rows, long long stride, long long width, size_t es) {
    return rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * es : 0;
}

// Whether two sets of rows share an element. Rows of one buffer (one stride, a fused projection's slices) are apart
// when their column windows are.
struct Rows {
    const void* p;
    long long stride, width, n;
    size_t es;
    ByteRange range() const { return ByteRange{p, span_bytes(n, stride, width, es)}; }
};
inline bool rows_meet(const Rows& a, const Rows& b) {
    if (!a.range().overlaps(b.range())) return false;
    const long long S = a.stride * (long long)a.es;
    if (S != b.stride * (long long)b.es) return true;
    long long d = (long long)((intptr_t)b.p - (intptr_t)a.p) % S;
    if (d < 0) d += S;  // b starts d bytes into a's row period
    return d < a.width * (long long)a.es || d + b.width * (long long)b.es > S;
}

inline kvd_status check_strided(const void* p, long long stride, long long width, size_t es) {
    if (!p || !aligned(p, 16) || stride < width || stride > (1LL << 40) || (stride * (long long)es) % 16 != 0)
        return KVD_ERR_INVALID_ARG;
    return KVD_OK;
}

kvd_status check_shape(int batch, int Hq, int Hkv, int D, kvd_out_dtype dt);
// Paged cache arguments, checked; s_max of the contiguous calls becomes
// max_blocks * page_size.
kvd_status check_paged(const int32_t* block_table, int max_blocks, int page_size, int num_pages, PagedCache* pg,
                       int* s_max);
kvd_status check_append(void* k_cache, void* v_cache, const void* k_new, const void* v_new, const int32_t* pos,
                        int batch, int s_max, int Hkv, int D, const int32_t* status);
kvd_status device_sms(int* sms);
// The frequencies of 8 to 128 pairs that share a table (api_fp4.cu).
kvd_status rope_turns(int pairs, double base, kvd_rope_scaling scaling, double scale, double original_len, double slow, double fast,
                      double attn_factor, uint64_t* turns_host, float* factor_out);
size_t workspace_for(int n_split, int batch, int Hq, int Hkv, int D);

}  // namespace kvd
