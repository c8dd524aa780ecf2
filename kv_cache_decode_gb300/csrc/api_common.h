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

kvd_status check_shape(int batch, int Hq, int Hkv, int D, kvd_out_dtype dt);
// Paged cache arguments, checked; s_max of the contiguous calls becomes
// max_blocks * page_size.
kvd_status check_paged(const int32_t* block_table, int max_blocks, int page_size, int num_pages, PagedCache* pg,
                       int* s_max);
kvd_status check_append(void* k_cache, void* v_cache, const void* k_new, const void* v_new, const int32_t* pos,
                        int batch, int s_max, int Hkv, int D, const int32_t* status);
kvd_status device_sms(int* sms);
size_t workspace_for(int n_split, int batch, int Hq, int Hkv, int D);

}  // namespace kvd
