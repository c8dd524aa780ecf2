// Page tables, slots and positions from request lengths. Sequence b goes from seq_lens[b] tokens to new_lens[b]: the pages
// it gives up go back on the stack of free ones, then pages that it needs come from its top, in order of sequence and
// block, as long as the running sum of what is needed fits. With prefix sums over the
// sequences every page's place on the stack is a matter of arithmetic, so nothing is counted by atomics and the
// same call always gives the same table. Released pages are laid down in reverse, so that a shrink right behind a growth leaves
// the stack as it was.
//
// One launch: a CTA, or a cluster of up to 16 where many slots are written; every CTA forms the prefix sums for itself in
// shared memory (a few thousand integers at most), and barriers part the release, the growth and the slots. Bound by latency.
#include <algorithm>

#include "../../include/kvdecode.h"
#include "api_common.h"
#include "blocks.h"
#include "cluster.cuh"

namespace kvd {

constexpr int kPagesThreads = 512;

// First index i in [0, n) with a[i + 1] > x, for a not decreasing with a[n] > x.
__device__ __forceinline__ int owner_of(const int* a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Exclusive prefix sums of two numbers over the block; tot receives their sums.
__device__ __forceinline__ void block_scan2(long long (&v)[2], long long (&tot)[2], long long (*s_warp)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long own[2] = {v[0], v[1]};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long n = __shfl_up_sync(0xffffffffu, v[k], off);
            if (lane >= off) v[k] += n;
        }
    if (lane == 31) s_warp[warp][0] = v[0], s_warp[warp][1] = v[1];
    __syncthreads();
    long long pre[2] = {0, 0};
    tot[0] = tot[1] = 0;
    for (int w = 0; w < kPagesThreads / 32; ++w)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (w < warp) pre[k] += s_warp[w][k];
            tot[k] += s_warp[w][k];
        }
    __syncthreads();
    v[0] += pre[0] - own[0];
    v[1] += pre[1] - own[1];
}

__global__ void __launch_bounds__(kPagesThreads, 1) pages_kernel(const PagesParams p, int parts) {
    extern __shared__ int s_dyn[];  // four arrays of B + 1
    __shared__ long long s_warp[kPagesThreads / 32][2];
    int* s_old = s_dyn;                 // length before
    int* s_rel = s_old + p.B + 1;       // pages released before sequence b, then by all
    int* s_need = s_rel + p.B + 1;      // pages taken before sequence b
    int* s_row = s_need + p.B + 1;      // new tokens before sequence b
    const int tid = threadIdx.x, rank = blockIdx.x, shift = p.page_shift, psize = 1 << shift;
    const int cap = p.max_blocks << shift;
    const int gtid = rank * kPagesThreads + tid, gthreads = parts * kPagesThreads;
    auto pages_of = [&](int len) { return (int)(((long long)len + psize - 1) >> shift); };
    auto sync = [&]() {
        if (parts > 1)
            cluster_sync();
        else
            __syncthreads();
    };
    int flags = 0;
    int F = __ldcg(p.free_count);
    if (F < 0 || F > p.num_pages) {
        F = F < 0 ? 0 : p.num_pages;
        flags |= KVD_STATUS_BAD_PAGE;
    }
    auto lengths = [&](int b, int& old, int& want) {
        const int raw = __ldcg(p.seq_lens + b);
        old = raw < 0 ? 0 : raw > cap ? cap : raw;
        if (raw != old) flags |= KVD_STATUS_SEQ_LEN_CLAMPED;
        want = __ldg(p.new_lens + b);
        if (want < 0 || want > cap) {  // a length the table cannot hold: the sequence stays as it is
            want = old;
            flags |= KVD_STATUS_POS_OUT_OF_RANGE;
        }
    };
    // ---- pages released and pages needed before each sequence (batch * max_blocks is below 2^31) ----
    long long released = 0, needed = 0, tot[2];
    for (int b0 = 0; b0 < p.B; b0 += kPagesThreads) {
        const int b = b0 + tid;
        int old = 0, want = 0;
        if (b < p.B) lengths(b, old, want);
        long long v[2] = {max(pages_of(old) - pages_of(want), 0), max(pages_of(want) - pages_of(old), 0)};
        block_scan2(v, tot, s_warp);
        if (b < p.B) {
            s_old[b] = old;
            s_row[b] = want;
            s_rel[b] = (int)(released + v[0]);
            s_need[b] = (int)(needed + v[1]);
        }
        released += tot[0];
        needed += tot[1];
    }
    const int R = (int)released;
    // ---- a sequence grows when all that is needed up to it fits; one that needs no page always ----
    const long long have = (long long)F + R;
    long long taken_l = 0, rows_l = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPagesThreads) {
        const int b = b0 + tid;
        int old = 0, want = 0, need = 0;
        if (b < p.B) {  // (this thread's own entries)
            old = s_old[b], want = s_row[b];
            need = max(pages_of(want) - pages_of(old), 0);
            if (need > 0 && (long long)s_need[b] + need > have) {
                need = 0;
                want = old;
                flags |= KVD_STATUS_NO_PAGES;
            }
        }
        long long v[2] = {need, max(want - old, 0)};
        block_scan2(v, tot, s_warp);
        if (b < p.B) {
            s_need[b] = (int)(taken_l + v[0]);
            s_row[b] = (int)min(rows_l + v[1], 0x7fffffffLL);
            if (rank == 0) {
                if (p.pos) p.pos[b] = old;
                if (p.offsets) p.offsets[b] = s_row[b];
            }
        }
        taken_l += tot[0];
        rows_l += tot[1];
    }
    const int taken = (int)taken_l, rows = (int)min(rows_l, 0x7fffffffLL);
    if (tid == 0) {
        s_rel[p.B] = R;
        s_need[p.B] = taken;
        s_row[p.B] = rows;
        if (rank == 0 && p.offsets) p.offsets[p.B] = rows;
    }
    if ((p.slots || p.positions) && rows > p.rows) flags |= KVD_STATUS_POS_OUT_OF_RANGE;  // rows behind the buffers are not written
    sync();  // every CTA has read the lengths and the count
    // ---- released pages: the r-th in order of sequence and block to place F + R - 1 - r of the stack ----
    for (int r = gtid; r < R; r += gthreads) {
        const int b = owner_of(s_rel, p.B, r), held = pages_of(s_old[b]), n = s_rel[b + 1] - s_rel[b];
        int32_t* e = p.table + (size_t)b * p.max_blocks + (held - n + (r - s_rel[b]));
        const int page = *e;
        const long long at = have - 1 - r;
        *e = -1;
        if ((unsigned)page >= (unsigned)p.num_pages) flags |= KVD_STATUS_BAD_PAGE;
        if (at < p.num_pages)
            p.free_pages[at] = page;
        else
            flags |= KVD_STATUS_BAD_PAGE;  // more pages come back than the pool has
    }
    const int top = (int)min(have, (long long)p.num_pages);
    sync();
    // ---- pages taken: the i-th from place top - 1 - i ----
    for (int i = gtid; i < taken; i += gthreads) {
        const int b = owner_of(s_need, p.B, i), held = pages_of(s_old[b]);
        const int at = top - 1 - i, page = at >= 0 ? __ldcg(p.free_pages + at) : -1;
        if ((unsigned)page >= (unsigned)p.num_pages) flags |= KVD_STATUS_BAD_PAGE;
        p.table[(size_t)b * p.max_blocks + held + (i - s_need[b])] = page;
    }
    if (rank == 0) {
        if (tid == 0) *p.free_count = max(top - taken, 0);
        for (int b = tid; b < p.B; b += kPagesThreads) {
            const int old = s_old[b], grown = s_row[b + 1] - s_row[b];
            int len = old + grown;
            if (grown == 0) {  // shorter, the same, or not given
                const int want = __ldg(p.new_lens + b);
                if (want >= 0 && want < old) len = want;
            }
            p.seq_lens[b] = len;
        }
    }
    if (p.slots || p.positions) {
        sync();
        const long long total = min((long long)rows, p.rows);
        // A warp takes a stretch of rows, 128 at a time, four neighbours a lane: the sequence is searched for once, then
        // followed; four steps' table entries are on the way at once.
        const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
        const int lane = tid & 31, gwarp = gtid >> 5, gwarps = gthreads >> 5;
        const long long per = ((p.rows + gwarps - 1) / gwarps + 127) & ~127LL;
        const long long end = min(p.rows, (gwarp + 1) * per);
        long long n0 = gwarp * per + 4 * lane;
        int b = n0 < total ? owner_of(s_row, p.B, (int)n0) : 0;
        for (; n0 < end; n0 += 512) {
            int slot[4][4], at[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const long long n = n0 + 128 * u + k;
                    slot[u][k] = at[u][k] = -1;
                    if (n < min(total, end)) {
                        while (n >= s_row[b + 1]) ++b;
                        at[u][k] = s_old[b] + ((int)n - s_row[b]);
                        slot[u][k] = __ldcg(p.table + (size_t)b * p.max_blocks + (at[u][k] >> shift));
                    }
                }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (at[u][k] >= 0) {
                        if ((unsigned)slot[u][k] >= (unsigned)p.num_pages) {
                            flags |= KVD_STATUS_BAD_PAGE;
                            slot[u][k] = -1;
                        } else {
                            slot[u][k] = (slot[u][k] << shift) + (at[u][k] & (psize - 1));
                        }
                    }
                const long long n = n0 + 128 * u;
                if (n >= end) break;
                if (wide && n + 4 <= end) {
                    if (p.slots) *reinterpret_cast<int4*>(p.slots + n) = make_int4(slot[u][0], slot[u][1], slot[u][2], slot[u][3]);
                    if (p.positions) *reinterpret_cast<int4*>(p.positions + n) = make_int4(at[u][0], at[u][1], at[u][2], at[u][3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (n + k < end) {
                            if (p.slots) p.slots[n + k] = slot[u][k];
                            if (p.positions) p.positions[n + k] = at[u][k];
                        }
                }
            }
        }
    }
    if (flags && p.status) atomicOr(p.status, flags);
}

cudaError_t launch_pages(const PagesParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    const int smem = 4 * (p.B + 1) * (int)sizeof(int);
    const cudaError_t e = allow_clusters(reinterpret_cast<const void*>(pages_kernel), 4 * (kPagesMaxBatch + 1) * (int)sizeof(int), &ready);
    if (e != cudaSuccess) return e;
    // A CTA for 4,096 rows, which it writes in two steps of its threads.
    int parts = 1;
    while (parts < 16 && (p.slots || p.positions) && (long long)parts * 4096 < p.rows) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)parts, 1, 1);
    cfg.blockDim = dim3(kPagesThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pages_kernel, p, parts);
}

}  // namespace kvd
