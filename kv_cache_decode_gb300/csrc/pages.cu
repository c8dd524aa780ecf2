// Page tables, slots and positions from request lengths. Sequence b goes from seq_lens[b] tokens to
// new_lens[b]: the pages it gives up go back on the stack of free ones, then pages that it needs come from its
// top, in order of sequence and block, as long as the running sum of what is needed fits. With prefix sums over
// the sequences every page's place on the stack is a matter of arithmetic, so nothing is counted by atomics and
// the same call always gives the same table. Released pages are laid down in reverse, so that a shrink right
// behind a growth leaves the stack as it was.
//
// One launch: a CTA, or a cluster of up to 16 where many slots are written; every CTA forms the prefix sums for
// itself in shared memory (16 bytes a sequence: up to 131 KB for 8,192 of them), and barriers part the release,
// the growth and the slots. Bound by latency (a growth by 5 tokens of 64 sequences and the shrink back: 9.6 us
// for the two), for prompts by the slots' stores from 16 multiprocessors (up to 4,096 tokens each with slots and
// positions, and back: 24 prompts 12 us, 256 30).
#include <algorithm>

#include "../../include/kvdecode.h"
#include "api_common.h"
#include "blocks.h"
#include "cluster.cuh"

namespace kvd {

constexpr int kPagesThreads = 1024;

// First index i in [0, n) with a[i + 1] > x, for a not decreasing with a[n] > x.
__device__ __forceinline__ int owner_of(const int* a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Exclusive prefix sums of two numbers over the block; tot receives their sums. s_warp: not used by the call
// before this one.
__device__ __forceinline__ void block_scan2(uint32_t (&v)[2], uint32_t (&tot)[2], uint32_t (*s_warp)[2]) {
    static_assert(kPagesThreads == 1024, "a lane a warp");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t own[2] = {v[0], v[1]};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, v[k], off);
            if (lane >= off) v[k] += n;
        }
    if (lane == 31) s_warp[warp][0] = v[0], s_warp[warp][1] = v[1];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t x = s_warp[lane][k];
        tot[k] = __reduce_add_sync(0xffffffffu, x);
        v[k] += __reduce_add_sync(0xffffffffu, lane < warp ? x : 0u) - own[k];
    }
}

__global__ void __launch_bounds__(kPagesThreads, 1) pages_kernel(const PagesParams p, int parts) {
    extern __shared__ int s_dyn[];  // four arrays of B + 1
    __shared__ uint32_t s_warp[2][kPagesThreads / 32][2];
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
    uint32_t released = 0, needed = 0, tot[2];
    int turn = 0;  // of the scan's two buffers
    for (int b0 = 0; b0 < p.B; b0 += kPagesThreads) {
        const int b = b0 + tid;
        int old = 0, want = 0;
        if (b < p.B) lengths(b, old, want);
        const int more = pages_of(want) - pages_of(old);
        uint32_t v[2] = {(uint32_t)max(-more, 0), (uint32_t)max(more, 0)};
        block_scan2(v, tot, s_warp[turn ^= 1]);
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
    // (Where lengths claim more pages than the pool has, the stack ends with the pool: never more than
    // num_pages are given out, so that the tokens of those, below 2^31, and of every sequence's last page
    // before are below 2^32.)
    const long long have = (long long)F + R;
    const int top = (int)min(have, (long long)p.num_pages);
    uint32_t taken_u = 0, rows_u = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPagesThreads) {
        const int b = b0 + tid;
        int old = 0, want = 0, need = 0;
        if (b < p.B) {  // (this thread's own entries)
            old = s_old[b], want = s_row[b];
            need = max(pages_of(want) - pages_of(old), 0);
            if (need > 0 && (long long)s_need[b] + need > top) {
                need = 0;
                want = old;
                flags |= KVD_STATUS_NO_PAGES;
            }
        }
        uint32_t v[2] = {(uint32_t)need, (uint32_t)max(want - old, 0)};
        block_scan2(v, tot, s_warp[turn ^= 1]);
        if (b < p.B) {
            s_need[b] = (int)(taken_u + v[0]);
            s_row[b] = (int)min(rows_u + v[1], 0x7fffffffu);
            if (rank == 0) {
                if (p.pos) p.pos[b] = old;
                if (p.offsets) p.offsets[b] = s_row[b];
            }
        }
        taken_u += tot[0];
        rows_u += tot[1];
    }
    const int taken = (int)taken_u, rows = (int)min(rows_u, 0x7fffffffu);
    if (tid == 0) {
        s_rel[p.B] = R;
        s_need[p.B] = taken;
        s_row[p.B] = rows;
        if (rank == 0 && p.offsets) p.offsets[p.B] = rows;
    }
    if ((p.slots || p.positions) && rows > p.rows) flags |= KVD_STATUS_POS_OUT_OF_RANGE;  // rows behind the buffers are not written
    sync();  // every CTA has read the lengths and the count
    // ---- released pages: the r-th in order of sequence and block to place F + R - 1 - r of the stack ----
#pragma unroll 4
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
    sync();
    // ---- pages taken: the i-th from place top - 1 - i (taken <= top) ----
#pragma unroll 4
    for (int i = gtid; i < taken; i += gthreads) {
        const int b = owner_of(s_need, p.B, i), held = pages_of(s_old[b]);
        const int page = __ldcg(p.free_pages + (top - 1 - i));
        if ((unsigned)page >= (unsigned)p.num_pages) flags |= KVD_STATUS_BAD_PAGE;
        p.table[(size_t)b * p.max_blocks + held + (i - s_need[b])] = page;
    }
    if (rank == 0) {
        if (tid == 0) *p.free_count = top - taken;
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
        // A warp takes a stretch of rows, 128 at a time, four neighbours a lane: the sequence is searched for
        // once, then followed; two steps' table entries are on the way at once.
        const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
        auto put = [&](long long n, long long end, const int (&slot)[4], const int (&at)[4]) {
            if (wide && n + 4 <= end) {
                if (p.slots) *reinterpret_cast<int4*>(p.slots + n) = make_int4(slot[0], slot[1], slot[2], slot[3]);
                if (p.positions) *reinterpret_cast<int4*>(p.positions + n) = make_int4(at[0], at[1], at[2], at[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (n + k < end) {
                        if (p.slots) p.slots[n + k] = slot[k];
                        if (p.positions) p.positions[n + k] = at[k];
                    }
            }
        };
        const int lane = tid & 31, gwarp = gtid >> 5, gwarps = gthreads >> 5;
        const long long per = ((total + gwarps - 1) / gwarps + 127) & ~127LL;
        const long long end = min(total, (gwarp + 1) * per);
        long long n0 = gwarp * per + 4 * lane;
        int b = n0 < end ? owner_of(s_row, p.B, (int)n0) : 0;
        for (; n0 < end; n0 += 256) {
            int slot[2][4], at[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const long long n = n0 + 128 * u + k;
                    slot[u][k] = at[u][k] = -1;
                    if (n < end) {
                        const int was = b;
                        while (n >= s_row[b + 1]) ++b;
                        at[u][k] = s_old[b] + ((int)n - s_row[b]);
                        // (neighbours of one sequence on one page: one entry for both)
                        if (k > 0 && b == was && (at[u][k] & (psize - 1)) != 0)
                            slot[u][k] = slot[u][k - 1];
                        else
                            slot[u][k] = __ldcg(p.table + (size_t)b * p.max_blocks + (at[u][k] >> shift));
                    }
                }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
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
                if (n0 + 128 * u < end) put(n0 + 128 * u, end, slot[u], at[u]);
            }
        }
        // What lies behind the last token.
        const int none[4] = {-1, -1, -1, -1};
        const long long tail = wide ? min((total + 3) & ~3LL, p.rows) : total;
        if (gtid < tail - total) {
            if (p.slots) p.slots[total + gtid] = -1;
            if (p.positions) p.positions[total + gtid] = -1;
        }
        for (long long n = tail + 4LL * gtid; n < p.rows; n += 4LL * gthreads) put(n, p.rows, none, none);
    }
    if (flags && p.status) atomicOr(p.status, flags);
}

cudaError_t launch_pages(const PagesParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0}, known[kMaxDevices];
    const void* kernel = reinterpret_cast<const void*>(pages_kernel);
    const int smem = 4 * (p.B + 1) * (int)sizeof(int), most = 4 * (kPagesMaxBatch + 1) * (int)sizeof(int);
    int at_once[5];
    cudaError_t e = allow_clusters(kernel, most, &ready);
    if (e == cudaSuccess) e = clusters_at_once(kernel, kPagesThreads, most, &ready, known, at_once);
    if (e != cudaSuccess) return e;
    // A CTA for 8,192 rows, two steps of its threads, and for 16,384 table entries (few of which change in a call).
    const long long rows = p.slots || p.positions ? p.rows : 0, entries = (long long)p.B * p.max_blocks;
    int parts = 1;
    for (int i = 1; i < 5 && at_once[i] > 0 && (parts * 8192LL < rows || parts * 16384LL < entries); ++i) parts *= 2;
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
    cfg.numAttrs = parts > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, pages_kernel, p, parts);
}

}  // namespace kvd
