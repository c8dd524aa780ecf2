// The blocks of tokens that a query attends to: every block is scored by its bounds (block_bounds.cu) and the
// K of the highest scores are kept. For query row r with codes c = round(q / s_r), s_r = max |q| / 127, and block j
// of KV head g:
//   I = sum_d (c_d > 0 ? c_d * hi_d : c_d * lo_d)   in whole numbers, below 2^23
//   score = fl(max over the group's rows of fl(I * s_r) * scale_j); NaN counts as +inf
// The first n_first and the last n_last blocks that the query token sees are always kept; ties go to the lowest index;
// the list ascends. Since I is a whole number, exact in float32 in whatever order it is summed, the selection is a
// matter of definition and not of the order of additions.
//
// Reads 2 D + 4 bytes a (block, KV head) once for all query tokens; bound by memory for batches, by latency for one
// sequence. A cluster of up to 16 CTAs takes a (sequence, KV head). First its warps score tiles of 16 blocks: f16 MMAs
// m16n8k16 with the blocks as rows and the query rows as columns, I = [hi lo] [max(c, 0) min(c, 0)]^T, exact since
// f16 holds the codes, products and sums. A lane's 16-byte load is 16 consecutive codes of a row; the MMA's k order is the permutation of
// columns that fits, the same for both operands, so codes go from the load to fragments in registers. Keys
// (scores as ordered integers) go to the workspace, the cluster meets at a barrier, and CTA i selects for the query tokens i, i + CTAs, ...: a
// histogram over 2,048 equal parts of the range [smallest, largest] of the keys, then over the part that holds the border, until
// the border's value or a part that fits whole is found (two rounds as a rule, three at most).
#include <math_constants.h>

#include <algorithm>

#include "../../include/kvdecode.h"
#include "blocks.h"
#include "cluster.cuh"
#include "common.cuh"

namespace kvd {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelTiles = 8;        // column tiles of 8 query rows scored at once
constexpr int kSelRoom = 64 * 1024; // shared memory: the query rows' fragments, later the keys

__device__ __forceinline__ uint32_t score_key(float s) {  // larger score, larger key; NaN as +inf, -0 as +0
    if (s != s) return 0xff800000u;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// How many query rows of a token share a column tile's 8 columns, in powers of two; a wider group takes whole tiles.
__host__ __device__ inline int sel_columns(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8; }

template <int D>
__global__ void __launch_bounds__(kSelThreads, D == 256 ? 1 : 2) block_select_kernel(const SelectParams p) {
    constexpr int KS = 2 * D / 16, LOADS = 2 * D / 64;  // k-steps; 16-byte loads of a lane and row
    extern __shared__ __align__(16) uint8_t smem[];
    uint2* s_q = reinterpret_cast<uint2*>(smem);         // [tile][k-step][lane]: B fragments
    uint32_t* s_key = reinterpret_cast<uint32_t*>(smem); // later: the keys of one query token
    __shared__ float s_sc[kSelTiles * 8];                // the columns' scales, NaN: no query row
    __shared__ uint32_t s_hist[kSelBins];
    __shared__ uint32_t s_a[kSelWarps], s_b[kSelWarps];
    __shared__ uint32_t s_lo, s_hi, s_need, s_done;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j4 = lane & 3, g8 = lane >> 2;
    const int rank = blockIdx.x % p.parts, pair = blockIdx.x / p.parts, h = pair % p.Hkv, b = pair / p.Hkv;
    const int bs = p.block_shift, G = p.G;
    const int raw = __ldg(p.seq_lens + b), L = raw < 0 ? 0 : raw > p.len_cap ? p.len_cap : raw;
    if (raw != L && h == 0 && rank == 0 && tid == 0 && p.status) atomicOr(p.status, KVD_STATUS_SEQ_LEN_CLAMPED);
    const int full = L >> bs;  // blocks with bounds
    uint32_t* keys = p.keys + (size_t)pair * p.T * p.key_stride;  // [T][key_stride]

    // ---- scores, unless the last query token keeps every block ----
    if ((int)(((long long)L + (1 << bs) - 1) >> bs) > p.K) {
        const int cols = sel_columns(G);                 // columns of a token in a tile
        const int per_tok = (G + 7) / 8;                 // tiles of a token (G > 8: several)
        const int toks = G > 8 ? kSelTiles / per_tok : kSelTiles * (8 / cols);  // tokens of a round
        for (int t0 = 0; t0 < p.T; t0 += toks) {
            const int nt = min(toks, p.T - t0);
            const int tiles = G > 8 ? nt * per_tok : (nt * cols + 7) / 8;
            // Column x of a round: token x / (8 per_tok) row x % (8 per_tok) for wide groups, else token x / cols, row x % cols.
            auto column = [&](int x, int& t, int& r) {
                const int w = G > 8 ? 8 * per_tok : cols;
                t = x / w;
                r = x - t * w;
                return t < nt && r < G;
            };
            __syncthreads();
            for (int x = warp; x < tiles * 8; x += kSelWarps) {  // the columns' scales
                int t, r;
                float s = __uint_as_float(0x7fffffffu);
                if (column(x, t, r)) {
                    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                          (((size_t)b * p.T + t0 + t) * p.Hq + (size_t)h * G + r) * D);
                    uint32_t a = 0;  // magnitudes as integers: a NaN is the largest
                    for (int i = lane; i < D / 2; i += 32) {
                        const uint32_t w = __ldg(q + i);
                        a = max(a, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
                    }
                    a = __reduce_max_sync(0xffffffffu, a);
                    if (a < 0x7f80u) s = __fdiv_rn(__uint_as_float(a << 16), 127.f);  // a row that is not finite takes no part
                }
                if (lane == 0) s_sc[x] = s;
            }
            __syncthreads();
            for (int i = tid; i < tiles * KS * 32; i += kSelThreads) {  // and their codes as fragments
                const int ln = i & 31, ks = (i >> 5) % KS, x = (i >> 5) / KS * 8 + (ln >> 2);
                const int col = 64 * (ks >> 2) + 16 * (ln & 3) + 4 * (ks & 3);  // the first of four, of the 2 D columns
                int t, r;
                uint2 f = make_uint2(0u, 0u);
                const float s = s_sc[x];
                if (column(x, t, r) && s > 0.f) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                         (((size_t)b * p.T + t0 + t) * p.Hq + (size_t)h * G + r) * D + (col & (D - 1))));
                    const float v[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
                    float c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        c[e] = fminf(fmaxf(rintf(__fdiv_rn(v[e], s)), -127.f), 127.f);
                        c[e] = col < D ? fmaxf(c[e], 0.f) : fminf(c[e], 0.f);
                    }
                    f = make_uint2(pack_f16x2(c[0], c[1]), pack_f16x2(c[2], c[3]));
                }
                s_q[i] = f;
            }
            __syncthreads();
            for (int j0 = (rank * kSelWarps + warp) * 16; j0 < full; j0 += p.parts * kSelWarps * 16) {
                // Rows j0 + g8 and j0 + g8 + 8: their codes, 16 bytes a load, and scales.
                uint4 w[2][LOADS];
                float sc[2];
                bool ok[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = j0 + g8 + 8 * e;
                    long long blk = -1;
                    if (j < full) {
                        if (p.pg.block_table) {
                            const int tok = j << bs;
                            const int page = __ldg(p.pg.block_table + (size_t)b * p.pg.max_blocks + (tok >> p.pg.page_shift));
                            if ((unsigned)page < (unsigned)p.pg.num_pages)
                                blk = ((long long)page << (p.pg.page_shift - bs)) + ((tok & ((1 << p.pg.page_shift) - 1)) >> bs);
                            else if (j4 == 0 && p.status)
                                atomicOr(p.status, KVD_STATUS_BAD_PAGE);
                        } else {
                            blk = (long long)b * (p.S_max >> bs) + j;
                        }
                    }
                    ok[e] = blk >= 0;
                    const size_t at = (size_t)(ok[e] ? blk : 0) * p.Hkv + h;
                    const uint4* src = reinterpret_cast<const uint4*>(p.codes + at * 2 * D) + j4;
#pragma unroll
                    for (int c = 0; c < LOADS; ++c) w[e][c] = ok[e] ? __ldg(src + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
                    sc[e] = ok[e] ? __ldg(p.scales + at) : 0.f;
                }
                float best[2][2];  // [block][column of the lane's two]
                for (int n = 0; n < tiles; ++n) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
                    const uint2* fq = s_q + (size_t)n * KS * 32 + lane;
#pragma unroll
                    for (int c = 0; c < LOADS; ++c) {
                        const uint32_t x[4] = {w[0][c].x, w[0][c].y, w[0][c].z, w[0][c].w};
                        const uint32_t y[4] = {w[1][c].x, w[1][c].y, w[1][c].z, w[1][c].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t a[4];
                            i8x4_to_f16x2x2(x[i], a[0], a[2]);
                            i8x4_to_f16x2x2(y[i], a[1], a[3]);
                            const uint2 f = fq[(4 * c + i) * 32];
                            mma_f16_16816((i & 1) ? acc2 : acc, a, f.x, f.y);
                        }
                    }
                    const float s0 = s_sc[8 * n + 2 * j4], s1 = s_sc[8 * n + 2 * j4 + 1];
                    const bool first = G <= 8 || n % per_tok == 0;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {  // (fmaxf passes the NaN of a column without a row over)
                        const float v0 = __fmul_rn(acc[2 * e] + acc2[2 * e], s0), v1 = __fmul_rn(acc[2 * e + 1] + acc2[2 * e + 1], s1);
                        best[e][0] = fmaxf(first ? -CUDART_INF_F : best[e][0], v0);
                        best[e][1] = fmaxf(first ? -CUDART_INF_F : best[e][1], v1);
                    }
                    if (G > 8 && n % per_tok != per_tok - 1) continue;
                    // The maximum over a token's columns, and its key: `cols` columns a token, tokens side by side.
                    const int width = G > 8 ? 8 : cols;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v0 = best[e][0], v1 = best[e][1];
                        if (width > 1) v0 = fmaxf(v0, v1);
                        if (width > 2) v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, v0, 1));
                        if (width > 4) v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, v0, 2));
                        const int j = j0 + g8 + 8 * e;
                        if (j >= full) continue;
                        const int t = G > 8 ? n / per_tok : (8 * n + 2 * j4) / cols;  // of this round
                        const uint32_t k0 = ok[e] ? score_key(__fmul_rn(v0, sc[e])) : 0u;
                        if (width == 1) {
                            if (t < nt) keys[(size_t)(t0 + t) * p.key_stride + j] = k0;
                            if (t + 1 < nt) keys[(size_t)(t0 + t + 1) * p.key_stride + j] = ok[e] ? score_key(__fmul_rn(v1, sc[e])) : 0u;
                        } else if ((2 * j4) % width == 0 && t < nt) {
                            keys[(size_t)(t0 + t) * p.key_stride + j] = k0;
                        }
                    }
                }
            }
        }
    }
    if (p.parts > 1)
        cluster_sync();
    else
        __syncthreads();

    // ---- the selection ----
    for (int t = rank; t < p.T; t += p.parts) {
        const int seen = L - p.T + 1 + t;
        const int nb = seen > 0 ? (int)(((long long)seen + (1 << bs) - 1) >> bs) : 0;  // blocks the token sees
        int32_t* out = p.blocks + (((size_t)b * p.T + t) * p.Hkv + h) * p.K;
        if (nb <= p.K) {
            for (int i = tid; i < p.K; i += kSelThreads) out[i] = i < nb ? i : -1;
            continue;
        }
        // Blocks [lo_j, hi_j) compete for the places that the first and last ones leave; all of them have bounds.
        const int lo_j = p.n_first, hi_j = nb - p.n_last, n = hi_j - lo_j, want = p.K - p.n_first - p.n_last;
        const uint32_t* src = keys + (size_t)t * p.key_stride + lo_j;
        const bool fits = n <= kSelRoom / 4;
        const int chunk = ((n + kSelThreads - 1) / kSelThreads) | 1;  // a thread's keys in a row; odd: lanes in different banks
        __syncthreads();
        uint32_t mn = 0xffffffffu, mx = 0u;
        for (int i = tid; i < n; i += kSelThreads) {
            const uint32_t k = __ldcg(src + i);
            if (fits) s_key[i] = k;
            mn = min(mn, k);
            mx = max(mx, k);
        }
        mn = __reduce_min_sync(0xffffffffu, mn);
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) s_a[warp] = mn, s_b[warp] = mx;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kSelWarps; ++w) mn = min(mn, s_a[w]), mx = max(mx, s_b[w]);
            s_lo = mn;
            s_hi = mx;
            s_need = (uint32_t)want;
            s_done = 0;
        }
        auto key = [&](int i) { return fits ? s_key[i] : __ldcg(src + i); };
        // Keys above s_hi are kept, s_need of those in [s_lo, s_hi] too.
        uint32_t lo, hi, need;
        bool whole = false;  // the border's part is kept whole
        if (want > 0) {
            while (true) {
                for (int i = tid; i < kSelBins; i += kSelThreads) s_hist[i] = 0;
                __syncthreads();
                lo = s_lo, hi = s_hi, need = s_need;
                const int shift = max(0, 21 - __clz(hi - lo));  // (hi - lo) >> shift is below 2,048
                for (int i = tid; i < n; i += kSelThreads) {
                    const uint32_t k = key(i);
                    if (k >= lo && k <= hi) atomicAdd(&s_hist[(k - lo) >> shift], 1u);
                }
                __syncthreads();
                // Thread i adds up 8 parts, from the top; the one in which the running sum reaches `need` has the border.
                constexpr int PER = kSelBins / kSelThreads;
                uint32_t cnt[PER], sum = 0;
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    cnt[e] = s_hist[kSelBins - 1 - (tid * PER + e)];
                    sum += cnt[e];
                }
                uint32_t incl = sum;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += x;
                }
                if (lane == 31) s_a[warp] = incl;
                __syncthreads();
                uint32_t before = incl - sum;
                for (int w = 0; w < warp; ++w) before += s_a[w];
                if (before < need && before + sum >= need) {
                    uint32_t at = before;
#pragma unroll
                    for (int e = 0; e < PER; ++e) {
                        if (at < need && at + cnt[e] >= need) {
                            const uint32_t part = kSelBins - 1 - (tid * PER + e), low = lo + (part << shift);
                            s_lo = low;
                            s_hi = shift == 0 ? low : min(hi, low + ((1u << shift) - 1));
                            s_need = need - at;
                            s_done = (shift == 0 || cnt[e] == need - at) ? 1 : 0;
                        }
                        at += cnt[e];
                    }
                }
                __syncthreads();
                if (s_done) break;
            }
            lo = s_lo, hi = s_hi, need = s_need;
            whole = lo != hi;  // (one value: the first `need` of them in order)
        } else {
            lo = hi = 0xffffffffu, need = 0;
        }
        // ---- kept blocks in order: a thread's run of keys, counted, then written behind the runs before ----
        const int i0 = min(tid * chunk, n), i1 = min(i0 + chunk, n);
        uint32_t above = 0, equal = 0;
        for (int i = i0; i < i1; ++i) {
            const uint32_t k = key(i);
            above += k > hi || (whole && k >= lo);
            equal += !whole && k == lo;
        }
        uint32_t ia = above, ie = equal;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, ia, off), y = __shfl_up_sync(0xffffffffu, ie, off);
            if (lane >= off) ia += x, ie += y;
        }
        __syncthreads();
        if (lane == 31) s_a[warp] = ia, s_b[warp] = ie;
        __syncthreads();
        uint32_t pa = ia - above, pe = ie - equal;
        for (int w = 0; w < warp; ++w) pa += s_a[w], pe += s_b[w];
        uint32_t at = pa + min(pe, need);
        for (int i = i0; i < i1; ++i) {
            const uint32_t k = key(i);
            bool keep = k > hi || (whole && k >= lo);
            if (!whole && k == lo) keep = pe++ < need;
            if (keep) out[p.n_first + at++] = lo_j + i;
        }
        for (int i = tid; i < p.n_first; i += kSelThreads) out[i] = i;
        for (int i = tid; i < p.n_last; i += kSelThreads) out[p.K - p.n_last + i] = hi_j + i;
    }
}

cudaError_t launch_block_select(const SelectParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> ready[3];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hkv * p.parts), 1, 1);
    cfg.blockDim = dim3(kSelThreads, 1, 1);
    cfg.dynamicSmemBytes = kSelRoom;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
#define KVD_SELECT(DD, i)                                                                                                \
    ([&]() {                                                                                                             \
        const cudaError_t e = allow_clusters(reinterpret_cast<const void*>(block_select_kernel<DD>), kSelRoom, &ready[i]); \
        return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, block_select_kernel<DD>, p) : e;                              \
    }())
    switch (p.D) {
        case 64: return KVD_SELECT(64, 0);
        case 128: return KVD_SELECT(128, 1);
        case 256: return KVD_SELECT(256, 2);
        default: return cudaErrorInvalidValue;
    }
#undef KVD_SELECT
}

}  // namespace kvd
