// The blocks of tokens that a query attends to: every block is scored by its bounds (block_bounds.cu) and the
// K of the highest scores are kept. For query row r with codes c = round(q / s_r), s_r = max |q| / 127, and block j
// of KV head g:
//   I = sum_d (c_d > 0 ? c_d * hi_d : c_d * lo_d)   in whole numbers, below 2^23
//   score = fl(max over the group's rows of fl(I * s_r) * scale_j); NaN counts as +inf
// The first n_first and the last n_last blocks that the query token sees are always kept; ties go to the lowest
// index; the list ascends. Since I is a whole number, exact in float32 in whatever order it is summed, the
// selection is a matter of definition and not of the order of additions.
//
// Reads 2 D + 4 bytes a (block, KV head) once for all query tokens. 32 sequences of 16,384 to 131,072 tokens in
// blocks of 32, 32 heads on 8 of 128: 41.5 us, 33 scoring (153 MB at 4.6 TB/s: some 500 instructions a tile of 16
// blocks, a third of them the rows' fragments) and 8 selecting; one of 131,072 in blocks of 64: 7.7, latency
// throughout; 65,536 keys a CTA, which it reads from L2, 44 to select. (Both in one launch of clusters: 53 and
// 9.9, since the cluster waits for its slowest part and the selection holds the scorers' places.) The first
// launch scores, some CTAs a (sequence, KV head), a warp tiles of 16 blocks: f16 MMAs m16n8k16 with the blocks
// as rows and the query rows as columns, I = [hi lo] [max(c, 0) min(c, 0)]^T. A code enters as code + 128 in
// the low bits of an f16, a subnormal; products and sums of these are whole numbers below 2^24 (times 2^-24),
// so exact. A lane's 16-byte copy is 16 consecutive codes of a row; the MMA's k order is the permutation of
// columns that fits, the same for both operands, so codes go from the lane's own place in shared memory to
// fragments without a shuffle, and a warp waits for its own copies alone. Keys (scores as ordered integers) go
// to the workspace. A second launch selects, a CTA a (sequence, query token, KV head): a histogram over 2,048
// equal parts of the range [smallest, largest] of the keys, then (seldom) over the part that holds the border,
// until that part has few keys, which are ranked one by one; the kept ones become bits, the bits the list.
#include <math_constants.h>

#include <algorithm>

#include "../../include/kvdecode.h"
#include "blocks.h"
#include "common.cuh"

namespace kvd {

constexpr uint32_t kSelNoPage = 1u; // key of a block that has no page: below every score's; 0 is below all
constexpr int kSelBins = 2048;
constexpr int kPickThreads = 512;
constexpr int kSelTiles = 8;        // column tiles of 8 query rows scored at once
constexpr int kSelTies = 64;        // keys around the border that are ranked one by one

// Shared memory of the scoring: the query rows' fragments, then a ring of tiles a warp, in which every lane has
// its own 16 bytes of each load and its two rows' scales. The selection puts the keys in its place.
template <int D>
struct SelectShape {
    static constexpr int KS = 2 * D / 16, LOADS = 2 * D / 64;  // k-steps; 16-byte loads of a lane and row
    static constexpr int WARPS = D == 256 ? 16 : 8, THREADS = 32 * WARPS;
    static constexpr int STAGES = D == 256 ? 1 : D == 128 ? 2 : 3;  // three CTAs an SM with one column tile, two
                                                                    // with more; at head_dim 256 one of twice the warps
    static constexpr int TILE = 2 * LOADS * 512 + 2 * 128;     // 16 blocks' codes, and scales
    static constexpr int RING = WARPS * STAGES * TILE;
    static constexpr int FRAG = KS * 32 * 8;                   // a column tile's fragments
    static constexpr int MOST = kSelTiles * FRAG + RING;
    static_assert(MOST + 2 * 1024 <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ uint32_t score_key(float s) {  // larger score, larger key; NaN as +inf, -0 as +0
    if (s != s) return 0xff800000u;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// How many query rows of a token share a column tile's 8 columns, in powers of two; a wider group takes whole tiles.
__host__ __device__ inline int sel_columns(int G) { return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8; }

// Column tiles that the query rows of T tokens take at once: 1, 2, 4, 6 or 8 (the last may be without rows).
static int select_tiles(int G, int T) {
    const int per_tok = (G + 7) / 8;
    const int n = std::min(kSelTiles, G > 8 ? std::min(T, kSelTiles / per_tok) * per_tok : (T * sel_columns(G) + 7) / 8);
    return n == 1 ? 1 : (n + 1) / 2 * 2;
}

// NT: column tiles of a round.
template <int D, int NT>
__global__ void __launch_bounds__(SelectShape<D>::THREADS, D == 256 ? 1 : NT == 1 ? 3 : 2) block_score_kernel(const SelectParams p) {
    using Sh = SelectShape<D>;
    constexpr int WARPS = Sh::WARPS;
    constexpr int KS = Sh::KS, LOADS = Sh::LOADS, STAGES = Sh::STAGES;
    extern __shared__ __align__(16) uint8_t smem[];
    uint2* s_q = reinterpret_cast<uint2*>(smem);         // [tile][k-step][lane]: B fragments
    __shared__ float s_sc[kSelTiles * 8];                // the columns' scales, NaN: no query row
    __shared__ float s_bias[kSelTiles * 8];              // what their sums start from
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j4 = lane & 3, g8 = lane >> 2;
    const int rank = blockIdx.x % p.parts, pair = blockIdx.x / p.parts, h = pair % p.Hkv, b = pair / p.Hkv;
    const int bs = p.block_shift, G = p.G;
    pdl_wait();
    pdl_launch_dependents();
    const int raw = __ldg(p.seq_lens + b), L = raw < 0 ? 0 : raw > p.len_cap ? p.len_cap : raw;
    const int full = L >> bs;  // blocks with bounds
    uint32_t* keys = p.keys + (size_t)pair * p.T * p.key_stride;  // [T][key_stride]

    // (Nothing to score where the last query token keeps every block.)
    const int first = (rank * WARPS + warp) * 16, step = p.parts * WARPS * 16;
    if ((int)(((long long)L + (1 << bs) - 1) >> bs) <= p.K || rank * WARPS * 16 >= full) return;
    {
        const int cols = sel_columns(G);                 // columns of a token in a tile
        const int per_tok = (G + 7) / 8;                 // tiles of a token (G > 8: several)
        const int toks = G > 8 ? NT / per_tok : NT * (8 / cols);  // tokens of a round
        uint8_t* ring = smem + NT * Sh::FRAG + warp * STAGES * Sh::TILE;
        // A tile's rows of this lane: blocks j0 + g8 and j0 + g8 + 8, by their place among all bounds (-1:
        // none). Lanes go different ways here; the warp comes together again at the end.
        auto look_up = [&](int j0, long long (&at)[2]) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = j0 + g8 + 8 * e;
                at[e] = -1;
                if (j < full) {
                    long long blk;
                    if (p.pg.block_table) {
                        const int tok = j << bs;
                        const int page = __ldg(p.pg.block_table + (size_t)b * p.pg.max_blocks + (tok >> p.pg.page_shift));
                        blk = -1;
                        if ((unsigned)page < (unsigned)p.pg.num_pages)
                            blk = ((long long)page << (p.pg.page_shift - bs)) + ((tok & ((1 << p.pg.page_shift) - 1)) >> bs);
                        else if (j4 == 0 && p.status)
                            atomicOr(p.status, KVD_STATUS_BAD_PAGE);
                    } else {
                        blk = (long long)b * (p.S_max >> bs) + j;
                    }
                    if (blk >= 0) at[e] = blk * p.Hkv + h;
                }
            }
            __syncwarp();
        };
        // Their codes and scales on the way to the lane's own places of a stage; `have` keeps which rows are there.
        uint32_t have = 0;
        const uint64_t policy = l2_evict_first_policy();
        auto fetch = [&](int stage, const long long (&at)[2]) {
            const uint32_t dst = smem_u32(ring) + stage * Sh::TILE + lane * 16;
            have &= ~(3u << (2 * stage));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool ok = at[e] >= 0;
                const size_t a = ok ? (size_t)at[e] : 0;
                have |= (ok ? 1u : 0u) << (2 * stage + e);
                const int8_t* src = p.codes + a * 2 * D + 16 * j4;
#pragma unroll
                for (int c = 0; c < LOADS; ++c) cp_async_16(dst + (e * LOADS + c) * 512, src + 64 * c, ok ? 16 : 0, policy);
                cp_async_4(dst - lane * 12 + 2 * LOADS * 512 + e * 128, p.scales + a, ok ? 4 : 0);
            }
        };
        for (int t0 = 0; t0 < p.T; t0 += toks) {
            const int nt = min(toks, p.T - t0);
            // Column x of a round: token x / (8 per_tok) row x % (8 per_tok) for wide groups, else token x /
            // cols, row x % cols.
            auto column = [&](int x, int& t, int& r) {
                const int w = G > 8 ? 8 * per_tok : cols;
                t = x / w;
                r = x - t * w;
                return t < nt && r < G;
            };
            // The first tiles' loads run while the query rows become fragments.
            constexpr int WORDS = D / 64;  // a lane's words of a query row
            uint32_t qw[WORDS];
            auto load_row = [&](int x) {
                int t, r;
                const bool live = column(x, t, r);
                const size_t row = ((size_t)b * p.T + t0 + (live ? t : 0)) * p.Hq + (size_t)h * G + (live ? r : 0);
                const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) + row * D);
#pragma unroll
                for (int i = 0; i < WORDS; ++i) qw[i] = live ? __ldg(q + lane + 32 * i) : 0x7fc07fc0u;  // no row: NaN
            };
            if (warp < NT * 8) load_row(warp);
            long long at[2];
            look_up(first, at);
#pragma unroll
            for (int k = 0; k < STAGES - 1; ++k) {
                fetch(k, at);
                cp_async_commit();
                look_up(first + (k + 1) * step, at);
            }
            if (t0 > 0) __syncthreads();
#pragma unroll 1
            for (int x = warp; x < NT * 8; x += WARPS) {
                if (x > warp) load_row(x);
                uint32_t a = 0;  // magnitudes as integers: a NaN is the largest
#pragma unroll
                for (int i = 0; i < WORDS; ++i) a = max(a, max(qw[i] & 0x7fffu, (qw[i] >> 16) & 0x7fffu));
                a = __reduce_max_sync(0xffffffffu, a);
                // A row that is not finite takes no part, as a column without a row: codes 0, scale NaN.
                const float s = a < 0x7f80u ? __fdiv_rn(__uint_as_float(a << 16), 127.f) : __uint_as_float(0x7fffffffu);
                int sum = 0;  // of the row's codes
                // round(q / s): by the reciprocal, but where that may lie on the other side of a half by the
                // quotient itself.
                const float inv = s > 1e-30f ? __frcp_rn(s) : 0.f;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    const int col = 2 * (lane + 32 * i);  // of two neighbours: their fragment's lane, k-step and half
                    float c[2] = {0.f, 0.f};
                    if (s > 0.f) {
                        bool near = inv == 0.f;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = (e ? bf16_hi(qw[i]) : bf16_lo(qw[i])) * inv;  // off by 2^-22 of itself at most, below 2^7
                            c[e] = rintf(x);
                            near |= fabsf(fabsf(x - c[e]) - 0.5f) < 1e-4f;
                        }
                        if (near) {  // (by lane; the warp meets again before the sum)
#pragma unroll
                            for (int e = 0; e < 2; ++e) c[e] = rintf(__fdiv_rn(e ? bf16_hi(qw[i]) : bf16_lo(qw[i]), s));
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) c[e] = fminf(fmaxf(c[e], -127.f), 127.f);
                    }
                    const int ks = 4 * (col >> 6) + ((col >> 2) & 3), ln = 4 * (x & 7) + ((col >> 4) & 3);
                    uint32_t* f = reinterpret_cast<uint32_t*>(s_q + ((size_t)(x >> 3) * KS + ks) * 32 + ln) + ((col >> 1) & 1);
                    f[0] = pack_f16x2(fmaxf(c[0], 0.f), fmaxf(c[1], 0.f));
                    f[KS / 2 * 64] = pack_f16x2(fminf(c[0], 0.f), fminf(c[1], 0.f));
                    sum += (int)c[0] + (int)c[1];
                }
                __syncwarp();
                sum = __reduce_add_sync(0xffffffffu, sum);
                if (lane == 0) s_sc[x] = s, s_bias[x] = (float)sum * -0x1p-17f;  // -128 of them, in units of 2^-24
            }
            __syncwarp();
            __syncthreads();
            int stage = 0;
            for (int j0 = first; j0 < full; j0 += step) {
                const int next = stage == 0 ? STAGES - 1 : stage - 1;  // the stage read last
                asm volatile("" ::: "memory");  // (a lane waits for its own copies alone: no barrier orders its loads)
                if (j0 + (STAGES - 1) * step < full) fetch(next, at);
                cp_async_commit();
                look_up(j0 + STAGES * step, at);
                cp_async_wait<STAGES - 1>();
                // The MMAs are .aligned: a warp's threads have to execute each of them together. What came
                // before (look-ups, the last tile's stores) let lanes go different ways, and only this makes
                // sure that they have met again.
                __syncwarp();
                const uint8_t* mine = ring + stage * Sh::TILE + lane * 16;
                // Codes enter the MMAs as code + 128 in the low bits of an f16, a subnormal of that many 2^-24;
                // the sums start from what that adds. Products and sums are whole numbers below 2^24 in these
                // units: exact.
                float acc[NT][4], acc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] = acc[n][2] = s_bias[8 * n + 2 * j4];
                    acc[n][1] = acc[n][3] = s_bias[8 * n + 2 * j4 + 1];
                }
#pragma unroll
                for (int c = 0; c < LOADS; ++c) {
                    const uint4 wx = *reinterpret_cast<const uint4*>(mine + c * 512);
                    const uint4 wy = *reinterpret_cast<const uint4*>(mine + (LOADS + c) * 512);
                    const uint32_t x[4] = {wx.x, wx.y, wx.z, wx.w}, y[4] = {wy.x, wy.y, wy.z, wy.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t ux = x[i] ^ 0x80808080u, uy = y[i] ^ 0x80808080u;
                        const uint32_t a[4] = {__byte_perm(ux, 0, 0x4140), __byte_perm(uy, 0, 0x4140), __byte_perm(ux, 0, 0x4342),
                                               __byte_perm(uy, 0, 0x4342)};
                        const uint2* fq = s_q + (4 * c + i) * 32 + lane;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 f = fq[n * KS * 32];
                            mma_f16_16816((NT == 1 && (i & 1)) ? acc2 : acc[n], a, f.x, f.y);
                        }
                    }
                }
                const bool ok[2] = {(bool)((have >> (2 * stage)) & 1u), (bool)((have >> (2 * stage + 1)) & 1u)};
                float sc[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[e] = *reinterpret_cast<const float*>(mine - lane * 12 + 2 * LOADS * 512 + e * 128);
                stage = stage + 1 == STAGES ? 0 : stage + 1;
                if constexpr (NT == 1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[0][e] += acc2[e];
                }
                float best[2][2];  // [block][column of the lane's two]
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float s0 = s_sc[8 * n + 2 * j4], s1 = s_sc[8 * n + 2 * j4 + 1];
                    const bool fresh = G <= 8 || n % per_tok == 0;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {  // (fmaxf passes the NaN of a column without a row over)
                        const float v0 = __fmul_rn(acc[n][2 * e] * 0x1p24f, s0), v1 = __fmul_rn(acc[n][2 * e + 1] * 0x1p24f, s1);
                        best[e][0] = fmaxf(fresh ? -CUDART_INF_F : best[e][0], v0);
                        best[e][1] = fmaxf(fresh ? -CUDART_INF_F : best[e][1], v1);
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
                        const bool here = j < full;
                        const int t = G > 8 ? n / per_tok : (8 * n + 2 * j4) / cols;  // among those scored at once
                        const uint32_t k0 = ok[e] ? score_key(__fmul_rn(v0, sc[e])) : kSelNoPage;
                        if (width == 1) {
                            if (here && t < nt) keys[(size_t)(t0 + t) * p.key_stride + j] = k0;
                            if (here && t + 1 < nt)
                                keys[(size_t)(t0 + t + 1) * p.key_stride + j] = ok[e] ? score_key(__fmul_rn(v1, sc[e])) : kSelNoPage;
                        } else if (here && (2 * j4) % width == 0 && t < nt) {
                            keys[(size_t)(t0 + t) * p.key_stride + j] = k0;
                        }
                        __syncwarp();
                    }
                }
            }
            cp_async_wait<0>();
        }
    }
}

// The selection: a CTA for a (sequence, query token, KV head).
__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(const SelectParams p, int room) {
    constexpr int WARPS = kPickThreads / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t* s_hist = reinterpret_cast<uint32_t*>(smem);
    uint2* s_tie = reinterpret_cast<uint2*>(s_hist + kSelBins);
    uint32_t* s_key = reinterpret_cast<uint32_t*>(s_tie + kSelTies);
    __shared__ uint32_t s_a[WARPS], s_b[WARPS];
    __shared__ uint32_t s_lo, s_hi, s_need, s_count, s_ties;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % p.Hkv, bt = blockIdx.x / p.Hkv, t = bt % p.T, b = bt / p.T, bs = p.block_shift;
    for (int i = tid; i < kSelBins / 4; i += kPickThreads) reinterpret_cast<uint4*>(s_hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) s_ties = 0;
    pdl_wait();
    pdl_launch_dependents();
    const int raw = __ldg(p.seq_lens + b), L = raw < 0 ? 0 : raw > p.len_cap ? p.len_cap : raw;
    if (raw != L && h == 0 && t == 0 && tid == 0 && p.status) atomicOr(p.status, KVD_STATUS_SEQ_LEN_CLAMPED);
    const int seen = L - p.T + 1 + t;
    const int nb = seen > 0 ? (int)(((long long)seen + (1 << bs) - 1) >> bs) : 0;  // blocks the token sees
    int32_t* out = p.blocks + (size_t)blockIdx.x * p.K;
    if (nb <= p.K) {
        for (int i = tid; i < p.K; i += kPickThreads) out[i] = i < nb ? i : -1;
        return;
    }
    // Blocks [lo_j, hi_j) compete for the places that the first and last ones leave; all of them have bounds.
    const int lo_j = p.n_first, hi_j = nb - p.n_last, want = p.K - p.n_first - p.n_last;
    const uint32_t* src = p.keys + (((size_t)b * p.Hkv + h) * p.T + t) * p.key_stride;
    for (int i = tid; i < p.n_first; i += kPickThreads) out[i] = i;
    for (int i = tid; i < p.n_last; i += kPickThreads) out[p.K - p.n_last + i] = hi_j + i;
    if (want == 0) return;
    // Keys in shared memory where they fit (0 for those of the first and last vector that do not compete), else
    // where they lie (the workspace, in L2).
    const int vecs = (hi_j + 3) / 4;
    const bool fits = (long long)vecs * 16 + kSelBins * 4 + kSelTies * 8 <= room;
    const uint32_t* key = fits ? s_key : src;
    uint32_t mn = 0xffffffffu, mx = 0u;
    for (int v0 = tid; v0 < vecs; v0 += 4 * kPickThreads) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int v = v0 + u * kPickThreads;
            x[u] = v < vecs ? __ldcg(reinterpret_cast<const uint4*>(src) + v) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int v = v0 + u * kPickThreads;
            uint32_t k[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = 4 * v + e >= lo_j && 4 * v + e < hi_j;
                if (!in) k[e] = 0u;
                mn = min(mn, in ? k[e] : 0xffffffffu);
                mx = max(mx, k[e]);
            }
            if (fits && v < vecs) reinterpret_cast<uint4*>(s_key)[v] = make_uint4(k[0], k[1], k[2], k[3]);
        }
    }
    mn = __reduce_min_sync(0xffffffffu, mn);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) s_a[warp] = mn, s_b[warp] = mx;
    __syncthreads();
    uint32_t lo = __reduce_min_sync(0xffffffffu, s_a[lane % WARPS]), hi = __reduce_max_sync(0xffffffffu, s_b[lane % WARPS]);
    uint32_t need = (uint32_t)want, count = 0;
    // The numbers of the warps before this one, and of all, of what each left in s_a.
    auto before_me = [&](uint32_t& all) {
        const uint32_t x = lane < WARPS ? s_a[lane] : 0u;
        all = __reduce_add_sync(0xffffffffu, x);
        return __reduce_add_sync(0xffffffffu, lane < warp ? x : 0u);
    };
    auto warp_scan = [&](uint32_t x) {  // inclusive
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        return x;
    };
    // Keys above hi are kept, `need` of those in [lo, hi] too: rounds of a histogram over 2,048 equal parts of
    // that range, until few keys are left in the part that has the border, or all of them are kept, or it is
    // one value. (A round takes 11 bits off the range: three at most.)
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
        const int shift = max(0, 21 - __clz(hi - lo));  // (hi - lo) >> shift is below 2,048
        for (int i0 = lo_j + tid; i0 < hi_j; i0 += 8 * kPickThreads) {  // (loads first: none is moved ahead of an atomic)
            uint32_t k[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) k[u] = i0 + u * kPickThreads < hi_j ? key[i0 + u * kPickThreads] : 0u;  // 0: below every lo
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k[u] >= lo && k[u] <= hi) atomicAdd(&s_hist[(k[u] - lo) >> shift], 1u);
        }
        __syncthreads();
        // Thread i adds up 4 parts, from the top, and leaves zeros; the one in which the running sum reaches
        // `need` has the border.
        static_assert(kSelBins == 4 * kPickThreads, "a vector of parts a thread");
        uint4* hp = reinterpret_cast<uint4*>(s_hist) + kPickThreads - 1 - tid;
        const uint4 x = *hp;
        *hp = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t sum = x.x + x.y + x.z + x.w, incl = warp_scan(sum);
        if (lane == 31) s_a[warp] = incl;
        __syncthreads();
        uint32_t all;
        const uint32_t before = before_me(all) + incl - sum;
        if (before < need && before + sum >= need) {
            const uint32_t c1 = before + x.w, c2 = c1 + x.z, c3 = c2 + x.y;  // running sums, from the top
            const int e = need <= c1 ? 3 : need <= c2 ? 2 : need <= c3 ? 1 : 0;
            const uint32_t low = lo + ((uint32_t)(4 * (kPickThreads - 1 - tid) + e) << shift);
            s_lo = low;
            s_hi = shift == 0 ? low : min(hi, low + ((1u << shift) - 1));
            s_need = need - (e == 3 ? before : e == 2 ? c1 : e == 1 ? c2 : c3);
            s_count = e == 3 ? x.w : e == 2 ? x.z : e == 1 ? x.y : x.x;
        }
        __syncthreads();
        lo = s_lo, hi = s_hi, need = s_need, count = s_count;
        if (lo == hi || count == need || count <= kSelTies) break;
    }
    // ---- which are kept, a bit a key; those at the border by their rank among each other; then the list from the bits ----
    const bool value = lo == hi;                                  // one value: the first `need` of them in order
    const bool ranked = !value && count != need && count <= kSelTies;
    constexpr int CHUNK = 32 * kPickThreads;                      // a word of bits a thread, in the histogram's place
    uint32_t* s_keep = s_hist;
    uint32_t* s_same = s_hist + kPickThreads;
    auto tie = [&](uint32_t k, int i) { s_tie[atomicAdd(&s_ties, 1u) & (kSelTies - 1)] = make_uint2(k, (uint32_t)i); };
    const bool one_chunk = hi_j - lo_j <= CHUNK;
    if (ranked && !one_chunk) {
        for (int i0 = lo_j + tid; i0 < hi_j; i0 += 8 * kPickThreads) {
            uint32_t k[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) k[u] = i0 + u * kPickThreads < hi_j ? key[i0 + u * kPickThreads] : 0u;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k[u] >= lo && k[u] <= hi) tie(k[u], i0 + u * kPickThreads);
        }
    }
    uint32_t base = 0;  // kept before this chunk
#pragma unroll 1
    for (int c0 = lo_j; c0 < hi_j; c0 += CHUNK) {
        const int words = (min(CHUNK, hi_j - c0) + 31) / 32;
        for (int w0 = warp; w0 < words; w0 += 4 * WARPS) {
            uint32_t k[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = c0 + 32 * (w0 + u * WARPS) + lane;
                k[u] = i < hi_j ? key[i] : 0u;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int w = w0 + u * WARPS;
                const bool border = k[u] >= lo && k[u] <= hi;
                const uint32_t keep = __ballot_sync(0xffffffffu, k[u] > hi || (border && !value && !ranked));
                const uint32_t same = __ballot_sync(0xffffffffu, border);
                if (w < words && lane == 0) s_keep[w] = keep;
                if (w < words && lane == 1) s_same[w] = same;
                if (ranked && one_chunk && border && w < words) tie(k[u], c0 + 32 * w + lane);
            }
        }
        __syncthreads();
        if (ranked) {
            if (tid < (int)count) {
                const uint2 x = s_tie[tid];
                uint32_t ahead = 0;
                for (uint32_t e = 0; e < count; ++e) ahead += s_tie[e].x > x.x || (s_tie[e].x == x.x && s_tie[e].y < x.y);
                const int at = (int)x.y - c0;
                if (ahead < need && at >= 0 && at < CHUNK) atomicOr(&s_keep[at >> 5], 1u << (at & 31));
            }
            __syncthreads();
        }
        uint32_t word = tid < words ? s_keep[tid] : 0u;
        const uint32_t same = value && tid < words ? s_same[tid] : 0u;
        const uint32_t cnt = __popc(word) | (__popc(same) << 16);  // (2^14 each at most)
        const uint32_t incl = warp_scan(cnt);
        if (lane == 31) s_a[warp] = incl;
        __syncthreads();
        uint32_t all;
        const uint32_t pre = before_me(all) + incl - cnt;
        // Of the border's value the first ones in order, as far as `need` goes.
        uint32_t seen_same = pre >> 16, to = base + (pre & 0xffffu) + min(seen_same, need);
        for (uint32_t m = same; m && seen_same < need; m &= m - 1, ++seen_same) word |= m & (0u - m);
        for (uint32_t m = word; m; m &= m - 1) {
            if (to < (uint32_t)want) out[p.n_first + to] = c0 + 32 * tid + __ffs(m) - 1;
            ++to;
        }
        const uint32_t taken = value ? min(all >> 16, need) : 0u;
        base += (all & 0xffffu) + taken;
        if (value) need -= taken;
        __syncthreads();
    }
}

cudaError_t launch_block_select(const SelectParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> ready[15], pick_ready;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hkv * p.parts), 1, 1);
    auto launch = [&](auto shape, auto kernel, int tiles, std::atomic<uint64_t>* done) {
        using Sh = decltype(shape);
        const int smem = tiles * Sh::FRAG + Sh::RING;
        const cudaError_t e = allow_clusters(reinterpret_cast<const void*>(kernel), smem, done);
        if (e != cudaSuccess) return e;
        cfg.blockDim = dim3(Sh::THREADS, 1, 1);
        cfg.dynamicSmemBytes = (size_t)smem;
        return cudaLaunchKernelEx(&cfg, kernel, p);
    };
#define KVD_SCORE(DD, i)                                                                                 \
    (tiles == 1   ? launch(SelectShape<DD>(), block_score_kernel<DD, 1>, 1, &ready[5 * i])               \
     : tiles == 2 ? launch(SelectShape<DD>(), block_score_kernel<DD, 2>, 2, &ready[5 * i + 1])           \
     : tiles == 4 ? launch(SelectShape<DD>(), block_score_kernel<DD, 4>, 4, &ready[5 * i + 2])           \
     : tiles == 6 ? launch(SelectShape<DD>(), block_score_kernel<DD, 6>, 6, &ready[5 * i + 3])           \
                  : launch(SelectShape<DD>(), block_score_kernel<DD, 8>, 8, &ready[5 * i + 4]))
    const int tiles = select_tiles(p.G, p.T);
    cudaError_t e = cudaSuccess;
    if (p.key_stride > 0) {  // (else no sequence has a full block)
        switch (p.D) {
            case 64: e = KVD_SCORE(64, 0); break;
            case 128: e = KVD_SCORE(128, 1); break;
            case 256: e = KVD_SCORE(256, 2); break;
            default: e = cudaErrorInvalidValue;
        }
    }
#undef KVD_SCORE
    if (e != cudaSuccess) return e;
    const long long most = 216 * 1024, room = kSelBins * 4 + kSelTies * 8 + (long long)p.key_stride * 4;
    const int smem = (int)(room <= most ? room : kSelBins * 4 + kSelTies * 8);
    if ((e = allow_clusters(reinterpret_cast<const void*>(block_pick_kernel), (int)most, &pick_ready)) != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.T * p.Hkv), 1, 1);
    cfg.blockDim = dim3(kPickThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    return cudaLaunchKernelEx(&cfg, block_pick_kernel, p, smem);
}

int select_ctas(int D, int G, int T) {
    const int tiles = select_tiles(G, T);
    const int smem = D == 64 ? tiles * SelectShape<64>::FRAG + SelectShape<64>::RING
                   : D == 128 ? tiles * SelectShape<128>::FRAG + SelectShape<128>::RING
                              : tiles * SelectShape<256>::FRAG + SelectShape<256>::RING;
    return std::max(1, std::min(D == 256 ? 1 : tiles == 1 ? 3 : 2, 227 * 1024 / (smem + 2048)));
}

}  // namespace kvd
