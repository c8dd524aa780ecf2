// Split-KV attention over an fp4 cache: the chunk kernel of split_kv_chunk.cuh
// for blocks of 16 tokens held in 4 bits (fp4.cuh).
//
//   s_t = scale * q . k_t,  out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m)   (base 2, log2(e) in the scale)
// with k_t = 2^ek_t * (code * block scale), v_t likewise. A code times its
// scale has at most 6 significant bits and enters the MMAs as f16 exactly; the
// row exponents stay out of them: ek_t multiplies the score, and ev_t is added
// to the exponent of the weight, w_t = 2^(s_t + ev_t - mo) with a running
// reference mo of its own, 12 to 15 below the largest s_t + ev_t, so that the f16 weights lie in the upper part of
// f16's range. A weight is off by 2^-12 of itself, or, 2^-26 of the largest and less, by up to 2^-37 of the largest. For
// fp32 output a second f16 holds 2^11 times the rest and meets A times 2^-11 (still exact: a code times its
// scale is a multiple of 2^-10): 2^-22 of the weight, or 2^-48 of the largest.
//
// The products are turned round so that tokens fill the 16 rows of m16n8k16 MMAs
// and the query rows its 8 columns: S^T = K q^T (A = K rows, B = q) and
// O^T = V^T w (A = V^T, B = w), which wastes no rows for groups of up to 8
// query heads. The codes go from shared memory to the A fragments in registers:
// * K: thread (r, c) = (lane / 4, lane % 4) takes 16 bytes (32 columns, two
//   scales) of its token's row and of the row 8 further on; the MMA's k order is
//   a permutation of the columns, the same for q.
// * V: thread (r, c) takes the 16 columns of scale block r for 4 tokens; the
//   nibbles of a token pair are interleaved first (4 logic operations for 16
//   codes), so that one conversion gives the pair a fragment register holds.
// * w: the score fragment, rounded to f16, transposed by movmatrix.
// Row i of a block is token i ^ ((i >> 1) & 1), which halves the shared-memory
// conflicts of the V loads.
//
// A group of WD warps shares a run of tokens: each warp forms the scores of its own
// blocks for all query rows (a K code is converted once), the weights go through
// shared memory to the group, and each warp accumulates D / WD columns of the
// output over all of the group's tokens (a V code is converted once). With few rows
// WD is 1 and the warps work alone; with many, accumulators of D / WD columns keep all
// rows in one CTA, so that nothing is converted once per 16 rows.
//
// A CTA walks its segments (a pair's tokens in the CTA's run) in tiles of its 8 warps' blocks. A ninth
// warp walks ahead and fills two rings of tiles, K's and V's, by bulk copies (a head's blocks
// are contiguous: a tile of a contiguous cache is one copy, a paged one a copy per page, each
// by the lane that looked it up), announcing each segment; K's place is filled
// again while V is still in use. Waits are bounded: one that gives up flags
// KVD_STATUS_TIMEOUT, and since a segment fixes its tiles, the working warps go on to its end
// together, on whatever the tiles hold, and stop there. The running maxima are only raised, after a vote, when a
// score passes them by 2^15. At a segment's end the warps' states are merged through shared memory.
//
// Measured: 128 sequences of 1,024 to 8,192 tokens, 32 query and 8 KV heads of 128: 144 us (691 MB, 4.8 of 6.8 TB/s
// copied; an instruction issues in 61 % of the cycles, the waits between are of many kinds). 64 sequences of 2,048, 48 query heads
// on one KV head of 256: 38.8 us, 5.5 for the first tile to arrive, 6.5 a tile of 256 tokens (3.2 of it the MMAs alone), 4 a merge. 9
// sequences of up to 4,001 with 5 drafted tokens, 32 and 8 heads of 128: 23.5 us. 12 or 16 working warps in place of 8 (with
// 152 or 112 registers) took 0.5 and 3 us more there, tiles of half the size 2, a schedule formed by the loading warp alone as long.
#pragma once

#include "fp4.cuh"
#include "split_kv_chunk.cuh"
#include "tc_common.cuh"

namespace kvd {

template <int D, int NT, bool F32OUT>
struct Fp4Shape {
    static constexpr int NW = 8, WORKERS = NW * 32;  // working threads
    static constexpr int ROWS = 8 * NT;          // query rows of a CTA
    static constexpr int KS = D / 16;            // k-steps of S^T; row tiles of O^T over the whole head
    // Warps of a group: accumulators (4 * KS / WD * NT registers) of at most 48, but no less than 64 columns a warp.
    static constexpr int WD = (KS * NT * 4 <= 48 || D == 64) ? 1 : (KS * NT * 2 <= 48 || D == 128) ? 2 : 4;
    static constexpr int GROUPS = NW / WD;
    static constexpr int DW = D / WD;            // columns of the output a warp holds
    static constexpr int ACC = KS / WD * NT * 4;
    // Blocks of 16 tokens of a warp per tile: two share each load of q's fragments; one where
    // two would leave room for a single CTA per SM.
    static constexpr int TB = (D == 256 && NT <= 3) ? 1 : 2;
    static constexpr int GB = TB * WD;           // blocks of a group's part of a tile
    static constexpr int CB = TB * NW;           // blocks of a tile: at most 16, a lane for each
    static constexpr int TILE = 16 * CB;
    static constexpr int BLK = Fp4Block<D>::BYTES;
    static constexpr int STAGE = CB * BLK;       // of K, or of V
    static constexpr int STAGES = D == 64 ? 3 : 2;
    static constexpr bool QREG = KS * NT * 2 <= 16;  // q fragments in registers, else in shared memory
    static constexpr int LD = D + 4;             // merge buffer row, floats
    static constexpr int RING = 2 * STAGES * STAGE;  // K stages, then V stages
    // With 8 query rows and warps that work alone every warp's state has room beside the rings, and one barrier stands
    // between them and the joined rows: 64 sequences of 500 to 1,500 tokens, 40 heads of 128, take 103.6 us, about 5 less than without.
    static constexpr bool FLAT = WD == 1 && NT == 1;
    static constexpr int MBUF = FLAT ? GROUPS : GROUPS / 2;          // merge buffers: the upper half of the groups hands over to the lower
    static constexpr int MERGE = MBUF * ROWS * LD * 4;
    static constexpr int PBYTES = WD > 1 ? GROUPS * GB * NT * 256 * (F32OUT ? 2 : 1) : 0;  // the weights' fragments
    static constexpr int SHARED = MERGE > PBYTES ? MERGE : PBYTES;  // weights, and at a segment's end the merge
    static constexpr int QBYTES = QREG ? 0 : KS * NT * 32 * 8;
    static constexpr int SMEM = RING + SHARED + QBYTES;
    static constexpr int STATIC = 4096 + (FLAT ? 3 : 2) * NW * ROWS * 4 + (QREG ? 28 + 4 * NW : 32) * ROWS;  // an upper bound of the static arrays
    static constexpr int MINB = (ACC <= 32 && 2 * (SMEM + STATIC + 1024) <= 228 * 1024) ? 2 : 1;
    // The loading warp is a ninth; a CTA alone on its SM launches a warpgroup for it, whose
    // registers the working warps then take (168 a thread at launch, 232 and 40 after: 2 * 232 + 40 = 3 * 168).
    static constexpr bool SPLIT = MINB == 1;
    static constexpr int THREADS = WORKERS + (SPLIT ? 128 : 32);
    static constexpr int SEG_COST = 1;           // tiles charged per pair
    static_assert(SMEM + STATIC <= 227 * 1024, "shared memory of a CTA");
};

// Schedule geometry: positions of a tile, a whole segment per step.
template <int U, int X>
struct Fp4Geom {
    KVD_HD constexpr int tt() const { return 1 << 30; }
    KVD_HD constexpr int unit() const { return U; }
    KVD_HD constexpr int x() const { return X; }
};

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
// The f16 MMA of common.cuh without its ordering against other instructions: the
// scheduler may move conversions and loads between the products.
__device__ __forceinline__ void mma_free(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int N>
struct Step {
    static constexpr int value = N;
};
template <class V>
__device__ __forceinline__ V lds(const uint8_t* a) {
    return *reinterpret_cast<const V*>(a);
}

// Two floats in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// The low halves of a's bytes and the high halves of b's: (a & 0x0f..) | (b & 0xf0..) in one operation.
__device__ __forceinline__ uint32_t nib(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xe4;" : "=r"(r) : "r"(a), "r"(b), "r"(0x0f0f0f0fu));
    return r;
}

constexpr float kNoMax = -3e38f;  // running maximum before any score
// How far (in powers of two) a score may pass its running maximum, and a weight's exponent its reference mo: 2^15 is still
// an f16 (the largest is 65504). Raising costs up to a fifth of a tile's time.
constexpr float kRoom = 15.f;
// Where mo is put when it is raised: so far below the largest exponent. What f16 has below its normal numbers' 2^-14 is lost to light
// weights, which the sum of the weights holds in 32 bits: 65,536 tokens of 2^-25 of the largest weight each were left out
// of the output when mo was put at the maximum itself. Maxima are raised more often so: 0.8 % of the grouped-query
// case above, 0.5 % with 10 and 0.4 % with 8.
constexpr float kLift = 12.f;
// 2^(x / 2), to be multiplied in twice: an output's factor 2^(mo - M) may lie below the smallest float where the output,
// of V rows near that, does not.
__device__ __forceinline__ float half_ex2(float x) { return tc::ex2_approx(0.5f * x); }
// Integers ordered as the floats they stand for.
__device__ __forceinline__ int float_order(float f) {
    const int i = __float_as_int(f);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float float_unorder(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// Barriers among the n threads of a group (id 1 + group), and among all working threads (id 15); the _any forms
// return whether any thread's v holds.
__device__ __forceinline__ void group_sync(int id, int n) { asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool group_any(int id, int n, bool v) {
    int r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.s32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n selp.s32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(id), "r"(n), "r"((int)v)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void workers_sync(int n) { group_sync(15, n); }
__device__ __forceinline__ bool workers_any(int n, bool v) { return group_any(15, n, v); }

// A segment, as the loading warp announces it.
struct Fp4Segment {
    int b, h, L;         // pair, its length
    int tok_lo, tok_hi;  // the segment's tokens
    bool full;           // it covers the pair
    bool end;            // no segment: the run is over
};

template <int D, int NT, bool F32OUT>
__global__ void __launch_bounds__(Fp4Shape<D, NT, F32OUT>::THREADS, Fp4Shape<D, NT, F32OUT>::MINB)
    split_kv_chunk_fp4_kernel(const __grid_constant__ DecodeParams p) {
    using Sh = Fp4Shape<D, NT, F32OUT>;
    using Blk = Fp4Block<D>;
    using Geo = Fp4Geom<Sh::TILE, Sh::SEG_COST>;
    constexpr int NW = Sh::NW, WORKERS = Sh::WORKERS, THREADS = Sh::THREADS, KS = Sh::KS, STAGES = Sh::STAGES, BLK = Sh::BLK, ROWS = Sh::ROWS;
    constexpr int WD = Sh::WD, TB = Sh::TB, GB = Sh::GB, TILE = Sh::TILE, DW = Sh::DW, MT = KS / WD;
    constexpr int KG = D > 128 ? D / 128 : 1;   // column groups of a K row
    constexpr int KW = D >= 128 ? 4 : 2;        // code words of a thread's K columns in one column group
    constexpr int VG = DW > 128 ? DW / 128 : 1; // column groups of this warp's output columns
    constexpr int VW = DW >= 128 ? 2 : 1;       // code words of a thread's V columns in one column group
    constexpr long long kBudget = 4000000000LL; // ~2 s: a wait that gives up

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_full[2 * STAGES], s_free[2 * STAGES];  // K stages, V stages
    constexpr int SEGS = 8;  // announced segments: the loading warp is at most STAGES + 1 ahead
    static_assert(STAGES + 2 <= SEGS, "announced segments");
    __shared__ Fp4Segment s_seg[SEGS];
    __shared__ __align__(8) uint64_t s_told[SEGS];
    __shared__ uint32_t s_bad[STAGES];  // bit x: block x of the tile names no page
    __shared__ long long s_red[THREADS / 32];
    __shared__ long long s_cum0;
    __shared__ int s_b0, s_abort;
    __shared__ __align__(8) float s_ml[NW][ROWS], s_l[NW][ROWS];  // running maxima and sums; s_ml also carries raised maxima
    __shared__ float s_qs[ROWS], s_inv[ROWS];
    __shared__ __align__(8) float s_qfar[Sh::QREG ? NW : 1][ROWS];  // the rest of the queries' factors above 2^10, else 1
    __shared__ float s_mo[Sh::FLAT ? NW : 1][ROWS];  // running maxima of the outputs
    __shared__ int s_max[ROWS];  // a segment's maxima, as ordered integers
    __shared__ long long s_dst[ROWS];
    __shared__ int s_short[ROWS];
    float* s_merge = reinterpret_cast<float*>(smem + Sh::RING);
    uint2* s_q = reinterpret_cast<uint2*>(smem + Sh::RING + Sh::SHARED);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = warp / WD, wg = warp % WD;
    const int r = lane >> 2, c4 = lane & 3;
    const int G = p.G, T = p.T, TG = T * G;
    const int c = blockIdx.x / p.row_blocks;
    const int rbase = (blockIdx.x - c * p.row_blocks) * ROWS;
    const int rend = min(TG, rbase + ROWS);
    auto out_row = [&](int b, int h, int rr) {  // row of out / lse ([B, T, Hq])
        const int i = rr / G;
        return ((size_t)b * T + i) * p.Hq + (size_t)h * G + (rr - i * G);
    };

    if (!p.early) pdl_wait();
    pdl_launch_dependents();

    if (tid < 2 * STAGES) tc::mbar_init(smem_u32(s_full + tid), 1), tc::mbar_init(smem_u32(s_free + tid), NW);
    if (tid < SEGS) tc::mbar_init(smem_u32(s_told + tid), 1);
    if (tid == 0) s_abort = 0, s_b0 = p.B, s_cum0 = 0;
    // Tokens a query row sees fewer than the last token's.
    if (tid < ROWS) s_short[tid] = T - 1 - min(rbase + tid, TG - 1) / G, s_max[tid] = float_order(kNoMax);
    tc::mbar_fence_init();

    // ---- this CTA's run of the line of (sequence, KV head) pairs, from one scan of the extents ----
    // Thread i takes sequences [i * per, (i + 1) * per). The first sequence of the run is the first b
    // that is_first_seq_candidate selects; that holds from some b on, so the thread that sees it begin knows.
    const DevLen len{p.seq_lens, p.len_cap, 1};
    const int per = (p.B + THREADS - 1) / THREADS, lo_b = min(p.B, tid * per), hi_b = min(p.B, lo_b + per);
    long long mine = 0;
    bool clamped = false;
#pragma unroll 1
    for (int b = lo_b; b < hi_b; ++b) {
        const int raw = __ldg(p.seq_lens + b);
        const int L = clamp_len(raw, p.len_cap);
        clamped |= (raw != L);
        mine += pair_extent(L, Geo{});
    }
    if (clamped && blockIdx.x == 0 && p.status) atomicOr(p.status, KVD_STATUS_SEQ_LEN_CLAMPED);
    mine *= p.Hkv;
    long long total;
    long long cum = block_incl_scan_ll<THREADS / 32>(mine, s_red, &total) - mine;
    const int C_eff = effective_ctas(p.n_split, total);
    if (c >= C_eff) {
        if (p.early) pdl_wait();
        return;
    }
    const long long S = run_begin(c, C_eff, total);
    {
        bool before = false;  // the sequence before this one is a candidate
        if (lo_b > 0 && lo_b < p.B) {
            const long long e = pair_extent(len(lo_b - 1), Geo{});
            before = is_first_seq_candidate(cum - e * p.Hkv, e, p.Hkv, S);
        }
#pragma unroll 1
        for (int b = lo_b; b < hi_b && !before; ++b) {
            const long long e = pair_extent(len(b), Geo{});
            before = is_first_seq_candidate(cum, e, p.Hkv, S);
            if (before) {
                s_b0 = b;
                s_cum0 = cum;
            }
            cum += e * p.Hkv;
        }
    }
    __syncthreads();
    volatile int* abort_flag = &s_abort;
    const uint32_t full = smem_u32(s_full), freed = smem_u32(s_free), told = smem_u32(s_told);
    auto give_up = [&]() {
        if (lane == 0 && p.status) atomicOr(p.status, KVD_STATUS_TIMEOUT);
    };

    if (warp >= NW) {
        if constexpr (Sh::SPLIT) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
            if (warp > NW) {
                if (p.early) pdl_wait();  // no warp is done before the preceding grid
                return;
            }
        }
        // ---- the loading warp: the walk of Walker::next (schedule.cuh), a segment of any length at a time ----
        constexpr int X = Sh::SEG_COST, CB = Sh::CB;
        const long long E = run_begin(c + 1, C_eff, total);
        long long pstart = s_cum0, pos = S;
        int b = s_b0, h = 0, L = b < p.B ? len(b) : 0;
        if (L > 0 && pstart < S) {
            const long long e = pair_extent(L, Geo{});
            h = (int)div_nonneg(S - pstart, e);
            pstart += (long long)h * e;
        }
        auto next_pair = [&]() {
            if (L == 0) {  // an empty pair of this run: zero rows
#pragma unroll 1
                for (int i = rbase * (D / 8) + lane; i < rend * (D / 8); i += 32) {
                    const size_t row = out_row(b, h, i / (D / 8)), e = row * D + (i % (D / 8)) * 8;
                    if constexpr (F32OUT) {
                        float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + e);
                        d[0] = d[1] = make_float4(0.f, 0.f, 0.f, 0.f);
                    } else {
                        *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + e) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    if (p.lse && i % (D / 8) == 0) p.lse[row] = -CUDART_INF_F;
                }
            }
            pstart += pair_extent(L, Geo{});
            if (++h == p.Hkv) {
                h = 0;
                ++b;
                L = b < p.B ? len(b) : 0;
            }
        };
        if (p.early) pdl_wait();  // the appended rows
        int stage = 0;
        uint32_t round = 0, nseg = 0;  // passes through the ring, segments announced
        bool fine = true;
        auto announce = [&](const Fp4Segment& sg) {
            if (lane == 0) {
                s_seg[nseg & (SEGS - 1)] = sg;
                tc::mbar_arrive(told + 8u * (nseg & (SEGS - 1)));
            }
            ++nseg;
        };
        auto take = [&](int which) {  // waits until a stage is free
            if (round > 0 && fine && !tc::mbar_wait(freed + 8u * (which * STAGES + stage), (round - 1) & 1u, abort_flag, kBudget)) {
                fine = false;
                give_up();
            }
        };
#pragma unroll 1
        while (fine && pos < E) {
#pragma unroll 1
            while (pos >= pstart + pair_extent(L, Geo{})) next_pair();
            const long long real0 = pstart + X, pend = pstart + pair_extent(L, Geo{});  // the pair's tokens
            if (pos < real0) pos = real0;
            if (pos >= E) break;
            const long long te = min(pend, E);
            const int tok_lo = (int)(pos - real0) * TILE, tok_hi = (int)min((te - real0) * TILE, (long long)L);
            const bool covers = real0 >= S && pend <= E;
            pos = te;
            announce(Fp4Segment{b, h, L, tok_lo, tok_hi, covers, false});
            if (lane < T)  // the segment's queries into L2, ahead of their loads
                tc::prefetch_l2(static_cast<const __nv_bfloat16*>(p.q) + (((size_t)b * T + lane) * p.Hq + (size_t)h * G) * D,
                                (uint32_t)(G * D * 2));
#pragma unroll 1
            for (int tok = tok_lo; tok < tok_hi && fine; tok += TILE) {
                const int n = min(CB, (tok_hi - tok + 15) >> 4);  // blocks of this tile
                size_t blk = 0;
                int run = 0;  // blocks to copy from this lane's on
                bool ok = true;
                if (!p.block_table) {
                    if (lane == 0) {
                        run = n;
                        blk = (size_t)((long long)b * p.Hkv + h) * (p.S_max >> 4) + (tok >> 4);
                    }
                } else {
                    const int in = 1 << (p.page_shift - 4), t = tok + 16 * lane, at = (t >> 4) & (in - 1);
                    if (lane < n && (lane == 0 || at == 0)) {
                        run = min(n - lane, in - at);
                        const int page = __ldg(p.block_table + (size_t)b * p.max_blocks + (t >> p.page_shift));
                        ok = (unsigned)page < (unsigned)p.num_pages;
                        if (!ok && p.status) atomicOr(p.status, KVD_STATUS_BAD_PAGE);
                        blk = (size_t)((long long)page * p.Hkv + h) * in + at;
                    }
                }
                const uint32_t bytes = ok ? (uint32_t)(run * BLK) : 0u;
                const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
                const uint32_t bad = __reduce_or_sync(0xffffffffu, ok ? 0u : ((1u << run) - 1u) << lane);
                // A CTA's codes are read once, unless row blocks share them.
                const uint64_t pol = p.row_blocks > 1 ? tc::l2_evict_last_policy() : l2_evict_first_policy();
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {
                    take(which);
                    if (!fine) break;
                    const uint32_t bar = full + 8u * (which * STAGES + stage);
                    if (lane == 0) {
                        if (which == 0) s_bad[stage] = bad;
                        tc::mbar_arrive_expect_tx(bar, sum);
                    }
                    __syncwarp();
                    if (bytes)
                        tc::bulk_load_1d(smem_u32(smem) + (uint32_t)((which * STAGES + stage) * Sh::STAGE + lane * BLK),
                                         static_cast<const uint8_t*>(which ? p.v : p.k) + blk * BLK, bytes, bar, pol);
                }
                if (++stage == STAGES) stage = 0, ++round;
            }
        }
        announce(Fp4Segment{0, 0, 0, 0, 0, false, true});
        if (c == C_eff - 1) {  // the last CTA also owns the empty pairs at the very end of the line
            pos = E;           // (the run may end inside a pair's charge)
#pragma unroll 1
            while (b < p.B && pos >= pstart + pair_extent(L, Geo{})) next_pair();
        }
        if (!fine) {  // bounded wait for copies in flight before the shared memory is given up
            int go = 0;
            const uint32_t parity = round;  // stages before `stage` were filled in this round, the others in the one before
#pragma unroll 1
            for (int s = 0; s < 2 * STAGES; ++s)
                tc::mbar_wait(full + 8u * s, (s % STAGES < stage ? parity : parity - 1) & 1u, &go, kBudget / 16);
        }
        return;
    }

    if constexpr (Sh::SPLIT) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n");
    uint2 qf[Sh::QREG ? KS * NT : 1];
    float qs[Sh::QREG ? NT : 1][2];  // |scale| * 2^(q's exponent) of this thread's query columns 8 j + 2 c4 + {0, 1}

    int stage = 0;
    uint32_t round = 0;
    bool fine = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (fine && !tc::mbar_wait(bar, parity & 1u, abort_flag, kBudget)) {
            fine = false;
            give_up();
        }
    };
    auto wait_tile = [&](int which) { wait(full + 8u * (which * STAGES + stage), round); };  // K (0) or V (1)
    auto done = [&](int which) {  // behind the tile's last use of K or V
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(freed + 8u * (which * STAGES + stage));
    };
    wait(told, 0);
    if (workers_any(WORKERS, !fine)) return;
#pragma unroll 1
    for (uint32_t n = 0;;) {
        const Fp4Segment ct = s_seg[n & (SEGS - 1)];
        if (ct.end) break;
        // ---- the pair's queries: f16 relative to each row's largest element, a negative scale's sign with them ----
        const uint4* qg = reinterpret_cast<const uint4*>(p.q);
        auto load_q = [&](int j, uint2* dst, int stride) {  // dst[k-step * stride]; returns the row's scale
            const int rr = rbase + 8 * j + r;
            uint4 w[KG * KW];
            float m = 0.f;
            const size_t e = (rr < TG ? out_row(ct.b, ct.h, rr) : 0) * (D / 8);
#pragma unroll
            for (int g = 0; g < KG; ++g)
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    w[g * KW + k] = rr < TG ? __ldg(qg + e + g * 16 + c4 * KW + k) : make_uint4(0, 0, 0, 0);
                    const uint32_t x[4] = {w[g * KW + k].x, w[g * KW + k].y, w[g * KW + k].z, w[g * KW + k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(x[i])), fabsf(bf16_hi(x[i]))));
                }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t eb = min(max(__float_as_uint(m) >> 23, 1u), 253u);
            const float dn = copysignf(__uint_as_float((254u - eb) << 23), p.scale_log2);
#pragma unroll
            for (int k = 0; k < KG * KW; ++k) {
                const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = pack_f16x2(bf16_lo(x[i]) * dn, bf16_hi(x[i]) * dn);
                dst[(2 * k) * stride] = make_uint2(y[0], y[1]);
                dst[(2 * k + 1) * stride] = make_uint2(y[2], y[3]);
            }
            // A factor above 2^10 goes in apart, behind the rest: with the cache row's it could overflow, and a score of zero become a NaN.
            const float f = fabsf(p.scale_log2) * __uint_as_float(eb << 23);
            if (c4 == 0) s_qfar[Sh::QREG ? warp : 0][8 * j + r] = f > 1024.f ? f * 9.765625e-4f : 1.f;
            return fminf(f, 1024.f);
        };
        if constexpr (Sh::QREG) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float sc = load_q(j, qf + j, NT);
                qs[j][0] = __shfl_sync(0xffffffffu, sc, 8 * c4);
                qs[j][1] = __shfl_sync(0xffffffffu, sc, 8 * c4 + 4);
            }
        } else {
            // One warp per column tile; the previous segment's readers are behind its merge.
            if (warp < NT) {
                const float sc = load_q(warp, s_q + warp * 32 + lane, NT * 32);
                if (c4 == 0) s_qs[warp * 8 + r] = sc;
            }
            workers_sync(WORKERS);
        }
        __syncwarp();
        bool far = false;  // some query's factor is in two parts
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int z = 0; z < 2; ++z) far |= s_qfar[Sh::QREG ? warp : 0][8 * j + 2 * c4 + z] != 1.f;
        far = __any_sync(0xffffffffu, far);
        float o[MT][NT][4];
        float ms[NT][2], mo[NT][2], l[NT][2];  // mo is the group's, ms and l this warp's
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) ms[j][x] = mo[j][x] = kNoMax, l[j][x] = 0.f;

#pragma unroll 1
        for (int tile = ct.tok_lo; tile < ct.tok_hi; tile += TILE) {  // (nothing in here but waits depends on memory)
            const int tile0 = tile + 16 * GB * group;       // the group's part
            const int tok0 = tile0 + 16 * TB * wg;          // this warp's blocks
            const uint8_t* kt = smem + stage * Sh::STAGE + GB * group * BLK;  // the group's K blocks, and its V blocks
            const uint8_t* vt = kt + Sh::RING / 2;
            const uint8_t* kb = kt + TB * wg * BLK;
            wait_tile(0);
            if (tile0 >= ct.tok_hi) {  // the segment ends before this group's part
                done(0);
                wait_tile(1);
            } else {
            // A block that names no page holds anything: its scales become zero, its exponents 2^0.
            const uint32_t badm = p.block_table ? (s_bad[stage] >> (TB * warp)) & ((1u << TB) - 1) : 0u;
            auto patch = [&](uint8_t* blk, bool none, int keep) {  // zero rows from token `keep` on, or all of them
                if (none) keep = 0;
#pragma unroll 1
                for (int i = lane; i < D; i += 32)  // scale byte i is token i / (D / 16)'s
                    if (i / (D / 16) >= keep) blk[Blk::SCALES + i] = 0;
                if (lane < 16 && lane >= keep) blk[Blk::EXPS + lane] = 127;
            };
            if (badm) {
#pragma unroll 1
                for (int x = 0; x < TB; ++x)
                    if ((badm >> x) & 1u) patch(smem + stage * Sh::STAGE + (TB * warp + x) * BLK, true, 0);
                __syncwarp();
                // These writes come before the bulk copy that fills the stage again.
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            }
            const int ta = r ^ ((r >> 1) & 1);  // token of MMA row r (row r + 8: 8 more)

            // ---- S^T = K q^T ----
            float s[TB][NT][4];
#pragma unroll
            for (int x = 0; x < TB; ++x)
#pragma unroll
                for (int j = 0; j < NT; ++j) s[x][j][0] = s[x][j][1] = s[x][j][2] = s[x][j][3] = 0.f;
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                uint32_t w[TB][2][KW];     // [block][row half][word]
                uint32_t sc[TB][2][2];     // [block][row half][scale of word / 2], twice in one register
#pragma unroll
                for (int x = 0; x < TB; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint8_t* a = kb + x * BLK + g * 16 * Blk::ROW + (ta + 8 * y) * Blk::ROW;
                        if constexpr (D >= 128) {
                            const uint4 v = lds<uint4>(a + c4 * 16);
                            w[x][y][0] = v.x, w[x][y][1] = v.y, w[x][y][2] = v.z, w[x][y][3] = v.w;
                            const uint32_t h = e4m3x2_to_f16x2(
                                lds<uint16_t>(kb + x * BLK + Blk::SCALES + (ta + 8 * y) * (D / 16) + 8 * g + 2 * c4));
                            sc[x][y][0] = __byte_perm(h, 0, 0x1010);
                            sc[x][y][1] = __byte_perm(h, 0, 0x3232);
                        } else {
                            const uint2 v = lds<uint2>(a + c4 * 8);
                            w[x][y][0] = v.x, w[x][y][1] = v.y;
                            sc[x][y][0] = e4m3x2_to_f16x2(
                                lds<uint8_t>(kb + x * BLK + Blk::SCALES + (ta + 8 * y) * (D / 16) + c4) * 0x101u);
                            sc[x][y][1] = sc[x][y][0];
                        }
                    }
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    const int ks = 2 * (g * KW + k);
                    uint32_t a0[TB][4], a1[TB][4];
#pragma unroll
                    for (int x = 0; x < TB; ++x) {
                        uint32_t h0[4], h1[4];
                        e2m1x8_to_f16(w[x][0][k], h0);
                        e2m1x8_to_f16(w[x][1][k], h1);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            a0[x][2 * i] = hmul2(h0[i], sc[x][0][k / 2]);
                            a0[x][2 * i + 1] = hmul2(h1[i], sc[x][1][k / 2]);
                            a1[x][2 * i] = hmul2(h0[2 + i], sc[x][0][k / 2]);
                            a1[x][2 * i + 1] = hmul2(h1[2 + i], sc[x][1][k / 2]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        uint2 qa, qb;
                        if constexpr (Sh::QREG) {
                            qa = qf[ks * NT + j], qb = qf[(ks + 1) * NT + j];
                        } else {
                            qa = s_q[(ks * NT + j) * 32 + lane], qb = s_q[((ks + 1) * NT + j) * 32 + lane];
                        }
#pragma unroll
                        for (int x = 0; x < TB; ++x) mma_free(s[x][j], a0[x], qa.x, qa.y);
#pragma unroll
                        for (int x = 0; x < TB; ++x) mma_free(s[x][j], a1[x], qb.x, qb.y);
                    }
                }
            }

            // ---- row exponents, masks, running maxima ----
            float ev[TB][2], kf[TB][2];
#pragma unroll
            for (int x = 0; x < TB; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) kf[x][y] = fp4_row_scale(lds<uint8_t>(kb + x * BLK + Blk::EXPS + ta + 8 * y));
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float q0, q1;
                if constexpr (Sh::QREG)
                    q0 = qs[j][0], q1 = qs[j][1];
                else
                    q0 = s_qs[8 * j + 2 * c4], q1 = s_qs[8 * j + 2 * c4 + 1];
#pragma unroll
                for (int x = 0; x < TB; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        // The two factors first: the row's (up to 2^117) alone may take a score out of range that the query's brings back.
                        const float2 v = mul2(make_float2(s[x][j][2 * y], s[x][j][2 * y + 1]),
                                              mul2(make_float2(kf[x][y], kf[x][y]), make_float2(q0, q1)));
                        s[x][j][2 * y] = v.x;
                        s[x][j][2 * y + 1] = v.y;
                    }
            }
            done(0);
            wait_tile(1);
            // Rows past the sequence or without a page hold anything: this warp's V blocks of the tile are put
            // right in shared memory, and scores that a query row does not see masked, so that nothing below has to ask.
            const bool edge = (tile0 + 16 * GB > ct.L - T + 1) || badm || far;
            if (edge) {
#pragma unroll 1
                for (int x = 0; x < TB; ++x)
                    patch(smem + Sh::RING / 2 + stage * Sh::STAGE + (TB * warp + x) * BLK, (badm >> x) & 1u, ct.L - tok0 - 16 * x);
                __syncwarp();
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            }
#pragma unroll
            for (int x = 0; x < TB; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)  // the byte b as 2^23 + b, less 2^23 + 127
                    ev[x][y] = __uint_as_float(0x4b000000u | lds<uint8_t>(kb + Sh::RING / 2 + x * BLK + Blk::EXPS + ta + 8 * y)) - 8388735.f;
            if (edge) {  // (a branch of its own for the large factors cost 1 to 2 % of every case)
#pragma unroll
                for (int x = 0; x < TB; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                s[x][j][2 * y + z] *= s_qfar[Sh::QREG ? warp : 0][8 * j + 2 * c4 + z];
                                if (tok0 + 16 * x + ta + 8 * y >= ct.L - s_short[8 * j + 2 * c4 + z]) s[x][j][2 * y + z] = -CUDART_INF_F;
                            }
            }
            bool raise = false;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int x = 0; x < TB; ++x)
                        raise |= fmaxf(s[x][j][z], s[x][j][2 + z]) > ms[j][z] + kRoom ||
                                 fmaxf(s[x][j][z] + ev[x][0], s[x][j][2 + z] + ev[x][1]) > mo[j][z] + kRoom;
            if constexpr (WD > 1) {
                raise = group_any(1 + group, 32 * WD, raise);  // also: the group is done with the previous tile's weights
            } else {
                raise = __any_sync(0xffffffffu, raise);
            }
            if (raise) {
                float ho[NT][2];
                if constexpr (WD == 1) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            float hs = fmaxf(s[0][j][z], s[0][j][2 + z]);
                            ho[j][z] = fmaxf(s[0][j][z] + ev[0][0], s[0][j][2 + z] + ev[0][1]);
                            if constexpr (TB > 1) {
                                hs = fmaxf(hs, fmaxf(s[TB - 1][j][z], s[TB - 1][j][2 + z]));
                                ho[j][z] = fmaxf(ho[j][z], fmaxf(s[TB - 1][j][z] + ev[TB - 1][0], s[TB - 1][j][2 + z] + ev[TB - 1][1]));
                            }
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) {
                                hs = fmaxf(hs, __shfl_xor_sync(0xffffffffu, hs, off));
                                ho[j][z] = fmaxf(ho[j][z], __shfl_xor_sync(0xffffffffu, ho[j][z], off));
                            }
                            const float ns = fmaxf(ms[j][z], hs);
                            l[j][z] *= tc::ex2_approx(ms[j][z] - ns);
                            ms[j][z] = ns;
                        }
                } else {
                    // Of the 2 NT maxima that the 8 lanes of a column hold, each exchange leaves a lane half (an odd number is
                    // exchanged whole); they go to s_l (scores, this warp's) and s_ml (with V's exponents, the group's).
                    auto fold = [&](float* to, bool with_ev) {
                        float v[2 * NT];
#pragma unroll
                        for (int i = 0; i < 2 * NT; ++i)
#pragma unroll
                            for (int x = 0; x < TB; ++x) {
                                const float a = s[x][i / 2][i % 2] + (with_ev ? ev[x][0] : 0.f),
                                            b = s[x][i / 2][2 + i % 2] + (with_ev ? ev[x][1] : 0.f);
                                v[i] = x ? fmaxf(v[i], fmaxf(a, b)) : fmaxf(a, b);
                            }
                        int n = 2 * NT, at = 0;  // v[i] is maximum at + i
#pragma unroll
                        for (int off = 16; off >= 4; off >>= 1) {
                            const bool up = lane & off;
                            if (n % 2 == 0) {
                                n /= 2;
                                at += up ? n : 0;
#pragma unroll
                                for (int i = 0; i < n; ++i) {
                                    const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                                    v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, off));
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < n; ++i) v[i] = fmaxf(v[i], __shfl_xor_sync(0xffffffffu, v[i], off));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < n; ++i) to[8 * ((at + i) >> 1) + 2 * c4 + ((at + i) & 1)] = v[i];
                    };
                    fold(s_l[warp], false);
                    fold(s_ml[warp], true);
                    group_sync(1 + group, 32 * WD);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float2 a = *reinterpret_cast<const float2*>(&s_l[warp][8 * j + 2 * c4]);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const float ns = fmaxf(ms[j][z], z ? a.y : a.x);
                            l[j][z] *= tc::ex2_approx(ms[j][z] - ns);
                            ms[j][z] = ns;
                        }
#pragma unroll
                        for (int w = 0; w < WD; ++w) {
                            const float2 b = *reinterpret_cast<const float2*>(&s_ml[group * WD + w][8 * j + 2 * c4]);
                            ho[j][0] = w ? fmaxf(ho[j][0], b.x) : b.x, ho[j][1] = w ? fmaxf(ho[j][1], b.y) : b.y;
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const float no = fmaxf(mo[j][z], ho[j][z] - kLift);
                        const float f = tc::ex2_approx(mo[j][z] - no);
                        mo[j][z] = no;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[i][j][z] *= f;
                            o[i][j][2 + z] *= f;
                        }
                    }
            }

            // ---- weights, as B fragments ----
            constexpr int PL = F32OUT ? 2 : 1;  // f16 parts of a weight, the second times 2^11
            uint2 wf[WD == 1 ? TB : 1][NT][PL];
            uint2* s_p = reinterpret_cast<uint2*>(s_merge) + group * (GB * NT * PL * 32) + lane;
#pragma unroll
            for (int x = 0; x < TB; ++x)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float2 v = make_float2(s[x][j][2 * y], s[x][j][2 * y + 1]);
                        const float2 a = add2(v, make_float2(-ms[j][0], -ms[j][1]));
                        const float2 b = add2(add2(v, make_float2(ev[x][y], ev[x][y])), make_float2(-mo[j][0], -mo[j][1]));
                        const float2 sum = add2(make_float2(l[j][0], l[j][1]), make_float2(tc::ex2_approx(a.x), tc::ex2_approx(a.y)));
                        l[j][0] = sum.x, l[j][1] = sum.y;
                        const float wv[2] = {tc::ex2_approx(b.x), tc::ex2_approx(b.y)};
                        const uint32_t h = pack_f16x2(wv[0], wv[1]);
                        hi[y] = movmatrix_trans(h);
                        if constexpr (F32OUT) lo[y] = movmatrix_trans(pack_f16x2(2048.f * (wv[0] - f16_lo(h)), 2048.f * (wv[1] - f16_hi(h))));
                    }
                    if constexpr (WD == 1) {
                        wf[x][j][0] = make_uint2(hi[0], hi[1]);
                        if constexpr (F32OUT) wf[x][j][1] = make_uint2(lo[0], lo[1]);
                    } else {
                        uint2* d = s_p + ((wg * TB + x) * NT + j) * PL * 32;
                        d[0] = make_uint2(hi[0], hi[1]);
                        if constexpr (F32OUT) d[32] = make_uint2(lo[0], lo[1]);
                    }
                }
            if constexpr (WD > 1) group_sync(1 + group, 32 * WD);

            // ---- O^T += V^T w over the group's blocks, this warp's columns ----
            const int t0 = (2 * c4) ^ (c4 & 1), t1 = t0 ^ 1;  // tokens of k = 2 c4, 2 c4 + 1 (and 8 more)
            const int d0 = wg * DW;                           // first column
            const int blocks = min(GB, (ct.tok_hi - tile0 + 15) >> 4);
            auto block_pv = [&](int x, const uint2 (&wx)[NT][PL]) {
                const uint8_t* base = vt + x * BLK;
#pragma unroll
                for (int g = 0; g < VG; ++g) {
                    uint32_t w[4][VW], sc[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint8_t* a = base + (d0 / 128 + g) * 16 * Blk::ROW + (d0 % 128) / 2 + 8 * y * Blk::ROW;
                        if constexpr (DW >= 128) {
                            const uint2 u0 = lds<uint2>(a + t0 * Blk::ROW + r * 8), u1 = lds<uint2>(a + t1 * Blk::ROW + r * 8);
                            w[2 * y][0] = u0.x, w[2 * y][1] = u0.y, w[2 * y + 1][0] = u1.x, w[2 * y + 1][1] = u1.y;
                        } else {
                            w[2 * y][0] = lds<uint32_t>(a + t0 * Blk::ROW + r * 4);
                            w[2 * y + 1][0] = lds<uint32_t>(a + t1 * Blk::ROW + r * 4);
                        }
                        const uint8_t* sb = base + Blk::SCALES + 8 * y * (D / 16) + d0 / 16 + (DW >= 128 ? 8 * g + r : r / 2);
                        sc[y] = e4m3x2_to_f16x2(lds<uint8_t>(sb + t0 * (D / 16)) | (lds<uint8_t>(sb + t1 * (D / 16)) << 8));
                    }
#pragma unroll
                    for (int v = 0; v < VW; ++v) {
                        uint32_t ev0[4], od0[4], ev1[4], od1[4];  // even and odd columns, token pairs 0 and 8 further
                        e2m1x8_to_f16(nib(w[0][v], w[1][v] << 4), ev0);
                        e2m1x8_to_f16(nib(w[0][v] >> 4, w[1][v]), od0);
                        e2m1x8_to_f16(nib(w[2][v], w[3][v] << 4), ev1);
                        e2m1x8_to_f16(nib(w[2][v] >> 4, w[3][v]), od1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a[4] = {hmul2(ev0[i], sc[0]), hmul2(od0[i], sc[0]), hmul2(ev1[i], sc[1]),
                                                   hmul2(od1[i], sc[1])};
                            const int m = (g * VW + v) * 4 + i;
#pragma unroll
                            for (int j = 0; j < NT; ++j) mma_free(o[m][j], a, wx[j][0].x, wx[j][0].y);
                            if constexpr (F32OUT) {
                                const uint32_t cut = 0x10001000u;  // 2^-11, twice
                                const uint32_t a1[4] = {hmul2(a[0], cut), hmul2(a[1], cut), hmul2(a[2], cut), hmul2(a[3], cut)};
#pragma unroll
                                for (int j = 0; j < NT; ++j) mma_free(o[m][j], a1, wx[j][1].x, wx[j][1].y);
                            }
                        }
                    }
                }
            };
            if constexpr (WD == 1) {
#pragma unroll
                for (int x = 0; x < TB; ++x) {
                    if (x >= blocks) break;
                    uint2 wx[NT][PL];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int k = 0; k < PL; ++k)
                            wx[j][k] = wf[x][j][k];
                    block_pv(x, wx);
                }
            } else {
#pragma unroll 1
                for (int x = 0; x < blocks; ++x) {
                    uint2 wx[NT][PL];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int k = 0; k < PL; ++k) wx[j][k] = s_p[((x * NT + j) * PL + k) * 32];
                    block_pv(x, wx);
                }
            }
            }
            done(1);
            if (++stage == STAGES) stage = 0, ++round;
        }

        if constexpr (Sh::FLAT) {
            // ---- merge the warps' states: each leaves its own as it is, and every thread joins 4 columns of a row ----
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                float sum = l[0][z];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (r == 0) {
                    s_ml[warp][2 * c4 + z] = ms[0][z];
                    s_l[warp][2 * c4 + z] = sum;
                    s_mo[warp][2 * c4 + z] = mo[0][z];
                }
            }
#pragma unroll
            for (int v = 0; v < VW; ++v)
#pragma unroll
                for (int z = 0; z < 2; ++z) {  // columns as in exchange below
                    float4* d = reinterpret_cast<float4*>(s_merge + (warp * ROWS + 2 * c4 + z) * Sh::LD + 8 * (VW * r + v));
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        d[x] = make_float4(o[4 * v + 2 * x][0][z], o[4 * v + 2 * x][0][2 + z], o[4 * v + 2 * x + 1][0][z],
                                           o[4 * v + 2 * x + 1][0][2 + z]);
                }
            workers_sync(WORKERS);
#pragma unroll 1
            for (int i = tid; i < (rend - rbase) * (D / 4); i += WORKERS) {
                const int row = i / (D / 4), col = (i - row * (D / 4)) * 4;
                float M = kNoMax, L = 0.f;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w][row]);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    L += s_l[w][row] * tc::ex2_approx(s_ml[w][row] - M);
                    const float m = s_mo[w][row], g = m > kNoMax ? half_ex2(m - M) : 0.f;
                    const float4 e = *reinterpret_cast<const float4*>(s_merge + (w * ROWS + row) * Sh::LD + col);
                    f = make_float4(f.x + g * e.x * g, f.y + g * e.y * g, f.z + g * e.z * g, f.w + g * e.w * g);
                }
                if (ct.full) {
                    const size_t orow = out_row(ct.b, ct.h, rbase + row);
                    const float inv = L > 0.f ? 1.f / L : 0.f;
                    if constexpr (F32OUT)
                        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + orow * D + col) =
                            make_float4(f.x * inv, f.y * inv, f.z * inv, f.w * inv);
                    else
                        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * D + col) =
                            make_uint2(pack_bf16x2(f.x * inv, f.y * inv), pack_bf16x2(f.z * inv, f.w * inv));
                    if (p.lse && col == 0) p.lse[orow] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -CUDART_INF_F;
                } else {
                    const size_t slot = ((size_t)c + ct.b * p.Hkv + ct.h) * TG + rbase + row;
                    *reinterpret_cast<float4*>(p.ws_o + slot * D + col) = f;
                    if (col == 0) p.ws_ml[slot] = make_float2(M, L);
                }
            }
        } else {
            // ---- merge the warps' states ----
            // The rows' maxima first, by atomics on ordered integers (a maximum does not depend on their order).
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    if (r == 0) atomicMax(&s_max[8 * j + 2 * c4 + z], float_order(ms[j][z]));
            workers_sync(WORKERS);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float M = float_unorder(s_max[8 * j + 2 * c4 + z]);
                    const float f = mo[j][z] > kNoMax ? half_ex2(mo[j][z] - M) : 0.f;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[i][j][z] = o[i][j][z] * f * f;
                        o[i][j][2 + z] = o[i][j][2 + z] * f * f;
                    }
                    float sum = l[j][z] * tc::ex2_approx(ms[j][z] - M);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    if (r == 0) s_l[warp][8 * j + 2 * c4 + z] = sum;
                }
            auto finish_rows = [&](int i) {  // a thread per row: sum, and where the row goes
                if (i < 0 || i >= rend - rbase) return;
                float L = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) L += s_l[w][i];
                const float M = float_unorder(s_max[i]);
                if (ct.full) {
                    const size_t orow = out_row(ct.b, ct.h, rbase + i);
                    s_inv[i] = L > 0.f ? 1.f / L : 0.f;
                    s_dst[i] = (long long)orow * D;
                    if (p.lse) p.lse[orow] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -CUDART_INF_F;
                } else {
                    const size_t slot = ((size_t)c + ct.b * p.Hkv + ct.h) * TG + rbase + i;
                    s_dst[i] = (long long)slot * D;
                    p.ws_ml[slot] = make_float2(M, L);
                }
            };
            auto emit = [&](int row, int col, const float4& f) {  // four columns of a merged row
                float* ws = p.ws_o + s_dst[row] + col;
                if (ct.full) {
                    const float inv = s_inv[row];
                    if constexpr (F32OUT)
                        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + s_dst[row] + col) =
                            make_float4(f.x * inv, f.y * inv, f.z * inv, f.w * inv);
                    else
                        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + s_dst[row] + col) =
                            make_uint2(pack_bf16x2(f.x * inv, f.y * inv), pack_bf16x2(f.z * inv, f.w * inv));
                } else {
                    *reinterpret_cast<float4*>(ws) = f;
                }
            };
            // Column of o[(g * VW + v) * 4 + i][j][0 / 2]: d0 + 128 g + 8 (VW r + v) + 2 i, + 1 for rows r + 8.
            // step 0: to the buffer; 1: the buffer added, and back to it.
            auto exchange = [&](auto step) {
#pragma unroll
                for (int g = 0; g < VG; ++g)
#pragma unroll
                    for (int v = 0; v < VW; ++v)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const int row = 8 * j + 2 * c4 + z, col = wg * DW + 128 * g + 8 * (VW * r + v);
                                float4* d = reinterpret_cast<float4*>(s_merge + ((group % Sh::MBUF) * ROWS + row) * Sh::LD + col);
                                const int m = (g * VW + v) * 4;
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    float4 f = make_float4(o[m + 2 * x][j][z], o[m + 2 * x][j][2 + z], o[m + 2 * x + 1][j][z],
                                                           o[m + 2 * x + 1][j][2 + z]);
                                    if constexpr (decltype(step)::value > 0) {
                                        const float4 e = d[x];
                                        f = make_float4(f.x + e.x, f.y + e.y, f.z + e.z, f.w + e.w);
                                    }
                                    d[x] = f;
                                }
                            }
            };
            // The last sum leaves from shared memory in a short loop of all threads: unrolled from the registers of half of
            // them it took twice as long, much of it fetching instructions that run once.
            if (group >= Sh::MBUF) exchange(Step<0>{});
            workers_sync(WORKERS);
            if (group < Sh::MBUF)
                exchange(Step<1>{});
            else
                finish_rows(tid - WORKERS / 2);
            workers_sync(WORKERS);
#pragma unroll 1
            for (int i = tid; i < (rend - rbase) * (D / 4); i += WORKERS) {
                const int row = i / (D / 4), col = (i - row * (D / 4)) * 4;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < Sh::MBUF; ++w) {
                    const float4 e = *reinterpret_cast<const float4*>(s_merge + (w * ROWS + row) * Sh::LD + col);
                    f = make_float4(f.x + e.x, f.y + e.y, f.z + e.z, f.w + e.w);
                }
                emit(row, col, f);
            }
            if (tid < ROWS) s_max[tid] = float_order(kNoMax);
        }
        ++n;
        wait(told + 8u * (n & (SEGS - 1)), n / SEGS);
        if (workers_any(WORKERS, !fine)) break;  // also: the merge buffers and q are free again
    }
}

template <int D, int NT, bool F32OUT>
cudaError_t launch_fp4_chunk(const ChunkKernel& k, const DecodeParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_split * p.row_blocks), 1, 1);  // row blocks of one run side by side
    cfg.blockDim = dim3((unsigned)k.threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)k.smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, split_kv_chunk_fp4_kernel<D, NT, F32OUT>, p);
}

template <int D, int NT, bool F32OUT>
inline ChunkKernel make_fp4_chunk_kernel(int index) {
    using Sh = Fp4Shape<D, NT, F32OUT>;
    ChunkKernel k;
    k.fn = reinterpret_cast<const void*>(split_kv_chunk_fp4_kernel<D, NT, F32OUT>);
    k.launch = launch_fp4_chunk<D, NT, F32OUT>;
    k.head_dim = D;
    k.threads = Sh::THREADS;
    k.smem_bytes = Sh::SMEM;
    k.tile_tokens = Sh::TILE;
    k.ctas_per_sm = Sh::MINB;
    k.seg_unit = Sh::TILE;
    k.seg_cost = Sh::SEG_COST;
    k.f32_out = F32OUT;
    k.tensor_core = false;
    k.mma_rows = Sh::ROWS;
    k.index = index;
    return k;
}

// Variants of one head dimension, by column tiles (8 query rows each) of a CTA.
#define KVD_FP4_TABLE(D)                                                                                              \
    const ChunkKernel* fp4_table_d##D(int nt, bool f32) {                                                             \
        static const ChunkKernel table[5][2] = {{make_fp4_chunk_kernel<D, 1, false>(0), make_fp4_chunk_kernel<D, 1, true>(1)}, \
                                                {make_fp4_chunk_kernel<D, 2, false>(2), make_fp4_chunk_kernel<D, 2, true>(3)}, \
                                                {make_fp4_chunk_kernel<D, 3, false>(4), make_fp4_chunk_kernel<D, 3, true>(5)}, \
                                                {make_fp4_chunk_kernel<D, 4, false>(6), make_fp4_chunk_kernel<D, 4, true>(7)}, \
                                                {make_fp4_chunk_kernel<D, 6, false>(8), make_fp4_chunk_kernel<D, 6, true>(9)}}; \
        return &table[nt <= 4 ? nt - 1 : 4][f32 ? 1 : 0];                                                             \
    }

}  // namespace kvd
