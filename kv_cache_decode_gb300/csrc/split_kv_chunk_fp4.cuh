// Split-KV attention over an fp4 cache: the chunk kernel of split_kv_chunk.cuh
// for blocks of 16 tokens held in 4 bits (fp4.cuh).
//
//   s_t = scale * q . k_t,  out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m)   (base 2, log2(e) in the scale)
// with k_t = 2^ek_t * (code * block scale), v_t likewise. A code times its
// scale has at most 6 significant bits and enters the MMAs as f16 exactly; the
// row exponents stay out of them: ek_t multiplies the score, and ev_t is added
// to the exponent of the weight, w_t = 2^(s_t + ev_t - mo) with a running
// maximum mo of its own, so that the f16 weights never leave f16's range
// however the rows' magnitudes differ.
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
// Every warp works alone inside a segment (a pair's tokens in the CTA's run):
// 32-token tiles are dealt round robin to the warps, each warp's lane 0 keeps its own ring
// of tiles filled by bulk copies (a head's blocks are contiguous), and the
// running maxima are only raised, by a vote, when a score passes them by 2^8.
// At a segment's end the warps' states are merged through shared memory.
#pragma once

#include "fp4.cuh"
#include "split_kv_chunk.cuh"
#include "tc_common.cuh"

namespace kvd {

template <int D, int NT>
struct Fp4Shape {
    static constexpr int NW = 8, THREADS = NW * 32;
    static constexpr int ROWS = 8 * NT;          // query rows of a CTA
    static constexpr int TILE = 32;              // tokens of a warp's stage: two blocks
    static constexpr int BLK = Fp4Block<D>::BYTES;
    static constexpr int STAGE = 4 * BLK;        // K blocks, then V blocks
    static constexpr int STAGES = D == 64 ? 3 : 2;
    static constexpr int KS = D / 16;            // k-steps of S^T, and row tiles of O^T
    static constexpr bool QREG = KS * NT * 2 <= 32;  // q fragments in registers, else in shared memory
    static constexpr int LD = D + 4;             // merge buffer row, floats
    static constexpr int RING = NW * STAGES * STAGE;
    static constexpr int MERGE = (NW / 2) * ROWS * LD * 4;
    static constexpr int QBYTES = QREG ? 0 : KS * NT * 32 * 8;
    static constexpr int SMEM = RING + MERGE + QBYTES;
    static constexpr int MINB = D == 256 ? 1 : 2;
    static constexpr int SEG_COST = 4;           // positions (tiles) charged per pair
    static_assert(MINB * (SMEM + 4096) <= 228 * 1024, "CTAs per SM");
};

// Schedule geometry: positions of 32 tokens, a whole segment per step.
template <int X>
struct Fp4Geom {
    KVD_HD constexpr int tt() const { return 1 << 30; }
    KVD_HD constexpr int unit() const { return 32; }
    KVD_HD constexpr int x() const { return X; }
};

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

constexpr float kNoMax = -3e38f;  // running maximum before any score

template <int D, int NT, bool F32OUT>
__global__ void __launch_bounds__(Fp4Shape<D, NT>::THREADS, Fp4Shape<D, NT>::MINB)
    split_kv_chunk_fp4_kernel(const DecodeParams p) {
    using Sh = Fp4Shape<D, NT>;
    using Blk = Fp4Block<D>;
    using Geo = Fp4Geom<Sh::SEG_COST>;
    constexpr int NW = Sh::NW, THREADS = Sh::THREADS, KS = Sh::KS, STAGES = Sh::STAGES, BLK = Sh::BLK, ROWS = Sh::ROWS;
    constexpr int CG = D > 128 ? D / 128 : 1;   // column groups
    constexpr int KW = D >= 128 ? 4 : 2;        // code words of a thread's K columns in one group
    constexpr int VW = D >= 128 ? 2 : 1;        // code words of a thread's V columns in one group
    constexpr long long kBudget = 4000000000LL; // ~2 s: a wait that gives up

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_bar[NW * STAGES];
    __shared__ long long s_red[NW];
    __shared__ int s_redi[NW];
    __shared__ long long s_cum0;
    __shared__ int s_abort;
    __shared__ float s_ml[NW][ROWS], s_l[NW][ROWS];
    __shared__ float s_qs[ROWS];
    float* s_merge = reinterpret_cast<float*>(smem + Sh::RING);
    uint2* s_q = reinterpret_cast<uint2*>(smem + Sh::RING + Sh::MERGE);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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

    if (tid < NW * STAGES) tc::mbar_init(smem_u32(s_bar + tid), 1);
    if (tid == 0) s_abort = 0;
    tc::mbar_fence_init();

    // ---- this CTA's run of the line of (sequence, KV head) pairs ----
    const DevLen len{p.seq_lens, p.len_cap, 1};
    long long mine = 0;
    bool clamped = false;
    for (int b = tid; b < p.B; b += THREADS) {
        const int raw = __ldg(p.seq_lens + b);
        const int L = clamp_len(raw, p.len_cap);
        clamped |= (raw != L);
        mine += pair_extent(L, Geo{});
    }
    if (clamped && blockIdx.x == 0 && p.status) atomicOr(p.status, KVD_STATUS_SEQ_LEN_CLAMPED);
    const long long total = block_sum_ll<NW>(mine, s_red) * p.Hkv;
    const int C_eff = effective_ctas(p.n_split, total);
    if (c >= C_eff) {
        if (p.early) pdl_wait();
        return;
    }
    const long long S = run_begin(c, C_eff, total);
    int b0 = p.B;
    long long cum0 = total;
    {
        long long base = 0;
        for (int chunk = 0; chunk < p.B; chunk += THREADS) {
            const int b = chunk + tid;
            const long long e = pair_extent(b < p.B ? len(b) : 0, Geo{});
            const long long v = e * p.Hkv;
            long long ctot;
            const long long cs = base + block_incl_scan_ll<NW>(v, s_red, &ctot) - v;
            const bool cand = (b < p.B) && is_first_seq_candidate(cs, e, p.Hkv, S);
            const int bmin = block_min_int<NW>(cand ? b : 0x7fffffff, s_redi);
            if (bmin != 0x7fffffff) {
                if (b == bmin) s_cum0 = cs;
                __syncthreads();
                b0 = bmin;
                cum0 = s_cum0;
                break;
            }
            base += ctot;
        }
    }
    Walker<DevLen, Geo> lw(len, Geo{}, p.B, p.Hkv, c, C_eff, total);
    lw.start(b0, cum0);
    Walker<DevLen, Geo> cw = lw;
    if (p.early) pdl_wait();  // the appended rows

    // ---- this warp's ring ----
    // The cache is streamed once per step unless several row blocks read it.
    const uint64_t policy = p.row_blocks > 1 ? tc::l2_evict_last_policy() : l2_evict_first_policy();
    const uint8_t* Kg = static_cast<const uint8_t*>(p.k);
    const uint8_t* Vg = static_cast<const uint8_t*>(p.v);
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * STAGES * Sh::STAGE);
    const uint32_t bars = smem_u32(s_bar + warp * STAGES);
    volatile int* abort_flag = &s_abort;

    Tile lt;                 // segment being loaded
    int lq = 0, li = 0, ln = 0;  // tiles before the segment, this warp's next tile of it, its tiles
    bool lmore = true;
    uint32_t bad = 0;        // bit 2 * stage + j: block j of the stage names no page
    auto block_index = [&](const Tile& t, int tok, bool& ok) -> long long {
        ok = true;
        if (!p.block_table) return ((long long)t.b * p.Hkv + t.h) * (p.S_max >> 4) + (tok >> 4);
        const int page = __ldg(p.block_table + (size_t)t.b * p.max_blocks + (tok >> p.page_shift));
        ok = (unsigned)page < (unsigned)p.num_pages;
        if (!ok && p.status && lane == 0) atomicOr(p.status, KVD_STATUS_BAD_PAGE);
        const int in_page = tok & ((1 << p.page_shift) - 1);
        return (((long long)page * p.Hkv + t.h) << (p.page_shift - 4)) + (in_page >> 4);
    };
    auto issue = [&](int stage) {  // the warp's next tile, if any, into a stage
        while (lmore && li >= ln) {
            lq += ln;
            lmore = lw.next(lt, NoOp{});
            ln = lmore ? (lt.tok_hi - lt.tok_lo + 31) >> 5 : 0;
            li = (warp - lq) & (NW - 1);
        }
        if (!lmore) return;
        const int tok = lt.tok_lo + 32 * li;
        li += NW;
        bool ok0, ok1 = false;
        const long long i0 = block_index(lt, tok, ok0);
        long long i1 = i0 + 1;
        const bool two = tok + 16 < lt.tok_hi;
        // The second block follows the first unless a page of 16 tokens ends between them.
        const bool joined = !p.block_table || p.page_shift > 4;
        if (two && joined) ok1 = ok0;
        if (two && !joined) i1 = block_index(lt, tok + 16, ok1);
        bad = (bad & ~(3u << (2 * stage))) | ((ok0 ? 0u : 1u) << (2 * stage)) | ((!two || ok1 ? 0u : 2u) << (2 * stage));
        if (lane == 0 && !*abort_flag) {
            const uint32_t bar = bars + 8u * stage, dst = ring + stage * Sh::STAGE;
            tc::mbar_arrive_expect_tx(bar, (uint32_t)(2 * BLK * ((ok0 ? 1 : 0) + (two && ok1 ? 1 : 0))));
            if (two && joined && ok0) {
                tc::bulk_load_1d(dst, Kg + (size_t)i0 * BLK, 2 * BLK, bar, policy);
                tc::bulk_load_1d(dst + 2 * BLK, Vg + (size_t)i0 * BLK, 2 * BLK, bar, policy);
            } else {
                if (ok0) {
                    tc::bulk_load_1d(dst, Kg + (size_t)i0 * BLK, BLK, bar, policy);
                    tc::bulk_load_1d(dst + 2 * BLK, Vg + (size_t)i0 * BLK, BLK, bar, policy);
                }
                if (two && ok1) {
                    tc::bulk_load_1d(dst + BLK, Kg + (size_t)i1 * BLK, BLK, bar, policy);
                    tc::bulk_load_1d(dst + 3 * BLK, Vg + (size_t)i1 * BLK, BLK, bar, policy);
                }
            }
        }
    };
    __syncthreads();  // barriers initialised
#pragma unroll
    for (int s = 0; s < STAGES; ++s) issue(s);

    auto write_empty = [&](int b, int h) {
        for (int i = rbase * D + tid; i < rend * D; i += THREADS) {
            const size_t e = out_row(b, h, i / D) * D + (i % D);
            if constexpr (F32OUT)
                reinterpret_cast<float*>(p.out)[e] = 0.f;
            else
                reinterpret_cast<__nv_bfloat16*>(p.out)[e] = __float2bfloat16_rn(0.f);
        }
        if (p.lse)
            for (int i = rbase + tid; i < rend; i += THREADS) p.lse[out_row(b, h, i)] = -CUDART_INF_F;
    };

    uint2 qf[Sh::QREG ? KS * NT : 1];
    float qs[NT][2];     // scale * 2^(q's exponent) of this thread's query columns 8 j + 2 c4 + {0, 1}
    int short_by[NT][2]; // tokens a query row sees fewer than the last token's
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) short_by[j][x] = T - 1 - min(rbase + 8 * j + 2 * c4 + x, TG - 1) / G;

    int stage = 0, cq = 0;
    uint32_t phase = 0;  // bit s: parity to wait for on stage s
    Tile ct;
    while (cw.next(ct, write_empty)) {
        // ---- the pair's queries: f16 relative to each row's largest element ----
        const uint4* qg = reinterpret_cast<const uint4*>(p.q);
        auto load_q = [&](int j, uint2* dst, int stride) {  // dst[k-step * stride]; returns the row's scale
            const int rr = rbase + 8 * j + r;
            uint4 w[CG * KW];
            float m = 0.f;
            const size_t e = (rr < TG ? out_row(ct.b, ct.h, rr) : 0) * (D / 8);
#pragma unroll
            for (int g = 0; g < CG; ++g)
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
            const float dn = __uint_as_float((254u - eb) << 23);
#pragma unroll
            for (int k = 0; k < CG * KW; ++k) {
                const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = pack_f16x2(bf16_lo(x[i]) * dn, bf16_hi(x[i]) * dn);
                dst[(2 * k) * stride] = make_uint2(y[0], y[1]);
                dst[(2 * k + 1) * stride] = make_uint2(y[2], y[3]);
            }
            return p.scale_log2 * __uint_as_float(eb << 23);
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
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                qs[j][0] = s_qs[8 * j + 2 * c4];
                qs[j][1] = s_qs[8 * j + 2 * c4 + 1];
            }
        }

        float o[KS][NT][4];
        float ms[NT][2], mo[NT][2], l[NT][2];
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) ms[j][x] = mo[j][x] = kNoMax, l[j][x] = 0.f;

        const int n_tiles = (ct.tok_hi - ct.tok_lo + 31) >> 5;
        for (int it = (warp - cq) & (NW - 1); it < n_tiles; it += NW) {
            const int tok0 = ct.tok_lo + 32 * it;
            if (!tc::mbar_wait(bars + 8u * stage, (phase >> stage) & 1u, abort_flag, kBudget) && lane == 0 && p.status)
                atomicOr(p.status, KVD_STATUS_TIMEOUT);
            phase ^= 1u << stage;
            const uint32_t kb = ring + stage * Sh::STAGE, vb = kb + 2 * BLK;
            const uint32_t badm = (bad >> (2 * stage)) & 3u;
            const bool two = tok0 + 16 < ct.tok_hi;
            // Tokens some query row does not see, or that name no page.
            const bool edge = (tok0 + 32 > ct.L - T + 1) || badm;
            const int ta = r ^ ((r >> 1) & 1);  // token of MMA row r (row r + 8: 8 more)

            // ---- S^T = K q^T ----
            float s[2][NT][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < NT; ++j) s[x][j][0] = s[x][j][1] = s[x][j][2] = s[x][j][3] = 0.f;
#pragma unroll
            for (int g = 0; g < CG; ++g) {
                uint32_t w[2][2][KW];     // [block][row half][word]
                uint32_t sc[2][2][2];     // [block][row half][scale of word / 2], twice in one register
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a = kb + x * BLK + (uint32_t)(g * 16 * Blk::ROW + (ta + 8 * y) * Blk::ROW);
                        if constexpr (D >= 128) {
                            const uint4 v = lds128(a + c4 * 16);
                            w[x][y][0] = v.x, w[x][y][1] = v.y, w[x][y][2] = v.z, w[x][y][3] = v.w;
                            const uint32_t h = e4m3x2_to_f16x2(
                                lds16(kb + x * BLK + (uint32_t)(Blk::SCALES + (ta + 8 * y) * (D / 16) + 8 * g + 2 * c4)));
                            sc[x][y][0] = __byte_perm(h, 0, 0x1010);
                            sc[x][y][1] = __byte_perm(h, 0, 0x3232);
                        } else {
                            const uint2 v = lds64(a + c4 * 8);
                            w[x][y][0] = v.x, w[x][y][1] = v.y;
                            sc[x][y][0] = e4m3x2_to_f16x2(
                                lds8(kb + x * BLK + (uint32_t)(Blk::SCALES + (ta + 8 * y) * (D / 16) + c4)) * 0x101u);
                            sc[x][y][1] = sc[x][y][0];
                        }
                    }
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    uint2 qa[NT], qb[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int ks = 2 * (g * KW + k);
                        if constexpr (Sh::QREG) {
                            qa[j] = qf[ks * NT + j], qb[j] = qf[(ks + 1) * NT + j];
                        } else {
                            qa[j] = s_q[(ks * NT + j) * 32 + lane], qb[j] = s_q[((ks + 1) * NT + j) * 32 + lane];
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t h0[4], h1[4];
                        e2m1x8_to_f16(w[x][0][k], h0);
                        e2m1x8_to_f16(w[x][1][k], h1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h0[i] = hmul2(h0[i], sc[x][0][k / 2]);
                            h1[i] = hmul2(h1[i], sc[x][1][k / 2]);
                        }
                        const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            mma_f16_16816(s[x][j], a0, qa[j].x, qa[j].y);
                            mma_f16_16816(s[x][j], a1, qb[j].x, qb[j].y);
                        }
                    }
                }
            }

            // ---- row exponents, masks, running maxima ----
            float ev[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t at = (uint32_t)(Blk::EXPS + ta + 8 * y);
                    const float kf = fp4_row_scale(lds8(kb + x * BLK + at));
                    ev[x][y] = (float)(int)lds8(vb + x * BLK + at) - 127.f;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        s[x][j][2 * y] *= kf * qs[j][0];
                        s[x][j][2 * y + 1] *= kf * qs[j][1];
                    }
                    if (edge) {
                        const int tok = tok0 + 16 * x + ta + 8 * y;
                        const bool none = (badm >> x) & 1u;
                        if (none) ev[x][y] = 0.f;
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                float& v = s[x][j][2 * y + z];
                                if (none) v = 0.f;
                                if (tok >= ct.L - short_by[j][z]) v = -CUDART_INF_F;
                            }
                        if (tok >= ct.L) ev[x][y] = 0.f;
                    }
                }
            bool raise = false;
            float hs[NT][2], ho[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    hs[j][z] = fmaxf(fmaxf(s[0][j][z], s[0][j][2 + z]), fmaxf(s[1][j][z], s[1][j][2 + z]));
                    ho[j][z] = fmaxf(fmaxf(s[0][j][z] + ev[0][0], s[0][j][2 + z] + ev[0][1]),
                                     fmaxf(s[1][j][z] + ev[1][0], s[1][j][2 + z] + ev[1][1]));
                    raise |= hs[j][z] > ms[j][z] + 8.f || ho[j][z] > mo[j][z] + 8.f;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) {
                            hs[j][z] = fmaxf(hs[j][z], __shfl_xor_sync(0xffffffffu, hs[j][z], off));
                            ho[j][z] = fmaxf(ho[j][z], __shfl_xor_sync(0xffffffffu, ho[j][z], off));
                        }
                        const float ns = fmaxf(ms[j][z], hs[j][z]), no = fmaxf(mo[j][z], ho[j][z]);
                        l[j][z] *= tc::ex2_approx(ms[j][z] - ns);
                        const float f = tc::ex2_approx(mo[j][z] - no);
                        ms[j][z] = ns;
                        mo[j][z] = no;
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            o[i][j][z] *= f;
                            o[i][j][2 + z] *= f;
                        }
                    }
            }

            // ---- weights, O^T += V^T w ----
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (x == 1 && !two) break;
                uint32_t bh[NT][2], bl[F32OUT ? NT : 1][2];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float wv[2];
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const float v = s[x][j][2 * y + z];
                            l[j][z] += tc::ex2_approx(v - ms[j][z]);
                            wv[z] = tc::ex2_approx(v + ev[x][y] - mo[j][z]);
                        }
                        const uint32_t hi = pack_f16x2(wv[0], wv[1]);
                        bh[j][y] = movmatrix_trans(hi);
                        if constexpr (F32OUT) bl[j][y] = movmatrix_trans(pack_f16x2(wv[0] - f16_lo(hi), wv[1] - f16_hi(hi)));
                    }
                const uint32_t base = vb + x * BLK;
                const int t0 = (2 * c4) ^ (c4 & 1), t1 = t0 ^ 1;  // tokens of k = 2 c4, 2 c4 + 1 (and 8 more)
#pragma unroll
                for (int g = 0; g < CG; ++g) {
                    uint32_t w[4][VW], sc[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a = base + (uint32_t)(g * 16 * Blk::ROW + 8 * y * Blk::ROW);
                        if constexpr (D >= 128) {
                            const uint2 u0 = lds64(a + t0 * Blk::ROW + r * 8), u1 = lds64(a + t1 * Blk::ROW + r * 8);
                            w[2 * y][0] = u0.x, w[2 * y][1] = u0.y, w[2 * y + 1][0] = u1.x, w[2 * y + 1][1] = u1.y;
                        } else {
                            w[2 * y][0] = lds32(a + t0 * Blk::ROW + r * 4);
                            w[2 * y + 1][0] = lds32(a + t1 * Blk::ROW + r * 4);
                        }
                        const uint32_t sb = base + (uint32_t)(Blk::SCALES + 8 * y * (D / 16) + (D >= 128 ? 8 * g + r : r / 2));
                        uint32_t s0 = lds8(sb + t0 * (D / 16)), s1 = lds8(sb + t1 * (D / 16));
                        if (edge) {  // rows past the sequence or without a page hold anything: their scale is zero
                            const int tok = tok0 + 16 * x + 8 * y;
                            const bool none = (badm >> x) & 1u;
                            if (none || tok + t0 >= ct.L) s0 = 0;
                            if (none || tok + t1 >= ct.L) s1 = 0;
                        }
                        sc[y] = e4m3x2_to_f16x2(s0 | (s1 << 8));
                    }
#pragma unroll
                    for (int v = 0; v < VW; ++v) {
                        uint32_t ev0[4], od0[4], ev1[4], od1[4];  // even and odd columns, token pairs 0 and 8 further
                        e2m1x8_to_f16((w[0][v] & 0x0f0f0f0fu) | ((w[1][v] << 4) & 0xf0f0f0f0u), ev0);
                        e2m1x8_to_f16(((w[0][v] >> 4) & 0x0f0f0f0fu) | (w[1][v] & 0xf0f0f0f0u), od0);
                        e2m1x8_to_f16((w[2][v] & 0x0f0f0f0fu) | ((w[3][v] << 4) & 0xf0f0f0f0u), ev1);
                        e2m1x8_to_f16(((w[2][v] >> 4) & 0x0f0f0f0fu) | (w[3][v] & 0xf0f0f0f0u), od1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a[4] = {hmul2(ev0[i], sc[0]), hmul2(od0[i], sc[0]), hmul2(ev1[i], sc[1]),
                                                   hmul2(od1[i], sc[1])};
                            const int m = (g * VW + v) * 4 + i;
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                mma_f16_16816(o[m][j], a, bh[j][0], bh[j][1]);
                                if constexpr (F32OUT) mma_f16_16816(o[m][j], a, bl[j][0], bl[j][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage
            issue(stage);
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }
        cq += n_tiles;

        // ---- merge the warps' states ----
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[j][z] += __shfl_xor_sync(0xffffffffu, l[j][z], off);
                if (r == 0) {
                    s_ml[warp][8 * j + 2 * c4 + z] = ms[j][z];
                    s_l[warp][8 * j + 2 * c4 + z] = l[j][z];
                }
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                float M = kNoMax;
#pragma unroll
                for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w][8 * j + 2 * c4 + z]);
                const float f = mo[j][z] > kNoMax ? tc::ex2_approx(mo[j][z] - M) : 0.f;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    o[i][j][z] *= f;
                    o[i][j][2 + z] *= f;
                }
            }
        // Column of o[(g * VW + v) * 4 + i][j][0 / 2]: 128 g + 8 (VW r + v) + 2 i, + 1 for rows r + 8.
        auto slot_of = [&](int g, int v, int j, int z) {
            return s_merge + ((warp & (NW / 2 - 1)) * ROWS + 8 * j + 2 * c4 + z) * Sh::LD + 128 * g + 8 * (VW * r + v);
        };
        auto exchange = [&](bool add) {
#pragma unroll
            for (int g = 0; g < CG; ++g)
#pragma unroll
                for (int v = 0; v < VW; ++v)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            float4* d = reinterpret_cast<float4*>(slot_of(g, v, j, z));
                            const int m = (g * VW + v) * 4;
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                float4 f = make_float4(o[m + 2 * x][j][z], o[m + 2 * x][j][2 + z], o[m + 2 * x + 1][j][z],
                                                       o[m + 2 * x + 1][j][2 + z]);
                                if (add) {
                                    const float4 e = d[x];
                                    f = make_float4(f.x + e.x, f.y + e.y, f.z + e.z, f.w + e.w);
                                }
                                d[x] = f;
                            }
                        }
        };
        if (warp >= NW / 2) exchange(false);
        __syncthreads();
        if (warp < NW / 2) exchange(true);
        __syncthreads();
        const int pair = ct.b * p.Hkv + ct.h;
        for (int i = tid; i < (rend - rbase) * (D / 4); i += THREADS) {
            const int row = i / (D / 4), col = (i - row * (D / 4)) * 4;
            float M = kNoMax, L = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w][row]);
#pragma unroll
            for (int w = 0; w < NW; ++w) L += s_l[w][row] * tc::ex2_approx(s_ml[w][row] - M);
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW / 2; ++w) {
                const float4 e = *reinterpret_cast<const float4*>(s_merge + (w * ROWS + row) * Sh::LD + col);
                f = make_float4(f.x + e.x, f.y + e.y, f.z + e.z, f.w + e.w);
            }
            if (ct.full) {
                const float inv = L > 0.f ? 1.f / L : 0.f;
                const size_t orow = out_row(ct.b, ct.h, rbase + row);
                if constexpr (F32OUT)
                    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + orow * D + col) =
                        make_float4(f.x * inv, f.y * inv, f.z * inv, f.w * inv);
                else
                    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * D + col) =
                        make_uint2(pack_bf16x2(f.x * inv, f.y * inv), pack_bf16x2(f.z * inv, f.w * inv));
                if (p.lse && col == 0) p.lse[orow] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -CUDART_INF_F;
            } else {
                const size_t slot = ((size_t)c + pair) * TG + rbase + row;
                *reinterpret_cast<float4*>(p.ws_o + slot * D + col) = f;
                if (col == 0) p.ws_ml[slot] = make_float2(M, L);
            }
        }
        __syncthreads();  // the merge buffers and q are free again
    }
    cw.finish(write_empty);
    if (s_abort) {  // bounded wait for copies in flight before the shared memory is given up
        int go = 0;
        for (int s = 0; s < STAGES; ++s) tc::mbar_wait(bars + 8u * s, (phase >> s) & 1u, &go, kBudget / 8);
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
    using Sh = Fp4Shape<D, NT>;
    ChunkKernel k;
    k.fn = reinterpret_cast<const void*>(split_kv_chunk_fp4_kernel<D, NT, F32OUT>);
    k.launch = launch_fp4_chunk<D, NT, F32OUT>;
    k.head_dim = D;
    k.threads = Sh::THREADS;
    k.smem_bytes = Sh::SMEM;
    k.tile_tokens = Sh::TILE;
    k.ctas_per_sm = Sh::MINB;
    k.seg_unit = 32;
    k.seg_cost = Sh::SEG_COST;
    k.f32_out = F32OUT;
    k.tensor_core = false;
    k.mma_rows = Sh::ROWS;
    k.index = index;
    return k;
}

#define KVD_FP4_TABLE(D)                                                                                    \
    const ChunkKernel* fp4_table_d##D(int nt, bool f32) {                                                   \
        static const ChunkKernel table[2][2] = {                                                            \
            {make_fp4_chunk_kernel<D, 1, false>(0), make_fp4_chunk_kernel<D, 1, true>(1)},                  \
            {make_fp4_chunk_kernel<D, 2, false>(2), make_fp4_chunk_kernel<D, 2, true>(3)}};                 \
        return &table[nt - 1][f32 ? 1 : 0];                                                                 \
    }

}  // namespace kvd
