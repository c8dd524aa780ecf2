// Attention over listed blocks of tokens: for every (sequence, query token, KV
// head), the softmax over the tokens of the blocks that its list names,
//   s_t = scale * q . k_t,  out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m)   (base 2, log2(e) in the scale).
// It reads K * block rows of K and V a pair where the attention over all tokens reads the sequence; bound by
// memory for batches (64 sequences, 32 heads on 8 of 128, 4,096 tokens each: 159 us for 1.07 GB, the copy
// rate), by latency for one sequence (2,048 tokens: 6.6 to 7 us). Wide groups: 64 sequences, 48 heads on one,
// 4,096 tokens take 72 us at head_dim 256 (3.8 TB/s; 32 heads 50.8), 39 at 128 and 28.6 at 64. Their 3 to 8 warps
// a team each read every K and V row: at 256 the shared-memory pipe is at 61 % of its peak over the whole time
// and 78 % where an SM works, tensor cores 29 %; at 128 and 64 it is at 32 and 24 %, and a warp mostly waits for
// its own last result (2 of 6 to 7 cycles an instruction) and its stages: latency of few warps.
//
// A stage is 32 tokens, K rows and V rows, brought by TMA into a ring (128-byte swizzle): as one box where
// blocks and pages have 32 tokens, else two units of 16 of any listed blocks. A loading warp looks the list up,
// 32 units at a time, and deals the stages to the CTA's teams in turn; a team works on its stages alone, so
// that nothing but its own loads holds it up. (Loads issued by the working warps themselves took 950 of a
// 16-token step's 2,200 cycles.) The products are turned round so that tokens fill the 16 rows of m16n8k16 MMAs
// and query rows their 8 columns (a group of 4 to 8 query heads is one column tile): S^T = K q^T, O^T = V^T w,
// the weights transposed by movmatrix. The running maximum of a column is raised only where a score passes it
// by 2^8 (a vote a stage otherwise): weights stay below 2^8 and keep their relative precision, bf16's 2^-8, the
// same rounding as the other attention kernels' of this library; for float32 output a second bf16 carries the
// rest to 2^-16. Teams are single warps for groups of up to 16 query heads (head_dim 256: 8); wider ones are
// shared out to the head_warps warps of a team.
//
// A pair's CTAs (parts, up to 16) are a cluster: their states are joined over distributed shared memory, each
// CTA writing a share of the output, without a second launch or a workspace. Where even 16 CTAs a pair leave
// SMs idle, `shards` such clusters a pair write normalised float32 results, which the shard merge of
// split_kv_merge.cu joins.
#pragma once

#include <cuda.h>
#include <float.h>
#include <math_constants.h>

#include <atomic>

#include "../../include/kvdecode.h"
#include "api_common.h"
#include "blocks.h"
#include "cluster.cuh"
#include "common.cuh"
#include "tc_common.cuh"

namespace kvd {

bool tc_encode_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box, bool u8);

struct BlocksMaps {
    CUtensorMap k;  // 3D: [rows of the cache, Hkv, D], box 32 or 16 x 1 x 64, 128-byte swizzle
    CUtensorMap v;
};

template <int D, int NT>
struct BlocksShape {
    static constexpr int ROWS_S = kBlocksStage;
    static constexpr int RW = 8 * NT;                    // query rows of a warp
    static constexpr int WARPS = blocks_warps(D);        // working warps of a CTA, at most
    static constexpr int CTAS = D == 256 ? 1 : 2;        // of an SM
    static constexpr int ELEM = ROWS_S * D * 2;          // a stage's rows of one tensor
    static constexpr int RING = (D == 256 ? 192 : 96) * 1024;  // shared out to the teams
    static constexpr int SLOTS = blocks_slots(D);
    static constexpr int ROWS = WARPS * RW;              // state rows of a CTA
    static constexpr int ST = D + 4;                     // floats between state rows: neighbours in different banks
    static constexpr int OFF_BAR = RING;                 // full and empty barriers
    static constexpr int OFF_N = OFF_BAR + 2 * SLOTS * 8;    // tokens of each stage
    static constexpr int OFF_ML = OFF_N + SLOTS * 8;         // m and the two sums of the states
    static constexpr int OFF_CML = OFF_ML + 3 * ROWS * 4;    // of the CTA's rows
    static constexpr int OFF_W = OFF_CML + 3 * 64 * 4;       // weights of the cluster's CTAs, and 1 / sum
    static constexpr int OFF_FLAG = OFF_W + 17 * 64 * 4;
    static constexpr int OFF_IN = OFF_FLAG + 16;             // what the cluster's CTAs send this one
    static constexpr int IN_FLOATS = 2048;
    static constexpr int SMEM = OFF_IN + IN_FLOATS * 4;
    static_assert(SLOTS * 2 * ELEM == RING, "stages fill the ring");
    static_assert(ROWS * ST * 4 <= RING, "the states take the ring's place");
    static_assert(CTAS * (SMEM + 1024) <= 227 * 1024, "shared memory of an SM");
};

// How often slot s (stage s % R of team s / R) is filled by `issued` stages, dealt to the teams' rings of R in turn.
__host__ __device__ constexpr int blocks_slot_uses(int issued, int s, int teams, int R) {
    return issued > s % R * teams + s / R ? (issued - (s % R * teams + s / R) - 1) / (teams * R) + 1 : 0;
}
// ... as counting them one by one gives it.
constexpr bool blocks_slot_uses_hold(int teams, int R) {
    int uses[64] = {};
    for (int issued = 0; issued < 5 * teams * R; ++issued) {
        for (int s = 0; s < teams * R; ++s)
            if (uses[s] != blocks_slot_uses(issued, s, teams, R)) return false;
        ++uses[issued % teams * R + issued / teams % R];
    }
    return true;
}
static_assert(blocks_slot_uses_hold(1, 12) && blocks_slot_uses_hold(4, 3) && blocks_slot_uses_hold(2, 5) &&
                  blocks_slot_uses_hold(3, 4),
              "the last phase of each slot");

// The bf16 MMA of common.cuh without its ordering against other instructions.
__device__ __forceinline__ void mma_bf16_free(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int NT, bool F32OUT>
__global__ void __launch_bounds__((BlocksShape<D, NT>::WARPS + 1) * 32, BlocksShape<D, NT>::CTAS)
    decode_blocks_kernel(const BlocksParams p, const __grid_constant__ BlocksMaps maps) {
    using Sh = BlocksShape<D, NT>;
    constexpr int RW = Sh::RW, KS = D / 16, MT = D / 16, ST = Sh::ST, U = kBlocksStage / 16;  // U: halves of 16 tokens of a stage
    constexpr long long kBudget = 4000000000LL;  // ~2 s of clock cycles a wait

    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t ring = smem_u32(smem), bars = ring + Sh::OFF_BAR;
    float* states = reinterpret_cast<float*>(smem);
    float* s_m = reinterpret_cast<float*>(smem + Sh::OFF_ML);
    float* s_l = s_m + Sh::ROWS;
    float* s_lr = s_l + Sh::ROWS;
    float* s_cm = reinterpret_cast<float*>(smem + Sh::OFF_CML);
    float* s_cl = s_cm + 64;
    float* s_clr = s_cl + 64;
    float* s_w = reinterpret_cast<float*>(smem + Sh::OFF_W);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Sh::OFF_FLAG);
    float* s_in = reinterpret_cast<float*>(smem + Sh::OFF_IN);
    volatile int* s_n = reinterpret_cast<volatile int*>(smem + Sh::OFF_N);  // tokens of a stage's halves (the second << 8); 0: the end

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthreads = blockDim.x;
    const int HT = p.head_warps, teams = p.teams, workers = teams * HT, team = warp / HT, wt = warp - team * HT;
    const bool loader = warp == workers;
    const int rank = blockIdx.x & (p.parts - 1), cl = blockIdx.x >> (__ffs(p.parts) - 1);  // (parts: a power of two)
    const int pair = cl % p.pairs, shard = cl / p.pairs;
    const int h = pair % p.Hkv, bt = pair / p.Hkv, t = bt % p.T, b = bt / p.T;
    const int R = Sh::SLOTS / teams;  // stages of a team's ring
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (Sh::SLOTS + s); };

    // ---- set-up that reads no input ----
    if (tid == 0) {
        for (int s = 0; s < Sh::SLOTS; ++s) {
            tc::mbar_init(bars + 8u * s, 1);
            tc::mbar_init(bars + 8u * (Sh::SLOTS + s), HT);
        }
        *abort_flag = 0;
        tc::mbar_fence_init();
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
    }
    // States of few rows are sent to the CTA that joins them, which has to have started by then.
    const bool send = p.parts > 1 && p.G <= 16 && p.G * D <= Sh::IN_FLOATS;
    if (send) cluster_arrive_relaxed();
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    float o[MT][NT][4], m[NT][2], l[NT][2], lr[F32OUT ? 1 : NT][2];
    bool dead = false;
    int issued = 0;  // stages the loading warp has issued
    if (loader) {
        // ---- the tokens this query token sees, and the units of this CTA ----
        const int us = p.unit_log2;
        const bool T16 = us == 4;  // a stage takes two units
        const int raw = __ldg(p.seq_lens + b), L = raw < 0 ? 0 : raw > p.S_max ? p.S_max : raw;
        const int32_t* list = p.blocks + (size_t)pair * p.K;
        const int units = p.K << (p.block_log2 - us), submask = (1 << (p.block_log2 - us)) - 1;
        const int W = p.shards * p.parts, last_block = (p.S_max - 1) >> p.block_log2;  // of the cache's
        const uint64_t policy = l2_evict_first_policy();
        if (raw != L && lane == 0 && p.status) atomicOr(p.status, KVD_STATUS_SEQ_LEN_CLAMPED);
        const int seen = L - p.T + 1 + t;  // <= 0: none
        int to_team = 0, slot = 0, phase = 1;  // phase: parity of the last release of the slots in turn
        auto next_stage = [&]() {  // the next stage's slot, or -1
            const int s = to_team * R + slot;
            if (issued >= teams * R && !__all_sync(0xffffffffu, tc::mbar_wait(empty(s), phase, abort_flag, kBudget))) return -1;
            ++issued;
            if (++to_team == teams) {
                to_team = 0;
                if (++slot == R) slot = 0, phase ^= 1;
            }
            return s;
        };
        auto issue = [&](int row0, int n0, int row1, int n1) {
            const int s = next_stage();
            if (s < 0) {
                dead = true;
                return;
            }
            if (lane == 0) {
                const uint32_t dst = ring + (uint32_t)s * 2 * Sh::ELEM, bar = full(s);
                s_n[s] = n0 | (n1 << 8);
                tc::mbar_arrive_expect_tx(bar, T16 && n1 == 0 ? Sh::ELEM : 2 * Sh::ELEM);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    tc::tma_load_3d(dst + c * (Sh::ROWS_S * 128), &maps.k, c * 64, h, row0, bar, policy);
                    tc::tma_load_3d(dst + Sh::ELEM + c * (Sh::ROWS_S * 128), &maps.v, c * 64, h, row0, bar, policy);
                }
                if (T16 && n1 > 0) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        tc::tma_load_3d(dst + c * (Sh::ROWS_S * 128) + 2048, &maps.k, c * 64, h, row1, bar, policy);
                        tc::tma_load_3d(dst + Sh::ELEM + c * (Sh::ROWS_S * 128) + 2048, &maps.v, c * 64, h, row1, bar, policy);
                    }
                }
            }
        };
        // Units are looked up 32 at a time, one a lane: how many of its tokens count, and its cache row. Those
        // of entries that name no block the token sees have none and are passed over.
        int row0 = 0, n0 = 0;  // a unit that waits for a second one
        for (long long u0 = shard * p.parts + rank; u0 < units && !dead; u0 += 32LL * W) {
            const long long u = u0 + (long long)lane * W;
            const int blk = u < units ? __ldg(list + ((int)u >> (p.block_log2 - us))) : -1;
            const bool named = blk >= 0 && blk <= last_block;
            const int tok = named ? (blk << p.block_log2) + (((int)u & submask) << us) : 0;
            const bool held = named && tok < p.S_max;
            int row = 0;
            bool bad = false;
            if (held) {
                if (p.pg.block_table) {
                    const int page = __ldg(p.pg.block_table + (size_t)b * p.pg.max_blocks + (tok >> p.pg.page_shift));
                    bad = (unsigned)page >= (unsigned)p.pg.num_pages;  // reads as zero rows: past the pool's end
                    row = bad ? p.pg.num_pages << p.pg.page_shift
                              : (page << p.pg.page_shift) + (tok & ((1 << p.pg.page_shift) - 1));
                } else {
                    row = b * p.S_max + tok;
                }
            }
            const int n = held ? min(1 << us, seen - tok) : 0;
            if (bad && n > 0 && p.status) atomicOr(p.status, KVD_STATUS_BAD_PAGE);
            for (uint32_t mask = __ballot_sync(0xffffffffu, n > 0); mask && !dead; mask &= mask - 1) {
                const int src = __ffs(mask) - 1, ru = __shfl_sync(0xffffffffu, row, src), nu = __shfl_sync(0xffffffffu, n, src);
                if (!T16) {
                    issue(ru, min(nu, 16), 0, max(nu - 16, 0));
                } else if (n0 == 0) {
                    row0 = ru, n0 = nu;
                } else {
                    issue(row0, n0, ru, nu);
                    n0 = 0;
                }
            }
        }
        if (n0 > 0 && !dead) issue(row0, n0, 0, 0);
        for (int j = 0; j < teams && !dead; ++j) {  // the end, for every team
            const int s = next_stage();
            if (s < 0) {
                dead = true;
            } else if (lane == 0) {
                s_n[s] = 0;
                tc::mbar_arrive(full(s));
            }
        }
    } else {
        // ---- q: column tile n's rows wt * RW + 8 n + lane / 4 as B fragments ----
        uint32_t qf[NT][KS][2];
        {
            const uint32_t* q32 = reinterpret_cast<const uint32_t*>(p.q);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = wt * RW + 8 * n + (lane >> 2);
                const uint32_t* qr = q32 + ((size_t)pair * p.G + r) * (D / 2) + (lane & 3);
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    qf[n][kk][0] = r < p.G ? __ldg(qr + kk * 8) : 0u;
                    qf[n][kk][1] = r < p.G ? __ldg(qr + kk * 8 + 4) : 0u;
                }
            }
        }
        // l: the weights' sum, for lse. lr: of the weights as V meets them, so that the output is a convex
        // combination of V rows (the same where float32 output carries both parts).
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -FLT_MAX;
            l[n][0] = l[n][1] = 0.f;
            if constexpr (!F32OUT) lr[n][0] = lr[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
        }
        auto chunk = [&](uint32_t base, int row, int c) {  // 16-byte chunk c of a swizzled row
            return base + (uint32_t)((c >> 3) * (Sh::ROWS_S * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        };
        int slot = 0, phase = 0;
        while (true) {
            const int st = team * R + slot;
            if (!__all_sync(0xffffffffu, tc::mbar_wait(full(st), phase, abort_flag, kBudget))) {
                dead = true;
                break;
            }
            __syncwarp();  // (lanes leave the wait one by one; what follows is .aligned and wants them together)
            const int counts = s_n[st];
            if (counts == 0) break;
            const int n_tok[2] = {counts & 0xff, counts >> 8};
            const uint32_t kb = ring + (uint32_t)st * 2 * Sh::ELEM, vb = kb + Sh::ELEM;
            // ---- scores: tokens 16 u + lane / 4 (s[u][n][0..1]) and + 8 (s[u][n][2..3]), query rows 8 n + 2 (lane % 4) + 0..1 ----
            float s[U][NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t a[4];
                    ldmatrix_x4(chunk(kb, 16 * u + (lane & 15), 2 * kk + (lane >> 4)), a[0], a[1], a[2], a[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_bf16_free(s[u][n], a, qf[n][kk][0], qf[n][kk][1]);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][n][e] *= p.scale_log2;
            bool raise = false;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (n_tok[u] < 16) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if ((lane >> 2) >= n_tok[u]) s[u][n][0] = s[u][n][1] = -CUDART_INF_F;
                        if ((lane >> 2) + 8 >= n_tok[u]) s[u][n][2] = s[u][n][3] = -CUDART_INF_F;
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    raise |= fmaxf(s[u][n][0], s[u][n][2]) > m[n][0] + 8.f;
                    raise |= fmaxf(s[u][n][1], s[u][n][3]) > m[n][1] + 8.f;
                }
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(fmaxf(s[0][n][e], s[0][n][e + 2]), fmaxf(s[1][n][e], s[1][n][e + 2]));
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                        const float up = fmaxf(m[n][e], x), f = exp2f(m[n][e] - up);
                        m[n][e] = up;
                        l[n][e] *= f;
                        if constexpr (!F32OUT) lr[n][e] *= f;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[i][n][e] *= f;
                            o[i][n][e + 2] *= f;
                        }
                    }
            }
            // ---- the weights as B fragments ----
            uint32_t ph[U][NT][2], pl[F32OUT ? U : 1][F32OUT ? NT : 1][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float e0 = tc::ex2_approx(s[u][n][2 * y] - m[n][0]), e1 = tc::ex2_approx(s[u][n][2 * y + 1] - m[n][1]);
                        const uint32_t hi = pack_bf16x2(e0, e1);
                        ph[u][n][y] = movmatrix_trans(hi);
                        l[n][0] += e0;
                        l[n][1] += e1;
                        if constexpr (F32OUT) {
                            pl[u][n][y] = movmatrix_trans(pack_bf16x2(e0 - bf16_lo(hi), e1 - bf16_hi(hi)));
                        } else {
                            lr[n][0] += bf16_lo(hi);
                            lr[n][1] += bf16_hi(hi);
                        }
                    }
            // ---- V rows past the last token hold anything: zero, since 0 * NaN is not 0 ----
            const bool part = n_tok[0] < 16 || n_tok[1] < 16;
            if (part) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    for (int i = lane + n_tok[u] * 8; i < 16 * 8; i += 32)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            *reinterpret_cast<uint4*>(smem + (vb - ring) + c * (Sh::ROWS_S * 128) + u * 2048 + i * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t a[4];
                    ldmatrix_x4_trans(chunk(vb, 16 * u + (lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)), a[0], a[1],
                                      a[2], a[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_bf16_free(o[i][n], a, ph[u][n][0], ph[u][n][1]);
                        if constexpr (F32OUT) mma_bf16_free(o[i][n], a, pl[u][n][0], pl[u][n][1]);
                    }
                }
            if (part) tc::fence_proxy_async_smem();  // the zeros come before the next load
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty(st));
            if (++slot == R) slot = 0, phase ^= 1;
        }
    }
    if (dead && lane == 0 && p.status) atomicOr(p.status, KVD_STATUS_TIMEOUT);

    // ---- where a wait of any warp gave up, copies may still be on their way: they are waited for (again with a ----
    // ---- limit), since the ring's place is used below and the CTA must not leave before them ----
    __syncthreads();
    if (*abort_flag) {  // (set before the barrier: every thread reads the same)
        if (loader)
            for (int s = 0; s < teams * R; ++s) {
                const int uses = blocks_slot_uses(issued, s, teams, R);
                if (uses > 0)
                    for (long long t0 = clock64(); !tc::mbar_test(full(s), (uses - 1) & 1) && clock64() - t0 < kBudget;) {
                    }
            }
        __syncthreads();
    }

    // ---- the states to shared memory, in the ring's place ----
    if (!loader) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
            if constexpr (!F32OUT) {
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) lr[n][e] += __shfl_xor_sync(0xffffffffu, lr[n][e], off);
            }
            const int r = warp * RW + 8 * n + 2 * (lane & 3) + e;
            if ((lane >> 2) == 0) {
                s_m[r] = m[n][e];
                s_l[r] = l[n][e];
                if constexpr (F32OUT)
                    s_lr[r] = l[n][e];
                else
                    s_lr[r] = lr[n][e];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                states[r * ST + 16 * i + (lane >> 2)] = o[i][n][e];
                states[r * ST + 16 * i + (lane >> 2) + 8] = o[i][n][e + 2];
            }
        }
    }
    __syncthreads();

    // ---- joined over the CTA's teams, then over the cluster ----
    // A state with no token has m = -FLT_MAX and sums of 0: its weight times anything is 0.
    const size_t out_base = (size_t)shard * p.pairs * p.G + (size_t)pair * p.G;  // row of out and lse
    auto put = [&](int r, int c, float inv, const float4& v) {
        const size_t e = (out_base + r) * D + 4 * c;
        if constexpr (F32OUT)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + e) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        else
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + e) =
                make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    };
    auto put_lse = [&](int r, float M, float sum) {
        if (p.lse) p.lse[out_base + r] = sum == 0.f ? -CUDART_INF_F : (M + log2f(sum)) * 0.69314718055994531f;
    };
    auto inverse = [](float sum) { return sum == 0.f ? 0.f : 1.f / sum; };
    const bool alone = p.parts == 1;
    const int vecs = p.G * (D / 4);             // float4 of the pair's output
    const int share = (vecs + p.parts - 1) / p.parts;  // of one CTA, where states are sent
    if (send) cluster_wait();  // the others have started
    for (int i = tid; i < vecs; i += nthreads) {
        const int r = i / (D / 4), c = i - r * (D / 4), step = HT * RW;  // team j's state of row r: r + j * step
        float M = -FLT_MAX, sum = 0.f, sumr = 0.f;
        for (int j = 0; j < teams; ++j) M = fmaxf(M, s_m[r + j * step]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < teams; ++j) {
            const float f = exp2f(s_m[r + j * step] - M);
            const float4 x = *reinterpret_cast<const float4*>(states + (r + j * step) * ST + 4 * c);
            sum += f * s_l[r + j * step];
            sumr += f * s_lr[r + j * step];
            v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
        }
        if (alone) {
            put(r, c, inverse(sumr), v);
            if (c == 0) put_lse(r, M, sum);
        } else if (send) {
            const int to = i / share;
            st_cluster4(map_to_rank(smem_u32(s_in + 4 * (rank * share + i - to * share)), to), v);
            if (c < p.parts) {  // (D / 4 >= 16 threads of a row, one a CTA)
                const uint32_t ml = map_to_rank(smem_u32(s_w + (rank * 16 + r) * 3), c);
                st_cluster(ml, M);
                st_cluster(ml + 4, sum);
                st_cluster(ml + 8, sumr);
            }
        } else {
            *reinterpret_cast<float4*>(states + r * ST + 4 * c) = v;  // only this thread reads it
            if (c == 0) s_cm[r] = M, s_cl[r] = sum, s_clr[r] = sumr;
        }
    }
    if (alone) return;
    cluster_sync();
    if (send) {  // all that came is here, and nothing more is read elsewhere
        for (int i = tid; i < share && rank * share + i < vecs; i += nthreads) {
            const int r = (rank * share + i) / (D / 4), c = rank * share + i - r * (D / 4);
            float M = -FLT_MAX, sum = 0.f, sumr = 0.f;
            for (int j = 0; j < p.parts; ++j) M = fmaxf(M, s_w[(j * 16 + r) * 3]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j = 0; j < p.parts; ++j) {
                const float* ml = s_w + (j * 16 + r) * 3;
                const float f = exp2f(ml[0] - M);
                const float4 x = *reinterpret_cast<const float4*>(s_in + 4 * (j * share + i));
                sum += f * ml[1];
                sumr += f * ml[2];
                v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
            }
            put(r, c, inverse(sumr), v);
            if (c == 0) put_lse(r, M, sum);
        }
        return;
    }
    for (int i = tid; i < p.G * p.parts; i += nthreads) {  // row r's maximum of CTA j
        const int r = i / p.parts, j = i - r * p.parts;
        s_w[j * 64 + r] = ld_cluster(map_to_rank(smem_u32(s_cm + r), j));
    }
    __syncthreads();
    for (int r = tid; r < p.G; r += nthreads) {
        float M = -FLT_MAX, sum = 0.f, sumr = 0.f;
        for (int j = 0; j < p.parts; ++j) M = fmaxf(M, s_w[j * 64 + r]);
        for (int j = 0; j < p.parts; ++j) {
            const float f = exp2f(s_w[j * 64 + r] - M);
            sum += f * ld_cluster(map_to_rank(smem_u32(s_cl + r), j));
            sumr += f * ld_cluster(map_to_rank(smem_u32(s_clr + r), j));
            s_w[j * 64 + r] = f;
        }
        s_w[16 * 64 + r] = inverse(sumr);
        if (rank == 0) put_lse(r, M, sum);
    }
    __syncthreads();
    for (int i = rank * nthreads + tid; i < p.G * (D / 4); i += p.parts * nthreads) {
        const int r = i / (D / 4), c = i - r * (D / 4);
        const uint32_t from = smem_u32(states + r * ST + 4 * c);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < p.parts; ++j) {
            const float f = s_w[j * 64 + r];
            const float4 x = ld_cluster4(map_to_rank(from, j));
            v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
        }
        put(r, c, s_w[16 * 64 + r], v);
    }
    cluster_sync();  // no CTA leaves while another reads its states
}

// Of the CTAs at D columns, whichever instance: their shared memory decides.
template <int D>
cudaError_t blocks_at_once(int (&n)[5]) {
    constexpr int NT = D < 256 ? 2 : 1;
    static std::atomic<uint64_t> ready{0}, known[kMaxDevices];
    return clusters_at_once(reinterpret_cast<const void*>(decode_blocks_kernel<D, NT, true>), (BlocksShape<D, NT>::WARPS + 1) * 32,
                            BlocksShape<D, NT>::SMEM, &ready, known, n);
}

template <int D, int NT, bool F32OUT>
cudaError_t launch_decode_blocks(const BlocksParams& p, cudaStream_t stream) {
    using Sh = BlocksShape<D, NT>;
    BlocksMaps maps;
    const cuuint64_t rows = p.pg.block_table ? (cuuint64_t)p.pg.num_pages << p.pg.page_shift : (cuuint64_t)p.B * p.S_max;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hkv, rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.Hkv * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)1 << p.unit_log2};
    if (!tc_encode_map(&maps.k, p.k, 3, dims, strides, box, false) || !tc_encode_map(&maps.v, p.v, 3, dims, strides, box, false))
        return cudaErrorInvalidValue;
    auto kern = decode_blocks_kernel<D, NT, F32OUT>;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory and clusters of 16
    const cudaError_t e = allow_clusters(reinterpret_cast<const void*>(kern), Sh::SMEM, &ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.shards * p.pairs * p.parts, 1, 1);
    cfg.blockDim = dim3((unsigned)(p.teams * p.head_warps + 1) * 32, 1, 1);
    cfg.dynamicSmemBytes = Sh::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p, maps);
}

#define KVD_BLOCKS_LAUNCH(DD)                                                                             \
    cudaError_t blocks_at_once_d##DD(int (&n)[5]) { return blocks_at_once<DD>(n); }                       \
    cudaError_t launch_decode_blocks_d##DD(const BlocksParams& p, bool f32_out, cudaStream_t stream) {    \
        if (p.head_rows == 8)                                                                             \
            return f32_out ? launch_decode_blocks<DD, 1, true>(p, stream) : launch_decode_blocks<DD, 1, false>(p, stream); \
        if constexpr (DD < 256)                                                                           \
            return f32_out ? launch_decode_blocks<DD, 2, true>(p, stream) : launch_decode_blocks<DD, 2, false>(p, stream); \
        return cudaErrorInvalidValue;                                                                     \
    }

}  // namespace kvd
