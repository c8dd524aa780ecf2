// Attention over listed blocks of tokens: for every (sequence, query token, KV
// head), the softmax over the tokens of the blocks that its list names,
//   s_t = scale * q . k_t,  out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m)   (base 2, log2(e) in the scale).
// It reads K * block rows of K and V a pair where the attention over all tokens reads the sequence;
// bound by memory for batches, by latency for one sequence.
//
// A unit is 16 tokens of a listed block, whose K rows and V rows a warp brings
// by TMA into its ring (128-byte swizzle) and works on alone: units are dealt to
// the warps of a pair's CTAs in turn, so every warp has its own loads in flight and waits for no other. The
// products are turned round so that tokens fill the 16 rows of m16n8k16 MMAs and query rows
// their 8 columns (a group of 4 to 8 query heads is one column tile): S^T = K q^T, O^T = V^T w, the weights
// transposed by movmatrix. The running maximum of a column is raised only where a score passes it by 2^8
// (a vote a unit otherwise): weights stay below 2^8 and keep their relative precision, bf16's 2^-8, the same
// rounding as the other attention kernels' of this library; for float32 output a second bf16 carries the rest to 2^-16.
// Groups of more than 16 query heads are shared out to head_warps warps over one ring.
//
// A pair's CTAs (parts, up to 16) are a cluster: their states are joined over
// distributed shared memory, each CTA writing a share of the output, without a second launch or a workspace. Where even
// 16 CTAs a pair leave SMs idle, `shards` such clusters a pair write normalised float32 results, which the
// shard merge of split_kv_merge.cu joins.
#pragma once

#include <cuda.h>
#include <float.h>
#include <math_constants.h>

#include <atomic>

#include "../../include/kvdecode.h"
#include "blocks.h"
#include "cluster.cuh"
#include "common.cuh"
#include "tc_common.cuh"

namespace kvd {

bool tc_encode_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box, bool u8);

struct BlocksMaps {
    CUtensorMap k;  // 3D: [rows of the cache, Hkv, D], box 16 x 1 x 64, 128-byte swizzle
    CUtensorMap v;
};

constexpr int kBlocksWarps = 4;

template <int D, int NT>
struct BlocksShape {
    static constexpr int RW = 8 * NT;                    // query rows of a warp
    static constexpr int ELEM = 16 * D * 2;              // a unit's rows of one tensor
    static constexpr int RING = 96 * 1024;               // shared out to the teams: two CTAs an SM
    static constexpr int SLOTS = RING / ELEM;
    static constexpr int ROWS = kBlocksWarps * RW;       // state rows of a CTA
    static constexpr int ST = D + 4;                     // floats between state rows: neighbours in different banks
    static constexpr int OFF_BAR = RING;                 // full and empty barriers
    static constexpr int OFF_ML = OFF_BAR + 2 * SLOTS * 8;   // m and the two sums of the states
    static constexpr int OFF_CML = OFF_ML + 3 * ROWS * 4;    // of the CTA's rows
    static constexpr int OFF_W = OFF_CML + 3 * 64 * 4;       // weights of the cluster's CTAs, and 1 / sum
    static constexpr int OFF_FLAG = OFF_W + 17 * 64 * 4;
    static constexpr int OFF_IN = OFF_FLAG + 16;             // what the cluster's CTAs send this one
    static constexpr int IN_FLOATS = 2048;
    static constexpr int SMEM = OFF_IN + IN_FLOATS * 4;
    static_assert(ROWS * ST * 4 <= RING, "the states take the ring's place");
    static_assert(2 * (SMEM + 1024) <= 227 * 1024, "two CTAs an SM");
};

// The bf16 MMA of common.cuh without its ordering against other instructions.
__device__ __forceinline__ void mma_bf16_free(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int NT, bool F32OUT>
__global__ void __launch_bounds__(kBlocksWarps * 32, 2) decode_blocks_kernel(const BlocksParams p,
                                                                          const __grid_constant__ BlocksMaps maps) {
    using Sh = BlocksShape<D, NT>;
    constexpr int RW = Sh::RW, KS = D / 16, MT = D / 16, ST = Sh::ST;
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

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthreads = blockDim.x;
    const int HT = p.head_warps, teams = (nthreads >> 5) / HT, team = warp / HT, wt = warp - team * HT;
    const int rank = blockIdx.x & (p.parts - 1), cl = blockIdx.x >> (__ffs(p.parts) - 1);  // (parts: a power of two)
    const int pair = cl % p.pairs, shard = cl / p.pairs;
    const int h = pair % p.Hkv, bt = pair / p.Hkv, t = bt % p.T, b = bt / p.T;
    const int R = Sh::SLOTS / teams, slot0 = team * R;  // this team's ring
    auto full = [&](int s) { return bars + 8u * (slot0 + s); };
    auto empty = [&](int s) { return bars + 8u * (Sh::SLOTS + slot0 + s); };

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

    // ---- the tokens this query token sees, and the units of this team ----
    const int raw = __ldg(p.seq_lens + b), L = raw < 0 ? 0 : raw > p.S_max ? p.S_max : raw;
    if (raw != L && tid == 0 && p.status) atomicOr(p.status, KVD_STATUS_SEQ_LEN_CLAMPED);
    const int seen = L - p.T + 1 + t;  // <= 0: none
    const int32_t* list = p.blocks + (size_t)pair * p.K;
    const int units = p.K << p.unit_shift, submask = (1 << p.unit_shift) - 1;
    const int W = p.shards * p.parts * teams, wid = (shard * p.parts + rank) * teams + team;
    const int last_block = (p.S_max - 1) >> (p.unit_shift + 4);  // of the cache's

    // Units are looked up 32 at a time, one a lane: how many of its tokens count, and its cache row. Those of entries
    // that name no block the token sees have none and are passed over. (List and table are read beside the length, not behind it.)
    struct Cursor {
        int u;          // the next look-up's first unit of this team
        uint32_t mask;  // lanes whose unit is still to come
        int row, n;
    };
    auto look_up = [&](Cursor& c, bool rows) {
        do {
            const long long u = c.u + (long long)lane * W;
            const int blk = u < units ? __ldg(list + ((int)u >> p.unit_shift)) : -1;
            const bool named = blk >= 0 && blk <= last_block;
            const int tok = named ? ((blk << p.unit_shift) + ((int)u & submask)) << 4 : 0;
            const bool held = named && tok < p.S_max;
            bool bad = false;
            if (rows && held) {
                if (p.pg.block_table) {
                    const int page = __ldg(p.pg.block_table + (size_t)b * p.pg.max_blocks + (tok >> p.pg.page_shift));
                    bad = (unsigned)page >= (unsigned)p.pg.num_pages;  // reads as zero rows: past the pool's end
                    c.row = bad ? p.pg.num_pages << p.pg.page_shift : (page << p.pg.page_shift) + (tok & ((1 << p.pg.page_shift) - 1));
                } else {
                    c.row = b * p.S_max + tok;
                }
            }
            c.n = held ? min(16, seen - tok) : 0;
            if (bad && c.n > 0 && p.status) atomicOr(p.status, KVD_STATUS_BAD_PAGE);
            c.mask = __ballot_sync(0xffffffffu, c.n > 0);
            const long long next = c.u + 32LL * W;
            c.u = next < units ? (int)next : units;
        } while (c.mask == 0 && c.u < units);
    };

    // ---- loads: K and V of each unit in turn, into the ring's slots in turn ----
    Cursor lc{min(wid, units), 0, 0, 0}, cc = lc;
    int issued = 0, islot = 0, iphase = 1, irow = 0;  // iphase: parity of the last release of slot islot
    bool more = true;
    const uint64_t policy = l2_evict_first_policy();
    bool dead = false;
    auto issue = [&]() {  // whole leading warps call this
        if (!(issued & 1)) {
            if (lc.mask == 0 && lc.u < units) look_up(lc, true);
            if (lc.mask == 0) {
                more = false;
                return;
            }
            const int i = __ffs(lc.mask) - 1;
            lc.mask &= lc.mask - 1;
            irow = __shfl_sync(0xffffffffu, lc.row, i);
        }
        if (HT > 1 && issued >= R && !dead && !tc::mbar_wait(empty(islot), iphase, abort_flag, kBudget)) dead = true;
        if (lane == 0 && !dead) {
            const CUtensorMap* map = (issued & 1) ? &maps.v : &maps.k;
            const uint32_t dst = ring + (uint32_t)(slot0 + islot) * Sh::ELEM, bar = full(islot);
            tc::mbar_arrive_expect_tx(bar, Sh::ELEM);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(dst + c * 2048, map, c * 64, h, irow, bar, policy);
        }
        ++issued;
        if (++islot == R) islot = 0, iphase ^= 1;
    };
    const bool lead = wt == 0;
    if (lead) {
        look_up(lc, true);
        for (int i = 0; i < R && more; ++i) issue();
    }

    // l: the weights' sum, for lse. lr: of the weights as V meets them, so that the output is a convex combination of V
    // rows (the same where float32 output carries both parts).
    float o[MT][NT][4], m[NT][2], l[NT][2], lr[F32OUT ? 1 : NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -FLT_MAX;
        l[n][0] = l[n][1] = 0.f;
        if constexpr (!F32OUT) lr[n][0] = lr[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }

    // ---- the units ----
    // A slot given back is filled again at once by a warp alone; a team's leader fills the slot of two elements before, so
    // that it seldom waits for the others.
    int done = 0, cslot = 0, cphase = 0;
    auto release = [&]() {
        __syncwarp();
        if (HT > 1) {
            if (lane == 0) tc::mbar_arrive(empty(cslot));
            if (lead && done >= 2 && more) issue();
        } else if (more) {
            issue();
        }
        ++done;
        if (++cslot == R) cslot = 0, cphase ^= 1;
    };
    auto chunk = [&](uint32_t base, int row, int c) {  // 16-byte chunk c of a swizzled row
        return base + (uint32_t)((c >> 3) * 2048 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
    };
    look_up(cc, false);
    while (cc.mask) {
        const int src = __ffs(cc.mask) - 1;
        const int n_tok = __shfl_sync(0xffffffffu, cc.n, src);
        cc.mask &= cc.mask - 1;
        if (cc.mask == 0 && cc.u < units) look_up(cc, false);

        if (!tc::mbar_wait(full(cslot), cphase, abort_flag, kBudget)) {
            dead = true;
            break;
        }
        float s[NT][4];
        {
            const uint32_t kb = ring + (uint32_t)(slot0 + cslot) * Sh::ELEM;
            const int row = lane & 15, half = lane >> 4;
            float s2[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                uint32_t a[4];
                ldmatrix_x4(chunk(kb, row, 2 * kk + half), a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16_free((kk & 1) ? s2[n] : s[n], a, qf[n][kk][0], qf[n][kk][1]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = (s[n][e] + s2[n][e]) * p.scale_log2;
        }
        release();
        // Tokens lane / 4 (s[n][0..1]) and lane / 4 + 8 (s[n][2..3]), query rows 8 n + 2 (lane % 4) + 0..1.
        if (n_tok < 16) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if ((lane >> 2) >= n_tok) s[n][0] = s[n][1] = -CUDART_INF_F;
                if ((lane >> 2) + 8 >= n_tok) s[n][2] = s[n][3] = -CUDART_INF_F;
            }
        }
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            raise |= fmaxf(s[n][0], s[n][2]) > m[n][0] + 8.f;
            raise |= fmaxf(s[n][1], s[n][3]) > m[n][1] + 8.f;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(s[n][e], s[n][e + 2]);
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
        uint32_t ph[NT][2], pl[F32OUT ? NT : 1][2];  // the weights as B fragments
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float e0 = tc::ex2_approx(s[n][2 * y] - m[n][0]), e1 = tc::ex2_approx(s[n][2 * y + 1] - m[n][1]);
                const uint32_t hi = pack_bf16x2(e0, e1);
                ph[n][y] = movmatrix_trans(hi);
                l[n][0] += e0;
                l[n][1] += e1;
                if constexpr (F32OUT) {
                    pl[n][y] = movmatrix_trans(pack_bf16x2(e0 - bf16_lo(hi), e1 - bf16_hi(hi)));
                } else {
                    lr[n][0] += bf16_lo(hi);
                    lr[n][1] += bf16_hi(hi);
                }
            }

        if (!tc::mbar_wait(full(cslot), cphase, abort_flag, kBudget)) {
            dead = true;
            break;
        }
        {
            const uint32_t vb = ring + (uint32_t)(slot0 + cslot) * Sh::ELEM;
            if (n_tok < 16) {  // rows past the last token hold anything: zero, since 0 * NaN is not 0
                for (int i = lane + n_tok * 8; i < 16 * 8; i += 32)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        *reinterpret_cast<uint4*>(smem + (vb - ring) + c * 2048 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                __syncwarp();
            }
            const int row = (lane & 7) + ((lane >> 4) << 3), odd = (lane >> 3) & 1;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t a[4];
                ldmatrix_x4_trans(chunk(vb, row, 2 * i + odd), a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16_free(o[i][n], a, ph[n][0], ph[n][1]);
                    if constexpr (F32OUT) mma_bf16_free(o[i][n], a, pl[n][0], pl[n][1]);
                }
            }
            if (n_tok < 16) tc::fence_proxy_async_smem();  // the zeros come before the next load
        }
        release();
    }
    if (dead) {
        if (lane == 0 && p.status) atomicOr(p.status, KVD_STATUS_TIMEOUT);
        // Copies still on their way are waited for (again with a limit), since the ring's place is used below.
        if (lead)
            for (; done < issued; ++done) {
                for (long long t0 = clock64(); !tc::mbar_test(full(cslot), cphase) && clock64() - t0 < kBudget;) {
                }
                if (++cslot == R) cslot = 0, cphase ^= 1;
            }
    }

    // ---- the states to shared memory, in the ring's place ----
    __syncthreads();
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

template <int D, int NT, bool F32OUT>
cudaError_t launch_decode_blocks(const BlocksParams& p, cudaStream_t stream) {
    using Sh = BlocksShape<D, NT>;
    BlocksMaps maps;
    const cuuint64_t rows = p.pg.block_table ? (cuuint64_t)p.pg.num_pages << p.pg.page_shift : (cuuint64_t)p.B * p.S_max;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hkv, rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.Hkv * D * 2};
    const cuuint32_t box[3] = {64, 1, 16};
    if (!tc_encode_map(&maps.k, p.k, 3, dims, strides, box, false) || !tc_encode_map(&maps.v, p.v, 3, dims, strides, box, false))
        return cudaErrorInvalidValue;
    auto kern = decode_blocks_kernel<D, NT, F32OUT>;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory and clusters of 16
    const cudaError_t e = allow_clusters(reinterpret_cast<const void*>(kern), Sh::SMEM, &ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.shards * p.pairs * p.parts, 1, 1);
    cfg.blockDim = dim3((unsigned)(kBlocksWarps / p.head_warps * p.head_warps) * 32, 1, 1);
    cfg.dynamicSmemBytes = Sh::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, maps);
}

#define KVD_BLOCKS_LAUNCH(DD)                                                                             \
    cudaError_t launch_decode_blocks_d##DD(const BlocksParams& p, bool f32_out, cudaStream_t stream) {    \
        if (p.G <= 8) return f32_out ? launch_decode_blocks<DD, 1, true>(p, stream) : launch_decode_blocks<DD, 1, false>(p, stream); \
        return f32_out ? launch_decode_blocks<DD, 2, true>(p, stream) : launch_decode_blocks<DD, 2, false>(p, stream);               \
    }

}  // namespace kvd
