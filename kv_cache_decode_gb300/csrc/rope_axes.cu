// Rotary positions of several axes (time, height and width of an image's or a video's tokens): pair i of a row
// turns by position[axes[i]] * w_i, the phases as in rope.cuh. Rows are turned as rope.cu turns them, and
// appended as kv_append_rope.cu appends them, but to cache rows that a slot map names, since a token's
// positions no longer say where it lies. One read of q, k and v and one write of each; bound by memory for
// prompts (turning 1.07 GB 156 us, appending 1.19 GB 177: the copy rate) and by latency for single tokens (3.5
// us). A warp takes a row, a share of its heads where there are few rows, or several rows where rows are short;
// a row's positions (4 at most) are loaded once and picked from registers.
#include <algorithm>

#include "append_unit.cuh"
#include "blocks.h"

namespace kvd {

constexpr int kAxesWarps = 4;

// Position of one row on any axis.
struct AxisPos {
    int p[4];
    __device__ __forceinline__ void load(const RopeAxes& r, long long row) {
#pragma unroll
        for (int a = 0; a < 4; ++a) p[a] = a < r.n_axes ? __ldg(r.positions + a * r.axis_stride + row) : 0;
    }
    __device__ __forceinline__ long long on(int axis) const {
        return axis == 0 ? p[0] : axis == 1 ? p[1] : axis == 2 ? p[2] : p[3];
    }
};

// The cosines and sines of rows row .. row + n - 1, [row][R / 2], by a whole warp (lane i holds row i's positions).
__device__ __forceinline__ void axes_table(const RopeAxes& rope, const AxisPos& mine, int n, float2* buf) {
    const int lane = threadIdx.x & 31, half = rope.table.rotary_dim >> 1;
    int tok = 0, i = lane;
    for (int e = 0; e < n * half; e += 32) {
        while (i >= half) i -= half, ++tok;
        AxisPos at;
#pragma unroll
        for (int a = 0; a < 4; ++a) at.p[a] = a < rope.n_axes ? __shfl_sync(0xffffffffu, mine.p[a], tok & 31) : 0;
        if (tok < n)
            rope_table_put(buf, tok * half + i,
                           rope_cos_sin(at.on(__ldg(rope.axes + i)), __ldg(rope.table.turns + i), rope.table.factor));
        i += 32;
    }
    __syncwarp();
}

template <bool IN32, bool OUT32, int DD>
__global__ void __launch_bounds__(kAxesWarps * 32) rope_axes_kernel(const RopeAxes rope, const void* x, long long xs, void* y,
                                                                    long long ys, long long rows, int parts, int H, int D) {
    extern __shared__ __align__(16) float2 s_cs[];  // [warps][R / 2]
    const long long w = (long long)blockIdx.x * kAxesWarps + (threadIdx.x >> 5);
    const long long row = w / parts;
    if (row >= rows) return;
    AxisPos at;
    at.load(rope, row);
    RopeWarp<DD> rw;
    rw.init(rope.table, D, s_cs + (threadIdx.x >> 5) * (rope.table.rotary_dim >> 1),
            [&](int i) { return at.on(__ldg(rope.axes + i)); });
    rw.template heads<IN32, OUT32>(x, (size_t)row * xs, y, (size_t)row * ys, H, (int)(w - row * parts), parts);
}

// Rows of few units: several to a warp.
template <bool IN32, bool OUT32>
__global__ void __launch_bounds__(kAxesWarps * 32) rope_axes_rows_kernel(const RopeAxes rope, const void* x, long long xs, void* y,
                                                                         long long ys, long long rows, int per_warp, int H, int D) {
    extern __shared__ __align__(16) float2 s_cs[];  // [warps][per_warp][R / 2]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = ((long long)blockIdx.x * kAxesWarps + warp) * per_warp;
    if (row >= rows) return;
    const int n = (int)min((long long)per_warp, rows - row);
    const RopeTokens rt{D, (D + 15) >> 4, rope.table.rotary_dim, n, rope.table.interleaved != 0, 0xffffffffu,
                        s_cs + (size_t)warp * per_warp * (rope.table.rotary_dim >> 1)};
    AxisPos at;
    at.load(rope, row + (lane < n ? lane : 0));
    rt.heads<IN32, OUT32, false>(x, (size_t)row * xs, (size_t)xs, y, (size_t)row * ys, (size_t)ys, H, rope.table, 0,
                                 [&]() { axes_table(rope, at, n, rt.s_cs); });
}

// Short rows of one head, where no thread shares a pair's cosine and sine with another: two units of 16 columns
// a thread, which forms its own. Rows of up to 128 columns: 134 MB of bf16 rows of 64 columns (all turned) take
// 38 us, 64 by the warps above; of 80 41 and 57, of 128 (half turned) 40.5 and 42; of 256, which stay with the
// warps, 40.5 and 32.
template <bool IN32, bool OUT32>
__global__ void __launch_bounds__(kAxesWarps * 32) rope_axes_one_kernel(const RopeAxes rope, const void* x, long long xs, void* y,
                                                                        long long ys, unsigned total, int D) {
    const unsigned units = (D + 15) >> 4, R = rope.table.rotary_dim;
    const bool inter = rope.table.interleaved;
    const unsigned step = gridDim.x * kAxesWarps * 32, j0 = blockIdx.x * kAxesWarps * 32 + threadIdx.x;
    RopeRaw<IN32> raw[2];
    AxisPos at[2];
    RopeUnit ru[2];
    long long row[2];
    int u[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const unsigned j = j0 + k * step < total ? j0 + k * step : j0 < total ? j0 : 0;
        row[k] = j / units;
        u[k] = (int)(j - (unsigned)row[k] * units);
        ru[k] = rope_unit(u[k], D, R, inter);
        raw[k].load(x, (size_t)row[k] * xs, ru[k]);
        at[k].load(rope, row[k]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (j0 + k * step >= total) return;
        const size_t e = (size_t)row[k] * ys;
        if (IN32 == OUT32 && !ru[k].turn) {
            raw[k].copy(y, e, ru[k]);
            continue;
        }
        float a[8], b[8];
        raw[k].get(a, b);
        if (ru[k].turn) {
            const uint2 ax = __ldg(reinterpret_cast<const uint2*>(rope.axes + 8 * u[k]));
            float2 cs[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                cs[i] = rope_cos_sin(at[k].on((int)(((i < 4 ? ax.x : ax.y) >> (8 * (i & 3))) & 0xffu)),
                                     __ldg(rope.table.turns + 8 * u[k] + i), rope.table.factor);
            rope_turn(a, b, cs, inter);
        }
        store8<OUT32>(y, e + ru[k].ca, a);
        if (ru[k].cb >= 0) store8<OUT32>(y, e + ru[k].cb, b);
    }
}

// Cache row that row's slot names, or -1: none (a negative slot), or none there is (flagged).
__device__ __forceinline__ long long slot_row(const int32_t* slots, long long row, long long cache_rows, int32_t* status) {
    const int s = __ldg(slots + row);
    if (s >= cache_rows) {
        if (status) atomicOr(status, KVD_STATUS_POS_OUT_OF_RANGE);
        return -1;
    }
    return s < 0 ? -1 : s;
}

// DD: head dimension 64, 128 or 256, or 0 for any other (bf16 cache only).
template <CacheForm FORM, int DD>
__global__ void __launch_bounds__(kAxesWarps * 32, 7) append_axes_kernel(const AppendTarget to, const RopeAxes rope, const NewRows in,
                                                                      const int32_t* __restrict__ slots, long long cache_rows,
                                                                      int parts, int32_t* status) {
    extern __shared__ __align__(16) float2 s_cs[];  // [warps][R / 2]
    pdl_launch_dependents();  // the attention that may follow waits for this grid before it reads anything
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * kAxesWarps + (threadIdx.x >> 5);
    const long long row = w / parts;
    const int part = (int)(w - row * parts);
    if (row >= in.rows) return;
    const long long dst = slot_row(slots, row, cache_rows, part == 0 && lane == 0 ? status : nullptr);
    if (dst < 0 && !in.q) return;
    AxisPos at;
    at.load(rope, row);
    RopeWarp<DD> rw;
    rw.init(rope.table, in.D, s_cs + (threadIdx.x >> 5) * (rope.table.rotary_dim >> 1),
            [&](int i) { return at.on(__ldg(rope.axes + i)); });
    const int D = rw.D, units = rw.units;
    if (in.q) rw.template heads<false, false>(in.q, (size_t)row * in.qs, in.q_out, (size_t)row * in.qos, in.Hq, part, parts);
    if (dst < 0) return;
    // ---- keys, then values, two steps' loads at a time; whole warps stay in the loop for the shuffles ----
    const int total = 2 * in.Hkv * units;
    for (int base = 32 * part; base < total; base += 64 * parts) {
        RopeRaw<false> raw[2];
        RopeUnit ru[2];
        int h[2], u[2];
        bool value[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j0 = base + k * 32 * parts + lane, j = j0 < total ? j0 : 0, hh = j / units;
            u[k] = j - hh * units;
            value[k] = hh >= in.Hkv;
            h[k] = value[k] ? hh - in.Hkv : hh;
            ru[k] = rope_unit(u[k], D, value[k] ? 0 : rw.R, rope.table.interleaved);
            if (j0 < total) raw[k].load(value[k] ? in.v : in.k, (size_t)row * (value[k] ? in.vs : in.ks) + (size_t)h[k] * D, ru[k]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j0 = base + k * 32 * parts;
            if (j0 >= total) break;
            put_unit<FORM, DD>(to, in, rope.table.interleaved, raw[k], ru[k], value[k] ? 0 : rw.R, value[k], h[k], u[k], D, dst, 0,
                               j0 + lane < total, [&](float(&a)[8], float(&b)[8]) { rw.turn(a, b, u[k]); });
        }
    }
}

// Tokens of few heads: several to a warp.
template <CacheForm FORM, int DD>
__global__ void __launch_bounds__(kAxesWarps * 32, 7) append_axes_rows_kernel(const AppendTarget to, const RopeAxes rope,
                                                                           const NewRows in, const int32_t* __restrict__ slots,
                                                                           long long cache_rows, int per_warp, int32_t* status) {
    extern __shared__ __align__(16) float2 s_cs[];  // [warps][per_warp][R / 2]
    pdl_launch_dependents();  // as above
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row0 = ((long long)blockIdx.x * kAxesWarps + warp) * per_warp;
    if (row0 >= in.rows) return;
    const int n = (int)min((long long)per_warp, in.rows - row0);
    const long long dst = lane < n ? slot_row(slots, row0 + lane, cache_rows, status) : -1;
    const int R = rope.table.rotary_dim, D = DD ? DD : in.D, units = DD ? DD / 16 : (D + 15) >> 4;
    const RopeTokens rt{D, units, R, n, rope.table.interleaved != 0, 0xffffffffu, s_cs + (size_t)warp * per_warp * (R >> 1)};
    AxisPos at;
    at.load(rope, row0 + (lane < n ? lane : 0));
    if (in.q)
        rt.heads<false, false, false>(in.q, (size_t)row0 * in.qs, (size_t)in.qs, in.q_out, (size_t)row0 * in.qos, (size_t)in.qos,
                                      in.Hq, rope.table, 0, [&]() { axes_table(rope, at, n, rt.s_cs); });
    const int total = n * 2 * in.Hkv * units;
    for (int base = 0; base < total; base += 64) {
        RopeRaw<false> raw[2];
        RopeUnit ru[2];
        int hh[2], u[2], tok[2];
        long long to_row[2];
        bool live[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = base + 32 * k + lane;
            rt.item(j, 2 * in.Hkv, tok[k], hh[k], u[k]);
            to_row[k] = __shfl_sync(0xffffffffu, dst, tok[k] & 31);
            live[k] = j < total && to_row[k] >= 0;
            const bool value = hh[k] >= in.Hkv;
            ru[k] = rope_unit(u[k], D, value ? 0 : R, rope.table.interleaved);
            if (live[k])
                raw[k].load(value ? in.v : in.k, (size_t)(row0 + tok[k]) * (value ? in.vs : in.ks) +
                                                     (size_t)(value ? hh[k] - in.Hkv : hh[k]) * D, ru[k]);
        }
        if (base == 0 && !in.q) axes_table(rope, at, n, rt.s_cs);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (base + 32 * k >= total) break;
            const bool value = hh[k] >= in.Hkv;
            put_unit<FORM, DD>(to, in, rope.table.interleaved, raw[k], ru[k], value ? 0 : R, value, value ? hh[k] - in.Hkv : hh[k],
                               u[k], D, to_row[k], 0, live[k], [&](float(&a)[8], float(&b)[8]) { rt.turn(a, b, tok[k], u[k]); });
        }
    }
}

cudaError_t launch_rope_axes(const RopeAxes& rope, const void* x, long long xs, bool in32, void* y, long long ys, bool out32,
                             long long rows, int H, int D, int num_sms, cudaStream_t stream) {
    const long long units = (long long)H * ((D + 15) / 16), steps = (units + 31) / 32;
    const int per_warp = rope_tokens(rows, units, 64, num_sms);
    const int parts = per_warp > 1 ? 1 : rope_parts(rows, steps, num_sms);
    cudaLaunchConfig_t cfg = {};
    if (H == 1 && units <= 8 && rows * units < (1LL << 31)) {
        cfg.gridDim = dim3((unsigned)((rows * units + 2 * kAxesWarps * 32 - 1) / (2 * kAxesWarps * 32)), 1, 1);
        cfg.blockDim = dim3(kAxesWarps * 32, 1, 1);
        cfg.stream = stream;
#define KVD_AXES(A, B) cudaLaunchKernelEx(&cfg, rope_axes_one_kernel<A, B>, rope, x, xs, y, ys, (unsigned)(rows * units), D)
        if (in32) return out32 ? KVD_AXES(true, true) : KVD_AXES(true, false);
        return out32 ? KVD_AXES(false, true) : KVD_AXES(false, false);
#undef KVD_AXES
    }
    cfg.gridDim = dim3((unsigned)(per_warp > 1 ? (rows + per_warp * kAxesWarps - 1) / (per_warp * kAxesWarps)
                                               : (rows * parts + kAxesWarps - 1) / kAxesWarps), 1, 1);
    cfg.blockDim = dim3(kAxesWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)kAxesWarps * per_warp * (rope.table.rotary_dim / 2) * sizeof(float2);
    cfg.stream = stream;
#define KVD_AXES_D(A, B, DD) cudaLaunchKernelEx(&cfg, rope_axes_kernel<A, B, DD>, rope, x, xs, y, ys, rows, parts, H, D)
#define KVD_AXES(A, B)                                                                                                \
    (per_warp > 1 ? cudaLaunchKernelEx(&cfg, rope_axes_rows_kernel<A, B>, rope, x, xs, y, ys, rows, per_warp, H, D)   \
     : D == 64 ? KVD_AXES_D(A, B, 64) : D == 128 ? KVD_AXES_D(A, B, 128) : D == 256 ? KVD_AXES_D(A, B, 256) : KVD_AXES_D(A, B, 0))
    if (in32) return out32 ? KVD_AXES(true, true) : KVD_AXES(true, false);
    return out32 ? KVD_AXES(false, true) : KVD_AXES(false, false);
#undef KVD_AXES
#undef KVD_AXES_D
}

cudaError_t launch_append_axes(const AppendTarget& to, const RopeAxes& rope, const NewRows& in, const int32_t* slots,
                               long long cache_rows, int32_t* status, int num_sms, cudaStream_t stream) {
    const long long units = (in.D + 15) / 16, hq = in.q ? in.Hq : 0;
    const int per_warp = rope_tokens(in.rows, (hq + 2LL * in.Hkv) * units, 256, num_sms);
    const long long steps = (std::max(hq, 2LL * in.Hkv) * units + 31) / 32;
    const int parts = per_warp > 1 ? 1 : rope_parts(in.rows, steps, num_sms);  // warps of a token
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(per_warp > 1 ? (in.rows + per_warp * kAxesWarps - 1) / (per_warp * kAxesWarps)
                                               : (in.rows * parts + kAxesWarps - 1) / kAxesWarps), 1, 1);
    cfg.blockDim = dim3(kAxesWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)kAxesWarps * per_warp * (rope.table.rotary_dim / 2) * sizeof(float2);
    cfg.stream = stream;
#define KVD_APP(F, DD)                                                                                                         \
    (per_warp > 1 ? cudaLaunchKernelEx(&cfg, append_axes_rows_kernel<CacheForm::F, DD>, to, rope, in, slots, cache_rows,       \
                                       per_warp, status)                                                                       \
                  : cudaLaunchKernelEx(&cfg, append_axes_kernel<CacheForm::F, DD>, to, rope, in, slots, cache_rows, parts, status))
#define KVD_APP_D(F) \
    (in.D == 64 ? KVD_APP(F, 64) : in.D == 128 ? KVD_APP(F, 128) : in.D == 256 ? KVD_APP(F, 256) : cudaErrorInvalidValue)
    switch (to.form) {
        case CacheForm::kBf16:
            return in.D == 64    ? KVD_APP(kBf16, 64)
                   : in.D == 128 ? KVD_APP(kBf16, 128)
                   : in.D == 256 ? KVD_APP(kBf16, 256)
                                 : KVD_APP(kBf16, 0);
        case CacheForm::kInt8: return KVD_APP_D(kInt8);
        case CacheForm::kFp8: return KVD_APP_D(kFp8);
        case CacheForm::kFp4: break;
    }
#undef KVD_APP_D
#undef KVD_APP
    return cudaErrorInvalidValue;
}

}  // namespace kvd
