"""The fp4 KV cache on the GPU: quantizer and reader bit for bit against the
oracle, attention over the rows read back against float64.

Tolerances (assert_close's): fp32 output 1e-4, bf16 output 1e-2 or half a step
plus the weights' rounding. The kernel's weights carry f16's 2^-11 (half a step,
bf16 output), the fp32 output's 2^-22, so both lie inside them; scores are fp32
sums of at most 256 products of |q| <= ~5 with |k| <= ~5, times scale
<= 1/8: within 256 * 25 / 8 * 2^-24 < 5e-5 absolute, a relative weight error of the same
size, spread over outputs of size 1."""
import math

import numpy as np
import pytest

import oracle
from gpu_helpers import assert_close, bf16_tensor_bits, cuda_or_skip, guarded, guards_intact, to_dev_bf16
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _rows(r, shape, spread=0.0):
    x = r.standard_normal(shape).astype(np.float32)
    if spread:
        x *= np.exp2(r.uniform(-spread, spread, shape[:-1] + (1,))).astype(np.float32)
    return f32_to_bf16_bits(x)


def _blocks(bits):
    """(blocks [B, Hkv, S / 16, ...], float64 rows [B, S, Hkv, D]) of bf16 rows [B, S, Hkv, D]."""
    c = oracle.quantize_fp4(np.ascontiguousarray(bits.transpose(0, 2, 1, 3)))
    return oracle.pack_fp4(*c), np.ascontiguousarray(oracle.dequantize_fp4(*c).transpose(0, 2, 1, 3))


def _poison(blocks, lens, D):
    """Rows past each length get codes, scales and exponents of all ones (NaN scales)."""
    codes, sb, exps = oracle.unpack_fp4(blocks, D)
    for b, L in enumerate(lens):
        codes[b, :, L:], sb[b, :, L:], exps[b, :, L:] = 15, 255, 255
    return oracle.pack_fp4(codes, sb, exps)


class Case:
    def __init__(self, seed, Hq, Hkv, D, lens, T=1, page=0, spread=0.0, dev=None):
        import torch
        r = np.random.default_rng(seed)
        self.T, self.D, self.Hq, self.Hkv, self.page = T, D, Hq, Hkv, page
        B, step = len(lens), page or 16
        self.lens = np.asarray(lens, np.int32)
        S = max(step, -(-max(max(lens), 1) // step) * step)
        self.S, self.B = S, B
        self.scale = float(np.float32(D ** -0.5))
        self.q = _rows(r, (B, T, Hq, D))
        kb, self.kd = _blocks(_rows(r, (B, S, Hkv, D), spread))
        vb, self.vd = _blocks(_rows(r, (B, S, Hkv, D), spread))
        kb, vb = _poison(kb, self.lens, D), _poison(vb, self.lens, D)
        self.bt = None
        if page:
            nb = S // page
            table = r.permutation(B * nb + 3)[:B * nb].reshape(B, nb).astype(np.int32)
            pool = [np.full((B * nb + 3, Hkv, page // 16, 9 * D + 16), 255, np.uint8) for _ in range(2)]
            for b in range(B):
                for j in range(nb):
                    for p, x in zip(pool, (kb, vb)):
                        p[table[b, j]] = x[b, :, j * (page // 16):(j + 1) * (page // 16)]
            for b in range(B):  # entries of blocks past the length name nothing
                table[b, -(-int(self.lens[b]) // page):] = -7
            kb, vb = pool
            self.bt = torch.from_numpy(table).to(dev)
        self.k, self.v = torch.from_numpy(kb).to(dev), torch.from_numpy(vb).to(dev)
        self.qd = to_dev_bf16(self.q, dev)
        self.lens_d = torch.from_numpy(self.lens).to(dev)

    def run(self, kvd, torch, dev, dtype, n_split=0, max_len=None, q=None):
        B, T, Hq, D = self.q.shape
        mx = self.S if max_len is None else max_len
        full, out = guarded((B, T, Hq, D), torch.bfloat16 if dtype == "bf16" else torch.float32, dev)
        lfull, lse = guarded((B, T, Hq), torch.float32, dev)
        _, n = kvd.decode_plan_fp4(B, T, Hq, self.Hkv, D, mx, 0, n_split)
        ws = torch.full((n + 512,), 0xa5, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        kvd.decode_fp4(self.qd if q is None else q, self.k, self.v, self.lens_d, mx, self.scale, out, block_table=self.bt,
                       workspace=ws[:n] if n else None, n_split=n_split, lse=lse, status=self.status)
        torch.cuda.synchronize()
        assert guards_intact(full) and guards_intact(lfull) and bool((ws[n:] == 0xa5).all())
        got = bf16_bits_to_f32(bf16_tensor_bits(out)) if dtype == "bf16" else out.cpu().numpy()
        return got.astype(np.float64), lse.cpu().numpy().astype(np.float64)

    def want(self):
        outs, lses = [], []
        for i in range(self.T):
            L = np.clip(self.lens - self.T + 1 + i, 0, None).astype(np.int32)
            o, l = oracle.decode_attention_f64kv(self.q[:, i], self.kd, self.vd, L, self.scale)
            outs.append(o)
            lses.append(l)
        return np.stack(outs, 1), np.stack(lses, 1)

    def check(self, kvd, torch, dev, dtype, **kw):
        got, lse = self.run(kvd, torch, dev, dtype, **kw)
        want, wl = self.want()
        assert int(self.status.item()) == 0
        assert_close(got, want, dtype, "fp4")
        none = np.isneginf(wl)
        assert np.array_equal(np.isneginf(lse), none) and np.abs(lse[~none] - wl[~none]).max(initial=0.0) < 1e-4
        assert (got[none] == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_quantize_and_read(D):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(D)
    B, S, Hkv = 5, 48, 3
    bits = _rows(r, (B, S, Hkv, D), 12.0)
    bits[0, 3] = 0
    bits[1, 2, 0, :16] = 0
    lens = np.array([48, 17, 0, 33, 60], np.int32)  # the last is clamped
    blocks = torch.full((B, Hkv, 4, 9 * D + 16), 0x5a, dtype=torch.uint8, device=dev)  # a longer cache
    kvd.kv_quantize_fp4(to_dev_bf16(bits, dev), blocks, torch.from_numpy(lens).to(dev), S)
    torch.cuda.synchronize()
    want, rows = _blocks(bits)
    want = np.concatenate([want, np.full((B, Hkv, 1, 9 * D + 16), 0x5a, np.uint8)], 2)
    old = [a.copy() for a in oracle.unpack_fp4(np.full_like(want, 0x5a), D)]
    new = oracle.unpack_fp4(want, D)
    for b in range(B):
        for o, n in zip(old, new):
            o[b, :, :min(lens[b], S)] = n[b, :, :min(lens[b], S)]
    assert np.array_equal(blocks.cpu().numpy(), oracle.pack_fp4(*old))
    # back: contiguous, then the same rows in pages
    out = torch.full((B, S + 7, Hkv, D), 3.0, dtype=torch.bfloat16, device=dev)
    ld = torch.from_numpy(lens).to(dev)
    kvd.kv_read_fp4(blocks, out, ld, S)
    torch.cuda.synchronize()
    exp = np.full((B, S + 7, Hkv, D), 3.0)
    for b in range(B):
        exp[b, :min(lens[b], S)] = rows[b, :min(lens[b], S)]
    assert np.array_equal(out.double().cpu().numpy(), exp)
    table = torch.randperm(B * 4 + 2, device=dev)[:B * 4].view(B, 4).int()
    pool = torch.zeros(B * 4 + 2, Hkv, 1, 9 * D + 16, dtype=torch.uint8, device=dev)
    pool[table.long()] = blocks.transpose(1, 2).unsqueeze(3)
    table[2] = -1  # an empty sequence's entries are not looked at
    table[3, 1] = 1 << 20
    exp[3, 16:32] = 0
    out.fill_(3.0)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kvd.kv_read_fp4(pool, out, ld, S, block_table=table, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvd.STATUS_BAD_PAGE
    assert np.array_equal(out.double().cpu().numpy(), exp)


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200, 257, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (32, 8, 128), (3, 3, 64), (9, 1, 64), (48, 1, 256), (5, 1, 256), (16, 1, 128),
                                      (64, 1, 128), (40, 2, 64)])
def test_attention(Hq, Hkv, D, dtype):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(Hq * D, Hq, Hkv, D, LENS, dev=dev)
    c.check(kvd, torch, dev, dtype)
    for n in (1, 2, 7, 600):  # every cut of the line gives the same answer
        c.check(kvd, torch, dev, dtype, n_split=n)


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("Hq,Hkv,D,T", [(8, 2, 128, 1), (24, 1, 64, 1), (6, 1, 256, 1), (8, 2, 128, 3), (12, 3, 64, 7), (4, 1, 256, 64)])
def test_attention_paged_multi(page, Hq, Hkv, D, T):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(page + T, Hq, Hkv, D, [300, 0, 1, T, 16, 47, 129], T=T, page=page, dev=dev)
    c.check(kvd, torch, dev, "f32")
    c.check(kvd, torch, dev, "bf16", n_split=5)


@pytest.mark.parametrize("Hq,Hkv,D,lens", [(8, 1, 128, [70001]), (4, 4, 64, [5000, 1, 12345]), (48, 1, 256, [9000, 4097]),
                                           (8, 8, 128, [3] * 200)])
def test_attention_long_and_many(Hq, Hkv, D, lens):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(1)
    c = Case(7, Hq, Hkv, D, lens, page=16, dev=dev)
    c.check(kvd, torch, dev, "f32")
    c.check(kvd, torch, dev, "bf16")


def test_magnitudes():
    """Rows whose sizes lie up to 2^60 apart, queries far below and above f16's range: the f16 weights
    keep their precision, checked relative to the terms that make up each output."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(31, 8, 2, 128, [200, 333, 40], dev=dev, spread=0.0)
    r = np.random.default_rng(5)
    # value rows spread over 2^+-30
    vb, c.vd = _blocks(_rows(r, (c.B, c.S, 2, 128), 30.0))
    c.v = torch.from_numpy(_poison(vb, c.lens, 128)).to(dev)
    # queries times 2^-40, keys times 2^40
    kb, c.kd = _blocks(f32_to_bf16_bits(bf16_bits_to_f32(_rows(r, (c.B, c.S, 2, 128))) * np.float32(2.0 ** 40)))
    c.k = torch.from_numpy(_poison(kb, c.lens, 128)).to(dev)
    c.q = f32_to_bf16_bits(bf16_bits_to_f32(c.q) * np.float32(2.0 ** -40))
    c.qd = to_dev_bf16(c.q, dev)
    got, lse = c.run(kvd, torch, dev, "f32")
    want, wl = c.want()
    mag, _ = oracle.decode_attention_f64kv(c.q[:, 0], c.kd, np.abs(c.vd), c.lens, c.scale)
    # weights to 2^-22 and scores to 5e-5, relative to sum_t w_t |v_t|
    assert (np.abs(got[:, 0] - want[:, 0]) <= 1e-4 * mag).all()
    assert np.abs(lse - wl).max() < 1e-4
    got, _ = c.run(kvd, torch, dev, "bf16")
    # bf16 output: f16 weights 2^-11 and half a bf16 step besides
    assert (np.abs(got[:, 0] - want[:, 0]) <= (1e-4 + 2.0 ** -10) * mag + np.abs(want[:, 0]) * 2.0 ** -8).all()


def test_rising_scores():
    """Scores that keep rising along the sequence raise the running maxima again and again."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(3, 8, 1, 64, [700], dev=dev)
    q = np.zeros((1, 1, 8, 64), np.float32)
    q[..., 0] = 8.0
    k = np.random.default_rng(0).standard_normal((1, c.S, 1, 64)).astype(np.float32) * 0.1
    k[0, :, 0, 0] = np.arange(c.S) * 0.5
    kb, c.kd = _blocks(f32_to_bf16_bits(k))
    c.k = torch.from_numpy(_poison(kb, c.lens, 64)).to(dev)
    c.q = f32_to_bf16_bits(q)
    c.qd = to_dev_bf16(c.q, dev)
    got, lse = c.run(kvd, torch, dev, "f32", n_split=3)
    want, wl = c.want()
    # scores up to 350: fp32 sums of that size are off by 2^-24 * 350 * a few
    assert np.abs(got - want).max() < 1e-3 and np.abs(lse - wl).max() < 1e-3


def test_status_and_clamp():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(9, 8, 2, 128, [100, 64, 90], page=16, dev=dev)
    # one block of sequence 1 names no page: zero rows
    c.bt[1, 2] = 99999
    c.kd[1, 32:48] = c.vd[1, 32:48] = 0
    got, _ = c.run(kvd, torch, dev, "f32")
    assert int(c.status.item()) == kvd.STATUS_BAD_PAGE
    assert_close(got, c.want()[0], "f32", "bad page")
    # lengths past max_seq_len and below zero are clamped
    c = Case(9, 8, 2, 128, [100, 64, 90], dev=dev)
    c.lens = np.array([80, 64, 0], np.int32)
    c.lens_d = torch.tensor([2 ** 31 - 1, 64, -5], dtype=torch.int32, device=dev)
    got, _ = c.run(kvd, torch, dev, "f32", max_len=80)
    assert int(c.status.item()) == kvd.STATUS_SEQ_LEN_CLAMPED
    assert_close(got, c.want()[0], "f32", "clamped")


def test_step_equals_append_then_attention():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    for T, page in ((1, 0), (1, 16), (4, 64)):
        c = Case(12 + T, 16, 4, 128, [300, 17, 100], T=T, page=page, dev=dev)
        r = np.random.default_rng(2)
        kn, vn = (to_dev_bf16(_rows(r, (c.B, T, 4, 128)), dev) for _ in range(2))
        pos = c.lens_d - T
        if c.T == 1:
            kn, vn = kn[:, 0], vn[:, 0]
        _, n = kvd.decode_plan_fp4(c.B, T, 16, 4, 128, c.S)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
        q = c.qd if T > 1 else c.qd[:, 0]
        k1, v1, k2, v2 = c.k.clone(), c.v.clone(), c.k.clone(), c.v.clone()
        a, b = torch.empty_like(q), torch.empty_like(q)
        kvd.kv_append_fp4(k1, v1, kn, vn, pos, block_table=c.bt)
        kvd.decode_fp4(q, k1, v1, c.lens_d, c.S, c.scale, a, block_table=c.bt, workspace=ws)
        kvd.decode_fp4(q, k2, v2, c.lens_d, c.S, c.scale, b, block_table=c.bt, workspace=ws, k_new=kn, v_new=vn, pos=pos)
        torch.cuda.synchronize()
        assert torch.equal(k1, k2) and torch.equal(v1, v2) and torch.equal(a, b)


def test_empty_batch():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=dev)
    k = kvd.alloc_cache_fp4(0, 2, 128, 64, device=dev)
    lens = torch.empty(0, dtype=torch.int32, device=dev)
    kvd.decode_fp4(q, k, k.clone(), lens, 64, 0.1, torch.empty_like(q))
    kvd.kv_quantize_fp4(torch.empty(0, 64, 2, 128, dtype=torch.bfloat16, device=dev), k, lens, 64)
    kvd.kv_append_fp4(k, k.clone(), q[:, :2], q[:, :2], lens)


def test_layers_together_in_a_graph():
    """A few layers' steps as a serving loop runs them: queries and keys turned and appended into a paged fp4
    cache, attention over it, several steps, captured once and replayed; against the oracle."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    B, Hq, Hkv, D, page, layers, steps = 3, 8, 2, 128, 16, 2, 20
    S, scale = 96, float(np.float32(128 ** -0.5))
    g = torch.Generator(device=dev).manual_seed(1)
    rope = kvd.RopeTable(64, scaling="linear", factor=2.0, device=dev)
    start = torch.tensor([40, 3, 11], dtype=torch.int32, device=dev)
    off = torch.tensor([0, 40, 43, 54], dtype=torch.int32, device=dev)
    nb = S // page
    bt = torch.randperm(B * nb, generator=g, device=dev).view(B, nb).int()
    k = [kvd.alloc_cache_fp4(B * nb, Hkv, D, page, device=dev) for _ in range(layers)]
    v = [kvd.alloc_cache_fp4(B * nb, Hkv, D, page, device=dev) for _ in range(layers)]
    zero = torch.zeros(B, dtype=torch.int32, device=dev)
    width = (Hq + 2 * Hkv) * D
    seen = [[[], []] for _ in range(layers)]  # rotated keys and values, [rows of the prompt] then steps

    def split(x):
        return (x[:, :Hq * D].view(-1, Hq, D), x[:, Hq * D:(Hq + Hkv) * D].view(-1, Hkv, D), x[:, (Hq + Hkv) * D:].view(-1, Hkv, D))
    prompt_pos = torch.cat([torch.arange(int(n), device=dev) for n in start]).int()
    for i in range(layers):  # the prompts, packed
        fused = torch.randn(54, width, generator=g, device=dev).bfloat16()
        _, kn, vn = split(fused)
        kvd.kv_append_fp4(k[i], v[i], kn, vn, zero, rope=rope, block_table=bt, row_offsets=off)
        kr = torch.empty_like(kn, memory_format=torch.contiguous_format)
        kvd.rope_apply(rope, kn, prompt_pos, kr)
        seen[i][0].append(kr.cpu())
        seen[i][1].append(vn.cpu())
    pos, lens = start.clone(), start + 1
    fused = [torch.zeros(B, width, device=dev, dtype=torch.bfloat16) for _ in range(layers)]
    q_rot = [torch.empty(B, Hq, D, device=dev, dtype=torch.bfloat16) for _ in range(layers)]
    out = [torch.empty(B, Hq, D, device=dev) for _ in range(layers)]
    ws = [torch.empty(max(kvd.decode_plan_fp4(B, 1, Hq, Hkv, D, S)[1], 1), device=dev, dtype=torch.uint8) for _ in range(layers)]

    def step():
        for i in range(layers):
            q, kn, vn = split(fused[i])
            kvd.kv_append_fp4(k[i], v[i], kn, vn, pos, rope=rope, q=q, q_out=q_rot[i], block_table=bt)
            kvd.decode_fp4(q_rot[i], k[i], v[i], lens, S, scale, out[i], block_table=bt, workspace=ws[i])
        pos.add_(1)
        lens.add_(1)
    draws = [[torch.randn(B, width, generator=g, device=dev).bfloat16() for _ in range(layers)] for _ in range(steps)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    for s in range(steps):
        for i in range(layers):
            fused[i].copy_(draws[s][i])
        at = pos.clone()
        if s == 0:
            with torch.cuda.stream(side):
                side.wait_stream(torch.cuda.default_stream())
                step()
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        for i in range(layers):
            q, kn, vn = split(draws[s][i])
            kr, qr = torch.empty(B, Hkv, D, device=dev, dtype=torch.bfloat16), torch.empty(B, Hq, D, device=dev, dtype=torch.bfloat16)
            kvd.rope_apply(rope, kn, at, kr)
            kvd.rope_apply(rope, q, at, qr)
            seen[i][0].append(kr.cpu())
            seen[i][1].append(vn.cpu())
            if s not in (0, 1, steps - 1):
                continue
            kd, vd = np.zeros((B, S, Hkv, D)), np.zeros((B, S, Hkv, D))
            L = (at + 1).cpu().numpy().astype(np.int32)
            for which, dst in ((0, kd), (1, vd)):
                for b in range(B):
                    lo, hi = int(off[b]), int(off[b + 1])
                    rows = torch.cat([seen[i][which][0][lo:hi]] + [x[b:b + 1] for x in seen[i][which][1:]])
                    assert rows.shape[0] == L[b]
                    dst[b, :L[b]] = oracle.dequantize_fp4(*oracle.quantize_fp4(bf16_tensor_bits(rows)))
            want, _ = oracle.decode_attention_f64kv(bf16_tensor_bits(qr), kd, vd, L, scale)
            assert_close(out[i].cpu().numpy().astype(np.float64), want, "f32", f"layer {i} step {s}")


def test_two_streams():
    """Two steps at once on two streams, each with its own workspace, give what they give alone."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    cs = [Case(20 + i, 32, 8, 128, [2000, 1500, 999], dev=dev) for i in range(2)]
    ws = [torch.empty(kvd.decode_plan_fp4(c.B, 1, 32, 8, 128, c.S)[1] + 1, dtype=torch.uint8, device=dev) for c in cs]
    alone = []
    for c, w in zip(cs, ws):
        out = torch.empty_like(c.qd)
        kvd.decode_fp4(c.qd, c.k, c.v, c.lens_d, c.S, c.scale, out, workspace=w)
        torch.cuda.synchronize()
        alone.append(out)
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [torch.zeros_like(c.qd) for c in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, w, o, s in zip(cs, ws, outs, streams):
            kvd.decode_fp4(c.qd, c.k, c.v, c.lens_d, c.S, c.scale, o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for a, o in zip(alone, outs))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 7), (3, 4), (3, 7), (4, 8), (5, 9), (7, 7)])
def test_every_number_of_column_tiles(D, T, G):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(D + T * G, 2 * G, 2, D, [290, 5, 0, 65], T=T, dev=dev)
    for dtype in ("bf16", "f32"):
        c.check(kvd, torch, dev, dtype)
        c.check(kvd, torch, dev, dtype, n_split=3)


def test_most_query_rows_and_no_tokens():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(3, 64, 1, 64, [100, 64, 1], T=64, dev=dev)
    c.check(kvd, torch, dev, "bf16")
    c.lens[:] = 0
    c.lens_d.zero_()
    c.check(kvd, torch, dev, "f32", max_len=0)


def test_offsets_past_32_bits():
    """Blocks further than 4 GB into a cache, by sequence, by page and within one sequence; two sequences with a
    page in common. The long sequence's first rows are zero: each adds 1 to the sum."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    D, BLK, n = 256, 9 * 256 + 16, 1 << 20
    big = [torch.zeros(3 * n, BLK, dtype=torch.uint8, device=dev) for _ in range(2)]  # 7.3 GB each
    c = Case(31, 8, 1, D, [1, 3, 500], dev=dev)
    small = [c.k, c.v]
    c.k, c.v = (x.view(3, 1, n, BLK) for x in big)
    for x, s in zip((c.k, c.v), small):
        x[:, :, :s.shape[2]] = s
    c.check(kvd, torch, dev, "f32")
    # an append to the last block of the last sequence, and the bulk conversion to the same place
    g = torch.Generator(device=dev).manual_seed(2)
    kn, vn = (torch.randn(3, 1, D, generator=g, device=dev).bfloat16() for _ in range(2))
    kvd.kv_append_fp4(c.k, c.v, kn, vn, torch.tensor([600, 600, 16 * n - 1], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    for x, new in ((c.k, kn), (c.v, vn)):
        want, _ = _blocks(bf16_tensor_bits(new).reshape(3, 1, 1, D).repeat(16, 1))
        for b, blk in ((1, 600 // 16), (2, n - 1)):
            w = [a[0, 0, 0] for a in oracle.unpack_fp4(want[b:b + 1], D)]
            got = [a[0, 0] for a in oracle.unpack_fp4(x[b, :, blk:blk + 1][None].cpu().numpy(), D)]
            at = 8 if b == 1 else 15
            assert all(np.array_equal(p[at], q) for p, q in zip(got, w))
            assert not any(np.delete(p, at, 0).any() for p in got)
    # pages at the end of the pool
    c = Case(32, 8, 1, D, [300, 290], page=16, dev=dev)
    c.bt[1, :5] = c.bt[0, :5]
    c.kd[1, :80], c.vd[1, :80] = c.kd[0, :80], c.vd[0, :80]
    m = c.k.shape[0]
    for x, s in zip(big, (c.k, c.v)):
        x[3 * n - m:] = s.view(m, BLK)
    c.k, c.v = (x.view(3 * n, 1, 1, BLK) for x in big)
    c.bt += 3 * n - m
    c.check(kvd, torch, dev, "f32")
    # one sequence: scores up to 256 * 25 * 8 / 16, each within 256 * 25 / 2 * 2^-24 < 2e-4, so the weights too, and
    # the outputs of size up to 5 within twice that
    for x in big:
        x.zero_()
    c = Case(33, 8, 1, D, [512], dev=dev)
    L = 48 * n - 3
    for x, s in zip(big, (c.k, c.v)):
        x[3 * n - 32:] = s.view(32, BLK)
    out, lse = torch.empty(1, 8, D, device=dev), torch.empty(1, 8, device=dev)
    _, nb = kvd.decode_plan_fp4(1, 1, 8, 1, D, L)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    k, v = (x.view(1, 1, 3 * n, BLK) for x in big)
    kvd.decode_fp4(c.qd[:, 0], k, v, torch.tensor([L], dtype=torch.int32, device=dev), L, 0.5, out, workspace=ws, lse=lse)
    torch.cuda.synchronize()
    q = bf16_bits_to_f32(c.q)[0, 0].astype(np.float64)
    s = 0.5 * q @ c.kd[0, :509, 0].T
    e = np.exp(s)
    total = e.sum(1) + (L - 509)
    assert np.abs(lse.cpu().numpy()[0] - np.log(total)).max() < 3e-4
    assert np.abs(out.cpu().numpy()[0] - (e @ c.vd[0, :509, 0]) / total[:, None]).max() < 2e-3
    assert (e.sum(1) > (L - 509)).any()  # the end of the sequence matters
    # rows of a bf16 cache past 4 GB, to blocks and back
    del c, big, k, v
    S = 1 << 23
    rows = torch.empty(2, S, 1, D, dtype=torch.bfloat16, device=dev)
    rows[1, :40] = torch.randn(40, 1, D, generator=g, device=dev).bfloat16()
    want, back = _blocks(np.pad(bf16_tensor_bits(rows[1, :40]), ((0, 8), (0, 0), (0, 0)))[None])
    lens = torch.tensor([0, 40], dtype=torch.int32, device=dev)
    blocks = kvd.alloc_cache_fp4(2, 1, D, S, device=dev)
    kvd.kv_quantize_fp4(rows, blocks, lens, S)
    rows[1, :40] = 0
    kvd.kv_read_fp4(blocks, rows, lens, S)
    torch.cuda.synchronize()
    assert np.array_equal(rows[1, :40].double().cpu().numpy(), back[0, :40])


@pytest.mark.parametrize("D,Hkv", [(64, 1), (64, 2), (64, 3), (128, 1), (128, 2), (256, 1)])
def test_quantize_and_read_few_heads(D, Hkv):
    """Few heads and many blocks: a CTA takes several blocks."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(D + Hkv)
    B, S = 40, 2080
    bits = _rows(r, (B, S, Hkv, D), 12.0)
    lens = r.integers(0, S, B).astype(np.int32)
    lens[[0, 3, 4, 5, 39]] = [S, 0, 1, 16, 17]
    blocks = torch.full((B, Hkv, S // 16 + 3, 9 * D + 16), 0x5a, dtype=torch.uint8, device=dev)
    kvd.kv_quantize_fp4(to_dev_bf16(bits, dev), blocks, torch.from_numpy(lens).to(dev), S)
    torch.cuda.synchronize()
    want, rows = _blocks(bits)
    old = [a.copy() for a in oracle.unpack_fp4(np.full((B, Hkv, S // 16 + 3, 9 * D + 16), 0x5a, np.uint8), D)]
    new = oracle.unpack_fp4(want, D)
    exp = np.full((B, S, Hkv, D), 3.0)
    for b in range(B):
        for o, n in zip(old, new):
            o[b, :, :lens[b]] = n[b, :, :lens[b]]
        exp[b, :lens[b]] = rows[b, :lens[b]]
    assert np.array_equal(blocks.cpu().numpy(), oracle.pack_fp4(*old))
    out = torch.full((B, S, Hkv, D), 3.0, dtype=torch.bfloat16, device=dev)
    ld = torch.from_numpy(lens).to(dev)
    kvd.kv_read_fp4(blocks, out, ld, S)
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), exp)
    # pages of 32 tokens, one of them unnamed
    nb = S // 32
    table = torch.randperm(B * nb + 1, device=dev)[:B * nb].view(B, nb).int()
    pool = torch.zeros(B * nb + 1, Hkv, 2, 9 * D + 16, dtype=torch.uint8, device=dev)
    pool[table.long()] = blocks[:, :, :2 * nb].reshape(B, Hkv, nb, 2, -1).transpose(1, 2).contiguous()
    table[0, 7] = -1
    exp[0, 7 * 32:8 * 32] = 0
    out.fill_(3.0)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kvd.kv_read_fp4(pool, out, ld, S, block_table=table, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvd.STATUS_BAD_PAGE
    assert np.array_equal(out.double().cpu().numpy(), exp)


@pytest.mark.parametrize("D,Hkv", [(64, 19), (128, 19), (256, 5), (128, 8)])
def test_quantize_and_read_few_blocks(D, Hkv):
    """Few blocks and many heads: several CTAs share a block's heads."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    bits = _rows(np.random.default_rng(D + Hkv), (3, 64, Hkv, D), 12.0)
    lens = np.array([64, 0, 23], np.int32)
    blocks = torch.full((3, Hkv, 4, 9 * D + 16), 0x5a, dtype=torch.uint8, device=dev)
    ld = torch.from_numpy(lens).to(dev)
    kvd.kv_quantize_fp4(to_dev_bf16(bits, dev), blocks, ld, 64)
    out = torch.full((3, 64, Hkv, D), 3.0, dtype=torch.bfloat16, device=dev)
    kvd.kv_read_fp4(blocks, out, ld, 64)
    torch.cuda.synchronize()
    want, rows = _blocks(bits)
    old = [a.copy() for a in oracle.unpack_fp4(np.full((3, Hkv, 4, 9 * D + 16), 0x5a, np.uint8), D)]
    exp = np.full((3, 64, Hkv, D), 3.0)
    for b in range(3):
        for o, n in zip(old, oracle.unpack_fp4(want, D)):
            o[b, :, :lens[b]] = n[b, :, :lens[b]]
        exp[b, :lens[b]] = rows[b, :lens[b]]
    assert np.array_equal(blocks.cpu().numpy(), oracle.pack_fp4(*old))
    assert np.array_equal(out.double().cpu().numpy(), exp)


def test_two_graphs_share_a_workspace():
    """Two captured calls of different shapes over one workspace, replayed in turn with new lengths and queries in place."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    cases = [Case(41, 16, 2, 128, [300, 0, 129], dev=dev), Case(42, 48, 1, 256, [900, 17], page=16, dev=dev)]
    need = max(kvd.decode_plan_fp4(c.B, 1, c.Hq, c.Hkv, c.D, c.S)[1] for c in cases)
    ws = torch.full((need,), 0xa5, dtype=torch.uint8, device=dev)
    outs = [torch.empty(c.B, c.Hq, c.D, device=dev) for c in cases]
    graphs = []
    for c, o in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvd.decode_fp4(c.qd[:, 0], c.k, c.v, c.lens_d, c.S, c.scale, o, block_table=c.bt, workspace=ws)
        graphs.append(g)
    for shrink in (0, 1, 5):
        for c in cases:
            c.lens = np.maximum(c.lens - shrink, 0).astype(np.int32)
            c.lens_d.copy_(torch.from_numpy(c.lens))
            c.qd.copy_(c.qd.flip(2))
            c.q = np.ascontiguousarray(c.q[:, :, ::-1])
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            assert_close(o.cpu().numpy().astype(np.float64), c.want()[0][:, 0], "f32", "graph")


def _tiled(first, rest, n, dev):
    """Blocks [1, 1, n / 16, ...]: 16 of `first`, then `rest`."""
    import torch
    f, r = (torch.from_numpy(x).to(dev) for x in (first, rest))
    return torch.cat([f.expand(16, -1), r.expand(n // 16 - 16, -1)]).contiguous()[None, None]


@pytest.mark.parametrize("gap", [23.6, 25.4, 31.0])
@pytest.mark.parametrize("rows,D", [(8, 64), (40, 64), (8, 128), (24, 128), (8, 256), (48, 256)])
def test_many_light_tokens_beside_heavy_ones(rows, D, gap):
    """16 tokens, one in each of the first 16 blocks, score `gap` powers of two above n like ones and have V rows of
    one value in the first column, so that an output in the others is the light tokens' share of the sum times their V row.

    Tolerance, relative to that: a weight of 2^-g of the heaviest term, g = gap, is off by 2^-12 or an absolute 2^-37 of that
    term (bf16 output), 2^-22 or 2^-48 of it (fp32 output); scores of 32 at most are off by 2^-22 of themselves in all
    (three roundings and scale * log2(e)). An output is summed from n / 16 / groups products of 16 tokens, twice that for fp32
    output, where the 8 / WD groups are 2 at the least, each sum cut to 24 bits (2^-23, all terms of one sign); the weights' sum from n / 64 to
    a thread, each rounded (2^-24). bf16 outputs half a step, 2^-8."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    n = 1 << 16
    k, v = np.zeros((2, 16, D), np.float32), np.ones((2, 16, D), np.float32)
    v *= 1.0 + np.arange(D, dtype=np.float32) / D
    k[0, 0, 0], v[0, 0, 1:] = 1.0, 0.0
    kc, vc = (oracle.quantize_fp4(f32_to_bf16_bits(x)) for x in (k, v))
    kb, vb = (oracle.pack_fp4(*x)[:, 0] for x in (kc, vc))
    kd, vd = (oracle.dequantize_fp4(*x) for x in (kc, vc))
    scale = float(np.float32(D ** -0.5))
    q = np.zeros((1, rows, D), np.float32)
    q[..., 0] = gap * math.log(2) / (scale * kd[0, 0, 0])
    q = f32_to_bf16_bits(q)
    g = scale * float(bf16_bits_to_f32(q)[0, 0, 0]) * kd[0, 0, 0]  # nats
    light = n - 16
    share = light / (16 * math.exp(g) + light)
    want = share * vd[1, 1, 1:]
    octaves = g / math.log(2)
    kt, vt = _tiled(kb[0], kb[1], n, dev), _tiled(vb[0], vb[1], n, dev)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    for n_split in (1, 0):
        _, nb = kvd.decode_plan_fp4(1, 1, rows, 1, D, n, 0, n_split)
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
        for dt, parts, tol in ((torch.bfloat16, 1, max(2.0 ** -12, 2.0 ** (octaves - 37)) + 2.0 ** -8),
                               (torch.float32, 2, max(2.0 ** -22, 2.0 ** (octaves - 48)))):
            tol += 2.0 ** -22 * 32 + parts * n / 32 * 2.0 ** -23 + n / 64 * 2.0 ** -24
            out, lse = torch.empty(1, rows, D, dtype=dt, device=dev), torch.empty(1, rows, device=dev)
            kvd.decode_fp4(to_dev_bf16(q, dev), kt, vt, lens, n, scale, out, workspace=ws, n_split=n_split, lse=lse)
            torch.cuda.synchronize()
            rel = np.abs(out[0, :, 1:].double().cpu().numpy() / want - 1).max()
            assert rel <= tol, (n_split, dt, rel, tol)
            assert np.abs(lse.cpu().numpy() - math.log(16 * math.exp(g) + light)).max() < 1e-4


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (40, 1, 64), (24, 1, 128), (48, 1, 256)])
def test_one_large_value(Hq, Hkv, D):
    """A token whose V row is 2^16 in one column and zero elsewhere takes no bits from the other tokens' weights: their
    terms, 2^-15 of its in V's exponent and 2^-11 at the least in the scores, stay above 2^-26 of the largest, so the other
    columns are as exact as ever (test_magnitudes' bounds, relative to the terms that make up an output)."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(51, Hq, Hkv, D, [300, 417], dev=dev)
    r = np.random.default_rng(6)
    v = bf16_bits_to_f32(_rows(r, (c.B, c.S, Hkv, D))).copy()
    v[:, 3::40] = 0
    v[:, 3::40, :, 5] = 2.0 ** 16
    vb, c.vd = _blocks(f32_to_bf16_bits(v))
    c.v = torch.from_numpy(_poison(vb, c.lens, D)).to(dev)
    other = np.arange(D) != 5
    want, wl = c.want()
    mag, _ = oracle.decode_attention_f64kv(c.q[:, 0], c.kd, np.abs(c.vd), c.lens, c.scale)
    for n_split in (0, 1):
        got, lse = c.run(kvd, torch, dev, "f32", n_split=n_split)
        err = np.abs(got[:, 0] - want[:, 0])
        assert (err <= 1e-4 * mag).all(), (err / mag).max()
        assert np.abs(lse - wl).max() < 1e-4
        got, _ = c.run(kvd, torch, dev, "bf16", n_split=n_split)
        err = np.abs(got[:, 0] - want[:, 0]) - np.abs(want[:, 0]) * 2.0 ** -8
        assert (err <= (1e-4 + 2.0 ** -11) * mag).all(), (err / mag)[..., other].max()


@pytest.mark.parametrize("up", [124, -126])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (24, 1, 64), (48, 1, 256)])
def test_keys_at_the_ends_of_the_range(Hq, Hkv, D, up):
    """Keys near the largest and the smallest bf16 numbers with queries as far the other way: ordinary scores."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(61, Hq, Hkv, D, [200, 333], dev=dev)
    x = bf16_bits_to_f32(_rows(np.random.default_rng(7), (c.B, c.S, Hkv, D)))
    kb, c.kd = _blocks(f32_to_bf16_bits((np.clip(x, -3.5, 3.5).astype(np.float64) * 2.0 ** up).astype(np.float32)))
    c.k = torch.from_numpy(_poison(kb, c.lens, D)).to(dev)
    c.q = f32_to_bf16_bits((np.clip(bf16_bits_to_f32(c.q), -3.5, 3.5).astype(np.float64) * 2.0 ** -up).astype(np.float32))
    c.qd = to_dev_bf16(c.q, dev)
    for dtype in ("f32", "bf16"):
        c.check(kvd, torch, dev, dtype)


@pytest.mark.parametrize("up", [-118, 100])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (40, 1, 64), (24, 1, 128), (48, 1, 256)])
def test_values_at_the_ends_of_the_range(Hq, Hkv, D, up):
    """V rows near the smallest and far towards the largest numbers: outputs as exact, relative to their terms, as of ordinary
    rows (test_magnitudes' bounds; below 2^-126 half a step of bf16 is 2^-134, of fp32 2^-150)."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(71, Hq, Hkv, D, [300, 17, 500], dev=dev)
    x = bf16_bits_to_f32(_rows(np.random.default_rng(8), (c.B, c.S, Hkv, D))).astype(np.float64)
    vb, c.vd = _blocks(f32_to_bf16_bits((x * 2.0 ** up).astype(np.float32)))
    c.v = torch.from_numpy(_poison(vb, c.lens, D)).to(dev)
    want, _ = c.want()
    mag, _ = oracle.decode_attention_f64kv(c.q[:, 0], c.kd, np.abs(c.vd), c.lens, c.scale)
    for n_split in (0, 1, 5):
        got, _ = c.run(kvd, torch, dev, "f32", n_split=n_split)
        assert (np.abs(got[:, 0] - want[:, 0]) <= 1e-4 * mag + 2.0 ** -148).all()
        got, _ = c.run(kvd, torch, dev, "bf16", n_split=n_split)
        assert (np.abs(got[:, 0] - want[:, 0]) <= (1e-4 + 2.0 ** -10) * mag + np.abs(want[:, 0]) * 2.0 ** -8 + 2.0 ** -134).all()


@pytest.mark.parametrize("Hq,Hkv,D,T,page", [(8, 1, 128, 1, 0), (32, 8, 128, 5, 16), (48, 1, 256, 1, 64), (40, 2, 64, 1, 16)])
def test_repeats_itself(Hq, Hkv, D, T, page):
    """The same call gives the same bits, whatever the workspace held."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(81, Hq, Hkv, D, [2300, 1, 700, 4001], T=T, page=page, dev=dev)
    _, n = kvd.decode_plan_fp4(c.B, T, Hq, Hkv, D, c.S)
    for dt in (torch.bfloat16, torch.float32):
        first = None
        for i in range(20):
            ws = torch.full((n + 1,), 17 * i % 256, dtype=torch.uint8, device=dev)
            out, lse = torch.empty(c.B, T, Hq, D, dtype=dt, device=dev), torch.empty(c.B, T, Hq, device=dev)
            kvd.decode_fp4(c.qd, c.k, c.v, c.lens_d, c.S, c.scale, out, block_table=c.bt, workspace=ws, lse=lse)
            torch.cuda.synchronize()
            if first is None:
                first = out, lse
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_quantizers_at_the_ends_of_the_range(D):
    """Rows from below the smallest row exponent to the largest numbers, rows of one large and otherwise tiny blocks of 16 columns: the
    bulk quantizer and the append give the oracle's bytes, and the reader the values, where bf16 holds them."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(D)
    B, S, Hkv = 2, 272, 3
    x = r.uniform(-1, 1, (B, S, Hkv, D))
    x *= np.exp2(np.linspace(-133, 127.9, S))[None, :, None, None]
    tiny = np.exp2(r.integers(-24, 1, (S, D // 16)).astype(np.float64)).repeat(16, -1)
    x[1] *= tiny[:, None, :]
    x[1, :, :, :16] *= 1.0 / tiny[:, None, :16]  # the first block keeps the row's size
    bits = f32_to_bf16_bits(x.astype(np.float32))
    assert (np.abs(bf16_bits_to_f32(bits)) < np.inf).all()
    want, rows = _blocks(bits)
    xd, lens = to_dev_bf16(bits, dev), torch.full((B,), S, dtype=torch.int32, device=dev)
    blocks = kvd.alloc_cache_fp4(B, Hkv, D, S, device=dev)
    kvd.kv_quantize_fp4(xd, blocks, lens, S)
    k, v = (kvd.alloc_cache_fp4(B, Hkv, D, S, device=dev) for _ in range(2))
    kvd.kv_append_fp4(k, v, xd, xd, torch.zeros(B, dtype=torch.int32, device=dev))
    k1, v1 = (kvd.alloc_cache_fp4(B, Hkv, D, S, device=dev) for _ in range(2))
    for t in range(S):  # a token at a time takes the other kernel
        kvd.kv_append_fp4(k1, v1, xd[:, t], xd[:, t], torch.full((B,), t, dtype=torch.int32, device=dev))
    out = torch.empty(B, S, Hkv, D, dtype=torch.bfloat16, device=dev)
    kvd.kv_read_fp4(blocks, out, lens, S)
    torch.cuda.synchronize()
    for got in (blocks, k, v, k1, v1):
        g = got.cpu().numpy()
        if not np.array_equal(g, want):
            a, b = oracle.unpack_fp4(g, D), oracle.unpack_fp4(want, D)
            raise AssertionError([np.argwhere(p != q)[:5].tolist() for p, q in zip(a, b)])
    held = bf16_bits_to_f32(f32_to_bf16_bits(np.where(np.abs(rows) < 3.3e38, rows, 0.0).astype(np.float32))).astype(np.float64) == rows
    assert held.mean() > 0.9 and np.array_equal(out.double().cpu().numpy()[held], rows[held])


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (24, 1, 128)])
def test_more_sequences_than_threads(Hq, Hkv, D):
    """A thread of the schedule's scan takes several sequences, many of them empty."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(9)
    lens = r.integers(0, 49, 1000) * (r.random(1000) < 0.6)
    lens[[0, 1, 500, 999]] = [0, 0, 300, 0]
    c = Case(91, Hq, Hkv, D, lens.tolist(), dev=dev)
    for n in (0, 1, 151, 3000):
        c.check(kvd, torch, dev, "f32", n_split=n)
    c.check(kvd, torch, dev, "bf16")


@pytest.mark.parametrize("Hq,Hkv,D,T", [(8, 2, 128, 1), (48, 1, 256, 1), (6, 3, 64, 4)])
def test_pages_longer_than_a_tile(Hq, Hkv, D, T):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(95, Hq, Hkv, D, [1100, 0, 511, 512, 513, T], T=T, page=512, dev=dev)
    c.check(kvd, torch, dev, "f32")
    c.check(kvd, torch, dev, "bf16", n_split=7)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (24, 1, 64), (48, 1, 256)])
@pytest.mark.parametrize("kup,qup", [(124, 100), (124, -100), (-124, 100), (-124, -124), (0, 124)])
def test_keys_that_queries_do_not_meet(Hq, Hkv, D, kup, qup):
    """Keys in the even columns, queries in the odd ones, however large or small: every score is zero, the output the mean."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    c = Case(67, Hq, Hkv, D, [200, 333], dev=dev)
    x = np.clip(bf16_bits_to_f32(_rows(np.random.default_rng(7), (c.B, c.S, Hkv, D))), -3.5, 3.5).astype(np.float64)
    x[..., 1::2] = 0
    kb, c.kd = _blocks(f32_to_bf16_bits((x * 2.0 ** kup).astype(np.float32)))
    c.k = torch.from_numpy(_poison(kb, c.lens, D)).to(dev)
    q = np.clip(bf16_bits_to_f32(c.q), -3.5, 3.5).astype(np.float64)
    q[..., 0::2] = 0
    c.q = f32_to_bf16_bits((q * 2.0 ** qup).astype(np.float32))
    c.qd = to_dev_bf16(c.q, dev)
    for dtype in ("f32", "bf16"):
        c.check(kvd, torch, dev, dtype)
