"""Rotary positions and the rotating appends on the GPU: rope_apply against
float64 (phases in exact integers), the appends bit for bit against rope_apply
followed by the oracle's placement and quantizers.

Tolerance of rope_apply, per element, for the pair (a, b) and factor f: the
phase's 24 bits move the angle by at most 2^-25 pi, sincospif is within 2 units in
the last place (2^-23 of a value up to 1), the factor's product, the inner product
and the fused sum round once each (2^-24): |f| (|a| + |b|) (2^-25 pi + 2^-23 +
3 * 2^-24) < 4.0e-7 |f| (|a| + |b|), and a bf16 result half a step of itself more."""
import numpy as np
import pytest

import oracle
from gpu_helpers import bf16_tensor_bits, cuda_or_skip
from workloads import bf16_bits_to_f32

pytestmark = pytest.mark.gpu


def _check(got, x, ph, factor, inter, dtype):
    import torch
    want = oracle.rope(x, ph, factor, inter)
    R = 2 * ph.shape[1]
    pair = np.zeros_like(x)
    ia, ib = (np.arange(0, R, 2), np.arange(1, R, 2)) if inter else (np.arange(R // 2), np.arange(R // 2, R))
    pair[..., ia] = pair[..., ib] = np.abs(x[..., ia]) + np.abs(x[..., ib])
    tol = 4.0e-7 * factor * pair
    if dtype == torch.bfloat16:
        tol = tol + np.abs(want) * (torch.finfo(dtype).eps / 2) * (1 + 1e-6) + 1e-40
    bad = np.abs(got - want) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want)[bad].max()))


@pytest.mark.parametrize("D,R,H,N,inter", [
    (128, 128, 32, 64, False), (128, 64, 40, 7, True), (64, 64, 1, 1, False), (256, 256, 48, 3, True), (80, 16, 5, 33, False),
    (80, 80, 2, 9, True), (72, 48, 3, 11, False), (128, 16, 8, 650, False), (1024, 256, 1, 5, False), (192, 112, 7, 5000, True),
])
def test_rope_apply(D, R, H, N, inter):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    rope = kvd.RopeTable(R, scaling="parts", factor=16.0, original_len=4096, interleaved=inter, device=dev)
    turns = rope.turns.cpu().numpy().view(np.uint64)
    g = torch.Generator(device=dev).manual_seed(D + N)
    pos = torch.randint(-5, 1 << 20, (N,), generator=g, device=dev).int()
    edge = torch.tensor([0, -1, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32, device=dev)[:N]
    pos[:edge.numel()] = edge
    ph = oracle.rope_phases(pos.cpu().numpy(), turns)
    for idt in (torch.bfloat16, torch.float32):
        x = torch.randn(N, H, D, generator=g, device=dev).to(idt)
        x[0, 0, :4] = 0
        for odt in (torch.bfloat16, torch.float32):
            out = torch.full_like(x, float("nan"), dtype=odt)
            kvd.rope_apply(rope, x, pos, out)
            torch.cuda.synchronize()
            _check(out.double().cpu().numpy(), x.double().cpu().numpy(), ph, rope.factor, inter, odt)
            if R < D and odt == idt:  # the other columns are copied
                assert torch.equal(out[..., R:], x[..., R:])
        y = x.clone()  # in place: the same bits
        out = torch.empty_like(x)
        kvd.rope_apply(rope, x, pos, out)
        kvd.rope_apply(rope, y, pos, y)
        torch.cuda.synchronize()
        assert torch.equal(y, out)


def test_rope_apply_strided_and_turned_back():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    rope = kvd.RopeTable(64, device=dev)
    N, H, D = 37, 6, 128
    g = torch.Generator(device=dev).manual_seed(5)
    wide = torch.randn(N, 10 * D, generator=g, device=dev)
    x = wide[:, 2 * D:8 * D].view(N, H, D)
    pos = torch.randint(0, 1 << 17, (N,), generator=g, device=dev).int()
    keep = wide.clone()
    ref = torch.empty(N, H, D, device=dev)
    kvd.rope_apply(rope, x.contiguous(), pos, ref)
    outw = torch.full((N, 9 * D), 7.0, device=dev)
    out = outw[:, D:7 * D].view(N, H, D)
    kvd.rope_apply(rope, x, pos, out)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(wide, keep)
    assert (outw[:, :D] == 7).all() and (outw[:, 7 * D:] == 7).all()
    kvd.rope_apply(rope, x, pos, x)  # a slice in place: its neighbours stay
    torch.cuda.synchronize()
    assert torch.equal(x, ref) and torch.equal(wide[:, :2 * D], keep[:, :2 * D]) and torch.equal(wide[:, 8 * D:], keep[:, 8 * D:])
    # [B, T, H, D] is B * T rows; negative positions turn back
    back = torch.empty(1, N, H, D, device=dev)
    kvd.rope_apply(rope, ref.view(1, N, H, D), -pos.view(1, N), back)
    torch.cuda.synchronize()
    # two turns, each within 4.0e-7 (|a| + |b|) with |a|, |b| <= 6
    assert (back[0] - keep[:, 2 * D:8 * D].view(N, H, D)).abs().max() < 2 * 4.0e-7 * 12


def test_what_is_not_turned_is_copied_bit_by_bit():
    """Every bf16 pattern, NaN payloads among them, in the columns past rotary_dim and in the value rows."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    bits = torch.arange(65536, dtype=torch.int32, device=dev).to(torch.int16)
    rope = kvd.RopeTable(16, device=dev)
    x = torch.zeros(586, 1, 128, dtype=torch.int16, device=dev)
    x.view(586, 128)[:, 16:] = torch.nn.functional.pad(bits, (0, 586 * 112 - 65536)).view(586, 112)
    out = torch.zeros_like(x)
    pos = torch.arange(586, dtype=torch.int32, device=dev)
    kvd.rope_apply(rope, x.view(torch.bfloat16), pos, out.view(torch.bfloat16))
    v = bits.view(512, 1, 128)
    kc = torch.zeros(1, 512, 1, 128, dtype=torch.int16, device=dev)
    vc = torch.zeros_like(kc)
    kvd.kv_append_rope(rope, kc.view(torch.bfloat16), vc.view(torch.bfloat16), torch.zeros_like(v).view(torch.bfloat16),
                       v.view(torch.bfloat16), torch.zeros(1, dtype=torch.int32, device=dev),
                       row_offsets=torch.tensor([0, 512], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert torch.equal(out[..., 16:], x[..., 16:]) and torch.equal(vc[0], v)


def test_rope_apply_refuses_views():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    rope = kvd.RopeTable(64, device=dev)
    x = torch.zeros(4, 8, 128, device=dev, dtype=torch.bfloat16)
    pos = torch.zeros(4, device=dev, dtype=torch.int32)
    bad = [lambda: kvd.rope_apply(rope, x.transpose(0, 1), pos, x), lambda: kvd.rope_apply(rope, x.half(), pos, x),
           lambda: kvd.rope_apply(rope, x, pos[:3], x), lambda: kvd.rope_apply(rope, x, pos.long(), x),
           lambda: kvd.rope_apply(rope, x, pos.cpu(), x), lambda: kvd.rope_apply(rope, x[..., :120], pos, x[..., :120]),
           lambda: kvd.rope_apply(rope, x[:, :, :32].contiguous(), pos, x[:, :, :32].contiguous()),
           lambda: kvd.rope_apply(kvd.RopeTable(64, device="cpu"), x, pos, x),
           lambda: kvd.rope_apply(rope, x, pos, x[:2])]
    for fn in bad:
        with pytest.raises((ValueError, TypeError, kvd.KvdError)):
            fn()


# ---------------------------------------------------------------------------
# the rotating appends
# ---------------------------------------------------------------------------

def _cache(kvd, torch, form, B, S, Hkv, D, page, dev, g):
    """(tensors by name, block table or None, bytes before): caches filled with a recognisable pattern."""
    lead = (B, S) if not page else (B * (S // page) + 2, page)
    bt = None
    if page:
        bt = torch.randperm(lead[0], generator=g, device=dev)[:B * (S // page)].view(B, S // page).int()
    t = {}
    for n in ("k", "v"):
        if form == "fp4":
            t[n] = torch.full((lead[0], Hkv, lead[1] // 16, 9 * D + 16), 0x5a, dtype=torch.uint8, device=dev)
        elif form == "bf16":
            t[n] = torch.full(lead + (Hkv, D), -3.0, dtype=torch.bfloat16, device=dev)
        else:
            t[n] = torch.full(lead + (Hkv, D), 85, dtype=torch.int8 if form == "int8" else torch.uint8, device=dev)
            t[n + "_scales"] = torch.full(lead + (Hkv,), -1.0, device=dev)
    return t, bt


def _expected(form, t, bt, S, page, k_bits, v_bits, seq, at):
    """numpy images of the cache tensors after rows (k_bits[n], v_bits[n]) go to position at[n] of sequence seq[n]."""
    e = {n: (bf16_tensor_bits(x) if x.dtype.is_floating_point and x.element_size() == 2 else x.cpu().numpy()).copy()
         for n, x in t.items()}
    table = None if bt is None else bt.cpu().numpy()
    for n, (b, p) in enumerate(zip(seq, at)):
        if p < 0 or p >= S:
            continue
        i, r = (b, p) if table is None else (table[b, p // page], p % page)
        for name, bits in (("k", k_bits[n]), ("v", v_bits[n])):
            if form == "bf16":
                e[name][i, r] = bits
            elif form == "fp4":
                codes, sb, exps = oracle.quantize_fp4(bits)
                H, D = codes.shape
                blk = e[name][i, :, r // 16]
                pad = lambda a: np.zeros((H, 16) + a.shape[1:], a.dtype)  # noqa: E731
                c16, s16, e16 = pad(codes), pad(sb), pad(exps)
                c16[:, r % 16], s16[:, r % 16], e16[:, r % 16] = codes, sb, exps
                new = oracle.pack_fp4(c16, s16, e16)[:, 0]
                m16 = [pad(a) for a in (codes, sb, exps)]
                m16[0][:, r % 16], m16[1][:, r % 16], m16[2][:, r % 16] = 15, 255, 255
                mask = oracle.pack_fp4(*m16)[:, 0]
                e[name][i, :, r // 16] = (blk & ~mask) | (new & mask)
            else:
                q = oracle.quantize_q8(bits) if form == "int8" else oracle.quantize_fp8(bits)
                e[name][i, r] = np.asarray(q[0]).view(e[name].dtype)
                e[name + "_scales"][i, r] = q[1]
    return e


def _same(t, e):
    import torch
    for n, x in t.items():
        got = bf16_tensor_bits(x) if x.dtype == torch.bfloat16 else x.cpu().numpy()
        bad = got != e[n]
        assert not bad.any(), (n, int(bad.sum()), np.argwhere(bad)[:5].tolist())


def _call(kvd, form, rope, t, *args, **kw):
    if form == "fp4":
        kvd.kv_append_fp4(t["k"], t["v"], *args, rope=rope, **kw)
    else:
        kvd.kv_append_rope(rope, t["k"], t["v"], *args, k_scales=t.get("k_scales"), v_scales=t.get("v_scales"), **kw)


@pytest.mark.parametrize("form", ["bf16", "int8", "fp8", "fp4"])
@pytest.mark.parametrize("D,R,inter,Hq,Hkv,page,T", [
    (128, 128, False, 32, 8, 0, 1), (128, 64, True, 8, 8, 16, 3), (64, 16, False, 6, 2, 32, 1), (64, 48, False, 5, 5, 16, 2),
    (256, 256, True, 48, 1, 64, 2), (256, 112, False, 3, 1, 0, 5),
])
def test_append_rope_uniform(form, D, R, inter, Hq, Hkv, page, T):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(D + R + T)
    B, S = 5, 128
    rope = kvd.RopeTable(R, scaling="wavelength", factor=8.0, original_len=64, interleaved=inter, device=dev)
    t, bt = _cache(kvd, torch, form, B, S, Hkv, D, page, dev, g)
    fused = torch.randn(B, T, (Hq + 2 * Hkv) * D, generator=g, device=dev).bfloat16()
    q = fused[..., :Hq * D].view(B, T, Hq, D)
    k = fused[..., Hq * D:(Hq + Hkv) * D].view(B, T, Hkv, D)
    v = fused[..., (Hq + Hkv) * D:].view(B, T, Hkv, D)
    k[1, 0, 0] = 0  # an all-zero head
    k[0, 0, 0] *= 1e-3
    pos = torch.tensor([0, 15, 61, S - T, 31], dtype=torch.int32, device=dev)
    positions = (pos[:, None] + torch.arange(T, device=dev, dtype=torch.int32)).contiguous()
    kr, qr = torch.empty(B, T, Hkv, D, device=dev, dtype=torch.bfloat16), torch.empty(B, T, Hq, D, device=dev, dtype=torch.bfloat16)
    kvd.rope_apply(rope, k, positions, kr)
    kvd.rope_apply(rope, q, positions, qr)
    torch.cuda.synchronize()
    seq = np.repeat(np.arange(B), T)
    want = _expected(form, t, bt, S, page, bf16_tensor_bits(kr).reshape(B * T, Hkv, D), bf16_tensor_bits(v).reshape(B * T, Hkv, D),
                     seq, positions.cpu().numpy().reshape(-1))
    q_out = torch.zeros_like(qr)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    before = fused.clone()
    _call(kvd, form, rope, t, k, v, pos, q=q, q_out=q_out, block_table=bt, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(fused, before)
    assert torch.equal(q_out, qr)
    _same(t, want)
    # queries turned in place in the fused rows, the cache as before
    _call(kvd, form, rope, t, k, v, pos, q=q, q_out=q, block_table=bt, status=status)
    torch.cuda.synchronize()
    assert torch.equal(q, qr) and torch.equal(k, before[..., Hq * D:(Hq + Hkv) * D].view(B, T, Hkv, D))
    _same(t, want)


@pytest.mark.parametrize("form,page", [("bf16", 32), ("int8", 0), ("fp8", 16), ("fp4", 16), ("fp4", 0)])
def test_append_rope_ragged(form, page):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    D, R, Hq, Hkv, S = 128, 64, 4, 2, 96
    lens = [0, 1, 17, 0, 40, 96, 3]
    B = len(lens)
    first = 2                       # rows before the first offset belong to nobody
    off = np.concatenate([[0], np.cumsum(lens)]) + first
    N = int(off[-1]) + 5            # nor do those behind the last
    g = torch.Generator(device=dev).manual_seed(11)
    rope = kvd.RopeTable(R, device=dev)
    t, bt = _cache(kvd, torch, form, B, S, Hkv, D, page, dev, g)
    q, k, v = (torch.randn(N, h, D, generator=g, device=dev).bfloat16() for h in (Hq, Hkv, Hkv))
    start = np.array([5, 7, 60, 3, 50, 0, S - 1])  # the last sequence runs over its end
    pos = torch.tensor(start, dtype=torch.int32, device=dev)
    seq = np.full(N, -1)
    at = np.full(N, -1)
    for b in range(B):
        seq[off[b]:off[b + 1]] = b
        at[off[b]:off[b + 1]] = start[b] + np.arange(lens[b])
    live = seq >= 0
    positions = torch.tensor(np.where(live, at, 0), dtype=torch.int32, device=dev)
    kr, qr = torch.empty_like(k), torch.empty_like(q)
    kvd.rope_apply(rope, k, positions, kr)
    kvd.rope_apply(rope, q, positions, qr)
    torch.cuda.synchronize()
    want = _expected(form, t, bt, S, page, bf16_tensor_bits(kr)[live], bf16_tensor_bits(v)[live], seq[live], at[live])
    q_out = torch.full_like(q, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    _call(kvd, form, rope, t, k, v, pos, q=q, q_out=q_out, block_table=bt, status=status,
          row_offsets=torch.tensor(off, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert int(status.item()) == kvd.STATUS_POS_OUT_OF_RANGE
    lt = torch.tensor(live, device=dev)
    assert torch.equal(q_out[lt], qr[lt]) and (q_out[~lt] == 9).all()
    _same(t, want)


@pytest.mark.parametrize("form", ["bf16", "fp4"])
def test_append_rope_bad_pages_and_positions(form):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    D, Hkv, S, page, B = 64, 3, 64, 16, 5
    g = torch.Generator(device=dev).manual_seed(4)
    rope = kvd.RopeTable(64, device=dev)
    t, bt = _cache(kvd, torch, form, B, S, Hkv, D, page, dev, g)
    bt[0, 1], bt[2, 0], bt[3, 3] = -1, t["k"].shape[0], 2 ** 30
    k, v = (torch.randn(B, Hkv, D, generator=g, device=dev).bfloat16() for _ in range(2))
    pos = torch.tensor([20, 63, 0, -1, 64], dtype=torch.int32, device=dev)
    kr = torch.empty_like(k)
    kvd.rope_apply(rope, k, pos, kr)
    torch.cuda.synchronize()
    want = _expected(form, t, bt, S, page, bf16_tensor_bits(kr)[1:2], bf16_tensor_bits(v)[1:2], [1], [63])
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    _call(kvd, form, rope, t, k, v, pos, block_table=bt, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvd.STATUS_POS_OUT_OF_RANGE | kvd.STATUS_BAD_PAGE
    _same(t, want)


def test_append_fp4_plain_and_many_rows():
    """No rotation, and enough rows for several tokens to a block."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    B, T, Hkv, D, S = 50, 64, 2, 64, 64
    g = torch.Generator(device=dev).manual_seed(8)
    t, _ = _cache(kvd, torch, "fp4", B, S, Hkv, D, 0, dev, g)
    k, v = (torch.randn(B, T, Hkv, D, generator=g, device=dev).bfloat16() for _ in range(2))
    pos = torch.zeros(B, dtype=torch.int32, device=dev)
    kvd.kv_append_fp4(t["k"], t["v"], k, v, pos)
    torch.cuda.synchronize()
    for n, x in (("k", k), ("v", v)):
        want = oracle.pack_fp4(*oracle.quantize_fp4(bf16_tensor_bits(x).transpose(0, 2, 1, 3)))
        assert np.array_equal(t[n].cpu().numpy(), want)


def test_rope_apply_to_other_columns_of_the_same_rows():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    rope = kvd.RopeTable(64, device=dev)
    N, H, D = 41, 3, 64
    g = torch.Generator(device=dev).manual_seed(6)
    wide = torch.randn(N, 2 * H * D, generator=g, device=dev).bfloat16()
    pos = torch.arange(N, dtype=torch.int32, device=dev)
    x, y = wide[:, :H * D].view(N, H, D), wide[:, H * D:].view(N, H, D)
    keep, ref = x.clone(), torch.empty(N, H, D, dtype=torch.bfloat16, device=dev)
    kvd.rope_apply(rope, keep, pos, ref)
    kvd.rope_apply(rope, x, pos, y)
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and torch.equal(x, keep)


def test_offsets_past_32_bits():
    """Rows further than 4 GB into a buffer or a cache turn as they do in a small one."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    rope = kvd.RopeTable(128, device=dev)
    g = torch.Generator(device=dev).manual_seed(9)
    N, H, D = (1 << 19) + 9, 32, 128
    x = torch.zeros(N, H, D, dtype=torch.bfloat16, device=dev)
    x[-9:] = torch.randn(9, H, D, generator=g, device=dev).bfloat16()
    last, pos = x[-9:].clone(), torch.arange(N, dtype=torch.int32, device=dev)
    ref = torch.empty_like(last)
    kvd.rope_apply(rope, last, pos[-9:].clone(), ref)
    kvd.rope_apply(rope, x, pos, x)
    torch.cuda.synchronize()
    assert torch.equal(x[-9:], ref) and not x[:-9].any()
    S = 1 << 23
    kc, vc = (torch.zeros(3, S, 1, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    k, v = (torch.randn(3, 1, D, generator=g, device=dev).bfloat16() for _ in range(2))
    at = torch.tensor([5, S - 1, S - 2], dtype=torch.int32, device=dev)
    kr = torch.empty_like(k)
    kvd.rope_apply(rope, k, at, kr)
    kvd.kv_append_rope(rope, kc, vc, k, v, at)
    torch.cuda.synchronize()
    i = torch.arange(3, device=dev)
    assert torch.equal(kc[i, at.long()], kr) and torch.equal(vc[i, at.long()], v)
    kc[i, at.long()] = 0
    vc[i, at.long()] = 0
    assert not kc.any() and not vc.any()


@pytest.mark.parametrize("D,R,H,inter", [(128, 128, 1, False), (64, 64, 1, True), (24, 16, 1, False), (16, 16, 1, True), (256, 240, 1, False),
                                         (80, 48, 3, False), (256, 256, 2, False), (64, 32, 4, True), (1024, 256, 1, True), (72, 64, 2, False)])
def test_many_short_rows(D, R, H, inter):
    """Rows of few heads go several to a warp when there are enough of them: the same bits as a few at a time."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    rope = kvd.RopeTable(R, interleaved=inter, device=dev)
    g = torch.Generator(device=dev).manual_seed(D + H)
    for N in (20003, 200003 if D <= 128 else 50003):
        wide = torch.randn(N, H * D + 8, generator=g, device=dev)
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (N,), generator=g, device=dev).int()
        for idt in (torch.bfloat16, torch.float32):
            x = wide.to(idt)[:, 8:].view(N, H, D)
            for odt in (torch.bfloat16, torch.float32):
                out, ref = (torch.full((N, H, D), float("nan"), dtype=odt, device=dev) for _ in range(2))
                kvd.rope_apply(rope, x, pos, out)
                for i in range(0, N, 5000):
                    kvd.rope_apply(rope, x[i:i + 5000], pos[i:i + 5000], ref[i:i + 5000])
                torch.cuda.synchronize()
                assert torch.equal(out, ref)
            full = wide.to(idt, copy=True)
            y = full[:, 8:].view(N, H, D)
            kvd.rope_apply(rope, y, pos, y)
            kvd.rope_apply(rope, x, pos, ref := torch.empty(N, H, D, dtype=idt, device=dev))
            torch.cuda.synchronize()
            assert torch.equal(y, ref) and torch.equal(full[:, :8], wide.to(idt)[:, :8])


@pytest.mark.parametrize("form,D,R,Hq,Hkv,page", [
    ("bf16", 64, 64, 2, 1, 16), ("bf16", 24, 16, 1, 1, 0), ("bf16", 256, 128, 1, 1, 64), ("int8", 128, 64, 2, 1, 0), ("fp8", 64, 48, 0, 2, 32),
    ("fp4", 64, 64, 0, 1, 16), ("fp4", 128, 128, 3, 1, 0), ("fp4", 256, 0, 0, 1, 32),
])
def test_append_many_short_rows(form, D, R, Hq, Hkv, page):
    """Likewise the appends: packed prompts in one call against a few sequences at a time, and uniform ones."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(D + Hq)
    rope = kvd.RopeTable(R, interleaved=Hq == 2, device=dev) if R else None
    B, S, G = 48, 2048, 4
    r = np.random.default_rng(D)
    lens = r.integers(0, 2000, B)
    lens[[0, 7, 8, 9, 20, B - 1]] = [0, 0, 0, 1, 2, 0]
    start = np.minimum(r.integers(0, 500, B), S - lens)
    start[[3, 30]] = [S - 100, -50]                       # past the end, before the start
    off = np.concatenate([[0], np.cumsum(lens)]) + 3
    N = int(off[-1]) + 70
    q, k, v = (torch.randn(N, max(h, 1), D, generator=g, device=dev).bfloat16() for h in (Hq, Hkv, Hkv))
    t, bt = _cache(kvd, torch, form, B, S, Hkv, D, page, dev, g)
    if page:
        bt[5, start[5] // page], bt[40, start[40] // page] = -1, t["k"].shape[0]  # pages that rows go to
    t2 = {n: x.clone() for n, x in t.items()}
    pos = torch.tensor(start, dtype=torch.int32, device=dev)
    outs = [torch.full_like(q, 9.0) for _ in range(2)]
    st = torch.zeros(2, dtype=torch.int32, device=dev)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    kw = lambda i, a, b: dict(q=q[a:b], q_out=outs[i][a:b]) if Hq else {}  # noqa: E731
    _call(kvd, form, rope, t, k, v, pos, row_offsets=i32(off), block_table=bt, status=st[:1], **kw(0, 0, N))
    for b in range(0, B, G):
        a, e = int(off[b]), int(off[b + G])
        if a == e:
            continue
        part = t2 if page else {n: x[b:b + G] for n, x in t2.items()}
        _call(kvd, form, rope, part, k[a:e], v[a:e], pos[b:b + G].contiguous(), row_offsets=i32(off[b:b + G + 1] - a),
              block_table=bt[b:b + G].contiguous() if page else None, status=st[1:], **kw(1, a, e))
    torch.cuda.synchronize()
    assert st.tolist() == [kvd.STATUS_POS_OUT_OF_RANGE | (kvd.STATUS_BAD_PAGE if page else 0)] * 2
    assert torch.equal(outs[0], outs[1])
    for n in t:
        assert torch.equal(t[n], t2[n]), n
    # uniform: T rows to each sequence
    T = 700
    a, pos = (x[:B * T].view(B, T, -1, D) for x in (k, v)), (pos.clamp(0, 400) + 3).contiguous()
    kk, vv = a
    if N >= B * T:
        _call(kvd, form, rope, t, kk, vv, pos, block_table=bt)
        for b in range(0, B, G):
            part = t2 if page else {n: x[b:b + G] for n, x in t2.items()}
            _call(kvd, form, rope, part, kk[b:b + G], vv[b:b + G], pos[b:b + G].contiguous(),
                  block_table=bt[b:b + G].contiguous() if page else None)
        torch.cuda.synchronize()
        for n in t:
            assert torch.equal(t[n], t2[n]), n


@pytest.mark.parametrize("inter", [False, True])
def test_cosines_and_sines(inter):
    """(a, b) = (1, 0) gives an angle's cosine and sine. The nearest quarter turn is taken off in integers, and what is left, x of at most
    1/4 in units of pi, is rounded to 24 bits: the angle is off by pi * 2^-27 at most (near the middle of a quarter
    turn by far less). The cosine 1 + u q(u), u = x^2 <= 1/16, |q| < 4.94: the sum's rounding 2^-25, q's and its first
    coefficient's 2^-22 each times u, u's own 2^-24 of u q < 0.31: 2^-25 + 2^-25 + 0.31 * 2^-24 + 2e-9 (the interpolation) < 8.1e-8. The
    sine x pi + x (...): the sum's 2^-24 of itself, the second term, below 0.08, 2^-22 of itself and the interpolation 2e-9 of x: 5 * 2^-24 of itself in all.
    Near a sine's or cosine's zero the small one of the two is that sine, and must be as exact relative to itself but for the angle."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    N, D = 200_000, 64
    rope = kvd.RopeTable(D, interleaved=inter, device=dev)
    turns = rope.turns.cpu().numpy().view(np.uint64)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (N,), device=dev, generator=torch.Generator(device=dev).manual_seed(1)).int()
    pos[:3] = torch.tensor([0, 1, -1], dtype=torch.int32)
    x = torch.zeros(N, 1, D, device=dev)
    ia, ib = (slice(0, D, 2), slice(1, D, 2)) if inter else (slice(0, D // 2), slice(D // 2, D))
    x[..., ia] = 1.0
    out = torch.empty_like(x)
    kvd.rope_apply(rope, x, pos, out)
    torch.cuda.synchronize()
    phase = (pos.cpu().numpy().astype(np.int64).view(np.uint64)[:, None] * turns[None]).view(np.int64)  # wraps
    half = phase.astype(np.float64) / 2.0 ** 63  # in units of pi, [-1, 1)
    near = np.where(half > 0, half - 1.0, half + 1.0)  # sin(pi half) = -sin(pi near)
    got = out[:, 0].double().cpu().numpy()
    sin = np.where(np.abs(half) > 0.5, -np.sin(np.pi * near), np.sin(np.pi * half))
    assert (got[0, ia] == 1).all() and (got[0, ib] == 0).all()
    for name, g, want, small in (("sin", got[:, ib], sin, np.abs(near) < 2.0 ** -6),
                                 ("cos", got[:, ia], np.cos(np.pi * half), np.abs(np.abs(half) - 0.5) < 2.0 ** -6)):
        err = np.abs(g - want)
        assert err.max() <= np.pi * 2.0 ** -27 + 8.1e-8, (name, err.max())
        tol = (np.pi * 2.0 ** -27 + np.abs(want) * 5 * 2.0 ** -24)[small]
        assert small.sum() > 10_000 and (err[small] <= tol).all(), (name, int((err[small] > tol).sum()), float(err[small].max()))
