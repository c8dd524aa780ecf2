"""Attention over selected blocks on the GPU: the bounds and the selection bit for
bit against their definitions, the attention against float64.

Tolerances of the attention. Scores are fp32 sums of at most 256 products of |q| <= ~5 and
|k| <= ~5, times scale <= 1/8: within 256 * 25 / 8 * 2^-24 < 5e-5, and the exponentials and sums add less than
that: 1e-4 absolute on lse, and relative on the weights, on outputs of size 1. bf16 output: weights rounded to bf16
(8 significant bits: off by u = 2^-8 of themselves at most) move an output by at most 2u / (1 - u) * sum_t w_t |v_t - out|,
and the output itself is rounded by half a step. float32 output: the weights' two parts leave u = 2^-16 of each."""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_helpers import bf16_tensor_bits, bf16_ulp, cuda_or_skip, guarded, guards_intact, to_dev_bf16
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

NAN = 0x7FC0


def _normal(r, shape):
    return f32_to_bf16_bits(r.standard_normal(shape).astype(np.float32))


class Cache:
    """K and V rows of B sequences, contiguous or in pages, rows past each length NaN."""

    def __init__(self, r, lens, Hkv, D, page, dev, S=None):
        import torch
        self.lens, self.Hkv, self.D, self.page = np.asarray(lens, np.int32), Hkv, D, page
        B = len(lens)
        S = S or max(int(max(lens)), 1)
        if page:
            S = -(-S // page) * page
        self.S, self.B = S, B
        self.k, self.v = (_normal(r, (B, S, Hkv, D)) for _ in range(2))
        for b, L in enumerate(lens):
            self.k[b, L:] = self.v[b, L:] = NAN
        self.bt, self.table = None, None
        k, v = self.k, self.v
        if page:
            nb = S // page
            n = B * nb + 3
            self.table = r.permutation(n)[:B * nb].reshape(B, nb).astype(np.int32)
            pools = [np.full((n, page, Hkv, D), NAN, np.uint16) for _ in range(2)]
            for b in range(B):
                for j in range(nb):
                    for p, x in zip(pools, (k, v)):
                        p[self.table[b, j]] = x[b, j * page:(j + 1) * page]
            for b in range(B):  # entries of blocks past the length name nothing
                self.table[b, -(-int(lens[b]) // page):] = -9
            k, v = pools
            self.bt = torch.from_numpy(self.table).to(dev)
        self.kd, self.vd = to_dev_bf16(k, dev), to_dev_bf16(v, dev)
        self.lens_d = torch.from_numpy(self.lens).to(dev)

    def rows(self):
        return (bf16_bits_to_f32(x).astype(np.float64) for x in (self.k, self.v))


def _run(c, q, lists, block, dev, dtype, lens=None):
    import torch
    import kv_cache_decode_gb300 as kvd
    B, T, Hq, D = q.shape
    full, out = guarded((B, T, Hq, D), torch.bfloat16 if dtype == "bf16" else torch.float32, dev)
    lfull, lse = guarded((B, T, Hq), torch.float32, dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    n = kvd.decode_blocks_plan(B, T, Hq, c.Hkv, D, lists.shape[-1], block)
    ws = torch.full((n + 512,), 0xa5, dtype=torch.uint8, device=dev)
    kvd.decode_blocks(to_dev_bf16(q, dev), c.kd, c.vd, torch.from_numpy(lists).to(dev), c.lens_d if lens is None else lens, block,
                      float(np.float32(D ** -0.5)), out, block_table=c.bt, workspace=ws[:n] if n else None, lse=lse, status=status)
    torch.cuda.synchronize()
    assert guards_intact(full) and guards_intact(lfull) and bool((ws[n:] == 0xa5).all())
    got = bf16_bits_to_f32(bf16_tensor_bits(out)) if dtype == "bf16" else out.cpu().numpy()
    return got.astype(np.float64), lse.cpu().numpy().astype(np.float64), int(status.item())


def _want(c, q, lists, block, lens=None):
    B, T, Hq, D = q.shape
    G = Hq // c.Hkv
    k, v = c.rows()
    q64 = bf16_bits_to_f32(q).astype(np.float64)
    out, lse, spread = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq)), np.zeros((B, T, Hq, D))
    for b in range(B):
        L = int((c.lens if lens is None else lens)[b])
        for i in range(T):
            for h in range(c.Hkv):
                g = slice(h * G, (h + 1) * G)
                out[b, i, g], lse[b, i, g], spread[b, i, g] = ref.attend(q64[b, i, g], k[b, :, h], v[b, :, h], lists[b, i, h].tolist(),
                                                                         L - T + 1 + i, block, float(np.float32(D ** -0.5)))
    return out, lse, spread


def _close(got, want, dtype):
    (o, l), (wo, wl, spread) = got, want
    none = np.isneginf(wl)
    assert np.array_equal(np.isneginf(l), none) and (o[none] == 0).all()
    assert np.isfinite(o).all() and np.abs(l[~none] - wl[~none]).max(initial=0.0) <= 1e-4
    tol = 1e-4 * np.maximum(1, spread)
    if dtype == "bf16":
        tol = tol + 0.5 * bf16_ulp(np.maximum(np.abs(o), np.abs(wo))) + 2 * 2.0 ** -8 / (1 - 2.0 ** -8) * spread
    else:
        tol = tol + 2 * 2.0 ** -16 / (1 - 2.0 ** -16) * spread
    assert (np.abs(o - wo) <= tol).all(), np.abs(o - wo).max()


def _lists(r, c, T, K, block, style="mixed"):
    """Lists of K entries: blocks in random order, some named twice, some past the end, some -1."""
    nb = -(-c.S // block)
    x = r.integers(0, nb, (c.B, T, c.Hkv, K)).astype(np.int32)
    if style == "mixed":
        x[r.random(x.shape) < 0.1] = -1
        x[r.random(x.shape) < 0.05] = nb + 5
        x[r.random(x.shape) < 0.02] = 2 ** 31 - 1
        x[r.random(x.shape) < 0.02] = -2 ** 31
    return x


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 65, 200, 257, 300, 511]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,block,page", [
    (8, 1, 128, 64, 0), (32, 8, 128, 64, 64), (3, 3, 64, 16, 16), (9, 1, 64, 32, 128), (48, 1, 256, 64, 0), (5, 1, 256, 16, 32),
    (16, 1, 128, 128, 16), (64, 1, 128, 32, 0), (40, 2, 64, 64, 16), (33, 1, 128, 16, 0), (64, 1, 256, 256, 64), (1, 1, 64, 4096, 0),
    (34, 2, 256, 32, 32), (2, 1, 128, 16, 0)])
def test_attention(Hq, Hkv, D, block, page, dtype):
    dev = cuda_or_skip()
    r = np.random.default_rng(Hq * D + block)
    c = Cache(r, LENS, Hkv, D, page, dev)
    q = _normal(r, (c.B, 1, Hq, D))
    for K in (1, 3, 40):
        x = _lists(r, c, 1, K, block)
        got = _run(c, q, x, block, dev, dtype)
        assert got[2] == 0
        _close(got[:2], _want(c, q, x, block), dtype)


@pytest.mark.parametrize("Hq,Hkv,D,T", [(8, 2, 128, 3), (24, 1, 64, 2), (6, 1, 256, 5), (12, 12, 64, 7), (4, 1, 128, 64)])
def test_attention_query_tokens(Hq, Hkv, D, T):
    dev = cuda_or_skip()
    r = np.random.default_rng(T)
    c = Cache(r, [300, 0, 1, T, 16, 47, 129], Hkv, D, 32, dev)
    q = _normal(r, (c.B, T, Hq, D))
    x = _lists(r, c, T, 9, 16)
    for dtype in ("f32", "bf16"):
        got = _run(c, q, x, 16, dev, dtype)
        assert got[2] == 0
        _close(got[:2], _want(c, q, x, 16), dtype)


@pytest.mark.parametrize("Hq,Hkv,D,block,K,lens", [
    (8, 1, 128, 128, 256, [32768]),           # one pair: several clusters
    (1, 1, 64, 16, 700, [11111]), (48, 1, 256, 64, 128, [9000, 4097]), (8, 8, 128, 64, 33, [5000]),
    (16, 8, 64, 32, 5, [900] * 90), (4, 2, 128, 16, 2, [33] * 300)])
def test_attention_long_and_many(Hq, Hkv, D, block, K, lens):
    dev = cuda_or_skip()
    r = np.random.default_rng(K)
    c = Cache(r, lens, Hkv, D, 16, dev)
    q = _normal(r, (c.B, 1, Hq, D))
    x = _lists(r, c, 1, K, block, "any")
    for dtype in ("f32", "bf16"):
        got = _run(c, q, x, block, dev, dtype)
        _close(got[:2], _want(c, q, x, block), dtype)
        again = _run(c, q, x, block, dev, dtype)
        assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.parametrize("Hq,D", [(8, 64), (48, 64), (3, 128), (48, 128), (8, 256), (20, 256)])
@pytest.mark.parametrize("B", [400, 100, 50, 12, 4])
def test_attention_by_how_many_pairs_there_are(Hq, D, B):
    """From one CTA a pair to clusters of 16, joined by sent and by fetched states."""
    dev = cuda_or_skip()
    r = np.random.default_rng(B + D)
    lens = r.integers(0, 180, B)
    c = Cache(r, lens, 1, D, 16, dev)
    q = _normal(r, (B, 1, Hq, D))
    for K in (9, 33):
        x = _lists(r, c, 1, K, 16)
        for dtype in ("f32", "bf16"):
            got = _run(c, q, x, 16, dev, dtype)
            assert got[2] == 0
            _close(got[:2], _want(c, q, x, 16), dtype)


def test_attention_scores():
    """Scores that rise along the list raise the maxima again and again; one that towers; equal ones."""
    dev = cuda_or_skip()
    r = np.random.default_rng(4)
    c = Cache(r, [1500, 1500, 1500], 1, 64, 0, dev)
    q = np.zeros((3, 1, 8, 64), np.float32)
    q[..., 0] = 8.0
    k = np.zeros((3, c.S, 1, 64), np.float32)
    k[0, :, 0, 0] = np.arange(c.S) * 0.25
    k[1, 777, 0, 0] = 100.0
    c.k = f32_to_bf16_bits(k)
    c.kd = to_dev_bf16(c.k, dev)
    x = np.tile(np.arange(-(-c.S // 32), dtype=np.int32), (3, 1, 1, 1))
    got = _run(c, f32_to_bf16_bits(q), x, 32, dev, "f32")
    out, lse, _ = _want(c, f32_to_bf16_bits(q), x, 32)
    # scores up to 375: fp32 roundings of that size, 375 * 2^-24 * a few
    assert np.abs(got[0] - out).max() < 1e-3 and np.abs(got[1] - lse).max() < 1e-3


def test_attention_not_finite():
    """A NaN or infinite key or value of a listed token shows in its KV head's rows; of a token that is not listed it does not."""
    dev = cuda_or_skip()
    r = np.random.default_rng(5)
    c = Cache(r, [200, 200, 200, 200], 2, 64, 0, dev)
    c.k[0, 40, 0, 3] = NAN
    c.k[1, 40, 1, 3] = 0x7F80
    c.v[2, 40, 0, 3] = NAN
    c.kd, c.vd = to_dev_bf16(c.k, dev), to_dev_bf16(c.v, dev)
    q = _normal(r, (4, 1, 4, 64))
    x = np.tile(np.array([0, 2, 5], np.int32), (4, 1, 2, 1))
    o, l, _ = _run(c, q, x, 32, dev, "f32")
    assert np.isfinite(o).all() and np.isfinite(l).all()
    x[..., 1] = 1
    o, l, _ = _run(c, q, x, 32, dev, "f32")
    assert np.isnan(o[0, 0, :2]).all() and np.isfinite(o[0, 0, 2:]).all()
    pos = bf16_bits_to_f32(q)[1, 0, 2:, 3] > 0  # q . k = +inf there, else -inf: a weight of 0
    assert np.isnan(o[1, 0, 2:][pos]).all() and np.isfinite(o[1, 0, 2:][~pos]).all() and np.isfinite(o[1, 0, :2]).all()
    assert np.isnan(o[2, 0, :2, 3]).all() and np.isfinite(np.delete(o[2, 0, :2], 3, -1)).all() and np.isfinite(o[3]).all()


def test_attention_status():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(6)
    c = Cache(r, [100, 64, 90], 2, 128, 16, dev)
    q = _normal(r, (3, 1, 8, 128))
    x = np.tile(np.arange(7, dtype=np.int32), (3, 1, 2, 1))
    c.bt[1, 2] = 99999  # names no page: zero rows
    c.k[1, 32:48] = c.v[1, 32:48] = 0
    got = _run(c, q, x, 16, dev, "f32")
    assert got[2] == kvd.STATUS_BAD_PAGE
    _close(got[:2], _want(c, q, x, 16), "f32")
    c = Cache(r, [112, 64, 0], 2, 128, 16, dev)
    lens = torch.tensor([2 ** 31 - 1, 64, -5], dtype=torch.int32, device=dev)
    got = _run(c, q, x, 16, dev, "f32", lens=lens)
    assert got[2] == kvd.STATUS_SEQ_LEN_CLAMPED
    _close(got[:2], _want(c, q, x, 16), "f32")


def test_attention_all_blocks_is_the_dense_one():
    """With every block listed the result is the attention over all tokens, within both kernels' bounds."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(7)
    c = Cache(r, [700, 33, 1, 512], 4, 128, 16, dev)
    q = _normal(r, (4, 1, 16, 128))
    x = np.tile(np.arange(-(-c.S // 64), dtype=np.int32), (4, 1, 4, 1))
    o, l, _ = _run(c, q, x, 64, dev, "f32")
    out, lse = torch.empty(4, 16, 128, device=dev), torch.empty(4, 16, device=dev)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=dev)
    kvd.decode_attention_paged(to_dev_bf16(q[:, 0], dev), c.kd, c.vd, c.bt, c.lens_d, c.S, float(np.float32(128 ** -0.5)), out,
                               workspace=ws, lse=lse)
    assert np.abs(o[:, 0] - out.double().cpu().numpy()).max() < 2e-4 and np.abs(l[:, 0] - lse.double().cpu().numpy()).max() < 2e-4


# ---------------------------------------------------------------------------
# bounds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D,Hkv,block,page", [(64, 3, 16, 0), (128, 8, 64, 64), (256, 1, 32, 128), (128, 2, 128, 128), (64, 1, 256, 0),
                                              (256, 5, 16, 16)])
def test_bounds(D, Hkv, block, page):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(D + block)
    lens = [0, 1, block - 1, block, block + 1, 5 * block + 3, 700, 8 * block]
    c = Cache(r, lens, Hkv, D, page, dev, S=max(700, 8 * block))
    c.k[5, 3, 0, 7] = 0x7F80             # infinity, NaN, zeros, tiny and huge keys
    c.k[5, block + 2, Hkv - 1, 5] = NAN
    c.k[6, :block, 0] = 0
    c.k[7, :block] = f32_to_bf16_bits(np.float32(1e-39) * r.standard_normal((block, Hkv, D)).astype(np.float32))
    c.k[7, block:2 * block] = f32_to_bf16_bits(np.float32(3e37) * np.clip(r.standard_normal((block, Hkv, D)), -9, 9).astype(np.float32))
    if page:
        for b in range(c.B):
            for j in range(-(-lens[b] // page)):
                c.kd[int(c.table[b, j])] = to_dev_bf16(c.k[b, j * page:(j + 1) * page], dev)
    else:
        c.kd = to_dev_bf16(c.k, dev)
    old = [0, 0, 5, block - 1, block, 2 * block, 3 * block + 1, 8 * block]
    for frm in (None, old):
        codes, scales = kvd.alloc_block_bounds(c.kd, block)
        codes.fill_(77)
        scales.fill_(-3.0)
        want_c, want_s = codes.cpu().numpy(), scales.cpu().numpy()
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        most = max(L - f for L, f in zip(lens, frm or [0] * len(lens)))
        kvd.kv_block_bounds(c.kd, codes, scales, c.lens_d, most, block, block_table=c.bt, status=status,
                            from_lens=None if frm is None else torch.tensor(frm, dtype=torch.int32, device=dev))
        torch.cuda.synchronize()
        k32 = bf16_bits_to_f32(c.k)
        for b, L in enumerate(lens):
            for j in range((frm or [0] * len(lens))[b] // block, L // block):
                n, sub = (b, j) if not page else (c.table[b, j * block // page], j * block % page // block)
                want_c[n, sub], want_s[n, sub] = ref.bounds(k32[b, j * block:(j + 1) * block])
        assert int(status.item()) == 0
        assert np.array_equal(codes.cpu().numpy(), want_c)
        assert np.array_equal(scales.cpu().numpy(), want_s, equal_nan=True)


def test_bounds_hold():
    """No key of a block scores above its bound with the query as it is: sum_d max(q_d hi_d, q_d lo_d) * scale."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(3)
    c = Cache(r, [640], 2, 128, 0, dev)
    codes, scales = kvd.alloc_block_bounds(c.kd, 64)
    kvd.kv_block_bounds(c.kd, codes, scales, c.lens_d, 640, 64)
    k, _ = c.rows()
    cd, sc = codes.double().cpu().numpy()[0], scales.double().cpu().numpy()[0]
    for _ in range(20):
        q = r.standard_normal(128)
        top = np.maximum(q * cd[:, :, 0], q * cd[:, :, 1]).sum(-1) * sc            # [10, 2]
        s = np.einsum("jthd,d->jth", k[0].reshape(10, 64, 2, 128), q).max(1)
        assert (s <= top * (1 + 1e-6)).all()


def test_bounds_status():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(8)
    c = Cache(r, [64, 100], 2, 64, 16, dev)
    codes, scales = kvd.alloc_block_bounds(c.kd, 16)

    def run(lens, most, frm=None):
        codes.fill_(5)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        kvd.kv_block_bounds(c.kd, codes, scales, torch.tensor(lens, dtype=torch.int32, device=dev), most, 16, block_table=c.bt,
                            status=status, from_lens=frm)
        torch.cuda.synchronize()
        return int(status.item()), codes.cpu().numpy()
    assert run([64, 96], 96)[0] == 0
    assert run([64, -1], 96)[0] == kvd.STATUS_SEQ_LEN_CLAMPED
    st, got = run([64, 96], 40)  # more tokens than said: three blocks a sequence at most
    assert st == kvd.STATUS_SEQ_LEN_CLAMPED and (got[c.table[0, 2]] != 5).any() and (got[c.table[0, 3]] == 5).all()
    c.bt[0, 1] = 1 << 28
    st, got = run([64, 96], 96)
    assert st == kvd.STATUS_BAD_PAGE and (got[c.table[0, 1]] == 5).all() and (got[c.table[0, 2]] != 5).any()


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------

def _select(dev, q, codes, scales, lens, max_len, block, K, first, last, bt=None):
    import torch
    import kv_cache_decode_gb300 as kvd
    B, T, Hq, D = q.shape
    Hkv = codes.shape[2]
    out = torch.full((B * T * Hkv * K + 64,), 123456, dtype=torch.int32, device=dev)
    n = kvd.block_select_plan(B, T, Hkv, max_len, block)
    ws = torch.full((n + 512,), 0xff, dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kvd.block_select(to_dev_bf16(q, dev), torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev),
                     torch.tensor(lens, dtype=torch.int32, device=dev), max_len, block, out[32:-32].view(B, T, Hkv, K), n_first=first,
                     n_last=last, block_table=None if bt is None else torch.from_numpy(bt).to(dev), workspace=ws[:n], status=status)
    torch.cuda.synchronize()
    assert bool((out[:32] == 123456).all()) and bool((out[-32:] == 123456).all()) and bool((ws[n:] == 0xff).all())
    return out[32:-32].view(B, T, Hkv, K).cpu().numpy(), int(status.item())


def _select_want(q, codes, scales, lens, block, K, first, last, bt=None, page=0):
    B, T, Hq, D = q.shape
    Hkv = codes.shape[2]
    G = Hq // Hkv
    q32 = bf16_bits_to_f32(q)
    out = np.zeros((B, T, Hkv, K), np.int64)
    for b, L in enumerate(lens):
        if bt is None:
            cb, sb, missing = codes[b], scales[b], ()
        else:
            ok = (bt[b] >= 0) & (bt[b] < len(codes))
            at = np.where(ok, bt[b], 0)
            cb, sb = (x[at].reshape((-1,) + x.shape[2:]) for x in (codes, scales))
            missing = set(np.nonzero(np.repeat(~ok, page // block))[0].tolist())
        for i in range(T):
            n = max(0, -(-(L - T + 1 + i) // block))
            for h in range(Hkv):
                s = np.full(n, 0, np.float32)
                m = min(n, len(sb))
                s[:m] = ref.score(q32[b, i, h * G:(h + 1) * G], cb[:m, h], sb[:m, h])
                out[b, i, h] = ref.select(s, K, first, last, missing)
    return out


def _codes(r, shape):
    hi = r.integers(-20, 128, shape + (1,))
    lo = hi - r.integers(0, 128, hi.shape)
    x = np.concatenate([hi, lo], -1)
    return np.ascontiguousarray(np.clip(np.moveaxis(x, -1, -2), -127, 127).astype(np.int8))


@pytest.mark.parametrize("Hq,Hkv,D,T,block,page", [
    (32, 8, 128, 1, 64, 0), (4, 4, 64, 1, 16, 16), (2, 1, 256, 3, 32, 64), (8, 1, 128, 5, 16, 0), (9, 1, 64, 2, 16, 32),
    (48, 1, 256, 2, 16, 0), (64, 1, 128, 9, 16, 0), (6, 2, 64, 17, 16, 128), (5, 5, 128, 64, 64, 64), (33, 1, 256, 1, 16, 16)])
def test_select(Hq, Hkv, D, T, block, page):
    dev = cuda_or_skip()
    r = np.random.default_rng(Hq + D + T)
    lens = [0, 1, block, 40 * block, 40 * block + 1, 57 * block - 1, 130 * block + 7, T]
    B, most = len(lens), 131 * block
    bt, n, per = None, B, 131
    if page:
        per = page // block
        nb = -(-131 // per)
        n = B * nb + 2
        bt = r.permutation(n)[:B * nb].reshape(B, nb).astype(np.int32)
        for b, L in enumerate(lens):
            bt[b, -(-L // page):] = -3
    codes = _codes(r, (n, per, Hkv, D))
    scales = r.uniform(0.01, 0.03, (n, per, Hkv)).astype(np.float32)
    q = _normal(r, (B, T, Hq, D))
    for K, first, last in ((1, 0, 1), (7, 2, 3), (40, 1, 2), (131, 0, 1), (200, 5, 6), (6, 3, 3)):
        got, st = _select(dev, q, codes, scales, lens, most, block, K, first, last, bt)
        assert st == 0
        assert np.array_equal(got, _select_want(q, codes, scales, lens, block, K, first, last, bt, page)), (K, first, last)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,T", [(1, 1), (8, 2), (8, 3), (8, 6), (8, 11), (3, 9), (12, 1), (12, 2), (12, 3), (12, 5), (2, 25), (64, 2)])
def test_select_widths(D, G, T):
    """Every number of query rows scored at once, in one round and several, for sequences of no block to many."""
    dev = cuda_or_skip()
    r = np.random.default_rng(D + G + T)
    Hkv, block = 2, 16
    for page in (0, 32):
        lens = [16 * 300 + 3, 0, 16 * 33, 16 * 8 - 1, 16 * 150, 31]
        nb, B = 301, len(lens)
        bt, n, per = None, B, nb
        if page:
            per = page // block
            n = B * 151 + 2
            bt = r.permutation(n)[:B * 151].reshape(B, 151).astype(np.int32)
            for b, L in enumerate(lens):
                bt[b, -(-L // page):] = -1
        codes = _codes(r, (n, per, Hkv, D))
        scales = r.uniform(0.01, 0.03, (n, per, Hkv)).astype(np.float32)
        q = _normal(r, (B, T, G * Hkv, D))
        for K, first, last in ((8, 1, 2), (100, 0, 1)):
            got, st = _select(dev, q, codes, scales, lens, nb * block, block, K, first, last, bt)
            assert st == 0
            assert np.array_equal(got, _select_want(q, codes, scales, lens, block, K, first, last, bt, page)), (K, page)


def test_select_whole_numbers_are_exact():
    """The largest sums there are, and neighbours one apart; many ties; scales that order blocks by their last bit."""
    dev = cuda_or_skip()
    r = np.random.default_rng(0)
    D, n = 256, 500
    codes = np.full((1, n, 1, 2, D), 127, np.int8)
    codes[..., 1, :] = -127
    codes[0, :, 0, 0, 17] -= r.integers(0, 3, n).astype(np.int8)
    scales = np.full((1, n, 1), np.float32(0.01))
    q = np.where(np.arange(8 * D).reshape(1, 1, 8, D) % 3 == 0, -1.0, 1.0).astype(np.float32)
    q[..., 17] = 1.0
    q = f32_to_bf16_bits(q)
    for K in (3, 100, 333, 499):
        got, _ = _select(dev, q, codes, scales, [n * 16], n * 16, 16, K, 0, 1)
        assert np.array_equal(got, _select_want(q, codes, scales, [n * 16], 16, K, 0, 1))
    scales = np.nextafter(np.float32(0.01), np.float32(1)) * np.ones((1, n, 1), np.float32)
    scales[0, r.random(n) < 0.5] = np.float32(0.01)
    for K in (3, 100, 333):
        got, _ = _select(dev, q, codes, scales, [n * 16], n * 16, 16, K, 1, 1)
        assert np.array_equal(got, _select_want(q, codes, scales, [n * 16], 16, K, 1, 1))


def test_select_odd_values():
    """Scales that are NaN, zero, infinite, tiny or huge; query rows of zeros, NaN, infinities, tiny and huge values."""
    dev = cuda_or_skip()
    r = np.random.default_rng(1)
    n, D = 90, 128
    codes = _codes(r, (7, n, 2, D))
    codes[:, 5] = 0
    scales = r.uniform(0.01, 0.03, (7, n, 2)).astype(np.float32)
    scales[:, 7], scales[:, 11], scales[:, 13], scales[:, 17] = np.nan, 0.0, 1e-42, 1e36
    scales[0, 20:80] = np.nan
    q = bf16_bits_to_f32(_normal(r, (7, 1, 8, D))).copy()
    q[1, 0, 1] = 0
    q[2, 0, 2, 3] = np.nan
    q[3, 0, 0:4] = np.inf
    q[4] *= np.float32(1e-38)
    q[5] *= np.float32(1e37)
    q[6] = 0
    q = f32_to_bf16_bits(q)
    lens = [n * 16] * 7
    for K in (4, 30, 62, 89):
        got, _ = _select(dev, q, codes, scales, lens, n * 16, 16, K, 0, 1)
        assert np.array_equal(got, _select_want(q, codes, scales, lens, 16, K, 0, 1)), K


@pytest.mark.parametrize("lens,block,K", [([400000], 16, 300), ([1 << 20, 70000, 16], 16, 4000), ([300000], 16, 18000)])
def test_select_long(lens, block, K):
    """More blocks than shared memory holds keys of."""
    dev = cuda_or_skip()
    r = np.random.default_rng(2)
    n = -(-max(lens) // block)
    codes = _codes(r, (len(lens), n, 1, 64))
    scales = r.uniform(0.01, 0.03, (len(lens), n, 1)).astype(np.float32)
    q = _normal(r, (len(lens), 2, 4, 64))
    got, st = _select(dev, q, codes, scales, lens, n * block, block, K, 1, 2)
    assert st == 0 and np.array_equal(got, _select_want(q, codes, scales, lens, block, K, 1, 2))


def test_select_status():
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(9)
    codes, scales = _codes(r, (60, 2, 1, 64)), r.uniform(0.01, 0.03, (60, 2, 1)).astype(np.float32)
    bt = r.permutation(60)[:50].reshape(1, 50).astype(np.int32)
    bt[0, 3], bt[0, 9] = -1, 60
    q = _normal(r, (1, 1, 4, 64))
    for K in (5, 90, 98):  # 98: one of the four blocks without a page is kept
        got, st = _select(dev, q, codes, scales, [1600], 1600, 16, K, 0, 1, bt)
        assert st == kvd.STATUS_BAD_PAGE
        assert np.array_equal(got, _select_want(q, codes, scales, [1600], 16, K, 0, 1, bt, 32))
    got, st = _select(dev, q, codes[:50], scales[:50], [99999], 1600, 16, 5, 0, 1, np.arange(50, dtype=np.int32).reshape(1, 50))
    assert st == kvd.STATUS_SEQ_LEN_CLAMPED
    assert np.array_equal(got, _select_want(q, codes[:50], scales[:50], [1600], 16, 5, 0, 1, np.arange(50).reshape(1, 50), 32))
