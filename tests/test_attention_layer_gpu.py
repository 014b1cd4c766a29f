"""Attention-layer operators on the GPU against the fp64 oracle.

Tolerances count roundings. u16 = 2^-8 and u32 = 2^-24 are half a step of bf16
and fp32 relative to the value.

  norm and rotation: the sum of D squares in 8 chains of 8 and log2(D/8) pair
    sums loses at most 13 u32, halved by the root; root, division, two
    products, weight + offset, sine and cosine (an angle off by 2^-25 turns =
    3.2 u32, 2 u32 of the function), product and difference: under 24 u32 of
    |a| + |b| in all, plus u16 of the result in bf16.
  write, read: exact.
  attention: logits from products exact in fp32, summed in fp32: at most D 2^-23
    (the tensor cores may truncate) of sum |q k| scale, and 4 u32 for the scale
    and the exponent's argument (relative to |z| <= sum |q k| scale); so each
    probability is off by e^(2 delta) - 1 <= 3 delta, delta = (D 2^-23 + 4 u32)
    sum |q k| scale, 2^-21 of the fast exponential; u16 for its rounding to
    bf16; the sum over L keys and its partial sums: L 2^-23. All relative to
    sum p |v|. Then u16 of the result.
    lse: delta + 2^-21 + L u32 in absolute terms, 4 u32 of its size.
"""
import numpy as np
import pytest
import torch

import uniform_state_text_b200 as dg
from oracle import attention as A

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24
F8 = torch.float8_e4m3fn
MASKS = {"full": dg.DG_MASK_FULL, "causal": dg.DG_MASK_CAUSAL, "tree": dg.DG_MASK_TREE}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from uniform_state_text_b200 import build
    build.build()
    dg.lib()


def f64(t):
    return t.double().cpu().numpy()


# ----------------------------------------------------------------------------- norm and rotation
def _check_norm(x, got, w, pos, freq, inter, eps, off, ulp):
    want, size = A.norm_rope(f64(x), None if w is None else f64(w), pos.cpu().numpy(), freq.cpu().numpy(),
                             inter, eps, off)
    tol = 24 * U32 * size + ulp * np.abs(want) + 1e-37
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,hq,hk,D,rot", [
    (1, 1, 1, 8, 0), (1, 16, 8, 128, 128), (7, 3, 1, 64, 64), (5, 5, 2, 80, 48), (33, 4, 0, 256, 64),
    (3, 2, 2, 256, 256), (9, 0, 3, 16, 16), (2, 9, 9, 136, 128), (1030, 22, 2, 128, 128)])
def test_norm_rope(tokens, hq, hk, D, rot, dt, inter):
    g = torch.Generator("cuda").manual_seed(tokens * 1000 + D)
    rows = (torch.randn(tokens, hq + 2 * hk + 1, D, generator=g, device="cuda") * 3).to(dt)
    q, k = rows[:, :hq], rows[:, hq:hq + hk]
    wq = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt)
    pos = torch.randint(-5, 1 << 20, (tokens,), generator=g, device="cuda").int()
    freq = dg.rope_frequencies(rot)
    qo, ko = dg.qk_norm_rope(q, k, wq, None, pos, freq, interleaved=inter, eps=1e-5, weight_offset=0.5)
    assert qo.shape == q.shape and ko.shape == k.shape and qo.is_contiguous()
    ulp = U16 if dt == torch.bfloat16 else 0.0
    _check_norm(q, qo, wq, pos, freq, inter, 1e-5, 0.5, ulp)
    _check_norm(k, ko, None, pos, freq, inter, 1e-5, 0.5, ulp)


def test_norm_rope_far_positions_and_small_rows():
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 0], dtype=torch.int32, device="cuda")
    freq = dg.rope_frequencies(64, 500000.0)
    x = torch.randn(4, 3, 64, device="cuda")
    x[1] *= 1e-6
    x[2, 1] = 0.0
    q, _ = dg.qk_norm_rope(x, x[:, :0], None, None, pos, freq)
    _check_norm(x, q, None, pos, freq, False, 1e-6, 0.0, 0.0)
    assert not q[2, 1].any()


def test_norm_rope_in_place_and_nan_stays_in_its_row():
    x = torch.randn(9, 4, 128, device="cuda").bfloat16()
    x[3, 1, 77] = float("nan")
    pos, freq = torch.arange(9, device="cuda").int(), dg.rope_frequencies(128)
    want, _ = dg.qk_norm_rope(x, x[:, :0], None, None, pos, freq)
    y = x.clone()
    dg.dg_qk_norm_rope(9, 4, 0, 128, 128, False, dg.DG_BF16, y.data_ptr(), 512, 128, 0, 0, 0, 0, 0, 0.0, 1e-6,
                       pos.data_ptr(), freq.data_ptr(), y.data_ptr(), 0,
                       torch.cuda.current_stream().cuda_stream)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    bad = want.isnan().any(-1)
    assert bad[3, 1] and bad.sum() == 1


# ----------------------------------------------------------------------------- the cache
class Setup:
    """A batch over a cache whose pages lie in random order; every row that no sequence owns is NaN."""

    def __init__(self, lengths, fmt, Hk, D, page, seed=0, pad=0, fill=True):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.past, self.new = [p for p, _ in lengths], [n for _, n in lengths]
        need = [-(-(p + n) // page) for p, n in lengths]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=self.g, device="cuda").int()
        self.table = torch.full((len(lengths), max(need + [1])), pages + 7, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        first = np.concatenate([[0], np.cumsum(self.new)])
        self.first, self.tokens = first, int(first[-1]) + pad
        dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        self.batch = dg.KVBatch(self.table, dev(first), dev(self.past), self.tokens)
        self.fmt, self.Hk, self.D, self.page = fmt, Hk, D, page
        self.cache = dg.KVCache.empty(pages, page, Hk, D, fmt)
        for n in "kv":
            t = getattr(self.cache, n)
            if fmt == dg.DG_KV_BF16:
                t.fill_(float("nan"))
            else:
                t.view(torch.uint8).fill_(0x7F)
                getattr(self.cache, n + "_exp").fill_(255)
        if fill:
            for b, (p, n) in enumerate(lengths):
                self.put(b, torch.randn(2, p + n, Hk, D, generator=self.g, device="cuda"))

    def at(self, b, start, stop):
        pos = torch.arange(start, stop, device="cuda")
        return self.table[b].long()[pos // self.page], pos % self.page

    def put(self, b, kv, start=0):
        """Rows of k and v (kv [2, n, Hk, D]) straight into the pages, quantised by torch."""
        page, place = self.at(b, start, start + kv.shape[1])
        for n, x in zip("kv", kv):
            t = getattr(self.cache, n)
            if self.fmt == dg.DG_KV_BF16:
                t[page, :, place] = x.bfloat16()
            else:
                e = torch.randint(120, 130, x.shape[:2], generator=self.g, device="cuda")
                t.view(torch.uint8)[page, :, place] = (x * 100).to(F8).view(torch.uint8)
                getattr(self.cache, n + "_exp")[page, :, place] = (e - 7).to(torch.uint8)

    def values(self, b, n, start, stop):
        """[positions, Hk, D] of sequence b in fp64 (numpy)."""
        page, place = self.at(b, start, stop)
        x = getattr(self.cache, n)[page, :, place].double()
        if self.fmt == dg.DG_KV_E4M3:
            e = getattr(self.cache, n + "_exp")[page, :, place].long()
            x = x * ((e - 127 + 1023) << 52).view(torch.float64)[..., None]
        return x.cpu().numpy()


LENGTHS = [(0, 1), (5, 0), (0, 0), (17, 3), (63, 1), (64, 65), (1, 130)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,Hk,D,page", [
    (dg.DG_KV_E4M3, 2, 128, 16), (dg.DG_KV_E4M3, 1, 16, 1), (dg.DG_KV_E4M3, 3, 80, 24),
    (dg.DG_KV_E4M3, 5, 256, 64), (dg.DG_KV_BF16, 2, 64, 16), (dg.DG_KV_BF16, 3, 112, 5)])
def test_write_then_read(fmt, Hk, D, page, dt):
    s = Setup(LENGTHS, fmt, Hk, D, page, pad=3, fill=False)
    rows = torch.randn(s.tokens, 2 * Hk + 1, D, generator=s.g, device="cuda")
    rows *= torch.exp(6 * torch.randn(s.tokens, 2 * Hk + 1, 1, generator=s.g, device="cuda"))
    rows[2, 0] = 0
    rows[1, 0, 3], rows[1, 0, 5], rows[3, 1, 0] = float("nan"), float("inf"), -float("inf")
    rows[4, 0] *= 1e-37
    rows[4, 1, 1] = 3.3e38
    rows = rows.to(dt)
    k, v = rows[:, :Hk], rows[:, Hk:2 * Hk]
    before = [getattr(s.cache, n).clone() for n in "kv"]
    s.cache.write(k, v, s.batch)
    s.cache.check()
    owned = torch.zeros(before[0].shape[:3], dtype=torch.bool, device="cuda")
    values = []
    for b, (p, n) in enumerate(LENGTHS):
        page_at, place = s.at(b, p, p + n)
        owned[page_at, :, place] = True
        for name, x in (("k", k), ("v", v)):
            src = f64(x[s.first[b]:s.first[b] + n])
            got = getattr(s.cache, name)[page_at, :, place]
            if fmt == dg.DG_KV_BF16:
                assert torch.equal(got.view(torch.int16),
                                   x[s.first[b]:s.first[b] + n].bfloat16().view(torch.int16))
                continue
            exps = getattr(s.cache, name + "_exp")[page_at, :, place].cpu().numpy()
            for i in range(n):
                for h in range(Hk):
                    codes, e = A.quantise(src[i, h])
                    assert exps[i, h] == e, (name, i, h, exps[i, h], e)
                    assert np.array_equal(f64(got[i, h]), codes, equal_nan=True), (name, i, h)
    for n, old in zip("kv", before):
        same = getattr(s.cache, n).view(torch.uint8) == old.view(torch.uint8)
        assert same.reshape(*owned.shape, -1)[~owned].all()
    for out_dt in (torch.float32, torch.bfloat16):
        out = tuple(torch.full((s.tokens, Hk, D), 7.0, dtype=out_dt, device="cuda") for _ in "kv")
        s.cache.read(s.batch, out_dt, out=out)
        s.cache.check()
        for name, o in zip("kv", out):
            for b, (p, n) in enumerate(LENGTHS):
                want = s.values(b, name, p, p + n)
                assert np.array_equal(f64(o[s.first[b]:s.first[b] + n]), want, equal_nan=True)
            assert (o[s.tokens - 3:] == 7.0).all()
    del values


@pytest.mark.parametrize("fmt", [dg.DG_KV_E4M3, dg.DG_KV_BF16])
def test_bad_pages_are_skipped_and_reported(fmt):
    s = Setup([(3, 20), (0, 4)], fmt, 2, 64, 8, seed=4)
    pages = s.cache.k.shape[0]
    s.table[0, 1], s.table[0, 2] = -1, pages          # positions 8..23: no page
    before = s.cache.k.clone()
    k = torch.randn(s.tokens, 2, 64, device="cuda")
    s.cache.write(k, k, s.batch)
    with pytest.raises(dg.DgError) as e:
        s.cache.check()
    assert e.value.code == dg.DG_EINVAL
    assert (s.cache.k.view(torch.uint8) != before.view(torch.uint8)).reshape(pages, -1).any(1).sum() == 2
    s.cache.status.zero_()
    out, _ = s.cache.read(s.batch, torch.float32)
    assert not out[5:20].any() and out[:5].any() and out[20:].any()
    assert int(s.cache.status) == dg.DG_EINVAL
    s.cache.status.zero_()
    # a past that runs over the table, and one below zero
    s.batch.past.copy_(torch.tensor([10 ** 6, -3], dtype=torch.int32))
    out, _ = s.cache.read(s.batch, torch.float32)
    assert not out[:20].any() and int(s.cache.status) == dg.DG_EINVAL
    before = s.cache.k.clone()
    s.cache.write(k, k, s.batch)
    changed = (s.cache.k.view(torch.uint8) != before.view(torch.uint8)).reshape(pages, -1).any(1)
    assert changed.sum() <= 1                         # position 0 of sequence 1 alone


# ----------------------------------------------------------------------------- attention
def _tree(new, seed, empty=()):
    """Ancestor bits of random trees; the tokens in `empty` see nothing."""
    r = np.random.default_rng(seed)
    words = max(1, -(-max(new) // 32))
    rows = []
    for n in new:
        seen = []
        for i in range(n):
            p = int(r.integers(-1, i)) if i else -1
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        rows += seen
    rows = [0 if t in empty else x for t, x in enumerate(rows)]
    return np.array([[(x >> 32 * w) & 0xFFFFFFFF for w in range(words)] for x in rows],
                    dtype=np.uint32).reshape(-1, words)


def _check_attention(s, q, mask, scale, out, lse, words=None, rows=None):
    group = q.shape[1] // s.Hk
    q, out, lse = f64(q), f64(out), f64(lse)
    for b, (p, n) in enumerate(zip(s.past, s.new)):
        if not n:
            continue
        K, V = (s.values(b, x, 0, p + n) for x in "kv")
        at = np.arange(n) if rows is None else np.unique([x % n for x in rows])
        t = s.first[b] + at
        seen = np.stack([A.seen_by(i, p, n, mask, None if words is None else words[s.first[b] + i]) for i in at])
        L = seen.sum(1)
        for h in range(q.shape[1]):
            want, wl, size, logit, spread = A.attend(q[t, h], K[:, h // group], V[:, h // group], seen, float(scale))
            got, gl = out[t, h], lse[t, h]
            assert not got[L == 0].any() and np.isneginf(gl[L == 0]).all(), (b, h)
            delta = (s.D * 2.0 ** -23 + 4 * U32) * logit
            tol = (3 * delta + 2.0 ** -21 + U16 + L * 2.0 ** -23)[:, None] * size + U16 * np.abs(want) + 1e-37
            fine = np.isfinite(want)           # a NaN among what a row sees comes out as one
            assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (b, h)
            err = np.abs(got - want)[fine] / tol[fine]
            assert (err <= 1).all(), (b, h, err.max())
            # each probability's rounding is its own, uniform to u16 of p at most: over keys and columns
            # the errors add as squares, at most u16 / sqrt(3) spread; three times that is far out
            fine = np.isfinite(want).all(1)
            norm = np.linalg.norm(got[fine] - want[fine], axis=1)
            lim = (3 * (U16 / 3 ** 0.5 + 3 * delta) * spread + 2.0 ** -20 * size.sum(1)
                   + U16 * np.linalg.norm(want, axis=1) + 1e-37)[fine]
            assert (norm <= lim).all(), (b, h, (norm / lim).max())
            fine = np.isfinite(wl)
            err = np.abs(gl - wl)[fine] / (delta + 2.0 ** -21 + L * U32 + 4 * U32 * np.abs(wl))[fine]
            assert (err <= 1).all(), (b, h, err.max())


def same(a, b):
    """Equal to the bit, but for which NaN it is."""
    return torch.equal(a.nan_to_num(123.0), b.nan_to_num(123.0))


def _tokens_q(s, G, seed=1):
    g = torch.Generator("cuda").manual_seed(seed)
    rows = torch.randn(s.tokens, s.Hk * G + 1, s.D, generator=g, device="cuda").bfloat16()
    return rows[:, 1:]


SHAPES = [  # fmt, D, Hk, G, page
    (dg.DG_KV_BF16, 128, 2, 4, 16), (dg.DG_KV_E4M3, 128, 2, 4, 64), (dg.DG_KV_BF16, 64, 1, 8, 1),
    (dg.DG_KV_E4M3, 256, 2, 1, 32), (dg.DG_KV_BF16, 256, 1, 3, 5), (dg.DG_KV_E4M3, 80, 3, 2, 24),
    (dg.DG_KV_BF16, 16, 1, 16, 128), (dg.DG_KV_E4M3, 176, 1, 5, 7)]


@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("fmt,D,Hk,G,page", SHAPES)
def test_attention_small(fmt, D, Hk, G, page, mask):
    lengths = [(0, 1), (300, 1), (0, 0), (9, 0), (127, 2), (128, 33), (0, 70), (255, 1), (61, 5)]
    s = Setup(lengths, fmt, Hk, D, page, seed=D + G, pad=2)
    q = _tokens_q(s, G)
    words = _tree(s.new, D, empty=(0, 2, 40)) if mask == "tree" else None
    tree = None
    if mask == "tree":
        tree = torch.zeros(s.tokens, words.shape[1], dtype=torch.int32, device="cuda")
        tree[:len(words)] = torch.from_numpy(words.view(np.int32))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    s.cache.attend(q, s.batch, MASKS[mask], tree=tree, scale=0.11, out=out, lse=lse)
    s.cache.check()
    assert (out[-2:] == 7.0).all() and (lse[-2:] == 7.0).all()
    _check_attention(s, q, mask, np.float32(0.11), out, lse, words)


@pytest.mark.parametrize("fmt,D,Hk,G,page,mask,lengths", [
    (dg.DG_KV_BF16, 128, 2, 2, 16, "causal", [(0, 600), (100, 300)]),      # prompts
    (dg.DG_KV_E4M3, 128, 1, 8, 64, "full", [(700, 256), (1, 256)]),        # canvases
    (dg.DG_KV_E4M3, 256, 1, 4, 32, "full", [(333, 256)]),
    (dg.DG_KV_BF16, 64, 1, 4, 24, "causal", [(513, 515)]),
    (dg.DG_KV_BF16, 128, 1, 5, 128, "tree", [(1000, 200), (0, 130)]),
    (dg.DG_KV_E4M3, 64, 2, 8, 8, "causal", [(20000, 1), (3, 1), (7000, 4)]),
    (dg.DG_KV_BF16, 256, 1, 1, 64, "causal", [(9000, 1)]),
    (dg.DG_KV_BF16, 128, 8, 2, 64, "causal", [(40001, 1)])])
def test_attention_long(fmt, D, Hk, G, page, mask, lengths):
    s = Setup(lengths, fmt, Hk, D, page, seed=D)
    q = _tokens_q(s, G, 3)
    words = _tree(s.new, 5) if mask == "tree" else None
    tree = torch.from_numpy(words.view(np.int32)).cuda() if mask == "tree" else None
    out, lse = s.cache.attend(q, s.batch, MASKS[mask], tree=tree)
    s.cache.check()
    _check_attention(s, q, mask, D ** -0.5, out, lse, words,
                     rows=[0, 1, 15, 16, 31, 32, 63, 64, 100, 127, 128, 129, 199, 255, 256, 299, 511, 514, 599])


@pytest.mark.parametrize("fmt,D,Hk,G,page,mask,lengths", [
    (dg.DG_KV_E4M3, 64, 2, 4, 8, "full", [(200, 256), (30, 100)]),         # two row tiles, codes
    (dg.DG_KV_E4M3, 128, 1, 2, 16, "causal", [(0, 700), (131, 400)]),
    (dg.DG_KV_E4M3, 96, 1, 6, 256, "tree", [(900, 61), (0, 90)]),          # G no power of two
    (dg.DG_KV_BF16, 64, 1, 64, 256, "causal", [(500, 9)]),                 # G above 32
    (dg.DG_KV_BF16, 128, 2, 12, 24, "tree", [(77, 40), (500, 33)]),
    (dg.DG_KV_BF16, 128, 3, 1, 128, "full", [(383, 129), (1, 513)]),
    (dg.DG_KV_BF16, 208, 1, 2, 64, "causal", [(70, 300)]),
    (dg.DG_KV_E4M3, 48, 1, 3, 16, "causal", [(300, 150)])])                # below 64: rows one by one
def test_attention_more_shapes(fmt, D, Hk, G, page, mask, lengths):
    s = Setup(lengths, fmt, Hk, D, page, seed=D + page)
    q = _tokens_q(s, G, 4)
    words = _tree(s.new, 8, empty=(3, 50)) if mask == "tree" else None
    tree = torch.from_numpy(words.view(np.int32)).cuda() if mask == "tree" else None
    out, lse = s.cache.attend(q, s.batch, MASKS[mask], tree=tree)
    s.cache.check()
    _check_attention(s, q, mask, D ** -0.5, out, lse, words)


@pytest.mark.parametrize("D", [64, 48])                  # queries by TMA, and row by row
def test_other_orders_of_the_rows(D):
    """Heads outermost, every other token of a buffer, and one row shared by all heads."""
    lengths, Hk, G = [(30, 40), (3, 7)], 2, 4
    s = Setup(lengths, dg.DG_KV_E4M3, Hk, D, 16, seed=D, fill=False)
    n = s.tokens
    kv = torch.randn(2, Hk, 2 * n, D, generator=s.g, device="cuda").bfloat16()
    k, v = kv[0, :, ::2].transpose(0, 1), kv[1, :, 1::2].transpose(0, 1)
    for b, (p, _) in enumerate(lengths):
        s.put(b, torch.randn(2, p, Hk, D, generator=s.g, device="cuda"))
    s.cache.write(k, v, s.batch)
    back = s.cache.read(s.batch, torch.float32)
    s2 = Setup(lengths, dg.DG_KV_E4M3, Hk, D, 16, seed=D, fill=False)
    s2.cache.write(k.contiguous(), v.contiguous(), s2.batch)
    for x, y in zip(back, s2.cache.read(s2.batch, torch.float32)):
        assert torch.equal(x, y)
    heads_outer = torch.randn(Hk * G, n, D, generator=s.g, device="cuda").bfloat16().transpose(0, 1)
    shared = heads_outer[:, :1].expand(-1, Hk * G, -1)
    for q in (heads_outer, shared):
        out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
        _check_attention(s, q, "causal", D ** -0.5, out, lse)
    pos, freq = torch.arange(n, device="cuda").int(), dg.rope_frequencies(32)
    a, b = dg.qk_norm_rope(heads_outer, k, None, None, pos, freq)
    _check_norm(heads_outer, a, None, pos, freq, False, 1e-6, 0.0, U16)
    _check_norm(k, b, None, pos, freq, False, 1e-6, 0.0, U16)
    with pytest.raises(ValueError):
        s.cache.attend(heads_outer.transpose(1, 2), s.batch, dg.DG_MASK_CAUSAL)


@pytest.mark.parametrize("fmt", [dg.DG_KV_BF16, dg.DG_KV_E4M3])
def test_shared_pages_and_a_page_twice(fmt):
    """Sequences over one prefix, and a table that names a page twice: the pasts are only read."""
    s = Setup([(96, 3), (96, 1), (80, 20)], fmt, 2, 128, 16, seed=6)
    s.table[1, :6] = s.table[0, :6]
    s.table[2, :3] = s.table[0, 1]
    q = _tokens_q(s, 4)
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    s.cache.check()
    _check_attention(s, q, "causal", 128 ** -0.5, out, lse)


@pytest.mark.parametrize("new", [1, 40])
def test_exponents_at_any_address(new):
    """Exponents that lie at an odd byte are read as the same ones."""
    s = Setup([(200, new), (33, 2)], dg.DG_KV_E4M3, 2, 128, 16, seed=8)
    c = s.cache
    room = [torch.zeros(c.k_exp.numel() + 1, dtype=torch.uint8, device="cuda") for _ in "kv"]
    odd = [r[1:].view(c.k_exp.shape) for r in room]
    for o, e in zip(odd, (c.k_exp, c.v_exp)):
        o.copy_(e)
    q = _tokens_q(s, 4)
    out, lse = dg.KVCache(c.k, c.v, *odd).attend(q, s.batch, dg.DG_MASK_CAUSAL)
    _check_attention(s, q, "causal", 128 ** -0.5, out, lse)


@pytest.mark.parametrize("words", [0, 1, 5])
def test_tree_rows_of_other_widths(words):
    """Words that are missing count as zero, those beyond the new tokens are not looked at."""
    s = Setup([(40, 50), (0, 3), (7, 64)], dg.DG_KV_BF16, 2, 64, 16, seed=9)
    q = _tokens_q(s, 2)
    bits = np.zeros((s.tokens, max(words, 2)), dtype=np.uint32)
    bits[:, :2] = _tree(s.new, 4)
    bits[:, 2:] = 0xFFFFFFFF
    tree = torch.from_numpy(bits[:, :words].copy().view(np.int32)).cuda()
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_TREE, tree=tree)
    s.cache.check()
    bits[:, words:] = 0
    _check_attention(s, q, "tree", 0.125, out, lse, bits)


def test_attention_of_the_largest_batch():
    s = Setup([(b % 37, 1 + (b % 5 == 0)) for b in range(1024)], dg.DG_KV_BF16, 1, 64, 16, seed=1)
    q = _tokens_q(s, 2)
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    s.cache.check()
    _check_attention(s, q, "causal", 0.125, out, lse)
    big = dg.KVBatch(torch.zeros(1025, 1, dtype=torch.int32, device="cuda"),
                     torch.zeros(1026, dtype=torch.int32, device="cuda"),
                     torch.zeros(1025, dtype=torch.int32, device="cuda"), s.tokens)
    with pytest.raises(dg.DgError):
        s.cache.attend(q, big, dg.DG_MASK_CAUSAL)


@pytest.mark.parametrize("kexp,vexp", [(-20, 30), (25, -40), (60, 90)])
def test_attention_over_rows_of_extreme_scale(kexp, vexp):
    """Exponents far from zero, beyond the range of fp16."""
    s = Setup([(150, 3), (20, 1)], dg.DG_KV_E4M3, 2, 128, 16, seed=2)
    for b in range(2):
        n = s.past[b] + s.new[b]
        rows = dg.KVBatch(s.table[b:b + 1].contiguous(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.zeros(1, dtype=torch.int32, device="cuda"), n)
        kv = torch.randn(2, n, 2, 128, generator=s.g, device="cuda")
        kv[1] *= torch.exp2(torch.randint(-6, 7, (n, 2, 1), generator=s.g, device="cuda").float())
        s.cache.write(kv[0] * 2.0 ** kexp, kv[1] * 2.0 ** vexp, rows)
    q = (_tokens_q(s, 4, 5).float() * 2.0 ** -kexp).bfloat16()
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    s.cache.check()
    _check_attention(s, q, "causal", 128 ** -0.5, out, lse)


def test_attention_large_logits_and_growing_maxima():
    """Logits up to hundreds, rising along the keys, so that the running maximum moves often."""
    s = Setup([(1000, 3)], dg.DG_KV_BF16, 1, 64, 16, seed=8)
    q = torch.ones(3, 4, 64, device="cuda").bfloat16()
    ramp = torch.linspace(-2, 2, 1003, device="cuda")[:, None, None].expand(-1, 1, 64)
    s.put(0, torch.stack((ramp, torch.randn(1003, 1, 64, generator=s.g, device="cuda"))))
    for scale in (0.01, 1.0, 4.0):
        out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL, scale=scale)
        _check_attention(s, q, "causal", scale, out, lse)


@pytest.mark.parametrize("fmt", [dg.DG_KV_BF16, dg.DG_KV_E4M3])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 2)])
def test_attention_single_tokens_of_a_ragged_batch(fmt, D, G):
    """Few rows in each tile, several items to a CTA and several CTAs to an item."""
    lengths = [(8000 - 233 * b, 1 if b % 8 != 7 else 0) for b in range(33)]
    s = Setup(lengths, fmt, 4, D, 64, seed=D)
    q = _tokens_q(s, G, 2)
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    s.cache.check()
    _check_attention(s, q, "causal", D ** -0.5, out, lse)


@pytest.mark.parametrize("fmt", [dg.DG_KV_BF16, dg.DG_KV_E4M3])
@pytest.mark.parametrize("D,G,new", [(128, 2, 40), (64, 1, 5), (256, 2, 70), (128, 8, 100)])
def test_what_is_masked_does_not_touch_a_row(fmt, D, G, new):
    """NaN (and infinities) in the keys and values of some new tokens: rows that do not see them are
    as before to the bit, rows that see them are not finite."""
    s = Setup([(130, new)], fmt, 1, D, 16, seed=D + new)
    q = _tokens_q(s, G, 5)
    words = _tree(s.new, 9)
    bad = [2, new // 2, new - 1]
    for i in range(new):                               # token 0 and its like see none of the bad ones
        for j in bad:
            if i % 3 == 0:
                words[i, j // 32] &= ~np.uint32(1 << (j % 32))
    tree = torch.from_numpy(words.view(np.int32)).cuda()
    good, good_lse = s.cache.attend(q, s.batch, dg.DG_MASK_TREE, tree=tree)
    causal, _ = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    for n, j in enumerate(bad):
        page, place = s.at(0, 130 + j, 131 + j)
        for name in "kv":
            t = getattr(s.cache, name)
            if fmt == dg.DG_KV_BF16:
                t[page, :, place, ::5] = [float("nan"), float("inf"), -float("inf")][n]
            else:
                t.view(torch.uint8)[page, :, place, ::5] = 0x7F
    for mask, want, seen in (
            (dg.DG_MASK_TREE, good, lambda i: any(words[i, j // 32] >> (j % 32) & 1 for j in bad)),
            (dg.DG_MASK_CAUSAL, causal, lambda i: i >= 2)):
        out, lse = s.cache.attend(q, s.batch, mask, tree=tree if mask == dg.DG_MASK_TREE else None)
        for i in range(new):
            if seen(i):
                assert not out[i].float().isfinite().all(), (mask, i)
            else:
                assert same(out[i], want[i]), (mask, i)
    # values alone: the infinities of a seen token come out as they are
    if fmt == dg.DG_KV_BF16:
        s = Setup([(4, 3)], fmt, 1, D, 16, seed=1)
        page, place = s.at(0, 5, 6)
        s.cache.v[page, :, place, 7] = float("inf")
        s.cache.v[page, :, place, 9] = -float("inf")
        out, lse = s.cache.attend(q[:3], s.batch, dg.DG_MASK_CAUSAL)
        assert out[0].float().isfinite().all() and lse.isfinite().all()
        assert (out[1:, :, 7] == float("inf")).all() and (out[1:, :, 9] == -float("inf")).all()
        rest = [d for d in range(D) if d not in (7, 9)]
        assert out[1:, :, rest].float().isfinite().all()


@pytest.mark.parametrize("G,new", [(1, 1), (8, 1), (8, 30)])
def test_infinite_values_of_the_past_come_out(G, new):
    s = Setup([(500, new), (40, new)], dg.DG_KV_BF16, 1, 128, 16, seed=G)
    q = _tokens_q(s, G, 5)
    want, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    for pos, d, x in ((3, 7, float("inf")), (300, 9, -float("inf")), (499, 11, float("nan")), (77, 7, 1.0)):
        page, place = s.at(0, pos, pos + 1)
        s.cache.v[page, :, place, d] = x
    out, lse2 = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    assert (out[:new, :, 7] == float("inf")).all() and (out[:new, :, 9] == -float("inf")).all()
    assert out[:new, :, 11].isnan().all() and torch.equal(lse, lse2)
    rest = [d for d in range(128) if d not in (7, 9, 11)]
    assert torch.equal(out[:, :, rest], want[:, :, rest]) and torch.equal(out[new:], want[new:])


def test_attention_reports_bad_pages():
    s = Setup([(40, 2)], dg.DG_KV_BF16, 1, 64, 16, seed=2)
    q = _tokens_q(s, 2)
    s.table[0, 1] = -5                                 # positions 16..31 read as zeros
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    assert int(s.cache.status) == dg.DG_EINVAL and out.float().isfinite().all()
    s.cache.status.zero_()
    s.batch.past.fill_(2 ** 31 - 1)
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    assert int(s.cache.status) == dg.DG_EINVAL


def test_attention_is_repeatable_and_keeps_nothing_in_its_scratch():
    s = Setup([(3000, 1), (500, 7), (0, 129)], dg.DG_KV_E4M3, 2, 128, 32, seed=6)
    q = _tokens_q(s, 4)
    a, la = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    n = dg.dg_cache_attention_scratch_bytes(s.cache.c, s.batch.c, q.shape[1])
    for fill in (0, 0xFF):
        scratch = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(a), torch.empty_like(la)
        dg.dg_cache_attention(s.cache.c, s.batch.c, q.shape[1], q.data_ptr(), q.stride(0), q.stride(1),
                              128 ** -0.5, dg.DG_MASK_CAUSAL, 0, 0, out.data_ptr(), lse.data_ptr(),
                              scratch.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert same(a, out) and same(la, lse)
        dg.dg_cache_attention(s.cache.c, s.batch.c, q.shape[1], q.data_ptr(), q.stride(0), q.stride(1),
                              128 ** -0.5, dg.DG_MASK_CAUSAL, 0, 0, out.data_ptr(), 0,
                              scratch.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert same(a, out)


@pytest.mark.parametrize("fmt", [dg.DG_KV_BF16, dg.DG_KV_E4M3])
@pytest.mark.parametrize("D,G,page,mask,lengths", [
    (128, 4, 64, "causal", [(3000 - 91 * b, 1) for b in range(33)]), (64, 8, 16, "causal", [(2500, 1), (9000, 1)]),
    (256, 2, 32, "full", [(1500, 128), (700, 100)]), (128, 2, 16, "causal", [(0, 1500), (200, 900)]),
    (64, 4, 128, "full", [(900, 300)]), (128, 3, 5, "causal", [(400, 200), (3000, 1)])])
def test_repeated_calls_agree_to_the_bit(fmt, D, G, page, mask, lengths):
    """Hand-overs between warps that went wrong now and then would show here."""
    s = Setup(lengths, fmt, 4, D, page, seed=D + G)
    q = _tokens_q(s, G, 2)
    want, lse = s.cache.attend(q, s.batch, MASKS[mask])
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    bits, lbits = want.view(torch.int16), lse.view(torch.int32)
    for _ in range(60):
        out, l = s.cache.attend(q, s.batch, MASKS[mask])
        off += (out.view(torch.int16) != bits).sum() + (l.view(torch.int32) != lbits).sum()
    assert int(off) == 0
    s.cache.check()


def test_captured_graph_follows_the_lengths():
    """One captured layer step replayed while the sequences grow, against eager calls."""
    Hk, G, D = 2, 4, 128
    s = Setup([(1000, 1), (64, 1)], dg.DG_KV_E4M3, Hk, D, 16, seed=3)
    x = torch.randn(2, Hk * G + 2 * Hk, D, device="cuda").bfloat16()
    pos, freq = torch.tensor([1000, 64], dtype=torch.int32, device="cuda"), dg.rope_frequencies(D)

    def step():
        q, k = dg.qk_norm_rope(x[:, :Hk * G], x[:, Hk * G:Hk * G + Hk], None, None, pos, freq)
        s.cache.write(k, x[:, Hk * G + Hk:], s.batch)
        return s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out, lse = step()
    for past in ([1000, 64], [990, 79], [5, 0], [700, 33]):
        s.batch.past.copy_(torch.tensor(past, dtype=torch.int32))
        pos.copy_(s.batch.past)
        x.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        want = step()
        assert same(got[0], want[0]) and same(got[1], want[1]), past
    s.cache.check()
    del graph


def test_two_streams_at_once():
    s = Setup([(2000, 3), (900, 5)], dg.DG_KV_BF16, 2, 128, 16, seed=7)
    q = _tokens_q(s, 4)
    want = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    full = s.cache.attend(q, s.batch, dg.DG_MASK_FULL)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for n, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[n].append(s.cache.attend(q, s.batch, [dg.DG_MASK_CAUSAL, dg.DG_MASK_FULL][n]))
    torch.cuda.synchronize()
    for n, ref in enumerate((want, full)):
        for o, l in got[n]:
            assert same(o, ref[0]) and same(l, ref[1])


def test_beside_the_denoise_step():
    """A denoise block on its own stream while attention calls run on another: both as when alone."""
    import synthetic
    w = synthetic.SMALL.replace(C=128, V=4096, d=256, tau=0.5 * 128 * np.log(2), max_steps=4)
    den = dg.Denoiser(w, synthetic.make_embedding(w).cuda())
    want, steps = den.block(0)
    want = want.clone()
    s = Setup([(3000, 2), (500, 9)], dg.DG_KV_E4M3, 2, 128, 16, seed=3)
    q = _tokens_q(s, 4)
    alone = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    torch.cuda.synchronize()
    for _ in range(5):
        got = [s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL) for _ in range(8)]
        out, n = den.block(0)
        torch.cuda.synchronize()
        assert n == steps and torch.equal(out, want)
        assert all(same(o, alone[0]) and same(l, alone[1]) for o, l in got)
    den.close()


def test_rows_beyond_four_gigabytes():
    """A cache of over 2^32 bytes (and elements); the sequence lies at its far end."""
    Hk, D, page = 8, 128, 64
    pages = 2 ** 32 // (Hk * page * D) + 100
    k = torch.empty(pages, Hk, page, D, dtype=torch.uint8, device="cuda").view(F8)
    v = torch.empty(pages, Hk, page, D, dtype=torch.uint8, device="cuda").view(F8)
    ke, ve = (torch.empty(pages, Hk, page, dtype=torch.uint8, device="cuda") for _ in "kv")
    cache = dg.KVCache(k, v, ke, ve)
    s = Setup([(0, 200)], dg.DG_KV_E4M3, Hk, D, page, seed=1)
    s.cache = cache
    s.table.copy_(torch.arange(pages - 4, pages, dtype=torch.int32)[None])
    x = torch.randn(2, 200, Hk, D, device="cuda").bfloat16()
    cache.write(x[0], x[1], s.batch)
    got = cache.read(s.batch, torch.float32)
    for n, (o, src) in enumerate(zip(got, x)):
        want = np.array([[A.dequantise(*A.quantise(r)) for r in t] for t in f64(src[::40])])
        assert np.array_equal(f64(o[::40]), want)
    q = _tokens_q(s, 2)
    out, lse = cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    cache.check()
    _check_attention(s, q, "causal", D ** -0.5, out, lse, rows=[0, 63, 64, 199])


def test_a_layer_through_a_prompt_a_canvas_and_a_draft():
    """norm and rotation, write, attention as a backbone runs them, against the oracle on the
    operators' own inputs at each stage: a causal prompt, two denoise steps of a canvas over it (each
    rewrites the canvas's rows), then a tree of drafts after the committed canvas."""
    Hk, G, D, page = 2, 2, 64, 16
    r = torch.Generator("cuda").manual_seed(12)
    s = Setup([(0, 150), (0, 41)], dg.DG_KV_E4M3, Hk, D, page, seed=12, fill=False)
    table = torch.randperm(64, generator=r, device="cuda").int().reshape(2, 32)
    s.cache, s.table = dg.KVCache.empty(64, page, Hk, D, dg.DG_KV_E4M3), table
    freq = dg.rope_frequencies(32)
    past = [0, 0]
    stages = [("causal", [150, 41]), ("full", [32, 32]), ("full", [32, 32]), ("commit", None), ("tree", [9, 17])]
    for n, (mask, new) in enumerate(stages):
        if mask == "commit":
            past = [p + 32 for p in past]
            continue
        s.past, s.new = past, new
        s.first = np.concatenate([[0], np.cumsum(new)])
        s.tokens = int(s.first[-1])
        dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        s.batch = dg.KVBatch(table, dev(s.first), dev(past), s.tokens)
        x = torch.randn(s.tokens, Hk * G + 2 * Hk, D, generator=r, device="cuda").bfloat16()
        pos = dev(np.concatenate([p + np.arange(m) for p, m in zip(past, new)]))
        q0, k0, v = x[:, :Hk * G], x[:, Hk * G:Hk * G + Hk], x[:, Hk * G + Hk:]
        q, k = dg.qk_norm_rope(q0, k0, None, None, pos, freq)
        _check_norm(k0, k, None, pos, freq, False, 1e-6, 0.0, U16)
        s.cache.write(k, v, s.batch)
        back, _ = s.cache.read(s.batch, torch.float32)
        err = np.abs(f64(back) - f64(k))
        assert (err <= 2.0 ** -4 * np.abs(f64(k)) + 2.0 ** -9 * np.abs(f64(k)).max(-1, keepdims=True) / 224).all()
        words = _tree(new, n) if mask == "tree" else None
        tree = torch.from_numpy(words.view(np.int32)).cuda() if mask == "tree" else None
        out, lse = s.cache.attend(q, s.batch, MASKS[mask], tree=tree)
        s.cache.check()
        _check_attention(s, q, mask, D ** -0.5, out, lse, words, rows=range(0, 150, 7))
        if mask == "causal":
            past = list(new)
