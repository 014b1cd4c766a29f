"""Attention-layer operators at the edges of their contract: against the fp64 oracle with the
tolerances of test_attention_layer_gpu.py, and against themselves."""
import numpy as np
import pytest
import torch

import uniform_state_text_b200 as dg
from oracle import attention as A
from test_attention_layer_gpu import MASKS, U16, U32, Setup, _check_attention, _check_norm, _tokens_q, _tree, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from uniform_state_text_b200 import build
    build.build()
    dg.lib()


# ----------------------------------------------------------------------------- the plan and the first copies
@pytest.mark.parametrize("batch,D,G", [(1, 128, 2), (1024, 64, 1), (1024, 128, 2), (1024, 256, 1), (33, 128, 150)])
def test_first_tiles_over_the_plan(batch, D, G):
    """The split's sums (one per sequence) lie where the first key tiles are copied to: the largest
    batch and the smallest, pages by TMA, a hundred times the same to the bit."""
    s = Setup([(120 + b % 9, 1) for b in range(batch)], dg.DG_KV_BF16, 1, D, 128, seed=D)
    q = _tokens_q(s, G, 3)
    want, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    s.cache.check()
    _check_attention(s, q, "causal", D ** -0.5, want, lse)
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        out, l = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
        off += (out.view(torch.int16) != want.view(torch.int16)).sum()
        off += (l.view(torch.int32) != lse.view(torch.int32)).sum()
    assert int(off) == 0
    s.cache.check()


# ----------------------------------------------------------------------------- infinite logits
class Setup16(Setup):
    """A cache whose rows may lie beyond bf16's range (an exponent above 246 in a caller's own cache):
    they enter the products as infinities."""

    def values(self, b, n, start, stop):
        x = super().values(b, n, start, stop)
        return np.where(np.abs(x) > float(torch.finfo(torch.bfloat16).max), np.copysign(np.inf, x), x)


def _infinite(s, name, b, pos, element, sign=1):
    """An infinity at one element of one row; in e4m3 by the largest code and an exponent of 2^127."""
    page, place = s.at(b, pos, pos + 1)
    t = getattr(s.cache, name)
    if s.fmt == dg.DG_KV_BF16:
        t[page, :, place, element] = sign * float("inf")
    else:
        t.view(torch.uint8)[page, :, place] = 0
        t.view(torch.uint8)[page, :, place, element] = 0x7E if sign > 0 else 0xFE
        getattr(s.cache, name + "_exp")[page, :, place] = 254


def _check_lse(s, q, mask, scale, lse):
    """lse is infinite or NaN where the oracle's is, and so."""
    for b, (p, n) in enumerate(zip(s.past, s.new)):
        K, V = (s.values(b, x, 0, p + n) for x in "kv")
        at = s.first[b] + np.arange(n)
        seen = np.stack([A.seen_by(i, p, n, mask) for i in range(n)])
        for h in range(0, q.shape[1], 3):
            g = h // (q.shape[1] // s.Hk)
            want = A.attend(f64(q)[at, h], K[:, g], V[:, g], seen, scale)[1]
            got = f64(lse)[at, h]
            bad = ~np.isfinite(want)
            assert np.array_equal(got[bad], want[bad], equal_nan=True) and np.isfinite(got[~bad]).all(), (b, h)


@pytest.mark.parametrize("fmt", [dg.DG_KV_BF16, dg.DG_KV_E4M3])
@pytest.mark.parametrize("D,G,new", [(64, 8, 30), (128, 8, 30), (128, 2, 3), (256, 2, 70)])
def test_infinite_logits_at_every_column(fmt, D, G, new):
    """One infinite element of one past key, at each place of 16 neighbours and in other tiles: rows whose
    logit is +inf are NaN, those whose logit is -inf have weight 0 there (times an infinite value: NaN)."""
    for pos in [*range(208, 224), 3, 499]:
        s = Setup16([(500, new)], fmt, 1, D, 16, seed=D + new)
        q = _tokens_q(s, G, 5)
        _infinite(s, "k", 0, pos, 5)
        _infinite(s, "v", 0, pos, 7)
        out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
        s.cache.check()
        _check_attention(s, q, "causal", D ** -0.5, out, lse)
        _check_lse(s, q, "causal", D ** -0.5, lse)


@pytest.mark.parametrize("D,G,new", [(64, 8, 30), (128, 8, 20), (128, 2, 3), (256, 2, 9)])
def test_infinite_logits_within_one_share(D, G, new):
    """Many sequences, so that one CTA goes through the tiles before and behind the infinite one."""
    s = Setup([(300, new)] * 60, dg.DG_KV_BF16, 4, D, 16, seed=D + new)
    q = _tokens_q(s, G, 5)
    for b in range(60):
        _infinite(s, "k", b, (b * 37) % (300 + new), 5)
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    s.cache.check()
    _check_attention(s, q, "causal", D ** -0.5, out, lse)
    _check_lse(s, q, "causal", D ** -0.5, lse)


@pytest.mark.parametrize("mask", ["causal", "full"])
@pytest.mark.parametrize("D,G,new,batch", [(64, 8, 40, 1), (128, 8, 30, 1), (128, 2, 3, 1), (256, 2, 70, 1),
                                           (64, 8, 40, 60), (128, 8, 30, 60), (128, 2, 3, 60)])
def test_rows_whose_logits_are_all_minus_infinity(D, G, new, batch, mask):
    """They weigh nothing, like rows that see nothing; and a row of +inf and finite logits is NaN."""
    s = Setup([(500, new)] * batch, dg.DG_KV_BF16, 1, D, 16, seed=D)
    q = _tokens_q(s, G, 5)
    s.cache.k[..., 5] = -float("inf")
    out, lse = s.cache.attend(q, s.batch, MASKS[mask])
    s.cache.check()
    _check_attention(s, q, mask, D ** -0.5, out, lse)
    down = q[..., 5] > 0
    assert not out[down].any() and (lse[down] == -float("inf")).all()
    assert out[~down].isnan().all() and lse[~down].isnan().all()


@pytest.mark.parametrize("batch", [1, 40])
@pytest.mark.parametrize("G,new", [(8, 30), (2, 3)])
def test_logits_beyond_fp32(G, new, batch):
    """q.k beyond fp32 counts as infinite; a finite q.k whose scaled logit lies beyond fp32, or is too
    large for its fraction to be held, still gets the softmax's weights."""
    s = Setup([(500, new)] * batch, dg.DG_KV_BF16, 1, 64, 16, seed=3)
    q = torch.ones_like(_tokens_q(s, G, 5))
    for big, qs, scale in ((2.0 ** 100, 2.0 ** 40, 1.0), (2.0 ** 115, 1.0, 2.0 ** 10)):
        for sign in (1, -1):
            for b in range(batch):
                page, place = s.at(b, 215, 216)
                s.cache.k[page, :, place] = sign * big
            out, lse = s.cache.attend(q * qs, s.batch, dg.DG_MASK_FULL, scale=scale)
            s.cache.check()
            if sign > 0 and scale == 1.0:
                assert out.isnan().all() and lse.isnan().all()
                continue
            # where one key is ahead by far it has all the weight
            for b in range(batch):
                K, V = (s.values(b, x, 0, 500 + new)[:, 0] for x in "kv")
                z = K.sum(1) * qs * scale
                top = int(z.argmax())
                rows = slice(int(s.first[b]), int(s.first[b + 1]))
                err = np.abs(f64(out[rows]) - V[top]).max() if np.sort(z)[-2] < z[top] - 1000 else 0.0
                assert err == 0.0, (b, err)
                assert not out[rows].isnan().any()
                got, want = f64(lse[rows]), z[top] + np.log(np.exp(z - z[top]).sum())
                delta = (64 * 2.0 ** -23 + 4 * U32) * (np.abs(K).sum(1) * qs * scale).max()   # of a logit, as there
                assert (np.isposinf(got) if want > 3.5e38 else np.abs(got - want) <= delta + 2.0 ** -20).all()


@pytest.mark.parametrize("step", [0.0, 0.5])
@pytest.mark.parametrize("size", [1e5, 3e7, 1e9, 1e20])
@pytest.mark.parametrize("G,new,batch", [(8, 30, 1), (8, 30, 30), (2, 3, 1), (2, 3, 60)])
def test_large_logits(G, new, batch, size, step):
    """Rows whose logits are all near one large number: the values' mean where they are equal, the weights
    of their differences where those are held; and never NaN."""
    s = Setup([(500, new)] * batch, dg.DG_KV_BF16, 1, 64, 16, seed=3)
    s.cache.k.zero_()
    s.cache.k[..., 0] = 1.0
    s.cache.k[..., 1] = step * torch.randint(0, 3, s.cache.k.shape[:3], generator=s.g, device="cuda")
    for sign in (1, -1):
        q = torch.zeros_like(_tokens_q(s, G, 5))
        q[..., 0] = sign * size
        q[..., 1] = torch.randn(q.shape[:2], generator=s.g, device="cuda")
        scale = 1.0 if size < 1e6 else 0.25
        out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL, scale=scale)
        s.cache.check()
        assert out.float().isfinite().all() and lse.isfinite().all()
        if step == 0.0 or size < 1e6:
            _check_attention(s, q, "causal", scale, out, lse)


# ----------------------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("mask", ["causal", "tree"])
@pytest.mark.parametrize("fmt", [dg.DG_KV_BF16, dg.DG_KV_E4M3])
@pytest.mark.parametrize("D,G,new,batch", [(64, 2, 20, 1), (128, 8, 30, 1), (128, 2, 140, 1), (256, 2, 70, 1),
                                           (128, 2, 20, 40), (64, 8, 24, 30), (256, 1, 9, 40)])
def test_values_that_are_not_finite_meet(fmt, D, G, new, batch, mask):
    """Infinities and NaN of the past and of new tokens in one column add up as numbers do, in the
    pieces of several CTAs and within one CTA's share."""
    s = Setup16([(500, new), (3, new)] * batch, fmt, 2 if batch == 1 else 4, D, 16, seed=D + new)
    q = _tokens_q(s, G, 5)
    nan = float("nan")
    for b, p in enumerate(s.past):
        for pos, e, sign in ((1, 7, -1), (p + 1, 7, 1), (p + 2, 9, 1), (p + 4, 9, -1), (p + 6, 12, -1), (0, 12, -1),
                             (p + new - 1, 15, 1)):
            _infinite(s, "v", b, pos, e, sign)
        page, place = s.at(b, 2, 3)
        if fmt == dg.DG_KV_BF16:
            s.cache.v[page, :, place, 11] = nan
        else:
            s.cache.v.view(torch.uint8)[page, :, place, 11] = 0x7F
        _infinite(s, "v", b, p + 3, 11)
    words = _tree(s.new, 3, empty=(5,)) if mask == "tree" else None
    tree = torch.from_numpy(words.view(np.int32)).cuda() if mask == "tree" else None
    out, lse = s.cache.attend(q, s.batch, MASKS[mask], tree=tree)
    s.cache.check()
    _check_attention(s, q, mask, D ** -0.5, out, lse, words)


# ----------------------------------------------------------------------------- the rotation's angle
def _turns(pos, freq):
    """pos freq / 2 pi mod 1 from whole numbers: pi by Machin's formula to 300 bits."""
    one = 1 << 300

    def arctan_inverse(n):
        total, term, k = 0, one // n, 0
        while term:
            total += term // (2 * k + 1) * (1 - 2 * (k & 1))
            term //= n * n
            k += 1
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    top, bottom = float(freq).as_integer_ratio()
    return (int(pos) * top * one * one // (bottom * 2 * pi) % one) / one


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_angles_at_far_positions(sign, interleaved):
    """Every angle is right to 2^-25 turns, for frequencies of either sign up to 1000. A pair (1, 0) comes
    out as one number times (cos t, sin t); sine, cosine and product add 3 u32 to the angle, in radians
    (2 u32 of the function and u32 of the product, relative, on either)."""
    r = np.random.default_rng(5)
    freq = sign * np.concatenate([10.0 ** r.uniform(-6, 2.99, 96), r.uniform(0, 2 * np.pi, 30), [0.0, 999.9]])
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1234567, -2 ** 30 - 1, 1, -1, 0, 131071]
    x = torch.zeros(len(pos), 1, 256, device="cuda")
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 128), slice(128, 256))
    x[..., first] = 1.0
    y, _ = dg.qk_norm_rope(x, x[:, :0], None, None, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                           torch.from_numpy(freq).cuda(), interleaved=interleaved, eps=0.0)
    y = f64(y)[:, 0]
    got = np.arctan2(y[:, second], y[:, first]) / (2 * np.pi)
    want = np.array([[_turns(p, f) for f in freq] for p in pos])
    err = np.abs((got - want + 0.5) % 1 - 0.5)
    assert err.max() <= 2.0 ** -25 + 3 * U32 / (2 * np.pi), err.max() * 2 ** 25


# ----------------------------------------------------------------------------- the owners
def test_a_refused_batch_leaves_no_size_behind():
    """A batch that the library refuses, then a right one of the same tokens, sequences and heads."""
    s = Setup([(40, 3)], dg.DG_KV_BF16, 1, 64, 1024, seed=1)
    q = _tokens_q(s, 2)
    wide = torch.zeros(1, 1 << 21, dtype=torch.int32, device="cuda")       # 2^31 positions
    bad = dg.KVBatch(wide, s.batch.first, s.batch.past, s.tokens)
    with pytest.raises(dg.DgError) as e:
        s.cache.attend(q, bad, dg.DG_MASK_CAUSAL)
    assert e.value.code == dg.DG_EUNSUPPORTED
    out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    _check_attention(s, q, "causal", 0.125, out, lse)


def test_sizes_kept_for_many_token_counts_are_bounded():
    s = Setup([(5, 600)], dg.DG_KV_BF16, 1, 64, 16, seed=1)
    q = _tokens_q(s, 1)
    for n in range(1, 600):
        s.cache.attend(q[:n], dg.KVBatch(s.table, s.batch.first.clamp(max=n), s.batch.past, n), dg.DG_MASK_CAUSAL)
    s.cache.check()
    assert len(s.cache._scratch) <= 64


# ----------------------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("fmt,D,G,page,new", [
    (dg.DG_KV_BF16, 128, 2, 64, 1), (dg.DG_KV_BF16, 128, 8, 64, 33), (dg.DG_KV_E4M3, 128, 2, 64, 1),
    (dg.DG_KV_E4M3, 64, 8, 64, 33), (dg.DG_KV_E4M3, 256, 2, 32, 4), (dg.DG_KV_BF16, 256, 3, 16, 5),
    (dg.DG_KV_BF16, 64, 3, 5, 70), (dg.DG_KV_E4M3, 48, 40, 5, 2)])      # single rows; queries row by row
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(fmt, D, G, page, new):
    """One hand-over withheld at a CTA's first, third or tenth key tile, limit 20 ms: the call returns with
    DG_ETIMEOUT in the status word, copies drained, and the next call is as before to the bit."""
    s = Setup([(3000 - 61 * b, new) for b in range(20)], fmt, 4, D, page, seed=D)
    q = _tokens_q(s, G, 2)
    want, lse = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
    s.cache.check()
    try:
        for tile in (1, 3, 10):
            dg.dg_cache_attention_inject_stall(20_000_000, tile)
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
            end.record()
            with pytest.raises(dg.DgError) as e:
                s.cache.check()
            assert e.value.code == dg.DG_ETIMEOUT
            assert 15 < start.elapsed_time(end) < 500            # ms; well under the default 2 s
            dg.dg_cache_attention_inject_stall(0, 0)
            s.cache.status.zero_()
            out, l = s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)
            s.cache.check()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
            assert torch.equal(l.view(torch.int32), lse.view(torch.int32))
    finally:
        dg.dg_cache_attention_inject_stall(0, 0)


@pytest.mark.parametrize("fmt", [dg.DG_KV_BF16, dg.DG_KV_E4M3])
def test_a_long_search_for_infinities_is_no_stall(fmt):
    """Searching a long tree's values for infinities takes each row longer than the (shortened) limit of a
    wait, and is progress all the same."""
    n = 4000
    s = Setup16([(0, n), (0, n)], fmt, 1, 64, 64, seed=2)
    q = _tokens_q(s, 1)
    _infinite(s, "v", 0, 0, 7)
    _infinite(s, "v", 1, n - 1, 7)
    bits = np.packbits(np.tri(n, 4000, dtype=np.uint8), axis=1, bitorder="little").view(np.uint32)
    bits = np.concatenate([bits, bits])
    tree = torch.from_numpy(bits.view(np.int32)).cuda()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    try:
        dg.dg_cache_attention_inject_stall(1_000_000, 0)
        start.record()
        out, lse = s.cache.attend(q, s.batch, dg.DG_MASK_TREE, tree=tree)
        end.record()
        s.cache.check()
    finally:
        dg.dg_cache_attention_inject_stall(0, 0)
    assert start.elapsed_time(end) > 2                  # ms: the search did take longer than the limit
    _check_attention(s, q, "tree", 0.125, out, lse, bits, rows=[0, 1, 77, 1999, 3000, n - 2, n - 1])


def test_check_waits_for_calls_of_other_streams():
    """A bad page met on a side stream, behind work that takes a while."""
    s = Setup([(40, 3)], dg.DG_KV_BF16, 1, 64, 16, seed=1)
    q = _tokens_q(s, 2)
    x = torch.randn(8192, 8192, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def work():
        y = x
        for _ in range(20):
            y = y @ y
            y /= y.norm()
        s.cache.attend(q, s.batch, dg.DG_MASK_CAUSAL)

    with torch.cuda.stream(side):                       # allocations, which would wait, made beforehand
        work()
    s.cache.check()
    s.table[0, 1] = -1
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        work()
    with pytest.raises(dg.DgError) as e:
        s.cache.check()
    assert e.value.code == dg.DG_EINVAL
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------- norms of very large and small rows
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-33, 1e30])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 32, False), (128, 128, True), (256, 64, False)])
def test_norms_of_rows_whose_squares_leave_fp32(D, rot, interleaved, eps, dt):
    """Rows from 1e-38 to 1e38, side by side: the squares' sum is far beyond fp32 or vanishes in it."""
    sizes = [1.0, 1e-38, 1e38, 1e-25, 1e25, 1e-20, 3e19, 1e-15, 1e-12, 1e15, 1e-30, 1e18]
    g = torch.Generator("cuda").manual_seed(D)
    x = torch.rand(7, 2 * len(sizes), D, generator=g, device="cuda") * 2 - 1
    x *= torch.tensor(sizes + sizes[::-1], device="cuda")[:, None]
    x = x.to(dt)
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt)
    pos, freq = torch.arange(7, device="cuda").int(), dg.rope_frequencies(rot)
    n = len(sizes)
    q, k = dg.qk_norm_rope(x[:, :n], x[:, n:], w, None, pos, freq, interleaved=interleaved, eps=eps)
    ulp = U16 if dt == torch.bfloat16 else 0.0
    eps = float(np.float32(eps))
    _check_norm(x[:, :n], q, w, pos, freq, interleaved, eps, 0.0, ulp)
    _check_norm(x[:, n:], k, None, pos, freq, interleaved, eps, 0.0, ulp)


def test_norm_of_the_most_tokens():
    """2^31 - 1 tokens of one head of 8: a row that all read, 34 GB of them written."""
    n = 2 ** 31 - 1
    x = torch.randn(1, 1, 8, device="cuda").bfloat16()
    out = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    dg.dg_qk_norm_rope(n, 1, 0, 8, 0, False, dg.DG_BF16, x.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0.0, 1e-6, 0, 0,
                       out.data_ptr(), 0, torch.cuda.current_stream().cuda_stream)
    want, _ = dg.qk_norm_rope(x, x[:, :0], None, None, torch.zeros(1, dtype=torch.int32, device="cuda"),
                              dg.rope_frequencies(0))
    for at in (0, n // 2, n - 33, n - 1):
        assert torch.equal(out[at], want[0, 0])
    assert (out[::4097] == want[0, 0]).all()
    del out
    torch.cuda.empty_cache()
