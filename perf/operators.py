"""Workloads of the attention-layer operators, with their plain forms.

Four operators that a backbone around the denoise step runs in every layer:

  norm    RMS norm of every query and key head, and the rotation by position
  write   keys and values of new tokens into a paged cache (bf16 or e4m3 with
          a power-of-two scale per row)
  read    those rows back out of the cache
  attend  attention of each sequence's new tokens over its cached prefix and,
          under a mask, over one another (a bidirectional canvas, a causal
          prompt, a tree of drafts, single tokens)

`own` selects the library's kernels; otherwise `run` computes the same result
with elementary torch operations in fp32 (angles in fp64), rounded once.
A case is a dict of plain values; lengths of ragged batches follow from it
alone, values and page orders from the seed.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
GOLDEN = 0.6180339887498949


def listed():
    return [
        # one token of one sequence between two layers: latency
        dict(name="norm, one token", op="norm", tokens=1, q_heads=16, k_heads=8, head_dim=128,
             rot=128, interleaved=False, dtype="bf16", packed=True, far=131072),
        # the 256-position canvas of one denoise step, wide heads, a quarter of each rotated
        dict(name="norm, canvas", op="norm", tokens=256, q_heads=8, k_heads=4, head_dim=256,
             rot=64, interleaved=True, dtype="f32", packed=False, far=8448),
        # a long prompt, width 2816 in heads of 128, rows of a packed projection
        dict(name="norm, prompt", op="norm", tokens=16384, q_heads=22, k_heads=2, head_dim=128,
             rot=128, interleaved=False, dtype="bf16", packed=True, far=16384),
        # four canvases rewritten into the cache in every denoise step
        dict(name="write, canvases e4m3", op="write", batch=4, new=256, past=4001, ragged=False,
             kv_heads=8, head_dim=128, page=64, fmt="e4m3", dtype="bf16", packed=True),
        # prompts of a ragged batch, small pages, fp32 keys and values
        dict(name="write, prompts e4m3", op="write", batch=7, new=4096, past=37, ragged=True,
             kv_heads=4, head_dim=256, page=16, fmt="e4m3", dtype="f32", packed=False),
        # a short reused prefix
        dict(name="read, short prefix", op="read", batch=1, new=131, past=0, ragged=False,
             kv_heads=8, head_dim=128, page=16, fmt="bf16", dtype="bf16"),
        # a long narrow cache handed to code that wants plain tensors
        dict(name="read, long e4m3", op="read", batch=3, new=40000, past=0, ragged=True,
             kv_heads=8, head_dim=128, page=64, fmt="e4m3", dtype="bf16"),
        # decoding: one token for each of 33 sequences of differing lengths
        dict(name="attend, single tokens e4m3", op="attend", mask="causal", batch=33, new=1,
             past=8000, ragged=True, q_heads=32, kv_heads=8, head_dim=128, page=64, fmt="e4m3"),
        # one token of one sequence over a long cache
        dict(name="attend, one long sequence", op="attend", mask="causal", batch=1, new=1,
             past=131071, ragged=False, q_heads=16, kv_heads=8, head_dim=128, page=128, fmt="bf16"),
        # trees of drafted tokens to be verified
        dict(name="attend, draft trees", op="attend", mask="tree", batch=5, new=63, past=6000,
             ragged=True, q_heads=16, kv_heads=2, head_dim=64, page=16, fmt="bf16"),
        # canvases of 256 positions over a committed prefix, wide heads
        dict(name="attend, canvases e4m3", op="attend", mask="full", batch=4, new=256, past=8192,
             ragged=False, q_heads=8, kv_heads=4, head_dim=256, page=32, fmt="e4m3"),
        # a prompt's prefill
        dict(name="attend, prompt", op="attend", mask="causal", batch=1, new=8192, past=0,
             ragged=False, q_heads=16, kv_heads=8, head_dim=128, page=64, fmt="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "write", "read", "attend", "attend"])
    if op == "norm":
        head_dim = rng.choice([64, 80, 96, 128, 256])
        k_heads = rng.choice([1, 2, 3, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 16384), q_heads=k_heads * rng.choice([1, 2, 4, 5]),
                    k_heads=k_heads, head_dim=head_dim, rot=rng.choice([head_dim, 32, 48]),
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    packed=rng.random() < 0.5, far=_log(rng, 16384, 1 << 20))
    fmt = rng.choice(["bf16", "e4m3"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([8, 16, 24, 32, 64, 128, 256])
    if op != "attend":
        batch = _log(rng, 1, 48)
        c = dict(op=op, batch=batch, new=_log(rng, 1, 40000 // batch), past=_log(rng, 1, 4000),
                 ragged=rng.random() < 0.6, kv_heads=kv_heads,
                 head_dim=rng.choice([64, 80, 128, 256]), page=page, fmt=fmt,
                 dtype=rng.choice(["bf16", "f32"]))
        if op == "write":
            c["packed"] = rng.random() < 0.5
        return c
    mask = rng.choice(["full", "causal", "causal", "tree"])
    group = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, mask=mask, batch=_log(rng, 1, 40),
             new=_log(rng, 1, {"full": 512, "causal": 6000, "tree": 130}[mask]),
             past=_log(rng, 1, 131072), ragged=rng.random() < 0.6, q_heads=group * kv_heads,
             kv_heads=kv_heads, head_dim=rng.choice([64, 80, 128, 128, 256]), page=page, fmt=fmt)
    # no drawn case costs more than the largest listed one, or fills the card in the plain form
    while (work(c)["flops"] > 2e11 or work(c)["bytes"] > 1e9 or _scores(c) > 5e8
           or c["batch"] * (c["past"] + c["new"]) * kv_heads * c["head_dim"] > 4e8):
        if c["past"] > c["new"]:
            c["past"] = max(1, c["past"] * 2 // 3)
        elif c["batch"] > 1:
            c["batch"] = c["batch"] * 2 // 3
        else:
            c["new"] = c["new"] * 2 // 3
    return c


def _scores(c):
    return c["batch"] * c["q_heads"] * c["new"] * (c["past"] + c["new"])


def _lengths(c):
    """(past, new) of each sequence: the case's own, or spread below them, some with nothing new."""
    past, new = [], []
    for b in range(c["batch"]):
        f = (b * GOLDEN) % 1.0 if c["ragged"] else 0.0
        past.append(c["past"] - int(f * 0.75 * c["past"]))
        new.append(0 if c["ragged"] and b % 8 == 7 else c["new"] - int(f * 0.5 * (c["new"] - 1)))
    return past, new


def work(c):
    if c["op"] == "norm":
        size = 2 if c["dtype"] == "bf16" else 4
        rows = c["tokens"] * (c["q_heads"] + c["k_heads"])
        return dict(bytes=rows * c["head_dim"] * size * 2 + 4 * c["tokens"] + 4 * c["rot"]
                    + 2 * c["head_dim"] * size,
                    flops=rows * (4 * c["head_dim"] + 3 * c["rot"]))
    past, new = _lengths(c)
    cached = c["head_dim"] * 2 if c["fmt"] == "bf16" else c["head_dim"] + 1
    if c["op"] != "attend":
        rows = 2 * sum(new) * c["kv_heads"]
        plain = c["head_dim"] * (2 if c["dtype"] == "bf16" else 4)
        return dict(bytes=rows * (cached + plain), flops=2 * rows * c["head_dim"])
    rows = 2 * sum(p + n for p, n in zip(past, new) if n) * c["kv_heads"]
    seen = sum(n * (p + (n if c["mask"] == "full" else (n + 1) / 2)) for p, n in zip(past, new))
    return dict(bytes=rows * cached + sum(new) * c["q_heads"] * (4 * c["head_dim"] + 4),
                flops=4 * c["head_dim"] * c["q_heads"] * seen)


# ----------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pow2(e):
    """2^e in fp32, exactly, for whole -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """Rows of fp32 to e4m3 codes (as bytes) and biased power-of-two exponents: the smallest
    exponent that brings the row's largest magnitude within 448."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = (e - 9 + (m > 0.875).int()).masked_fill(m == 0, 0).clamp(-100, 119)
    codes = (x * _pow2(-e)[..., None]).clamp(-448, 448).to(F8).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _tree_words(g, new):
    """Ancestor masks of random trees, one bit per node of the same sequence, itself included."""
    width = max(1, (max(new) + 31) // 32)
    out = []
    for n in new:
        parent = [int(f * (i + 1)) - 1 for i, f in
                  enumerate(torch.rand(n, generator=g, device="cuda").cpu().tolist())]
        seen = []
        for i, p in enumerate(parent):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        out += [[(s >> (32 * w)) & 0xFFFFFFFF for w in range(width)] for s in seen]
    words = torch.tensor(out, dtype=torch.int64).reshape(-1, width)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()


def prepare(c, seed):
    g = _generator(seed)
    if c["op"] == "norm":
        t, d, hq, hk = c["tokens"], c["head_dim"], c["q_heads"], c["k_heads"]
        dt = _type(c["dtype"])
        if c["packed"]:                       # queries, keys and values of one projection
            rows = _randn(g, t, hq + 2 * hk, d).mul_(1.5).to(dt)
            q, k = rows[:, :hq], rows[:, hq:hq + hk]
        else:
            q, k = _randn(g, t, hq, d).to(dt), _randn(g, t, hk, d).mul_(2).to(dt)
        i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
        start = int(torch.randint(0, c["far"] - t + 1, (1,), generator=g, device="cuda"))
        return dict(case=c, q=q, k=k, wq=(1 + 0.2 * _randn(g, d)).to(dt),
                    wk=(1 + 0.2 * _randn(g, d)).to(dt), inv_freq=10000.0 ** (-2 * i / c["rot"]),
                    positions=(start + torch.arange(t, device="cuda")).int())
    past, new = _lengths(c)
    page, hk, d = c["page"], c["kv_heads"], c["head_dim"]
    need = [-(-(p + n) // page) for p, n in zip(past, new)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.zeros(c["batch"], max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    first = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()
    s = dict(case=c, table=table, first=first, past=torch.tensor(past, dtype=torch.int32).cuda(),
             tokens=sum(new), most_new=max(new), most=max(p + n for p, n in zip(past, new)))
    shape = (pages, hk, page, d)
    if c["op"] == "write":
        if c["fmt"] == "bf16":
            s["k_pages"], s["v_pages"] = torch.zeros(2, *shape, dtype=torch.bfloat16, device="cuda")
        else:
            s["k_pages"], s["v_pages"] = torch.zeros(2, *shape, dtype=torch.uint8, device="cuda")
            s["k_exp"], s["v_exp"] = torch.zeros(2, *shape[:3], dtype=torch.uint8, device="cuda")
    else:
        for n in ("k", "v"):
            x = _randn(g, *shape)
            if c["fmt"] == "bf16":
                s[n + "_pages"] = x.to(torch.bfloat16)
            else:
                s[n + "_pages"], s[n + "_exp"] = _quantise(x)
    if c["op"] == "write":
        rows = _randn(g, s["tokens"], 2 * hk, d).to(_type(c["dtype"]))
        s["k"], s["v"] = rows[:, :hk], rows[:, hk:]
        if not c["packed"]:
            s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
    if c["op"] == "attend":
        s["q"] = _randn(g, s["tokens"], c["q_heads"], d).mul_(1.5).to(torch.bfloat16)
        s["tree"] = _tree_words(g, new) if c["mask"] == "tree" else None
    if own:                                   # the handles that a program keeps for its cache and batch
        import uniform_state_text_b200 as dg
        as_pages = lambda x: x if c["fmt"] == "bf16" else x.view(F8)  # noqa: E731
        s["cache"] = dg.KVCache(as_pages(s["k_pages"]), as_pages(s["v_pages"]), s.get("k_exp"),
                                s.get("v_exp"))
        s["batch"] = dg.KVBatch(table, first, s["past"], s["tokens"])
    return s


# ----------------------------------------------------------------------------- one pass
def run(s):
    return {"norm": _norm, "write": _write, "read": _read, "attend": _attend}[s["case"]["op"]](s)


def _norm(s):
    c = s["case"]
    if own:
        import uniform_state_text_b200 as dg
        return dg.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"],
                               interleaved=c["interleaved"], eps=1e-6)
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return tuple(_plain_norm(x, w, cos, sin, c["rot"], c["interleaved"])
                 for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))


def _plain_norm(x, w, cos, sin, rot, interleaved):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    r = y[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, y[..., rot:]), -1).to(x.dtype)


def _slots(s):
    """Page and place in the page of every new token."""
    token = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["first"].long(), token, right=True) - 1
    pos = s["past"].long()[b] + token - s["first"].long()[b]
    page = s["case"]["page"]
    return s["table"][b, pos // page].long(), pos % page


def _written(s):
    out = {}
    for n in ("k", "v"):
        pages = s[n + "_pages"]
        out[n] = pages if pages.dtype == torch.bfloat16 else pages.view(F8)
        if pages.dtype != torch.bfloat16:
            out[n + "_exp"] = s[n + "_exp"]
    return out


def _write(s):
    if own:
        s["cache"].write(s["k"], s["v"], s["batch"])
        return _written(s)
    page, place = _slots(s)
    for n in ("k", "v"):
        if s["case"]["fmt"] == "bf16":
            s[n + "_pages"][page, :, place] = s[n].to(torch.bfloat16)
        else:
            codes, e = _quantise(s[n].float())
            s[n + "_pages"][page, :, place] = codes
            s[n + "_exp"][page, :, place] = e
    return _written(s)


def _values(s, n):
    """The cache's pages as fp32."""
    x = s[n + "_pages"]
    if x.dtype == torch.bfloat16:
        return x.float()
    return x.view(F8).float() * _pow2(s[n + "_exp"].int() - 127)[..., None]


def _read(s):
    if own:
        return s["cache"].read(s["batch"], _type(s["case"]["dtype"]))
    page, place = _slots(s)
    return tuple(_values(s, n)[page, :, place].to(_type(s["case"]["dtype"])) for n in ("k", "v"))


def _attend(s):
    c = s["case"]
    if own:
        import uniform_state_text_b200 as dg
        mask = {"full": dg.DG_MASK_FULL, "causal": dg.DG_MASK_CAUSAL, "tree": dg.DG_MASK_TREE}
        return s["cache"].attend(s["q"], s["batch"], mask[c["mask"]], tree=s["tree"])
    hq, hk, d, most = c["q_heads"], c["kv_heads"], c["head_dim"], s["most"]
    first, past = s["first"].long(), s["past"].long()
    i = torch.arange(max(1, s["most_new"]), device="cuda")
    new = first[1:] - first[:-1]
    token = (first[:-1, None] + i).clamp(max=s["tokens"] - 1)               # [B, n]
    q = s["q"].float()[token].unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k, v = (_values(s, n)[s["table"].long()].transpose(1, 2).flatten(2, 3)[:, :, :most]
            for n in ("k", "v"))                                            # [B, hk, L, d]
    node = torch.arange(most, device="cuda") - past[:, None]                # [B, L]
    inside = (node >= 0) & (node < new[:, None])
    seen = (node < 0)[:, None].expand(-1, len(i), -1)
    if c["mask"] == "full":
        seen = seen | inside[:, None]
    elif c["mask"] == "causal":
        seen = seen | (inside[:, None] & (node[:, None] <= i[:, None]))
    else:
        at = node.clamp(0, 32 * s["tree"].shape[1] - 1)
        words = torch.gather(s["tree"][token].long(), 2,
                             (at // 32)[:, None].expand(-1, len(i), -1))
        seen = seen | (inside[:, None] & ((words >> (at % 32)[:, None]) & 1).bool())
    score = (q @ k.transpose(2, 3)).mul_(d ** -0.5).unflatten(2, (hq // hk, len(i)))
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == -math.inf, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, (hq // hk, len(i)))
    out = out / total.masked_fill(total == 0, 1)
    lse = (top + total.log())[..., 0]
    token_b = torch.searchsorted(first, torch.arange(s["tokens"], device="cuda"), right=True) - 1
    token_i = torch.arange(s["tokens"], device="cuda") - first[token_b]
    out, lse = out.permute(0, 3, 1, 2, 4)[token_b, token_i], lse.permute(0, 3, 1, 2)[token_b, token_i]
    return out.flatten(1, 2).to(torch.bfloat16), lse.flatten(1, 2)


# ----------------------------------------------------------------------------- 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "write": _exact_write, "read": _exact_read,
            "attend": _exact_attend}[c["op"]](s, c)


def _exact_norm(s, c):
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["head_dim"] + 1e-6).sqrt() * w.double()
        half = c["rot"] // 2
        y = x.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
            t = (s["positions"].double() * s["inv_freq"][i])[:, None]
            y[..., a] = x[..., a] * t.cos() - x[..., b] * t.sin()
            y[..., b] = x[..., a] * t.sin() + x[..., b] * t.cos()
        out.append(y)
    return tuple(out)


def _exact_rows(s, c):
    """(sequence, token, position) runs of the batch."""
    past, new = _lengths(c)
    at = 0
    for b, (p, n) in enumerate(zip(past, new)):
        yield b, at, p, n
        at += n


def _exact_pages(s, c, b, p, n):
    pos = torch.arange(p, p + n, device="cuda")
    return s["table"][b].long()[pos // c["page"]], pos % c["page"]


def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_write(s, c):
    out = {}
    for n in ("k", "v"):
        pages = torch.zeros(s[n + "_pages"].shape, dtype=torch.float64, device="cuda")
        exps = torch.zeros(pages.shape[:3], dtype=torch.uint8, device="cuda")
        for b, at, p, m in _exact_rows(s, c):
            page, place = _exact_pages(s, c, b, p, m)
            x = s[n][at:at + m].double()
            if c["fmt"] == "e4m3":
                top = x.abs().amax(-1, keepdim=True)
                e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).long()
                e = e + (top > 448 * _exact_pow2(e)).long() - (top <= 448 * _exact_pow2(e - 1)).long()
                e = torch.where(top > 0, e, 0)
                x = x / _exact_pow2(e)
                step = _exact_pow2(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
                x = torch.round(x / step) * step
                exps[page, :, place] = (e[..., 0] + 127).to(torch.uint8)
            pages[page, :, place] = x
        out[n] = pages
        if c["fmt"] == "e4m3":
            out[n + "_exp"] = exps
    return out


def _exact_values(s, c, n, b, p, m):
    page, place = _exact_pages(s, c, b, p, m)
    x = s[n + "_pages"][page, :, place]
    if c["fmt"] == "bf16":
        return x.double()
    return x.view(F8).double() * _exact_pow2(s[n + "_exp"][page, :, place].long() - 127)[..., None]


def _exact_read(s, c):
    return tuple(torch.cat([_exact_values(s, c, n, b, p, m) for b, _, p, m in _exact_rows(s, c)])
                 for n in ("k", "v"))


def _exact_attend(s, c):
    group = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["tokens"], c["q_heads"], c["head_dim"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], c["q_heads"], dtype=torch.float64, device="cuda")
    for b, at, p, n in _exact_rows(s, c):
        if not n:
            continue
        k, v = (_exact_values(s, c, x, b, 0, p + n) for x in ("k", "v"))
        i = torch.arange(n, device="cuda")
        if c["mask"] == "full":
            own_block = torch.ones(n, n, dtype=torch.bool, device="cuda")
        elif c["mask"] == "causal":
            own_block = i[:, None] >= i
        else:
            own_block = torch.stack([(s["tree"][at:at + n, j // 32] >> (j % 32)) & 1
                                     for j in range(n)], 1).bool()
        hidden = torch.cat((torch.zeros(n, p, dtype=torch.bool, device="cuda"), ~own_block), 1)
        for h in range(c["q_heads"]):
            z = s["q"][at:at + n, h].double() @ k[:, h // group].T / c["head_dim"] ** 0.5
            z[hidden] = -math.inf
            lse[at:at + n, h] = torch.logsumexp(z, 1)
            out[at:at + n, h] = torch.softmax(z, 1) @ v[:, h // group]
    return out, lse
