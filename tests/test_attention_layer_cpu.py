"""Refusals and layout of the attention-layer calls (no GPU needed: every refusal comes before a launch)."""
import ctypes
import os
import subprocess

import pytest

import uniform_state_text_b200 as dg
from uniform_state_text_b200 import build as dgbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096        # stands for a device pointer; no refused call reads it


@pytest.fixture(scope="module", autouse=True)
def lib():
    dgbuild.build()
    return dg.lib()


@pytest.mark.parametrize("struct", [dg.dg_kv_cache, dg.dg_kv_batch])
def test_struct_layout_matches_header(tmp_path, struct):
    name = struct.__name__
    fields = [f[0] for f in struct._fields_]
    body = "".join(f'  printf("{f} %zu\\n", offsetof({name}, {f}));\n' for f in fields)
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dg.h"\nint main(void){\n'
                    f'  printf("size %zu\\n", sizeof({name}));\n{body}  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)],
                   check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(struct)
    for f in fields:
        assert int(got[f]) == getattr(struct, f).offset, f


def _cache(**kw):
    a = dict(k=P, v=P, k_exp=P, v_exp=P, status=P, pages=4, page_size=16, kv_heads=2, head_dim=64,
             format=dg.DG_KV_E4M3)
    return dg.dg_kv_cache(**{**a, **kw})


def _batch(**kw):
    a = dict(page_table=P, first=P, past=P, batch=2, table_stride=3, tokens=5)
    return dg.dg_kv_batch(**{**a, **kw})


BAD = [
    (dict(format=2), {}, dg.DG_EINVAL), (dict(page_size=0), {}, dg.DG_EINVAL),
    (dict(pages=-1), {}, dg.DG_EINVAL), (dict(kv_heads=0), {}, dg.DG_EINVAL),
    (dict(head_dim=8), {}, dg.DG_EUNSUPPORTED), (dict(head_dim=72), {}, dg.DG_EUNSUPPORTED),
    (dict(head_dim=272), {}, dg.DG_EUNSUPPORTED), (dict(k=0), {}, dg.DG_EINVAL),
    (dict(v_exp=0), {}, dg.DG_EINVAL), (dict(status=0), {}, dg.DG_EINVAL),
    (dict(k=P + 8), {}, dg.DG_EINVAL),
    (dict(pages=1 << 20, page_size=1 << 10, kv_heads=2), {}, dg.DG_EUNSUPPORTED),
    (dict(pages=2, page_size=(1 << 31) - 1, kv_heads=(1 << 31) - 1), {}, dg.DG_EUNSUPPORTED),
    ({}, dict(batch=-1), dg.DG_EINVAL), ({}, dict(batch=1025), dg.DG_EUNSUPPORTED),
    ({}, dict(tokens=-1), dg.DG_EINVAL), ({}, dict(first=0), dg.DG_EINVAL),
    ({}, dict(past=0), dg.DG_EINVAL), ({}, dict(page_table=0), dg.DG_EINVAL),
    ({}, dict(table_stride=1 << 30), dg.DG_EUNSUPPORTED), ({}, dict(table_stride=-1), dg.DG_EINVAL),
]


def _attend(lib, c, b, **kw):
    a = dict(q_heads=4, q=P, ts=256, hs=64, scale=0.1, mask=dg.DG_MASK_CAUSAL, tree=0, words=0, out=P, lse=0,
             scratch=P, n=1 << 40)
    a.update(kw)
    return lib.dg_cache_attention(c, b, *a.values(), None)


@pytest.mark.parametrize("cache,batch,code", BAD)
def test_cache_and_batch_are_checked(lib, cache, batch, code):
    c, b = _cache(**cache), _batch(**batch)
    assert lib.dg_cache_write(c, b, dg.DG_BF16, P, 128, 64, P, 128, 64, None) == code
    assert dg.dg_last_error(None)
    assert lib.dg_cache_read(c, b, dg.DG_BF16, P, P, None) == code
    assert _attend(lib, c, b) == code
    assert lib.dg_cache_attention_scratch_bytes(c, b, 4) == 0


def test_null_structs(lib):
    assert lib.dg_cache_write(None, _batch(), 1, P, 8, 8, P, 8, 8, None) == dg.DG_EINVAL
    assert lib.dg_cache_read(_cache(), None, 1, P, P, None) == dg.DG_EINVAL
    assert lib.dg_cache_attention_scratch_bytes(None, None, 4) == 0


@pytest.mark.parametrize("args", [
    (7, P, 128, 64, P, 128, 64), (dg.DG_BF16, 0, 128, 64, P, 128, 64),
    (dg.DG_BF16, P + 2, 128, 64, P, 128, 64), (dg.DG_BF16, P, 129, 64, P, 128, 64),
    (dg.DG_F32, P, 128, 64, P, 128, 60)])
def test_write_refusals(lib, args):
    assert lib.dg_cache_write(_cache(), _batch(), *args, None) == dg.DG_EINVAL


@pytest.mark.parametrize("args", [(7, P, P), (dg.DG_F32, 0, P), (dg.DG_F32, P, P + 4)])
def test_read_refusals(lib, args):
    assert lib.dg_cache_read(_cache(), _batch(), *args, None) == dg.DG_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(q_heads=0), dg.DG_EINVAL), (dict(q_heads=3), dg.DG_EINVAL), (dict(q=0), dg.DG_EINVAL),
    (dict(ts=7), dg.DG_EINVAL), (dict(scale=0.0), dg.DG_EINVAL), (dict(scale=-1.0), dg.DG_EINVAL),
    (dict(scale=float("nan")), dg.DG_EINVAL), (dict(scale=float("inf")), dg.DG_EINVAL),
    (dict(mask=3), dg.DG_EINVAL), (dict(mask=-1), dg.DG_EINVAL),
    (dict(mask=dg.DG_MASK_TREE, words=2), dg.DG_EINVAL),
    (dict(mask=dg.DG_MASK_TREE, tree=P, words=-1), dg.DG_EINVAL), (dict(out=0), dg.DG_EINVAL),
    (dict(out=P + 2), dg.DG_EINVAL), (dict(scratch=0), dg.DG_EINVAL), (dict(scratch=P + 16), dg.DG_EINVAL),
    (dict(n=8), dg.DG_ENOMEM)])
def test_attention_refusals(lib, kw, code):
    assert _attend(lib, _cache(), _batch(), **kw) == code
    assert dg.dg_last_error(None)


def test_more_rows_than_the_kernels_index(lib):
    b = _batch(tokens=1 << 29)
    assert _attend(lib, _cache(), b) == dg.DG_EUNSUPPORTED
    assert lib.dg_cache_attention_scratch_bytes(_cache(), b, 4) == 0 and dg.dg_last_error(None)
    assert lib.dg_cache_attention_scratch_bytes(_cache(), _batch(), 3) == 0
    n = lib.dg_cache_attention_scratch_bytes(_cache(), _batch(), 4)
    assert n > 0 and n % 256 == 0
    assert _attend(lib, _cache(), _batch(), n=n - 1) == dg.DG_ENOMEM


def _norm(lib, **kw):
    a = dict(tokens=3, qh=4, kh=2, D=64, rot=64, inter=0, dtype=dg.DG_BF16, q=P, qts=256, qhs=64, k=P,
             kts=128, khs=64, wq=0, wk=0, off=0.0, eps=1e-6, pos=P, freq=P, qo=P, ko=P)
    a.update(kw)
    return lib.dg_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), dg.DG_EINVAL), (dict(qh=-1), dg.DG_EINVAL), (dict(D=4), dg.DG_EUNSUPPORTED),
    (dict(D=60), dg.DG_EUNSUPPORTED), (dict(D=264), dg.DG_EUNSUPPORTED), (dict(rot=8), dg.DG_EUNSUPPORTED),
    (dict(rot=80), dg.DG_EUNSUPPORTED), (dict(rot=-16), dg.DG_EUNSUPPORTED), (dict(dtype=9), dg.DG_EINVAL),
    (dict(eps=-1.0), dg.DG_EINVAL), (dict(eps=float("nan")), dg.DG_EINVAL),
    (dict(off=float("inf")), dg.DG_EINVAL), (dict(q=0), dg.DG_EINVAL), (dict(k=P + 4), dg.DG_EINVAL),
    (dict(qts=260), dg.DG_EINVAL), (dict(qo=0), dg.DG_EINVAL), (dict(ko=P + 8), dg.DG_EINVAL),
    (dict(wq=P + 2), dg.DG_EINVAL), (dict(pos=0), dg.DG_EINVAL), (dict(freq=0), dg.DG_EINVAL)])
def test_norm_refusals(lib, kw, code):
    assert _norm(lib, **kw) == code
    assert dg.dg_last_error(None)


def test_nothing_to_do_is_no_error(lib):
    assert _norm(lib, tokens=0) == dg.DG_OK
    assert _norm(lib, qh=0, kh=0) == dg.DG_OK
    for b in (_batch(tokens=0), _batch(batch=0), _batch(batch=0, page_table=0, first=0, past=0)):
        assert lib.dg_cache_write(_cache(), b, dg.DG_BF16, 0, 0, 0, 0, 0, 0, None) == dg.DG_OK
        assert lib.dg_cache_read(_cache(), b, dg.DG_BF16, 0, 0, None) == dg.DG_OK
        assert _attend(lib, _cache(), b, q=0, out=0, scratch=0) == dg.DG_OK


def test_owners_refuse_host_tensors():
    import torch
    with pytest.raises(ValueError):
        dg.KVCache(torch.zeros(1, 1, 1, 16, dtype=torch.bfloat16), torch.zeros(1, 1, 1, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        dg.KVCache(torch.zeros(1, 1, 1, 16), torch.zeros(1, 1, 1, 16))
    with pytest.raises(ValueError):
        dg.KVBatch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                   torch.zeros(1, dtype=torch.int32), 1)
    x = torch.zeros(1, 1, 16)
    with pytest.raises(ValueError):
        dg.qk_norm_rope(x, x, None, None, torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.float64))
