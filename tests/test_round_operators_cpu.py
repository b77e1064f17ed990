"""Refusals of process_logits, page_plan and prefix_attention: every argument
error returns its status before anything is enqueued (no device is touched),
and the Python layer refuses tensors of the wrong place, type or shape."""

import ctypes

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
PTR = 0x10000


@pytest.fixture(scope="module")
def L():
    ssd.build()
    return ssd.lib()


def _logits_call(L, B=2, N=3, V=64, stride=64, dtype=0, out_dtype=0, out_ptr=2 * PTR,
                 out_stride=64, parent=None, rules=(), **kw):
    a = ssd._Logits(PTR, dtype, kw.get("pad", 0), stride)
    b = ssd._Logits(out_ptr, out_dtype, 0, out_stride)
    r = ssd._LogitRules(fill=-1.0)
    for k, v in rules:
        setattr(r, k, v)
    if parent is not None:
        r.parent = np.asarray(parent, dtype=np.int32).tobytes()
    return L.ssd_process_logits(ctypes.byref(a), ctypes.byref(b), B, N, V, ctypes.byref(r), None,
                                None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(V=0), INVALID),
    (dict(V=65), INVALID),                                   # longer than the row stride
    (dict(dtype=2, out_dtype=2), INVALID), (dict(out_dtype=1), INVALID),
    (dict(pad=1), INVALID), (dict(out_ptr=None), INVALID),
    (dict(out_ptr=2 * PTR + 1), INVALID),
    (dict(out_ptr=PTR, out_stride=80), INVALID),             # in place with another stride
    (dict(N=257, stride=64), UNSUPPORTED),
    (dict(V=1 << 24, stride=1 << 24, out_stride=1 << 24), UNSUPPORTED),
    (dict(rules=[("fill", float("nan"))]), INVALID),
    (dict(rules=[("pad_", 1)]), INVALID),
    (dict(rules=[("history", PTR)]), INVALID),               # no lengths
    (dict(rules=[("history", PTR), ("history_len", PTR), ("history_max", -1)]), INVALID),
    (dict(rules=[("n_bias", 1)]), INVALID), (dict(rules=[("n_bias", -1)]), INVALID),
    (dict(rules=[("n_bias", 65536), ("bias_ids", PTR), ("bias", PTR)]), INVALID),
    (dict(rules=[("mask", PTR), ("mask_row_stride", -1)]), INVALID),
    (dict(parent=[0, 0, 1]), INVALID), (dict(parent=[-1, 1, 0]), INVALID),
    (dict(parent=[-1, 0, -1]), INVALID),
])
def test_process_logits_refusals(L, kw, status):
    assert _logits_call(L, **kw) == status


def _plan_call(L, **kw):
    a = dict(lens=PTR, new=PTR, held=2 * PTR, B=4, tables=PTR, stride=8, cols=8, free=PTR, cap=4,
             count=PTR, page=16, rows=10, slots=PTR, pos=None, own=None, cu=PTR, kv=3 * PTR,
             held_out=PTR, served=PTR, free_out=4 * PTR)
    a.update(kw)
    return L.ssd_page_plan(*a.values(), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(B=8193), UNSUPPORTED), (dict(lens=None), INVALID),
    (dict(tables=None), INVALID), (dict(cu=None), INVALID), (dict(slots=None), INVALID),
    (dict(stride=7), INVALID), (dict(cols=0), INVALID), (dict(page=0), INVALID),
    (dict(cap=-1), INVALID), (dict(free=None), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=1 << 28, stride=1 << 28, B=5), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(free_out=PTR), INVALID), (dict(kv=PTR), INVALID), (dict(held_out=2 * PTR), INVALID),
])
def test_page_plan_refusals(L, kw, status):
    assert _plan_call(L, **kw) == status


def _attention(**kw):
    kv = ssd._Paged(PTR, 4096, 512, 128)
    a = ssd._Attention(dtype=0, R=4, Hq=8, Hkv=4, D=128, G=2, num_pages=10, page_size=8, q=PTR,
                       q_row_stride=1024, q_head_stride=128, k=kv, v=kv, prefix_tables=PTR,
                       prefix_len=PTR, group_off=PTR, tables=PTR, lens=PTR,
                       prefix_table_stride=5, table_stride=2, prefix_cols=5, cols=2, out=PTR,
                       out_row_stride=1024, out_head_stride=128, lse=PTR, scale=0.1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), INVALID), (dict(R=0), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(G=-1), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(scale=float("inf")), INVALID), (dict(pad_=1), INVALID),
    (dict(prefix_len=None), INVALID), (dict(group_off=None), INVALID),
    (dict(prefix_table_stride=4), INVALID), (dict(lens=None), INVALID),
    (dict(table_stride=1), INVALID), (dict(q=None), INVALID), (dict(q=PTR + 2), INVALID),
    (dict(q_head_stride=4), INVALID), (dict(out_row_stride=-8), INVALID),
    (dict(k=ssd._Paged(PTR, 4096, 516, 128)), INVALID), (dict(v=ssd._Paged(None, 8, 8, 8)), INVALID),
    (dict(prefix_cols=1 << 30, prefix_table_stride=1 << 30, page_size=64), UNSUPPORTED),
    (dict(), WORKSPACE),
])
def test_prefix_attention_refusals(L, kw, status):
    a = _attention(**kw)
    assert L.ssd_prefix_attention(ctypes.byref(a), None, 0, None, None) == status
    if status == UNSUPPORTED:
        assert L.ssd_prefix_attention_workspace_size(ctypes.byref(a)) == 0


def test_prefix_attention_workspace(L):
    a = _attention()
    n = L.ssd_prefix_attention_workspace_size(ctypes.byref(a))
    assert n > 0 and n % 256 == 0
    assert L.ssd_prefix_attention(ctypes.byref(a), PTR, n - 1, None, None) == WORKSPACE
    assert L.ssd_prefix_attention(ctypes.byref(a), PTR + 16, n, None, None) == WORKSPACE
    assert L.ssd_prefix_attention_workspace_size(ctypes.byref(_attention(R=400))) > n
    assert L.ssd_prefix_attention_workspace_size(ctypes.byref(_attention(G=0))) > 0
    # no own tokens
    assert L.ssd_prefix_attention_workspace_size(ctypes.byref(_attention(tables=None, lens=None))) > 0


def test_cpu_tensors_are_refused(L):
    import torch

    z = torch.zeros((2, 3, 32))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ssd.SSDError):
        ssd.process_logits(z)
    with pytest.raises(ssd.SSDError):
        ssd.page_plan(i, i, i, torch.zeros((2, 4), dtype=torch.int32), i, i[:1], 16, 4)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    c = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    t = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ssd.SSDError):
        ssd.prefix_attention(q, c, c, t, i[:1], i)


def test_structures_match_the_header(tmp_path):
    """The ctypes structures have the sizes and offsets of the C ones."""
    import os
    import shutil
    import subprocess

    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no host compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    names = {"ssd_logit_rules": ssd._LogitRules, "ssd_paged": ssd._Paged,
             "ssd_attention": ssd._Attention}
    body = "".join(
        f'printf("%zu\\n", sizeof({c}));' +
        "".join(f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in t._fields_)
        for c, t in names.items())
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "ssd.h"\nint main(void) {' + body + "return 0; }\n")
    exe = str(tmp_path / "t")
    subprocess.run([cc, "-I", inc, str(src), "-o", exe], check=True)
    got = list(map(int, subprocess.run([exe], capture_output=True, text=True).stdout.split()))
    want = [x for t in names.values()
            for x in [ctypes.sizeof(t)] + [getattr(t, f).offset for f, _ in t._fields_]]
    assert got == want
