"""Calls of process_logits, page_plan and prefix_attention whose outcome is settled before
anything is enqueued: no device is touched."""

import ctypes

import pytest

import sampling_ssd_verify_gb300 as ssd
from tests.test_round_operators_cpu import INVALID, PTR, UNSUPPORTED, WORKSPACE, _attention


def test_tensors_of_a_gpu_that_is_not_current_are_refused(monkeypatch):
    """A launch goes to the current GPU, whatever the tensors' is."""
    import torch

    class Elsewhere(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    def there(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype).as_subclass(Elsewhere)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    i = there(2)
    c = there(3, 16, 2, 64, dtype=torch.bfloat16)
    z = there(2, 3, 32, dtype=torch.float32)
    for call in (lambda: ssd.process_logits(z),
                 lambda: ssd.page_plan(i, i, i, there(2, 4), i, there(1), 16, 4),
                 lambda: ssd.prefix_attention(there(2, 4, 64, dtype=torch.bfloat16), c, c,
                                              there(1, 2), there(1), i),
                 lambda: ssd._logits(z),           # verification and sampling
                 lambda: ssd.cache_build(i, i, i, i, table=i),
                 lambda: ssd.cache_build_guesses(there(2, 3, 2), table=i),
                 lambda: ssd.cache_lookup(i, i, i)):
        with pytest.raises(ssd.SSDError, match="cuda:1.*cuda:0"):
            call()


@pytest.mark.parametrize("T", [0, 1, 40])
def test_outputs_of_a_plan_are_known_again_in_inference_mode(T):
    """Views made in inference mode know no base."""
    import torch

    for mode in (torch.inference_mode, torch.no_grad):
        with mode():
            o = ssd._plan_views(torch, 9, T, torch.device("cpu"))
            at = ssd._plan_pointers(o, 9, T, torch.int32, -1)
            assert [p for p, k in zip(at, ssd._PLAN) if o[k].numel()] == \
                [o[k].data_ptr() for k in ssd._PLAN if o[k].numel()]
            for B, rows, out in ((8, T, o), (9, T + 17, o), (9, T, dict(o, cu=o["cu"].clone())),
                                 (9, T, dict(o, held=o["served"]))):
                with pytest.raises(ssd.SSDError):
                    ssd._plan_pointers(out, B, rows, torch.int32, -1)


def test_outputs_of_a_plan_come_whole():
    import torch

    o = ssd._plan_views(torch, 4, 8, torch.device("cpu"))
    for name in o:
        with pytest.raises(ssd.SSDError):
            ssd._plan_pointers({k: v for k, v in o.items() if k != name}, 4, 8, torch.int32, -1)


@pytest.mark.parametrize("kw,status", [
    (dict(prefix_tables=None, prefix_cols=0), WORKSPACE), (dict(tables=None, cols=0), WORKSPACE),
    (dict(tables=None, lens=None), WORKSPACE),
    (dict(tables=None, lens=None, cols=2 ** 31 - 1), WORKSPACE),
    (dict(prefix_tables=None), INVALID), (dict(tables=None), INVALID),
    (dict(lens=None, cols=0), INVALID),
])
def test_tables_without_columns_have_no_address(kw, status):
    """A tensor of no elements has a null address."""
    ssd.build()
    L = ssd.lib()
    a = _attention(**kw)
    assert L.ssd_prefix_attention(ctypes.byref(a), None, 0, None, None) == status
    assert (L.ssd_prefix_attention_workspace_size(ctypes.byref(a)) > 0) == (status == WORKSPACE)


@pytest.mark.parametrize("kw,status", [
    (dict(), WORKSPACE), (dict(out_row_stride=2048), INVALID), (dict(out_head_stride=136), INVALID),
])
def test_attention_in_place_keeps_the_strides(kw, status):
    ssd.build()
    a = _attention(out=_attention().q, **kw)
    assert ssd.lib().ssd_prefix_attention(ctypes.byref(a), None, 0, None, None) == status


@pytest.mark.parametrize("out", ["slots", "pos", "own", "cu", "kv", "held_out", "served", "free_out"])
@pytest.mark.parametrize("of", ["lens", "new", "held", "tables", "free", "count"])
def test_outputs_of_a_plan_are_not_its_inputs(out, of):
    """The kernel reads its inputs again after the first outputs are written."""
    ssd.build()
    a = dict(lens=1, new=2, held=3, B=4, tables=4, stride=8, cols=8, free=5, cap=4, count=6,
             page=16, rows=10, slots=7, pos=8, own=9, cu=10, kv=11, held_out=12, served=13,
             free_out=14)
    a = {k: v if k in ("B", "stride", "cols", "cap", "page", "rows") else v * PTR
         for k, v in a.items()}
    a[out] = a[of]
    assert ssd.lib().ssd_page_plan(*a.values(), None, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(prefix_cols=1, page_size=2 ** 31 - 1), UNSUPPORTED),
    (dict(cols=1, prefix_cols=0, page_size=2 ** 31 - 2 ** 20), UNSUPPORTED),
    (dict(cols=1, prefix_cols=1, page_size=2 ** 31 - 2 ** 20 - 8), WORKSPACE),
])
def test_lengths_leave_room_for_a_step_below_32_bits(kw, status):
    """Tokens are counted in steps and stretches past the last one."""
    ssd.build()
    a = _attention(R=1, G=1, **kw)
    assert ssd.lib().ssd_prefix_attention(ctypes.byref(a), None, 0, None, None) == status
