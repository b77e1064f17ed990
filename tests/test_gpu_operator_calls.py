"""How process_logits, page_plan and prefix_attention are called: in inference mode, from
several threads, with the dict of another call, with tables of no columns."""

import ctypes
import threading

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd
from tests import test_gpu_attention as attention
from tests import test_gpu_logits as logits
from tests import test_gpu_pages as pages
from tests.parity import i32, torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ssd.build()
    ssd.lib()


def test_no_own_tables_whatever_their_columns():
    """NULL tables and lens: no own tokens, whatever `cols` says."""
    torch, dev = torch_dev()
    s = attention.make([3, 2], [50, 7], [0] * 5, 4, 2, 64, 16, torch.bfloat16, own=False)
    want = attention.call(s)
    L = ssd.lib()
    q, k, v = s["q"], s["k"], s["v"]
    for cols in (2, 1000):
        out, lse = torch.full_like(q, 7), torch.empty((5, 4), device=dev)
        a = ssd._Attention(
            0, 5, 4, 2, 64, 2, k.shape[0], 16, q.data_ptr(), q.stride(0), q.stride(1),
            (k.data_ptr(), *k.stride()[:3]), (v.data_ptr(), *v.stride()[:3]), s["pt"].data_ptr(),
            s["pl"].data_ptr(), s["off"].data_ptr(), None, None, s["pt"].stride(0), cols,
            s["pt"].shape[1], cols, out.data_ptr(), out.stride(0), out.stride(1), lse.data_ptr(),
            64 ** -0.5, 0)
        n = L.ssd_prefix_attention_workspace_size(ctypes.byref(a))
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        st = L.ssd_prefix_attention(ctypes.byref(a), ws.data_ptr(), n, None,
                                    torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"])


@pytest.mark.parametrize("room", [0, 60])
def test_inference_mode(room):
    """A serving program's mode, in which views have no base: outputs new and used again."""
    torch, dev = torch_dev()
    rng = np.random.default_rng(2)
    state = list(pages.random_state(rng, 9, 16, 90, 5, 40, 60))
    state[-1] = room
    with torch.inference_mode():
        pages.run(*state)                 # three calls, two of them with out=
        z, d, parent = logits.make(2, 3, 500, 9, torch.float32, seed=1)
        o = logits.run_case(z, d, parent)
        logits.run_case(z, d, parent, out=o)
        s = attention.make([2, 3], [40, 7], [3] * 5, 4, 2, 64, 16, torch.bfloat16)
        o = attention.call(s)
        attention.check(s, attention.call(s, out=o))


def test_plan_outputs_that_are_not_an_earlier_calls():
    torch, dev = torch_dev()
    i = torch.zeros(4, dtype=torch.int32, device=dev)
    args = (i, i, i, torch.zeros((4, 5), dtype=torch.int32, device=dev), i, i[:1], 16, 8)
    o = ssd.page_plan(*args)
    for out in ({"slots": o["slots"]}, {k: v for k, v in o.items() if k != "served"},
                dict(o, cu=o["cu"].long()), dict(o, cu=o["cu"].cpu()),
                {k: v.clone() for k, v in o.items()}):
        with pytest.raises(ssd.SSDError):
            ssd.page_plan(*args, out=out)
    with torch.inference_mode():
        ssd.page_plan(*args, out=o)       # made outside, used inside
