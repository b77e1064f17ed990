"""Refusals of tree_attention, append_path and fork_rows: every argument error returns its status
before anything is enqueued (no device is touched), and the Python layer refuses tensors of the
wrong place, type or shape."""

import ctypes

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd

class _TreeAttn(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("N", ctypes.c_int32),
                ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_seq_stride", ctypes.c_int64),
                ("q_node_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k", ssd._Paged), ("v", ssd._Paged), ("k_cache", ssd._Paged), ("v_cache", ssd._Paged),
                ("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("parent", ctypes.c_char_p),
                ("out", ctypes.c_void_p), ("out_seq_stride", ctypes.c_int64),
                ("out_node_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("lse", ctypes.c_void_p), ("cols", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Layers(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _Append(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int32), ("B", ctypes.c_int32), ("N", ctypes.c_int32),
                ("H", ctypes.c_int32), ("row_bytes", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("rows", ctypes.c_int32), ("path_cols", ctypes.c_int32), ("pad_", ctypes.c_int32),
                ("k", _Layers), ("v", _Layers), ("k_cache", _Layers), ("v_cache", _Layers),
                ("slots", ctypes.c_void_p), ("owner", ctypes.c_void_p), ("cu", ctypes.c_void_p),
                ("path", ctypes.c_void_p), ("path_stride", ctypes.c_int64)]


class _Fork(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("B", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("free_cap", ctypes.c_int32), ("L", ctypes.c_int32), ("H", ctypes.c_int32),
                ("row_bytes", ctypes.c_int32), ("pad_", ctypes.c_int32),
                ("src", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("tables", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("shares", ctypes.c_void_p), ("free_pages", ctypes.c_void_p),
                ("free_count", ctypes.c_void_p), ("k_cache", _Layers), ("v_cache", _Layers),
                ("tables_out", ctypes.c_void_p), ("lens_out", ctypes.c_void_p),
                ("held_out", ctypes.c_void_p), ("served", ctypes.c_void_p),
                ("shares_out", ctypes.c_void_p), ("free_out", ctypes.c_void_p)]


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
PTR = 0x10000


@pytest.fixture(scope="module")
def L():
    ssd.build()
    return ssd.lib()


def _tree(**kw):
    a = _TreeAttn(dtype=0, B=2, N=3, Hq=4, Hkv=2, D=64, num_pages=9, page_size=16, q=PTR,
                      q_seq_stride=768, q_node_stride=256, q_head_stride=64,
                      k=(2 * PTR, 384, 128, 64), v=(3 * PTR, 384, 128, 64),
                      k_cache=(4 * PTR, 2048, 128, 64), v_cache=(5 * PTR, 2048, 128, 64),
                      tables=6 * PTR, lens=7 * PTR, table_stride=4, parent=None, out=8 * PTR,
                      out_seq_stride=768, out_node_stride=256, out_head_stride=64, lse=None,
                      cols=4, scale=0.125)
    for k, v in kw.items():
        if k == "parent":
            v = np.asarray(v, dtype=np.int32).tobytes()
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(), WORKSPACE), (dict(dtype=1), INVALID), (dict(dtype=7), INVALID), (dict(B=0), INVALID),
    (dict(N=0), INVALID), (dict(N=257), UNSUPPORTED), (dict(N=256), WORKSPACE),
    (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(D=80), UNSUPPORTED), (dict(D=0), UNSUPPORTED), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(q=None), INVALID), (dict(q=PTR + 8), INVALID),
    (dict(q_seq_stride=764), INVALID), (dict(q_node_stride=-256), INVALID),
    (dict(q_head_stride=65), INVALID), (dict(out=None), INVALID), (dict(out_head_stride=4), INVALID),
    (dict(k=(0, 384, 128, 64)), INVALID), (dict(v=(3 * PTR + 2, 384, 128, 64)), INVALID),
    (dict(k=(2 * PTR, 380, 128, 64)), INVALID), (dict(k_cache=(4 * PTR, 2048, 100, 64)), INVALID),
    (dict(v_cache=(0, 2048, 128, 64)), INVALID), (dict(v_cache=(PTR, -2048, 128, 64)), INVALID),
    (dict(tables=None), INVALID), (dict(lens=None), INVALID), (dict(table_stride=3), INVALID),
    (dict(tables=None, cols=0), WORKSPACE), (dict(cols=-1), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=-1.0), WORKSPACE), (dict(scale=0.0), WORKSPACE),
    (dict(parent=[-1, 0, 0]), WORKSPACE), (dict(parent=[0, 0, 0]), INVALID),
    (dict(parent=[-1, 1, 0]), INVALID), (dict(parent=[-1, 0, -1]), INVALID),
    (dict(parent=[-2, 0, 0]), INVALID),
    (dict(cols=1, page_size=2 ** 31 - 2 ** 20), UNSUPPORTED),
    (dict(B=2 ** 30), UNSUPPORTED), (dict(Hq=2 ** 30, Hkv=2 ** 29), UNSUPPORTED),
    (dict(out=PTR), WORKSPACE), (dict(out=PTR, out_node_stride=512), INVALID),
    (dict(out=PTR, out_seq_stride=1536), INVALID), (dict(out=PTR, out_head_stride=128), INVALID),
])
def test_tree_attention_refusals(L, kw, status):
    a = _tree(**kw)
    assert L.ssd_tree_attention(ctypes.byref(a), None, 0, None, None) == status
    if status == WORKSPACE:
        n = L.ssd_tree_attention_workspace_size(ctypes.byref(a))
        assert n > 0 and n % 256 == 0
        assert L.ssd_tree_attention(ctypes.byref(a), PTR + 128, n, None, None) == WORKSPACE
        assert L.ssd_tree_attention(ctypes.byref(a), PTR, n - 1, None, None) == WORKSPACE
    assert L.ssd_tree_attention(None, None, 0, None, None) == INVALID
    assert L.ssd_tree_attention_workspace_size(None) == 0


def _append(**kw):
    row = (1 << 20, 4096, 256, 128)
    a = _Append(L=2, B=3, N=4, H=2, row_bytes=128, num_pages=9, page_size=16, rows=0,
                    path_cols=3, pad_=0, k=(PTR, *row), v=(2 * PTR, *row), k_cache=(3 * PTR, *row),
                    v_cache=(4 * PTR, *row), slots=PTR, owner=PTR, cu=PTR, path=PTR, path_stride=3)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


ROW = (1 << 20, 4096, 256, 128)
APPEND = [
    (dict(), 0), (dict(L=0), INVALID), (dict(B=0), INVALID), (dict(N=0), INVALID),
    (dict(H=0), INVALID), (dict(row_bytes=0), INVALID), (dict(row_bytes=24), INVALID),
    (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(rows=-1), INVALID),
    (dict(path_cols=-1), INVALID), (dict(pad_=1), INVALID), (dict(cu=None), INVALID),
    (dict(rows=4, slots=None), INVALID), (dict(rows=4, owner=None), INVALID),
    (dict(path_stride=2), INVALID), (dict(path=None, path_stride=0), 0),
    (dict(k=(0, *ROW)), INVALID), (dict(k=(PTR + 8, *ROW)), INVALID),
    (dict(v=(0, *ROW)), INVALID), (dict(v_cache=(0, *ROW)), INVALID),
    (dict(v=(0, *ROW), v_cache=(0, *ROW)), 0), (dict(k_cache=(3 * PTR, -16, 4096, 256, 128)), INVALID),
    (dict(k_cache=(3 * PTR, 1 << 20, 4096, 250, 128)), INVALID),
    (dict(k_cache=(PTR, *ROW)), INVALID), (dict(k_cache=(2 * PTR, *ROW)), INVALID),
    (dict(v_cache=(3 * PTR, *ROW)), INVALID), (dict(v_cache=(PTR, *ROW)), INVALID),
    (dict(v_cache=(2 * PTR, *ROW)), INVALID),
    (dict(row_bytes=1 << 24, H=2), UNSUPPORTED), (dict(rows=2 ** 31 - 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", APPEND)
def test_append_path_refusals(L, kw, status):
    a = _append(**kw)                  # no rows: nothing is launched
    assert L.ssd_append_path(ctypes.byref(a), None, None) == status
    assert L.ssd_append_path(None, None, None) == INVALID


def _fork(**kw):
    a = _Fork(S=3, B=4, cols=5, page_size=16, num_pages=9, free_cap=8, L=2, H=2, row_bytes=128,
                  pad_=0, src=PTR, lens=2 * PTR, held=3 * PTR, tables=4 * PTR, table_stride=5,
                  shares=5 * PTR, free_pages=6 * PTR, free_count=7 * PTR, k_cache=(8 * PTR, *ROW),
                  v_cache=(9 * PTR, *ROW), tables_out=10 * PTR, lens_out=11 * PTR,
                  held_out=12 * PTR, served=13 * PTR, shares_out=14 * PTR, free_out=15 * PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(), WORKSPACE), (dict(S=0), INVALID), (dict(B=0), INVALID), (dict(cols=0), INVALID),
    (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID), (dict(free_cap=-1), INVALID),
    (dict(L=-1), INVALID), (dict(H=0), INVALID), (dict(row_bytes=20), INVALID),
    (dict(pad_=1), INVALID), (dict(S=8193), UNSUPPORTED), (dict(B=8193), UNSUPPORTED),
    (dict(S=8192, cols=2 ** 18, table_stride=2 ** 18), UNSUPPORTED), (dict(row_bytes=1 << 25), UNSUPPORTED),
    (dict(num_pages=2 ** 30 + 1), UNSUPPORTED),
    (dict(src=None), INVALID), (dict(lens=None), INVALID), (dict(held=None), INVALID),
    (dict(tables=None), INVALID), (dict(shares=None), INVALID), (dict(free_pages=None), INVALID),
    (dict(free_pages=None, free_cap=0), WORKSPACE), (dict(free_count=None), INVALID),
    (dict(table_stride=4), INVALID), (dict(tables_out=None), INVALID), (dict(lens_out=None), INVALID),
    (dict(held_out=None), INVALID), (dict(served=None), INVALID), (dict(shares_out=None), INVALID),
    (dict(free_out=None), INVALID), (dict(k_cache=(0, *ROW)), INVALID),
    (dict(k_cache=(0, *ROW), v_cache=(0, *ROW)), INVALID),
    (dict(L=0, k_cache=(0, 0, 0, 0, 0), v_cache=(0, 0, 0, 0, 0)), WORKSPACE),
    (dict(v_cache=(0, *ROW)), WORKSPACE), (dict(v_cache=(8 * PTR, *ROW)), INVALID),
    (dict(v_cache=(9 * PTR, 8, 4096, 256, 128)), INVALID),
    *[({out: i * PTR}, INVALID) for out in ("tables_out", "lens_out", "held_out", "served",
                                            "shares_out", "free_out") for i in range(1, 8)],
])
def test_fork_rows_refusals(L, kw, status):
    f = _fork(**kw)
    assert L.ssd_fork_rows(ctypes.byref(f), None, 0, None, None) == status
    if status == WORKSPACE:
        n = L.ssd_fork_rows_workspace_size(ctypes.byref(f))
        assert n > 0 and n % 256 == 0
        assert L.ssd_fork_rows(ctypes.byref(f), PTR + 128, n, None, None) == WORKSPACE
        assert L.ssd_fork_rows(ctypes.byref(f), PTR, n - 1, None, None) == WORKSPACE
    assert L.ssd_fork_rows(None, None, 0, None, None) == INVALID
    assert L.ssd_fork_rows_workspace_size(None) == 0


def test_python_layer_wants_gpu_tensors():
    import torch

    c = torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16)
    x = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    for call in (lambda: ssd.tree_attention(x, x[:, :, :2], x[:, :, 2:], c, c, t, i),
                 lambda: ssd.append_path(x[:, :, :2], x[:, :, 2:], c, c, i.long(), i, i),
                 lambda: ssd.fork_rows(i, i, i, t, i, i, i[:1], 16)):
        with pytest.raises(ssd.SSDError):
            call()


def test_tensors_of_a_gpu_that_is_not_current_are_refused(monkeypatch):
    import torch

    class Elsewhere(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    def there(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype).as_subclass(Elsewhere)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    c = there(9, 16, 2, 64, dtype=torch.bfloat16)
    q, k = there(2, 3, 4, 64, dtype=torch.bfloat16), there(2, 3, 2, 64, dtype=torch.bfloat16)
    i, t = there(2), there(2, 4)
    for call in (lambda: ssd.tree_attention(q, k, k, c, c, t, i),
                 lambda: ssd.append_path(k, k, c, c, i, i, i),
                 lambda: ssd.fork_rows(i, i, i, t, i, i, there(1), 16)):
        with pytest.raises(ssd.SSDError, match="cuda:1.*cuda:0"):
            call()


def test_packed_descriptors_are_the_structs():
    """What the binding packs has the size of the structs, field after field."""
    for pack, kind, floats in ((ssd._PACK_TREE, _TreeAttn, 1), (ssd._PACK_APPEND, _Append, 0),
                               (ssd._PACK_FORK, _Fork, 0)):
        leaves = []

        def walk(prefix, t):
            for name, f in t._fields_:
                if issubclass(f, ctypes.Structure):
                    walk(prefix + [name], f)
                else:
                    leaves.append(prefix + [name])

        walk([], kind)
        values = [i + 1 for i in range(len(leaves))]
        b = pack(*values)
        assert len(b) == ctypes.sizeof(kind)
        if kind is _TreeAttn:            # a pointer to bytes reads them
            kind = type("T", (ctypes.Structure,), {"_fields_": [
                (n, ctypes.c_void_p if f is ctypes.c_char_p else f) for n, f in kind._fields_]})
        x = kind.from_buffer_copy(b)
        for want, at in zip(values, leaves):
            y = x
            for name in at:
                y = getattr(y, name)
            assert y == want, at


def test_outputs_of_a_fork_are_known_again_and_come_whole():
    import torch

    counts = (4 * 7, 4, 4, 4, 33, 1)
    for mode in (torch.inference_mode, torch.no_grad):
        with mode():
            o = ssd._fork_views(torch, counts, 7, torch.device("cpu"))
            assert ssd._fork_pointers(o, counts, torch.int32, -1) == [o[k].data_ptr() for k in ssd._FORK]
            for name in ssd._FORK:
                for bad in ({k: v for k, v in o.items() if k != name},
                            dict(o, **{name: o[name].clone()})):
                    with pytest.raises(ssd.SSDError):
                        ssd._fork_pointers(bad, counts, torch.int32, -1)
            for other in ((4 * 7, 4, 4, 4, 49, 1), (5 * 7, 5, 5, 5, 33, 1), (4 * 7, 20, 4, 4, 33, 1)):
                with pytest.raises(ssd.SSDError):
                    ssd._fork_pointers(o, other, torch.int32, -1)


@pytest.mark.parametrize("made,asked", [
    ((4, 7, 33), (7, 4, 33)), ((4, 7, 33), (14, 2, 48)), ((4, 7, 33), (4, 7, 40)),
    ((4, 6, 30), (6, 4, 30)), ((8, 10, 97), (10, 8, 112)), ((2, 3, 100), (2, 3, 110)),
    ((16, 16, 16), (16, 16, 15)), ((3, 5, 20), (5, 3, 20)),
])
def test_outputs_of_a_fork_of_other_sizes_are_refused(made, asked):
    """Rows, columns and pages that take the same room in the buffer are told apart."""
    import torch

    def counts(B, cols, pages):
        return B * cols, B, B, B, pages, 1

    o = ssd._fork_views(torch, counts(*made), made[1], torch.device("cpu"))
    assert ssd._fork_pointers(o, counts(*made), torch.int32, -1) == [o[k].data_ptr() for k in ssd._FORK]
    with pytest.raises(ssd.SSDError, match="earlier call"):
        ssd._fork_pointers(o, counts(*asked), torch.int32, -1)


def test_outputs_of_a_fork_seen_otherwise_are_refused():
    import torch

    counts = (4 * 4, 4, 4, 4, 33, 1)
    o = ssd._fork_views(torch, counts, 4, torch.device("cpu"))
    for bad in (dict(tables=o["tables"].t()), dict(tables=o["tables"].view(-1)),
                dict(lens=o["lens"][:3]), dict(shares=o["shares"][:32])):
        with pytest.raises(ssd.SSDError, match="earlier call"):
            ssd._fork_pointers(dict(o, **bad), counts, torch.int32, -1)


class _Library:
    """Keeps the descriptors of its calls."""

    def __init__(self):
        self.seen = []

    def __getattr__(self, name):
        def call(a, *rest):
            self.seen.append((name, a))
            return 256 if name.endswith("workspace_size") else 0
        return call


@pytest.fixture
def here(monkeypatch):
    """The binding with a library that launches nothing, and CPU tensors that pass for the current
    GPU's."""
    import torch

    class Here(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

    library = _Library()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(ssd, "lib", lambda: library)
    monkeypatch.setattr(ssd, "_torch_module", torch)
    return library, lambda t: t.as_subclass(Here)


def test_a_path_of_no_columns_is_a_path(here):
    import torch

    library, on = here
    k, c = (on(torch.zeros(shape, dtype=torch.bfloat16)) for shape in ((2, 3, 2, 64), (9, 16, 2, 64)))
    slots, owner, cu = on(torch.zeros(4, dtype=torch.int64)), on(torch.zeros(4, dtype=torch.int32)), \
        on(torch.tensor([0, 2, 4], dtype=torch.int32))
    for path in (None, on(torch.zeros((2, 0), dtype=torch.int32)),
                 on(torch.zeros((2, 2), dtype=torch.int32)[:, :0]),
                 on(torch.zeros((2, 2), dtype=torch.int32))):
        ssd.append_path(k, None, c, None, slots, owner, cu, path)
        a = _Append.from_buffer_copy(library.seen.pop()[1])
        assert a.path_cols == (0 if path is None else path.shape[1])
        assert bool(a.path) == (path is not None)  # without an address: a chain


def _drafts(on, N):
    import torch

    q, k = (on(torch.zeros((2, N, H, 64), dtype=torch.bfloat16)) for H in (4, 2))
    c = on(torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16))
    return q, k, k, c, c, on(torch.zeros((2, 4), dtype=torch.int32)), \
        on(torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("parent", [
    [-1, 0, 2 ** 31], [-1, 0, -2 ** 40], [-1, 0, 2 ** 70], [-1, 0.5, 1], np.array([-1.0, 0.0, 0.9]),
    np.array([[-1, 5], [0, 5], [1, 5]]), [[-1], [0], [1]], [-1, 0], [-1, 0, 1, 1], [-1, None, 0],
    ["-1", "0", "1"], [-1, [0], 0], 3, np.int64(3), np.array([2 ** 40, 0, 0]),
    np.array([2 ** 64 - 1, 0, 0], dtype=np.uint64),
])
def test_parents_that_are_no_tree_of_the_nodes_are_refused(here, parent):
    library, on = here
    with pytest.raises(ssd.SSDError, match="parent"):
        ssd.tree_attention(*_drafts(on, 3), parent=parent, lse=False)
    assert not library.seen


def test_parents_of_any_whole_type(here):
    import torch

    library, on = here
    for parent in ([-1, 0, 0], (-1, 0, 0), np.array([-1, 0, 0]), np.array([-1, 0, 0], dtype=np.int8),
                   np.array([[-1, 0, 0]] * 2)[0], torch.tensor([-1, 0, 0]), [np.int64(-1), 0, 0],
                   [-1.0, 0.0, 0.0], np.array([-1, 0, 0], dtype=object),
                   np.array([-1, 7, 0, 7, 0])[::2]):
        ssd.tree_attention(*_drafts(on, 3), parent=parent, lse=False)
        name, a = library.seen.pop()
        library.seen.clear()
        assert name == "ssd_tree_attention"
        at = type("T", (ctypes.Structure,), {"_fields_": [
            (n, ctypes.c_void_p if f is ctypes.c_char_p else f) for n, f in _TreeAttn._fields_]}) \
            .from_buffer_copy(a).parent
        assert np.frombuffer(ctypes.string_at(at, 12), dtype=np.int32).tolist() == [-1, 0, 0]


@pytest.mark.parametrize("kw,status", [
    *[({f"out_{d}_stride": x}, INVALID) for d in ("seq", "node", "head") for x in (0, 8, 56)],
    ({"out_head_stride": 64}, WORKSPACE),
    ({"B": 1, "out_seq_stride": 0}, WORKSPACE), ({"N": 1, "out_node_stride": 0}, WORKSPACE),
    ({"Hq": 1, "Hkv": 1, "out_head_stride": 0}, WORKSPACE),
])
def test_outputs_that_lie_on_one_another_are_refused(L, kw, status):
    assert L.ssd_tree_attention(ctypes.byref(_tree(**kw)), None, 0, None, None) == status


@pytest.mark.parametrize("at,n", list(enumerate(("L", "num_pages", "page_size", "H"))))
@pytest.mark.parametrize("name", ["k_cache", "v_cache"])
def test_caches_that_lie_on_themselves_are_refused(L, at, n, name):
    """An expanded cache, or one whose rows overlap, takes several tokens in one place."""
    for x in (0, 16, 112):
        row = [*ROW]
        row[at] = x
        kw = {name: ((3 if name == "k_cache" else 4) * PTR, *row)}
        assert L.ssd_append_path(ctypes.byref(_append(**kw)), None, None) == INVALID
        assert L.ssd_append_path(ctypes.byref(_append(**kw, **{n: 1})), None, None) == 0
        # nodes are only read
        assert L.ssd_append_path(ctypes.byref(_append(k=(PTR, *row))), None, None) == 0


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38])
def test_scales_that_pass_float32_in_base_2_are_refused(L, scale):
    a = _tree(scale=scale)
    assert L.ssd_tree_attention(ctypes.byref(a), None, 0, None, None) == INVALID
    assert L.ssd_tree_attention_workspace_size(ctypes.byref(a)) == 0
    assert L.ssd_tree_attention(ctypes.byref(_tree(scale=scale * 0.9)), None, 0, None, None) == \
        (WORKSPACE if abs(scale) < 2.5e38 else INVALID)
