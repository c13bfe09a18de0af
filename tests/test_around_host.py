"""Argument checks of the operators around the attention, without a GPU: every refusal comes before
any pointer is used."""
import ctypes
import math

import pytest

from conftest import has_gpu

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def ffi():
    from diffusion_transformer_ultra_b200 import _ffi, build
    build.build()
    return _ffi


@pytest.fixture()
def mem():
    buf = ctypes.create_string_buffer(1 << 12)
    return ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16, buf


def norm(ffi, **kw):
    n = dict(batch=2, rows=3, cols=64, dtype=0, wdtype=0, per_sample=0, plus_one=0, eps=1e-6, x_row=64, x_batch=192, y_row=64,
             y_batch=192, dy_row=64, dy_batch=192)
    n.update(kw)
    return ffi.NormSizes(**n)


def adapter(ffi, **kw):
    c = dict(rows=4, k=64, n=32, rank=8, adapters=2, dtype=0, x_row=64, y_row=32)
    c.update(kw)
    return ffi.AdapterSizes(**c)


def cross(ffi, **kw):
    c = dict(batch=2, nq=5, ns=7, heads=4, kv_heads=2, head_dim=64, dtype=0, masked=0, scale=0.125)
    c.update(kw)
    s = ffi.CrossSizes(**c)
    for t in range(8):
        s.stride[t][:] = (1 << 12, 256, 64)
    return s


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dtype=9), INVALID),
    (dict(wdtype=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(cols=16385), UNSUPPORTED), (dict(batch=1 << 16, rows=1 << 16), UNSUPPORTED),
    (dict(batch=1 << 16, per_sample=1), UNSUPPORTED)])
def test_layer_norm_sizes(ffi, mem, bad, status):
    a, _ = mem
    L, n, need = ffi.lib(), norm(ffi, **bad), ctypes.c_size_t()
    assert L.ultragen_layer_norm(n, a, None, None, a, None, None, None) == status
    assert L.ultragen_layer_norm_backward_workspace(n, ctypes.byref(need)) == status
    assert L.ultragen_layer_norm_backward(n, a, a, None, a, a, a, None, None, 0, None, 0, None) == status


def test_layer_norm_pointers(ffi, mem):
    a, _ = mem
    L, n, need = ffi.lib(), norm(ffi), ctypes.c_size_t()
    assert L.ultragen_layer_norm(n, None, None, None, a, None, None, None) == INVALID
    assert L.ultragen_layer_norm(n, a, None, None, None, None, None, None) == INVALID
    assert L.ultragen_layer_norm(None, a, None, None, a, None, None, None) == INVALID
    assert L.ultragen_layer_norm(norm(ffi, rows=0), None, None, None, None, None, None, None) == OK
    for hole in range(5):
        p = [a] * 5
        p[hole] = None
        assert L.ultragen_layer_norm_backward(n, p[0], p[1], None, p[2], p[3], p[4], None, None, 0, None, 0, None) == INVALID
    assert L.ultragen_layer_norm_backward(n, a, a, None, a, a, a, None, None, 7, None, 0, None) == INVALID
    assert L.ultragen_layer_norm_backward_workspace(n, None) == INVALID
    assert L.ultragen_layer_norm_backward_workspace(n, ctypes.byref(need)) == OK and need.value % 16 == 0 and need.value > 0


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), INVALID), (dict(k=0), INVALID), (dict(n=0), INVALID), (dict(rank=0), INVALID), (dict(adapters=0), INVALID),
    (dict(dtype=5), INVALID), (dict(rank=129), UNSUPPORTED), (dict(n=4194241), UNSUPPORTED)])
def test_adapter_sizes(ffi, mem, bad, status):
    a, _ = mem
    L, c, need = ffi.lib(), adapter(ffi, **bad), ctypes.c_size_t()
    assert L.ultragen_adapter_project_workspace(c, ctypes.byref(need)) == status
    assert L.ultragen_adapter_project(c, a, a, None, a, a, None, a, a, a, 1 << 20, None) == status


def test_adapter_sizes_whose_tiles_would_pass_32_bits(ffi, mem):
    """A tile of rows, or the warps' pieces of k, behind the last one must still have an index."""
    a, _ = mem
    L, need = ffi.lib(), ctypes.c_size_t()
    for most in (dict(rows=2 ** 31 - 256), dict(k=2 ** 31 - 512, x_row=2 ** 31)):
        c = adapter(ffi, **most)
        assert L.ultragen_adapter_project_workspace(c, ctypes.byref(need)) == OK and need.value > 0
        assert L.ultragen_adapter_project(c, a, a, None, a, a, None, a, a, None, 0, None) == INVALID      # (no workspace)
    for past in (dict(rows=2 ** 31 - 255), dict(rows=2 ** 31 - 1), dict(k=2 ** 31 - 511), dict(k=2 ** 31 - 1)):
        c = adapter(ffi, **past)
        assert L.ultragen_adapter_project_workspace(c, ctypes.byref(need)) == UNSUPPORTED
        assert L.ultragen_adapter_project(c, a, a, None, a, a, None, a, a, a, 1 << 20, None) == UNSUPPORTED


def test_adapter_pointers(ffi, mem):
    a, _ = mem
    L, c, need = ffi.lib(), adapter(ffi), ctypes.c_size_t()
    assert L.ultragen_adapter_project_workspace(c, ctypes.byref(need)) == OK
    order = ("x", "w", "a", "b", "ids", "y", "ws")

    def call(**p):
        q = dict.fromkeys(order, a)
        size = p.pop("size", need.value)
        q.update(p)
        return L.ultragen_adapter_project(c, q["x"], q["w"], None, q["a"], q["b"], None, q["ids"], q["y"], q["ws"], size, None)
    for name in order:
        assert call(**{name: None}) == INVALID
    assert call(size=need.value - 1) == INVALID
    assert call(ws=a + 8) == INVALID
    assert L.ultragen_adapter_project(adapter(ffi, rows=0), *[None] * 9, 0, None) == OK


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), INVALID), (dict(nq=-1), INVALID), (dict(ns=-1), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(heads=3), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(dtype=1), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(heads=258, kv_heads=2), UNSUPPORTED),
    (dict(batch=1 << 15, nq=1 << 14), UNSUPPORTED)])
def test_cross_sizes(ffi, mem, bad, status):
    a, _ = mem
    L, c, need = ffi.lib(), cross(ffi, **bad), ctypes.c_size_t()
    for back in (0, 1):
        assert L.ultragen_cross_attention_workspace(c, back, ctypes.byref(need)) == status
    assert L.ultragen_cross_attention(c, a, a, a, None, None, a, None, a, 1 << 20, None) == status
    assert L.ultragen_cross_attention_backward(c, a, a, a, a, a, a, None, None, a, a, a, a, 1 << 20, None) == status


def test_cross_pointers_and_strides(ffi, mem):
    a, _ = mem
    L, need = ffi.lib(), ctypes.c_size_t()
    c = cross(ffi, masked=1)
    assert L.ultragen_cross_attention_workspace(c, 0, ctypes.byref(need)) == OK and need.value > 0
    assert L.ultragen_cross_attention_workspace(c, 2, ctypes.byref(need)) == INVALID
    assert L.ultragen_cross_attention_workspace(c, 0, None) == INVALID
    assert L.ultragen_cross_attention_workspace(c, 0, ctypes.byref(need)) == OK
    assert L.ultragen_cross_attention(c, a, a, a, None, a, a, None, a, need.value - 1, None) == INVALID
    assert L.ultragen_cross_attention(c, a, a, a, None, a, a, None, None, need.value, None) == INVALID
    for hole in range(4):
        p = [a] * 4
        p[hole] = None
        assert L.ultragen_cross_attention(c, *p[:3], None, a, p[3], None, a, need.value, None) == INVALID
        p[hole] = a + 8
        assert L.ultragen_cross_attention(c, *p[:3], None, a, p[3], None, a, need.value, None) == INVALID
    # a mask the workspace was not sized for
    assert L.ultragen_cross_attention(cross(ffi), a, a, a, None, a, a, None, a, 1 << 20, None) == INVALID
    for t in range(8):
        c = cross(ffi)
        c.stride[t][1] = 60
        if t < 4:
            assert L.ultragen_cross_attention(c, a, a, a, None, None, a, None, a, 1 << 20, None) == INVALID
        assert L.ultragen_cross_attention_backward(c, a, a, a, a, a, a, None, None, a, a, a, a, 1 << 20, None) == INVALID
    assert L.ultragen_cross_attention(cross(ffi, batch=0), *[None] * 8, 0, None) == OK


def test_an_output_that_is_an_operand(ffi):
    """Outputs that begin where an operand does that the call still reads are refused; the pairs that the
    header allows get past the checks (to the device, of which there need be none)."""
    L, need = ffi.lib(), ctypes.c_size_t()
    buf = ctypes.create_string_buffer(1 << 16)
    base = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    names = iter(range(64))

    def place():
        return base + 16 * next(names)
    x, y, w, b, mean, rstd, dy, dw, db = (place() for _ in range(9))
    n = norm(ffi)
    fwd = dict(x=x, w=w, b=b, y=y, mean=mean, rstd=rstd)

    def forward(n=n, **kw):
        q = dict(fwd, **kw)
        return L.ultragen_layer_norm(n, *(q[k] for k in ("x", "w", "b", "y", "mean", "rstd")), None)
    for other in ("w", "b", "mean", "rstd"):
        assert forward(y=fwd[other]) == INVALID
    assert forward(mean=rstd) == INVALID
    assert forward(norm(ffi, y_row=65), y=x) == INVALID and forward(norm(ffi, y_batch=256), y=x) == INVALID
    bwd = dict(dy=dy, x=x, w=w, mean=mean, rstd=rstd, dx=y, dw=None, db=None)

    def backward(n=n, ws=None, **kw):
        q = dict(bwd, **kw)
        return L.ultragen_layer_norm_backward(n, *(q[k] for k in ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db")), 1, ws,
                                              1 << 20 if ws else 0, None)
    for other in ("w", "mean", "rstd"):
        assert backward(dx=bwd[other]) == INVALID
    assert backward(norm(ffi, y_row=65), dx=x) == INVALID and backward(norm(ffi, dy_row=65), dx=dy) == INVALID
    assert backward(ws=base, dw=dw, db=dw) == INVALID and backward(ws=base, dx=dw, dw=dw, db=db) == INVALID
    c = adapter(ffi)
    assert L.ultragen_adapter_project_workspace(c, ctypes.byref(need)) == OK
    order = ("x", "w", "bias", "a", "b", "scales", "ids")
    ops = {k: place() for k in order}
    ws = place()
    for other in order:
        assert L.ultragen_adapter_project(c, *(ops[k] for k in order), ops[other], ws, need.value, None) == INVALID
    q, k, v, o, do, dq, dk, dv, lse = (place() for _ in range(9))
    c = cross(ffi, nq=7, kv_heads=4, batch=200)                # (enough items: no workspace forward)
    assert L.ultragen_cross_attention_workspace(c, 0, ctypes.byref(need)) == OK and need.value == 0

    def attend(c=c, out=o):
        return L.ultragen_cross_attention(c, q, k, v, None, None, out, lse, None, 0, None)
    assert attend(out=k) == INVALID and attend(out=v) == INVALID and attend(out=lse) == INVALID
    other = cross(ffi, nq=7, kv_heads=4, batch=200)
    other.stride[3][1] = 512
    assert attend(other, out=q) == INVALID
    assert L.ultragen_cross_attention_workspace(c, 1, ctypes.byref(need)) == OK
    back = dict(do=do, q=q, k=k, v=v, o=o, lse=lse, dq=dq, dk=dk, dv=dv)

    def grad(**kw):
        p = dict(back, **kw)
        return L.ultragen_cross_attention_backward(c, p["do"], p["q"], p["k"], p["v"], p["o"], p["lse"], None, None, p["dq"], p["dk"],
                                                   p["dv"], ws, need.value, None)
    for other in ("q", "k", "v", "do", "dk", "dv", "lse"):
        assert grad(dq=back[other]) == INVALID
    for out in ("dk", "dv"):
        for other in ("q", "do"):
            assert grad(**{out: back[other]}) == INVALID
    assert grad(dk=dv) == INVALID
    if not has_gpu():                                          # (host addresses: nothing may be launched)
        NO_DEVICE = 7
        assert forward() == forward(y=x) == backward() == backward(dx=x) == backward(dx=dy) == NO_DEVICE
        assert attend() == attend(out=q) == grad() == NO_DEVICE


def test_binding_refuses_host_tensors():
    import torch
    import diffusion_transformer_ultra_b200 as ug
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ug.layer_norm(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        ug.layer_norm_backward(x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        ug.adapter_project(x, x, x, x, x, x)
    q = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ug.cross_attention(q, q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        ug.cross_attention_backward(q, q, q, q, q, q, q, q, q)


@pytest.fixture()
def devices(monkeypatch):
    """Two devices without a GPU: the current one is a list's only entry, streams know theirs."""
    import contextlib
    import torch
    current = [torch.device("cuda", 0)]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d)
        yield
        current[0] = before

    class Stream:
        def __init__(self, index):
            self.device, self.cuda_stream = torch.device("cuda", index), 100 + index
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0].index)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream((current[0] if d is None else torch.device(d)).index))
    return current, Stream


def test_status_is_asked_of_the_streams_device(ffi, devices, monkeypatch):
    import diffusion_transformer_ultra_b200 as ug
    from diffusion_transformer_ultra_b200 import around
    current, stream = devices
    asked = []

    class Library:
        @staticmethod
        def ultragen_operator_status(s):
            asked.append((current[0].index, s))
            return 0
    monkeypatch.setattr(around, "lib", lambda: Library)
    assert ug.operator_status() == ug.operator_status(stream(1)) == ug.operator_status(stream(0)) == 0
    assert asked == [(0, 100), (1, 101), (0, 100)] and current[0].index == 0


def test_a_projected_layer_runs_on_its_own_device(devices, monkeypatch):
    """Every step, the joint attention's too, with the buffers' device current; an output elsewhere is refused."""
    import types
    import torch
    from diffusion_transformer_ultra_b200 import around
    current, _ = devices
    ran = []
    one, zero = torch.device("cuda", 1), torch.device("cuda", 0)

    class Fake(torch.Tensor):
        device = one
    pl = object.__new__(around.ProjectedLayer)
    pl.norm = types.SimpleNamespace(device=one, view=lambda *s: None)
    pl.shape = (1, 2, 3, 4)
    pl.q = pl.k = pl.v = pl.xq = types.SimpleNamespace(view=lambda *s: None)
    pl.layer = lambda q, k, v, o, stream: ran.append(("layer", current[0])) or o
    monkeypatch.setattr(around, "layer_norm", lambda *a, **k: ran.append(("norm", current[0])))
    monkeypatch.setattr(around, "adapter_project", lambda *a, **k: ran.append(("project", current[0])))
    o = torch.zeros(1).as_subclass(Fake)
    three = [None] * 3
    assert pl(None, o, three, three, three, None) is o
    assert ran == [("norm", one)] + [("project", one)] * 3 + [("layer", one)] and current[0] == zero
    with pytest.raises(ValueError, match="cuda:1"):
        pl(None, torch.zeros(1), three, three, three, None)
    assert len(ran) == 5
