"""Layer norm, forward and backward, against a plain implementation in float64.

Tolerances, with u half a step of the output type (bf16 2^-8, fp16 2^-11, fp32 2^-24), e = 2^-24 and
C columns; every sum of n fp32 terms is off by at most n e of the sum of their absolute values (trees
and warps make the kernels' shorter than that).
  mean: (C + 1) e mean|x|.   d = x - mean is off by that plus e |d|, called ed.
  var:  (C + 3) e var + 2 mean|d ed|;  rstd: half the relative error of var + eps, plus 3 e (the
        division and the root).
  y:    with xh = d rstd: |w'| (|xh| (rel rstd + 3 e) + ed rstd) + 2 e (|y| + |b|) + u |y|.
  backward, from the given mean and rstd: xh off by ex = 3 e (|xh| + |mean| rstd) + 0;
        g = dy w' by 2 e |g|; a = mean g by (C + 4) e mean|g|; c = mean(g xh) by
        (C + 6) e mean|g xh| + mean(|g| ex);
        dx: rstd (2 e |g| + err a + |xh| err c + |c| ex + 6 e (|g| + |a| + |xh c|)) + u |dx|;
        dw: sum (n + 4) e |dy xh| + |dy| ex over its n rows, db: n e sum|dy|, plus u of each.
fp16 results have 2^-25 (half their smallest step) on top.
"""
import pytest

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module")
def ug(gpu_required):
    from diffusion_transformer_ultra_b200 import build
    build.build()
    import diffusion_transformer_ultra_b200 as pkg
    return pkg


def dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def rnd(t, ref):
    import torch
    return torch.finfo(t).eps / 2 * ref.abs() + (2.0 ** -25 if t == torch.float16 else 0.0) + 1e-30


def make(B, R, C, dtype, weight, wdtype=None, seed=0, offset=0.3):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(7 + seed)

    def r(*s):
        return torch.randn(s, generator=g, device="cuda")
    t, wt = dt(dtype), dt(wdtype or dtype)
    shape = {"shared": (C,), "sample": (B, C), "none": None}[weight]
    w = b = None
    if shape:
        w, b = (1 + 0.3 * r(*shape)).to(wt), (0.2 * r(*shape)).to(wt)
    return (r(B, R, C) + offset * r(C)).to(t), r(B, R, C).to(t), w, b


def bcast(w, per_sample):
    return w[:, None] if per_sample else w


def forward_reference(x, w, b, plus, eps, t):
    import torch
    C = x.shape[-1]
    xd = x.double()
    mean = xd.mean(-1, keepdim=True)
    d = xd - mean
    emean = (C + 1) * E * xd.abs().mean(-1, keepdim=True)
    ed = emean + E * d.abs()
    var = (d * d).mean(-1, keepdim=True)
    evar = (C + 3) * E * var + 2 * (d.abs() * ed).mean(-1, keepdim=True) + (ed * ed).mean(-1, keepdim=True)
    rstd = (var + eps) ** -0.5
    rel = 0.5 * evar / (var + eps) + 3 * E
    per = w is not None and w.dim() == 2
    wd = torch.ones((), dtype=torch.float64, device="cuda") if w is None else bcast(w.double(), per) + plus
    bd = 0.0 * wd if b is None else bcast(b.double(), per)
    xh = d * rstd
    y = xh * wd + bd
    tol = wd.abs() * (xh.abs() * (rel + 3 * E) + ed * rstd) + 2 * E * (y.abs() + bd.abs()) + rnd(t, y)
    return (y, tol), (mean.squeeze(-1), emean.squeeze(-1) + 1e-30), (rstd.squeeze(-1), (rel * rstd).squeeze(-1))


def backward_reference(dy, x, mean, rstd, w, plus, t, gt, per_sample):
    import torch
    C = x.shape[-1]
    m, r = mean.double()[..., None], rstd.double()[..., None]
    per = w is not None and w.dim() == 2
    wd = torch.ones((), dtype=torch.float64, device="cuda") if w is None else bcast(w.double(), per) + plus
    g, xh = dy.double() * wd, (x.double() - m) * r
    ex = 3 * E * (xh.abs() + m.abs() * r)
    a, c = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    ea = (C + 4) * E * g.abs().mean(-1, keepdim=True)
    ec = (C + 6) * E * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * ex).mean(-1, keepdim=True)
    dx = r * (g - a - xh * c)
    tol = r * (2 * E * g.abs() + ea + xh.abs() * ec + c.abs() * ex + 6 * E * (g.abs() + a.abs() + (xh * c).abs()))
    over = (1,) if per_sample else (0, 1)
    n = x.shape[1] * (1 if per_sample else x.shape[0])
    d = dy.double()
    dw, db = (d * xh).sum(over), d.sum(over)
    tw = ((n + 4) * E * (d * xh).abs() + d.abs() * ex).sum(over)
    tb = n * E * d.abs().sum(over)
    return (dx, tol + rnd(t, dx)), (dw, tw + rnd(gt, dw)), (db, tb + rnd(gt, db))


def check(name, got, ref):
    want, tol = ref
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} off, first at {i}: {got[i]} for {want[i]} +- {tol[i]}")


def run(ug, B, R, C, dtype, weight, wdtype=None, plus=False, eps=1e-6, grad="fp32", offset=0.3):
    import torch
    x, dy, w, b = make(B, R, C, dtype, weight, wdtype, offset=offset)
    y = torch.full_like(x, float("nan"))
    mean, rstd = (torch.full((B, R), float("nan"), device="cuda") for _ in range(2))
    ug.layer_norm(x, y, w, b, eps=eps, plus_one=plus, mean=mean, rstd=rstd)
    ry, rm, rr = forward_reference(x, w, b, float(plus), eps, x.dtype)
    check("y", y, ry)
    check("mean", mean, rm)
    check("rstd", rstd, rr)
    dx = torch.full_like(x, float("nan"))
    shape = (B, C) if weight == "sample" else (C,)
    dw, db = (torch.full(shape, float("nan"), dtype=dt(grad), device="cuda") for _ in range(2))
    ug.layer_norm_backward(dy, x, mean, rstd, dx, w, plus_one=plus, dweight=dw, dbias=db)
    rx, rw, rb = backward_reference(dy, x, mean, rstd, w, float(plus), x.dtype, dt(grad), weight == "sample")
    check("dx", dx, rx)
    check("dweight", dw, rw)
    check("dbias", db, rb)


SHAPES = [(1, 1, 1), (1, 1, 8), (2, 3, 7), (1, 5, 511), (3, 77, 512), (2, 9, 513), (2, 33, 1153), (1, 40, 1536), (2, 17, 2048),
          (1, 3, 8191), (1, 4, 8192), (2, 2, 16384), (1, 3000, 64), (2, 700, 256), (4, 130, 1000)]


@pytest.mark.parametrize("weight", ["none", "shared", "sample"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_sizes(ug, shape, dtype, weight):
    run(ug, *shape, dtype, weight, plus=weight == "sample")


@pytest.mark.parametrize("dtype,wdtype,grad", [("bf16", "fp32", "bf16"), ("fp16", "fp32", "fp16"), ("fp16", "fp16", "fp32")])
@pytest.mark.parametrize("weight", ["shared", "sample"])
def test_types(ug, dtype, wdtype, grad, weight):
    run(ug, 3, 50, 768, dtype, weight, wdtype, plus=True, grad=grad, eps=1e-3)


def test_mean_far_above_the_spread(ug):
    """A sum of squares would cancel: the variance comes from the distances to the mean."""
    run(ug, 2, 20, 1536, "fp32", "shared", offset=300.0)


def test_rows_of_equal_values(ug):
    """The variance is zero: y = bias, rstd = eps^-1/2, and every gradient is finite."""
    import torch
    x = torch.full((1, 4, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    w, b = torch.ones(200, device="cuda"), torch.linspace(-1, 1, 200, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(1, 4, device="cuda"), torch.empty(1, 4, device="cuda")
    ug.layer_norm(x, y, w, b, eps=1e-4, mean=mean, rstd=rstd)
    assert torch.equal(y, b.to(torch.bfloat16).expand_as(y)) and (mean == 3).all()
    assert ((rstd - 100).abs() <= 100 * 4 * E).all()
    dx = torch.empty_like(x)
    ug.layer_norm_backward(torch.ones_like(x), x, mean, rstd, dx, w)
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("C", [200, 515, 1536])
def test_a_row_of_nan_stays_alone(ug, C):
    import torch
    x, dy, w, b = make(2, 9, C, "bf16", "shared")
    want, dwant = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(2, 9, device="cuda"), torch.empty(2, 9, device="cuda")
    ug.layer_norm(x, want, w, b, mean=mean, rstd=rstd)
    ug.layer_norm_backward(dy, x, mean, rstd, dwant, w)
    x[1, 4, C // 2] = float("nan")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    ug.layer_norm(x, y, w, b, mean=mean, rstd=rstd)
    ug.layer_norm_backward(dy, x, mean, rstd, dx, w)
    rest = torch.ones(2, 9, dtype=torch.bool, device="cuda")
    rest[1, 4] = False
    assert torch.isnan(y[1, 4]).all() and torch.equal(y[rest], want[rest]) and torch.equal(dx[rest], dwant[rest])


@pytest.mark.parametrize("C,step", [(64, 65), (1536, 1544), (1153, 1160), (520, 1)])
def test_strides_and_in_place(ug, C, step):
    """Rows apart, samples in any order, y over x and dx over dy; what lies between stays."""
    import torch
    B, R = 2, 31
    x, dy, w, b = make(B, R, C, "bf16", "sample")

    def apart(t):
        big = torch.full((R, B, max(step, C)), 7.0, dtype=t.dtype, device="cuda")
        v = big[..., :C].transpose(0, 1)
        v.copy_(t)
        return big, v
    bigx, xv = apart(x)
    bigd, dv = apart(dy)
    mean, rstd = torch.empty(B, R, device="cuda"), torch.empty(B, R, device="cuda")
    y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty(B, C, device="cuda"), torch.empty(B, C, device="cuda")
    ug.layer_norm(x, y, w, b, mean=mean, rstd=rstd)
    check("y", y, forward_reference(x, w, b, 0.0, 1e-6, x.dtype)[0])
    ug.layer_norm_backward(dy, x, mean, rstd, dx, w, dweight=dw, dbias=db)
    dw2 = torch.empty_like(dw)
    ug.layer_norm_backward(dv, xv, mean, rstd, dv, w, dweight=dw2, dbias=db)
    ug.layer_norm(xv, xv, w, b)
    # (unaligned rows sum in another order than aligned ones: compare with the formula instead)
    rx, rw, _ = backward_reference(dy, x, mean, rstd, w, 0.0, x.dtype, torch.float32, True)
    check("y in place", xv, forward_reference(x, w, b, 0.0, 1e-6, x.dtype)[0])
    check("dx in place", dv, rx)
    check("dweight", dw2, rw)
    assert (bigx[..., C:] == 7).all() and (bigd[..., C:] == 7).all()


def test_two_dimensions_and_parts_of_the_gradients(ug):
    import torch
    x, dy, w, b = make(1, 50, 320, "fp16", "shared")
    mean, rstd = torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
    y = torch.empty_like(x[0])
    ug.layer_norm(x[0], y, w, mean=mean, rstd=rstd)
    check("y", y[None], forward_reference(x, w, None, 0.0, 1e-6, x.dtype)[0])
    rx, rw, rb = backward_reference(dy, x, mean[None], rstd[None], w, 0.0, x.dtype, torch.float32, False)
    for want_w, want_b in ((True, False), (False, True), (False, False)):
        dx = torch.empty_like(y)
        dw, db = torch.empty(320, device="cuda"), torch.empty(320, device="cuda")
        ug.layer_norm_backward(dy[0], x[0], mean, rstd, dx, w, dweight=dw if want_w else None, dbias=db if want_b else None)
        check("dx", dx[None], rx)
        if want_w:
            check("dw", dw, rw)
        if want_b:
            check("db", db, rb)


def test_no_rows(ug):
    import torch
    x = torch.empty(2, 0, 64, device="cuda")
    ug.layer_norm(x, torch.empty_like(x))
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    st = torch.empty(2, 0, device="cuda")
    ug.layer_norm_backward(x, x, st, st, torch.empty_like(x), dweight=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


def test_same_bits_every_time_and_from_graphs(ug):
    import torch
    x, dy, w, b = make(2, 900, 1536, "bf16", "shared", "fp32")

    def buffers():
        return [torch.empty_like(x), torch.empty(2, 900, device="cuda"), torch.empty(2, 900, device="cuda"), torch.empty_like(x),
                torch.empty(1536, device="cuda"), torch.empty(1536, device="cuda")]

    def once(o):
        ug.layer_norm(x, o[0], w, b, mean=o[1], rstd=o[2])
        ug.layer_norm_backward(dy, x, o[1], o[2], o[3], w, dweight=o[4], dbias=o[5])
    sets = [buffers() for _ in range(4)]
    once(sets[0])
    once(sets[1])
    graphs = []
    for o in sets[2:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            once(o)
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for o in sets[1:] for a, c in zip(sets[0], o))


def test_gradients_against_differences(ug):
    import torch
    B, R, C = 2, 6, 96
    x, dy, w, b = make(B, R, C, "fp32", "sample")
    mean, rstd = torch.empty(B, R, device="cuda"), torch.empty(B, R, device="cuda")
    ug.layer_norm(x, torch.empty_like(x), w, b, plus_one=True, mean=mean, rstd=rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ug.layer_norm_backward(dy, x, mean, rstd, dx, w, plus_one=True, dweight=dw, dbias=db)
    refs = backward_reference(dy, x, mean, rstd, w, 1.0, x.dtype, torch.float32, True)

    def loss(x, w, b):
        m = x.mean(-1, keepdim=True)
        v = ((x - m) ** 2).mean(-1, keepdim=True)
        return (((x - m) / torch.sqrt(v + 1e-6) * (1 + w[:, None]) + b[:, None]) * dy.double()).sum()
    args = [t.double() for t in (x, w, b)]
    for i, (got, ref) in enumerate(zip((dx, dw, db), refs)):
        g = torch.Generator(device="cuda")
        g.manual_seed(i)
        d = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        slope = (loss(*up) - loss(*down)) / (2 * h)
        # mean and rstd come rounded from the forward pass: 4 (C + 4) e relative at most, on top
        extra = 4 * (C + 4) * E * (ref[0].abs() + dy.double().abs().amax()) * d.abs()
        assert abs((got.double() * d).sum() - slope) <= (ref[1] * d.abs()).sum() + extra.sum() + 1e-7 * slope.abs()


# Rows enough for a warp to a row (64 to each of 148 multiprocessors): row ends inside and at a lane's piece,
# and one to sixteen pieces of it; samples that end between the two rows of a pair.
MANY = [(3, 3333, 516), (1, 10000, 1024), (3, 3200, 1028), (2, 5000, 1536), (7, 1400, 2044), (1, 9999, 2048)]


@pytest.mark.parametrize("weight", ["none", "shared", "sample"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
@pytest.mark.parametrize("shape", MANY)
def test_many_rows(ug, shape, dtype, wdtype, weight):
    run(ug, *shape, dtype, weight, wdtype, plus=weight == "sample")


@pytest.mark.parametrize("shape,dtype", [((3, 3333, 515), "bf16"), ((2, 5000, 1153), "fp32"), ((1, 400, 16384), "bf16"), ((2, 300, 8191), "fp16"),
                                         ((1, 5000, 4096), "bf16"), ((2, 5000, 2052), "fp16"), ((1, 10000, 640), "fp32")])
def test_many_rows_of_other_widths_and_types(ug, shape, dtype):
    run(ug, *shape, dtype, "sample", plus=True)


@pytest.mark.parametrize("C", [516, 1536, 2048])
def test_many_rows_in_place_and_a_row_of_nan(ug, C):
    """Rows apart and y over x; a row of NaN changes no other row's bits; what lies between the rows stays."""
    import torch
    B, R = 2, 5000
    x, _, w, b = make(B, R, C, "bf16", "sample", "fp32")
    x[1, 77, C // 3] = float("nan")
    want, mean, rstd = torch.empty_like(x), torch.empty(B, R, device="cuda"), torch.empty(B, R, device="cuda")
    ug.layer_norm(x, want, w, b, mean=mean, rstd=rstd)
    rest = torch.ones(B, R, dtype=torch.bool, device="cuda")
    rest[1, 77] = False
    clean = x.clone()
    clean[1, 77] = 0
    ry, rm, rr = forward_reference(clean, w, b, 0.0, 1e-6, x.dtype)
    assert torch.isnan(want[1, 77]).all() and torch.isnan(mean[1, 77])
    for name, got, ref in (("y", want, ry), ("mean", mean, rm), ("rstd", rstd, rr)):
        check(name, got[rest], [t.expand_as(got)[rest] for t in ref])
    big = torch.full((R, B, C + 8), 7.0, dtype=x.dtype, device="cuda")
    v = big[..., :C].transpose(0, 1)
    v.copy_(x)
    ug.layer_norm(v, v, w, b)
    assert torch.equal(v[rest], want[rest]) and torch.isnan(v[1, 77]).all() and (big[..., C:] == 7).all()


def test_one_row_for_all(ug):
    """x and dy of stride zero."""
    import torch
    x, dy, w, b = make(3, 40, 200, "bf16", "shared")
    for xx, dd in ((x[:1].expand_as(x), dy), (x[:, :1].expand_as(x), dy[:1, :1].expand_as(dy))):
        y, mean, rstd = torch.empty_like(dy), torch.empty(3, 40, device="cuda"), torch.empty(3, 40, device="cuda")
        ug.layer_norm(xx, y, w, b, mean=mean, rstd=rstd)
        check("y", y, forward_reference(xx, w, b, 0.0, 1e-6, x.dtype)[0])
        dx, dw = torch.empty_like(dy), torch.empty(200, device="cuda")
        ug.layer_norm_backward(dd, xx, mean, rstd, dx, w, dweight=dw)
        rx, rw, _ = backward_reference(dd, xx, mean, rstd, w, 0.0, x.dtype, torch.float32, False)
        check("dx", dx, rx)
        check("dw", dw, rw)


@pytest.mark.parametrize("shape", [(1, 9471, 1024), (1, 9472, 1024), (65535, 1, 64), (4001, 3, 520)])
def test_row_and_sample_counts_at_the_kernels_borders(ug, shape):
    run(ug, *shape, "bf16", "sample", "fp32", plus=True)


def test_two_streams_at_once(ug):
    import torch
    sets = []
    for seed in range(2):
        x, dy, w, b = make(2, 4000, 1536, "bf16", "shared", "fp32", seed=seed)

        def once(o, a=(x, dy, w, b), stream=None):
            x, dy, w, b = a
            ug.layer_norm(x, o[0], w, b, mean=o[1], rstd=o[2], stream=stream)
            ug.layer_norm_backward(dy, x, o[1], o[2], o[3], w, dweight=o[4], dbias=o[5], stream=stream)
        outs = [[torch.empty_like(x), torch.empty(2, 4000, device="cuda"), torch.empty(2, 4000, device="cuda"), torch.empty_like(x),
                 torch.empty(1536, device="cuda"), torch.empty(1536, device="cuda")] for _ in range(9)]
        once(outs[0])
        sets.append((once, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(1, 9):
        for once, outs, stream in sets:
            once(outs[i], stream=stream)
    torch.cuda.synchronize()
    assert ug.operator_status() == 0
    assert all(torch.equal(a, c) for _, outs, _ in sets for o in outs[1:] for a, c in zip(outs[0], o))


def test_calls_of_several_threads_that_take_unequal_shared_memory(ug):
    """The same kernel for many rows and for few, from host threads at once (through the C call, which runs
    without Python's lock): each launch is accepted."""
    import ctypes
    import threading
    import torch
    from diffusion_transformer_ultra_b200 import around
    call = ctypes.CDLL(ug._ffi.LIB_PATH).ultragen_layer_norm
    call.argtypes = ug.lib().ultragen_layer_norm.argtypes
    jobs, answers = [], []
    for R in (2000, 300, 2000, 300):
        x, _, w, b = make(1, R, 1000, "bf16", "shared")
        y = torch.empty_like(x)
        n, _ = around._norm_sizes(x, w, b, False, 1e-6)
        n.y_row, n.y_batch = y.stride(1), y.stride(0)
        jobs.append((x, y, w, b, n, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(x, y, w, b, n, stream):
        torch.cuda.set_device(x.device)
        args = (ctypes.byref(n), x.data_ptr(), w.data_ptr(), b.data_ptr(), y.data_ptr(), None, None, stream.cuda_stream)
        answers.append({call(*args) for _ in range(20000)})
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert answers == [{0}] * len(jobs)
    for x, y, w, b, *_ in jobs:
        check("y", y, forward_reference(x, w, b, 0.0, 1e-6, x.dtype)[0])


def test_as_many_rows_as_are_taken(ug):
    """2^31 - 1 rows of two columns: a row index plus the walk's step passes 2^31.  Sampled rows at the start,
    in the middle and at the end against the formula; every output is written."""
    import torch
    R, C = 2 ** 31 - 1, 2
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    part = 2 ** 28
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for i in range(0, R, part):                                # (a fill in parts: the generator's own limits)
        x[i:i + part].normal_(generator=g)
    w, b = torch.tensor([1.5, -0.75], device="cuda"), torch.tensor([0.25, -2.0], device="cuda")
    y = torch.full_like(x, float("nan"))
    mean, rstd = (torch.full((R,), float("nan"), device="cuda") for _ in range(2))
    ug.layer_norm(x, y, w, b, eps=1e-3, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    assert ug.operator_status() == 0
    spots = [slice(i, min(i + 5000, R)) for i in (0, R // 3, 2 ** 30 - 2500, R - 5000)]
    for s in spots:
        ry, rm, rr = forward_reference(x[None, s], w, b, 0.0, 1e-3, x.dtype)
        check("y", y[None, s], ry)
        check("mean", mean[None, s], rm)
        check("rstd", rstd[None, s], rr)
    assert not any(torch.isnan(t[i:i + part]).any() for t in (y, mean, rstd) for i in range(0, R, part))
    dx, dw = y, torch.full((C,), float("nan"), device="cuda")
    dx.fill_(float("nan"))
    ug.layer_norm_backward(x, x, mean, rstd, dx, w, dweight=dw)
    torch.cuda.synchronize()
    assert ug.operator_status() == 0 and torch.isfinite(dw).all()
    for s in spots:
        check("dx", dx[None, s], backward_reference(x[None, s], x[None, s], mean[None, s], rstd[None, s], w, 0.0, x.dtype,
                                                    torch.float32, False)[0])
    assert not any(torch.isnan(dx[i:i + part]).any() for i in range(0, R, part))
