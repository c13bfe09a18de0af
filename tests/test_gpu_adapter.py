"""The projection with low-rank adapters against a plain implementation in float64.

Tolerances, with u half a step of the output type (bf16 2^-8, fp16 2^-11, fp32 2^-24) and sub 2^-25
for fp16 (half its smallest step):
  * the sums over k, and over the rank twice (high and low parts), run in fp32; a tensor core may cut
    off instead of rounding, so each of the K + 2 R + 2 additions is off by at most 2^-23 of the sum of
    absolute products;
  * t = scale A x is held as two 16-bit numbers: off by 2^-16 |t| at most (bf16; fp16 less) + sub;
  * y is rounded once: u |y| + sub.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ug(gpu_required):
    from diffusion_transformer_ultra_b200 import build
    build.build()
    import diffusion_transformer_ultra_b200 as pkg
    return pkg


def dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def make(M, K, N, R, A, dtype, ids="mixed", bias=True, seed=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(100 + seed)
    t = dt(dtype)

    def r(*s, f=1.0):
        return (torch.randn(s, generator=g, device="cuda") * f).to(t)
    rows = torch.arange(M, device="cuda")
    kinds = {
        "mixed": (rows * 7 + 3) % (A + 2) - 1,                 # -1 and A: no adapter
        "none": rows * 0 - 1,
        "runs": rows * A // max(M, 1),
        "late": torch.where(rows >= M - M // 5 - 1, rows % A, -1),
        "one": rows * 0 + A - 1,
    }
    return dict(x=r(M, K), w=r(N, K, f=K ** -0.5), a=r(A, R, K, f=K ** -0.5), b=r(A, N, R, f=0.5 * R ** -0.5),
                ids=kinds[ids].to(torch.int32), scales=0.5 + torch.rand(A, generator=g, device="cuda"),
                bias=r(N, f=0.1) if bias else None)


def reference(s, scales=True):
    import torch
    x, w, a, b = (s[k].double() for k in ("x", "w", "a", "b"))
    u = torch.finfo(s["x"].dtype).eps / 2
    sub = 2.0 ** -25 if s["x"].dtype == torch.float16 else 0.0
    K, (A, R) = x.shape[1], a.shape[:2]
    y, mag = x @ w.T, x.abs() @ w.abs().T
    low = torch.zeros_like(y)
    if s["bias"] is not None:
        y = y + s["bias"].double()
        mag = mag + s["bias"].double().abs()
    for i in range(A):
        m = (s["ids"] == i).nonzero().squeeze(1)
        f = s["scales"][i].double() if scales else 1.0
        t = f * (x[m] @ a[i].T)
        y[m] += t @ b[i].T
        mag[m] += f * (x[m].abs() @ a[i].abs().T) @ b[i].abs().T
        low[m] += (2.0 ** -16 * t.abs() + sub) @ b[i].abs().T
    return y, u * y.abs() + sub + low + (K + 2 * R + 2) * 2.0 ** -23 * mag


def check(got, ref, tol):
    import torch
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i]} for {ref[i]} +- {tol[i]}")
    assert torch.isfinite(got).all()


def run(ug, s, **kw):
    import torch
    y = torch.full((s["x"].shape[0], s["w"].shape[0]), float("nan"), dtype=s["x"].dtype, device="cuda")
    ug.adapter_project(s["x"], s["w"], y, s["a"], s["b"], s["ids"], scales=s["scales"], bias=s["bias"], **kw)
    torch.cuda.synchronize()
    assert ug.operator_status() == 0
    return y


# rows, k, n, rank, adapters: one row to several tiles, odd widths, ranks that fill no granule
SHAPES = [
    (1, 64, 64, 16, 1), (1, 8, 1, 1, 1), (8, 2048, 640, 16, 8), (9, 136, 77, 4, 3), (16, 520, 130, 8, 5), (31, 256, 333, 64, 2),
    (32, 72, 100, 24, 40), (33, 64, 64, 16, 2), (100, 264, 65, 12, 7), (257, 512, 513, 16, 3), (300, 88, 1000, 64, 8),
    (1000, 1536, 384, 32, 4), (513, 40, 256, 128, 9), (2500, 192, 2050, 16, 2), (700, 64, 8, 20, 300),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_sizes(ug, shape, dtype):
    s = make(*shape, dtype)
    check(run(ug, s), *reference(s))


@pytest.mark.parametrize("ids", ["none", "runs", "late", "one"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("shape", [(12, 256, 96, 16, 4), (900, 320, 520, 16, 4), (3000, 128, 250, 64, 3)])
def test_which_rows_have_adapters(ug, shape, ids, bias):
    s = make(*shape, "bf16", ids=ids, bias=bias)
    check(run(ug, s), *reference(s))


@pytest.mark.parametrize("shape", [(1, 5, 3, 2, 1), (70, 100, 130, 7, 3), (130, 64, 64, 16, 2)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_general_kernel(ug, shape, dtype):
    """fp32, and k that 16-byte accesses cannot read."""
    M, K, N, R, A = shape
    s = make(M, K if dtype == "fp32" else K - K % 8 + 3, N, R, A, dtype)
    check(run(ug, s), *reference(s))


@pytest.mark.parametrize("M", [20, 400])
@pytest.mark.parametrize("gap", [8, 3])
def test_strided_rows(ug, M, gap):
    """Rows apart, of x (aligned or not) and of y; what lies between y's rows stays."""
    import torch
    s = make(M, 128, 136, 16, 3, "bf16")
    xs = torch.full((M, 128 + gap), float("nan"), dtype=torch.bfloat16, device="cuda")
    xs[:, :128] = s["x"]
    s["x"] = xs[:, :128]
    ys = torch.full((M + 1, 136 + gap), 7.0, dtype=torch.bfloat16, device="cuda")
    ug.adapter_project(s["x"], s["w"], ys[:M, :136], s["a"], s["b"], s["ids"], scales=s["scales"], bias=s["bias"])
    check(ys[:M, :136], *reference(s))
    assert (ys[:, 136:] == 7).all() and (ys[M] == 7).all()


def test_without_scales_and_on_a_side_stream(ug):
    import torch
    s = make(300, 256, 264, 16, 3, "fp16")
    s["scales"] = None
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = run(ug, s, stream=st)
    check(y, *reference(s, scales=False))


def test_no_rows(ug):
    s = make(0, 64, 64, 16, 2, "bf16")
    assert run(ug, s).shape == (0, 64)


@pytest.mark.parametrize("M", [24, 600])
def test_an_adapter_of_infinities_and_nan_stays_with_its_rows(ug, M):
    import torch
    s = make(M, 192, 200, 16, 3, "bf16")
    ref, tol = reference(s)
    s["b"][1, 5, 3] = float("inf")
    s["b"][1, 70:90] = float("nan")
    s["b"][1, 199, 15] = float("-inf")
    s["a"][0, 2] = float("nan")                                # reaches every column of its rows
    y = run(ug, s)
    own, sick = s["ids"] == 1, s["ids"] == 0
    cols = torch.zeros(200, dtype=torch.bool, device="cuda")
    cols[5] = cols[199] = True
    cols[70:90] = True
    hit = own[:, None] & cols[None]
    assert not torch.isfinite(y[hit]).any()
    assert torch.isnan(y[sick]).all()
    rest = ~hit & ~sick[:, None]
    assert ((y.double() - ref).abs() <= tol)[rest].all()


@pytest.mark.parametrize("M", [7, 900])
def test_same_bits_every_time_and_from_graphs(ug, M):
    import torch
    s = make(M, 512, 384, 16, 4, "bf16")
    first = run(ug, s)
    assert torch.equal(first, run(ug, s))
    outs, graphs = [torch.zeros_like(first) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ug.adapter_project(s["x"], s["w"], o, s["a"], s["b"], s["ids"], scales=s["scales"], bias=s["bias"])
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    s["x"].mul_(2)
    s["ids"].copy_(s["ids"].flip(0))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = run(ug, s)
    assert all(torch.equal(want, o) for o in outs)


def test_two_streams_at_once(ug):
    import torch
    ss = [make(700, 256, 300, 16, 3, "bf16", seed=i) for i in range(2)]
    want = [run(ug, s) for s in ss]
    streams = [torch.cuda.Stream() for _ in ss]
    got = [[torch.empty_like(w) for _ in range(8)] for w in want]
    torch.cuda.synchronize()
    for i in range(8):
        for k, s in enumerate(ss):
            ug.adapter_project(s["x"], s["w"], got[k][i], s["a"], s["b"], s["ids"], scales=s["scales"], bias=s["bias"],
                               stream=streams[k])
    torch.cuda.synchronize()
    assert all(torch.equal(w, o) for w, os in zip(want, got) for o in os)


def test_rows_past_32_bit_offsets(ug):
    """Row strides that put the last rows of x and y behind 2^31 elements."""
    import torch
    M, far = 300, 2 ** 31 // 256
    s = make(M, 64, 64, 16, 2, "bf16")
    big = torch.empty(M * far, dtype=torch.bfloat16, device="cuda")
    xf, yf = big.as_strided((M, 64), (far, 1)), big.as_strided((M, 64), (far, 1), 1024)
    xf.copy_(s["x"])
    ref = reference(s)
    s["x"] = xf
    ug.adapter_project(xf, s["w"], yf, s["a"], s["b"], s["ids"], scales=s["scales"], bias=s["bias"])
    check(yf, *ref)


@pytest.mark.parametrize("M", [24, 600])
@pytest.mark.parametrize("tsize,bsize", [(2.0 ** -18, 1024.0), (2.0 ** -10, 64.0), (2.0 ** 9, 2.0 ** -13), (2.0 ** -4, 1.0)])
def test_fp16_products_of_unequal_sizes(ug, M, tsize, bsize):
    """s A x far below B, where a 16-bit low part alone would end at fp16's smallest step, and far above it.
    The adapter's terms alone (W = 0): each t b is off by what the header states, 2^-22 |t b| + 2^-36 |b| +
    min(2^-26 |t|, 2^-12 |t b|); the fp32 sums that make t by K 2^-23 of their absolute products, those over
    the rank by (2 R + K) 2^-23; y is rounded once."""
    import torch
    K, N, R, A = 64, 136, 16, 2
    s = make(M, K, N, R, A, "fp16", bias=False)
    s["w"].zero_()
    s["x"] = (s["x"].float() * tsize ** 0.5).half()
    s["a"] = (s["a"].float() * tsize ** 0.5).half()
    s["b"] = (s["b"].float() * bsize / (0.5 * R ** -0.5)).half()
    y = run(ug, s)
    x, a, b = (s[k].double() for k in ("x", "a", "b"))
    want, tol = torch.zeros(M, N, dtype=torch.float64, device="cuda"), torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for i in range(A):
        m = (s["ids"] == i).nonzero().squeeze(1)
        f = s["scales"][i].double()
        t, mag = f * (x[m] @ a[i].T), f * (x[m].abs() @ a[i].abs().T)
        want[m] = t @ b[i].T
        tb = t.abs()[:, None] * b[i].abs()[None]               # [rows, N, R]
        off = 2.0 ** -22 * tb + 2.0 ** -36 * b[i].abs() + torch.minimum(2.0 ** -26 * t.abs()[:, None], 2.0 ** -12 * tb)
        tol[m] = off.sum(-1) + (2 * K + 2 * R) * 2.0 ** -23 * (mag @ b[i].abs().T)
    check(y, want, tol + 2.0 ** -11 * want.abs() + 2.0 ** -25)


# Tiles of 256 columns, several to a pair of blocks, as a layer's projections take them (74 pairs), and
# several of 128; rows and columns that end inside a tile.
LAYERS = [(9728, 136, 4608, 16, 5), (9700, 64, 4600, 32, 2), (4864, 1536, 1536, 16, 2), (20000, 72, 1001, 24, 3), (5000, 320, 2048, 64, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ids", ["mixed", "late", "runs"])
@pytest.mark.parametrize("shape", LAYERS)
def test_layers(ug, shape, ids, dtype):
    s = make(*shape, dtype, ids=ids, bias=ids != "runs")
    check(run(ug, s), *reference(s))


@pytest.mark.parametrize("shape", LAYERS[:2])
def test_infinities_and_nan_of_an_adapter_in_a_layer(ug, shape):
    """As above with few tiles, here with the flags of tiles that follow one another in a block."""
    import torch
    M, _, N, R, A = shape
    s = make(*shape, "bf16")
    s["ids"][M // 3:M // 2] = 0                                # tiles without the sick adapter between tiles with it
    ref, tol = reference(s)
    s["b"][1, 5, 3] = float("inf")
    s["b"][1, N // 2:N // 2 + 40] = float("nan")
    s["b"][1, N - 1, R - 1] = float("-inf")
    y = run(ug, s)
    cols = torch.zeros(N, dtype=torch.bool, device="cuda")
    cols[5] = cols[N - 1] = True
    cols[N // 2:N // 2 + 40] = True
    hit = (s["ids"] == 1)[:, None] & cols[None]
    assert not torch.isfinite(y[hit]).any()
    assert ((y.double() - ref).abs() <= tol)[~hit].all()


def test_same_bits_in_a_layer(ug):
    import torch
    s = make(*LAYERS[0], "bf16")
    first = run(ug, s)
    side, noise = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    for i in range(10):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(i):
                noise = (noise @ noise).tanh()
        assert torch.equal(first, run(ug, s))


@pytest.mark.parametrize("M", [20, 400])
def test_one_row_for_all(ug, M):
    """x of stride zero: the same row for every adapter."""
    s = make(M, 128, 136, 16, 3, "bf16")
    s["x"] = s["x"][:1].expand(M, 128)
    check(run(ug, s), *reference(s))


@pytest.mark.parametrize("M", [7, 8, 9, 16, 17, 32, 33, 64, 65, 255, 256, 513])
def test_row_counts_at_the_kernels_borders(ug, M):
    s = make(M, 520, 300, 16, 8, "bf16")
    check(run(ug, s), *reference(s))


@pytest.mark.parametrize("M", [577, 1000, 2000])
@pytest.mark.parametrize("R", [16, 64])
def test_several_adapters_in_some_hundreds_of_rows(ug, M, R):
    s = make(M, 512, 520, R, 8, "fp16")
    check(run(ug, s), *reference(s))
