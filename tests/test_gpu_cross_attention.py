"""Cross attention, forward and backward, against a plain implementation in float64.

Tolerances, with u half a step of the 16-bit type (bf16 2^-8, fp16 2^-11):
  * a logit is an fp32 sum of D products, so it is off by at most D 2^-24 scale sum|q k| (called
    e), and a weight p by the factor 1 +- (2 e + 2^-20) (its own and its row sum's logit, plus the
    approximate exponential); lse by e + 2^-20 (1 + |lse|);
  * P is rounded to 16 bits for P V: o is off by (u + 2 e + 2^-20) sum p|v| + u |o|; in fp16 a
    weight below 2^-14 of the row's largest is off by 2^-25 of it instead: 2^-25 sum|v|;
  * backward: delta = do . o with the rounded o is off by u sum|do||o|; dS is rounded to 16 bits
    (fp16: 2^-25 at least), so each ds is off by
    d = p u sum|do||o| + u |ds| + 2^-25 [fp16] + (3 e + 2^-18) p (sum|do||v| + sum|do||o|),
    and dq by scale sum_j d |k_j| + u |dq|, dk by scale sum_i d |q_i| + u |dk|; dv by
    sum_i (u p + 2^-25 [fp16] + (3 e + 2^-18) p) |do| + u |dv|.  (3 e: lse comes from a pass that had its own
    e, on top of the weight's.)
An fp16 result below 2^-14 is a multiple of 2^-24, so its rounding is off by up to 2^-25 whatever
its size: every fp16 output has that much on top of u times its value.
"""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ug(gpu_required):
    from diffusion_transformer_ultra_b200 import build
    build.build()
    import diffusion_transformer_ultra_b200 as pkg
    return pkg


def inputs(B, N, S, H, G, D, dtype, seed=0, qscale=1.3):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 + seed)

    def r(*s):
        return torch.randn(s, generator=g, device="cuda")
    q, k, v, do = r(B, N, H, D) * qscale, r(B, S, G, D), r(B, S, G, D), r(B, N, H, D)
    return tuple(t.to(dtype) for t in (q, k, v, do))


def visible(B, S, lens, mask):
    import torch
    keep = torch.ones(B, S, dtype=torch.bool, device="cuda")
    if lens is not None:
        keep &= torch.arange(S, device="cuda")[None] < lens[:, None]
    if mask is not None:
        keep &= mask.bool()
    return keep


def reference(q, k, v, do, lens, mask, scale):
    """float64 outputs, and the tolerances of the module's docstring."""
    import torch
    B, N, H, D = q.shape
    S, G = k.shape[1:3]
    u = torch.finfo(q.dtype).eps / 2
    sub = 2.0 ** -25 if q.dtype == torch.float16 else 0.0
    keep = visible(B, S, lens, mask)[:, None, None, :]
    # hidden keys may hold anything: the definition never reads them
    hide = ~visible(B, S, lens, mask)[:, :, None, None]
    k, v = (t.masked_fill(hide, 0.0) for t in (k, v))
    q, do = (t.double().transpose(1, 2) for t in (q, do))                       # [B, H, N, D]
    k, v = (t.double().transpose(1, 2).repeat_interleave(H // G, 1) for t in (k, v))
    s = (q @ k.mT) * scale
    s = s.masked_fill(~keep, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.where(keep & (lse > -math.inf), torch.exp(s - lse), 0.0)
    o = p @ v
    e = D * 2.0 ** -24 * scale * (q.abs() @ k.abs().mT).masked_fill(~keep, 0.0)
    em = e.amax(-1, keepdim=True) if S else torch.zeros_like(lse)
    po = p @ v.abs()
    # sum|v| over the visible keys alone: the hidden ones were zeroed above
    tol_o = (u + 2 * em + 2.0 ** -20) * po + u * o.abs() + sub + sub * v.abs().sum(-2, keepdim=True) + 1e-9
    tol_lse = (em + 2.0 ** -20 * (1 + lse.abs())).squeeze(-1)
    dp = do @ v.mT
    delta = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    ado = (do.abs() * o.abs()).sum(-1, keepdim=True)
    rel = 3 * em + 2.0 ** -18
    live = keep & (lse > -math.inf)
    d = p * u * ado + u * ds.abs() + sub * live + rel * p * (do.abs() @ v.abs().mT + ado)
    dq, tol_dq = scale * ds @ k, scale * d @ k.abs()
    dk, tol_dk = scale * ds.mT @ q, scale * d.mT @ q.abs()
    dv, tol_dv = p.mT @ do, ((u + rel) * p + sub * live).mT @ do.abs()

    def heads(t):
        return t.view(B, G, H // G, S, D).sum(2)
    dk, tol_dk, dv, tol_dv = map(heads, (dk, tol_dk, dv, tol_dv))
    out = dict(o=(o, tol_o), dq=(dq, tol_dq + u * dq.abs() + sub + 1e-9), dk=(dk, tol_dk + u * dk.abs() + sub + 1e-9),
               dv=(dv, tol_dv + u * dv.abs() + sub + 1e-9))
    out = {n: (a.transpose(1, 2), t.transpose(1, 2)) for n, (a, t) in out.items()}
    out["lse"] = (lse.squeeze(-1), tol_lse)
    return out


def check(name, got, ref, tol):
    import torch
    got = got.double()
    same = (got == ref) | ((got - ref).abs() <= tol)
    bad = int((~same).sum())
    if bad:
        i = (~same).nonzero()[0].tolist()
        raise AssertionError(f"{name}: {bad} of {same.numel()} off, first at {i}: {got[tuple(i)]} for {ref[tuple(i)]}")
    assert not torch.isnan(got).any()


def strided(t, how):
    """A copy of t [B, L, H, D] with another memory layout."""
    import torch
    if how == "heads_first":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if how == "packed":                                       # a slice of a wider projection's output
        B, L, H, D = t.shape
        big = torch.full((B, L, H + 2, D + 8), float("nan"), dtype=t.dtype, device=t.device)
        view = big[:, :, 1:H + 1, 8:]
        view.copy_(t)
        return view
    return t.clone()


def run(ug, B, N, S, H, G, D, dtype, lens=None, mask=None, backward=True, layout="plain", scale=None, qscale=1.3,
        poison=True, seed=0):
    import torch
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    q, k, v, do = inputs(B, N, S, H, G, D, dt, seed, qscale)
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if mask is not None:
        mask = mask(B, S).cuda()
    if poison:                                                # what is hidden may hold anything
        hide = ~visible(B, S, lens, mask)
        k[hide], v[hide] = float("nan"), float("inf")
    q, k, v, do = (strided(t, layout) for t in (q, k, v, do))
    sc = D ** -0.5 if scale is None else scale
    ref = reference(q, k, v, do, lens, mask, sc)
    o = strided(torch.full_like(q, float("nan")), layout)
    lse = torch.full((B, H, N), float("nan"), device="cuda")
    ug.cross_attention(q, k, v, o, kv_lens=lens, key_mask=mask, scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert ug.operator_status() == 0
    check("o", o, *ref["o"])
    check("lse", lse, *ref["lse"])
    if not backward:
        return o
    dq, dk, dv = (strided(torch.full_like(t, float("nan")), layout) for t in (q, k, v))
    ug.cross_attention_backward(do, q, k, v, o, lse, dq, dk, dv, kv_lens=lens, key_mask=mask, scale=scale)
    torch.cuda.synchronize()
    assert ug.operator_status() == 0
    check("dv", dv, *ref["dv"])
    check("dk", dk, *ref["dk"])
    check("dq", dq, *ref["dq"])
    hide = ~visible(B, S, lens, mask)
    assert (dk[hide] == 0).all() and (dv[hide] == 0).all()
    return o, dq, dk, dv


# batch, queries, states, heads, kv heads, head dim
SHAPES = [
    (1, 1, 1, 1, 1, 64), (2, 1, 2, 2, 1, 128), (1, 7, 129, 3, 3, 64), (2, 128, 128, 2, 2, 128),
    (1, 257, 77, 2, 2, 128), (3, 130, 513, 6, 2, 64), (1, 500, 300, 5, 1, 128), (1, 43, 40, 7, 1, 64),
    (2, 1, 2000, 8, 2, 128), (1, 3, 4099, 4, 1, 64), (1, 2000, 1, 2, 2, 64), (1, 300, 200, 128, 1, 64),
    (2, 1500, 260, 24, 24, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_every_key_visible(ug, shape, dtype):
    run(ug, *shape, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape,lens", [
    ((4, 130, 200, 4, 2, 128), [200, 0, 1, 129]), ((3, 1, 700, 8, 1, 64), [1, 700, 0]),
    ((2, 64, 64, 2, 2, 64), [0, 0]), ((2, 300, 256, 3, 1, 128), [128, 127]), ((2, 9, 50, 2, 2, 128), [-3, 99]),
    ((2, 40, 300, 2, 2, 128), [1, 1])])
def test_lengths(ug, shape, lens, dtype):
    run(ug, *shape, dtype, lens=lens)


MASKS = {
    "none": lambda B, S: _zeros(B, S), "scattered": lambda B, S: _scatter(B, S),
    "last": lambda B, S: _only(B, S, S - 1), "late": lambda B, S: _late(B, S),
}


def _zeros(B, S):
    import torch
    return torch.zeros(B, S, dtype=torch.bool)


def _scatter(B, S):
    import torch
    return (torch.arange(S)[None] * 7 + torch.arange(B)[:, None]) % 3 != 0


def _only(B, S, j):
    m = _zeros(B, S)
    m[:, j] = True
    return m


def _late(B, S):
    """Nothing visible in the first tiles (a left-padded prompt)."""
    m = _zeros(B, S)
    m[:, S * 3 // 4:] = True
    m[-1] = False
    return m


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("which", list(MASKS))
@pytest.mark.parametrize("shape", [(2, 140, 300, 4, 2, 128), (2, 2, 1030, 6, 2, 64), (3, 65, 5, 2, 2, 64)])
def test_masks(ug, shape, which, dtype):
    run(ug, *shape, dtype, mask=MASKS[which])


def test_mask_of_bytes_and_lengths_together(ug):
    run(ug, 3, 70, 400, 4, 4, 64, "bf16", lens=[390, 130, 0], mask=lambda B, S: _scatter(B, S).byte() * 5)


@pytest.mark.parametrize("layout", ["heads_first", "packed"])
@pytest.mark.parametrize("shape", [(2, 150, 140, 4, 2, 128), (2, 3, 600, 3, 1, 64)])
def test_strides(ug, shape, layout):
    run(ug, *shape, "bf16", lens=[shape[2], shape[2] // 2], layout=layout)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_peaked_logits_whose_maximum_rises_along_the_keys(ug, dtype):
    """Logits up to some hundreds: the running maximum grows by far more than its slack."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    B, N, S, H, D = 1, 200, 640, 2, 64
    q, k, v, do = inputs(B, N, S, H, H, D, dt, 5)
    k = (k * torch.linspace(0.2, 8, S, device="cuda")[None, :, None, None]).to(dt)
    ref = reference(q, k, v, do, None, None, 0.5)
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    ug.cross_attention(q, k, v, o, scale=0.5, lse=lse)
    check("o", o, *ref["o"])
    check("lse", lse, *ref["lse"])


def test_without_lse_and_on_a_side_stream(ug):
    import torch
    q, k, v, _ = inputs(2, 100, 90, 2, 2, 64, torch.bfloat16)
    want = torch.empty_like(q)
    ug.cross_attention(q, k, v, want)
    torch.cuda.synchronize()
    got = torch.empty_like(q)
    s = torch.cuda.Stream()
    ug.cross_attention(q, k, v, got, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("shape", [(4, 3000, 300, 24, 24, 64), (2, 300, 700, 4, 2, 128), (1, 500, 300, 5, 1, 128), (2, 1, 2000, 8, 2, 128)])
def test_output_in_place_of_the_queries(ug, shape):
    """o may be q: one and two query tiles to an item, split keys, heads that share keys."""
    import torch
    q, k, v, _ = inputs(*shape, torch.bfloat16)
    want = torch.empty_like(q)
    ug.cross_attention(q, k, v, want)
    ug.cross_attention(q, k, v, q)
    assert torch.equal(q, want)


def test_empty_sequences(ug):
    import torch
    q, k, v, do = inputs(2, 5, 0, 4, 2, 64, torch.bfloat16)
    o, lse = torch.full_like(q, float("nan")), torch.zeros(2, 4, 5, device="cuda")
    ug.cross_attention(q, k, v, o, lse=lse)
    assert (o == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = torch.full_like(q, float("nan")), torch.empty_like(k), torch.empty_like(v)
    ug.cross_attention_backward(do, q, k, v, o, lse, dq, dk, dv)
    assert (dq == 0).all()
    q, k, v, do = inputs(2, 0, 70, 4, 2, 64, torch.bfloat16)
    o, lse = torch.empty_like(q), torch.zeros(2, 4, 0, device="cuda")
    ug.cross_attention(q, k, v, o, lse=lse)
    dq, dk, dv = torch.empty_like(q), torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    ug.cross_attention_backward(do, q, k, v, o, lse, dq, dk, dv)
    assert (dk == 0).all() and (dv == 0).all()


def test_one_visible_key_has_no_gradient_of_the_logits(ug):
    """Its weight is one whatever the logit: dq and dk are exactly zero."""
    for lens, mask in (([1, 1], None), (None, lambda B, S: _only(B, S, 150))):
        _, dq, dk, _ = run(ug, 2, 140, 200, 4, 2, 64, "bf16", lens=lens, mask=mask)
        assert (dq == 0).all() and (dk == 0).all()


def test_same_bits_every_time_and_from_a_graph(ug):
    import torch
    q, k, v, do = inputs(2, 300, 700, 4, 2, 128, torch.bfloat16)
    lens = torch.tensor([700, 333], dtype=torch.int32, device="cuda")
    mask = _scatter(2, 700).cuda()

    def once(out):
        o, lse, dq, dk, dv = out
        ug.cross_attention(q, k, v, o, kv_lens=lens, key_mask=mask, lse=lse)
        ug.cross_attention_backward(do, q, k, v, o, lse, dq, dk, dv, kv_lens=lens, key_mask=mask)

    def buffers():
        return (torch.empty_like(q), torch.empty(2, 4, 300, device="cuda"), torch.empty_like(q), torch.empty_like(k),
                torch.empty_like(v))
    first, second = buffers(), buffers()
    once(first)
    once(second)
    torch.cuda.synchronize()
    assert ug.operator_status() == 0
    assert [int((a != b).sum()) for a, b in zip(first, second)] == [0] * 5
    # two graphs from the same inputs, replayed in turn, then with other inputs in the same memory
    outs, graphs = [buffers(), buffers()], []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            once(out)
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out in outs for a, b in zip(first, out))
    q.mul_(0.5)
    lens.copy_(torch.tensor([5, 700], dtype=torch.int32))
    graphs[0].replay()
    once(second)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(second, outs[0]))


def test_gradients_against_differences(ug):
    """Central differences of the float64 loss along a random direction, against the kernel's
    gradients projected on it: off by at most the element tolerances' projection."""
    import torch
    q, k, v, do = inputs(1, 40, 60, 4, 2, 64, torch.float16, 9)
    scale = 64 ** -0.5
    ref = reference(q, k, v, do, None, None, scale)
    o, lse = torch.empty_like(q), torch.empty(1, 4, 40, device="cuda")
    ug.cross_attention(q, k, v, o, lse=lse)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    ug.cross_attention_backward(do, q, k, v, o, lse, *grads)

    def loss(q, k, v):
        qq, kk, vv = (t.transpose(1, 2) for t in (q, k, v))
        kk, vv = (t.repeat_interleave(2, 1) for t in (kk, vv))
        p = torch.softmax(scale * qq @ kk.mT, -1)
        return ((p @ vv).transpose(1, 2) * do.double()).sum()
    for i, name in enumerate(("dq", "dk", "dv")):
        g = torch.Generator(device="cuda")
        g.manual_seed(i)
        args = [t.double() for t in (q, k, v)]
        d = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        slope = (loss(*up) - loss(*down)) / (2 * h)
        got = (grads[i].double() * d).sum()
        assert abs(got - slope) <= (ref[name][1] * d.abs()).sum() + 1e-6 * slope.abs()


def test_long_states_past_32_bit_offsets(ug):
    """Strides that put the last sample's states behind 2^31 elements."""
    import torch
    B, N, S, G, D = 3, 20, 130, 1, 64
    far = 2 ** 30 + 64                                         # elements between samples
    big = torch.empty(2 * far + S * G * D, dtype=torch.bfloat16, device="cuda")
    q, k, v, do = inputs(B, N, S, 2, G, D, torch.bfloat16)
    kf = big.as_strided((B, S, G, D), (far, D, D, 1))
    kf.copy_(k)
    ref = reference(q, k, v, do, None, None, D ** -0.5)
    o, lse = torch.empty_like(q), torch.empty(B, 2, N, device="cuda")
    ug.cross_attention(q, kf, v, o, lse=lse)
    check("o", o, *ref["o"])
    dq, dk, dv = torch.empty_like(q), kf, torch.empty_like(v)
    dkf = torch.empty_like(big).as_strided((B, S, G, D), (far, D, D, 1))
    ug.cross_attention_backward(do, q, kf, v, o, lse, dq, dkf, dv)
    check("dq", dq, *ref["dq"])
    check("dk", dkf, *ref["dk"])
    check("dv", dv, *ref["dv"])


# More work items than multiprocessors in every kernel, so that blocks go from item to item (accumulators,
# barriers and constants handed over), as a layer's sizes have it.  At 148 multiprocessors: two query tiles
# to an item, the last with one; heads that share keys (42 queries to a tile); all keys in one tile; two
# samples' key tiles to a block; split keys (4 parts) and split queries (4 parts) with several items a block.
LAYERS = [(4, 600, 300, 24, 24, 128), (4, 600, 300, 24, 24, 64), (4, 700, 260, 24, 8, 128), (3, 1100, 520, 16, 4, 64),
          (4, 1300, 77, 24, 24, 128), (8, 130, 1000, 16, 16, 128), (10, 20, 4096, 15, 15, 64), (10, 20, 4096, 15, 15, 128),
          (10, 4096, 100, 15, 15, 128), (10, 4096, 100, 15, 15, 64)]


def prompts(B, S):
    """Lengths of padded prompts, an empty one and one of a single state among them."""
    return [(S, 0, 1, S // 2 + 1, S - 1)[i % 5] for i in range(B)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hidden", ["nothing", "lengths", "scattered", "late and lengths"])
@pytest.mark.parametrize("shape", LAYERS)
def test_several_items_to_a_block(ug, shape, hidden, dtype):
    lens = prompts(shape[0], shape[2]) if "lengths" in hidden else None
    mask = {"scattered": _scatter, "late and lengths": _late}.get(hidden)
    run(ug, *shape, dtype, lens=lens, mask=mask)


@pytest.mark.parametrize("shape", LAYERS)
def test_same_bits_with_several_items_to_a_block(ug, shape):
    """Ten runs beside other work of unequal length, which shifts the blocks' timing."""
    import torch
    B, N, S, H, G, D = shape
    q, k, v, do = inputs(*shape, torch.bfloat16)
    lens = torch.tensor(prompts(B, S), dtype=torch.int32, device="cuda")
    side, noise = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    first = None
    for i in range(10):
        o, lse = torch.full_like(q, float("nan")), torch.full((B, H, N), float("nan"), device="cuda")
        dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, k, v))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(i):
                noise = (noise @ noise).tanh()
        ug.cross_attention(q, k, v, o, kv_lens=lens, lse=lse)
        ug.cross_attention_backward(do, q, k, v, o, lse, dq, dk, dv, kv_lens=lens)
        torch.cuda.synchronize()
        assert ug.operator_status() == 0
        got = (o, lse, dq, dk, dv)
        first = first or got
        assert [int((a != b).sum()) for a, b in zip(first, got)] == [0] * 5


@pytest.mark.parametrize("D", [64, 128])
def test_broadcast_inputs(ug, D):
    """Strides of zero: one prompt for all samples, one key/value head for all, one do for all queries; the
    gradients come for each of them."""
    import torch
    B, N, S, H, dt = 3, 150, 140, 4, torch.bfloat16
    q, k, v, do = inputs(B, N, S, H, H, D, dt)
    for kk, vv, dd in ((k[:1].expand_as(k), v[:1].expand_as(v), do), (k[:, :, :1].expand_as(k), v, do[:, :1].expand_as(do)),
                       (k, v[:1, :, :1].expand_as(v), do[:1, :1, :1].expand_as(do))):
        ref = reference(q, kk, vv, dd, None, None, D ** -0.5)
        o, lse = torch.full_like(q, float("nan")), torch.full((B, H, N), float("nan"), device="cuda")
        ug.cross_attention(q, kk, vv, o, lse=lse)
        check("o", o, *ref["o"])
        check("lse", lse, *ref["lse"])
        dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, k, v))
        ug.cross_attention_backward(dd, q, kk, vv, o, lse, dq, dk, dv)
        check("dv", dv, *ref["dv"])
        check("dk", dk, *ref["dk"])
        check("dq", dq, *ref["dq"])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [512.0, 2.0 ** -10])
def test_scaled_losses(ug, size, dtype):
    """do of another size, as a scaled loss or a mean over many tokens gives it."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    B, N, S, H, G, D = 2, 300, 260, 4, 2, 128
    q, k, v, do = inputs(B, N, S, H, G, D, dt)
    do = (do.float() * size).to(dt)
    ref = reference(q, k, v, do, None, None, D ** -0.5)
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    ug.cross_attention(q, k, v, o, lse=lse)
    dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, k, v))
    ug.cross_attention_backward(do, q, k, v, o, lse, dq, dk, dv)
    check("dv", dv, *ref["dv"])
    check("dk", dk, *ref["dk"])
    check("dq", dq, *ref["dq"])


def test_both_passes_on_two_streams_at_once(ug):
    import torch
    sets = []
    for seed in range(2):
        q, k, v, do = inputs(3, 500, 400, 8, 4, 128, torch.bfloat16, seed)
        lens, mask = torch.tensor([400, 77, 0], dtype=torch.int32, device="cuda"), _scatter(3, 400).cuda()

        def once(out, a=(q, k, v, do, lens, mask), stream=None):
            q, k, v, do, lens, mask = a
            ug.cross_attention(q, k, v, out[0], kv_lens=lens, key_mask=mask, lse=out[1], stream=stream)
            ug.cross_attention_backward(do, q, k, v, out[0], out[1], *out[2:], kv_lens=lens, key_mask=mask, stream=stream)
        outs = [(torch.empty_like(q), torch.empty(3, 8, 500, device="cuda"), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
                for _ in range(9)]
        once(outs[0])
        sets.append((once, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(1, 9):
        for once, outs, stream in sets:
            once(outs[i], stream=stream)
    torch.cuda.synchronize()
    assert ug.operator_status() == 0
    assert all(torch.equal(a, b) for _, outs, _ in sets for out in outs[1:] for a, b in zip(outs[0], out))


def test_more_samples_than_a_grid_dimension_holds(ug):
    run(ug, 70000, 2, 130, 1, 1, 64, "bf16", poison=False)
