"""Norm, adapter projection, joint attention and cross attention together, each step against float64 on
the buffers the step before left, with the tolerances of the operators' own tests; and the binding's
refusals of mismatched tensors."""
import dataclasses

import pytest

from helpers import check_attention, geometry
from oracle import hla_oracle as O

import test_gpu_adapter as ta
import test_gpu_cross_attention as tc
import test_gpu_layer_norm as tn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ug(gpu_required):
    from diffusion_transformer_ultra_b200 import build
    build.build()
    import diffusion_transformer_ultra_b200 as pkg
    return pkg


def make(ug, C=192, R=8, adapters=2, ns=100):
    import torch
    wl = dataclasses.replace(ug.WORKLOADS["1k"], name="small", H=16, W=16, l=8, b=2, rho=4, T=20, heads=2, D=64, axes=(16, 24, 24),
                             batch=2)
    plan = ug.plan_for(wl)
    N, HD = plan.info["N_raster"], wl.heads * wl.D
    g = torch.Generator(device="cuda")
    g.manual_seed(11)

    def r(*s, f=1.0):
        return (torch.randn(s, generator=g, device="cuda") * f).bfloat16()
    rows = torch.arange(wl.batch * N, device="cuda")
    low = rows % N >= N - 16                                   # adapters on the low-resolution tokens
    s = dict(x=r(wl.batch, N, C), w=[r(HD, C, f=C ** -0.5) for _ in range(4)], a=[r(adapters, R, C, f=C ** -0.5) for _ in range(4)],
             b=[r(adapters, HD, R, f=0.3) for _ in range(4)], ids=torch.where(low, rows // N, -1).to(torch.int32),
             scales=torch.tensor([0.7, 1.3], device="cuda"), weight=r(wl.batch, C, f=0.2), shift=r(wl.batch, C, f=0.2),
             k=r(wl.batch, ns, wl.heads, wl.D), v=r(wl.batch, ns, wl.heads, wl.D),
             lens=torch.tensor([ns, 37], dtype=torch.int32, device="cuda"))
    return wl, plan, s


def run(ug, pl, s, o, xo, stream=None):
    pl(s["x"], o, s["w"][:3], s["a"][:3], s["b"][:3], s["ids"], s["scales"], weight=s["weight"], shift=s["shift"], stream=stream)
    pl.cross(xo, s["w"][3], s["a"][3], s["b"][3], s["ids"], s["k"], s["v"], s["scales"], kv_lens=s["lens"], stream=stream)


def test_every_step(ug):
    import torch
    wl, plan, s = make(ug)
    pl = ug.ProjectedLayer(plan, wl.batch, s["x"].shape[-1])
    o, xo = torch.empty(pl.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(pl.shape, dtype=torch.bfloat16, device="cuda")
    run(ug, pl, s, o, xo)
    torch.cuda.synchronize()
    assert plan.sync_status() == 0 and ug.operator_status() == 0
    tn.check("norm", pl.norm, tn.forward_reference(s["x"], s["weight"], s["shift"], 1.0, 1e-6, torch.bfloat16)[0])
    B, N, H, D = pl.shape
    for i, out in enumerate((pl.q, pl.k, pl.v, pl.xq)):
        ta.check(out.view(B * N, H * D), *ta.reference(dict(x=pl.norm.view(B * N, -1), w=s["w"][i], a=s["a"][i], b=s["b"][i],
                                                            ids=s["ids"], scales=s["scales"], bias=None)))
    g = geometry(wl)
    # check_attention's absolute bound is stated for values of unit size; output and error are linear in V,
    # so both are taken relative to the largest token's root mean square.
    size = float(pl.v.double().square().mean(-1).sqrt().max())
    for h in range(H):
        ref, _ = O.forward(*(t[:, :, h:h + 1].cpu().double().numpy() for t in (pl.q, pl.k, pl.v)), g, wl.axes)
        check_attention(o[:, :, h:h + 1].cpu().double().numpy() / size, O.unpermute(ref, g) / size, f"head {h}")
    ref = tc.reference(pl.xq, s["k"], s["v"], torch.zeros_like(pl.xq), s["lens"], None, D ** -0.5)
    tc.check("cross", xo, *ref["o"])


def test_the_same_from_a_graph_and_a_side_stream(ug):
    import torch
    wl, plan, s = make(ug)
    pl = ug.ProjectedLayer(plan, wl.batch, s["x"].shape[-1])
    outs = [[torch.empty(pl.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(3)]
    run(ug, pl, s, *outs[0])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    run(ug, pl, s, *outs[1], stream=st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        run(ug, pl, s, *outs[2])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out in outs[1:] for a, b in zip(outs[0], out))
    del g


def test_refusals(ug):
    import torch
    f = dict(device="cuda")
    x, h = torch.zeros(4, 64, **f), torch.zeros(4, 64, dtype=torch.bfloat16, **f)
    st = torch.zeros(4, **f)
    i = torch.zeros(4, dtype=torch.int32, **f)
    a, b = torch.zeros(2, 8, 64, dtype=torch.bfloat16, **f), torch.zeros(2, 32, 8, dtype=torch.bfloat16, **f)
    w, y = torch.zeros(32, 64, dtype=torch.bfloat16, **f), torch.zeros(4, 32, dtype=torch.bfloat16, **f)
    q, k = torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16, **f), torch.zeros(1, 5, 2, 64, dtype=torch.bfloat16, **f)
    lse = torch.zeros(1, 4, 3, **f)
    bad = [
        lambda: ug.layer_norm(x, h), lambda: ug.layer_norm(x, x[:3]), lambda: ug.layer_norm(x.t(), x.t()),
        lambda: ug.layer_norm(x, x, weight=torch.zeros(63, **f)), lambda: ug.layer_norm(x, x, weight=torch.zeros(4, 64, **f)),
        lambda: ug.layer_norm(h, h, weight=torch.zeros(64, dtype=torch.float16, **f)), lambda: ug.layer_norm(x, x, mean=st[:3]),
        lambda: ug.layer_norm(x, x[:1].expand(4, 64)), lambda: ug.layer_norm(x, x.cpu()),
        lambda: ug.layer_norm_backward(x, x, st, st, h), lambda: ug.layer_norm_backward(x, x, st, st[:2], x),
        lambda: ug.layer_norm_backward(x, x, st, st, x, dweight=torch.zeros(64, **f), dbias=torch.zeros(63, **f)),
        lambda: ug.adapter_project(h, w, y, a, b, i.long()), lambda: ug.adapter_project(h, w, y, a, b, i[:3]),
        lambda: ug.adapter_project(h, w[:, :60], y, a, b, i), lambda: ug.adapter_project(h, w, y, a, b[:1], i),
        lambda: ug.adapter_project(h, w, y.float(), a, b, i), lambda: ug.adapter_project(h, w, y, a, b, i, scales=st[:1]),
        lambda: ug.cross_attention(q, k, k[:, :4], q.clone()), lambda: ug.cross_attention(q, k[:, :, :1].expand(1, 5, 3, 64), k, q),
        lambda: ug.cross_attention(q, k, k, q.float()), lambda: ug.cross_attention(q, k, k, q.clone(), kv_lens=i),
        lambda: ug.cross_attention(q, k, k, q.clone(), key_mask=torch.ones(1, 4, dtype=torch.bool, **f)),
        lambda: ug.cross_attention(q[..., :32], k[..., :32], k[..., :32], q[..., :32].clone()),
        lambda: ug.cross_attention(q, k, k, q.clone(), lse=lse[:, :3]), lambda: ug.cross_attention(q, k, k, q.clone(), scale=-1.0),
        lambda: ug.cross_attention_backward(q, q, k, k, q, lse, q.clone(), k, k[:, :4]),
    ]
    for n, call in enumerate(bad):
        with pytest.raises((ValueError, ug.UltragenError)):
            call()
            raise AssertionError(f"case {n} was taken")


def test_two_instances_at_once_and_one_behind_an_event(ug):
    """Instances with a plan each overlap on two streams; one instance moves to another stream behind an event."""
    import torch
    sets = []
    for i in range(2):
        wl, plan, s = make(ug)
        if i:
            s["x"] = s["x"].flip(0).contiguous()
        pl = ug.ProjectedLayer(plan, wl.batch, s["x"].shape[-1])
        want = [torch.empty(pl.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        run(ug, pl, s, *want)
        sets.append((pl, s, want, torch.cuda.Stream(), [[torch.zeros_like(w) for w in want] for _ in range(10)]))
    torch.cuda.synchronize()
    assert not torch.equal(sets[0][2][0], sets[1][2][0])
    for k in range(10):
        for pl, s, _, st, outs in sets:
            run(ug, pl, s, *outs[k], stream=st)
    torch.cuda.synchronize()
    for _, _, want, _, outs in sets:
        assert all(torch.equal(a, b) for out in outs for a, b in zip(want, out))
    (pl, s, want, first, outs), second = sets[0], sets[1][3]
    last = torch.cuda.Event()
    for k, st in enumerate((first, second) * 5):
        for o in outs[k]:
            o.zero_()
        st.wait_stream(torch.cuda.current_stream())
        if k:
            st.wait_event(last)
        run(ug, pl, s, *outs[k], stream=st)
        last.record(st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out in outs for a, b in zip(want, out))
