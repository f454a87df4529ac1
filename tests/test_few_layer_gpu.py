"""The few-token layer (moe_forward_few) against a plain 64-bit implementation.

Bounds.  Let G = W_g x, U = W_u x (contraction length d), h = gate * SiLU(G) * U, y = sum of
W_d h over experts and hidden columns (length n = experts * F), and |.|-sums written with
absolute values throughout.  With u = 2^-24 (fp32) and r = eps/2 of the storage type:
  * an fp32 sum of d products is off by at most (d + 2) u sum|w x| in any order, so
    dh <= gate (1.1 |U| (d + 2) u |W_g||x| + |SiLU(G)| (d + 2) u |W_u||x|) (|SiLU'| <= 1.1),
    plus 16 u |h| for exp, the division and the products;
  * a logit is off by dz = (d + 2) u |w_r||x| + u |z|, a gate by a factor of 2 dz + 64 u;
  * the choice of experts is checked against the 64-bit logits up to 2 dz per comparison, and
    everything that follows from it against the 64-bit layer over the chosen experts;
  * H is rounded once: r |h|; y is summed in fp32: (n + 4) u |W_d||h|, and rounded: r |y|.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def N():
    from routing_dispatch_expert_gemm_b200 import build, native
    build.build()
    return native


def make(T, d, E, k, F, dtype="bf16", shared=False, bias=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dtype])

    p = {"x": rn((T, d), 1.0), "w_router": rn((E, d), d ** -0.5),
         "w_gate": rn((E, F, d), 0.05), "w_up": rn((E, F, d), 0.05), "w_down": rn((E, d, F), 0.05),
         "logit_bias": None if bias is None else torch.tensor(bias, device="cuda")}
    for n, s in (("shared_gate", (F, d)), ("shared_up", (F, d)), ("shared_down", (d, F))):
        p[n] = rn(s, 0.05) if shared else None
    return p


def reference(p, out, k, gate_mode, capacity=-1, residual=False, live=None):
    """y, gates and their bounds for the experts in out["ids"], which are checked first."""
    x = p["x"].double()
    T, d = x.shape
    E, F = p["w_gate"].shape[:2]
    live = T if live is None else live
    r = torch.finfo(p["x"].dtype).eps / 2
    z = x @ p["w_router"].double().t()
    dz = (d + 2) * U * (x.abs() @ p["w_router"].double().abs().t()) + U * z.abs()
    if p["logit_bias"] is not None:
        z = z + p["logit_bias"].double()
        dz = dz + U * torch.nan_to_num(z.abs(), posinf=0.0)
    ids = out["ids"].long().clone()
    ids[live:] = torch.arange(k, device="cuda")
    chosen = torch.gather(z, 1, ids)
    slack = 2 * dz.max(1, keepdim=True).values
    assert all(len(set(row)) == k for row in ids.tolist())
    rest = z.scatter(1, ids, -float("inf")).max(1, keepdim=True).values
    following = torch.cat([chosen[:, 1:], rest], 1)
    assert bool((chosen >= following - slack)[:live].all()), "not the top-k"
    top = chosen[:, :1]
    dead = torch.isinf(top)  # every expert masked
    e = torch.exp(chosen - torch.where(dead, 0.0, top))
    over = z if gate_mode == "softmax_topk" else chosen
    den = torch.exp(over - torch.where(dead, 0.0, top)).sum(1, keepdim=True)
    gates = torch.where(dead, torch.zeros_like(e), e / torch.where(dead, 1.0, den))
    rel_gate = 2 * dz.max(1, keepdim=True).values + 64 * U
    y, by = torch.zeros_like(x), torch.zeros_like(x)
    n = (E + 1) * F

    def add(t, g, wg, wu, wd, rel_g):
        wg, wu, wd = wg.double(), wu.double(), wd.double()
        G, V = wg @ x[t], wu @ x[t]
        s = G * torch.sigmoid(G)
        h = g * s * V
        dh = (g * (d + 2) * U * (1.1 * V.abs() * (wg.abs() @ x[t].abs())
                                 + s.abs() * (wu.abs() @ x[t].abs()))
              + (16 * U + rel_g + r) * h.abs())
        y[t] += wd @ h
        by[t] += wd.abs() @ (dh + (n + 4) * U * h.abs())

    count = [0] * E
    for t in range(live):
        for j in range(k):
            ex = int(ids[t, j])
            count[ex] += 1
            if 0 <= capacity < count[ex]:
                continue
            add(t, gates[t, j], p["w_gate"][ex], p["w_up"][ex], p["w_down"][ex],
                float(rel_gate[t]))
        if p["shared_gate"] is not None:
            add(t, 1.0, p["shared_gate"], p["shared_up"], p["shared_down"], 0.0)
        if residual:
            y[t] += x[t]
    by = by * 1.01 + (r + 2 * U) * y.abs() * 1.01 + 1e-30
    return dict(y=y, by=by, gates=gates, bg=rel_gate * gates + 1e-30, demand=count)


def call(N, cfg, p, n_tokens=None, ws=None, y=None):
    T, k, E = cfg.T, cfg.k, cfg.E
    ws = N.workspace(cfg) if ws is None else ws
    y = torch.full_like(p["x"], 7.0) if y is None else y
    out = dict(y=y, ids=torch.full((T, k), -9, dtype=torch.int32, device="cuda"),
               gates=torch.full((T, k), -9.0, device="cuda"),
               demand=torch.full((E,), -9, dtype=torch.int32, device="cuda"),
               offsets=torch.full((E + 2,), -9, dtype=torch.int32, device="cuda"))
    nt = None if n_tokens is None else torch.tensor([n_tokens], dtype=torch.int32, device="cuda")
    N.moe_forward_few(cfg, p["x"], p["w_router"], p["logit_bias"], p["w_gate"], p["w_up"],
                      p["w_down"], p["shared_gate"], p["shared_up"], p["shared_down"], y,
                      out["ids"], out["gates"], out["demand"], out["offsets"], nt, ws)
    assert N.moe_get_device_status(ws) == 0
    return out


def check(out, ref, live):
    gerr = (out["gates"][:live].double() - ref["gates"][:live]).abs()
    assert bool((gerr <= ref["bg"][:live]).all())
    if live:
        worst = ((out["y"][:live].double() - ref["y"][:live]).abs() / ref["by"][:live]).max()
        assert worst <= 1.0, f"error is {float(worst):.2f} of its bound"
    assert bool((out["y"][live:] == 7.0).all()) and bool((out["ids"][live:] == -9).all())
    assert bool((out["gates"][live:] == -9.0).all())


CASES = [
    # T, d, E, k, F, dtype, gate mode, shared, residual, capacity, live
    (1, 128, 4, 2, 128, "bf16", "topk_softmax", False, False, -1, None),
    (1, 1024, 32, 8, 512, "bf16", "topk_softmax", False, True, -1, None),
    (3, 256, 1, 1, 384, "bf16", "softmax_topk", True, False, -1, None),
    (7, 640, 9, 3, 128, "bf16", "softmax_topk_renorm", True, True, -1, 5),
    (8, 128, 5, 5, 896, "bf16", "softmax_topk", False, False, -1, None),
    (9, 384, 40, 8, 256, "bf16", "topk_softmax", False, True, -1, None),
    (16, 1152, 65, 4, 1152, "bf16", "softmax_topk_renorm", True, False, 1, None),
    (17, 512, 7, 2, 640, "bf16", "topk_softmax", True, True, 3, 16),
    (32, 256, 200, 6, 128, "bf16", "softmax_topk", False, False, -1, None),
    (32, 2048, 4, 4, 512, "bf16", "topk_softmax", True, True, -1, 31),
    (32, 4736 + 128, 2, 1, 128, "bf16", "topk_softmax", False, False, -1, None),
    (2, 4, 3, 2, 4, "f32", "topk_softmax", False, False, -1, None),
    (5, 772, 13, 3, 300, "f32", "softmax_topk", True, True, -1, 4),
    (13, 68, 256, 32, 132, "f32", "softmax_topk_renorm", False, True, 2, None),
    (32, 516, 6, 2, 260, "f32", "topk_softmax", True, False, -1, None),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:6]))
def test_against_64_bits(N, case):
    T, d, E, k, F, dtype, mode, shared, residual, cap, live = case
    p = make(T, d, E, k, F, dtype, shared, bias=[0.1 * (i % 7) for i in range(E)], seed=T)
    cfg = N.make_config(T, d, E, k, F, dtype=dtype, gate_mode=mode, capacity=cap,
                        has_shared=shared, add_residual=residual)
    n = T if live is None else live
    out = call(N, cfg, p, live)
    ref = reference(p, out, k, mode, cap, residual, n)
    check(out, ref, n)
    assert out["demand"].tolist() == ref["demand"]
    kept = [c if cap < 0 else min(c, cap) for c in ref["demand"]]
    starts = [sum(kept[:e]) for e in range(E + 1)]
    assert out["offsets"].tolist() == starts + [starts[-1] + (n if shared else 0)]


@pytest.mark.parametrize("live", [0, 1])
def test_padded_batch(N, live):
    p = make(6, 256, 8, 2, 128, shared=True)
    cfg = N.make_config(6, 256, 8, 2, 128, has_shared=True)
    out = call(N, cfg, p, live)
    check(out, reference(p, out, 2, "topk_softmax", live=live), live)
    assert int(out["offsets"][-1]) == live * 3 and int(out["demand"].sum()) == live * 2
    for beyond, same in ((-3, 0), (99, 6)):  # clamped to 0..T
        assert int(call(N, cfg, p, beyond)["offsets"][-1]) == same * 3


@pytest.mark.parametrize("shared,residual", [(False, False), (False, True), (True, True)])
def test_capacity_zero(N, shared, residual):
    p = make(4, 128, 4, 2, 128, shared=shared)
    cfg = N.make_config(4, 128, 4, 2, 128, capacity=0, has_shared=shared, add_residual=residual)
    out = call(N, cfg, p)
    check(out, reference(p, out, 2, "topk_softmax", 0, residual), 4)
    if not shared:
        assert torch.equal(out["y"], p["x"] if residual else torch.zeros_like(p["x"]))


@pytest.mark.parametrize("mode", ["topk_softmax", "softmax_topk", "softmax_topk_renorm"])
def test_masked_experts(N, mode):
    inf = float("inf")
    for bias, alone in (([0.0, -inf, 0.0, -inf, 0.0, 0.0], False),  # two experts closed
                        ([-inf, -inf, 0.3, -inf, -inf, -inf], True),  # fewer than k are open
                        ([-inf] * 6, None)):                          # none is
        p = make(5, 256, 6, 3, 128, bias=bias, shared=True)
        cfg = N.make_config(5, 256, 6, 3, 128, gate_mode=mode, has_shared=True)
        out = call(N, cfg, p)
        ref = reference(p, out, 3, mode)
        assert bool(torch.isfinite(out["y"]).all())
        err = (out["y"].double() - ref["y"]).abs()
        assert bool((err <= ref["by"]).all())
        if alone:
            assert out["ids"].tolist() == [[2, 0, 1]] * 5
            assert bool((out["gates"][:, 1:] == 0).all())
        if alone is None:
            assert out["ids"].tolist() == [[0, 1, 2]] * 5
            assert bool((out["gates"] == 0).all())
        if alone is False:
            assert not bool(((out["ids"] == 1) | (out["ids"] == 3)).any())


def test_ties_and_nan_rank(N):
    """Equal logits go to the lower index; a NaN logit ranks below every number."""
    p = make(2, 128, 6, 3, 128)
    p["w_router"].zero_()
    p["logit_bias"] = torch.tensor([float("nan"), 1.0, 2.0, 2.0, -0.0, 0.0], device="cuda")
    cfg = N.make_config(2, 128, 6, 3, 128)
    assert call(N, cfg, p)["ids"].tolist() == [[2, 3, 1]] * 2
    p["logit_bias"] = torch.tensor([float("nan"), -0.0, 0.0, -0.0, -1.0, -1.0], device="cuda")
    assert call(N, cfg, p)["ids"].tolist() == [[1, 2, 3]] * 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_routing_as_moe_forward(N, dtype):
    p = make(16, 512, 24, 4, 256, dtype, shared=True)
    cfg = N.make_config(16, 512, 24, 4, 256, dtype=dtype, has_shared=True, add_residual=True)
    ws = N.workspace(cfg)
    out = call(N, cfg, p, ws=ws)
    y = torch.empty_like(p["x"])
    ids, gates = torch.empty_like(out["ids"]), torch.empty_like(out["gates"])
    demand, offsets = torch.empty_like(out["demand"]), torch.empty_like(out["offsets"])
    N.moe_forward(cfg, p["x"], p["w_router"], None, p["w_gate"], p["w_up"], p["w_down"],
                  p["shared_gate"], p["shared_up"], p["shared_down"], y, ids, gates, demand,
                  offsets, ws)
    ref = reference(p, out, 4, "topk_softmax", -1, True)
    assert torch.equal(ids, out["ids"]) and torch.equal(demand, out["demand"])
    assert torch.equal(offsets, out["offsets"])
    assert float((gates - out["gates"]).abs().max()) <= 2 * float(ref["bg"].max())
    again = call(N, cfg, p, ws=ws)  # after another kind of call on the same workspace
    assert torch.equal(again["y"], out["y"])


def test_in_place_graph_and_streams(N):
    """y = x; repeated, captured and replayed; two calls at once on two workspaces."""
    p = make(12, 1024, 16, 4, 512, shared=True)
    cfg = N.make_config(12, 1024, 16, 4, 512, has_shared=True, add_residual=True)
    want = call(N, cfg, p)["y"]
    q = dict(p, x=p["x"].clone())
    ws = N.workspace(cfg)
    call(N, cfg, q, ws=ws, y=q["x"])
    assert torch.equal(q["x"], want)

    args = (p["w_router"], None, p["w_gate"], p["w_up"], p["w_down"], p["shared_gate"],
            p["shared_up"], p["shared_down"])
    x, y = p["x"].clone(), torch.empty_like(p["x"])
    count = torch.tensor([12], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        N.moe_forward_few(cfg, x, *args, y, None, None, None, None, count, ws)
        N.moe_forward_few(cfg, y, *args, y, None, None, None, None, count, ws)
    step2 = call(N, cfg, dict(p, x=want.clone()))["y"]
    for _ in range(3):
        y.zero_()
        graph.replay()
        assert torch.equal(y, step2)
    count.fill_(5)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert not bool(y[5:].any()) and bool(y[:5].any())

    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(y), N.workspace(cfg)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (o, w) in zip(streams, outs):
            with torch.cuda.stream(s):
                N.moe_forward_few(cfg, p["x"], *args, o, None, None, None, None, None, w)
    torch.cuda.synchronize()
    for o, w in outs:
        assert torch.equal(o, want) and N.moe_get_device_status(w) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [4, 15, 30])
def test_broken_expert_reaches_its_own_tokens_only(N, T, dtype):
    """Infinities and NaNs in an expert's weights, and in a token, stay with the tokens that
    chose the expert and with that token."""
    p = make(T, 256, 8, 2, 128, dtype, seed=T)
    cfg = N.make_config(T, 256, 8, 2, 128, dtype=dtype)
    before = call(N, cfg, p)
    hit = (before["ids"] == 3).any(1)
    p["w_down"][3, 5, 7], p["w_down"][3, 9, 1] = float("nan"), float("inf")
    p["w_up"][3, 0, 0] = float("inf")
    after = call(N, cfg, p)
    assert torch.equal(before["ids"], after["ids"])
    assert torch.equal(before["y"][~hit], after["y"][~hit])
    assert not bool(torch.isfinite(after["y"][hit][:, 5]).any())
    p = make(T, 256, 8, 2, 128, dtype, seed=T)
    ref = reference(p, before, 2, "topk_softmax")
    p["x"][1, 17] = float("nan")  # it routes to the first experts, which changes the others' shares
    after = call(N, cfg, p)
    rest = torch.arange(T, device="cuda") != 1
    assert torch.equal(before["ids"][rest], after["ids"][rest])
    assert bool(((after["y"].double() - ref["y"]).abs() <= ref["by"])[rest].all())
    assert bool(torch.isnan(after["y"][1]).all())


def test_unaligned_output_and_wide_shapes(N):
    """y at an address that is not 16-byte aligned; a hidden width of many chunks beside a narrow
    model width, and the other way round."""
    for d, F, E, T in ((128, 8192, 6, 5), (6144, 128, 3, 9), (256, 2048, 250, 31)):
        p = make(T, d, E, 3, F, shared=True, seed=d)
        cfg = N.make_config(T, d, E, 3, F, has_shared=True, add_residual=True)
        flat = torch.full((T * d + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = flat[3:3 + T * d].view(T, d)
        out = call(N, cfg, p, n_tokens=T - 1, y=y)
        check(out, reference(p, out, 3, "topk_softmax", -1, True, T - 1), T - 1)
        assert bool((flat[:3] == 7.0).all()) and bool((flat[3 + T * d:] == 7.0).all())


@pytest.mark.parametrize("T", [5, 14, 29])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [False, True])
def test_masked_experts_with_broken_weights(N, T, dtype, shared):
    """A route at a logit of -inf is counted, but does not run: NaNs and infinities in the weights
    of a masked expert reach nobody, also where fewer than k experts are open, or none is."""
    inf = float("inf")
    for bias, cap in (([-inf, -inf, 0.3, -inf, -inf, -inf], -1), ([-inf] * 6, -1),
                      ([-inf, 0.0, -inf, 0.5, -inf, -inf], 2)):
        p = make(T, 256, 6, 3, 128, dtype, shared, bias=bias, seed=T)
        cfg = N.make_config(T, 256, 6, 3, 128, dtype=dtype, has_shared=shared, capacity=cap)
        clean = call(N, cfg, p)
        ref = reference(p, clean, 3, "topk_softmax", cap)
        q = dict(p)
        for name, value in (("w_gate", float("nan")), ("w_up", inf), ("w_down", float("nan"))):
            q[name] = p[name].clone()
            q[name][torch.tensor(bias) == -inf] = value
        out = call(N, cfg, q)
        check(out, ref, T)
        for name in ("ids", "gates", "demand", "offsets", "y"):
            assert torch.equal(out[name], clean[name]), name
        assert out["demand"].tolist() == ref["demand"]
        kept = [c if cap < 0 else min(c, cap) for c in ref["demand"]]
        assert out["offsets"].tolist()[:-1] == [sum(kept[:e]) for e in range(7)]
