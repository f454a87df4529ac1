"""Projections with per-token low-rank adapters (moe_adapter_linear, moe_adapter_gate_up)
against a plain 64-bit implementation.

Bounds.  u = 2^-24, r = eps/2 of the storage type, |.|-sums with absolute values throughout.
An fp32 sum of n products in any order is off by at most (n + 2) u times its |.|-sum, so
  v = A x            dv <= (d_in + 2) u |A||x|
  s B v              dd <= |s| |B| dv + (rank + 6) u |s| |B||v| (+ 2^-16 |s| |B||v|: the
                     tensor-core form may keep v in two bf16 halves, 16 bits in all)
  p = W x + s B v    dp <= (d_in + 2) u |W||x| + dd + 4 u (|W||x| + |s||B||v|)
  y = p + addend     dp + 2 u |y| + r |y|
  h = SiLU(g) up     1.1 |up| dg + |SiLU(g)| dup + dg dup + 16 u |h| + r |h|
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


def make(T, d_in, d_out, n, rank, dtype="bf16", mix="tokens", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dtype])

    p = {"x": rn((T, d_in), 1.0), "scale": torch.rand(n, generator=g, device="cuda") + 0.5,
         "addend": rn((T, d_out), 1.0),
         "w": [rn((d_out, d_in), 0.05) for _ in range(2)],
         "a": [rn((n, rank, d_in), d_in ** -0.5) for _ in range(2)],
         "b": [rn((n, d_out, rank), 0.3) for _ in range(2)]}
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda")
    if mix == "requests":  # a few runs of tokens
        ids = ids[(torch.arange(T, device="cuda") * 5 // T) * (T // 5 if T >= 5 else 1)]
    elif mix == "one":
        ids = torch.full((T,), n - 1, device="cuda")
    elif mix == "none":
        ids = torch.full((T,), -1, device="cuda")
    p["ids"] = ids.to(torch.int32)
    return p


def projection(p, i, scale=True):
    """p[t] and its bound, in 64 bits."""
    x, w = p["x"].double(), p["w"][i].double()
    d_in, rank = x.shape[1], p["a"][i].shape[1]
    base, mag = x @ w.t(), x.abs() @ w.abs().t()
    out, dp = base.clone(), (d_in + 6) * U * mag
    for j in range(p["a"][i].shape[0]):
        rows = torch.nonzero(p["ids"] == j).flatten()
        if rows.numel() == 0:
            continue
        a, b = p["a"][i][j].double(), p["b"][i][j].double()
        s = float(p["scale"][j]) if scale else 1.0
        v = x[rows] @ a.t()
        dv = (d_in + 2) * U * (x[rows].abs() @ a.abs().t())
        out[rows] += s * (v @ b.t())
        dp[rows] += s * (dv @ b.abs().t()) + ((rank + 10) * U + 2.0 ** -16) * s * (
            (v.abs() + dv) @ b.abs().t())
    return out, dp


def reference(p, pair, addend=False, scale=True):
    r = torch.finfo(p["x"].dtype).eps / 2
    g, dg = projection(p, 0, scale)
    if not pair:
        y = g + (p["addend"].double() if addend else 0.0)
        return y, (dg + (2 * U + r) * y.abs()) * 1.01 + 1e-30
    up, du = projection(p, 1, scale)
    s = g * torch.sigmoid(g)
    h = s * up
    return h, (1.1 * up.abs() * dg + s.abs() * du + 1.1 * dg * du
               + (16 * U + r) * h.abs()) * 1.01 + 1e-30


def call(N, p, pair, addend=False, n_tokens=None, ws=None, y=None, scale=True, status=0):
    T, d_in = p["x"].shape
    n, rank = p["a"][0].shape[:2]
    d_out = p["w"][0].shape[0]
    dtype = "bf16" if p["x"].dtype == torch.bfloat16 else "f32"
    cfg = N.make_adapter_config(T, d_in, d_out, n, rank, dtype=dtype)
    ws = N.adapter_workspace(cfg) if ws is None else ws
    y = torch.full((T, d_out), 7.0, dtype=p["x"].dtype, device="cuda") if y is None else y
    nt = None if n_tokens is None else torch.tensor([n_tokens], dtype=torch.int32, device="cuda")
    sc = p["scale"] if scale else None
    if pair:
        N.moe_adapter_gate_up(cfg, p["x"], p["w"][0], p["w"][1], p["a"][0], p["b"][0], p["a"][1],
                              p["b"][1], sc, p["ids"], y, nt, ws)
    else:
        N.moe_adapter_linear(cfg, p["x"], p["w"][0], p["a"][0], p["b"][0], sc, p["ids"],
                             p["addend"] if addend else None, y, nt, ws)
    assert N.moe_get_device_status(ws, clear=True) == status
    return y


def check(y, ref, live):
    want, bound = ref
    if live:
        worst = ((y[:live].double() - want[:live]).abs() / bound[:live]).max()
        assert worst <= 1.0, f"error is {float(worst):.2f} of its bound"
    assert bool((y[live:] == 7.0).all())


CASES = [
    # T, d_in, d_out, adapters, rank, dtype, mix, live
    (1, 8, 8, 1, 8, "bf16", "one", None),
    (1, 4096, 1024, 8, 16, "bf16", "one", None),
    (2, 520, 264, 3, 8, "bf16", "tokens", None),
    (7, 1032, 136, 40, 24, "bf16", "tokens", 5),
    (8, 256, 2048, 4, 128, "bf16", "requests", None),
    (9, 512, 4744, 2, 64, "bf16", "none", None),
    (16, 1000, 328, 16, 16, "bf16", "tokens", 16),
    (24, 2056, 64, 1000, 16, "bf16", "tokens", None),
    (31, 128, 5000, 5, 40, "bf16", "requests", 30),
    (32, 72, 40, 32, 128, "bf16", "tokens", None),
    (1, 4, 4, 1, 4, "f32", "one", None),
    (5, 516, 132, 3, 12, "f32", "tokens", 4),
    (13, 1028, 68, 6, 128, "f32", "tokens", None),
    (32, 260, 500, 40, 20, "f32", "requests", None),
    (33, 256, 128, 4, 16, "bf16", "tokens", None),
    (64, 64, 128, 1, 8, "bf16", "one", None),
    (65, 72, 8, 3, 8, "bf16", "tokens", 64),
    (100, 1000, 264, 100, 40, "bf16", "tokens", 97),
    (130, 520, 1032, 5, 128, "bf16", "requests", None),
    (200, 4096, 512, 64, 16, "bf16", "tokens", None),
    (257, 128, 4096, 7, 16, "bf16", "requests", 256),
    (300, 648, 392, 3, 24, "bf16", "none", None),
    (400, 264, 9000, 100, 16, "bf16", "tokens", 390),
    (777, 512, 2048, 6, 32, "bf16", "requests", 700),
    (1031, 264, 5000, 9, 16, "bf16", "tokens", None),
    (1024, 136, 4872, 3, 8, "bf16", "requests", None),
    (1500, 264, 4104, 200, 16, "bf16", "tokens", None),
    (2047, 72, 2056, 5, 128, "bf16", "requests", 1900),
    (2500, 1032, 1944, 40, 24, "bf16", "one", 2305),
    (33, 68, 36, 5, 4, "f32", "tokens", 33),
    (77, 1000, 516, 5, 12, "f32", "tokens", 70),
    (300, 132, 260, 3, 64, "f32", "requests", None),
]


@pytest.mark.parametrize("pair", [False, True], ids=["linear", "gate_up"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:7]))
def test_against_64_bits(N, case, pair):
    T, d_in, d_out, n, rank, dtype, mix, live = case
    p = make(T, d_in, d_out, n, rank, dtype, mix, seed=T + d_in)
    for addend in ((False,) if pair else (False, True)):
        y = call(N, p, pair, addend, live)
        check(y, reference(p, pair, addend), T if live is None else live)


@pytest.mark.parametrize("T", [6, 70])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_ids_and_scale(N, T, dtype):
    p = make(T, 256, 128, 3, 8, dtype)
    for live, seen in ((0, 0), (-5, 0), (1, 1), (T + 9, T)):
        for pair in (False, True):
            check(call(N, p, pair, False, live), reference(p, pair), seen)
    check(call(N, p, False, scale=False), reference(p, False, scale=False), T)
    bad = dict(p, ids=p["ids"].clone())
    bad["ids"][2], bad["ids"][4] = 3, -2  # out of range: no adapter, and flagged
    ref = dict(p, ids=bad["ids"].clone())
    ref["ids"][2] = ref["ids"][4] = -1
    for pair in (False, True):
        check(call(N, bad, pair, status=7), reference(ref, pair), T)
    # behind the last token an id is not looked at
    assert bool((call(N, bad, False, n_tokens=2)[2:] == 7.0).all())


@pytest.mark.parametrize("T", [12, 150, 5000])
def test_in_place_repeat_and_graph(N, T):
    p = make(T, 1024, 512, 6, 16)
    want = call(N, p, False, True)
    y = p["addend"].clone()
    q = dict(p, addend=y)
    call(N, q, False, True, y=y)  # addend is y
    assert torch.equal(y, want)
    assert torch.equal(call(N, p, False, True), want)

    cfg = N.make_adapter_config(T, 1024, 512, 6, 16)
    back = N.make_adapter_config(T, 512, 1024, 6, 16)
    ws = N.adapter_workspace(back)
    down = make(T, 512, 1024, 6, 16, seed=3)
    h, out = torch.empty((T, 512), dtype=torch.bfloat16, device="cuda"), torch.empty_like(p["x"])
    count = torch.tensor([T], dtype=torch.int32, device="cuda")

    def ffn():
        N.moe_adapter_gate_up(cfg, p["x"], p["w"][0], p["w"][1], p["a"][0], p["b"][0], p["a"][1],
                              p["b"][1], p["scale"], p["ids"], h, count, ws)
        N.moe_adapter_linear(back, h, down["w"][0], down["a"][0], down["b"][0], down["scale"],
                             p["ids"], p["x"], out, count, ws)

    ffn()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffn()
    for _ in range(3):
        h.zero_()
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    check(h, reference(p, True), T)
    p["ids"].fill_(-1)  # the adapters of a replay are read when it runs
    graph.replay()
    check(h, reference(p, True), T)

    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(want), N.adapter_workspace(cfg)) for _ in streams]
    want = call(N, p, False, True)
    for _ in range(4):
        for s, (o, w) in zip(streams, outs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                N.moe_adapter_linear(cfg, p["x"], p["w"][0], p["a"][0], p["b"][0], p["scale"],
                                     p["ids"], p["addend"], o, None, w)
    torch.cuda.synchronize()
    for o, _ in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("T", [9, 48])
def test_layer_with_adapted_shared_expert(N, T):
    """The layer's routed part, then the shared expert with each request's adapters, added in
    place: what a decode step runs."""
    d, F, E, k = 512, 256, 8, 2
    g = torch.Generator(device="cuda").manual_seed(5)

    def rn(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()

    up, down = make(T, d, F, 4, 16, seed=1), make(T, F, d, 4, 16, seed=2)
    x, ids = up["x"], up["ids"]
    wr, wg, wu, wd = rn((E, d), d ** -0.5), rn((E, F, d), .05), rn((E, F, d), .05), rn((E, d, F), .05)
    cfg = N.make_config(T, d, E, k, F, add_residual=True)
    ws = N.workspace(cfg)
    y = torch.empty_like(x)
    fwd = N.moe_forward_few if T <= 32 else N.moe_forward
    extra = (None, ws) if T <= 32 else (ws,)
    fwd(cfg, x, wr, None, wg, wu, wd, None, None, None, y, None, None, None, None, *extra)
    routed = y.clone()
    c1, c2 = N.make_adapter_config(T, d, F, 4, 16), N.make_adapter_config(T, F, d, 4, 16)
    h = torch.empty((T, F), dtype=torch.bfloat16, device="cuda")
    aws = N.adapter_workspace(c2)
    N.moe_adapter_gate_up(c1, x, up["w"][0], up["w"][1], up["a"][0], up["b"][0], up["a"][1],
                          up["b"][1], up["scale"], ids, h, None, aws)
    N.moe_adapter_linear(c2, h, down["w"][0], down["a"][0], down["b"][0], down["scale"], ids, y, y,
                         None, aws)
    check(h, reference(up, True), T)
    check(y, reference(dict(down, x=h, ids=ids, addend=routed), False, True), T)
    assert N.moe_get_device_status(ws) == 0 and N.moe_get_device_status(aws) == 0


@pytest.mark.parametrize("T,d_out", [(6, 64), (90, 64), (700, 5000), (700, 64), (1000, 5000)])
def test_broken_adapter_reaches_its_own_tokens_only(N, T, d_out):
    """Infinities and NaNs in one request's adapter, also in matrices that no token uses."""
    for dtype in ("bf16", "f32"):
        for mix in ("tokens", "requests"):
            p = make(T, 128, d_out, 5, 16, dtype, mix, seed=7)
            p["ids"][T // 2] = 2
            clean = [call(N, p, pair) for pair in (False, True)]
            for i in range(2):
                p["a"][i][1, 3, 5] = float("inf")
                p["b"][i][2, 7, 3] = float("nan")
                p["b"][i][2, d_out - 1, 0] = float("inf")
                p["a"][i][4].fill_(float("nan"))
            p["ids"][p["ids"] == 1] = 0
            p["ids"][p["ids"] == 4] = -1
            good = p["ids"] != 2
            for pair in (False, True):
                q = dict(p, a=[a.clone() for a in p["a"]], b=[b.clone() for b in p["b"]])
                for i in range(2):
                    q["a"][i][1, 3, 5], q["b"][i][2, 7, 3], q["b"][i][2, -1, 0] = 0.0, 0.0, 0.0
                    q["a"][i][4].fill_(0.0)
                y = call(N, p, pair)
                want, bound = reference(q, pair)
                err = (y.double() - want).abs() <= bound
                assert bool(err[good].all())
                own = ~good
                assert bool(torch.isnan(y[own][:, 7]).all())
                assert not bool(torch.isfinite(y[own][:, -1]).any())
                rest = [c for c in range(d_out) if c not in (7, d_out - 1)]
                assert bool(err[own][:, rest].all())
            del clean


@pytest.mark.parametrize("T,d_out", [(20, 64), (200, 512), (777, 2048), (5000, 2048)])
def test_few_live_tokens_and_unaligned_outputs(N, T, d_out):
    """A batch padded to many times its tokens; y and the addend at addresses that are not
    16-byte aligned."""
    p = make(T, 64, d_out, 4, 8, mix="requests", seed=2)
    for live in (0, 1, T // 3):
        for pair in (False, True):
            check(call(N, p, pair, n_tokens=live), reference(p, pair), live)
    flat = torch.full((T * d_out + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    add = torch.empty_like(flat)
    add[3:3 + T * d_out] = p["addend"].flatten()
    y = flat[1:1 + T * d_out].view(T, d_out)
    q = dict(p, addend=add[3:3 + T * d_out].view(T, d_out))
    check(call(N, q, False, True, n_tokens=T - 1, y=y), reference(p, False, True), T - 1)
    assert bool((flat[1 + T * d_out:] == 7.0).all()) and float(flat[0]) == 7.0
    check(call(N, p, True, y=y), reference(p, True), T)


def test_adapters_of_another_stream_and_order(N):
    """The tensors of one stream used on another, after an event: the call runs on the stream it
    is given."""
    p = make(50, 512, 256, 3, 16)
    want = call(N, p, False)
    cfg = N.make_adapter_config(50, 512, 256, 3, 16)
    ws = N.adapter_workspace(cfg)
    y = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    N.moe_adapter_linear(cfg, p["x"], p["w"][0], p["a"][0], p["b"][0], p["scale"], p["ids"], None,
                         y, None, ws, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("T,d_out", [(6, 64), (90, 64), (700, 5000), (700, 64), (1000, 5000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_shrink(N, T, d_out, dtype):
    """A x of one adapter is +inf in one rank and its B is positive there: the formula gives
    +inf in every output of its tokens, and the others know nothing of it."""
    p = make(T, 128, d_out, 4, 16, dtype, "requests", seed=3)
    p["ids"][T // 2] = 2
    p["a"][0][2, 5, 9] = float("inf")
    p["x"][:, 9] = 1.0
    p["b"][0][2, :, 5] = 0.5
    own = p["ids"] == 2
    y = call(N, p, False)
    assert bool((y[own] == float("inf")).all())
    q = dict(p, a=[p["a"][0].clone()])
    q["a"][0][2, 5, 9] = 0.0
    want, bound = reference(q, False)
    assert bool(((y.double() - want).abs() <= bound)[~own].all())


def test_broken_rows_of_rare_adapters(N):
    """Adapters in the first token block alone: the tiles between two of its tiles have none.
    Infinities in B in the rows of its first tiles, which the later ones do not meet."""
    T, d_out = 8192, 10240
    p = make(T, 64, d_out, 3, 8, mix="none", seed=4)
    p["ids"][:100] = 1
    p["b"][0][1, :256, 2] = float("inf")
    y = call(N, p, False)
    v = (p["x"][:100].double() @ p["a"][0][1].double().t())[:, 2]
    sign = torch.where(v > 0, float("inf"), float("-inf"))  # v is no zero: 64 random products
    assert bool((y[:100, :256].double() == sign[:, None]).all())
    q = dict(p, w=[p["w"][0][256:]], b=[p["b"][0][:, 256:].contiguous()])
    want, bound = reference(q, False)
    assert bool(((y[:, 256:].double() - want).abs() <= bound).all())
    assert bool(torch.isfinite(y[100:]).all())


@pytest.mark.parametrize("pair", [False, True], ids=["linear", "gate_up"])
def test_calls_on_two_streams_at_once(N, pair):
    """Calls whose kernels wait for all of their CTAs, on two streams, each with its own
    workspace: the same bits as one after the other."""
    shapes = [(3, 512, 1024), (24, 2048, 4096), (40, 4096, 512), (100, 512, 512)]
    ps = [make(T, d_in, d_out, 6, 16, seed=T) for T, d_in, d_out in shapes]
    want = [call(N, p, pair) for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(6):
        for i, p in enumerate(ps):
            for s in streams:
                with torch.cuda.stream(s):
                    T, d_in, d_out = shapes[i]
                    cfg = N.make_adapter_config(T, d_in, d_out, 6, 16)
                    ws = N.adapter_workspace(cfg)
                    y = torch.zeros((T, d_out), dtype=torch.bfloat16, device="cuda")
                    if pair:
                        N.moe_adapter_gate_up(cfg, p["x"], p["w"][0], p["w"][1], p["a"][0],
                                              p["b"][0], p["a"][1], p["b"][1], p["scale"],
                                              p["ids"], y, None, ws)
                    else:
                        N.moe_adapter_linear(cfg, p["x"], p["w"][0], p["a"][0], p["b"][0],
                                             p["scale"], p["ids"], None, y, None, ws)
                    got.append((i, y, ws))
    torch.cuda.synchronize()
    for i, y, ws in got:
        assert torch.equal(y, want[i]) and N.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("T,d_in,d_out,n,mix", [
    (16, 4096, 8192, 16, "tokens"), (24, 14336, 264, 64, "tokens"), (33, 1032, 520, 40, "tokens"),
    (64, 1024, 1024, 64, "tokens"), (64, 4104, 136, 3, "requests"), (128, 520, 264, 9, "one"),
    (12, 16384, 4096, 5, "none"), (129, 2048, 256, 129, "tokens")])
def test_shrink_inside_the_gemm(N, T, d_in, d_out, n, mix):
    """Shapes whose GEMM splits the contraction, around the sizes where it shrinks by itself;
    the same workspace again and again, with other counts of tokens, eagerly and from a graph."""
    p = make(T, d_in, d_out, n, 16, mix=mix, seed=5)
    cfg = N.make_adapter_config(T, d_in, d_out, n, 16)
    ws = N.adapter_workspace(cfg)
    for pair in (False, True):
        ref = reference(p, pair)
        check(call(N, p, pair, ws=ws), ref, T)
        for live in (0, 1, T // 2 + 1):
            check(call(N, p, pair, n_tokens=live, ws=ws), ref, live)
        y = torch.full((T, d_out), 7.0, dtype=torch.bfloat16, device="cuda")
        count = torch.tensor([T], dtype=torch.int32, device="cuda")
        args = ((p["w"][0], p["w"][1], p["a"][0], p["b"][0], p["a"][1], p["b"][1]) if pair else
                (p["w"][0], p["a"][0], p["b"][0]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if pair:
                N.moe_adapter_gate_up(cfg, p["x"], *args, p["scale"], p["ids"], y, count, ws)
            else:
                N.moe_adapter_linear(cfg, p["x"], *args, p["scale"], p["ids"], None, y, count, ws)
        for live in (T, 2, T - 1):
            y.fill_(7.0)
            count.fill_(live)
            g.replay()
            check(y, ref, live)
        assert N.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("T,d_in,d_out", [
    (18688, 128, 64), (18689, 128, 64), (18816, 72, 128), (18944, 256, 128), (18945, 128, 128)])
def test_prompts_beside_a_narrow_projection(N, T, d_in, d_out):
    """A row block or two of W and so many tokens that SM pairs run the GEMM: around the token
    counts where as many CTAs could also split the contraction."""
    p = make(T, d_in, d_out, 6, 16, mix="requests", seed=9)
    for pair in (False, True):
        check(call(N, p, pair), reference(p, pair), T)


# T, d_in, d_out: streaming, split, one CTA per tile (twice), SM pairs
BROKEN_SHAPES = [(6, 128, 64), (90, 128, 64), (90, 64, 64), (700, 128, 5000), (1000, 128, 5000)]


@pytest.mark.parametrize("T,d_in,d_out", BROKEN_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_shrink_beside_a_broken_adapter(N, T, d_in, d_out, dtype):
    """One request's A x is +inf in one rank (its outputs are +inf), another's B holds a NaN and
    an infinity: neither knows of the other, whatever tile they share."""
    p = make(T, d_in, d_out, 4, 16, dtype, "requests", seed=3)
    p["ids"][T // 2], p["ids"][T // 2 + 1] = 2, 1
    p["a"][0][2, 5, 9] = float("inf")
    p["x"][:, 9] = 1.0
    p["b"][0][2, :, 5] = 0.5
    p["b"][0][1, 7, 3], p["b"][0][1, d_out - 1, 4] = float("nan"), float("inf")
    y = call(N, p, False)
    assert bool((y[p["ids"] == 2] == float("inf")).all())
    broken = p["ids"] == 1
    assert bool(torch.isnan(y[broken][:, 7]).all())
    assert not bool(torch.isfinite(y[broken][:, d_out - 1]).any())
    q = dict(p, a=[p["a"][0].clone()], b=[p["b"][0].clone()])
    q["a"][0][2, 5, 9] = q["b"][0][1, 7, 3] = q["b"][0][1, d_out - 1, 4] = 0.0
    want, bound = reference(q, False)
    good = (y.double() - want).abs() <= bound
    assert bool(good[(p["ids"] != 2) & ~broken].all())
    rest = [c for c in range(d_out) if c not in (7, d_out - 1)]
    assert bool(good[broken][:, rest].all())


@pytest.mark.parametrize("side", [0, 1], ids=["gate", "up"])
@pytest.mark.parametrize("T,d_in,d_out", BROKEN_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_shrink_of_one_projection(N, T, d_in, d_out, dtype, side):
    """A x of one request is +inf for the gate or for the up projection alone: h is the infinity
    that SiLU(gate) up gives, since the other projection stays finite."""
    p = make(T, d_in, d_out, 4, 16, dtype, "requests", seed=6)
    p["ids"][T // 2] = 2
    p["a"][side][2, 5, 9] = float("inf")
    p["x"][:, 9] = 1.0
    p["b"][side][2, :, 5] = 0.5
    own = p["ids"] == 2
    h = call(N, p, True)
    other, slack = projection(p, 1 - side)  # SiLU has the sign of its argument
    clear = other.abs() > slack
    want = torch.where(other > 0, float("inf"), float("-inf"))
    assert float(clear[own].double().mean()) > 0.9
    assert bool((h.double() == want)[own[:, None] & clear].all())
    q = dict(p, a=[a.clone() for a in p["a"]])
    q["a"][side][2, 5, 9] = 0.0
    want, bound = reference(q, True)
    assert bool(((h.double() - want).abs() <= bound)[~own].all())


@pytest.mark.parametrize("T,d_in,d_out", BROKEN_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_shrink_meets_an_infinite_row(N, T, d_in, d_out, dtype):
    """inf * inf and inf * -inf in the same rank are infinities, not NaNs."""
    p = make(T, d_in, d_out, 4, 16, dtype, "requests", seed=8)
    p["ids"][T // 2] = 2
    p["a"][0][2, 5, 9] = float("inf")
    p["x"][:, 9] = 1.0
    p["b"][0][2, :, 5] = 0.5
    p["b"][0][2, 3, 5], p["b"][0][2, 6, 5] = float("inf"), float("-inf")
    y = call(N, p, False)[p["ids"] == 2].float()
    assert bool((y[:, 6] == float("-inf")).all())
    assert bool((y[:, [c for c in range(d_out) if c != 6]] == float("inf")).all())


@pytest.mark.parametrize("T,d_in,d_out", [(3, 512, 256), (24, 2048, 1024), (700, 128, 5000)])
def test_clear_then_call_on_a_side_stream(N, T, d_in, d_out):
    """A recorded error clears the whole header, on the stream that is named and before the call
    returns: the next launch on it finds all counts zero."""
    p = make(T, d_in, d_out, 4, 16, seed=2)
    want = call(N, p, False)
    bad = dict(p, ids=p["ids"].clone())
    bad["ids"][0] = 99
    cfg = N.make_adapter_config(T, d_in, d_out, 4, 16)
    ws = N.adapter_workspace(cfg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(want)

    def run(q):
        N.moe_adapter_linear(cfg, q["x"], q["w"][0], q["a"][0], q["b"][0], q["scale"], q["ids"],
                             None, y, None, ws, stream=side)

    for _ in range(20):
        run(bad)
        assert N.moe_get_device_status(ws, stream=side) == 7  # kept until it is cleared
        assert N.moe_get_device_status(ws, stream=side, clear=True) == 7
        run(p)
        assert N.moe_get_device_status(ws, stream=side, clear=True) == 0
        assert torch.equal(y, want)
    header = ws[:256].view(torch.int32)
    header.copy_(torch.arange(1, 65))  # as a launch that timed out may leave it
    torch.cuda.synchronize()
    assert N.moe_get_device_status(ws, stream=side, clear=True) == 1
    assert not bool(header.any())
    run(p)
    assert N.moe_get_device_status(ws, stream=side) == 0 and torch.equal(y, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_workspace_of_the_largest_batch(N, dtype):
    """A workspace sized for the largest batch and rank serves the smaller calls of a server, of
    either projection, and nothing behind it is written."""
    most = N.moe_adapter_workspace_bytes(N.make_adapter_config(513, 64, 64, 1, 32, dtype))
    buf = torch.full((most + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    ws = buf[:most]
    N.moe_workspace_init(ws)
    for T, d_in, d_out, rank in ((513, 2048, 512, 16), (512, 2048, 512, 32), (257, 4096, 1024, 16),
                                 (256, 4096, 1024, 32), (64, 2048, 2048, 32), (17, 16384, 256, 16),
                                 (3, 128, 4096, 32), (1, 64, 64, 8), (480, 4096, 128, 32)):
        p = make(T, d_in, d_out, 5, rank, dtype, seed=T)
        for pair in (False, True):
            check(call(N, p, pair, ws=ws), reference(p, pair), T)
    assert bool((buf[most:] == 0x5a).all())


@pytest.mark.parametrize("used", [4, 5, 8, 15, 16, 17, 40])
@pytest.mark.parametrize("T,d_in,d_out,rank", [
    (300, 64, 264, 8), (300, 64, 264, 32), (1024, 72, 5000, 8), (1279, 128, 5000, 16)])
def test_adapters_of_a_token_block(N, T, d_in, d_out, rank, used):
    """Around the number of adapters that a token block passes through K blocks, evenly mixed and
    with the first one on nearly all tokens; the last block is a short one."""
    p = make(T, d_in, d_out, 64, rank, seed=used)
    even = torch.arange(T, device="cuda") % used
    skewed = torch.where(torch.arange(T, device="cuda") % 256 < used, even, 0)
    for ids in (even, skewed):
        p["ids"] = (63 - ids).to(torch.int32)
        for pair in (False, True):
            check(call(N, p, pair), reference(p, pair), T)


@pytest.mark.parametrize("pair", [False, True], ids=["linear", "gate_up"])
def test_a_wait_that_runs_out(N, pair):
    """A ticket word past the work: no CTA shrinks, and the wait for the pieces ends at its time
    limit with MOE_ERR_TIMEOUT, y as it was.  Cleared, the workspace serves again."""
    T, d_in, d_out = 33, 1032, 520  # the split form that shrinks by itself
    p = make(T, d_in, d_out, 6, 16, seed=1)
    want = call(N, p, pair)
    cfg = N.make_adapter_config(T, d_in, d_out, 6, 16)
    ws = N.adapter_workspace(cfg)
    assert torch.equal(call(N, p, pair, ws=ws), want)
    ws[200:204].view(torch.int32).fill_(1 << 20)  # zero between launches
    y = call(N, p, pair, ws=ws, status=6)
    assert bool((y == 7.0).all())
    assert not bool(ws[:256].any())
    for _ in range(3):
        assert torch.equal(call(N, p, pair, ws=ws), want)


@pytest.mark.parametrize("pair", [False, True], ids=["linear", "gate_up"])
@pytest.mark.parametrize("case", [
    (1, 1028, 132, 3, 12, "f32", None), (3, 2052, 516, 40, 20, "f32", None),
    (4, 1024, 2048, 4, 128, "f32", 3), (5, 1540, 260, 3, 8, "f32", None),
    (8, 2052, 1028, 9, 64, "f32", 7), (8, 1028, 1032, 9, 16, "f32", None),
    (9, 1540, 260, 5, 8, "f32", None), (2, 132, 4100, 2, 4, "f32", None),
    (16, 516, 4360, 16, 36, "f32", None), (11, 72, 5000, 40, 128, "f32", 10),
    (17, 516, 4360, 5, 8, "f32", 16), (32, 8, 4100, 5, 8, "f32", None),
    (8, 4096, 8200, 16, 16, "bf16", None), (8, 4096, 8200, 16, 32, "bf16", None),
    (16, 4096, 4104, 16, 128, "bf16", None), (32, 4096, 2056, 16, 128, "bf16", 31),
    (32, 4096, 2056, 16, 64, "bf16", None), (16, 8, 4096, 4, 32, "bf16", None),
    (40, 8, 136, 4, 8, "bf16", None), (70, 56, 5000, 9, 48, "bf16", 65),
    (300, 16, 5000, 9, 48, "bf16", None), (1024, 8, 5000, 3, 16, "bf16", None)],
    ids=lambda c: "-".join(str(v) for v in c[:6]))
def test_where_the_kernels_change(N, case, pair):
    """On both sides of the sizes, types and ranks that decide between the kernels, and
    contractions shorter than a K block."""
    T, d_in, d_out, n, rank, dtype, live = case
    p = make(T, d_in, d_out, n, rank, dtype, seed=T + rank)
    check(call(N, p, pair, n_tokens=live), reference(p, pair), T if live is None else live)


@pytest.mark.parametrize("pair", [False, True], ids=["linear", "gate_up"])
@pytest.mark.parametrize("T,d_in,d_out,n", [(90, 64, 64, 4), (700, 128, 5000, 16), (1000, 128, 5000, 16)])
def test_nothing_of_a_broken_call_stays(N, T, d_in, d_out, n, pair):
    """A call with a broken request, then clean ones on the same workspace: the bits of a fresh
    one, also where requests without an adapter came between."""
    p = make(T, d_in, d_out, n, 16, seed=4)
    want = call(N, p, pair)
    ws = N.adapter_workspace(N.make_adapter_config(T, d_in, d_out, n, 16))
    q = dict(p, x=p["x"].clone(), b=[b.clone() for b in p["b"]])
    q["x"][::3, 1] = float("inf")
    q["b"][0][1, 3, 4] = float("nan")
    gone = dict(p, ids=torch.full_like(p["ids"], -1))
    for before in (q, gone, q):
        call(N, before, pair, ws=ws)
        assert torch.equal(call(N, p, pair, ws=ws), want)
        live = T // 2
        check(call(N, p, pair, n_tokens=live, ws=ws), reference(p, pair), live)


@pytest.mark.parametrize("dtype,T", [("bf16", 5), ("bf16", 64), ("bf16", 200), ("bf16", 1200),
                                     ("f32", 4), ("f32", 16), ("f32", 200)])
def test_adapters_past_32_bit_offsets(N, dtype, T):
    """More than 2^31 elements in A and in B: the first and the last adapter in use."""
    d, d_out, rank, n = 2056, 4104, 128, 8192
    g = torch.Generator(device="cuda").manual_seed(T)
    p = make(T, d, d_out, 2, rank, dtype, seed=T)
    big = dict(p, scale=torch.ones(n, device="cuda"))
    ids = torch.randint(-1, 2, (T,), generator=g, device="cuda").to(torch.int32)
    ids[-1] = 1
    a = torch.empty((n, rank, d), dtype=DT[dtype], device="cuda")
    b = torch.empty((n, d_out, rank), dtype=DT[dtype], device="cuda")
    assert a.numel() > 2 ** 31 and b.numel() > 2 ** 31
    for big_m, small_m in ((a, p["a"]), (b, p["b"])):
        big_m[0], big_m[n - 1] = small_m[0][0], small_m[0][1]
    big["a"], big["b"] = [a, a], [b, b]
    big["scale"][0], big["scale"][n - 1] = p["scale"][0], p["scale"][1]
    big["ids"] = torch.where(ids == 1, n - 1, ids).to(torch.int32)
    p["ids"], p["a"], p["b"] = ids, [p["a"][0]] * 2, [p["b"][0]] * 2
    for pair in (False, True):
        check(call(N, big, pair), reference(p, pair), T)


@pytest.mark.parametrize("dtype,pair", [("bf16", False), ("bf16", True), ("f32", False),
                                        ("f32", True)])
def test_outputs_past_32_bit_offsets(N, dtype, pair):
    """More than 2^31 outputs: the rows at the beginning, around 2^31 elements and at the end."""
    T, d_in, d_out = 262400, 64, 8200
    p = make(T, d_in, d_out, 3, 16, dtype, "requests", seed=1)
    y = torch.full((T, d_out), 7.0, dtype=DT[dtype], device="cuda")
    call(N, p, pair, not pair, T - 3, y=y)
    middle = 2 ** 31 // d_out
    rows = torch.cat([torch.arange(0, 300), torch.arange(middle - 150, middle + 150),
                      torch.arange(T - 300, T - 3)]).cuda()
    q = dict(p, x=p["x"][rows], ids=p["ids"][rows], addend=p["addend"][rows])
    check(y[rows], reference(q, pair, not pair), len(rows))
    assert bool((y[T - 3:] == 7.0).all())
