"""Cases and plain forms of the operators that serve a decode step with per-request adapters:

  few      the whole MoE layer (router, top-k, experts, combine) for at most 32 tokens
           (``moe_forward_few``)
  linear   a projection shared by all tokens plus each token's own low-rank adapter
           (``moe_adapter_linear``):  y[t] = addend[t] + W x[t] + s_a B_a (A_a x[t])
  gate_up  the SwiGLU pair of such projections (``moe_adapter_gate_up``)

``run`` computes a case in elementary torch operations, or through the package's entry points
when ``own`` is true.
"""
import math

import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _few(name, T, d, E, k, F, dtype="bf16", gate_mode="topk_softmax", shared=False,
         residual=False, bias="none", active=None):
    return {"name": name, "op": "few", "T": T, "d": d, "E": E, "k": k, "F": F, "dtype": dtype,
            "gate_mode": gate_mode, "shared": shared, "residual": residual, "bias": bias,
            "active": T if active is None else active}


def _adapt(name, op, T, d_in, d_out, n, rank, dtype="bf16", mix="tokens", addend=False,
           active=None):
    return {"name": name, "op": op, "T": T, "d_in": d_in, "d_out": d_out, "n": n, "rank": rank,
            "dtype": dtype, "mix": mix, "addend": addend, "active": T if active is None else active}


def listed():
    return [
        # one sequence decoding on a layer of many small experts: latency is everything
        _few("few_granite_T1", 1, 1024, 32, 8, 512, residual=True),
        # a small decode batch on the same layer: nearly every expert is touched
        _few("few_granite_T16", 16, 1024, 32, 8, 512, residual=True),
        # a decode batch on a few large experts with a skewed router: all weights stream
        _few("few_mixtral_T16", 16, 4096, 8, 2, 14336, bias="zipf"),
        # one sequence beside a shared expert: most of the work is the shared expert's
        _few("few_shared16_T1", 1, 4096, 16, 2, 8192, gate_mode="softmax_topk_renorm",
             shared=True, bias="normal"),
        # fp32 at odd sizes, the batch padded to a captured length (4 of 5 rows hold tokens)
        _few("few_f32_odd", 5, 772, 13, 3, 300, dtype="f32", gate_mode="softmax_topk",
             shared=True, residual=True, bias="normal", active=4),
        # one token of one request through an adapted projection
        _adapt("linear_T1", "linear", 1, 4096, 4096, 8, 16, addend=True),
        # a decode batch, every token another request, some of them without an adapter; the
        # down projection of a large expert, its result added to the layer's output
        _adapt("linear_T24_mixed", "linear", 24, 14336, 4096, 64, 16, addend=True),
        # prompts of a few requests back to back (ragged lengths), tensor-core bound
        _adapt("linear_T4099", "linear", 4099, 4096, 4096, 8, 16, mix="requests"),
        # fp32 at odd sizes, padded batch
        _adapt("linear_f32_odd", "linear", 77, 1000, 516, 5, 12, dtype="f32", addend=True,
               active=70),
        # a decode batch through the shared expert's first half
        _adapt("gate_up_T16", "gate_up", 16, 4096, 8192, 32, 16),
        # a wide decode batch, all requests different, larger rank, small projection
        _adapt("gate_up_T200", "gate_up", 200, 1024, 512, 256, 32),
        # prompts through the first half of a large expert: the largest case
        _adapt("gate_up_T1531", "gate_up", 1531, 4096, 14336, 6, 32, mix="requests"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("few", "few", "linear", "gate_up"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    while True:
        if op == "few":
            T = _log(rng, 1, 32)
            unit = 128 if dtype == "bf16" else 4
            d = unit * _log(rng, 256 // unit, 4096 // unit)
            F = unit * _log(rng, 256 // unit, 8192 // unit)
            E = _log(rng, 4, 64)
            k = rng.randint(1, min(8, E))
            case = _few("", T, d, E, k, F, dtype,
                        rng.choice(("topk_softmax", "softmax_topk_renorm", "softmax_topk")),
                        rng.random() < 0.5, rng.random() < 0.5,
                        rng.choice(("none", "normal", "zipf")),
                        T if rng.random() < 0.7 else rng.randint(1, T))
            size = 4 if dtype == "f32" else 2
            if 3 * (E + 1) * d * F * size > 1.5e9:
                continue
        else:
            unit = 8 if dtype == "bf16" else 4
            T = _log(rng, 1, 4096 if dtype == "bf16" else 256)
            d_in = unit * _log(rng, 256 // unit, 8192 // unit)
            d_out = unit * _log(rng, 256 // unit, 8192 // unit)
            rank = unit * rng.choice((1, 2, 4, 8))
            n = _log(rng, 1, 64)
            mix = rng.choice(("tokens", "requests"))
            case = _adapt("", op, T, d_in, d_out, n, rank, dtype, mix,
                          op == "linear" and rng.random() < 0.5,
                          T if rng.random() < 0.7 else rng.randint(1, T))
            cost = T * d_in * d_out * (2 if op == "gate_up" else 1)
            if cost > (4e10 if dtype == "bf16" else 2e9):
                continue
        del case["name"]
        return case


def _randn(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _stack(gen, n, shape, std, dtype):
    out = torch.empty((n,) + shape, dtype=dtype, device="cuda")
    for i in range(n):  # one matrix at a time keeps the fp32 temporaries small
        out[i] = _randn(gen, shape, std, dtype)
    return out


def _requests(gen, T, n):
    """Adapter of each token when requests lie back to back: at most 8 runs of tokens."""
    cuts = (torch.rand(7, generator=gen, device="cuda") * T).long().sort().values
    run = (torch.arange(T, device="cuda")[:, None] >= cuts[None, :]).sum(1)
    owner = torch.randint(-1, n, (8,), generator=gen, device="cuda")
    return owner[run].to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, T = TORCH[case["dtype"]], case["T"]
    st = {"case": case, "n_tokens": torch.tensor([case["active"]], dtype=torch.int32,
                                                 device="cuda")}
    if case["op"] == "few":
        d, E, F = case["d"], case["E"], case["F"]
        st["x"] = _randn(gen, (T, d), 1.0, dt)
        st["w_router"] = _randn(gen, (E, d), d ** -0.5, dt)
        st["logit_bias"] = {
            "none": lambda: None,
            "normal": lambda: torch.randn(E, generator=gen, device="cuda") * 0.5,
            "zipf": lambda: torch.tensor([-1.1 * math.log(e + 1) for e in range(E)],
                                         device="cuda")}[case["bias"]]()
        st["w_gate"] = _stack(gen, E, (F, d), 0.02, dt)
        st["w_up"] = _stack(gen, E, (F, d), 0.02, dt)
        st["w_down"] = _stack(gen, E, (d, F), 0.02, dt)
        sh = case["shared"]
        st["shared_gate"] = _randn(gen, (F, d), 0.02, dt) if sh else None
        st["shared_up"] = _randn(gen, (F, d), 0.02, dt) if sh else None
        st["shared_down"] = _randn(gen, (d, F), 0.02, dt) if sh else None
        st["y"] = _randn(gen, (T, d), 1.0, dt)  # rows without a token stay as they are
    else:
        d, N, n, r = case["d_in"], case["d_out"], case["n"], case["rank"]
        st["x"] = _randn(gen, (T, d), 1.0, dt)
        pair = 2 if case["op"] == "gate_up" else 1
        st["w"] = [_randn(gen, (N, d), 0.02, dt) for _ in range(pair)]
        st["a"] = [_stack(gen, n, (r, d), d ** -0.5, dt) for _ in range(pair)]
        st["b"] = [_stack(gen, n, (N, r), 0.2, dt) for _ in range(pair)]
        st["scale"] = torch.rand(n, generator=gen, device="cuda") + 0.5
        if case["mix"] == "requests":
            st["ids"] = _requests(gen, T, n)
        else:
            st["ids"] = torch.randint(-1, n, (T,), generator=gen, device="cuda").to(torch.int32)
        st["addend"] = _randn(gen, (T, N), 1.0, dt) if case["addend"] else None
        st["y"] = _randn(gen, (T, N), 1.0, dt)
    if own:
        from routing_dispatch_expert_gemm_b200 import native as N_
        if case["op"] == "few":
            st["cfg"] = N_.make_config(T, case["d"], case["E"], case["k"], case["F"],
                                       dtype=case["dtype"], gate_mode=case["gate_mode"],
                                       has_shared=case["shared"], add_residual=case["residual"])
            st["ws"] = N_.workspace(st["cfg"])
            st["ids_out"] = torch.zeros((T, case["k"]), dtype=torch.int32, device="cuda")
            st["gates_out"] = torch.zeros((T, case["k"]), dtype=torch.float32, device="cuda")
        else:
            st["cfg"] = N_.make_adapter_config(T, case["d_in"], case["d_out"], case["n"],
                                               case["rank"], dtype=case["dtype"])
            st["ws"] = N_.adapter_workspace(st["cfg"])
    return st


def _run_own(st):
    from routing_dispatch_expert_gemm_b200 import native as N_
    op = st["case"]["op"]
    if op == "few":
        N_.moe_forward_few(st["cfg"], st["x"], st["w_router"], st["logit_bias"], st["w_gate"],
                           st["w_up"], st["w_down"], st["shared_gate"], st["shared_up"],
                           st["shared_down"], st["y"], st["ids_out"], st["gates_out"], None,
                           None, st["n_tokens"], st["ws"])
        return {"y": st["y"], "ids": st["ids_out"], "gates": st["gates_out"]}
    if op == "linear":
        N_.moe_adapter_linear(st["cfg"], st["x"], st["w"][0], st["a"][0], st["b"][0],
                              st["scale"], st["ids"], st["addend"], st["y"], st["n_tokens"],
                              st["ws"])
    else:
        N_.moe_adapter_gate_up(st["cfg"], st["x"], st["w"][0], st["w"][1], st["a"][0],
                               st["b"][0], st["a"][1], st["b"][1], st["scale"], st["ids"],
                               st["y"], st["n_tokens"], st["ws"])
    return {"y": st["y"]}


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _ffn(x, wg, wu, wd):
    return (_silu(x @ wg.float().t()) * (x @ wu.float().t())) @ wd.float().t()


def _few_plain(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    # 64 bits for the logits: the order of close ones decides which experts run
    z = st["x"].double() @ st["w_router"].double().t()
    if st["logit_bias"] is not None:
        z = z + st["logit_bias"].double()
    top, ids = torch.sort(z, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    e = torch.exp(top - top[:, :1])
    if c["gate_mode"] == "softmax_topk":
        gates = e / torch.exp(z - top[:, :1]).sum(1, keepdim=True)
    else:  # renormalised over the selected experts, or softmax over them: the same value
        gates = e / e.sum(1, keepdim=True)
    gates = gates.float()
    x = st["x"].float()
    weight = torch.zeros((T, E), device=x.device).scatter(1, ids, gates)
    y = torch.zeros_like(x)
    for j in range(E):
        y = y + weight[:, j:j + 1] * _ffn(x, st["w_gate"][j], st["w_up"][j], st["w_down"][j])
    if c["shared"]:
        y = y + _ffn(x, st["shared_gate"], st["shared_up"], st["shared_down"])
    if c["residual"]:
        y = y + x
    live = (torch.arange(T, device=x.device) < st["n_tokens"])[:, None]
    zero = torch.zeros((), device=x.device)
    return {"y": torch.where(live, y.to(st["x"].dtype), st["y"]),
            "ids": torch.where(live, ids, zero.long()).to(torch.int32),
            "gates": torch.where(live, gates, zero)}


def _project(st, i, x):
    out = x @ st["w"][i].float().t()
    for j in range(st["case"]["n"]):
        mine = (st["ids"] == j)[:, None]
        part = (x @ st["a"][i][j].float().t()) @ st["b"][i][j].float().t()
        out = out + torch.where(mine, st["scale"][j] * part, torch.zeros_like(part))
    return out


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "few":
        return _few_plain(state)
    x = state["x"].float()
    y = _project(state, 0, x)
    if c["op"] == "gate_up":
        y = _silu(y) * _project(state, 1, x)
    elif state["addend"] is not None:
        y = y + state["addend"].float()
    live = (torch.arange(c["T"], device=x.device) < state["n_tokens"])[:, None]
    return {"y": torch.where(live, y.to(state["x"].dtype), state["y"])}


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    T = case["active"]
    if case["op"] == "few":
        d, E, k, F = case["d"], case["E"], case["k"], case["F"]
        # experts that T tokens touch, if they choose them evenly
        touched = E * (1.0 - (1.0 - k / E) ** T)
        n_w = touched + (1 if case["shared"] else 0)
        rows = T * (k + (1 if case["shared"] else 0))
        return {"bytes": (3 * n_w * d * F + E * d + 2 * T * d) * size + 8 * T * k,
                "flops": 6 * rows * d * F + 2 * T * d * E}
    d, N, n, r = case["d_in"], case["d_out"], case["n"], case["rank"]
    pair = 2 if case["op"] == "gate_up" else 1
    used = min(n, 8) if case["mix"] == "requests" else n * (1.0 - (1.0 - 1.0 / (n + 1)) ** T)
    used = min(used, T)
    return {"bytes": (pair * (N * d + used * r * (d + N)) + T * (d + N)
                      + (T * N if case["addend"] else 0)) * size + 4 * T,
            "flops": 2 * pair * T * (N * d + r * (d + N))}


def exact(case, seed):
    st = prepare(case, seed)
    x = st["x"].double()
    live = case["active"]
    if case["op"] != "few":
        parts = []
        for w, a, b in zip(st["w"], st["a"], st["b"]):
            out = torch.matmul(x, w.double().transpose(0, 1))
            for t0 in range(0, case["T"], 64):  # every token with its own pair of matrices
                ids = st["ids"][t0:t0 + 64].long()
                has = torch.nonzero(ids >= 0).flatten()
                own_a, own_b = a[ids[has]].double(), b[ids[has]].double()
                u = torch.einsum("trd,td->tr", own_a, x[t0 + has])
                out[t0 + has] += (torch.einsum("tnr,tr->tn", own_b, u)
                                  * st["scale"][ids[has]].double()[:, None])
            parts.append(out)
        y = st["y"].double()
        if case["op"] == "gate_up":
            y[:live] = (parts[0] * torch.sigmoid(parts[0]) * parts[1])[:live]
        else:
            add = 0.0 if st["addend"] is None else st["addend"].double()
            y[:live] = (parts[0] + add)[:live]
        return {"y": y}
    k = case["k"]
    y = st["y"].double()
    ids_all = torch.zeros((case["T"], k), dtype=torch.int32, device=x.device)
    gates_all = torch.zeros((case["T"], k), dtype=torch.float64, device=x.device)

    def expert(v, wg, wu, wd):
        g = torch.mv(wg.double(), v)
        return torch.mv(wd.double(), g * torch.sigmoid(g) * torch.mv(wu.double(), v))

    for t in range(live):  # the definition, token by token
        z = torch.mv(st["w_router"].double(), x[t])
        if st["logit_bias"] is not None:
            z = z + st["logit_bias"].double()
        logits = z.tolist()
        order = sorted(range(case["E"]), key=lambda e: (-logits[e], e))[:k]
        p = torch.softmax(z, 0)[order]
        if case["gate_mode"] != "softmax_topk":
            p = p / p.sum()
        out = torch.zeros_like(x[t])
        for j, e in enumerate(order):
            out += p[j] * expert(x[t], st["w_gate"][e], st["w_up"][e], st["w_down"][e])
        if case["shared"]:
            out += expert(x[t], st["shared_gate"], st["shared_up"], st["shared_down"])
        if case["residual"]:
            out += x[t]
        y[t] = out
        ids_all[t] = torch.tensor(order, dtype=torch.int32)
        gates_all[t] = p
    return {"y": y, "ids": ids_all, "gates": gates_all}
