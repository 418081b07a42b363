"""Cases for the tensor-parallel layer operators: the gated feed-forward block
and the linear cross entropy over a split vocabulary, each over N rank
buffers of one GPU.

With ``own`` false ``run`` computes a case from elementary torch operations in
fp32 (rounded once to the payload type); with ``own`` true it makes the calls a
user makes of the library.

A case: ``op`` ("ffn" or "xent"), ``train`` (forward alone, or forward and
backward), ``ranks`` N, ``rows`` T, ``hidden`` H, ``size`` (the rank's share I of
the inner size, or the whole vocabulary V), ``act`` (feed-forward only) and
``dtype``.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, train, ranks, rows, hidden, size, dtype, act="silu"):
    c = {"name": name, "op": op, "train": train, "ranks": ranks, "rows": rows, "hidden": hidden, "size": size,
         "dtype": dtype, "act": act if op == "ffn" else ""}
    return c


def listed():
    return [
        # One decoded token through a layer split 8 ways (hidden 5120, the
        # tensor-parallel activations of the benchmark): weights streamed once.
        _case("ffn-decode-t1", "ffn", False, 8, 1, 5120, 1728, "bf16"),
        # A small layer on one GPU, a few tokens: the latency of a call.
        _case("ffn-small-t5", "ffn", False, 1, 5, 1024, 2816, "bf16"),
        # A decode batch, between weight streaming and matrix products.
        _case("ffn-decode-t64", "ffn", False, 8, 64, 5120, 1728, "bf16"),
        # A prompt of 512 tokens.
        _case("ffn-prefill-t512", "ffn", False, 8, 512, 5120, 1728, "bf16"),
        # A training step of the same layer.
        _case("ffn-train-t8192", "ffn", True, 8, 8192, 5120, 1728, "bf16"),
        # Sizes that fill no tile and no 16-byte vector.
        _case("ffn-train-ragged", "ffn", True, 3, 777, 1001, 363, "bf16", "gelu"),
        # Training in full precision.
        _case("ffn-train-f32", "ffn", True, 2, 1024, 2048, 2816, "f32", "gelu_tanh"),
        # The log-likelihood of one next token.
        _case("xent-score-t1", "xent", False, 8, 1, 5120, 131072, "bf16"),
        # Scoring a short continuation with a small model.
        _case("xent-score-t48", "xent", False, 4, 48, 2048, 32000, "bf16"),
        # The loss of a training step, vocabulary split 8 ways.
        _case("xent-train-t4096", "xent", True, 8, 4096, 5120, 131072, "bf16"),
        # Ragged rows, hidden size and vocabulary (shards of unequal length).
        _case("xent-train-ragged", "xent", True, 3, 611, 1003, 10007, "bf16"),
        # Training in full precision.
        _case("xent-train-f32", "xent", True, 2, 1024, 1024, 16000, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "xent"])
    train = rng.random() < 0.5
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    ranks = rng.choice([1, 2, 3, 4, 8])
    while True:
        rows = _log_int(rng, 2, 8192) if train else _log_int(rng, 1, 1024)
        hidden = _log_int(rng, 128, 8192)
        size = _log_int(rng, 64, 8192) if op == "ffn" else _log_int(rng, 1000, 131072)
        # Most models have sizes of whole vectors; one draw in four keeps its own.
        if rng.random() < 0.75:
            hidden = (hidden + 63) // 64 * 64
            size = (size + 31) // 32 * 32
        flops = (3 if train else 1) * rows * hidden * size * (6 * ranks if op == "ffn" else 2)
        nbytes = hidden * size * (3 * ranks if op == "ffn" else 1) * (2 if dtype == "bf16" else 4)
        if flops <= (4e12 if dtype == "bf16" else 8e11) and nbytes <= 1.4e9:
            break
    act = rng.choice(["silu", "gelu", "gelu_tanh"]) if op == "ffn" else ""
    return {"op": op, "train": train, "ranks": ranks, "rows": rows, "hidden": hidden, "size": size, "dtype": dtype,
            "act": act}


def _shards(case):
    """Vocabulary rows of each rank: blocks of ceil(V / N)."""
    v, n = case["size"], case["ranks"]
    b = -(-v // n)
    return [max(0, min((r + 1) * b, v) - r * b) for r in range(n)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    n, rows, hidden, size = case["ranks"], case["rows"], case["hidden"], case["size"]

    def normal(*shape, scale=1.0):
        t = torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)
        return t.mul_(scale).to(dt)

    state = {"case": dict(case)}
    if case["op"] == "ffn":
        # Activations as a normalisation leaves them, one copy per rank;
        # weights that keep the variance.
        x = normal(rows, hidden)
        state["x"] = [x.clone() for _ in range(n)]
        state["w_gate"] = [normal(size, hidden, scale=hidden ** -0.5) for _ in range(n)]
        state["w_up"] = [normal(size, hidden, scale=hidden ** -0.5) for _ in range(n)]
        state["w_down"] = [normal(hidden, size, scale=(n * size) ** -0.5) for _ in range(n)]
        if case["train"]:
            dout = normal(rows, hidden, scale=0.05)
            state["dout"] = [dout.clone() for _ in range(n)]
        return state
    shards = _shards(case)
    w = [normal(v, hidden, scale=1.5 * hidden ** -0.5) for v in shards]
    target = torch.randint(0, size, (rows,), generator=gen, device=dev)
    # A model that has learned something: the hidden state leans towards its
    # target's weights, by an amount that differs from row to row.
    lean = torch.rand(rows, 1, generator=gen, device=dev) * 4.0
    x = torch.randn(rows, hidden, generator=gen, device=dev)
    x = (x + lean * torch.cat(w)[target].float()).to(dt)
    # Padding and prompt tokens carry no loss.
    if rows > 8:
        target = torch.where(torch.rand(rows, generator=gen, device=dev) < 0.1,
                             torch.full_like(target, -100), target)
    state["x"] = [x.clone() for _ in range(n)]
    state["w"] = w
    state["target"] = target
    if case["train"]:
        valid = (target >= 0).float()
        state["grad_loss"] = valid / valid.sum().clamp(min=1.0)
    return state


# ---- plain forms: elementary operations in fp32 ----


def _act(z, act):
    """(act(z), act'(z))"""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        phi = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    k, c = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(k * (z + c * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3.0 * c * z * z)


def _plain_ffn(state):
    case = state["case"]
    dt = DTYPES[case["dtype"]]
    res = {"out": []}
    if case["train"]:
        res.update(dx=[], dw_gate=[], dw_up=[], dw_down=[])
    for r in range(case["ranks"]):
        x, wg, wu, wd = (state[k][r].float() for k in ("x", "w_gate", "w_up", "w_down"))
        g, u = x @ wg.T, x @ wu.T
        a, da = _act(g, case["act"])
        h = a * u
        res["out"].append((h @ wd.T).to(dt))
        if case["train"]:
            dout = state["dout"][r].float()
            dh = dout @ wd
            dg, du = dh * u * da, dh * a
            res["dx"].append((dg @ wg + du @ wu).to(dt))
            res["dw_gate"].append((dg.T @ x).to(dt))
            res["dw_up"].append((du.T @ x).to(dt))
            res["dw_down"].append((dout.T @ h).to(dt))
    return res


def _plain_xent(state):
    case = state["case"]
    dt = DTYPES[case["dtype"]]
    n = case["ranks"]
    target, shards = state["target"], _shards(case)
    valid = (target >= 0) & (target < case["size"])
    xs = [x.float() for x in state["x"]]
    logits = [xs[r] @ state["w"][r].float().T for r in range(n)]
    top = torch.stack([z.amax(1) for z in logits if z.shape[1]]).amax(0)
    total = sum(torch.exp(z - top[:, None]).sum(1) for z in logits)
    lse = top + torch.log(total)
    at = torch.zeros_like(lse)
    row = torch.arange(case["rows"], device=lse.device)
    first, hits = 0, []
    for r in range(n):
        mine = valid & (target >= first) & (target < first + shards[r])
        local = torch.where(mine, target - first, torch.zeros_like(target))
        if shards[r]:
            at = torch.where(mine, logits[r][row, local], at)
        hits.append((mine, local))
        first += shards[r]
    loss = torch.where(valid, lse - at, torch.zeros_like(lse))
    res = {"loss": [loss.clone() for _ in range(n)], "lse": [lse.clone() for _ in range(n)]}
    if case["train"]:
        grad = torch.where(valid, state["grad_loss"], torch.zeros_like(lse))
        res["dx"], res["dw"] = [], []
        for r in range(n):
            mine, local = hits[r]
            d = torch.exp(logits[r] - lse[:, None])
            if shards[r]:
                d[row, local] -= mine.float()
            d *= grad[:, None]
            res["dx"].append((d @ state["w"][r].float()).to(dt))
            res["dw"].append((d.T @ xs[r]).to(dt))
    return res


# ---- the library's calls ----


def _own_ffn(state):
    import all_reduce_reduction_rank_amd as ar

    case = state["case"]
    x, wg, wu, wd = (state[k] for k in ("x", "w_gate", "w_up", "w_down"))
    if not case["train"]:
        return {"out": ar.gated_ffn(x, wg, wu, wd, act=case["act"])}
    shape = (case["rows"], case["size"])
    gate = [torch.empty(shape, dtype=torch.float32, device=t.device) for t in x]
    up = [torch.empty(shape, dtype=torch.float32, device=t.device) for t in x]
    out = ar.gated_ffn(x, wg, wu, wd, gate=gate, up=up, act=case["act"])
    dx, dwg, dwu, dwd = ar.gated_ffn_backward(state["dout"], x, wg, wu, wd, gate, up, act=case["act"])
    return {"out": out, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}


def _own_xent(state):
    import all_reduce_reduction_rank_amd as ar

    x, w, target = state["x"], state["w"], state["target"]
    loss, lse = ar.linear_cross_entropy(x, w, target)
    res = {"loss": loss, "lse": lse}
    if state["case"]["train"]:
        res["dx"], res["dw"] = ar.linear_cross_entropy_backward(state["grad_loss"], x, w, target, lse)
    return res


def run(state):
    if state["case"]["op"] == "ffn":
        return _own_ffn(state) if own else _plain_ffn(state)
    return _own_xent(state) if own else _plain_xent(state)


def work(case):
    """Inputs read once, outputs written once; the products of the formulas
    (the backward pass counts 2 products per forward product)."""
    n, t, h, s = case["ranks"], case["rows"], case["hidden"], case["size"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "ffn":
        nbytes = n * (2 * t * h + 3 * h * s) * es
        flops = 6.0 * n * t * h * s
        if case["train"]:
            nbytes += n * (2 * t * h + 3 * h * s) * es
            flops *= 3
    else:
        nbytes = (n * t * h + h * s) * es + 8 * t + 8 * n * t
        flops = 2.0 * t * h * s
        if case["train"]:
            nbytes += (n * t * h + h * s) * es + 4 * t
            flops *= 3
    return {"bytes": nbytes, "flops": flops}


# ---- definitions in 64 bits ----


def _exact_act(z, act):
    if act == "silu":
        sig = torch.sigmoid(z)
        return z * sig, sig + z * sig * torch.sigmoid(-z)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / 2.0 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) / (2.0 * math.pi) ** 0.5
    inner = (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
    slope = (2.0 / math.pi) ** 0.5 * (1.0 + 0.134145 * z ** 2)
    th = torch.tanh(inner)
    return z * (1.0 + th) / 2, (1.0 + th) / 2 + z * slope * (1.0 - th.square()) / 2


def exact(case, seed):
    """The operators' definitions, row block by row block, in fp64."""
    state = prepare(case, seed)
    n, rows = case["ranks"], case["rows"]
    f64 = torch.float64
    if case["op"] == "ffn":
        names = ["out"] + (["dx", "dw_gate", "dw_up", "dw_down"] if case["train"] else [])
        res = {k: [] for k in names}
        for r in range(n):
            x = state["x"][r].to(f64)
            wg, wu, wd = (state[k][r].to(f64) for k in ("w_gate", "w_up", "w_down"))
            gate, up = torch.mm(x, wg.t()), torch.mm(x, wu.t())
            value, slope = _exact_act(gate, case["act"])
            res["out"].append(torch.mm(value * up, wd.t()))
            if case["train"]:
                dout = state["dout"][r].to(f64)
                dhid = torch.mm(dout, wd)
                dgate, dup = dhid * up * slope, dhid * value
                res["dx"].append(torch.mm(dgate, wg) + torch.mm(dup, wu))
                res["dw_gate"].append(torch.mm(dgate.t().contiguous(), x))
                res["dw_up"].append(torch.mm(dup.t().contiguous(), x))
                res["dw_down"].append(torch.mm(dout.t().contiguous(), value * up))
        return res
    shards = _shards(case)
    starts = [sum(shards[:r]) for r in range(n)]
    whole = torch.cat(state["w"]).to(f64)
    target = state["target"]
    valid = (target >= 0) & (target < case["size"])
    x = state["x"][0].to(f64)
    loss = torch.zeros(rows, dtype=f64, device=x.device)
    lse = torch.zeros(rows, dtype=f64, device=x.device)
    if case["train"]:
        dx = [torch.zeros_like(x) for _ in range(n)]
        dw = torch.zeros_like(whole)
    for i in range(0, rows, 1024):
        j = min(rows, i + 1024)
        z = torch.mm(x[i:j], whole.t())
        logp = torch.log_softmax(z, dim=1)
        lse[i:j] = torch.logsumexp(z, dim=1)
        ok = valid[i:j]
        pick = target[i:j].clamp(0, case["size"] - 1)[:, None]
        loss[i:j] = torch.where(ok, -logp.gather(1, pick)[:, 0], torch.zeros_like(loss[i:j]))
        if case["train"]:
            d = logp.exp()
            d.scatter_add_(1, pick, torch.full_like(pick, -1, dtype=f64))
            d *= torch.where(ok, state["grad_loss"][i:j].to(f64), torch.zeros_like(loss[i:j]))[:, None]
            for r in range(n):
                a, b = starts[r], starts[r] + shards[r]
                dx[r][i:j] = torch.mm(d[:, a:b].contiguous(), whole[a:b])
            dw += torch.mm(d.t().contiguous(), x[i:j])
    res = {"loss": [loss] * n, "lse": [lse] * n}
    if case["train"]:
        res["dx"] = dx
        res["dw"] = [dw[starts[r]:starts[r] + shards[r]] for r in range(n)]
    return res
