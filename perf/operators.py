"""Cases for the products at original precision (grouped by expert, and dense
with an epilogue) and for token sampling.

``run`` computes the operators in elementary torch operations in 32 bits (64
for sampling) when ``own`` is false, and calls ``bit_routed_moe_amd`` when it
is true.  ``exact`` gives the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------------------------------

def _grouped(name, dir, dtype, T, k, E, K, N, act, gather, bias=False, skew=0.0, save=False):
    return {"name": name, "op": "grouped", "dir": dir, "dtype": dtype, "T": T, "k": k, "E": E, "K": K, "N": N,
            "act": act, "gather": gather, "bias": bias, "skew": skew, "save": save}


def _linear(name, dir, dtype, M, K, N, act, bias, residual, save=False):
    return {"name": name, "op": "linear", "dir": dir, "dtype": dtype, "M": M, "K": K, "N": N, "act": act,
            "bias": bias, "residual": residual, "save": save}


def _sample(name, dtype, B, V, std, mix, masked):
    return {"name": name, "op": "sample", "dtype": dtype, "B": B, "V": V, "std": std, "mix": mix, "masked": masked}


def listed():
    return [
        # one token's gate/up products over bf16 experts (the 7168/2048, 256-expert, top-8 layer): latency of decode
        _grouped("grouped_decode_up", "fwd", "bf16", 1, 8, 256, 7168, 4096, "swiglu", True),
        # a 4096-token chunk's down products of the same layer, ragged by a skewed router: prefill
        _grouped("grouped_prefill_down", "fwd", "bf16", 4096, 8, 256, 2048, 7168, "none", False, skew=0.6),
        # the gate/up products' gradients on one of eight expert shards (32 experts), a training microbatch
        _grouped("grouped_train_up_bwd", "bwd", "bf16", 2048, 4, 32, 7168, 4096, "swiglu", True, skew=0.4),
        # the tiny layer in fp32 mode with biases, forward: a parity run, or a test model
        _grouped("grouped_tiny_f32", "fwd", "f32", 16, 2, 8, 256, 128, "silu", True, bias=True),
        # odd widths in fp32 mode, gradients: a small model trained at full precision
        _grouped("grouped_odd_f32_bwd", "bwd", "f32", 301, 3, 7, 459, 331, "gelu", True, bias=True, skew=0.5),
        # one token through a square projection with residual: the smallest serving call
        _linear("linear_decode", "fwd", "bf16", 1, 7168, 7168, "none", True, True),
        # output head for a batch of decoding sessions: logits over a large vocabulary
        _linear("linear_head", "fwd", "bf16", 16, 7168, 131072, "none", False, False),
        # dense SwiGLU FFN up-projection of a 4096-token chunk, pre-activations kept for training
        _linear("linear_train_up", "fwd", "bf16", 4096, 7168, 4096, "swiglu", True, False, save=True),
        # an ordinary layer's gradients (input, weights, bias) over a 4096-token microbatch
        _linear("linear_train_bwd", "bwd", "bf16", 4096, 7168, 2048, "gelu_tanh", True, False),
        # one session's next token, everything switched on: latency of serving
        _sample("sample_one", "f32", 1, 131072, 3.0, "all", False),
        # a serving batch with every session's own settings, a grammar masking some rows' tokens
        _sample("sample_batch", "f32", 64, 131072, 2.5, "mixed", True),
        # a large batch over a smaller odd vocabulary with bf16 logits and flat distributions (top-p alone)
        _sample("sample_wide_bf16", "bf16", 256, 50003, 1.0, "topp", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "linear", "linear", "sample"])
    if op == "grouped":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        E = _log(rng, 2, 64)
        k = rng.randint(1, min(E, 8))
        big = 4096 if dtype == "bf16" else 700
        T = _log(rng, 1, big)
        K, N = _log(rng, 64, big), _log(rng, 64, big)
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
        if act == "swiglu":
            N += N % 2
        return _grouped("", rng.choice(["fwd", "bwd"]), dtype, T, k, E, K, N, act, rng.random() < 0.7,
                        bias=rng.random() < 0.5, skew=rng.uniform(0.0, 1.0), save=rng.random() < 0.5)
    if op == "linear":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        big = 8192 if dtype == "bf16" else 1500
        M = _log(rng, 1, 4096 if dtype == "bf16" else 1000)
        K, N = _log(rng, 64, big), _log(rng, 64, big)
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
        if act == "swiglu":
            N += N % 2
        return _linear("", rng.choice(["fwd", "fwd", "bwd"]), dtype, M, K, N, act, rng.random() < 0.6,
                       rng.random() < 0.5, save=rng.random() < 0.5)
    return _sample("", rng.choice(["f32", "bf16"]), _log(rng, 1, 256), _log(rng, 200, 131072), rng.uniform(0.5, 5.0),
                   rng.choice(["all", "mixed", "topp", "greedy"]), rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------------------------------------------

def _pad(n, dtype):
    """Row stride in elements: rows start at 16-byte boundaries."""
    q = 8 if dtype == "bf16" else 4
    return (n + q - 1) // q * q


def _rows(g, n, cols, dtype, scale=1.0):
    """[n][cols] normal values, rows at 16-byte boundaries."""
    t = torch.empty(n, _pad(cols, dtype), dtype=DT[dtype], device="cuda").normal_(0.0, scale, generator=g)
    return t[:, :cols]


def _empty(n, cols, dtype):
    return torch.empty(n, _pad(cols, dtype), dtype=DT[dtype], device="cuda")[:, :cols]


def _out_cols(c):
    return c["N"] // 2 if c["act"] == "swiglu" else c["N"]


def _route(c, seed):
    """Distinct experts for each token under a skewed router, and the pairs by expert (tokens ascending): the
    permutation that the layer makes from a router's choice."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    T, k, E = c["T"], c["k"], c["E"]
    bias = -c["skew"] * torch.log(1.0 + torch.randperm(E, generator=g).float())
    gumbel = -torch.log(-torch.log(torch.rand(T, E, generator=g).clamp_(1e-9, 1 - 1e-7)))
    idx = torch.topk(bias + gumbel, k, dim=1).indices
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return offsets, order


def _matmul_state(c, s):
    """The framework's handle and workspace for the case's product."""
    import bit_routed_moe_amd as ds4
    bwd = c["dir"] == "bwd"
    m = ds4.make_matmul(c["K"], c["N"], groups=c.get("E", 1), dtype=c["dtype"], act=c["act"], grad=c["dtype"],
                        ldx=_pad(c["K"], c["dtype"]), ldw=_pad(c["K"], c["dtype"]),
                        ldy=_pad(_out_cols(c), c["dtype"]), ldz=_pad(c["N"], c["dtype"]))
    s["m"] = m
    n = ds4.matmul_workspace_bytes(m, s["rows"], backward=bwd)
    s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


def _prepare_product(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    K, N, dt = c["K"], c["N"], c["dtype"]
    grouped = c["op"] == "grouped"
    s = {"case": c}
    if grouped:
        E, k = c["E"], c["k"]
        offsets, order = _route(c, seed)
        rows = c["T"] * k
        s["host_offsets"] = offsets.tolist()
        s["offsets"] = offsets.cuda()
        s["sorted_pair"] = order.cuda() if c["gather"] else None
        x = _rows(g, c["T"] if c["gather"] else rows, K, dt)
    else:
        E, rows = 1, c["M"]
        s["host_offsets"] = [0, rows]
        x = _rows(g, rows, K, dt)
    s["rows"], s["x"] = rows, x
    w = torch.empty(E, N, _pad(K, dt), dtype=DT[dt], device="cuda")
    for e in range(E):
        w[e].normal_(0.0, K ** -0.5, generator=g)
    s["w"] = w[:, :, :K]
    s["bias"] = (torch.empty(E, N, device="cuda").normal_(0.0, 0.1, generator=g).to(DT[dt]) if c["bias"] else None)
    oc = _out_cols(c)
    if c["dir"] == "fwd":
        s["residual"] = _rows(g, rows, oc, dt) if c.get("residual") else None
        s["y"] = _empty(rows, oc, dt)
        s["z"] = _empty(rows, N, dt) if c["save"] else None
    else:
        s["dy"] = _rows(g, rows, oc, dt)
        s["z"] = None
        if c["act"] != "none":     # the forward pass's pre-activations
            s["z"] = _empty(rows, N, dt)
            s["z"].copy_(_rows(g, rows, N, dt))
        s["dx"] = _empty(rows, K, dt)
        s["dw"] = torch.empty(E, N, _pad(K, dt), dtype=DT[dt], device="cuda")[:, :, :K]
        s["dbias"] = torch.empty(E, N, dtype=DT[dt], device="cuda") if c["bias"] else None
    if own:
        _matmul_state(c, s)
    return s


def _prepare_sample(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator(device="cpu").manual_seed(seed)
    B, V = c["B"], c["V"]
    logits = torch.empty(B, V, device="cuda").normal_(0.0, c["std"], generator=g)
    if c["masked"]:     # a grammar leaves every other row a fifth of its tokens
        drop = torch.rand(B, V, device="cuda", generator=g) < 0.8
        drop[::2] = False
        drop[:, 0] = False
        logits.masked_fill_(drop, float("-inf"))
    s = {"case": c, "logits": logits.to(DT[c["dtype"]])}
    u = torch.rand(B, generator=h)
    temp = 0.3 + 1.2 * torch.rand(B, generator=h)
    top_k = torch.randint(1, 200, (B,), generator=h, dtype=torch.int32)
    top_p = 0.5 + 0.5 * torch.rand(B, generator=h)
    min_p = 0.1 * torch.rand(B, generator=h)
    if c["mix"] == "mixed":      # 0, 1 and 0 switch a filter off; temperature 0 is the greedy choice
        r = torch.randint(0, 4, (4, B), generator=h)
        temp[r[0] == 0] = 0.0
        top_k[r[1] >= 2] = 0
        top_p[r[2] >= 2] = 1.0
        min_p[r[3] >= 2] = 0.0
    if c["mix"] == "greedy":
        temp.zero_()
    if c["mix"] == "topp":
        temp.fill_(1.0)
        top_k.zero_()
        top_p.fill_(0.9)
        min_p.zero_()
    for n, t in (("u", u), ("temperature", temp), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p)):
        s[n] = t.cuda()
    s["token"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["prob"] = torch.empty(B, dtype=torch.float32, device="cuda")
    if own:
        import bit_routed_moe_amd as ds4
        s["ws"] = torch.empty(ds4.sample_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    return _prepare_sample(case, seed) if case["op"] == "sample" else _prepare_product(case, seed)


# ---- the framework's calls -------------------------------------------------------------------------------------

def _run_own(s):
    import bit_routed_moe_amd as ds4
    c = s["case"]
    if c["op"] == "sample":
        ds4.sample(c["B"], c["V"], s["logits"], s["u"], s["token"], temperature=s["temperature"], top_k=s["top_k"],
                   top_p=s["top_p"], min_p=s["min_p"], prob=s["prob"], workspace=s["ws"])
        return [s["token"], s["prob"]]
    if c["op"] == "linear":
        if c["dir"] == "fwd":
            ds4.linear(s["m"], s["rows"], s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"], z=s["z"],
                       workspace=s["ws"])
        else:
            ds4.linear_backward(s["m"], s["rows"], s["x"], s["w"], s["dy"], z=s["z"], dx=s["dx"], dw=s["dw"],
                                dbias=s["dbias"], workspace=s["ws"])
    else:
        at = {"sorted_pair": s["sorted_pair"], "top_k": c["k"], "x_rows": s["x"].shape[0]}
        if c["dir"] == "fwd":
            ds4.grouped_matmul(s["m"], s["rows"], s["x"], s["w"], s["offsets"], s["y"], bias=s["bias"], z=s["z"],
                               workspace=s["ws"], **at)
        else:
            ds4.grouped_matmul_backward(s["m"], s["rows"], s["x"], s["w"], s["offsets"], s["dy"], z=s["z"],
                                        dx=s["dx"], dw=s["dw"], dbias=s["dbias"], workspace=s["ws"], **at)
    if c["dir"] == "fwd":
        return [s["y"]] + ([s["z"]] if c["save"] else [])
    return [s["dx"], s["dw"]] + ([s["dbias"]] if c["bias"] else [])


# ---- the plain form --------------------------------------------------------------------------------------------

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    n = z.shape[1] // 2
    a, b = z[:, :n], z[:, n:]
    return a / (1 + torch.exp(-a)) * b


def _act_grad(dy, z, act):
    """dz = dy * act'(z)."""
    if act == "none":
        return dy
    if act == "relu":
        return dy * (z > 0)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return dy * (p * (1 + z * (1 - p)))
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5)
    if act == "gelu_tanh":
        r = (2 / math.pi) ** 0.5
        t = torch.tanh(r * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * r * (1 + 3 * 0.044715 * z * z))
    n = z.shape[1] // 2
    a, b = z[:, :n], z[:, n:]
    p = 1 / (1 + torch.exp(-a))
    return torch.cat([dy * b * (p * (1 + a * (1 - p))), dy * a * p], dim=1)


def _plain_product(s):
    c = s["case"]
    off, x, w = s["host_offsets"], s["x"], s["w"]
    E, fwd, out = len(off) - 1, c["dir"] == "fwd", DT[c["dtype"]]
    gather = c["op"] == "grouped" and c["gather"]
    if gather:
        x = x[(s["sorted_pair"] // c["k"]).long()]
    if fwd:
        y = torch.empty(s["rows"], _out_cols(c), dtype=out, device="cuda")
        zs = torch.empty(s["rows"], c["N"], dtype=out, device="cuda") if c["save"] else None
    else:
        dx = torch.empty(s["rows"], c["K"], dtype=out, device="cuda")
        dw = torch.zeros(E, c["N"], c["K"], dtype=out, device="cuda")
        db = torch.zeros(E, c["N"], dtype=out, device="cuda") if c["bias"] else None
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        xe, we = x[a:b].float(), w[e].float()
        if fwd:
            z = xe @ we.t()
            if s["bias"] is not None:
                z = z + s["bias"][e].float()
            v = _act(z, c["act"])
            if s["residual"] is not None:
                v = v + s["residual"][a:b].float()
            y[a:b] = v
            if c["save"]:
                zs[a:b] = z
        else:
            dz = _act_grad(s["dy"][a:b].float(), None if s["z"] is None else s["z"][a:b].float(), c["act"])
            dx[a:b] = dz @ we
            dw[e] = dz.t() @ xe
            if c["bias"]:
                db[e] = dz.sum(0)
    if fwd:
        return [y] + ([zs] if c["save"] else [])
    return [dx, dw] + ([db] if c["bias"] else [])


def _plain_sample(s):
    """Rows sorted by logit descending (ties: lower index first), the three filters as prefixes of that order, and
    the first token whose running sum of weights exceeds u times the kept sum; in 64 bits, as borders matter."""
    l = s["logits"].double()
    B, V = l.shape
    v, at = torch.sort(l, dim=1, descending=True, stable=True)
    t = s["temperature"].double()
    greedy = t <= 0
    w = torch.exp((v - v[:, :1]) / torch.where(greedy, torch.ones_like(t), t)[:, None])
    pos = torch.arange(V, device="cuda")[None, :]
    k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
    w = w * (pos < k)
    c = torch.cumsum(w, dim=1)
    p = s["top_p"].double()[:, None]
    keep = (p >= 1) | (c - w < p * c[:, -1:]) | (pos == 0)
    w = w * (keep & ((w >= s["min_p"].double()[:, None]) | (pos == 0)))
    w = w * ((pos == 0) | ~greedy[:, None])
    c = torch.cumsum(w, dim=1)
    total = c[:, -1:]
    first = torch.argmax((c > s["u"].double()[:, None] * total).int(), dim=1, keepdim=True)
    return [at.gather(1, first)[:, 0].int(), (w.gather(1, first) / total)[:, 0].float()]


def run(state):
    if own:
        return _run_own(state)
    return _plain_sample(state) if state["case"]["op"] == "sample" else _plain_product(state)


# ---- what a pass cannot do without -----------------------------------------------------------------------------

def _active(c):
    """Experts that are expected to have rows."""
    q = [(1.0 + i) ** -c["skew"] for i in range(c["E"])]
    t = sum(q)
    return sum(1.0 - (1.0 - min(1.0, c["k"] * p / t)) ** c["T"] for p in q)


def work(case):
    c = case
    if c["op"] == "sample":
        n = c["B"] * c["V"]
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + c["B"] * 28, "flops": 4 * n}
    eb = 2 if c["dtype"] == "bf16" else 4
    K, N, oc = c["K"], c["N"], _out_cols(c)
    if c["op"] == "grouped":
        rows, E, live = c["T"] * c["k"], c["E"], _active(c)
        xr = c["T"] if c["gather"] else rows
    else:
        rows, E, live, xr = c["M"], 1, 1, c["M"]
    if c["dir"] == "fwd":
        b = xr * K + live * N * K + rows * oc + (rows * N if c["save"] else 0) + (live * N if c["bias"] else 0)
        b += rows * oc if c.get("residual") else 0
        return {"bytes": int(eb * b), "flops": 2 * rows * K * N}
    b = xr * K + live * N * K + rows * oc + (rows * N if c["act"] != "none" else 0) + rows * K + E * N * K
    b += E * N if c["bias"] else 0
    return {"bytes": int(eb * b), "flops": 4 * rows * K * N}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------

def _exact_act(z, act):
    if act == "none":
        return z.clone()
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    a, b = z.chunk(2, dim=1)
    return a * torch.sigmoid(a) * b


def _exact_product(s):
    c = s["case"]
    grouped, fwd = c["op"] == "grouped", c["dir"] == "fwd"
    bounds = s["host_offsets"]
    src = (torch.div(s["sorted_pair"].long(), c["k"], rounding_mode="floor") if grouped and c["gather"]
           else torch.arange(s["rows"], device="cuda"))
    parts = [[], [], []]
    for e, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        x, w = s["x"].double()[src[a:b]] if c["op"] == "linear" else s["x"][src[a:b]].double(), s["w"][e].double()
        if fwd:
            z = torch.matmul(x, w.t())
            z = z if s["bias"] is None else z + s["bias"][e].double()
            y = _exact_act(z, c["act"])
            parts[0].append(y if s["residual"] is None else y + s["residual"][a:b].double())
            parts[1].append(z)
        else:
            dy = s["dy"][a:b].double()
            if c["act"] == "none":
                dz = dy
            else:       # the activation's derivative, by differentiating its definition
                z = s["z"][a:b].double().requires_grad_()
                dz, = torch.autograd.grad(_exact_act(z, c["act"]), z, dy)
                if c["act"] == "relu":
                    dz = torch.where(z.detach() > 0, dz, torch.zeros_like(dz))
            parts[0].append(torch.matmul(dz, w))
            parts[1].append(torch.matmul(dz.t(), x)[None])
            parts[2].append(dz.sum(dim=0)[None])
    if fwd:
        return [torch.cat(parts[0])] + ([torch.cat(parts[1])] if c["save"] else [])
    return [torch.cat(parts[0]), torch.cat(parts[1])] + ([torch.cat(parts[2])] if c["bias"] else [])


def _exact_sample(s):
    """Row by row: the kept set is built from the definition, then walked to the running sum."""
    tokens, probs = [], []
    c = s["case"]
    for r in range(c["B"]):
        l = s["logits"][r].double()
        T, k, p, q = (float(s[n][r]) for n in ("temperature", "top_k", "top_p", "min_p"))
        order = torch.argsort(-l, stable=True)
        if T <= 0:
            tokens.append(int(order[0]))
            probs.append(1.0)
            continue
        z = l[order] / T
        if k > 0:
            z = z[: int(k)]
        w = torch.softmax(z, 0)
        if p < 1:
            n = int((torch.cumsum(w, 0) < p).sum()) + 1     # the shortest prefix that reaches p
            w = w[:n]
        w = w[: max(1, int((w >= q * w[0]).sum()))]
        run_sum = torch.cumsum(w, 0) / w.sum()
        i = min(int((run_sum <= float(s["u"][r])).sum()), w.numel() - 1)
        tokens.append(int(order[i]))
        probs.append(float(w[i] / w.sum()))
    return [torch.tensor(tokens, dtype=torch.int32, device="cuda"),
            torch.tensor(probs, dtype=torch.float64, device="cuda")]


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_sample(s) if case["op"] == "sample" else _exact_product(s)
