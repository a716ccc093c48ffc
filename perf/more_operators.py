"""Cases for tokens sorted by expert and back (with weights, dropped pairs and
gradients), for products in 8-bit integers with a scale for each token and
channel, and for penalties, biases and grammar masks on logits.

``run`` computes the operators in elementary torch operations when ``own`` is
false, and calls ``bit_routed_moe_amd`` when it is true.  ``exact`` gives the
same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------------------------------

def _tokens(name, op, dir, dtype, T, k, E, H, weighted, layout="sorted", base=False, skew=0.3):
    return {"name": name, "op": op, "dir": dir, "dtype": dtype, "T": T, "k": k, "E": E, "H": H, "weighted": weighted,
            "layout": layout, "base": base, "skew": skew}


def _linear8(name, dtype, M, K, N, act, bias, residual):
    return {"name": name, "op": "linear8", "dtype": dtype, "M": M, "K": K, "N": N, "act": act, "bias": bias,
            "residual": residual}


def _grouped8(name, dtype, T, k, E, K, N, act, gather, bias=False, skew=0.0):
    return {"name": name, "op": "grouped8", "dtype": dtype, "T": T, "k": k, "E": E, "K": K, "N": N, "act": act,
            "gather": gather, "bias": bias, "skew": skew}


def _logits(name, dtype, out, B, V, history, repetition, counts, bias, mask):
    return {"name": name, "op": "logits", "dtype": dtype, "out": out, "B": B, "V": V, "history": history,
            "repetition": repetition, "counts": counts, "bias": bias, "mask": mask}


def listed():
    return [
        # a 4096-token chunk's rows laid out by expert (the 7168-wide, 256-expert, top-8 layer): prefill
        _tokens("dispatch_prefill", "dispatch", "fwd", "bf16", 4096, 8, 256, 7168, False),
        # gradients of weighted rows with a fixed capacity for each expert (some pairs dropped, some rows empty), odd
        # width, fp32: a small model trained at full precision
        _tokens("dispatch_odd_f32_bwd", "dispatch", "bwd", "f32", 1501, 3, 24, 459, True, layout="capacity"),
        # decoding sessions' expert outputs back to their tokens, the shared expert's added: latency of serving
        _tokens("collect_decode", "collect", "fwd", "bf16", 16, 8, 256, 7168, True, base=True),
        # a training microbatch: gradients of the experts' rows, of the router's weights and of its logits
        _tokens("collect_train_bwd", "collect", "bwd", "bf16", 2048, 8, 256, 7168, True),
        # one token through a square projection with residual: the smallest serving call
        _linear8("linear8_decode", "bf16", 1, 7168, 7168, "none", True, True),
        # the gate/up projection of a 4096-token chunk: prefill
        _linear8("linear8_prefill", "bf16", 4096, 7168, 4096, "swiglu", False, False),
        # odd sizes with fp32 rows: a test model
        _linear8("linear8_odd_f32", "f32", 301, 1459, 331, "gelu", True, False),
        # one token's gate/up products of 8 experts of 256: latency of decode
        _grouped8("grouped8_decode_up", "bf16", 1, 8, 256, 7168, 4096, "swiglu", True),
        # a 4096-token chunk's down products of the same layer, ragged by a skewed router: prefill
        _grouped8("grouped8_prefill_down", "bf16", 4096, 8, 256, 2048, 7168, "none", False, skew=0.6),
        # one session's next token, everything switched on, a long conversation behind it: latency of serving
        _logits("logits_one", "f32", "f32", 1, 131072, 8000, True, True, 100, True),
        # a serving batch, conversations of every length, half of them under a grammar
        _logits("logits_batch", "f32", "f32", 64, 131072, 4000, True, True, 30, True),
        # a large batch over a smaller odd vocabulary, bf16 logits to fp32, counts alone
        _logits("logits_wide_bf16", "bf16", "f32", 256, 50003, 700, False, True, 0, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tokens", "tokens", "linear8", "grouped8", "logits"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
    if op == "tokens":
        k = rng.randint(1, 8)
        return _tokens("", rng.choice(["dispatch", "collect"]), rng.choice(["fwd", "bwd"]), dtype, _log(rng, 1, 4096),
                       k, _log(rng, max(k, 2), 256), _log(rng, 64, 7168 if dtype == "bf16" else 3600),
                       rng.random() < 0.7, layout=rng.choice(["sorted", "sorted", "capacity"]),
                       base=rng.random() < 0.5, skew=rng.uniform(0.0, 1.0))
    if op == "linear8":
        N = _log(rng, 64, 8192)
        return _linear8("", dtype, _log(rng, 1, 4096), _log(rng, 64, 8192), N + N % 2 if act == "swiglu" else N, act,
                        rng.random() < 0.5, rng.random() < 0.5)
    if op == "grouped8":
        E = _log(rng, 2, 64)
        N = _log(rng, 64, 4096)
        return _grouped8("", dtype, _log(rng, 1, 4096), rng.randint(1, min(E, 8)), E, _log(rng, 64, 4096),
                         N + N % 2 if act == "swiglu" else N, act, rng.random() < 0.6, bias=rng.random() < 0.5,
                         skew=rng.uniform(0.0, 1.0))
    lt = rng.choice(["f32", "f32", "bf16"])
    return _logits("", lt, rng.choice([lt, "f32"]), _log(rng, 1, 256), _log(rng, 200, 131072), _log(rng, 1, 8000),
                   rng.random() < 0.7, rng.random() < 0.7, rng.choice([0, 0, 5, 100]), rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------------------------------------------

def _pad(n, dtype):
    """Row stride in elements: rows start at 16-byte boundaries."""
    q = {"bf16": 8, "f32": 4, "i8": 16}[dtype]
    return (n + q - 1) // q * q


def _rows(g, n, cols, dtype, scale=1.0):
    """[n][cols] normal values, rows at 16-byte boundaries."""
    t = torch.empty(n, _pad(cols, dtype), dtype=DT[dtype], device="cuda").normal_(0.0, scale, generator=g)
    return t[:, :cols]


def _empty(n, cols, dtype):
    return torch.empty(n, _pad(cols, dtype), dtype=DT[dtype], device="cuda")[:, :cols]


def _route(c, seed):
    """Distinct experts for each token under a skewed router, their weights, and the pairs by expert (tokens
    ascending): what the layer's route and permute give."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    T, k, E = c["T"], c["k"], c["E"]
    bias = -c["skew"] * torch.log(1.0 + torch.randperm(E, generator=g).float())
    logits = bias - torch.log(-torch.log(torch.rand(T, E, generator=g).clamp_(1e-9, 1 - 1e-7)))
    top = torch.topk(logits, k, dim=1)
    flat = top.indices.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    count = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64)
    offsets[1:] = count.cumsum(0)
    pos = torch.empty(T * k, dtype=torch.int64)
    pos[order] = torch.arange(T * k)
    return top.indices.int(), torch.softmax(top.values, 1), offsets, order, pos, flat


def _prepare_tokens(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, k, H, dt = c["T"], c["k"], c["H"], c["dtype"]
    idx, w, offsets, order, pos, flat = _route(c, seed)
    rows = T * k
    if c["layout"] == "capacity":   # a fixed number of rows for each expert: what is over is dropped, the rest empty
        cap = max(1, rows // c["E"])
        slot = pos - offsets[flat]
        pos = torch.where(slot < cap, flat * cap + slot, torch.full_like(pos, -1))
        rows = c["E"] * cap
        order = torch.full((rows,), -1, dtype=torch.int64)
        kept = pos >= 0
        order[pos[kept]] = torch.arange(T * k)[kept]
    s = {"case": c, "rows": rows, "pair_pos": pos.int().cuda(), "sorted_pair": order.int().cuda(),
         "topk_idx": idx.cuda(), "topk_w": w.float().cuda() if c["weighted"] else None}
    token, sorted_rows = _rows(g, T, H, dt), _rows(g, rows, H, dt)
    if c["op"] == "dispatch":
        s["x"] = token
        if c["dir"] == "fwd":
            s["out"] = _empty(rows, H, dt)
        else:
            s["dout"] = sorted_rows
            s["dx"] = _empty(T, H, dt)
    else:
        s["expert_rows"] = sorted_rows
        if c["dir"] == "fwd":
            s["base"] = token if c["base"] else None
            s["y"] = _empty(T, H, dt)
        else:
            s["dy"] = token
            s["drows"] = _empty(rows, H, dt)
            s["dlogits"] = torch.empty(T, c["E"], device="cuda")
    s["dtopk_w"] = torch.empty(T, k, device="cuda") if c["dir"] == "bwd" and c["weighted"] else None
    if own:
        import bit_routed_moe_amd as ds4
        s["d"] = ds4.make_rows(H, k, dtype=dt, ldx=_pad(H, dt), ldr=_pad(H, dt))
        s["cfg"] = ds4.make_config(256, 128, c["E"], k)
    return s


def _codes(w):
    """Codes and scales of rows of weights: done once, when a model is loaded."""
    scale = w.abs().amax(dim=-1) / 127
    return torch.round(w / scale[..., None]).to(torch.int8), scale


def _prepare_product(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    K, N, dt = c["K"], c["N"], c["dtype"]
    s = {"case": c, "sorted_pair": None}
    if c["op"] == "grouped8":
        E = c["E"]
        _, _, offsets, order, _, _ = _route(c, seed)
        rows = c["T"] * c["k"]
        xr = c["T"] if c["gather"] else rows
        s["host_offsets"] = offsets.tolist()
        s["offsets"] = offsets.int().cuda()
        s["sorted_pair"] = order.int().cuda() if c["gather"] else None
    else:
        E, rows, xr = 1, c["M"], c["M"]
        s["host_offsets"] = [0, rows]
    s["rows"], s["x"] = rows, _rows(g, xr, K, dt)
    codes = torch.zeros(E, N, _pad(K, "i8"), dtype=torch.int8, device="cuda")
    s["w_scale"] = torch.empty(E, N, device="cuda")
    for e in range(E):
        codes[e, :, :K], s["w_scale"][e] = _codes(torch.empty(N, K, device="cuda").normal_(0.0, K ** -0.5, generator=g))
    s["w"] = codes[:, :, :K]
    oc = N // 2 if c["act"] == "swiglu" else N
    s["bias"] = torch.empty(E, N, device="cuda").normal_(0.0, 0.1, generator=g).to(DT[dt]) if c["bias"] else None
    s["residual"] = _rows(g, rows, oc, dt) if c.get("residual") else None
    s["y"] = _empty(rows, oc, dt)
    s["xq"] = torch.empty(xr, _pad(K, "i8"), dtype=torch.int8, device="cuda")[:, :K]
    s["x_scale"] = torch.empty(xr, device="cuda")
    if own:
        import bit_routed_moe_amd as ds4
        m = ds4.make_matmul_int8(K, N, groups=E, dtype=dt, act=c["act"], ldx=_pad(K, "i8"), ldw=_pad(K, "i8"),
                                 ldy=_pad(oc, dt))
        s["m"] = m
        s["ws"] = torch.empty(max(16, ds4.matmul_int8_workspace_bytes(m, rows)), dtype=torch.uint8, device="cuda")
    return s


def _prepare_logits(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator(device="cpu").manual_seed(seed)
    B, V = c["B"], c["V"]
    s = {"case": c, "logits": torch.empty(B, V, device="cuda").normal_(0.0, 3.0, generator=g).to(DT[c["dtype"]])}
    s["out"] = torch.empty(B, V, dtype=DT[c["out"]], device="cuda")
    # conversations of every length up to `history`, their prompts first; frequent tokens come often
    L = c["history"]
    n = torch.randint(0, L + 1, (B,), generator=h)
    n[0] = L
    offsets = torch.zeros(B + 1, dtype=torch.int64)
    offsets[1:] = n.cumsum(0)
    total = int(offsets[-1])
    tokens = (V * torch.rand(max(total, 1), generator=h).pow(4)).long().clamp_(max=V - 1)
    s["history"], s["history_offsets"] = tokens.int().cuda(), offsets.int().cuda()
    s["prompt_len"] = (n * torch.rand(B, generator=h)).int().cuda()
    s["n_history"] = total
    s["repetition"] = (1.0 + 0.5 * torch.rand(B, generator=h)).cuda() if c["repetition"] else None
    s["presence"] = (1.5 * torch.rand(B, generator=h)).cuda() if c["counts"] else None
    s["frequency"] = (0.7 * torch.rand(B, generator=h)).cuda() if c["counts"] else None
    s["bias_token"] = s["bias_value"] = s["bias_offsets"] = s["mask"] = s["mask_row"] = None
    if c["bias"]:   # up to `bias` tokens of a row, some of them banned
        m = torch.randint(0, min(c["bias"], V) + 1, (B,), generator=h)
        off = torch.zeros(B + 1, dtype=torch.int64)
        off[1:] = m.cumsum(0)
        s["bias_offsets"] = off.int().cuda()
        step = V // min(c["bias"], V)
        i = torch.arange(max(int(off[-1]), 1))
        s["bias_token"] = (((i - off[torch.searchsorted(off, i, right=True).clamp_(max=B) - 1]) * step) % V).int().cuda()
        v = 5.0 * torch.randn(i.numel(), generator=h)
        v[torch.rand(i.numel(), generator=h) < 0.2] = float("-inf")
        s["bias_value"] = v.cuda()
        s["n_bias"] = int(off[-1])
    if c["mask"]:   # the states of a few grammars, for about half of the rows
        G = max(1, min(8, B))
        W = (V + 31) // 32
        bits = torch.randint(-2 ** 31, 2 ** 31, (G, W), generator=h, dtype=torch.int64)
        bits &= torch.randint(-2 ** 31, 2 ** 31, (G, W), generator=h, dtype=torch.int64)
        bits[torch.rand(G, W, generator=h) < 0.7] = 0
        s["mask"] = bits.int().cuda()
        row = torch.randint(0, G, (B,), generator=h)
        row[1::2] = -1
        s["mask_row"] = row.int().cuda()
    return s


def prepare(case, seed):
    if case["op"] in ("dispatch", "collect"):
        return _prepare_tokens(case, seed)
    return _prepare_logits(case, seed) if case["op"] == "logits" else _prepare_product(case, seed)


# ---- the framework's calls -------------------------------------------------------------------------------------

def _run_own(s):
    import bit_routed_moe_amd as ds4
    c = s["case"]
    op = c["op"]
    if op == "logits":
        ds4.adjust_logits(c["B"], c["V"], s["logits"], s["out"], history=s["history"],
                          history_offsets=s["history_offsets"], prompt_len=s["prompt_len"],
                          repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                          bias_token=s["bias_token"], bias_value=s["bias_value"], bias_offsets=s["bias_offsets"],
                          mask=s["mask"], mask_row=s["mask_row"])
        return [s["out"]]
    if op in ("linear8", "grouped8"):
        ds4.quantize_rows_int8(s["x"].shape[0], c["K"], s["x"], s["xq"], s["x_scale"])
        if op == "linear8":
            ds4.linear_int8(s["m"], s["rows"], s["xq"], s["x_scale"], s["w"], s["w_scale"], s["y"], bias=s["bias"],
                            residual=s["residual"], workspace=s["ws"])
        else:
            ds4.grouped_matmul_int8(s["m"], s["rows"], s["xq"], s["x_scale"], s["w"], s["w_scale"], s["offsets"],
                                    s["y"], sorted_pair=s["sorted_pair"], top_k=c["k"], x_rows=s["x"].shape[0],
                                    bias=s["bias"], workspace=s["ws"])
        return [s["y"]]
    d, T, rows, pos = s["d"], c["T"], s["rows"], s["pair_pos"]
    empty = s["sorted_pair"] if c["layout"] == "capacity" else None
    if op == "dispatch":
        if c["dir"] == "fwd":
            ds4.dispatch(d, T, rows, s["x"], pos, s["out"], topk_w=s["topk_w"], sorted_pair=empty)
            return [s["out"]]
        ds4.dispatch_backward(d, T, rows, s["dout"], pos, topk_w=s["topk_w"], x=s["x"], dx=s["dx"],
                              dtopk_w=s["dtopk_w"])
        return [s["dx"]] + ([s["dtopk_w"]] if c["weighted"] else [])
    if c["dir"] == "fwd":
        ds4.collect(d, T, rows, s["expert_rows"], pos, s["y"], topk_w=s["topk_w"], base=s["base"])
        return [s["y"]]
    ds4.collect_backward(d, T, rows, s["dy"], pos, expert_rows=s["expert_rows"], topk_w=s["topk_w"], sorted_pair=empty,
                         drows=s["drows"], dtopk_w=s["dtopk_w"])
    if not c["weighted"]:
        return [s["drows"]]
    ds4.route_backward(s["cfg"], T, s["topk_idx"], s["topk_w"], s["dtopk_w"], s["dlogits"])
    return [s["drows"], s["dtopk_w"], s["dlogits"]]


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


def _plain_tokens(s):
    c = s["case"]
    T, k, H, rows, dt = c["T"], c["k"], c["H"], s["rows"], DT[c["dtype"]]
    pos = s["pair_pos"].long()
    there = (pos >= 0).float()[:, None]
    w = s["topk_w"].reshape(-1, 1) if s["topk_w"] is not None else torch.ones(T * k, 1, device="cuda")

    def to_rows(x):         # the tokens' rows by expert, with their weights; empty rows are zero
        pair = s["sorted_pair"].long()
        full = (pair >= 0)[:, None]
        pair = pair.clamp(min=0)
        return torch.where(full, x.float()[pair // k] * w[pair], torch.zeros((), device="cuda")).to(dt)

    def of_pairs(r):        # the pairs' rows in the tokens' order; dropped pairs have none
        return r[pos.clamp(min=0)].float() * there

    if c["op"] == "dispatch":
        if c["dir"] == "fwd":
            return [to_rows(s["x"])]
        p = of_pairs(s["dout"])
        dx = (p * w).reshape(T, k, H).sum(1).to(dt)
        if not c["weighted"]:
            return [dx]
        return [dx, (p.reshape(T, k, H) * s["x"].float()[:, None]).sum(2)]
    if c["dir"] == "fwd":
        y = (of_pairs(s["expert_rows"]) * w).reshape(T, k, H).sum(1)
        return [(y if s["base"] is None else y + s["base"].float()).to(dt)]
    drows = to_rows(s["dy"])
    if not c["weighted"]:
        return [drows]
    dw = (of_pairs(s["expert_rows"]).reshape(T, k, H) * s["dy"].float()[:, None]).sum(2)
    tw = s["topk_w"]        # a softmax over the chosen logits
    dl = tw * (dw - (tw * dw).sum(1, keepdim=True))
    return [drows, dw, torch.zeros(T, c["E"], device="cuda").scatter_(1, s["topk_idx"].long(), dl)]


def _plain_product(s):
    """Codes by the nearest whole number (64 bits: values next to a border), products of codes in fp32."""
    c = s["case"]
    off, oc = s["host_offsets"], s["y"].shape[1]
    x = s["x"].float()
    top = x.abs().amax(1, keepdim=True)
    scale = top / 127
    q = torch.round(x.double() * 127 / torch.where(top > 0, top, torch.ones_like(top)).double()).float()
    if s["sorted_pair"] is not None:
        src = (s["sorted_pair"] // c["k"]).long()
        q, scale = q[src], scale[src]
    y = torch.empty(s["rows"], oc, dtype=DT[c["dtype"]], device="cuda")
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        z = (q[a:b] @ s["w"][e].float().t()) * scale[a:b] * s["w_scale"][e]
        if s["bias"] is not None:
            z = z + s["bias"][e].float()
        v = _act(z, c["act"])
        if s["residual"] is not None:
            v = v + s["residual"][a:b].float()
        y[a:b] = v
    return [y]


def _plain_logits(s):
    c = s["case"]
    B, V = c["B"], c["V"]
    l = s["logits"].float()
    at = torch.arange(s["n_history"], device="cuda")
    off = s["history_offsets"].long()
    row = torch.searchsorted(off, at, right=True) - 1
    flat = row * V + s["history"][:s["n_history"]].long()
    made = (at - off[row] >= s["prompt_len"].long()[row]).float()
    count = torch.zeros(B * V, device="cuda").index_put_((flat,), made, accumulate=True).reshape(B, V)
    if s["repetition"] is not None:
        seen = torch.zeros(B * V, dtype=torch.bool, device="cuda")
        seen[flat] = True
        r = s["repetition"][:, None]
        l = torch.where(seen.reshape(B, V), torch.where(l > 0, l / r, l * r), l)
    if s["frequency"] is not None:
        l = l - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias_token"] is not None:
        n = s["n_bias"]
        row = torch.searchsorted(s["bias_offsets"].long(), torch.arange(n, device="cuda"), right=True) - 1
        add = torch.zeros(B * V, device="cuda")
        add[row * V + s["bias_token"][:n].long()] = s["bias_value"][:n]
        l = l + add.reshape(B, V)
    if s["mask"] is not None:
        bit = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        allowed = (bit.reshape(s["mask"].shape[0], -1)[:, :V] == 1)[s["mask_row"].clamp(min=0).long()]
        l = torch.where(allowed | (s["mask_row"] < 0)[:, None], l, torch.full((), float("-inf"), device="cuda"))
    return [l.to(DT[c["out"]])]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op in ("dispatch", "collect"):
        return _plain_tokens(state)
    return _plain_logits(state) if op == "logits" else _plain_product(state)


# ---- what a pass cannot do without -----------------------------------------------------------------------------

def _active(c):
    """Experts that are expected to have rows."""
    q = [(1.0 + i) ** -c["skew"] for i in range(c["E"])]
    t = sum(q)
    return sum(1.0 - (1.0 - min(1.0, c["k"] * p / t)) ** c["T"] for p in q)


def work(case):
    c = case
    if c["op"] in ("dispatch", "collect"):
        eb = 2 if c["dtype"] == "bf16" else 4
        P = c["T"] * c["k"]
        dots = c["dir"] == "bwd" and c["weighted"]
        tokens, rows = c["T"] * c["H"], P * c["H"]
        if c["op"] == "dispatch":     # forward: x read, rows written; backward: rows read, dx written, x read
            n = tokens + rows + (tokens if dots else 0)
        elif c["dir"] == "fwd":
            n = rows + tokens + (tokens if c["base"] else 0)
        else:                         # dy read, rows' gradients written, rows read
            n = tokens + rows + (rows if dots else 0)
        b = eb * n + 4 * P + (4 * P if c["weighted"] else 0) + (4 * P if dots else 0)
        if dots and c["op"] == "collect":
            b += 4 * c["T"] * c["E"] + 4 * P
        return {"bytes": b, "flops": 2 * rows * (2 if dots else 1)}
    if c["op"] == "logits":
        n = c["B"] * c["V"]
        b = n * ((4 if c["dtype"] == "f32" else 2) + (4 if c["out"] == "f32" else 2))
        b += 4 * c["B"] * (c["history"] // 2 + 8) + 4 * c["B"] * c["bias"]
        b += min(8, c["B"]) * c["V"] // 8 if c["mask"] else 0
        return {"bytes": b, "flops": 4 * n}
    eb = 2 if c["dtype"] == "bf16" else 4
    K, N = c["K"], c["N"]
    oc = N // 2 if c["act"] == "swiglu" else N
    if c["op"] == "grouped8":
        rows, live = c["T"] * c["k"], _active(c)
        xr = c["T"] if c["gather"] else rows
    else:
        rows, live, xr = c["M"], 1, c["M"]
    b = eb * (xr * K + rows * oc * (2 if c.get("residual") else 1)) + live * N * (K + 4)
    b += live * N * eb if c["bias"] else 0
    return {"bytes": int(b), "flops": 2 * rows * K * N}


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


def _exact_tokens(s):
    """Slot by slot: slot j of every token names one sorted row, or none."""
    c = s["case"]
    T, k, H, rows = c["T"], c["k"], c["H"], s["rows"]
    new = lambda *n: torch.zeros(*n, dtype=torch.float64, device="cuda")
    pos = s["pair_pos"].view(T, k).long()
    weight = s["topk_w"].double() if c["weighted"] else torch.ones(T, k, dtype=torch.float64, device="cuda")
    to_rows = (c["op"], c["dir"]) in (("dispatch", "fwd"), ("collect", "bwd"))
    token = s["x" if c["op"] == "dispatch" else "dy"].double() if to_rows or c["op"] == "dispatch" else None
    out = new(rows, H) if to_rows else (s["base"].double().clone() if s.get("base") is not None else new(T, H))
    dots = new(T, k)
    theirs = s.get("dout", s.get("expert_rows"))
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        p = pos[t, j]
        if to_rows:
            out[p] = token[t] * weight[t, j:j + 1]
        else:
            out[t] += theirs[p].double() * weight[t, j:j + 1]
        if c["dir"] == "bwd" and c["weighted"]:
            dots[t, j] = torch.einsum("th,th->t", theirs[p].double(), token[t])
    if c["dir"] == "fwd" or not c["weighted"]:
        return [out]
    if c["op"] == "dispatch":
        return [out, dots]
    # the logits' gradient, by differentiating the softmax over the chosen ones
    chosen = torch.log(weight).requires_grad_()
    d, = torch.autograd.grad(torch.softmax(chosen, 1), chosen, dots)
    full = new(T, c["E"])
    full[torch.arange(T, device="cuda")[:, None], s["topk_idx"].long()] = d
    return [out, dots, full]


def _exact_product(s):
    c = s["case"]
    x = s["x"].double()
    scale = x.abs().amax(dim=1) / 127.0
    codes = torch.where(scale[:, None] > 0, x * 127.0 / (scale * 127.0)[:, None], x).round()
    src = (torch.arange(s["rows"], device="cuda") if s["sorted_pair"] is None
           else torch.div(s["sorted_pair"].long(), c["k"], rounding_mode="floor"))
    parts = []
    for e, (a, b) in enumerate(zip(s["host_offsets"][:-1], s["host_offsets"][1:])):
        if b > a:
            at = src[a:b]
            z = torch.matmul(codes[at], s["w"][e].double().t())
            z = z * (scale[at][:, None] * s["w_scale"][e].double()[None, :])
            y = _exact_act(z if s["bias"] is None else z + s["bias"][e].double(), c["act"])
            parts.append(y if s["residual"] is None else y + s["residual"][a:b].double())
    return [torch.cat(parts)]


def _exact_logits(s):
    """Row by row, each rule at the tokens that it names."""
    c = s["case"]
    V = c["V"]
    out = torch.empty(c["B"], V, dtype=torch.float64, device="cuda")
    hist, boff = s["history_offsets"].tolist(), s["bias_offsets"].tolist() if s["bias_offsets"] is not None else None
    plen = s["prompt_len"].tolist()
    mrow = s["mask_row"].tolist() if s["mask_row"] is not None else None
    for r in range(c["B"]):
        l = s["logits"][r].double()
        said = s["history"][hist[r]:hist[r + 1]].long()
        made, n = torch.unique(said[plen[r]:], return_counts=True)
        if s["repetition"] is not None:
            seen = torch.unique(said)
            p = s["repetition"][r].double()
            l[seen] = torch.maximum(l[seen], torch.zeros_like(l[seen])) / p + l[seen].clamp(max=0) * p
        if s["frequency"] is not None:
            l[made] -= s["frequency"][r].double() * n + s["presence"][r].double()
        if boff is not None:
            l[s["bias_token"][boff[r]:boff[r + 1]].long()] += s["bias_value"][boff[r]:boff[r + 1]].double()
        if mrow is not None and mrow[r] >= 0:
            words = s["mask"][mrow[r]].long() & 0xFFFFFFFF
            bits = torch.div(words[:, None], 2 ** torch.arange(32, device="cuda"), rounding_mode="floor") % 2
            l[bits.reshape(-1)[:V] == 0] = float("-inf")
        out[r] = l
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("dispatch", "collect"):
        return _exact_tokens(s)
    return _exact_logits(s) if case["op"] == "logits" else _exact_product(s)
