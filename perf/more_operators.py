"""Operators around the experts that training a router and serving 4-bit experts need, as a program
calls them, with their plain forms: token slots sorted by expert, the gradients of the way into
expert order, of the weighted way back and of the gating, and products of few rows with 4-bit
weights whose scales (and zero points) belong to groups along K.

``run`` computes either the plain form (elementary torch operations) or, with ``own`` set, calls
the library.  A slot is one of a token's k choices; an id of -1 is a slot without an expert
(padding), which has no row: its position is -1.
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token's 8 experts of 256: a decode step whose ids come from another router
        dict(name="sort_token", op="sort", T=1, E=256, k=8, skew=0.7, drop=0.0),
        # a training batch of 32768 tokens, a few slots of it padding
        dict(name="sort_train", op="sort", T=32768, E=256, k=8, skew=0.7, drop=0.03),
        # an odd, padded batch on small experts; the rows' gradient joins the residual's in fp32
        dict(name="permute_back_odd", op="permute_back", T=333, E=60, k=4, H=2048, skew=1.0,
             drop=0.1, add=True, out="fp32"),
        # a training batch on the 256-expert layer
        dict(name="permute_back_train", op="permute_back", T=8192, E=256, k=8, H=7168, skew=0.7,
             drop=0.0, add=False, out="bf16"),
        # a small padded batch, two experts a token and a gated shared expert
        dict(name="combine_back_odd", op="combine_back", T=37, E=8, k=2, H=4096, skew=0.5,
             drop=0.1, shared="gated"),
        # a training batch on the 256-expert layer and its shared expert
        dict(name="combine_back_train", op="combine_back", T=8192, E=256, k=8, H=7168, skew=0.7,
             drop=0.0, shared="plain"),
        # an odd batch on the 60-expert softmax router
        dict(name="gate_back_odd", op="gate_back", T=333, E=60, k=4, gating="softmax", scale=1.0,
             drop=0.1),
        # a training batch on the 256-expert sigmoid router
        dict(name="gate_back_train", op="gate_back", T=32768, E=256, k=8,
             gating="sigmoid_bias_renorm", scale=2.5, drop=0.0),
        # one token through a dense 4-bit layer: the weights are read once, latency counts
        dict(name="gemv_token", op="gemv", T=1, E=1, k=1, N=4096, K=7168, group=128, zero=False,
             out="bf16", skew=0.0),
        # one token's 8 experts of 256, small groups: a decode step's gate and up products
        dict(name="gemv_experts", op="gemv", T=1, E=256, k=8, N=4096, K=7168, group=32, zero=False,
             out="bf16", skew=0.7),
        # ragged: 8 experts of uneven, odd row counts, N that ends inside a tile, K inside a group
        dict(name="gemv_ragged", op="gemv", T=21, E=8, k=3, N=1000, K=1440, group=64, zero=True,
             out="fp32", skew=1.0),
        # a decode batch of 64 on 256 experts: nearly every expert has rows
        dict(name="gemv_batch64", op="gemv", T=64, E=256, k=8, N=4096, K=7168, group=128, zero=True,
             out="bf16", skew=0.7),
    ]


def draw(rng):
    def log(lo, hi):
        return math.exp(rng.uniform(math.log(lo), math.log(hi)))

    def odd(lo, hi):
        """An odd number of lo .. hi, spread over the logarithm: tiles and batches end unevenly."""
        return max(lo | 1, min((hi - 1) | 1, int(log(lo, hi)) | 1))

    op = rng.choice(("sort", "permute_back", "combine_back", "gate_back", "gemv", "gemv"))
    skew, drop = rng.choice((0.0, 0.4, 0.7, 1.1)), rng.choice((0.0, 0.03, 0.3))
    E = int(log(2, 257))
    k = rng.randint(1, min(8, E))
    if op == "sort":
        return dict(op=op, T=odd(1, 32768), E=E, k=k, skew=skew, drop=drop)
    if op == "permute_back":
        return dict(op=op, T=odd(1, 8192), E=E, k=k, H=8 * odd(8, 896), skew=skew, drop=drop,
                    add=rng.random() < 0.5, out=rng.choice(("bf16", "fp32")))
    if op == "combine_back":
        return dict(op=op, T=odd(1, 8192), E=E, k=k, H=8 * odd(8, 896), skew=skew, drop=drop,
                    shared=rng.choice(("none", "plain", "gated")))
    if op == "gate_back":
        gating = rng.choice(("softmax_renorm", "softmax", "sigmoid_bias_renorm"))
        return dict(op=op, T=odd(1, 32768), E=E, k=k, gating=gating, scale=rng.choice((1.0, 2.5)),
                    drop=drop)
    while True:
        E = rng.choice((1, int(log(2, 257))))
        c = dict(op=op, T=odd(1, 64), E=E, k=1 if E == 1 else rng.randint(1, min(8, E)),
                 N=odd(63, 14336), K=32 * odd(3, 448), group=rng.choice((32, 64, 128)),
                 zero=rng.random() < 0.5, out=rng.choice(("bf16", "fp32")), skew=skew)
        if c["E"] * c["N"] * c["K"] <= 256 * 4096 * 7168:
            return c


# ------------------------------------------------------------------------------------- inputs
def _choose(T, E, k, skew, drop, g):
    """ids [T][k] int32 of a router with Zipf(skew) popularity (each row's experts distinct and
    ascending); `drop` of the tokens are padding, all their slots -1, and as many single slots."""
    dev = "cuda"
    pop = -skew * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    pop = pop[torch.randperm(E, generator=g, device=dev)]
    u = torch.rand((T, E), generator=g, device=dev).clamp_(1e-7, 1 - 1e-7)
    ids = (pop - torch.log(-torch.log(u))).topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
    if drop:
        ids[torch.rand(T, generator=g, device=dev) < drop] = -1
        ids[torch.rand((T, k), generator=g, device=dev) < drop] = -1
    return ids


def _positions(ids, E):
    """(counts, offsets, pos, src) of ids [T][k]: slots in expert order, stable; slots without an
    expert have pos -1, and the end of src that no slot takes is -1."""
    flat = ids.reshape(-1).long()
    has = (flat >= 0) & (flat < E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    key = torch.where(has, flat, E)
    counts.scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts[:E], 0)])
    order = torch.sort(key, stable=True).indices
    n = torch.arange(flat.numel(), device=flat.device)
    taken = n < offsets[E]
    src = torch.where(taken, order, -1)
    pos = torch.empty_like(src)
    pos[order] = torch.where(taken, n, -1)
    i32 = torch.int32
    return counts[:E].to(i32), offsets.to(i32), pos.view(ids.shape).to(i32), src.to(i32)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 29)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    st = dict(case)
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    bf16 = torch.bfloat16
    if op == "gate_back":
        z = randn(T, E)
        sig = case["gating"] == "sigmoid_bias_renorm"
        choice = 1.0 / (1.0 + torch.exp(-z)) + randn(E) * 0.1 if sig else z
        ids = choice.topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
        if case["drop"]:
            ids[torch.rand((T, k), generator=g, device=dev) < case["drop"]] = -1
        st["logits"], st["ids"], st["dw"] = z, ids, randn(T, k)
    else:
        ids = _choose(T, E, k, case["skew"], case.get("drop", 0.0), g)
        if op == "sort":
            st["ids"] = ids
        else:
            _, st["offsets"], st["pos"], st["src"] = _positions(ids, E)
    if op == "permute_back":
        st["dx_perm"] = randn(T * k, case["H"], dtype=bf16)
        st["add_to"] = randn(T, case["H"], dtype=bf16) if case["add"] else None
    elif op == "combine_back":
        H = case["H"]
        st["dout"], st["y_perm"] = randn(T, H, dtype=bf16), randn(T * k, H, dtype=bf16)
        w = torch.rand((T, k), generator=g, device=dev) + 0.05
        st["w"] = w / w.sum(dim=1, keepdim=True)
        st["shared_y"] = randn(T, H, dtype=bf16) if case["shared"] != "none" else None
        st["shared_gate"] = (torch.rand(T, generator=g, device=dev) if case["shared"] == "gated"
                             else None)
    elif op == "gemv":
        N, K, G = case["N"], case["K"], case["group"]
        ng = -(-K // G)
        words = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), generator=g, device=dev,
                              dtype=torch.int32)
        st["w4"] = words.view(torch.uint8).view(E, N, K // 2)
        st["scales"] = ((0.5 + torch.rand((E, N, ng), generator=g, device=dev)) * 0.005).to(bf16)
        st["zeros"] = (torch.randint(6, 11, (E, N, ng), generator=g, device=dev, dtype=torch.uint8)
                       if case["zero"] else None)
        st["bounds"] = st["offsets"].tolist()
        st["x"] = randn(st["bounds"][-1], K, dtype=bf16)
    if own:
        _own_buffers(st)
    return st


def _own_buffers(st):
    """What a program keeps beside the inputs: outputs and workspaces."""
    import expert_dispatch_streaming_gb300 as moe
    dev, op, T, E, k = "cuda", st["op"], st["T"], st["E"], st["k"]
    f32, bf16 = torch.float32, torch.bfloat16
    if op == "sort":
        i32 = dict(dtype=torch.int32, device=dev)
        st["res"] = dict(counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                         pos=torch.empty((T, k), **i32), src=torch.empty(T * k, **i32))
        st["ws_bytes"] = moe.moe_sort_tokens_workspace_size(T, E, k)
        st["ws"] = torch.empty(max(st["ws_bytes"], 256), dtype=torch.uint8, device=dev)
    elif op == "permute_back":
        st["res"] = dict(dx=torch.empty((T, st["H"]), device=dev,
                                        dtype=bf16 if st["out"] == "bf16" else f32))
    elif op == "combine_back":
        H = st["H"]
        r = dict(dy_perm=torch.zeros((T * k, H), dtype=bf16, device=dev),
                 dw=torch.empty((T, k), dtype=f32, device=dev))
        if st["shared_y"] is not None:
            r["dshared"] = torch.empty((T, H), dtype=bf16, device=dev)
        if st["shared_gate"] is not None:
            r["dshared_gate"] = torch.empty(T, dtype=f32, device=dev)
        st["res"] = r
    elif op == "gate_back":
        st["res"] = dict(dlogits=torch.empty((T, E), dtype=f32, device=dev))
    else:
        rows = st["bounds"][-1]
        st["res"] = dict(y=torch.empty((rows, st["N"]), device=dev,
                                       dtype=bf16 if st["out"] == "bf16" else f32))
        st["ws_bytes"] = moe.moe_grouped_gemv_int4_workspace_size(rows, E, st["N"], st["K"])
        st["ws"] = torch.empty(max(st["ws_bytes"], 256), dtype=torch.uint8, device=dev)


# ------------------------------------------------------------------------------------- run
def run(st):
    if own:
        return _run_own(st)
    return {"sort": _sort, "permute_back": _permute_back, "combine_back": _combine_back,
            "gate_back": _gate_back, "gemv": _gemv}[st["op"]](st)


def _run_own(st):
    import expert_dispatch_streaming_gb300 as moe
    op, T, E, k, r = st["op"], st["T"], st["E"], st["k"], st["res"]
    if op == "sort":
        moe.moe_sort_tokens(st["ids"], T, E, k, r["counts"], r["offsets"], r["pos"], r["src"],
                            st["ws"], st["ws_bytes"])
    elif op == "permute_back":
        moe.moe_permute_backward(st["dx_perm"], st["pos"], st["add_to"], T, k, st["H"], st["out"],
                                 r["dx"])
    elif op == "combine_back":
        moe.moe_combine_backward(st["dout"], st["y_perm"], st["pos"], st["w"], T, k, st["H"],
                                 st["shared_y"], st["shared_gate"], r["dy_perm"], r["dw"],
                                 r.get("dshared"), r.get("dshared_gate"))
    elif op == "gate_back":
        moe.moe_gate_backward(st["logits"], st["ids"], st["dw"], T, E, k, st["gating"],
                              st["scale"], r["dlogits"])
    else:
        moe.moe_grouped_gemv_int4(st["x"], st["w4"], st["scales"], st["zeros"], st["offsets"], E,
                                  st["N"], st["K"], st["group"], st["bounds"][-1], st["out"],
                                  r["y"], st["ws"], st["ws_bytes"])
    return r


# ------------------------------------------------------------------------------- plain forms
def _sort(st):
    counts, offsets, pos, src = _positions(st["ids"], st["E"])
    return dict(counts=counts, offsets=offsets, pos=pos, src=src)


def _slots(st, j):
    """(tokens whose slot j has a row, those rows)."""
    p = st["pos"][:, j].long()
    t = torch.nonzero(p >= 0).view(-1)
    return t, p[t]


def _permute_back(st):
    dx = torch.zeros((st["T"], st["H"]), dtype=torch.float32, device="cuda")
    for j in range(st["k"]):
        t, p = _slots(st, j)
        dx[t] += st["dx_perm"][p].float()
    if st["add_to"] is not None:
        dx += st["add_to"].float()
    return dict(dx=dx if st["out"] == "fp32" else dx.to(torch.bfloat16))


def _combine_back(st):
    T, k, H = st["T"], st["k"], st["H"]
    dout = st["dout"].float()
    dy = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float32, device="cuda")
    for j in range(k):
        t, p = _slots(st, j)
        d = dout[t]
        dw[t, j] = (d * st["y_perm"][p].float()).sum(dim=1)
        dy[p] = (d * st["w"][t, j, None]).to(torch.bfloat16)
    out = dict(dy_perm=dy, dw=dw)
    if st["shared_y"] is not None:
        gate = st["shared_gate"]
        out["dshared"] = (dout if gate is None else dout * gate[:, None]).to(torch.bfloat16)
        if gate is not None:
            out["dshared_gate"] = (dout * st["shared_y"].float()).sum(dim=1)
    return out


def _gate_back(st):
    z, ids, scale = st["logits"], st["ids"].long(), st["scale"]
    has = ids >= 0
    at = ids.clamp_min(0)
    dw = torch.where(has, st["dw"], 0.0)
    zj = torch.where(has, z.gather(1, at), -math.inf)
    if st["gating"] == "softmax":
        p = torch.exp(z - z.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
        pj = torch.where(has, p.gather(1, at), 0.0)
        inner = (pj * dw).sum(dim=1, keepdim=True)
        return dict(dlogits=(p * -inner).scatter_add(1, at, pj * dw) * scale)
    if st["gating"] == "softmax_renorm":
        v, slope = torch.exp(zj - zj.amax(dim=1, keepdim=True).clamp_min(-1e30)), 1.0
    else:
        v = 1.0 / (1.0 + torch.exp(-zj))
        slope = torch.where(has, 1.0 / (1.0 + torch.exp(zj)), 0.0)
    r = v / v.sum(dim=1, keepdim=True).clamp_min(1e-30)
    inner = (r * dw).sum(dim=1, keepdim=True)
    return dict(dlogits=torch.zeros_like(z).scatter_add(1, at, scale * r * (dw - inner) * slope))


def _gemv(st):
    b, G, K = st["bounds"], st["group"], st["K"]
    dtype = torch.bfloat16 if st["out"] == "bf16" else torch.float32
    parts = []
    for e in range(st["E"]):
        if b[e + 1] == b[e]:
            continue
        w = st["w4"][e]
        # two codes a byte, the lower half first
        q = torch.stack([w & 15, w >> 4], dim=2).view(w.shape[0], K).float()
        z = 8.0 if st["zeros"] is None else st["zeros"][e].float().repeat_interleave(G, 1)[:, :K]
        q = (q - z) * st["scales"][e].float().repeat_interleave(G, 1)[:, :K]
        parts.append((st["x"][b[e]:b[e + 1]].float() @ q.T).to(dtype))
    return dict(y=torch.cat(parts))


# ------------------------------------------------------------------------------------- work
def _rows_of(case):
    """Rows of each expert by rank, as a Zipf(skew) router gives them on average (the products'
    work depends on the chosen experts a little)."""
    T, E, k = case["T"], case["E"], case["k"]
    p = [(r + 1.0) ** -case["skew"] for r in range(E)]
    s = sum(p)
    # P(expert has a row) for T tokens that take k of E without repetition, near enough
    return sum(1.0 - (1.0 - min(1.0, k * v / s)) ** T for v in p), T * k


def work(case):
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    if op == "sort":
        return {"bytes": 12 * T * k + 8 * E + 4, "flops": T * k}
    if op == "gate_back":
        read = T * E if case["gating"] == "softmax" else T * k
        return {"bytes": 4 * (read + T * E) + 8 * T * k, "flops": 4 * read + 4 * T * k}
    if op == "gemv":
        used, rows = _rows_of(case)
        used = min(used, rows)
        N, K, ng = case["N"], case["K"], -(-case["K"] // case["group"])
        ob = 2 if case["out"] == "bf16" else 4
        return {"bytes": int(used * N * (K // 2 + ng * (3 if case["zero"] else 2)))
                + rows * (2 * K + ob * N), "flops": 2 * rows * N * K}
    H, live = case["H"], (1.0 - case["drop"]) ** 2
    rows = int(T * k * live)
    if op == "permute_back":
        ob = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * rows * H + (ob + (2 if case["add"] else 0)) * T * H + 4 * T * k,
                "flops": rows * H}
    per = {"none": 0, "plain": 2, "gated": 4}[case["shared"]]
    return {"bytes": 4 * rows * H + (2 + per) * T * H + 12 * T * k, "flops": 3 * rows * H}


# ------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits; the gradients by automatic differentiation of the forward
    operators' formulas."""
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    if op == "sort":
        return None                 # whole numbers
    st = prepare(case, seed)
    f64 = torch.float64
    if op == "permute_back":
        tok = torch.div(st["src"].long(), k, rounding_mode="floor")
        rows = int((st["src"] >= 0).sum())
        dx = torch.zeros((T, case["H"]), dtype=f64, device="cuda")
        dx.index_add_(0, tok[:rows], st["dx_perm"][:rows].to(f64))
        return dict(dx=dx if st["add_to"] is None else dx + st["add_to"].to(f64))
    if op == "combine_back":
        src = st["src"].long()
        rows = int((src >= 0).sum())
        src = src[:rows]
        w = st["w"].to(f64).view(-1)
        dy = torch.zeros((T * k, case["H"]), dtype=f64, device="cuda")
        dw = torch.zeros(T * k, dtype=f64, device="cuda")
        for lo in range(0, rows, 8192):
            s = src[lo:lo + 8192]
            d = st["dout"][s // k].to(f64)
            dy[lo:lo + s.numel()] = d * w[s, None]
            dw[s] = torch.einsum("rh,rh->r", d, st["y_perm"][lo:lo + s.numel()].to(f64))
        out = dict(dy_perm=dy, dw=dw.view(T, k))
        if st["shared_y"] is not None:
            g = st["shared_gate"]
            d = st["dout"].to(f64)
            out["dshared"] = d if g is None else torch.einsum("th,t->th", d, g.to(f64))
            if g is not None:
                out["dshared_gate"] = torch.einsum("th,th->t", d, st["shared_y"].to(f64))
        return out
    if op == "gate_back":
        z = st["logits"].to(f64).requires_grad_(True)
        chosen = torch.zeros((T, E + 1), dtype=torch.bool, device="cuda")
        chosen.scatter_(1, torch.where(st["ids"] < 0, E, st["ids"].long()), True)
        chosen = chosen[:, :E]
        up = torch.zeros((T, E + 1), dtype=f64, device="cuda")
        up.scatter_(1, torch.where(st["ids"] < 0, E, st["ids"].long()), st["dw"].to(f64))
        up = up[:, :E]
        if case["gating"] == "softmax":
            w = torch.softmax(z, 1)
        else:
            v = torch.sigmoid(z) if case["gating"] == "sigmoid_bias_renorm" else torch.exp(z)
            v = torch.where(chosen, v, 0.0)
            total = v.sum(1, keepdim=True)
            w = v / torch.where(total > 0, total, 1.0)
        loss = (w * up).masked_select(chosen).sum() * case["scale"]
        return dict(dlogits=torch.autograd.grad(loss, z)[0])
    b, out = st["bounds"], []
    col = torch.arange(case["K"], device="cuda")
    for e in range(E):
        if b[e + 1] == b[e]:
            continue
        byte = st["w4"][e][:, col // 2].int()
        code = torch.where(col % 2 == 1, byte // 16, byte % 16).to(f64)
        zero = 8.0 if st["zeros"] is None else st["zeros"][e].to(f64)[:, col // case["group"]]
        w = (code - zero) * st["scales"][e].to(f64)[:, col // case["group"]]
        out.append(torch.einsum("rk,nk->rn", st["x"][b[e]:b[e + 1]].to(f64), w))
    return dict(y=torch.cat(out, 0))
