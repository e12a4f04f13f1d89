"""Cases of the operators around the router and the int8 expert products.

Four kinds of work, each as a user's program calls it:

  balance  load-balance loss of a routed batch with its per-expert counts, then
           its gradient with respect to the router logits (moe_balance_fwd,
           moe_balance_bwd);
  router   backward of the router: the input gradient of the balance loss
           added to the layer's, the gates' gradient added to the logits'
           gradient, and the router's weight and bias gradients
           (moe_router_bwd, moe_gate_bwd);
  linear   rows quantized to int8 with a scale per row, then their product
           with an int8 matrix (one, or one per expert) with a scale per
           output channel (moe_quant_i8, moe_i8_linear); direction "grad" is
           the gradient of the rows, by the same two calls on the transposed
           matrix;
  experts  a SwiGLU expert forward from int8 matrices: quantize the tokens,
           gate and up in one product, SwiGLU and quantization of its rows,
           the down product.

With own = False every kind runs in elementary torch operations in float32
(float64 where a value next to a rounding border is decided); with own = True
it runs through this repository's library.
"""
import math

import torch

own = False

F32, F64, I32 = torch.float32, torch.float64, torch.int32
ACT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a micro-batch of the small float32 layer: latency
        dict(name="balance_t64_e8", kind="balance", T=64, E=8, k=2, pad=0.0),
        # a padded training batch; odd length
        dict(name="balance_t4095_e64_pad", kind="balance", T=4095, E=64, k=6, pad=0.25),
        # eight 8K sequences over 460 experts
        dict(name="balance_t65536_e460", kind="balance", T=65536, E=460, k=12, pad=0.0),
        # the small float32 layer
        dict(name="router_t64_d128_e8_f32", kind="router", T=64, d=128, E=8, k=2, act="f32", pad=0.0),
        # a padded training batch over 64 experts
        dict(name="router_t4096_d2048_e64", kind="router", T=4096, d=2048, E=64, k=6, act="bf16", pad=0.25),
        # one 8K sequence over 460 experts
        dict(name="router_t8192_d2048_e460", kind="router", T=8192, d=2048, E=460, k=12, act="bf16", pad=0.0),
        # one matrix, odd sizes, float32 rows
        dict(name="linear_m777_n1001_k1111_f32", kind="linear", T=777, E=1, k=1, N=1001, K=1111, act="f32", grad=False),
        # one matrix over an 8K sequence: a dense projection beside the experts
        dict(name="linear_m8192_n2048_k2048", kind="linear", T=8192, E=1, k=1, N=2048, K=2048, act="bf16", grad=False),
        # row gradient of the down products of 64 experts in training
        dict(name="grad_t4096_e64_n2048_k1408", kind="linear", T=4096, E=64, k=6, N=2048, K=1408, act="bf16", grad=True),
        # one token of a serving loop
        dict(name="experts_t1_e460", kind="experts", T=1, E=460, k=12, d=2048, f=768),
        # a decode batch: every used expert's weights are read once
        dict(name="experts_t64_e460", kind="experts", T=64, E=460, k=12, d=2048, f=768),
        # a prompt of 8K tokens
        dict(name="experts_t8192_e460", kind="experts", T=8192, E=460, k=12, d=2048, f=768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["balance", "router", "linear", "linear", "experts", "experts"])
    E = _log(rng, 4, 460)
    k = min(E, rng.choice([1, 2, 4, 6, 8, 12]))
    if kind == "balance":
        return dict(kind=kind, T=_log(rng, 1, 65536), E=E, k=k, pad=rng.choice([0.0, 0.1, 0.5]))
    if kind == "router":
        return dict(kind=kind, T=_log(rng, 1, 8192), d=32 * rng.randint(4, 64), E=E, k=k,
                    act=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0.0, 0.25]))
    if kind == "linear":
        E = rng.choice([1, _log(rng, 2, 64)])
        return dict(kind=kind, T=_log(rng, 1, 8192 if E == 1 else 4096), E=E, k=min(E, rng.choice([1, 2, 4, 6])),
                    N=rng.randint(64, 2048), K=rng.randint(64, 2048) if E == 1 else rng.randint(64, 1408),
                    act=rng.choice(["bf16", "bf16", "f32"]), grad=rng.random() < 0.4)
    return dict(kind=kind, T=_log(rng, 1, 8192), E=E, k=k, d=16 * rng.randint(8, 128), f=16 * rng.randint(4, 48))


def _used(E, k, T):
    """Experts with rows, about, under even routing."""
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["kind"] == "balance":
        # logits read by both directions, selection read, gradient written
        return {"bytes": 3 * T * E * 4 + T * k * 4 + E * 8, "flops": 12 * T * E}
    if case["kind"] == "router":
        d, ab = case["d"], 4 if case["act"] == "f32" else 2
        io = T * d * ab * 4 + T * k * d * ab + 2 * T * E * 4 + T * k * 12 + 2 * d * E * 4 + E * 4
        return {"bytes": io, "flops": 4 * T * d * E + 2 * T * k * d}
    if case["kind"] == "linear":
        N, K, ab = case["N"], case["K"], 4 if case["act"] == "f32" else 2
        S = T * k
        rows = S * N * ab + S * K * ab if case["grad"] else T * K * ab + S * N * ab
        return {"bytes": rows + int(_used(E, k, T) * (N * K + N * 4)), "flops": 2 * S * N * K}
    d, f, S = case["d"], case["f"], T * k
    weights = int(_used(E, k, T) * (3 * d * f + (2 * f + d) * 4))
    # (the rows between the two products stay inside the operator's definition)
    return {"bytes": T * d * 2 + S * d * 2 + weights, "flops": 6 * S * d * f}


# ----------------------------------------------------------------- inputs --

def _routing(T, E, k, g):
    """A skewed selection of k of E experts per token and its stable
    expert-contiguous permutation."""
    dev = "cuda"
    logits = torch.randn(T, E, device=dev, generator=g) + torch.randn(E, device=dev, generator=g) * math.sqrt(0.5)
    top = torch.topk(logits, k, dim=1)
    idx = top.indices.to(I32)
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=I32, device=dev)
    offsets[1:] = torch.cumsum(counts, 0)
    slot_pos = torch.empty(T * k, dtype=I32, device=dev)
    slot_pos[order] = torch.arange(T * k, dtype=I32, device=dev)
    return dict(logits=logits, topk_idx=idx, gates=torch.softmax(top.values, 1), offsets=offsets,
                perm_src=order.to(I32), slot_pos=slot_pos, most=int(counts.max()), used=int((counts > 0).sum()))


def _int8(shape, g):
    return torch.randn(shape, device="cuda", generator=g, dtype=torch.float16).mul_(36).round_().clamp_(-127, 127).to(torch.int8)


def _channel(shape, K, g):
    """Scales of the output channels of matrices of variance 1/K."""
    return (torch.rand(shape, device="cuda", generator=g) * 0.5 + 0.75) / (36 * math.sqrt(K))


def _valid(T, pad, g):
    return torch.rand(T, device="cuda", generator=g) >= pad if pad > 0 else None


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = "cuda"
    T, E, k, kind = case["T"], case["E"], case["k"], case["kind"]
    s = dict(case, **_routing(T, E, k, g))
    rand = lambda *n, dt=F32: torch.randn(*n, device=dev, generator=g).to(dt)  # noqa: E731
    if kind == "balance":
        s["valid"] = _valid(T, case["pad"], g)
        if s["valid"] is not None:      # what stands behind a padded token is no number
            s["logits"] = torch.where(s["valid"][:, None], s["logits"], float("nan"))
        s["dloss"] = torch.full((1,), 0.01, device=dev)
    elif kind == "router":
        d, act = case["d"], ACT[case["act"]]
        s["valid"] = _valid(T, case["pad"], g)
        s["x"], s["dy"], s["dx_in"] = rand(T, d, dt=act), rand(T, d, dt=act), rand(T, d, dt=act)
        s["e_out"] = rand(T * k, d, dt=act)
        s["w_router"] = rand(d, E) / math.sqrt(d)
        p = torch.softmax(s["logits"], 1)
        s["dlogits"] = p * (rand(E) * 0.1)
        if s["valid"] is not None:
            s["dlogits"] = s["dlogits"] * s["valid"][:, None]
    elif kind == "linear":
        N, K, act = case["N"], case["K"], ACT[case["act"]]
        if case["grad"]:
            s["rows"] = rand(T * k, N, dt=act)
        else:
            s["rows"] = rand(T, K, dt=act)
        # the stored rows of a matrix start at multiples of 16 bytes
        s["w"] = _padded(_int8((E, N, K), g))
        s["w_scale"] = _channel((E, N), K, g)
        if case["grad"]:
            s["w_t"] = _padded(s["w"].transpose(1, 2))
    else:
        d, f = case["d"], case["f"]
        s["rows"] = rand(T, d, dt=torch.bfloat16)
        s["w_gu"], s["s_gu"] = _padded(_int8((E, 2 * f, d), g)), _channel((E, 2 * f), d, g)
        s["w_dn"], s["s_dn"] = _padded(_int8((E, d, f), g)), _channel((E, d), f, g)
    if own:
        _keep(s)
    return s


def _padded(w):
    """The matrices with their rows at a stride of 16 bytes."""
    E, N, K = w.shape
    if K % 16 == 0:
        return w.contiguous()
    room = torch.zeros(E, N, (K + 15) // 16 * 16, dtype=w.dtype, device=w.device)
    room[:, :, :K] = w
    return room[:, :, :K]


def _keep(s):
    """The dims, workspaces and output buffers that a program keeps."""
    from sparse_moe_expert_fp32_amd import binding as B
    new = lambda *n, dt=F32: torch.empty(*n, dtype=dt, device="cuda")  # noqa: E731
    T, E, k = s["T"], s["E"], s["k"]
    S = T * k
    if s["kind"] in ("balance", "router"):
        d = s.get("d", 128)
        s["dm"] = dm = B.dims(T, d, E, k, 32, 1, 32, s.get("act", "bf16"))
        call = B.CALL_BALANCE_FWD if s["kind"] == "balance" else B.CALL_ROUTER_BWD
        s["ws"] = new(max(1, B.moe_workspace_size(dm, call)), dt=torch.uint8)
        if s["kind"] == "balance":
            s.update(loss=new(1), counts=new(E + 1, dt=I32), prob=new(E), stats=new(T, 2), out=new(T, E))
        else:
            s.update(out=new(T, E), dx=new(T, d, dt=s["x"].dtype), dw=new(d, E), db=new(E))
    elif s["kind"] == "linear":
        width, M = s["rows"].shape[1], s["rows"].shape[0]
        s.update(q=new(M, B.moe_i8_stride(width), dt=torch.int8), q_scale=new(M),
                 out=new(S, s["K"] if s["grad"] else s["N"], dt=s["rows"].dtype))
    else:
        d, f = s["d"], s["f"]
        s.update(q=new(T, B.moe_i8_stride(d), dt=torch.int8), q_scale=new(T), gu=new(S, 2 * f, dt=torch.bfloat16),
                 hq=new(S, B.moe_i8_stride(f), dt=torch.int8), h_scale=new(S), out=new(S, d, dt=torch.bfloat16))


# -------------------------------------------------------------------- run --

def run(s):
    return (_own if own else _plain)[s["kind"]](s)


def _own_balance(s):
    from sparse_moe_expert_fp32_amd import binding as B
    B.moe_balance_fwd(s["dm"], s["logits"], s["topk_idx"], s["valid"], s["loss"], s["counts"], s["prob"], s["stats"], s["ws"])
    B.moe_balance_bwd(s["dm"], s["logits"], s["stats"], s["counts"], s["valid"], s["dloss"], s["out"])
    return dict(loss=s["loss"], counts=s["counts"], prob=s["prob"], dlogits=s["out"])


def _own_router(s):
    from sparse_moe_expert_fp32_amd import binding as B
    dm, x, w, v = s["dm"], s["x"], s["w_router"], s["valid"]
    B.moe_router_bwd(dm, x, w, v, s["dlogits"], s["dx_in"], s["dx"], None, None, s["ws"])
    B.moe_gate_bwd(dm, s["dy"], s["e_out"], s["topk_idx"], s["gates"], s["slot_pos"], v, s["dlogits"], s["out"])
    B.moe_router_bwd(dm, x, w, v, s["out"], None, None, s["dw"], s["db"], s["ws"])
    return dict(dlogits=s["out"], dx=s["dx"], dw=s["dw"], db=s["db"])


def _own_linear(s):
    from sparse_moe_expert_fp32_amd import binding as B
    if s["grad"]:
        B.moe_quant_i8(s["rows"], s["q"], s["q_scale"], col_scale=s["w_scale"], offsets=s["offsets"])
        B.moe_i8_linear(s["q"], s["q_scale"], s["w_t"], None, s["out"], offsets=s["offsets"])
    else:
        B.moe_quant_i8(s["rows"], s["q"], s["q_scale"])
        B.moe_i8_linear(s["q"], s["q_scale"], s["w"], s["w_scale"], s["out"], offsets=s["offsets"],
                        row_src=s["perm_src"], row_div=s["k"])
    return dict(scale=s["q_scale"], out=s["out"])


def _own_experts(s):
    from sparse_moe_expert_fp32_amd import binding as B
    f = s["f"]
    B.moe_quant_i8(s["rows"], s["q"], s["q_scale"])
    B.moe_i8_linear(s["q"], s["q_scale"], s["w_gu"], s["s_gu"], s["gu"], offsets=s["offsets"],
                    row_src=s["perm_src"], row_div=s["k"])
    B.moe_quant_i8(s["gu"][:, :f], s["hq"], s["h_scale"], mul=s["gu"][:, f:])
    B.moe_i8_linear(s["hq"], s["h_scale"], s["w_dn"], s["s_dn"], s["out"], offsets=s["offsets"])
    return dict(scale=s["q_scale"], out=s["out"])


_own = dict(balance=_own_balance, router=_own_router, linear=_own_linear, experts=_own_experts)


# ------------------------------------------------------------- plain form --

def _plain_balance(s):
    l, E, k = s["logits"], s["E"], s["k"]
    T = l.shape[0]
    on = torch.ones(T, dtype=torch.bool, device=l.device) if s["valid"] is None else s["valid"]
    l = torch.where(on[:, None], l, 0.0)
    z = torch.exp(l - l.amax(1, keepdim=True))
    p = z / z.sum(1, keepdim=True) * on[:, None]
    hit = torch.where(on[:, None], s["topk_idx"].long(), E)     # (one bin more for padded tokens)
    counts = torch.bincount(hit.reshape(-1), minlength=E + 1)[:E]
    n = on.sum()
    some = n.clamp_min(1)       # (without a token the loss and its gradient are 0)
    prob = (p.sum(0, dtype=F64) / some).float()
    share = counts.double() * E / (some.double() * k)
    loss = (share * prob.double()).sum().float().reshape(1)
    w = (share / some * s["dloss"].double()).float()
    dlogits = p * (w - (p * w).sum(1, keepdim=True))
    return dict(loss=loss, counts=torch.cat([counts, n.reshape(1)]).to(I32), prob=prob, dlogits=dlogits)


def _plain_router(s):
    T, d = s["x"].shape
    E, k = s["E"], s["k"]
    on = torch.ones(T, dtype=torch.bool, device=s["x"].device) if s["valid"] is None else s["valid"]
    dl = torch.where(on[:, None], s["dlogits"], 0.0)
    dx = (s["dx_in"].float() + dl @ s["w_router"].t()).to(s["x"].dtype)
    o = s["e_out"].float()[s["slot_pos"].long()].reshape(T, k, d)
    dg = (s["dy"].float()[:, None, :] * o).sum(2)
    ga = s["gates"]
    dsel = ga * (dg - (ga * dg).sum(1, keepdim=True))
    dsel = torch.where(on[:, None], dsel, 0.0)
    total = dl.scatter_add(1, s["topk_idx"].long(), dsel)
    x = torch.where(on[:, None], s["x"].float(), 0.0)
    return dict(dlogits=total, dx=dx, dw=x.t() @ total, db=total.sum(0))


def _quantized(v):
    """float32 rows -> (whole values in float32, scale): scale = max|v| / 127,
    the quotients in 64 bits because they stand next to rounding borders."""
    scale = (v.abs().amax(1).double() / 127.0).float()
    safe = torch.where(scale > 0, scale, 1.0)
    return torch.round(v.double() / safe.double()[:, None]).clamp(-127, 127).float(), scale


def _expert_of(s, M):
    return torch.searchsorted(s["offsets"][1:].contiguous(), torch.arange(M, device="cuda", dtype=I32), right=True)


def _grouped(a, a_scale, w, w_scale, s, dt):
    """Rows a of whole values by the matrix of each row's expert.  The rows of
    the experts that have any are laid out as one padded batch; whole values
    up to 2^24 are exact in float32."""
    M, E = a.shape[0], s["E"]
    if E == 1:
        acc = a @ w[0].float().t()
        scale = a_scale[:, None] * (w_scale[0][None, :] if w_scale is not None else 1.0)
        return (acc * scale).to(dt)
    e, at, most, used = _expert_of(s, M), s["offsets"].long(), s["most"], s["used"]
    some = torch.argsort((at[1:] == at[:-1]).to(I32), stable=True)[:used]
    place = torch.zeros(E, dtype=torch.int64, device="cuda")
    place[some] = torch.arange(used, device="cuda")
    row = place[e] * most + torch.arange(M, device="cuda") - at[e]
    wide = torch.zeros(used * most, a.shape[1], device="cuda")
    wide[row] = a
    acc = torch.bmm(wide.reshape(used, most, -1), w[some].float().transpose(1, 2).contiguous())
    acc = acc.reshape(used * most, -1)[row]
    scale = a_scale[:, None] * (w_scale[e] if w_scale is not None else 1.0)
    return (acc * scale).to(dt)


def _plain_linear(s):
    dt = s["rows"].dtype
    if s["grad"]:
        e = _expert_of(s, s["rows"].shape[0])
        a, scale = _quantized(s["rows"].float() * s["w_scale"][e])
        return dict(scale=scale, out=_grouped(a, scale, s["w_t"], None, s, dt))
    a, scale = _quantized(s["rows"].float())
    src = s["perm_src"].long() // s["k"]
    return dict(scale=scale, out=_grouped(a[src], scale[src], s["w"], s["w_scale"], s, dt))


def _plain_experts(s):
    f = s["f"]
    a, scale = _quantized(s["rows"].float())
    src = s["perm_src"].long() // s["k"]
    gu = _grouped(a[src], scale[src], s["w_gu"], s["s_gu"], s, torch.bfloat16).float()
    h, h_scale = _quantized(gu[:, :f] / (1.0 + torch.exp(-gu[:, :f])) * gu[:, f:])
    return dict(scale=scale, out=_grouped(h, h_scale, s["w_dn"], s["s_dn"], s, torch.bfloat16))


_plain = dict(balance=_plain_balance, router=_plain_router, linear=_plain_linear, experts=_plain_experts)


# ---------------------------------------------------------- from 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    return dict(balance=_exact_balance, router=_exact_router, linear=_exact_linear, experts=_exact_experts)[case["kind"]](s)


def _rows_on(s):
    T = s["T"]
    return torch.arange(T, device="cuda") if s["valid"] is None else s["valid"].nonzero()[:, 0]


def _exact_balance(s):
    E, k, T = s["E"], s["k"], s["T"]
    rows = _rows_on(s)
    n = rows.numel()
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    prob, dlogits = torch.zeros(E, dtype=F64, device="cuda"), torch.zeros(T, E, dtype=F64, device="cuda")
    if n == 0:      # (nothing routed: nothing lost)
        return dict(loss=torch.zeros(1, dtype=F64), counts=counts.to(I32), prob=prob, dlogits=dlogits)
    l = s["logits"][rows].double()
    logp = l - torch.logsumexp(l, 1, keepdim=True)
    p = logp.exp()
    chosen = torch.zeros(n, E, dtype=F64, device="cuda")
    chosen.scatter_(1, s["topk_idx"][rows].long(), 1.0)
    fraction = chosen.mean(0) / k
    prob = p.mean(0)
    counts[:E] = chosen.sum(0).round().long()
    counts[E] = n
    loss = E * torch.dot(fraction, prob)
    # d loss / d p[t][e] = E fraction[e] / n, through the softmax
    gp = s["dloss"].double() * E * fraction / n
    dlogits[rows] = p * gp - p * (p @ gp)[:, None]
    return dict(loss=loss.reshape(1), counts=counts.to(I32), prob=prob, dlogits=dlogits)


def _exact_router(s):
    T, k = s["T"], s["k"]
    rows = _rows_on(s)
    dl = torch.zeros(T, s["E"], dtype=F64, device="cuda")
    dl[rows] = s["dlogits"][rows].double()
    dx = s["dx_in"].double() + torch.mm(dl, s["w_router"].double().t())
    slots = s["slot_pos"].long().reshape(T, k)
    g = s["gates"].double()
    dg = torch.stack([(s["dy"].double() * s["e_out"][slots[:, j]].double()).sum(1) for j in range(k)], 1)
    dsel = g * dg - g * (g * dg).sum(1, keepdim=True)
    total = dl.clone()
    for j in range(k):
        total[rows, s["topk_idx"][rows, j].long()] += dsel[rows, j]
    x = s["x"][rows].double()
    return dict(dlogits=total, dx=dx, dw=torch.mm(x.t(), total[rows]), db=total[rows].sum(0))


def _exact_rows(v):
    """The quantized rows as the values they stand for, and the scales.  The
    definition quantizes float32 values by a float32 scale: both roundings
    belong to it, and the quotient is rounded once, from 64 bits."""
    v = v.float().double()
    scale = (v.abs().max(1).values / 127).float().double()
    q = (v / scale.clamp_min(1e-300)[:, None]).round().clamp(-127, 127)
    return q * scale[:, None], scale


def _exact_products(a, w, w_scale, offsets):
    out = torch.zeros(a.shape[0], w.shape[1], dtype=F64, device="cuda")
    at = offsets.tolist()
    for e in range(w.shape[0]):
        if at[e + 1] > at[e]:
            m = w[e].double()
            if w_scale is not None:
                m = m * w_scale[e].double()[:, None]
            out[at[e]:at[e + 1]] = a[at[e]:at[e + 1]] @ m.t()
    return out


def _exact_linear(s):
    if s["grad"]:
        at = s["offsets"].long()
        per_row = torch.repeat_interleave(s["w_scale"], at[1:] - at[:-1], dim=0)
        a, scale = _exact_rows(s["rows"].float() * per_row)
        return dict(scale=scale, out=_exact_products(a, s["w"].transpose(1, 2), None, s["offsets"]))
    a, scale = _exact_rows(s["rows"])
    token = torch.div(s["perm_src"], s["k"], rounding_mode="floor").long()
    return dict(scale=scale, out=_exact_products(a[token], s["w"], s["w_scale"], s["offsets"]))


def _exact_experts(s):
    f = s["f"]
    a, scale = _exact_rows(s["rows"])
    token = torch.div(s["perm_src"], s["k"], rounding_mode="floor").long()
    # (the first product's rows are stored in bf16: that rounding belongs to the chain)
    gu = _exact_products(a[token], s["w_gu"], s["s_gu"], s["offsets"]).float().bfloat16().double()
    h, h_scale = _exact_rows(gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:])
    return dict(scale=scale, out=_exact_products(h, s["w_dn"], s["s_dn"], s["offsets"]))
