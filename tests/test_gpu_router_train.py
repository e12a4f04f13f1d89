"""Load-balance loss, gate gradient and router backward on the GPU against the
formulas in float64, at the sizes and masks where they can go wrong.

Tolerances count float32 roundings (U = 2^-24): n additions in any order carry
at most n U of the sum of magnitudes; expf and the argument's rounding carry
(|x| + 4) U of the exponential."""
import numpy as np
import pytest
import torch

from sparse_moe_expert_fp32_amd import binding as B, configs, inputs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = "cuda:0"
HALF_ACT = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dims(T, d, E, k, act="bf16"):
    return B.dims(T, d, E, k, 32, 1, 32, act)


def f64(t):
    return t.double().cpu()


def route(T, E, k, seed, spread=1.0):
    g = gen(seed)
    l = torch.randn(T, E, generator=g) * spread
    top = torch.topk(l, k, 1)
    return l, top.indices.to(torch.int32), torch.softmax(top.values, 1)


# ------------------------------------------------------------------ balance --

def balance_ref(l, idx, valid, dloss):
    T, E = l.shape
    k = idx.shape[1]
    on = torch.ones(T, dtype=torch.bool) if valid is None else valid
    n = int(on.sum())
    counts = torch.zeros(E + 1, dtype=torch.int64)
    p = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        if on[t]:
            row = l[t].double()
            m = row.max()
            if m > -np.inf:
                z = torch.exp(row - m)
                p[t] = z / z.sum()
            for e in idx[t].tolist():
                if 0 <= e < E:
                    counts[e] += 1
    counts[E] = n
    if n == 0:
        return 0.0, counts, torch.zeros(E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64), p
    prob = p.sum(0) / n
    loss = E * float((counts[:E] / (n * k) * prob).sum())
    w = dloss * E * counts[:E].double() / (n * n * k)
    return loss, counts, prob, p * (w - (p * w).sum(1, keepdim=True)), p


def balance_gpu(l, idx, valid, dloss, in_place=False):
    T, E = l.shape
    dm = dims(T, 32, E, idx.shape[1])
    new = lambda *n, dt=torch.float32: torch.full(n, -77, dtype=dt, device=DEV)  # noqa: E731
    loss, counts, prob, stats = new(1), new(E + 1, dt=torch.int32), new(E), new(T, 2)
    ws = new(max(1, B.moe_workspace_size(dm, B.CALL_BALANCE_FWD)), dt=torch.int8)
    ld, idxd = l.to(DEV), idx.to(DEV)
    v = None if valid is None else valid.to(DEV)
    dl = torch.tensor([dloss], device=DEV)
    out = ld if in_place else new(T, E)
    B.moe_balance_fwd(dm, ld, idxd, v, loss, counts, prob, stats, ws)
    B.moe_balance_bwd(dm, ld, stats, counts, v, dl, out)
    torch.cuda.synchronize()
    return loss, counts, prob, stats, out


def check_balance(l, idx, valid, dloss=0.5, in_place=False):
    loss, counts, prob, stats, out = balance_gpu(l, idx, valid, dloss, in_place)
    rl, rc, rp, rd, p = balance_ref(l, idx, valid, dloss)
    T, E = l.shape
    n, k = int(rc[E]), idx.shape[1]
    assert torch.equal(counts.cpu().long(), rc)
    fin = torch.where(torch.isfinite(l), l, torch.zeros_like(l)).double()
    span = float((fin.max() - fin.min())) if n else 0.0
    rel_p = (span + 4 + E // 64 + 8 + 4) * U           # exp, the row's sum, two multiplications
    rel = rel_p + (T + 8) * U                          # the sum over tokens, all terms >= 0
    assert torch.all((f64(prob) - rp).abs() <= rel * rp + 1e-38)
    assert abs(float(loss) - rl) <= (rel + 4 * U) * rl + 1e-38
    wmax = abs(dloss) * E * float(rc[:E].max()) / max(1, n * n * k)
    assert torch.all((f64(out) - rd).abs() <= (3 * rel_p + (E // 64 + 12) * U) * p * wmax * 2 + 1e-38)
    if valid is not None:
        assert torch.all(out.cpu()[~valid] == 0) and torch.all(stats.cpu()[~valid] == 0)


@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 8, 2), (3, 64, 6), (64, 8, 2), (77, 65, 5), (130, 256, 32), (61, 257, 1),
    (200, 460, 12), (33, 513, 8), (19, 1024, 32), (2600, 12, 3),
])
def test_balance(cuda_ok, T, E, k):
    l, idx, _ = route(T, E, k, T + E)
    check_balance(l, idx, None)


@pytest.mark.parametrize("T,E,k", [(5, 8, 2), (301, 100, 4), (65, 460, 12)])
def test_balance_masked_tokens_hold_anything(cuda_ok, T, E, k):
    l, idx, _ = route(T, E, k, 3 * T)
    valid = torch.rand(T, generator=gen(T)) > 0.4
    valid[0], valid[-1] = False, True
    l[~valid] = float("nan")
    idx[~valid] = 1 << 30
    check_balance(l, idx, valid)
    check_balance(l, idx, valid, in_place=True)


def test_balance_without_a_token(cuda_ok):
    l, idx, _ = route(9, 20, 3, 1)
    check_balance(l * float("inf"), idx, torch.zeros(9, dtype=torch.bool))


@pytest.mark.parametrize("T,cut,E,k", [(300, 7, 40, 3), (513, 256, 460, 12)])
def test_balance_counts_added_over_two_halves(cuda_ok, T, cut, E, k):
    """A batch in two parts whose counts are added between the two calls: the
    gradient has the whole batch's loads."""
    l, idx, _ = route(T, E, k, T)
    valid = torch.rand(T, generator=gen(1)) > 0.2
    whole = balance_gpu(l, idx, valid, 0.5)
    dl = torch.tensor([0.5], device=DEV)
    parts = []
    for s in (slice(0, cut), slice(cut, T)):
        n = s.stop - s.start
        dm = dims(n, 32, E, k)
        new = lambda *n_, dt=torch.float32: torch.full(n_, -77, dtype=dt, device=DEV)  # noqa: E731
        ld, v = l[s].to(DEV), valid[s].to(DEV)
        loss, counts, prob, stats = new(1), new(E + 1, dt=torch.int32), new(E), new(n, 2)
        ws = new(max(1, B.moe_workspace_size(dm, B.CALL_BALANCE_FWD)), dt=torch.int8)
        B.moe_balance_fwd(dm, ld, idx[s].to(DEV), v, loss, counts, prob, stats, ws)
        parts.append((dm, ld, v, stats, counts))
    total = parts[0][4] + parts[1][4]
    assert torch.equal(total, whole[1])
    outs = []
    for dm, ld, v, stats, _ in parts:
        out = torch.empty_like(ld)
        B.moe_balance_bwd(dm, ld, stats, total, v, dl, out)
        outs.append(out)
    assert torch.equal(torch.cat(outs), whole[4])   # (a row's arithmetic is the same)


def test_balance_masked_experts_and_empty_rows(cuda_ok):
    """-inf logits have probability 0, a row of them adds nothing; the type's
    lowest value is a finite logit like others; same index twice, and indices
    out of range."""
    l, idx, _ = route(70, 90, 4, 2)
    l[:, 7] = -np.inf
    l[3] = -np.inf
    l[4, 5:] = -np.inf
    l[5] = torch.finfo(torch.float32).min
    l[6, 10] = torch.finfo(torch.float32).min
    idx[8] = 2
    idx[9, 1], idx[9, 2] = -1, 90
    T, E = l.shape
    loss, counts, prob, stats, out = balance_gpu(l, idx, None, 1.0)
    rl, rc, rp, rd, p = balance_ref(l, idx, None, 1.0)
    assert torch.equal(counts.cpu().long(), rc) and counts[2] >= 4
    rel = (16 + 4 + 2 + 12 + T + 8) * U
    assert torch.all((f64(prob) - rp).abs() <= rel * rp)
    assert abs(float(loss) - rl) <= rel * rl
    others = [t for t in range(T) if t != 5]        # (row 5 is even over all experts)
    assert torch.all(out[3] == 0) and torch.all(out[others, 7] == 0)
    assert torch.all((f64(out) - rd).abs() <= 8 * rel * p * float(rc[:E].max()) * E / (T * T * 4))


def test_balance_nan_is_not_hidden(cuda_ok):
    l, idx, _ = route(40, 70, 4, 5)
    l[13, 50] = float("nan")
    loss, counts, prob, stats, out = balance_gpu(l, idx, None, 1.0)
    assert torch.isnan(loss).all() and torch.isnan(prob).all()
    assert torch.isnan(out[13]).all() and torch.isfinite(out[14]).all()
    assert counts[70] == 40


def test_balance_gradient_against_differences(cuda_ok):
    """Central differences of the float64 loss with the counts held fixed."""
    l, idx, _ = route(6, 9, 2, 8)
    *_, out = balance_gpu(l, idx, None, 1.0)
    counts = balance_ref(l, idx, None, 1.0)[1][:9].double()
    def loss(x):
        return 9 * float((counts / 12 * torch.softmax(x, 1).mean(0)).sum())
    h = 1e-5
    for t, e in ((0, 0), (2, 5), (5, 8), (3, 3)):
        a, b = l.double().clone(), l.double().clone()
        a[t, e] += h
        b[t, e] -= h
        # (the differences' own error: h^2 of the third derivative, and 2^-52 / h)
        assert abs((loss(a) - loss(b)) / (2 * h) - float(out[t, e])) <= 1e-9 + 60 * U


# --------------------------------------------------------------------- gate --

def act_t(act):
    return torch.bfloat16 if act == "bf16" else torch.float32


def gate_case(T, d, E, k, act, seed):
    g = gen(seed)
    l, idx, gates = route(T, E, k, seed)
    dy = torch.randn(T, d, generator=g).to(act_t(act))
    e_out = torch.randn(T * k, d, generator=g).to(act_t(act))
    pos = torch.randperm(T * k, generator=g).to(torch.int32).reshape(T, k)
    dl = torch.randn(T, E, generator=g)
    return dy, e_out, idx, gates, pos, dl


def gate_ref(dy, e_out, idx, gates, pos, valid, dl):
    T, k = idx.shape
    o = e_out.double()[pos.long()]
    prod = dy.double()[:, None, :] * o
    dg, mag = prod.sum(2), prod.abs().sum(2)
    g = gates.double()
    dsel = g * (dg - (g * dg).sum(1, keepdim=True))
    size = g * (mag + (g * mag).sum(1, keepdim=True))
    tot = torch.zeros(T, dl.shape[1] if dl is not None else 0, dtype=torch.float64)
    return dsel, size


def check_gate(T, d, E, k, act, valid=None, dl_given=True, in_place=False, dup=False):
    dy, e_out, idx, gates, pos, dl = gate_case(T, d, E, k, act, T + 7 * k)
    if dup:
        idx[:, 1] = idx[:, 0]
    if valid is not None:
        dy[~valid] = float("nan")
    dm = dims(T, d, E, k, act)
    dd = [t.to(DEV) for t in (dy, e_out, idx, gates, pos)]
    v = None if valid is None else valid.to(DEV)
    src = dl.to(DEV) if dl_given else None
    out = src if in_place else torch.full((T, E), -77.0, device=DEV)
    B.moe_gate_bwd(dm, *dd, v, src, out)
    torch.cuda.synchronize()
    dsel, size = gate_ref(dy, e_out, idx, gates, pos, valid, dl)
    ref = dl.double().clone() if dl_given else torch.zeros(T, E, dtype=torch.float64)
    tol = ref.abs() * 4 * U
    tol.scatter_add_(1, idx.long(), (d / 64 + 3 * k + 24) * U * size)
    ref.scatter_add_(1, idx.long(), dsel)
    on = torch.ones(T, dtype=torch.bool) if valid is None else valid
    assert torch.all((f64(out) - ref).abs()[on] <= tol[on] + 1e-38)
    assert torch.all(out.cpu()[~on] == 0)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,E,k", [
    (1, 32, 1, 1), (1, 128, 8, 2), (5, 2048, 460, 12), (63, 96, 65, 3), (33, 1056, 20, 5),
    (18, 544, 40, 8), (9, 320, 1024, 32), (130, 64, 64, 6), (7, 256, 48, 13),
])
def test_gate_bwd(cuda_ok, T, d, E, k, act):
    check_gate(T, d, E, k, act)


@pytest.mark.parametrize("kw", [
    dict(dl_given=False), dict(in_place=True), dict(dup=True), dict(dup=True, in_place=True),
    dict(valid=True), dict(valid=True, in_place=True), dict(valid=True, dl_given=False),
])
def test_gate_bwd_variants(cuda_ok, kw):
    kw = dict(kw)
    if kw.get("valid"):
        kw["valid"] = torch.arange(50) % 3 != 0
    check_gate(50, 160, 70, 6, "bf16", **kw)


def test_gate_bwd_most_tokens(cuda_ok):
    """2^26 slots, one a token: more than a launch takes."""
    T, d = 1 << 26, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    new = lambda *n: torch.randn(*n, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    dy, e_out = new(T, d), new(T, d)
    gates = torch.rand(T, generator=g, device=DEV)
    idx = torch.zeros(T, dtype=torch.int32, device=DEV)
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)
    valid = torch.ones(T, dtype=torch.uint8, device=DEV)
    valid[5], valid[T - 7] = 0, 0
    out = torch.full((T, 1), -77.0, device=DEV)
    B.moe_gate_bwd(dims(T, d, 1, 1), dy, e_out, idx, gates, pos, valid, None, out)
    for t in (0, (1 << 24) - 500, 1 << 25, T - 1000):      # (both sides of a launch's end)
        s = slice(t, t + 1000)
        prod = dy[s].double() * e_out[pos[s].long()].double()
        dg, mag, ga = prod.sum(1), prod.abs().sum(1), gates[s].double()
        ref = torch.where(valid[s] > 0, ga * (dg - ga * dg), 0.0)
        assert torch.all((out[s, 0].double() - ref).abs() <= 32 * U * ga * mag * 2)
    assert int((out == -77).sum()) == 0


# ------------------------------------------------------------------- router --

def router_case(T, d, E, act, seed):
    g = gen(seed)
    x = torch.randn(T, d, generator=g).to(act_t(act))
    w = torch.randn(d, E, generator=g) / d ** 0.5
    dl = torch.randn(T, E, generator=g) * torch.rand(T, 1, generator=g)
    dx_in = torch.randn(T, d, generator=g).to(act_t(act))
    return x, w, dl, dx_in


def run_router(dm, x, w, valid, dl, dx_in, want, alias=False):
    T, d, E, dt = dm.T, dm.d_model, dm.n_experts, x.dtype
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    xin = to(dx_in) if "x" in want else None
    dx = (xin if alias else torch.full((T, d), -77.0, device=DEV, dtype=dt)) if "x" in want else None
    dw = torch.full((d, E), -77.0, device=DEV) if "w" in want else None
    db = torch.full((E,), -77.0, device=DEV) if "b" in want else None
    ws = torch.full((max(1, B.moe_workspace_size(dm, B.CALL_ROUTER_BWD)),), 255, dtype=torch.uint8, device=DEV)
    B.moe_router_bwd(dm, to(x), to(w), to(valid), to(dl), xin, dx, dw, db, ws)
    torch.cuda.synchronize()
    return dx, dw, db


def check_router(T, d, E, act, want="xwb", valid=None, dx_given=True, alias=False):
    x, w, dl, dx_in = router_case(T, d, E, act, T + d + E)
    on = torch.ones(T, dtype=torch.bool) if valid is None else valid
    xd, dld = x.double(), dl.double()
    xd[~on], dld[~on] = 0, 0
    if valid is not None:
        x[~on], dl[~on] = float("nan"), float("inf")
    dx, dw, db = run_router(dims(T, d, E, 1, act), x, w, valid, dl, dx_in if dx_given else None, want, alias)
    if dx is not None:
        ref = dld @ w.double().t() + (dx_in.double() if dx_given else 0.0)
        mag = dld.abs() @ w.double().abs().t()
        half = 2.0 ** -8 if act == "bf16" else 2.0 ** -24
        # float32: E + 4 additions; bf16 output: each operand kept to 16 bits
        # or more (2^-17 each, and the product of two remainders 2^-16)
        tol = half * ref.abs() * (1 + half) + (E + 8) * U * (mag + ref.abs()) + (2.0 ** -15 * mag if act == "bf16" else 0)
        assert torch.all((f64(dx) - ref).abs() <= tol + 1e-38)
    n = int(on.sum())
    if dw is not None:
        ref, mag = xd.t() @ dld, xd.abs().t() @ dld.abs()
        assert torch.all((f64(dw) - ref).abs() <= (n + 12) * U * mag + 1e-38)
        if n > 1000:   # far from the worst case: additions of random sign
            assert float((f64(dw) - ref).norm() / ref.norm()) <= 2e-6
    if db is not None:
        assert torch.all((f64(db) - dld.sum(0)).abs() <= (n + 12) * U * dld.abs().sum(0) + 1e-38)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,E", [
    (1, 32, 1), (1, 128, 8), (64, 128, 8), (3, 2048, 460), (130, 96, 65), (257, 416, 33),
    (100, 1120, 1024), (511, 160, 127), (1500, 256, 130),
])
def test_router_bwd(cuda_ok, T, d, E, act):
    check_router(T, d, E, act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [
    dict(want="x"), dict(want="w"), dict(want="b"), dict(want="xb"), dict(want="wb"),
    dict(dx_given=False), dict(alias=True), dict(valid=True), dict(valid=True, alias=True),
    dict(valid=True, dx_given=False, want="x"), dict(valid="none"),
])
def test_router_bwd_variants(cuda_ok, act, kw):
    kw = dict(kw)
    if kw.get("valid") == "none":
        kw["valid"] = torch.zeros(150, dtype=torch.bool)
    elif kw.get("valid"):
        kw["valid"] = torch.rand(150, generator=gen(4)) > 0.3
    check_router(150, 224, 70, act, **kw)


def same_or_near(got, ref, tol):
    """Infinities and NaN as in ref, the rest within tol."""
    got = f64(got)
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.isinf(), ref.isinf()) and torch.equal(got[ref.isinf()], ref[ref.isinf()])
    fin = ref.isfinite()
    assert torch.all(((got - ref).abs() <= tol)[fin])


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,E", [(12, 64, 1), (70, 96, 20), (300, 256, 130), (600, 160, 65)])
def test_router_bwd_infinities(cuda_ok, T, d, E, act, masked):
    """Infinities and NaN in rows that take part give what float32 sums give
    and stay in their rows and columns; in masked rows they reach nothing."""
    x, w, dl, dx_in = router_case(T, d, E, act, T * d)
    x[3, 5], x[4, 7], x[9, 30] = np.inf, -np.inf, np.nan
    x[1, 2] = np.inf
    dl[1] = torch.where(torch.arange(E) % 2 == 0, 0.5, -2.0)     # (one bf16 plane)
    x[8, 40] = np.inf
    dl[8] = 0
    dl[2, 0], dl[6, E - 1] = -np.inf, np.nan
    w[1, 0], w[8, E - 1] = np.inf, np.nan
    dx_in[5, 3] = -np.inf
    valid = torch.arange(T) % 4 != 2 if masked else None
    if masked:      # (the rows 2 and 6 of dl are masked now; so is this one)
        x[10], dl[10] = np.nan, np.inf
    dx, dw, db = run_router(dims(T, d, E, 1, act), x, w, valid, dl, dx_in, "xwb")
    on = torch.ones(T, dtype=torch.bool) if valid is None else valid
    xd, dld, wd = x[on].double(), dl[on].double(), w.double()
    share = dld[:, None, :] * wd[None]
    ref, mag = dx_in.double(), torch.zeros(T, d, dtype=torch.float64)
    ref[on] += share.sum(2)
    mag[on] = share.abs().sum(2)
    half = HALF_ACT[act]
    same_or_near(dx, ref, half * ref.abs() * (1 + half) + (E + 8) * U * (mag + ref.abs()) +
                 (2.0 ** -15 * mag if act == "bf16" else 0))
    prod = xd[:, :, None] * dld[:, None, :]
    same_or_near(dw, prod.sum(0), (T + 12) * U * prod.abs().sum(0))
    same_or_near(db, dld.sum(0), (T + 12) * U * dld.abs().sum(0))


def hard_values(n, seed):
    """Significands whose lower bits are most when the leading 8 or 16 are
    taken off: just below and above the steps of bf16, all ones, random ones."""
    g = gen(seed)
    near = torch.tensor([2.0 ** -7 - 2.0 ** -23, 2.0 ** -8 - 2.0 ** -23, 2.0 ** -8 + 2.0 ** -23,
                         2.0 ** -7 + 2.0 ** -15 - 2.0 ** -23, 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -23,
                         1 - 2.0 ** -23, 2.0 ** -7 - 2.0 ** -16 - 2.0 ** -22, 2.0 ** -6 - 2.0 ** -23])
    v = 1 + torch.where(torch.rand(n, generator=g) < 0.5, near[torch.randint(0, 8, (n,), generator=g)],
                        torch.rand(n, generator=g) * 2.0 ** -6)
    return v * 2.0 ** torch.randint(-20, 20, (n,), generator=g) * torch.sign(torch.randn(n, generator=g))


def test_router_bwd_single_products_keep_float32(cuda_ok):
    """One product per sum: at most 2^-24 of it left out (1 U, and 2^-10 of
    that), five additions of plane products to the sum (5 U)."""
    T, d, E = 300, 256, 130
    dl, w = hard_values(T, 1)[:, None], hard_values(d, 2)[:, None]
    dx, _, _ = run_router(dims(T, d, 1, 1, "f32"), torch.zeros(T, d), w, None, dl, None, "x")
    ref = dl.double() @ w.double().t()
    assert torch.all((f64(dx) - ref).abs() <= 7 * U * ref.abs())
    for n, act in ((E, "f32"), (7, "f32"), (E, "bf16")):
        x, dl = hard_values(d, 3)[None].to(act_t(act)), hard_values(n, 4)[None]
        _, dw, _ = run_router(dims(1, d, n, 1, act), x, torch.zeros(d, n), None, dl, None, "w")
        ref = x.double().t() @ dl.double()
        assert torch.all((f64(dw) - ref).abs() <= 7 * U * ref.abs())


def test_router_bwd_bf16_dx_where_the_sum_cancels(cuda_ok):
    """dx_in takes the product's bf16 value off, so that the operands' 16 bits
    show: 2^-17 of each (rounded), 2^-16 for the product of what is below their
    leading 8 bits, float32 additions, one rounding of what is left."""
    T, d = 300, 256
    dl, w = hard_values(T, 5)[:, None], hard_values(d, 6)[:, None]
    prod = dl.double() @ w.double().t()
    dx_in = (-prod).to(torch.bfloat16)
    dx, _, _ = run_router(dims(T, d, 1, 1, "bf16"), torch.zeros(T, d).bfloat16(), w, None, dl, dx_in, "x")
    ref = prod + dx_in.double()
    tol = (2.0 ** -15 * (1 + 2.0 ** -7) + 8 * U) * prod.abs()
    assert torch.all((f64(dx) - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_router_bwd_next_to_the_largest_number(cuda_ok, act):
    """Operands and sums that a rounding to 8 bits would take to infinity."""
    T, d, E = 40, 64, 33
    big = torch.finfo(torch.float32).max
    x, w, dl = torch.zeros(T, d), torch.zeros(d, E), torch.zeros(T, E)
    dl[3, 4], dl[5, 6], dl[7, 8] = big, -big * (1 - 2.0 ** -9), 2.0 ** -100
    w[1, 4], w[2, 6], w[3, 4] = 2.0 ** -110, 1.0, 0.75
    w[5, 4] = 2.0                         # (past the largest number: infinite)
    x[3, 9], x[5, 10], x[7, 11] = 2.0 ** -100, 1.0, 2.0 ** 127
    if act == "f32":
        w[4, 8], x[7, 12] = big, big
    x = x.to(act_t(act))
    dx, dw, _ = run_router(dims(T, d, E, 1, act), x, w, None, dl, None, "xw")
    rx, rw = dl.double() @ w.double().t(), x.double().t() @ dl.double()
    rx[rx > big] = np.inf
    half = HALF_ACT[act]
    if act == "bf16":
        # bf16's last step ends at top; operands kept to 16 bits move a sum by up
        # to 2^-15 of it, so one that is 2^-24 from top may end on either side
        top = (2 - 2.0 ** -8) * 2.0 ** 127
        edge = (rx.abs() / top - 1).abs() <= 2.0 ** -15
        assert int(edge.sum()) == 1 and float(f64(dx)[edge].abs()) >= top * (1 - 2.0 ** -8)
        dx = torch.where(edge.to(DEV), 0, dx)
        rx = torch.where(edge, 0.0, torch.where(rx.abs() >= top, torch.sign(rx) * np.inf, rx))
    same_or_near(dx, rx, (half + 7 * U + (2.0 ** -15 * 1.01 if act == "bf16" else 0)) * rx.abs())
    same_or_near(dw, rw, 7 * U * rw.abs())


def test_router_bwd_workspace_is_for_the_weight_gradient(cuda_ok):
    """dx and db alone need none; dw_router without one is refused."""
    T, d, E = 2000, 96, 20
    x, w, dl, dx_in = router_case(T, d, E, "bf16", 3)
    dm = dims(T, d, E, 1)
    assert B.moe_workspace_size(dm, B.CALL_ROUTER_BWD) > 0
    ref_dx, _, ref_db = run_router(dm, x, w, None, dl, dx_in, "xb")
    t = [v.to(DEV) for v in (x, w, dl, dx_in)]
    dx, dw, db = torch.empty_like(t[0]), torch.empty_like(t[1]), torch.empty(E, device=DEV)
    B.moe_router_bwd(dm, None, t[1], None, t[2], t[3], dx, None, db, None)
    torch.cuda.synchronize()
    assert torch.equal(dx, ref_dx) and torch.equal(db, ref_db)
    with pytest.raises(B.MoeError, match="workspace"):
        B.moe_router_bwd(dm, t[0], t[1], None, t[2], t[3], dx, dw, db, None)


def test_router_bwd_is_repeatable(cuda_ok):
    x, w, dl, dx_in = router_case(2000, 256, 100, "bf16", 9)
    a = run_router(dims(2000, 256, 100, 1), x, w, None, dl, dx_in, "xwb")
    b = run_router(dims(2000, 256, 100, 1), x, w, None, dl, dx_in, "xwb")
    assert all(torch.equal(p, q) for p, q in zip(a, b))


# ----------------------------------------------------------------- together --

def layer(T=300, E=24, k=4, act="bf16", seed=0, d=256):
    from sparse_moe_expert_fp32_amd.layer import DeviceLayer
    cfg = configs.LayerConfig("rt", 500, T=T, d=d, E=E, k=k, f=128, r=16,
                              group=128, act=act, router_bias_var=0.5, train=True)
    L = DeviceLayer(cfg, inputs.generate(cfg, seed), device=DEV, want_logits=True)
    L.init_router_training()
    L.bal_dloss.fill_(0.3)
    return cfg, L


RESULTS = ("bal_loss", "bal_counts", "bal_prob", "dlogits", "dx", "dw_router", "db_router")


def test_layer_router_training_step(cuda_ok):
    """A float32 layer: the router's gradients of loss = <dy, y> + 0.3 balance
    against float64 autograd through router, softmax gates and the experts'
    outputs, with the selection held fixed."""
    cfg, L = layer(T=60, E=12, k=3, act="f32", d=128)
    L.router_train_step()
    torch.cuda.synchronize()
    x, w, b = (f64(L.t[n]) for n in ("x", "w_router", "b_router"))
    w.requires_grad_(True)
    b.requires_grad_(True)
    logits = x @ w + b
    idx = L.topk_idx.cpu().long()
    gates = torch.softmax(logits.gather(1, idx), 1)
    o = f64(L.e_out)[L.slot_pos.cpu().long()].reshape(cfg.T, cfg.k, cfg.d)
    y = (gates[:, :, None] * o).sum(1)
    counts = torch.bincount(idx.reshape(-1), minlength=cfg.E).double()
    bal = cfg.E * (counts / cfg.S * torch.softmax(logits, 1).mean(0)).sum()
    ((y * f64(L.t["dy"])).sum() + 0.3 * bal).backward()
    assert abs(float(L.bal_loss) - float(bal.detach())) <= 1e-5 * float(bal.detach())
    # float32 logits over d = 128 and dot products over d: 1e-5 of the norm
    for got, ref in ((L.dw_router, w.grad), (L.db_router, b.grad)):
        assert float((f64(got) - ref).norm() / ref.norm()) <= 1e-5


def test_router_training_dx_adds_the_balance_share(cuda_ok):
    cfg, L = layer()
    L.train_step()
    torch.cuda.synchronize()
    before = f64(L.dx)
    L.balance()
    L.router_bwd()
    torch.cuda.synchronize()
    share = f64(L.dlogits_bal) @ f64(L.t["w_router"]).t()
    ref = before + share
    assert torch.all((f64(L.dx) - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + 1e-6 * share.abs().max())


def test_router_training_without_a_balance_weight(cuda_ok):
    """A step whose caller has filled no bal_dloss: the balance loss weighs
    nothing, whatever the memory held."""
    cfg, L = layer()
    torch.use_deterministic_algorithms(True)      # (fills new memory with NaN)
    try:
        L.init_router_training()
    finally:
        torch.use_deterministic_algorithms(False)
    L.train_step()
    torch.cuda.synchronize()
    dx = L.dx.clone()
    L.router_train_step()
    torch.cuda.synchronize()
    assert float(L.bal_dloss) == 0 and torch.all(L.dlogits_bal == 0)
    assert torch.equal(L.dx, dx) and torch.isfinite(L.dw_router).all()


def test_router_training_on_a_side_stream_and_in_a_graph(cuda_ok):
    """The step captured once and replayed between eager steps of the same
    layer gives the eager bits on every replay."""
    cfg, L = layer()
    valid = (torch.arange(cfg.T) % 5 != 0).to(DEV)
    L.router_train_step(valid)
    torch.cuda.synchronize()
    ref = {n: getattr(L, n).clone() for n in RESULTS}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.router_train_step(valid)
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(L, n), ref[n]) for n in RESULTS)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.router_train_step(valid)
    for _ in range(4):
        for n in RESULTS:
            getattr(L, n).fill_(-3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(L, n), ref[n]) for n in RESULTS)
        L.router_train_step(valid)
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(L, n), ref[n]) for n in RESULTS)


def test_router_optimizer_step(cuda_ok):
    """The router's own AdamW step moves w_router and b_router as the call on
    copies of them does."""
    cfg, L = layer(T=50, E=8, k=2)
    L.router_train_step()
    w, b = L.t["w_router"].clone(), L.t["b_router"].clone()
    L.router_optimizer_step(lr=1e-2)
    h = B.adamw_hparams(1e-2, 0.9, 0.95, 1e-8, 0.0, 1)
    for master, g in ((w, L.dw_router), (b, L.db_router)):
        m, v = torch.zeros_like(master), torch.zeros_like(master)
        B.moe_adamw_step(h, master, g, m, v)
    torch.cuda.synchronize()
    assert torch.equal(L.t["w_router"], w) and torch.equal(L.t["b_router"], b)


def test_two_layers_on_two_streams(cuda_ok):
    """Each layer has its own workspaces: steps of two layers that overlap on
    two streams give the bits that they give alone."""
    a, b = layer(T=300, seed=1)[1], layer(T=900, E=40, seed=2)[1]
    ref = []
    for L in (a, b):
        L.router_train_step()
        torch.cuda.synchronize()
        ref.append({n: getattr(L, n).clone() for n in RESULTS})
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for L in (a, b):
            for n in RESULTS:
                getattr(L, n).fill_(-3)
        torch.cuda.synchronize()
        a.router_train_step(stream=sa)
        b.router_train_step(stream=sb)
        torch.cuda.synchronize()
        for L, r in zip((a, b), ref):
            assert all(torch.equal(getattr(L, n), r[n]) for n in RESULTS)


def test_binding_refuses_wrong_tensors(cuda_ok):
    cfg, L = layer(T=20, E=8, k=2)
    L.forward()
    with pytest.raises(B.MoeError, match="counts"):
        B.moe_balance_fwd(L.dm, L.logits, L.topk_idx, None, L.bal_loss, L.bal_counts[:-1],
                          L.bal_prob, L.bal_stats, L.ws[B.CALL_BALANCE_FWD])
    with pytest.raises(B.MoeError, match="logits"):
        B.moe_balance_bwd(L.dm, L.logits.t(), L.bal_stats, L.bal_counts, None, L.bal_dloss, L.dlogits)
    with pytest.raises(B.MoeError, match="dx "):
        B.moe_router_bwd(L.dm, L.t["x"], L.t["w_router"], None, L.dlogits, None, L.dx.float(),
                         None, None, L.ws[B.CALL_ROUTER_BWD])
    with pytest.raises(B.MoeError, match="valid"):
        B.moe_gate_bwd(L.dm, L.t["dy"], L.e_out, L.topk_idx, L.gates, L.slot_pos,
                       torch.ones(19, dtype=torch.bool, device=DEV), None, L.dlogits)
