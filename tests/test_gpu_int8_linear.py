"""Int8 rows and products on the GPU against the definition in float64: the
quantized values and the integer sums are exact, the scales carry counted
float32 roundings (U = 2^-24) and one rounding to the output type."""
import numpy as np
import pytest
import torch

from sparse_moe_expert_fp32_amd import binding as B, configs, inputs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = "cuda:0"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.double().cpu()


# -------------------------------------------------------------------- rows --

def quant_ref(v):
    """v float32 [M][K] -> (q, scale): the quotient rounded from 64 bits (a
    quotient of two float32 numbers never falls on the wrong side of a border
    there)."""
    scale = (v.abs().max(1).values.double() / 127).float()
    s = scale.double()
    q = torch.where(s[:, None] > 0, torch.round(v.double() / s.clamp_min(1e-300)[:, None]), 0.0)
    return q.clamp(-127, 127).to(torch.int8), scale


def run_quant(x, K, **kw):
    M = x.shape[0]
    ld = kw.pop("ldq", B.moe_i8_stride(K))
    q = torch.full((M, ld), 55, dtype=torch.int8, device=DEV)
    s = torch.full((M,), -77.0, device=DEV)
    B.moe_quant_i8(x, q, s, **kw)
    torch.cuda.synchronize()
    return q, s


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 2048), (5, 7), (33, 128), (64, 129), (9, 1000),
                                 (3, 4096), (2, 5001), (300, 768), (2, 20000)])
def test_quant_rows(cuda_ok, M, K, dt):
    x = torch.randn(M, K, generator=gen(M + K)).to(dt)
    q, s = run_quant(x.to(DEV), K)
    rq, rs = quant_ref(x.float())
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu()[:, :K], rq) and torch.all(q[:, K:] == 0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [200, 768, 1027, 2048, 3001, 4096, 4100])
def test_quant_many_rows(cuda_ok, K, dt):
    """Row counts at which a wave takes a row; also by expert, and with rows
    behind the last expert."""
    M = 2100
    x = torch.randn(M, K, generator=gen(K)).to(dt)
    q, s = run_quant(x.to(DEV), K)
    rq, rs = quant_ref(x.float())
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu()[:, :K], rq)
    assert torch.all(q[:, K:] == 0)
    E = 70
    counts = torch.randint(0, 60, (E,), generator=gen(1))
    off = torch.cat([torch.zeros(1), torch.cumsum(counts, 0).clamp(max=M - 3)]).to(torch.int32)
    S = int(off[-1])
    cs = torch.rand(E, K, generator=gen(2)) + 0.1
    q, s = run_quant(x.to(DEV), K, col_scale=cs.to(DEV), offsets=off.to(DEV))
    e = torch.searchsorted(off[1:].contiguous(), torch.arange(S, dtype=torch.int32), right=True)
    rq, rs = quant_ref(x[:S].float() * cs[e])
    assert torch.equal(s.cpu()[:S], rs) and torch.equal(q.cpu()[:S, :K], rq)
    assert torch.all(q[S:] == 55) and torch.all(s[S:] == -77)


def test_quant_more_rows_than_a_launch(cuda_ok):
    """Rows of more than one launch (2^22 each), with the last expert's end in
    the second one."""
    M, K = (1 << 22) + 700, 24
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(M, K, generator=g, device=DEV)
    off = torch.tensor([0, 5, (1 << 22) + 100, M - 300], dtype=torch.int32, device=DEV)
    cs = torch.rand(3, K, generator=g, device=DEV) + 0.1
    q, s = run_quant(x, K, col_scale=cs, offsets=off)
    S = M - 300
    for i, j, e in ((0, 5, 0), (5, 2000, 1), ((1 << 22) - 500, (1 << 22) + 100, 1), ((1 << 22) + 100, S, 2)):
        rq, rs = quant_ref(x[i:j].cpu() * cs[e].cpu())
        assert torch.equal(s[i:j].cpu(), rs) and torch.equal(q[i:j, :K].cpu(), rq)
    assert torch.all(q[:S, K:] == 0) and torch.all(q[S:] == 55) and torch.all(s[S:] == -77)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_quant_ties_and_extremes(cuda_ok, dt):
    """Quotients that end in one half go to the even side; zeros, subnormal
    and huge rows, and rows with values that are no numbers."""
    K = 300
    x = torch.zeros(12, K)
    ints = torch.arange(K) % 255 - 127
    x[0] = ints.float() * 0.5                      # scale 0.5: halves at odd places
    x[0, 0] = 63.5
    x[1] = torch.where(torch.arange(K) % 2 == 0, 63.5, -31.75)   # amax / 2, amax / 4
    x[1, 5] = 127.0
    x[3] = torch.randn(K, generator=gen(1)) * 1e-39
    x[4] = torch.randn(K, generator=gen(2)) * 1e-45
    x[5] = torch.randn(K, generator=gen(3)) * 1e37
    x[6, 17] = float("nan")
    x[7] = 1.0
    x[7, 100] = float("inf")
    x[8, 3] = -5.0
    x[9] = torch.randn(K, generator=gen(4)) * 1e-30
    x[10, :] = torch.finfo(torch.float32).max if dt == torch.float32 else 3e38
    x[11] = torch.linspace(-1, 1, K)
    x = x.to(dt)
    q, s = run_quant(x.to(DEV), K)
    fine = [i for i in range(12) if i not in (6, 7)]
    rq, rs = quant_ref(x.float()[fine])
    assert torch.equal(s.cpu()[fine], rs)
    assert torch.equal(q.cpu()[fine][:, :K], rq)
    assert s[2] == 0 and torch.all(q[2] == 0)
    for i in (6, 7):
        assert torch.isnan(s[i]) and torch.all(q[i] == 0)


@pytest.mark.parametrize("M", [40, 2100])
def test_quant_next_to_a_half(cuda_ok, M):
    """Quotients a few float32 steps to either side of n + 1/2, and on it, in
    the first columns, in the middle of a row and in its last chunk."""
    K = 1500
    g = gen(M)
    top = (torch.rand(M, 1, generator=g) + 0.5) * 2.0 ** torch.randint(-40, 40, (M, 1), generator=g)
    s = (top.double() / 127).float()
    half = torch.randint(-127, 127, (M, K), generator=g).double() + 0.5
    v = (half * s.double()).float()
    step = torch.randint(-3, 4, (M, K), generator=g)
    v = (v.view(torch.int32) + step.to(torch.int32)).view(torch.float32)
    v[:, 700:1490] = torch.randn(M, 790, generator=g) * top / 8   # (most chunks are ordinary)
    v = torch.minimum(torch.maximum(v, -top), top)
    v[:, 9] = top[:, 0]
    q, sc = run_quant(v.to(DEV), K)
    rq, rs = quant_ref(v)
    assert torch.equal(sc.cpu(), rs) and torch.equal(q.cpu()[:, :K], rq)


def test_quant_strides_and_wider_rows(cuda_ok):
    """Rows of a wider matrix off a 16-byte boundary, and q wider than needed."""
    for off in (0, 1, 8):
        wide = torch.randn(20, 333, generator=gen(off)).bfloat16()
        x = wide.to(DEV)[:, off:off + 200]
        q, s = run_quant(x, 200, ldq=272)
        rq, rs = quant_ref(wide[:, off:off + 200].float())
        assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu()[:, :200], rq)
        assert torch.all(q[:, 200:] == 0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [1, 100, 768, 4100])
def test_quant_channel_scales_by_expert(cuda_ok, K, dt):
    """The row's expert picks the multipliers; rows behind the last expert
    stay as they were."""
    counts = [0, 3, 0, 1, 7, 0, 5, 0]
    E, S = len(counts), sum(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    x = torch.randn(S + 4, K, generator=gen(K)).to(dt)
    cs = torch.rand(E, K, generator=gen(9)) + 0.1
    q, s = run_quant(x.to(DEV), K, col_scale=cs.to(DEV), offsets=off.to(DEV))
    e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    rq, rs = quant_ref(x[:S].float() * cs[e])       # one float32 product
    assert torch.equal(s.cpu()[:S], rs) and torch.equal(q.cpu()[:S, :K], rq)
    assert torch.all(q[S:] == 55) and torch.all(s[S:] == -77)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 1), (4, 768), (37, 1001), (3, 5000), (2050, 768), (2048, 130)])
def test_quant_swiglu(cuda_ok, M, K, dt):
    gu = (torch.randn(M, 2 * K, generator=gen(M * K)) * 3).to(dt)
    gu[0, 0] = -200.0                                # exp(200) overflows: silu is 0
    d = gu.to(DEV)
    q, s = run_quant(d[:, :K], K, mul=d[:, K:])
    g, u = gu[:, :K].double(), gu[:, K:].double()
    v = g * torch.sigmoid(g) * u
    amax = v.abs().max(1).values
    # exp, 1 + e, the quotient and the product: at most 8 roundings of v
    assert torch.all((f64(s) - amax / 127).abs() <= 10 * U * amax / 127 + 1e-44)
    got = f64(q)[:, :K] * f64(s)[:, None]
    assert torch.all((got - v).abs() <= f64(s)[:, None] * (0.5 + 127 * 10 * U) + 8 * U * v.abs() + 1e-44)
    assert torch.all(q[:, K:] == 0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lo,hi", [(-30, -20), (-86, -70), (-86, 5)])
@pytest.mark.parametrize("M,K", [(3, 300), (2100, 129), (2050, 768)])
def test_quant_swiglu_negative_gates(cuda_ok, M, K, lo, hi, dt):
    """Gates far below 0 in the whole row: the row's values are e^x in size, and
    every one keeps float32's accuracy (expf 2 U, 1 + e, the quotient, the
    product, the scale's quotient: 6 U)."""
    g = gen(M + K)
    gu = torch.rand(M, 2 * K, generator=g) * (hi - lo) + lo
    gu[:, K:] = torch.randn(M, K, generator=g)
    gu = gu.to(dt)
    d = gu.to(DEV)
    q, s = run_quant(d[:, :K], K, mul=d[:, K:])
    x, u = gu[:, :K].double(), gu[:, K:].double()
    v = x * torch.sigmoid(x) * u
    amax = v.abs().max(1).values
    assert torch.all((f64(s) - amax / 127).abs() <= 7 * U * amax / 127)
    got = f64(q)[:, :K] * f64(s)[:, None]
    assert torch.all((got - v).abs() <= f64(s)[:, None] * (0.5 + 127 * 8 * U) + 8 * U * v.abs())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [100, 129, 768, 4100])
@pytest.mark.parametrize("M", [30, 2100])
def test_quant_swiglu_with_channel_scales(cuda_ok, M, K, dt):
    """SwiGLU and the expert's channel scales in one call; rows behind the last
    expert stay as they were."""
    E = 9
    g = gen(M * K)
    cut = torch.sort(torch.randint(0, M - 2, (E - 1,), generator=g)).values
    off = torch.cat([torch.zeros(1), cut, torch.tensor([M - 3.0])]).to(torch.int32)
    S = int(off[-1])
    gu = (torch.randn(M, 2 * K, generator=g) * 3).to(dt)
    cs = torch.rand(E, K, generator=g) + 0.1
    d = gu.to(DEV)
    q, s = run_quant(d[:, :K], K, mul=d[:, K:], col_scale=cs.to(DEV), offsets=off.to(DEV))
    e = torch.searchsorted(off[1:].contiguous(), torch.arange(S, dtype=torch.int32), right=True)
    x, u = gu[:S, :K].double(), gu[:S, K:].double()
    v = x * torch.sigmoid(x) * u * cs[e].double()
    amax = v.abs().max(1).values
    assert torch.all((f64(s)[:S] - amax / 127).abs() <= 8 * U * amax / 127)   # (one product more)
    got = f64(q)[:S, :K] * f64(s)[:S, None]
    assert torch.all((got - v).abs() <= f64(s)[:S, None] * (0.5 + 127 * 9 * U) + 9 * U * v.abs())
    assert torch.all(q[:S, K:] == 0) and torch.all(q[S:] == 55) and torch.all(s[S:] == -77)


# ---------------------------------------------------------------- products --

def linear_case(counts, N, K, dt, seed, div=1, pad=0, scales=True, src=True):
    g = gen(seed)
    E, S = len(counts), sum(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    R = max(1, (S + div - 1) // div)
    a = torch.zeros(R, B.moe_i8_stride(K), dtype=torch.int8)
    a[:, :K] = torch.randint(-127, 128, (R, K), generator=g).to(torch.int8)
    ldw = (K + 15) // 16 * 16 + 16 * pad
    w = torch.randint(-128, 128, (E, N, ldw), generator=g).to(torch.int8)   # what stands behind K is not used
    a_s = torch.rand(R, generator=g) + 0.01
    w_s = (torch.rand(E, N, generator=g) + 0.01) * 1e-3 if scales else None
    rows = torch.randint(0, R * div, (S,), generator=g).to(torch.int32) if src else None
    return off, a, w[:, :, :K], a_s, w_s, rows


def linear_ref(off, a, w, a_s, w_s, rows, div):
    S, K = int(off[-1]), w.shape[2]
    r = (rows.long() // div) if rows is not None else torch.arange(S)
    out = torch.zeros(S, w.shape[1], dtype=torch.float64)
    for e in range(w.shape[0]):
        i, j = int(off[e]), int(off[e + 1])
        if j > i:
            out[i:j] = a[r[i:j], :K].double() @ w[e].double().t()
            out[i:j] *= a_s[r[i:j]].double()[:, None] * (w_s[e].double() if w_s is not None else 1.0)
    return out


def check_linear(counts, N, K, dt, seed=0, div=1, pad=0, scales=True, src=True, extra=3, wide=5,
                 no_offsets=False):
    off, a, w, a_s, w_s, rows = linear_case(counts, N, K, dt, seed, div, pad, scales, src)
    S = int(off[-1])
    if no_offsets:
        extra = 0
    if not src and S + extra > a.shape[0]:
        extra = a.shape[0] - S
    out = torch.full((S + extra, N + wide), -77.0, dtype=dt, device=DEV)
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    wd = torch.empty(w.shape[0], N, w.stride(1), dtype=torch.int8, device=DEV)
    wd.copy_(torch.as_strided(w, wd.shape, w.stride()))
    src_d = None
    if rows is not None:
        src_d = torch.zeros(S + extra, dtype=torch.int32)
        src_d[:S] = rows
        src_d = src_d.to(DEV)
    B.moe_i8_linear(to(a), to(a_s), wd[:, :, :K], to(w_s), out[:, :N],
                    offsets=None if no_offsets else to(off), row_src=src_d, row_div=div)
    torch.cuda.synchronize()
    ref = linear_ref(off, a, w, a_s, w_s, rows, div)
    got = f64(out)
    # the sum to float32, the product of the scales, their product: 3 roundings
    tol = ref.abs() * (3.1 * U + HALF[dt] * (1 + 4 * U))
    bad = (got[:S, :N] - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4])
    assert torch.all(got[S:] == -77) and torch.all(got[:, N:] == -77)   # left as it was
    return out


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 2048, 2048), (2, 33, 65), (16, 16, 64), (17, 100, 128), (64, 64, 192),
    (65, 129, 1000), (127, 257, 511), (300, 1001, 1111), (512, 768, 384), (1030, 130, 260),
])
def test_linear_one_matrix(cuda_ok, M, N, K, dt):
    check_linear([M], N, K, dt, seed=M + N, src=False)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K,div", [
    ([0, 3, 0, 1, 16, 0, 17, 2], 96, 160, 4),        # decode-like
    ([0] * 20 + [1] + [0] * 30, 64, 128, 1),         # a single row
    ([5, 130, 0, 64, 300, 1], 200, 272, 6),
    ([700, 0, 0, 20], 144, 129, 12),
    ([257, 255, 256, 129], 520, 640, 3),
    ([1] * 90, 70, 100, 2),
    ([33, 40, 31, 65, 50, 0, 48, 90], 300, 2000, 5),
])
def test_linear_experts(cuda_ok, counts, N, K, div, dt):
    check_linear(counts, N, K, dt, seed=N + K, div=div)


def spread(E, total, seed, odd=()):
    """E row counts of about `total` in all: the given ones, empty ones, and
    skewed ones."""
    c = -torch.log1p(-torch.rand(E, generator=gen(seed)) * 0.999)
    c = (c / c.sum() * total).int().tolist()
    c[: len(odd)] = odd
    c[len(odd)] = 0
    return c


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,total,odd,N,K", [
    (64, 300, (16, 17, 32, 33, 1), 1000, 200),                    # a few rows a matrix
    (100, 500, (40,), 513, 1040),
    (24, 700, (64, 65, 128, 129, 1), 700, 384),                   # tens of rows
    (32, 2600, (64, 65, 128, 129, 256, 3), 1030, 272),            # about a hundred
    (32, 6000, (64, 65, 128, 129, 192, 193, 256, 257, 600, 1), 1030, 160),   # hundreds
    (40, 7000, (255, 31), 904, 129),
])
def test_linear_every_tile_height(cuda_ok, E, total, odd, N, K, dt):
    check_linear(spread(E, total, E + K, list(odd)), N, K, dt, seed=E, div=3)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,total,odd,N,K", [
    (24, 1800, (64, 65, 96, 97, 128, 129, 1, 33, 31), 8203, 200),        # a hundred rows, much work
    (24, 5200, (1, 31, 33, 63, 65, 95, 97, 127, 129, 159, 161, 191, 193, 223, 225, 255, 257, 600),
     14001, 129),                                                       # hundreds
    (1, 0, (), 7300, 70),                                               # one matrix, 2300 rows
])
def test_linear_every_tile_height_with_many_channels(cuda_ok, E, total, odd, N, K, dt):
    counts = [2300] if E == 1 else spread(E, total, E + K, list(odd))
    check_linear(counts, N, K, dt, seed=E, div=3 if E > 1 else 1, src=E > 1)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(3, 100, 6000), (17, 40, 8192), (5, 33, 8300), (20, 130, 4100),
                                   (2100, 300, 5000), (1500, 2100, 70)])
def test_linear_long_rows_and_many_rows(cuda_ok, M, N, K, dt):
    check_linear([M], N, K, dt, seed=K, src=False)


@pytest.mark.parametrize("kw", [
    dict(scales=False), dict(pad=3), dict(wide=0), dict(wide=8), dict(wide=1), dict(src=False),
    dict(extra=0), dict(extra=200),
])
def test_linear_variants(cuda_ok, kw):
    for dt in (torch.float32, torch.bfloat16):
        check_linear([40, 0, 150, 7], 136, 208, dt, div=1, **kw)


def test_linear_no_rows_at_all(cuda_ok):
    check_linear([0, 0, 0], 64, 128, torch.bfloat16, extra=9)
    out = torch.full((0, 64), 1.0, device=DEV)
    a = torch.zeros(1, 128, dtype=torch.int8, device=DEV)
    B.moe_i8_linear(a, torch.ones(1, device=DEV), torch.zeros(1, 64, 128, dtype=torch.int8, device=DEV),
                    None, out, row_src=torch.zeros(0, dtype=torch.int32, device=DEV))


def test_linear_without_offsets_takes_every_row(cuda_ok):
    for M in (1, 40, 333):
        check_linear([M], 160, 224, torch.bfloat16, src=False, no_offsets=True)


def test_linear_largest_sums_and_lowest_weights(cuda_ok):
    """-128 weights against +-127 rows over K = 65536: sums near 2^30, exact."""
    K, N, M = 65536, 8, 20
    a = torch.full((M, K), 127, dtype=torch.int8)
    a[1::2] = -127
    w = torch.full((1, N, K), -128, dtype=torch.int8)
    w[0, 3] = 127
    out = torch.empty(M, N, device=DEV)
    B.moe_i8_linear(a.to(DEV), torch.ones(M, device=DEV), w.to(DEV), None, out)
    ref = a.double() @ w[0].double().t()
    assert torch.all((f64(out) - ref).abs() <= U * ref.abs())


def test_linear_nan_scale_marks_its_row_only(cuda_ok):
    off, a, w, a_s, w_s, rows = linear_case([30, 20], 50, 96, torch.bfloat16, 3, src=False)
    a_s[13] = float("nan")
    out = torch.empty(50, 50, device=DEV)
    B.moe_i8_linear(a.to(DEV), a_s.to(DEV), w.contiguous().to(DEV), w_s.to(DEV), out, offsets=off.to(DEV))
    nan = torch.isnan(out).cpu()
    assert nan[13].all() and int(nan.sum()) == 50


@pytest.mark.parametrize("short", [True, False])
def test_linear_matrices_past_32_bits(cuda_ok, short):
    """540 matrices of 4 MiB: byte offsets past 2^31; the rows of the last
    experts come from there."""
    E, N, K = 540, 2048, 2048
    counts = [0] * E
    counts[0], counts[-1], counts[E - 3] = (3, 5, 2) if short else (200, 300, 1500)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    S = sum(counts)
    w = torch.zeros(E, N, K, dtype=torch.int8, device=DEV)
    for e in (0, E - 3, E - 1):
        w[e] = torch.randint(-128, 128, (N, K), generator=gen(e)).to(torch.int8).to(DEV)
    a = torch.randint(-127, 128, (S, K), generator=gen(1)).to(torch.int8)
    a_s = torch.rand(S, generator=gen(2))
    out = torch.empty(S, N, device=DEV)
    B.moe_i8_linear(a.to(DEV), a_s.to(DEV), w, None, out, offsets=off.to(DEV))
    for e in (0, E - 3, E - 1):
        i, j = int(off[e]), int(off[e + 1])
        ref = (a[i:j].to(DEV).double() @ w[e].double().t()) * a_s[i:j].to(DEV).double()[:, None]
        assert torch.all((out[i:j].double() - ref).abs() <= ref.abs() * 3.1 * U)


@pytest.mark.parametrize("looked_up", [False, True])
def test_linear_rows_past_32_bits(cuda_ok, looked_up):
    """2097452 rows of 2 KiB: the last ones lie behind 2^32 bytes."""
    R, N, K = 2097152 + 300, 32, 2048
    at = torch.tensor([0, 5, 255, 256, 2097151, 2097152, R - 257, R - 1])
    a = torch.zeros(R, K, dtype=torch.int8, device=DEV)
    vals = torch.randint(-127, 128, (len(at), K), generator=gen(1)).to(torch.int8).to(DEV)
    a[at.to(DEV)] = vals
    a_s = torch.rand(R, device=DEV)
    w = torch.randint(-128, 128, (1, N, K), generator=gen(2)).to(torch.int8).to(DEV)
    out = torch.empty(len(at) if looked_up else R, N, device=DEV)
    B.moe_i8_linear(a, a_s, w, None, out,
                    row_src=at.to(torch.int32).to(DEV) if looked_up else None)
    got = out if looked_up else out[at.to(DEV)]
    ref = (vals.double() @ w[0].double().t()) * a_s[at.to(DEV)].double()[:, None]
    assert torch.all((got.double() - ref).abs() <= ref.abs() * 3.1 * U)
    if not looked_up:
        assert int((out != 0).any(1).sum()) == len(at)   # (the other rows are 0)


def test_linear_many_rows_looked_up_past_32_bits(cuda_ok):
    """3000 rows looked up on both sides of 2^32 bytes, one matrix and several."""
    R, N, K, M = 2097152 + 300, 300, 2048, 3000
    g = torch.Generator(device=DEV).manual_seed(3)
    a = torch.randint(-127, 128, (R, K), generator=g, dtype=torch.int8, device=DEV)
    a_s = torch.rand(R, generator=g, device=DEV)
    src = torch.randint(0, R, (M,), generator=g, device=DEV).to(torch.int32)
    src[:1000] = torch.randint(2097152 - 300, R, (1000,), generator=g, device=DEV)
    rows = a[src.long()].double()
    for E in (1, 6):
        w = torch.randint(-128, 128, (E, N, K), generator=g, dtype=torch.int8, device=DEV)
        off = torch.linspace(0, M, E + 1, device=DEV).to(torch.int32) if E > 1 else None
        out = torch.empty(M, N, device=DEV)
        B.moe_i8_linear(a, a_s, w, None, out, offsets=off, row_src=src)
        at = off.tolist() if E > 1 else [0, M]
        ref = torch.cat([rows[at[e]:at[e + 1]] @ w[e].double().t() for e in range(E)])
        ref = ref * a_s[src.long()].double()[:, None]
        assert torch.all((out.double() - ref).abs() <= ref.abs() * 3.1 * U)


@pytest.mark.parametrize("wider", [0, 64])
def test_linear_one_matrix_past_32_bits(cuda_ok, wider):
    """The largest matrix there may be, 65536 x 65536, and at a longer stride."""
    N = K = 65536
    g = torch.Generator(device=DEV).manual_seed(4)
    w = torch.randint(-128, 128, (1, N, K + wider), generator=g, dtype=torch.int8, device=DEV)
    w = w[:, :, :K]
    a = torch.randint(-127, 128, (40, K), generator=g, dtype=torch.int8, device=DEV)
    out = torch.empty(40, N, device=DEV)
    B.moe_i8_linear(a, torch.ones(40, device=DEV), w, None, out)
    rows = a.double()
    for n in (0, 30000, N - 2048):
        ref = rows @ w[0, n:n + 2048].double().t()
        assert torch.all((out[:, n:n + 2048].double() - ref).abs() <= ref.abs() * U)


def test_row_sources_out_of_range_are_clamped(cuda_ok):
    a = torch.randint(-127, 128, (4, 128), generator=gen(0)).to(torch.int8)
    w = torch.randint(-128, 128, (1, 40, 128), generator=gen(1)).to(torch.int8)
    src = torch.tensor([-9, 0, 7, 8, 1 << 30], dtype=torch.int32)
    out = torch.empty(5, 40, device=DEV)
    B.moe_i8_linear(a.to(DEV), torch.ones(4, device=DEV), w.to(DEV), None, out,
                    row_src=src.to(DEV), row_div=2)
    ref = (a.double() @ w[0].double().t())[torch.tensor([0, 0, 3, 3, 3])]
    assert torch.equal(f64(out), ref)


def test_offsets_behind_the_rows_are_clamped(cuda_ok):
    """Offsets that say more rows than there are reach no row behind M."""
    off, a, w, a_s, w_s, rows = linear_case([6, 10], 40, 96, torch.float32, 3, src=False)
    big = off.clone()
    big[2] = 4000
    out = torch.full((20, 40), -77.0, device=DEV)
    B.moe_i8_linear(a.to(DEV), a_s.to(DEV), w.contiguous().to(DEV), w_s.to(DEV), out[:16], offsets=big.to(DEV))
    ref = linear_ref(off, a, w, a_s, w_s, None, 1)
    assert torch.all((f64(out)[:16] - ref).abs() <= ref.abs() * 4.1 * U) and torch.all(out[16:] == -77)


# ---------------------------------------------------------------- together --

def experts_case(T, E, k, d, f, seed=0):
    from sparse_moe_expert_fp32_amd.layer import DeviceLayer, Int8Experts
    cfg = configs.LayerConfig("i8", 600 + T, T=T, d=d, E=E, k=k, f=128, r=4, group=32, act="bf16",
                              router_bias_var=0.5)
    L = DeviceLayer(cfg, inputs.generate(cfg, seed), device=DEV)
    g = gen(seed)
    gu = torch.randint(-127, 128, (E, 2 * f, d), generator=g).to(torch.int8)
    dn = torch.randint(-127, 128, (E, d, f), generator=g).to(torch.int8)
    s_gu = (torch.rand(E, 2 * f, generator=g) + 0.5) / (73 * d ** 0.5)
    s_dn = (torch.rand(E, d, generator=g) + 0.5) / (73 * f ** 0.5)
    X = Int8Experts(gu.to(DEV), s_gu.to(DEV), dn.to(DEV), s_dn.to(DEV))
    return cfg, L, X


@pytest.mark.parametrize("T,E,k,d,f", [(1, 40, 4, 256, 96), (64, 24, 3, 384, 112), (700, 6, 2, 256, 80)])
def test_int8_experts_forward(cuda_ok, T, E, k, d, f):
    """route -> permute -> int8 experts -> combine, stage by stage: each stage
    against the definition on the GPU's own inputs to it."""
    cfg, L, X = experts_case(T, E, k, d, f)
    L.route()
    L.permute()
    gu = X.forward(L)
    L.combine()
    torch.cuda.synchronize()
    x = L.t["x"].float().cpu()
    q, s = quant_ref(x)
    tok = L.perm_src.cpu().long() // k
    off = L.offsets.cpu().tolist()
    o = torch.zeros(cfg.S, d, dtype=torch.float64)
    for e in range(E):
        i, j = off[e], off[e + 1]
        if j == i:
            continue
        # (the sums first, exact: a sum of 0 then stays 0)
        ref = q[tok[i:j]].double() @ X.gate_up[e].cpu().double().t()
        ref = ref * s[tok[i:j]].double()[:, None] * f64(X.s_gate_up[e])
        assert torch.all((f64(gu[i:j]) - ref).abs() <= ref.abs() * (HALF[torch.bfloat16] + 5 * U))
        g, u = f64(gu[i:j])[:, :f], f64(gu[i:j])[:, f:]
        h = g * torch.sigmoid(g) * u
        hs = h.abs().max(1).values / 127
        wd = X.down[e].cpu().double() * f64(X.s_down[e])[:, None]
        hq = torch.round(h / hs.clamp_min(1e-300)[:, None])
        o[i:j] = (hq @ X.down[e].cpu().double().t()) * hs[:, None] * f64(X.s_down[e])
        # a value next to a border may fall on either side: at most one step each
        near = ((h / hs.clamp_min(1e-300)[:, None]).frac().abs() - 0.5).abs() < 1e-3
        slack = near.double() * hs[:, None] @ wd.abs().t()
        assert torch.all((f64(L.e_out[i:j]) - o[i:j]).abs() <=
                         o[i:j].abs() * (HALF[torch.bfloat16] + 20 * U) + slack +
                         20 * U * (h.abs() @ wd.abs().t()))
    pos = L.slot_pos.cpu().long()
    y = (f64(L.gates)[:, :, None] * f64(L.e_out)[pos].reshape(T, k, d)).sum(1)
    assert torch.all((f64(L.y) - y).abs() <= y.abs() * HALF[torch.bfloat16] + 1e-5 * y.abs().max())


@pytest.mark.parametrize("which", ["gate_up", "down"])
def test_row_gradient(cuda_ok, which):
    """The gradient of a product's rows by the same int8 product on the
    transposed matrices: against the exact gradient of <dout, out>, off by at
    most half a quantization step of every gradient value."""
    cfg, L, X = experts_case(120, 5, 2, 256, 80)
    L.route()
    L.permute()
    w, cs = (X.gate_up, X.s_gate_up) if which == "gate_up" else (X.down, X.s_down)
    dout = torch.randn(cfg.S, w.shape[1], generator=gen(5)).bfloat16().to(DEV)
    dx = X.rows_grad(which, dout, L.offsets)
    torch.cuda.synchronize()
    off = L.offsets.cpu().tolist()
    for e in range(5):
        i, j = off[e], off[e + 1]
        if j == i:
            continue
        W = w[e].cpu().double()
        v = f64(dout[i:j]) * f64(cs[e])
        ref = v @ W                                  # d <dout, out> / d rows
        step = v.abs().max(1).values / 127
        tol = 0.5 * step[:, None] * W.abs().sum(0) * (1 + 1e-5) + HALF[torch.bfloat16] * ref.abs()
        assert torch.all((f64(dx[i:j]) - ref).abs() <= tol * (1 + HALF[torch.bfloat16]) + 1e-30)
        # and exactly the quantized definition
        q, s = quant_ref(dout[i:j].float().cpu() * cs[e].cpu())
        d = (q.double() @ W) * s.double()[:, None]
        assert torch.all((f64(dx[i:j]) - d).abs() <= d.abs() * (HALF[torch.bfloat16] + 4 * U))


def test_row_gradient_against_differences(cuda_ok):
    """<dout, out(rows)> of the dequantized product is linear in the rows:
    its difference along a direction is the gradient's product with it, up to
    half a step of every quantized gradient value."""
    N, K, M = 96, 64, 20
    g = gen(2)
    w = torch.randint(-127, 128, (1, N, K), generator=g).to(torch.int8).to(DEV)
    cs = (torch.rand(1, N, generator=g) + 0.5).to(DEV) / 500
    dout = torch.randn(M, N, generator=g).to(DEV)
    from sparse_moe_expert_fp32_amd.layer import Int8Experts
    X = Int8Experts(w, cs, w.transpose(1, 2).contiguous(), None)
    dx = X.rows_grad("gate_up", dout, None)
    W = f64(w[0]) * f64(cs[0])[:, None]
    f = lambda r: (f64(dout) * (r @ W.t())).sum(1)  # noqa: E731
    r0, step = torch.randn(M, K, generator=g).double(), torch.randn(M, K, generator=g).double()
    diff = (f(r0 + step) - f(r0 - step)) / 2
    v = f64(dout) * f64(cs[0])
    slack = 0.5 * (v.abs().max(1).values / 127) * (step.abs() @ f64(w[0]).abs().t()).sum(1) * 1.001
    assert torch.all((diff - (f64(dx) * step).sum(1)).abs() <= slack + 1e-6)


def test_int8_experts_on_a_stream_and_in_a_graph(cuda_ok):
    """Captured once, replayed between eager calls: the eager bits each time."""
    cfg, L, X = experts_case(90, 12, 3, 256, 96)

    def step():
        L.route()
        L.permute()
        X.forward(L)
        L.combine()

    step()
    torch.cuda.synchronize()
    ref = L.y.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    assert torch.equal(L.y, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        L.y.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(L.y, ref)
        step()
        torch.cuda.synchronize()
        assert torch.equal(L.y, ref)


def test_binding_refuses_wrong_tensors(cuda_ok):
    z = lambda *n, dt=torch.int8: torch.zeros(*n, dtype=dt, device=DEV)  # noqa: E731
    f = torch.float32
    with pytest.raises(B.MoeError, match="adjacent"):
        B.moe_quant_i8(z(64, 4, dt=f).t(), z(4, 128), z(4, dt=f))
    with pytest.raises(B.MoeError, match="q must"):
        B.moe_quant_i8(z(4, 200, dt=f), z(4, 128), z(4, dt=f))
    with pytest.raises(B.MoeError, match="mul"):
        B.moe_quant_i8(z(4, 100, dt=f), z(4, 128), z(4, dt=f), mul=z(4, 99, dt=f))
    with pytest.raises(B.MoeError, match="w must"):
        B.moe_i8_linear(z(4, 128), z(4, dt=f), z(1, 40, 128, dt=f), None, z(4, 40, dt=f))
    with pytest.raises(B.MoeError, match="reach its stride"):
        B.moe_i8_linear(z(4, 128), z(4, dt=f), z(1, 40 * 112)[:, :40 * 112 - 8].as_strided((1, 40, 100), (4480, 112, 1), 8),
                        None, z(4, 40, dt=f))
    with pytest.raises(B.MoeError, match="w_scale"):
        B.moe_i8_linear(z(4, 128), z(4, dt=f), z(1, 40, 112), z(41, dt=f), z(4, 40, dt=f))
    with pytest.raises(B.MoeError, match="multiple of 16"):
        B.moe_i8_linear(z(4, 128), z(4, dt=f), z(1, 40, 100), None, z(4, 40, dt=f))


def test_quant_writes_nothing_beside_its_rows(cuda_ok):
    """q as a part of a wider buffer: rows that are not adjacent are refused,
    one row is written to its own end."""
    x = torch.randn(5, 100, generator=gen(3)).to(DEV)
    room = torch.full((6, 384), 55, dtype=torch.int8, device=DEV)
    for part in (room[:5, :128], room[:5, 128:256], room[1:6, 256:]):
        with pytest.raises(B.MoeError, match="one after another"):
            B.moe_quant_i8(x, part, torch.empty(5, device=DEV))
    s = torch.empty(1, device=DEV)
    B.moe_quant_i8(x[:1], room[5:, 128:256], s)
    torch.cuda.synchronize()
    rq, rs = quant_ref(x[:1].cpu())
    assert torch.equal(room[5:, 128:228].cpu(), rq) and torch.equal(s.cpu(), rs)
    assert torch.all(room[5, 228:256] == 0)
    room[5, 128:256] = 55
    assert torch.all(room == 55)


def large_experts(E=24, N=1024, K=2048, S=600, seed=7):
    """Down products whose layout takes the GPU a while, and a gradient of them."""
    from sparse_moe_expert_fp32_amd.layer import Int8Experts
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randint(-127, 128, (E, N, K), generator=g, dtype=torch.int8, device=DEV)
    gu = torch.randint(-127, 128, (E, 2 * K, 128), generator=g, dtype=torch.int8, device=DEV)
    cs = (torch.rand(E, N, generator=g, device=DEV) + 0.5) / 1000
    off = torch.linspace(0, S, E + 1, device=DEV).to(torch.int32)
    dout = torch.randn(S, N, generator=g, device=DEV).bfloat16()
    return Int8Experts(gu, torch.ones(E, 2 * K, device=DEV), w, cs), dout, off


def rows_grad_ref(X, dout, off):
    """The quantized definition in float64, on the CPU's quantizer."""
    out, at = torch.zeros(dout.shape[0], X.down.shape[2], dtype=torch.float64), off.tolist()
    for e in range(X.E):
        i, j = at[e], at[e + 1]
        q, s = quant_ref(dout[i:j].float().cpu() * X.s_down[e].cpu())
        out[i:j] = (q.double() @ X.down[e].cpu().double()) * s.double()[:, None]
    return out


def near_bf16(got, ref):
    return bool(torch.all((f64(got) - ref).abs() <= ref.abs() * (HALF[torch.bfloat16] + 4 * U)))


def test_row_gradient_first_on_a_side_stream(cuda_ok):
    """The first call, which lays the matrices out, on a side stream while the
    current one is busy; then calls on other streams, which find the layout."""
    X, dout, off = large_experts()
    ref = rows_grad_ref(X, dout, off)
    torch.cuda.synchronize()
    s, s2, busy = torch.cuda.Stream(), torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    for _ in range(20):
        busy = busy @ busy * 1e-3
    s.wait_stream(torch.cuda.current_stream())
    first = X.rows_grad("down", dout, off, stream=s)
    other = X.rows_grad("down", dout, off, stream=s2)
    here = X.rows_grad("down", dout, off)
    torch.cuda.synchronize()
    assert near_bf16(first, ref)
    assert torch.equal(first, here) and torch.equal(first, other)


def test_row_gradient_follows_its_matrices(cuda_ok):
    """Matrices written in place or replaced after a first gradient."""
    X, dout, off = large_experts(E=5, N=272, K=160, S=90)
    assert near_bf16(X.rows_grad("down", dout, off), rows_grad_ref(X, dout, off))
    X.down.copy_(torch.flip(X.down, (2,)))
    assert near_bf16(X.rows_grad("down", dout, off), rows_grad_ref(X, dout, off))
    X.down = torch.flip(X.down, (1,)).contiguous()
    assert near_bf16(X.rows_grad("down", dout, off), rows_grad_ref(X, dout, off))
    with torch.inference_mode():
        X.down = torch.flip(X.down, (1,)).contiguous()
        assert near_bf16(X.rows_grad("down", dout, off), rows_grad_ref(X, dout, off))
        X.down.zero_()
    X.transpose()
    assert not X.rows_grad("down", dout, off).any()


def test_row_gradient_in_a_graph(cuda_ok):
    """A capture needs the layout before it; the captured product reads the
    layout that transpose() renews in place."""
    X, dout, off = large_experts(E=5, N=256, K=128, S=90)
    dx, y = torch.zeros(90, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(4, device=DEV)
    B.moe_quant_i8(dout, torch.empty(90, 256, dtype=torch.int8, device=DEV),
                   torch.empty(90, device=DEV))   # (the library is loaded on this GPU)
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        y.add_(1)
        with pytest.raises(RuntimeError, match="transpose"):
            X.rows_grad("down", dout, off)
    X.transpose()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dx.copy_(X.rows_grad("down", dout, off))
    for step in range(4):
        ref = X.rows_grad("down", dout, off)
        dx.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, ref) and near_bf16(dx, rows_grad_ref(X, dout, off))
        X.down.copy_(torch.flip(X.down, (1 + step % 2,)))
        X.transpose()


def test_linear_refuses_unsigned_matrices(cuda_ok):
    """uint8 values have no sign to read; their bytes do, as a view in int8."""
    w = torch.arange(256, device=DEV).repeat(1, 4, 1).to(torch.uint8)
    a = torch.ones(2, 256, dtype=torch.int8, device=DEV)
    out = torch.zeros(2, 4, device=DEV)
    with pytest.raises(B.MoeError, match="w must be int8"):
        B.moe_i8_linear(a, torch.ones(2, device=DEV), w, None, out)
    assert not out.any()
    B.moe_i8_linear(a, torch.ones(2, device=DEV), w.view(torch.int8), None, out)
    assert torch.all(out == -128)


def test_row_gradient_after_a_layout_that_failed(cuda_ok):
    """A matrix that cannot be laid out leaves nothing half kept."""
    X, dout, off = large_experts(E=5, N=272, K=160, S=90)
    good, X.down = X.down, X.down[0]
    with pytest.raises(ValueError):
        X.transpose()                       # (gate_up was laid out before it)
    g = torch.randn(90, X.gate_up.shape[1], generator=gen(1)).bfloat16().to(DEV)
    first = X.rows_grad("gate_up", g, off)
    X.down = good
    assert near_bf16(X.rows_grad("down", dout, off), rows_grad_ref(X, dout, off))
    assert torch.equal(X.rows_grad("gate_up", g, off), first)
