"""Host-side checks of the load-balance, router-backward and int8 calls (no
GPU needed): bad arguments are refused with the documented status before the
GPU is touched."""
import ctypes

import pytest
import torch

from sparse_moe_expert_fp32_amd import binding as B

P = 0x1000   # never dereferenced: validation fails before any HIP call


def dm(**kw):
    base = dict(T=64, d=128, E=8, k=2, f=256, r=4, group=32, act="f32")
    base.update(kw)
    return ctypes.byref(B.dims(**base))


def err():
    return B.LIB.moe_last_error().decode()


def test_workspace_sizes_of_the_new_calls():
    big = B.dims(8192, 2048, 460, 12, 768, 16, 128, "bf16")
    for c in (B.CALL_BALANCE_FWD, B.CALL_ROUTER_BWD):
        assert 0 <= B.moe_workspace_size(big, c) < 256 << 20
    assert B.moe_workspace_size(big, B.CALL_BALANCE_FWD) > 0
    out = ctypes.c_size_t(7)
    assert B.LIB.moe_workspace_size(ctypes.byref(big), 7, ctypes.byref(out)) == -1 and out.value == 7


@pytest.mark.parametrize("hole", range(2, 9))
def test_balance_fwd_refuses_null(hole):
    a = [dm(), P, P, None, P, P, P, P, P, 1 << 30, None]
    need = {2: 1, 3: 2, 4: 4, 5: 5, 6: 6, 7: 7}.get(hole)
    if need is None:                       # the workspace: missing, then too small
        a[8] = None
        assert B.LIB.moe_balance_fwd(*a) == -3
        a[8], a[9] = P, 8
        assert B.LIB.moe_balance_fwd(*a) == -3 and "workspace" in err()
        return
    a[need] = None
    assert B.LIB.moe_balance_fwd(*a) == -1 and err().startswith("moe_balance_fwd")


def test_balance_refuses_bad_dims_and_alignment():
    assert B.LIB.moe_balance_fwd(dm(E=1025), P, P, None, P, P, P, P, P, 1 << 30, None) == -1
    assert B.LIB.moe_balance_fwd(dm(), P, P, None, P, P, P, P + 4, P, 1 << 30, None) == -1
    assert B.LIB.moe_balance_fwd(dm(), P, P, None, P, P, P, P, P + 8, 1 << 30, None) == -1
    assert B.LIB.moe_balance_bwd(None, P, P, P, None, P, P, None) == -1
    for i in (1, 2, 3, 5, 6):
        a = [dm(), P, P, P, None, P, P, None]
        a[i] = None
        assert B.LIB.moe_balance_bwd(*a) == -1 and err().startswith("moe_balance_bwd")
    assert B.LIB.moe_balance_bwd(dm(), P, P + 4, P, None, P, P, None) == -1


def test_gate_bwd_refuses():
    for i in (1, 2, 3, 4, 5, 8):
        a = [dm(), P, P, P, P, P, None, None, P, None]
        a[i] = None
        assert B.LIB.moe_gate_bwd(*a) == -1 and err().startswith("moe_gate_bwd")
    assert B.LIB.moe_gate_bwd(dm(), P + 8, P, P, P, P, None, None, P, None) == -1
    assert "16-byte" in err()


def test_router_bwd_refuses():
    def call(x=P, w=P, dl=P, dx_in=None, dx=P, dw=P, db=P, ws=P, n=1 << 30):
        return B.LIB.moe_router_bwd(dm(), x, w, None, dl, dx_in, dx, dw, db, ws, n, None)
    assert call(dl=None) == -1
    assert call(dx=None, dw=None, db=None) == -1 and "at least one" in err()
    assert call(w=None) == -1
    assert call(x=None) == -1
    assert call(dx=None, dx_in=P) == -1
    assert call(dx=P + 2) == -1 and "16-byte" in err()
    assert call(x=P + 4) == -1
    if B.moe_workspace_size(B.dims(64, 128, 8, 2, 256, 4, 32, "f32"), B.CALL_ROUTER_BWD):
        assert call(ws=None) == -3


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), -1), (dict(M=(1 << 26) + 1), -1), (dict(K=0), -1), (dict(K=65537), -1),
    (dict(E=0), -1), (dict(E=1025), -1), (dict(act=3), -2), (dict(ldx=99), -1),
    (dict(ldq=120), -1), (dict(ldq=136), -1), (dict(mul=P, ldm=99), -1), (dict(E=2), -1),
    (dict(x=None), -1), (dict(q=None), -1), (dict(scale=None), -1), (dict(q=P + 8), -1),
    (dict(M=0, x=None, q=None, scale=None), 0),
])
def test_quant_refuses(kw, status):
    a = dict(M=4, K=100, act=0, x=P, ldx=100, mul=None, ldm=0, cs=None, off=None, E=1, q=P,
             ldq=128, scale=P)
    a.update(kw)
    assert B.LIB.moe_quant_i8(*a.values(), None) == status
    if status:
        assert err().startswith("moe_quant_i8")


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), -1), (dict(M=(1 << 26) + 1), -1), (dict(N=0), -1), (dict(N=65537), -1),
    (dict(K=0), -1), (dict(K=65537), -1), (dict(E=0), -1), (dict(E=1025), -1),
    (dict(act=2), -2), (dict(lda=112), -1), (dict(lda=136), -1), (dict(ldw=96), -1),
    (dict(ldw=120), -1), (dict(ldo=39), -1), (dict(E=2), -1), (dict(a_rows=3), -1),
    (dict(src=P, a_rows=0), -1), (dict(src=P, div=0), -1), (dict(a=None), -1),
    (dict(a_scale=None), -1), (dict(w=None), -1), (dict(out=None), -1), (dict(a=P + 8), -1),
    (dict(w=P + 4), -1), (dict(M=0, a=None, a_scale=None, w=None, out=None, a_rows=0), 0),
])
def test_linear_refuses(kw, status):
    a = dict(a=P, lda=128, a_scale=P, a_rows=4, src=None, div=1, off=None, w=P, ldw=112, ws=None,
             out=P, ldo=40)
    d = dict(M=4, N=40, K=100, E=1, act=1)
    for k, v in kw.items():
        (d if k in d else a)[k] = v
    assert B.LIB.moe_i8_linear(ctypes.byref(B.I8Dims(*d.values())), *a.values(), None) == status
    if status:
        assert err().startswith("moe_i8_linear")
    assert B.LIB.moe_i8_linear(None, *a.values(), None) == -1


def test_binding_refuses_tensors_off_the_gpu():
    z = torch.zeros
    with pytest.raises(B.MoeError, match="GPU"):
        B.moe_quant_i8(z(4, 100), z(4, 128, dtype=torch.int8), z(4))
    with pytest.raises(B.MoeError, match="GPU"):
        B.moe_i8_linear(z(4, 128, dtype=torch.int8), z(4), z(1, 40, 112, dtype=torch.int8), None,
                        z(4, 40))
    with pytest.raises(B.MoeError, match="GPU"):
        B.moe_balance_bwd(B.dims(4, 128, 8, 2, 256, 4, 32, "f32"), z(4, 8), z(4, 2),
                          z(9, dtype=torch.int32), None, z(1), z(4, 8))


@pytest.mark.parametrize("gu,s_gu,down,s_down", [
    ((2, 7, 8), (2, 7), (2, 8, 3), (2, 8)),       # an odd number of gate/up channels
    ((2, 8, 8), (2, 8), (2, 8, 5), (2, 8)),       # down reads another width
    ((2, 8, 8), (2, 8), (3, 8, 4), (3, 8)),       # another number of experts
    ((2, 8, 8), (2, 4), (2, 8, 4), (2, 8)),       # scales of gate only
    ((2, 8, 8), (2, 8), (2, 8, 4), (2, 4)),
])
def test_int8_experts_refuse_shapes_that_do_not_match(gu, s_gu, down, s_down):
    from sparse_moe_expert_fp32_amd.layer import Int8Experts
    X = Int8Experts(torch.zeros(gu, dtype=torch.int8), torch.zeros(s_gu),
                    torch.zeros(down, dtype=torch.int8), torch.zeros(s_down))
    with pytest.raises(ValueError, match="Int8Experts"):
        X.forward(None)


def test_int8_experts_are_copied_and_pickled():
    import copy
    import pickle

    from sparse_moe_expert_fp32_amd.layer import Int8Experts
    X = Int8Experts(torch.ones(2, 8, 8, dtype=torch.int8), torch.ones(2, 8),
                    torch.ones(2, 8, 4, dtype=torch.int8), torch.ones(2, 8))
    for Y in (copy.deepcopy(X), pickle.loads(pickle.dumps(X))):
        assert torch.equal(Y.gate_up, X.gate_up) and Y.f == 4 and Y.t is None
