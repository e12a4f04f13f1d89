"""ctypes binding of libmoe_tqp.so (see include/moe_tqp.h).

Argument marshalling only: torch tensors are passed by device pointer and the
current HIP stream; every step of the layer runs in the library's kernels.
Importing this module loads the library and raises if it was not built.
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_tqp.so")

MOE_F32, MOE_BF16 = 0, 1
CALL_ROUTE, CALL_PERMUTE, CALL_EXPERT_FWD, CALL_COMBINE, CALL_ADAPTER_BWD = range(5)
CALL_BALANCE_FWD, CALL_ROUTER_BWD = 5, 6
# workspace flags OR-ed into a call id of moe_workspace_size
WS_SAVE_GIVEN, WS_PACKED_GIVEN = 0x100, 0x200
MAT_GATE_UP, MAT_DOWN = 0, 1


class MoeError(RuntimeError):
    pass


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("group", ctypes.c_int32), ("act", ctypes.c_int32),
                ("lora_scale", ctypes.c_float), ("base_bits", ctypes.c_int32)]


class QLora(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("qt", ctypes.c_void_p),
                ("qf", ctypes.c_void_p)]


class I8Dims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("act", ctypes.c_int32)]


class AdamWHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("step", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise MoeError(f"{LIB_PATH} is missing: build it with "
                       "`python -m sparse_moe_expert_fp32_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    I64 = ctypes.c_int64
    DP = ctypes.POINTER(Dims)
    sig = {
        "moe_route": [DP, P, P, P, P, P, P, P, SZ, P],
        "moe_permute": [DP, P, P, P, P, P, P, P, P, SZ, P],
        "moe_expert_fwd": [DP, P, P, P, QLora, QLora, QLora, P, P, P, SZ, P],
        "moe_expert_fwd_noalloc": [DP, P, P, P, QLora, QLora, QLora, P, P, P],
        "moe_combine": [DP, P, P, P, P, P, SZ, P],
        "moe_adapter_bwd": [DP, P, P, P, P, P, P, P, P, QLora, QLora, QLora, P, P, P,
                            P, P, P, P, P, P, P, SZ, P],
        "moe_workspace_size": [DP, I32, ctypes.POINTER(SZ)],
        "moe_save_size": [DP, ctypes.POINTER(SZ)],
        "moe_status_string": [I32],
        "moe_last_error": [],
        "moe_abi_version": [],
        "moe_timer_start": [I32],
        "moe_timer_stop": [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(I32)],
        "moe_adamw_step": [ctypes.POINTER(AdamWHparams), ctypes.c_int64, P, P, P, P, P, I32, P],
        "moe_pack_base_t_size": [DP, ctypes.POINTER(SZ)],
        "moe_pack_base_t": [DP, I32, P, P, P, SZ, P],
        "moe_pack_base_f_size": [DP, ctypes.POINTER(SZ)],
        "moe_pack_base_f": [DP, I32, P, P, P, SZ, P],
        "moe_rev_couple": [DP, P, P, P, I32, P],
        "moe_balance_fwd": [DP, P, P, P, P, P, P, P, P, SZ, P],
        "moe_balance_bwd": [DP, P, P, P, P, P, P, P],
        "moe_gate_bwd": [DP, P, P, P, P, P, P, P, P, P],
        "moe_router_bwd": [DP, P, P, P, P, P, P, P, P, P, SZ, P],
        "moe_quant_i8": [I32, I32, I32, P, I64, P, I64, P, P, I32, P, I64, P, P],
        "moe_i8_linear": [ctypes.POINTER(I8Dims), P, I64, P, I32, P, I32, P, P, I64, P, P, I64,
                          P],
        "moe_grow_copy": [P, P, ctypes.c_int64, I32, I32, P],
        "moe_grow_router": [I32, I32, I32, P, P, P, ctypes.c_float, P, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = I32
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_last_error.restype = ctypes.c_char_p
    return lib


LIB = _load()
EXPORTS = ("moe_route", "moe_permute", "moe_expert_fwd", "moe_expert_fwd_noalloc", "moe_combine",
           "moe_adapter_bwd",
           "moe_workspace_size", "moe_save_size", "moe_status_string", "moe_last_error",
           "moe_abi_version", "moe_timer_start", "moe_timer_stop", "moe_adamw_step",
           "moe_pack_base_t_size", "moe_pack_base_t", "moe_pack_base_f_size", "moe_pack_base_f",
           "moe_rev_couple", "moe_grow_copy", "moe_grow_router", "moe_balance_fwd",
           "moe_balance_bwd", "moe_gate_bwd", "moe_router_bwd", "moe_quant_i8", "moe_i8_linear")

# kernel tags of moe_timer_start (moe_kernel_tag)
KT = {"router_logits": 0, "router_topk": 1, "permute": 2, "gateup": 3, "down": 4, "combine": 5,
      "gate_grad": 6, "bwd_down": 7, "bwd_gateup": 8}


def _check(status: int, name: str):
    if status != 0:
        raise MoeError(f"{name}: {LIB.moe_status_string(status).decode()}: "
                       f"{LIB.moe_last_error().decode()}")


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dims(T, d, E, k, f, r, group, act, lora_scale=1.0, bits=4) -> Dims:
    a = {"f32": MOE_F32, "bf16": MOE_BF16}.get(act, act)
    return Dims(T, d, E, k, f, r, group, a, lora_scale, bits)


def dims_of(cfg, T: int | None = None) -> Dims:
    return dims(cfg.T if T is None else T, cfg.d, cfg.E, cfg.k, cfg.f, cfg.r, cfg.group,
                cfg.act, cfg.lora_scale, getattr(cfg, "bits", 4))


def qlora(q, scale, A, B, qt=None, qf=None) -> QLora:
    return QLora(_p(q), _p(scale), _p(A), _p(B), _p(qt), _p(qf))


def moe_workspace_size(dm: Dims, call: int) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.moe_workspace_size(ctypes.byref(dm), call, ctypes.byref(out)), "moe_workspace_size")
    return out.value


def moe_save_size(dm: Dims) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.moe_save_size(ctypes.byref(dm), ctypes.byref(out)), "moe_save_size")
    return out.value


def moe_abi_version() -> int:
    return LIB.moe_abi_version()


def moe_timer_start(tag) -> None:
    _check(LIB.moe_timer_start(KT.get(tag, tag)), "moe_timer_start")


def moe_timer_stop():
    ms, n = ctypes.c_float(0), ctypes.c_int32(0)
    _check(LIB.moe_timer_stop(ctypes.byref(ms), ctypes.byref(n)), "moe_timer_stop")
    return ms.value, n.value


def moe_route(dm, x, w_router, b_router, topk_idx, gates, logits, ws, stream=None):
    _check(LIB.moe_route(ctypes.byref(dm), _p(x), _p(w_router), _p(b_router), _p(topk_idx),
                         _p(gates), _p(logits), _p(ws), ws.numel() if ws is not None else 0,
                         _stream(stream)), "moe_route")


def moe_permute(dm, topk_idx, x, counts, offsets, perm_src, slot_pos, x_perm, ws, stream=None):
    _check(LIB.moe_permute(ctypes.byref(dm), _p(topk_idx), _p(x), _p(counts), _p(offsets),
                           _p(perm_src), _p(slot_pos), _p(x_perm), _p(ws),
                           ws.numel() if ws is not None else 0, _stream(stream)), "moe_permute")


def moe_expert_fwd(dm, x, offsets, perm_src, gate, up, down, e_out, save, ws, stream=None):
    _check(LIB.moe_expert_fwd(ctypes.byref(dm), _p(x), _p(offsets), _p(perm_src), gate, up, down,
                              _p(e_out), _p(save), _p(ws), ws.numel() if ws is not None else 0,
                              _stream(stream)), "moe_expert_fwd")


def moe_expert_fwd_noalloc(dm, x, offsets, perm_src, gate, up, down, e_out, save, stream=None):
    _check(LIB.moe_expert_fwd_noalloc(ctypes.byref(dm), _p(x), _p(offsets), _p(perm_src), gate,
                                      up, down, _p(e_out), _p(save), _stream(stream)),
           "moe_expert_fwd_noalloc")


def moe_combine(dm, e_out, slot_pos, gates, y, ws=None, stream=None):
    _check(LIB.moe_combine(ctypes.byref(dm), _p(e_out), _p(slot_pos), _p(gates), _p(y), _p(ws),
                           ws.numel() if ws is not None else 0, _stream(stream)), "moe_combine")


def moe_adapter_bwd(dm, dy, x, topk_idx, gates, offsets, perm_src, slot_pos, w_router, gate, up,
                    down, e_out, save, dx, dA_gate, dB_gate, dA_up, dB_up, dA_down, dB_down, ws,
                    stream=None):
    _check(LIB.moe_adapter_bwd(ctypes.byref(dm), _p(dy), _p(x), _p(topk_idx), _p(gates),
                               _p(offsets), _p(perm_src), _p(slot_pos), _p(w_router), gate, up,
                               down, _p(e_out), _p(save), _p(dx), _p(dA_gate), _p(dB_gate),
                               _p(dA_up), _p(dB_up), _p(dA_down), _p(dB_down), _p(ws),
                               ws.numel() if ws is not None else 0, _stream(stream)),
           "moe_adapter_bwd")


def pack_base_supported(dm: Dims) -> bool:
    """Whether these dims have a packed transposed base (the matrix-core path)."""
    out = ctypes.c_size_t(0)
    return LIB.moe_pack_base_t_size(ctypes.byref(dm), ctypes.byref(out)) == 0


def moe_pack_base_t_size(dm: Dims) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.moe_pack_base_t_size(ctypes.byref(dm), ctypes.byref(out)), "moe_pack_base_t_size")
    return out.value


def moe_pack_base_t(dm: Dims, matrix: int, q, scale, packed, stream=None):
    _check(LIB.moe_pack_base_t(ctypes.byref(dm), matrix, _p(q), _p(scale), _p(packed),
                               packed.numel() if packed is not None else 0, _stream(stream)),
           "moe_pack_base_t")


def moe_rev_couple(dm: Dims, x, m, out, sign: int, stream=None):
    _check(LIB.moe_rev_couple(ctypes.byref(dm), _p(x), _p(m), _p(out), sign, _stream(stream)),
           "moe_rev_couple")


def moe_grow_copy(src, dst, block_bytes: int, n_experts: int, factor: int, stream=None):
    _check(LIB.moe_grow_copy(_p(src), _p(dst), block_bytes, n_experts, factor, _stream(stream)),
           "moe_grow_copy")


def moe_grow_router(d: int, n_experts: int, factor: int, w, b, noise, noise_scale: float,
                    w_out, b_out, stream=None):
    _check(LIB.moe_grow_router(d, n_experts, factor, _p(w), _p(b), _p(noise), noise_scale,
                               _p(w_out), _p(b_out), _stream(stream)), "moe_grow_router")


def moe_pack_base_f_size(dm: Dims) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.moe_pack_base_f_size(ctypes.byref(dm), ctypes.byref(out)), "moe_pack_base_f_size")
    return out.value


def moe_pack_base_f(dm: Dims, matrix: int, q, scale, packed, stream=None):
    _check(LIB.moe_pack_base_f(ctypes.byref(dm), matrix, _p(q), _p(scale), _p(packed),
                               packed.numel() if packed is not None else 0, _stream(stream)),
           "moe_pack_base_f")


def adamw_hparams(lr, beta1, beta2, eps, weight_decay, step) -> AdamWHparams:
    return AdamWHparams(lr, beta1, beta2, eps, weight_decay, step)


def moe_adamw_step(h: AdamWHparams, master, grad, m, v, param=None, stream=None):
    if param is None:
        pdt = MOE_F32
    else:
        pdt = MOE_BF16 if param.dtype == torch.bfloat16 else MOE_F32
    n = master.numel()
    _check(LIB.moe_adamw_step(ctypes.byref(h), n, _p(master), _p(grad), _p(m), _p(v), _p(param),
                              pdt, _stream(stream)), "moe_adamw_step")


# ---- load balance, router training, int8 rows and products.  The tensors'
# types, sizes and layouts are checked here (the C ABI sees pointers only),
# and the call runs with the tensors' device current.

_F32, _I32, _I8, _U8, _BF16 = (torch.float32, torch.int32, torch.int8, torch.uint8,
                               torch.bfloat16)
_ACT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_DT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def _gpu(name, t) -> int:
    """Index of the GPU that t is on."""
    dev = t.get_device()
    if dev < 0:
        raise MoeError(f"{name}: tensors must be on the GPU, got {t.device}")
    return dev


def _dense(name, arg, t, dtype, numel, dev):
    """Pointer of a contiguous tensor of `numel` elements on GPU `dev`."""
    if t.dtype is not dtype or t.numel() != numel or t.get_device() != dev or \
            not t.is_contiguous():
        raise MoeError(f"{name}: {arg} must be a contiguous {dtype} tensor of {numel} elements "
                       f"on GPU {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _opt(name, arg, t, dtype, numel, dev):
    return None if t is None else _dense(name, arg, t, dtype, numel, dev)


def _valid(name, t, T, dev):
    if t is None:
        return None
    return _dense(name, "valid", t, _U8 if t.dtype is _U8 else torch.bool, T, dev)


def _ws(name, ws, dev):
    if ws is None:
        return None, 0
    n = ws.numel() * ws.element_size()
    return _dense(name, "ws", ws, ws.dtype, ws.numel(), dev), n


def _call(name, dev, fn, args, stream):
    """fn(*args, stream) with GPU `dev` current, on its current stream unless
    one is given."""
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None
                    else _stream(stream))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(stream))
    if status:
        _check(status, name)


def moe_balance_fwd(dm: Dims, logits, topk_idx, valid, loss, counts, prob, stats, ws, stream=None):
    """Load-balance loss, per-expert counts (and the number of tokens, last)
    and mean probabilities; `stats` is what moe_balance_bwd reads."""
    f, T, E, dev = "moe_balance_fwd", dm.T, dm.n_experts, _gpu("moe_balance_fwd", logits)
    _call(f, dev, LIB.moe_balance_fwd,
          (dm, _dense(f, "logits", logits, _F32, T * E, dev),
           _dense(f, "topk_idx", topk_idx, _I32, T * dm.top_k, dev), _valid(f, valid, T, dev),
           _dense(f, "loss", loss, _F32, 1, dev), _dense(f, "counts", counts, _I32, E + 1, dev),
           _dense(f, "prob", prob, _F32, E, dev), _dense(f, "stats", stats, _F32, 2 * T, dev),
           *_ws(f, ws, dev)), stream)


def moe_balance_bwd(dm: Dims, logits, stats, counts, valid, dloss, dlogits, stream=None):
    """Gradient of the load-balance loss with respect to the logits."""
    f, T, E, dev = "moe_balance_bwd", dm.T, dm.n_experts, _gpu("moe_balance_bwd", logits)
    _call(f, dev, LIB.moe_balance_bwd,
          (dm, _dense(f, "logits", logits, _F32, T * E, dev),
           _dense(f, "stats", stats, _F32, 2 * T, dev),
           _dense(f, "counts", counts, _I32, E + 1, dev), _valid(f, valid, T, dev),
           _dense(f, "dloss", dloss, _F32, 1, dev),
           _dense(f, "dlogits", dlogits, _F32, T * E, dev)), stream)


def moe_gate_bwd(dm: Dims, dy, e_out, topk_idx, gates, slot_pos, valid, dlogits_in, dlogits,
                 stream=None):
    """dlogits = dlogits_in + the gates' gradient with respect to the logits."""
    f, T, E, k, d, act = "moe_gate_bwd", dm.T, dm.n_experts, dm.top_k, dm.d_model, _DT.get(dm.act)
    dev = _gpu(f, dy)
    _call(f, dev, LIB.moe_gate_bwd,
          (dm, _dense(f, "dy", dy, act, T * d, dev),
           _dense(f, "e_out", e_out, act, T * k * d, dev),
           _dense(f, "topk_idx", topk_idx, _I32, T * k, dev),
           _dense(f, "gates", gates, _F32, T * k, dev),
           _dense(f, "slot_pos", slot_pos, _I32, T * k, dev), _valid(f, valid, T, dev),
           _opt(f, "dlogits_in", dlogits_in, _F32, T * E, dev),
           _dense(f, "dlogits", dlogits, _F32, T * E, dev)), stream)


def moe_router_bwd(dm: Dims, x, w_router, valid, dlogits, dx_in, dx, dw_router, db_router, ws,
                   stream=None):
    """dx = dx_in + dlogits W_r^T, dw_router = x^T dlogits, db_router = the
    column sums of dlogits; each output may be None."""
    f, T, E, d, act = "moe_router_bwd", dm.T, dm.n_experts, dm.d_model, _DT.get(dm.act)
    dev = _gpu(f, dlogits)
    _call(f, dev, LIB.moe_router_bwd,
          (dm, _opt(f, "x", x, act, T * d, dev), _opt(f, "w_router", w_router, _F32, d * E, dev),
           _valid(f, valid, T, dev), _dense(f, "dlogits", dlogits, _F32, T * E, dev),
           _opt(f, "dx_in", dx_in, act, T * d, dev), _opt(f, "dx", dx, act, T * d, dev),
           _opt(f, "dw_router", dw_router, _F32, d * E, dev),
           _opt(f, "db_router", db_router, _F32, E, dev), *_ws(f, ws, dev)), stream)


def moe_i8_stride(K: int) -> int:
    """Row stride of int8 rows of K values (moe_quant_i8, moe_i8_linear)."""
    return (K + 127) // 128 * 128


def _rows(name, arg, t, dtype, dev):
    """(rows, columns, row stride) of a matrix whose columns are adjacent."""
    if t.dim() == 2 and t.dtype is dtype and t.get_device() == dev:
        M, N = t.shape
        ld, one = t.stride()
        if one == 1 or N <= 1:
            return M, N, ld if ld > N or M > 1 else N
    raise MoeError(f"{name}: {arg} must be a {dtype} matrix on GPU {dev} with adjacent columns, "
                   f"got {t.dtype} {tuple(t.shape)} {t.stride()} on {t.device}")


def _act_code(name, arg, t) -> int:
    a = _ACT.get(t.dtype)
    if a is None:
        raise MoeError(f"{name}: {arg} must be float32 or bfloat16, got {t.dtype}")
    return a


def moe_quant_i8(x, q, scale, mul=None, col_scale=None, offsets=None, stream=None):
    """Rows of x (or silu(x) mul, or x col_scale[expert]) -> int8 rows q
    [M][moe_i8_stride(K)] or wider, one row after another (all of a row is
    written: 0 behind column K), and their scales [M]."""
    f, dev, act = "moe_quant_i8", _gpu("moe_quant_i8", x), _act_code("moe_quant_i8", "x", x)
    M, K, ldx = _rows(f, "x", x, x.dtype, dev)
    Mq, Kq, ldq = _rows(f, "q", q, _I8, dev)
    if Mq != M or Kq < moe_i8_stride(K):
        raise MoeError(f"{f}: q must have {M} rows of at least {moe_i8_stride(K)} values, "
                       f"got {tuple(q.shape)}")
    if ldq != Kq and M > 1:   # (the columns up to the stride would be another tensor's)
        raise MoeError(f"{f}: q's rows must lie one after another, got {tuple(q.shape)} at "
                       f"stride {ldq}")
    ldm, E = 0, 1
    if mul is not None:
        Mm, Km, ldm = _rows(f, "mul", mul, x.dtype, dev)
        if Mm != M or Km != K:
            raise MoeError(f"{f}: mul must be {(M, K)}, got {tuple(mul.shape)}")
    if offsets is not None:
        E = offsets.numel() - 1
    _call(f, dev, LIB.moe_quant_i8,
          (M, K, act, x.data_ptr(), ldx, _p(mul), ldm,
           _opt(f, "col_scale", col_scale, _F32, E * K, dev),
           _opt(f, "offsets", offsets, _I32, E + 1, dev), E, q.data_ptr(), Kq,
           _dense(f, "scale", scale, _F32, M, dev)), stream)


def moe_i8_linear(a, a_scale, w, w_scale, out, offsets=None, row_src=None, row_div=1,
                  stream=None):
    """out[p] = rows a (int8, as moe_quant_i8 writes them) by the int8 matrix
    w[e] [N][K] of the row's expert, scaled per row and per channel.  (Rows and
    scales of a float matrix come from moe_quant_i8 over its output channels;
    two's-complement bytes kept as uint8 go in as w.view(torch.int8).)"""
    f, dev, act = "moe_i8_linear", _gpu("moe_i8_linear", a), _act_code("moe_i8_linear", "out", out)
    R, Ka, lda = _rows(f, "a", a, _I8, dev)
    M, N, ldo = _rows(f, "out", out, out.dtype, dev)
    E, Nw, K = w.shape if w.dim() == 3 else (0, 0, 0)
    es, ldw, one = w.stride() if E else (0, 0, 0)
    if not E or Nw != N or w.dtype is not _I8 or w.get_device() != dev or (one != 1 and K > 1):
        raise MoeError(f"{f}: w must be int8 [E][{N}][K] with adjacent columns on GPU {dev}, got "
                       f"{w.dtype} {tuple(w.shape)} {w.stride()} on {w.device}")
    if K % 16 or not w.is_contiguous():
        if N == 1:
            ldw = es if E > 1 else max(ldw, K)
        if E > 1 and es != N * ldw:
            raise MoeError(f"{f}: the experts' matrices must lie one after another")
        if w.untyped_storage().nbytes() - w.storage_offset() < E * N * ldw:
            raise MoeError(f"{f}: the last row of w must reach its stride")
    else:
        ldw = K
    if Ka < moe_i8_stride(K):
        raise MoeError(f"{f}: a must have rows of at least {moe_i8_stride(K)} values")
    _call(f, dev, LIB.moe_i8_linear,
          (I8Dims(M, N, K, E, act), a.data_ptr(), lda,
           _dense(f, "a_scale", a_scale, _F32, R, dev), R,
           _opt(f, "row_src", row_src, _I32, M, dev), row_div,
           _opt(f, "offsets", offsets, _I32, E + 1, dev), w.data_ptr(), ldw,
           _opt(f, "w_scale", w_scale, _F32, E * N, dev), out.data_ptr(), ldo), stream)
