"""Convenience calls over the C ABI: allocate outputs / workspaces with torch (device
memory only) and run one IntLoRA step through libintlora.so.  No arithmetic of the
method happens here."""
from __future__ import annotations

import ctypes
import importlib

import torch

from . import binding as B


def _dev(t):
    return t.device


def gen_r(d, n, seed, layer_id, c, aux_dist=0):
    out = torch.empty((d, n), dtype=torch.float32, device=_dev(c))
    B.intlora_gen_r(B.desc(d, n, 1, 8, seed, layer_id, aux_dist), c, out)
    return out


def sigma_w(W):
    d, n = W.shape
    out = torch.empty(d, dtype=torch.float32, device=_dev(W))
    B.intlora_stats(B.desc(d, n, 1, 8), B.INTLORA_SIGMA_W, W=W, out0=out)
    return out


def vmc_scale(sigma, alpha, aux_dist=0):
    c = torch.empty_like(sigma)
    if aux_dist == 0:
        B.intlora_vmc_scale(sigma.numel(), sigma, alpha, c)
    else:
        B.intlora_vmc_scale_dist(sigma.numel(), sigma, alpha, aux_dist, c)
    return c


def code_bytes(d, n, w_bits):
    return (d, n) if w_bits == 8 else (d, n // 2)


def base_quant(W, c, w_bits, seed, layer_id, aux_dist=0):
    d, n = W.shape
    wr = torch.empty(code_bytes(d, n, w_bits), dtype=torch.uint8, device=_dev(W))
    z = torch.empty(d, dtype=torch.int32, device=_dev(W))
    s = torch.empty(d, dtype=torch.float32, device=_dev(W))
    B.intlora_base_quant(B.desc(d, n, 1, w_bits, seed, layer_id, aux_dist), W, c, wr, z, s)
    return wr, z, s


def setup_layer(W, w_bits, seed, layer_id, alpha=1.5, aux_dist=0):
    """AQS + VMC set-up of a pretrained layer on the GPU: sigma_W, c, Q[W - R*].  The
    auxiliary law (aux_dist) is kept with the state and used by every merge of it."""
    sig = sigma_w(W)
    c = vmc_scale(sig, alpha, aux_dist)
    wr, z, s = base_quant(W, c, w_bits, seed, layer_id, aux_dist)
    return dict(sigma=sig, c=c, wround=wr, z=z, s=s, aux_dist=aux_dist)


def workspace(op, d, n, r, w_bits, device):
    nbytes = B.intlora_workspace_bytes(op, B.desc(d, n, r, w_bits))
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def u_minmax(st, A, Bm, w_bits, seed, layer_id, ws=None):
    d, r = A.shape
    n = Bm.shape[1]
    dsc = B.desc(d, n, r, w_bits, seed, layer_id, st.get("aux_dist", 0))
    ws = workspace(B.INTLORA_OP_STATS_UMINMAX, d, n, r, w_bits, A.device) if ws is None else ws
    umin = torch.empty(d, dtype=torch.float32, device=A.device)
    umax = torch.empty_like(umin)
    B.intlora_stats(dsc, B.INTLORA_U_MINMAX, None, B.base(st["wround"], st["z"], st["s"], st["c"]), B.lora(A, Bm),
                    umin, umax, ws)
    return umin, umax


def merge_mul(st, A, Bm, w_bits, u_bits, seed, layer_id, dbg=False, ws=None, out=None, u_range=None):
    """u_range: optional (u_min, u_max) device tensors [d] used in place of the row range."""
    d, r = A.shape
    n = Bm.shape[1]
    dev = A.device
    dsc = B.desc(d, n, r, w_bits, seed, layer_id, st.get("aux_dist", 0))
    ws = workspace(B.INTLORA_OP_MERGE_MUL, d, n, r, w_bits, dev) if ws is None else ws
    o = out or dict(m=torch.empty((d, n), dtype=torch.int16, device=dev),
                    sbar=torch.empty(d, dtype=torch.float32, device=dev),
                    zbar=torch.empty(d, dtype=torch.int32, device=dev),
                    split=torch.empty(d, dtype=torch.uint8, device=dev),
                    sat=torch.zeros(2, dtype=torch.int64, device=dev))
    if dbg and "uround" not in o:
        o["uround"] = torch.empty((d, n), dtype=torch.uint8, device=dev)
    B.intlora_merge_mul(dsc, B.base(st["wround"], st["z"], st["s"], st["c"]), B.lora(A, Bm), u_bits, o["m"],
                        o["sbar"], o["zbar"], m_split=o.get("split"), u_round_dbg=o.get("uround") if dbg else None,
                        sat_count=o["sat"], ws=ws, u_min=u_range[0] if u_range else None,
                        u_max=u_range[1] if u_range else None)
    return o


def merge_mul_planes(st, A, Bm, w_bits, u_bits, seed, layer_id, dbg=False, ws=None, out=None, u_range=None):
    """MUL merge writing the merged integers as their two int8 byte planes (d x 2n
    bytes) with per-row plane codes, for the linear layer's INT16_PLANES format."""
    d, r = A.shape
    n = Bm.shape[1]
    dev = A.device
    dsc = B.desc(d, n, r, w_bits, seed, layer_id, st.get("aux_dist", 0))
    ws = workspace(B.INTLORA_OP_MERGE_MUL, d, n, r, w_bits, dev) if ws is None else ws
    o = out or dict(planes=torch.empty((d, 2 * n), dtype=torch.uint8, device=dev),
                    sbar=torch.empty(d, dtype=torch.float32, device=dev),
                    zbar=torch.empty(d, dtype=torch.int32, device=dev),
                    code=torch.empty(d, dtype=torch.uint8, device=dev),
                    sat=torch.zeros(2, dtype=torch.int64, device=dev))
    if dbg and "uround" not in o:
        o["uround"] = torch.empty((d, n), dtype=torch.uint8, device=dev)
    B.intlora_merge_mul_planes(dsc, B.base(st["wround"], st["z"], st["s"], st["c"]), B.lora(A, Bm), u_bits,
                               o["planes"], o["sbar"], o["zbar"], o["code"],
                               u_round_dbg=o.get("uround") if dbg else None, sat_count=o["sat"], ws=ws,
                               u_min=u_range[0] if u_range else None, u_max=u_range[1] if u_range else None)
    return o


def merge_mul_noalloc(st, A, Bm, w_bits, u_bits, seed, layer_id, dbg=False, out=None, u_range=None):
    """MUL merge with the library's own per-device scratch (no workspace); same outputs
    as merge_mul."""
    d, r = A.shape
    n = Bm.shape[1]
    dev = A.device
    dsc = B.desc(d, n, r, w_bits, seed, layer_id, st.get("aux_dist", 0))
    o = out or dict(m=torch.empty((d, n), dtype=torch.int16, device=dev),
                    sbar=torch.empty(d, dtype=torch.float32, device=dev),
                    zbar=torch.empty(d, dtype=torch.int32, device=dev),
                    split=torch.empty(d, dtype=torch.uint8, device=dev),
                    sat=torch.zeros(2, dtype=torch.int64, device=dev))
    if dbg and "uround" not in o:
        o["uround"] = torch.empty((d, n), dtype=torch.uint8, device=dev)
    B.intlora_merge_mul_noalloc(dsc, B.base(st["wround"], st["z"], st["s"], st["c"]), B.lora(A, Bm), u_bits, o["m"],
                                o["sbar"], o["zbar"], m_split=o.get("split"),
                                u_round_dbg=o.get("uround") if dbg else None, sat_count=o["sat"],
                                u_min=u_range[0] if u_range else None, u_max=u_range[1] if u_range else None)
    return o


def merge_mul_fused(st, A, Bm, w_bits, u_bits, seed, layer_id, dbg=False, out=None):
    """Fused single-pass MUL merge (no workspace); same outputs as merge_mul."""
    d, r = A.shape
    n = Bm.shape[1]
    dev = A.device
    dsc = B.desc(d, n, r, w_bits, seed, layer_id, st.get("aux_dist", 0))
    o = out or dict(m=torch.empty((d, n), dtype=torch.int16, device=dev),
                    sbar=torch.empty(d, dtype=torch.float32, device=dev),
                    zbar=torch.empty(d, dtype=torch.int32, device=dev),
                    split=torch.empty(d, dtype=torch.uint8, device=dev),
                    sat=torch.zeros(2, dtype=torch.int64, device=dev))
    if dbg and "uround" not in o:
        o["uround"] = torch.empty((d, n), dtype=torch.uint8, device=dev)
    B.intlora_merge_mul_fused(dsc, B.base(st["wround"], st["z"], st["s"], st["c"]), B.lora(A, Bm), u_bits, o["m"],
                              o["sbar"], o["zbar"], m_split=o.get("split"),
                              u_round_dbg=o.get("uround") if dbg else None, sat_count=o["sat"])
    return o


def merge_mul_codes(st, A, Bm, w_bits, u_bits, seed, layer_id, ws=None, out=None):
    """MUL merge keeping U's codes (packed nibbles d x n/2) with s_bar, z_bar, for the
    merge-on-load linear layer."""
    d, r = A.shape
    n = Bm.shape[1]
    dev = A.device
    dsc = B.desc(d, n, r, w_bits, seed, layer_id, st.get("aux_dist", 0))
    ws = workspace(B.INTLORA_OP_MERGE_MUL, d, n, r, w_bits, dev) if ws is None else ws
    o = out or dict(ucode=torch.empty((d, n // 2), dtype=torch.uint8, device=dev),
                    sbar=torch.empty(d, dtype=torch.float32, device=dev),
                    zbar=torch.empty(d, dtype=torch.int32, device=dev))
    B.intlora_merge_mul_codes(dsc, B.base(st["wround"], st["z"], st["s"], st["c"]), B.lora(A, Bm), u_bits, o["ucode"],
                              o["sbar"], o["zbar"], ws=ws)
    return o


def merge_shift(st, A, Bm, w_bits, v_bits, seed, layer_id, dbg=False, ws=None, out=None, u_range=None):
    """u_range: optional (u_min, u_max) device tensors [d] used in place of the row range."""
    d, r = A.shape
    n = Bm.shape[1]
    dev = A.device
    dsc = B.desc(d, n, r, w_bits, seed, layer_id, st.get("aux_dist", 0))
    ws = workspace(B.INTLORA_OP_MERGE_SHIFT, d, n, r, w_bits, dev) if ws is None else ws
    o = out or dict(m=torch.empty(code_bytes(d, n, w_bits), dtype=torch.uint8, device=dev),
                    sbar=torch.empty(d, dtype=torch.float32, device=dev),
                    sat=torch.zeros(2, dtype=torch.int64, device=dev))
    if dbg and "shift" not in o:
        o["shift"] = torch.empty((d, n), dtype=torch.uint8, device=dev)
    B.intlora_merge_shift(dsc, B.base(st["wround"], st["z"], st["s"], st["c"]), B.lora(A, Bm), v_bits, o["m"],
                          o["sbar"], o.get("shift") if dbg else None, o["sat"], ws,
                          u_min=u_range[0] if u_range else None, u_max=u_range[1] if u_range else None)
    return o


def merge_ptq(st, A, Bm, w_bits, bits, seed, layer_id, ws=None, out=None):
    """QLoRA-style comparison path: x = (s w + R*) + AB, per-row requant at `bits`."""
    d, r = A.shape
    n = Bm.shape[1]
    dev = A.device
    dsc = B.desc(d, n, r, w_bits, seed, layer_id, st.get("aux_dist", 0))
    ws = workspace(B.INTLORA_OP_MERGE_PTQ, d, n, r, w_bits, dev) if ws is None else ws
    o = out or dict(code=torch.empty(code_bytes(d, n, bits), dtype=torch.uint8, device=dev),
                    s=torch.empty(d, dtype=torch.float32, device=dev),
                    z=torch.empty(d, dtype=torch.int32, device=dev))
    B.intlora_merge_ptq(dsc, B.base(st["wround"], st["z"], st["s"], st["c"]), B.lora(A, Bm), bits, o["code"], o["s"],
                        o["z"], ws)
    return o


def ste_backward(st, A, Bm, G, w_bits, ws=None, out=None):
    """Straight-through backward to the LoRA factors: dA = (G.[w != 0]) B^T, dB = A^T (G.[w != 0])."""
    d, r = A.shape
    n = Bm.shape[1]
    dev = A.device
    dsc = B.desc(d, n, r, w_bits)
    if ws is None:
        nb = B.intlora_workspace_bytes(B.INTLORA_OP_STE_BACKWARD, dsc)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    o = out or dict(dA=torch.empty((d, r), dtype=torch.float32, device=dev),
                    dB=torch.empty((r, n), dtype=torch.float32, device=dev))
    B.intlora_ste_backward(dsc, st["wround"], st["z"], A, Bm, G, o["dA"], o["dB"], ws)
    return o


def quant_act(X):
    M, n = X.shape
    xq = torch.empty((M, n), dtype=torch.int8, device=X.device)
    sx = torch.empty(M, dtype=torch.float32, device=X.device)
    rs = torch.empty(M, dtype=torch.int32, device=X.device)
    B.intlora_quant_act(M, n, X, xq, sx, rs)
    return xq, sx, rs


def linear(xq, sx, rowsum, wfmt, m, sbar, d, acc_dbg=False, out=None, split=None):
    """split: the MUL merge's per-row split codes (INT16 only); None = bias split for
    every row."""
    M, n = xq.shape
    Y = torch.empty((M, d), dtype=torch.int16, device=xq.device) if out is None else out
    planes = 2 if wfmt in (B.INTLORA_W_INT16, B.INTLORA_W_INT16_PLANES) else 1
    acc = torch.empty((planes, M, d), dtype=torch.int32, device=xq.device) if acc_dbg else None
    B.intlora_linear_fwd(M, d, n, xq, sx, rowsum, wfmt, m, split, sbar, Y, acc)
    return Y, acc


def linear_codes(xq, sx, ucode, wcode, z, zbar, sbar, d, acc_dbg=False, out=None):
    """Merge-on-load linear layer: m = (U_round - z_bar) (W_round - z) formed in the GEMM
    from the packed 4-bit codes (d x n/2 each)."""
    M, n = xq.shape
    Y = torch.empty((M, d), dtype=torch.int16, device=xq.device) if out is None else out
    acc = torch.empty((2, M, d), dtype=torch.int32, device=xq.device) if acc_dbg else None
    B.intlora_linear_fwd_codes(M, d, n, xq, sx, ucode, wcode, z, zbar, sbar, Y, acc)
    return Y, acc


# ---------------------------------------------------------------- floating-point layers
_FLOAT = {torch.bfloat16: B.INTLORA_BF16, torch.float16: B.INTLORA_FP16, torch.float32: B.INTLORA_FP32}
_HALF = (torch.bfloat16, torch.float16)
_E4M3 = (torch.float8_e4m3fn,)
_BYTES = (torch.uint8,)


def _want(name, t, shape, dtypes, dev):
    """The address of t, which has this shape, one of these types, is contiguous and lies on
    the current device `dev` (where the call is enqueued); ValueError otherwise."""
    if t.get_device() != dev:  # -1 for a host tensor
        raise ValueError(f"{name}: expected a tensor on the current device, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _dims(name, t, *dims):
    if t.dim() not in dims:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dims))} dimensions, got shape {tuple(t.shape)}")
    return t.shape


def _offsets(offsets, E, dev):
    if offsets is None:
        if E != 1:
            raise ValueError("offsets: needed with more than one group")
        return None
    return _want("offsets", offsets, (E + 1,), (torch.int64,), dev)


def _output(out, shape, dtype, like, dev):
    if out is None:
        out = like.new_empty(shape, dtype=dtype)
        return out, out.data_ptr()
    return out, _want("out", out, shape, (dtype,), dev)


def fp8_scale_bytes(n):
    """Scale bytes per row of n columns: one per 128, in whole groups of four."""
    return 4 * ((n + 511) // 512)


def fp8_quant_act(X, out=None):
    """e4m3 codes of X [M, n] (bf16, fp16 or fp32) and their scale bytes, one per 128 columns:
    (xq [M, n] float8_e4m3fn, sx [M, fp8_scale_bytes(n)] uint8)."""
    M, n = _dims("X", X, 2)
    dev = torch.cuda.current_device()
    x = _want("X", X, (M, n), _FLOAT, dev)
    xq, xp = _output(out[0] if out else None, (M, n), torch.float8_e4m3fn, X, dev)
    sx, sp = _output(out[1] if out else None, (M, fp8_scale_bytes(n)), torch.uint8, X, dev)
    B.intlora_fp8_quant_act(M, n, _FLOAT[X.dtype], x, xp, sp)
    return xq, sx


def fp8_quant_weight(W, transpose=False):
    """e4m3 codes of a weight [d, n] or of E of them [E, d, n] with one scale per 128 x 128
    block: dict(wq, sw), and with `transpose` the same codes transposed (wq_t, sw_t), on which
    fp8_linear computes the input gradient dY W from dY's codes."""
    shape = _dims("W", W, 2, 3)
    w = _want("W", W, shape, _FLOAT, torch.cuda.current_device())
    E, (d, n) = (shape[0] if len(shape) == 3 else 1), shape[-2:]
    lead = shape[:-2]
    o = dict(wq=W.new_empty(shape, dtype=torch.float8_e4m3fn),
             sw=W.new_empty((*lead, (d + 127) // 128, fp8_scale_bytes(n)), dtype=torch.uint8))
    if transpose:
        o["wq_t"] = W.new_empty((*lead, n, d), dtype=torch.float8_e4m3fn)
        o["sw_t"] = W.new_empty((*lead, (n + 127) // 128, fp8_scale_bytes(d)), dtype=torch.uint8)
    B.intlora_fp8_quant_weight(E, d, n, _FLOAT[W.dtype], w, o["wq"], o["sw"], o.get("wq_t"), o.get("sw_t"))
    return o


def _fp8_operands(xq, sx, wq, sw, lead, dev):
    M, n = _dims("xq", xq, 2)
    d, s = wq.shape[-2], fp8_scale_bytes(n)
    return M, d, n, (_want("xq", xq, (M, n), _E4M3, dev), _want("sx", sx, (M, s), _BYTES, dev),
                     _want("wq", wq, (*lead, d, n), _E4M3, dev), _want("sw", sw, (*lead, (d + 127) // 128, s), _BYTES, dev))


def fp8_linear(xq, sx, wq, sw, out=None):
    """Y [M, d] (bf16) of codes and scales as fp8_quant_act and fp8_quant_weight make them."""
    _dims("wq", wq, 2)
    dev = torch.cuda.current_device()
    M, d, n, p = _fp8_operands(xq, sx, wq, sw, (), dev)
    Y, y = _output(out, (M, d), torch.bfloat16, xq, dev)
    B.intlora_fp8_linear_fwd(M, d, n, *p, y)
    return Y


def fp8_grouped_linear(xq, sx, offsets, wq, sw, out=None):
    """As fp8_linear with one weight per group of rows: wq [E, d, n], rows offsets[e] ..
    offsets[e + 1] - 1 take weight e.  Rows in no group are left as they are in `out`; without
    `out` they are not initialised."""
    E = _dims("wq", wq, 3)[0]
    dev = torch.cuda.current_device()
    M, d, n, (x, s, w, v) = _fp8_operands(xq, sx, wq, sw, (E,), dev)
    Y, y = _output(out, (M, d), torch.bfloat16, xq, dev)
    B.intlora_fp8_grouped_linear_fwd(M, E, d, n, x, s, _offsets(offsets, E, dev), w, v, y)
    return Y


def grouped_linear(X, offsets, W, out=None):
    """Y [M, d] of X [M, n] and W [E, d, n] (bf16 or fp16): rows offsets[e] .. offsets[e + 1] - 1
    are multiplied by W[e]^T.  Rows in no group are left as they are in `out`; without `out` they
    are not initialised."""
    M, n = _dims("X", X, 2)
    E, d, _ = _dims("W", W, 3)
    dev = torch.cuda.current_device()
    x, w = _want("X", X, (M, n), _HALF, dev), _want("W", W, (E, d, n), (X.dtype,), dev)
    Y, y = _output(out, (M, d), X.dtype, X, dev)
    B.intlora_grouped_linear_fwd(M, E, d, n, _FLOAT[X.dtype], x, _offsets(offsets, E, dev), w, y)
    return Y


def grouped_linear_dx(dY, offsets, W, out=None):
    """The gradient of grouped_linear's X: dX [M, n] of dY [M, d] and W [E, d, n].  Rows in no
    group are left as they are in `out` (their gradient is zero: clear them there); without
    `out` they are not initialised."""
    M, d = _dims("dY", dY, 2)
    E, _, n = _dims("W", W, 3)
    dev = torch.cuda.current_device()
    y, w = _want("dY", dY, (M, d), _HALF, dev), _want("W", W, (E, d, n), (dY.dtype,), dev)
    dX, x = _output(out, (M, n), dY.dtype, dY, dev)
    B.intlora_grouped_linear_dx(M, E, d, n, _FLOAT[dY.dtype], y, _offsets(offsets, E, dev), w, x)
    return dX


def grouped_linear_dw(dY, X, offsets, dtype=None, out=None):
    """The gradient of grouped_linear's W: dW [E, d, n] of dY [M, d] and X [M, n], in their type
    or in fp32 (dtype).  With offsets = None one group of all rows: dW [1, d, n], whose fp32
    form is the G of ste_backward."""
    M, d = _dims("dY", dY, 2)
    n = _dims("X", X, 2)[1]
    dev = torch.cuda.current_device()
    y, x = _want("dY", dY, (M, d), _HALF, dev), _want("X", X, (M, n), (dY.dtype,), dev)
    E = 1 if offsets is None else offsets.numel() - 1
    dtype = dtype or (dY.dtype if out is None else out.dtype)
    if dtype not in (dY.dtype, torch.float32):
        raise ValueError(f"dtype: expected {dY.dtype} or torch.float32, got {dtype}")
    dW, w = _output(out, (E, d, n), dtype, dY, dev)
    B.intlora_grouped_linear_dw(M, E, d, n, _FLOAT[dY.dtype], _FLOAT[dtype], y, x, _offsets(offsets, E, dev), w)
    return dW


# ---------------------------------------------------------------- gradient norm, clipping
_tensor_list = None


def _tensors(name, ts):
    """A list of them.  The call holds it until its kernels are enqueued: what an iterator made on
    the way may have no other owner, and its memory could become the workspace."""
    if isinstance(ts, torch.Tensor):
        raise ValueError(f"{name}: expected a list of tensors")
    return list(ts)


def _read(name, ts, dev):
    """Addresses, element counts and types of a list of contiguous bf16, fp16 or fp32 tensors on
    device `dev` as C arrays, read in one pass in compiled code."""
    global _tensor_list
    if _tensor_list is None:
        try:
            _tensor_list = importlib.import_module("._tensor_list", __package__)
        except ImportError as e:
            raise RuntimeError(f"_tensor_list.so does not load ({e}): build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')") from e
    n = len(ts)
    ptrs, numel, types = _tensor_list.read(name, ts, dev)
    return ((ctypes.c_void_p * n).from_buffer_copy(ptrs), (ctypes.c_int64 * n).from_buffer_copy(numel),
            (ctypes.c_int32 * n).from_buffer_copy(types))


def _sumsq(ptrs, numel, types, dev):
    size = B.intlora_grad_ws_bytes(numel)
    ws = torch.empty(8 + size // 8, dtype=torch.float64, device=dev)  # the sum, then the parts
    at = ws.data_ptr()
    B.intlora_grad_sumsq(ptrs, numel, types, at, at + 64, ws_bytes=size)
    return ws


def _clip(ptrs, numel, types, sumsq, max_norm, out, dev):
    outs = ptrs
    if out is not None:
        out = _tensors("out", out)
        outs, n, t = _read("out", out, dev)
        if bytes(n) != bytes(numel) or bytes(t) != bytes(types):
            raise ValueError("out: expected tensors of the gradients' sizes and types")
    norm = torch.empty(1, dtype=torch.float32, device=dev)
    B.intlora_grad_clip(ptrs, outs, numel, types, sumsq, max_norm, norm)
    return norm


def clip_grad_norm(grads, max_norm, out=None):
    """Scales a list of gradients (bf16, fp16, fp32) by min(1, max_norm / (norm + 1e-6)), norm
    being the 2-norm over all of them, in place or into `out` (tensors of the same sizes and
    types), and returns the norm as a device tensor [1] (fp32); nothing waits for the GPU.
    Tensors are contiguous, on the current device, and start at multiples of 16 bytes.
    Ranks that each hold a part call grad_sumsq, add their sums and call grad_clip."""
    dev, grads = torch.cuda.current_device(), _tensors("grads", grads)
    a = _read("grads", grads, dev)
    ws = _sumsq(*a, dev)
    return _clip(*a, ws.data_ptr(), max_norm, out, dev)


def grad_sumsq(grads):
    """The sum of all squared gradients, a device tensor [1] (fp64)."""
    dev, grads = torch.cuda.current_device(), _tensors("grads", grads)
    return _sumsq(*_read("grads", grads, dev), dev)[:1]


def grad_clip(grads, sumsq, max_norm, out=None):
    """The second half of clip_grad_norm, from a sum of squares (fp64 [1]) over all ranks."""
    dev, grads = torch.cuda.current_device(), _tensors("grads", grads)
    a = _read("grads", grads, dev)
    return _clip(*a, _want("sumsq", sumsq, (1,), (torch.float64,), dev), max_norm, out, dev)
