"""Torch-facing binding of the tiledq C ABI.

Argument marshalling only: device pointers, sizes and the current HIP stream
go to libtiledq.so; every step of the computation runs in its HIP kernels.
Tensors must live on the GPU; outputs are allocated with torch unless given.
"""
import ctypes
import functools
import threading

import torch

from ._lib import TiledqError, check, lib

Q4_0, Q8_0, IQ4_NL, MXFP4, Q4_1, Q4_K = 0, 1, 2, 3, 4, 5
F32, BF16, F16 = 0, 1, 2
PATH_GEMV, PATH_GEMM, PATH_GEMV_FLAT, PATH_GEMM_FLAT, PATH_GEMM_MX, PATH_GEMM_SPLIT = 0, 1, 2, 3, 4, 5

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _ptr(t):
    """Device address as an int (the C-ABI's pointer arguments take ints)."""
    return t.data_ptr() if t is not None else None


# torch's raw handle of a device's current stream (what
# torch.cuda.current_stream(device).cuda_stream returns, without building a
# Stream object on every call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t):
    """The current HIP stream of tensor t's device, as an int handle."""
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


@functools.lru_cache(maxsize=4096)
def _size_query(name, *args):
    """A size / workspace query of the C ABI; they depend on their arguments
    alone, so results are cached."""
    return getattr(lib(), name)(*args)


def _need_cuda(*ts, out=None):
    """Inputs must be contiguous GPU tensors; `out` a GPU tensor (its row
    stride is passed to the library as ldy, checked by _check_out)."""
    for t in ts:
        if t is not None and not t.is_cuda:
            raise TiledqError("tiledq operates on GPU tensors only")
        if t is not None and not t.is_contiguous():
            raise TiledqError("tiledq expects contiguous tensors")
    if out is not None and not out.is_cuda:
        raise TiledqError("tiledq operates on GPU tensors only")


def _nbytes(t):
    return t.numel() * t.element_size()


def _need_bytes(name, what, t, nbytes):
    if t is not None and _nbytes(t) < nbytes:
        raise TiledqError(f"{name}: {what} holds {_nbytes(t)} bytes, needs {nbytes}")


def _check_weights(name, qtype, w, K, N, flat=False):
    """The weight buffer covers the tiles (or flat blocks) of (qtype, K, N)."""
    nbytes = _size_query("tq_flat_bytes" if flat else "tq_tiled_bytes", qtype, K, N)
    if nbytes == 0 and N > 0:
        raise TiledqError(f"{name}: type {qtype} with K={K}, N={N} is not a valid shape")
    _need_bytes(name, "flat" if flat else "tiles", w, nbytes)


def _check_act(name, q, d, K):
    """q is int8 [M, K] and d fp16 with M * K/32 elements; returns M."""
    if q.dim() != 2 or q.dtype != torch.int8 or q.shape[1] != K:
        raise TiledqError(f"{name}: q must be int8 [M, K={K}], got {q.dtype} {tuple(q.shape)}")
    M = q.shape[0]
    if d is not None:
        if d.dtype != torch.float16:
            raise TiledqError(f"{name}: d must be float16, got {d.dtype}")
        if d.numel() < M * (K // 32):
            raise TiledqError(f"{name}: d holds {d.numel()} scales, needs {M * (K // 32)}")
    return M


def _check_out(name, out, M, N):
    """out is fp32 with unit column stride, at least M rows and N columns."""
    if out is None:
        return
    if out.dim() != 2 or out.dtype != torch.float32 or out.stride(1) != 1 or \
            out.shape[0] < M or out.shape[1] < N:
        raise TiledqError(f"{name}: out must be float32 [>={M}, >={N}] with unit column "
                          f"stride, got {out.dtype} {tuple(out.shape)}")


def _lut_arg(lut):
    if lut is None:
        return None
    vals = [int(v) for v in (lut.tolist() if hasattr(lut, "tolist") else lut)]
    if len(vals) != 16 or any(v < -128 or v > 127 for v in vals):
        raise TiledqError("lut must hold 16 int8 values")
    return (ctypes.c_int8 * 16)(*vals)


def tile_bytes(qtype):
    return lib().tq_tile_bytes(qtype)


def block_bytes(qtype):
    return lib().tq_block_bytes(qtype)


def tiled_bytes(qtype, K, N):
    return lib().tq_tiled_bytes(qtype, K, N)


def flat_bytes(qtype, K, N):
    return lib().tq_flat_bytes(qtype, K, N)


def supported(qtype, K, N, M, path=PATH_GEMV):
    return bool(lib().tq_supported(qtype, K, N, M, path))


def repack_tiles(qtype, flat, K, N, out=None):
    """Flat GGML blocks (uint8 GPU tensor) -> tiles (uint8 GPU tensor)."""
    nbytes = tiled_bytes(qtype, K, N)
    _check_weights("repack_tiles", qtype, flat, K, N, flat=True)
    _need_bytes("repack_tiles", "out", out, nbytes)
    _need_cuda(flat, out)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=flat.device)
    check(lib().tq_repack_tiles(qtype, _ptr(flat), K, N, _ptr(out), _stream(flat)),
          "tq_repack_tiles")
    return out


def quantize_act(x, K=None, q=None, d=None):
    """x [M, >=K] fp32 / bf16 / fp16 -> (q int8 [M, K], d fp16 [M, K/32])."""
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise TiledqError("quantize_act: x must be 2-D fp32, bf16 or fp16")
    if x.stride(1) != 1:
        raise TiledqError("quantize_act: x must have unit column stride")
    M, Kx = x.shape
    K = Kx if K is None else K
    if K > Kx:
        raise TiledqError(f"quantize_act: K={K} exceeds the {Kx} columns of x")
    if q is not None and q.dtype != torch.int8:
        raise TiledqError("quantize_act: q must be int8")
    if d is not None and d.dtype != torch.float16:
        raise TiledqError("quantize_act: d must be float16")
    _need_bytes("quantize_act", "q", q, M * K)
    _need_bytes("quantize_act", "d", d, 2 * M * (K // 32))
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if d is None:
        d = torch.empty((M, K // 32), dtype=torch.float16, device=x.device)
    if not x.is_cuda:
        raise TiledqError("tiledq operates on GPU tensors only")
    _need_cuda(q, d)
    check(lib().tq_quantize_act(_DTYPES[x.dtype], _ptr(x), M, K, x.stride(0), _ptr(q), _ptr(d),
                                _stream(x)), "tq_quantize_act")
    return q, d


def _out(q, N, out):
    """`out` as given (the caller has checked it with _check_out), else a new
    fp32 [M, N] tensor on q's device."""
    if out is None:
        out = torch.empty((q.shape[0], N), dtype=torch.float32, device=q.device)
    return out


# Zero-filled qgemv workspaces, one per (device, stream): every call leaves
# its workspace zero-filled, so it is reused by later calls on the same stream
# without clearing (on one stream no call's launches overlap another's, and
# _with_workspace lets none come between them).  A HIP graph captured
# on a stream keeps that stream's workspace: replaying it on another stream
# while calls run on the capture stream would share the workspace, so replay
# it on the capture stream or keep the two apart in time.  A workspace that has
# become too small is kept: a captured graph may still write to it.  Calls that
# are captured before a workspace large enough was there share one of the
# graph's own, in its memory, of which every replay clears once what has to be
# zero.  It is held until a later capture on that stream or an eager call there:
# the capture's own tensors must not get its memory.
_workspaces = {}
_outgrown = []
_captured = {}                       # (device, stream): capture's number, workspace
_COUNTERS = 1 << 20                  # TQ_NOALLOC_SCRATCH_BYTES: what lies behind is scratch


def _capture_of(stream_handle):
    """Number of the capture that a stream is part of, 0 if none."""
    n = ctypes.c_uint64()
    check(lib().tq_capture_id(stream_handle, ctypes.byref(n)), "tq_capture_id")
    return n.value


def _captured_workspace(device, stream_handle, capture, nbytes):
    key = (device, stream_handle)
    number, ws = _captured.get(key, (0, None))
    if number != capture or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        ws[:_COUNTERS].zero_()
        _captured[key] = (capture, ws)
    return ws


def workspace(device, stream_handle, nbytes):
    key = (device, stream_handle)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        size = max(nbytes, 1 << 16)
        capture = _capture_of(stream_handle) if device.type == "cuda" else 0
        if capture:
            return _captured_workspace(device, stream_handle, capture, size)
        _captured.pop(key, None)
        if ws is not None:
            _outgrown.append(ws)
            size = max(size, 2 * ws.numel())     # so that they stay few
        ws = torch.zeros(size, dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


# A call may be several launches that hand something on in the workspace, and
# threads may share a stream: each stream's calls are enqueued one at a time.
_turns = {}


def _with_workspace(entry, device, st, need, *args):
    """entry(*args, workspace, its bytes, stream): its status."""
    if not need:
        return entry(*args, None, 0, st)
    turn = _turns.get(st)
    if turn is None:
        turn = _turns.setdefault(st, threading.Lock())
    with turn:
        return entry(*args, workspace(device, st, need).data_ptr(), need, st)


def qgemv(qtype, tiles, K, N, q, d, lut=None, out=None, split=True):
    """Decode product y [M, N] = W (tiles) x A (q, d), M <= 8.  split=False
    runs one workgroup per stripe (no workspace)."""
    M = _check_act("tq_qgemv", q, d, K)
    _check_weights("tq_qgemv", qtype, tiles, K, N)
    _check_out("tq_qgemv", out, M, N)
    _need_cuda(tiles, q, d, out=out)
    out = _out(q, N, out)
    st = _stream(q)
    need = _size_query("tq_qgemv_workspace_bytes", qtype, K, N, M) if split else 0
    check(_with_workspace(lib().tq_qgemv, q.device, st, need, qtype, _ptr(tiles), K, N, _ptr(q),
                          _ptr(d), M, _lut_arg(lut), _ptr(out), out.stride(0)), "tq_qgemv")
    return out


def qgemv_noalloc(qtype, tiles, K, N, q, d, lut=None, out=None):
    """qgemv through the entry point that allocates nothing (its K-split
    scratch is a device array inside the library, shared by all calls on a
    GPU: calls that overlap on one GPU race).  Pass `out` to allocate
    nothing here either."""
    M = _check_act("tq_qgemv_noalloc", q, d, K)
    _check_weights("tq_qgemv_noalloc", qtype, tiles, K, N)
    _check_out("tq_qgemv_noalloc", out, M, N)
    _need_cuda(tiles, q, d, out=out)
    out = _out(q, N, out)
    check(lib().tq_qgemv_noalloc(qtype, _ptr(tiles), K, N, _ptr(q), _ptr(d), M, _lut_arg(lut),
                                 _ptr(out), out.stride(0), _stream(q)), "tq_qgemv_noalloc")
    return out


def qgemv_x(qtype, tiles, K, N, x, lut=None, out=None, split=True):
    """Decode in one launch: quantize x [M, >=K] (fp32 / bf16 / fp16) and
    multiply, y [M, N]; bit-identical to quantize_act followed by qgemv."""
    if x.dim() != 2 or x.dtype not in _DTYPES or x.stride(1) != 1:
        raise TiledqError("qgemv_x: x must be 2-D fp32, bf16 or fp16 with unit column stride")
    if x.shape[1] < K:
        raise TiledqError(f"qgemv_x: x has {x.shape[1]} columns, K={K}")
    _check_weights("tq_qgemv_x", qtype, tiles, K, N)
    _check_out("tq_qgemv_x", out, x.shape[0], N)
    _need_cuda(tiles, out=out)
    if not x.is_cuda:
        raise TiledqError("tiledq operates on GPU tensors only")
    M = x.shape[0]
    out = _out(x, N, out)
    st = _stream(x)
    need = _size_query("tq_qgemv_workspace_bytes", qtype, K, N, M) if split else 0
    check(_with_workspace(lib().tq_qgemv_x, x.device, st, need, qtype, _ptr(tiles), K, N,
                          _DTYPES[x.dtype], _ptr(x), x.stride(0), M, _lut_arg(lut), _ptr(out),
                          out.stride(0)), "tq_qgemv_x")
    return out


def qgemm(qtype, tiles, K, N, q, d, lut=None, out=None):
    """Prefill product y [M, N] on int8 MFMA, any M."""
    M = _check_act("tq_qgemm", q, d, K)
    _check_weights("tq_qgemm", qtype, tiles, K, N)
    _check_out("tq_qgemm", out, M, N)
    _need_cuda(tiles, q, d, out=out)
    out = _out(q, N, out)
    check(lib().tq_qgemm(qtype, _ptr(tiles), K, N, _ptr(q), _ptr(d), q.shape[0], _lut_arg(lut),
                         _ptr(out), out.stride(0), _stream(q)), "tq_qgemm")
    return out


def matmul_path(qtype, K, N, M):
    """The path matmul takes: PATH_GEMV, PATH_GEMM_SPLIT or PATH_GEMM."""
    return lib().tq_matmul_path(qtype, K, N, M)


def matmul(qtype, tiles, K, N, q, d, lut=None, out=None):
    """y [M, N] for any M: the library picks qgemv (M <= 8), one qgemv pass
    per 8 rows (up to 64 rows, where estimated faster), the GEMM with K split
    over workgroups (small output grids) or qgemm (matmul_path)."""
    M = _check_act("tq_matmul", q, d, K)
    _check_weights("tq_matmul", qtype, tiles, K, N)
    _check_out("tq_matmul", out, M, N)
    _need_cuda(tiles, q, d, out=out)
    out = _out(q, N, out)
    st = _stream(q)
    need = _size_query("tq_matmul_workspace_bytes", qtype, K, N, M)
    check(_with_workspace(lib().tq_matmul, q.device, st, need, qtype, _ptr(tiles), K, N, _ptr(q),
                          _ptr(d), M, _lut_arg(lut), _ptr(out), out.stride(0)), "tq_matmul")
    return out


def matmul_x(qtype, tiles, K, N, x, lut=None, out=None):
    """y [M, N] from fp32 / bf16 / fp16 activations x [M, >=K], any M: the
    fused decode where it is cheaper, else quantize_act into the workspace
    followed by matmul's path."""
    if x.dim() != 2 or x.dtype not in _DTYPES or x.stride(1) != 1:
        raise TiledqError("matmul_x: x must be 2-D fp32, bf16 or fp16 with unit column stride")
    if x.shape[1] < K:
        raise TiledqError(f"matmul_x: x has {x.shape[1]} columns, K={K}")
    M = x.shape[0]
    _check_weights("tq_matmul_x", qtype, tiles, K, N)
    _check_out("tq_matmul_x", out, M, N)
    _need_cuda(tiles, out=out)
    if not x.is_cuda:
        raise TiledqError("tiledq operates on GPU tensors only")
    out = _out(x, N, out)
    st = _stream(x)
    need = _size_query("tq_matmul_x_workspace_bytes", qtype, K, N, M)
    check(_with_workspace(lib().tq_matmul_x, x.device, st, need, qtype, _ptr(tiles), K, N,
                          _DTYPES[x.dtype], _ptr(x), x.stride(0), M, _lut_arg(lut), _ptr(out),
                          out.stride(0)), "tq_matmul_x")
    return out


def unpack_tiles(qtype, tiles, K, N, out=None):
    """Tiles (uint8 GPU tensor) -> flat GGML blocks (uint8 GPU tensor)."""
    nbytes = flat_bytes(qtype, K, N)
    _check_weights("unpack_tiles", qtype, tiles, K, N)
    _need_bytes("unpack_tiles", "out", out, nbytes)
    _need_cuda(tiles, out)
    if out is None:
        out = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=tiles.device)
    check(lib().tq_unpack_tiles(qtype, _ptr(tiles), K, N, _ptr(out), _stream(tiles)),
          "tq_unpack_tiles")
    return out[:nbytes]


def quantize_act_mx(x, K=None, q=None, e=None):
    """x [M, >=K] fp32 / bf16 / fp16 -> MXFP8 (q uint8 E4M3 codes [M, K],
    e uint8 E8M0 scales [M, K/32])."""
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise TiledqError("quantize_act_mx: x must be 2-D fp32, bf16 or fp16")
    if x.stride(1) != 1:
        raise TiledqError("quantize_act_mx: x must have unit column stride")
    M, Kx = x.shape
    K = Kx if K is None else K
    if K > Kx:
        raise TiledqError(f"quantize_act_mx: K={K} exceeds the {Kx} columns of x")
    _need_bytes("quantize_act_mx", "q", q, M * K)
    _need_bytes("quantize_act_mx", "e", e, M * (K // 32))
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if e is None:
        e = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    if not x.is_cuda:
        raise TiledqError("tiledq operates on GPU tensors only")
    _need_cuda(q, e)
    check(lib().tq_quantize_act_mx(_DTYPES[x.dtype], _ptr(x), M, K, x.stride(0), _ptr(q),
                                   _ptr(e), _stream(x)), "tq_quantize_act_mx")
    return q, e


def qgemm_mx(tiles, K, N, q, e, out=None):
    """MXFP4 tiles x MXFP8 activations on the block-scaled matrix cores:
    y [M, N] fp32, any M."""
    M = q.shape[0]
    if tiles.numel() * tiles.element_size() < tiled_bytes(MXFP4, K, N) or \
            q.numel() < M * K or e.numel() < M * (K // 32):
        raise TiledqError("qgemm_mx: buffer too small")
    _check_out("tq_qgemm_mx", out, M, N)
    _need_cuda(tiles, q, e, out=out)
    out = _out(q, N, out)
    check(lib().tq_qgemm_mx(_ptr(tiles), K, N, _ptr(q), _ptr(e), M, _ptr(out), out.stride(0),
                            _stream(q)), "tq_qgemm_mx")
    return out


def matmul_mx(tiles, K, N, q, e, out=None):
    """qgemm_mx with K split over workgroups where the output grid is small
    (tq_matmul_mx; the per-stream workspace holds the partial planes)."""
    M = q.shape[0]
    if tiles.numel() * tiles.element_size() < tiled_bytes(MXFP4, K, N) or \
            q.numel() < M * K or e.numel() < M * (K // 32):
        raise TiledqError("matmul_mx: buffer too small")
    _check_out("tq_matmul_mx", out, M, N)
    _need_cuda(tiles, q, e, out=out)
    out = _out(q, N, out)
    st = _stream(q)
    need = _size_query("tq_matmul_mx_workspace_bytes", K, N, M)
    check(_with_workspace(lib().tq_matmul_mx, q.device, st, need, _ptr(tiles), K, N, _ptr(q),
                          _ptr(e), M, _ptr(out), out.stride(0)), "tq_matmul_mx")
    return out


def _flat_product(name, qtype, flat, K, N, q, d, lut, out):
    M = _check_act(name, q, d, K)
    _check_weights(name, qtype, flat, K, N, flat=True)
    _check_out(name, out, M, N)
    _need_cuda(flat, q, d, out=out)
    out = _out(q, N, out)
    check(getattr(lib(), name)(qtype, _ptr(flat), K, N, _ptr(q), _ptr(d), q.shape[0],
                               _lut_arg(lut), _ptr(out), out.stride(0), _stream(q)), name)
    return out


def qgemv_flat(qtype, flat, K, N, q, d, lut=None, out=None):
    """Decode product over flat (un-repacked) GGML blocks, M <= 8."""
    return _flat_product("tq_qgemv_flat", qtype, flat, K, N, q, d, lut, out)


def qgemm_flat(qtype, flat, K, N, q, d, lut=None, out=None):
    """Prefill product over flat GGML blocks, any M."""
    return _flat_product("tq_qgemm_flat", qtype, flat, K, N, q, d, lut, out)


def matmul_flat(qtype, flat, K, N, q, d, lut=None, out=None):
    """Product over flat GGML blocks for any M (qgemv_flat for M <= 8)."""
    return _flat_product("tq_matmul_flat", qtype, flat, K, N, q, d, lut, out)


def block_dots(qtype, tiles, K, N, q, lut=None, path=PATH_GEMV, out=None):
    """Integer block dots int32 [M, N, K/32] as computed inside qgemv / qgemm
    (paths PATH_GEMV_FLAT / PATH_GEMM_FLAT: `tiles` holds flat blocks)."""
    M = _check_act("tq_block_dots", q, None, K)
    _check_weights("tq_block_dots", qtype, tiles, K, N,
                   flat=path in (PATH_GEMV_FLAT, PATH_GEMM_FLAT))
    if out is not None and out.dtype != torch.int32:
        raise TiledqError("tq_block_dots: out must be int32")
    _need_bytes("tq_block_dots", "out", out, 4 * M * N * (K // 32))
    _need_cuda(tiles, q, out)
    if out is None:
        out = torch.empty((M, N, K // 32), dtype=torch.int32, device=q.device)
    check(lib().tq_block_dots(qtype, _ptr(tiles), K, N, _ptr(q), M, _lut_arg(lut), _ptr(out),
                              path, _stream(q)), "tq_block_dots")
    return out


# The decode-step operators run once or more per layer and token, so their
# checks are written for few Python operations: one condition per tensor,
# details only once it has failed.

def _refuse(name, what, want, t):
    if not t.is_cuda:
        raise TiledqError("tiledq operates on GPU tensors only")
    raise TiledqError(f"{name}: {what} must be {want}, got {t.dtype} {tuple(t.shape)} with strides "
                      f"{t.stride()} on {t.device}")


def _check_index(name, what, t, n, dev):
    """t is a contiguous int32 vector of at least n elements on device dev."""
    if t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] < n or t.get_device() != dev or \
            not t.is_contiguous():
        _refuse(name, what, f"contiguous int32, 1-D, >= {n} elements, on device {dev}", t)


def _check_heads(name, what, t, shape, dtype, dev):
    """t is `shape` of dtype on device dev with contiguous rows; returns its
    token and head strides."""
    if t.shape != shape or t.dtype is not dtype or (t.stride(2) != 1 and shape[2] > 1) or \
            t.get_device() != dev:
        _refuse(name, what, f"{dtype} {tuple(shape)} with contiguous rows on device {dev}", t)
    return t.stride(0), t.stride(1)


def _heads_of(name, what, t, dtypes):
    """Shape, strides, device of t [tokens, heads, D] on the GPU."""
    code = dtypes.get(t.dtype)
    dev = t.get_device()
    if t.dim() != 3 or code is None or dev < 0:
        _refuse(name, what, f"[tokens, heads, D] of {[str(d) for d in dtypes]}", t)
    shape = t.shape
    ts, hs, es = t.stride()
    if es != 1 and shape[2] > 1:
        _refuse(name, what, "[tokens, heads, D] with contiguous rows", t)
    return shape, ts, hs, dev, code


def _stream_of(dev):
    """The current HIP stream of GPU number dev, as an int handle."""
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None):
    """RMS norm of each head of q [T, Hq, D] and k [T, Hk, D] (fp32 / bf16 /
    fp16, any token and head strides) with weights [D] (None: no norm), then
    the rotation of its first 2 * len(inv_freq) elements by the angles
    positions [T] (int32) * inv_freq (fp32): pairs (i, i + half), or
    neighbours if interleaved.  q_out, k_out may be q, k.  Returns both."""
    name = "tq_qk_norm_rope"
    qshape, q_ts, q_hs, dev, code = _heads_of(name, "q", q, _DTYPES)
    T, Hq, D = qshape
    dtype = q.dtype
    if k.dim() != 3:
        _refuse(name, "k", f"[{T}, heads, {D}]", k)
    Hk = k.shape[1]
    kshape = (T, Hk, D)
    k_ts, k_hs = _check_heads(name, "k", k, kshape, dtype, dev)
    _check_index(name, "positions", positions, T, dev)
    if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or \
            inv_freq.get_device() != dev or not inv_freq.is_contiguous():
        _refuse(name, "inv_freq", f"contiguous float32, 1-D, on device {dev}", inv_freq)
    wcode = code
    qw = kw = None
    for what, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            wcode = _DTYPES.get(w.dtype)
            if wcode is None or w.dim() != 1 or w.shape[0] != D or w.get_device() != dev or \
                    not w.is_contiguous():
                _refuse(name, what, f"contiguous fp32, bf16 or fp16 [{D}] on device {dev}", w)
    if q_weight is not None:
        qw = q_weight.data_ptr()
    if k_weight is not None:
        if q_weight is not None and q_weight.dtype is not k_weight.dtype:
            raise TiledqError(f"{name}: q_weight and k_weight must share a type")
        kw = k_weight.data_ptr()
    if q_out is None:
        q_out = torch.empty_like(q)
        qo_ts, qo_hs, _ = q_out.stride()
    else:
        qo_ts, qo_hs = _check_heads(name, "q_out", q_out, qshape, dtype, dev)
    if k_out is None:
        k_out = torch.empty_like(k)
        ko_ts, ko_hs, _ = k_out.stride()
    else:
        ko_ts, ko_hs = _check_heads(name, "k_out", k_out, kshape, dtype, dev)
    status = lib().tq_qk_norm_rope(
        code, q.data_ptr(), q_ts, q_hs, Hq, k.data_ptr(), k_ts, k_hs, Hk, T, D,
        2 * inv_freq.shape[0], 1 if interleaved else 0, wcode, qw, kw, eps, positions.data_ptr(),
        inv_freq.data_ptr(), q_out.data_ptr(), qo_ts, qo_hs, k_out.data_ptr(), ko_ts, ko_hs,
        _stream_of(dev))
    if status:
        check(status, name)
    return q_out, k_out


def cache_bytes(ctype, n_pages, page_size, kv_heads, D):
    """Bytes of one of the two buffers (keys, values) of a paged cache."""
    return lib().tq_cache_bytes(ctype, n_pages, page_size, kv_heads, D)


def _cache_pages(name, ctype, k_cache, v_cache, page_size, kv_heads, D, dev):
    """Pages of a cache, from its buffers' size."""
    page = _size_query("tq_cache_bytes", ctype, 1, page_size, kv_heads, D)
    if page == 0:
        raise TiledqError(f"{name}: no cache of type {ctype} with {kv_heads} heads of {D} and "
                          f"pages of {page_size}")
    for what, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if c.dtype is not torch.uint8 or c.get_device() != dev or not c.is_contiguous():
            _refuse(name, what, f"contiguous uint8 on device {dev}", c)
    n = k_cache.numel()
    if n != v_cache.numel() or n == 0 or n % page:
        raise TiledqError(f"{name}: caches hold {n} and {v_cache.numel()} bytes, not the same "
                          f"whole number of pages of {page}")
    return n // page


def cache_write(ctype, k, v, k_cache, v_cache, slots, page_size):
    """Quantize k, v [T, H, D] (fp32 / bf16 / fp16) into slots [T] (int32,
    page * page_size + position; one outside the cache is skipped) of a paged
    Q8_0 or Q4_0 cache (uint8 buffers of cache_bytes)."""
    name = "tq_cache_write"
    shape, k_ts, k_hs, dev, code = _heads_of(name, "k", k, _DTYPES)
    T, H, D = shape
    if v.dim() != 3:
        _refuse(name, "v", f"{tuple(shape)}", v)
    v_ts, v_hs = _check_heads(name, "v", v, shape, k.dtype, dev)
    _check_index(name, "slots", slots, T, dev)
    n_pages = _cache_pages(name, ctype, k_cache, v_cache, page_size, H, D, dev)
    status = lib().tq_cache_write(
        ctype, code, k.data_ptr(), k_ts, k_hs, v.data_ptr(), v_ts, v_hs, T, H, D,
        slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), n_pages, page_size,
        _stream_of(dev))
    if status:
        check(status, name)


def cache_read(ctype, k_cache, v_cache, slots, kv_heads, D, page_size, dtype=torch.float32):
    """The values of cache slots [T]: (k, v) [T, kv_heads, D] of dtype; a slot
    outside the cache reads as zeros."""
    name = "tq_cache_read"
    code = _DTYPES.get(dtype)
    if code is None:
        raise TiledqError(f"{name}: dtype must be float32, bfloat16 or float16")
    dev = slots.get_device()
    if dev < 0 or slots.dim() != 1:
        _refuse(name, "slots", "int32, 1-D", slots)
    T = slots.shape[0]
    _check_index(name, "slots", slots, T, dev)
    n_pages = _cache_pages(name, ctype, k_cache, v_cache, page_size, kv_heads, D, dev)
    k = torch.empty((T, kv_heads, D), dtype=dtype, device=slots.device)
    v = torch.empty_like(k)
    status = lib().tq_cache_read(
        ctype, code, k_cache.data_ptr(), v_cache.data_ptr(), n_pages, page_size, kv_heads, D,
        slots.data_ptr(), T, k.data_ptr(), v.data_ptr(), _stream_of(dev))
    if status:
        check(status, name)
    return k, v


_ATTN_DTYPES = {torch.bfloat16: BF16, torch.float16: F16}


def tree_attention(ctype, q, k_cache, v_cache, page_table, ctx_lens, starts, kv_heads, page_size,
                   max_nodes=None, max_ctx=None, scale=None, mask=None, out=None):
    """Attention of new tokens q [T, Hq, D] (bf16 / fp16) over a paged cache
    that already holds their keys and values.  Sequence b: rows starts[b] ..
    starts[b+1]-1 of q, pages page_table[b] (int32 [B, pages]), ctx_lens[b]
    tokens before the new ones.  mask: int32 [T, words], bit j of a row = new
    token j of the sequence is seen (None: the chain, j <= i).  max_nodes and
    max_ctx bound the new and the cached tokens of a sequence; they default
    to all rows of q and all of the table.  scale defaults to D ** -0.5."""
    name = "tq_tree_attention"
    shape, q_ts, q_hs, dev, code = _heads_of(name, "q", q, _ATTN_DTYPES)
    T, Hq, D = shape
    if page_table.dim() != 2 or page_table.dtype is not torch.int32 or \
            page_table.get_device() != dev or (page_table.shape[1] > 1 and
                                               page_table.stride(1) != 1):
        _refuse(name, "page_table", f"int32 [batch, pages], rows contiguous, on device {dev}",
                page_table)
    B, width = page_table.shape
    _check_index(name, "ctx_lens", ctx_lens, B, dev)
    _check_index(name, "starts", starts, B + 1, dev)
    n_pages = _cache_pages(name, ctype, k_cache, v_cache, page_size, kv_heads, D, dev)
    words = stride = 0
    mp = None
    if mask is not None:
        if mask.dim() != 2 or mask.dtype is not torch.int32 or mask.shape[0] < T or \
                mask.get_device() != dev or (mask.shape[1] > 1 and mask.stride(1) != 1):
            _refuse(name, "mask", f"int32 [{T}, words], rows contiguous, on device {dev}", mask)
        words, stride, mp = mask.shape[1], mask.stride(0), mask.data_ptr()
    if max_nodes is None:
        max_nodes = max(T, 1)
    if max_ctx is None:
        max_ctx = width * page_size
    if out is None:
        out = torch.empty_like(q)
        o_ts, o_hs, _ = out.stride()
    else:
        if out.dim() != 3 or out.shape[0] < T:
            _refuse(name, "out", f"[>= {T}, {Hq}, {D}]", out)
        o_ts, o_hs = _check_heads(name, "out", out, (out.shape[0], Hq, D), q.dtype, dev)
    st = _stream_of(dev)
    need = _size_query("tq_tree_attention_workspace_bytes", B, Hq, kv_heads, D, max_nodes, max_ctx)
    status = _with_workspace(
        lib().tq_tree_attention, q.device, st, need, ctype, code, q.data_ptr(), q_ts, q_hs, T, Hq,
        kv_heads, D, k_cache.data_ptr(), v_cache.data_ptr(), n_pages, page_size,
        page_table.data_ptr(), page_table.stride(0), width, B, ctx_lens.data_ptr(),
        starts.data_ptr(), mp, stride, words, max_nodes, max_ctx,
        D ** -0.5 if scale is None else scale, out.data_ptr(), o_ts, o_hs)
    if status:
        check(status, name)
    return out


def verify_draft(target, tokens, starts, uniforms, final_uniforms, draft=None, parents=None,
                 max_nodes=None):
    """Accept drafted tokens against the target's probabilities.  Sequence b:
    nodes starts[b] .. starts[b+1]-1, node 0 the last certain token; target
    [N, V] (fp32 / bf16 / fp16): row n the target's distribution after node n;
    draft [N, V]: the one n's children were drawn from (None: tokens chosen
    without chance); tokens, parents int32 [N] (parents None: chains);
    uniforms fp32 [N], final_uniforms fp32 [B].  Returns int32 (accepted [B],
    tokens [B, max_nodes]: the accepted tokens, the next one, -1s; nodes [B,
    max_nodes]: the accepted nodes, -1s).  max_nodes bounds the nodes of a
    sequence; it defaults to all of them."""
    name = "tq_verify_draft"
    code = _DTYPES.get(target.dtype)
    dev = target.get_device()
    if target.dim() != 2 or code is None or dev < 0 or \
            (target.shape[1] > 1 and target.stride(1) != 1):
        _refuse(name, "target", "[nodes, vocab] fp32, bf16 or fp16 with contiguous rows", target)
    N, V = target.shape
    dp = parp = None
    d_stride = 0
    if draft is not None:
        if draft.shape != target.shape or draft.dtype is not target.dtype or \
                draft.get_device() != dev or (V > 1 and draft.stride(1) != 1):
            _refuse(name, "draft", f"{target.dtype} {tuple(target.shape)} with contiguous rows on "
                                   f"device {dev}", draft)
        dp, d_stride = draft.data_ptr(), draft.stride(0)
    _check_index(name, "tokens", tokens, N, dev)
    if parents is not None:
        _check_index(name, "parents", parents, N, dev)
        parp = parents.data_ptr()
    _check_index(name, "starts", starts, 1, dev)
    B = starts.shape[0] - 1
    for what, t, n in (("uniforms", uniforms, N), ("final_uniforms", final_uniforms, B)):
        if t.dtype is not torch.float32 or t.dim() != 1 or t.shape[0] < n or \
                t.get_device() != dev or not t.is_contiguous():
            _refuse(name, what, f"contiguous float32, 1-D, >= {n} elements, on device {dev}", t)
    width = max(N, 1) if max_nodes is None else max_nodes
    if width < 1:
        raise TiledqError(f"{name}: max_nodes must be at least 1")
    device = target.device
    accepted = torch.empty(B, dtype=torch.int32, device=device)
    out_tokens = torch.empty((B, width), dtype=torch.int32, device=device)
    nodes = torch.empty_like(out_tokens)
    st = _stream_of(dev)
    need = _size_query("tq_verify_draft_workspace_bytes", B, V)
    status = _with_workspace(
        lib().tq_verify_draft, device, st, need, code, target.data_ptr(), target.stride(0), dp,
        d_stride, N, V, tokens.data_ptr(), parp, starts.data_ptr(), B, uniforms.data_ptr(),
        final_uniforms.data_ptr(), width, accepted.data_ptr(), out_tokens.data_ptr(),
        nodes.data_ptr())
    if status:
        check(status, name)
    return accepted, out_tokens, nodes


STREAM_READ_BLOCKS = 2048       # TQ_STREAM_READ_BLOCKS: words of the sink


def stream_read(buf, nbytes=None, sink=None):
    """Measurement instrument: read the first `nbytes` bytes of `buf` (all of
    it by default) once with the library's streaming-read kernel.  Returns
    the int32 sink [STREAM_READ_BLOCKS]; the XOR of its words is the XOR of
    every 32-bit word read."""
    nbytes = _nbytes(buf) if nbytes is None else nbytes
    _need_bytes("tq_stream_read", "buf", buf, nbytes)
    if sink is not None and sink.dtype != torch.int32:
        raise TiledqError("tq_stream_read: sink must be int32")
    _need_bytes("tq_stream_read", "sink", sink, 4 * STREAM_READ_BLOCKS)
    _need_cuda(buf, sink)
    if sink is None:
        sink = torch.empty(STREAM_READ_BLOCKS, dtype=torch.int32, device=buf.device)
    check(lib().tq_stream_read(_ptr(buf), nbytes, _ptr(sink), _stream(buf)), "tq_stream_read")
    return sink
