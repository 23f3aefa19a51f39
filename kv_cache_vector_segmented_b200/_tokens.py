"""ctypes binding of rotary positions and the exact token cache (the
ri_rotary* and ri_token_* calls of include/retroinfer.h).

Argument marshalling only, as in _binding: tensors are checked for device,
dtype, shape and layout, and the calls run on torch's current stream of the
tensors' device, made current around the call where it is not.

rotary is differentiable; the cache's calls serve and record no gradient.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import (_need, _P, _ptr, _sz, _vp, RI_OK, RIError, STATUS_CODES,
                       alloc_workspace, check, lib)

# the current device and a device's current stream without torch.cuda's
# wrappers: a decode step makes these calls once each, and they are cheap
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream

BF16, FP16, FP32 = 0, 1, 2
_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


class CHeads(ctypes.Structure):
    _fields_ = [("data", _vp), ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


class RotaryConfig(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_len", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double)]


class CRope(ctypes.Structure):
    _fields_ = [("turns", _vp), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_float)]


class CTokenCache(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("K", _vp), ("V", _vp), ("pos", _vp),
                ("weight", _vp), ("lens", _vp)]


class CTokenPrefix(ctypes.Structure):
    _fields_ = [("K", _vp), ("V", _vp), ("length", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


_i32, _i64 = ctypes.c_int32, ctypes.c_int64
lib.ri_rotary_table.restype = ctypes.c_int
lib.ri_rotary_table.argtypes = [_P(RotaryConfig), _vp, _vp, _P(ctypes.c_double)]
lib.ri_rotary.restype = ctypes.c_int
lib.ri_rotary.argtypes = [_i32, _i32, _i32, _i32, _i32, _P(CHeads), _vp, _i64, _P(CRope),
                          _P(CHeads), _i32, _vp]
lib.ri_token_append.restype = ctypes.c_int
lib.ri_token_append.argtypes = [_P(CTokenCache), _i32, _P(CHeads), _P(CHeads), _vp, _i64,
                                _P(CRope), _P(CHeads), _vp, _vp, _vp, _vp]
lib.ri_token_attend_workspace.restype = _sz
lib.ri_token_attend_workspace.argtypes = [_P(CTokenCache), _i32]
lib.ri_token_attend.restype = ctypes.c_int
lib.ri_token_attend.argtypes = [_P(CTokenCache), _vp, _P(CTokenPrefix), _vp, _vp, _i32, _vp, _sz,
                                _vp]
lib.ri_selftest_token_attend_timeout.restype = ctypes.c_int
lib.ri_selftest_token_attend_timeout.argtypes = [_P(CTokenCache), _vp, _P(CTokenPrefix), _vp, _vp,
                                                 _i32, _vp, _sz, _i32, ctypes.c_uint64, _vp]
lib.ri_token_evict_workspace.restype = _sz
lib.ri_token_evict_workspace.argtypes = [_P(CTokenCache), _i32]
lib.ri_token_evict.restype = ctypes.c_int
lib.ri_token_evict.argtypes = [_P(CTokenCache), _i32, _i32, _i32, _P(CTokenCache), _vp, _sz, _vp]


def _run(dev: torch.device, fn, where: str, *args) -> None:
    """fn(*args, stream) on torch's current stream of the tensors' device, which
    is made current around the call where it is not."""
    if dev.type != "cuda":
        raise ValueError("the token cache's calls need CUDA tensors")
    i = dev.index
    if i == _current_device():
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            rc = fn(*args, _raw_stream(i))
    if rc != RI_OK:
        raise RIError(rc, where)


def _dense(t, name: str, dtype: torch.dtype, shape: tuple, dev) -> int:
    """The address of a contiguous tensor of this dtype, shape and device."""
    if type(t) is not torch.Tensor or t.dtype != dtype or t.shape != shape or \
            t.device != dev or not t.is_contiguous():
        _need(t, name, dtype, shape, dev)
    return t.data_ptr()


class RotaryTable:
    """Angles of rotary positions on a device: per rotated pair the turns per
    position as a 64-bit fraction (ri_rotary_table), the layout of the pairs
    and the factor on the rotated values."""

    def __init__(self, turns: torch.Tensor, magnitude: float = 1.0, interleaved: bool = False,
                 frequencies: Optional[torch.Tensor] = None):
        _need(turns, "turns", torch.int64, (turns.shape[0],) if turns.dim() == 1 else (-1,))
        self.turns, self.frequencies = turns, frequencies
        self.rotary_dim = 2 * turns.shape[0]
        self.magnitude, self.interleaved = float(magnitude), bool(interleaved)
        self._c = CRope(turns.data_ptr(), self.rotary_dim, int(self.interleaved), self.magnitude)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def make(cls, rotary_dim: int = 128, base: float = 10000.0, scaling: str = "none",
             factor: float = 1.0, original_len: int = 8192, low: Optional[float] = None,
             high: Optional[float] = None, interleaved: bool = False, device="cuda"):
        """The table of frequencies base^(-2i / rotary_dim), scaled for long
        contexts as ri_rotary_config says; low / high default to 1 and 4
        ("bands") or 1 and 32 ("yarn")."""
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
        low = 1.0 if low is None else low
        high = (32.0 if scaling == "yarn" else 4.0) if high is None else high
        cfg = RotaryConfig(rotary_dim, ROPE_SCALINGS[scaling], original_len, 0, base, factor, low,
                           high)
        n = max(1, min(rotary_dim, 256) // 2)
        turns = torch.zeros(n, dtype=torch.int64)
        freq = torch.zeros(n, dtype=torch.float64)
        mag = ctypes.c_double(1.0)
        check(lib.ri_rotary_table(ctypes.byref(cfg), turns.data_ptr(), freq.data_ptr(),
                                  ctypes.byref(mag)), "ri_rotary_table")
        return cls(turns.to(device), mag.value, interleaved, freq)


def _heads(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, dev,
           measure: bool = False) -> CHeads:
    """A strided [B][T][heads][d] tensor as the C struct; only d must be
    contiguous.  (The stride of an extent of one says nothing: it is passed as 0.)
    `measure`: dtype, shape and dev are the tensor's own."""
    if not measure:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
    sb, st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    B, T, H, _ = shape
    return CHeads(t.data_ptr(), sb if B > 1 else 0, st if T > 1 else 0, sh if H > 1 else 0)


def _positions(pos: torch.Tensor, B: int, T: int, dev) -> int:
    """Checks int32 positions [B][T] (tokens contiguous); the sequences' stride."""
    if not isinstance(pos, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    if pos.dtype != torch.int32:
        raise TypeError(f"positions must be torch.int32, got {pos.dtype}")
    if pos.shape != (B, T):
        raise ValueError(f"positions must have shape {(B, T)}, got {tuple(pos.shape)}")
    if pos.device != dev:
        raise ValueError(f"positions must be on {dev}, got {pos.device}")
    sb, st = pos.stride()
    if T > 1 and st != 1:
        raise ValueError("positions must be contiguous over the tokens")
    return sb


def _no_overlap(out: torch.Tensor, name: str) -> None:
    """A written tensor addresses every element once (no stride-0 views)."""
    if 0 in out.stride() and any(s == 0 and n > 1 for s, n in zip(out.stride(), out.shape)):
        raise ValueError(f"{name} must not repeat elements (a stride of 0)")


class _Rotary(torch.autograd.Function):
    """The rotation is linear and orthogonal up to its magnitude: the gradient
    of its input is the inverse rotation of its output's."""

    @staticmethod
    def forward(ctx, x, positions, table, inverse):
        ctx.save_for_backward(positions)
        ctx.table, ctx.inverse = table, inverse
        return rotary(x, positions, table, inverse=inverse)

    @staticmethod
    def backward(ctx, grad):
        if grad.stride(-1) != 1:
            grad = grad.contiguous()
        return rotary(grad, *ctx.saved_tensors, ctx.table, inverse=not ctx.inverse), None, None, \
            None


def rotary(x: torch.Tensor, positions: torch.Tensor, table: RotaryTable,
           out: Optional[torch.Tensor] = None, inverse: bool = False) -> torch.Tensor:
    """Rotary positions (ri_rotary) on heads x [B][T][heads][d] (bf16, fp16 or
    fp32; any strides with d contiguous), positions int32 [B][T].  `out` may
    be x itself, or a tensor or view of x's shape (the transpose of
    [B][heads][T][d], say: the layout build_index takes); a new dense tensor
    when not given.  inverse=True turns back: the backward pass of the
    rotation on its output's gradient.  Differentiable in x, without `out`."""
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError("x must be a tensor [batch][tokens][heads][head_dim]")
    if x.dtype not in _DTYPES:
        raise TypeError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    if (x.requires_grad or (out is not None and out.requires_grad)) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("rotary records no gradient with `out`: leave it out, or call under "
                             "torch.no_grad()")
        return _Rotary.apply(x, positions, table, inverse)
    dev, shape, dtype = x.device, x.shape, x.dtype
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    cx = _heads(x, "x", dtype, shape, dev, measure=True)
    co = _heads(out, "out", dtype, shape, dev)
    _no_overlap(out, "out")
    B, T, H, d = shape
    sb = _positions(positions, B, T, dev)
    if table.turns.device != dev:
        raise ValueError(f"table must be on {dev}, got {table.turns.device}")
    if x.numel() == 0:
        return out
    _run(dev, lib.ri_rotary, "ri_rotary", B, T, H, d, _DTYPES[dtype], ctypes.byref(cx),
         positions.data_ptr(), sb, table._ref, ctypes.byref(co), 1 if inverse else 0)
    return out


class TokenCache:
    """The exact tokens of every (sequence, KV head) (ri_token_cache): K, V
    bf16 [B][H_kv][capacity][128], pos int32 and weight fp32
    [B][H_kv][capacity], lens int32 [B][H_kv].  The tensors are the caller's
    and stay where they are; `status` is a 256-byte status region for
    token_append (read_device_status(cache.status))."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor, pos: torch.Tensor,
                 weight: torch.Tensor, lens: torch.Tensor, group_size: int = 1):
        if not isinstance(K, torch.Tensor) or K.dim() != 4:
            raise ValueError("K must be a tensor [batch][num_kv_heads][capacity][head_dim]")
        B, H, cap, d = K.shape
        dev = K.device
        _need(K, "K", torch.bfloat16, (B, H, cap, d), dev)
        _need(V, "V", torch.bfloat16, (B, H, cap, d), dev)
        _need(pos, "pos", torch.int32, (B, H, cap), dev)
        _need(weight, "weight", torch.float32, (B, H, cap), dev)
        _need(lens, "lens", torch.int32, (B, H), dev)
        self.K, self.V, self.pos, self.weight, self.lens = K, V, pos, weight, lens
        self.batch, self.num_kv_heads, self.capacity = B, H, cap
        self.group_size, self.head_dim, self.device = group_size, d, dev
        self._c = CTokenCache(B, H, group_size, d, cap, K.data_ptr(), V.data_ptr(),
                              pos.data_ptr(), weight.data_ptr(), lens.data_ptr())
        self._ref = ctypes.byref(self._c)
        token_attend_workspace_bytes(self, 0)  # the library's checks of the sizes
        self.status = alloc_workspace(256, dev)

    @classmethod
    def empty(cls, batch: int, num_kv_heads: int, group_size: int, capacity: int, device="cuda",
              head_dim: int = 128):
        """A cache without tokens."""
        shape = (batch, num_kv_heads, capacity)
        kv = [torch.empty(shape + (head_dim,), dtype=torch.bfloat16, device=device)
              for _ in range(2)]
        return cls(*kv, torch.zeros(shape, dtype=torch.int32, device=device),
                   torch.zeros(shape, dtype=torch.float32, device=device),
                   torch.zeros(shape[:2], dtype=torch.int32, device=device), group_size)


def token_append(cache: TokenCache, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                 table: Optional[RotaryTable] = None, q: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None,
                 lens_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """ri_token_append: stores k (rotated by `table`; None: as it is) and v
    bf16 [B][T][H_kv][128] behind every sequence's last token, and returns the
    step's queries q [B][T][H_q][128] rotated (None without q).  positions
    int32 [B][T].  The lengths advance in place, or into lens_out.  A head
    without room stores nothing and RI_ERR_CAPACITY is recorded in
    cache.status."""
    B, H, d, dev = cache.batch, cache.num_kv_heads, cache.head_dim, cache.device
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a tensor [batch][tokens][num_kv_heads][head_dim]")
    T = k.shape[1]
    ck = _heads(k, "k", torch.bfloat16, (B, T, H, d), dev)
    cv = _heads(v, "v", torch.bfloat16, (B, T, H, d), dev)
    sb = _positions(positions, B, T, dev)
    if table is not None and table.turns.device != dev:
        raise ValueError(f"table must be on {dev}, got {table.turns.device}")
    cq = None
    if q is not None:
        shape = (B, T, H * cache.group_size, d)
        cq = ctypes.byref(_heads(q, "q", torch.bfloat16, shape, dev))
        if q_out is None:
            q_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        _dense(q_out, "q_out", torch.bfloat16, shape, dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if lens_out is None:
        lens_out = cache.lens
    else:
        _dense(lens_out, "lens_out", torch.int32, (B, H), dev)
    _run(dev, lib.ri_token_append, "ri_token_append", cache._ref, T, ctypes.byref(ck),
         ctypes.byref(cv), positions.data_ptr(), sb, None if table is None else table._ref, cq,
         _ptr(q_out), lens_out.data_ptr(), cache.status.data_ptr())
    return q_out


def token_attend_workspace_bytes(cache: TokenCache, prefix_len: int = 0) -> int:
    n = lib.ri_token_attend_workspace(cache._ref, prefix_len)
    if n == 0:
        raise RIError(STATUS_CODES["RI_ERR_INVALID_ARG"], "ri_token_attend_workspace")
    return n


def token_attend(q: torch.Tensor, cache: TokenCache, prefix: Optional[tuple] = None,
                 add_weight: bool = True, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None):
    """ri_token_attend: one query token per sequence, q bf16 [B][H_q][128],
    over the shared prefix (K, V bf16 [H_kv][P][128] each, of equal strides
    with 128 contiguous; None: none) and the cache's own tokens, whose
    attention weights are added to cache.weight unless add_weight is False.
    Returns (out bf16 [B][H_q][128], lse fp32 [B][H_q])."""
    return _attend(q, cache, prefix, add_weight, out, lse, workspace, lib.ri_token_attend,
                   "ri_token_attend")


def selftest_token_attend_timeout(q: torch.Tensor, cache: TokenCache, prefix: tuple,
                                  workspace: torch.Tensor, hand_off: int, limit_ns: int,
                                  add_weight: bool = True):
    """ri_selftest_token_attend_timeout: a call whose first block over the
    prefix leaves one hand-off undone (1: a tile's copy, 2: the scores'
    signal), every wait limited to limit_ns."""
    return _attend(q, cache, prefix, add_weight, None, None, workspace,
                   lib.ri_selftest_token_attend_timeout, "ri_selftest_token_attend_timeout",
                   hand_off, limit_ns)


def _attend(q, cache, prefix, add_weight, out, lse, workspace, fn, where, *test):
    B, H, d, dev = cache.batch, cache.num_kv_heads, cache.head_dim, cache.device
    shape = (B, H * cache.group_size, d)
    q_ptr = _dense(q, "q", torch.bfloat16, shape, dev)
    cp, P = None, 0
    if prefix is not None:
        K, V = prefix
        for t, name in ((K, "prefix K"), (V, "prefix V")):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be a torch.bfloat16 tensor")
            if t.dim() != 3 or t.shape[0] != H or t.shape[2] != d:
                raise ValueError(f"{name} must have shape ({H}, length, {d}), got "
                                 f"{tuple(t.shape)}")
            if t.device != dev:
                raise ValueError(f"{name} must be on {dev}, got {t.device}")
        P = K.shape[1]
        if V.shape != K.shape:
            raise ValueError("prefix K and V must have equal shapes and strides")
        if P:
            (sh, st, sd), (vh, vt, vd) = K.stride(), V.stride()
            if (H > 1 and vh != sh) or (P > 1 and vt != st):
                raise ValueError("prefix K and V must have equal shapes and strides")
            if sd != 1 or vd != 1:
                raise ValueError("prefix: the head dimension must be contiguous")
            if P == 1:
                st = d
            cp = ctypes.byref(CTokenPrefix(K.data_ptr(), V.data_ptr(), P, 0, st, sh))
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _dense(out, "out", torch.bfloat16, shape, dev)
    if lse is None:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=dev)
    else:
        _dense(lse, "lse", torch.float32, shape[:2], dev)
    if workspace is None:
        workspace = alloc_workspace(token_attend_workspace_bytes(cache, P), dev)
    elif workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}, got {workspace.device}")
    _run(dev, fn, where, cache._ref, q_ptr, cp, out.data_ptr(), lse.data_ptr(),
         1 if add_weight else 0, workspace.data_ptr(), workspace.numel(), *test)
    return out, lse


def token_evict_workspace_bytes(cache: TokenCache, budget: int) -> int:
    n = lib.ri_token_evict_workspace(cache._ref, budget)
    if n == 0:
        raise RIError(STATUS_CODES["RI_ERR_INVALID_ARG"], "ri_token_evict_workspace")
    return n


def token_evict(cache: TokenCache, budget: int, keep_first: int = 4, keep_recent: int = 64,
                out: Optional[TokenCache] = None,
                workspace: Optional[torch.Tensor] = None) -> TokenCache:
    """ri_token_evict: reduces every (sequence, KV head) to its `budget` tokens
    of most attention weight, those at positions < keep_first and the
    keep_recent newest positions before all others (by row, where they alone
    are more than the budget); in place, or into `out`
    (which may share some of the cache's tensors).  Returns the cache that
    holds the result."""
    dev = cache.device
    out = cache if out is None else out
    if out.device != dev:
        raise ValueError(f"out must be on {dev}, got {out.device}")
    if workspace is None:
        workspace = alloc_workspace(token_evict_workspace_bytes(cache, budget), dev)
    elif workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}, got {workspace.device}")
    _run(dev, lib.ri_token_evict, "ri_token_evict", cache._ref, budget, keep_first, keep_recent,
         out._ref, workspace.data_ptr(), workspace.numel())
    return out
