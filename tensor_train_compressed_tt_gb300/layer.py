"""PyTorch-facing wrappers over the libttc C ABI.

PyTorch supplies device memory and the stream; each method marshals tensor
pointers into one libttc call.  No arithmetic happens here.
"""

from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import ttc

_DT = {torch.float32: ttc.TT_DT_F32, torch.bfloat16: ttc.TT_DT_BF16}
# E4M3 activations: x / dy hold one-byte codes (a float8_e4m3fn tensor, or
# uint8 holding the same bytes); y / dx come back in bf16.
if hasattr(torch, "float8_e4m3fn"):
    _DT[torch.float8_e4m3fn] = ttc.TT_DT_E4M3
_DT[torch.uint8] = ttc.TT_DT_E4M3


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    """The stream's handle, by default the current one's: asked for without the
    torch.cuda.Stream object around it, which takes 2.9 us, a quarter of a small
    call on the host."""
    if stream is not None:
        return int(stream.cuda_stream)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _filled(shape, dtype: torch.dtype, device, fill: Optional[float]) -> torch.Tensor:
    if fill is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return torch.full(shape, fill, dtype=dtype, device=device)


def _new(shape, dtype: torch.dtype, device, stream: Optional[torch.cuda.Stream],
         fill: Optional[float] = None) -> torch.Tensor:
    """An output that the caller did not give: of the memory of the stream that the
    kernels run on, so that nothing else still uses it there, and held for the
    caller's stream, which reads it afterwards.  fill: what it holds where the
    kernels do not write it."""
    if stream is None:
        return _filled(shape, dtype, device, fill)
    with torch.cuda.stream(stream):
        t = _filled(shape, dtype, device, fill)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _grad_fill(accumulate: bool) -> Optional[float]:
    """What a gradient that the call makes starts from: it is added to, or overwritten."""
    return 0.0 if accumulate else None


def _scratch(stream: Optional[torch.cuda.Stream], workspace, *args) -> torch.Tensor:
    """A workspace that is dropped at the call's end: of the memory of the call's
    stream, where it is next used after the call's kernels."""
    if stream is None:
        return workspace(*args)
    with torch.cuda.stream(stream):
        return workspace(*args)


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else int(t.data_ptr())


class TTLinear:
    """One TT linear layer: y (T x M) = x (T x N) W^T, W given by packed cores."""

    def __init__(self, in_modes: Sequence[int], out_modes: Sequence[int],
                 ranks: Sequence[int], dtype: torch.dtype = torch.bfloat16,
                 accumulate: bool = False, reuse_merge: bool = False, reuse_z: bool = False,
                 deterministic: bool = False):
        self.in_modes = tuple(in_modes)
        self.out_modes = tuple(out_modes)
        self.ranks = tuple(ranks)
        self.dtype = dtype
        self.fill = _grad_fill(accumulate)
        # dtype of y and dx
        self.out_dtype = torch.bfloat16 if _DT[dtype] == ttc.TT_DT_E4M3 else dtype
        flags = (ttc.TT_ACCUMULATE if accumulate else 0) | \
            (ttc.TT_REUSE_MERGE if reuse_merge else 0) | (ttc.TT_REUSE_Z if reuse_z else 0) | \
            (ttc.TT_DETERMINISTIC if deterministic else 0)
        self.desc = ttc.make_desc(in_modes, out_modes, ranks, _DT[dtype], flags)
        self.plan = ttc.tt_plan(self.desc)
        self.core_off, self.diag_off, self.n_params = ttc.tt_param_layout(self.plan)
        self.N = 1
        self.M = 1
        for n in in_modes:
            self.N *= n
        for m in out_modes:
            self.M *= m

    def workspace_bytes(self, T: int) -> int:
        return ttc.tt_workspace_size(self.plan, T)

    def workspace(self, T: int, device="cuda") -> torch.Tensor:
        return torch.empty(self.workspace_bytes(T), dtype=torch.uint8, device=device)

    def forward(self, x: torch.Tensor, params: torch.Tensor, y: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        if y is None:
            y = _new((T, self.M), self.out_dtype, x.device, stream)
        if ws is None:
            ws = _scratch(stream, self.workspace, T, x.device)
        ttc.check(ttc.tt_forward(self.plan, T, _ptr(x), _ptr(params), _ptr(y), _ptr(ws),
                                 ws.numel(), _stream(stream)), "tt_forward")
        return y

    def backward(self, x: torch.Tensor, dy: torch.Tensor, params: torch.Tensor,
                 dx: Optional[torch.Tensor] = None, dparams: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, stream=None):
        T = x.shape[0]
        if dx is None:
            dx = _new((T, self.N), self.out_dtype, x.device, stream)
        if dparams is None:
            dparams = _new((self.n_params,), torch.float32, x.device, stream, self.fill)
        if ws is None:
            ws = _scratch(stream, self.workspace, T, x.device)
        ttc.check(ttc.tt_backward(self.plan, T, _ptr(x), _ptr(dy), _ptr(params), _ptr(dx),
                                  _ptr(dparams), _ptr(ws), ws.numel(), _stream(stream)),
                  "tt_backward")
        return dx, dparams


    def rank_update(self, params: torch.Tensor, dparams: torch.Tensor, gamma: float,
                    beta: float, lr: float = 0.0, stream=None) -> None:
        """In place: dparams += penalty sub-gradient (lr == 0), or one
        proximal gradient step on params (lr > 0)."""
        ttc.check(ttc.tt_rank_update(self.plan, _ptr(params), _ptr(dparams), gamma, beta, lr,
                                     _stream(stream)), "tt_rank_update")


class TTFFN:
    """y = TT_down(GELU(TT_up(x))), exact erf GELU, both layers through one plan."""

    def __init__(self, up: Sequence[Sequence[int]], down: Sequence[Sequence[int]],
                 dtype: torch.dtype = torch.bfloat16, accumulate: bool = False,
                 reuse_merge: bool = False, reuse_z: bool = False, deterministic: bool = False):
        flags = (ttc.TT_ACCUMULATE if accumulate else 0) | \
            (ttc.TT_REUSE_MERGE if reuse_merge else 0) | (ttc.TT_REUSE_Z if reuse_z else 0) | \
            (ttc.TT_DETERMINISTIC if deterministic else 0)
        self.dtype = dtype
        self.fill = _grad_fill(accumulate)
        self.up_desc = ttc.make_desc(up[0], up[1], up[2], _DT[dtype], flags)
        self.down_desc = ttc.make_desc(down[0], down[1], down[2], _DT[dtype], flags)
        self.plan = ttc.tt_ffn_plan(self.up_desc, self.down_desc)
        self.layout = [ttc.tt_ffn_param_layout(self.plan, i) for i in (0, 1)]
        self.N = 1
        self.M = 1
        for n in up[0]:
            self.N *= n
        for m in down[1]:
            self.M *= m

    def workspace(self, T: int, device="cuda") -> torch.Tensor:
        return torch.empty(ttc.tt_workspace_size(self.plan, T), dtype=torch.uint8,
                           device=device)

    def forward(self, x, p_up, p_down, y=None, ws=None, stream=None):
        T = x.shape[0]
        if y is None:
            y = _new((T, self.M), self.dtype, x.device, stream)
        if ws is None:
            ws = _scratch(stream, self.workspace, T, x.device)
        ttc.check(ttc.tt_ffn_forward(self.plan, T, _ptr(x), _ptr(p_up), _ptr(p_down), _ptr(y),
                                     _ptr(ws), ws.numel(), _stream(stream)), "tt_ffn_forward")
        return y

    def backward(self, x, dy, p_up, p_down, dx=None, dp_up=None, dp_down=None, ws=None,
                 stream=None):
        T = x.shape[0]
        if dx is None:
            dx = _new((T, self.N), self.dtype, x.device, stream)
        if dp_up is None:
            dp_up = _new((self.layout[0][2],), torch.float32, x.device, stream, self.fill)
        if dp_down is None:
            dp_down = _new((self.layout[1][2],), torch.float32, x.device, stream, self.fill)
        if ws is None:
            ws = _scratch(stream, self.workspace, T, x.device)
        ttc.check(ttc.tt_ffn_backward(self.plan, T, _ptr(x), _ptr(dy), _ptr(p_up),
                                      _ptr(p_down), _ptr(dx), _ptr(dp_up), _ptr(dp_down),
                                      _ptr(ws), ws.numel(), _stream(stream)),
                  "tt_ffn_backward")
        return dx, dp_up, dp_down


class TTMulti:
    """Up to three TT layers on one input x (the Q, K and V projections):
    y_g = x W_g^T for each layer; the backward returns dx = sum_g dy_g W_g
    and each layer's packed gradients."""

    def __init__(self, layers: Sequence[Sequence[Sequence[int]]],
                 dtype: torch.dtype = torch.bfloat16, accumulate: bool = False,
                 reuse_merge: bool = False, reuse_z: bool = False, deterministic: bool = False):
        flags = (ttc.TT_ACCUMULATE if accumulate else 0) | \
            (ttc.TT_REUSE_MERGE if reuse_merge else 0) | (ttc.TT_REUSE_Z if reuse_z else 0) | \
            (ttc.TT_DETERMINISTIC if deterministic else 0)
        self.dtype = dtype
        self.fill = _grad_fill(accumulate)
        self.out_dtype = torch.bfloat16 if _DT[dtype] == ttc.TT_DT_E4M3 else dtype
        self.descs = [ttc.make_desc(i, o, r, _DT[dtype], flags) for i, o, r in layers]
        self.plan = ttc.tt_multi_plan(self.descs)
        self.G = len(self.descs)
        self.layout = [ttc.tt_multi_param_layout(self.plan, g) for g in range(self.G)]
        self.N = 1
        for n in layers[0][0]:
            self.N *= n
        self.M = []
        for _, o, _ in layers:
            m = 1
            for v in o:
                m *= v
            self.M.append(m)

    def workspace(self, T: int, device="cuda") -> torch.Tensor:
        return torch.empty(ttc.tt_workspace_size(self.plan, T), dtype=torch.uint8,
                           device=device)

    def forward(self, x, params, y=None, ws=None, stream=None):
        T = x.shape[0]
        if y is None:
            y = [_new((T, m), self.out_dtype, x.device, stream) for m in self.M]
        if ws is None:
            ws = _scratch(stream, self.workspace, T, x.device)
        ttc.check(ttc.tt_multi_forward(self.plan, T, _ptr(x), [_ptr(p) for p in params],
                                       [_ptr(t) for t in y], _ptr(ws), ws.numel(),
                                       _stream(stream)), "tt_multi_forward")
        return y

    def backward(self, x, dy, params, dx=None, dparams=None, ws=None, stream=None):
        T = x.shape[0]
        if dx is None:
            dx = _new((T, self.N), self.out_dtype, x.device, stream)
        if dparams is None:
            dparams = [_new((lay[2],), torch.float32, x.device, stream, self.fill)
                       for lay in self.layout]
        if ws is None:
            ws = _scratch(stream, self.workspace, T, x.device)
        ttc.check(ttc.tt_multi_backward(self.plan, T, _ptr(x), [_ptr(t) for t in dy],
                                        [_ptr(p) for p in params], _ptr(dx),
                                        [_ptr(t) for t in dparams], _ptr(ws), ws.numel(),
                                        _stream(stream)), "tt_multi_backward")
        return dx, dparams


class TTMEmbedding:
    """TT-matrix embedding table: lookup of rows for int32 indices and its
    backward into the packed cores/diagonals (float32)."""

    def __init__(self, row_modes: Sequence[int], col_modes: Sequence[int],
                 ranks: Sequence[int], accumulate: bool = False, reuse: bool = False):
        # reuse: backward() takes the batch's distinct rows from the lookup()
        # of the same indices on the same workspace (TT_REUSE_MERGE)
        flags = (ttc.TT_ACCUMULATE if accumulate else 0) | (ttc.TT_REUSE_MERGE if reuse else 0)
        self.fill = _grad_fill(accumulate)
        self.desc = ttc.make_ttm_desc(row_modes, col_modes, ranks, flags)
        self.plan = ttc.tt_ttm_plan(self.desc)
        self.core_off, self.diag_off, self.n_params = ttc.tt_param_layout(self.plan)
        self.V = 1
        self.Dm = 1
        for m in row_modes:
            self.V *= m
        for n in col_modes:
            self.Dm *= n

    def workspace(self, B: int, device="cuda") -> torch.Tensor:
        return torch.empty(ttc.tt_workspace_size(self.plan, B), dtype=torch.uint8, device=device)

    def lookup(self, idx: torch.Tensor, params: torch.Tensor, out=None, ws=None, stream=None):
        B = idx.shape[0]
        if out is None:
            out = _new((B, self.Dm), torch.float32, idx.device, stream)
        if ws is None:
            ws = _scratch(stream, self.workspace, B, idx.device)
        ttc.check(ttc.tt_ttm_lookup(self.plan, B, _ptr(idx), _ptr(params), _ptr(out), _ptr(ws),
                                    ws.numel(), _stream(stream)), "tt_ttm_lookup")
        return out

    def backward(self, idx: torch.Tensor, dout: torch.Tensor, params: torch.Tensor,
                 dparams=None, ws=None, stream=None):
        B = idx.shape[0]
        if dparams is None:
            dparams = _new((self.n_params,), torch.float32, idx.device, stream, self.fill)
        if ws is None:
            ws = _scratch(stream, self.workspace, B, idx.device)
        ttc.check(ttc.tt_ttm_lookup_backward(self.plan, B, _ptr(idx), _ptr(dout), _ptr(params),
                                             _ptr(dparams), _ptr(ws), ws.numel(),
                                             _stream(stream)), "tt_ttm_lookup_backward")
        return dparams

    def stats(self, ws: torch.Tensor, stream=None):
        """(distinct rows, distinct (i_1, i_2) prefixes) of the last call on ws."""
        return ttc.tt_ttm_stats(self.plan, _ptr(ws), _stream(stream))


def _dense(t: Optional[torch.Tensor], shape, dtype: torch.dtype, name: str) -> int:
    """Pointer of a dense CUDA tensor of the given shape and type (0 for None)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of shape {shape} and "
                         f"{dtype}, got {tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


class TTNorm:
    """Layer normalisation of (T, N) rows with an optional residual sum in
    front of it: s = x + res, y = (s - mean(s)) / sqrt(var(s) + eps) gamma + beta."""

    def __init__(self, N: int, dtype: torch.dtype = torch.bfloat16, eps: float = 1e-5,
                 accumulate: bool = False):
        self.N = int(N)
        self.dtype = dtype
        self.fill = _grad_fill(accumulate)
        self.plan = ttc.tt_norm_plan(N, eps, _DT[dtype], ttc.TT_ACCUMULATE if accumulate else 0)

    def workspace(self, T: int, device="cuda") -> torch.Tensor:
        return torch.empty(ttc.tt_workspace_size(self.plan, T), dtype=torch.uint8, device=device)

    def forward(self, x, gamma=None, beta=None, res=None, y=None, sum=None, stats=None,
                stream=None):
        """(y, s, stats): s is None without a residual (it would be x), stats
        holds each row's mean and 1 / sqrt(var + eps) for the backward."""
        T, N = x.shape[0], self.N
        if y is None:
            y = _new((T, N), self.dtype, x.device, stream)
        if res is not None and sum is None:
            sum = _new((T, N), self.dtype, x.device, stream)
        if stats is None:
            stats = _new((T, 2), torch.float32, x.device, stream)
        f32, sh = torch.float32, (T, N)
        ttc.check(ttc.tt_norm_forward(
            self.plan, T, _dense(x, sh, self.dtype, "x"), _dense(res, sh, self.dtype, "res"),
            _dense(gamma, (N,), f32, "gamma"), _dense(beta, (N,), f32, "beta"),
            _dense(sum, sh, self.dtype, "sum"), _dense(y, sh, self.dtype, "y"),
            _dense(stats, (T, 2), f32, "stats"), _stream(stream)), "tt_norm_forward")
        return y, sum, stats

    def backward(self, s, dy, gamma, stats, dsum=None, dx=None, dgamma=None, dbeta=None, ws=None,
                 stream=None):
        """(dx, dgamma, dbeta); dx is the gradient of x and of res.  dsum is
        the gradient that reaches s along the residual path."""
        T, N = s.shape[0], self.N
        if dx is None:
            dx = _new((T, N), self.dtype, s.device, stream)
        if dgamma is None:
            dgamma = _new((N,), torch.float32, s.device, stream, self.fill)
        if dbeta is None:
            dbeta = _new((N,), torch.float32, s.device, stream, self.fill)
        if ws is None:
            ws = _scratch(stream, self.workspace, T, s.device)
        f32, sh = torch.float32, (T, N)
        ttc.check(ttc.tt_norm_backward(
            self.plan, T, _dense(s, sh, self.dtype, "s"), _dense(dy, sh, self.dtype, "dy"),
            _dense(dsum, sh, self.dtype, "dsum"), _dense(gamma, (N,), f32, "gamma"),
            _dense(stats, (T, 2), f32, "stats"), _dense(dx, sh, self.dtype, "dx"),
            _dense(dgamma, (N,), f32, "dgamma"), _dense(dbeta, (N,), f32, "dbeta"), _ptr(ws),
            ws.numel(), _stream(stream)), "tt_norm_backward")
        return dx, dgamma, dbeta


class TTSeqs:
    """The sequences of a batch: int32 device arrays of first and past-the-end
    rows of each one's queries and keys, the buffers' row counts and bounds on
    a sequence's lengths.  Keeps the arrays alive.  gaps: rows of the buffers may
    belong to no sequence (a cache's unused ones).  The kernels leave those rows of
    their outputs as they are; outputs that TTAttention makes hold zeros there (and
    lse -infinity).  With gaps=False, for sequences that cover every row, it does not
    fill them first."""

    def __init__(self, q_begin, q_end, k_begin, k_end, Tq: int, Tk: int, max_q: int, max_k: int,
                 gaps: bool = True):
        B = q_begin.shape[0]
        self.arrays = (q_begin, q_end, k_begin, k_end)
        for t in self.arrays:
            _dense(t, (B,), torch.int32, "sequence rows")
        self.Tq, self.Tk = int(Tq), int(Tk)
        self.gaps = bool(gaps)
        self.c = ttc.tt_attn_seqs(B, int(max_q), int(max_k), self.Tq, self.Tk,
                                  *(t.data_ptr() for t in self.arrays))

    @classmethod
    def packed(cls, offsets: torch.Tensor, T: int, max_len: int) -> "TTSeqs":
        """Self-attention over sequences packed one after another: sequence b
        is rows offsets[b] .. offsets[b + 1] of T, from row 0 to row T without a gap."""
        return cls(offsets[:-1], offsets[1:], offsets[:-1], offsets[1:], T, T, max_len, max_len,
                   gaps=False)


class TTAttention:
    """Attention between the Q, K, V projections and O: query i sees key j
    when j <= i + right (right >= 0) and j >= i - left (left >= 0) or j < sinks;
    kv_heads key heads are shared by heads / kv_heads query heads each."""

    def __init__(self, heads: int, dim: int, kv_heads: Optional[int] = None,
                 dtype: torch.dtype = torch.bfloat16, left: int = -1, right: int = -1,
                 sinks: int = 0, scale: float = 0.0):
        self.heads, self.dim = int(heads), int(dim)
        self.kv_heads = self.heads if kv_heads is None else int(kv_heads)
        self.dtype = dtype
        self.plan = ttc.tt_attn_plan(heads, self.kv_heads, dim, left, right, sinks, scale,
                                     _DT[dtype])

    def workspace(self, seqs: TTSeqs, backward: bool = True, device="cuda") -> torch.Tensor:
        """Enough for a forward of seqs and, unless backward is False, for a backward
        (either can be the larger: a few tokens against a long cache need theirs for
        the forward)."""
        n = ttc.tt_attn_workspace_size(self.plan, seqs.c, False)
        if backward:
            n = max(n, ttc.tt_attn_workspace_size(self.plan, seqs.c, True))
        return torch.empty(n, dtype=torch.uint8, device=device)

    def _heads(self, t: torch.Tensor, rows: int, heads: int, name: str) -> ttc.tt_heads:
        """(rows, heads, dim) of any row and head stride, or (rows, heads * dim)."""
        shape, st = t.shape, t.stride()
        if t.dtype == self.dtype and t.is_cuda and shape[0] == rows:
            if len(shape) == 3 and shape[1] == heads and shape[2] == self.dim and \
                    (st[2] == 1 or self.dim == 1):
                return ttc.tt_heads(t.data_ptr(), st[0], st[1])
            if len(shape) == 2 and shape[1] == heads * self.dim and \
                    (st[1] == 1 or shape[1] == 1):
                return ttc.tt_heads(t.data_ptr(), st[0], self.dim)
        raise ValueError(f"{name}: expected a CUDA tensor of ({rows}, {heads}, {self.dim}) "
                         f"{self.dtype} with its last axis dense, got {tuple(shape)} {t.dtype} "
                         f"on {t.device}, strides {tuple(st)}")

    def forward(self, q, k, v, seqs: TTSeqs, o=None, lse=None, ws=None, stream=None):
        """(o, lse); o like q but dense, lse (heads, Tq) fp32.  Rows of no sequence stay
        as they are in tensors that the caller gives."""
        if o is None:
            o = _new(q.shape, self.dtype, q.device, stream, 0.0 if seqs.gaps else None)
        if lse is None:
            lse = _new((self.heads, seqs.Tq), torch.float32, q.device, stream,
                       -math.inf if seqs.gaps else None)
        if ws is None:
            ws = _scratch(stream, self.workspace, seqs, False, q.device)
        H, G = self.heads, self.kv_heads
        ttc.check(ttc.tt_attn_forward(
            self.plan, seqs.c, self._heads(q, seqs.Tq, H, "q"), self._heads(k, seqs.Tk, G, "k"),
            self._heads(v, seqs.Tk, G, "v"), self._heads(o, seqs.Tq, H, "o"),
            _dense(lse, (H, seqs.Tq), torch.float32, "lse"), _ptr(ws), ws.numel(),
            _stream(stream)), "tt_attn_forward")
        return o, lse

    def backward(self, q, k, v, o, lse, do, seqs: TTSeqs, dq=None, dk=None, dv=None, ws=None,
                 stream=None):
        """(dq, dk, dv) for the gradient do of o.  Rows of no sequence stay as they are
        in tensors that the caller gives."""
        fill = 0.0 if seqs.gaps else None
        if dq is None:
            dq = _new(q.shape, self.dtype, q.device, stream, fill)
        if dk is None:
            dk = _new(k.shape, self.dtype, q.device, stream, fill)
        if dv is None:
            dv = _new(v.shape, self.dtype, q.device, stream, fill)
        if ws is None:
            ws = _scratch(stream, self.workspace, seqs, True, q.device)
        H, G = self.heads, self.kv_heads
        ttc.check(ttc.tt_attn_backward(
            self.plan, seqs.c, self._heads(q, seqs.Tq, H, "q"), self._heads(k, seqs.Tk, G, "k"),
            self._heads(v, seqs.Tk, G, "v"), self._heads(o, seqs.Tq, H, "o"),
            _dense(lse, (H, seqs.Tq), torch.float32, "lse"),
            self._heads(do, seqs.Tq, H, "do"), self._heads(dq, seqs.Tq, H, "dq"),
            self._heads(dk, seqs.Tk, G, "dk"), self._heads(dv, seqs.Tk, G, "dv"), _ptr(ws),
            ws.numel(), _stream(stream)), "tt_attn_backward")
        return dq, dk, dv
