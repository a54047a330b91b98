"""The TT layers of one transformer encoder block as one step.

The CoMERA project page tensorises every linear layer of its encoder blocks
(the attention projections Q, K, V, O and the feed-forward pair) and runs the
whole training step as one CUDA graph to remove launch overhead ("Making small
tensor operations fast on GPUs", bullet "CUDA Graph": 14.3 -> 7.2 minutes an
epoch).  This module composes the library's calls for one block: the forward
of Q, K, V (on the same x: one multi-layer plan, whose kernels stream x once
for all three), O and the FFN pair, then their backward in reverse order, all
on one stream so that a CUDA graph captures the block with the
programmatic-launch edges between consecutive kernels.  The backward of Q, K
and V returns their summed input gradient dx_q + dx_k + dx_v, which is what
the block's x receives.  The attention between
the projections is not a TT layer and is not part of this step.
TTTransformerBlock is the whole block: the same layers with the normalisations,
residual sums and attention between them, its training step, and the step of
single tokens against a cache of keys and values.

Argument marshalling only: every product runs in libttc's kernels.
"""

from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from . import synth, ttc
from .layer import TTAttention, TTFFN, TTLinear, TTMulti, TTNorm, TTSeqs

PROJ = ("q", "k", "v", "o")
QKV = ("q", "k", "v")


class TTEncoderBlock:
    """Q, K, V, O (768 x 768) and the GELU FFN pair (768 -> 3072 -> 768), each
    a rank-30 TT layer, bf16 activations; the backward of every layer reuses
    its forward's merges and kept z' (TT_REUSE_Z)."""

    def __init__(self, reuse_z: bool = True, deterministic: bool = False,
                 fuse_qkv: bool = True):
        L = synth.ENCODER_LAYERS
        self.fuse_qkv = fuse_qkv
        single = ("o",) if fuse_qkv else PROJ
        self.proj = {nm: TTLinear(L[nm].in_modes, L[nm].out_modes, L[nm].ranks, torch.bfloat16,
                                  reuse_z=reuse_z, deterministic=deterministic) for nm in single}
        self.qkv = TTMulti([(L[nm].in_modes, L[nm].out_modes, L[nm].ranks) for nm in QKV],
                           torch.bfloat16, reuse_z=reuse_z,
                           deterministic=deterministic) if fuse_qkv else None
        up, dn = L["up"], L["down"]
        self.ffn = TTFFN((up.in_modes, up.out_modes, up.ranks),
                         (dn.in_modes, dn.out_modes, dn.ranks), torch.bfloat16,
                         reuse_z=reuse_z, deterministic=deterministic)

    def buffers(self, T: int, device="cuda") -> Dict[str, torch.Tensor]:
        """Workspaces, outputs and gradients of one step (allocated once)."""
        b = {}
        if self.fuse_qkv:
            b["ws_qkv"] = self.qkv.workspace(T, device)
            b["dx_qkv"] = torch.empty((T, self.qkv.N), dtype=torch.bfloat16, device=device)
            for g, nm in enumerate(QKV):
                b[f"y_{nm}"] = torch.empty((T, self.qkv.M[g]), dtype=torch.bfloat16,
                                           device=device)
                b[f"dp_{nm}"] = torch.empty(self.qkv.layout[g][2], dtype=torch.float32,
                                            device=device)
        for nm in self.proj:
            lay = self.proj[nm]
            b[f"ws_{nm}"] = lay.workspace(T, device)
            b[f"y_{nm}"] = torch.empty((T, lay.M), dtype=torch.bfloat16, device=device)
            b[f"dx_{nm}"] = torch.empty((T, lay.N), dtype=torch.bfloat16, device=device)
            b[f"dp_{nm}"] = torch.empty(lay.n_params, dtype=torch.float32, device=device)
        b["ws_ffn"] = self.ffn.workspace(T, device)
        b["y_ffn"] = torch.empty((T, self.ffn.M), dtype=torch.bfloat16, device=device)
        b["dx_ffn"] = torch.empty((T, self.ffn.N), dtype=torch.bfloat16, device=device)
        b["dp_up"] = torch.empty(self.ffn.layout[0][2], dtype=torch.float32, device=device)
        b["dp_down"] = torch.empty(self.ffn.layout[1][2], dtype=torch.float32, device=device)
        return b

    def step(self, x, xo, xf, dy: Dict[str, torch.Tensor], params: Dict[str, torch.Tensor],
             b: Dict[str, torch.Tensor], stream=None) -> None:
        """Forward of Q, K, V, O and the FFN pair, then the backward in reverse
        order; outputs in b (y_* and dp_* per layer, dx_* per input: dx_qkv
        for the fused Q, K, V)."""
        xin = {"q": x, "k": x, "v": x, "o": xo}
        if self.fuse_qkv:
            self.qkv.forward(x, [params[nm] for nm in QKV], y=[b[f"y_{nm}"] for nm in QKV],
                             ws=b["ws_qkv"], stream=stream)
        for nm in self.proj:
            self.proj[nm].forward(xin[nm], params[nm], y=b[f"y_{nm}"], ws=b[f"ws_{nm}"],
                                  stream=stream)
        self.ffn.forward(xf, params["up"], params["down"], y=b["y_ffn"], ws=b["ws_ffn"],
                         stream=stream)
        self.ffn.backward(xf, dy["ffn"], params["up"], params["down"], dx=b["dx_ffn"],
                          dp_up=b["dp_up"], dp_down=b["dp_down"], ws=b["ws_ffn"], stream=stream)
        for nm in reversed(list(self.proj)):
            self.proj[nm].backward(xin[nm], dy[nm], params[nm], dx=b[f"dx_{nm}"],
                                   dparams=b[f"dp_{nm}"], ws=b[f"ws_{nm}"], stream=stream)
        if self.fuse_qkv:
            self.qkv.backward(x, [dy[nm] for nm in QKV], [params[nm] for nm in QKV],
                              dx=b["dx_qkv"], dparams=[b[f"dp_{nm}"] for nm in QKV],
                              ws=b["ws_qkv"], stream=stream)

    def capture(self, T, x, xo, xf, dy, params, b) -> torch.cuda.CUDAGraph:
        """The step as one CUDA graph (replay() runs the whole block)."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step(x, xo, xf, dy, params, b)  # on the capture stream
        return g


class TTTransformerBlock(TTEncoderBlock):
    """The whole pre-norm block on a residual stream kept as a sum of two parts,
    so that each residual sum is one with the normalisation that reads it:

        s1 = x + res             h1 = norm(s1; g1, b1)
        a  = O(attention(Q h1, K h1, V h1))
        s2 = a + s1              h2 = norm(s2; g2, b2)
        out = (FFN(h2), s2)      the next block's (x, res)

    Sequences are packed (TTSeqs); the window and the first tokens that stay
    visible are those of TTAttention.  params holds the six layers' packed
    parameters and the fp32 norm weights g1, b1, g2, b2; their gradients are
    b["dp_*"] and b["dg1"], b["db1"], b["dg2"], b["db2"]."""

    def __init__(self, heads: int = 12, left: int = -1, right: int = -1, sinks: int = 0,
                 eps: float = 1e-5, reuse_z: bool = True, deterministic: bool = False):
        super().__init__(reuse_z, deterministic)
        self.N = self.qkv.N
        self.norm = TTNorm(self.N, torch.bfloat16, eps)
        self.attn = TTAttention(heads, self.N // heads, left=left, right=right, sinks=sinks)

    def buffers(self, T: int, seqs: TTSeqs, device="cuda") -> Dict[str, torch.Tensor]:
        """Everything a step of T tokens of seqs writes (allocated once): a training
        step, or decode's."""
        b = super().buffers(T, device)
        for nm in ("s1", "h1", "s2", "h2", "att", "datt", "dq", "dk", "dv", "ds1", "ds2"):
            b[nm] = torch.empty((T, self.N), dtype=torch.bfloat16, device=device)
        for nm in ("st1", "st2"):
            b[nm] = torch.empty((T, 2), dtype=torch.float32, device=device)
        for nm in ("dg1", "db1", "dg2", "db2"):
            b[nm] = torch.empty(self.N, dtype=torch.float32, device=device)
        b["lse"] = torch.empty((self.attn.heads, T), dtype=torch.float32, device=device)
        b["ws_attn"] = self.attn.workspace(seqs, True, device)
        b["ws_norm"] = self.norm.workspace(T, device)
        return b

    def _project(self, x, res, params, b, stream) -> None:
        """s1, h1 and the projections Q, K, V of h1."""
        self.norm.forward(x, params["g1"], params["b1"], res, y=b["h1"],
                          sum=None if res is None else b["s1"], stats=b["st1"], stream=stream)
        self.qkv.forward(b["h1"], [params[nm] for nm in QKV], y=[b[f"y_{nm}"] for nm in QKV],
                         ws=b["ws_qkv"], stream=stream)

    def _finish(self, s1, params, b, stream) -> Tuple[torch.Tensor, torch.Tensor]:
        """From the attention's output to the block's (FFN output, s2)."""
        self.proj["o"].forward(b["att"], params["o"], y=b["y_o"], ws=b["ws_o"], stream=stream)
        self.norm.forward(b["y_o"], params["g2"], params["b2"], s1, y=b["h2"], sum=b["s2"],
                          stats=b["st2"], stream=stream)
        self.ffn.forward(b["h2"], params["up"], params["down"], y=b["y_ffn"], ws=b["ws_ffn"],
                         stream=stream)
        return b["y_ffn"], b["s2"]

    def forward(self, x, res: Optional[torch.Tensor], seqs: TTSeqs,
                params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor], stream=None):
        """(FFN output, s2); res is None for the first block."""
        self._project(x, res, params, b, stream)
        self.attn.forward(b["y_q"], b["y_k"], b["y_v"], seqs, o=b["att"], lse=b["lse"],
                          ws=b["ws_attn"], stream=stream)
        return self._finish(x if res is None else b["s1"], params, b, stream)

    def backward(self, x, res: Optional[torch.Tensor], dffn, ds2: Optional[torch.Tensor],
                 seqs: TTSeqs, params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor],
                 stream=None) -> torch.Tensor:
        """The gradient of x and of res, for dffn and ds2, those of forward's
        outputs (ds2 None where nothing reads s2)."""
        self.ffn.backward(b["h2"], dffn, params["up"], params["down"], dx=b["dx_ffn"],
                          dp_up=b["dp_up"], dp_down=b["dp_down"], ws=b["ws_ffn"], stream=stream)
        self.norm.backward(b["s2"], b["dx_ffn"], params["g2"], b["st2"], ds2, dx=b["ds2"],
                           dgamma=b["dg2"], dbeta=b["db2"], ws=b["ws_norm"], stream=stream)
        self.proj["o"].backward(b["att"], b["ds2"], params["o"], dx=b["datt"],
                                dparams=b["dp_o"], ws=b["ws_o"], stream=stream)
        self.attn.backward(b["y_q"], b["y_k"], b["y_v"], b["att"], b["lse"], b["datt"], seqs,
                           dq=b["dq"], dk=b["dk"], dv=b["dv"], ws=b["ws_attn"], stream=stream)
        self.qkv.backward(b["h1"], [b["dq"], b["dk"], b["dv"]], [params[nm] for nm in QKV],
                          dx=b["dx_qkv"], dparams=[b[f"dp_{nm}"] for nm in QKV],
                          ws=b["ws_qkv"], stream=stream)
        self.norm.backward(x if res is None else b["s1"], b["dx_qkv"], params["g1"], b["st1"],
                           b["ds2"], dx=b["ds1"], dgamma=b["dg1"], dbeta=b["db1"],
                           ws=b["ws_norm"], stream=stream)
        return b["ds1"]

    def step(self, x, res: Optional[torch.Tensor], dffn, ds2: Optional[torch.Tensor],
             seqs: TTSeqs, params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor],
             stream=None) -> None:
        """A training step: forward, then backward for the gradients dffn and ds2 of its
        outputs; everything in b (y_ffn and s2, ds1, dp_*, dg1, db1, dg2, db2)."""
        self.forward(x, res, seqs, params, b, stream)
        self.backward(x, res, dffn, ds2, seqs, params, b, stream)

    def capture(self, x, res: Optional[torch.Tensor], dffn, ds2: Optional[torch.Tensor],
                seqs: TTSeqs, params: Dict[str, torch.Tensor],
                b: Dict[str, torch.Tensor]) -> torch.cuda.CUDAGraph:
        """The training step as one CUDA graph (replay() runs the whole block)."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step(x, res, dffn, ds2, seqs, params, b)  # on the capture stream
        return g

    def decode(self, x, res: Optional[torch.Tensor], keys, values, rows, seqs: TTSeqs,
               params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor], stream=None):
        """forward for a few new tokens: their keys and values go to `rows` (int64)
        of the caches keys and values (rows, heads, dim), which seqs names as the
        sequences' keys; (FFN output, s2)."""
        self._project(x, res, params, b, stream)
        shape = (-1, self.attn.kv_heads, self.attn.dim)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            keys.index_copy_(0, rows, b["y_k"].view(shape))
            values.index_copy_(0, rows, b["y_v"].view(shape))
        self.attn.forward(b["y_q"], keys, values, seqs, o=b["att"], lse=b["lse"],
                          ws=b["ws_attn"], stream=stream)
        return self._finish(x if res is None else b["s1"], params, b, stream)
