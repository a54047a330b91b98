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
residual sums and attention between them (with positions and dropout where they are
asked for), its training step, and the step of single tokens against a cache of keys
and values.  TTTokenHead is what follows the last block: the output layer, the log
probabilities of tokens and their loss.

Argument marshalling only: every product runs in libttc's kernels.
"""

from __future__ import annotations

from typing import Dict, Optional, Sequence, Tuple, Union

import torch

from . import synth, ttc
from .layer import (TTAttention, TTDropNorm, TTFFN, TTLinear, TTLogProbs, TTMulti, TTNorm,
                    TTRotary, TTSeqs, _filled)

PROJ = ("q", "k", "v", "o")
QKV = ("q", "k", "v")


def _drop_norms(N: int, p: float, eps: float, site: Optional[int], places: int):
    """The dropouts of a part of a model, at sites from `site` on; None for p = 0."""
    if not 0 <= p <= 1:
        raise ValueError(f"dropout: expected 0 to 1, got {p}")
    if p == 0:
        return None
    if site is None:
        raise ValueError("site: parts with dropout need sites of their own (two at the same one "
                         "drop the same elements)")
    return [TTDropNorm(N, p, torch.bfloat16, eps, site + i) for i in range(places)]


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
    b["dp_*"] and b["dg1"], b["db1"], b["dg2"], b["db2"].

    rotary: Q h1 and K h1 pass through it in front of the attention, at the tokens'
    positions pos (int32; None: their rows, which serves packed sequences as well, where
    the distances alone count).  With a norm, params may hold its weights gq, gk, whose
    gradients are b["dgq"], b["dgk"] (of a rotary with accumulate the sums over the steps,
    from zeros on).
    dropout: of x and of a in front of their sums, in a pass that is given the state rng
    (TTDropout.state; None: nothing is dropped).  The block takes the sites `site` and
    `site` + 1, which nothing else in the model may have: with dropout, site has to be
    given."""

    def __init__(self, heads: int = 12, left: int = -1, right: int = -1, sinks: int = 0,
                 eps: float = 1e-5, reuse_z: bool = True, deterministic: bool = False,
                 rotary: Optional[TTRotary] = None, dropout: float = 0.0,
                 site: Optional[int] = None):
        super().__init__(reuse_z, deterministic)
        self.N = self.qkv.N
        self.norm = TTNorm(self.N, torch.bfloat16, eps)
        self.attn = TTAttention(heads, self.N // heads, left=left, right=right, sinks=sinks)
        if rotary is not None and (rotary.heads, rotary.kv_heads, rotary.dim, rotary.dtype) != \
                (heads, heads, self.attn.dim, torch.bfloat16):
            raise ValueError(f"rotary: expected {heads} heads of {self.attn.dim} for q and k in "
                             f"bfloat16")
        self.rotary = rotary
        self.drops = _drop_norms(self.N, dropout, eps, site, 2)

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
        if self.rotary is not None:
            for nm in ("rq", "rk"):
                b[nm] = torch.empty((T, self.N), dtype=torch.bfloat16, device=device)
            if self.rotary.norm:
                for nm in ("dgq", "dgk"):  # zeros where the rotary adds to them
                    b[nm] = _filled((self.attn.dim,), torch.float32, device, self.rotary.fill)
            b["ws_rope"] = self.rotary.workspace(T, device)
        if self.drops is not None:
            for nm in ("dx", "da"):
                b[nm] = torch.empty((T, self.N), dtype=torch.bfloat16, device=device)
        b["lse"] = torch.empty((self.attn.heads, T), dtype=torch.float32, device=device)
        b["ws_attn"] = self.attn.workspace(seqs, True, device)
        b["ws_norm"] = self.norm.workspace(T, device)
        return b

    def _dropping(self, rng) -> bool:
        if rng is not None and self.drops is None:
            raise ValueError("rng: this block has no dropout")
        return rng is not None

    def _project(self, x, res, params, b, stream, rng=None) -> torch.Tensor:
        """s1, h1 and the projections Q, K, V of h1; returns s1."""
        if self._dropping(rng):
            self.drops[0].forward(x, rng, params["g1"], params["b1"], res, y=b["h1"],
                                  sum=b["s1"], stats=b["st1"], stream=stream)
        else:
            self.norm.forward(x, params["g1"], params["b1"], res, y=b["h1"],
                              sum=None if res is None else b["s1"], stats=b["st1"],
                              stream=stream)
        self.qkv.forward(b["h1"], [params[nm] for nm in QKV], y=[b[f"y_{nm}"] for nm in QKV],
                         ws=b["ws_qkv"], stream=stream)
        return x if res is None and rng is None else b["s1"]

    def _finish(self, s1, params, b, stream, rng=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """From the attention's output to the block's (FFN output, s2)."""
        self.proj["o"].forward(b["att"], params["o"], y=b["y_o"], ws=b["ws_o"], stream=stream)
        if rng is not None:
            self.drops[1].forward(b["y_o"], rng, params["g2"], params["b2"], s1, y=b["h2"],
                                  sum=b["s2"], stats=b["st2"], stream=stream)
        else:
            self.norm.forward(b["y_o"], params["g2"], params["b2"], s1, y=b["h2"], sum=b["s2"],
                              stats=b["st2"], stream=stream)
        self.ffn.forward(b["h2"], params["up"], params["down"], y=b["y_ffn"], ws=b["ws_ffn"],
                         stream=stream)
        return b["y_ffn"], b["s2"]

    def _turned(self, b) -> Tuple[torch.Tensor, torch.Tensor]:
        """The attention's queries and keys."""
        return (b["y_q"], b["y_k"]) if self.rotary is None else (b["rq"], b["rk"])

    def forward(self, x, res: Optional[torch.Tensor], seqs: TTSeqs,
                params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor], stream=None,
                pos: Optional[torch.Tensor] = None, rng: Optional[torch.Tensor] = None):
        """(FFN output, s2); res is None for the first block."""
        s1 = self._project(x, res, params, b, stream, rng)
        if self.rotary is not None:
            self.rotary.forward(b["y_q"], b["y_k"], pos, params.get("gq"), params.get("gk"),
                                q_out=b["rq"], k_out=b["rk"], stream=stream)
        q, k = self._turned(b)
        self.attn.forward(q, k, b["y_v"], seqs, o=b["att"], lse=b["lse"], ws=b["ws_attn"],
                          stream=stream)
        return self._finish(s1, params, b, stream, rng)

    def backward(self, x, res: Optional[torch.Tensor], dffn, ds2: Optional[torch.Tensor],
                 seqs: TTSeqs, params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor],
                 stream=None, pos: Optional[torch.Tensor] = None,
                 rng: Optional[torch.Tensor] = None) \
            -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
        """The gradient of x and of res, for dffn and ds2, those of forward's
        outputs (ds2 None where nothing reads s2).  With rng (forward's) the two differ:
        (that of x, that of res)."""
        dropping = self._dropping(rng)
        self.ffn.backward(b["h2"], dffn, params["up"], params["down"], dx=b["dx_ffn"],
                          dp_up=b["dp_up"], dp_down=b["dp_down"], ws=b["ws_ffn"], stream=stream)
        if dropping:
            self.drops[1].backward(b["s2"], b["dx_ffn"], rng, params["g2"], b["st2"], ds2,
                                   dx=b["da"], dres=b["ds2"], dgamma=b["dg2"], dbeta=b["db2"],
                                   ws=b["ws_norm"], stream=stream)
        else:
            self.norm.backward(b["s2"], b["dx_ffn"], params["g2"], b["st2"], ds2, dx=b["ds2"],
                               dgamma=b["dg2"], dbeta=b["db2"], ws=b["ws_norm"], stream=stream)
        self.proj["o"].backward(b["att"], b["da"] if dropping else b["ds2"], params["o"],
                                dx=b["datt"], dparams=b["dp_o"], ws=b["ws_o"], stream=stream)
        q, k = self._turned(b)
        self.attn.backward(q, k, b["y_v"], b["att"], b["lse"], b["datt"], seqs, dq=b["dq"],
                           dk=b["dk"], dv=b["dv"], ws=b["ws_attn"], stream=stream)
        if self.rotary is not None:  # in place: dq and dk become those of Q h1 and K h1
            norm = self.rotary.norm
            self.rotary.backward(b["dq"], b["dk"], pos, b["y_q"] if norm else None,
                                 b["y_k"] if norm else None, params.get("gq"), params.get("gk"),
                                 dq_in=b["dq"], dk_in=b["dk"], dgq=b.get("dgq"),
                                 dgk=b.get("dgk"), ws=b["ws_rope"], stream=stream)
        self.qkv.backward(b["h1"], [b["dq"], b["dk"], b["dv"]], [params[nm] for nm in QKV],
                          dx=b["dx_qkv"], dparams=[b[f"dp_{nm}"] for nm in QKV],
                          ws=b["ws_qkv"], stream=stream)
        if dropping:
            self.drops[0].backward(b["s1"], b["dx_qkv"], rng, params["g1"], b["st1"], b["ds2"],
                                   dx=b["dx"], dres=b["ds1"], dgamma=b["dg1"], dbeta=b["db1"],
                                   ws=b["ws_norm"], stream=stream)
            return b["dx"], b["ds1"]
        self.norm.backward(x if res is None else b["s1"], b["dx_qkv"], params["g1"], b["st1"],
                           b["ds2"], dx=b["ds1"], dgamma=b["dg1"], dbeta=b["db1"],
                           ws=b["ws_norm"], stream=stream)
        return b["ds1"]

    def step(self, x, res: Optional[torch.Tensor], dffn, ds2: Optional[torch.Tensor],
             seqs: TTSeqs, params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor],
             stream=None, pos: Optional[torch.Tensor] = None,
             rng: Optional[torch.Tensor] = None) -> None:
        """A training step: forward, then backward for the gradients dffn and ds2 of its
        outputs; everything in b (y_ffn and s2, ds1, with dropout dx, dp_*, dg1, db1, dg2,
        db2)."""
        self.forward(x, res, seqs, params, b, stream, pos, rng)
        self.backward(x, res, dffn, ds2, seqs, params, b, stream, pos, rng)

    def capture(self, x, res: Optional[torch.Tensor], dffn, ds2: Optional[torch.Tensor],
                seqs: TTSeqs, params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor],
                pos: Optional[torch.Tensor] = None,
                rng: Optional[torch.Tensor] = None) -> torch.cuda.CUDAGraph:
        """The training step as one CUDA graph (replay() runs the whole block)."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step(x, res, dffn, ds2, seqs, params, b, pos=pos, rng=rng)  # capture stream
        return g

    def decode(self, x, res: Optional[torch.Tensor], keys, values, rows, seqs: TTSeqs,
               params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor], stream=None,
               pos: Optional[torch.Tensor] = None):
        """forward for a few new tokens: their keys and values go to `rows` (int64, or
        int32 with a rotary) of the caches keys and values (rows, heads, dim), which seqs
        names as the sequences' keys; (FFN output, s2).  With a rotary pos (int32) is
        the tokens' positions, as the cached keys had them, and rows of int64 are converted
        in each call."""
        s1 = self._project(x, res, params, b, stream)
        shape = (-1, self.attn.kv_heads, self.attn.dim)
        here = stream if stream is not None else torch.cuda.current_stream()
        if self.rotary is not None:
            if pos is None:
                raise ValueError("pos: a cache needs the tokens' positions")
            with torch.cuda.stream(here):
                rows = rows.to(torch.int32)
            self.rotary.to_cache(b["y_q"], b["y_k"], b["y_v"], pos, rows, keys, values,
                                 params.get("gq"), params.get("gk"), q_out=b["rq"],
                                 stream=stream)
        else:
            with torch.cuda.stream(here):
                keys.index_copy_(0, rows, b["y_k"].view(shape))
                values.index_copy_(0, rows, b["y_v"].view(shape))
        self.attn.forward(self._turned(b)[0], keys, values, seqs, o=b["att"], lse=b["lse"],
                          ws=b["ws_attn"], stream=stream)
        return self._finish(s1, params, b, stream)


class TTTokenHead:
    """What follows the last block's (x, res):

        s = dropout(x) + res    h = norm(s; gf, bf)    logits = W h
        logp, lse (and the entropy) of each token's target, and the top alternatives

    with W a TT layer of N inputs and at least `vocab` outputs (a product of modes; the
    ones behind `vocab` are not read).  params holds the packed parameters "head" and the
    fp32 weights gf, bf; their gradients are b["dp_head"], b["dgf"], b["dbf"].  dropout
    and rng as in TTTransformerBlock."""

    def __init__(self, in_modes: Sequence[int], out_modes: Sequence[int], ranks: Sequence[int],
                 vocab: Optional[int] = None, eps: float = 1e-5, scale: float = 1.0,
                 top: int = 0, dropout: float = 0.0, site: Optional[int] = None,
                 reuse_z: bool = True, deterministic: bool = False):
        self.linear = TTLinear(in_modes, out_modes, ranks, torch.bfloat16, reuse_z=reuse_z,
                               deterministic=deterministic)
        self.N, self.M = self.linear.N, self.linear.M
        self.vocab = self.M if vocab is None else int(vocab)
        if not 1 <= self.vocab <= self.M:
            raise ValueError(f"vocab: expected 1 to {self.M}, got {vocab}")
        self.norm = TTNorm(self.N, torch.bfloat16, eps)
        drops = _drop_norms(self.N, dropout, eps, site, 1)
        self.drop = drops[0] if drops else None
        self.probs = TTLogProbs(self.vocab, torch.bfloat16, scale, top)

    def buffers(self, T: int, device="cuda") -> Dict[str, torch.Tensor]:
        """Everything that T tokens write (allocated once).  The gradient of the logits
        takes their place, unless outputs behind `vocab` have to have zeros."""
        bf = lambda n: torch.empty((T, n), dtype=torch.bfloat16, device=device)  # noqa: E731
        f32 = lambda *n: torch.empty(n, dtype=torch.float32, device=device)  # noqa: E731
        b = {nm: bf(self.N) for nm in ("s", "h", "dh", "ds")}
        b["logits"] = bf(self.M)
        b["dlogits"] = b["logits"] if self.vocab == self.M else bf(self.M).zero_()
        b["st"] = f32(T, 2)
        b.update({nm: f32(T) for nm in ("logp", "lse", "entropy")})
        if self.probs.top:
            b["top"] = torch.empty((T, self.probs.top), dtype=torch.int32, device=device)
            b["top_logp"] = f32(T, self.probs.top)
        if self.drop is not None:
            b["dx"] = bf(self.N)
        b.update({nm: f32(self.N) for nm in ("dgf", "dbf")})
        b["dp_head"] = f32(self.linear.n_params)
        b["ws_head"] = self.linear.workspace(T, device)
        b["ws_norm"] = self.norm.workspace(T, device)
        return b

    def _logits(self, x, res, params, b, stream, rng) -> None:
        if rng is not None and self.drop is None:
            raise ValueError("rng: this head has no dropout")
        if rng is not None:
            self.drop.forward(x, rng, params["gf"], params["bf"], res, y=b["h"], sum=b["s"],
                              stats=b["st"], stream=stream)
        else:
            self.norm.forward(x, params["gf"], params["bf"], res, y=b["h"],
                              sum=None if res is None else b["s"], stats=b["st"], stream=stream)
        self.linear.forward(b["h"], params["head"], y=b["logits"], ws=b["ws_head"],
                            stream=stream)

    def forward(self, x, res: Optional[torch.Tensor], params: Dict[str, torch.Tensor],
                b: Dict[str, torch.Tensor], targets: Optional[torch.Tensor] = None, stream=None):
        """(logp, lse, entropy, top, top_logp) of the logits b["logits"] (logp None
        without targets, top and top_logp None where the head has none)."""
        self._logits(x, res, params, b, stream, None)
        return self.probs.forward(b["logits"][:, :self.vocab], targets,
                                  logp=None if targets is None else b["logp"], lse=b["lse"],
                                  entropy=b["entropy"], top=b.get("top"),
                                  top_logp=b.get("top_logp"), stream=stream)

    def step(self, x, res: Optional[torch.Tensor], targets: torch.Tensor, dlogp: torch.Tensor,
             params: Dict[str, torch.Tensor], b: Dict[str, torch.Tensor], stream=None,
             rng: Optional[torch.Tensor] = None, dentropy: Optional[torch.Tensor] = None):
        """A training step for the gradients dlogp (-1 / T for a mean loss) and dentropy
        of the log probabilities and entropies: (logp, the gradient of x, that of res)."""
        self._logits(x, res, params, b, stream, rng)
        V = self.vocab
        self.probs.loss(b["logits"][:, :V], targets, dlogp, dentropy, logp=b["logp"],
                        lse=b["lse"], entropy=None if dentropy is None else b["entropy"],
                        dlogits=b["dlogits"][:, :V], stream=stream)
        self.linear.backward(b["h"], b["dlogits"], params["head"], dx=b["dh"],
                             dparams=b["dp_head"], ws=b["ws_head"], stream=stream)
        if rng is not None:
            self.drop.backward(b["s"], b["dh"], rng, params["gf"], b["st"], dx=b["dx"],
                               dres=b["ds"], dgamma=b["dgf"], dbeta=b["dbf"], ws=b["ws_norm"],
                               stream=stream)
            return b["logp"], b["dx"], b["ds"]
        self.norm.backward(x if res is None else b["s"], b["dh"], params["gf"], b["st"], None,
                           dx=b["ds"], dgamma=b["dgf"], dbeta=b["dbf"], ws=b["ws_norm"],
                           stream=stream)
        return b["logp"], b["ds"], b["ds"]
