"""The forward pass of a pre-norm decoder stack over a paged cache, for what calibration reads of it.

``affinity_up`` and ``affinity_down`` score a layer from its attention output `a` and the residual `x` that enters
its FFN's pre-norm.  ``Forward`` computes both for a batch of sequences that may share a prefix (a system prompt is
run once and read by every sequence), and goes on from the cache token by token, so that calibration can also read
what the model writes itself:

    fwd = Forward(layers, H, G, d_head, n_pages=512, n_pos=8192)
    prefix = fwd.new_sequence()
    fwd.run(embedded_system_prompt, [prefix])
    seqs = [fwd.new_sequence() for _ in prompts]
    S_up, S_down = stack.calibrate_stack(fwd.layer_inputs(embedded_prompts, seqs, lengths, prefix=prefix), N, dims)

The appends, the attention and the norms are the library's; the projections are plain matrix products.  A layer is
a dict of tensors on the GPU under the names of ``stack.realise_layout``'s weights and its gains: g_attn, Wq, Wk, Wv, Wo,
gamma, Wg, Wu, Wd, and optionally qn, kn (per-head norm gains of queries and keys).
"""
from __future__ import annotations

import dataclasses
from typing import Callable, Dict, Iterator, List, Optional, Sequence

from . import binding as B


@dataclasses.dataclass
class CachedSequence:
    """A sequence in the cache: its pages and the tokens they hold."""
    pages: List[int] = dataclasses.field(default_factory=list)
    length: int = 0


def rotary_tables(n_pos: int, rot: int, base: float = 10000.0, device="cuda"):
    """cos and sin of position t times base^(-2 j / rot), j < rot / 2, from 64-bit angles."""
    import torch
    inv = base ** (-torch.arange(rot // 2, dtype=torch.float64, device=device) * 2.0 / rot)
    angle = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


class Forward:
    """A layer stack with its paged caches: n_pages pages of page_size tokens per layer, positions up to n_pos."""

    def __init__(self, layers: Sequence[Dict[str, object]], H: int, G: int, d_head: int, n_pages: int, n_pos: int,
                 page_size: int = 64, eps: float = 1e-6, base: float = 10000.0):
        import torch
        self.layers, self.H, self.G, self.d, self.eps = list(layers), H, G, d_head, eps
        w = self.layers[0]["Wq"]
        self.page_size, self.n_pos = page_size, n_pos
        pools = torch.empty(len(self.layers), 2, n_pages, G, page_size, d_head, dtype=w.dtype, device=w.device)
        self.caches = [B.kv_cache(p[0], p[1]) for p in pools]
        cos, sin = rotary_tables(n_pos, d_head, base, w.device)
        self.rotaries = [B.rotary(cos, sin, q_gain=l.get("qn"), k_gain=l.get("kn"), eps=eps) for l in self.layers]
        self.free = list(range(n_pages - 1, -1, -1))

    def new_sequence(self) -> CachedSequence:
        return CachedSequence()

    def release(self, seq: CachedSequence) -> None:
        """Gives a sequence's pages back."""
        self.free.extend(reversed(seq.pages))
        seq.pages, seq.length = [], 0

    def _grow(self, seqs: Sequence[CachedSequence], lengths: Sequence[int], prefix_len: int) -> None:
        need = [-(-(s.length + n) // self.page_size) - len(s.pages) for s, n in zip(seqs, lengths)]
        if sum(n for n in need if n > 0) > len(self.free):
            raise ValueError("the cache has too few free pages")
        if any(prefix_len + s.length + n > self.n_pos for s, n in zip(seqs, lengths)):
            raise ValueError("a sequence would pass n_pos")
        for s, n, k in zip(seqs, lengths, need):
            for _ in range(k):
                s.pages.append(self.free.pop())
            s.length += n

    def blocks(self, x, seqs: Sequence[CachedSequence], lengths: Optional[Sequence[int]] = None,
               prefix: Optional[CachedSequence] = None, check: bool = False) -> Iterator[tuple]:
        """One step, a layer at a time.  x [T, D]: the embedded new tokens, sequence by sequence, lengths[b] of
        sequence b (equal ones if not given); all sequences stand behind `prefix`.  Yields (i, a, x) of every layer:
        the attention output [T, H d_head] and the residual entering the FFN's pre-norm [T, D], which are
        overwritten when the iteration goes on; x holds the stack's output [T, D] when it ends.  The step's status is
        read at the end, with `check` (which waits for the stream) before every yield too."""
        import torch
        T, D = x.shape
        B_ = len(seqs)
        if lengths is None:
            if T % B_:
                raise ValueError("lengths are needed where tokens do not divide among the sequences")
            lengths = [T // B_] * B_
        if len(lengths) != B_ or sum(lengths) != T or min(lengths) < 0:
            raise ValueError(f"lengths must be {B_} counts that add up to {T}")
        if len(set(map(id, seqs))) != B_ or any(s is prefix for s in seqs):
            raise ValueError("a sequence can stand in a step only once")
        prefix_len = prefix.length if prefix is not None else 0
        self._grow(seqs, lengths, prefix_len)

        def ints(v):
            return torch.tensor(v, dtype=torch.int32).to(x.device)

        starts = [0]
        for n in lengths:
            starts.append(starts[-1] + n)
        width = max([len(s.pages) for s in seqs] + [1])
        table = [s.pages + [0] * (width - len(s.pages)) for s in seqs]
        step = B.step(T, self.H, ints(starts), ints([s.length for s in seqs]), ints(table).reshape(B_, width),
                      ints(prefix.pages) if prefix_len else None, prefix_len)
        plan = torch.empty(B.step_plan_size(step, self.caches[0]), dtype=torch.uint8, device=x.device)
        B.step_plan(step, self.caches[0], plan)
        h, a = torch.empty_like(x), torch.empty(T, self.H * self.d, dtype=x.dtype, device=x.device)
        # the first block's input norm: nothing is added yet
        B.block_norm(x, x, x, h, pre_gain=self.layers[0]["g_attn"], scale=0.0, eps=self.eps)
        for i, w in enumerate(self.layers):
            q, k, v = h @ w["Wq"].T, h @ w["Wk"].T, h @ w["Wv"].T
            B.kv_append(q, k, v, self.caches[i], step, self.rotaries[i], q, plan)
            B.prefix_attention(q, self.caches[i], step, self.d ** -0.5, a, None, plan)
            B.block_norm(x, a @ w["Wo"].T, x, h, pre_gain=w["gamma"], eps=self.eps)
            if check:
                self._status(plan)
            yield i, a, x
            f = (torch.nn.functional.silu(h @ w["Wg"].T) * (h @ w["Wu"].T)) @ w["Wd"].T
            if i + 1 < len(self.layers):
                B.block_norm(x, f, x, h, pre_gain=self.layers[i + 1]["g_attn"], eps=self.eps)
            else:
                B.block_norm(x, f, x, eps=self.eps)
        self._status(plan)

    @staticmethod
    def _status(plan) -> None:
        st = B.device_status(plan)
        if st != B.AFF_OK:
            raise B.AffinityError(st, "forward step", B.strerror(st))

    def run(self, x, seqs: Sequence[CachedSequence], lengths: Optional[Sequence[int]] = None,
            prefix: Optional[CachedSequence] = None):
        """One step through every layer: the stack's output [T, D].  x is left as it is."""
        y = x.clone()
        for _ in self.blocks(y, seqs, lengths, prefix):
            pass
        return y

    def layer_inputs(self, x, seqs: Sequence[CachedSequence], lengths: Optional[Sequence[int]] = None,
                     prefix: Optional[CachedSequence] = None) -> Callable[[int], Dict[str, object]]:
        """The `layer_inputs` of ``stack.calibrate_stack`` for one step: called with rising layer numbers (some may
        be left out, as a resumed run does), each time the stack goes on to that layer."""
        run = self.blocks(x.clone(), seqs, lengths, prefix, check=True)

        def inputs(i: int) -> Dict[str, object]:
            for j, a, residual in run:
                if j == i:
                    break
            else:
                raise ValueError(f"layer {i} has been passed")
            w = self.layers[i]
            t = {"a": a, "x": residual, "Wo": w["Wo"], "gamma": w["gamma"], "Wg": w["Wg"], "Wu": w["Wu"], "Wd": w["Wd"]}
            if i + 1 < len(self.layers):
                n = self.layers[i + 1]
                t.update(gamma_next=n["g_attn"], Wq_next=n["Wq"], Wk_next=n["Wk"], Wv_next=n["Wv"])
            return t

        return inputs
