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
    step: Optional["_Step"] = dataclasses.field(default=None, repr=False, compare=False)   # until every layer's cache has it


class _Step:
    """A step that has begun: its sequences have grown, but not every layer's cache holds the new tokens yet."""

    def __init__(self, seqs: Sequence[CachedSequence], lengths: Sequence[int], prefix: Optional[CachedSequence]):
        self.seqs, self.lengths, self.prefix = list(seqs), list(lengths), prefix
        self.prefix_len = prefix.length if prefix is not None else 0
        self.prefix_pages = list(prefix.pages) if self.prefix_len else None
        self.rest = None           # the layers still to run, where the step may be ended without its caller
        self.closed = False        # a sequence of it was released

    def check(self) -> None:
        changed = self.prefix_len and (self.prefix.length < self.prefix_len or
                                       self.prefix.pages[:len(self.prefix_pages)] != self.prefix_pages)
        if self.closed or changed:
            raise ValueError("a sequence of this step was released")


def _begin(fwd: "Forward", x, seqs: Sequence[CachedSequence], lengths: Optional[Sequence[int]],
           prefix: Optional[CachedSequence]) -> _Step:
    """Checks a step, ends the steps that its sequences still stand in, and grows the sequences."""
    T, n = x.shape[0], len(seqs)
    if lengths is None:
        if T % n:
            raise ValueError("lengths are needed where tokens do not divide among the sequences")
        lengths = [T // n] * n
    if len(lengths) != n or sum(lengths) != T or min(lengths) < 0:
        raise ValueError(f"lengths must be {n} counts that add up to {T}")
    if len(set(map(id, seqs))) != n or any(s is prefix for s in seqs):
        raise ValueError("a sequence can stand in a step only once")
    used = list(seqs) + ([prefix] if prefix is not None else [])
    for s in used:
        if s.step is not None and s.step.rest is not None:
            for _ in s.step.rest:
                pass
    if any(s.step is not None for s in used):
        raise ValueError("a step of a sequence was left before its last layer: release the sequence")
    step = _Step(seqs, lengths, prefix)
    fwd._grow(seqs, lengths, step.prefix_len)
    for s in seqs:
        s.step = step
    return step


def _layers(fwd: "Forward", x, step: _Step, check: bool) -> Iterator[tuple]:
    """A step that has begun, a layer at a time (see Forward.blocks)."""
    import torch
    T, n = x.shape[0], len(step.seqs)
    step.check()

    def ints(v):
        return torch.tensor(v, dtype=torch.int32).to(x.device)

    starts = [0]
    for k in step.lengths:
        starts.append(starts[-1] + k)
    width = max([len(s.pages) for s in step.seqs] + [1])
    table = [s.pages + [0] * (width - len(s.pages)) for s in step.seqs]
    at = B.step(T, fwd.H, ints(starts), ints([s.length for s in step.seqs]), ints(table).reshape(n, width),
                ints(step.prefix_pages) if step.prefix_len else None, step.prefix_len)
    plan = torch.empty(B.step_plan_size(at, fwd.caches[0]), dtype=torch.uint8, device=x.device)
    B.step_plan(at, fwd.caches[0], plan)
    h, a = torch.empty_like(x), torch.empty(T, fwd.H * fwd.d, dtype=x.dtype, device=x.device)
    # the first block's input norm: nothing is added yet
    B.block_norm(x, x, x, h, pre_gain=fwd.layers[0]["g_attn"], scale=0.0, eps=fwd.eps)
    for i, w in enumerate(fwd.layers):
        last = i + 1 == len(fwd.layers)
        q, k, v = h @ w["Wq"].T, h @ w["Wk"].T, h @ w["Wv"].T
        B.kv_append(q, k, v, fwd.caches[i], at, fwd.rotaries[i], q, plan)
        B.prefix_attention(q, fwd.caches[i], at, fwd.d ** -0.5, a, None, plan)
        B.block_norm(x, a @ w["Wo"].T, x, h, pre_gain=w["gamma"], eps=fwd.eps)
        if check:
            _status(plan)
        if last:
            for s in step.seqs:
                s.step = None
        yield i, a, x
        if not last:
            step.check()
        f = (torch.nn.functional.silu(h @ w["Wg"].T) * (h @ w["Wu"].T)) @ w["Wd"].T
        if last:
            B.block_norm(x, f, x, eps=fwd.eps)
        else:
            B.block_norm(x, f, x, h, pre_gain=fwd.layers[i + 1]["g_attn"], eps=fwd.eps)
    _status(plan)


def _status(plan) -> None:
    st = B.device_status(plan)
    if st != B.AFF_OK:
        raise B.AffinityError(st, "forward step", B.strerror(st))


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
        """Gives a sequence's pages back.  A step that it still stands in ends there, for the others too."""
        if seq.step is not None:
            seq.step.closed, seq.step.rest = True, None
            seq.step = None
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
        read at the end, with `check` (which waits for the stream) before every yield too.  Left before its last
        layer, a step leaves caches without its tokens: its sequences are refused until they are released."""
        yield from _layers(self, x, _begin(self, x, seqs, lengths, prefix), check)

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
        be left out, as a resumed run does), each time the stack goes on to that layer.  The sequences have grown at once;
        the next step that uses one of them first runs the layers that were not asked for."""
        step = _begin(self, x, seqs, lengths, prefix)
        run = step.rest = _layers(self, x.clone(), step, check=True)

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
