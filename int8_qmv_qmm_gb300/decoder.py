"""A whole decoder from the library's calls: packed linears, norms with the
residual's addition, rotary positions with the append to the 8-bit cache,
attention over it, and sampling, for prompts and, as one CUDA graph, for decode
steps.  Weights are random (seeded), as everywhere in this package.

    d = Decoder("cuda", slots=4, max_tokens=4096)
    first = d.prefill([[5, 17, 99], [3], [], [8, 8]])  # an empty list: nothing new
    d.capture()
    for _ in range(100):
        tokens = d.decode()                              # int32 [slots], on the device

What stands between the calls in torch is the embedding's rows and the
activation silu(gate) * up.  Each layer is

    h, r  = add_rms_norm(y, w1, r)        r: the residual stream, float32
    q     = rope_append(linear(h, qkv))   keys and values go to the layer's cache
    y     = linear(cache_attention(q), o)
    h, r  = add_rms_norm(y, w2, r)
    y     = linear(silu(gate) * up, down)

With experts the last line is one of a mixture of them, and q and k can be normed for
each head before they turn (qk_norm):

    routing = route_experts(linear(h, router), top_experts)
    a       = silu(gate) * up of expert_linear(h, routing, gate_up)
    y       = combine_experts(expert_linear(a, routing, down), routing)

python -m int8_qmv_qmm_gb300.decoder times decode steps at Llama-3.2-1B's layer
shapes."""

from __future__ import annotations

import torch
import torch.nn.functional as F

from . import (KV_BLOCK, KVCache, add_rms_norm, attention_workspace, cache_attention,
               combine_experts, expert_linear, linear, quantize_affine, rope_append, rope_table,
               route_experts, sample, token_logprobs)
from . import synthetic as S


class Decoder:
    """Sampling settings are the tensors temperature, top_k, top_p and min_p
    [slots], as sample() takes them (the largest logit by default); write to
    them at any time, also after capture().

    experts and top_experts make the layers mixtures of experts, qk_norm adds the norms of
    query and key heads.  With logprobs = n, logprobs, entropy, top_tokens and top_logprobs are
    those of each slot's last token (token_logprobs with the n likeliest; the whole
    distribution's, whatever the sampling settings leave out of it).

    A slot whose logits have no token (all NaN or -infinity, as after an overflow) gets -1,
    and goes on from token 0; its neighbours are not affected."""

    def __init__(self, device="cuda", slots: int = 4, max_tokens: int = 4096, layers: int = 2,
                 hidden: int = 256, q_heads: int = 4, kv_heads: int = 2, head_dim: int = 64,
                 ffn: int = 512, vocab: int = 1024, bits: int = 8,
                 dtype: torch.dtype = torch.float16, rope_base: float = 10000.0, seed: int = 2,
                 experts: int = 0, top_experts: int = 2, qk_norm: bool = False,
                 logprobs: int | None = None):
        self.device, self.dtype, self.bits = torch.device(device), dtype, bits
        self.slots, self.max_tokens, self.q_heads, self.ffn = slots, max_tokens, q_heads, ffn
        self._seed = S.weight_seed(seed, 0)
        self.experts, self.top_experts = experts, top_experts
        width = (q_heads + 2 * kv_heads) * head_dim
        ones = torch.ones(hidden, dtype=dtype, device=self.device)
        # the page table and the lengths serve every layer
        lens = torch.zeros(slots, dtype=torch.int32, device=self.device)
        blocks = (max_tokens + KV_BLOCK - 1) // KV_BLOCK
        table = torch.arange(slots * blocks, dtype=torch.int32,
                             device=self.device).view(slots, blocks)
        self.embed = self._weights(vocab, hidden).to(dtype)
        heads = torch.ones(head_dim, dtype=dtype, device=self.device)
        norms = dict(q_norm=heads, k_norm=heads) if qk_norm else {}
        self.layers = [dict(norm1=ones, norm2=ones, qkv=self._packed(width, hidden),
                            o=self._packed(hidden, q_heads * head_dim),
                            gate_up=self._packed(2 * ffn, hidden, experts),
                            down=self._packed(hidden, ffn, experts),
                            router=self._packed(experts, hidden) if experts else None,
                            norms=norms,
                            cache=KVCache.empty(slots, max_tokens, kv_heads, head_dim, dtype,
                                                self.device, table=table, lens=lens,
                                                n_pages=slots * blocks))
                       for _ in range(layers)]
        self.norm, self.lm_head = ones, self._packed(vocab, hidden)
        self.rope = rope_table(max_tokens, head_dim, rope_base, device=self.device)
        self.workspace = attention_workspace(head_dim, self.device)
        self.lens = lens
        self.held = [0] * slots  # the same on the host
        # of the last call, float32 [slots, vocab] (rows of slots that got no tokens in it
        # are not theirs)
        self.logits = None
        self._top = logprobs
        self.logprobs = self.entropy = self.top_tokens = self.top_logprobs = None

        def row(value, dt=torch.float32):
            return torch.full((slots,), value, dtype=dt, device=self.device)

        self.temperature, self.top_p, self.min_p = row(0.0), row(1.0), row(0.0)
        self.top_k, self.tokens = row(0, torch.int32), row(0, torch.int32)
        self.u = row(0.0)  # the step's uniform numbers
        self._one_each = torch.arange(slots + 1, dtype=torch.int32, device=self.device)
        self._graph = None

    def _weights(self, n, k):
        self._seed += 1
        return torch.from_numpy(S.weights_f32(self._seed, n, k)).to(self.device)

    def _packed(self, n, k, experts=0):
        """Packed weights, or (experts in front) those of all experts."""
        if not experts:
            return quantize_affine(self._weights(n, k), self.bits, sdtype=self.dtype)
        return tuple(torch.stack(t) for t in zip(*(self._packed(n, k) for _ in range(experts))))

    def _linear(self, x, w, out_dtype=None):
        return linear(x, *w, self.bits, out_dtype=out_dtype)

    def _mixture(self, h, layer):
        routing = route_experts(self._linear(h, layer["router"], torch.float32), self.top_experts,
                                overlap_previous=True)
        gate_up = expert_linear(h, routing, *layer["gate_up"], self.bits, overlap_previous=True)
        y = expert_linear(F.silu(gate_up[:, :self.ffn]) * gate_up[:, self.ffn:], routing,
                          *layer["down"], self.bits)
        return combine_experts(y, routing, overlap_previous=True)

    def _forward(self, tokens, starts, max_new):
        """Logits of each slot's last new token; the caches and lens move on."""
        y = F.embedding(tokens, self.embed)
        r = None
        for layer in self.layers:
            if r is None:
                r = y.float()
                h, _ = add_rms_norm(y, layer["norm1"])
            else:
                h, _ = add_rms_norm(y, layer["norm1"], r, residual_out=r, overlap_previous=True)
            q = rope_append(self._linear(h, layer["qkv"]), self.rope, layer["cache"], starts,
                            self.q_heads, overlap_previous=True, **layer["norms"])
            a = cache_attention(q, layer["cache"], starts, max_new, self.workspace,
                                overlap_previous=True)
            y = self._linear(a.view(len(tokens), -1), layer["o"])
            h, _ = add_rms_norm(y, layer["norm2"], r, residual_out=r, overlap_previous=True)
            if self.experts:
                y = self._mixture(h, layer)
                continue
            gate_up = self._linear(h, layer["gate_up"])
            y = self._linear(F.silu(gate_up[:, :self.ffn]) * gate_up[:, self.ffn:],
                             layer["down"])
        self.lens += starts.diff()
        if len(tokens) != self.slots or max_new != 1:
            last = (starts[1:] - 1).clamp_(min=0).long()
            y, r = y[last], r[last]
        h, _ = add_rms_norm(y, self.norm, r)
        return self._linear(h, self.lm_head, torch.float32)

    def _sample(self, logits, tokens):
        sample(logits, self.u, self.temperature, self.top_k, self.top_p, self.min_p,
               tokens=tokens, overlap_previous=True)
        if self._top is not None:
            self.logprobs, self.entropy, self.top_tokens, self.top_logprobs = token_logprobs(
                logits, tokens, self._top, overlap_previous=True)

    _OF_TOKENS = ("logprobs", "entropy", "top_tokens", "top_logprobs")
    _ANSWERS = ("logits",) + _OF_TOKENS

    def _answers(self):
        return [getattr(self, name) for name in self._ANSWERS]

    def _answer(self, values):
        for name, value in zip(self._ANSWERS, values):
            setattr(self, name, value)

    def _check_room(self, new):
        for s, n in enumerate(new):
            if self.held[s] + n > self.max_tokens:
                raise ValueError(f"slot {s} holds {self.held[s]} tokens; {n} more would pass "
                                 f"max_tokens = {self.max_tokens}")

    def prefill(self, prompts):
        """Appends prompts[s] (a list of token ids, or of none) to each slot and
        samples the next token of those that got any.  Returns tokens [slots]."""
        new = [len(p) for p in prompts]
        if len(prompts) != self.slots or not any(new):
            raise ValueError("prefill takes a list of token ids for each slot, not all empty")
        self._check_room(new)
        flat = torch.tensor([t for p in prompts for t in p], dtype=torch.int32)
        if not 0 <= int(flat.min()) <= int(flat.max()) < len(self.embed):
            raise ValueError("a token id is outside the vocabulary")
        starts = torch.zeros(self.slots + 1, dtype=torch.int32)
        starts[1:] = torch.tensor(new).cumsum(0)
        starts = starts.to(self.device)
        self.u.uniform_()
        self.logits = self._forward(flat.to(self.device), starts, max(new))
        tokens, got = torch.empty_like(self.tokens), starts.diff() > 0
        before = [getattr(self, name) for name in self._OF_TOKENS]
        self._sample(self.logits, tokens)
        self.tokens.copy_(torch.where(got, tokens, self.tokens))
        for name, old in zip(self._OF_TOKENS, before):
            if old is not None:  # (a slot that got none keeps its last token's)
                own = got if old.dim() == 1 else got[:, None]
                setattr(self, name, torch.where(own, getattr(self, name), old))
        self.held = [h + n for h, n in zip(self.held, new)]
        return self.tokens

    def _step(self):
        # (a row of logits without a token gives -1, which has no embedding)
        self.logits = self._forward(self.tokens.clamp(min=0), self._one_each, 1)
        self._sample(self.logits, self.tokens)

    def capture(self):
        """Records the decode step as a CUDA graph; decode() then replays it.
        (A warm-up step runs first and is undone: the next step writes its token to
        the same place of the caches.)"""
        self._check_room([1] * self.slots)
        tokens, lens, before = self.tokens.clone(), self.lens.clone(), self._answers()
        side = torch.cuda.Stream(self.device)
        side.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(side):
            self._step()
        torch.cuda.current_stream(self.device).wait_stream(side)
        self.tokens.copy_(tokens)
        self.lens.copy_(lens)
        self._graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self._graph):
            self._step()
        self._graph_answers = self._answers()
        self._answer(before)

    def decode(self):
        """One decode step of every slot.  Returns the new tokens [slots] (one tensor,
        written to by every call; after capture() logits is one too, and the log
        probabilities)."""
        self._check_room([1] * self.slots)
        self.u.uniform_()
        if self._graph is None:
            self._step()
        else:
            self._graph.replay()
            self._answer(self._graph_answers)
        self.held = [h + 1 for h in self.held]
        return self.tokens


def main():
    import argparse

    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--slots", type=int, default=32)
    p.add_argument("--context", type=int, default=1000)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--steps", type=int, default=50)
    p.add_argument("--experts", type=int, default=0, help="a mixture of them in every layer")
    p.add_argument("--top-experts", type=int, default=2)
    p.add_argument("--ffn", type=int, default=0, help="an expert's (default: the layer shapes')")
    p.add_argument("--bits", type=int, default=8)
    a = p.parse_args()
    shape = {name: (n, k) for name, n, k in S.LLAMA_1B_LINEARS}
    d = Decoder("cuda", a.slots, a.context + a.steps + 8, a.layers, hidden=shape["q_proj"][1],
                q_heads=32, kv_heads=8, head_dim=64, ffn=a.ffn or shape["gate_proj"][0],
                vocab=S.LLAMA_1B_LM_HEAD[1], bits=a.bits, experts=a.experts, top_experts=a.top_experts,
                qk_norm=a.experts > 0)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    prompt = [[(7 * i + s) % 1000 for i in range(a.context)] for s in range(a.slots)]
    d.temperature.fill_(0.8)
    d.top_p.fill_(0.95)
    start.record()
    d.prefill(prompt)
    stop.record()
    torch.cuda.synchronize()
    print(f"prefill of {a.slots} x {a.context} tokens, {a.layers} layers: "
          f"{start.elapsed_time(stop):.2f} ms (first call)")
    d.capture()
    for _ in range(3):
        d.decode()
    start.record()
    for _ in range(a.steps):
        d.decode()
    stop.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(stop) / a.steps
    print(f"decode, {a.slots} slots: {ms * 1e3:.1f} us a step, {a.slots / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
