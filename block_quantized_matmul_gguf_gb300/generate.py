"""A small generation loop over the library's calls, as a serving program runs
them: plan the pages of a step, project q, k and v with Q4_0 weights, append
keys and values to the 4-bit cache, attend, project back, apply the Q8_0 LM
head, adjust the logits, take the largest.

One attention layer with a residual, random weights of the given sizes and no
tokenizer: it shows how the calls fit together, not a language model.

    python -m block_quantized_matmul_gguf_gb300.generate --steps 16
"""
from __future__ import annotations

import argparse

import torch

from . import qmm, synth


class Layer:
    """Random weights of one attention layer, an embedding and an LM head."""

    def __init__(self, hidden=512, heads=8, kv_heads=2, head_dim=64, vocab=2048, seed=0, device="cuda"):
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.vocab = hidden, heads, kv_heads, head_dim, vocab
        self.device = torch.device(device)

        def blocks(a):
            return torch.from_numpy(a).to(self.device)

        width, kv_width = heads * head_dim, kv_heads * head_dim
        self.wq = blocks(synth.q4_0_weights(width, hidden, seed=seed, stream=0))
        self.wk = blocks(synth.q4_0_weights(kv_width, hidden, seed=seed, stream=1))
        self.wv = blocks(synth.q4_0_weights(kv_width, hidden, seed=seed, stream=2))
        self.wo = blocks(synth.q4_0_weights(hidden, width, seed=seed, stream=3))
        self.head = blocks(synth.q8_0_weights(vocab, hidden, seed=seed, stream=4))
        self.embedding = blocks(synth.activations_f32(vocab, hidden, seed=seed, stream=5))


class Generator:
    """Requests that share a paged Q4_0 cache and take their steps together."""

    def __init__(self, layer: Layer, batch: int, num_pages: int = 256, page_size: int = 16, max_pages: int = 64):
        self.layer, self.batch, dev = layer, batch, layer.device
        self.cache = qmm.kv_cache_q4_0(num_pages, page_size, layer.kv_heads, layer.head_dim, dev)
        self.workspace = qmm.attn_workspace(self.cache, layer.heads)
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((batch, max_pages), -1, **i32)
        self.free = torch.arange(num_pages, **i32)
        self.free_at = 0  # pages taken so far
        self.kv_len = torch.zeros(batch, **i32)
        self.history = [[] for _ in range(batch)]
        self.hidden = torch.zeros((batch, layer.hidden), device=dev)  # last row of each request
        self.prompt_len = torch.zeros(batch, **i32)

    def _project(self, weights, x, n_out, k):
        """Rows of x times a Q4_0 matrix: fp32 up to 16 rows, else bf16 in and fp32 out."""
        if x.dtype == torch.float32:
            return qmm.gemv("q4_0", weights, x, n_out, k)
        return qmm.gemm("q4_0", weights, x, n_out, k)

    def forward(self, tokens):
        """tokens: a list of new token ids for each request; one without any keeps
        its last row's hidden state (zeros before its first token).
        Returns those states [batch][hidden]."""
        layer, dev = self.layer, self.layer.device
        if not any(tokens):
            return self.hidden
        added = torch.tensor([len(t) for t in tokens], dtype=torch.int32, device=dev)
        total, most = sum(len(t) for t in tokens), max(len(t) for t in tokens)
        page = self.cache.page_size
        lens = self.kv_len.tolist()
        taken = sum(-(-(n + len(t)) // page) - -(-n // page) for n, t in zip(lens, tokens))
        if self.free_at + taken > self.free.numel():
            raise RuntimeError("the cache is full")
        if max(n + len(t) for n, t in zip(lens, tokens)) > self.table.shape[1] * page:
            raise RuntimeError("a request is longer than its row of the page table")
        q_start = torch.empty(self.batch + 1, dtype=torch.int32, device=dev)
        kv_len, used = torch.empty_like(self.kv_len), torch.empty(1, dtype=torch.int32, device=dev)
        slots = torch.empty(total, dtype=torch.int64, device=dev)
        positions = torch.empty(total, dtype=torch.int32, device=dev)
        qmm.qmm_kv_plan(self.kv_len, added, self.free[self.free_at:], self.table, page, q_start, kv_len, slots,
                        positions, used)
        self.free_at += taken

        flat = torch.tensor([t for row in tokens for t in row], dtype=torch.int64, device=dev)
        x = layer.embedding[flat]
        small = total <= qmm.QMM_GEMV_MAX_M
        act = x if small else x.bfloat16()
        width, kv_width = layer.heads * layer.head_dim, layer.kv_heads * layer.head_dim
        if small:  # three projections in one launch
            q, k, v = (torch.empty((total, n), device=dev) for n in (width, kv_width, kv_width))
            qmm.qmm_gemv_q4_0_multi([(layer.wq, q, width), (layer.wk, k, kv_width), (layer.wv, v, kv_width)],
                                    act, total, layer.hidden)
        else:
            q, k, v = (self._project(w, act, n, layer.hidden)
                       for w, n in ((layer.wq, width), (layer.wk, kv_width), (layer.wv, kv_width)))
        heads = (total, layer.kv_heads, layer.head_dim)
        qmm.qmm_kv_append_q4_0(self.cache, k.view(heads), v.view(heads), slots)
        out = torch.empty((total, layer.heads, layer.head_dim), dtype=act.dtype, device=dev)
        qmm.qmm_attn_q4_0(self.cache, q.view(out.shape), out, self.table, q_start, kv_len, most,
                          layer.head_dim ** -0.5, workspace=self.workspace)
        x = x + self._project(layer.wo, out.view(total, width), layer.hidden, width)
        self.kv_len = kv_len
        self.last = dict(q=q.view(out.shape), out=out, q_start=q_start, slots=slots, positions=positions)
        ends = x[(q_start[1:] - 1).long().clamp(min=0)]  # of a request without new tokens, another's
        self.hidden = torch.where((added > 0)[:, None], ends, self.hidden)
        return self.hidden

    def logits(self, rows, repetition=1.1, frequency=0.1, presence=0.1, bias=None, allowed=None):
        """LM head and adjustment of [batch][hidden] rows (at most 16)."""
        layer, dev = self.layer, self.layer.device
        y = qmm.gemv("q8_0", layer.head, rows, layer.vocab, layer.hidden)
        ends = [0]
        for h in self.history:
            ends.append(ends[-1] + len(h))

        def f32(v):
            return torch.full((self.batch,), v, dtype=torch.float32, device=dev)

        more = {}
        if bias:
            more = dict(bias_ids=torch.tensor(list(bias) * self.batch, dtype=torch.int32, device=dev),
                        bias_values=torch.tensor(list(bias.values()) * self.batch, dtype=torch.float32, device=dev),
                        bias_start=torch.arange(self.batch + 1, dtype=torch.int32, device=dev) * len(bias))
        qmm.qmm_logits_adjust(y, y, history=torch.tensor([t for h in self.history for t in h], dtype=torch.int32, device=dev),
                              hist_start=torch.tensor(ends, dtype=torch.int32, device=dev), prompt_len=self.prompt_len,
                              repetition=f32(repetition), frequency=f32(frequency), presence=f32(presence),
                              allowed=allowed, **more)
        return y

    def step(self, tokens, **adjust):
        """New tokens of each request in, the next token of each out."""
        rows = self.forward(tokens)
        for h, t in zip(self.history, tokens):
            h.extend(t)
        return self.logits(rows, **adjust).argmax(-1).tolist()

    def run(self, prompts, steps, **adjust):
        """Prompts first, then one token a request and step; the tokens generated."""
        self.prompt_len = torch.tensor([len(h) + len(p) for h, p in zip(self.history, prompts)], dtype=torch.int32,
                                       device=self.layer.device)
        made = [[] for _ in prompts]
        tokens = prompts
        for _ in range(steps):
            new = self.step(tokens, **adjust)
            for m, t in zip(made, new):
                m.append(t)
            tokens = [[t] for t in new]
        return made


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    layer = Layer(seed=a.seed)
    prompts = [[1, 2, 3, 4, 5], list(range(40, 120)), [7]]
    made = Generator(layer, len(prompts)).run(prompts, a.steps)
    for p, m in zip(prompts, made):
        print(f"{len(p)} prompt tokens -> {m}")


if __name__ == "__main__":
    main()
