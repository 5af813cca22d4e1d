"""A small hybrid model decoded through the library: gated-delta-rule layers and a full-attention
layer between RMS norms, random weights.

    python examples/hybrid_decode.py

The prompt goes through the fused prologue and the chunked rule; every further token through one
step of the recurrent rule per layer (activations fused in), one new token against the paged
key-value cache (written by the same call) and the norms with the residual's addition, the last
one in 8 bits with a scale per row.  The plain products in between are torch's.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunked_prefill_gb300 import gdn  # noqa: E402

K = 128


@dataclass
class Config:
    hidden: int = 512
    layers: tuple = ("gdn", "gdn", "attention")
    hqk: int = 2
    hv: int = 4
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    vocab: int = 1000
    page: int = 16
    dtype: torch.dtype = torch.bfloat16


class HybridModel:
    def __init__(self, cfg: Config, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.cfg, self.device = cfg, device

        def w(*shape, dtype=cfg.dtype):
            return (torch.randn(*shape, generator=gen, device=device) / shape[0] ** 0.5).to(dtype)

        self.embed, self.head = w(cfg.vocab, cfg.hidden) * 20, w(cfg.hidden, cfg.vocab)
        self.norms = [torch.ones(cfg.hidden, device=device, dtype=cfg.dtype) for _ in range(len(cfg.layers) + 1)]
        self.weights = []
        for kind in cfg.layers:
            if kind == "gdn":
                self.weights.append(dict(
                    qkv=w(cfg.hidden, (2 * cfg.hqk + cfg.hv) * K), ab=w(cfg.hidden, 2 * cfg.hv), out=w(cfg.hv * K, cfg.hidden),
                    A_log=torch.zeros(cfg.hv, device=device) - 2, dt_bias=torch.randn(cfg.hv, generator=gen, device=device)))
            else:
                self.weights.append(dict(qkv=w(cfg.hidden, (cfg.heads + 2 * cfg.kv_heads) * cfg.head_dim),
                                         out=w(cfg.heads * cfg.head_dim, cfg.hidden)))

    def new_cache(self, slots: int, pages: int):
        """The pools a server keeps: states by slot, keys and values by page."""
        c, pools = self.cfg, []
        for kind in c.layers:
            if kind == "gdn":
                pools.append(torch.zeros(slots, c.hv, K, K, device=self.device))
            else:
                pools.append([torch.zeros(pages, c.page, c.kv_heads, c.head_dim, device=self.device, dtype=c.dtype) for _ in range(2)])
        return pools

    # ------------------------------------------------------------------ parts of a layer
    def _gdn_inputs(self, w, y):
        """q, k, v and the gates' pre-activations as views of the projections' rows."""
        c = self.cfg
        qkv, ab = y @ w["qkv"], (y @ w["ab"]).float()
        q, k, v = (x.unflatten(-1, (-1, K)) for x in qkv.split([c.hqk * K, c.hqk * K, c.hv * K], -1))
        return q, k, v, ab[..., :c.hv], ab[..., c.hv:]

    def _attention_inputs(self, w, y):
        c = self.cfg
        n = [c.heads * c.head_dim, c.kv_heads * c.head_dim, c.kv_heads * c.head_dim]
        return (x.unflatten(-1, (-1, c.head_dim)) for x in (y @ w["qkv"]).split(n, -1))

    def _logits(self, y, residual):
        y8, scale, _ = gdn.rms_norm_quant(y, self.norms[-1], residual=residual)
        return (y8.float() * scale) @ self.head.float()

    # --------------------------------------------------------------------------- prompt
    @torch.no_grad()
    def prefill(self, tokens, pools, slots, table):
        """Logits [N, vocab] after the prompt [N, T]; states and pages are filled."""
        c, (N, T) = self.cfg, tokens.shape
        x, residual = self.embed[tokens], None
        for kind, w, pool, norm in zip(c.layers, self.weights, pools, self.norms):
            if residual is None:
                (y, _), residual = gdn.rms_norm(x, norm), x
            else:
                y, residual = gdn.rms_norm(x, norm, residual=residual)
            if kind == "gdn":
                q, k, v, a, b = (t.contiguous() for t in self._gdn_inputs(w, y))
                q, k, g, beta = gdn.gated_delta_rule_prologue(q, k, a, b, w["A_log"], w["dt_bias"])
                o, state = gdn.chunk_gated_delta_rule(q, k, v, g, beta, output_final_state=True)
                pool[slots.long()] = state
            else:
                q, k, v = self._attention_inputs(w, y)
                at = torch.arange(T, device=self.device)
                page = table[:, at // c.page].long()
                pool[0][page, at % c.page], pool[1][page, at % c.page] = k, v
                G = c.heads // c.kv_heads
                z = torch.einsum("nqhd,nkhd->nhqk", q.float(), k.float().repeat_interleave(G, 2)) * c.head_dim ** -0.5
                z = z.masked_fill(at[None, :] > at[:, None], float("-inf"))
                o = torch.einsum("nhqk,nkhd->nqhd", z.softmax(-1), v.float().repeat_interleave(G, 2)).to(c.dtype)
            x = o.flatten(2) @ w["out"]
        return self._logits(x[:, -1], residual[:, -1])

    # ------------------------------------------------------------------------ one token
    @torch.no_grad()
    def decode(self, tokens, pools, slots, table, lens):
        """Logits [N, vocab] after one more token [N] per sequence; lens counts it."""
        c = self.cfg
        x, residual = self.embed[tokens], None
        for kind, w, pool, norm in zip(c.layers, self.weights, pools, self.norms):
            if residual is None:
                (y, _), residual = gdn.rms_norm(x, norm), x
            else:
                y, residual = gdn.rms_norm(x, norm, residual=residual)
            if kind == "gdn":
                q, k, v, a, b = (t[:, None] for t in self._gdn_inputs(w, y))
                o, _ = gdn.gated_delta_rule_step(q, k, v, a, b, state=pool, slots=slots, A_log=w["A_log"], dt_bias=w["dt_bias"])
            else:
                q, k, v = self._attention_inputs(w, y)
                o = gdn.paged_attention_decode(q, pool[0], pool[1], table, lens, k_new=k, v_new=v)
            x = o.flatten(1) @ w["out"]
        return self._logits(x, residual)


def main():
    cfg = Config()
    model = HybridModel(cfg)
    N, T, new, max_pages = 4, 100, 32, 10
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randint(0, cfg.vocab, (N, T), generator=gen, device="cuda")
    pools = model.new_cache(slots=N + 2, pages=N * max_pages)
    slots = torch.tensor([3, 0, 5, 1], dtype=torch.int32, device="cuda")
    table = torch.randperm(N * max_pages, generator=gen, device="cuda").to(torch.int32).view(N, max_pages)
    logits = model.prefill(prompt, pools, slots, table)
    token = logits.argmax(-1)
    lens = torch.full((N,), T, dtype=torch.int32, device="cuda")

    # the step as a captured graph: lengths, slots and pages are read on the device
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kept = [p.clone() if torch.is_tensor(p) else [t.clone() for t in p] for p in pools]
        model.decode(token, kept, slots, table, lens + 1)  # warm-up on copies
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            lens += 1
            token.copy_(model.decode(token, pools, slots, table, lens).argmax(-1))
    torch.cuda.current_stream().wait_stream(side)
    out = [token.clone()]
    for _ in range(new):
        graph.replay()
        out.append(token.clone())
    for n, row in enumerate(torch.stack(out, 1).tolist()):
        print(f"sequence {n}: {row}")


if __name__ == "__main__":
    main()
