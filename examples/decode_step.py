"""The end of a decoding step, from the residual stream to the next token and
back: the tied embedding's row of the last token (int4 head), residual addition
and RMS norm straight to microscaled 8-bit codes, the product with a microscaled
4-bit head, and the draw with temperature, top-k, top-p and min-p.

    python examples/decode_step.py [--batch 4] [--vocab 151936] [--hidden 1024] [--steps 16]

There is no model between the embedding and the norm: a fixed random mixing of
the hidden state stands in for it, and the weights are random.  The step is run
eagerly and as one CUDA graph; both give the same tokens.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_wql_gb300 as wql  # noqa: E402


@dataclass
class Head:
    """What a serving process keeps: laid out once."""
    embed: wql.QuantizedWeight     # int4, for the gather
    logits: wql.MXMatrix           # e2m1 blocks, for the product
    gamma: torch.Tensor
    mix: torch.Tensor              # stands in for the model

    @staticmethod
    def random(vocab: int, hidden: int, seed: int = 0) -> "Head":
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        w = 0.02 * torch.randn(vocab, hidden, generator=g, device="cuda")
        gamma = 1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")
        mix = torch.randn(hidden, hidden, generator=g, device="cuda") / hidden ** 0.5
        return Head(wql.wql_quantize(w, 4, 64), wql.wql_mx_quantize(w), gamma.bfloat16(),
                    mix.bfloat16())


@dataclass
class Sequences:
    """A batch's state between steps."""
    ids: torch.Tensor              # int32 [batch], last tokens
    residual: torch.Tensor         # bf16 [batch, hidden]
    temperature: torch.Tensor
    top_k: torch.Tensor
    top_p: torch.Tensor
    min_p: torch.Tensor

    @staticmethod
    def start(batch: int, hidden: int) -> "Sequences":
        def full(v, dtype=torch.float32):
            return torch.full((batch,), v, dtype=dtype, device="cuda")
        return Sequences(torch.arange(batch, dtype=torch.int32, device="cuda"),
                         torch.zeros(batch, hidden, dtype=torch.bfloat16, device="cuda"),
                         full(0.8), full(50, torch.int32), full(0.95), full(0.02))


def step(head: Head, seq: Sequences, u: torch.Tensor, workspace: wql.Workspace):
    """One step for the whole batch; updates seq.ids and seq.residual in place
    and returns the drawn tokens' log-probabilities."""
    x = wql.wql_embed_gather(seq.ids, head.embed, torch.bfloat16) @ head.mix
    y, _, _ = wql.wql_add_rmsnorm(x, head.gamma, seq.residual, fmt=wql.NORM_MX_FP8,
                                  residual_out=seq.residual)
    logits = wql.wql_mx_logits(y, head.logits, torch.bfloat16, workspace=workspace)
    ids, logp = wql.wql_sample(logits, u, seq.temperature, seq.top_k, seq.top_p, seq.min_p)
    seq.ids.copy_(ids)
    return logp


def decode(batch: int, vocab: int, hidden: int, steps: int, graph: bool, seed: int = 0):
    """Token ids [steps, batch] and their log-probabilities."""
    head, seq = Head.random(vocab, hidden, seed), Sequences.start(batch, hidden)
    workspace = wql.Workspace("cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    draws = torch.rand(steps, batch, generator=g, device="cuda")
    u = torch.zeros(batch, device="cuda")
    run = lambda: step(head, seq, u, workspace)  # noqa: E731
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()                               # loads and sizes everything once
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            logp = run()
        again = Sequences.start(batch, hidden)
        seq.ids.copy_(again.ids)
        seq.residual.copy_(again.residual)
    tokens, logps = [], []
    for i in range(steps):
        u.copy_(draws[i])
        if graph:
            captured.replay()
        else:
            logp = run()
        tokens.append(seq.ids.clone())
        logps.append(logp.clone())
    torch.cuda.synchronize()
    if workspace.error_word():
        raise RuntimeError(f"a wait ran out: error word {workspace.error_word():#x}")
    ids = torch.stack(tokens).cpu()
    if (ids == -2).any():
        raise RuntimeError("a wait of the sampler ran out")
    return ids, torch.stack(logps).cpu()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=151936)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    eager, logp = decode(a.batch, a.vocab, a.hidden, a.steps, graph=False)
    graph, _ = decode(a.batch, a.vocab, a.hidden, a.steps, graph=True)
    for b in range(a.batch):
        print(f"sequence {b}: {eager[:, b].tolist()}  mean logp {logp[:, b].mean():.3f}")
    print("the graph draws the same tokens" if torch.equal(eager, graph) else "TOKENS DIFFER")


if __name__ == "__main__":
    main()
