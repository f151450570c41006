"""Beam search over a head that every request has its own low-rank adapter for:
the int4 head's logits, what the adapters add to them, the selection over beams
and vocabulary, and the beams' states following it in place.

    python examples/beam_step.py [--batch 2] [--beams 4] [--vocab 50304] [--hidden 512]
                                 [--steps 16]

There is no model in front of the head: a fixed random mixing of a recurrent
hidden state stands in for it, and the weights are random.  The step is run
eagerly and as one CUDA graph; both find the same sequences.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_wql_gb300 as wql  # noqa: E402

EOS = 1


@dataclass
class Model:
    """What a serving process keeps: laid out once."""
    head: wql.QuantizedWeight
    adapters: wql.LoraAdapters     # of the head
    mix: torch.Tensor              # stands in for the model

    @staticmethod
    def random(vocab: int, hidden: int, adapters: int, seed: int = 0) -> "Model":
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        a = (randn(adapters, 16, hidden) / hidden ** 0.5).half()
        b = (0.3 * randn(adapters, vocab, 16)).half()
        return Model(wql.wql_quantize(0.3 * randn(vocab, hidden), 4, 64),
                     wql.LoraAdapters(a, b, torch.ones(adapters, device="cuda")),
                     (randn(hidden, hidden) / hidden ** 0.5).half())


@dataclass
class Search:
    """A batch's state between steps."""
    hidden: torch.Tensor           # fp16 [batch * beams, hidden]
    history: torch.Tensor          # int32 [batch * beams, steps]
    tokens: torch.Tensor           # int32 [batch, beams], last ones
    scores: torch.Tensor           # float [batch, beams]
    best_end: torch.Tensor         # float [batch], of the sequences that have ended
    length: torch.Tensor           # int32 [batch]
    ids: torch.Tensor              # int32 [batch * beams], adapters

    @staticmethod
    def start(model: Model, batch: int, beams: int, steps: int) -> "Search":
        rows, k = batch * beams, model.head.k
        scores = torch.full((batch, beams), float("-inf"), device="cuda")
        scores[:, 0] = 0                            # the first step has one beam
        count = model.adapters.a.shape[0]
        # one request more than there are adapters goes without
        ids = (torch.arange(rows, device="cuda") // beams % (count + 1) - 1).int()
        return Search(torch.zeros(rows, k, dtype=torch.float16, device="cuda"),
                      torch.zeros(rows, steps, dtype=torch.int32, device="cuda"),
                      torch.zeros(batch, beams, dtype=torch.int32, device="cuda"), scores,
                      torch.full((batch,), float("-inf"), device="cuda"),
                      torch.zeros(batch, dtype=torch.int32, device="cuda"), ids)

    def copy_(self, other: "Search") -> None:
        for name, value in vars(other).items():
            getattr(self, name).copy_(value)


def step(model: Model, s: Search, workspace: wql.Workspace) -> None:
    """One step for the whole batch, in place."""
    x = wql.wql_embed_gather(s.tokens.view(-1), model.head, torch.float16)
    s.hidden.copy_(torch.tanh((s.hidden + x) @ model.mix))
    logits, _, _ = wql.wql_logits(s.hidden, model.head, workspace=workspace)
    wql.wql_lora_add(logits, s.hidden, model.adapters, s.ids, out=logits)
    # surviving beams stay in their rows: less to move
    tokens, parents, scores, ended = wql.wql_beam_select(logits, s.scores, EOS, wql.BEAM_ANCHORED)
    wql.wql_beam_reorder([s.hidden], parents)
    wql.wql_beam_reorder([s.history], parents, s.length, 1)
    here = torch.arange(s.history.shape[1], device="cuda") == s.length[0]
    s.history.copy_(torch.where(here, tokens.view(-1, 1), s.history))
    s.best_end.copy_(torch.maximum(s.best_end, ended.amax(-1)))
    s.tokens.copy_(tokens)
    s.scores.copy_(scores)
    s.length.add_(1)


def search(batch: int, beams: int, vocab: int, hidden: int, steps: int, graph: bool, seed: int = 0):
    """(histories [batch, beams, steps], scores [batch, beams], best ended scores)."""
    model = Model.random(vocab, hidden, 3, seed)
    s = Search.start(model, batch, beams, steps)
    workspace = wql.Workspace("cuda")
    run = lambda: step(model, s, workspace)  # noqa: E731
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()                               # loads and sizes everything once
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            run()
        s.copy_(Search.start(model, batch, beams, steps))
    for _ in range(steps):
        captured.replay() if graph else run()
    torch.cuda.synchronize()
    if workspace.error_word():
        raise RuntimeError(f"a wait ran out: error word {workspace.error_word():#x}")
    return s.history.view(batch, beams, steps).cpu(), s.scores.cpu(), s.best_end.cpu()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=50304)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    eager = search(a.batch, a.beams, a.vocab, a.hidden, a.steps, graph=False)
    graph = search(a.batch, a.beams, a.vocab, a.hidden, a.steps, graph=True)
    for i in range(a.batch):
        best = int(eager[1][i].argmax())
        print(f"sequence {i}: {eager[0][i, best].tolist()}  score {eager[1][i, best]:.3f}  "
              f"best ended {eager[2][i]:.3f}")
    same = all(torch.equal(x, y) for x, y in zip(eager, graph))
    print("the graph finds the same sequences" if same else "SEQUENCES DIFFER")


if __name__ == "__main__":
    main()
