"""The end of a decode step for a batch of requests, captured once and replayed per token.

Each request has its own low-rank adapter on the head, its own sampling keys and its own random numbers.  A stand-in
for the model's layers (an embedding of the last token mixed into the hidden row) feeds the tail:

    hidden, residual -> norm_rows (8-bit rows, one scale each) -> project_rows (8-bit head + the request's adapter)
    -> draw_rows (the request's temperature, top_k, top_p, min_p, and a number in [0, 1) per token)

    python examples/decode_tail.py --slots 8 --vocab 32000 --hidden 1024 --tokens 16
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class DecodeTail:
    """Weights and per-slot state on the GPU; step() draws the next token of every slot."""

    def __init__(self, slots, vocab, hidden, rank=16, adapters=4, seed=0):
        import torch
        self.torch = torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        bf16 = torch.bfloat16
        self.embed = rand(vocab, hidden).to(bf16)
        self.norm_weight = (1 + 0.1 * rand(hidden)).to(bf16)
        head = rand(vocab, hidden) * 3 * hidden ** -0.5
        self.head_scale = head.abs().amax(1) / 448
        self.head = (head / self.head_scale[:, None]).to(torch.float8_e4m3fn)
        self.a = (rand(adapters, rank, hidden) * hidden ** -0.5).to(bf16)
        self.b = (rand(adapters, vocab, rank) * rank ** -0.5).to(bf16)
        self.adapter_scale = torch.full((adapters,), 0.5, device="cuda")
        # one request per slot: the last slot uses the head alone
        self.row_adapter = torch.tensor([s % adapters if s + 1 < slots else -1 for s in range(slots)], dtype=torch.int32, device="cuda")
        self.temperature = torch.linspace(0.0, 1.2, slots, device="cuda")     # slot 0 is greedy
        self.top_k = torch.tensor([(0, 40, 200, 5000)[s % 4] % vocab for s in range(slots)], dtype=torch.int32, device="cuda")
        self.top_p = torch.tensor([(1.0, 0.95, 0.9)[s % 3] for s in range(slots)], device="cuda")
        self.min_p = torch.tensor([(0.0, 0.02)[s % 2] for s in range(slots)], device="cuda")
        # what a step reads and writes in place, so that it can be replayed
        self.last = torch.arange(slots, device="cuda", dtype=torch.int32)
        self.residual = rand(slots, hidden).to(bf16)
        self.u = torch.zeros(slots, device="cuda")
        self.lps = torch.zeros(slots, device="cuda")

    def step(self):
        import request_token_sampling_gb300 as G
        hidden = self.embed[self.last.long()]
        n = G.norm_rows(hidden, self.norm_weight, residual=self.residual, y=False, f8=True, out=dict(residual=self.residual))
        logits = G.project_rows(n["q"], self.head, x_scale=n["scale"], w_scale=self.head_scale, a=self.a, b=self.b,
                                row_adapter=self.row_adapter, adapter_scale=self.adapter_scale)
        G.draw_rows(logits, self.u, self.temperature, self.top_k, self.top_p, self.min_p, V=logits.shape[1],
                    out=dict(ids=self.last, lps=self.lps))
        return logits

    def capture(self):
        """The step as a CUDA graph; the state is as before the capture."""
        torch = self.torch
        state = [t.clone() for t in (self.last, self.residual)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        for t, s in zip((self.last, self.residual), state):
            t.copy_(s)
        return graph


def decode(slots, vocab, hidden, tokens, seed=0, graph=True):
    """[tokens, slots] ids and their log-probabilities."""
    import torch
    import request_token_sampling_gb300 as G
    tail = DecodeTail(slots, vocab, hidden, seed=seed)
    step = tail.capture().replay if graph else tail.step
    numbers = torch.rand(tokens, slots, generator=torch.Generator(device="cuda").manual_seed(seed + 1), device="cuda")
    ids, lps = [], []
    for t in range(tokens):
        tail.u.copy_(numbers[t])
        step()
        ids.append(tail.last.clone())
        lps.append(tail.lps.clone())
    torch.cuda.synchronize()
    if G.tail_errors():
        raise RuntimeError("a kernel gave up waiting")
    return torch.stack(ids), torch.stack(lps)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("slots", 8), ("vocab", 32000), ("hidden", 1024), ("tokens", 16), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    if a.hidden % 16:
        ap.error("the hidden width is a multiple of 16")
    ids, lps = decode(a.slots, a.vocab, a.hidden, a.tokens, a.seed)
    for s in range(a.slots):
        print(f"slot {s}: {' '.join(map(str, ids[:, s].tolist()))}   mean log-probability {lps[:, s].mean().item():.3f}")


if __name__ == "__main__":
    main()
