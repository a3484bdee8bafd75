"""Speculative decoding end to end on the quantized products and the paged 4-bit K/V cache.

A small synthetic decoder (random weights, quantized to 4 bits; its head makes
the next token often a fixed successor of the last one, so that drafts are
right now and then) continues one prompt in several ways at once:

  1. the prompt goes through in pieces of up to 64 tokens, once;
  2. the other sequences fork from it and share its whole pages;
  3. every step drafts two branches of `depth` tokens each from the
     sequence's own history, verifies the tree of 1 + 2 * depth rows in one
     pass (products of M = sequences * rows, rotary positions, append,
     attention under the tree's mask, gated blocks, the likeliest tokens with
     their log probabilities), accepts the longer branch, and appends its keys
     and values again, now in a row: what was rejected lies behind the length;
  4. half of the sequences end, their pages are freed and the rest compacted,
     and the others go on.

With a window, the layers attend to the last tokens and the first few only.
Nothing in a step waits for the device.  ``python -m
affine_quantized_gemm_amd.spec_decode --help`` for the sizes.
"""

from __future__ import annotations

import argparse
import time

import torch

import affine_quantized_gemm_amd as Q

BITS, GROUP = 4, 64


class Decoder:
    """Weights of a decoder with shared kv heads, gated MLP and rotary positions."""

    def __init__(self, layers=2, hidden=1024, heads=8, kv_heads=2, head_dim=128, ffn=2048, vocab=2048,
                 dtype=torch.bfloat16, cycle=13, habit=7.0, seed=0, window=None, sinks=0):
        self.layers, self.heads, self.kv_heads, self.head_dim, self.dtype = layers, heads, kv_heads, head_dim, dtype
        if sinks and window is None:
            raise ValueError("sinks need a window")
        self.window, self.sinks = window, sinks
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
        weight = lambda n, k: Q.quantize((rand(n, k) * k ** -0.5).to(dtype), BITS, GROUP)
        self.qkv = [weight((heads + 2 * kv_heads) * head_dim, hidden) for _ in range(layers)]
        self.o = [weight(hidden, heads * head_dim) for _ in range(layers)]
        self.gate_up = [weight(2 * ffn, hidden) for _ in range(layers)]
        self.down = [weight(hidden, ffn) for _ in range(layers)]
        self.embedding = rand(vocab, hidden).to(dtype)
        # logits of deviation 1, to which t + 1 (or the first of t's `cycle` tokens) adds `habit` after token t
        t = torch.arange(vocab, device="cuda")
        before = torch.where(t % cycle == 0, (t + cycle - 1).clamp(max=vocab - 1), t - 1)
        head = rand(vocab, hidden) + habit * hidden ** -0.5 * self.embedding[before].float()
        self.head = Q.quantize((head * hidden ** -0.5).to(dtype), BITS, GROUP)
        self.freq = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda") / head_dim)

    def cache(self, pages: int, page_size: int = 64) -> Q.KVCache:
        return Q.KVCache.empty(self.layers, pages, self.kv_heads, self.head_dim, GROUP, page_size, self.dtype)

    def _mul(self, x, w):
        return Q.small_m(x, *w, BITS, GROUP)

    def _norm(self, x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(self.dtype)

    def forward(self, cache, tokens, positions, tables, lens, mask=None, max_len=None):
        """New tokens (at most 64, as many for each sequence) through all layers: logits, and every layer's k and v."""
        rows, H, kv = tokens.shape[0], self.heads, []
        x = self.embedding[tokens]
        for layer in range(self.layers):
            qkv = self._mul(self._norm(x), self.qkv[layer]).view(rows, H + 2 * self.kv_heads, self.head_dim)
            q, k, v = qkv.split([H, self.kv_heads, self.kv_heads], 1)
            turned = qkv[:, :H + self.kv_heads]
            Q.rotary(turned, positions, self.freq, out=turned)  # q and k, in place
            cache.append(layer, k, v, tables, lens)
            y = cache.attend(layer, q, tables, lens, mask=mask, max_len=max_len, window=self.window, sinks=self.sinks)
            x = x + self._mul(y.view(rows, -1), self.o[layer])
            x = x + self._mul(Q.gated(self._norm(x), *self.gate_up[layer], BITS, GROUP), self.down[layer])
            kv.append((k, v))
        return self._mul(self._norm(x), self.head), kv


class Sequences:
    """Page tables, lengths and histories of a batch that shares one cache."""

    def __init__(self, model: Decoder, seqs: int, most_tokens: int, depth: int = 3, page_size: int = 64):
        width = -(-most_tokens // page_size)
        int32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
        self.model, self.cache, self.most = model, model.cache(seqs * width, page_size), width * page_size
        self.tables, self.lens, self.refs = int32(seqs, width) - 1, int32(seqs), int32(seqs * width)
        self.history = torch.zeros(seqs, most_tokens + 64, dtype=torch.int64, device="cuda")
        self.said = torch.zeros(seqs, most_tokens + 64, device="cuda")     # the tokens' log probabilities (the first's is 0)
        self.tokens = torch.zeros(seqs, dtype=torch.int64, device="cuda")  # in the history; the last is not cached yet
        self.sound = torch.ones((), dtype=torch.int32, device="cuda")     # every page asked for was there
        self.least = torch.zeros((), dtype=torch.int64, device="cuda")    # -1: a token was picked from NaN or infinite logits
        # the draft tree: rows 0, 1..depth and depth + 1..2 * depth, what each sees, and its two paths
        self.depth, branch = depth, range(1, depth + 1)
        self.level = torch.tensor([0, *branch, *branch], device="cuda")
        self.sees = torch.tensor([1, *((2 << i) - 1 for i in branch),
                                  *(1 | ((1 << i) - 1) << (depth + 1) for i in branch)], device="cuda")
        self.paths = torch.tensor([[0, *branch], [0, *(depth + i for i in branch)]], device="cuda")
        self.branch = torch.tensor([*branch], device="cuda")

    def _reserve(self, tables, lens, add: int):
        ok = self.cache.reserve(tables, lens, self.refs, torch.full_like(lens, add))
        self.sound = torch.minimum(self.sound, ok.min())

    def prefill(self, prompt: torch.Tensor) -> torch.Tensor:
        """The prompt into sequence 0; logits of all its tokens."""
        out, tables, lens = [], self.tables[:1], self.lens[:1]
        for at in range(0, prompt.numel(), 64):
            piece = prompt[at:at + 64]
            self._reserve(tables, lens, piece.numel())
            positions = torch.arange(at, at + piece.numel(), device="cuda")
            out.append(self.model.forward(self.cache, piece, positions, tables, lens, max_len=self.most)[0])
        logits = torch.cat(out)
        self.history[0, :prompt.numel()] = prompt
        self.said[0, 1:prompt.numel()] = Q.log_probs(logits[:-1], prompt[1:]).tokens
        self.tokens[0] = prompt.numel()
        return logits

    def fork(self, logits: torch.Tensor) -> None:
        """All other sequences from sequence 0, each with another of the likeliest next tokens."""
        seqs = self.lens.numel()
        if seqs > 1:
            dst = torch.arange(1, seqs, dtype=torch.int32, device="cuda")
            ok = self.cache.fork(self.tables, self.lens, self.refs, torch.zeros_like(dst), dst)
            self.sound = torch.minimum(self.sound, ok.min())
        self.history[1:], self.tokens[1:] = self.history[0].clone(), self.tokens[0].clone()
        self.said[1:] = self.said[0].clone()
        first = Q.log_probs(logits[None], top=seqs)
        self.least = torch.minimum(self.least, first.top_ids.min())
        self.history.scatter_(1, self.tokens[:, None], first.top_ids.T.clamp(min=0))
        self.said.scatter_(1, self.tokens[:, None], first.top_values.T)
        self.tokens += 1

    def _drafts(self):
        """[seqs, depth] twice: what followed the last token where it stood last before, and where it stood first."""
        most = self.history.shape[1]
        at = torch.arange(most, device="cuda")
        stood = (self.history == self.history.gather(1, self.tokens[:, None] - 1)) & (at < self.tokens[:, None] - 1)
        late, early = torch.where(stood, at, -1).amax(1), torch.where(stood, at, most).amin(1)
        return [self.history.gather(1, (i[:, None] + self.branch).clamp(0, most - 1)) for i in (late, early)]

    def step(self) -> None:
        """One draft tree of 1 + 2 * depth rows a sequence: verified, its longer right branch kept."""
        seqs, R = self.lens.numel(), self.level.numel()
        root = self.history.gather(1, self.tokens[:, None] - 1)
        tree = torch.cat([root, *self._drafts()], 1)
        start = self.lens.clone()
        self._reserve(self.tables, self.lens, R)
        positions = (start[:, None] + self.level).flatten()
        logits, kv = self.model.forward(self.cache, tree.flatten(), positions, self.tables, self.lens,
                                        self.sees.repeat(seqs), self.most)
        likeliest = Q.log_probs(logits, top=1)
        picks, said = likeliest.top_ids.view(seqs, R), likeliest.top_values.view(seqs, R)
        # a draft is right if its parent's pick is that token
        right = [(tree[:, p[1:]] == picks[:, p[:-1]]).long().cumprod(1).sum(1) for p in self.paths]
        path, kept = self.paths[(right[1] > right[0]).long()], torch.maximum(*right)
        # the branch's keys and values next to the root's (past the kept ones: places of the next step)
        rows = (path + R * torch.arange(seqs, device="cuda")[:, None]).flatten()
        self.lens.copy_(start + self.depth + 1)
        for layer, (k, v) in enumerate(kv):
            self.cache.append(layer, k[rows], v[rows], self.tables, self.lens)
        self.lens.copy_(start + kept + 1)
        places = self.tokens[:, None] + torch.arange(self.depth + 1, device="cuda")
        taken = picks.gather(1, path)
        self.least = torch.minimum(self.least, torch.where(places <= self.tokens[:, None] + kept[:, None], taken, 0).min())
        self.history.scatter_(1, places, taken.clamp_(min=0))
        self.said.scatter_(1, places, said.gather(1, path))
        self.tokens += kept + 1

    def end(self, which: list[int]) -> None:
        """The sequences' pages freed, the others' packed together, their rows taken out."""
        self.cache.free(self.tables, self.lens, self.refs, torch.tensor(which, dtype=torch.int32, device="cuda"))
        self.tables, self.refs = self.cache.compact(self.tables, self.refs)[:2]
        keep = [i for i in range(self.lens.numel()) if i not in which]
        self.tables, self.lens = self.tables[keep].contiguous(), self.lens[keep]
        self.history, self.said, self.tokens = self.history[keep], self.said[keep], self.tokens[keep]

    def texts(self) -> list[list[int]]:
        """Every sequence's tokens so far."""
        assert int(self.sound) == 1, "the cache has too few pages"
        assert int(self.least) == 0, "a token's logits were NaN or infinite"
        return [row[:n] for row, n in zip(self.history.tolist(), self.tokens.tolist())]

    def scores(self) -> list[list[float]]:
        """The log probability with which every one of those tokens came (the first's is 0)."""
        return [row[:n] for row, n in zip(self.said.tolist(), self.tokens.tolist())]


def logits_of(model: Decoder, tokens: list[int]) -> torch.Tensor:
    """Logits after each of the tokens, without drafts, in a cache of their own."""
    s = Sequences(model, 1, len(tokens))
    return s.prefill(torch.tensor(tokens, device="cuda"))


def main(argv=None) -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--seqs", type=int, default=4)
    p.add_argument("--prompt", type=int, default=200, help="tokens")
    p.add_argument("--steps", type=int, default=40, help="before half of the sequences end, and after")
    p.add_argument("--depth", type=int, default=3, help="drafted tokens of a branch")
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--ffn", type=int, default=14336)
    p.add_argument("--dtype", choices=["f16", "bf16"], default="bf16")
    p.add_argument("--window", type=int, default=0, help="tokens that a row attends to (0: all)")
    p.add_argument("--sinks", type=int, default=0, help="first tokens that it attends to besides")
    a = p.parse_args(argv)
    if a.seqs * (1 + 2 * a.depth) > 64:
        p.error("seqs * (1 + 2 * depth) rows: at most 64")
    if a.window < 0 or a.sinks < 0 or a.sinks and not a.window:
        p.error("window and sinks: 0 or more, and sinks only with a window")
    model = Decoder(a.layers, a.hidden, a.heads, a.kv_heads, a.hidden // a.heads, a.ffn,
                    dtype=torch.float16 if a.dtype == "f16" else torch.bfloat16,
                    window=a.window or None, sinks=a.sinks)
    s = Sequences(model, a.seqs, a.prompt + 1 + (2 * a.steps + 3) * (1 + 2 * a.depth), a.depth)
    prompt = torch.randint(0, model.embedding.shape[0], (a.prompt,), generator=torch.Generator().manual_seed(1)).cuda()
    s.fork(s.prefill(prompt)[-1])
    for part in range(2):
        s.step()
        torch.cuda.synchronize()
        before, t0 = s.tokens.clone(), time.perf_counter()
        for _ in range(a.steps):
            s.step()
        torch.cuda.synchronize()
        dt, n = time.perf_counter() - t0, int((s.tokens - before).sum())
        seqs = s.lens.numel()
        print(f"{seqs} sequences, {seqs * (1 + 2 * a.depth)} rows a step: {1e3 * dt / a.steps:.2f} ms a step, "
              f"{n / a.steps / seqs:.2f} tokens a step and sequence, {n / dt:.0f} tokens/s")
        if part == 0 and seqs > 1:
            s.end(list(range(seqs // 2, seqs)))
    for text, said in zip(s.texts(), s.scores()):
        said = said[a.prompt:]
        print(f"  ... {text[a.prompt:a.prompt + 16]} ({len(text)} tokens, {sum(said) / len(said):.2f} nats each)")


if __name__ == "__main__":
    main()
