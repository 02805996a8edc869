"""Serving a small KDA:GQA hybrid (three KDA layers, one softmax-attention
layer, and so on) with random weights: prompts packed together, decode steps,
samples forked from one prompt, ended sequences released and the cache
compacted.

Every sequence-mixing step runs in the library: the chunk scan and the decode
step of the KDA layers with the norm and gate of their outputs, the paged
key-value cache of the others, and the residual sums with the norms between
layers.  The projections around them are plain matrix products.

    python examples/serve_hybrid.py [--layers 8] [--steps 32] [--cache e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gated_delta_rule_41_gb300 as kda  # noqa: E402

BF16 = torch.bfloat16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Hybrid:
    """Weights, and the state of up to ``rows`` sequences: per KDA layer the
    recurrent states, per attention layer a pair of page pools, and one block
    table for all of them."""

    def __init__(self, layers=8, width=512, heads=4, kv_heads=2, head=64, vocab=1000, rows=16,
                 pages=256, page=16, max_pages=64, cache="bf16", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[0] ** -0.5).to(BF16)

        self.H, self.HKV, self.D, self.rows = heads, kv_heads, head, rows
        self.emb = w(vocab, width)
        self.layers = []
        pools = []
        for i in range(layers):
            n = heads * head
            if i % 4 != 3:
                self.layers.append(dict(kind="kda", qkv=w(width, 3 * n), g=w(width, n),
                                        beta=w(width, heads), out=w(n, width), z=w(width, n),
                                        norm=torch.ones(head, device="cuda"),
                                        state=torch.zeros(rows, heads, head, head, device="cuda")))
            else:
                t = BF16 if cache == "bf16" else torch.float8_e4m3fn
                k, v = (torch.zeros(pages, page, kv_heads, head, device="cuda").to(t)
                        for _ in range(2))
                # what a code is worth: values of a few units on a scale of 448
                s = None if cache == "bf16" else torch.full((kv_heads,), 1 / 32, device="cuda")
                pools += [k, v]
                self.layers.append(dict(kind="attn", qkv=w(width, n + 2 * kv_heads * head),
                                        out=w(n, width),
                                        kv=kda.KVPages(k, v, k_scale=s, v_scale=s)))
        self.book = kda.PageBook(pages, page, pools)
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        # tokens that rows gained in this step: none where the pages ran out
        self.granted = torch.zeros(rows, dtype=torch.int32, device="cuda")
        first = next(l for l in self.layers if l["kind"] == "attn")["kv"]
        self.ws = kda.paged_decode_workspace(first, rows, heads)

    def _gated(self, l, o, y):
        """The norm of a KDA layer's output with its gate, per head."""
        z = (y @ l["z"]).view(-1, self.H, self.D)
        return kda.gated_norm_fwd(o.reshape(z.shape), z, l["norm"], eps=1e-6)

    def _run(self, x, mix):
        """The layers on token embeddings: each mixes the norm of the residual stream and adds
        to it; ``mix(layer, y)`` gives a layer's heads.  Returns the norm of the stream behind the last."""
        x, y = kda.add_norm_fwd(x, None, eps=1e-6)
        for l in self.layers:
            o = mix(l, y)
            x, y = kda.add_norm_fwd(x, o.reshape(x.shape[0], -1) @ l["out"], eps=1e-6, out_residual=x)
        return y

    def _kda_inputs(self, l, x):
        n, H, D = x.shape[0], self.H, self.D
        q, k, v = (x @ l["qkv"]).view(n, 3, H, D).unbind(1)
        g = -torch.nn.functional.softplus((x @ l["g"]).float()).to(BF16).view(n, H, D)
        return q.contiguous(), k.contiguous(), v.contiguous(), g, torch.sigmoid(x @ l["beta"])

    def prompts(self, slots, tokens):
        """Run new prompts (lists of token ids) in idle rows; logits of each
        one's last token."""
        n = [len(t) for t in tokens]
        add = [0] * self.rows
        cu = [0] * (self.rows + 1)
        order = sorted(range(len(slots)), key=lambda i: slots[i])   # packed by row
        for i in order:
            add[slots[i]] = n[i]
        for s in range(self.rows):
            cu[s + 1] = cu[s] + add[s]
        ids = torch.tensor([t for i in order for t in tokens[i]], device="cuda")
        cu = ints(cu)
        self.book.extend(ints(add), self.table, self.lens, self.refs, granted=self.granted)

        def mix(l, y):
            if l["kind"] == "attn":
                return self._attend(l, y, cu)
            q, k, v, g, beta = (t[None] for t in self._kda_inputs(l, y))
            o, ht = kda.chunk_kda_fwd_varlen(q, k, v, g, beta, cu, output_final_state=True,
                                             use_qk_l2norm_in_kernel=True)
            rows = torch.tensor(slots, device="cuda")
            l["state"][rows] = ht[rows]
            return self._gated(l, o[0], y)

        y = self._run(self.emb[ids], mix)
        last = torch.tensor([sum(add[:s]) + add[s] - 1 for s in slots], device="cuda")
        return y[last].float() @ self.emb.float().T

    def _attend(self, l, y, cu=None):
        H, HKV, D = self.H, self.HKV, self.D
        qkv = (y @ l["qkv"]).view(y.shape[0], H + 2 * HKV, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + HKV], qkv[:, H + HKV:]
        kda.paged_append(l["kv"], k, v, self.table, self.lens, cu, granted=self.granted)
        if cu is not None:
            return kda.paged_prefill(q, l["kv"], self.table, self.lens, cu)
        return kda.paged_decode(q, l["kv"], self.table, self.lens, workspace=self.ws)

    def step(self, ids):
        """One token for each row (idle rows go along); logits [rows, vocab]."""
        self.book.extend(1, self.table, self.lens, self.refs, granted=self.granted)

        def mix(l, y):
            if l["kind"] == "attn":
                return self._attend(l, y)
            o = kda.recurrent_step(*self._kda_inputs(l, y), l["state"], use_qk_l2norm_in_kernel=True)
            return self._gated(l, o, y)

        return self._run(self.emb[ids], mix).float() @ self.emb.float().T

    def fork(self, parents, children):
        p, c = ints(parents), ints(children)
        self.book.fork(p, c, self.table, self.lens, self.refs)
        kda.pages_copy([l["state"] for l in self.layers if l["kind"] == "kda"], p, c)

    def release(self, slots):
        self.book.free(ints(slots), self.table, self.lens, self.refs)
        self.book.compact(self.table, self.lens, self.refs)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    args = ap.parse_args(argv)
    m = Hybrid(layers=args.layers, cache=args.cache)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1000, (n,), generator=g).tolist() for n in (300, 45, 7)]
    logits = m.prompts([0, 1, 2], prompts)
    m.fork([0, 0, 1], [5, 6, 7])                       # two more samples of prompt 0, one of 1
    ids = torch.zeros(m.rows, dtype=torch.long, device="cuda")
    for slot, row in ((0, 0), (1, 1), (2, 2), (5, 0), (6, 0), (7, 1)):
        ids[slot] = torch.multinomial(torch.softmax(logits[row], -1), 1)[0]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(args.steps):
        ids = torch.multinomial(torch.softmax(m.step(ids), -1), 1)[:, 0]
        if i == args.steps // 2:
            m.release([1, 5])
    torch.cuda.synchronize()
    kda.check()
    held = int((m.refs > 0).sum())
    ms = (time.perf_counter() - t) / args.steps * 1e3
    print(f"{args.steps} steps of {args.layers} layers, {ms:.2f} ms each; "
          f"lengths {m.lens.tolist()}, {held} pages held")


if __name__ == "__main__":
    main()
