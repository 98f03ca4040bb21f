"""A small hybrid decoder: gated delta rule layers with a softmax-attention layer among them,
trained for a few steps and then served from its recurrent states and its paged cache, in 4 or 8
bits, a token a sequence at a time or by beam search.

    python examples/hybrid_decoder.py [--steps 20] [--tokens 64] [--beams 4] [--bits 4]

Training runs gdn_fwd / gdn_bwd and gdn_rope / gdn_rope_bwd on dense batches.  Serving takes
ragged prompts packed in one pass (gdn_fwd_varlen, gdn_kv_append, gdn_kv_attn) and then a token
a sequence at a time (gdn_decode, gdn_kv_append, gdn_kv_attn), the step captured in a CUDA graph.
With --bits 8 the cache is gdn_kv8_append's.  Beam search adds gdn_beam_select and gdn_beam_reorder
to the step: states are lanes of a pool, full pages are shared by the beams.  Random weights,
synthetic tokens.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import gated_deltanet_recurrence_gdn_gb300 as gdn  # noqa: E402


class GdnFn(torch.autograd.Function):
    """gdn_fwd from a zero state, with gdn_bwd as its gradient."""

    @staticmethod
    def forward(ctx, q, k, v, log_alpha, beta):
        ctx.save_for_backward(q, k, v, log_alpha, beta)
        return gdn.gdn_fwd(q, k, v, log_alpha, beta, final_state=False)[0]

    @staticmethod
    def backward(ctx, do):
        q, k, v, log_alpha, beta = ctx.saved_tensors
        return tuple(gdn.gdn_bwd(q, k, v, log_alpha, beta, None, do.contiguous())[:5])


class RopeFn(torch.autograd.Function):
    """gdn_rope of q and k, with gdn_rope_bwd as its gradient."""

    @staticmethod
    def forward(ctx, q, k, cos, sin, pos):
        ctx.save_for_backward(cos, sin, pos)
        return gdn.gdn_rope(q, k, cos, sin, pos)

    @staticmethod
    def backward(ctx, dq, dk):
        return (*gdn.gdn_rope_bwd(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors),
                None, None, None)


class Decoder(torch.nn.Module):
    """Layers "g" (gated delta rule) and "a" (softmax attention with grouped heads)."""

    def __init__(self, layers="gag", vocab=256, width=256, heads=4, kv_heads=2, d=64, max_len=1024,
                 page=16, dtype=torch.bfloat16, device="cuda", seed=0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)
        self.layers, self.heads, self.kv_heads, self.d, self.dtype = layers, heads, kv_heads, d, dtype
        self.max_len, self.page = max_len, page

        def weight(*shape):
            w = torch.randn(*shape, generator=gen) * shape[0] ** -0.5
            return torch.nn.Parameter(w.to(device))

        self.embed = torch.nn.Parameter(torch.randn(vocab, width, generator=gen).to(device))
        self.w = torch.nn.ParameterList()
        for kind in layers:
            # g: q, k, v and the gate and write strength of every head; a: q and the shared k, v
            n = heads * (3 * d + 2) if kind == "g" else (heads + 2 * kv_heads) * d
            self.w += [weight(width, n), weight(heads * d, width)]
        self.cos, self.sin = gdn.gdn_rope_table(max_len, d, device=device)

    def project(self, i, x):
        """The i-th layer's inputs from hidden rows x [..., width], heads in front of d."""
        H, Hk, d = self.heads, self.kv_heads, self.d
        y = F.rms_norm(x, x.shape[-1:]) @ self.w[2 * i]
        if self.layers[i] == "a":
            y = y.unflatten(-1, (H + 2 * Hk, d)).to(self.dtype)
            return y[..., :H, :], y[..., H:H + Hk, :], y[..., H + Hk:, :]
        q, k, v, gates = y.split([H * d] * 3 + [2 * H], -1)
        q, k = (F.normalize(t.unflatten(-1, (H, d)), dim=-1).to(self.dtype) for t in (q, k))
        return (q, k, v.unflatten(-1, (H, d)).to(self.dtype), F.logsigmoid(gates[..., :H] + 2),
                torch.sigmoid(gates[..., H:]))

    def add(self, i, x, o):
        return x + o.flatten(-2).float() @ self.w[2 * i + 1]

    def logits(self, x):
        return F.rms_norm(x, x.shape[-1:]) @ self.embed.t() * x.shape[-1] ** -0.5

    def forward(self, tokens):
        """Logits of dense batches [B, T], with gradients."""
        x = self.embed[tokens]
        pos = torch.arange(tokens.shape[1], dtype=torch.int32, device=x.device)
        for i, kind in enumerate(self.layers):
            p = [t.transpose(1, 2) for t in self.project(i, x)]     # [B, heads, T, d]
            if kind == "g":
                o = GdnFn.apply(*(t.contiguous() for t in p))
            else:
                q, k = RopeFn.apply(p[0], p[1], self.cos, self.sin, pos)
                o = F.scaled_dot_product_attention(q, k, p[2], is_causal=True, enable_gqa=True)
            x = self.add(i, x, o.transpose(1, 2))
        return self.logits(x)


class Serving:
    """States, pages and lengths of `batch` sequences of a decoder, the cache in 4 or 8 bits."""

    def __init__(self, model, batch, bits=4):
        m, dev = model, model.embed.device
        per = -(-m.max_len // m.page)
        self.m, self.batch = m, batch
        pages, self.append, self.attn = {
            4: (gdn.gdn_kv_pages, gdn.gdn_kv_append, gdn.gdn_kv_attn),
            8: (gdn.gdn_kv8_pages, gdn.gdn_kv8_append, gdn.gdn_kv8_attn)}[bits]
        self.state = [torch.zeros(batch, m.heads, m.d, m.d, device=dev) if kind == "g" else
                      pages(batch * per, m.kv_heads, m.page, m.d, device=dev)
                      for kind in m.layers]
        # pages dealt out in turn: a sequence's lie apart
        self.table = torch.arange(batch * per, dtype=torch.int32,
                                  device=dev).view(per, batch).t().contiguous()
        self.len = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.slots = None
        self.graph = None

    def _attend(self, i, p, pos, cu, most, table=None, length=None):
        pages, kw = self.state[i], dict(cu_seqlens=cu)
        at = (self.table if table is None else table, self.len if length is None else length)
        q = self.append(pages, p[1], p[2], *at, q=p[0], cos=self.m.cos, sin=self.m.sin, pos=pos, **kw)
        return self.attn(q, pages, *at, max_new=most, **kw)

    @torch.no_grad()
    def extend(self, tokens, counts):
        """Packed tokens, counts[b] more of every sequence: their logits [sum(counts), vocab]."""
        m, dev = self.m, tokens.device
        n = torch.tensor(counts, dtype=torch.int32, device=dev)
        cu = F.pad(n.cumsum(0), (1, 0)).int()
        pos = (torch.arange(sum(counts), device=dev)
               - (cu[:-1] - self.len).repeat_interleave(n)).int()
        self.len += n
        x = m.embed[tokens]
        for i, kind in enumerate(m.layers):
            p = m.project(i, x)
            if kind == "g":
                p = [t.transpose(0, 1).contiguous() for t in p]
                o, h = gdn.gdn_fwd_varlen(*p, cu, h0=self.state[i])
                self.state[i].copy_(h)
                o = o.transpose(0, 1)
            else:
                o = self._attend(i, p, pos, cu, max(counts))
            x = m.add(i, x, o)
        return m.logits(x)

    def _token(self):
        m = self.m
        pos = self.len.clone()
        self.len += 1
        x = m.embed[self.tokens]
        for i, kind in enumerate(m.layers):
            p = m.project(i, x)
            if kind == "g":
                o = gdn.gdn_decode(*(t.contiguous() for t in p), self.state[i], slots=self.slots)
            else:
                o = self._attend(i, p, pos, None, 1)
            x = m.add(i, x, o)
        return m.logits(x)

    @torch.no_grad()
    def step(self, tokens):
        """One more token of every sequence: its logits [batch, vocab].  The second call captures
        the step, later ones replay it."""
        if self.graph is None:
            self.graph, self.tokens = False, tokens.clone()
            return self._token()
        self.tokens.copy_(tokens)
        if not self.graph:
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self._token()
        self.graph.replay()
        return self.out.clone()


class BeamServing(Serving):
    """Beam search: `batch` prompts with `beams` beams each.  Beam w of prompt b has lane
    slots[b, w], a row of the recurrent layers' pools and of `own`, the pages that it may write."""

    def __init__(self, model, batch, beams, bits=4, eos=None):
        super().__init__(model, batch * beams, bits)
        dev = model.embed.device
        self.groups, self.beams, self.eos = batch, beams, eos
        self.own = self.table.clone()
        self.slots = torch.arange(batch * beams, dtype=torch.int32, device=dev)
        self.scores = torch.zeros(batch, beams, device=dev)
        self.done = torch.zeros(batch, beams, dtype=torch.bool, device=dev)
        self.tokens = torch.zeros(batch * beams, dtype=torch.long, device=dev)
        self.beam = torch.zeros(batch, beams, dtype=torch.int32, device=dev)
        self.made = []                      # (beam that each goes on from, token) of every step

    def _go_on(self, logits, scores, done):
        """The best continuations take the beams' places."""
        kw = {} if self.eos is None else dict(done=done, eos=self.eos)
        best, beam, token = gdn.gdn_beam_select(logits, scores, self.beams, **kw)
        g = [t for t, kind in zip(self.state, self.m.layers) if kind == "g"]
        a = [t for t, kind in zip(self.state, self.m.layers) if kind == "a"]
        slots, table = gdn.gdn_beam_reorder(
            beam, self.slots.view(self.groups, self.beams), states=g, caches=a,
            page_table=self.table, own_pages=self.own, kv_len=self.len, page_size=self.m.page)
        self.slots.copy_(slots.flatten())
        self.table.copy_(table)
        self.scores.copy_(best)
        self.beam.copy_(beam)
        self.tokens.copy_(token.flatten())
        if self.eos is not None:
            self.done.copy_(done.gather(1, beam.long()) | (token == self.eos))

    @torch.no_grad()
    def start(self, tokens, counts):
        """Packed prompts of counts[b] tokens, by the first beam of each; then all go on from it."""
        m, dev = self.m, tokens.device
        n = torch.tensor(counts, dtype=torch.int32, device=dev)
        cu = F.pad(n.cumsum(0), (1, 0)).int()
        pos = (torch.arange(sum(counts), device=dev) - cu[:-1].repeat_interleave(n)).int()
        lane = self.slots.view(self.groups, self.beams)[:, 0].long()
        table = self.table.view(self.groups, self.beams, -1)[:, 0].contiguous()
        x = m.embed[tokens]
        for i, kind in enumerate(m.layers):
            p = m.project(i, x)
            if kind == "g":
                p = [t.transpose(0, 1).contiguous() for t in p]
                o, h = gdn.gdn_fwd_varlen(*p, cu)
                self.state[i][lane] = h
                o = o.transpose(0, 1)
            else:
                o = self._attend(i, p, pos, cu, max(counts), table, n)
            x = m.add(i, x, o)
        self.len.copy_(n.repeat_interleave(self.beams))
        last = m.logits(x)[cu[1:].long() - 1]
        one = torch.zeros(self.groups, 1, device=dev)
        self._go_on(last[:, None], one, one.bool())
        self.made.append((self.beam.clone(), self.tokens.view_as(self.beam).clone()))

    @torch.no_grad()
    def step(self):
        """One more token of every beam.  The second call captures the step, later ones replay it."""
        def body():
            logits = self._token()
            self._go_on(logits, self.scores, self.done)
        if self.graph is None:
            self.graph = False
            body()
        else:
            if not self.graph:
                self.graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(self.graph):
                    body()
            self.graph.replay()
        self.made.append((self.beam.clone(), self.tokens.view_as(self.beam).clone()))

    def sequences(self):
        """The tokens of every beam, [batch, beams, steps], best first."""
        at = torch.arange(self.beams, device=self.beam.device).expand(self.groups, -1)
        out = []
        for beam, token in reversed(self.made):
            out.append(token.gather(1, at))
            at = beam.long().gather(1, at)
        return torch.stack(out[::-1], -1)


def train(model, steps, batch=8, T=256, lr=3e-3, seed=1):
    """Learns to go on with a sequence of period 16; returns the loss of every step."""
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        x = torch.randint(0, 256, (batch, 16), generator=gen).repeat(1, T // 16 + 1)[:, :T + 1]
        x = x.to(model.embed.device)
        loss = F.cross_entropy(model(x[:, :-1]).flatten(0, 1), x[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--bits", type=int, default=4, choices=(4, 8))
    args = ap.parse_args()
    model = Decoder()
    losses = train(model, args.steps)
    print("loss %.3f -> %.3f in %d steps" % (losses[0], losses[-1], args.steps))

    counts = [1, 37, 130, 256]
    gen = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, 256, (n,), generator=gen) for n in counts]
    serve = Serving(model, len(counts), args.bits)
    ends = torch.tensor(counts).cumsum(0) - 1
    logits = serve.extend(torch.cat(prompts).cuda(), counts)[ends.cuda()]
    made = []
    for _ in range(args.tokens):
        made.append(logits.argmax(-1))
        logits = serve.step(made[-1])
    gdn.sync_check()
    made = torch.stack(made, 1).cpu()

    # the same rows from the training pass, whose cache rounds nothing
    worst = 0.0
    for b, p in enumerate(prompts):
        with torch.no_grad():
            want = model(torch.cat([p, made[b]])[None].cuda())[0, -1]
        worst = max(worst, ((logits[b] - want).norm() / want.norm()).item())
    print("%d sequences, %d tokens each; logits against the unrounded pass: %.3f apart"
          % (len(counts), args.tokens, worst))

    search = BeamServing(model, len(counts), args.beams, args.bits)
    search.start(torch.cat(prompts).cuda(), counts)
    for _ in range(args.tokens - 1):
        search.step()
    gdn.sync_check()
    print("%d beams each: best log-probabilities %s" % (args.beams, " ".join(
        "%.2f" % x for x in search.scores[:, 0].tolist())))


if __name__ == "__main__":
    main()
