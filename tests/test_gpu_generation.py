"""The page operators, the cached keys and values and the beam selection together, as a program that generates text uses them."""
import math

import pytest
import torch

import device_wide_prefix_amd as dws
from gpu_util import note

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, VOCAB, LAYERS = 4, 2, 32, 101, 2


class Model:
    """Random layers of attention alone, keys and queries turned by their positions."""

    def __init__(self, dtype):
        gen = torch.Generator().manual_seed(1)
        width = HEADS * DIM

        def weights(*shape):
            return (torch.randn(*shape, generator=gen, dtype=torch.float64) / math.sqrt(shape[0])).to(dtype)

        self.embed = weights(VOCAB, width) * math.sqrt(VOCAB)
        self.qkv = [weights(width, (HEADS + 2 * KV) * DIM) * 1.7 for _ in range(LAYERS)]
        self.out = [weights(width, width) for _ in range(LAYERS)]
        self.head = weights(width, VOCAB) * 2
        self.freqs = (100.0 ** (-torch.arange(DIM // 2, dtype=torch.float64) / (DIM // 2))).float()
        self.dtype = dtype

    def split(self, layer, x):
        q, k, v = (x @ self.qkv[layer]).split([HEADS * DIM, KV * DIM, KV * DIM], dim=1)
        return q.view(-1, HEADS, DIM), k.view(-1, KV, DIM), v.view(-1, KV, DIM)

    def on_gpu(self):
        m = Model.__new__(Model)
        m.dtype, m.freqs, m.embed, m.head = self.dtype, self.freqs.cuda(), self.embed.cuda(), self.head.cuda()
        m.qkv, m.out = [x.cuda() for x in self.qkv], [x.cuda() for x in self.out]
        return m

    def logits_of_last(self, tokens):
        """Of the whole text, in 64 bits and without a cache."""
        x = self.embed.double()[tokens]
        n = len(tokens)
        angle = torch.arange(n).double()[:, None, None] * self.freqs.double()
        hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
        for layer in range(LAYERS):
            q, k, v = (x @ self.qkv[layer].double()).split([HEADS * DIM, KV * DIM, KV * DIM], dim=1)
            q, k, v = q.view(n, HEADS, DIM), k.view(n, KV, DIM), v.view(n, KV, DIM)

            def turn(y):
                a, b = y.chunk(2, -1)
                return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)

            q, k = turn(q), turn(k)
            k, v = (y.repeat_interleave(HEADS // KV, 1) for y in (k, v))
            s = torch.einsum("qhd,khd->hqk", q, k) * DIM ** -0.5
            p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
            x = x + torch.einsum("hqk,khd->qhd", p, v).reshape(n, -1) @ self.out[layer].double()
        return x[-1] @ self.head.double()


class Server:
    """A pool of pages of all layers, (layers, pages, 2, kv, page_tokens, dim), and its rows."""

    def __init__(self, model, rows, pages=200, page=8, most=12):
        self.m, self.page = model, page
        self.pool = torch.full((LAYERS, pages, 2, KV, page, DIM), math.nan, dtype=model.dtype, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((rows, most), -1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(rows, dtype=torch.int32, device="cuda")

    def cache(self):
        return self.refs, self.table, self.lengths

    def forward(self, tokens, rows, offsets=None, groups=None, shared=None):
        """Logits of all tokens, appended to rows that were grown for them."""
        x = self.m.embed[tokens]
        for layer in range(LAYERS):
            q, k, v = self.m.split(layer, x)
            keys, values = (self.pool[layer, :, i].transpose(1, 2) for i in (0, 1))
            q = dws.pages_append(keys, values, self.table, self.lengths, k, v, rows=rows, offsets=offsets, freqs=self.m.freqs, q=q)
            o = dws.pages_attention(q, keys, values, self.table, self.lengths, rows=rows, offsets=offsets, groups=groups, shared=shared)
            x = x + o.reshape(len(x), -1) @ self.m.out[layer]
        return x @ self.m.head

    def grow(self, rows, by):
        granted = dws.pages_grow(*self.cache(), rows, self.lengths[rows.long()] + by, page_tokens=self.page)
        assert granted.all()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def beams_of(model, prompts, beams, steps, end):
    """The search with the whole texts computed again at every step, in 64 bits."""
    found = []
    for prompt in prompts:
        live = [(0.0, list(prompt), False)]
        for _ in range(steps):
            options = []
            for w, (score, text, over) in enumerate(live):
                if over:
                    options.append((-score, w, end))
                    continue
                x = torch.log_softmax(model.logits_of_last(torch.tensor(text)), 0)
                options += [(-(score + float(x[t])), w, t) for t in range(VOCAB)]
            options.sort()
            # the choice must not hang on rounding
            assert all(b[0] - a[0] > 1e-4 for a, b in zip(options[:beams], options[1: beams + 1]))
            live = [(-s, live[w][1] + [t], live[w][2] or t == end) for s, w, t in options[:beams]]
        found.append([(score, text) for score, text, _ in live])
    return found


def test_beam_search_over_pages(gpu):
    """Prompts in one packed call, then beams that share them: fork, grow, append, attend, select, and rows reordered by
    freeing and forking. Texts equal those of a search without any cache."""
    note("generation: beam search")
    model, beams, steps, end = Model(torch.float32), 4, 14, 7
    prompts = [[3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5, 8, 9, 7, 9, 3, 2, 3, 8], [2, 7, 1, 8], [1] * 16]
    want = beams_of(model, prompts, beams, steps, end)
    n = len(prompts)
    s = Server(model.on_gpu(), n * beams)
    rows = torch.arange(n * beams, dtype=torch.int32, device="cuda").view(n, beams)
    first = rows[:, 0].contiguous()
    new = ints([len(p) for p in prompts])
    s.grow(first, new)
    offsets = torch.cat([ints([0], torch.int64), new.long().cumsum(0)])
    logits = s.forward(ints(sum(prompts, [])).long(), first, offsets)[offsets[1:] - 1]
    # all beams begin as the first one
    parents = first.repeat_interleave(beams - 1)
    granted, src, dst, count = dws.pages_fork(*s.cache(), parents, rows[:, 1:].reshape(-1).contiguous(), page_tokens=s.page)
    assert granted.all()
    dws.pages_copy(s.pool, src, dst, count, page_dim=1)
    logits = logits[:, None].expand(n, beams, VOCAB)
    scores = torch.full((n, beams), -math.inf, device="cuda")
    scores[:, 0] = 0
    over = torch.zeros(n, beams, dtype=torch.bool, device="cuda")
    texts = torch.zeros(n, beams, 0, dtype=torch.int64, device="cuda")
    groups = torch.arange(0, n * beams + 1, beams, device="cuda")
    shared = ints([len(p) // s.page * s.page for p in prompts])
    for step in range(steps):
        scores, parents, tokens, rows, src, dst = dws.beam_select(logits, scores, finished=over, end_token=end, rows=rows)
        at = parents.long()
        texts = torch.cat([texts.gather(1, at[..., None].expand(-1, -1, step)), tokens[..., None]], 2)
        over = over.gather(1, at) | (tokens == end)
        dws.pages_free(*s.cache(), dst, page_tokens=s.page)
        _, a, b, count = dws.pages_fork(*s.cache(), src, dst, page_tokens=s.page)
        dws.pages_copy(s.pool, a, b, count, page_dim=1)
        flat = rows.reshape(-1)
        s.grow(flat, 1)
        logits = s.forward(tokens.reshape(-1).long(), flat, groups=groups, shared=shared).view(n, beams, VOCAB)
    for i, prompt in enumerate(prompts):
        for w, (score, text) in enumerate(want[i]):
            assert prompt + texts[i, w].tolist() == text
            assert abs(float(scores[i, w]) - score) < 1e-4
    dws.pages_free(*s.cache(), rows.reshape(-1), page_tokens=s.page)
    assert not s.refs.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_in_parts(gpu, dtype):
    """A prompt at once, in parts and token by token, a refused row beside it: the same logits, to the type's rounding."""
    note(f"generation: prompt in parts {dtype}")
    gen = torch.Generator().manual_seed(2)
    text = torch.randint(0, VOCAB, (60,), generator=gen)
    model = Model(dtype)
    want = torch.stack([model.logits_of_last(text[: i + 1]) for i in range(60)])
    for cuts in ([60], [17, 31, 60], list(range(1, 61))):
        s = Server(model.on_gpu(), 3)
        rows = ints([2, -1])
        got, at = [], 0
        for cut in cuts:
            n = cut - at
            granted = dws.pages_grow(*s.cache(), rows, ints([cut, 5]), page_tokens=s.page)
            assert granted.tolist() == [1, 0]
            tokens = torch.cat([text[at: cut], text[:1]]).cuda()
            got.append(s.forward(tokens, rows, ints([0, n, n + 1], torch.int64))[:n])
            at = cut
        off = (torch.cat(got).double().cpu() - want).norm() / want.norm()
        assert off < (1e-5 if dtype == torch.float32 else 0.05), off
