"""Cached keys and values and beam selection from their definitions, in 64 bits, one row and head after another."""
import math
import random

import torch

LOG2E = 1.4426950408889634


class Cache:
    """A pool of pages and the rows in it. Places that no row holds are NaN."""

    def __init__(self, seed, lens, dtype, kv=2, dk=64, dv=64, page=16, layout="heads", shared=None, spare=3, device="cpu"):
        """shared: [(first row, rows, tokens)]: rows that begin with the first one's pages."""
        rng = random.Random(seed)
        gen = torch.Generator().manual_seed(seed)
        self.page, self.lens, self.kv, self.dk, self.dv, self.dtype = page, list(lens), kv, dk, dv, dtype
        of = {}
        for first, rows, tokens in shared or []:
            assert tokens % page == 0
            of.update({r: (first, tokens // page) for r in range(first + 1, first + rows)})
        need = [max(0, -(-n // page) - (of[r][1] if r in of else 0)) for r, n in enumerate(lens)]
        pages = sum(need) + spare
        order = rng.sample(range(pages), pages)
        most = max([-(-n // page) for n in lens] + [1]) + 1
        table, at = [], 0
        for r, n in enumerate(need):
            row = (table[of[r][0]][: of[r][1]] if r in of else []) + order[at: at + n]
            at += n
            table.append(row + [-1] * (most - len(row)))
        self.table = torch.tensor(table, dtype=torch.int32).reshape(len(lens), most).to(device)
        self.lengths = torch.tensor(lens, dtype=torch.int32, device=device)

        def pool(dim):
            if layout == "beside":      # keys and values beside each other in a token's row
                return torch.full((pages, page, kv, dk + dv), math.nan, dtype=dtype)
            x = torch.full((pages, kv, page, dim) if layout == "heads" else (pages, page, kv, dim), math.nan, dtype=dtype)
            return x.transpose(1, 2) if layout == "heads" else x

        if layout == "beside":
            self.pool = pool(0)
            self.keys, self.values = self.pool.split([dk, dv], dim=3)
        else:
            self.keys, self.values = pool(dk), pool(dv)
        for r, n in enumerate(lens):
            for t in range(n):
                p, s = table[r][t // page], t % page
                if r in of and t < of[r][1] * page:
                    continue
                self.keys[p, s] = torch.randn(kv, dk, generator=gen).to(dtype)
                self.values[p, s] = torch.randn(kv, dv, generator=gen).to(dtype)
        if layout == "beside":
            self.pool = self.pool.to(device)
            self.keys, self.values = self.pool.split([dk, dv], dim=3)
        elif device != "cpu":
            self.keys, self.values = (self._moved(x, device, layout) for x in (self.keys, self.values))

    @staticmethod
    def _moved(x, device, layout):
        return x.transpose(1, 2).contiguous().to(device).transpose(1, 2) if layout == "heads" else x.contiguous().to(device)

    def args(self):
        return self.keys, self.values, self.table, self.lengths


def attention(q, keys, values, table, lengths, rows, offsets, scale):
    """(out, lse, spread, largest) in 64 bits: `spread` is the average of |v| with the probabilities, `largest` the largest
    sum of scale |q_d k_d| of a row of queries; for the tolerance. What a query does not see is not touched."""
    q, keys, values = q.double().cpu(), keys.cpu(), values.cpu()
    table, lengths = table.tolist(), lengths.tolist()
    pages, page, kv, _ = keys.shape
    tokens, heads, _ = q.shape
    dv = values.shape[3]
    out = torch.zeros(tokens, heads, dv, dtype=torch.float64)
    spread = torch.zeros_like(out)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    largest = torch.zeros(tokens, heads, dtype=torch.float64)
    for i, row in enumerate(rows):
        b, e = offsets[i], offsets[i + 1]
        if not 0 <= row < len(table) or e - b > lengths[row] or lengths[row] > len(table[row]) * page:
            continue
        n = lengths[row]
        there = [t for t in range(n) if 0 <= table[row][t // page] < pages]
        at = torch.tensor(there, dtype=torch.long)
        p, s = torch.tensor([table[row][t // page] for t in there], dtype=torch.long), at % page
        k, v = keys[p, s].double(), values[p, s].double()
        for j in range(b, e):
            seen = at <= n - (e - j)
            if not seen.any():
                continue
            for h in range(heads):
                g = h // (heads // kv)
                x = scale * (k[seen, g] @ q[j, h])
                lse[j, h] = torch.logsumexp(x, 0)
                w = torch.softmax(x, 0)
                out[j, h] = w @ v[seen, g]
                spread[j, h] = w @ v[seen, g].abs()
                largest[j, h] = abs(scale) * (k[seen, g].abs() @ q[j, h].abs()).max()
    return out, lse, spread, largest


def attention_bound(out, spread, largest, n, dk, dtype):
    """How far an element of the output may be off.

    The result is rounded once: eps / 2 of it. 16-bit probabilities are rounded before their product with the values: eps / 2
    of what they weigh, `spread`. In units u = 2^-24 of fp32: a score's products are summed in at most dk / 2 steps, each off
    by u of a partial sum that is at most `largest`; scaling and the exponent's argument are off by 4 u of it and the
    exponential by 2 u of itself; a sum over n tokens has n / 16 + 16 steps; joining parts costs 8 u more. All of it enters
    the sum of products and the sum of the probabilities."""
    half = torch.finfo(dtype).eps / 2
    u = 2.0 ** -24
    relative = 2 * u * ((dk / 2 + 4) * largest + n / 16 + 16 + 10)
    return half * out.abs() * (1 + half) + (relative[..., None] + (half if dtype != torch.float32 else 0)) * spread * (1 + half) + 1e-30


def turned(x, position, freqs, adjacent):
    """One token's (heads, dim) with its pairs turned, in 64 bits."""
    x = x.double().clone()
    n = freqs.numel()
    if n:
        angle = position * freqs.double()
        a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
        cos, sin, first, second = angle.cos(), angle.sin(), x[:, a].clone(), x[:, b].clone()
        x[:, a], x[:, b] = first * cos - second * sin, first * sin + second * cos
    return x


def select(logits, scores, k, finished=None, end_token=0):
    """(scores, parents, tokens) of the k best, as lists of requests. score + x - norm rises with x, so a beam's own tokens are
    ordered by their logits: 64 bits of the sum would make equal ones of logits that are 1e-30 apart."""
    out = []
    for b in range(logits.shape[0]):
        best = []
        vocab = logits.shape[2]
        for w in range(logits.shape[1]):
            x, s = logits[b, w].double(), float(scores[b, w])
            norm = float(torch.logsumexp(x, 0))
            if finished is not None and finished[b, w]:
                # (its logits are not looked at)
                x, norm = torch.full((vocab,), -math.inf, dtype=torch.float64), 0.0
                x[end_token] = 0.0
            alive = math.isfinite(s) and math.isfinite(norm)
            if not alive:
                x = torch.full((vocab,), -math.inf, dtype=torch.float64)
            order = torch.sort(x, descending=True, stable=True).indices[:k].tolist()
            best += [(-(s + (float(x[t]) - norm)) if alive else math.inf, w, place, t) for place, t in enumerate(order)]
        out.append([(-key, w, t) for key, w, _, t in sorted(best)[:k]])
    return out


def moves(parents, rows):
    """(rows, src, dst) of one request."""
    free, seen = [r for w, r in enumerate(rows) if w not in parents], set()
    new, src, dst = [], [], []
    for p in parents:
        first = p not in seen
        seen.add(p)
        new.append(rows[p] if first else free.pop(0))
        src.append(-1 if first else rows[p])
        dst.append(-1 if first else new[-1])
    return new, src, dst
