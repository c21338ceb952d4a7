"""Cases and plain forms of the operators that write, read and reorder a paged cache while tokens are generated.

A cache of keys and values lies in pages: ``table[row]`` lists the pages of a row and ``lengths[row]`` its tokens, the
latest included, so that token t of a row is at place ``t % page_tokens`` of page ``table[row][t // page_tokens]``. The
tokens of a call are packed, sequence after sequence, and are the last ones of their rows.

- ``append`` writes the keys and values of the tokens into the pages. Pairs of the first ``rot`` dimensions of keys and
  queries are turned by the angle position * freqs[pair] on the way.
- ``attend`` is attention of the tokens' queries with everything in their rows up to their own position,

      out = sum_t p_t v_t,   p = softmax over t <= position of scale q . k_t

  Sequences come in groups whose first ``shared`` tokens are in the same pages, as rows forked from one prompt have them.
- ``select`` extends beams: of all (beam, token) pairs of a request the k with the largest
  score[beam] + log_softmax(logits[beam])[token], the lowest index first among equal ones. A finished beam goes on with
  the end token alone, at its score. Rows (of the cache, or of states) go on with a beam's first continuation; further
  ones take the rows of beams that end, into which ``src`` has to be copied.

With ``own`` false run() computes all of it with elementary torch operations; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # one new token of one sequence of a small model: nothing but latency
        {"name": "append_one", "kind": "append", "seqs": 1, "low": 1, "high": 1, "lens": 1, "far": 900, "heads": 8, "kv": 2,
         "dk": 64, "dv": 64, "rot": 64, "adjacent": False, "page": 16, "layout": "heads", "pads": 0, "type": "bf16"},
        # a token for each sequence of a full batch, half of each head turned, in adjacent pairs, far positions
        {"name": "append_batch", "kind": "append", "seqs": 256, "low": 1, "high": 1, "lens": 2, "far": 100000, "heads": 32,
         "kv": 8, "dk": 128, "dv": 128, "rot": 64, "adjacent": True, "page": 16, "layout": "tokens", "pads": 3, "type": "fp16"},
        # packed prompts of unequal lengths, the first of them behind tokens that are there already
        {"name": "append_prompts", "kind": "append", "seqs": 9, "low": 100, "high": 5000, "lens": 3, "far": 5000, "heads": 32,
         "kv": 8, "dk": 128, "dv": 128, "rot": 128, "adjacent": False, "page": 16, "layout": "heads", "pads": 0, "type": "bf16"},
        # one token of one short sequence: latency
        {"name": "attend_one", "kind": "attend", "groups": 1, "members": 1, "low": 1, "high": 1, "prefix": "0,0",
         "behind": "700,700", "lens": 1, "heads": 8, "kv": 2, "dk": 64, "dv": 64, "page": 16, "layout": "heads", "pads": 0,
         "type": "bf16"},
        # a token for each sequence of a batch that shares nothing, of very unequal lengths, some places empty
        {"name": "attend_ragged", "kind": "attend", "groups": 96, "members": 1, "low": 1, "high": 1, "prefix": "0,0",
         "behind": "1,16000", "lens": 2, "heads": 32, "kv": 8, "dk": 128, "dv": 128, "page": 16, "layout": "heads", "pads": 3,
         "type": "bf16"},
        # a batch that answers questions about one long text
        {"name": "attend_shared", "kind": "attend", "groups": 1, "members": 64, "low": 1, "high": 1, "prefix": "32773,32773",
         "behind": "1,600", "lens": 3, "heads": 32, "kv": 8, "dk": 128, "dv": 128, "page": 16, "layout": "heads", "pads": 0,
         "type": "bf16"},
        # beams of some requests, each request with its own prompt
        {"name": "attend_beams", "kind": "attend", "groups": 12, "members": 8, "low": 1, "high": 1, "prefix": "300,6000",
         "behind": "1,40", "lens": 4, "heads": 24, "kv": 4, "dk": 96, "dv": 96, "page": 32, "layout": "tokens", "pads": 0,
         "type": "fp16"},
        # the prompts of three requests, computed behind a text that they share
        {"name": "attend_prompts", "kind": "attend", "groups": 1, "members": 3, "low": 900, "high": 2000, "prefix": "4097,4097",
         "behind": "0,100", "lens": 5, "heads": 32, "kv": 8, "dk": 128, "dv": 128, "page": 16, "layout": "heads", "pads": 0,
         "type": "bf16"},
        # a few drafted tokens a sequence, in 32 bits, with odd pages and head dimensions
        {"name": "attend_fp32_odd", "kind": "attend", "groups": 2, "members": 5, "low": 1, "high": 4, "prefix": "99,700",
         "behind": "1,90", "lens": 6, "heads": 6, "kv": 3, "dk": 72, "dv": 40, "page": 7, "layout": "tokens", "pads": 1,
         "type": "fp32"},
        # the beams of one request
        {"name": "select_one", "kind": "select", "batch": 1, "beams": 4, "k": 4, "vocab": 32000, "type": "fp32"},
        # a full batch with a large vocabulary, twice as many candidates as beams
        {"name": "select_batch", "kind": "select", "batch": 64, "beams": 8, "k": 16, "vocab": 131071, "type": "bf16"},
        # wide beams, whose rows are reordered
        {"name": "select_wide", "kind": "select", "batch": 5, "beams": 32, "k": 32, "vocab": 50001, "type": "fp16"},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.99)))))))


def _cost(case):
    """About the time of the floor, in units of a byte."""
    w = work(case)
    return max(w["bytes"], w["flops"] / (200 if case["type"] != "fp32" else 25))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "select"])
    most = max(_cost(c) for c in listed() if c["kind"] == kind)
    t = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if kind == "select":
        while True:
            beams = _log_int(rng, 1, 32)
            case = {"kind": kind, "batch": _log_int(rng, 1, 64), "beams": beams, "k": beams * rng.choice([1, 1, 2]),
                    "vocab": _log_int(rng, 1000, 150000), "type": t}
            if _cost(case) <= most:
                return case
    kv = rng.choice([1, 2, 3, 4, 8, 8])
    head = rng.choice([64, 128, 128, 96, 80, 256, 8 * rng.randint(2, 32), rng.randint(16, 200)])
    case = {"kind": kind, "heads": kv * rng.choice([1, 2, 3, 4, 4, 8]), "kv": kv, "dk": head,
            "dv": rng.choice([head, head, head, 64, 8 * rng.randint(2, 32)]), "page": rng.choice([16, 16, 32, 64, 1, rng.randint(2, 100)]),
            "layout": rng.choice(["heads", "tokens"]), "type": t, "lens": rng.randint(10, 1000000)}
    while True:
        if kind == "append":
            seqs = _log_int(rng, 1, 256)
            low, high = (1, 1) if rng.random() < 0.4 else (1, _log_int(rng, 4, 5000))
            case.update(seqs=seqs, low=low, high=high, far=_log_int(rng, 16, 100000), rot=rng.choice([head // 2 * 2, head // 4 * 2]),
                        adjacent=rng.random() < 0.5, pads=rng.randint(0, seqs // 16))
        else:
            groups, members = (1, _log_int(rng, 1, 64)) if rng.random() < 0.5 else (_log_int(rng, 1, 96), _log_int(rng, 1, 8))
            low, high = (1, 1) if rng.random() < 0.6 else ((1, rng.randint(2, 8)) if rng.random() < 0.6 else (1, _log_int(rng, 10, 2000)))
            first, behind = _log_int(rng, 1, 32000), _log_int(rng, 1, 16000)
            case.update(groups=groups, members=members, low=low, high=high,
                        prefix="%d,%d" % (first, _log_int(rng, first, 33000)) if members > 1 else "0,0",
                        behind="%d,%d" % (rng.randint(0, behind), behind), pads=rng.randint(0, groups * members // 16))
        if _cost(case) <= most and _plain_bytes(case) < 24e9:
            return case


def _plain_bytes(case):
    """What the plain form of attention holds of scores, keys and values behind the shared tokens."""
    if case["kind"] == "append":
        return 0
    groups = _lengths(case)
    n = sum(len(m) for _, m in groups)
    own_tokens = max(length for _, m in groups for _, length in m)
    new = max(t for _, m in groups for t, _ in m)
    first = max(p for p, _ in groups)
    return 4 * n * (own_tokens * (case["kv"] * (case["dk"] + case["dv"]) + 3 * case["heads"] * new) + 3 * case["heads"] * new * first)


def _lengths(case):
    """The case's groups: [(shared tokens, [(new tokens, tokens behind the shared ones, new ones included), ...]), ...].
    Only whole pages are shared; the rest of the prefix lies in each row's own pages."""
    rng, page = random.Random(case["lens"]), case["page"]

    def between(low, high):
        return _log_int(rng, max(1, low), max(1, high)) if high else 0

    if case["kind"] == "append":
        out = []
        for _ in range(case["seqs"]):
            new = between(case["low"], case["high"])
            out.append((0, [(new, new + rng.randint(0, case["far"]))]))
        return out
    low, high = (int(x) for x in case["prefix"].split(","))
    behind = [int(x) for x in case["behind"].split(",")]
    out = []
    for _ in range(case["groups"]):
        prefix = between(low, high)
        shared = prefix // page * page if case["members"] > 1 else 0
        members = []
        for _ in range(case["members"]):
            new = between(case["low"], case["high"])
            members.append((new, prefix - shared + between(*behind) + new))
        out.append((shared, members))
    return out


# ---- the inputs --------------------------------------------------------------

def _pool(gen, case, pages):
    """(keys, values) of one layer, (pages, page_tokens, heads, dim) views of a pool; its pages hold old values."""
    dev, t = _device(), _TYPES[case["type"]]
    out = []
    for dim in (case["dk"], case["dv"]):
        shape = (pages, case["kv"], case["page"], dim) if case["layout"] == "heads" else (pages, case["page"], case["kv"], dim)
        x = torch.empty(shape, dtype=t, device=dev)
        for part in x.split(max(1, (1 << 27) // max(1, x[0].numel()))):
            part.copy_(torch.randn(part.shape, generator=gen, device=dev))
        out.append(x.transpose(1, 2) if case["layout"] == "heads" else x)
    return out


def _rows_of(gen, case, state):
    """The table, lengths and places of the case's sequences in a cache of some more rows and pages. (Where tokens are
    only appended, one page stands for all those before them: their values do not matter, and the pool stays small.)"""
    dev, page = _device(), case["page"]
    groups = _lengths(case)
    n = sum(len(m) for _, m in groups)
    pages = [(shared // page, [-(-length // page) for _, length in m]) for shared, m in groups]
    before = [(m[0][1] - m[0][0]) // page if case["kind"] == "append" else 0 for _, m in groups]
    need = sum(s + sum(own) - gone for (s, own), gone in zip(pages, before))
    most = max(s + max(own) for s, own in pages) + 1
    count = need + 7
    order = torch.randperm(count, generator=gen, device=dev).to(torch.int32).cpu()
    rows = torch.randperm(n + 3, generator=gen, device=dev)[:n].to(torch.int32).cpu()
    table = torch.full((n + 3, most), -1, dtype=torch.int32)
    lengths = torch.zeros(n + 3, dtype=torch.int32)
    at = i = 0
    for (shared, members), (first, own), gone in zip(groups, pages, before):
        prefix = order[at: at + first]
        at += first
        for (_, length), more in zip(members, own):
            r = int(rows[i])
            table[r, :first] = prefix
            table[r, :gone] = order[-1]
            table[r, first + gone: first + more] = order[at: at + more - gone]
            lengths[r] = shared + length
            at += more - gone
            i += 1
    live = torch.ones(n, dtype=torch.bool)
    if case["pads"]:        # empty places of a batch of fixed size
        live[torch.randperm(n, generator=gen, device=dev)[: case["pads"]].cpu()] = False
    new = [t for _, m in groups for t, _ in m]
    offsets = torch.tensor([0] + new, dtype=torch.int64).cumsum(0)
    with_row = torch.repeat_interleave(live, torch.tensor(new)).nonzero().reshape(-1)
    state.update(table=table.to(dev), lengths=lengths.to(dev), rows=torch.where(live, rows, -1).to(torch.int32).to(dev),
                 offsets=offsets.to(dev), live=live.tolist(), with_row=with_row.to(dev), groups=groups, new=new, n=n,
                 pages=count, page=page)
    return sum(new)


def prepare(case, seed):
    dev, t = _device(), _TYPES[case["type"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    state = {"kind": case["kind"]}
    if case["kind"] == "select":
        b, w, v = case["batch"], case["beams"], case["vocab"]
        logits = torch.empty(b, w, v, dtype=t, device=dev)
        for part in logits:
            part.copy_(2.5 * normal(w, v))
        state.update(logits=logits, scores=-5 - 0.7 * normal(b, w).abs().cumsum(1), k=case["k"],
                     finished=torch.rand(b, w, generator=gen, device=dev) < 0.1, end=v // 3)
        if case["k"] == w:
            state["rows"] = torch.randperm(b * w + 5, generator=gen, device=dev)[: b * w].to(torch.int32).reshape(b, w)
        return state
    tokens = _rows_of(gen, case, state)
    state["keys"], state["values"] = _pool(gen, case, state["pages"])
    heads, kv, dk, dv = case["heads"], case["kv"], case["dk"], case["dv"]
    if case["kind"] == "append":
        # queries, keys and values are parts of one projection's output, as they are in a model
        parts = normal(tokens, heads * dk + kv * dk + kv * dv).to(t).split([heads * dk, kv * dk, kv * dv], dim=1)
        state.update(q=parts[0].view(tokens, heads, dk), k=parts[1].view(tokens, kv, dk), v=parts[2].view(tokens, kv, dv))
        pairs = torch.arange(case["rot"] // 2, device=dev, dtype=torch.float32)
        state.update(freqs=10000.0 ** (-2 * pairs / max(1, case["rot"])), adjacent=case["adjacent"])
        return state
    state.update(q=(1.5 * normal(tokens, heads, dk)).to(t), scale=dk ** -0.5)
    ends = [0]
    for _, members in state["groups"]:
        ends.append(ends[-1] + len(members))
    state["group_offsets"] = torch.tensor(ends, dtype=torch.int64, device=dev)
    state["shared"] = torch.tensor([s for s, _ in state["groups"]], dtype=torch.int32, device=dev)
    state["groups_of_one"] = case["members"] == 1
    return state


# ---- the plain forms ---------------------------------------------------------

def _turned(x, at, state):
    """x (tokens, heads, dim) with the pairs of its first dimensions turned, in 32 bits; the angles in 64."""
    freqs = state["freqs"]
    angle = at.double()[:, None, None] * freqs.double()
    cos, sin = angle.cos().float(), angle.sin().float()
    x, half = x.float(), freqs.numel()
    if state["adjacent"]:
        a, b = x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half: 2 * half]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_append(state):
    dev, table, page = state["table"].device, state["table"], state["page"]
    tokens = state["q"].shape[0]
    offsets, rows = state["offsets"], state["rows"].long()
    seq = torch.repeat_interleave(torch.arange(state["n"], device=dev), offsets[1:] - offsets[:-1], output_size=tokens)
    row = rows[seq]
    there = row >= 0
    row = row.clamp(min=0)
    at = state["lengths"][row].long() - (offsets[seq + 1] - torch.arange(tokens, device=dev))
    at = torch.where(there, at, torch.zeros_like(at))
    place = table[row, at // page].long()
    q = _turned(state["q"], at, state).to(state["q"].dtype)
    k = _turned(state["k"], at, state).to(state["k"].dtype)
    q = torch.where(there[:, None, None], q, torch.zeros_like(q))
    keys, values = state["keys"], state["values"]
    some = state["with_row"]
    keys[place[some], at[some] % page] = k[some]
    values[place[some], at[some] % page] = state["v"][some]
    return {"q": q, "keys": keys, "values": values}


def _gathered(pool, pages, first, count):
    """Tokens first .. first + count - 1 of rows with these pages (rows, pages): (rows, heads, count, dim) in 32 bits."""
    page = pool.shape[1]
    at = torch.arange(first, first + count, device=pages.device)
    held = pages[:, at // page].long().clamp(min=0)
    return pool[held, at % page].float().transpose(1, 2)


def _plain_attend(state):
    """The shared tokens once for each group, what lies behind them for all sequences at once; joined by their largest
    scores and sums. Sequences are padded to the longest."""
    dev, kv = state["q"].device, state["keys"].shape[2]
    heads, dk = state["q"].shape[1:]
    dv, n, share = state["values"].shape[3], state["n"], heads // kv
    groups, longest = state["groups"], max(state["new"])
    tokens = state["q"].shape[0]
    rows = state["rows"].long().clamp(min=0)
    table, length = state["table"][rows], state["lengths"][rows].long()
    length = torch.where(state["rows"] >= 0, length, torch.zeros_like(length))
    offsets = state["offsets"]
    new = offsets[1:] - offsets[:-1]
    step = torch.arange(longest, device=dev)
    packed = (offsets[:-1, None] + step).clamp(max=tokens - 1)
    inside = step < new[:, None]
    at = torch.where(inside, length[:, None] - new[:, None] + step, -1)                         # positions, (n, longest)
    q = state["q"].float()[packed] * state["scale"]
    q = q.reshape(n, longest, kv, share, dk).permute(0, 2, 1, 3, 4).reshape(n, kv, longest * share, dk)
    at = at.repeat_interleave(share, 1)[:, None, :, None]

    def part(q, k, v, t, at):
        s = q @ k.transpose(-1, -2)
        s = torch.where(t <= at, s, -math.inf)
        m = s.amax(-1, keepdim=True).clamp(min=-1e30)
        p = torch.exp(s - m)
        return m, p.sum(-1, keepdim=True), p @ v

    # behind the shared tokens
    first = torch.tensor([s for s, members in groups for _ in members], device=dev)
    behind = max(x for _, members in groups for _, x in members)
    t = first[:, None] + torch.arange(behind, device=dev)
    held = table.gather(1, (t // state["page"]).clamp(max=table.shape[1] - 1)).long().clamp(min=0)
    k, v = (pool[held, t % state["page"]].float().transpose(1, 2) for pool in (state["keys"], state["values"]))
    m, z, o = part(q, k, v, t[:, None, None], at)
    # the shared ones
    i = 0
    for shared, members in groups:
        live = state["live"][i: i + len(members)]
        if shared and any(live):
            g, lead = slice(i, i + len(members)), i + live.index(True)
            k, v = (_gathered(pool, table[lead: lead + 1], 0, shared)[0] for pool in (state["keys"], state["values"]))
            rest = (len(members) * longest * share, -1)
            flat = q[g].transpose(0, 1).reshape(kv, *rest)
            m1, z1, o1 = (x.reshape(kv, len(members), longest * share, -1).transpose(0, 1) for x in
                          part(flat, k, v, torch.arange(shared, device=dev), at[g].reshape(*rest)))
            top = torch.maximum(m[g], m1)
            a, b = torch.exp(m[g] - top), torch.exp(m1 - top)
            m[g], z[g], o[g] = top, a * z[g] + b * z1, a * o[g] + b * o1
        i += len(members)
    out = torch.where(z > 0, o / z, torch.zeros_like(o)).to(state["q"].dtype)
    out = out.reshape(n, kv, longest, share, dv).permute(0, 2, 1, 3, 4).reshape(n, longest, heads, dv)
    return out[inside]


def _moves(parents, rows):
    """New rows of the beams, and which rows to copy where (-1: none)."""
    b, w = rows.shape
    beams = torch.arange(w, device=rows.device)
    same = parents[:, :, None] == beams                                     # (request, continuation, beam)
    first = (same.long().cumsum(1) * same).gather(2, parents[:, :, None].long())[..., 0] == 1
    over = ~same.any(1)                                                     # beams that end
    free = torch.sort((~over).long(), dim=1, stable=True).indices           # those first, in order
    rank = ((~first).long().cumsum(1) - 1).clamp(min=0)
    kept = rows.gather(1, parents.long())
    new = torch.where(first, kept, rows.gather(1, free.gather(1, rank)))
    none = torch.full_like(kept, -1)
    return new, torch.where(first, none, kept).reshape(-1), torch.where(first, none, new).reshape(-1)


def _plain_select(state):
    """In 64 bits: neighbours at the border of the k best are close."""
    logits, scores, k = state["logits"], state["scores"], state["k"]
    b, w, v = logits.shape
    x = logits.double()
    top = x.amax(-1, keepdim=True)
    total = top + torch.exp(x - top).sum(-1, keepdim=True).log()
    key = scores.double()[..., None] + (x - total)
    end = torch.arange(v, device=x.device) == state["end"]
    key = torch.where(state["finished"][..., None], torch.where(end, scores.double()[..., None], -math.inf), key).reshape(b, w * v)
    # the k-th largest; those above it, and of the equal ones those of the lowest index
    value, index = torch.topk(key, k, dim=1)
    last = value[:, -1:]
    place = torch.arange(w * v, device=x.device)
    equal = torch.topk(torch.where(key == last, place, w * v), k, dim=1, largest=False).values
    both = torch.cat([torch.where(value > last, index, w * v), equal], 1)
    both = torch.sort(both, dim=1).values
    value = key.gather(1, both.clamp(max=w * v - 1))
    value = torch.where(both < w * v, value, torch.full_like(value, math.nan))
    order = torch.sort(torch.where(value.isnan(), -math.inf, value), dim=1, descending=True, stable=True).indices[:, :k]
    best, value = both.gather(1, order), value.gather(1, order)
    parents, tokens = (best // v).to(torch.int32), (best % v).to(torch.int32)
    out = {"scores": value.float(), "parents": parents, "tokens": tokens}
    if "rows" in state:
        out["rows"], out["src"], out["dst"] = _moves(parents, state["rows"])
    return out


def _own_run(state):
    import device_wide_prefix_amd as dws
    if state["kind"] == "append":
        q = dws.pages_append(state["keys"], state["values"], state["table"], state["lengths"], state["k"], state["v"],
                             rows=state["rows"], offsets=state["offsets"], freqs=state["freqs"], adjacent=state["adjacent"],
                             q=state["q"])
        return {"q": q, "keys": state["keys"], "values": state["values"]}
    if state["kind"] == "attend":
        groups = {} if state["groups_of_one"] else {"groups": state["group_offsets"], "shared": state["shared"]}
        return dws.pages_attention(state["q"], state["keys"], state["values"], state["table"], state["lengths"],
                                   rows=state["rows"], offsets=state["offsets"], scale=state["scale"], **groups)
    more = {"rows": state["rows"]} if "rows" in state else {}
    got = dws.beam_select(state["logits"], state["scores"], k=state["k"], finished=state["finished"], end_token=state["end"], **more)
    return dict(zip(("scores", "parents", "tokens", "rows", "src", "dst"), got))


def run(state):
    if own:
        return _own_run(state)
    return {"append": _plain_append, "attend": _plain_attend, "select": _plain_select}[state["kind"]](state)


# ---- the definitions in 64 bits ----------------------------------------------

def _places(state, row, count):
    t = torch.arange(count, device=state["table"].device)
    return state["table"][row].long()[t // state["page"]], t % state["page"]


def _exact_append(state):
    keys, values = state["keys"].double(), state["values"].double()
    turned = {"q": state["q"].double().clone(), "k": state["k"].double().clone()}
    freqs, ends = state["freqs"].double(), state["offsets"].tolist()
    pairs = torch.arange(freqs.numel(), device=keys.device)
    a, b = (2 * pairs, 2 * pairs + 1) if state["adjacent"] else (pairs, pairs + freqs.numel())
    for i, row in enumerate(state["rows"].tolist()):
        s = slice(ends[i], ends[i + 1])
        if row < 0:
            turned["q"][s] = 0
            continue
        length = int(state["lengths"][row])
        page, place = (x[length - (ends[i + 1] - ends[i]):] for x in _places(state, row, length))
        at = torch.arange(length - (ends[i + 1] - ends[i]), length, device=keys.device).double()
        z = torch.polar(torch.ones((), dtype=torch.float64, device=keys.device).expand(at.numel(), pairs.numel()).contiguous(),
                        at[:, None] * freqs)[:, None]
        for x in turned.values():
            y = torch.complex(x[s][..., a], x[s][..., b]) * z
            x[s][..., a], x[s][..., b] = y.real, y.imag
        keys[page, place] = turned["k"][s]
        values[page, place] = state["v"][s].double()
    return {"q": turned["q"], "keys": keys, "values": values}


def _exact_attend(state):
    q = state["q"].double()
    heads, kv = q.shape[1], state["keys"].shape[2]
    out = torch.zeros(q.shape[0], heads, state["values"].shape[3], dtype=torch.float64, device=q.device)
    ends = state["offsets"].tolist()
    for i, row in enumerate(state["rows"].tolist()):
        new = ends[i + 1] - ends[i]
        if row < 0 or new == 0:
            continue
        length = int(state["lengths"][row])
        page, place = _places(state, row, length)
        hidden = torch.ones(new, length, device=q.device).triu(length - new + 1) > 0
        for h in range(kv):
            k, v = state["keys"][:, :, h][page, place].double(), state["values"][:, :, h][page, place].double()
            for one in range(h * heads // kv, (h + 1) * heads // kv):
                s = (q[ends[i]: ends[i + 1], one] @ k.T) * state["scale"]
                out[ends[i]: ends[i + 1], one] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v
    return out


def _exact_select(state):
    scores, parents, tokens = [], [], []
    for x, s, over in zip(state["logits"], state["scores"], state["finished"]):
        key = torch.log_softmax(x.double(), -1) + s.double()[:, None]
        key[over] = -math.inf
        key[over, state["end"]] = s.double()[over]
        value, index = torch.sort(key.reshape(-1), descending=True, stable=True)
        scores.append(value[: state["k"]])
        parents.append(index[: state["k"]] // x.shape[1])
        tokens.append(index[: state["k"]] % x.shape[1])
    out = {"scores": torch.stack(scores), "parents": torch.stack(parents).to(torch.int32),
           "tokens": torch.stack(tokens).to(torch.int32)}
    if "rows" in state:
        out.update(rows=state["rows"].clone(), src=torch.full_like(state["rows"].reshape(-1), -1),
                   dst=torch.full_like(state["rows"].reshape(-1), -1))
        w = state["rows"].shape[1]
        for b, (row, chosen) in enumerate(zip(state["rows"].tolist(), out["parents"].tolist())):
            free, seen = [r for j, r in enumerate(row) if j not in chosen], set()
            for c, parent in enumerate(chosen):
                if parent in seen:
                    out["src"][b * w + c], out["dst"][b * w + c] = row[parent], free[0]
                    out["rows"][b, c] = free.pop(0)
                else:
                    out["rows"][b, c] = row[parent]
                    seen.add(parent)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "select": _exact_select}[case["kind"]](state)


# ---- the work ----------------------------------------------------------------

def work(case):
    size = _BYTES[case["type"]]
    if case["kind"] == "select":
        n = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": n * size + case["batch"] * (case["beams"] * 9 + case["k"] * 12), "flops": 4 * n}
    heads, kv, dk, dv = case["heads"], case["kv"], case["dk"], case["dv"]
    groups = _lengths(case)
    new = sum(t for _, m in groups for t, _ in m)
    if case["kind"] == "append":
        return {"bytes": 2 * new * size * ((heads + kv) * dk + kv * dv), "flops": 3 * new * (heads + kv) * case["rot"]}
    cached = sum(shared + sum(length for _, length in m) for shared, m in groups)
    seen = sum(t * (shared + length) - t * (t - 1) // 2 for shared, m in groups for t, length in m)
    return {"bytes": size * (cached * kv + new * heads) * (dk + dv), "flops": 2 * seen * heads * (dk + dv)}
