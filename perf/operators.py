"""Cases and plain forms of the gated delta rule and of the page operators.

The gated delta rule is a scan of matrix-valued affine maps along the tokens of a sequence: with S the (dim_k x dim_v)
state of a head,

    S' = exp(g_t) S;   u_t = beta_t (v_t - S'^T k_t);   S = S' + k_t u_t^T;   o_t = scale S^T q_t

Three of its forms are measured: ``prefill`` (the outputs of whole sequences and the state after each), ``train`` (the
outputs, then every gradient) and ``step`` (a few tokens more for each sequence of a batch, states in a pool).

The page operators keep a cache in pages: ``refs[p]`` counts the rows that hold page p (0: free), ``table[row]`` lists
the pages of a row and ``lengths[row]`` its tokens. ``copy`` moves pages, ``grow`` gives rows more of them, ``fork`` makes
rows that share another row's pages, ``free`` gives pages back and ``compact`` moves the pages in use to the front.

With ``own`` false run() computes all of it with elementary torch operations in 32 bits; with ``own`` true it calls the
library.
"""
import math

import torch

own = False

_CHUNK = 64
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # one token for one sequence of a small model: nothing but latency
        {"name": "step_one_small", "kind": "step", "n": 1, "tokens": 1, "hk": 4, "hv": 8, "dk": 64, "dv": 64, "slots": 5,
         "pads": 0, "type": "bf16"},
        # one token for each sequence of a full serving batch, a few of its places empty
        {"name": "step_batch", "kind": "step", "n": 128, "tokens": 1, "hk": 16, "hv": 32, "dk": 128, "dv": 128,
         "slots": 160, "pads": 3, "type": "bf16"},
        # the first tokens of one short prompt, 16-bit floats, heads shared by three
        {"name": "prefill_short", "kind": "prefill", "lens": "201", "hk": 2, "hv": 6, "dk": 64, "dv": 96, "init": False,
         "type": "fp16"},
        # packed prompts of very unequal lengths, one of a single token and one empty, each continuing a state
        {"name": "prefill_packed", "kind": "prefill", "lens": "6001,1,2048,63,64,0,65,4097,130,3915", "hk": 16, "hv": 32,
         "dk": 128, "dv": 128, "init": True, "type": "bf16"},
        # a training step in 32 bits with odd head dimensions
        {"name": "train_fp32_odd", "kind": "train", "lens": "333,70", "hk": 3, "hv": 3, "dk": 72, "dv": 40, "init": True,
         "type": "fp32"},
        # a training step on four sequences, keys and queries shared by two value heads
        {"name": "train_packed", "kind": "train", "lens": "2048,2048,1531,2500", "hk": 8, "hv": 16, "dk": 128, "dv": 128,
         "init": False, "type": "bf16"},
        # key and value pages of a prefix copied to other places of the pool
        {"name": "copy_many", "kind": "copy", "pages": 16384, "layers": 2, "elems": 16384, "n": 6000, "pads": 37,
         "type": "bf16"},
        # one request that asks for four samples
        {"name": "fork_few", "kind": "fork", "pages": 509, "layers": 1, "elems": 4096, "rows": 24, "max_pages": 40,
         "page_tokens": 16, "n": 4, "pads": 0, "type": "bf16"},
        # recurrent states: one page each, which every fork has to copy
        {"name": "fork_states", "kind": "fork", "pages": 400, "layers": 1, "elems": 524288, "rows": 256, "max_pages": 1,
         "page_tokens": 1 << 30, "n": 64, "pads": 2, "type": "fp32"},
        # a batch of long requests ends
        {"name": "free_long", "kind": "free", "pages": 1000000, "rows": 512, "max_pages": 4096, "page_tokens": 16, "n": 128,
         "pads": 5},
        # a small pool put in order
        {"name": "compact_small", "kind": "compact", "pages": 777, "layers": 1, "elems": 1000, "rows": 30, "max_pages": 50,
         "page_tokens": 16, "type": "fp16"},
        # a large pool, about half of it in use, put in order
        {"name": "compact_large", "kind": "compact", "pages": 60000, "layers": 2, "elems": 8192, "rows": 200,
         "max_pages": 512, "page_tokens": 16, "type": "bf16"},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.99)))))))


def draw(rng):
    kind = rng.choice(["step", "step", "prefill", "prefill", "train", "train", "copy", "grow", "fork", "free", "compact"])
    if kind in ("step", "prefill", "train"):
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        hv = hk * rng.choice([1, 1, 2, 3]) if hk < 16 else hk * rng.choice([1, 2])
        dk = rng.choice([64, 128, 128, 32, 96, 100, 256, 8 * rng.randint(1, 32)])
        dv = rng.choice([64, 128, 128, 32, 96, 36, 256, 8 * rng.randint(1, 32)])
        case = {"kind": kind, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
        if kind == "step":
            most = max(1, min(300, int(128 * 32 * 128 * 128 / (hv * dk * dv))))
            n = _log_int(rng, 1, most)
            case.update(n=n, tokens=rng.choice([1, 1, 1, 2, 4, 7]), slots=n + rng.randint(0, n // 4 + 2),
                        pads=rng.randint(0, n // 8))
            return case
        most = (16384 * 32 if kind == "prefill" else 8127 * 16) * 128 * 128 // (hv * max(dk, 64) * max(dv, 64))
        if case["type"] == "fp32":
            most //= 8
        total = _log_int(rng, 60, max(61, min(most, 16384 if kind == "prefill" else 8127)))
        count = rng.randint(1, max(1, min(12, total // 40)))
        cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        case.update(lens=",".join(str(x) for x in lens), init=rng.random() < 0.5)
        return case
    bits = rng.choice(["bf16", "fp16", "fp32"])
    if kind == "copy":
        pages = _log_int(rng, 64, 16384)
        elems = _log_int(rng, 500, 16384)
        n = rng.randint(1, pages // 3)
        return {"kind": kind, "pages": pages, "layers": rng.randint(1, 2), "elems": elems, "n": n,
                "pads": rng.randint(0, n // 8), "type": bits if bits != "fp32" else "bf16"}
    rows = _log_int(rng, 8, 512)
    max_pages = _log_int(rng, 4, 512)
    pages = rows * max_pages * 3 // 4 + rng.randint(8, 64)
    case = {"kind": kind, "pages": pages, "rows": rows, "max_pages": max_pages, "page_tokens": rng.choice([1, 16, 16, 64, 100])}
    if kind in ("grow", "fork", "free"):
        n = rng.randint(1, max(1, rows // 4))
        case.update(n=n, pads=rng.randint(0, n // 4))
    if kind in ("fork", "compact"):
        layers = rng.randint(1, 2)
        case.update(layers=layers, type=bits, elems=_log_int(rng, 64, max(65, min(16384, 60000 * 8192 // (pages * layers)))))
    return case


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ---- the inputs --------------------------------------------------------------

def _heads(gen, tokens, case):
    """q, k of unit length (as a model normalises them), v, log decays between about 0 and -5, and beta in (0, 1)."""
    dev, t = _device(), _TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    # q, k and v are parts of one projection's output, as they are in a model
    parts = torch.empty(tokens, 2 * hk * dk + hv * dv, dtype=t, device=dev)
    q, k, v = parts.split([hk * dk, hk * dk, hv * dv], dim=1)
    q, k, v = q.view(tokens, hk, dk), k.view(tokens, hk, dk), v.view(tokens, hv, dv)
    for x in (q, k):
        x.copy_(torch.nn.functional.normalize(normal(tokens, hk, dk), dim=-1))
    v.copy_(normal(tokens, hv, dv))
    rate = torch.exp(torch.rand(hv, generator=gen, device=dev) * 6 - 5)
    g = -rate * torch.nn.functional.softplus(normal(tokens, hv))
    beta = torch.sigmoid(normal(tokens, hv)).to(t)
    return {"q": q, "k": k, "v": v, "g": g, "beta": beta}


def _cache(gen, case):
    """A pool's counts, table and lengths after rows were filled, forked and freed in no order."""
    dev = _device()
    rows, max_pages, pages, pt = case["rows"], case["max_pages"], case["pages"], case["page_tokens"]
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    n = torch.randint(0, max_pages + 1, (rows,), generator=gen, device=dev)
    if max_pages == 1:
        n.fill_(1)
    n[torch.randperm(rows, generator=gen, device=dev)[: max(1, rows // 3)]] = 0      # empty rows
    end = torch.cumsum(n, 0)
    n = torch.where(end <= pages * 3 // 4, n, torch.zeros_like(n))
    start = torch.cumsum(n, 0) - n
    at = start[:, None] + torch.arange(max_pages, device=dev)
    held = torch.arange(max_pages, device=dev) < n[:, None]
    table = torch.where(held, order[at.clamp(max=pages - 1)], -1).to(torch.int32)
    short = torch.randint(0, pt, (rows,), generator=gen, device=dev)
    lengths = torch.clamp(n * pt - short, min=0)
    lengths = torch.where(n > 0, torch.maximum(lengths, (n - 1) * pt + 1), lengths).to(torch.int32)
    # half of the empty rows share the whole pages of another row
    empty, full = (lengths == 0).nonzero().reshape(-1), (lengths > 0).nonzero().reshape(-1)
    if full.numel():
        heir = empty[: empty.numel() // 2]
        parent = full[torch.randint(0, full.numel(), (heir.numel(),), generator=gen, device=dev)]
        whole = lengths[parent] // pt
        table[heir] = torch.where(torch.arange(max_pages, device=dev) < whole[:, None], table[parent], -1)
        lengths[heir] = whole * pt
    refs = torch.zeros(pages + 1, dtype=torch.int32, device=dev)
    refs.index_add_(0, torch.where(table >= 0, table, pages).reshape(-1).long(), torch.ones(rows * max_pages, dtype=torch.int32, device=dev))
    refs = refs[:pages].contiguous()
    return {"refs": refs, "table": table, "lengths": lengths, "page_tokens": pt}


def _padded(x, pads, gen):
    """x with `pads` of its places set to -1, as a batch of fixed size has them."""
    if pads:
        x = x.clone()
        x[torch.randperm(x.numel(), generator=gen, device=x.device)[:pads]] = -1
    return x


def _pool(gen, case):
    shape = (case["layers"], case["pages"], case["elems"])
    return torch.randn(shape, generator=gen, device=_device(), dtype=_TYPES[case["type"]])


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    kind = case["kind"]
    if kind == "step":
        n = case["n"]
        state = _heads(gen, n * case["tokens"], case)
        state["pool"] = 0.3 * torch.randn(case["slots"], case["hv"], case["dk"], case["dv"], generator=gen, device=dev)
        slots = torch.randperm(case["slots"], generator=gen, device=dev)[:n].to(torch.int32)
        state["slots"] = _padded(slots, case["pads"], gen)
        state["out"] = torch.zeros(n * case["tokens"], case["hv"], case["dv"], dtype=_TYPES[case["type"]], device=dev)
        state["scale"] = case["dk"] ** -0.5
    elif kind in ("prefill", "train"):
        lens = _lens(case)
        state = _heads(gen, sum(lens), case)
        ends = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
        state["offsets"] = ends.to(dev)
        state["lens"] = lens
        shape = (len(lens), case["hv"], case["dk"], case["dv"])
        state["initial"] = 0.3 * torch.randn(shape, generator=gen, device=dev) if case["init"] else None
        state["scale"] = case["dk"] ** -0.5
        if kind == "train":
            state["d_out"] = torch.randn(sum(lens), case["hv"], case["dv"], generator=gen, device=dev).to(_TYPES[case["type"]])
    elif kind == "copy":
        both = torch.randperm(case["pages"], generator=gen, device=dev)[: 2 * case["n"]].to(torch.int32)
        state = {"pool": _pool(gen, case), "src": _padded(both[: case["n"]].contiguous(), case["pads"], gen),
                 "dst": both[case["n"]:].contiguous()}
    else:
        state = _cache(gen, case)
        if kind in ("fork", "compact"):
            state["pool"] = _pool(gen, case)
        if kind == "compact":
            # half of the rows ended, their pages are holes now
            gone = torch.randperm(case["rows"], generator=gen, device=dev)[: case["rows"] // 2]
            held = state["table"][gone]
            state["refs"].index_add_(0, held[held >= 0].long(), torch.full((int((held >= 0).sum()),), -1, dtype=torch.int32, device=dev))
            state["table"][gone] = -1
            state["lengths"][gone] = 0
        elif kind == "free":
            state["rows"] = _padded(torch.randperm(case["rows"], generator=gen, device=dev)[: case["n"]].to(torch.int32), case["pads"], gen)
        elif kind == "grow":
            rows = torch.randperm(case["rows"], generator=gen, device=dev)[: case["n"]].to(torch.int32)
            state["rows"] = _padded(rows, case["pads"], gen)
            most = case["max_pages"] * case["page_tokens"]
            more = torch.randint(0, 3 * case["page_tokens"] + 1, (case["n"],), generator=gen, device=dev)
            state["new_lengths"] = torch.clamp(state["lengths"][rows.long()] + more, max=most).to(torch.int32)
        elif kind == "fork":
            empty = (state["lengths"] == 0).nonzero().reshape(-1)
            full = (state["lengths"] > 0).nonzero().reshape(-1)
            n = min(case["n"], empty.numel())
            state["children"] = empty[torch.randperm(empty.numel(), generator=gen, device=dev)[:n]].to(torch.int32)
            pick = torch.randint(0, max(1, full.numel()), (n,), generator=gen, device=dev)
            parents = full[pick] if full.numel() else empty[pick % empty.numel()]
            state["parents"] = _padded(parents.to(torch.int32), min(case["pads"], n), gen)
    state["kind"] = kind
    return state


# ---- the plain forms ---------------------------------------------------------

def _inverse(low):
    """(I + low)^-1 for strictly lower triangular `low`, by doubling the inverted diagonal blocks."""
    c = low.shape[-1]
    inv = torch.ones(*low.shape[:-2], c, 1, 1, device=low.device, dtype=low.dtype)
    b = 1
    while b < c:
        blocks = low.reshape(*low.shape[:-2], c // (2 * b), 2 * b, c // (2 * b), 2 * b)
        blocks = torch.movedim(torch.diagonal(blocks, dim1=-4, dim2=-2), -1, -3)
        first, second = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        left = -(second @ blocks[..., b:, :b] @ first)
        inv = torch.cat([torch.cat([first, torch.zeros_like(first)], -1), torch.cat([left, second], -1)], -2)
        b *= 2
    return inv[..., 0, :, :]


def _plain_rule(q, k, v, g, beta, s, scale):
    """Outputs and last states for q, k, v [n, heads, tokens, dim], g, beta [n, heads, tokens] and states s, in 32 bits;
    tokens of g = 0, beta = 0, k = 0 behind a sequence change nothing. Chunks of _CHUNK tokens: within one, the u solve
    a triangular system; from chunk to chunk only the state goes on."""
    n, h, length, dk = q.shape
    chunks = -(-length // _CHUNK)
    more = chunks * _CHUNK - length

    def split(x):
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 3) + (0, more))
        return x.reshape(n, h, chunks, _CHUNK, *x.shape[3:])

    q, k, v, g, beta = split(q), split(k), split(v), split(g), split(beta)
    total = torch.cumsum(g.double(), -1)
    lower = torch.ones(_CHUNK, _CHUNK, device=q.device).tril() > 0
    decay = torch.exp(torch.where(lower, total[..., :, None] - total[..., None, :], -math.inf).float())
    kt = k.transpose(-1, -2).contiguous()
    t = _inverse((beta[..., None] * decay * (k @ kt)).tril(-1))
    p = scale * decay * (q @ kt)
    into = torch.exp(total.float())[..., None]
    out_of = torch.exp((total[..., -1:] - total).float())[..., None]
    outs = []
    for c in range(chunks):
        x = beta[:, :, c, :, None] * (v[:, :, c] - into[:, :, c] * (k[:, :, c] @ s))
        u = t[:, :, c] @ x
        outs.append(scale * into[:, :, c] * (q[:, :, c] @ s) + p[:, :, c] @ u)
        s = into[:, :, c, -1:] * s + kt[:, :, c] @ (out_of[:, :, c] * u)
    return torch.cat(outs, 2)[:, :, :length] if outs else v.reshape(n, h, 0, v.shape[-1]), s


def _rows_of(state):
    """Where the packed rows lie in a [sequences, longest] layout."""
    offsets, longest = state["offsets"], max(state["lens"] + [1])
    at = torch.arange(longest, device=offsets.device)
    inside = at < (offsets[1:] - offsets[:-1])[:, None]
    return (offsets[:-1, None] + at).clamp(max=max(0, sum(state["lens"]) - 1)), inside


def _laid_out(x, rows, inside, heads):
    """Packed [tokens, h, ...] as [sequences, heads, longest, ...] in 32 bits, zero behind each sequence."""
    x = x.float()
    x = x.repeat_interleave(heads // x.shape[1], 1)[rows]
    x = torch.where(inside.reshape(*inside.shape, *(1,) * (x.dim() - 2)), x, torch.zeros_like(x))
    return x.transpose(1, 2).contiguous()


def _plain_prefill(state, leaves=None):
    src = leaves or state
    heads = state["v"].shape[1]
    rows, inside = _rows_of(state)
    parts = [_laid_out(src[x], rows, inside, heads) for x in ("q", "k", "v", "g", "beta")]
    s = src["initial"]
    if s is None:
        s = torch.zeros(len(state["lens"]), heads, state["q"].shape[2], state["v"].shape[2], device=parts[0].device)
    o, s = _plain_rule(*parts, s, state["scale"])
    return o.transpose(1, 2)[inside], s


def _plain_train(state):
    names = ["q", "k", "v", "g", "beta"] + (["initial"] if state["initial"] is not None else [])
    leaves = {x: state[x].float().detach().requires_grad_() for x in names}
    leaves.setdefault("initial", None)
    with torch.enable_grad():
        o, _ = _plain_prefill(state, leaves)
        grads = torch.autograd.grad(o, [leaves[x] for x in names], state["d_out"].float())
    t = state["q"].dtype
    return {"out": o.detach().to(t), **{"d_" + x: y.to(t) for x, y in zip(names, grads)}}


def _plain_step(state):
    pool, slots, out = state["pool"], state["slots"], state["out"]
    n, hv = slots.numel(), pool.shape[1]
    some = (slots >= 0).nonzero().reshape(-1)
    at = slots[some].long()

    def part(x):
        x = x.reshape(n, -1, *x.shape[1:])[some].float()
        return x.repeat_interleave(hv // x.shape[2], 2)

    q, k, v, g, beta = (part(state[x]) for x in ("q", "k", "v", "g", "beta"))
    s = pool[at]
    outs = []
    for i in range(q.shape[1]):
        s = torch.exp(g[:, i])[..., None, None] * s
        u = beta[:, i, :, None] * (v[:, i] - (k[:, i, :, None, :] @ s)[:, :, 0])
        s = s + k[:, i, :, :, None] * u[:, :, None, :]
        outs.append(state["scale"] * (q[:, i, :, None, :] @ s)[:, :, 0])
    out.view(n, q.shape[1], hv, -1)[some] = torch.stack(outs, 1).to(out.dtype)
    pool[at] = s
    return {"out": out, "state": pool}


def _moved(pool, src, dst):
    """pool[dst] = pool[src] in every layer for the pairs with src and dst from 0."""
    some = ((src >= 0) & (dst >= 0)).nonzero().reshape(-1)
    pool[:, dst[some].long()] = pool[:, src[some].long()]
    return pool


def _ceil(x, by):
    return (x + by - 1) // by


def _plain_grow(state):
    refs, table, lengths, pt = state["refs"].clone(), state["table"].clone(), state["lengths"].clone(), state["page_tokens"]
    rows, new = state["rows"], state["new_lengths"].long()
    row = rows.clamp(min=0).long()
    old = lengths[row].long()
    good = (rows >= 0) & (new >= old) & (_ceil(new, pt) <= table.shape[1])
    need = torch.where(good, _ceil(new, pt) - _ceil(old, pt), 0)
    first = torch.cumsum(need, 0) - need
    free = (refs <= 0).nonzero().reshape(-1)
    granted = good & ((need == 0) | (first + need <= free.numel()))
    need = torch.where(granted, need, 0)
    which = torch.repeat_interleave(torch.arange(rows.numel(), device=rows.device), need)
    k = torch.arange(which.numel(), device=rows.device) - (torch.cumsum(need, 0) - need)[which]
    page = free[first[which] + k]
    table[row[which], _ceil(old, pt)[which] + k] = page.to(torch.int32)
    refs[page] = 1
    lengths[row[granted]] = new[granted].to(torch.int32)
    return {"refs": refs, "table": table, "lengths": lengths, "granted": granted.to(torch.int32)}


def _plain_fork(state):
    refs, table, lengths, pt = state["refs"].clone(), state["table"].clone(), state["lengths"].clone(), state["page_tokens"]
    parents, children = state["parents"], state["children"]
    good = (parents >= 0) & (children >= 0)
    parent, child = parents.clamp(min=0).long(), children.clamp(min=0).long()
    good &= lengths[child] == 0
    length = torch.where(good, lengths[parent], 0).long()
    need = (length % pt != 0).long()
    first = torch.cumsum(need, 0) - need
    free = (refs <= 0).nonzero().reshape(-1)
    granted = good & ((need == 0) | (first < free.numel()))
    copied = (granted & (need > 0)).nonzero().reshape(-1)
    page = torch.full_like(length, -1)
    page[copied] = free[first[copied]]
    whole = (length // pt)[:, None]
    at = torch.arange(table.shape[1], device=table.device)
    held = table[parent]
    shared = (at < whole) & granted[:, None]
    refs.index_add_(0, held[shared].long(), torch.ones_like(held[shared]))
    refs[page[copied]] = 1
    rows = torch.where(shared, held, torch.where((at == whole) & (need > 0)[:, None], page[:, None].to(torch.int32), -1))
    table[child[granted]] = rows[granted]
    lengths[child[granted]] = length[granted].to(torch.int32)
    src = held[copied, (length // pt)[copied]]
    pool = _moved(state["pool"], src, page[copied])
    return {"pool": pool, "refs": refs, "table": table, "lengths": lengths, "granted": granted.to(torch.int32)}


def _plain_free(state):
    refs, table, lengths, pt = state["refs"].clone(), state["table"].clone(), state["lengths"].clone(), state["page_tokens"]
    row = state["rows"][state["rows"] >= 0].long()
    held = table[row]
    mine = (torch.arange(table.shape[1], device=table.device) < _ceil(lengths[row].long(), pt)[:, None]) & (held >= 0)
    was = refs > 0
    refs.index_add_(0, held[mine].long(), torch.full_like(held[mine], -1))
    table[row] = -1
    lengths[row] = 0
    return {"refs": refs, "table": table, "lengths": lengths, "freed": (was & (refs <= 0)).sum().reshape(1)}


def _plain_compact(state):
    refs, table = state["refs"].clone(), state["table"].clone()
    live = refs > 0
    count = live.sum()
    at = torch.arange(refs.numel(), device=refs.device)
    src, dst = (live & (at >= count)).nonzero().reshape(-1), (~live & (at < count)).nonzero().reshape(-1)
    remap = torch.where(live, at, -1)
    remap[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    new = remap[table.clamp(min=0).long()]
    table = torch.where((table >= 0) & (new >= 0), new, table.long()).to(torch.int32)
    pool = _moved(state["pool"], src, dst)
    return {"pool": pool, "refs": refs, "table": table, "count": count.reshape(1), "remap": remap.to(torch.int32)}


# ---- one pass ----------------------------------------------------------------

def _own_run(state):
    import device_wide_prefix_amd as dws
    kind = state["kind"]
    if kind == "step":
        out = dws.delta_rule_step(state["q"], state["k"], state["v"], state["g"], state["beta"], state["pool"],
                                  slots=state["slots"], scale=state["scale"], out=state["out"])
        return {"out": out, "state": state["pool"]}
    if kind in ("prefill", "train"):
        args = [state[x] for x in ("q", "k", "v", "g", "beta")]
        more = {"offsets": state["offsets"], "initial_state": state["initial"], "scale": state["scale"]}
        if kind == "prefill":
            out, final = dws.delta_rule(*args, final_state=True, **more)
            return {"out": out, "state": final}
        out = dws.delta_rule(*args, **more)
        grads = dws.delta_rule_backward(state["d_out"], *args, **more)
        return {"out": out, **{"d_" + x: y for x, y in zip(("q", "k", "v", "g", "beta", "initial"), grads) if y is not None}}
    if kind == "copy":
        return {"pool": dws.pages_copy(state["pool"], state["src"], state["dst"], page_dim=1)}
    refs, table, lengths = state["refs"].clone(), state["table"].clone(), state["lengths"].clone()
    if kind == "grow":
        granted = dws.pages_grow(refs, table, lengths, state["rows"], state["new_lengths"], state["page_tokens"])
        return {"refs": refs, "table": table, "lengths": lengths, "granted": granted}
    if kind == "fork":
        granted, src, dst, count = dws.pages_fork(refs, table, lengths, state["parents"], state["children"], state["page_tokens"])
        pool = dws.pages_copy(state["pool"], src, dst, count=count, page_dim=1)
        return {"pool": pool, "refs": refs, "table": table, "lengths": lengths, "granted": granted}
    if kind == "free":
        freed = dws.pages_free(refs, table, lengths, state["rows"], state["page_tokens"])
        return {"refs": refs, "table": table, "lengths": lengths, "freed": freed}
    count, remap, src, dst, moves = dws.pages_compact(refs, table)
    pool = dws.pages_copy(state["pool"], src, dst, count=moves, page_dim=1)
    return {"pool": pool, "refs": refs, "table": table, "count": count, "remap": remap}


def run(state):
    if own:
        return _own_run(state)
    kind = state["kind"]
    if kind == "step":
        return _plain_step(state)
    if kind == "prefill":
        o, s = _plain_prefill(state)
        return {"out": o.to(state["q"].dtype), "state": s}
    if kind == "train":
        return _plain_train(state)
    if kind == "copy":
        return {"pool": _moved(state["pool"], state["src"], state["dst"])}
    return {"grow": _plain_grow, "fork": _plain_fork, "free": _plain_free, "compact": _plain_compact}[kind](state)


# ---- the definition in 64 bits ----------------------------------------------

def _wide(x, lens, heads):
    """Packed [tokens, h, ...] as a list over time of [sequences, heads, ...] in 64 bits, zero behind each sequence."""
    x = x.double()
    x = x.repeat_interleave(heads // x.shape[1], 1)
    wide = torch.zeros(max(lens + [1]), len(lens), *x.shape[1:], dtype=x.dtype, device=x.device)
    first = 0
    for i, n in enumerate(lens):
        wide[:n, i] = x[first: first + n]
        first += n
    return wide


def _narrow(wide, lens, shared):
    """The inverse of _wide; a head that `shared` heads used gets their sum."""
    x = torch.cat([wide[:n, i] for i, n in enumerate(lens)])
    return x.reshape(x.shape[0], x.shape[1] // shared, shared, *x.shape[2:]).sum(2) if shared > 1 else x


def exact(case, seed):
    if case["kind"] not in ("step", "prefill", "train"):
        return None
    state = prepare(case, seed)
    train, hv, scale = case["kind"] == "train", case["hv"], state["scale"]
    lens = [case["tokens"]] * case["n"] if case["kind"] == "step" else state["lens"]
    q, k, v, g, b = (_wide(state[x], lens, hv) for x in ("q", "k", "v", "g", "beta"))
    if case["kind"] == "step":
        some = state["slots"] >= 0
        s = state["pool"][state["slots"].clamp(min=0).long()].double()
    elif state["initial"] is not None:
        s = state["initial"].double()
    else:
        s = torch.zeros(len(lens), hv, case["dk"], case["dv"], dtype=torch.float64, device=q.device)
    out = torch.zeros_like(v)
    before = torch.zeros(v.shape[0], *s.shape, dtype=s.dtype, device=s.device) if train else None
    for t in range(v.shape[0]):
        if train:
            before[t] = s
        s = s * g[t].exp()[..., None, None]
        u = b[t][..., None] * (v[t] - torch.matmul(k[t][..., None, :], s).squeeze(-2))
        s = s + k[t][..., :, None] * u[..., None, :]
        out[t] = scale * torch.matmul(q[t][..., None, :], s).squeeze(-2)
    if case["kind"] == "step":
        new = state["pool"].double()
        new[state["slots"][some].long()] = s[some]
        out = torch.where(some[None, :, None, None], out, torch.zeros_like(out)).transpose(0, 1)
        return {"out": out.reshape(state["out"].shape), "state": new}
    if not train:
        return {"out": _narrow(out, lens, 1), "state": s}
    d_out = _wide(state["d_out"], lens, hv)
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, b))
    ds = torch.zeros_like(s)
    for t in reversed(range(v.shape[0])):
        decayed = before[t] * g[t].exp()[..., None, None]
        off = v[t] - torch.matmul(k[t][..., None, :], decayed).squeeze(-2)
        u = b[t][..., None] * off
        after = decayed + k[t][..., :, None] * u[..., None, :]
        ds = ds + scale * q[t][..., :, None] * d_out[t][..., None, :]
        dq[t] = scale * torch.matmul(after, d_out[t][..., None]).squeeze(-1)
        du = torch.matmul(k[t][..., None, :], ds).squeeze(-2)
        db[t] = (du * off).sum(-1)
        dv[t] = b[t][..., None] * du
        dk[t] = torch.matmul(ds, u[..., None]).squeeze(-1) - torch.matmul(decayed, dv[t][..., None]).squeeze(-1)
        ds = ds - k[t][..., :, None] * dv[t][..., None, :]
        dg[t] = (ds * decayed).sum((-1, -2))
        ds = ds * g[t].exp()[..., None, None]
    shared = hv // case["hk"]
    grads = {"out": _narrow(out, lens, 1), "d_q": _narrow(dq, lens, shared), "d_k": _narrow(dk, lens, shared),
             "d_v": _narrow(dv, lens, 1), "d_g": _narrow(dg, lens, 1), "d_beta": _narrow(db, lens, 1)}
    if case["init"]:
        grads["d_initial"] = ds
    return grads


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    kind = case["kind"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}.get(case.get("type"), 0)
    if kind in ("step", "prefill", "train"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        count = case["n"] - case["pads"] if kind == "step" else len(_lens(case))
        tokens = count * case["tokens"] if kind == "step" else sum(_lens(case))
        states = count * hv * dk * dv
        inputs = tokens * (2 * hk * dk * size + hv * (dv * size + size + 4))
        outputs = tokens * hv * dv * size
        if kind == "step":
            return {"bytes": inputs + outputs + 8 * states, "flops": 6 * tokens * hv * dk * dv}
        if kind == "prefill":
            return {"bytes": inputs + outputs + states * (8 if case["init"] else 4), "flops": 6 * tokens * hv * dk * dv}
        grads = tokens * (2 * hk * dk + hv * (dv + 2)) * size
        initial = states * (8 + size) if case["init"] else 0
        # forward: inputs in, outputs out; backward: inputs and d_out in, gradients out
        return {"bytes": 2 * inputs + 2 * outputs + grads + initial, "flops": 20 * tokens * hv * dk * dv}
    if kind == "copy":
        return {"bytes": (case["n"] - case["pads"]) * (2 * case["layers"] * case["elems"] * size + 8), "flops": 0}
    pages, rows, most = case["pages"], case["rows"], case["max_pages"]
    if kind == "compact":
        # about a sixth of the pages are in use, in no order: five sixths of those lie behind the front
        moved = pages * 5 // 36
        return {"bytes": 2 * moved * case["layers"] * case["elems"] * size + 12 * pages + 8 * rows * most, "flops": 0}
    n = case["n"] - case["pads"]
    if kind == "fork":
        return {"bytes": n * (2 * case["layers"] * case["elems"] * size + 8 * most) + 4 * pages, "flops": 0}
    if kind == "grow":
        return {"bytes": n * 24 + 4 * pages, "flops": 0}
    return {"bytes": n * most * 6, "flops": 0}
