"""The page operators on the GPU against one request after another. All results are whole numbers or bytes: equal."""
import random

import pytest
import torch

import device_wide_prefix_amd as dws
from gpu_util import note
from pages_reference import Cache, filled, pages_of

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class OnGpu:
    def __init__(self, c: Cache):
        self.refs, self.table, self.lengths, self.page_tokens = ints(c.refs), ints(c.table), ints(c.lengths), c.page_tokens
        if self.table.dim() != 2:
            self.table = self.table.reshape(len(c.table), -1)

    def args(self):
        return self.refs, self.table, self.lengths

    def same(self, c: Cache):
        assert self.refs.tolist() == c.refs
        assert self.table.tolist() == c.table
        assert self.lengths.tolist() == c.lengths


# pages, rows, most pages of a row, tokens of a page
CACHES = [(1, 1, 1, 1), (7, 3, 2, 4), (64, 9, 20, 16), (4095, 40, 150, 16), (4096, 40, 130, 1), (4097, 33, 200, 5),
          (20000, 70, 700, 16), (9000, 5, 4500, 3)]


@pytest.mark.parametrize("shape", CACHES)
def test_grow(gpu, shape):
    note(f"pages grow {shape}")
    rng = random.Random(1)
    c = filled(2, *shape)
    most = shape[2] * shape[3]
    for step in range(3):
        g = OnGpu(c)
        n = rng.randint(1, 2 * shape[1])
        rows = [rng.randint(-2, shape[1] + 1) for _ in range(n)]            # some twice, some outside
        new = [max(0, (c.lengths[r] if 0 <= r < shape[1] else 0) + rng.randint(-2, most // (step + 1) + 2)) for r in rows]
        granted = dws.pages_grow(*g.args(), ints(rows), ints(new), g.page_tokens)
        assert granted.tolist() == c.grow(rows, new)
        g.same(c)


@pytest.mark.parametrize("shape", CACHES)
def test_fork(gpu, shape):
    note(f"pages fork {shape}")
    rng = random.Random(3)
    c = filled(4, *shape)
    for _ in range(3):
        c.free(rng.sample(range(shape[1]), shape[1] // 3))
        g = OnGpu(c)
        n = rng.randint(1, 2 * shape[1])
        parents = [rng.randint(-1, shape[1]) for _ in range(n)]
        children = [rng.randint(-1, shape[1]) for _ in range(n)]
        granted, src, dst, count = dws.pages_fork(*g.args(), ints(parents), ints(children), g.page_tokens)
        want, a, b = c.fork(parents, children)
        assert granted.tolist() == want
        assert count.tolist() == [len(a)]
        assert src.tolist() == a + [-1] * (n - len(a)) and dst.tolist() == b + [-1] * (n - len(b))
        g.same(c)


@pytest.mark.parametrize("shape", CACHES)
def test_free(gpu, shape):
    note(f"pages free {shape}")
    rng = random.Random(5)
    c = filled(6, *shape)
    g = OnGpu(c)
    rows = [rng.randint(-2, shape[1] + 1) for _ in range(shape[1])]
    assert dws.pages_free(*g.args(), ints(rows), g.page_tokens).tolist() == [c.free(rows)]
    g.same(c)
    rows = list(range(shape[1]))
    assert dws.pages_free(*g.args(), ints(rows), g.page_tokens).tolist() == [c.free(rows)]
    g.same(c)
    assert not any(c.refs)


@pytest.mark.parametrize("shape", CACHES)
@pytest.mark.parametrize("state", ["mixed", "empty", "full", "front", "back"])
def test_compact(gpu, shape, state):
    note(f"pages compact {shape} {state}")
    c = filled(7, *shape)
    pages = shape[0]
    if state != "mixed":
        c = Cache(*shape)
        for p in range(pages):
            c.refs[p] = {"empty": 0, "full": 2, "front": int(p < pages // 2), "back": int(p >= pages // 2)}[state]
        c.table[0] = [(5 * i) % pages for i in range(shape[2])]
    g = OnGpu(c)
    count, remap, src, dst, moves = dws.pages_compact(g.refs, g.table)
    n, want, a, b = c.compact()
    assert count.tolist() == [n] and moves.tolist() == [len(a)] and remap.tolist() == want
    assert src.tolist() == a + [-1] * (pages // 2 - len(a)) and dst.tolist() == b + [-1] * (pages // 2 - len(b))
    g.same(c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
@pytest.mark.parametrize("layers,pages,elems", [(1, 2, 1), (1, 9, 7), (3, 50, 1000), (2, 40, 8192), (2, 33, 20001), (1, 20, 100000)])
def test_copy(gpu, layers, pages, elems, dtype):
    note(f"pages copy {layers} {pages} {elems} {dtype}")
    gen = torch.Generator().manual_seed(1)
    pool = torch.randint(0, 200, (layers, pages, elems), generator=gen).to(dtype)
    order = torch.randperm(pages, generator=gen)
    n = pages // 2
    src, dst = order[:n].clone(), order[n: 2 * n].clone()
    src[::5] = -1
    if n > 2:
        dst[1], src[2] = pages, 1 << 30                                     # outside the pool
    want = pool.clone()
    pairs = [(int(a), int(b)) for a, b in zip(src, dst) if 0 <= a < pages and 0 <= b < pages]
    for a, b in pairs:
        want[:, b] = pool[:, a]
    # a buffer around the pool that has to stay, and a start that is not a multiple of 16 bytes
    size = pool.numel()
    for shift in (0, 16 // pool.element_size(), 1):
        around = torch.full((size + 64,), 3, dtype=dtype, device="cuda")
        inside = around[shift: shift + size].view(pool.shape)
        inside.copy_(pool)
        assert dws.pages_copy(inside, src.int().cuda(), dst.int().cuda(), page_dim=1) is inside
        assert torch.equal(inside.cpu(), want)
        assert (around[:shift] == 3).all() and (around[shift + size:] == 3).all()
    if layers == 1:
        flat = pool[0].cuda()
        dws.pages_copy(flat, src.int().cuda(), dst.int().cuda())
        assert torch.equal(flat.cpu(), want[0])
    # only the first pairs, counted on the GPU
    for k in (-1, 0, 1, n, n + 5):
        some = pool.cuda()
        dws.pages_copy(some, src.int().cuda(), dst.int().cuda(), count=torch.tensor([k], device="cuda"), page_dim=1)
        want = pool.clone()
        for a, b in zip(src[:max(0, k)], dst[:max(0, k)]):
            if 0 <= a < pages and 0 <= b < pages:
                want[:, b] = pool[:, a]
        assert torch.equal(some.cpu(), want)


def test_copy_beyond_32_bits(gpu):
    """Pages whose bytes lie beyond 2^32."""
    pool = torch.zeros(3, 1 << 31, dtype=torch.uint8, device="cuda")
    pool[0] = 7
    pool[0, -1] = 9
    dws.pages_copy(pool, ints([0]), ints([2]))
    assert int(pool[2, 0]) == 7 and int(pool[2, -1]) == 9 and bool((pool[2, 1:-1] == 7).all()) and not pool[1].any()


def test_no_requests(gpu):
    c = filled(8, 50, 6, 5, 4)
    g = OnGpu(c)
    none = ints([])
    assert dws.pages_grow(*g.args(), none, none, 4).numel() == 0
    granted, src, dst, count = dws.pages_fork(*g.args(), none, none, 4)
    assert granted.numel() == src.numel() == dst.numel() == 0 and count.tolist() == [0]
    assert dws.pages_free(*g.args(), none, 4).tolist() == [0]
    pool = torch.ones(50, 3, device="cuda")
    dws.pages_copy(pool, none, none)
    g.same(c)


def test_a_cache_that_is_wrong_touches_nothing_outside(gpu):
    """Entries outside the pool, lengths beyond the table and counts below 0 are skipped or taken as free."""
    c = filled(9, 100, 8, 10, 4)
    around = torch.full((3, 200), 77, dtype=torch.int32, device="cuda")
    refs, table, lengths = around[0, 50:150], around[1, 50:130].view(8, 10), around[2, 50:58]
    refs.copy_(ints(c.refs))
    table.copy_(ints(c.table))
    lengths.copy_(ints(c.lengths))
    table[0] = ints([1 << 30, -5, 100, 99, 0, -(1 << 31), 101, 3, 2, 1])
    table[5] = -1
    lengths[0], lengths[1], lengths[2], lengths[5] = 40, 2**31 - 1, -7, 0
    refs[3] = -4
    dws.pages_fork(refs, table, lengths, ints([0, 1, 2]), ints([5, 6, 7]), 4)
    dws.pages_grow(refs, table, lengths, ints([0, 1, 2, 3]), ints([2**31 - 1, 2**31 - 1, 4, -1]), 4)
    dws.pages_compact(refs, table)
    dws.pages_free(refs, table, lengths, ints(list(range(8))), 4)
    torch.cuda.synchronize()
    for row, (a, b) in zip(around, ((50, 150), (50, 130), (50, 58))):
        assert (row[:a] == 77).all() and (row[b:] == 77).all()


def test_many_requests(gpu):
    """More requests than one pass over them takes, and more rows than a workgroup."""
    c = filled(10, 6000, 3000, 3, 4)
    g = OnGpu(c)
    rng = random.Random(11)
    rows = [rng.randrange(3000) for _ in range(5000)]
    new = [min(12, c.lengths[r] + rng.randint(0, 3)) for r in rows]
    assert dws.pages_grow(*g.args(), ints(rows), ints(new), 4).tolist() == c.grow(rows, new)
    g.same(c)
    gone = rng.sample(range(3000), 1400)
    assert dws.pages_free(*g.args(), ints(gone), 4).tolist() == [c.free(gone)]
    parents, children = [rng.randrange(3000) for _ in range(2500)], [rng.choice(gone) for _ in range(2500)]
    granted, src, dst, count = dws.pages_fork(*g.args(), ints(parents), ints(children), 4)
    want, a, b = c.fork(parents, children)
    assert granted.tolist() == want and src[:len(a)].tolist() == a and dst[:len(b)].tolist() == b
    g.same(c)


def test_a_cache_in_use(gpu):
    """Rows grow, fork, end and are compacted, their tokens written and read back: what a row holds is its own."""
    pages, rows, max_pages, pt = 300, 20, 12, 8
    c = Cache(pages, rows, max_pages, pt)
    g = OnGpu(c)
    keys, values = (torch.full((2, pages, pt, 3), -1.0, device="cuda") for _ in range(2))
    content = {r: [] for r in range(rows)}
    rng = random.Random(12)
    stamp = 0

    def write(r, new):
        nonlocal stamp
        for t in range(len(content[r]), new):
            stamp += 1
            content[r].append(stamp)
            page = c.table[r][t // pt]
            keys[:, page, t % pt] = stamp
            values[:, page, t % pt] = -stamp

    for step in range(12):
        some = rng.sample(range(rows), 6)
        new = [min(max_pages * pt, c.lengths[r] + rng.randint(0, 20)) for r in some]
        assert dws.pages_grow(*g.args(), ints(some), ints(new), pt).tolist() == c.grow(some, new)
        for r in some:
            write(r, c.lengths[r])
        empty = [r for r in range(rows) if not c.lengths[r]][:3]
        full = [r for r in range(rows) if c.lengths[r]]
        parents = [rng.choice(full) for _ in empty]
        granted, src, dst, count = dws.pages_fork(*g.args(), ints(parents), ints(empty), pt)
        assert granted.tolist() == c.fork(parents, empty)[0]
        for pool in (keys, values):
            dws.pages_copy(pool, src, dst, count=count, page_dim=1)
        for p, r, ok in zip(parents, empty, granted.tolist()):
            content[r] = list(content[p]) if ok else []
        gone = rng.sample(range(rows), 4)
        assert dws.pages_free(*g.args(), ints(gone), pt).tolist() == [c.free(gone)]
        for r in gone:
            content[r] = []
        if step % 3 == 2:
            n, remap, src, dst, moves = dws.pages_compact(g.refs, g.table)
            assert n.tolist() == [c.compact()[0]]
            for pool in (keys, values):
                dws.pages_copy(pool, src, dst, count=moves, page_dim=1)
        g.same(c)
        for r in range(rows):
            for t, want in enumerate(content[r]):
                page = c.table[r][t // pt]
                assert float(keys[1, page, t % pt, 2]) == want and float(values[0, page, t % pt, 0]) == -want
        assert all(pages_of(len(content[r]), pt) == sum(p >= 0 for p in c.table[r]) for r in range(rows))


def test_states_in_pages(gpu):
    """Recurrent states as one-page rows: a beam forks, its copies go on with other tokens, ends, and the pool is
    compacted; the table is what dws.delta_rule_step takes as slots."""
    from delta_reference import close, inputs, reference
    names = ("q", "k", "v", "g", "beta")
    hv, dk, dv, beams = 2, 32, 24, 3
    lens = [40] * beams
    x, offsets, _ = inputs(20, lens, 1, hv, dk, dv, torch.float32, init=False)
    pool = torch.randn(9, hv, dk, dv, device="cuda")
    c = Cache(9, 6, 1, 1 << 30)
    g = OnGpu(c)
    rows = [4, 1, 3]
    assert dws.pages_grow(*g.args(), ints([4]), ints([10]), g.page_tokens).tolist() == [1]
    c.grow([4], [10])
    prompt = {y: x[y][:10] for y in names}
    dws.delta_rule(*(prompt[y] for y in names), final_state=pool, slots=g.table[4])
    granted, src, dst, count = dws.pages_fork(*g.args(), ints([4, 4]), ints([1, 3]), g.page_tokens)
    c.fork([4, 4], [1, 3])
    dws.pages_copy(pool, src, dst, count=count)
    outs = []
    for t in range(10, 30):
        if t == 20:                                     # the first one ends, the others move down
            dws.pages_free(*g.args(), ints([4]), g.page_tokens)
            c.free([4])
            n, _, src, dst, moves = dws.pages_compact(g.refs, g.table)
            dws.pages_copy(pool, src, dst, count=moves)
            assert n.tolist() == [c.compact()[0]] == [2]
        g.same(c)
        at = torch.arange(beams, device="cuda") * 40 + t
        slots = g.table[torch.tensor(rows, device="cuda"), 0].contiguous()
        outs.append(dws.delta_rule_step(*(x[y][at] for y in names), pool, slots=slots))
    for b in range(beams):
        seq = {y: torch.cat([x[y][:10], x[y][b * 40 + 10: b * 40 + 30]]) for y in names}
        want, final = reference(*(seq[y] for y in names), [0, 30], None, dk ** -0.5)
        last = 10 if b == 0 else 20
        close(torch.stack([o[b] for o in outs[:last]]), want[10: 10 + last], torch.float32, "out")
        if b:
            close(pool[c.table[rows[b]][0]], final[0], torch.float32, "state")
        else:
            assert all((o[0] == 0).all() for o in outs[10:])


@pytest.mark.parametrize("pages,most", [(5000, 150), (9000, 300)])
def test_graphs_and_streams(gpu, pages, most):
    """All five captured once and replayed between eager calls, from the same start each time; in one launch each, and
    in three."""
    c = filled(13, pages, 40, most, 16)
    start = OnGpu(c)
    empty = [r for r in range(40) if not c.lengths[r]]
    full = [r for r in range(40) if c.lengths[r]]
    rows, new = ints(full[:8]), ints([min(2400, c.lengths[r] + 33) for r in full[:8]])
    parents, children, gone = ints(full[:len(empty)]), ints(empty), ints(full[-5:])
    gen = torch.Generator().manual_seed(1)
    first = torch.randn(pages, 33, generator=gen).cuda()

    def everything(work):
        refs, table, lengths, pool = work
        for a, b in zip(work, (start.refs, start.table, start.lengths, first)):
            a.copy_(b)
        out = [dws.pages_grow(refs, table, lengths, rows, new, 16)]
        granted, src, dst, count = dws.pages_fork(refs, table, lengths, parents, children, 16)
        dws.pages_copy(pool, src, dst, count=count)
        out += [granted, src, dst, count, dws.pages_free(refs, table, lengths, gone, 16)]
        n, remap, src, dst, moves = dws.pages_compact(refs, table)
        dws.pages_copy(pool, src, dst, count=moves)
        return out + [n, remap, src, dst, moves, refs, table, lengths, pool]

    def room():
        return [torch.empty_like(a) for a in (start.refs, start.table, start.lengths, first)]

    want = [t.clone() for t in everything(room())]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        work = room()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = everything(work)
        graphs.append((graph, got))
    side = torch.cuda.Stream()
    for _ in range(3):
        for _, got in graphs:
            for t in got:
                t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            aside = everything(room())
        for graph, _ in graphs:
            graph.replay()
        eager = everything(room())
        torch.cuda.synchronize()
        for got in (aside, eager, graphs[0][1], graphs[1][1]):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows", [4097, 200001])
def test_far_more_rows_than_pages(gpu, rows):
    """One tile of pages and many of rows, whose claims of the call before are all forgotten."""
    note(f"pages rows {rows}")
    pages, most, page_tokens, n = 300, 2, 4, 150
    c = Cache(pages, rows, most, page_tokens)
    rng = random.Random(11)
    g = OnGpu(c)
    for step in range(3):
        named = [rng.choice([0, 1, rows - 1, rows, rng.randrange(rows)]) for _ in range(n)]
        new = [rng.randint(0, most * page_tokens) for _ in range(n)]
        granted = dws.pages_grow(*g.args(), ints(named), ints(new), page_tokens)
        assert granted.tolist() == c.grow(named, new)
        parents = [rng.choice(named) for _ in range(n)]
        children = [rng.choice([rows - 2, rng.randrange(rows), rng.randrange(rows)]) for _ in range(n)]
        granted, src, dst, count = dws.pages_fork(*g.args(), ints(parents), ints(children), page_tokens)
        want, a, b = c.fork(parents, children)
        assert granted.tolist() == want and count.tolist() == [len(a)] and src.tolist()[:len(a)] == a
        some = named[::2]
        assert dws.pages_free(*g.args(), ints(some), page_tokens).tolist() == [c.free(some)]
    g.same(c)
