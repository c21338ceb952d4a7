"""Cached keys and values on the GPU: what is written, and attention over it, against 64 bits."""
import math
import random
from fractions import Fraction

import pytest
import torch

import device_wide_prefix_amd as dws
from cache_reference import Cache, attention, attention_bound, turned
from gpu_util import note

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def freqs_of(pairs):
    return (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(1, pairs))).float().cuda()


# ---- appending ----------------------------------------------------------------

APPEND = [
    # lens after, new tokens, heads, kv, dk, dv, pairs, adjacent, page, layout
    ([1], [1], 2, 1, 64, 64, 32, False, 16, "heads"),
    ([17, 5, 0, 40, 33], [1, 5, 0, 9, 33], 4, 2, 128, 128, 64, False, 16, "heads"),
    ([17, 5, 40, 33], [3, 5, 9, 32], 6, 3, 128, 64, 32, True, 7, "tokens"),
    ([100, 64, 65], [70, 1, 2], 8, 8, 96, 80, 40, False, 1, "tokens"),
    ([9, 30], [4, 11], 3, 1, 33, 17, 16, True, 5, "tokens"),
    ([9, 30], [4, 11], 3, 3, 33, 17, 13, False, 5, "heads"),
    ([9, 30], [4, 11], 0, 2, 36, 20, 6, False, 100, "beside"),
    ([50, 4], [2, 4], 2, 2, 256, 256, 128, True, 16, "beside"),
    ([50, 4], [2, 4], 2, 2, 256, 8, 0, False, 16, "heads"),
    ([50, 4], [2, 4], 5, 1, 1, 1, 0, False, 3, "tokens"),
    ([50, 4], [2, 4], 5, 1, 2, 3, 1, False, 3, "tokens"),
]


def check_append(c, rows, offsets, k, v, q, freqs, adjacent, before, took, positions=None, skip=()):
    """The pools against `before`, with the tokens of sequences not in `skip` written; `took`: q_out."""
    keys, values = (x.clone() for x in before)
    at = {}
    for i, row in enumerate(rows):
        b, e = offsets[i], offsets[i + 1]
        for j in range(b, e):
            if i in skip:
                if took is not None:
                    assert (took[j] == 0).all()
                continue
            t = c.lens[row] - (e - j)
            position = t if positions is None else positions[j]
            p, s = int(c.table[row, t // c.page]), t % c.page
            if 0 <= p < keys.shape[0]:
                at[p, s] = j
                keys[p, s], values[p, s] = math.inf, v[j].to(values.dtype)
                close_turn(c.keys[p, s], k[j], position, freqs, adjacent)
            if took is not None:
                close_turn(took[j], q[j], position, freqs, adjacent)
    same = torch.ones(keys.shape[:2], dtype=torch.bool)
    for p, s in at:
        same[p, s] = False
    bits = {2: torch.int16, 4: torch.int32}[keys.element_size()]
    assert torch.equal(c.keys.cpu().contiguous().view(bits)[same], keys.cpu().contiguous().view(bits)[same])
    assert torch.equal(c.values.cpu().contiguous().view(bits), values.cpu().contiguous().view(bits))


def close_turn(got, x, position, freqs, adjacent):
    """Rounded once from fp32: half a step of the result, and of (|a| + |b|) 4 units of fp32 for cosine and sine (one each),
    their products and the sum."""
    got, x, freqs = got.double().cpu(), x.cpu(), freqs.cpu()
    want = turned(x, position, freqs, adjacent)
    n, both = freqs.numel(), x.double().abs()
    if n:
        a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
        pair = both[:, a] + both[:, b]
        both[:, a], both[:, b] = pair, pair
        both[:, 2 * n:] = 0
    else:
        both = both * 0
    half = torch.finfo(x.dtype).eps / 2
    # below the normal numbers a step is that of the smallest one
    tiny = torch.finfo(x.dtype).tiny * half
    assert ((got - want).abs() <= half * want.abs() + (1 + half) * 4 * 2.0 ** -24 * both + tiny).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(gpu, case, dtype):
    lens, new, heads, kv, dk, dv, pairs, adjacent, page, layout = APPEND[case]
    note(f"append {case} {dtype}")
    gen = torch.Generator().manual_seed(case)
    c = Cache(case, lens, dtype, kv, dk, dv, page, layout, device="cuda")
    order = random.Random(case).sample(range(len(lens)), len(lens))
    offsets = [0]
    for r in order:
        offsets.append(offsets[-1] + new[r])
    tokens = offsets[-1] + 2                                        # two rows in no sequence
    # parts of one projection, which starts at an odd place
    width = heads * dk + kv * dk + kv * dv
    wide = torch.randn(tokens * width + 1, generator=gen).to(dtype).cuda()[1 if case % 2 else 0:][: tokens * width].view(tokens, width)
    q, k, v = wide.split([heads * dk, kv * dk, kv * dv], dim=1)
    q, k, v = q.view(tokens, heads, dk), k.view(tokens, kv, dk), v.view(tokens, kv, dv)
    freqs = freqs_of(pairs)
    before = c.keys.clone(), c.values.clone()
    got = dws.pages_append(*c.args(), k, v, rows=ints(order), offsets=ints(offsets, torch.int64), freqs=freqs if pairs else None,
                           adjacent=adjacent, q=q if heads else None)
    check_append(c, order, offsets, k, v, q, freqs, adjacent, before, got)
    if heads:
        assert (got[offsets[-1]:] == 0).all()
        # in place, and into a given tensor: the same bits
        given = torch.full((tokens, heads, dk), 3.0, dtype=dtype, device="cuda")
        more = dict(rows=ints(order), offsets=ints(offsets, torch.int64), freqs=freqs if pairs else None, adjacent=adjacent)
        assert dws.pages_append(*c.args(), k, v, q=q, q_out=given, **more) is given
        assert torch.equal(given[: offsets[-1]], got[: offsets[-1]]) and (given[offsets[-1]:] == 3).all()
        rest = wide[:, heads * dk:].clone()
        dws.pages_append(*c.args(), k, v, q=q, q_out=q, **more)
        assert torch.equal(q[: offsets[-1]], got[: offsets[-1]]) and torch.equal(wide[:, heads * dk:], rest)


def test_append_evenly_and_positions(gpu):
    note("append evenly, given positions")
    c = Cache(1, [20, 31, 8], FP32, 2, 64, 64, 16, device="cuda")
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(6, 2, 64, generator=gen).cuda() for _ in range(2))
    q = torch.randn(6, 4, 64, generator=gen).cuda()
    positions = [0, 5, 2**31 - 1, 1000003, -7, 12]
    before = c.keys.clone(), c.values.clone()
    got = dws.pages_append(*c.args(), k, v, freqs=freqs_of(32), positions=ints(positions), q=q)
    check_append(c, [0, 1, 2], [0, 2, 4, 6], k, v, q, freqs_of(32), False, before, got, positions)


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def test_angles_of_far_positions(gpu):
    """Cosine and sine of position * frequency, in whole numbers until the angle is below pi: one unit of fp32 each, as near the
    beginning, one for the correction and two for the function that gives them."""
    note("append, far positions")
    gen = torch.Generator().manual_seed(7)
    positions = [1, 1000003, 2**24 + 1, 999999937, 1 << 30, 2**31 - 1, 2**31 - 2, 2147483629, -(2**31), -1999999973, 1234567891, -5]
    n, pairs = len(positions), 128
    freqs = (0.5 + torch.rand(pairs, generator=gen) * 0.5)
    freqs[:40] *= 4.0 ** -torch.arange(40) % 1 + 0.001
    freqs[0], freqs[1], freqs[2] = 1.0, 6.2831855, 1e-7
    c = Cache(30, [n], FP32, 1, 256, 4, 16, device="cuda")
    k, v, q = (torch.zeros(n, 1, d, device="cuda") for d in (256, 4, 256))
    k[..., :pairs] = 1          # (cos, sin)
    q[..., pairs:] = 1          # (-sin, cos)
    got = dws.pages_append(*c.args(), k, v, freqs=freqs.cuda(), positions=ints(positions), q=q).double().cpu()
    keys = torch.stack([c.keys[int(c.table[0, 0]), t] for t in range(n)]).double().cpu()
    for t, p in enumerate(positions):
        want = []
        for f in freqs.tolist():
            x = p * Fraction(f)
            x = float(x - round(x / (2 * PI)) * 2 * PI)
            want.append((math.cos(x), math.sin(x)))
        cos, sin = torch.tensor(want, dtype=torch.float64).T
        for a, b in ((keys[t, 0, :pairs], cos), (keys[t, 0, pairs:], sin), (got[t, 0, :pairs], -sin), (got[t, 0, pairs:], cos)):
            off = (a - b).abs().max()
            assert off <= 4 * 2.0 ** -24, f"position {p}: {off * 2 ** 24:.3g} units"


def test_append_leaves_out(gpu):
    """Rows outside the table, named twice, not granted, shorter than the tokens or longer than the table; pages that are not there."""
    note("append left out")
    c = Cache(2, [20, 31, 8, 40, 3, 12, 64], BF16, 1, 64, 64, 16, device="cuda")
    c.lengths[6] = c.lens[6] = c.table.shape[1] * 16 + 1
    rows = [0, -1, 1, 7, 1, 2, 3, 4, 5, 6, 2**31 - 1]
    new = [2, 1, 3, 1, 2, 1, 2, 4, 2, 1, 1]
    c.table[5, 0], c.table[0, 1] = -1, 1 << 24
    offsets = [sum(new[:i]) for i in range(len(new) + 1)]
    gen = torch.Generator().manual_seed(4)
    k, v = (torch.randn(sum(new), 1, 64, generator=gen).to(BF16).cuda() for _ in range(2))
    q = torch.randn(sum(new), 2, 64, generator=gen).to(BF16).cuda()
    granted = [1, 1, 1, 1, 1, 0, 7, 1, -1, 1, 1]
    before = c.keys.clone(), c.values.clone()
    got = dws.pages_append(*c.args(), k, v, rows=ints(rows), offsets=ints(offsets, torch.int64), granted=ints(granted),
                           freqs=freqs_of(32), q=q)
    check_append(c, rows, offsets, k, v, q, freqs_of(32), False, before, got, skip=(1, 3, 4, 5, 7, 9, 10))


def test_append_many_sequences(gpu):
    """More sequences than a search round takes, a row named again at the far end."""
    note("append many sequences")
    n = 5000
    rng = random.Random(5)
    rows = rng.sample(range(n), n)
    rows[-1] = rows[0]
    new = [rng.choice([0, 1, 1, 2, 3]) for _ in range(n)]
    new[0], new[-1] = 1, 2
    offsets = [0]
    for x in new:
        offsets.append(offsets[-1] + x)
    table = ints(rng.sample(range(n), n)).view(n, 1)
    lengths = torch.full((n,), 4, dtype=torch.int32, device="cuda")
    keys, values = (torch.zeros(n, 4, 1, 8, device="cuda") for _ in range(2))
    k = torch.arange(offsets[-1] * 8, dtype=torch.float32, device="cuda").view(-1, 1, 8) + 1
    dws.pages_append(keys, values, table, lengths, k, -k, rows=ints(rows), offsets=ints(offsets, torch.int64))
    want = torch.zeros(n, 4, 1, 8)
    pages, k = table.view(-1).tolist(), k.cpu()
    for i, row in enumerate(rows[:-1]):
        for j in range(new[i]):
            want[pages[row], 4 - new[i] + j] = k[offsets[i] + j]
    assert torch.equal(keys.cpu(), want) and torch.equal(values.cpu(), -want)


def test_append_as_many_tokens_as_a_launch_has(gpu):
    note("append, the most tokens")
    tokens, page = 4 * ((2**32 - 1) // 256), 64
    pages = -(-tokens // page)
    k = torch.arange(tokens, dtype=torch.int32, device="cuda").to(torch.int16).view(FP16).view(tokens, 1, 1)
    v = k.view(torch.int16).bitwise_not().view(FP16)
    keys, values = (torch.zeros(pages, page, 1, 1, dtype=FP16, device="cuda") for _ in range(2))
    table = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    dws.pages_append(keys, values, table, ints([tokens]), k, v)
    for pool, x in ((keys, k), (values, v)):
        assert torch.equal(pool.view(torch.int16).flip(0).reshape(-1)[:tokens], x.view(torch.int16).reshape(-1))


@pytest.mark.parametrize("begin,end", [(-(2**62), 2**62), (-(2**63), 5), (-(2**63), 40), (-(2**63), 2**63 - 1), (-1, 2**63 - 1), (-3, 40)])
def test_append_offsets_before_the_first_row(gpu, begin, end):
    """A sequence that says it begins before the call's first token is left out, however far: its length is no 64-bit number, and
    places reckoned with it would lie before the row, or in other rows and pages."""
    note(f"append, offsets {begin} {end}")
    c = Cache(23, [40, 0, 7, 64], BF16, 2, 64, 64, 16, device="cuda")
    gen = torch.Generator().manual_seed(6)
    k, v = (torch.randn(44, 2, 64, generator=gen).to(BF16).cuda() for _ in range(2))
    q = torch.randn(44, 4, 64, generator=gen).to(BF16).cuda()
    bits = [x.clone().view(torch.int16) for x in (c.keys, c.values)]
    for row in range(4):
        got = dws.pages_append(*c.args(), k, v, rows=ints([row]), offsets=ints([begin, end], torch.int64), q=q, freqs=freqs_of(32))
        assert (got == 0).all()
        assert torch.equal(c.keys.view(torch.int16), bits[0]) and torch.equal(c.values.view(torch.int16), bits[1])
    # the sequences beside it are written
    before = c.keys.clone(), c.values.clone()
    offsets = [begin, 2, 5]
    got = dws.pages_append(*c.args(), k, v, rows=ints([0, 2]), offsets=ints(offsets, torch.int64), q=q, freqs=freqs_of(32))
    check_append(c, [0, 2], [0, 2, 5], k, v, q, freqs_of(32), False, before, got, skip=(0,))
    assert (got[5:] == 0).all()


# ---- attention ----------------------------------------------------------------

def run_attention(c, rows, new, heads, scale=None, groups=None, shared=None, seed=0, q=None, lse=True, **more):
    gen = torch.Generator().manual_seed(seed)
    offsets = [0]
    for x in new:
        offsets.append(offsets[-1] + x)
    if q is None:
        q = (1.5 * torch.randn(offsets[-1], heads, c.dk, generator=gen)).to(c.dtype).cuda()
    scale = c.dk ** -0.5 if scale is None else scale
    if groups is not None:
        more.update(groups=ints(groups, torch.int64), shared=ints(shared))
    got = dws.pages_attention(q, *c.args(), rows=ints(rows), offsets=ints(offsets, torch.int64), scale=scale, lse=True, **more)
    return q, offsets, scale, got


def check_attention(c, rows, new, heads, **more):
    q, offsets, scale, (out, lse) = run_attention(c, rows, new, heads, **more)
    want, want_lse, spread, largest = attention(q, *c.args(), rows, offsets, scale)
    bound = attention_bound(want, spread, largest, max(c.lens + [1]), c.dk, c.dtype)
    out, lse = out.double().cpu(), lse.double().cpu()
    nan = want.isnan()
    assert torch.equal(out.isnan(), nan)
    wild = ~want.isfinite()
    assert torch.equal(out[wild & ~nan], want[wild & ~nan])
    off = (out - want).abs()[~wild]
    assert (off <= bound[~wild]).all(), f"off by up to {(off / bound[~wild]).max():.3g} of the bound"
    blind = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, blind) and (out[blind] == 0).all()
    fine = want_lse.isfinite()
    # twice the relative error of a probability, and the logarithm's rounding
    tolerance = (c.dk + 8) * 2.0 ** -24 * largest + (max(c.lens + [1]) / 8 + 64) * 2.0 ** -24 + 4 * 2.0 ** -24 * want_lse.abs()
    assert ((lse - want_lse).abs()[fine] <= tolerance[fine]).all()
    return out


HEADS = [(1, 1), (4, 1), (6, 3), (8, 8), (32, 1), (40, 1), (9, 3)]
DIMS = [(64, 64), (128, 128), (96, 96), (72, 40), (256, 256), (20, 12), (33, 65), (1, 1), (160, 8), (16, 200)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("dims", DIMS)
def test_decode_dimensions(gpu, dims, dtype):
    note(f"attention decode {dims} {dtype}")
    c = Cache(1, [1, 31, 32, 33, 129, 300], dtype, 2, *dims, 16, "heads", device="cuda")
    check_attention(c, [5, 0, 3, 1, 2, 4], [1] * 6, 6)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads,kv", HEADS)
@pytest.mark.parametrize("page,layout", [(16, "heads"), (7, "tokens"), (1, "beside"), (100, "heads")])
def test_decode_heads_and_pages(gpu, heads, kv, page, layout, dtype):
    note(f"attention decode {heads} {kv} {page} {layout} {dtype}")
    c = Cache(2, [127, 128, 1, 513], dtype, kv, 64, 64, page, layout, device="cuda")
    check_attention(c, [1, 3, 0, 2], [1] * 4, heads)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("new", [[2, 1, 3, 4], [33, 0, 200, 1], [1, 300, 17, 64], [0, 0, 0, 5]])
def test_several_tokens(gpu, new, dtype):
    """Drafts and prompts, whose own tokens are seen only by those behind them."""
    note(f"attention {new} {dtype}")
    c = Cache(3, [max(x, 40) + 37 * i for i, x in enumerate(new)], dtype, 2, 128, 128, 16, device="cuda")
    check_attention(c, [0, 1, 2, 3], new, 8)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("share,members,tokens,new", [(4, 3, 64, 1), (4, 8, 512, 1), (8, 17, 320, 1), (4, 5, 96, 3), (3, 40, 32, 2),
                                                      (4, 3, 160, 50), (1, 2, 16, 1)])
def test_groups(gpu, share, members, tokens, new, dtype):
    """A group that shares its first tokens between two sequences that share nothing, and the same without being told."""
    note(f"attention groups {share} {members} {tokens} {new} {dtype}")
    rng = random.Random(4)
    lens = [50] + [tokens + new + rng.randint(0, 150) for _ in range(members)] + [77]
    c = Cache(4, lens, dtype, 2, 64, 96, 16, shared=[(1, members, tokens)], device="cuda")
    rows, counts = list(range(members + 2)), [1] + [new] * members + [2]
    groups = [0, 1, members + 1, members + 2]
    out = check_attention(c, rows, counts, 2 * share, groups=groups, shared=[16, tokens, 32])
    apart = check_attention(c, rows, counts, 2 * share)
    half = torch.finfo(dtype).eps
    assert (out - apart).norm() <= 2 * half * apart.norm()
    # sequences outside any group, and groups without sequences
    check_attention(c, rows, counts, 2 * share, groups=[1, 1, members + 1, members + 1], shared=[5, tokens, 9])


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("dims", [(128, 128), (96, 96), (40, 128), (128, 24), (64, 64), (8, 56), (256, 72), (33, 65), (117, 117), (5, 3),
                                  (142, 64), (170, 170), (256, 256), (136, 248)])
def test_tiles_of_many_queries(gpu, dims, dtype):
    """36, 80 and 160 rows of queries a key head, pages that are not there, and NaN where the pool begins."""
    note(f"attention many queries {dims} {dtype}")
    c = Cache(21, [61, 40, 230], dtype, 2, *dims, 16, "heads", device="cuda")
    c.table[c.table == 0] = -1
    c.table[2, 5] = -1
    c.table[2, 9] = c.keys.shape[0]
    c.keys[0] = c.values[0] = math.nan
    check_attention(c, [0, 1, 2], [20, 9, 40], 8)
    # the tile's end is that of the cache, and of a page
    c = Cache(22, [64, 128, 192], dtype, 1, *dims, 16, "tokens", device="cuda")
    check_attention(c, [2, 0, 1], [33, 64, 17], 4)


def check_own_rounding(c, rows, new, heads, **more):
    """Nothing but the result's own rounding: half a step of it, h = eps / 2. The first part of a weight is less than it is by up to
    two steps, 4 h of it; rounding that costs 4 h^2 of the weight, and 2^-20 of it may be added. The rest is fp32's, as
    attention_bound has it for that type."""
    q, offsets, scale, (out, _) = run_attention(c, rows, new, heads, **more)
    want, _, spread, largest = attention(q, *c.args(), rows, offsets, scale)
    half = torch.finfo(c.dtype).eps / 2
    bound = attention_bound(want, spread, largest, max(c.lens), c.dk, FP32) + half * (1 + half) * want.abs() + (4 * half ** 2 + 2.0 ** -20) * spread
    off = (out.double().cpu() - want).abs()
    assert (off <= bound).all(), f"off by up to {(off / bound).max():.3g} of the bound"


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dims", [(128, 128), (64, 64), (96, 80), (33, 65), (160, 200), (256, 256)])
def test_weights_lose_nothing(gpu, dims, dtype):
    """Tiles of up to 32, 64 and 128 queries, of tokens and of sequences that share their first ones."""
    note(f"attention, weights in two parts {dims} {dtype}")
    c = Cache(26, [150, 230, 90, 400], dtype, 2, *dims, 16, shared=[(0, 2, 96)], device="cuda")
    for new, heads in (([1, 1, 1, 1], 4), ([3, 1, 2, 4], 8), ([5, 9, 7, 8], 14), ([70, 30, 64, 20], 4)):
        check_own_rounding(c, [0, 1, 2, 3], new, heads)
    check_own_rounding(c, [0, 1, 2, 3], [1, 1, 1, 1], 60, groups=[0, 2], shared=[96])


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("dims", [(128, 128), (64, 64), (33, 65), (160, 200)])
def test_weights_in_one_part_where_asked_for(gpu, dims, dtype):
    """Rounded once in tiles of more than 32 queries, and nothing else: the others, and fp32, have the same bits."""
    note(f"attention, weights in one part {dims} {dtype}")
    c = Cache(27, [150, 230, 90, 400], dtype, 2, *dims, 16, shared=[(0, 2, 96)], device="cuda")
    c.values[int(c.table[1, 2]), 3, 0, 5] = math.inf
    for new, heads, more in (([1, 1, 1, 1], 4, {}), ([5, 9, 7, 8], 14, {}), ([70, 30, 64, 20], 4, {}),
                             ([1, 1, 1, 1], 60, {"groups": [0, 2], "shared": [96]})):
        one = check_attention(c, [0, 1, 2, 3], new, heads, one_part=True, **more)
        two = check_attention(c, [0, 1, 2, 3], new, heads, **more)
        same = torch.equal(one.nan_to_num(nan=7.0), two.nan_to_num(nan=7.0))
        assert same == (dtype == FP32 or max(new) * heads // 2 <= 32 and not more)


def test_groups_with_odd_places(gpu):
    """Fewer shared tokens than whole pages, more than the rows have, none; empty places first and last in a group."""
    note("attention groups, odd places")
    c = Cache(5, [200 + i for i in range(6)], BF16, 2, 64, 64, 16, shared=[(0, 6, 192)], device="cuda")
    for shared in (0, 1, 31, 150, 192, -5):
        check_attention(c, list(range(6)), [1] * 6, 4, groups=[0, 6], shared=[shared])
    for rows in ([-1, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, -1], [0, 9, -3, 3, 4, 5], [-1] * 6):
        check_attention(c, rows, [1] * 6, 4, groups=[0, 6], shared=[192])
    # rows that have only the shared pages, and more said to be shared than there is
    c = Cache(6, [192] * 6, BF16, 2, 64, 64, 16, shared=[(0, 6, 192)], device="cuda")
    for shared in (191, 192, 10**9):
        check_attention(c, list(range(6)), [1] * 6, 4, groups=[0, 6], shared=[shared])
    check_attention(c, list(range(6)), [2, 1, 0, 3, 1, 1], 4, groups=[0, 6], shared=[192])


@pytest.mark.parametrize("members,empty", [(6, []), (6, [0]), (6, [3]), (6, [5]), (6, [0, 1, 2, 4]), (6, [0, 1, 2, 3, 4]), (40, list(range(33))),
                                           (40, list(range(0, 40, 2))), (300, list(range(270)))])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_groups_share_whatever_places_are_empty(gpu, members, empty, dtype):
    """The shared tokens are read through the first sequence that has a row, for all of a group: here no other row's table has them."""
    note(f"attention groups, empty places {members} {len(empty)} {dtype}")
    c = Cache(29, [96 + 1 + 7 * (r % 9) for r in range(members)], dtype, 2, 64, 64, 16, shared=[(0, members, 96)], device="cuda")
    rows = [-1 if r in empty else r for r in range(members)]
    for odd in (False, True):       # among the shared values, too
        if odd:
            c.values[int(c.table[0, 3]), 5, 1, 7] = math.inf
        for heads, new in ((4, [1] * members), (16, [1 + r % 2 for r in range(members)])):
            q, offsets, scale, got = run_attention(c, rows, new, heads, groups=[0, members], shared=[96])
            want, _, spread, largest = attention(q, *c.args(), rows, offsets, scale)
            off = (got[0].double().cpu() - want).abs()
            fine = want.isfinite()
            assert torch.equal(got[0].double().cpu()[~fine], want[~fine])
            assert (off <= attention_bound(want, spread, largest, 200, 64, dtype))[fine].all()
            if odd:                 # (rows that are computed again read their own tables)
                continue
            table, live = c.table.clone(), [r for r in range(members) if r not in empty]
            for r in live[1:]:
                table[r, :6] = -1
            again = dws.pages_attention(q, c.keys, c.values, table, c.lengths, rows=ints(rows), offsets=ints(offsets, torch.int64), scale=scale,
                                        groups=ints([0, members], torch.int64), shared=ints([96]), lse=True)
            assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_that_see_nothing(gpu, dtype):
    note(f"attention empty rows {dtype}")
    c = Cache(7, [0, 5, 100, 3, 64, 40], dtype, 2, 64, 64, 16, device="cuda")
    c.table[2, 3] = -1                      # a page in the middle
    c.table[4] = -1                         # all pages
    c.table[5, 0] = c.keys.shape[0]         # a page behind the pool
    check_attention(c, [0, 1, 2, 3, 4, 5, -1, 6, 2**31 - 1, 1], [0, 5, 1, 4, 2, 3, 1, 1, 2, 1], 4)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_values_that_are_not_finite(gpu, dtype):
    """Infinities and NaN reach the queries that see them, in tiles of one and of many queries, and no others; what lies
    behind a row's end is NaN in all of these tests."""
    note(f"attention not finite {dtype}")
    for new in ([1, 1, 1], [9, 4, 1], [60, 40, 70]):
        c = Cache(8, [100, 90, 200], dtype, 2, 64, 64, 16, device="cuda")

        def at(pool, row, t):
            return pool[int(c.table[row, t // 16]), t % 16]

        at(c.values, 0, 97)[0, 3] = math.inf
        at(c.values, 0, 95)[1, 5] = math.nan
        at(c.values, 1, 89)[0] = -math.inf
        at(c.keys, 2, 198)[1, 7] = math.nan
        at(c.keys, 2, 150)[0, 7] = math.inf
        q, offsets, scale, (out, _) = run_attention(c, [0, 1, 2], new, 4)
        want, _, spread, largest = attention(q, *c.args(), [0, 1, 2], offsets, scale)
        out = out.double().cpu()
        assert torch.equal(out.isfinite(), want.isfinite())
        fine = want.isfinite()
        bound = attention_bound(want, spread, largest.nan_to_num(posinf=1e3), 200, 64, dtype)
        assert ((out - want).abs() <= bound)[fine].all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("new,heads,groups", [([1, 1, 1, 1], 4, None), ([1, 1, 1, 1], 4, 96), ([4, 1, 3, 2], 8, None), ([9, 4, 1, 9], 8, None),
                                              ([60, 40, 70, 33], 4, None), ([40, 2, 1, 33], 16, 96), ([1, 1, 1, 1], 64, 96)])
@pytest.mark.parametrize("dims", [(64, 64), (128, 96), (33, 17), (160, 200)])
def test_infinities_among_the_values(gpu, new, heads, groups, dims, dtype):
    """Values that are not finite in the middle of rows, where every query sees them: infinities stay infinities of their sign,
    both signs in one dimension give NaN, and other dimensions nothing of it."""
    note(f"attention infinities {new} {heads} {groups} {dims} {dtype}")
    shared = [(0, 4, groups)] if groups else None
    more = {"groups": [0, 4], "shared": [groups]} if groups else {}
    for row, tokens in ((0, 40), (3, 165)):
        c = Cache(24, [300, 261, 200, 333], dtype, 2, *dims, 16, shared=shared, device="cuda")

        def at(t):
            return c.values[int(c.table[row, t // 16]), t % 16]

        at(tokens)[0, 3] = math.inf
        at(tokens)[1, 5] = -math.inf
        at(tokens + 1)[1, 6] = math.inf
        at(tokens + 20)[1, 6] = -math.inf
        at(tokens + 50)[0, 11] = math.nan
        check_attention(c, [0, 1, 2, 3], new, heads, **more)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("new,heads", [(1, 4), (9, 7), (40, 4), (70, 3)])
def test_infinities_of_any_weight(gpu, new, heads, dtype):
    """Infinite values of tokens whose weights are whole powers of two, from the largest to 2^-30 of it, which 16 bits hold
    exactly and in one part."""
    note(f"attention, infinities of any weight {new} {heads} {dtype}")
    c = Cache(31, [333, 200, 400], dtype, 1, 64, 64, 16, device="cuda")
    c.keys[c.keys.isfinite()] = 0
    q = torch.zeros(3 * new, heads, 64, dtype=dtype, device="cuda")
    q[..., 0] = 1
    for row in range(3):
        for i, (below, at) in enumerate(((0, 37), (1, 33), (5, 64), (10, 70), (14, 71), (20, 90), (24, 95), (27, 96), (30, 100))):
            page, place = int(c.table[row, at // 16]), at % 16
            c.keys[page, place, 0, 0] = -below
            c.values[page, place, 0, 2 * i] = math.inf
            c.values[page, place, 0, 2 * i + 1] = -math.inf
    for more in ({}, {"one_part": True}) if dtype == BF16 else ({},):
        check_attention(c, [0, 1, 2], [new] * 3, heads, q=q, scale=math.log(2.0), **more)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 3.0])
def test_scales(gpu, scale):
    note(f"attention scale {scale}")
    c = Cache(9, [100, 33, 300], FP32, 2, 64, 64, 16, device="cuda")
    check_attention(c, [0, 1, 2], [1, 33, 2], 4, scale=scale)


def test_far_apart_scores(gpu):
    """Scores that rise and fall by hundreds along the row."""
    note("attention far apart scores")
    for dtype in (BF16, FP32):
        c = Cache(10, [700, 700], dtype, 1, 64, 64, 16, device="cuda")
        for r, sign in ((0, 1), (1, -1)):
            for t in range(700):
                c.keys[int(c.table[r, t // 16]), t % 16] = sign * (t - 350) / 8
        q = torch.full((8, 2, 64), 0.5, dtype=dtype, device="cuda")
        check_attention(c, [0, 1], [4, 4], 2, q=q, scale=0.25)


def test_strides(gpu):
    """Queries inside a projection, results inside a wider array, not at multiples of 16 bytes."""
    note("attention strides")
    for dtype, shift in ((BF16, 0), (BF16, 1), (FP16, 2), (FP32, 1)):
        c = Cache(11, [90, 130, 40], dtype, 2, 48, 48, 16, "tokens", device="cuda")
        gen = torch.Generator().manual_seed(1)
        wide = torch.randn(20, 500, generator=gen).to(dtype).cuda()
        q = wide[:, shift: shift + 4 * 48].view(20, 4, 48)[:15]
        out = torch.full((20, 333), 7.0, dtype=dtype, device="cuda")
        inside = out[:, shift: shift + 192].view(20, 4, 48)[:15]
        new = [4, 10, 1]
        got = check_attention(c, [2, 0, 1], new, 4, q=q, out=inside)
        assert torch.equal(inside.double().cpu(), got)
        assert (out[15:] == 7).all() and (out[:, :shift] == 7).all() and (out[:, shift + 192:] == 7).all()


def test_rest_of_the_rows(gpu):
    note("attention rest")
    c = Cache(12, [90, 130], BF16, 2, 64, 64, 16, device="cuda")
    q = torch.randn(12, 4, 64, device="cuda").to(BF16)
    offsets = ints([3, 5, 9], torch.int64)
    out, lse = dws.pages_attention(q, *c.args(), offsets=offsets, lse=True)
    assert (out[:3] == 0).all() and (out[9:] == 0).all() and (lse[:3] == -math.inf).all() and (lse[9:] == -math.inf).all()
    given, given_lse = torch.full_like(out, 5), torch.full_like(lse, 5)
    assert dws.pages_attention(q, *c.args(), offsets=offsets, out=given, lse=given_lse)[0] is given
    assert torch.equal(given[3:9], out[3:9]) and (given[:3] == 5).all() and (given[9:] == 5).all()
    assert torch.equal(given_lse[3:9], lse[3:9]) and (given_lse[:3] == 5).all() and (given_lse[9:] == 5).all()
    alone = dws.pages_attention(q[3:9].contiguous(), *c.args(), offsets=offsets - 3)
    assert torch.equal(alone, out[3:9])
    # no sequences, no tokens
    none = dws.pages_attention(q, *c.args(), rows=ints([]), offsets=ints([0], torch.int64))
    assert (none == 0).all()
    assert dws.pages_attention(q[:0], *c.args()).shape == (0, 4, 64)


def test_rest_of_given_and_new_results(gpu):
    """Rows in no sequence stay as they were in a given tensor, and are set in a new one, whichever of the two results is which."""
    note("attention, rest of given and new results")
    c = Cache(28, [90, 130], FP32, 2, 64, 64, 16, device="cuda")
    q = torch.randn(12, 4, 64, device="cuda")
    offsets = ints([3, 5, 9], torch.int64)
    want, want_lse = dws.pages_attention(q, *c.args(), offsets=offsets, lse=True)
    rest = [0, 1, 2, 9, 10, 11]
    for new_out in (False, True):
        for new_lse in (False, True):
            out, lse = (torch.full_like(x, 5) for x in (want, want_lse))
            got, got_lse = dws.pages_attention(q, *c.args(), offsets=offsets, out=None if new_out else out, lse=True if new_lse else lse)
            assert (got is out) != new_out and (got_lse is lse) != new_lse
            assert torch.equal(got[3:9], want[3:9]) and torch.equal(got_lse[3:9], want_lse[3:9])
            assert (got[rest] == (0 if new_out else 5)).all(), (new_out, new_lse)
            assert (got_lse[rest] == (-math.inf if new_lse else 5)).all(), (new_out, new_lse)


def test_offsets_that_are_wrong(gpu):
    """Offsets, groups and lengths that make no sense: nothing outside the arrays is touched, and the right sequences of
    another call are as before."""
    note("attention wrong offsets")
    c = Cache(13, [90, 130, 40, 64], BF16, 2, 64, 64, 16, device="cuda")
    q = torch.randn(40, 8, 64, device="cuda").to(BF16)
    right = dws.pages_attention(q[:4], *c.args())
    around = torch.full((3, 40, 8, 64), 2.0, dtype=BF16, device="cuda")
    for offsets in ([0, 50, 3, 40, 40], [-7, 5, 10**12, 2, 30], [40, 0, 40, 0, 40], [5, 4, 3, 2, 1], [-(2**62), 2**62, 0, 40, 2**62]):
        for groups, shared in ((None, None), ([0, 3, 1, 4], [32, 64, 2**31 - 1]), ([-5, 2**60, 0, 9], [-(2**31), 80, 80])):
            more = {} if groups is None else {"groups": ints(groups, torch.int64), "shared": ints(shared)}
            dws.pages_attention(q, *c.args(), offsets=ints(offsets, torch.int64), out=around[1], **more)
            k = torch.randn(40, 2, 64, device="cuda").to(BF16)
            kept = c.keys.clone(), c.values.clone()
            dws.pages_append(*c.args(), k, k, offsets=ints(offsets, torch.int64), q=q)
            c.keys.copy_(kept[0])
            c.values.copy_(kept[1])
    lengths = ints([2**31 - 1, -5, 81, 10**6])
    dws.pages_attention(q[:4], *c.args()[:3], lengths, out=around[1][:4])
    assert (around[0] == 2).all() and (around[2] == 2).all()
    assert torch.equal(dws.pages_attention(q[:4], *c.args()), right)


@pytest.mark.parametrize("n", [700, 2500])
def test_many_sequences(gpu, n):
    """More sequences and groups than the plan takes at a time or keeps beside it."""
    note(f"attention many sequences {n}")
    rng = random.Random(14)
    lens = [rng.choice([1, 2, 17, 30, 33]) for _ in range(n)]
    shared = [(i, 4, 16) for i in range(0, n - 8, 4) if min(lens[i: i + 4]) > 16]
    c = Cache(14, lens, FP32, 1, 8, 8, 16, shared=shared, device="cuda")
    bounds = list(range(0, n - 8, 4)) + [n - 8]
    of = {first: tokens for first, _, tokens in shared}
    check_attention(c, list(range(n)), [1] * n, 2, groups=bounds, shared=[of.get(b, 0) for b in bounds[:-1]])
    many = [rng.choice([0, 1, 1, 3]) for _ in range(n)]
    many = [min(x, y) for x, y in zip(many, lens)]
    check_attention(c, list(range(n)), many, 2)


def wide_reference(q, k, v, scale):
    """One sequence's last tokens, (heads, tokens, dim) in 64 bits on the GPU."""
    x = (q.double() @ k.double().transpose(1, 2)) * scale
    new, n = x.shape[1:]
    hidden = torch.ones(new, n, dtype=torch.bool, device=x.device).triu(n - new + 1)
    return torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v.double()


@pytest.mark.parametrize("dtype,dim,new,length", [(BF16, 128, 1, 300001), (BF16, 64, 700, 5003), (FP16, 256, 130, 9000), (FP32, 128, 3, 40000)])
def test_long_rows(gpu, dtype, dim, new, length):
    note(f"attention long {dtype} {dim} {new} {length}")
    gen = torch.Generator(device="cuda").manual_seed(15)
    page, kv, heads = 16, 2, 8
    pages = -(-length // page)
    keys, values = (torch.randn(pages, kv, page, dim, generator=gen, device="cuda").to(dtype).transpose(1, 2) for _ in range(2))
    table = torch.randperm(pages, generator=gen, device="cuda").int()[None].contiguous()
    q = torch.randn(new, heads, dim, generator=gen, device="cuda").to(dtype)
    out = dws.pages_attention(q, keys, values, table, ints([length]), offsets=ints([0, new], torch.int64))
    k, v = (x[table[0].long()].permute(2, 0, 1, 3).reshape(kv, -1, dim)[:, :length] for x in (keys, values))
    per = heads // kv
    want = torch.cat([wide_reference(q[:, h * per: (h + 1) * per].transpose(0, 1), k[h: h + 1], v[h: h + 1], dim ** -0.5) for h in range(kv)])
    off = (out.double() - want.transpose(0, 1)).norm() / want.norm()
    # rounding the result and the probabilities: each at most half a step of every value; fp32 as the scores' sums
    assert off <= (2 * torch.finfo(dtype).eps / 2 if dtype != FP32 else 64 * 2.0 ** -24), off


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("below", [11.0, 14.0, 16.3, 17.7, 20.0])
@pytest.mark.parametrize("new,heads", [(1, 2), (3, 8), (1, 48), (40, 3)])
def test_one_token_far_above_many(gpu, new, heads, below, dtype):
    """A token that outweighs each of 100,000 others by e^below, which together still weigh what counts: first, in the middle and
    last, in tiles of up to 32 queries and of more. What a weight loses to its type's range is a loss in one direction. As many
    rows (with the same pages) as workgroups, so that each row's maximum goes along with all of it."""
    note(f"attention one above many {new} {heads} {below} {dtype}")
    n, rows, dim, page = 100001, 530, 64, 64
    gen = torch.Generator(device="cuda").manual_seed(25)
    pages = -(-n // page)
    table = torch.randperm(pages, generator=gen, device="cuda").int().expand(rows, pages).contiguous()
    values = (0.5 + torch.rand(pages, page, 1, dim, generator=gen, device="cuda")).to(dtype)
    q = torch.zeros(rows * new, heads, dim, device="cuda", dtype=dtype)
    q[..., 0] = 1
    offsets = torch.arange(0, rows * new + 1, new, device="cuda")
    for place in (0, n // 2, n - new):
        keys = torch.zeros(pages, page, 1, dim, device="cuda", dtype=dtype)
        at = table[0, place // page].long(), place % page
        keys[at][0, 0] = below
        kept = values[at].clone()
        values[at] = 0.0625
        out, lse = dws.pages_attention(q, keys, values, table, ints([n] * rows), offsets=offsets, scale=1.0, lse=True)
        k, v = (x[table[0].long()].reshape(-1, dim)[:n].double() for x in (keys, values))
        values[at] = kept
        for j in {0, new - 1}:
            seen = n - new + 1 + j
            x = k[:seen, 0]
            w = torch.softmax(x, 0)
            want = w @ v[:seen]
            largest = torch.full((1,), float(x.max()), dtype=torch.float64)
            # (fp32 products add two tokens a step, not 16: n / 2 steps of a sum)
            bound = attention_bound(want[None].cpu(), want[None].cpu(), largest, 8 * n if dtype == FP32 else n, 1, dtype)[0].cuda()
            off = (out.view(rows, new, heads, dim)[:, j].double() - want).abs()
            assert (off <= bound).all(), f"off by up to {(off / bound).max():.3g} of the bound"
            exact = float(torch.logsumexp(x, 0))
            assert (lse.view(rows, new, heads)[:, j].double() - exact).abs().max() <= (n / 8 + 64 + 9 * below + 4 * exact) * 2.0 ** -24


def test_far_apart_scores_in_fp16(gpu):
    """Scores that rise and fall by hundreds along the row, with the range of fp16."""
    note("attention far apart scores, fp16")
    for tokens, heads in ((4, 2), (4, 24), (60, 2)):
        c = Cache(10, [700, 700], FP16, 1, 64, 64, 16, device="cuda")
        for r, sign in ((0, 1), (1, -1)):
            for t in range(700):
                c.keys[int(c.table[r, t // 16]), t % 16] = sign * (t - 350) / 8
        for scale in (0.25, 0.01):
            q = torch.full((2 * tokens, heads, 64), 0.5, dtype=FP16, device="cuda")
            check_attention(c, [0, 1], [tokens, tokens], heads, q=q, scale=scale)


def test_pool_beyond_32_bits(gpu):
    """Pages more than 2^32 bytes and 2^31 elements from the pool's beginning, written and read."""
    note("attention beyond 32 bits")
    page, kv, dim = 16, 8, 128
    pages = (1 << 31) // (page * kv * dim) + 40
    keys, values = (torch.empty(pages, page, kv, dim, dtype=BF16, device="cuda") for _ in range(2))
    n = 200
    table = torch.tensor([[pages - 1 - 3 * i if i % 2 else i for i in range(13)]], dtype=torch.int32, device="cuda")
    for x in (keys, values):
        x[table[0].long()] = math.nan
    gen = torch.Generator().manual_seed(16)
    k, v = (torch.randn(n, kv, dim, generator=gen).to(BF16).cuda() for _ in range(2))
    q = torch.randn(1, 16, dim, generator=gen).to(BF16).cuda()
    lengths = ints([n])
    dws.pages_append(keys, values, table, lengths, k, v)
    out = dws.pages_attention(q, keys, values, table, lengths)
    kk, vv = (x.transpose(0, 1).double() for x in (k, v))
    want = torch.cat([wide_reference(q[:, 2 * h: 2 * h + 2].transpose(0, 1), kk[h: h + 1], vv[h: h + 1], dim ** -0.5) for h in range(kv)])
    assert (out.double() - want.transpose(0, 1)).norm() / want.norm() <= torch.finfo(BF16).eps


@pytest.mark.parametrize("new", [1, 30])
def test_pages_far_apart(gpu, new):
    """Three pages 33 GiB apart, keys and values beside each other in their rows."""
    note(f"attention pages far apart {new}")
    page, kv, dk, dv, n = 16, 2, 64, 96, 43
    step = 33 * 2 ** 30 // 2
    pool = torch.empty(2 * step + page * kv * (dk + dv), dtype=BF16, device="cuda")
    pool = pool.as_strided((3, page, kv, dk + dv), (step, kv * (dk + dv), dk + dv, 1))
    pool.fill_(math.nan)
    keys, values = pool.split([dk, dv], dim=3)
    table, lengths = ints([[2, 0, 1]]), ints([n])
    gen = torch.Generator().manual_seed(17)
    k, v = (torch.randn(n, kv, d, generator=gen).to(BF16).cuda() for d in (dk, dv))
    q = torch.randn(new, 4 * kv, dk, generator=gen).to(BF16).cuda()
    dws.pages_append(keys, values, table, lengths, k, v)
    out = dws.pages_attention(q, keys, values, table, lengths, offsets=ints([0, new], torch.int64))
    kk, vv = (x.transpose(0, 1) for x in (k, v))
    want = torch.cat([wide_reference(q[:, 4 * h: 4 * h + 4].transpose(0, 1), kk[h: h + 1], vv[h: h + 1], dk ** -0.5) for h in range(kv)])
    assert (out.double() - want.transpose(0, 1)).norm() / want.norm() <= torch.finfo(BF16).eps


def test_tables_for_very_long_rows(gpu):
    """Tables that could hold 2^31 tokens a row: what a row may cost is counted in larger units, and rounded."""
    note("attention, tables for very long rows")
    page, kv, dim = 1024, 2, 64
    lens = [1, 70, 5000, 1024, 30011, 2, 900, 4096] * 3
    gen = torch.Generator().manual_seed(18)
    need = [-(-n // page) for n in lens]
    keys, values = (torch.randn(sum(need), page, kv, dim, generator=gen).to(BF16).cuda() for _ in range(2))
    table = torch.full((len(lens), 2 ** 21 - 1), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(need), generator=gen).int(), 0
    for r, x in enumerate(need):
        table[r, :x] = order[at: at + x]
        at += x
    new = [min(n, (1, 40, 3)[r % 3]) for r, n in enumerate(lens)]
    offsets = torch.tensor([0] + new).cumsum(0)
    q = torch.randn(int(offsets[-1]), 8, dim, generator=gen).to(BF16).cuda()
    out = dws.pages_attention(q, keys, values, table.cuda(), ints(lens), offsets=offsets.cuda())
    for r, n in enumerate(lens):
        pages, b, e = table[r, : need[r]].long().cuda(), int(offsets[r]), int(offsets[r + 1])
        k, v = (x[pages].reshape(-1, kv, dim)[:n].transpose(0, 1) for x in (keys, values))
        want = torch.cat([wide_reference(q[b:e, 4 * h: 4 * h + 4].transpose(0, 1), k[h: h + 1], v[h: h + 1], dim ** -0.5) for h in range(kv)])
        assert (out[b:e].double() - want.transpose(0, 1)).norm() / want.norm() <= torch.finfo(BF16).eps, (r, n)


def test_same_bits_every_time(gpu):
    note("attention same bits")
    c = Cache(17, [500, 700, 20, 300], BF16, 2, 128, 128, 16, shared=[(0, 2, 480)], device="cuda")
    one = run_attention(c, [0, 1, 2, 3], [1, 2, 5, 100], 8, groups=[0, 2, 4], shared=[480, 0])[3]
    for _ in range(20):
        again = run_attention(c, [0, 1, 2, 3], [1, 2, 5, 100], 8, groups=[0, 2, 4], shared=[480, 0])[3]
        assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])


def test_streams(gpu):
    """Calls on streams of their own at the same time."""
    note("attention streams")
    c = Cache(18, [900, 1200, 64], BF16, 2, 128, 128, 16, device="cuda")
    q = torch.randn(3, 8, 128, device="cuda").to(BF16)
    want = dws.pages_attention(q, *c.args())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(12):
        s = streams[i % 3]
        if i % 2:
            with torch.cuda.stream(s):
                got.append(dws.pages_attention(q, *c.args()))
        else:
            got.append(dws.pages_attention(q, *c.args(), stream=s.cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


def test_graph_follows_the_cache(gpu):
    """A captured step of appending and attending, replayed as the rows grow, beside another one on the same cache."""
    note("attention graph")
    c = Cache(19, [20, 33, 64], BF16, 2, 64, 64, 16, device="cuda")
    table = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
    table[:, : c.table.shape[1]] = c.table
    keys, values = (torch.cat([x, torch.zeros(20, *x.shape[1:], dtype=BF16, device="cuda")]) for x in (c.keys, c.values))
    fresh = iter(range(c.keys.shape[0], c.keys.shape[0] + 20))
    lengths = c.lengths.clone()
    q, k, v = (torch.randn(3, h, 64, device="cuda").to(BF16) for h in (4, 2, 2))
    freqs = freqs_of(32)

    def step():
        turned_q = dws.pages_append(keys, values, table, lengths, k, v, freqs=freqs, q=q)
        return dws.pages_attention(turned_q, keys, values, table, lengths, lse=True)

    lens = list(c.lens)

    def grow():
        for r in range(3):
            if lens[r] % 16 == 0:
                table[r, lens[r] // 16] = next(fresh)
            lens[r] += 1
        lengths.copy_(ints(lens))

    grow()
    step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    for i in range(8):
        grow()
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        want = step()
        for g, got in graphs:
            for x in got:
                x.fill_(9)
            g.replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


def test_refusals(gpu):
    c = Cache(20, [20, 33], BF16, 2, 64, 32, 16, device="cuda")
    q, k, v = (torch.randn(2, h, d, device="cuda").to(BF16) for h, d in ((4, 64), (2, 64), (2, 32)))
    keys, values, table, lengths = c.args()
    for call in (lambda: dws.pages_attention(q[:, :3], *c.args()), lambda: dws.pages_attention(q.float(), *c.args()),
                 lambda: dws.pages_attention(q[0], *c.args()), lambda: dws.pages_attention(q, keys, values[:-1], table, lengths),
                 lambda: dws.pages_attention(q, keys, values, table.long(), lengths),
                 lambda: dws.pages_attention(q, keys, values, table, lengths[:1]),
                 lambda: dws.pages_attention(q[:1], *c.args()), lambda: dws.pages_attention(q, *c.args(), groups=ints([0, 2], torch.int64)),
                 lambda: dws.pages_attention(q, *c.args(), groups=ints([0, 2], torch.int64), shared=ints([1, 2])),
                 lambda: dws.pages_attention(q, *c.args(), rows=ints([0, 1], torch.int64)),
                 lambda: dws.pages_attention(q, *c.args(), lse=torch.zeros(2, 4, device="cuda", dtype=BF16)),
                 lambda: dws.pages_attention(q, *c.args(), out=q),
                 lambda: dws.pages_append(*c.args(), k, v[:1]), lambda: dws.pages_append(*c.args(), k, k),
                 lambda: dws.pages_append(*c.args(), k, v, freqs=freqs_of(33)), lambda: dws.pages_append(*c.args(), k, v, q_out=q),
                 lambda: dws.pages_append(*c.args(), k, v, granted=ints([1])), lambda: dws.pages_append(*c.args(), k, v, q=k[..., :32])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(dws.ScanError):
        dws.pages_attention(keys[0, :2], *c.args(), out=keys[0, :2, :, :32])
    with pytest.raises(dws.ScanError):
        dws.pages_append(*c.args(), keys[0, :2], v)
    with pytest.raises(dws.ScanError):
        dws.pages_attention(q, *c.args(), scale=math.inf)
