"""Beam selection on the GPU against 64 bits. Parents, tokens and rows are whole numbers: equal."""
import math
import random

import pytest
import torch

import device_wide_prefix_amd as dws
from cache_reference import moves, select
from gpu_util import note

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
# A term of the sum of exponentials is off by 2 units u = 2^-24 of the exponential and by its argument's rounding, at most 40 u
# where the term counts (exp(-28) and above); eight terms are summed in fp32, the rest in fp64. The logarithm takes that as it is.
NORM = 50 * 2.0 ** -24


def check(logits, scores, k=None, finished=None, end=0, rows=None):
    k = logits.shape[1] if k is None else k
    got = dws.beam_select(logits.cuda() if not logits.is_cuda else logits, scores.cuda(), k=k,
                          finished=None if finished is None else finished.cuda(), end_token=end,
                          rows=None if rows is None else rows.cuda())
    want = select(logits.cpu(), scores, k, finished, end)
    value, parents, tokens = (x.cpu() for x in got[:3])
    assert parents.tolist() == [[w for _, w, _ in r] for r in want]
    assert tokens.tolist() == [[t for _, _, t in r] for r in want]
    best = torch.tensor([[s for s, _, _ in r] for r in want], dtype=torch.float64)
    assert torch.equal(value == -math.inf, best == -math.inf)
    fine = best.isfinite()
    assert ((value.double() - best).abs()[fine] <= (best.abs() * 2.0 ** -24 + NORM)[fine]).all()
    if rows is not None:
        new, src, dst = got[3].tolist(), got[4].view(rows.shape).tolist(), got[5].view(rows.shape).tolist()
        for b, p in enumerate(parents.tolist()):
            assert (new[b], src[b], dst[b]) == moves(p, rows[b].tolist())
    return got


def made(seed, batch, beams, vocab, dtype):
    gen = torch.Generator().manual_seed(seed)
    logits = (2.5 * torch.randn(batch, beams, vocab, generator=gen)).to(dtype)
    return logits, -3 - torch.rand(batch, beams, generator=gen) * 2, gen


SHAPES = [(1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 7, 3), (3, 4, 63, 8), (2, 2, 64, 64), (1, 4, 513, 4), (5, 8, 2049, 16), (2, 32, 1003, 64),
          (1, 64, 300, 64), (70, 2, 999, 2), (3, 5, 20011, 5), (1, 1, 70001, 64), (2, 9, 40000, 33), (300, 4, 129, 4)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_select(gpu, shape, dtype):
    note(f"beam {shape} {dtype}")
    batch, beams, vocab, k = shape
    logits, scores, gen = made(1, batch, beams, vocab, dtype)
    check(logits, scores, k)
    finished = torch.rand(batch, beams, generator=gen) < 0.4
    check(logits, scores, k, finished, vocab // 2)
    check(logits, scores, k, torch.ones(batch, beams, dtype=torch.uint8), vocab - 1)
    if k == beams:
        rows = torch.randperm(batch * beams + 9, generator=gen)[: batch * beams].int().view(batch, beams)
        check(logits, scores, rows=rows)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "steps", "few", "alternating"])
def test_orders(gpu, kind, dtype):
    """Ties go to the lowest beam and token, and no order of the logits is special."""
    note(f"beam order {kind} {dtype}")
    for vocab in (700, 9001):
        at = torch.arange(vocab)
        x = {"equal": at * 0, "rising": at / 64, "falling": -at / 64, "steps": at // 300, "few": (at % 977 == 5) * 3,
             "alternating": (at % 2) * 2 + at / vocab}[kind].to(dtype)
        logits = x.expand(2, 3, vocab).clone()
        for k in (3, 40):
            check(logits, torch.tensor([[-1.0, -1.0, -1.0], [-2.0, -1.0, -3.0]]), k)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_masked_logits(gpu, dtype):
    """Tokens that are not allowed; beams without any; NaN and infinities; the type's lowest value as a mask; signed zeros."""
    note(f"beam masked {dtype}")
    logits, scores, gen = made(2, 9, 4, 3001, dtype)
    logits[0, :, 10:] = -math.inf                       # ten tokens each
    logits[1, 1] = -math.inf                            # a beam without any
    logits[2, :, 5:] = -math.inf                        # fewer than are wanted
    logits[2, 0, 1:] = -math.inf
    logits[3, 2, 77] = math.nan
    logits[4, 0, 2500] = math.inf
    logits[5] = -math.inf
    logits[6, :, 100:] = torch.finfo(dtype).min
    logits[7] = 0.0
    logits[7, :, ::2] = -0.0
    logits[8, 3] = math.nan
    scores[8, 0], scores[8, 1] = -math.inf, math.nan
    for k in (4, 30):
        check(logits, scores, k)
    check(logits, scores, 30, torch.rand(9, 4, generator=gen) < 0.5, 3000)
    # the first step of a search: all beams but the first are not there yet
    scores[:, 1:] = -math.inf
    check(logits, scores, 4, rows=torch.arange(36, dtype=torch.int32).view(9, 4))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("bad", [math.nan, -math.inf, math.inf])
def test_finished_beams_whatever_their_logits_hold(gpu, bad, dtype):
    """A finished beam goes on with the end token at its own score, its logits computed or not: one value of them that is not
    finite, or all; first, in the middle and last among the beams."""
    note(f"beam finished, logits {bad} {dtype}")
    for vocab in (5, 700, 9001):
        logits, scores, gen = made(9, 6, 4, vocab, dtype)
        over = torch.zeros(6, 4, dtype=torch.bool)
        for b in range(3):
            for at, w in ((slice(vocab // 3, vocab // 3 + 1), b), (slice(None), 3 - b)):
                logits[b, w, at] = bad
                over[b, w] = True
        logits[3:5] = bad                           # all of a request's beams have ended
        over[3:5] = True
        scores[5, 2], over[5, 2] = -math.inf, True  # one that has no score
        end = vocab - 2
        for k in (2, 4, 5):
            value, parents, tokens = (x.cpu() for x in dws.beam_select(logits.cuda(), scores.cuda(), k=k, finished=over.cuda(), end_token=end))
            for b in range(6):
                best = sorted((-float(scores[b, w]), w) for w in range(4) if over[b, w] and scores[b, w].isfinite())
                got = [(-s, w) for s, w, t in zip(value[b].tolist(), parents[b].tolist(), tokens[b].tolist()) if over[b, w] and s > -math.inf]
                assert all(tokens[b, i] == end for i in range(k) if over[b, parents[b, i]] and value[b, i] > -math.inf)
                assert got == best[: len(got)]
                if over[b].all():
                    assert len(got) == min(k, 4) and (value[b, 4:] == -math.inf).all()
                # what is left out is below what was chosen
                assert all(-x <= float(value[b, -1]) for x, _ in best[len(got):])
        check(logits, scores, 4, over, end, rows=torch.randperm(24, generator=gen).int().view(6, 4))


def test_far_apart(gpu):
    """Logits and scores of any size; the largest far above the others."""
    note("beam far apart")
    for dtype, size in ((FP32, 1e30), (FP32, 1e-30), (BF16, 1e30), (FP16, 6e4), (FP32, 80.0)):
        logits, scores, _ = made(3, 3, 4, 5000, FP32)
        check((logits / logits.abs().max() * size).to(dtype), scores * 1000, 8)


def test_strides_and_places(gpu):
    """Logits inside wider arrays that start anywhere, the last of several positions, one row for all beams."""
    note("beam strides")
    for dtype in (BF16, FP32):
        gen = torch.Generator().manual_seed(4)
        wide = (2 * torch.randn(4, 3, 5, 2100, generator=gen)).to(dtype).cuda()
        scores = -torch.rand(4, 3, generator=gen)
        for shift in range(9):
            check(wide[:, :, -1, shift: 2001 + shift], scores, 6)
        check(wide[:, :1, 0].expand(4, 3, 2100), scores, 6)
        check(wide[0, :, 1:, 3:].transpose(0, 1), -torch.rand(4, 3, generator=gen), 3)


def test_states_follow_their_beams(gpu):
    """Slots of states are reordered in place: pages_copy of the moves."""
    note("beam states")
    logits, scores, gen = made(5, 20, 6, 40, FP32)
    rows = torch.randperm(150, generator=gen)[:120].int().view(20, 6)
    pool = torch.randn(150, 33, generator=gen).cuda()
    want = pool.cpu()
    _, parents, _, new, src, dst = check(logits, scores, rows=rows)
    dws.pages_copy(pool, src, dst)
    for b in range(20):
        assert sorted(new[b].tolist()) == sorted(rows[b].tolist())
        for c in range(6):
            assert torch.equal(pool[int(new[b, c])].cpu(), want[int(rows[b, parents[b, c]])])
    rest = [i for i in range(150) if i not in rows.flatten().tolist()]
    assert torch.equal(pool[rest].cpu(), want[rest])


def test_same_bits_streams_and_graphs(gpu):
    note("beam streams and graphs")
    logits, scores, gen = made(6, 7, 8, 30001, BF16)
    logits, scores = logits.cuda(), scores.cuda()
    rows = torch.arange(56, dtype=torch.int32, device="cuda").view(7, 8)
    want = dws.beam_select(logits, scores, rows=rows)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(12):
        got.append(dws.beam_select(logits, scores, rows=rows, stream=streams[i % 3].cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, dws.beam_select(logits, scores, rows=rows)))
    for i in range(5):
        logits.copy_(2 * torch.randn(logits.shape, generator=gen))
        want = dws.beam_select(logits, scores, rows=rows)
        for g, out in graphs:
            for x in out:
                x.fill_(3)
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(x, y) for x, y in zip(out, want)), i


def test_beyond_32_bits(gpu):
    """Rows more than 2^31 elements from the first."""
    note("beam beyond 32 bits")
    gen = torch.Generator().manual_seed(7)
    wide = torch.empty(3, (1 << 30) + 12345, dtype=BF16, device="cuda")
    part = (2 * torch.randn(3, 2, 3001, generator=gen)).to(BF16)
    logits = wide[:, : 2 * 4000].unflatten(1, (2, 4000))[..., :3001]
    logits.copy_(part)
    got = dws.beam_select(logits, -torch.ones(3, 2, device="cuda"), k=5)
    want = dws.beam_select(part.cuda(), -torch.ones(3, 2, device="cuda"), k=5)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_refusals(gpu):
    logits, scores, _ = made(8, 2, 3, 50, FP32)
    logits, scores = logits.cuda(), scores.cuda()
    rows = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    for call in (lambda: dws.beam_select(logits[0], scores), lambda: dws.beam_select(logits, scores[:1]),
                 lambda: dws.beam_select(logits, scores.half()), lambda: dws.beam_select(logits, scores, rows=rows.long()),
                 lambda: dws.beam_select(logits, scores, k=2, rows=rows), lambda: dws.beam_select(logits, scores, finished=rows),
                 lambda: dws.beam_select(logits.transpose(1, 2), scores)):
        with pytest.raises(ValueError):
            call()
    for more in ({"k": 0}, {"k": 65}, {"k": -1}, {"finished": scores < 0, "end_token": 50}, {"finished": scores < 0, "end_token": -1}):
        with pytest.raises((dws.ScanError, RuntimeError)):
            dws.beam_select(logits, scores, **more)
    with pytest.raises(dws.ScanError):
        dws.beam_select(logits[:, :, :1], scores, k=4)
    with pytest.raises(TypeError):
        dws.beam_select(logits.long(), scores)


def test_empty_batch(gpu):
    got = dws.beam_select(torch.zeros(0, 3, 50, device="cuda"), torch.zeros(0, 3, device="cuda"))
    assert [tuple(x.shape) for x in got] == [(0, 3)] * 3
