"""Host-side checks of the calls on cached keys and values and of the beam selection: refusals before any HIP call."""
import ctypes
import os

import pytest
import torch

import device_wide_prefix_amd as dws

FAKE = 0x10000000      # never dereferenced: every call here fails its checks, or has no tokens
BAD, UNSUPPORTED, OVERLAP, MISALIGNED = dws.ERR_INVALID_ARG, dws.ERR_UNSUPPORTED, dws.ERR_OVERLAP, dws.ERR_MISALIGNED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dws.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dws.load_library()


def room(k):
    return FAKE + 0x1000000 * k


def put(a, changes):
    """Sets members by their dotted names."""
    for name, x in changes.items():
        at = a
        *path, last = name.split(".")
        for part in path:
            at = getattr(at, part)
        setattr(at, last, x)
    return a


def shared_parts(a, tokens=64):
    """A bf16 cache of 10 pages of 16 tokens, 2 heads of 64 and 32 dimensions, and the tokens of 4 sequences."""
    put(a, {"cache.keys": dws.PagePool(room(1), 16 * 128, 128, 64), "cache.values": dws.PagePool(room(2), 16 * 64, 64, 32),
            "cache.d_table": room(3), "cache.d_lengths": room(4), "cache.n_pages": 10, "cache.n_rows": 6, "cache.max_pages": 5,
            "cache.page_tokens": 16, "cache.heads": 2, "cache.dim_k": 64, "cache.dim_v": 32, "cache.dtype": dws.BFLOAT16,
            "seqs.tokens": tokens, "seqs.n": 4, "seqs.d_offsets": room(5), "seqs.d_rows": room(6), "heads_q": 4})
    a.q = dws.Rows(room(7), 256, 64)
    return a


def append_args(**more):
    a = shared_parts(dws.PagesAppendArgs())
    a.q_out, a.k, a.v = dws.Rows(room(8), 256, 64), dws.Rows(room(9), 128, 64), dws.Rows(room(10), 64, 32)
    put(a, {"pairs": 16, "d_freqs": room(11), "d_granted": room(12), "d_positions": room(13)})
    return put(a, more)


def attention_args(**more):
    a = shared_parts(dws.PagesAttentionArgs())
    a.out = dws.Rows(room(8), 128, 32)
    put(a, {"scale": 0.1, "n_groups": 2, "d_groups": room(9), "d_shared": room(10), "d_lse": room(11)})
    return put(a, more)


def beam_args(**more):
    a = dws.BeamArgs(d_logits=room(1), batch=3, beams=4, vocab=1000, batch_stride=4000, beam_stride=1000, dtype=dws.FLOAT16, k=4,
                     d_scores=room(2), d_finished=room(3), end_token=7, d_rows=room(4), d_out_scores=room(5), d_parents=room(6),
                     d_tokens=room(7), d_out_rows=room(8), d_src=room(9), d_dst=room(10))
    return put(a, more)


def status(lib, a):
    name = {dws.PagesAppendArgs: "dws_pages_append", dws.PagesAttentionArgs: "dws_pages_attention",
            dws.BeamArgs: "dws_beam_select"}[type(a)]
    return getattr(lib, name)(ctypes.byref(a), None)


SHARED = [
    ({"cache.dtype": dws.INT32}, BAD), ({"cache.dtype": 9}, BAD), ({"cache.n_pages": 0}, BAD), ({"cache.n_rows": -1}, BAD),
    ({"cache.max_pages": -1}, BAD), ({"cache.page_tokens": 0}, BAD), ({"cache.heads": 0}, BAD), ({"cache.dim_k": 0}, BAD),
    ({"cache.dim_v": -5}, BAD), ({"heads_q": -1}, BAD), ({"seqs.tokens": -1}, BAD), ({"seqs.n": -1}, BAD),
    ({"seqs.n": 0, "seqs.d_offsets": None}, BAD), ({"seqs.n": 5, "seqs.d_offsets": None}, BAD),
    ({"cache.n_pages": (1 << 24) + 1}, UNSUPPORTED), ({"cache.n_rows": 1 << 31}, UNSUPPORTED),
    ({"cache.max_pages": 1 << 31}, UNSUPPORTED), ({"cache.page_tokens": 1 << 31}, UNSUPPORTED),
    ({"cache.n_rows": 1 << 30, "cache.max_pages": 1 << 30}, UNSUPPORTED), ({"cache.heads": 65536}, UNSUPPORTED),
    ({"cache.dim_k": 257}, UNSUPPORTED), ({"cache.dim_v": 300}, UNSUPPORTED), ({"seqs.tokens": 1 << 31}, UNSUPPORTED),
    ({"seqs.n": 1 << 31}, UNSUPPORTED),
    ({"cache.keys.data": None}, BAD), ({"cache.values.data": None}, BAD), ({"cache.d_table": None}, BAD),
    ({"cache.d_lengths": None}, BAD), ({"q.data": None}, BAD), ({"cache.keys.page_stride": -1}, BAD),
    ({"cache.values.head_stride": (1 << 40) + 1}, BAD), ({"q.token_stride": -1}, BAD), ({"q.head_stride": 1 << 41}, BAD),
    ({"cache.keys.page_stride": 1 << 40, "cache.n_pages": 1 << 24}, BAD), ({"q.data": 2**64 - 64}, BAD),
    ({"cache.keys.data": room(1) + 1}, MISALIGNED), ({"cache.d_table": room(3) + 2}, MISALIGNED),
    ({"seqs.d_offsets": room(5) + 4}, MISALIGNED), ({"seqs.d_rows": room(6) + 2}, MISALIGNED), ({"q.data": room(7) + 1}, MISALIGNED),
]


@pytest.mark.parametrize("make", [append_args, attention_args])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared_refusals(lib, make, case):
    changes, want = SHARED[case]
    assert status(lib, make(**changes)) == want, changes


def test_refusals_of_append(lib):
    assert lib.dws_pages_append(None, None) == BAD
    for changes, want in (
            ({"pairs": -1}, BAD), ({"pairs": 33}, BAD), ({"d_freqs": None}, BAD), ({"k.data": None}, BAD), ({"v.data": None}, BAD),
            ({"q_out.data": None}, BAD), ({"d_freqs": room(11) + 2}, MISALIGNED), ({"d_granted": room(12) + 1}, MISALIGNED),
            ({"d_positions": room(13) + 1}, MISALIGNED),
            # written twice
            ({"cache.keys.head_stride": 32}, BAD), ({"cache.keys.head_stride": 0}, BAD), ({"cache.values.page_stride": 0}, BAD),
            ({"cache.values.token_stride": 33}, BAD), ({"q_out.token_stride": 255}, BAD), ({"q_out.head_stride": 63}, BAD),
            # written over what is read, or written twice
            ({"cache.values.data": room(1) + 64}, OVERLAP), ({"k.data": room(1) + 2 * 16 * 128}, OVERLAP),
            ({"q_out.data": room(7) + 2}, OVERLAP), ({"q_out.data": room(9)}, OVERLAP), ({"cache.d_lengths": room(1)}, OVERLAP),
            ({"cache.d_table": room(2) + 8}, OVERLAP), ({"d_positions": room(8) + 16}, OVERLAP),
            # queries half beside the keys in rows of 300: the last head reaches into them
            ({"q_out.data": room(9) - 2 * 150, "q_out.token_stride": 300, "q_out.head_stride": 40, "k.token_stride": 300,
              "cache.dim_k": 40, "cache.keys.head_stride": 64}, OVERLAP)):
        assert status(lib, append_args(**changes)) == want, changes
    # nothing to write: accepted without a launch
    assert status(lib, append_args(**{"seqs.tokens": 0, "k.data": None, "v.data": None, "q.data": None, "q_out.data": None})) == dws.OK


def test_append_refuses_more_tokens_than_a_launch_has(lib):
    """A wave of 64 threads a token, four to a workgroup, and at most 2^32 - 1 threads: refused before any HIP call."""
    far = {"cache.n_rows": 1, "cache.max_pages": 1 << 24, "cache.n_pages": 1 << 24, "cache.page_tokens": 128, "heads_q": 0, "pairs": 0,
           "cache.heads": 1, "cache.dim_k": 1, "cache.dim_v": 1, "cache.keys": dws.PagePool(1 << 40, 128, 1, 1),
           "cache.values": dws.PagePool(1 << 41, 128, 1, 1), "k": dws.Rows(1 << 42, 1, 1), "v": dws.Rows(1 << 43, 1, 1),
           "d_granted": None, "d_positions": None}
    for tokens in (4 * ((2**32 - 1) // 256) + 1, 1 << 26, 1 << 28, (1 << 31) - 1):
        assert status(lib, append_args(**{**far, "seqs.tokens": tokens})) == UNSUPPORTED, tokens


def test_parts_of_one_pool_do_not_overlap(lib):
    """Keys beside values in every page, in every token's row, and with heads outside."""
    empty = {"seqs.tokens": 0, "cache.dim_v": 64}
    for keys, values in (((2 * 2048, 128, 64), 2048), ((16 * 256, 256, 64), 128), ((2 * 16 * 128, 128, 16 * 128), 64),
                         ((16 * 256, 256, 128), 64), ((2 * 2 * 1024, 64, 1024), 2048)):
        def pools(shift):
            return {**empty, "cache.keys": dws.PagePool(room(1), *keys), "cache.values": dws.PagePool(room(1) + 2 * shift, *keys)}

        assert status(lib, append_args(**pools(values))) == dws.OK, keys
        assert status(lib, append_args(**pools(values - 8))) == OVERLAP, keys
        assert status(lib, append_args(**pools(values + 8))) == OVERLAP, keys
        assert status(lib, append_args(**pools(0))) == OVERLAP, keys


def test_pools_that_lie_in_one_another(lib):
    """Equal strides of any size, none a multiple of another: refused exactly where an element is in both, told element by
    element. (A call without tokens that is not refused ends well, and launches nothing.)"""
    for page, token, head, dim in ((5000, 301, 150, 70), (1203, 600, 75, 37), (700, 40, 20, 10), (80, 20, 641, 9)):
        pages, page_tokens, heads = 3, 2, 2

        def elements(at):
            return {at + i * page + j * token + k * head + d for i in range(pages) for j in range(page_tokens) for k in range(heads)
                    for d in range(dim)}

        keys = elements(0)
        for shift in list(range(-2 * head, 2 * head)) + [page - 3, page + 1, token + dim, -page + dim, -token - dim]:
            a = append_args(**{"seqs.tokens": 0, "heads_q": 0, "cache.n_pages": pages, "cache.page_tokens": page_tokens,
                               "cache.heads": heads, "cache.dim_k": dim, "cache.dim_v": dim, "pairs": 0,
                               "cache.keys": dws.PagePool(room(21), page, token, head),
                               "cache.values": dws.PagePool(room(21) + 2 * shift, page, token, head)})
            want = OVERLAP if keys & elements(shift) else dws.OK
            assert status(lib, a) == want, (page, token, head, dim, shift)


def test_refusals_of_attention(lib):
    assert lib.dws_pages_attention(None, None) == BAD
    need = ctypes.c_size_t(0)
    size = lib.dws_pages_attention_workspace
    assert size(None, ctypes.byref(need)) == BAD and size(ctypes.byref(attention_args()), None) == BAD
    assert size(ctypes.byref(attention_args()), ctypes.byref(need)) == dws.OK and need.value > 0
    work = {"d_workspace": room(20), "workspace_bytes": need.value}
    for changes, want in (
            ({"heads_q": 0}, BAD), ({"heads_q": 3}, BAD), ({"scale": NAN}, BAD), ({"scale": INF}, BAD), ({"n_groups": -1}, BAD),
            ({"n_groups": 1 << 31}, UNSUPPORTED), ({"d_groups": None}, BAD), ({"d_shared": None}, BAD), ({"out.data": None}, BAD),
            ({"d_groups": room(9) + 4}, MISALIGNED), ({"d_shared": room(10) + 2}, MISALIGNED), ({"d_lse": room(11) + 2}, MISALIGNED),
            ({"out.head_stride": 31}, BAD), ({"out.token_stride": 100}, BAD), ({"out.data": room(1)}, OVERLAP),
            ({"out.data": room(7) + 64}, OVERLAP), ({"d_lse": room(8) + 16}, OVERLAP), ({"d_lse": room(3)}, OVERLAP),
            ({"d_workspace": None}, BAD), ({"workspace_bytes": need.value - 1}, BAD), ({"d_workspace": room(20) + 64}, MISALIGNED),
            ({"d_workspace": room(7)}, OVERLAP)):
        assert status(lib, attention_args(**{**work, **changes})) == want, changes
    for changes in ({"cache.dtype": dws.INT32}, {"heads_q": 5}, {"n_groups": -1}, {"cache.dim_k": 0}):
        assert size(ctypes.byref(attention_args(**changes)), ctypes.byref(need)) == BAD, changes
    # more tiles of queries than a launch's numbers hold
    assert size(ctypes.byref(attention_args(**{"seqs.tokens": (1 << 31) - 1, "heads_q": 65534})), ctypes.byref(need)) == UNSUPPORTED
    # without tokens nothing is launched
    none = {"seqs.tokens": 0, "q.data": None, "out.data": None, "d_lse": None}
    assert status(lib, attention_args(**{**work, **none})) == dws.OK


def test_scales_of_attention(lib):
    """scale log2(e) has to be a number, too: a score of 0 would be NaN with an infinite one."""
    need = ctypes.c_size_t(0)
    assert lib.dws_pages_attention_workspace(ctypes.byref(attention_args()), ctypes.byref(need)) == dws.OK
    none = {"seqs.tokens": 0, "q.data": None, "out.data": None, "d_lse": None, "d_workspace": room(20), "workspace_bytes": need.value}
    for scale, want in ((0.0, dws.OK), (2.3e38, dws.OK), (-2.3e38, dws.OK), (1e-45, dws.OK), (2.4e38, BAD), (-3.4e38, BAD), (NAN, BAD), (-INF, BAD)):
        assert status(lib, attention_args(**none, scale=scale)) == want, scale


def test_options_of_attention(lib):
    need = ctypes.c_size_t(0)
    assert lib.dws_pages_attention_workspace(ctypes.byref(attention_args()), ctypes.byref(need)) == dws.OK
    none = {"seqs.tokens": 0, "q.data": None, "out.data": None, "d_lse": None, "d_workspace": room(20), "workspace_bytes": need.value}
    for options, want in ((0, dws.OK), (dws.ATTENTION_ONE_PART, dws.OK), (2, BAD), (3, BAD), (-1, BAD), (1 << 30, BAD)):
        assert status(lib, attention_args(**none, options=options)) == want, options


def test_workspace_of_attention_does_not_grow_with_prompts_alone(lib):
    def bytes_of(**changes):
        need = ctypes.c_size_t(0)
        assert lib.dws_pages_attention_workspace(ctypes.byref(attention_args(**changes)), ctypes.byref(need)) == dws.OK
        return need.value

    few, many = bytes_of(**{"n_groups": 0, "seqs.tokens": 1 << 16}), bytes_of(**{"n_groups": 0, "seqs.tokens": 1 << 20})
    # (what is noted down of a tile, 72 bytes for 128 queries of a key head)
    assert few < many < few + (1 << 20) * 4 * 72 / 128 + 4096
    # with groups, partial results of at most half a tile a sequence
    assert bytes_of(**{"seqs.tokens": 1 << 20}) < many + (1 << 20) * 4 * 72 / 128 + (1 << 19)


def test_refusals_of_beam_select(lib):
    assert lib.dws_beam_select(None, None) == BAD
    need = ctypes.c_size_t(0)
    size = lib.dws_beam_select_workspace
    assert size(None, ctypes.byref(need)) == BAD and size(ctypes.byref(beam_args()), None) == BAD
    assert size(ctypes.byref(beam_args()), ctypes.byref(need)) == dws.OK and need.value >= 12 * (4 * 8 + 16)
    work = {"d_workspace": room(20), "workspace_bytes": need.value}
    for changes, want in (
            ({"dtype": dws.INT32}, BAD), ({"batch": -1}, BAD), ({"beams": 0}, BAD), ({"vocab": 0}, BAD), ({"k": 0}, BAD),
            ({"k": 3}, BAD), ({"vocab": 0}, BAD), ({"beams": 65}, UNSUPPORTED), ({"k": 65, "d_rows": None}, UNSUPPORTED),
            ({"vocab": 1 << 31}, UNSUPPORTED), ({"batch": 1 << 30}, UNSUPPORTED), ({"batch": 1 << 40}, UNSUPPORTED),
            ({"vocab": 1, "k": 5, "d_rows": None}, BAD), ({"batch_stride": -1}, BAD), ({"beam_stride": (1 << 40) + 1}, BAD),
            ({"end_token": -1}, BAD), ({"end_token": 1000}, BAD),
            ({"d_logits": None}, BAD), ({"d_scores": None}, BAD), ({"d_out_scores": None}, BAD), ({"d_parents": None}, BAD),
            ({"d_tokens": None}, BAD), ({"d_out_rows": None}, BAD), ({"d_src": None}, BAD), ({"d_dst": None}, BAD),
            ({"d_logits": room(1) + 1}, MISALIGNED), ({"d_scores": room(2) + 2}, MISALIGNED), ({"d_tokens": room(7) + 2}, MISALIGNED),
            ({"d_out_scores": room(2)}, OVERLAP), ({"d_parents": room(7) + 4}, OVERLAP), ({"d_out_rows": room(4)}, OVERLAP),
            ({"d_dst": room(1) + 100}, OVERLAP), ({"d_workspace": None}, BAD), ({"workspace_bytes": 8}, BAD),
            ({"d_workspace": room(20) + 8}, MISALIGNED), ({"d_workspace": room(1)}, OVERLAP)):
        assert status(lib, beam_args(**{**work, **changes})) == want, changes
    assert status(lib, beam_args(batch=0)) == dws.OK
    # without finished beams the end token is not looked at
    assert status(lib, beam_args(**{**work, "d_finished": None, "end_token": -1, "d_tokens": None})) == BAD


@pytest.mark.parametrize("packed,kind", [("_APPEND", dws.PagesAppendArgs), ("_ATTENTION", dws.PagesAttentionArgs),
                                         ("_BEAM", dws.BeamArgs)])
def test_packed_arguments_are_the_structures(packed, kind):
    packed = getattr(dws, packed)

    def leaves(c, path=()):
        for name, t in c._fields_:
            if issubclass(t, ctypes.Structure):
                yield from leaves(t, path + (name,))
            else:
                yield path + (name,), t

    a, values = kind(), []
    for i, (path, t) in enumerate(leaves(kind)):
        x = float(i) if t is ctypes.c_float else i + 1
        values.append(x)
        put(a, {".".join(path): x})
    assert packed.size == ctypes.sizeof(kind) and packed.pack(*values) == bytes(a)


def test_binding_refuses_cpu_tensors_and_graphs():
    x = torch.zeros(3, 4, 2, 8)
    table, lengths = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 2, 8)
    for call in (lambda: dws.pages_append(x, x, table, lengths, t, t), lambda: dws.pages_attention(t, x, x, table, lengths),
                 lambda: dws.beam_select(t, torch.zeros(2, 2))):
        with pytest.raises(TypeError):
            call()
    wants = torch.zeros(2, 2, 8, requires_grad=True)
    for call in (lambda: dws.pages_append(x, x, table, lengths, wants, t), lambda: dws.pages_attention(wants, x, x, table, lengths),
                 lambda: dws.beam_select(wants, torch.zeros(2, 2))):
        with pytest.raises(RuntimeError, match="records no graph"):
            call()
