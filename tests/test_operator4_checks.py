"""What the 4-bit cache and its attention, beam selection and reordering refuse on the host, before any CUDA call: the C entry
points' own checks (addresses that are never dereferenced) and the binding's (CPU tensors: a call that passes every check stops at
the device check)."""
import ctypes
import os

import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv

FAKE = 1 << 20          # an aligned, never-dereferenced address
MAX_DRAFT, MAX_BATCH = 1023, 4096
BIG = 1 << 30           # bytes of a workspace that is large enough
DEVICE_MSG = "libsv takes device tensors"
I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_verification_74_gb300 import build
    try:
        build.build()
    except RuntimeError as e:  # no nvcc on this machine
        if not os.path.exists(sv.LIB_PATH):
            pytest.skip(str(e))
    return sv.lib()


def call(fn, names, good, **over):
    """fn with the named arguments of `good`, some of them replaced."""
    assert not set(over) - set(names), set(over) - set(names)
    return fn(*[{**good, **over}[n] for n in names])


HEAD = 16 * 9 * 64 // 8  # bytes of a head's page


def cache4(**over):
    good = dict(pool=FAKE, layer_stride=8 * 2 * HEAD, page_stride=2 * HEAD, head_stride=HEAD, layers=2, pages=8, page_size=16,
                kv_heads=2, head_dim=64, page_refs=FAKE, k_scale=1.0, v_scale=0.5)
    return sv.sv_cache4(**{**good, **over})


BAD_CACHES = [dict(pool=None), dict(page_refs=None), dict(pool=FAKE + 8), dict(layers=0), dict(pages=0), dict(pages=(1 << 22) + 1),
              dict(page_size=4), dict(page_size=24), dict(page_size=2048), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=96),
              dict(head_dim=128), dict(head_stride=HEAD - 16), dict(head_stride=HEAD + 8), dict(page_stride=0), dict(layer_stride=-16),
              dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=float("nan")), dict(v_scale=float("inf")), dict(k_scale=1e-39)]

# every call on a cache: its arguments after the cache, and what a valid call passes
CALLS = {
    "sv_cache4_reserve": ("table width lens extra B ok ws ws_bytes stream".split(), {}),
    "sv_cache4_append": ("layer layers table width lens offsets n_rows k_new v_new new_layer_stride new_row_stride B ws "
                         "ws_bytes stream".split(), dict(layers=2)),
    "sv_cache4_commit": ("table width lens offsets path accept B Nmax out_len ws ws_bytes stream".split(), {}),
    "sv_cache4_fork": ("table width rows lens src dst n ok ws ws_bytes stream".split(), {}),
    "sv_cache4_release": ("table width rows lens seqs n ws ws_bytes stream".split(), {}),
    "sv_cache4_reorder": ("table width rows lens src ok ws ws_bytes stream".split(), {}),
    "sv_tree_attention4": ("layer q q_row q_head q_heads table width lens offsets n_rows parent B Nmax scale window sinks out "
                           "out_row out_head lse ws ws_bytes stream".split(), {}),
}
GOOD = dict(table=FAKE, width=4, lens=FAKE, extra=FAKE, B=3, ok=FAKE, ws=FAKE, ws_bytes=BIG, stream=None, layer=0, layers=1,
            offsets=FAKE, n_rows=12, k_new=FAKE, v_new=FAKE, new_layer_stride=12 * 128, new_row_stride=128, path=FAKE,
            accept=FAKE, Nmax=4, out_len=FAKE, rows=3, src=FAKE, dst=FAKE, n=2, seqs=FAKE, q=FAKE, q_row=256, q_head=64,
            q_heads=4, parent=FAKE, scale=0.125, window=0, sinks=0, out=FAKE, out_row=256, out_head=64, lse=FAKE)


def on_cache(L, name, c=None, **over):
    names, mine = CALLS[name]
    c = cache4() if c is None else c
    return call(lambda *a: getattr(L, name)(ctypes.addressof(c), *a), names, {**GOOD, **mine}, **over)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("over", BAD_CACHES)
def test_bad_caches_are_refused(L, name, over):
    assert on_cache(L, name, cache4(**over)) == sv.SV_ERR_INVALID_ARG


@pytest.mark.parametrize("name", CALLS)
def test_cache_workspaces(L, name):
    for over in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=255)):
        assert on_cache(L, name, **over) == sv.SV_ERR_WORKSPACE
    assert getattr(L, name)(None, *[{**GOOD, **CALLS[name][1]}[n] for n in CALLS[name][0]]) == sv.SV_ERR_INVALID_ARG


@pytest.mark.parametrize("name,over", [
    *[(n, o) for n in CALLS for o in (dict(table=None), dict(lens=None), dict(width=0), dict(width=(1 << 20) + 1))],
    *[(n, o) for n in ("sv_cache4_reserve", "sv_cache4_append", "sv_cache4_commit", "sv_tree_attention4")
      for o in (dict(B=-1), dict(B=MAX_BATCH + 1))],
    ("sv_cache4_reserve", dict(extra=None)), ("sv_cache4_reserve", dict(B=4096, width=1 << 20)),
    *[("sv_cache4_append", o) for o in (
        dict(layer=-1), dict(layer=1), dict(layers=-1), dict(n_rows=-1), dict(offsets=None), dict(k_new=None), dict(v_new=None),
        dict(k_new=FAKE + 8), dict(new_row_stride=132), dict(new_row_stride=120), dict(new_layer_stride=4))],
    *[("sv_cache4_commit", o) for o in (
        dict(Nmax=0), dict(Nmax=MAX_DRAFT + 2), dict(offsets=None), dict(path=None), dict(accept=None), dict(out_len=None))],
    *[("sv_cache4_fork", o) for o in (
        dict(n=-1), dict(n=MAX_BATCH + 1), dict(src=None), dict(dst=None), dict(rows=0), dict(rows=-1))],
    *[("sv_cache4_release", o) for o in (dict(n=-1), dict(n=MAX_BATCH + 1), dict(seqs=None), dict(rows=0))],
    *[("sv_cache4_reorder", o) for o in (dict(src=None), dict(rows=-1), dict(rows=MAX_BATCH + 1))],
    *[("sv_tree_attention4", o) for o in (
        dict(layer=2), dict(layer=-1), dict(q_heads=0), dict(q_heads=3), dict(q_heads=258), dict(Nmax=0),
        dict(Nmax=MAX_DRAFT + 2), dict(n_rows=-1), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")),
        dict(window=-1), dict(sinks=-1), dict(q=None), dict(out=None), dict(offsets=None), dict(q=FAKE + 8), dict(out=FAKE + 2),
        dict(q_row=252), dict(q_head=56), dict(out_row=-256), dict(out_head=32))],
])
def test_bad_arguments_are_refused(L, name, over):
    assert on_cache(L, name, **over) == sv.SV_ERR_INVALID_ARG
    assert L.sv_last_error_string()


def test_reorder_of_a_bf16_cache(L):
    c = sv.sv_cache(k=FAKE, v=FAKE, layer_stride=8 * 16 * 2 * 64, page_stride=16 * 2 * 64, slot_stride=2 * 64, head_stride=64, layers=2,
                    pages=8, page_size=16, kv_heads=2, head_dim=64, page_refs=FAKE)
    names = "table width rows lens src ok ws ws_bytes stream".split()
    go = lambda **over: call(lambda *a: L.sv_cache_reorder(ctypes.addressof(c), *a), names, GOOD, **over)  # noqa: E731
    for over in (dict(src=None), dict(rows=-1), dict(rows=MAX_BATCH + 1), dict(table=None), dict(lens=None), dict(width=0)):
        assert go(**over) == sv.SV_ERR_INVALID_ARG
    for over in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=255)):
        assert go(**over) == sv.SV_ERR_WORKSPACE
    assert go(rows=0, src=None, table=None, lens=None) == sv.SV_OK
    c.head_dim = 32
    assert go() == sv.SV_ERR_INVALID_ARG


def test_scales_whose_product_leaves_float32(L):
    assert on_cache(L, "sv_tree_attention4", cache4(k_scale=1e-30), scale=1e-30) == sv.SV_ERR_INVALID_ARG
    assert on_cache(L, "sv_tree_attention4", cache4(k_scale=1e30), scale=1e30) == sv.SV_ERR_INVALID_ARG
    assert b"k_scale" in L.sv_last_error_string()


def test_attention_of_too_many_tiles_is_refused(L):
    wide = dict(page_size=1024, head_stride=64 * HEAD, page_stride=2 * 64 * HEAD, layer_stride=16 * 64 * HEAD)
    assert on_cache(L, "sv_tree_attention4", cache4(**wide), B=4096, width=1 << 20) == sv.SV_ERR_INVALID_ARG
    assert b"too many" in L.sv_last_error_string()


def test_empty_calls_are_no_ops(L):
    assert on_cache(L, "sv_cache4_reserve", B=0, lens=None, extra=None, table=None) == sv.SV_OK
    assert on_cache(L, "sv_cache4_append", n_rows=0, k_new=None, v_new=None) == sv.SV_OK
    assert on_cache(L, "sv_cache4_append", layers=0, k_new=None, v_new=None) == sv.SV_OK
    assert on_cache(L, "sv_cache4_commit", B=0, lens=None, table=None) == sv.SV_OK
    assert on_cache(L, "sv_cache4_fork", n=0, src=None, dst=None) == sv.SV_OK
    assert on_cache(L, "sv_cache4_release", n=0, seqs=None) == sv.SV_OK
    assert on_cache(L, "sv_cache4_reorder", rows=0, src=None, table=None, lens=None) == sv.SV_OK
    assert on_cache(L, "sv_tree_attention4", B=0, lens=None, table=None, q=None) == sv.SV_OK
    assert on_cache(L, "sv_tree_attention4", n_rows=0, q=None, out=None) == sv.SV_OK


def test_attention_workspace_sizes(L):
    def size(heads, **over):
        c = cache4(**over)
        return L.sv_attention4_workspace_size(ctypes.addressof(c), heads)

    big = 2 * HEAD
    assert 0 < size(4) < size(4, head_dim=128, head_stride=big, page_stride=2 * big, layer_stride=16 * big)
    assert size(0) == size(3) == size(258) == size(4, page_size=7) == 0
    assert size(256) == size(2)


# ---- beam selection ---------------------------------------------------------------------------------

BEAM = "logits row_stride dt B W V scores finished pad K out_scores out_rows out_tokens ws ws_bytes stream".split()
BEAM_GOOD = dict(logits=FAKE, row_stride=104, dt=sv.SV_BF16, B=2, W=4, V=100, scores=FAKE, finished=None, pad=0, K=8, out_scores=FAKE,
                 out_rows=FAKE, out_tokens=FAKE, ws=FAKE, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("over", [
    dict(dt=2), dict(B=-1), dict(W=0), dict(W=65), dict(B=(1 << 16) // 4 + 1), dict(B=1 << 30), dict(V=0), dict(V=(1 << 18) + 1), dict(K=0),
    dict(K=129), dict(pad=-1), dict(logits=None), dict(scores=None), dict(out_scores=None), dict(out_rows=None), dict(out_tokens=None),
    dict(logits=FAKE + 1), dict(logits=FAKE + 2, dt=sv.SV_F32), dict(row_stride=99)])
def test_beam_refuses(L, over):
    assert call(L.sv_beam_select, BEAM, BEAM_GOOD, **over) == sv.SV_ERR_INVALID_ARG
    assert L.sv_last_error_string()


def test_beam_sizes_and_no_ops(L):
    for over in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=255)):
        assert call(L.sv_beam_select, BEAM, BEAM_GOOD, **over) == sv.SV_ERR_WORKSPACE
    need = L.sv_beam_workspace_size(8, 100, 8)
    assert call(L.sv_beam_select, BEAM, BEAM_GOOD, ws_bytes=need - 1) == sv.SV_ERR_WORKSPACE
    assert L.sv_beam_workspace_size(-1, 100, 8) == L.sv_beam_workspace_size(8, 0, 8) == L.sv_beam_workspace_size(8, 100, 0) == 0
    assert L.sv_beam_workspace_size((1 << 16) + 1, 100, 8) == L.sv_beam_workspace_size(8, 100, 129) == 0
    assert 0 < need < L.sv_beam_workspace_size(64, 100, 8) < L.sv_beam_workspace_size(64, 100, 64)
    nothing = {n: None for n in BEAM if n not in ("row_stride", "dt", "B", "W", "V", "pad", "K", "ws_bytes")}
    assert call(L.sv_beam_select, BEAM, BEAM_GOOD, B=0, **{n: None for n in nothing}) == sv.SV_OK


# ---- the binding --------------------------------------------------------------------------------------

def _raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def beam(**over):
    a = dict(logits=torch.zeros(8, 64, dtype=BF16), scores=torch.zeros(2, 4), candidates=4, finished=torch.zeros(2, 4, dtype=I32),
             ws=torch.zeros(1 << 16, dtype=torch.uint8))
    a.update(over)
    x, s, k = (a.pop(n) for n in ("logits", "scores", "candidates"))
    return sv.beam_select(x, s, k, **a)


def test_beam_checks(L):
    _raises(lambda: beam(), DEVICE_MSG)                                            # every check passes
    _raises(lambda: beam(logits=torch.zeros(2, 4, 64, dtype=BF16)), "takes logits")
    _raises(lambda: beam(logits=torch.zeros(7, 64, dtype=BF16)), "takes logits")
    _raises(lambda: beam(scores=torch.zeros(8)), "takes logits")
    _raises(lambda: beam(logits=torch.zeros(8, 64, dtype=torch.float16)), "bfloat16")
    _raises(lambda: beam(finished=torch.zeros(8, dtype=I32)), "shape of scores")
    _raises(lambda: beam(logits=torch.zeros(64, 8).T), "logit rows must be contiguous")
    with pytest.raises(ValueError):
        sv.beam_workspace(8, 0, 4)


def low_beam(**over):
    a = dict(logits=torch.zeros(8, 64), row_stride=64, dt=sv.SV_F32, B=2, W=4, V=64, scores=torch.zeros(2, 4),
             finished=torch.zeros(2, 4, dtype=I32), pad=0, K=4, out_scores=torch.zeros(2, 4), out_rows=torch.zeros(2, 4, dtype=I32),
             out_tokens=torch.zeros(2, 4, dtype=I32), ws=torch.zeros(1 << 16, dtype=torch.uint8))
    a.update(over)
    sv.sv_beam_select(*a.values())


def test_low_level_beam_checks(L):
    _raises(lambda: low_beam(), DEVICE_MSG)
    _raises(lambda: low_beam(logits=torch.zeros(7, 64)), "logits holds")
    _raises(lambda: low_beam(dt=sv.SV_BF16), "logits must be torch.bfloat16")
    for name, short, wrong in (("scores", torch.zeros(7), torch.zeros(8, dtype=torch.float64)),
                               ("finished", torch.zeros(7, dtype=I32), torch.zeros(8, dtype=torch.bool)),
                               ("out_scores", torch.zeros(7), torch.zeros(8, dtype=BF16)),
                               ("out_rows", torch.zeros(7, dtype=I32), torch.zeros(8, dtype=torch.int64)),
                               ("out_tokens", torch.zeros(7, dtype=I32), torch.zeros(8, dtype=torch.int64))):
        _raises(lambda: low_beam(**{name: short}), f"{name} holds")
        _raises(lambda: low_beam(**{name: wrong}), f"{name} must be")


def test_cache4_checks(L):
    def make(**over):
        a = dict(pool=torch.zeros(2, 8, 2, HEAD, dtype=torch.uint8), page_refs=torch.zeros(8, dtype=I32),
                 page_table=torch.full((3, 4), -1, dtype=I32), page_size=16, head_dim=64)
        a.update(over)
        return sv.PagedCache4(**a)

    _raises(lambda: make(), DEVICE_MSG)
    pool = torch.zeros(2, 8, 2, HEAD, dtype=torch.uint8)
    _raises(lambda: make(pool=pool[0]), "must be \\[layers")
    _raises(lambda: make(pool=pool[..., 16:]), "must be \\[layers")
    _raises(lambda: make(pool=pool.to(torch.int8)), "pool must be torch.uint8")
    _raises(lambda: make(pool=torch.zeros(2, 8, HEAD, 2, dtype=torch.uint8).transpose(2, 3)), "must be contiguous")
    _raises(lambda: make(page_table=torch.zeros(4, dtype=I32)), "page_table must be")


class HostCache4(sv.PagedCache4):
    """A cache whose struct holds addresses that nothing dereferences."""

    def __init__(self):
        self.c, self.kv_heads, self.head_dim, self.rows, self.width = cache4(), 2, 64, 3, 4
        self._c, self._table, self._ws, self._ws_bytes = ctypes.addressof(self.c), FAKE, FAKE, BIG


def test_call_checks(L):
    c = HostCache4()
    i = lambda n: torch.zeros(n, dtype=I32)  # noqa: E731
    kv = torch.zeros(2, 12, 2, 64, dtype=BF16)
    _raises(lambda: c.reserve(i(3), i(3)), DEVICE_MSG)
    _raises(lambda: c.append(kv, kv, i(3), i(4)), DEVICE_MSG)
    _raises(lambda: c.append(kv.float(), kv.float(), i(3), i(4)), "must be torch.bfloat16")
    _raises(lambda: c.commit(i(4), i(5), i(16).view(4, 4), i(4)), "page table has 3 rows")
    _raises(lambda: c.reorder(i(3), i(3)), DEVICE_MSG)
    _raises(lambda: c.reorder(i(3), i(2)), "src must name a row")
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    go = lambda q: sv.tree_attention(q, c, 0, i(3), i(4), i(12), 4, ws=ws)  # noqa: E731
    _raises(lambda: go(torch.zeros(12, 4, 64, dtype=BF16)), DEVICE_MSG)
    _raises(lambda: go(torch.zeros(12, 4, 64)), "must be torch.bfloat16")
    with pytest.raises(ValueError):
        sv.attention_workspace(c, 3)
