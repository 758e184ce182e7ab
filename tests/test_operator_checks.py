"""What sampling, the paged cache and tree attention refuse on the host, before any CUDA call: the C entry points' own
checks (addresses that are never dereferenced) and the binding's checks of types and extents (CPU tensors: a call that
passes every check stops at the device check)."""
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


# ---- C entry points ---------------------------------------------------------------------------------

def call(fn, names, good, **over):
    """fn with the named arguments of `good`, some of them replaced."""
    assert not set(over) - set(names), set(over) - set(names)
    return fn(*[{**good, **over}[n] for n in names])


SAMPLE = ("logits row_stride dt R V temperature top_k top_p min_p uniforms M out_tokens out_probs out_rows out_stride ws "
          "ws_bytes stream").split()
SAMPLE_GOOD = dict(logits=FAKE, row_stride=104, dt=sv.SV_BF16, R=4, V=100, temperature=FAKE, top_k=FAKE, top_p=FAKE,
                   min_p=FAKE, uniforms=FAKE, M=2, out_tokens=FAKE, out_probs=FAKE, out_rows=None, out_stride=0, ws=FAKE,
                   ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("over", [
    dict(dt=2), dict(R=-1), dict(R=(1 << 20) + 1), dict(V=0), dict(V=(1 << 18) + 1), dict(M=-1), dict(M=1025),
    dict(logits=None), dict(temperature=None), dict(uniforms=None), dict(out_tokens=None), dict(logits=FAKE + 1),
    dict(logits=FAKE + 2, dt=sv.SV_F32), dict(row_stride=99), dict(out_rows=FAKE + (1 << 22), out_stride=99),
    dict(out_rows=FAKE + (1 << 22) + 1, out_stride=104), dict(out_rows=FAKE, out_stride=112)])
def test_sample_refuses(L, over):
    assert call(L.sv_sample_rows, SAMPLE, SAMPLE_GOOD, **over) == sv.SV_ERR_INVALID_ARG
    assert L.sv_last_error_string()


@pytest.mark.parametrize("over", [dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=255)])
def test_sample_workspace(L, over):
    assert call(L.sv_sample_rows, SAMPLE, SAMPLE_GOOD, **over) == sv.SV_ERR_WORKSPACE


def test_sample_sizes_and_no_ops(L):
    assert L.sv_sample_workspace_size(-1, 100) == L.sv_sample_workspace_size(4, 0) == 0
    assert L.sv_sample_workspace_size(4, (1 << 18) + 1) == L.sv_sample_workspace_size((1 << 20) + 1, 100) == 0
    assert 0 < L.sv_sample_workspace_size(4, 100) < L.sv_sample_workspace_size(64, 100) < L.sv_sample_workspace_size(64, 9999)
    need = L.sv_sample_workspace_size(4, 100)
    assert call(L.sv_sample_rows, SAMPLE, SAMPLE_GOOD, ws_bytes=need - 1) == sv.SV_ERR_WORKSPACE
    nothing = {n: None for n in SAMPLE if n not in ("row_stride", "dt", "R", "V", "M", "out_stride", "ws_bytes")}
    assert call(L.sv_sample_rows, SAMPLE, SAMPLE_GOOD, R=0, **nothing) == sv.SV_OK
    assert call(L.sv_sample_rows, SAMPLE, SAMPLE_GOOD, M=0, **nothing) == sv.SV_OK      # no draw and no cut rows


def cache(**over):
    good = dict(k=FAKE, v=FAKE, layer_stride=8 * 16 * 2 * 64, page_stride=16 * 2 * 64, slot_stride=2 * 64, head_stride=64,
                layers=2, pages=8, page_size=16, kv_heads=2, head_dim=64, page_refs=FAKE)
    return sv.sv_cache(**{**good, **over})


BAD_CACHES = [dict(k=None), dict(v=None), dict(page_refs=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(layers=0), dict(pages=0),
              dict(pages=(1 << 22) + 1), dict(page_size=4), dict(page_size=24), dict(page_size=2048), dict(kv_heads=0),
              dict(kv_heads=1025), dict(head_dim=96), dict(slot_stride=132), dict(head_stride=-64), dict(page_stride=0)]

# every call on a cache: its arguments after the cache, and what a valid call passes
CALLS = {
    "sv_cache_reserve": ("table width lens extra B ok ws ws_bytes stream".split(), {}),
    "sv_cache_append": ("layer layers table width lens offsets n_rows k_new v_new new_layer_stride new_row_stride B ws "
                        "ws_bytes stream".split(), dict(layers=2)),
    "sv_cache_commit": ("table width lens offsets path accept B Nmax out_len ws ws_bytes stream".split(), {}),
    "sv_cache_fork": ("table width rows lens src dst n ok ws ws_bytes stream".split(), {}),
    "sv_cache_release": ("table width rows lens seqs n ws ws_bytes stream".split(), {}),
    "sv_tree_attention": ("layer q q_row q_head q_heads table width lens offsets n_rows parent B Nmax scale window sinks out "
                          "out_row out_head lse ws ws_bytes stream".split(), {}),
}
GOOD = dict(table=FAKE, width=4, lens=FAKE, extra=FAKE, B=3, ok=FAKE, ws=FAKE, ws_bytes=BIG, stream=None, layer=0, layers=1,
            offsets=FAKE, n_rows=12, k_new=FAKE, v_new=FAKE, new_layer_stride=12 * 128, new_row_stride=128, path=FAKE,
            accept=FAKE, Nmax=4, out_len=FAKE, rows=3, src=FAKE, dst=FAKE, n=2, seqs=FAKE, q=FAKE, q_row=256, q_head=64,
            q_heads=4, parent=FAKE, scale=0.125, window=0, sinks=0, out=FAKE, out_row=256, out_head=64, lse=FAKE)


def on_cache(L, name, c=None, **over):
    names, mine = CALLS[name]
    c = cache() if c is None else c
    return call(lambda *a: getattr(L, name)(ctypes.addressof(c), *a), names, {**GOOD, **mine}, **over)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("over", BAD_CACHES)
def test_bad_caches_are_refused(L, name, over):
    assert on_cache(L, name, cache(**over)) == sv.SV_ERR_INVALID_ARG


@pytest.mark.parametrize("name", CALLS)
def test_cache_workspaces(L, name):
    for over in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=255)):
        assert on_cache(L, name, **over) == sv.SV_ERR_WORKSPACE
    assert getattr(L, name)(None, *[{**GOOD, **CALLS[name][1]}[n] for n in CALLS[name][0]]) == sv.SV_ERR_INVALID_ARG


@pytest.mark.parametrize("name,over", [
    *[(n, o) for n in CALLS for o in (dict(table=None), dict(lens=None), dict(width=0), dict(width=(1 << 20) + 1))],
    *[(n, o) for n in ("sv_cache_reserve", "sv_cache_append", "sv_cache_commit", "sv_tree_attention")
      for o in (dict(B=-1), dict(B=MAX_BATCH + 1))],
    ("sv_cache_reserve", dict(extra=None)), ("sv_cache_reserve", dict(B=4096, width=1 << 20)),
    *[("sv_cache_append", o) for o in (
        dict(layer=-1), dict(layer=1), dict(layers=-1), dict(n_rows=-1), dict(offsets=None), dict(k_new=None), dict(v_new=None),
        dict(k_new=FAKE + 8), dict(new_row_stride=132), dict(new_row_stride=120), dict(new_layer_stride=4))],
    *[("sv_cache_commit", o) for o in (
        dict(Nmax=0), dict(Nmax=MAX_DRAFT + 2), dict(offsets=None), dict(path=None), dict(accept=None), dict(out_len=None))],
    *[("sv_cache_fork", o) for o in (
        dict(n=-1), dict(n=MAX_BATCH + 1), dict(src=None), dict(dst=None), dict(rows=0), dict(rows=-1))],
    *[("sv_cache_release", o) for o in (dict(n=-1), dict(n=MAX_BATCH + 1), dict(seqs=None), dict(rows=0))],
    *[("sv_tree_attention", o) for o in (
        dict(layer=2), dict(layer=-1), dict(q_heads=0), dict(q_heads=3), dict(q_heads=258), dict(Nmax=0),
        dict(Nmax=MAX_DRAFT + 2), dict(n_rows=-1), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")),
        dict(window=-1), dict(sinks=-1), dict(q=None), dict(out=None), dict(offsets=None), dict(q=FAKE + 8), dict(out=FAKE + 2),
        dict(q_row=252), dict(q_head=56), dict(out_row=-256), dict(out_head=32))],
])
def test_bad_arguments_are_refused(L, name, over):
    assert on_cache(L, name, **over) == sv.SV_ERR_INVALID_ARG
    assert L.sv_last_error_string()


def test_attention_of_too_many_tiles_is_refused(L):
    # 4096 requests of up to 2^30 slots, 2 heads: their tiles cannot be counted in 32 bits
    assert on_cache(L, "sv_tree_attention", cache(page_size=1024), B=4096, width=1 << 20) == sv.SV_ERR_INVALID_ARG
    assert b"too many" in L.sv_last_error_string()


def test_empty_calls_are_no_ops(L):
    assert on_cache(L, "sv_cache_reserve", B=0, lens=None, extra=None, table=None) == sv.SV_OK
    assert on_cache(L, "sv_cache_append", n_rows=0, k_new=None, v_new=None) == sv.SV_OK
    assert on_cache(L, "sv_cache_append", layers=0, k_new=None, v_new=None) == sv.SV_OK
    assert on_cache(L, "sv_cache_commit", B=0, lens=None, table=None) == sv.SV_OK
    assert on_cache(L, "sv_cache_fork", n=0, src=None, dst=None) == sv.SV_OK
    assert on_cache(L, "sv_cache_release", n=0, seqs=None) == sv.SV_OK
    assert on_cache(L, "sv_tree_attention", B=0, lens=None, table=None, q=None) == sv.SV_OK
    assert on_cache(L, "sv_tree_attention", n_rows=0, q=None, out=None) == sv.SV_OK


def test_attention_workspace_sizes(L):
    def size(heads, **over):
        c = cache(**over)
        return L.sv_attention_workspace_size(ctypes.addressof(c), heads)

    assert 0 < size(4) < size(4, head_dim=128, head_stride=128, slot_stride=256, page_stride=4096, layer_stride=1 << 15)
    assert size(0) == size(3) == size(258) == size(4, page_size=7) == 0
    assert size(256) == size(2)


# ---- the binding --------------------------------------------------------------------------------------

def _raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def sample(R=3, V=64, M=2, **over):
    a = dict(logits=torch.zeros(R, V, dtype=BF16), temperature=torch.ones(R), uniforms=torch.zeros(R, M),
             top_k=torch.zeros(R, dtype=I32), top_p=torch.ones(R), min_p=torch.zeros(R),
             ws=torch.zeros(1 << 16, dtype=torch.uint8))
    a.update(over)
    x, t, u = (a.pop(n) for n in ("logits", "temperature", "uniforms"))
    return sv.sample(x, t, u, **a)


def test_sample_checks(L):
    _raises(lambda: sample(), DEVICE_MSG)                                          # every check passes
    _raises(lambda: sample(logits=torch.zeros(3, 4, 64, dtype=BF16)), "takes logits")
    _raises(lambda: sample(uniforms=torch.zeros(2, 2)), "takes logits")
    _raises(lambda: sample(uniforms=torch.zeros(3)), "takes logits")
    _raises(lambda: sample(logits=torch.zeros(3, 64, dtype=torch.float16)), "bfloat16")
    _raises(lambda: sample(filtered=torch.zeros(3, 64)), "filtered must have")
    _raises(lambda: sample(filtered=torch.zeros(3, 63, dtype=BF16)), "filtered must have")


def low_sample(R=3, V=64, M=2, **over):
    a = dict(logits=torch.zeros(R, V), row_stride=V, dt=sv.SV_F32, R=R, V=V, temperature=torch.ones(R),
             top_k=torch.zeros(R, dtype=I32), top_p=torch.ones(R), min_p=torch.zeros(R), uniforms=torch.zeros(R, M), M=M,
             out_tokens=torch.zeros(R, M, dtype=I32), out_probs=torch.zeros(R, M), out_rows=torch.zeros(R, V), out_stride=V,
             ws=torch.zeros(1 << 16, dtype=torch.uint8))
    a.update(over)
    sv.sv_sample_rows(*a.values())


def test_low_level_sample_checks(L):
    _raises(lambda: low_sample(), DEVICE_MSG)
    _raises(lambda: low_sample(logits=torch.zeros(2, 64)), "logits holds")
    _raises(lambda: low_sample(dt=sv.SV_BF16), "logits must be torch.bfloat16")
    for name, short, wrong in (("temperature", torch.ones(2), torch.ones(3, dtype=torch.float64)),
                               ("top_k", torch.zeros(2, dtype=I32), torch.zeros(3, dtype=torch.int64)),
                               ("top_p", torch.ones(2), torch.ones(3, dtype=BF16)),
                               ("min_p", torch.ones(2), torch.ones(3, dtype=I32)),
                               ("uniforms", torch.zeros(5), torch.zeros(6, dtype=torch.float64)),
                               ("out_tokens", torch.zeros(5, dtype=I32), torch.zeros(6, dtype=torch.int64)),
                               ("out_probs", torch.zeros(5), torch.zeros(6, dtype=BF16))):
        _raises(lambda: low_sample(**{name: short}), f"{name} holds")
        _raises(lambda: low_sample(**{name: wrong}), f"{name} must be")
    _raises(lambda: low_sample(out_rows=torch.zeros(3, 63)), "out_rows holds")


def pool(**over):
    a = dict(k=torch.zeros(2, 8, 16, 2, 64, dtype=BF16), v=torch.zeros(2, 8, 16, 2, 64, dtype=BF16),
             page_refs=torch.zeros(8, dtype=I32), page_table=torch.full((3, 4), -1, dtype=I32))
    a.update(over)
    return sv.PagedCache(**a)


def test_cache_checks(L):
    _raises(lambda: pool(), DEVICE_MSG)
    k = torch.zeros(2, 8, 16, 2, 64, dtype=BF16)
    _raises(lambda: pool(k=k[0]), "must be \\[layers")
    _raises(lambda: pool(v=k[:, :7]), "alike")
    _raises(lambda: pool(k=k.float(), v=k.float()), "k must be torch.bfloat16")
    _raises(lambda: pool(k=k.transpose(3, 4), v=k.transpose(3, 4)), "head dimension must be contiguous")
    _raises(lambda: pool(page_table=torch.zeros(4, dtype=I32)), "page_table must be")


class HostCache(sv.PagedCache):
    """A cache whose struct holds addresses that nothing dereferences."""

    def __init__(self):
        self.c, self.kv_heads, self.head_dim, self.rows, self.width = cache(), 2, 64, 3, 4
        self.k = torch.zeros(1, dtype=BF16)
        self._c, self._table, self._ws, self._ws_bytes = ctypes.addressof(self.c), FAKE, FAKE, BIG


def test_cache_call_checks(L):
    c = HostCache()
    i = lambda n: torch.zeros(n, dtype=I32)  # noqa: E731
    kv = torch.zeros(2, 12, 2, 64, dtype=BF16)
    _raises(lambda: c.reserve(i(3), i(3)), DEVICE_MSG)
    _raises(lambda: c.reserve(i(4), i(4)), "page table has 3 rows")
    _raises(lambda: c.append(kv, kv, i(3), i(4)), DEVICE_MSG)
    _raises(lambda: c.append(kv, kv[:1], i(3), i(4)), "k_new and v_new must be")
    _raises(lambda: c.append(kv[..., :32], kv[..., :32], i(3), i(4)), "k_new and v_new must be")
    _raises(lambda: c.append(kv.float(), kv.float(), i(3), i(4)), "must be torch.bfloat16")
    wide = torch.zeros(2, 12, 2, 128, dtype=BF16)[..., :64]
    _raises(lambda: c.append(wide, wide, i(3), i(4)), "contiguous")
    _raises(lambda: c.append(kv, kv, i(4), i(5)), "page table has 3 rows")
    _raises(lambda: c.commit(i(3), i(4), i(12), i(3)), "path must be")
    _raises(lambda: c.commit(i(4), i(5), i(16).view(4, 4), i(4)), "page table has 3 rows")


def test_attention_checks(L):
    c = HostCache()
    i = lambda n: torch.zeros(n, dtype=I32)  # noqa: E731
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    q = torch.zeros(12, 4, 64, dtype=BF16)
    go = lambda q=q, lens=i(3), offsets=i(4), parent=i(12), **kw: sv.tree_attention(q, c, 0, lens, offsets, parent, 4, ws=ws, **kw)  # noqa: E731
    _raises(lambda: go(), DEVICE_MSG)
    _raises(lambda: go(q=q[0]), "q must be")
    _raises(lambda: go(q=q[..., :32]), "q must be")
    _raises(lambda: go(q=q.float()), "must be torch.bfloat16")
    _raises(lambda: go(out=torch.zeros(12, 4, 64)), "must be torch.bfloat16")
    _raises(lambda: go(out=torch.zeros(11, 4, 64, dtype=BF16)), "shape of q")
    _raises(lambda: go(q=torch.zeros(12, 64, 4, dtype=BF16).transpose(1, 2)), "must be contiguous")
    _raises(lambda: go(lens=i(4), offsets=i(5)), "page table has 3 rows")
    with pytest.raises(ValueError):
        sv.attention_workspace(c, 3)
    with pytest.raises(ValueError):
        sv.sample_workspace(4, 0)
