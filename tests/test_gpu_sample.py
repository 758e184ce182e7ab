"""sv_sample_rows on the GPU: against the float64 oracle outside its near-boundary bands, and bit for
bit against the documented arithmetic (float32 exponents, integer weights) spelled out in torch."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_74_gb300 as sv
from oracle.sample import sample_row

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def rows(kind, R, V, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "ties":       # few distinct values: long runs of equal logits
        x = torch.randint(-3, 4, (R, V), generator=g, device="cuda").float()
    elif kind == "zeros":    # +0 and -0 are one value
        x = torch.where(torch.rand((R, V), generator=g, device="cuda") < 0.5, 0.0, -0.0)
    elif kind == "masked":   # most tokens masked, the last row but one of the lowest value, one row all masked
        x = torch.randn((R, V), generator=g, device="cuda") * 2
        x[torch.rand((R, V), generator=g, device="cuda") < 0.9] = -math.inf
        x[0] = -math.inf
        if R > 1:
            x[1] = torch.finfo(torch.bfloat16).min
    elif kind == "wide":     # weights far below 2^-40 beside ordinary ones
        x = torch.randn((R, V), generator=g, device="cuda") * 40
    else:
        x = torch.randn((R, V), generator=g, device="cuda") * 3
    return x.to(dtype)


def share(total, part24):
    return (total >> 24) * part24 + (((total & 0xFFFFFF) * part24) >> 24)


def defined(x, T, u, k=None, p=None, q=None):
    """The documented arithmetic: float32 exponents and 2^y, integer weights, exact sums."""
    xf = x.float()
    R, V = xf.shape
    greedy = T == 0
    steep = torch.div(torch.full_like(T, 1.4426950408889634), torch.where(greedy, torch.ones_like(T), T))
    top = xf.amax(1, keepdim=True)
    y = torch.where(top == -math.inf, torch.full_like(xf, -math.inf), (xf - top) * steep[:, None])
    w = torch.round(torch.exp2(y) * 2.0 ** 40).long()
    order = torch.sort(xf, dim=1, descending=True, stable=True).indices
    kk = torch.full((R,), V, device="cuda") if k is None else torch.where(k <= 0, V, k.long())
    keep = torch.arange(V, device="cuda") < torch.where(greedy, 1, kk)[:, None]
    ws = w.gather(1, order) * keep
    if p is not None:
        pp = torch.where(greedy, torch.ones_like(T), p)
        limit = share(ws.sum(1), torch.round(pp * 2.0 ** 24).long()).clamp(min=1)
        keep &= (pp >= 1)[:, None] | ((ws.cumsum(1) - ws) < limit[:, None])
    if q is not None:
        keep &= y.gather(1, order) >= torch.where(greedy, torch.zeros_like(T), torch.log2(q))[:, None]
    kept = torch.zeros_like(keep).scatter(1, order, keep) & (xf > -math.inf)
    c = (w * kept).cumsum(1)
    Z = c[:, -1:]
    tok = torch.searchsorted(c, share(Z, (u * 2.0 ** 24).long()), right=True)
    prob = w.gather(1, tok.clamp(max=V - 1)).float() / Z.clamp(min=1).float()
    none = Z == 0
    return (torch.where(none, -1, tok).int(), torch.where(none, torch.zeros_like(prob), prob),
            xf.masked_fill(~kept, -math.inf).to(x.dtype))


def params(R, seed, which):
    g = torch.Generator(device="cuda").manual_seed(seed + 7)
    pick = lambda v: torch.tensor(v, device="cuda")[torch.randint(len(v), (R,), generator=g, device="cuda")]  # noqa: E731
    T = pick([1.0, 0.3, 0.7, 0.0, 2.5])
    k = pick([0, 1, 2, 50, 1000, 10 ** 9]).to(torch.int32) if "k" in which else None
    p = pick([1.0, 0.9, 0.5, 0.999, 1e-6]) if "p" in which else None
    q = pick([0.0, 0.05, 1.0, 0.3]) if "q" in which else None
    return T, k, p, q


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 255, 1000, 4097, 32000, 65543, 151936, 262144])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
def test_bit_exact_over_sizes(V, kind, dtype):
    R = 9
    x = rows(kind, R, V, dtype, V)
    T, k, p, q = params(R, V, "kpq")
    u = torch.randint(1 << 24, (R, 3), device="cuda", generator=torch.Generator(device="cuda").manual_seed(V)) / 2.0 ** 24
    ws = sv.sample_workspace(R, V)
    tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
    a, b, c = defined(x, T, u, k, p, q)
    assert torch.equal(cut.view(torch.int16 if dtype == torch.bfloat16 else torch.int32),
                       c.view(torch.int16 if dtype == torch.bfloat16 else torch.int32))
    assert torch.equal(tok, a) and torch.equal(prob, b)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


@pytest.mark.parametrize("which", ["", "k", "p", "q", "kp", "kq", "pq"])
@pytest.mark.parametrize("kind", ["normal", "ties", "zeros", "wide", "masked"])
def test_bit_exact_over_filters(which, kind):
    R, V = 24, 50021
    for dtype in (torch.bfloat16, torch.float32):
        x = rows(kind, R, V, dtype, len(which) + len(kind))
        T, k, p, q = params(R, 3, which)
        u = torch.rand((R, 5), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).clamp(max=1 - 2 ** -24)
        u[0, :2] = torch.tensor([0.0, 1 - 2.0 ** -24])
        tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True)
        a, b, c = defined(x, T, u, k, p, q)
        assert torch.equal(cut, c) and torch.equal(tok, a) and torch.equal(prob, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_against_the_oracle(dtype):
    """Tokens, probabilities and kept sets of the float64 oracle.  A weight differs from the real one by at
    most |y| 2^-23 ln 2 (two roundings of its exponent) + 2^-22 (ex2.approx) + 2^-41 / w: below 2e-6 wherever a weight of
    2^-12 or more decides; what hangs on less is left out, and is rare."""
    R, V = 32, 20011
    x = rows("normal", R, V, dtype, 5)
    T, k, p, q = params(R, 5, "kpq")
    u = torch.randint(1 << 24, (R, 4), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) / 2.0 ** 24
    tok, prob, cut = (t.cpu() for t in sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True))
    left_out = 0
    for r in range(R):
        o = sample_row(x[r].double().cpu().numpy(), float(T[r]), int(k[r]), float(p[r]), float(q[r]), u[r].double().cpu().numpy())
        kept = (cut[r] > -math.inf).numpy()
        differs = np.nonzero(kept != o["kept"])[0]
        assert set(differs) <= set(o["near_cut"].tolist())
        if len(differs):
            left_out += 1
            continue
        clear = ~o["near_draw"]
        left_out += int((~clear).sum())
        assert np.array_equal(tok[r].numpy()[clear], o["tokens"][clear])
        assert np.allclose(prob[r].numpy()[clear], o["probs"][clear], rtol=4e-6, atol=1e-12)
    assert left_out <= 3


def test_strides_alignment_and_in_place():
    V = 3001
    for dtype in (torch.bfloat16, torch.float32):
        for shift in range(0, 9):
            base = rows("normal", 6, V + 13, dtype, shift)
            x = base[:, shift:shift + V]
            T, k, p, q = params(6, shift, "kpq")
            u = torch.full((6, 2), 0.37, device="cuda")
            a, b, c = defined(x, T, u, k, p, q)
            keep = base.clone()
            out = torch.full((6, V + 5), 7.0, dtype=dtype, device="cuda")
            tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=out[:, 2:2 + V])
            assert torch.equal(tok, a) and torch.equal(prob, b) and torch.equal(cut, c)
            assert torch.all(out[:, :2] == 7) and torch.all(out[:, 2 + V:] == 7) and torch.equal(base, keep)
            sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=x)        # in place
            assert torch.equal(x, c)
            keep[:, shift:shift + V] = c
            assert torch.equal(base, keep)                                   # nothing beside the rows changed


def test_bad_rows_are_flagged_and_others_stand():
    R, V = 12, 5000
    x = rows("normal", R, V, torch.float32, 1)
    T, k = torch.ones(R, device="cuda"), torch.full((R,), 20, dtype=torch.int32, device="cuda")
    p, q, u = torch.full((R,), 0.9, device="cuda"), torch.zeros(R, device="cuda"), torch.full((R, 2), 0.5, device="cuda")
    x[0, 4321], x[1, 17], x[2] = math.nan, math.inf, -math.inf
    T[3], T[4], T[5] = -1.0, math.nan, math.inf
    k[6], p[7], p[8], q[9], u[10, 1] = -1, 0.0, 1.5, -0.1, 1.0
    ws = sv.sample_workspace(R, V)
    tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True, ws=ws)
    st, bits = sv.sv_query_status(ws)
    assert st == sv.SV_ERR_DEVICE_INPUT
    assert bits == sv.SV_DEV_BAD_LOGIT | sv.SV_DEV_BAD_TEMPERATURE | sv.SV_DEV_BAD_FILTER
    for r in range(11):
        assert torch.all(tok[r] == -1) and torch.all(cut[r] == -math.inf)
        assert torch.all(prob[r] == 0) if r == 2 else torch.all(torch.isnan(prob[r]))
    a, b, c = defined(x[11:], T[11:], u[11:], k[11:], p[11:], q[11:])
    assert torch.equal(tok[11:], a) and torch.equal(prob[11:], b) and torch.equal(cut[11:], c)
    assert sv.sv_query_status(ws) == (sv.SV_OK, 0)


def test_no_draws_no_probs_many_draws():
    x = rows("normal", 3, 1000, torch.bfloat16, 1)
    T = torch.tensor([1.0, 0.0, 0.5], device="cuda")
    p = torch.full((3,), 0.8, device="cuda")
    _, _, cut = sv.sample(x, T, torch.empty((3, 0), device="cuda"), top_p=p, filtered=True)
    assert torch.equal(cut, defined(x, T, torch.zeros((3, 1), device="cuda"), p=p)[2])
    u = torch.arange(1024, device="cuda").expand(3, 1024).contiguous() / 1024
    tok, prob, _ = sv.sample(x, T, u, top_p=p, probs=False)
    assert prob is None and torch.equal(tok, defined(x, T, u, p=p)[0])
    assert torch.all(tok[:, 1:] >= tok[:, :-1])        # an inverse CDF in vocabulary order


def test_extreme_temperatures():
    x = rows("normal", 4, 3000, torch.float32, 3)
    T = torch.tensor([1e-30, 1e-39, 1e4, 3e38], device="cuda")
    u = torch.full((4, 3), 0.61, device="cuda")
    tok, prob, _ = sv.sample(x, T, u)
    assert torch.all(tok[:2] == x[:2].argmax(1, keepdim=True)) and torch.all(prob[:2] == 1)
    assert torch.all((prob[2:] * 3000 - 1).abs() < 1e-2)
    assert torch.all((tok[3] - 1830).abs() <= 1)


def test_losslessness_with_cut_rows():
    """Drafts drawn from cut rows, verified with the cut rows as both distributions' rows: a draft that equals its
    target is always accepted."""
    B, K, V = 8, 3, 8000
    t = rows("normal", B * (K + 1), V, torch.bfloat16, 9)
    T = torch.ones(B * (K + 1), device="cuda")
    p = torch.full((B * (K + 1),), 0.9, device="cuda")
    u = torch.rand((B * (K + 1), 1), device="cuda").clamp(max=0.9999999)
    tok, _, cut = sv.sample(t, T, u, top_p=p, filtered=True)
    cut = cut.view(B, K + 1, V)
    drafts = tok.view(B, K + 1)[:, :K].contiguous()
    out, n, _, _, _ = sv.verify_sample(cut.reshape(-1, V), cut[:, :K].reshape(-1, V).contiguous(), drafts,
                                       torch.ones(B, device="cuda"), K, seed=3)
    assert torch.all(n == K) and torch.equal(out[:, :K], drafts)


def test_stream_and_graph():
    R, V = 5, 9000
    x = rows("normal", R, V, torch.bfloat16, 2)
    T, k, p, q = params(R, 2, "kpq")
    u = torch.full((R, 1), 0.4, device="cuda")
    want = defined(x, T, u, k, p, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        tok, prob, cut = sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=True)
    side.synchronize()
    assert torch.equal(tok, want[0]) and torch.equal(cut, want[2])
    ws = sv.sample_workspace(R, V)
    out, cut = (torch.empty_like(tok), torch.empty_like(prob)), torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sample(x, T, u, top_k=k, top_p=p, min_p=q, filtered=cut, out=out, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(cut, want[2])
