"""Sampling against the definition evaluated row by row in 64 bits (numpy)."""
import numpy as np
import pytest
import torch

import int4_weight_only_gemm_amd as w4
from gpu_helpers import log

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# prob is rounded once to binary32; a weight sum of V <= 2^18 terms of half a unit of 2^-44 each is
# off by at most 2^-27 of a sum that is at least 1
PROB = 2.0 ** -24 + 2.0 ** -26


def draw(z, u, t=1.0, k=0, p=1.0, mp=0.0):
    """(token, prob) of one row by the definition."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    if z.max() == -np.inf:
        return -1, 0.0
    if not t > 0:
        return int(z.argmax()), 1.0
    by = np.lexsort((np.arange(z.size), -z))
    w = np.where(z == z.max(), 1.0, 0.0) if z.max() == np.inf else np.exp((z - z.max()) / t)
    w = np.where(z == -np.inf, 0.0, w)
    if 0 < k < z.size:
        by = by[:k]
    if p < 1:
        run = np.cumsum(w[by])
        by = by[:max(1, int(np.searchsorted(run, max(p, 0.0) * run[-1], side="left")) + 1)]
    if mp > 0:
        by = by[w[by] >= min(mp, 1.0)]
    by = np.sort(by)
    run = np.cumsum(w[by])
    at = int(np.searchsorted(run, min(max(u, 0.0), 1.0) * run[-1], side="right"))
    if at >= by.size:
        at = int(np.nonzero(w[by])[0][-1])
    return int(by[at]), float(w[by[at]] / run[-1])


def check(logits, u, t=None, k=None, p=None, mp=None, what=""):
    B = logits.shape[0]
    log(f"sample {what} {tuple(logits.shape)} {logits.dtype}")
    dev = [None if x is None else x.cuda() for x in (t, k, p, mp)]
    token, prob = w4.sample(logits.cuda() if not logits.is_cuda else logits, u.cuda(), *dev)
    token, prob = token.cpu().numpy(), prob.cpu().numpy()
    z = logits.float().cpu().numpy()
    for b in range(B):
        a = [d if x is None else x[b].item() for x, d in ((t, 1.0), (k, 0), (p, 1.0), (mp, 0.0))]
        want, pw = draw(z[b], float(u[b]), *a)
        assert token[b] == want, f"{what}: row {b} of {B}: token {token[b]}, not {want} (settings {a}, u={float(u[b])})"
        assert abs(prob[b] - pw) <= PROB * pw + 2.0 ** -44, f"{what}: row {b}: prob {prob[b]}, not {pw}"
    return token


def settings(B, g):
    r = lambda: torch.rand(B, generator=g)  # noqa: E731
    t = torch.where(r() < 0.1, torch.zeros(B), 0.3 + 1.2 * r())
    k = torch.where(r() < 0.3, torch.zeros(B), 1 + 200 * r() ** 3).int()
    p = torch.where(r() < 0.3, torch.ones(B), 0.2 + 0.79 * r())
    mp = torch.where(r() < 0.5, torch.zeros(B), 0.2 * r())
    return t, k, p, mp


@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (5, 63), (7, 1000), (4, 4099), (40, 32000), (1, 152064), (6, 151936),
                                 (160, 8200)])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_mixed_settings(B, V, kind):
    g = torch.Generator().manual_seed(B + V)
    z = (2.5 * torch.randn(B, V, generator=g))
    z[:, :min(V, 40)] += 6 * torch.rand(B, min(V, 40), generator=g)
    z = z.to(kind)
    t, k, p, mp = settings(B, g)
    u = torch.rand(B, generator=g)
    check(z, u, t, k, p, mp, "all cuts")
    check(z, u, t, None, p, None, "top-p")
    check(z, u, t, k, None, None, "top-k")
    check(z, u, t, None, None, mp, "min-p")
    check(z, u, None, None, None, None, "plain")


def test_every_u_of_a_small_row():
    # the whole line of u through one row: each kept token in turn, in the order of the vocabulary
    z = torch.tensor([[0.0, 2.0, -1.0, 2.0, 1.0, float("-inf"), 0.5]]).repeat(401, 1)
    u = torch.linspace(0, 1, 401) * (1 - 2.0 ** -24)
    full = lambda v, kind=F32: torch.full((401,), v, dtype=kind)  # noqa: E731
    assert set(check(z, u, what="plain")) == {0, 1, 2, 3, 4, 6}
    assert set(check(z, u, k=full(3, torch.int32), what="k=3")) == {1, 3, 4}
    assert set(check(z, u, k=full(1, torch.int32), what="k=1: the first of two equal ones")) == {1}
    assert set(check(z, u, p=full(0.5), what="p=.5")) == {1, 3}
    assert set(check(z, u, p=full(0.0), what="p=0 keeps one")) == {1}
    assert set(check(z, u, mp=full(0.3), what="min-p")) == {1, 3, 4}
    assert set(check(z, u, mp=full(7.0), what="min-p above 1")) == {1, 3}


def test_ties_and_degenerate_rows():
    V = 20000
    z = torch.zeros(12, V)
    z[1] = -3.0                                           # all equal, more than a row's list holds
    z[2, 777] = 5.0
    z[3] = float("-inf")                                  # nothing to draw
    z[4] = float("nan")
    z[5, ::2] = float("nan")
    z[6, 5], z[6, 9] = float("inf"), float("inf")
    z[7] = float("-inf")
    z[7, 4321] = -1e30
    z[8] = torch.linspace(-1e-4, 1e-4, V)                 # nearly equal: one bin
    z[9, 100:] = -0.0                                     # -0 and 0 are equal
    z[10] = torch.randn(V, generator=torch.Generator().manual_seed(3)).round()   # a few values, long ties
    z[11] = 1e38 * torch.randn(V, generator=torch.Generator().manual_seed(4))
    g = torch.Generator().manual_seed(5)
    for i in range(4):
        u = torch.rand(12, generator=g)
        t = torch.full((12,), (1.0, 0.5, 2.0, 1.0)[i])
        k = torch.full((12,), (7, 5000, 19999, 0)[i], dtype=torch.int32)
        p = torch.full((12,), (1.0, 0.6, 0.9, 0.35)[i])
        check(z, u, t, k, p, None, f"ties {i}")
        check(z, u, t, None, None, None, f"ties plain {i}")
        check(z.to(BF16), u, t, k, None, None, f"ties bf16 {i}")


@pytest.mark.parametrize("V", [152064, 400000])
def test_deep_cuts(V):
    # flat rows: cuts deep in the bulk, top-k of tens of thousands, long vocabularies
    g = torch.Generator().manual_seed(V)
    z = torch.cat([1.3 * torch.randn(3, V, generator=g), 0.01 * torch.randn(1, V, generator=g)])
    p = torch.tensor([0.9, 0.5, 0.99, 0.3])
    k = torch.tensor([0, 60000, 30000, 0], dtype=torch.int32)
    u = torch.rand(4, generator=g)
    t = torch.tensor([1.0, 0.7, 1.5, 1.0])
    check(z, u, t, k, p, None, "deep cuts")
    check(z, u, t, k, p, torch.full((4,), 0.01), "deep cuts, min-p")
    check(z, u, None, None, None, torch.full((4,), 1e-5), "min-p below the near weights")
    check((4 * z).to(BF16), u, t, k, p, None, "deep cuts bf16")
    check((2 * z).round() / 2, u, t, k, p, None, "a few values, cuts in long runs of equal logits")


def test_extreme_settings():
    g = torch.Generator().manual_seed(11)
    z = 3 * torch.randn(8, 5000, generator=g)
    t = torch.tensor([-1.0, 0.0, float("nan"), 1e-6, 1e-30, 1e6, 0.7, 0.7])
    k = torch.tensor([5, 5, 5, 5, 5, 0, -3, 1 << 30], dtype=torch.int32)
    p = torch.tensor([0.9, 0.9, 0.9, 0.9, 0.9, 1.5, float("nan"), -1.0])
    mp = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.0, -1.0, float("nan"), 0.0])
    check(z, torch.tensor([0.5, 0.5, 0.5, 0.5, 0.5, 0.25, 1.5, -2.0]), t, k, p, mp, "extremes")


def test_strides_streams_graph_and_repeat():
    g = torch.Generator().manual_seed(13)
    B, V = 9, 12345
    wide = torch.randn(B, V + 7, generator=g).cuda()
    t, k, p, mp = (x.cuda() for x in settings(B, g))
    u = torch.rand(B, generator=g).cuda()
    for kind in (F32, BF16):
        x = wide.to(kind)[:, 3:3 + V]
        a, b = w4.sample(x, u, t, k, p, mp), w4.sample(x.contiguous(), u, t, k, p, mp)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = wide[:, :V].contiguous()
    with torch.cuda.stream(s):
        first = w4.sample(z, u, t, k, p, mp)              # sizes the stream's workspace
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = w4.sample(z, u, t, k, p, mp)
        for i in range(5):
            z.copy_(torch.randn(B, V, generator=g))
            u.copy_(torch.rand(B, generator=g))
            graph.replay()
            s.synchronize()
            again = [x.clone() for x in got]
            eager = w4.sample(z, u, t, k, p, mp)
            s.synchronize()
            assert torch.equal(again[0], eager[0]) and torch.equal(again[1], eager[1]), f"replay {i}"
    assert first[0].shape == (B,)
    assert w4.sample(z[:0], u[:0])[0].shape == (0,)


def test_many_rows():
    # more rows than one set of launches takes
    g = torch.Generator().manual_seed(17)
    B, V = 1500, 300
    z = 2 * torch.randn(B, V, generator=g)
    t, k, p, mp = settings(B, g)
    check(z, torch.rand(B, generator=g), t, k, p, mp, "many rows")


def test_refusals():
    z, u = torch.zeros(3, 10, device="cuda"), torch.zeros(3, device="cuda")
    for change in (dict(u=u[:2]), dict(u=u.double()), dict(top_k=u), dict(top_p=u.half()), dict(logits=z.half()),
                   dict(logits=z.t()), dict(temperature=u.cpu()), dict(min_p=u[None])):
        args = dict(logits=z, u=u)
        args.update(change)
        with pytest.raises((ValueError, TypeError)):
            w4.sample(**args)
    with pytest.raises(w4.W4Error):
        w4.sample(torch.zeros(1, (1 << 19) + 1, device="cuda"), u[:1])
