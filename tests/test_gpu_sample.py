"""Sampling on the GPU against the sorting oracle: tokens equal, log
probabilities within 2^-22 of their size (one fp32 rounding is 2^-24; the rest
is 64-bit arithmetic).  The inputs come with the generator's seed; a draw lands
within 1e-12 of a border between tokens with probability below 1e-6 per test."""
import numpy as np
import pytest
import torch

import slq_synth as S
import weight_only_mixed_amd as slq
from oracle import serve as orc
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def dev(a, t=None):
    return None if a is None else torch.from_numpy(np.asarray(a)).to(DEV if t is None else t)


def check(logits, u, what="", **cuts):
    """logits: a device tensor, the cuts numpy arrays or None."""
    tok, lp = slq.slq_sample(logits, dev(u), **{n: dev(c) for n, c in cuts.items()})
    tok2, lp2 = slq.slq_sample(logits, dev(u), **{n: dev(c) for n, c in cuts.items()})
    torch.cuda.synchronize()
    rt, rl, kept = orc.sample(logits.double().cpu().numpy(), u, **cuts)
    t, l = tok.cpu().numpy(), lp.double().cpu().numpy()
    say(f"sample {what} {tuple(logits.shape)} {logits.dtype}: kept {kept.min()}..{kept.max()}, differing {int((t != rt).sum())}")
    assert np.array_equal(t, rt), (what, np.flatnonzero(t != rt)[:5], t[t != rt][:5], rt[t != rt][:5], kept[t != rt][:5])
    fin = np.isfinite(rl)
    assert np.array_equal(fin, np.isfinite(l)) and np.all(np.abs(l - rl)[fin] <= 2.0 ** -22 * np.abs(rl[fin]) + 1e-12)
    assert torch.equal(tok, tok2) and torch.equal(lp, lp2)
    return t, kept


def rows_of(g, rows, vocab, dtype, sigma=2.5, boost=8.0):
    l = g.standard_normal((rows, vocab)) * sigma
    for r in range(rows):
        l[r, g.integers(0, vocab, 20)] += boost * g.random(20)
    return torch.from_numpy(l.astype(np.float32)).to(T[dtype]).to(DEV)


def settings(g, rows, vocab):
    f = np.float32
    return {
        "free": {},
        "temperature": dict(temperature=g.uniform(0.2, 3, rows).astype(f)),
        "top-k": dict(top_k=g.integers(1, max(2, min(vocab, 100)), rows).astype(np.int32)),
        "wide top-k": dict(top_k=g.integers(1, vocab + 5, rows).astype(np.int32)),
        "top-p": dict(top_p=g.uniform(0.05, 1.05, rows).astype(f), temperature=g.uniform(0.5, 1.5, rows).astype(f)),
        "min-p": dict(min_p=(10.0 ** g.uniform(-6, 0, rows)).astype(f)),
        "all": dict(temperature=g.uniform(0.5, 2, rows).astype(f), top_k=g.integers(-2, 300, rows).astype(np.int32),
                    top_p=g.uniform(0.3, 1.1, rows).astype(f), min_p=g.uniform(-0.01, 0.05, rows).astype(f)),
        "greedy": dict(temperature=np.zeros(rows, f), top_k=np.full(rows, 5, np.int32)),
    }


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 63), (5, 64), (4, 65), (9, 1000), (3, 4097), (6, 50257), (2, 151936)])
def test_shapes_and_settings(dtype, rows, vocab):
    g = np.random.default_rng(rows * 31 + vocab)
    logits = rows_of(g, rows, vocab, dtype)
    for what, cuts in settings(g, rows, vocab).items():
        check(logits, g.random(rows).astype(np.float32), what, **cuts)


@pytest.mark.parametrize("vocab", [1, 7, 1000, 20000, 151936])
def test_ties(vocab):
    """All logits equal, two values only, and a coarse grid."""
    g = np.random.default_rng(vocab)
    for l in (np.zeros((4, vocab)), g.integers(0, 2, (4, vocab)) * 0.5, np.round(g.standard_normal((4, vocab)) * 4) / 2):
        logits = torch.from_numpy(l.astype(np.float32)).to(DEV)
        u = np.array([0.0, 0.3, 0.77, 1 - 2.0 ** -24], np.float32)
        check(logits, u, "free")
        check(logits, u, "top-k", top_k=np.array([1, 3, max(1, vocab // 2), vocab - 1], np.int32))
        check(logits, u, "top-p", top_p=np.array([0.0, 0.2, 0.5001, 0.9999], np.float32))
        check(logits, u, "both", top_k=np.array([2, 5, 600, vocab], np.int32), top_p=np.array([0.4, 0.61, 0.3, 0.8], np.float32))
        check(logits, u, "greedy", temperature=np.zeros(4, np.float32))
        check(logits, u, "min-p 1", min_p=np.array([1, 1, 2, 0.5], np.float32))


def test_draws_reach_every_kept_token():
    """u over a fine grid: shares of the draws as the probabilities say."""
    p = np.array([0.02, 0.5, 0.08, 0.3, 0.1])
    n = 1000
    logits = torch.from_numpy(np.log(np.tile(p, (n, 1))).astype(np.float32)).to(DEV)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    t, _ = check(logits, u, "grid")
    assert np.array_equal(np.bincount(t, minlength=5), (p * n).round())
    t, _ = check(logits, u, "grid top-k 2", top_k=np.full(n, 2, np.int32))
    assert np.array_equal(np.bincount(t, minlength=5), [0, 625, 0, 375, 0])


def test_infinities_nan_and_empty_rows():
    inf = np.inf
    g = np.random.default_rng(1)
    l = g.standard_normal((10, 3001)).astype(np.float32)
    l[0] = -inf
    l[1, 1:] = -inf
    l[2, ::2] = -inf
    l[3, 5] = inf
    l[4, [5, 9]] = inf
    l[5, ::3] = np.nan
    l[6] = np.nan
    l[7] = 3e38 * np.sign(l[7])
    l[8] = np.where(np.arange(3001) % 2, 1e-42, -1e-42)
    l[9] = np.where(np.arange(3001) % 2, 0.0, -0.0)
    u = g.random(10).astype(np.float32)
    for t in ("fp32", "bf16"):
        logits = torch.from_numpy(l).to(T[t]).to(DEV)
        for what, cuts in settings(g, 10, 3001).items():
            check(logits, u, what, **cuts)
        check(logits, u, "hot", temperature=np.full(10, inf, np.float32))
        check(logits, u, "cold", temperature=np.full(10, 1e-30, np.float32), top_p=np.full(10, 0.5, np.float32))
        check(logits, u, "not a number", temperature=np.full(10, np.nan, np.float32))
        check(logits, u, "no cuts", top_p=np.full(10, np.nan, np.float32), min_p=np.full(10, np.nan, np.float32),
              top_k=np.full(10, -7, np.int32))


def test_lists_that_end_at_zero():
    """Units whose listed elements reach down to exactly +-0, and to the numbers beside it."""
    g = np.random.default_rng(17)
    l = -np.abs(g.standard_normal((6, 9000))).astype(np.float32)
    for r in range(6):
        at = g.permutation(9000)[:600]
        l[r, at] = np.float32([0.0, -0.0, 1e-45, -1e-45, 0.0, 0.0])[r] * np.ones(600, np.float32)
        l[r, at[:100]] = g.random(100)
    u = g.random(6).astype(np.float32)
    logits = torch.from_numpy(l).to(DEV)
    for k in (20, 101, 350, 700):
        check(logits, u, f"zeros top-k {k}", top_k=np.full(6, k, np.int32))
    check(logits, u, "zeros top-p", top_p=np.float32([0.01, 0.05, 0.1, 0.12, 0.2, 0.5]))


def test_strided_and_unaligned_rows():
    g = np.random.default_rng(3)
    wide = rows_of(g, 5, 5003, "bf16")
    u = g.random(5).astype(np.float32)
    for v in (wide[:, 1:4097], wide[:, :777], wide[::2, 3:]):
        check(v, u[:v.shape[0]], "view", top_p=np.full(v.shape[0], 0.9, np.float32))
    one = wide[:1].expand(5, 5003)
    check(one, u, "one row for all", top_k=np.full(5, 40, np.int32))


@pytest.mark.parametrize("sigma", [0.01, 1.0, 6.0])
def test_flat_and_steep_rows(sigma):
    g = np.random.default_rng(int(sigma * 100))
    logits = rows_of(g, 8, 60001, "fp32", sigma=sigma, boost=0.0)
    u = g.random(8).astype(np.float32)
    for what, cuts in settings(g, 8, 60001).items():
        check(logits, u, f"sigma {sigma} {what}", **cuts)


@pytest.mark.parametrize("order", ["ascending", "descending"])
def test_sorted_rows(order):
    base = np.linspace(-20, 20, 40000).astype(np.float32)
    l = np.stack([base if order == "ascending" else base[::-1]] * 4)
    u = np.array([0.01, 0.4, 0.8, 0.999], np.float32)
    logits = torch.from_numpy(l).to(DEV)
    check(logits, u, order)
    check(logits, u, order, top_k=np.array([1, 64, 65, 5000], np.int32))
    check(logits, u, order, top_p=np.array([0.1, 0.9, 0.99, 0.9999], np.float32))


def test_fidelity_workload_rows():
    a, _ = S.fidelity_logits(64, S.VOCAB, 0.05, S.seed_for(6))
    g = np.random.default_rng(11)
    u = g.random(64).astype(np.float32)
    check(torch.from_numpy(a).to(DEV), u, "workload", top_k=np.full(64, 50, np.int32), top_p=np.full(64, 0.95, np.float32))
    check(torch.from_numpy(a).to(DEV), u, "workload top-p", top_p=np.full(64, 0.95, np.float32))


def test_more_rows_than_compute_units():
    g = np.random.default_rng(21)
    logits = torch.from_numpy((g.standard_normal((5000, 300)) * 3).astype(np.float32)).to(DEV)
    u = g.random(5000).astype(np.float32)
    check(logits, u, "rows", **settings(g, 5000, 300)["all"])


@pytest.mark.parametrize("vocab", [2041, 2047, 2048, 2049, 2050, 4095, 8193])
@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_sizes_around_the_whole_row_list(vocab, dtype):
    g = np.random.default_rng(vocab)
    logits = rows_of(g, 3, vocab, dtype)
    u = g.random(3).astype(np.float32)
    for what, cuts in settings(g, 3, vocab).items():
        check(logits, u, what, **cuts)


def test_very_many_rows():
    g = np.random.default_rng(41)
    logits = torch.from_numpy((g.standard_normal((70000, 12)) * 2).astype(np.float32)).to(DEV)
    check(logits, g.random(70000).astype(np.float32), "rows", **settings(g, 70000, 12)["top-p"])


def test_two_streams_at_once():
    g = np.random.default_rng(43)
    a, b = rows_of(g, 6, 40009, "fp32"), rows_of(g, 50, 9001, "bf16")
    ua, ub = (torch.from_numpy(g.random(n).astype(np.float32)).to(DEV) for n in (6, 50))
    pa, pb = torch.full((6,), 0.95, device=DEV), torch.full((50,), 0.6, device=DEV)
    ra, rb = slq.slq_sample(a, ua, top_p=pa), slq.slq_sample(b, ub, top_p=pb)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s[0]):
            ta = slq.slq_sample(a, ua, top_p=pa)
        with torch.cuda.stream(s[1]):
            tb = slq.slq_sample(b, ub, top_p=pb)
        torch.cuda.synchronize()
        assert torch.equal(ta[0], ra[0]) and torch.equal(tb[0], rb[0]) and torch.equal(tb[1], rb[1])


def test_graph_replays_with_eager_calls_between():
    g = np.random.default_rng(31)
    logits, u = rows_of(g, 4, 30011, "fp32"), torch.zeros(4, device=DEV)
    p = torch.full((4,), 0.97, device=DEV)
    slq.slq_sample(logits, u, top_p=p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tok, lp = slq.slq_sample(logits, u, top_p=p)
    for r in range(5):
        logits.copy_(rows_of(g, 4, 30011, "fp32"))
        u.copy_(torch.from_numpy(g.random(4).astype(np.float32)))
        graph.replay()
        t2, l2 = slq.slq_sample(logits, u, top_p=p)
        torch.cuda.synchronize()
        assert torch.equal(tok, t2) and torch.equal(lp, l2)
        assert np.array_equal(tok.cpu().numpy(), orc.sample(logits.cpu().numpy(), u.cpu().numpy(), top_p=p.cpu().numpy())[0])


def test_binding_refusals():
    l, u = torch.zeros(2, 8, device=DEV), torch.zeros(2, device=DEV)
    for bad in (dict(temperature=u[:1]), dict(top_k=u), dict(top_p=u.double()), dict(min_p=u.cpu())):
        with pytest.raises(slq.SlqError):
            slq.slq_sample(l, u, **bad)
    for bl, bu in ((l.double(), u), (l[:, :0], u), (l.t(), u), (l[0], u), (l, None), (l, u.bfloat16())):
        with pytest.raises(slq.SlqError):
            slq.slq_sample(bl, bu)
    t, lp = slq.slq_sample(l[:0], u[:0])
    assert t.numel() == 0 and lp.numel() == 0
