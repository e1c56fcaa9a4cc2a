"""Verification of drafted tokens (include/draft.h) on the GPU, against the
definition in 64 bits (numpy, exact sums).  Tokens and counts are whole
numbers and must be equal; where a drawn token lies within 2^-40 of the total
of a running sum's border, either side of it is right (no test's does)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rank_latent_kv_gb300 import palu
    palu.lib()
    return palu


def reference(target, draft, drafts, au, su, n_drafts):
    B, k = drafts.shape
    V = target.shape[2]
    toks, kept = np.full((B, k + 1), -1, np.int64), np.zeros(B, np.int32)
    for b in range(B):
        n, a = int(n_drafts[b]), 0
        while a < n:
            x = drafts[b, a]
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, a, x])
            if not float(au[b, a]) * q < float(target[b, a, x]):
                break
            a += 1
        p = target[b, a].astype(np.float64)
        w = p.copy()
        if a < n:
            if draft is not None:
                w = p - draft[b, a].astype(np.float64)
            elif 0 <= drafts[b, a] < V:
                w[drafts[b, a]] = 0
        with np.errstate(invalid="ignore"):
            w = np.where(w > 0, w, 0.0)
            if not w.sum() > 0:
                w = np.where(p > 0, p, 0.0)
        kept[b] = a
        toks[b, :a] = drafts[b, :a]
        total = math.fsum(w)
        if total > 0:
            cum = np.cumsum(w.astype(np.longdouble))
            toks[b, a] = int(np.searchsorted(cum, np.longdouble(su[b]) * cum[-1], side="right"))
    return toks, kept


def inputs(B, k, V, seed, sharp=3.0, near=1.0, draft=True):
    rng = np.random.default_rng(seed)
    logits = sharp * rng.standard_normal((B, k + 1, V))
    soft = lambda z: (np.exp(z - z.max(-1, keepdims=True)) / np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)).astype(np.float32)
    t = soft(logits)
    d = soft(logits[:, :k] + near * rng.standard_normal((B, k, V))) if draft else None
    src = d if draft else t[:, :k]
    x = np.array([[rng.choice(V, p=(src[b, i].astype(np.float64) / src[b, i].astype(np.float64).sum())) for i in range(k)]
                  for b in range(B)], dtype=np.int64)
    return t, d, x, rng.random((B, k), dtype=np.float32), rng.random(B, dtype=np.float32)


def call(P, t, d, x, au, su, **kw):
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    out, kept, new = P.draft_verify(dev(t), dev(d), dev(x), dev(au), dev(su), **kw)
    return out.cpu().numpy(), kept.cpu().numpy(), None if new is None else new.cpu().numpy()


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,k,V", [(1, 1, 1), (1, 1, 2), (3, 2, 31), (2, 4, 127), (5, 3, 129), (4, 7, 1000), (2, 1, 4097),
                                   (9, 5, 32003), (2, 3, 152065), (1, 40, 77)])
def test_against_the_definition(P, B, k, V, draft):
    t, d, x, au, su = inputs(B, k, V, B * 100 + k + V, draft=draft)
    n = np.array([(k - i * 3) % (k + 1) for i in range(B)], np.int32)
    lengths = np.arange(B, dtype=np.int64) + 50
    out, kept, new = call(P, t, d, x, au, su, n_drafts=torch.from_numpy(n).to(DEV), lengths=torch.from_numpy(lengths).to(DEV))
    rt, rk = reference(t, d, x, au, su, n)
    assert np.array_equal(kept, rk) and np.array_equal(out, rt)
    assert np.array_equal(new, lengths - (n - rk))


def test_many_draws_follow_exact_sums(P):
    """Flat, long rows: gaps between running sums far below an fp32 ulp of the total."""
    B, k, V = 64, 1, 60000
    t, d, x, au, su = inputs(B, k, V, 7, sharp=0.5, near=0.3)
    out, kept, _ = call(P, t, d, x, au, su)
    rt, rk = reference(t, d, x, au, su, np.full(B, k))
    assert np.array_equal(kept, rk) and np.array_equal(out, rt)


def test_borders_ties_and_extremes(P):
    V, k = 300, 2
    t = np.zeros((7, k + 1, V), np.float32)
    d = np.zeros((7, k, V), np.float32)
    x = np.zeros((7, k), np.int64)
    au, su = np.zeros((7, k), np.float32), np.zeros(7, np.float32)
    # 0: u q == p exactly is not kept; the drawn token is the lowest with a weight at u = 0
    t[0, 0, 5], d[0, 0, 5], t[0, 0, 200], x[0, 0], au[0, 0] = 0.25, 0.5, 0.75, 5, 0.5
    # 1: everything kept, drawn from the last row with the largest u below 1
    t[1, :, 7] = 1.0
    d[1, :, 7], x[1] = 1.0, 7
    t[1, 2, 7], t[1, 2, 299], au[1], su[1] = 0.5, 0.5, 1 - 2.0 ** -24, 1 - 2.0 ** -24
    # 2: target and draft equal but the draft's token has no probability: no weight is left, the target's row is used
    t[2, 0, 3] = t[2, 0, 4] = d[2, 0, 3] = d[2, 0, 4] = 0.5
    x[2, 0], su[2] = 9, 0.5                                      # 0.5 * 1.0: not above, so token 4
    # 3: a row of zeros: no token
    x[3, 0], au[3, 0] = 1, 0.5
    # 4: NaN weights count as nothing
    t[4, 0] = np.nan
    t[4, 0, 250], x[4, 0] = 0.125, 8
    # 5: tokens outside the vocabulary are never kept
    x[5] = [V, -1]
    t[5, 0, 11] = 1.0
    # 6: subnormal weights
    t[6, 0, 100], t[6, 0, 101], x[6, 0], su[6] = 2.0 ** -140, 2.0 ** -140, 5, 0.75
    out, kept, _ = call(P, t, d, x, au, su)
    rt, rk = reference(t, d, x, au, su, np.full(7, k))
    assert np.array_equal(kept, rk) and np.array_equal(out, rt)
    assert out[0, 0] == 200 and out[1].tolist() == [7, 7, 299] and out[2, 0] == 4 and out[3, 0] == -1
    assert out[4, 0] == 250 and out[5, 0] == 11 and out[6, 0] == 101


def test_clamped_counts_strided_tables_and_given_outputs(P):
    B, k, V = 4, 3, 501
    t, d, x, au, su = inputs(B, k, V, 77)
    n = np.array([-5, 9, 2, 0], np.int32)
    tt = torch.zeros(B + 1, k + 3, V + 5, device=DEV)
    tt[:B, :k + 1, :V] = torch.from_numpy(t).to(DEV)
    dd = torch.zeros(k, B, V, device=DEV)
    dd[:] = torch.from_numpy(d).to(DEV).transpose(0, 1)
    toks = torch.full((B, k + 1), 99, dtype=torch.int64, device=DEV)
    lengths = torch.full((B,), 1 << 40, dtype=torch.int64, device=DEV)
    dev = lambda a: torch.from_numpy(a).to(DEV)
    out, kept, new = P.draft_verify(tt[:B, :k + 1, :V], dd.transpose(0, 1), dev(x), dev(au), dev(su), n_drafts=dev(n),
                                    lengths=lengths, tokens=toks, new_lengths=lengths)
    m = np.clip(n, 0, k)
    rt, rk = reference(t, d, x, au, su, m)
    assert out is toks and new is lengths
    assert np.array_equal(toks.cpu().numpy(), rt) and np.array_equal(kept.cpu().numpy(), rk)
    assert np.array_equal(lengths.cpu().numpy(), (1 << 40) - (m - rk).astype(np.int64))


def test_distribution_is_the_targets(P):
    """The first token, over many random numbers, has the target's distribution: the 5-sigma bar of 40 binomials."""
    V, N = 40, 20000
    rng = np.random.default_rng(5)
    t = rng.dirichlet(np.ones(V) * 0.5, 2).astype(np.float32)
    q = rng.dirichlet(np.ones(V) * 0.5).astype(np.float32)
    x = rng.choice(V, (N, 1), p=q.astype(np.float64) / q.astype(np.float64).sum())
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    out, _, _ = P.draft_verify(dev(t)[None].expand(N, -1, -1), dev(q)[None, None].expand(N, -1, -1), dev(x),
                               dev(rng.random((N, 1), dtype=np.float32)), dev(rng.random(N, dtype=np.float32)))
    count = np.bincount(out[:, 0].cpu().numpy(), minlength=V)
    p = t[0].astype(np.float64)
    p /= p.sum()
    assert (np.abs(count - N * p) <= 5 * np.sqrt(N * p * (1 - p)) + 1).all()


def test_captured_graph(P):
    B, k, V = 3, 4, 5000
    t, d, x, au, su = inputs(B, k, V, 3)
    dev = lambda a: torch.from_numpy(a).to(DEV)
    t1, d1, x1, a1, s1 = map(dev, (t, d, x, au, su))
    toks, kept = torch.zeros(B, k + 1, dtype=torch.int64, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.draft_verify(t1, d1, x1, a1, s1, tokens=toks, n_kept=kept)
    for seed in (4, 5):
        new = inputs(B, k, V, seed)
        for a, b in zip((t1, d1, x1, a1, s1), new):
            a.copy_(torch.from_numpy(b))
        g.replay()
        rt, rk = reference(*new, np.full(B, k))
        assert np.array_equal(toks.cpu().numpy(), rt) and np.array_equal(kept.cpu().numpy(), rk)


def test_refusals(P):
    B, k, V = 2, 3, 50
    t, d = torch.zeros(B, k + 1, V, device=DEV), torch.zeros(B, k, V, device=DEV)
    x, au, su = torch.zeros(B, k, dtype=torch.int64, device=DEV), torch.zeros(B, k, device=DEV), torch.zeros(B, device=DEV)
    n = torch.zeros(B, dtype=torch.int32, device=DEV)
    for f in (lambda: P.draft_verify(t.half(), d, x, au, su), lambda: P.draft_verify(t[:, :k], d, x, au, su),
              lambda: P.draft_verify(t, d[:, :2], x, au, su), lambda: P.draft_verify(t, d.double(), x, au, su),
              lambda: P.draft_verify(t, d, x.int(), au, su), lambda: P.draft_verify(t, d, x, au[:, :2], su),
              lambda: P.draft_verify(t, d, x, au, su[:1]), lambda: P.draft_verify(t, d, x, au, su, n_drafts=n.long()),
              lambda: P.draft_verify(t, d, x, au, su, lengths=n), lambda: P.draft_verify(t, d, x, au, su, new_lengths=n.long()),
              lambda: P.draft_verify(t[:, :, ::2], d[:, :, ::2], x, au, su), lambda: P.draft_verify(t, d.cpu(), x, au, su),
              lambda: P.draft_verify(t[:, :1, :0], None, x[:, :0], au[:, :0], su)):
        with pytest.raises((ValueError, P.PaluError)):
            f()


def test_kept_lengths_roll_a_latent_cache_back(P):
    """Drafts appended to a ragged latent cache, verified, and rolled back by the lengths that come out."""
    B, H, k, V, S = 3, 2, 4, 64, 37
    rng = np.random.default_rng(1)
    xk = torch.from_numpy(rng.standard_normal((B, H, S, 128)).astype(np.float16)).to(DEV)
    cfg = P.palu_config_default(n_head_groups=1, rank=16)
    basis, mu, _, _, _ = P.fit(cfg, xk)
    kc = P.LatentCache(cfg, P.PALU_ROLE_KEY, 16, B, H, 128, basis, mu)
    kc.append(xk)
    n = np.array([4, 2, 0], np.int32)
    new = torch.from_numpy(rng.standard_normal((B, H, k + 1, 128)).astype(np.float16)).to(DEV)
    kc.append_ragged(new, torch.from_numpy(n + 1).to(DEV))
    t, d, x, au, su = inputs(B, k, V, 12, near=2.0)
    dev = lambda a: torch.from_numpy(a).to(DEV)
    _, kept, keep = P.draft_verify(dev(t), dev(d), dev(x), dev(au), dev(su), n_drafts=dev(n),
                                   lengths=torch.tensor(kc.lengths(), dtype=torch.int64, device=DEV))
    kc.truncate_ragged(keep)
    assert kc.sync() == 0
    rt, rk = reference(t, d, x, au, su, n)
    assert kc.lengths() == [S + 1 + int(a) for a in rk] and np.array_equal(kept.cpu().numpy(), rk)
