"""The serving operators together, as a speculative decode loop uses them: the
new tokens' keys normalised, rotated and appended to pages, attention over the
pages behind a shared prompt, the drafts verified, the lengths rolled back, and
the next step on what remains; and the same queries and keys through
qk_norm_rope into a latent cache.  Every step against 64-bit references."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_draft import reference as verify_reference
from test_gpu_paged import D, DEV, DT, _table, attend_close, close, make_cache, offsets_of, ref_attend, ref_transform

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rank_latent_kv_gb300 import palu
    palu.lib()
    return palu


@pytest.mark.parametrize("dt,Hq,Hk,page,prompt", [("fp16", 24, 8, 16, 64), ("bf16", 7, 1, 64, 256), ("bf16", 16, 2, 32, 0)])
def test_speculative_steps(P, dt, Hq, Hk, page, prompt):
    d, B, k, V, steps = DT[dt], 3, 4, 97, 5
    rng = np.random.default_rng(Hq)
    g = torch.Generator().manual_seed(Hq)
    shared = prompt // page
    lengths = [prompt + n for n in (30, 1, 100)]
    width = -(-(max(lengths) + steps * (k + 1)) // page)
    pools, dev, c = make_cache(P, d, lengths, page, Hk, width=width, shared=shared, seed=3)
    ids = c.page_table.cpu()
    cs = _table(1000, 64)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(d) for _ in range(2)]
    csd, wd = cs.to(DEV), [x.to(DEV) for x in w]
    for _ in range(steps):
        n_drafts = rng.integers(0, k + 1, B).astype(np.int32)
        new = [int(n) + 1 for n in n_drafts]                 # the last token and its drafts
        n = sum(new)
        c.lengths += torch.tensor(new, device=DEV)
        lengths = [a + b for a, b in zip(lengths, new)]
        qkv = torch.randn(n, Hq + 2 * Hk, D, generator=g).to(d)
        x = qkv.to(DEV)
        off = offsets_of(new)
        q = c.append(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], off, q=x[:, :Hq], cos_sin=csd, q_weight=wd[0], k_weight=wd[1])
        out = c.attend(q, off, k + 1, shared_pages=shared)
        # references: the queries and the new rows of the pages, then attention over the pages as stored
        row, host = 0, [t.cpu() for t in dev]
        for b, m in enumerate(new):
            pos = torch.arange(lengths[b] - m, lengths[b])
            sl = slice(row, row + m)
            ref, scale = ref_transform(qkv[sl, :Hq], w[0], cs[pos], False, 1e-6)
            close(q[sl], ref, scale, d)
            at = ids[b].long()[pos // page], slice(None), pos % page
            ref, scale = ref_transform(qkv[sl, Hq:Hq + Hk], w[1], cs[pos], False, 1e-6)
            close(host[0][at], ref, scale, d)
            assert torch.equal(host[1][at], qkv[sl, Hq + Hk:])
            row += m
        ref, mag = ref_attend(q.cpu(), host, ids, lengths, new, page)
        attend_close(out, ref, mag, d)
        # verification, and the rollback by the lengths that come out
        t = rng.dirichlet(np.ones(V) * 0.2, (B, k + 1)).astype(np.float32)
        dr = rng.dirichlet(np.ones(V) * 0.2, (B, k)).astype(np.float32)
        drafts = rng.integers(0, V, (B, k))
        au, su = rng.random((B, k), dtype=np.float32), rng.random(B, dtype=np.float32)
        to = lambda a: torch.from_numpy(a).to(DEV)
        tokens, kept, keep = P.draft_verify(to(t), to(dr), to(drafts), to(au), to(su), n_drafts=to(n_drafts),
                                            lengths=c.lengths, new_lengths=c.lengths)
        assert keep is c.lengths
        rt, rk = verify_reference(t, dr, drafts, au, su, n_drafts)
        assert np.array_equal(tokens.cpu().numpy(), rt) and np.array_equal(kept.cpu().numpy(), rk)
        lengths = [a - int(m) + int(r) for a, m, r in zip(lengths, n_drafts, rk)]
        assert c.lengths.tolist() == lengths and c.sync() == 0


def test_normalised_and_rotated_keys_in_a_latent_cache(P):
    """qk_norm_rope's outputs go straight into the fit, the append and the decode of the latent cache."""
    B, T, Hq, Hk = 2, 70, 6, 2
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(B, T, Hq + 2 * Hk, D, generator=g).half().to(DEV)
    pos = torch.arange(T, device=DEV).expand(B, T).contiguous()
    cs, w = _table(200, 128).to(DEV), torch.ones(D).half().to(DEV)
    q, key = P.qk_norm_rope(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], pos, cs, q_weight=w, k_weight=w)
    val = qkv[:, :, Hq + Hk:].transpose(1, 2).contiguous()
    caches = []
    for role, x in ((P.PALU_ROLE_KEY, key), (P.PALU_ROLE_VALUE, val)):
        cfg = P.palu_config_default(n_head_groups=2, rank=64)
        basis, mu, _, r, _ = P.fit(cfg, x)
        c = P.LatentCache(cfg, role, r, B, Hk, 128, basis, mu)
        c.append(x)
        caches.append(c)
    out = P.decode(*caches, q[:, :, -1].contiguous())
    views = []
    for c, role in zip(caches, (O.ROLE_KEY, O.ROLE_VALUE)):
        Vr, mu = c.basis_array()
        views.append(O.OracleCache.from_buffers(role, Vr, mu, c.c.rank, B, Hk, c.c.capacity, True, c.record_array(),
                                                c.tail_array(), c.c.length))
    err = O.relative_error(out.cpu().numpy(), O.attend(q[:, :, -1].cpu().numpy(), *views))
    assert np.isfinite(err).all() and err.max() < 2e-3
