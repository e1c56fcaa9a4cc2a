"""Draft verification at the edges of its range: more clusters than the GPU
holds, with rows so short that most of a cluster's segments are empty.  Against
the definition in 64 bits, as in test_gpu_draft.py."""
import numpy as np
import pytest
import torch

from test_gpu_draft import DEV, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rank_latent_kv_gb300 import palu
    palu.lib()
    return palu


@pytest.mark.parametrize("B,V", [(1, 3), (18, 70), (2500, 5), (1200, 130)])
def test_short_rows_of_many_sequences(P, B, V):
    """Segments without a value send their sums at once: not before every CTA of the cluster has begun.  Beside another
    stream's work, which holds CTAs of a cluster back."""
    k = 2
    t, d, x, au, su = inputs(B, k, V, B + V)
    rt, rk = reference(t, d, x, au, su, np.full(B, k))
    dev = [torch.from_numpy(a).to(DEV) for a in (t, d, x, au, su)]
    busy, s = torch.zeros(1 << 24, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        with torch.cuda.stream(s):
            busy.add_(1)
        outs.append(P.draft_verify(*dev)[:2])
    torch.cuda.synchronize()
    for out, kept in outs:
        assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(out.cpu().numpy(), rt)


@pytest.mark.parametrize("B", [18, 64])
def test_long_rows_keep_the_stated_bound(P, B):
    """A row of 41 million weights that are whole numbers, so that the definition is exact in integers: every drawn token's
    border lies within (278 + 12 ceil(V / 16384)) 2^-48 of the total (include/draft.h).  Its first half is flat: equal
    values round alike, so that what is lost adds up; the powers of two behind it lose nothing."""
    V, k = 41_000_003, 1
    g = torch.Generator(device=DEV).manual_seed(B)
    w = torch.full((V,), 1 << 23, device=DEV)
    w[:V // 2] = 12345679
    ui = torch.randint(0, 1 << 24, (B,), generator=g, device=DEV)
    t = (w.double() * 2.0 ** -24).float()[None, None].expand(B, k + 1, V)
    z = torch.zeros(B, k, dtype=torch.int64, device=DEV)
    out, kept, _ = P.draft_verify(t, None, z, torch.zeros(B, k, device=DEV), (ui.double() * 2.0 ** -24).float(),
                                  n_drafts=torch.zeros(B, dtype=torch.int32, device=DEV))
    cum = w.cumsum(0).cpu()
    total = int(cum[-1])
    tol = total * (278 + 12 * -(-V // 16384)) / 2 ** 48
    assert (kept == 0).all()
    for token, u in zip(out[:, 0].tolist(), ui.tolist()):
        want = total * u / 2 ** 24                        # 73 bits, rounded to 53: far below tol
        assert (int(cum[token - 1]) if token else 0) - tol <= want < int(cum[token]) + tol, (token, u)


def test_counts_and_lengths_in_place(P):
    """n_kept may be n_drafts, new_lengths may be lengths; a view shifted by one sequence is refused."""
    B, k, V = 200, 3, 301
    t, d, x, au, su = inputs(B, k, V, 5)
    n = np.arange(B, dtype=np.int32) % (k + 1)
    rt, rk = reference(t, d, x, au, su, n)
    dev = lambda a: torch.from_numpy(a).to(DEV)
    t, d, x, au, su = map(dev, (t, d, x, au, su))
    for _ in range(5):
        count, length = torch.zeros(B + 1, dtype=torch.int32, device=DEV), torch.full((B + 1,), 100, device=DEV)
        count[:B] = dev(n)
        toks, kept, new = P.draft_verify(t, d, x, au, su, n_drafts=count[:B], lengths=length[:B], n_kept=count[:B],
                                         new_lengths=length[:B])
        assert np.array_equal(toks.cpu().numpy(), rt) and np.array_equal(kept.cpu().numpy(), rk)
        assert np.array_equal(new.cpu().numpy(), 100 - (n - rk))
    with pytest.raises(P.PaluError, match="overlap"):
        P.draft_verify(t, d, x, au, su, n_drafts=count[:B], n_kept=count[1:])
    with pytest.raises(P.PaluError, match="overlap"):
        P.draft_verify(t, d, x, au, su, lengths=length[:B], new_lengths=length[1:])
