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
