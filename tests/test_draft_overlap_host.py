"""palu_draft_verify refuses outputs that overlap an input or another output
(sequences run independently: one would overwrite what another has yet to
read), without a GPU.  The arrays lie in one buffer of made-up addresses;
nothing is launched by a refused call."""
import ctypes

import pytest

from tests.test_abi import palu  # noqa: F401  (fixture)

I64x2 = ctypes.c_int64 * 2
B, K, V = 3, 2, 50
M = 1 << 20
SIZE = dict(target=B * (K + 1) * V * 4, draft=B * K * V * 4, drafts=B * K * 8, n_drafts=B * 4, accept_u=B * K * 4, sample_u=B * 4,
            lengths=B * 8, tokens=B * (K + 1) * 8, n_kept=B * 4, new_lengths=B * 8)
AT = {name: (i + 1) * M for i, name in enumerate(SIZE)}
OUT = ("tokens", "n_kept", "new_lengths")


def verify(palu, ts=((K + 1) * V, V), ds=(K * V, V), **at):
    a = dict(AT, **at)
    st = palu.lib().palu_draft_verify(B, K, V, a["target"], I64x2(*ts), a["draft"], I64x2(*ds), a["drafts"], a["n_drafts"],
                                      a["accept_u"], a["sample_u"], a["lengths"], a["tokens"], a["n_kept"], a["new_lengths"], None)
    return st, palu.lib().palu_last_error()


@pytest.mark.parametrize("out", OUT)
def test_each_output_against_everything_else(palu, out):
    for other, size in SIZE.items():
        if other == out:
            continue
        for at in (AT[other] + size - 8, AT[other] - SIZE[out] + 8, AT[other] + 8):
            st, msg = verify(palu, **{out: at})
            assert st == 1 and b"overlap" in msg, (out, other, at)
    # the same array is refused too, but for lengths and new_lengths, n_drafts and n_kept: each sequence its own element
    for other in SIZE:
        if other != out and (out, other) not in (("new_lengths", "lengths"), ("n_kept", "n_drafts")):
            st, msg = verify(palu, **{out: AT[other]})
            assert st == 1 and b"overlap" in msg, (out, other)


def test_strided_tables(palu):
    """A table's extent follows from its strides: behind the last row, and not between rows only."""
    far = AT["target"] + ((B - 1) * 7 * V + K * 2 * V + V) * 4
    st, msg = verify(palu, ts=(7 * V, 2 * V), n_kept=far - 8)
    assert st == 1 and b"overlap" in msg
    for strides in ((1 << 62, V), (V, 1 << 61)):               # an extent that no address space has
        assert verify(palu, ts=strides)[0] == 1
        assert verify(palu, ds=strides)[0] == 1
