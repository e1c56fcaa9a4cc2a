"""The 4-bit page format's oracle against facts worked out by hand."""
import numpy as np

from oracle import paged4_oracle as O4


def test_every_nibble_of_a_block_has_one_owner():
    used = np.zeros((O4.BLOCK, 2), int)
    for place in (O4.PLACES[0], O4.PLACES[2]):
        for at, shift in place.reshape(-1, 2):
            used[at, shift // 4] += 1
    for place in (O4.PLACES[1], O4.PLACES[3]):
        for at in place.reshape(-1):
            used[at:at + 2] += 1
    assert (used == 1).all()


def test_a_value_byte_belongs_to_one_token():
    owner = {}
    for t in range(16):
        for d in range(O4.D):
            assert owner.setdefault(O4.value_place(t, d)[0], t) == t


def test_places_by_hand():
    assert O4.key_place(0, 0) == (0, 0) and O4.key_place(0, 1) == (2, 0) and O4.key_place(0, 2) == (0, 4)
    assert O4.key_place(3, 32 + 8 + 7) == (64 * 3 + 16 + 4 + 3, 4)
    assert O4.value_place(0, 8) == (1280, 4) and O4.value_place(9, 64 + 16 + 1) == (1280 + 512 + 64 + 4 + 3, 0)
    assert O4.key_scale_place(15, 3) == (1278 - 8, 1278) and O4.value_scale_place(15, 3) == (2304 + 126, 2304 + 254)


def test_quantiser_by_hand():
    x = np.zeros(O4.D, np.float32)
    x[:32] = np.arange(32) / 2.0 - 3                              # -3 .. 12.5: s = 15.5 / 15, z = -3
    x[32:64] = 7                                                  # no range: s = 0, reads back exactly
    x[64:96] = [0, 15] * 16                                       # s = 1: codes are the values
    x[65] = 2.5                                                   # a tie goes to the even code
    x[96] = np.inf
    c, s, z = O4.quantise(x)
    assert s[0] == np.float16(15.5 / 15) and z[0] == -3 and c[0] == 0 and c[31] == 15
    assert s[1] == 0 and z[1] == 7 and (c[32:64] == 0).all()
    assert s[2] == 1 and z[2] == 0 and c[65] == 2 and c[64] == 0 and c[67] == 15
    assert s[3] == 0 and np.isnan(z[3]) and (c[96:] == 0).all()
    h = O4.held(x)
    assert (h[32:64] == 7).all() and np.isnan(h[96:]).all() and (np.abs(h[:32] - x[:32]) <= float(s[0]) / 2 + 0.02).all()


def test_write_and_read_back():
    rng = np.random.default_rng(0)
    block = rng.integers(0, 256, O4.BLOCK, dtype=np.uint8)
    k, v = rng.standard_normal((2, 16, O4.D)).astype(np.float16).astype(np.float32)
    for t in rng.permutation(16):
        O4.write(block, t, k[t], v[t])
    assert np.array_equal(O4.rows(block, False), O4.held(k)) and np.array_equal(O4.rows(block, True), O4.held(v))


def test_what_is_held_is_finite_in_fp16():
    x = np.zeros(O4.D, np.float32)
    x[:32] = np.linspace(-65504, 65504, 32)
    x[32:64] = np.linspace(65000, 65504, 32)
    x[64:96] = np.linspace(-3e38, 1e38, 32)                       # bf16's range: cut
    c, s, z = O4.quantise(x)
    assert (O4.held(x) <= 65504).all() and s[0] == np.float16(8728) and z[2] == -65504 and c[95] == 15
