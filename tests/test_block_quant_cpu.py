"""The 64-bit reference of the 4-bit formats and the norm against hand-worked cases and differences."""
import numpy as np

from tests import _block_quant as bq


def test_e2m1_rounding_by_hand():
    v = np.array([0.0, -0.0, 0.24, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.0, -0.3, -5.0, -100.0])
    want = [0, 8, 0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 9, 14, 15]
    assert bq.encode(v, bq.E2M1, 8).tolist() == want


def test_e4m3_values():
    assert bq.E4M3[-1] == 448 and bq.E4M3[8] == 2.0 ** -6 and len(bq.E4M3) == 127
    assert bq.E5M2[-1] == 57344 and len(bq.E5M2) == 124
    assert bq.encode(np.array([1.0, 448.0, 500.0, 2.0 ** -10, 2.0 ** -9]), bq.E4M3, 128).tolist() == \
        [0x38, 0x7E, 0x7E, 0, 1]


def bits(v):
    return (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_mxfp4_blocks_by_hand():
    x = np.zeros((1, 128), np.float32)
    x[0, 0], x[0, 1] = 6.0, -1.5                    # amax 6 = 1.5 * 2^2: X = 0
    x[0, 32] = 7.0                                  # saturates: X = 0, 7 -> 6
    x[0, 64], x[0, 65] = np.inf, 1.0                # X = 127: infinity -> 6, 1 -> 0
    x[0, 96] = np.nan
    codes, sf = bq.quantise(bits(x), bq.MXFP4)
    assert sf.tolist() == [[127, 127, 254, 255]]
    assert codes[0, 0] == 7 and codes[0, 1] == 0xB and codes[0, 32] == 7 and codes[0, 64] == 7 and codes[0, 65] == 0
    zero, sz = bq.quantise(np.zeros((1, 32), np.uint16), bq.MXFP4)
    assert sz[0, 0] == 0 and not zero.any()


def test_nvfp4_blocks_by_hand():
    x = np.zeros((1, 32), np.float32)
    x[0, :3] = [6.0, 3.0, -0.5]                     # g = 1: s = e4m3(6 / 6) = 1
    x[0, 16] = 2.0 ** -9                            # s = e4m3(2^-9 / 6) = 0: zero codes
    codes, sf = bq.quantise(bits(x), bq.NVFP4, 1.0)
    assert sf.tolist() == [[0x38, 0]] and codes[0, :3].tolist() == [7, 5, 9] and codes[0, 16] == 0
    codes, sf = bq.quantise(bits(x), bq.NVFP4, 448.0)
    assert sf[0, 0] == 0x7E and codes[0, :3].tolist() == [7, 5, 9]


def test_atom_layout_round_trip():
    rng = np.random.default_rng(0)
    for kind, n in ((bq.MXFP8, 5), (bq.MXFP4, 9), (bq.NVFP4, 18)):
        sf = rng.integers(1, 255, (200, n)).astype(np.uint8)
        a = bq.atoms(sf, kind)
        back, pad = bq.from_atoms(a, 200, n, kind)
        assert np.array_equal(back, sf) and not pad.any()
        per = {bq.MXFP8: 4, bq.MXFP4: 8, bq.NVFP4: 16}[kind]
        row_atoms = -(-n // per) * per // 4
        for r, j in ((0, 0), (31, 4), (32, 1), (130, n - 1), (199, 3)):   # the documented byte
            off = ((r // 128) * row_atoms + j // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + j % 4
            assert a[off] == sf[r, j]


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    h, gamma, w = rng.standard_normal((5, 16)), rng.standard_normal(16), rng.standard_normal((5, 16))
    eps = 1e-3

    def loss(h, gamma):
        return (bq.rmsnorm(h, None, gamma, eps)[2] * w).sum()

    rstd = bq.rmsnorm(h, None, gamma, eps)[1]
    dh, dgamma = bq.rmsnorm_grad(w, h, gamma, rstd)
    d = 1e-5                                        # central differences: error O(d^2) + 1e-16 / d
    for i, j in ((0, 0), (2, 7), (4, 15)):
        e = np.zeros_like(h)
        e[i, j] = d
        assert abs((loss(h + e, gamma) - loss(h - e, gamma)) / (2 * d) - dh[i, j]) < 1e-8
    for j in (0, 9):
        e = np.zeros(16)
        e[j] = d
        assert abs((loss(h, gamma + e) - loss(h, gamma - e)) / (2 * d) - dgamma[j]) < 1e-8
