"""The latent-cache oracle against hand-worked values and its own definition."""
import numpy as np
import pytest
import torch

import oracle


def _row(entries):
    r = np.zeros(576)
    r[:len(entries)] = entries
    return r


def test_elements():
    e2m1 = oracle.latent_elements("mx4")
    assert e2m1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    e4m3 = oracle.latent_elements("mx8")
    assert len(e4m3) == 127 and e4m3[1] == 2.0 ** -9 and e4m3[8] == 2.0 ** -6 and e4m3[-1] == 448
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3, codes)


@pytest.mark.parametrize("form,entries,byte,values", [
    # 6 fits at e = 0; 0.25 is a tie to 0, 0.75 a tie to 1, 2.5 to 2, 5 to 4
    ("mx4", [6, 0.25, 0.75, 2.5, 5, -3.5], 127, [6, 0, 1, 2, 4, -4]),
    # 6.25 does not: e = 1, quanta of 1 below 4 and of 4 between 8 and 12
    ("mx4", [6.25, 1, 0.5, -0.5, 7], 128, [6, 1, 0, 0, 8]),
    ("mx8", [448, 1 / 1024, 3 / 1024, 17, 19], 127, [448, 0, 4 / 1024, 16, 20]),
    ("mx8", [450, 17], 128, [448, 16]),
    ("mx8", [0.0], 10, [0]),                               # an empty group: the smallest scale
    ("mx4", [2.0 ** -125], 10, [0]),
])
def test_hand_worked_groups(form, entries, byte, values):
    _, scales, _ = oracle.latent_quantise(_row(entries), form)
    assert scales[0] == byte and (scales[1:] == 10).all()
    assert oracle.latent_values(_row(entries), form)[:len(values)].tolist() == values


@pytest.mark.parametrize("form", ["mx8", "mx4"])
def test_invariants(form):
    rng = np.random.default_rng(3)
    rows = torch.from_numpy(rng.standard_normal((40, 576)) * 2.0 ** rng.integers(-30, 30, (40, 1))).bfloat16().double().numpy()
    v = oracle.latent_values(rows, form)
    assert np.array_equal(oracle.latent_values(v, form), v)                    # quantising again changes nothing
    assert np.array_equal(oracle.latent_values(-rows, form), -v)
    assert np.array_equal(oracle.latent_values(rows * 8, form), v * 8)         # powers of two pass through
    assert np.array_equal(torch.from_numpy(v).bfloat16().double().numpy(), v)  # each value is a bf16 number
    assert np.array_equal(v[:, 512:], rows[:, 512:])
    # half a step of the element: 2^-4 (2^-2) of the entry, or half the smallest
    # step of a group whose largest entry uses at least the upper half of the range
    amax = np.abs(rows[:, :512]).reshape(40, 16, 32).max(-1).repeat(32, -1)
    step = (2.0 ** -4, 2.0 ** -10 / 224) if form == "mx8" else (2.0 ** -2, 0.25 / 3)
    assert (np.abs(v - rows)[:, :512] <= np.maximum(step[0] * np.abs(rows[:, :512]), step[1] * amax)).all()


def test_non_finite_and_huge():
    big = float(torch.finfo(torch.bfloat16).max)
    for form, top in (("mx8", 448 * 2.0 ** 119), ("mx4", 6 * 2.0 ** 125)):
        v = oracle.latent_values(_row([big, -big, 1.0]), form)
        assert v[0] == top and v[1] == -top and v[2] == 0
        for bad in (np.inf, -np.inf, np.nan):
            v = oracle.latent_values(_row([1.0, bad]), form)
            assert np.isnan(v[:32]).all() and (v[32:] == 0).all()


def test_bytes():
    row = _row([6, -0.5, 1.5])
    row[512] = -2.0
    b = oracle.latent_bytes(row, "mx4")
    assert b.shape == (400,) and b[0] == 0x97 and b[1] == 0x03 and b[256] == 127 and b[257] == 10
    assert b[272:274].tolist() == [0x00, 0xC0]      # bf16(-2) = 0xC000
    b = oracle.latent_bytes(row, "mx8")
    # amax 6 = 1.5 * 2^2: e = -6, entries 384, -32, 96
    assert b.shape == (656,) and b[512] == 121 and b[0] == 0x7C and b[1] == 0xE0 and b[2] == 0x6C
