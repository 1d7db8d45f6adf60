"""Pins of the paged cache's float64 oracle on cases that can be checked by hand."""
import numpy as np
import pytest
import torch

from oracle import paged


def test_round_e4m3_against_torch():
    x = torch.cat([torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 40,
                   torch.linspace(-0.05, 0.05, 4001), torch.tensor([0.0, 448.0, -448.0, 2 ** -9, 2 ** -10, 3 * 2 ** -10])])
    x = x.clamp(-448, 448)
    assert np.array_equal(paged.round_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    assert paged.round_e4m3(np.array([1e9, -np.inf, np.nan])).tolist() == [448.0, -448.0, 0.0]


@pytest.mark.parametrize("absmax,exp", [(448.0, 0), (448.0001, 1), (224.0, -1), (224.1, 0), (1.75, -8), (1.7500001, -7),
                                        (1e-45, -100), (0.0, -100), (3.4028234e38, 119)])
def test_page_scale(absmax, exp):
    assert paged.page_scale(absmax) == 2.0 ** exp


def test_growth_rounds_the_page_again():
    p = paged.Pages(1, 1, 1)
    p.append(np.array([[[1.0625]]]), np.array([[[1.0]]]), [0])      # 1.0625 ties to 1.0 (even) in E4M3
    assert p.gather([0])[0][0, 0, 0] == 1.0
    first = p.scales[0][0, 0]
    p.append(np.array([[[900.0]]]), np.array([[[1.0]]]), [1])
    assert p.scales[0][0, 0] == 4.0 and p.scales[0][0, 0] > first
    assert p.gather([0, 1])[0][:, 0, 0].tolist() == [1.0, 896.0]
    p.append(np.array([[[2.0]]]), np.array([[[1.0]]]), [0])         # the page starts over
    assert p.scales[0][0, 0] == 2.0 ** -7 and p.gather([0, 1])[0][:, 0, 0].tolist() == [2.0, 0.0]


def test_plan_denies_in_order():
    free = np.array([5, 6, 7, 8])
    table = np.full((4, 3), -1)
    p = paged.plan([0, 0, 3, 47], [17, 33, 2, 2], table, free, 4, 60)
    assert p["denied"] == 2 and p["count"] == 2                     # 2 pages, then 3 of 2, then none, then past the table
    assert p["table"][0].tolist() == [8, 7, -1] and p["kv_len"].tolist() == [17, 0, 5, 47]
    assert p["row_start"].tolist() == [0, 17, 50, 52, 54]
    assert p["slots"][:18].tolist() == [128 + i for i in range(16)] + [112, -1]


def test_attend_by_hand():
    p = paged.Pages(2, 1, 1)
    p.append(np.array([[[0.0]], [[0.0]], [[8.0]]]), np.array([[[1.0]], [[3.0]], [[100.0]]]), [16, 17, 18])
    table = np.array([[1]])
    a = p.attend(np.ones((1, 2, 1)), table, [2])
    assert np.allclose(a["out"], 2.0) and np.allclose(a["mass"], 1.0)
    w = np.exp(8.0) / (np.exp(8.0) + 2)
    a = p.attend(np.ones((2, 1, 1)), table, [3], [0, 2])
    assert np.allclose(a["out"][:, 0, 0], [2.0, 96 * w + 4 * (1 - w) / 2])     # 100 rounds to 96 (even) at scale 2^-2
    assert np.allclose(p.attend(np.ones((1, 1, 1)), table, [3], window=1)["out"], 96.0)
    assert np.allclose(p.attend(np.ones((1, 1, 1)), np.array([[-1]]), [3])["out"], 0.0)
