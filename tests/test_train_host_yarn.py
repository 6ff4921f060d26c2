"""YaRN's frequencies, pinned: a blend linear in the pair's index between two whole pairs, as
checkpoints of that scaling are trained with, and not one linear in the number of turns."""
import math
import os

import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import _native, api, build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(_native.LIB_PATH):
        build.build()


def yarn(dim, base, factor, length, low, high):
    """The definition, with the two pairs given."""
    out = []
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        m = min(max((i - low) / (high - low), 0), 1)
        out.append(f * (1 - m) + f / factor * m)
    return torch.tensor(out, dtype=torch.float64).float()


@pytest.mark.parametrize("dim,base,factor,length,fast,slow,low,high", [
    # 128 ln(4096 / 64 pi) / (2 ln 10^4) = 20.94, 128 ln(4096 / 2 pi) / (2 ln 10^4) = 45.03
    (128, 10000.0, 16.0, 4096, 32, 1, 20, 46),
    # 64 ln(8192 / 64 pi) / (2 ln 5 10^5) = 9.04, 64 ln(8192 / 2 pi) / (2 ln 5 10^5) = 17.49
    (64, 500000.0, 8.0, 8192, 32, 1, 9, 18),
    # 32 ln(128 / 64 pi) is below 0; 32 ln(128 / 2 pi) / (2 ln 100) = 10.47
    (32, 100.0, 4.0, 128, 32, 1, 0, 11),
    # 8 ln(10^9 / 4 pi) / (2 ln 10) = 31.6, so the first pair lies behind the last
    (8, 10.0, 2.0, 10 ** 9, 2, 1, 31, 31.001),
    # 16 ln(512 / 2 pi) / (2 ln 3) = 32.04: cut to 15; 16 ln(512 / 64 pi) / (2 ln 3) = 6.80
    (16, 3.0, 4.0, 512, 32, 1, 6, 15),
    # no pair makes a turn: all but the first are scaled
    (16, 10000.0, 4.0, 5, 32, 1, 0, 0.001),
    (64, 10000.0, 4.0, 4096, 32, 0, 10, 63),   # slow = 0: up to the width
])
def test_blend(dim, base, factor, length, fast, slow, low, high):
    got, scale = api.la_rotary_frequencies(dim, base, "yarn", factor, length, fast, slow)
    assert math.isclose(scale, 1 + 0.1 * math.log(factor), rel_tol=2.0 ** -23)
    want = yarn(dim, base, factor, length, low, high)
    assert torch.allclose(got, want, rtol=2.0 ** -22, atol=0), (got, want)


def test_values():
    """A few worked by hand: 128 values, base 10^4, factor 16, trained on 4096 tokens; pairs 20..46."""
    f, _ = api.la_rotary_frequencies(128, 10000.0, "yarn", 16.0, 4096.0)
    plain = lambda i: 10.0 ** (-i / 16)  # noqa: E731
    for pair, share in ((0, 0), (20, 0), (21, 1 / 26), (33, 0.5), (38, 18 / 26), (45, 25 / 26),
                        (46, 1), (63, 1)):
        assert math.isclose(f[pair], plain(pair) * (1 - share * 15 / 16), rel_tol=1e-6), pair


def test_base_of_one_has_no_pairs_to_blend():
    for base in (1.0, 0.5):
        with pytest.raises(api.LAError):
            api.la_rotary_frequencies(16, base, "yarn", 4.0, 4096.0)
        api.la_rotary_frequencies(16, base)
