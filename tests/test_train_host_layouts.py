"""Which layouts the training pass's calls take, without a GPU: packed projections' parts interleave
in any order of their axes, and an output that shares an element with another tensor is refused.
Every call here is refused before device work, by what is checked behind the layouts."""
import itertools
import os
import random

import pytest

from causal_linear_attention_chunkwise_gb300 import _native, build

P = 0x10000000  # never dereferenced: validation fails first
BEHIND = "inv_freq, positions"  # refused for the frequencies' place: the layouts have passed


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        build.build()
    return _native.load()


def packed(order, sizes, part, first=0):
    """Address and (b,h,t) strides of part `part` of a packed tensor: `order` names its axes from
    the outermost on (p: the parts), `sizes` their allocated sizes."""
    stride, at = 1, {}
    for axis in reversed(order):
        at[axis] = stride
        stride *= sizes[axis]
    return first + part * at.get("p", 0), (at["b"], at["h"], at["t"])


def rotary(lib, q, k, qo, ko, B=2, H=4, Hk=None, L=8, d=64, elt=2, backward=False):
    """The message of a call whose frequencies lie in q_out."""
    def args(x):
        return (None, 0, 0, 0) if x is None else (P + x[0] * elt, *x[1])
    Hk = H if Hk is None else Hk
    status = (lib.la_rotary_bwd if backward else lib.la_rotary_fwd)(
        *args(q), H, *args(k), Hk if k else 0, 1 if elt == 2 else 0, B, L, d, d, 0,
        (P + qo[0] * elt) & ~3, 1.0, None, None, None, *args(qo), *args(ko), None)
    assert status == 1
    return lib.la_last_error().decode()


LAYOUTS = ["bpthd", "bphtd", "btphd", "bthpd", "tbphd", "pbthd", "bhptd", "tbhpd"]
DENSE = (1 << 24, (4 * 8 * 64, 8 * 64, 64))


def sizes(longer=0, **kw):
    return {"b": 2, "h": 4, "t": 8 + longer, "d": 64, "p": 3, **kw}


@pytest.mark.parametrize("order", LAYOUTS)
@pytest.mark.parametrize("longer", [0, 5])
def test_parts_of_a_packed_projection(lib, order, longer):
    q, k, v = (packed(order, sizes(longer), i) for i in range(3))
    # in place; into another packed tensor; from and to dense ones
    other = [packed(order, sizes(longer), i, 1 << 22) for i in range(3)]
    dense, dense2 = DENSE, (DENSE[0] * 2, DENSE[1])
    for at in ((q, k, q, k), (q, k, *other[:2]), (q, k, other[1], other[2]), (dense, dense2, q, k),
               (q, k, v, dense), (q, None, k, None)):
        assert BEHIND in rotary(lib, *at, backward=longer > 0), (order, at)


@pytest.mark.parametrize("order", LAYOUTS)
def test_parts_that_share_elements(lib, order):
    q, k, v = (packed(order, sizes(), i) for i in range(3))
    one = packed(order, sizes(), 0, 1)       # an element further on
    head = (q[0] + q[1][1], q[1])            # a head further on
    late = (q[0] + q[1][2], q[1])            # a token further on
    for at in ((q, k, one, v), (q, k, k, v), (q, k, head, v), (q, k, late, v), (q, k, v, v),
               (one, None, q, None)):
        assert "overlap" in rotary(lib, *at) and BEHIND not in rotary(lib, *at), (order, at)


def test_heads_of_their_own_numbers(lib):
    """Queries and keys of unlike head counts in one projection, full and cut to a prefix."""
    for Lmax in (8, 11):
        row = (6 + 2 * 2) * 64
        s = (Lmax * row, 64, row)
        q, k = (0, s), (6 * 64, s)
        assert BEHIND in rotary(lib, q, k, q, k, H=6, Hk=2)
        assert BEHIND in rotary(lib, q, (6 * 64, (s[0], 7, row)), q, (7 * 64, (s[0], 9, row)), H=6,
                                Hk=1)
        assert BEHIND not in rotary(lib, q, k, q, (5 * 64, s), H=6, Hk=2)
    one = (0, (640, 64, 3))  # one token: its stride means nothing
    assert BEHIND in rotary(lib, one, (384, (640, 64, 5)), one, (384, (640, 64, 5)), H=6, Hk=2, L=1)


def elements(x, n, d):
    b, h, t = x[1]
    return {x[0] + i * b + j * h + m * t + e for i in range(n[0]) for j in range(n[1])
            for m in range(n[2]) for e in range(d)}


def own(x, n, d):
    return len(elements(x, n, d)) == n[0] * n[1] * n[2] * d


def test_against_counting_elements(lib):
    """Small random layouts, each of the same strides for both or of unlike ones: what shares an
    element is refused; of the same strides what does not is taken."""
    rng = random.Random(1)
    taken = refused = 0
    for _ in range(4000):
        d = rng.choice([2, 4])
        n = tuple(rng.randint(1, 3) for _ in range(3))
        order = rng.sample(range(3), 3)
        strides, at = [0, 0, 0], d * rng.randint(1, 3)
        for i in order:
            strides[i] = at
            at = at * n[i] + rng.choice([0, 0, 2, 4])
        x = (64, tuple(strides))
        other = tuple(strides) if rng.random() < 0.8 else \
            tuple(s * rng.choice([1, 1, 2]) for s in strides)
        y = (64 + 2 * rng.randint(-20, 40), other)
        if not (own(x, n, d) and own(y, n, d)):
            continue
        shared = bool(elements(x, n, d) & elements(y, n, d))
        same = x[0] == y[0] and all(a == b for a, b, m in zip(x[1], y[1], n) if m > 1)
        got = BEHIND in rotary(lib, x, None, y, None, B=n[0], H=n[1], L=n[2], d=d)
        unlike = any(a != b for a, b, m in zip(x[1], y[1], n) if m > 1)
        if same or not shared and not unlike:
            assert got, (n, d, x, y)
            taken += 1
        elif shared:
            assert not got, (n, d, x, y)
            refused += 1
    assert taken > 300 and refused > 300


def gated(lib, x, dx, B=2, H=4, L=8, d=64, gate=1 << 22, dgate=1 << 23):
    """The message of a call that has no workspace for dweight."""
    row = H * d
    status = lib.la_gated_norm_bwd(
        P + (3 << 23), row, P + x[0] * 2, *x[1], P + gate * 2, row, 1, B, H, L, d, 0, 1, 0,
        P + (5 << 23), None, 1, 1e-5, P + dx[0] * 2, *dx[1], P + dgate * 2, row, P + (6 << 23), None,
        None, 0, None)
    assert status == 1
    return lib.la_last_error().decode()


@pytest.mark.parametrize("order", LAYOUTS)
@pytest.mark.parametrize("longer", [0, 5])
def test_gated_norm_between_parts(lib, order, longer):
    q, k, v = (packed(order, sizes(longer), i) for i in range(3))
    for x, dx in itertools.product((q, k, v), repeat=2):
        assert "workspace" in gated(lib, x, dx), (order, x, dx)
    assert "overlap" in gated(lib, q, (q[0] + 8, q[1]))
    assert "overlap" in gated(lib, q, (q[0] + q[1][1], q[1]))


def test_gated_norm_forward_between_parts(lib):
    """y in the rows of a packed tensor, x the other part of it at the same strides."""
    B, H, L, d = 2, 4, 8, 64

    def call(x, xs, y, ys, weight):
        status = lib.la_gated_norm_fwd(P + x * 2, *xs, None, 0, 1, B, H, L, d, 0, 0, 0, weight, None,
                                       1, 1e-5, P + y * 2, ys, None)
        assert status == 1
        return lib.la_last_error().decode()

    for Lmax in (L, L + 3):
        s = packed("btphd", {"b": B, "h": H, "t": Lmax, "d": d, "p": 3}, 0)[1]
        row = s[2]
        weight = P + (H * d) * 2  # in y: seen behind the layouts
        assert ("weight or bias" in call(0, s, H * d, row, weight)) == (Lmax == L)
        assert "y overlaps an input" in call(0, s, 0, row, None)
        assert "y overlaps an input" in call(H * d, s, H * d + 8, row, None)
