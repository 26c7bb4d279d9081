"""CPU tests of the requests whose rows' references move: that they do, where they are meant to, with a share of the
row's weight on both sides; and that a result that is not scaled down then leaves the bound of the GPU's tests."""
import numpy as np
import pytest

from oracle import chunk

from tree_scores import UNIT, both_halves, kinds, leveled, moves_once, run, scores


def walk(c, unit, mistake=None):
    """Of request 0's rows: the moves behind the first unit, and whether any row is outside the bound."""
    rows = np.arange(min(c.new[0], 6))
    x, V = scores(c, 0, rows)
    exact = c.oracle(0, rows)[1]
    lim = chunk.attention_bound(*exact)
    g = c.hq // c.hkv
    single = c.new[0] * g <= 128
    n_units = -(-x.shape[-1] // UNIT)
    found, wrong = [], 0
    for i in range(len(rows)):
        for h in range(c.hq):
            parts = [run(x[i, h], V[:, h // g], units, mistake)
                     for units in ([range(0, n_units, 2), range(1, n_units, 2)] if single else [range(n_units)])]
            ref = max(p[0] for p in parts)
            total = sum(p[1] * np.exp2(p[0] - ref) for p in parts)
            out = sum(p[2] * np.exp2(p[0] - ref) for p in parts) / total
            wrong += bool((np.abs(out - exact[0][i, h]) > lim[i, h]).any())
            found += [(kinds(c)[i, h], *m) for p in parts for m in p[3]]
    return found, wrong


@pytest.mark.parametrize("nodes", [20, 50])                # one row tile, two
@pytest.mark.parametrize("unit,half", [(2, 0), (2, 1), (3, 0), (3, 1), (5, 0), (5, 1)])
def test_the_reference_moves_where_it_is_meant_to(nodes, unit, half):
    c = leveled([moves_once(unit, half)], [nodes])
    found, wrong = walk(c, unit)
    assert wrong == 0
    here = [m for m in found if m[1:3] == (unit, half)]
    assert {m[0] for m in here} == {0, 1, 2} and all(2.0 ** -40 < m[3] < 1.0 for m in here)
    assert walk(c, unit, "kept")[1] > 0


def test_the_second_unit_of_two_row_tiles_moves():
    for half in (0, 1):
        c = leveled([moves_once(1, half)], [50])
        found, wrong = walk(c, 1)
        assert wrong == 0 and {m[0] for m in found if m[1:3] == (1, half)} == {0, 1, 2}
        assert walk(c, 1, "kept")[1] > 0


@pytest.mark.parametrize("nodes", [20, 50])
@pytest.mark.parametrize("unit", [2, 3, 5])
def test_both_halves_of_a_unit_move(nodes, unit):
    c = leveled([both_halves(unit)], [nodes])
    found, wrong = walk(c, unit)
    assert wrong == 0
    assert {m[:2] + (m[2],) for m in found} >= {(0, unit, 0), (1, unit, 1), (2, unit, 0)}
    for mistake in ("kept", "half"):
        assert walk(c, unit, mistake)[1] > 0, mistake


@pytest.mark.parametrize("nodes", [20, 50])
def test_a_unit_moves_twice_and_two_units_move(nodes):
    c = leveled([moves_once(2, 0, (2, 1))], [nodes])
    found, wrong = walk(c, 2)
    assert wrong == 0 and {m[1:3] for m in found} >= {(2, 0), (2, 1)}
    assert walk(c, 2, "first")[1] > 0
    c = leveled([moves_once(2, 0, (4, 1))], [nodes])
    found, wrong = walk(c, 2)
    assert wrong == 0 and {m[1:3] for m in found} >= {(2, 0), (4, 1)}
    assert walk(c, 2, "kept")[1] > 0
