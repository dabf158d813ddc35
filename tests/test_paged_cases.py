"""CPU tests of the attention tests' own means: the patterns of scores move the
reference of the softmax inside a share, and a rescale that is left out is off by
more than the error bound."""
import math

import pytest
import torch

import paged_cases as ref


@pytest.mark.parametrize("tiles,ctas", [([11] * 185, 148), ([1], 148), ([3, 0, 5, 1, 0], 4), ([938, 0, 1, 2, 2, 313], 148)])
def test_shares_are_the_whole_list(tiles, ctas):
    got = ref.shares(tiles, ctas)
    assert len(got) == min(ctas, sum(tiles))
    flat = [(p, t) for own in got for p, a, b in own for t in range(a, b)]
    assert flat == [(p, t) for p, n in enumerate(tiles) for t in range(n)]
    sizes = [sum(b - a for _, a, b in own) for own in got]
    assert max(sizes) - min(sizes) <= 1


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kind", ["rising", "falling", "saw", "spikes"])
def test_a_missing_rescale_exceeds_the_bound(kind, mx):
    n, H, C, page = 704, 6, 128, 32
    q, codes, sf, scale = ref.stepped(kind, n, H, C, mx, torch.Generator().manual_seed(3), "cpu")
    table = torch.arange(n // page, dtype=torch.int32)[None]
    fp4, sfp = codes.view(n // page, page, -1), sf.view(n // page, page, -1)
    want, lse, bound, lse_bound = ref.attend(q, fp4, sfp, table, [n], scale, mx=mx)
    rows = ref.dequant(codes, sf, mx)
    x = scale * (q[0].double() @ rows.T)
    assert 100 < float(x.max()) < 125

    def run(moved):
        out, got, count = ref.online(x / math.log(2.0), rows, moved)
        out_off = ((out - want[0]).abs() > bound[0]).any(-1)  # of each head
        return out_off, (got - lse[0]).abs() > lse_bound[0], count

    out_off, lse_off, count = run(lambda o, l, f: (o * f[:, None], l * f))
    assert not out_off.any() and not lse_off.any()
    if kind == "falling":
        assert int(count.max()) == 0
        return
    assert int(count.min()) >= (4 if kind == "rising" else 2)
    out_off, _, _ = run(lambda o, l, f: (o, l * f))
    assert out_off.all()  # the sums of rows not rescaled
    _, lse_off, _ = run(lambda o, l, f: (o * f[:, None], l))
    assert lse_off.all()  # the sum of weights not rescaled
    out_off, lse_off, _ = run(lambda o, l, f: (o, l))
    assert out_off.all() and lse_off.all()
