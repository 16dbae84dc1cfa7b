"""That the whole-number data of group4_exact.py shows a fault of one lane or one group in the longest rows (CPU; the fault is put into
the sums that the tests compare with)."""
import pytest

torch = pytest.importorskip("torch")
from tests import group4_exact as ex, group4_ref as g4  # noqa: E402


@pytest.mark.parametrize("K", [14001, 26656, 30031, 32766])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_a_lane_or_a_scale_shows(K, group):
    x, code, e = ex.layer(1, 9, K, group, K, "cpu")
    w = ex.weights(code, e, group)
    y = ex.product(x, w)[0]
    part = torch.nn.functional.pad(x[0].double() * w, (0, -K % 32)).view(9, -1, 32).sum(2)          # what each 32 columns add
    assert bool((part != 0).any(0).all()) and float((part != 0).double().mean()) > 0.95
    # each group under the scale of the one after it, or before it
    of_group = torch.nn.functional.pad(x[0].double() * code.double(), (0, -K % group)).view(9, -1, group).sum(2)
    s = torch.exp2(e.double())
    for by in (1, -1):
        off = of_group * (torch.roll(s, by, 1) - s)
        inner = off[:, 1:] if by == 1 else off[:, :-1]
        assert bool((inner != 0).any(0).all())
    assert torch.equal((of_group * s).sum(1), y)


def test_packing_is_the_stored_form():
    _, code, _ = ex.layer(1, 5, 101, 32, 1, "cpu")
    assert (ex.pack(code).numpy() == g4.pack(code.numpy())).all()
