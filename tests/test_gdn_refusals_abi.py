"""Host-side refusals of outputs whose rows or heads lie over one another, and of an infinite eps (no GPU needed)."""
import math

import pytest

from test_gdn_abi import fak, ref, structs  # noqa: F401


@pytest.mark.parametrize("stride", [0, 64, 120, -64])
@pytest.mark.parametrize("field", ["out_row", "out_head"])
def test_attn_outputs_over_one_another(fak, field, stride):  # noqa: F811
    b, r, a, n = structs()
    setattr(a, field, stride)
    assert fak.lib.fak_gdn_attn(ref(b), ref(a), None) == 1
    a.rows = a.nk = a.nv = 1  # never taken
    b.n_seqs = 0
    assert fak.lib.fak_gdn_attn(ref(b), ref(a), None) == 0


@pytest.mark.parametrize("stride", [0, 1, 5119, -5000])
def test_norm_rows_over_one_another(fak, stride):  # noqa: F811
    for field in ("h_row", "n_row"):
        n = structs()[3]
        setattr(n, field, stride)
        assert fak.lib.fak_residual_norm(ref(n), None) == 1
        n.rows = 0
        assert fak.lib.fak_residual_norm(ref(n), None) == 0
    n = structs()[3]
    n.h_row, n.y, n.n = stride, None, None  # h is read alone: nothing to do
    assert fak.lib.fak_residual_norm(ref(n), None) == 0


def test_an_infinite_eps(fak):  # noqa: F811
    b, r, a, n = structs()
    r.eps = a.eps = n.eps = math.inf
    assert fak.lib.fak_gdn_conv(ref(b), ref(r), None) == 1 and fak.lib.fak_gdn_attn(ref(b), ref(a), None) == 1
    assert fak.lib.fak_residual_norm(ref(n), None) == 1
