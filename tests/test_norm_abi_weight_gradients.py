"""rope_norm_qk_bwd without a GPU: weight gradients of tensors that have no rows are outputs like others."""
import pytest

import rotary_position_embedding_rope_gb300 as R
from test_norm_abi import A, INV, UNS, bwd, lib  # noqa: F401 (lib: a fixture)


@pytest.mark.parametrize("none", [dict(Hq=0, q=None, gq=None, dq=None), dict(Hq=0, Hk=0), dict(S=0), dict(B=0, Hq=0)])
@pytest.mark.parametrize("over,status", [
    (dict(dwq=13 * A + 2), UNS), (dict(dwk=13 * A), INV), (dict(ws=13 * A), INV), (dict(dwq=5 * A), INV), (dict(ws=None), INV),
    (dict(wsb=100), INV)])
def test_refusals_without_rows(lib, none, over, status):  # noqa: F811
    assert bwd(lib, **none, **over) == status


def test_nothing_wanted_without_heads(lib):  # noqa: F811
    none = dict(q=None, k=None, gq=None, gk=None, dq=None, dk=None, dwq=None, dwk=None, ws=None, wsb=0, cos=None, sin=None)
    assert bwd(lib, Hq=0, Hk=0, **none) == R.ROPE_OK
