"""attention_paged: a query that sees no key gets zeros, whatever the keys and values of its sequence hold, in each kind of
work (few rows, twice as many, tiles, several pieces a tile)."""
import pytest

import serving_ref as S
from gpu_util import lib, require_gpu
from test_gpu_attention_paged import case, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q,k,Hq,Hk,D,page", [
    ([3], [2], 2, 2, 128, 16), ([2, 3], [1, 2], 4, 4, 64, 16), ([12], [4], 1, 1, 128, 64), ([8, 1], [3, 5], 2, 1, 64, 32),
    ([40], [20], 4, 2, 128, 64), ([300], [100], 4, 4, 64, 16), ([300, 1], [170, 3], 8, 2, 128, 128), ([700], [650], 1, 1, 128, 64)])
@pytest.mark.parametrize("of", ["keys", "values"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_without_keys(q, k, Hq, Hk, D, page, of, bad, dtype):
    require_gpu()
    R = lib()
    x = make(case(q, k, Hq, Hk, D, D, page, dtype))
    for row in x[3]:
        x[1 if of == "keys" else 2][int(row[0]), :, 0] = bad       # the first key's
    got = run(R, *x, *S.tables(1e4, D, 1024))
    for start, n, m in zip(x[4].tolist(), q, k):
        assert not got[start:start + max(n - m, 0)].any()
