"""The serving calls where offsets pass 32 bits: bit for bit what the same rows
give in small tensors (the path a call takes does not depend on where they lie)."""
import pytest
import torch

import serving_ref as S
from gpu_util import lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    require_gpu()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    yield
    torch.cuda.empty_cache()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B", [2, 20])
def test_pages_at_the_end_of_a_large_pool(B):
    """Append, then decode (with the prefix beside the suffixes, and in a kernel of its own): 45000 pages, 2.9e9 elements."""
    R = lib()
    Hq, Hk, page, D, n_pages, prefix = 16, 8, 64, 128, 45000, 500
    g = torch.Generator().manual_seed(31)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    cos, sin = (x.cuda() for x in S.tables(1e4, D, 1024))
    used = 8 + 3 * B
    place = torch.randperm(used, generator=g)
    where = (n_pages - used + place).int()                 # of the small pool's pages
    old, new = [(i * 17) % 100 for i in range(B)], [1 + (i * 5) % 9 for i in range(B)]
    cu = ints(0, *[sum(new[:i + 1]) for i in range(B)])
    k, v, q = rnd(sum(new), Hk, D), rnd(sum(new), Hk, D), rnd(B, Hq, D)
    small = [rnd(used, Hk, page, D) for _ in range(2)]
    large = [torch.zeros(n_pages, Hk, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert large[0].numel() > 1 << 31
    for a, b in zip(small, large):
        b[where.long().cuda()] = a
    outs = []
    for pools, ids in ((small, torch.arange(used, dtype=torch.int32)), (large, where)):
        ids = ids.cuda()
        table, shared = ids[8:].view(B, 3).contiguous(), ids[:8].contiguous()
        R.cache_append(k, v, *pools, table, cu, ints(*old), cos, sin, pos_offset=prefix)
        outs.append(R.attention_shared_prefix(q, *pools, table, ints(*[a + b for a, b in zip(old, new)]), shared,
                                              prefix, cos, sin))
    assert R.rope_check_errors() == R.ROPE_OK
    assert torch.equal(outs[0], outs[1]) and outs[0].isfinite().all()
    for a, b in zip(small, large):
        assert torch.equal(a, b[where.long().cuda()])
        assert torch.count_nonzero(b[:n_pages - used]) == 0


def test_sequences_at_the_end_of_long_packed_tensors():
    R = lib()
    lens, at, Hq, D = [300, 1, 77, 130], 600_000, 32, 128
    total = at + sum(lens) + 5
    assert at * Hq * D > 1 << 31
    g = torch.Generator().manual_seed(37)
    small = [torch.randn(sum(lens), Hq, D, generator=g).bfloat16().cuda() for _ in range(3)]
    large = [torch.zeros(total, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    for a, b in zip(small, large):
        b[at:at + sum(lens)] = a
    cos, sin = (x.cuda() for x in S.tables(1e4, D, 512))
    cu = ints(0, *[sum(lens[:i + 1]) for i in range(len(lens))])
    out = torch.full((total, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    for causal in (True, False):
        want = R.attention_packed(*small, cu, cos, sin, causal=causal)
        R.attention_packed(*large, cu + at, cos, sin, causal=causal, out=out)
        assert R.rope_check_errors() == R.ROPE_OK
        assert torch.equal(out[at:at + sum(lens)], want)
        assert (out[:at] == 7).all() and (out[at + sum(lens):] == 7).all()
