"""How a decode call is dealt out: the suffixes behind the prefix on the same CTAs, and what the merge goes by, which
is in the workspace whatever becomes of the CTAs that do the work."""
import pytest
import torch

import serving_ref as S
from gpu_util import lib, require_gpu
from test_gpu_attention_decode import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D, page, layout, dtype", [(128, 64, "split_half", "bf16"), (64, 16, "interleaved", "f16")])
def test_suffixes_behind_the_prefix(D, page, layout, dtype):
    """76 row tiles of 16 sequences (16 heads over one): with a cluster fewer than one each the prefix would take two
    rounds, so every CTA has prefix work, and the suffixes follow on all of them."""
    require_gpu()
    R = lib()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms < 152:
        pytest.skip("the deal is that of 152 SMs")
    keys = 16 if D == 128 else 32                          # of a chunk
    B, prefix = 76 * 16, 1500
    c = dict(lens=[(i * 5) % 61 * keys // 16 for i in range(B)], prefix=prefix, Hq=16, Hk=1, D=D, rd=D, page=page, dtype=dtype,
             layout=layout)
    q, kp, vp, table, lens, ptable = make(c)
    cos, sin = S.tables(1e4, D, prefix + max(c["lens"]) + 1)
    ws = torch.full((R.rope_attention_decode_workspace(B, 16, 1, D, page, table.shape[1], prefix),), 255, dtype=torch.uint8,
                    device="cuda")
    got = R.attention_shared_prefix(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), ptable.cuda(), prefix, cos.cuda(),
                                    sin.cuda(), layout=layout, workspace=ws)
    assert R.rope_check_errors() == R.ROPE_OK
    # the deal: chunks of a warp, (head, key tile)s of a group of clusters; chunks of the sequences before each
    chunks = [-(-n // keys) for n in c["lens"]]
    per = -(-sum(chunks) // (152 * 8))
    assert per >= 3 and int(ws[:8].view(torch.int64)) == per          # (on fewer SMs it would be more)
    assert int(ws[8:12].view(torch.int32)) == -(-prefix // 128)
    starts = torch.tensor([0] + chunks).cumsum(0)
    assert torch.equal(ws[128:128 + 4 * (B + 1)].view(torch.int32).cpu().long(), starts)
    ref = S.shared_prefix(q, kp, vp, table, lens, ptable, prefix, cos, sin, layout=layout)
    check(got.cpu(), ref, c, "decode suffixes behind the prefix D%d" % D)
