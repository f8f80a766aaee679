"""The serving calls beside autograd: they carry no graph, and what they write in place counts as written."""
import pytest
import torch

from gpu_util import lib, require_gpu
from test_gpu_streams import decode, packed, serving_inputs

pytestmark = pytest.mark.gpu


def append(R, t, n=7):
    cu = torch.tensor([0, 5, n], dtype=torch.int32, device="cuda")
    old = torch.tensor([14, 3], dtype=torch.int32, device="cuda")
    R.cache_append(t["k"][:n], t["v"][:n], t["kp"], t["vp"], t["table"], cu, old, t["cos"], t["sin"])


def test_outputs_carry_no_graph():
    require_gpu()
    R = lib()
    t = serving_inputs()
    want = packed(R, t), decode(R, t)
    for n in ("q", "k", "v", "d"):
        t[n].requires_grad_()
    got = packed(R, t), decode(R, t)
    assert not any(x.requires_grad for x in got) and all(torch.equal(a, b) for a, b in zip(got, want))
    append(R, t)
    assert not t["kp"].requires_grad and not t["vp"].requires_grad
    assert R.rope_check_errors() == R.ROPE_OK


def test_what_is_written_counts_as_written():
    require_gpu()
    R = lib()
    t = serving_inputs()
    x = torch.ones_like(t["kp"]).requires_grad_()
    y = (x * t["kp"]).sum()                                # saves the pool
    before = [t[n]._version for n in ("kp", "vp")]
    append(R, t)
    assert [t[n]._version for n in ("kp", "vp")] == [v + 1 for v in before]
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    for call, like in ((packed, "q"), (decode, "d")):
        out = torch.empty_like(t[like])
        v = out._version
        assert call(R, t, out=out) is out and out._version == v + 1
    # a refused call writes nothing
    before = t["kp"]._version
    with pytest.raises(R.RopeError):
        R.cache_append(t["k"][:7], t["v"][:7], t["kp"], t["kp"], t["table"], t["cu"], t["lens"], t["cos"], t["sin"])
    assert t["kp"]._version == before


def test_inference_tensors():
    require_gpu()
    R = lib()
    t = serving_inputs()
    with torch.inference_mode():
        kp, vp = t["kp"].clone(), t["vp"].clone()
    append(R, t)
    append(R, dict(t, kp=kp, vp=vp))                       # outside the mode they were made in
    with torch.inference_mode():
        append(R, dict(t, kp=kp, vp=vp))
        out = torch.empty_like(t["q"])
        assert torch.equal(packed(R, t, out=out), packed(R, t))
    assert torch.equal(kp, t["kp"]) and torch.equal(vp, t["vp"])
    assert R.rope_check_errors() == R.ROPE_OK
