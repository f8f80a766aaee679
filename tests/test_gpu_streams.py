"""Calls on a stream other than the current one: what a call allocates comes
from the memory of its own stream (a block of the current one may still be in
use there), and calls of two streams do not disturb one another."""
import contextlib

import pytest
import torch

import serving_ref as S
from gpu_util import lib, require_gpu

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def allocations(streams):
    """Collects the stream of every block handed out inside."""
    torch.cuda.memory._record_memory_history(enabled="all", context=None)
    try:
        yield
        trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
        streams += [e["stream"] for e in trace if e["action"] == "alloc"]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)


def serving_inputs(seed=3):
    g = torch.Generator().manual_seed(seed)
    x = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    t = dict(q=x(700, 4, 64), k=x(700, 2, 64), v=x(700, 2, 64), d=x(2, 4, 64), kp=x(8, 2, 16, 64), vp=x(8, 2, 16, 64),
             cu=i(0, 450, 700), table=i([0, 1], [2, 3]), lens=i(19, 5), prefix=i(4, 5))
    t["cos"], t["sin"] = (y.cuda() for y in S.tables(1e4, 64, 512))
    return t


def packed(R, t, **more):
    return R.attention_packed(t["q"], t["k"], t["v"], t["cu"], t["cos"], t["sin"], causal=True, **more)


def decode(R, t, **more):
    return R.attention_shared_prefix(t["d"], t["kp"], t["vp"], t["table"], t["lens"], t["prefix"], 20, t["cos"], t["sin"],
                                     **more)


@pytest.mark.parametrize("call", [packed, decode])
@pytest.mark.parametrize("raw", [False, True])
def test_serving_blocks_come_from_the_calls_stream(call, raw):
    require_gpu()
    R = lib()
    t = serving_inputs()
    want = call(R, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    with allocations(got):
        a = call(R, t, stream=side.cuda_stream if raw else side)
    assert len(got) == 2 and set(got) == {side.cuda_stream}            # the output and the workspace
    got = []
    with torch.cuda.stream(side), allocations(got):
        b = call(R, t, stream=0 if raw else torch.cuda.default_stream())
    assert len(got) == 2 and set(got) == {0}
    got = []
    with allocations(got):
        c = call(R, t)
    assert len(got) == 2 and set(got) == {0}
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in (a, b, c)) and R.rope_check_errors() == R.ROPE_OK


@pytest.mark.parametrize("call", [packed, decode])
def test_serving_calls_of_two_streams_at_once(call):
    """A call on the current stream, then at once one of the same sizes on another, with nothing between them."""
    require_gpu()
    R = lib()
    a, b = serving_inputs(3), serving_inputs(4)
    want = call(R, a), call(R, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        busy = torch.randn(2048, 2048, device="cuda")
        for _ in range(4):
            busy = busy @ busy                                          # the current stream is behind the host
        x = call(R, a)
        y = call(R, b, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    assert R.rope_check_errors() == R.ROPE_OK


def dense_inputs(seed=3):
    g = torch.Generator().manual_seed(seed)
    x = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    t = dict(q=x(2, 4, 600, 128), k=x(2, 2, 600, 128), v=x(2, 2, 600, 128))
    t["mask"] = torch.ones(2, 600, dtype=torch.bool, device="cuda")
    t["mask"][1, 500:] = False
    t["cos"], t["sin"] = (y.cuda() for y in S.tables(1e4, 128, 600))
    return t


def dense(R, t, **more):
    return R.attention(t["q"], t["k"], t["v"], t["cos"], t["sin"], causal=True, **more),


def masked(R, t, **more):
    return R.attention(t["q"], t["k"], t["v"], t["cos"], t["sin"], attn_mask=t["mask"], **more),


def rotated(R, t, **more):
    return R.rotate_qk(t["q"], t["k"], t["cos"], t["sin"], **more)


def tables(R, t, **more):
    return R.build_tables(1e4, 64, 100, **more)


def tables_ex(R, t, **more):
    return R.build_tables_ex("pixel", 64, 100, **more)


@pytest.mark.parametrize("call", [dense, masked, rotated, tables, tables_ex])
@pytest.mark.parametrize("raw", [False, True])
def test_blocks_come_from_the_calls_stream(call, raw):
    require_gpu()
    R = lib()
    t = dense_inputs()
    want = call(R, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for current, other in ((torch.cuda.default_stream(), side), (side, torch.cuda.default_stream())):
        got = []
        with torch.cuda.stream(current), allocations(got):
            outs.append(call(R, t, stream=other.cuda_stream if raw else other))
        assert len(got) == 2 and set(got) == {other.cuda_stream}
    got = []
    with allocations(got):
        outs.append(call(R, t))
    assert len(got) == 2 and set(got) == {0}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want)) and R.rope_check_errors() == R.ROPE_OK


def test_host_staging_comes_from_the_copy_streams_memory():
    require_gpu()
    R = lib()
    from rotary_position_embedding_rope_gb300.host import HostAttention, HostRotator

    t = dense_inputs()
    want = rotated(R, t), dense(R, t)
    torch.cuda.synchronize()
    q, k, v = (t[n].cpu().pin_memory() for n in "qkv")
    qo, ko, o = (torch.empty_like(x).pin_memory() for x in (q, k, q))
    rot, att = HostRotator(chunks=2), HostAttention(chunks=2)
    for run, s_in in ((lambda: rot.apply_qk(q, k, t["cos"], t["sin"], qo, ko), rot.s_in),
                      (lambda: att.forward(q, k, v, o, t["cos"], t["sin"], causal=True), att.s_in)):
        got = []
        with allocations(got):
            run().synchronize()
        assert got and set(got) == {s_in.cuda_stream}
    assert torch.equal(qo, want[0][0].cpu()) and torch.equal(ko, want[0][1].cpu()) and torch.equal(o, want[1][0].cpu())


@pytest.mark.parametrize("call", [packed, decode, dense])
def test_a_captured_call_on_a_forked_stream(call):
    """A graph whose call runs on a second stream, forked from and joined with the captured one; replayed on new data, with
    eager calls of the same sizes between the replays."""
    require_gpu()
    R = lib()
    make = dense_inputs if call is dense else serving_inputs
    one = lambda o: o[0] if isinstance(o, tuple) else o
    t, new = make(3), make(4)
    want, want_new = one(call(R, t)), one(call(R, new))
    torch.cuda.synchronize()
    main, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        out = one(call(R, t, stream=side))
        main.wait_stream(side)
        twice = out * 2                                    # what follows on the captured stream
    for _ in range(2):
        graph.replay()
        other = one(call(R, new))
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(twice, want * 2) and torch.equal(other, want_new)
    for n in t:
        t[n].copy_(new[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want_new) and torch.equal(twice, want_new * 2)
    assert R.rope_check_errors() == R.ROPE_OK
