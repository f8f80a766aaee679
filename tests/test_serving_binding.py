"""What the binding of the serving calls refuses before any of them reaches the
library, and that calls of two threads do not disturb one another."""
import threading

import pytest
import torch

import rotary_position_embedding_rope_gb300 as R
import serving_ref as S
from gpu_util import require_gpu

X = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
POOL = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
I = torch.zeros(5, dtype=torch.int32)
TABLE = torch.zeros(4, 1, dtype=torch.int32)
T = torch.zeros(8, 32)


@pytest.mark.parametrize("call", [
    lambda **o: R.cache_append(X, X, POOL, POOL, TABLE, I, I[:4], T, T, **o),
    lambda **o: R.attention_packed(X, X, X, I, T, T, **o),
    lambda **o: R.attention_shared_prefix(X, POOL, POOL, TABLE, I[:4], None, 0, T, T, **o),
])
def test_host_tensors_and_layouts(call):
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(KeyError):
        call(layout="pairs")


@pytest.mark.parametrize("bad", [None, 3, "q", [1.0]])
def test_what_is_no_tensor(bad):
    with pytest.raises(TypeError, match="expected a tensor"):
        R.cache_append(bad, X, POOL, POOL, TABLE, I, I[:4], T, T)
    with pytest.raises(TypeError, match="expected a tensor"):
        R.attention_packed(bad, X, X, I, T, T)
    with pytest.raises(TypeError, match="expected a tensor"):
        R.attention_shared_prefix(bad, POOL, POOL, TABLE, I[:4], None, 0, T, T)


def _calls(seed):
    """The three calls on tensors of their own; what each returns or writes."""
    g = torch.Generator().manual_seed(seed)
    x = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    k, v, kp, vp = x(7, 2, 64), x(7, 2, 64), x(6, 2, 16, 64), x(6, 2, 16, 64)
    q, d = x(7, 4, 64), x(2, 4, 64)
    table, cu, old, lens, prefix = i([0, 1], [2, 3]), i(0, 5, 7), i(14, 3), i(19, 5), i(4, 5)
    cos, sin = (t.cuda() for t in S.tables(1e4, 64, 64))
    torch.cuda.synchronize()

    def step(stream):
        pools = kp.clone(), vp.clone()
        R.cache_append(k, v, *pools, table, cu, old, cos, sin, pos_offset=20, stream=stream)
        a = R.attention_packed(q, k, v, cu, cos, sin, stream=stream)
        b = R.attention_shared_prefix(d, *pools, table, lens, prefix, 20, cos, sin, stream=stream)
        return (*pools, a, b)

    return step


@pytest.mark.gpu
def test_calls_of_two_threads():
    require_gpu()
    steps = [_calls(11), _calls(12)]
    want = [s(None) for s in steps]
    torch.cuda.synchronize()
    wrong, met = [], threading.Barrier(2)

    def work(n):
        try:
            stream = torch.cuda.Stream()
            met.wait(60)
            with torch.cuda.stream(stream):
                for _ in range(100):
                    got = steps[n](stream)
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                        wrong.append(n)
        except BaseException as e:
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [] and R.rope_check_errors() == R.ROPE_OK


@pytest.mark.gpu
def test_refusals_name_what_is_wrong():
    require_gpu()
    x, pool, i, table, t = (a.cuda() for a in (X, POOL, I, TABLE, T))
    packed = dict(q=x, k=x, v=x, cu_seqlens_q=i, cos=t, sin=t)
    for over, err, name in [
            (dict(k=None), TypeError, "k: expected a tensor"), (dict(cos=t.double(), sin=t), ValueError, "cos"),
            (dict(cos=t[:, ::2], sin=t[:, ::2]), ValueError, "cos must be contiguous"),
            (dict(sin=t[:7]), ValueError, "same shape"), (dict(cu_seqlens_q=I), ValueError, "cu_seqlens_q must be on cuda"),
            (dict(cu_seqlens_q=i[:0]), ValueError, "n_seqs"), (dict(v=x[:3]), ValueError, "same tokens"),
            (dict(out=torch.zeros_like(x)[:3]), ValueError, "out must be"), (dict(scale="1"), TypeError, None),
            (dict(workspace=3), TypeError, "workspace"), (dict(workspace=I), ValueError, "workspace"),
            (dict(stream=2.5), AttributeError, None), (dict(scale=float("nan")), R.RopeError, None)]:
        with pytest.raises(err, match=name):
            R.attention_packed(**dict(packed, **over))
    decode = dict(q=x, k_pages=pool, v_pages=pool, block_table=table, seq_lens=i[:4], prefix_table=None, prefix_len=0,
                  cos=t, sin=t)
    for over, err, name in [
            (dict(v_pages=pool[:1]), ValueError, "one shape"), (dict(k_pages=pool.half()), ValueError, "k_pages"),
            (dict(q=x[:, :, :32].contiguous()), ValueError, "features"), (dict(block_table=table[:3]), ValueError, "block_table"),
            (dict(block_table=table.long()), ValueError, "block_table"), (dict(prefix_len=1), ValueError, "prefix_table"),
            (dict(prefix_len=1.5, prefix_table=i), TypeError, None), (dict(prefix_len=2 ** 70, prefix_table=i), OverflowError, None),
            (dict(prefix_table=i.float()), ValueError, "prefix_table")]:
        with pytest.raises(err, match=name):
            R.attention_shared_prefix(**dict(decode, **over))
    append = dict(k=x, v=x, k_pages=pool, v_pages=torch.zeros_like(pool), block_table=table, cu_seqlens=i,
                  cache_lens=i[:4], cos=t, sin=t)
    for over, err, name in [
            (dict(k=x.float()), TypeError, "bf16 or fp16"), (dict(v=x[:, :1]), ValueError, "v must be"),
            (dict(cu_seqlens=i[:4]), ValueError, "cu_seqlens"), (dict(cache_lens=i), ValueError, "cache_lens"),
            (dict(pos=i), ValueError, "pos must be"), (dict(block_table=i), ValueError, "block_table"),
            (dict(pos_offset=None), TypeError, None), (dict(v_pages=pool), R.RopeError, None)]:
        with pytest.raises(err, match=name):
            R.cache_append(**dict(append, **over))
    assert R.rope_check_errors() == R.ROPE_OK
