"""A transformer block's MLP on quantized rows, as it is used: norm and modulation to quantized rows,
colwise product with GELU, quantization, rowwise partials of every rank, and the boundary to the
next block.  Each step is checked against 64 bits on the step's own inputs; the chain is also
captured in a HIP graph, run on another stream, and by threads at once."""
import threading

import pytest
import torch

import block_reference as ref
import tensor_sharded_linear_amd as tsl

pytestmark = pytest.mark.gpu
BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
D, F, P = 512, 1024, 2


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    w1 = torch.randn(F, D, generator=g).mul_(D ** -0.5).to(BF).cuda()
    w2 = torch.randn(D, F, generator=g).mul_(F ** -0.5).to(BF).cuda()
    b1, b2 = torch.randn(F, generator=g).to(BF).cuda(), torch.randn(D, generator=g).to(BF).cuda()
    w = dict(b2=b2, mod=torch.randn(1, 6 * D, generator=g).mul_(0.5).to(BF).cuda())
    w["ranks"] = []
    for r in range(P):
        s1, sb = tsl.tp_plan_shard_slice(w1, b1, "colwise", P, r)
        s2, _ = tsl.tp_plan_shard_slice(w2, None, "rowwise", P, r)
        w["ranks"].append((tsl.tp_quantize_fp8(s1), sb, tsl.tp_quantize_fp8(s2)))
    return w


def _chain(x, w, stream=None, keep=None):
    mod = [w["mod"][:, i * D:(i + 1) * D] for i in range(5)]
    m = x.shape[0]
    _, z = tsl.tp_block_norm(x, scale=mod[0], shift=mod[1], z_dtype=FP8, stream=stream, group_rows=m)
    parts = []
    for q1, b1, q2 in w["ranks"]:
        hid = tsl.tp_linear_colwise_fp8(*z, *q1, b1, act="gelu_tanh", stream=stream)
        q = tsl.tp_quantize_fp8(hid, stream=stream)
        parts.append(tsl.tp_linear_rowwise_fp8(*q, *q2, stream=stream))
        if keep is not None:
            keep.append((z, q1, b1, q2, hid, q, parts[-1]))
    return tsl.tp_block_norm(x, parts, bias=w["b2"], gate=mod[2], scale=mod[3], shift=mod[4], group_rows=m, stream=stream)


@pytest.mark.parametrize("m", [1, 7, 64, 200, 700, 3001])
def test_chain_step_by_step(m):
    w = _weights(m)
    x = torch.randn(m, D, generator=torch.Generator().manual_seed(m)).to(BF).cuda()
    keep = []
    h, z = _chain(x, w, keep=keep)
    for z8, q1, b1, q2, hid, q, part in keep:
        ref.check(hid, *ref.linear(ref.values(*z8), ref.values(*q1), b1, "gelu_tanh", m > 96))
        ref.check(part, *ref.linear(ref.values(*q), ref.values(*q2), None, "none"))
    mod = [w["mod"][:, i * D:(i + 1) * D] for i in range(5)]
    (wh, eh), (wz, ez) = ref.block_norm(x, [k[-1] for k in keep], w["b2"], ("none", None, None), mod[2], 1.0,
                                        ("layer", None, None), mod[3], mod[4], 1e-6, torch.zeros(m, dtype=torch.int64))
    ref.check(h, wh, eh)
    ref.check(z, wz, ez)


@pytest.mark.parametrize("m", [5, 300, 3001])
def test_graph_replays_equal_eager(m):
    """Replays with eager work and synchronisations between them, each against the eager result."""
    w = _weights(1)
    x = torch.randn(m, D, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _chain(x, w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, z = _chain(x, w)
    for i in range(4):
        x.copy_(torch.randn(m, D, generator=torch.Generator().manual_seed(10 + i)).to(BF).cuda())
        eh, ez = _chain(x, w)
        torch.cuda.synchronize()
        h.fill_(float("nan"))
        z.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, eh) and torch.equal(z, ez), i


def test_another_stream_and_threads():
    """Each thread on its own stream (given explicitly, not current): the same bits as alone."""
    ws = [_weights(s) for s in range(3)]
    xs = [torch.randn(m, D, generator=torch.Generator().manual_seed(m)).to(BF).cuda() for m in (3, 120, 2500)]
    want = [_chain(x, w) for x, w in zip(xs, ws)]
    torch.cuda.synchronize()
    got, bad = [None] * 3, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):   # outputs are allocated on the stream that writes them
                for _ in range(5):
                    got[i] = _chain(xs[i], ws[i], stream=s)
                    with pytest.raises(ValueError):
                        tsl.tp_linear_rowwise_fp8(*ws[i]["ranks"][0][0], *ws[i]["ranks"][0][0], stream=s,
                                                  out=torch.empty(F // P, F // P + 2, device="cuda")[:, 1:-1])
                    assert "tp_linear_rowwise_fp8" in tsl.tp_last_error()
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert not bad and not any(t.is_alive() for t in threads), bad
    for (h, z), (wh, wz) in zip(got, want):
        assert torch.equal(h, wh) and torch.equal(z, wz)
