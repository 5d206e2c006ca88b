"""The binding's calls on another stream than the current one, given as a torch
stream, as a handle and as the default stream's handle 0: the bits of the
current stream's."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from bit_kv_cache_qvg_b200 import build
    build.build()
    from bit_kv_cache_qvg_b200 import qvg
    return qvg


def everything(q, X, Q, pos, **kw):
    """What a program computes of one block of keys and one of values."""
    cfg = q.config(K=64, T=2, group_size=64, iters=3)
    k, v = q.quantize(X[0], cfg, **kw), q.quantize(X[1], cfg, **kw)
    static = q.quantize_static(X[0], cfg, **kw)
    tables = q.rope_tables(4000, **kw)
    cache = q.Cache(cfg, X[0].shape[0], 4000, 2)
    cache.append(X[0], **kw)
    whole = cache.dequantize(**kw)
    O = q.attention(k, v, Q, pos, tables, **kw)
    W = q.attention_weights(k, Q[None], pos[None], tables, **kw)
    e = q.evict(k, v, W, 700, **kw)
    out = [k.codes, k.assign, k.centroids, v.scale, v.zero, static.codes, q.dequantize(k, **kw), whole, tables[256:], O, W,    # (of the header only the status word is set)
           q.attention_batch(k, v, Q[None], pos[None], tables, **kw), e.kept, e.k.codes, q.dequantize(e.v, **kw)]
    return out, cache


@pytest.mark.parametrize("of", [lambda s: s, lambda s: s.cuda_stream], ids=["stream", "handle"])
def test_calls_on_a_side_stream(q, of):
    from bit_kv_cache_qvg_b200 import synth
    X = [synth.block_batch(2, synth.KVShape(1, 30, 52), seed=s, kinds=[kind] * 2).cuda() for s, kind in ((3, 0), (4, 1))]
    Q = torch.randn((2, 90, 128), device="cuda").to(torch.bfloat16)
    pos = 1560 + torch.arange(90, device="cuda")
    want, keep = everything(q, X, Q, pos)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        torch.cuda._sleep(2_000_000)
        busy = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 20, 1 << 24)]
        del busy                                        # let go of, with its work still queued
        got, cache = everything(q, X, Q, pos, stream=of(side))
        torch.cuda.current_stream().wait_stream(side)
        same = [torch.equal(a, b) for a, b in zip(got, want)]
        assert all(same), same
        side.synchronize()
        del got, cache
    with torch.cuda.stream(side):                       # the default stream, from another one
        got, cache = everything(q, X, Q, pos, stream=0)
        side.wait_stream(torch.cuda.default_stream())
        same = [torch.equal(a, b) for a, b in zip(got, want)]
        torch.cuda.synchronize()
    assert all(same), same


def test_a_side_stream_inside_a_capture(q):
    """A captured graph with a branch on another stream: what the branch allocates is the
    graph's, results that nobody keeps among them."""
    g = torch.Generator(device="cuda").manual_seed(5)
    cfg = q.config(K=32, T=1, group_size=64)
    k, v = (q.quantize(torch.randn((2, 3000, 128), generator=g, device="cuda"), cfg) for _ in range(2))
    k, v = (q.Packed(codes=p.codes, scale=p.scale, zero=p.zero, assign=p.assign, centroids=p.centroids.to(torch.bfloat16),
                     cfg=cfg, N=3000, H=2, d=128, dtype=q.BF16) for p in (k, v))
    tables = q.rope_tables(4000)
    Q = [torch.randn((1, 2, n, 128), generator=g, device="cuda").to(torch.bfloat16) for n in (3, 300)]
    pos = [3000 + torch.arange(x.shape[2], device="cuda")[None] for x in Q]

    def step(**kw):
        W = q.attention_weights(k, Q[1], pos[1], tables, **kw)
        q.attention_batch(k, v, Q[0], pos[0], tables, **kw)              # not kept
        return q.attention_batch(k, v, Q[1], pos[1], tables, **kw), q.attention_batch(k, v, Q[0], pos[0], tables, **kw), W, \
            q.evict(k, v, W, 1000, **kw).k.codes

    want = step()
    torch.cuda.synchronize()
    side, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        a, b = step(stream=side), step()
        here.wait_stream(side)
    for _ in range(3):
        for x in (*a, *b):
            x.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for r in (a, b) for x, y in zip(r, want))


def test_a_stream_of_another_device_is_refused(q):
    class Elsewhere(torch.cuda.Stream):
        device = torch.device("cuda", 1)

    p = q.alloc_packed(q.config(K=16, T=1, group_size=64), 10, 1)
    with pytest.raises(q.QvgError) as e:
        q.dequantize(p, stream=Elsewhere())
    assert e.value.status == 1
