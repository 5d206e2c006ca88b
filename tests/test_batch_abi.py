"""CPU checks of qvg_attention_batch, qvg_attention_weights and qvg_evict: what
they refuse, and that they refuse it before they touch the GPU."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def q():
    from bit_kv_cache_qvg_b200 import build
    build.build()
    from bit_kv_cache_qvg_b200 import qvg
    qvg.lib()
    return qvg


def packed(q, **kw):
    a = dict(codes=0x2000, scale=0x3000, zero=0x4000, assign=0x5000, centroids=0x6000)
    a.update(kw)
    return q._Packed(*(a[k] for k in ("codes", "scale", "zero", "assign", "centroids")))


def batch(q, **kw):
    a = dict(B=2, group=1, Nq=1, Nt=16, Q=0x10000, q_pos=0x20000, k_pos=None, tail_k=0x30000, tail_v=0x40000,
             tail_pos=0x50000, tail_len=0x60000, causal=1)
    a.update(kw)
    return q._Batch(**a)


def both(q, cfg=None, k=None, v=None, Nk=1000, H=4, d=128, b=None, tables=0x70000, positions=1000, O=0x80000, received=None,
         out=0x90000, ws=0xA0000, ws_bytes=0):
    """The status of the two calls on a batch (a workspace of no bytes: no call gets past it)."""
    L = q.lib()
    cfg = cfg or q.config(K=16, T=1, group_size=16, iters=4)
    k, v, b = k or packed(q), v or packed(q), b or batch(q)
    n = 256 + 512 * positions
    return (L.qvg_attention_batch(C.byref(cfg), C.byref(k), C.byref(v), Nk, H, d, C.byref(b), tables, n, O, ws, ws_bytes, None),
            L.qvg_attention_weights(C.byref(cfg), C.byref(k), Nk, H, d, C.byref(b), tables, n, received, out, ws, ws_bytes, None))


def test_a_valid_call_gets_as_far_as_the_workspace(q):
    assert both(q) == (6, 6)
    assert both(q, b=batch(q, Nt=0, tail_k=None, tail_v=None, tail_pos=None, tail_len=None)) == (6, 6)
    assert both(q, b=batch(q, tail_pos=None, tail_len=None, causal=0)) == (6, 6)
    assert both(q, b=batch(q, k_pos=0x100000), positions=10) == (6, 6)          # positions of its own: any table
    sym = q.config(K=16, T=1, group_size=16, scale_mode=q.SYM)
    assert both(q, cfg=sym, k=packed(q, zero=None), v=packed(q, zero=None)) == (6, 6)
    plain = q.config(K=16, T=0, group_size=16)
    assert both(q, cfg=plain, k=packed(q, assign=None, centroids=None), v=packed(q, assign=None, centroids=None)) == (6, 6)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(B=-1), dict(group=0), dict(Nq=0), dict(Nt=-1), dict(causal=2), dict(Q=None), dict(q_pos=None),
    dict(Q=0x10008), dict(q_pos=0x20004), dict(k_pos=0x100004), dict(tail_k=None), dict(tail_k=0x30008),
    dict(tail_pos=0x50004), dict(tail_len=0x60002),
])
def test_bad_batches_are_refused(q, kw):
    assert both(q, b=batch(q, **kw)) == (1, 1)


def test_the_values_of_a_tail_are_asked_for_where_they_are_read(q):
    assert both(q, b=batch(q, tail_v=None)) == (1, 6)
    assert both(q, b=batch(q, tail_v=0x40008)) == (1, 6)


@pytest.mark.parametrize("kw", [dict(Nq=1 << 23), dict(Nt=1 << 23), dict(B=1 << 12, group=1 << 11), dict(B=1 << 21), dict(B=4, Nq=1 << 21)])
def test_sizes_beyond_the_kernels_are_unsupported(q, kw):
    assert both(q, b=batch(q, **kw)) == (2, 2)


def test_bad_arguments_are_refused(q):
    assert both(q, Nk=0) == (1, 1)
    assert both(q, Nk=1 << 23) == (2, 2)
    assert both(q, H=0) == (1, 1)
    assert both(q, d=64) == (2, 2)
    assert both(q, cfg=q.config(K=300, T=1, group_size=16)) == (1, 1)
    assert both(q, cfg=q.config(K=16, T=9, group_size=16)) == (2, 2)
    assert both(q, positions=999) == (1, 1)                      # token 999 is beyond the tables
    assert both(q, positions=0) == (1, 1)
    assert both(q, tables=None) == (1, 1)
    assert both(q, tables=0x70010) == (1, 1)                     # 32-byte aligned
    assert both(q, ws=None) == (1, 1)
    assert both(q, ws=0xA0008, ws_bytes=1 << 30) == (1, 1)
    assert both(q, O=None)[0] == 1 and both(q, O=0x80008)[0] == 1
    assert both(q, out=None)[1] == 1 and both(q, out=0x90002)[1] == 1 and both(q, received=0x90001)[1] == 1
    for bad in (dict(codes=None), dict(codes=0x2008), dict(scale=None), dict(scale=0x3004), dict(zero=None), dict(zero=0x4001),
                dict(assign=None), dict(centroids=None), dict(centroids=0x6008)):
        assert both(q, k=packed(q, **bad)) == (1, 1), bad
        assert both(q, v=packed(q, **bad)) == (1, 6), bad
    L, cfg, p = q.lib(), q.config(K=16, T=1, group_size=16), packed(q)
    assert L.qvg_attention_batch(C.byref(cfg), C.byref(p), C.byref(p), 10, 1, 128, None, 0x70000, 1 << 20, 0x80000, 0xA0000, 0, None) == 1
    assert L.qvg_attention_weights(C.byref(cfg), None, 10, 1, 128, C.byref(batch(q)), 0x70000, 1 << 20, None, 0x90000, 0xA0000, 0, None) == 1
    assert q.attention_batch_workspace_bytes(cfg, 0, 1, 1, 1, 1) == 0
    assert q.attention_weights_workspace_bytes(cfg, 10, 1, 0, 1, 1) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory: without a device the launch fails instead")
@pytest.mark.parametrize("b", [dict(B=4, Nq=380, Nt=380), dict(B=1, Nq=1560, Nt=0), dict(B=8, group=4, Nt=512), dict(B=16, group=4, Nt=0), dict(B=1, Nt=33)])
def test_a_workspace_for_some_of_the_heads_is_enough(q, b):
    """32 heads of 38,000 tokens ask for up to 1.3 GB; 64 MiB hold a few heads at a
    time, 64 KiB not even one."""
    cfg = q.config(K=256, T=2, group_size=64)
    kw = dict(cfg=cfg, Nk=38000, H=32, positions=40000, b=batch(q, **b))
    assert both(q, ws_bytes=64 << 20, **kw) == (4, 4)             # as far as the launch
    assert both(q, ws_bytes=4096, **kw) == (6, 6)


def evict(q, cfg=None, k=None, v=None, Nk=1000, H=4, d=128, weights=0x10000, k_pos=None, keep=500, first=4, recent=32, ko=None,
          vo=None, kept=0x20000, pos=0x30000, wout=0x40000):
    cfg = cfg or q.config(K=16, T=1, group_size=16)
    k, v = k or packed(q), v or packed(q, codes=0x7000, scale=0x8000, zero=0x9000, assign=0xA000)
    ko = ko or packed(q, codes=0x102000, scale=0x103000, zero=0x104000, assign=0x105000)
    vo = vo or packed(q, codes=0x107000, scale=0x108000, zero=0x109000, assign=0x10A000)
    return q.lib().qvg_evict(C.byref(cfg), C.byref(k), C.byref(v), Nk, H, d, weights, k_pos, keep, first, recent, C.byref(ko), C.byref(vo),
                             kept, pos, wout, None)


@pytest.mark.parametrize("kw,status", [
    (dict(keep=0), 1), (dict(keep=1001), 1), (dict(first=-1), 1), (dict(recent=-1), 1), (dict(first=469), 1), (dict(recent=497), 1),
    (dict(first=1 << 62, recent=1 << 62), 1),
    (dict(weights=None), 1), (dict(weights=0x10002), 1), (dict(kept=None), 1), (dict(kept=0x20001), 1), (dict(k_pos=0x30004), 1),
    (dict(pos=0x30004), 1), (dict(wout=0x40002), 1), (dict(Nk=0, keep=1), 1), (dict(H=0), 1), (dict(d=96), 2), (dict(Nk=1 << 23), 2),
    (dict(wout=0x10000), 1), (dict(k_pos=0x30000), 1),
])
def test_evict_refuses(q, kw, status):
    cfg = q.config(K=16, T=1, group_size=16)
    if kw.get("d") == 96:
        cfg = q.config(K=16, T=1, group_size=32)
    assert evict(q, cfg=cfg, **kw) == status


def test_evict_refuses_outputs_that_are_inputs(q):
    for field, at in (("codes", 0x2000), ("scale", 0x3000), ("zero", 0x4000), ("assign", 0x5000)):
        out = dict(codes=0x102000, scale=0x103000, zero=0x104000, assign=0x105000)
        out[field] = at
        assert evict(q, ko=packed(q, **out)) == 1, field
        assert evict(q, vo=packed(q, **{**out, "codes": out["codes"] + (0 if field == "codes" else 0x5000)})) == 1, field
    for field, at in (("codes", 0x102000), ("scale", 0x103000), ("zero", 0x104000), ("assign", 0x105000)):
        out = dict(codes=0x107000, scale=0x108000, zero=0x109000, assign=0x10A000)
        out[field] = at                       # both caches' outputs in one place
        assert evict(q, vo=packed(q, **out)) == 1, field
    for bad in (dict(codes=None), dict(codes=0x2008), dict(scale=0x3004), dict(zero=None), dict(assign=None)):
        assert evict(q, k=packed(q, **bad)) == 1, bad


def test_the_binding_checks_before_it_calls(q):
    cfg = q.config(K=16, T=1, group_size=64)
    p = q.alloc_packed(cfg, 100, 2, device="cpu")
    Q = torch.zeros((1, 4, 3, 128), dtype=torch.bfloat16)
    pos = torch.zeros((1, 3), dtype=torch.int64)
    tables = torch.zeros(256 + 512 * 200, dtype=torch.uint8)
    for kw in (dict(Q=Q.float()), dict(Q=Q[0]), dict(Q=Q[:, :3]), dict(Q=Q.transpose(1, 2)), dict(q_pos=pos.int()), dict(q_pos=pos[0]),
               dict(k_pos=torch.zeros((2, 99), dtype=torch.int64)), dict(tables=tables.float()),
               dict(tail=q.Tail(k=torch.zeros((1, 2, 5, 64), dtype=torch.bfloat16))),
               dict(tail=q.Tail(k=torch.zeros((2, 5, 128), dtype=torch.bfloat16))),
               dict(tail=q.Tail(k=torch.zeros((1, 2, 5, 128), dtype=torch.bfloat16), length=torch.zeros(1))),
               dict()):                       # a CPU cache
        args = dict(Q=Q, q_pos=pos, tables=tables)
        args.update(kw)
        for call in (lambda: q.attention_batch(p, p, **args), lambda: q.attention_weights(p, **args)):
            with pytest.raises(q.QvgError) as e:
                call()
            assert e.value.status == 1, kw
    w = torch.zeros((2, 100))
    for kw in (dict(keep=0), dict(keep=101), dict(keep=5, first=3, recent=3), dict(keep=5, first=-1), dict(keep=5, weights=w.double()),
               dict(keep=5, weights=w[:1]), dict(keep=5)):
        with pytest.raises(q.QvgError) as e:
            q.evict(p, p, kw.pop("weights", w), **kw)
        assert e.value.status == 1
    with pytest.raises(q.QvgError):
        q.evict(p, q.alloc_packed(q.config(K=16, T=2, group_size=64), 100, 2, device="cpu"), w, 5)
    with pytest.raises(q.QvgError) as e:
        q.attention_weights(q.alloc_packed(cfg, 100, 2, dtype=q.FP32, device="cpu"), Q, pos, tables)
    assert e.value.status == 2


# ------------------------------------------------------------------ packed streams

def damaged(q, cfg, H=2, N=100):
    """A packed form, and what one of its tensors could be that is not laid out as its sizes say."""
    import dataclasses
    p = q.alloc_packed(cfg, N, H, device="cpu")
    wide = q.alloc_packed(cfg, N, 2 * H, device="cpu")
    tall = q.alloc_packed(cfg, 2 * N, H, device="cpu")
    for name in ("codes", "scale", "zero", "assign", "centroids"):
        if getattr(p, name).numel() == 0:
            continue
        by_head = 1 if name in ("assign", "centroids") else 0
        every_other = torch.narrow(getattr(wide, name), by_head, 0, 2 * H).unflatten(by_head, (H, 2)).select(by_head + 1, 0)
        yield name, dataclasses.replace(p, **{name: every_other})              # heads with a gap between them
        yield name, dataclasses.replace(p, **{name: getattr(p, name).narrow(by_head, 0, H - 1)})          # a head short
        if name != "centroids":
            part = getattr(tall, name).narrow(by_head + 1, 0, N)              # a part of longer streams
            assert part.shape == getattr(p, name).shape
            yield name, dataclasses.replace(p, **{name: part})
            yield name, dataclasses.replace(p, **{name: getattr(tall, name)})
        yield name, dataclasses.replace(p, **{name: getattr(p, name).float()})


@pytest.mark.parametrize("T,mode", [(2, 0), (1, 1), (0, 0)])
def test_packed_streams_that_are_not_laid_out_as_their_sizes_say_are_refused(q, T, mode, monkeypatch):
    """Every call reads (or writes) a packed form's tensors as contiguous arrays of its
    sizes: a strided view, a short or a long one, another element size is refused
    before the library is called."""
    cfg = q.config(K=16, T=T, group_size=64, scale_mode=mode)
    good = q.alloc_packed(cfg, 100, 2, device="cpu")
    good.struct()
    Q, pos = torch.zeros((1, 4, 3, 128), dtype=torch.bfloat16), torch.zeros((1, 3), dtype=torch.int64)
    tables, w, X = torch.zeros(256 + 512 * 200, dtype=torch.uint8), torch.zeros((2, 100)), torch.zeros((2, 100, 128), dtype=torch.bfloat16)

    class Library:
        def __getattr__(self, name):
            def call(*a):
                assert name.endswith("_bytes"), f"{name} was called"
                return 4096
            return call

    monkeypatch.setattr(q, "lib", Library)
    monkeypatch.setattr(q, "_on_device", lambda *t: torch.device("cpu"))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)
    monkeypatch.setattr(q, "_stream", lambda s: 0)
    n = 0
    for name, p in damaged(q, cfg):
        for call in (lambda: q.attention_batch(p, good, Q, pos, tables), lambda: q.attention_batch(good, p, Q, pos, tables),
                     lambda: q.attention_weights(p, Q, pos, tables), lambda: q.evict(p, good, w, 50), lambda: q.evict(good, p, w, 50),
                     lambda: q.attention(p, good, Q[0, :2], pos[0], tables), lambda: q.dequantize(p),
                     lambda: q.quantize(X, cfg, out=p, workspace=torch.zeros(4096, dtype=torch.uint8)), lambda: q.quantize_static(X, cfg, out=p)):
            with pytest.raises(q.QvgError) as e:
                call()
            assert e.value.status == 1 and name in str(e.value), (name, str(e.value))
            n += 1
    assert n > 50


def test_heads_of_a_packed_form_that_are_contiguous_are_taken(q):
    """A part whose strides say no more than its sizes is a packed form."""
    p = q.alloc_packed(q.config(K=16, T=1, group_size=64), 100, 5, device="cpu")
    one = q.Packed(codes=p.codes[-2:], scale=p.scale[-2:], zero=p.zero[-2:], assign=p.assign[:, -2:], centroids=p.centroids[:, -2:],
                   cfg=p.cfg, N=100, H=2, d=128, dtype=q.BF16)
    s = one.struct()
    assert s.codes == p.codes.data_ptr() + 3 * 100 * 32 and s.assign == p.assign.data_ptr() + 300
