"""qvg_attention_batch, qvg_attention_weights and qvg_evict against plain
implementations in 64 bits, at the sizes and masks where they can go wrong.

Tolerances, from the kernels' arithmetic, with u = 2^-8 (half a bf16 step) and
v = 2^-11 (half an fp16 step; below 2^-14 the rounding is at most 2^-25):

* attention_batch: rotated queries and keys rounded to fp16, so a score is off
  by at most eps_j = (2v + v^2 + 2^-16) sum_c |q'_c k'_jc| / sqrt(d) + 2^-25
  sum_c (|q'_c| + |k'_jc|) / sqrt(d), where 2^-16 covers the fp32 rotations and
  sums (128 terms, 2^-24 each); a weight rounded to bf16 (u) and a base-2
  exponential (2^-21).  A normalised weight then changes by a factor between
  1/F and F, F = (1 + u + 2^-21) / (1 - u - 2^-21) e^(2 eps), eps the row's
  largest, so that element c of O is off by at most (F - 1) sum_j w_j |v_jc|,
  plus the output's rounding u |O_c| and the fp32 sums over the keys (2^-24 a
  key).
* attention_weights: operands of two fp16 halves leave v^2 of each operand (or
  2^-25) and drop the product of the low halves (v^2): eps_j = (3 v^2 + 2^-16)
  sum |q' k'| / sqrt(d) + 2^-25 sum (|q'| + |k'|) / sqrt(d), F = e^(2 eps)
  (1 + 2^-20) with the scores' and the logarithm's fp32 rounding, 2^-23 (|s| +
  |lse|), in the exponent; each row adds (F - 1) w, and the sums over rows and
  onto `received` 2^-24 a term."""
import numpy as np
import pytest
import torch

from gpu_util import np_bits, values

pytestmark = pytest.mark.gpu
D = 128
U, V = 2.0 ** -8, 2.0 ** -11


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from bit_kv_cache_qvg_b200 import build
    build.build()
    from bit_kv_cache_qvg_b200 import qvg
    return qvg


def streams(q, g, cfg, H, N, spread=1.0):
    """A packed form of H blocks of N tokens with random codes, scales and tables."""
    u8 = lambda *s, hi=256: torch.randint(0, hi, s, generator=g, dtype=torch.uint8)  # noqa: E731
    e4m3 = lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    ng, T, K = D // cfg.group_size, cfg.T, cfg.K
    scale = torch.rand((H, N, ng), generator=g) * 0.3 + 0.02
    zero = e4m3(scale * (torch.rand(scale.shape, generator=g) - 2.0)) if cfg.scale_mode == q.ASYM else torch.empty((0,), dtype=torch.uint8)
    tables = (torch.randn((T, H, K, D), generator=g) * spread).to(torch.bfloat16)
    p = dict(codes=u8(H, N, D // 4), scale=e4m3(scale), zero=zero, assign=u8(T, H, N, hi=min(K + 1, 256)),
             centroids=tables)
    return q.Packed(**{k: v.cuda() for k, v in p.items()}, cfg=cfg, N=N, H=H, d=D, dtype=q.BF16)


def rebuilt(ora, p):
    """The oracle's reconstruction [H][N][d] in fp64 (the kernels clamp centroid
    indices to K - 1, the oracle is given them clamped)."""
    c = p.cfg
    named = dict(codes=np_bits(p.codes), scale=np_bits(p.scale), zero=np_bits(p.zero),
                 assign=np.minimum(np_bits(p.assign), c.K - 1), centroids=np_bits(p.centroids))
    return values(ora.dequantize(named, K=c.K, T=c.T, G=c.group_size, N=p.N, H=p.H, d=D, scale_mode=c.scale_mode))


def rotated(x, pos, base=10000.0):
    a = np.asarray(pos, np.float64)[:, None] * base ** (-2.0 * np.arange(D // 2) / D)
    re, im = x[:, 0::2], x[:, 1::2]
    out = np.empty_like(x)
    out[:, 0::2], out[:, 1::2] = re * np.cos(a) - im * np.sin(a), re * np.sin(a) + im * np.cos(a)
    return out


class Case:
    """One batch: its device arguments, and every row's keys, values and scores in 64 bits."""

    def __init__(self, q, ora, seed, H=2, group=1, B=1, Nq=1, Nk=100, Nt=0, K=16, T=1, G=64, mode=0, causal=False,
                 gaps=False, lens=None, q_pos=None, spread=1.0, q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.cfg = q.config(K=K, T=T, group_size=G, scale_mode=mode)
        self.kp, self.vp = streams(q, g, self.cfg, H, Nk, spread), streams(q, g, self.cfg, H, Nk, spread)
        self.H, self.group, self.B, self.Nq, self.Nk, self.Nt, self.causal = H, group, B, Nq, Nk, Nt, causal
        self.Q = (torch.randn((B, H * group, Nq, D), generator=g) * q_scale).to(torch.bfloat16)
        self.k_pos = torch.cumsum(torch.randint(1, 4, (H, Nk), generator=g), 1) - 1 if gaps else None
        past = 3 * Nk if gaps else Nk
        self.tail = None
        self.lens = [Nt] * B if lens is None else lens
        if Nt:
            tk, tv = (torch.randn((B, H, Nt, D), generator=g).to(torch.bfloat16) for _ in range(2))
            for b, n in enumerate(self.lens):       # what lies behind a tail's length may hold anything
                tk[b, :, n:], tv[b, :, n:] = float("nan"), float("inf")
            self.tail_pos = past + torch.arange(Nt).repeat(B, 1)
            self.tk, self.tv = tk, tv
            self.tail = q.Tail(k=tk.cuda(), v=tv.cuda(), pos=self.tail_pos.cuda(),
                               length=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
        if q_pos is None:
            q_pos = past + torch.arange(Nq).repeat(B, 1) + (max(0, Nt - Nq) if causal else 0)
        self.q_pos = q_pos
        self.tables = q.rope_tables(past + Nt + Nq + 10)
        self.Kh, self.Vh = rebuilt(ora, self.kp), rebuilt(ora, self.vp)

    def args(self):
        return dict(Q=self.Q.cuda(), q_pos=self.q_pos.cuda(), tables=self.tables, tail=self.tail,
                    k_pos=None if self.k_pos is None else self.k_pos.cuda(), causal=self.causal)

    def rows(self):
        """(b, j, h, scores, sum |q' k'| / sqrt(d), 2^-25 sum (|q'| + |k'|) / sqrt(d), mask, values) of the Nq rows of each sequence and query head."""
        for b in range(self.B):
            n = self.lens[b] if self.Nt else 0
            pos = self.q_pos[b].numpy()
            for h in range(self.H):
                at = np.arange(self.Nk) if self.k_pos is None else self.k_pos[h].numpy()
                k, v = rotated(self.Kh[h], at), self.Vh[h]
                if n:
                    tp = self.tail_pos[b, :n].numpy()
                    k = np.concatenate([k, rotated(values(np_bits(self.tk[b, h, :n])), tp)])
                    v = np.concatenate([v, values(np_bits(self.tv[b, h, :n]))])
                    at = np.concatenate([at, tp])
                sees = np.broadcast_to(pos[:, None] >= 0, (self.Nq, len(at)))
                if self.causal:
                    sees = sees & (at[None] <= pos[:, None])
                for j in range(h * self.group, (h + 1) * self.group):
                    qr = rotated(values(np_bits(self.Q[b, j])), np.maximum(pos, 0))
                    small = 2.0 ** -25 * (np.abs(qr).sum(1)[:, None] + np.abs(k).sum(1)[None]) / np.sqrt(D)
                    yield b, j, h, qr @ k.T / np.sqrt(D), np.abs(qr) @ np.abs(k).T / np.sqrt(D), small, sees, v


def softmax(s, sees):
    s = np.where(sees, s, -np.inf)
    m = s.max(1, keepdims=True, initial=-1e300)
    e = np.exp(s - m)
    z = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = m[:, 0] + np.log(z[:, 0])
    return e / np.maximum(z, 1e-300), lse


def check_attention(case, O):
    O = values(np_bits(O))
    assert np.isfinite(O).all()
    for b, j, h, s, mag, small, sees, v in case.rows():
        w, _ = softmax(s, sees)
        ref = w @ v
        eps = np.where(sees, (2 * V + V * V + 2.0 ** -16) * mag + small, 0.0).max(1)
        F = (1 + U + 2.0 ** -21) / (1 - U - 2.0 ** -21) * np.exp(2 * eps)
        bound = (F - 1 + s.shape[1] * 2.0 ** -24)[:, None] * (w @ np.abs(v))
        bound = bound + U * (np.abs(ref) + bound) + 1e-30
        err = np.abs(O[b, j] - ref)
        assert np.all(err <= bound), (b, j, float((err / bound).max()), float(err.max()))
        assert np.all(O[b, j][~sees.any(1)] == 0.0)


def check_weights(case, out, received=None):
    H, Nk = case.H, case.Nk
    out = out.cpu().numpy().astype(np.float64)
    ref = np.zeros((H, Nk)) if received is None else received.cpu().numpy().astype(np.float64).copy()
    bound = np.abs(ref) * 2.0 ** -23 + 1e-30
    rows = case.B * case.group * case.Nq
    for b, j, h, s, mag, small, sees, v in case.rows():
        w, lse = softmax(s, sees)
        eps = np.where(sees, (3 * V * V + 2.0 ** -16) * mag + small, 0.0).max(1)
        eps = eps + 2.0 ** -23 * (np.abs(np.where(sees, s, 0.0)).max(1) + np.where(np.isfinite(lse), np.abs(lse), 0.0))
        F = np.exp(2 * eps) * (1 + 2.0 ** -20 + s.shape[1] * 2.0 ** -24)
        ref[h] += w[:, :Nk].sum(0)
        bound[h] += ((F - 1 + rows * 2.0 ** -24)[:, None] * w[:, :Nk]).sum(0)
    bound += np.abs(ref) * 2.0 ** -23
    err = np.abs(out - ref)
    assert np.all(err <= bound), (float((err / bound).max()), float(err.max()))


SHAPES = [
    dict(Nk=1),                                                                   # one key, one row
    dict(Nk=1, Nt=1, causal=True, B=2),
    dict(Nk=77, Nt=5, B=3, group=2, causal=True, T=0, G=32, lens=[5, 0, 2]),      # plain rounding, an empty tail
    dict(Nk=512, Nt=16, B=2, causal=True, G=16, lens=[16, 3]),
    dict(Nk=1000, Nt=33, B=5, group=4, T=2, K=256, lens=[33, 1, 32, 0, 17], gaps=True),
    dict(Nk=700, Nq=4, B=2, group=2, Nt=40, T=4, G=16, mode=1, causal=True, K=200),
    dict(Nk=333, Nq=37, Nt=37, causal=True, T=3, G=8, K=64),
    dict(H=1, Nk=2049, Nq=130, B=2, Nt=130, T=2, G=128, mode=1, gaps=True, K=64),
    dict(H=3, Nk=1300, Nq=300, B=2, Nt=300, causal=True, T=2, K=64, lens=[300, 150]),
    dict(H=1, Nk=900, Nq=520, T=1, G=32, mode=1, K=256),
    dict(H=1, Nk=400, Nq=3, T=5, K=32, B=2, Nt=9),                                # the stage count at run time
    dict(H=1, Nk=515, Nq=290, T=6, K=32, group=2, causal=True, gaps=True),
    dict(Nk=260, B=2, Nt=3, lens=[0, 3], G=8, K=256, mode=1),                     # two rows, the smallest groups
    dict(Nk=131, B=3, Nt=70, lens=[70, 64, 1], T=8, G=128),                       # three rows, eight stages
    dict(H=1, Nk=200, Nq=64, Nt=1, T=2),                                          # the most rows without the tensor-core kernels' tiles
    dict(H=1, Nk=129, Nq=65, Nt=129, T=0, G=32, causal=True),                     # one more
    dict(H=2, Nk=256, Nq=129, B=3, Nt=200, lens=[0, 200, 128], T=1),              # an empty tail among long ones
    dict(H=1, Nk=100, Nq=20, B=4, group=2, Nt=40, lens=[40, 0, 7, 39], causal=True, G=8),   # many rows, few to a sequence
    # enough blocks of 64 rows x 64 keys for the tensor-core kernels
    dict(H=2, Nk=2601, Nq=130, B=2, Nt=130, T=2, G=128, mode=1, gaps=True, K=64),
    dict(H=3, Nk=1700, Nq=300, B=2, Nt=300, causal=True, T=2, K=64, lens=[300, 150]),
    dict(H=3, Nk=2300, Nq=300, T=1, G=32, mode=1, K=256),
    dict(H=2, Nk=2700, Nq=290, T=6, K=32, group=2, causal=True, gaps=True),
    dict(H=3, Nk=4600, Nq=65, Nt=129, T=0, G=32, causal=True),
    dict(H=2, Nk=2690, Nq=129, B=3, Nt=200, lens=[0, 200, 128], T=4, G=16),
    dict(H=3, Nk=3200, Nq=20, B=4, group=2, Nt=40, lens=[40, 0, 7, 39], causal=True, T=3, G=8),
    dict(H=2, Nk=64, Nq=1000, Nt=1000, causal=True, T=2),                         # the tail is the most of it
]


@pytest.mark.parametrize("kw", SHAPES, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items() if k != "lens"))
def test_attention_batch_matches_64_bits(q, ora, kw):
    case = Case(q, ora, seed=len(str(kw)), **kw)
    O = q.attention_batch(case.kp, case.vp, **case.args())
    torch.cuda.synchronize()
    assert q.workspace_status(case.tables) == 0
    check_attention(case, O)


@pytest.mark.parametrize("kw", SHAPES, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items() if k != "lens"))
def test_attention_weights_match_64_bits(q, ora, kw):
    case = Case(q, ora, seed=len(str(kw)), **kw)
    received = torch.rand((case.H, case.Nk), generator=torch.Generator().manual_seed(3)).cuda()
    out = q.attention_weights(case.kp, received=received, **case.args())
    alone = q.attention_weights(case.kp, **case.args())
    again = received.clone()
    q.attention_weights(case.kp, received=again, out=again, **case.args())        # in place
    torch.cuda.synchronize()
    assert q.workspace_status(case.tables) == 0
    check_weights(case, out, received)
    check_weights(case, alone)
    assert torch.equal(again, out)                                                # the same bits every time


@pytest.mark.parametrize("Nq", [3, 200, 490])                         # positions below 900: see the cache moved there
def test_rows_that_see_nothing(q, ora, Nq):
    """Padding rows (negative positions), and causal rows before every key:
    zeros, and no weight given."""
    pos = torch.arange(Nq).repeat(2, 1) + 400
    pos[0, 0], pos[1, 1:] = -1, -7
    pos[0, 2] = 2                                       # sees the keys at positions 0 .. 2 only
    case = Case(q, ora, seed=5, B=2, Nq=Nq, Nk=390, Nt=4, causal=True, q_pos=pos, group=2)
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    check_weights(case, q.attention_weights(case.kp, **case.args()))
    case.k_pos = torch.arange(case.Nk).repeat(case.H, 1) + 900      # all of the prefix lies ahead; the tail does not
    case.tables = q.rope_tables(2000)
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    out = q.attention_weights(case.kp, **case.args())
    assert torch.count_nonzero(out) == 0
    case = Case(q, ora, seed=6, B=1, Nq=Nq, Nk=300, q_pos=torch.full((1, Nq), -1))
    assert torch.count_nonzero(q.attention_batch(case.kp, case.vp, **case.args())) == 0
    assert torch.count_nonzero(q.attention_weights(case.kp, **case.args())) == 0


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq", [2, 40, 300])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_padding_rows_may_hold_anything(q, ora, Nq, causal, fill):
    """Queries of padding rows that nobody wrote, and of rows before every key:
    the other rows and the weights are what they are without them."""
    pos = torch.arange(Nq).repeat(2, 1) + 700
    pos[0, 0], pos[1, Nq // 2:] = -1, -5
    case = Case(q, ora, seed=41, H=2, B=2, Nq=Nq, Nk=700, Nt=6, causal=causal, q_pos=pos, group=2, T=2)
    if causal:                                          # a row before every key: the cache moved behind it
        case.k_pos = torch.arange(case.Nk).repeat(case.H, 1) + 3
        case.tail_pos = case.tail_pos + 3
        case.tail.pos = case.tail_pos.cuda()
        pos[0, 1] = 2
    calls = (lambda: q.attention_batch(case.kp, case.vp, **case.args()), lambda: q.attention_weights(case.kp, **case.args()))
    O, W = (f() for f in calls)
    check_attention(case, O)
    check_weights(case, W)
    unseen = (pos < 0) | (causal & (pos < 3))
    case.Q = torch.where(unseen[:, None, :, None], fill, case.Q)
    O2, W2 = (f() for f in calls)
    assert torch.equal(O, O2) and torch.equal(W, W2)


@pytest.mark.parametrize("kw", [dict(Nk=32), dict(Nk=64, Nq=5, B=2, group=2), dict(Nk=40, Nq=50, T=2), dict(Nk=63, Nq=300, gaps=True),
                                dict(Nk=1, Nq=33, B=3, T=3, G=8), dict(Nk=17, B=20, group=4, T=6, K=32)],
                         ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_one_range_needs_no_joining(q, ora, kw):
    """So few keys that a row's CTA writes O itself; some rows see nothing."""
    B, Nq = kw.get("B", 1), kw.get("Nq", 1)
    pos = torch.randint(0, 2 * kw["Nk"], (B, Nq), generator=torch.Generator().manual_seed(2))
    if Nq > 1:
        pos[:, ::4] = -3
    case = Case(q, ora, seed=29, causal=True, q_pos=pos, **kw)
    case.tables = q.rope_tables(4 * kw["Nk"] + 100)     # to cover every position above
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    check_weights(case, q.attention_weights(case.kp, **case.args()))


@pytest.mark.parametrize("Nq", [1, 300, 1500])
def test_large_scores_and_far_positions(q, ora, Nq):
    """Scores of several tens (a weight near 1 at one key), and a cache whose
    positions lie far out in the tables."""
    case = Case(q, ora, seed=8, Nk=640, Nq=Nq, B=2, T=1, K=64, spread=2.0, q_scale=3.0)
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    check_weights(case, q.attention_weights(case.kp, **case.args()))
    case = Case(q, ora, seed=9, Nk=640, Nq=Nq, T=1, K=64, gaps=True)
    case.k_pos += 500_000
    case.q_pos = case.q_pos + 500_000
    case.tables = q.rope_tables(510_000)
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    check_weights(case, q.attention_weights(case.kp, **case.args()))


@pytest.mark.parametrize("Nq", [1, 5, 400])
def test_small_keys_and_large_queries(q, ora, Nq):
    """Keys of a few thousandths and queries of some hundreds: the rounding of a
    key's low half is absolute there."""
    case = Case(q, ora, seed=67, Nk=900, Nq=Nq, B=2, T=1, K=64, mode=1, spread=2.0 ** -9, q_scale=300.0)
    case.kp.scale.fill_(0x01)                           # 2^-9
    case.Kh = rebuilt(ora, case.kp)
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    check_weights(case, q.attention_weights(case.kp, **case.args()))


@pytest.mark.parametrize("Nq", [5, 400])
def test_keys_beyond_fp16_saturate(q, ora, Nq, monkeypatch):
    """A quarter of the keys' rotated channels beyond 65504: attention is that of the clipped ones."""
    import sys
    case = Case(q, ora, seed=71, Nk=900, Nq=Nq, B=2, T=1, K=64, mode=1, spread=6e4, q_scale=2e-5)
    O = q.attention_batch(case.kp, case.vp, **case.args())
    plain = rotated
    assert 0.15 < (np.abs(plain(case.Kh[0], np.arange(case.Nk))) > 65504).mean() < 0.4
    monkeypatch.setattr(sys.modules[__name__], "rotated", lambda x, pos: np.clip(plain(x, pos), -65504, 65504))
    check_attention(case, O)


@pytest.mark.parametrize("kw", [
    dict(H=1, Nk=20000),                                                          # as many ranges as one head is cut into
    dict(H=1, Nk=9000, Nq=3, Nt=9000, causal=True),                               # of the prefix and of the tail
    dict(H=1, Nk=20000, Nq=70),
    dict(H=1, Nk=20, Nq=65, Nt=66000),                                            # a tail much longer than the prefix
    dict(H=1, Nk=9000, Nq=10, B=7, Nt=9000, lens=[9000, 0, 1, 4500, 64, 65, 8999]),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items() if k != "lens"))
def test_few_heads_are_cut_into_many_ranges(q, ora, kw):
    case = Case(q, ora, seed=len(str(kw)), **kw)
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    check_weights(case, q.attention_weights(case.kp, **case.args()))
    assert q.workspace_status(case.tables) == 0


@pytest.mark.parametrize("kw", [
    dict(H=12, Nk=100, Nq=1111),                                                  # one range: O by the CTA that has the rows
    dict(H=12, Nk=100, Nq=1025, Nt=3),                                            # and a tail's: a single row in the last block
    dict(H=1, Nk=12800, Nq=159, causal=True),                                     # cut into ranges, 31 rows behind a tile
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_last_warps_with_fewer_rows_than_lanes(q, ora, kw):
    case = Case(q, ora, seed=59, T=2, **kw)
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    check_weights(case, q.attention_weights(case.kp, **case.args()))
    assert q.workspace_status(case.tables) == 0


@pytest.mark.parametrize("kw", [
    dict(Nk=2000, Nq=130, B=2, Nt=130, lens=[130, 77], T=2, K=64, causal=True, gaps=True),      # tiles of prefix and tails
    dict(Nk=3200, Nq=20, B=4, group=2, Nt=40, lens=[40, 0, 7, 39], T=1),                        # tails of few rows
    dict(Nk=6000, Nq=300, T=2),                                                                # one head alone has tiles, too
    dict(Nk=90, Nq=900, B=2),                                                                  # sums by key in cuts of the rows
    dict(Nk=3000, Nq=3, B=2, Nt=70, lens=[70, 1], T=3, G=8),
    dict(Nk=3000, Nt=9, causal=True),
], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items() if k != "lens"))
def test_smaller_workspaces_take_fewer_heads_at_a_time(q, ora, kw):
    """From what a call asks for down to what it asks for with one head: the same
    formula for every head, and not a byte behind the workspace is written.  Five
    heads go in groups of 5, of 3 and 2, of 2, 2 and 1, and one by one."""
    case = Case(q, ora, seed=61, H=5, **kw)
    for call, size, check in (
            (lambda ws: q.attention_batch(case.kp, case.vp, workspace=ws, **case.args()), q.attention_batch_workspace_bytes, check_attention),
            (lambda ws: q.attention_weights(case.kp, workspace=ws, **case.args()), q.attention_weights_workspace_bytes, check_weights)):
        full, least = (size(case.cfg, case.Nk, H, case.B, case.group, case.Nq, case.Nt) for H in (5, 1))
        assert 0 < least <= full
        for n in sorted({full, full - 1, full * 3 // 4, full // 2, full * 2 // 5, full // 4, least}, reverse=True):
            n = max(n, least)
            room = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
            out = call(room[:n])
            assert torch.all(room[n:] == 0xA5)
            check(case, out)
        with pytest.raises(q.QvgError) as e:
            call(torch.empty(16, dtype=torch.uint8, device="cuda"))
        assert e.value.status == 6
    assert q.workspace_status(case.tables) == 0


def test_heads_that_do_not_go_at_once_go_in_equal_groups(q):
    """32 heads whose tiles or scores fit the workspace 29 or 31 at a time go as 16
    and 16: what they ask for is what 16 heads do."""
    cfg = q.config(K=256, T=2, group_size=64)
    for size, Nk, rows in ((q.attention_batch_workspace_bytes, 66_000, 256), (q.attention_batch_workspace_bytes, 70_000, 1560),
                           (q.attention_weights_workspace_bytes, 70_000, 1560), (q.attention_weights_workspace_bytes, 140_000, 64)):
        two, one = (size(cfg, Nk, H, 1, 1, rows) for H in (32, 16))
        assert 0 < two == one


def test_every_sequence_alone_gives_the_same(q, ora):
    """A batch of sequences gives each row what it gets alone, within the
    rounding of the weights against other running maxima."""
    case = Case(q, ora, seed=11, B=4, Nq=60, Nk=1500, Nt=20, T=2, K=64, lens=[20, 0, 7, 13])
    O = q.attention_batch(case.kp, case.vp, **case.args())
    args = case.args()
    for b in range(4):
        t = q.Tail(k=case.tail.k[b:b + 1], v=case.tail.v[b:b + 1], pos=case.tail.pos[b:b + 1], length=case.tail.length[b:b + 1])
        one = q.attention_batch(case.kp, case.vp, args["Q"][b:b + 1], args["q_pos"][b:b + 1], case.tables, tail=t)
        assert (one.float() - O[b:b + 1].float()).abs().max() <= 2.0 ** -6 * O.float().abs().max()


@pytest.mark.parametrize("Nq", [2, 300, 700])
def test_other_streams_and_captured_graphs(q, ora, Nq):
    """The calls on a side stream, and captured into two graphs with workspaces
    of their own that replay at the same time, give the bits of the eager call."""
    case = Case(q, ora, seed=13, B=2, Nq=Nq, Nk=900, Nt=8, T=2, K=64)
    args = case.args()
    O = q.attention_batch(case.kp, case.vp, **args)
    W = q.attention_weights(case.kp, **args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    O1 = q.attention_batch(case.kp, case.vp, **args, stream=side)
    W1 = q.attention_weights(case.kp, **args, stream=side)
    side.synchronize()
    assert torch.equal(O, O1) and torch.equal(W, W1)
    graphs = []
    sizes = (case.cfg, case.Nk, case.H, case.B, case.group, case.Nq, case.Nt)
    for _ in range(2):
        ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
              (q.attention_batch_workspace_bytes(*sizes), q.attention_weights_workspace_bytes(*sizes))]
        o, w = torch.zeros_like(O), torch.zeros_like(W)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            q.attention_batch(case.kp, case.vp, **args, O=o, workspace=ws[0])
            q.attention_weights(case.kp, **args, out=w, workspace=ws[1])
        graphs.append((gr, o, w, ws))
    streams_ = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (gr, *_), s in zip(graphs, streams_):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for _, o, w, _ws in graphs:
        assert torch.equal(O, o) and torch.equal(W, w)
    assert q.workspace_status(case.tables) == 0


def test_the_batch_agrees_with_qvg_attention(q, ora):
    """One sequence, one query head to each K/V head, no tail: the same formula
    as qvg_attention, within both calls' bf16 roundings."""
    case = Case(q, ora, seed=17, H=2, Nq=200, Nk=1500, T=2, K=64)
    O = q.attention_batch(case.kp, case.vp, **case.args())
    P = q.attention(case.kp, case.vp, case.Q[0].cuda(), case.q_pos[0].cuda(), case.tables)
    check_attention(case, O)
    assert (O[0].float() - P).abs().max() <= 2.0 ** -6 * P.abs().max()


def test_a_recorded_timeout_and_a_failed_launch_are_reported(q, ora, monkeypatch):
    """The status word that a kernel's expired wait would leave in the tables is
    reported by the calls whose kernels wait, until it is read; few rows wait for
    nothing and go on."""
    case = Case(q, ora, seed=19, H=2, Nq=300, Nk=3000)
    few = dict(case.args(), Q=case.Q[:, :, :2].contiguous().cuda(), q_pos=case.q_pos[:, :2].contiguous().cuda())
    want = q.attention_batch(case.kp, case.vp, **few)
    case.tables[:4] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8)
    for call in (lambda: q.attention_batch(case.kp, case.vp, **case.args()), lambda: q.attention_weights(case.kp, **case.args())):
        torch.cuda.synchronize()
        with pytest.raises(q.QvgError) as e:
            call()
        assert e.value.status == 5
    assert torch.equal(q.attention_batch(case.kp, case.vp, **few), want)
    assert q.workspace_status(case.tables) == 5 and q.workspace_status(case.tables) == 0
    check_attention(case, q.attention_batch(case.kp, case.vp, **case.args()))
    monkeypatch.setenv("QVG_FAULT_INJECT", "stream")
    w = torch.rand((2, 3000), device="cuda")
    for call in (lambda: q.attention_batch(case.kp, case.vp, **case.args()), lambda: q.attention_weights(case.kp, **case.args()),
                 lambda: q.evict(case.kp, case.vp, w, 100)):
        with pytest.raises(q.QvgError) as e:
            call()
        assert e.value.status == 4
    torch.cuda.synchronize()


def test_weights_survive_a_recorded_timeout(q, ora):
    """A captured call looks at no status word on the host.  Once an expired wait
    is recorded its kernels leave the weights received before as they are, in
    place or not; cleared, the next replay adds them again."""
    for kw in (dict(H=2, Nq=300, Nk=3000), dict(H=1, Nq=1500, Nk=66, B=2, Nt=4)):       # the second: sums by key in cuts of the rows
        case = Case(q, ora, seed=43, **kw)
        received = torch.rand((case.H, case.Nk), generator=torch.Generator().manual_seed(4)).cuda()
        want = q.attention_weights(case.kp, received=received, **case.args())
        args, inplace, out, alone = case.args(), received.clone(), torch.full_like(received, 7.0), torch.full_like(received, 7.0)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            q.attention_weights(case.kp, received=inplace, out=inplace, **args)
            q.attention_weights(case.kp, received=received, out=out, **args)
            q.attention_weights(case.kp, out=alone, **args)
        case.tables[:4] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(inplace, received) and torch.equal(out, received) and torch.count_nonzero(alone) == 0
        assert q.workspace_status(case.tables) == 5 and q.workspace_status(case.tables) == 0
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(inplace, want) and torch.equal(out, want)
        check_weights(case, alone)


def test_packed_streams_on_another_device_are_refused(q, ora):
    import dataclasses
    case = Case(q, ora, seed=53, H=2, Nk=200, T=2)
    w = torch.rand((2, 200), device="cuda")
    for name in ("scale", "zero", "assign", "centroids"):
        p = dataclasses.replace(case.kp, **{name: getattr(case.kp, name).cpu()})
        for call in (lambda: q.attention_batch(p, case.vp, **case.args()), lambda: q.attention_batch(case.kp, p, **case.args()),
                     lambda: q.attention_weights(p, **case.args()), lambda: q.evict(p, case.vp, w, 50), lambda: q.dequantize(p)):
            with pytest.raises(q.QvgError) as e:
                call()
            assert e.value.status == 1 and name in str(e.value)


def test_two_threads_at_once(q, ora):
    """Calls from two threads on streams of their own give the bits of one."""
    import threading
    cases = [Case(q, ora, seed=23 + i, H=2, Nq=n, Nk=2500, Nt=8, T=2, K=64) for i, n in enumerate((3, 400))]
    args = [c.args() for c in cases]
    call = [lambda c=c, a=a, **kw: (q.attention_batch(c.kp, c.vp, **a, **kw), q.attention_weights(c.kp, **a, **kw)) for c, a in zip(cases, args)]
    want = [f() for f in call]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i].append(call[i](stream=s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))


@pytest.mark.parametrize("Nq", [1, 24, 400])
def test_a_side_stream_leaves_the_current_one_s_blocks_alone(q, ora, Nq):
    """A block that the current stream has let go of while its work is still
    queued is not what a call on another stream gets; the results are those of
    the current stream, with work of both queued at once."""
    case = Case(q, ora, seed=47, B=2, Nq=Nq, Nk=3000, Nt=8, T=2, K=64)
    args = case.args()
    w = torch.rand((case.H, case.Nk), device="cuda")
    calls = [lambda **kw: q.attention_batch(case.kp, case.vp, **args, **kw), lambda **kw: q.attention_weights(case.kp, **args, **kw),
             lambda **kw: q.evict(case.kp, case.vp, w, 1500, **kw).k.codes]
    want = [f() for f in calls]
    sizes = (case.cfg, case.Nk, case.H, case.B, case.group, case.Nq, case.Nt)
    need = (q.attention_batch_workspace_bytes(*sizes), q.attention_weights_workspace_bytes(*sizes), 1 << 20)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for f, r, n in zip(calls, want, need):
        held = torch.empty(n, dtype=torch.uint8, device="cuda")
        at = held.data_ptr()
        torch.cuda._sleep(2_000_000)
        held.fill_(255)
        del held
        got = f(stream=side)
        assert not at <= got.data_ptr() < at + n
        assert torch.empty(n, dtype=torch.uint8, device="cuda").data_ptr() == at      # it is still the current stream's
        torch.cuda.synchronize()
        assert torch.equal(got, r)
    for _ in range(10):                                 # both streams, and results freed while they are read
        a = [f() for f in calls]
        b = [f(stream=side) for f in calls]
        c = [f(stream=side.cuda_stream) for f in calls]
        torch.cuda.current_stream().wait_stream(side)
        same = [torch.equal(x, r) for g in (a, b, c) for x, r in zip(g, want)]
        del a, b, c
        assert all(same)


# ------------------------------------------------------------------ eviction

def kept_plain(w, keep, first, recent):
    """The kept indices of one head, from the definition."""
    n = len(w)
    key = np.where(np.isnan(w), -np.inf, w.astype(np.float64))
    order = sorted(range(first, n - recent), key=lambda i: (-key[i], not np.isnan(w[i]) and 0 or int(np.isnan(w[i])), i))
    return np.sort(np.array(list(range(first)) + order[:keep - first - recent] + list(range(n - recent, n)), np.int64))


def check_evict(q, kp, vp, w, keep, first, recent, k_pos=None):
    e = q.evict(kp, vp, w, keep, first=first, recent=recent, k_pos=k_pos)
    torch.cuda.synchronize()
    wn = w.cpu().numpy()
    for h in range(kp.H):
        want = torch.from_numpy(kept_plain(wn[h], keep, first, recent)).cuda()
        assert torch.equal(e.kept[h].long(), want), h
        assert torch.equal(e.pos[h], want if k_pos is None else k_pos[h][want])
        assert torch.equal(e.weights[h].view(torch.int32), w[h][want].view(torch.int32))
        for a, p in ((e.k, kp), (e.v, vp)):
            assert torch.equal(a.codes[h], p.codes[h][want]) and torch.equal(a.scale[h], p.scale[h][want])
            if p.cfg.scale_mode == 0:
                assert torch.equal(a.zero[h], p.zero[h][want])
            assert torch.equal(a.assign[:, h], p.assign[:, h][:, want])
            assert a.centroids is p.centroids and a.N == keep
    return e


@pytest.mark.parametrize("H,N,keep,first,recent,T,G,mode", [
    (1, 1, 1, 0, 0, 1, 64, 0), (2, 2, 1, 0, 1, 0, 32, 0), (1, 3, 3, 1, 1, 2, 64, 0), (2, 37, 20, 4, 16, 1, 8, 0),
    (3, 500, 376, 4, 32, 2, 16, 1), (2, 1025, 1, 0, 0, 4, 128, 0), (1, 4097, 4000, 7, 100, 8, 128, 1),
    (2, 10240, 5000, 0, 0, 1, 64, 0),           # the shared memory of a head's weights just above 40 KB
    (2, 12289, 5001, 3, 9, 3, 32, 0), (1, 49152, 30000, 11, 13, 1, 64, 1), (2, 60001, 777, 5, 10, 2, 64, 0), (2, 300, 123, 5, 10, 0, 32, 0),
])
def test_evict_matches_the_definition(q, H, N, keep, first, recent, T, G, mode):
    g = torch.Generator().manual_seed(N + keep)
    cfg = q.config(K=16, T=T, group_size=G, scale_mode=mode)
    kp, vp = streams(q, g, cfg, H, N), streams(q, g, cfg, H, N)
    w = (torch.randn((H, N), generator=g) * 2).exp()
    w[:, N // 2:N // 2 + N // 5] = 0.0                          # many equal weights
    k_pos = (torch.cumsum(torch.randint(1, 9, (H, N), generator=g), 1)).cuda()
    check_evict(q, kp, vp, w.cuda(), keep, first, recent, k_pos)
    check_evict(q, kp, vp, w.cuda(), keep, first, recent)


@pytest.mark.parametrize("seed", range(3))
def test_evict_orders_every_kind_of_weight(q, seed):
    """Negative weights, infinities, NaN (below everything), both zeros (equal),
    subnormals, ties at the border; all equal."""
    g = torch.Generator().manual_seed(seed)
    N = 777
    cfg = q.config(K=16, T=1, group_size=64)
    kp, vp = streams(q, g, cfg, 2, N), streams(q, g, cfg, 2, N)
    kinds = torch.tensor([0.0, -0.0, 1.0, -1.0, float("inf"), -float("inf"), float("nan"), 1e-42, -1e-42, 3.5, 1e38, -1e38])
    w = kinds[torch.randint(0, len(kinds), (2, N), generator=g)]
    for keep, first, recent in ((1, 0, 0), (300, 0, 0), (N - 1, 0, 0), (N, 3, 4), (500, 100, 400), (411, 17, 0)):
        check_evict(q, kp, vp, w.cuda(), keep, first, recent)
    check_evict(q, kp, vp, torch.full((2, N), 2.5).cuda(), 100, 10, 10)
    check_evict(q, kp, vp, torch.full((2, N), float("nan")).cuda(), 100, 10, 10)


def test_evict_of_many_heads(q):
    """So many heads that a head has one CTA, and more tokens than its shared
    memory holds weights of."""
    g = torch.Generator().manual_seed(1)
    H, N = 80, 49_200
    cfg = q.config(K=16, T=1, group_size=128, scale_mode=1)
    kp = streams(q, g, cfg, H, N)
    w = torch.rand((H, N), generator=g)
    w[:, ::3] = 0.25
    check_evict(q, kp, kp, w.cuda(), 30_001, 100, 200)


def test_evict_of_more_heads_than_a_grid_is_high(q):
    g = torch.Generator().manual_seed(4)
    H, N = 70_000, 5
    kp = streams(q, g, q.config(K=16, T=0, group_size=128, scale_mode=1), H, N)
    w = torch.argsort(torch.rand((H, N), generator=g), dim=1).float().cuda()      # a permutation of 0 .. 4 each
    e = q.evict(kp, kp, w, 2, first=1)
    best = w[:, 1:].argmax(1) + 1
    assert torch.equal(e.kept.long(), torch.stack([torch.zeros_like(best), best], 1))
    assert torch.equal(e.k.codes, torch.gather(kp.codes, 1, e.kept.long()[:, :, None].expand(-1, -1, D // 4)))
    assert torch.equal(e.v.scale, torch.gather(kp.scale, 1, e.kept.long()[:, :, None]))


def test_evict_on_another_stream_and_captured(q):
    g = torch.Generator().manual_seed(2)
    cfg = q.config(K=16, T=2, group_size=64)
    kp, vp = streams(q, g, cfg, 2, 9000), streams(q, g, cfg, 2, 9000)
    w = [torch.rand((2, 9000), generator=g).cuda() for _ in range(2)]
    want = [q.evict(kp, vp, x, 5000, first=3, recent=70) for x in w]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    e = q.evict(kp, vp, w[0], 5000, first=3, recent=70, stream=side)
    side.synchronize()
    assert torch.equal(e.kept, want[0].kept) and torch.equal(e.v.codes, want[0].v.codes)
    now = w[0].clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        e = q.evict(kp, vp, now, 5000, first=3, recent=70)
    for x, r in zip(w, want):
        now.copy_(x)
        gr.replay()
        torch.cuda.synchronize()
        for a, b in ((e.kept, r.kept), (e.pos, r.pos), (e.weights, r.weights), (e.k.codes, r.k.codes), (e.k.assign, r.k.assign),
                     (e.v.scale, r.v.scale), (e.v.zero, r.v.zero)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits(q):
    """The last head of a cache of more than 4 GiB of codes gives the bits that
    it gives alone."""
    H, N = 18, 8_000_000
    cfg = q.config(K=16, T=1, group_size=128, scale_mode=1)
    g = torch.Generator(device="cuda").manual_seed(3)
    big = q.alloc_packed(cfg, N, H)
    assert big.codes.numel() > 1 << 32
    big.codes.random_(0, 256, generator=g)
    big.scale.fill_(0x28)                               # 2^-2
    big.assign.random_(0, 16, generator=g)
    big.centroids.normal_(generator=g)
    one = q.Packed(codes=big.codes[-1:], scale=big.scale[-1:], zero=big.zero, assign=big.assign[:, -1:],
                   centroids=big.centroids[:, -1:], cfg=cfg, N=N, H=1, d=D, dtype=q.BF16)
    tables = q.rope_tables(N + 200)
    for Nq in (1, 16, 80):
        Q = torch.randn((1, H, Nq, D), generator=g, device="cuda").to(torch.bfloat16)
        pos = (N + torch.arange(Nq, device="cuda")).reshape(1, -1)
        O = q.attention_batch(big, big, Q, pos, tables)
        alone = q.attention_batch(one, one, Q[:, -1:].contiguous(), pos, tables)
        # cut into other ranges: the weights round against other references
        assert (O[0, -1].float() - alone[0, 0].float()).abs().max() <= 2.0 ** -6 * alone.float().abs().max()
        W = q.attention_weights(big, Q, pos, tables)
        alone = q.attention_weights(one, Q[:, -1:].contiguous(), pos, tables)
        assert (W[-1] - alone[0]).abs().max() <= 1e-5 * alone.max()
        del O, alone
    w = torch.rand((H, N), generator=g, device="cuda")
    e = q.evict(big, big, w, 1_000_000)
    a = q.evict(one, one, w[-1:].contiguous(), 1_000_000)
    assert torch.equal(e.kept[-1], a.kept[0]) and torch.equal(e.k.codes[-1], a.k.codes[0]) and torch.equal(e.k.assign[:, -1], a.k.assign[:, 0])
    assert torch.equal(e.weights[-1], a.weights[0])
    assert q.workspace_status(tables) == 0


def test_attend_accumulate_evict_together(q, ora):
    """A cache kept within a budget, as it would be used: chunks are quantised
    once, every step attends and adds up the weights, and eviction thins the
    cache, after which the kept tokens are read at their own positions."""
    from bit_kv_cache_qvg_b200 import synth
    cfg = q.config(K=64, T=2, group_size=64, iters=3)
    H, N = 2, 1560
    X = [synth.block_batch(H, synth.KVShape(1, 30, 52), seed=s, kinds=[kind] * H).cuda() for s, kind in ((31, 0), (32, 1))]
    kp, vp = q.quantize(X[0], cfg), q.quantize(X[1], cfg)
    pos, got = None, None
    case = Case.__new__(Case)
    for step, keep in enumerate((1200, 777, 300)):
        g = torch.Generator().manual_seed(step)
        case.cfg, case.kp, case.vp, case.H, case.group, case.B, case.Nq, case.Nk = cfg, kp, vp, H, 2, 2, 30, kp.N
        case.Nt, case.lens, case.causal = 30, [30, 12], True
        case.Q = (torch.randn((2, H * 2, 30, D), generator=g) * 0.05).to(torch.bfloat16)
        case.tk, case.tv = (torch.randn((2, H, 30, D), generator=g).to(torch.bfloat16) for _ in range(2))
        case.tail_pos = N + 30 * step + torch.arange(30).repeat(2, 1)
        case.q_pos = case.tail_pos.clone()
        case.q_pos[1, 12:] = -1
        case.k_pos = None if pos is None else pos.cpu()
        case.tail = q.Tail(k=case.tk.cuda(), v=case.tv.cuda(), pos=case.tail_pos.cuda(),
                           length=torch.tensor([30, 12], dtype=torch.int32).cuda())
        case.tables = q.rope_tables(2000)
        case.Kh, case.Vh = rebuilt(ora, kp), rebuilt(ora, vp)
        check_attention(case, q.attention_batch(kp, vp, **case.args()))
        out = q.attention_weights(kp, received=got, **case.args())
        check_weights(case, out, got)
        e = check_evict(q, kp, vp, out, keep, 16, 64, pos)
        before = q.dequantize(kp)
        kp, vp, pos, got = e.k, e.v, e.pos, e.weights
        for h in range(H):
            assert torch.equal(q.dequantize(kp)[h], before[h][e.kept[h].long()])
