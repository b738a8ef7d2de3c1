"""GPU tests of the eviction operators at the edges of their range: values and queries of
extreme size, blocks that are not there, queries that are not numbers, long contexts."""
import numpy as np
import pytest
import torch

import workloads as W
from evict_util import check_weights, weight_tolerance, weights_reference
from parity_util import check_attention
from workloads import bf16_bits

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _cuda(*a):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in a]


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


class Seq:
    """One sequence of keys and values [L][Hkv][d] (bf16) in a cache of its own, and the
    oracle's rows of the same tokens (float64)."""

    def __init__(self, tq, orc, K, V, kind="tq", spare=0):
        L, Hkv, d = K.shape
        nblk = (L + 15) // 16
        self.cache = tq.Cache(nblk + spare, Hkv, d, rotate=kind != "unrotated", bf16=kind == "bf16")
        self.cache.data.fill_(0xFF)  # what lies behind the tokens reaches nothing
        slots = np.arange(L, dtype=np.int32)
        st = _status()
        tq.quantize_append(K.cuda(), V.cuda(), *_cuda(slots), self.cache, status=st)
        assert int(st.item()) == 0
        self.bt = torch.arange(nblk, dtype=torch.int32, device="cuda").view(1, nblk)
        self.lens = torch.tensor([L], dtype=torch.int32, device="cuda")
        if kind == "bf16":
            self.K, self.V = K.double().numpy()[None], V.double().numpy()[None]
            return
        rec = np.zeros((nblk, Hkv, orc.record_bytes(d)), np.uint8)
        rot = kind != "unrotated"
        orc.quantize_append(bf16_bits(K), bf16_bits(V), slots, rec, rotate=rot)
        self.K, self.V = orc.dequantize(rec, Hkv, d, np.arange(nblk, dtype=np.int32)[None], np.array([L], np.int32), L,
                                        rotate=rot)


# ------------------------------------------------------------------ values of extreme size
@pytest.mark.parametrize("d,L,n,window,spans", [
    (128, 600, 40, 0, [(100, 101, 0.0, 7e4), (333, 340, -3e4, 9e4)]),  # few tokens of two steps
    (128, 600, 40, 9, [(0, 600, 0.0, 7e4)]),                           # every token
    (64, 700, 130, 5, [(695, 700, -6e4, 6e4)]),                        # only in the sight of the last rows
    (64, 700, 130, 0, [(64, 128, 0.0, 9e5), (300, 301, -6.4e4, 9e5)]),
    (128, 3000, 3, 0, [(1000, 1001, 0.0, 7e4), (2999, 3000, -3e4, 9e4)]),  # contexts cut into parts
])
def test_prefill_weights_value_ranges(tq, orc, d, L, n, window, spans):
    """Groups whose scale and zero point fit fp16 while n s + z passes 65504, beside groups of
    ordinary size: finite, and the rows that do not see such a token keep their accuracy.

    Per dim the output is off by the weights' relative error times the mean of |v|; by the
    fp16 parts of weights and values (2^-22 each, 2^-22 for the product of the low parts, and
    2^-24 for n s + z); by a step's products, 12 or, where its four records are held at a
    sixteenth, 192, cut by 2^-23 each, and the sum over L / 64 steps (2^-23 each); and by half a
    step of the low part at a sixteenth, 2^-25 x 16."""
    Hkv, G = 2, 4
    rng = np.random.default_rng(L + d)
    K = _bf16(rng.standard_normal((L, Hkv, d)))
    V = rng.standard_normal((L, Hkv, d)).astype(np.float32)
    for a, b, lo, hi in spans:
        V[a:b] = rng.uniform(lo, hi, (b - a, Hkv, d))
        V[a:b, :, :32] = rng.standard_normal((b - a, Hkv, 32))  # one group stays ordinary
        V[a:b, :, 32], V[a:b, :, 33] = lo, hi                   # one spans the range
    s = Seq(tq, orc, K, _bf16(V))
    q = _bf16(rng.standard_normal((n, Hkv * G, d)))
    qs = np.array([0, n], np.int32)
    tw = torch.zeros((1, Hkv, L), device="cuda")
    st = _status()
    out = tq.prefill_attention_weights(q.cuda(), s.cache, s.bt, s.lens, *_cuda(qs), n, d ** -0.5, tw, window=window,
                                       status=st).cpu().numpy()
    assert int(st.item()) == 0 and np.isfinite(out).all()
    qd = q.double().numpy()
    want, add = weights_reference(qd, s.K, s.V, [L], d ** -0.5, qs, window)
    tol = weight_tolerance(qd, s.K, [L], d ** -0.5, 0.0, (window or n) * G)
    check_weights(tw.cpu().numpy(), add, tol(add))
    mean_v = weights_reference(qd, s.K, np.abs(s.V), [L], d ** -0.5, qs, window)[0]
    bound = (tol(np.float64(1.0)) + 3.25 * 2.0 ** -22 + (192 + L / 64) * 2.0 ** -23) * mean_v + 2.0 ** -21
    err = np.abs(out - want)
    assert np.all(err <= bound), float(np.max(err / bound))


# ------------------------------------------------------------------ blocks that are not there
def _chunk_reference(q, K, V, L, scale, window, there):
    """fp64 attention of a chunk over the tokens that are there (bool [L]); rows that see none
    are 0 and have no vote.  q [n][Hq][d], K, V [L][Hkv][d]."""
    n, Hq, _ = q.shape
    Hkv = K.shape[1]
    out, w = np.zeros(q.shape), np.zeros((Hkv, L))
    seen = (np.arange(L)[None] <= (L - n + np.arange(n))[:, None]) & there[None]
    some = seen.any(1)
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        x = np.where(seen, q[:, h] @ K[:, kv].T * scale, -np.inf)
        p = np.where(seen, np.exp(x - np.where(some, x.max(1), 0)[:, None]), 0)
        p /= np.where(some, p.sum(1), 1)[:, None]
        out[:, h] = p @ V[:, kv]
        w[kv] += p[max(0, n - (window or n)):].sum(0)
    return out, w


@pytest.mark.parametrize("d,Hkv,G,L,n,window,bad", [
    (128, 2, 4, 400, 30, 0, [3, 24]),                       # one inside, one under the causal limits
    (128, 2, 4, 400, 30, 7, [0, 1, 2, 3]),                  # a whole step
    (64, 2, 8, 500, 100, 40, [30, 31]),                     # the last block among them
    (128, 1, 4, 64, 64, 0, [0]),                            # the first rows see no token
    (64, 1, 3, 200, 20, 0, list(range(13))),                # none is there
    (128, 2, 4, 3000, 3, 0, [90] + list(range(100, 164))),  # contexts in parts, more than a part gone
    (128, 8, 4, 3000, 3, 2, list(range(188))),
])
def test_prefill_weights_leave_absent_blocks_out(tq, orc, d, Hkv, G, L, n, window, bad):
    """Tokens of a block id outside the cache are not there: they take no part in any row's
    softmax, as in the decode."""
    rng = np.random.default_rng(L + len(bad))
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))))
    bt = s.bt.clone()
    bt[0, bad] = torch.tensor([-1 if i % 2 else s.cache.num_blocks for i in bad], dtype=torch.int32, device="cuda")
    there = np.ones(L, bool)
    for i in bad:
        there[16 * i:16 * i + 16] = False
    q = _bf16(rng.standard_normal((n, Hkv * G, d)))
    before = rng.random((1, Hkv, L)).astype(np.float32)
    tw = torch.from_numpy(before).cuda()
    st = _status()
    out = tq.prefill_attention_weights(q.cuda(), s.cache, bt, s.lens, *_cuda(np.array([0, n], np.int32)), n, d ** -0.5,
                                       tw, window=window, status=st)
    assert int(st.item()) == tq.STATUS_BAD_BLOCK
    qd = q.double().numpy()
    want, add = _chunk_reference(qd, s.K[0], s.V[0], L, d ** -0.5, window, there)
    check_attention(out.cpu().numpy(), want)
    got = tw.cpu().numpy()
    assert np.array_equal(got[..., ~there], before[..., ~there])
    tol = weight_tolerance(qd, s.K, [L], d ** -0.5, before.astype(np.float64), (window or n) * G)
    check_weights(got, before.astype(np.float64) + add, tol(add))


# ------------------------------------------------------------------ queries that are not numbers
@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("kind,d", [("tq", 128), ("tq", 64), ("unrotated", 128), ("bf16", 128), ("bf16", 64)])
def test_a_decode_query_that_is_not_a_number(tq, orc, kind, d, num_splits):
    """Its output is NaN however the context is cut, the other heads' rows are bit by bit those
    without it, and the sums are those of the other heads."""
    Hkv, G, L = 2, 5, 300
    rng = np.random.default_rng(d)
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))), kind)
    q = _bf16(rng.standard_normal((1, Hkv * G, d))).cuda()
    bad = q.clone()
    bad[0, 1, 3] = float("nan")
    bad[0, 7] = float("inf")
    lost = torch.zeros(Hkv * G, dtype=torch.bool)
    lost[1] = lost[7] = True
    good, tw = (torch.zeros((1, Hkv, L), device="cuda") for _ in range(2))
    want = tq.decode_attention_weights(q, s.cache, s.bt, s.lens, L, d ** -0.5, good, num_splits=num_splits)
    out = tq.decode_attention_weights(bad, s.cache, s.bt, s.lens, L, d ** -0.5, tw, num_splits=num_splits)
    assert torch.isnan(out[0, lost]).all() and torch.equal(out[0, ~lost], want[0, ~lost])
    total = tw.sum(-1)[0].cpu()
    assert torch.isfinite(tw).all() and torch.allclose(total, torch.tensor([G - 1.0, G - 1.0]), rtol=1e-5)


# ------------------------------------------------------------------ parts that are not numbers
@pytest.mark.parametrize("call,kind,d", [("decode", "tq", 128), ("decode", "tq", 64), ("decode", "bf16", 128),
                                         ("prefill", "tq", 128), ("prefill", "tq", 64)])
def test_a_part_without_a_sum_leaves_its_rows_without_weights(tq, orc, call, kind, d):
    """Records whose scores are not numbers, as many as one part of a cut context (what a part
    that gave up waiting leaves looks the same): their head's rows are NaN and add nothing, as
    where the context is whole, and the other head is as without them."""
    Hkv, G, L, n = 2, 4, 3000, 3
    rng = np.random.default_rng(d)
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))), kind)
    q = _bf16(rng.standard_normal((1 if call == "decode" else n, Hkv * G, d))).cuda()
    before = torch.from_numpy(rng.random((1, Hkv, L)).astype(np.float32)).cuda()

    def run(splits):
        tw = before.clone()
        if call == "decode":
            out = tq.decode_attention_weights(q, s.cache, s.bt, s.lens, L, d ** -0.5, tw, num_splits=splits)
        else:
            out = tq.prefill_attention_weights(q, s.cache, s.bt, s.lens, *_cuda(np.array([0, n], np.int32)), n,
                                               d ** -0.5, tw)
        return out, tw

    # ranges of at least one record (decode), parts of eight steps and more (prompt: from an
    # eighth of the context on, far more than one part)
    splits = 188 if call == "decode" else 0
    want, sums = run(splits)
    bad = slice(6, 7) if call == "decode" else slice(24, 120)
    if kind == "bf16":
        s.cache.data[bad, 0, :32 * d].view(torch.int16)[:] = 0x7fc0
    else:
        s.cache.data[bad, 0, 8 * d:8 * d + 32].view(torch.int16)[:] = 0x7e00
    for k in (splits, 1):
        out, tw = run(k)
        assert torch.isnan(out[:, :G]).all() and torch.equal(tw[0, 0], before[0, 0])
        if k == splits:
            assert torch.equal(out[:, G:], want[:, G:]) and torch.equal(tw[0, 1], sums[0, 1])


# ------------------------------------------------------------------ queries of extreme size
@pytest.mark.parametrize("kind", ["tq", "unrotated"])
@pytest.mark.parametrize("call", ["decode", "prefill", "prefill in parts"])
def test_queries_at_the_limit_of_fp16(tq, orc, kind, call):
    """A query is held as fp16 parts of scale log2(e) times its rotated elements.  Up to 65504
    they give the fp64 result (small keys bring the scores back to ordinary size); a row that
    passes it sets TQ_STATUS_RANGE and has no weights, and the other rows are as without it."""
    Hkv, G, d, L = 2, 4, 128, 1500 if call == "prefill in parts" else 300
    n = 3 if call == "prefill in parts" else 1 if call == "decode" else 40
    rng = np.random.default_rng(n)
    small = 2.0 ** -14
    s = Seq(tq, orc, _bf16(small * rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))), kind)
    qs = np.array([0, n], np.int32)
    # rotated elements of normal numbers stay below 5.5 here; scaled by 2^15 / 5.5, below 2^15
    scale = d ** -0.5
    q = _bf16(rng.standard_normal((n, Hkv * G, d)) * (2.0 ** 15 / 5.5 / 1.4427 / scale * 0.99))

    def run(q, status):
        tw = torch.zeros((1, Hkv, L), device="cuda")
        if call == "decode":
            return tq.decode_attention_weights(q.cuda(), s.cache, s.bt, s.lens, L, scale, tw, status=status), tw
        return tq.prefill_attention_weights(q.cuda(), s.cache, s.bt, s.lens, *_cuda(qs), n, scale, tw, status=status), tw

    st = _status()
    out, tw = run(q, st)
    assert int(st.item()) == 0
    qd = q.double().numpy()
    want, add = weights_reference(qd, s.K, s.V, [L], scale, None if call == "decode" else qs)
    check_attention(out.cpu().numpy(), want)
    tol = weight_tolerance(qd, s.K, [L], scale, 0.0, n * G)
    check_weights(tw.cpu().numpy(), add, tol(add))
    big = q.clone()
    big[0, 2] *= 64  # its largest element passes 2^16
    out2, tw2 = run(big, st)
    assert int(st.item()) == tq.STATUS_RANGE
    keep = torch.ones((n, Hkv * G), dtype=torch.bool)
    keep[0, 2] = False
    assert torch.equal(out2.cpu()[keep], out.cpu()[keep]) and torch.isfinite(tw2).all()
    # a row's weights sum to 1 as closely as each of them is good
    assert torch.allclose(tw2.sum(-1)[0].cpu(), torch.tensor([n * G - 1.0, n * G]), rtol=float(tol(np.float64(1.0))))


@pytest.mark.parametrize("num_splits", [0, 1])
@pytest.mark.parametrize("kind", ["tq", "bf16"])
def test_padded_rows_of_a_batch_may_hold_anything(tq, orc, kind, num_splits):
    """Sequences of no token beside a real one, their queries not numbers: output 0, no status, and
    sums as they were."""
    Hkv, G, L, d = 2, 4, 200, 128
    rng = np.random.default_rng(3)
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))), kind)
    q = _bf16(rng.standard_normal((4, Hkv * G, d))).cuda()
    alone, tw1 = torch.zeros((1, Hkv, L), device="cuda"), torch.full((4, Hkv, L), 3.0, device="cuda")
    want = tq.decode_attention_weights(q[2:3].contiguous(), s.cache, s.bt, s.lens, L, d ** -0.5, alone)
    q[[0, 1, 3]] = float("nan")
    q[1, 0] = float("inf")
    lens = torch.tensor([0, 0, L, 0], dtype=torch.int32, device="cuda")
    bt = torch.full((4, s.bt.shape[1]), -1, dtype=torch.int32, device="cuda")
    bt[2] = s.bt[0]
    st = _status()
    out = tq.decode_attention_weights(q, s.cache, bt, lens, L, d ** -0.5, tw1, num_splits=num_splits, status=st)
    assert int(st.item()) == 0 and torch.all(out[[0, 1, 3]] == 0) and torch.all(tw1[[0, 1, 3]] == 3.0)
    check_attention(out[2:3].cpu().numpy(), want.double().cpu().numpy())
    assert torch.allclose(tw1[2], 3.0 + alone[0], rtol=1e-5)


# ------------------------------------------------------------------ chunks outside the rows
@pytest.mark.parametrize("weights", [False, True])
def test_prefill_chunks_outside_the_rows_touch_nothing(tq, orc, weights):
    """Row offsets that no chunk can have, those whose difference leaves 32 bits among them: the
    status, and neither out nor the sums are touched."""
    Hkv, G, L, d, n = 2, 4, 100, 128, 10
    rng = np.random.default_rng(1)
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))))
    q = _bf16(rng.standard_normal((n, Hkv * G, d))).cuda()
    low, high = -2 ** 31, 2 ** 31 - 1
    for a, b in [(5, low), (9, low + 3), (low, 5), (-1, 5), (6, 5), (0, n + 1), (5, high), (high, low), (high, high)]:
        out = torch.full((n, Hkv * G, d), 7.0, device="cuda")
        tw = torch.full((1, Hkv, L), 3.0, device="cuda")
        st = _status()
        qs = _cuda(np.array([a, b], np.int32))
        if weights:
            tq.prefill_attention_weights(q, s.cache, s.bt, s.lens, *qs, n, d ** -0.5, tw, out=out, status=st)
        else:
            tq.prefill_attention(q, s.cache, s.bt, s.lens, *qs, n, d ** -0.5, out=out, status=st)
        assert int(st.item()) == tq.STATUS_BAD_LEN, (a, b)
        assert torch.all(out == 7.0) and torch.all(tw == 3.0), (a, b)


# ------------------------------------------------------------------ long contexts
def _long_reference(q, K, V, scale, window):
    """weights_reference of one sequence's last rows, in 64 bits on the device."""
    n, Hq, d = q.shape
    L, Hkv = K.shape[:2]
    K, V = (torch.from_numpy(x).cuda() for x in (K, V))
    q = q.cuda().double()
    out, w = torch.zeros((n, Hq, d), dtype=torch.float64), torch.zeros((Hkv, L), dtype=torch.float64)
    hidden = torch.ones((n, L), dtype=torch.bool, device="cuda").triu(L - n + 1)
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        p = torch.softmax((q[:, h] @ K[:, kv].T * scale).masked_fill(hidden, -np.inf), 1)
        out[:, h] = (p @ V[:, kv]).cpu()
        w[kv] += p[max(0, n - window):].sum(0).cpu()
    return out.numpy(), w.numpy()


@pytest.mark.parametrize("kind,d,num_splits", [("tq", 128, 0), ("tq", 128, 1), ("tq", 64, 0), ("unrotated", 64, 3),
                                               ("bf16", 128, 1), ("bf16", 64, 0)])
def test_decode_weights_over_a_long_context(tq, orc, kind, d, num_splits):
    """65536 tokens, where sums cut towards zero at every tensor-core step show.

    The output is near sqrt(e / L) = 0.0064 a dim (for weights that sum to 1).  Independent
    errors of the weights average as the weights themselves: their share of it is the rms of
    a weight's relative error, a score of rms 1.4 cut by 2^-24 in each of 16 steps, 2^-20 at
    most.  What does not average are the zero-point sums, 0.13 against codes of the opposite
    sign (the middle of 32 normal values, 4.14 / 30): a record's product cut by up to 2^-23,
    0.13 / 0.0064 x 2^-23 = 2.4e-6, and the rounded additions of 683 records a warp (one
    split, six warps), twice, sqrt(2) 2^-25 0.13 / 0.0064 sqrt(683 / 9 / 6) = 3e-6.  (Summed on
    in the accumulators, 683 steps cut by 2^-24: 4e-5 x 0.13 / 0.0064 = 8e-4.)  bf16 values
    have no such pair of sums; theirs are 2^-25 sqrt(1024) = 1e-6 (summed on, 2048 steps cut
    by 2^-24: 1.2e-4)."""
    L, G = 65536, 4
    rng = np.random.default_rng(L + d)
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, 1, d))), _bf16(rng.standard_normal((L, 1, d))), kind)
    q = _bf16(rng.standard_normal((1, G, d)))
    tw = torch.zeros((1, 1, L), device="cuda")
    out = tq.decode_attention_weights(q.cuda(), s.cache, s.bt, s.lens, L, d ** -0.5, tw, num_splits=num_splits)
    want, add = _long_reference(q, s.K[0], s.V[0], d ** -0.5, 1)
    err = np.linalg.norm(out.cpu().numpy() - want) / np.linalg.norm(want)
    assert err <= 1e-5, err
    tol = weight_tolerance(q.double().numpy(), s.K, [L], d ** -0.5, 0.0, G)
    check_weights(tw[0].cpu().numpy(), add, tol(add))


@pytest.mark.parametrize("d,Hkv,L,n", [(128, 1, 32768, 5), (64, 8, 16384, 600)])
def test_prefill_weights_over_a_long_context(tq, orc, d, Hkv, L, n):
    """Contexts cut into parts (few rows) and whole.  The values' sums have no large partner, so
    the output's error is that of the weights, 2^-20 at most as in the decode, and of the sums
    over up to 512 steps, 2^-25 sqrt(512) = 7e-7.  (Summed on in tensor memory, 256 steps of 12
    products cut by 2^-24: 1.8e-4 of the sum at the end.)"""
    G = 4
    rng = np.random.default_rng(L + n)
    K, V = (_bf16(rng.standard_normal((L, 1, d))).expand(L, Hkv, d).contiguous() for _ in range(2))
    s = Seq(tq, orc, K, V)
    q = _bf16(rng.standard_normal((n, Hkv * G, d)))
    tw = torch.zeros((1, Hkv, L), device="cuda")
    out = tq.prefill_attention_weights(q.cuda(), s.cache, s.bt, s.lens, *_cuda(np.array([0, n], np.int32)), n,
                                       d ** -0.5, tw, window=3)
    want, add = _long_reference(q, s.K[0], s.V[0], d ** -0.5, 3)
    err = np.linalg.norm(out.cpu().numpy() - want) / np.linalg.norm(want)
    assert err <= 1e-5, err
    tol = weight_tolerance(q.double().numpy(), s.K, [L], d ** -0.5, 0.0, 3 * G)
    check_weights(tw[0].cpu().numpy(), add, tol(add))


@pytest.mark.parametrize("kind,max_len,attended", [("tq", 208, 208), ("tq", 200, 208), ("bf16", 200, 200)])
def test_decode_weights_of_a_length_beyond_the_maximum(tq, orc, kind, max_len, attended):
    """The sequence is cut as the plain decode cuts it (the 4-bit caches at a whole block), and
    sums at or past max_seq_len keep their values."""
    Hkv, G, L, d = 2, 4, 400, 128
    rng = np.random.default_rng(7)
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))), kind)
    q = _bf16(rng.standard_normal((1, Hkv * G, d)))
    before = rng.random((1, Hkv, L)).astype(np.float32)
    tw = torch.from_numpy(before).cuda()
    st = _status()
    out = tq.decode_attention_weights(q.cuda(), s.cache, s.bt, s.lens, max_len, d ** -0.5, tw, status=st)
    assert int(st.item()) == tq.STATUS_BAD_LEN
    qd = q.double().numpy()
    want, add = weights_reference(qd, s.K, s.V, [attended], d ** -0.5)
    check_attention(out.cpu().numpy(), want)
    got = tw.cpu().numpy()
    assert np.array_equal(got[..., max_len:], before[..., max_len:])
    old = before[..., :max_len].astype(np.float64)
    tol = weight_tolerance(qd, s.K, [attended], d ** -0.5, old, G)
    check_weights(got[..., :max_len], old + add[..., :max_len], tol(add[..., :max_len]))


@pytest.mark.parametrize("d,Hkv,G,L,n,bad", [
    (128, 2, 4, 400, 30, [3, 24]),
    (128, 2, 4, 400, 30, [0, 1, 2, 3]),
    (64, 2, 8, 500, 100, [30, 31]),
    (128, 1, 4, 64, 64, [0]),
    (64, 1, 3, 200, 20, list(range(13))),
])
def test_prefill_leaves_absent_blocks_out(tq, orc, d, Hkv, G, L, n, bad):
    """The same of the prefill without weights."""
    rng = np.random.default_rng(L + len(bad))
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))))
    bt = s.bt.clone()
    bt[0, bad] = torch.tensor([-1 if i % 2 else s.cache.num_blocks for i in bad], dtype=torch.int32, device="cuda")
    there = np.ones(L, bool)
    for i in bad:
        there[16 * i:16 * i + 16] = False
    q = _bf16(rng.standard_normal((n, Hkv * G, d)))
    st = _status()
    out = tq.prefill_attention(q.cuda(), s.cache, bt, s.lens, *_cuda(np.array([0, n], np.int32)), n, d ** -0.5, status=st)
    assert int(st.item()) == tq.STATUS_BAD_BLOCK
    want, _ = _chunk_reference(q.double().numpy(), s.K[0], s.V[0], L, d ** -0.5, 0, there)
    check_attention(out.cpu().numpy(), want)


@pytest.mark.parametrize("d,L,n,spans", [
    (128, 600, 40, [(100, 101, 0.0, 7e4), (333, 340, -3e4, 9e4)]),
    (128, 600, 40, [(0, 600, 0.0, 7e4)]),
    (64, 700, 130, [(695, 700, -6e4, 6e4)]),
    (64, 700, 130, [(64, 128, 0.0, 9e5), (300, 301, -6.4e4, 9e5)]),
])
def test_prefill_value_ranges(tq, orc, d, L, n, spans):
    """The same of the prefill without weights, which sums on in tensor memory: every one of its
    products (up to 192 a step) is cut by 2^-23 of the sum so far, and weights of at least
    the largest's 1 keep 2^-25 in their two parts."""
    Hkv, G = 2, 4
    rng = np.random.default_rng(L + d)
    K = _bf16(rng.standard_normal((L, Hkv, d)))
    V = rng.standard_normal((L, Hkv, d)).astype(np.float32)
    for a, b, lo, hi in spans:
        V[a:b] = rng.uniform(lo, hi, (b - a, Hkv, d))
        V[a:b, :, :32] = rng.standard_normal((b - a, Hkv, 32))
        V[a:b, :, 32], V[a:b, :, 33] = lo, hi
    s = Seq(tq, orc, K, _bf16(V))
    q = _bf16(rng.standard_normal((n, Hkv * G, d)))
    qs = np.array([0, n], np.int32)
    st = _status()
    out = tq.prefill_attention(q.cuda(), s.cache, s.bt, s.lens, *_cuda(qs), n, d ** -0.5, status=st).cpu().numpy()
    assert int(st.item()) == 0 and np.isfinite(out).all()
    qd = q.double().numpy()
    want, _ = weights_reference(qd, s.K, s.V, [L], d ** -0.5, qs)
    mean_v = weights_reference(qd, s.K, np.abs(s.V), [L], d ** -0.5, qs)[0]
    all_v = np.zeros_like(mean_v)
    for i in range(n):
        all_v[i] = np.repeat(np.abs(s.V[0, :L - n + i + 1]).sum(0), G, 0)
    tol = weight_tolerance(qd, s.K, [L], d ** -0.5, 0.0, 0)
    bound = (tol(np.float64(1.0)) + 3.25 * 2.0 ** -22 + (L / 64 + 1) * 192 * 2.0 ** -23) * mean_v
    bound += 2.0 ** -25 * all_v + 2.0 ** -21
    err = np.abs(out - want)
    assert np.all(err <= bound), float(np.max(err / bound))


# ------------------------------------------------------------------ nothing there yet
@pytest.mark.parametrize("kind", ["tq", "bf16"])
def test_sequences_and_sums_of_no_token(tq, orc, kind):
    """Before the first token: sums of no place, lengths of 0."""
    cache = tq.Cache(4, 2, 128, bf16=kind == "bf16")
    bt = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    tw = torch.empty((3, 2, 0), device="cuda")
    st = _status()
    q = torch.randn((3, 8, 128), device="cuda").to(torch.bfloat16)
    out = tq.decode_attention_weights(q, cache, bt, lens, 0, 0.1, tw, status=st)
    kept, n = tq.evict_select(tw, lens, 0, 5, sink=1, recent=1, status=st)
    tq.compact_cache(cache, bt, lens, kept, n, status=st)
    assert int(st.item()) == 0 and torch.all(out == 0) and torch.all(kept == -1) and torch.all(n == 0)


# ------------------------------------------------------------------ captured and replayed
@pytest.mark.parametrize("L,n", [(3000, 5), (400, 300)])
def test_prefill_weights_in_a_graph(tq, orc, L, n):
    """Captured once, replayed with other lengths and queries: what the calls give one by one."""
    Hkv, G, d = 8, 4, 64
    rng = np.random.default_rng(L)
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))))
    q = torch.empty((n, Hkv * G, d), dtype=torch.bfloat16, device="cuda")
    qs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ws = torch.empty(tq.prefill_weights_workspace_bytes(1, Hkv * G, Hkv, d, n, 3), dtype=torch.uint8, device="cuda")
    out, tw = torch.empty((n, Hkv * G, d), device="cuda"), torch.empty((1, Hkv, L), device="cuda")

    def call(q, lens, qs, out, tw, ws=None):
        tq.prefill_attention_weights(q, s.cache, s.bt, lens, qs, n, d ** -0.5, tw, window=3, out=out, workspace=ws)

    lens = s.lens.clone()
    call(q.zero_(), lens, qs, out, tw.zero_(), ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q, lens, qs, out, tw, ws)
    for length, rows in ((L, n), (L - 77, n), (L, n - 4), (n, n)):
        q.copy_(_bf16(rng.standard_normal(tuple(q.shape))))
        lens.fill_(length)
        qs[1] = rows
        start = torch.rand_like(tw)
        want, sums = torch.full_like(out, 7.0), start.clone()
        call(q, lens, qs, want, sums)
        tw.copy_(start)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(tw, sums)


@pytest.mark.parametrize("d,L,n", [(128, 1290, 10), (64, 1290, 100)])
def test_prefill_weights_add_small_products_first(tq, orc, d, L, n):
    """A tensor-core step cuts its sum by 2^-24 of it on average.  A score (rms 1.44, base 2)
    takes its d / 16 <= 8 large products behind the small ones, 8 x 2^-24 x 1.44 ln 2 =
    4.8e-7 of a weight, a step's output its four, 2.4e-7; the query's parts (2^-23) and the
    exponential (2 ulp) add 2.4e-7.  (Large products first: 16 and 12 such cuts, 1.7e-6.)"""
    Hkv, G = 4, 4
    rng = np.random.default_rng(L + d)
    s = Seq(tq, orc, _bf16(rng.standard_normal((L, Hkv, d))), _bf16(rng.standard_normal((L, Hkv, d))))
    q = _bf16(rng.standard_normal((n, Hkv * G, d)))
    qs = np.array([0, n], np.int32)
    tw = torch.zeros((1, Hkv, L), device="cuda")
    out = tq.prefill_attention_weights(q.cuda(), s.cache, s.bt, s.lens, *_cuda(qs), n, d ** -0.5, tw, window=1)
    want, add = weights_reference(q.double().numpy(), s.K, s.V, [L], d ** -0.5, qs, 1)
    for got, ref in ((out, want), (tw, add)):
        err = np.linalg.norm(got.cpu().numpy() - ref) / np.linalg.norm(ref)
        assert err <= 1e-6, err
