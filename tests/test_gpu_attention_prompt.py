"""int8_attention_prompt against masked softmax attention in 64 bits.

Tolerance, per value o = sum_k w_k v_k with A = sum_k w_k |v_k|, X = scale * max_k sum_d |q_d k_kd|
and n keys:
  * the result's rounding: 2^-11 |o| (2^-25 among the subnormals);
  * the softmax weights rounded to fp16 before the second product: 2^-11 A, and
    at most 2^-25 for each weight that is subnormal there (the largest is at least 1);
  * fp32 arithmetic, a whole step 2^-23 each (the tensor cores may truncate):
    D + 8 of them on scores no larger than X, which the exponential turns into a
    relative error of the weights (numerator and sum), and n/8 + 64 in the sums over keys.
"""
import itertools

import numpy as np
import pytest
import torch

import int8_quantized_row_b200 as i8
from gpu_helpers import device_status_clean

pytestmark = pytest.mark.gpu


def cum(lens):
    return torch.tensor([0, *itertools.accumulate(lens)], dtype=torch.int32, device="cuda")


def inputs(seed, nq, nk, Hq, H, D, more=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").half()
    return rand(sum(nq) + more, Hq, D), rand(sum(nk) + more, H, D), rand(sum(nk) + more, H, D)


def definition(Q, K, V, nq, nk, scale):
    """(o, tol) in double for the rows of all sequences."""
    Hq, H, D = Q.shape[1], K.shape[1], Q.shape[2]
    G, a, c = Hq // H, 0, 0
    o = torch.zeros(sum(nq), Hq, D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    for n, m in zip(nq, nk):
        live = torch.ones(n, m, device="cuda").tril(m - n).bool()
        for h in range(Hq if m else 0):
            q, k, v = Q[a:a + n, h].double(), K[c:c + m, h // G].double(), V[c:c + m, h // G].double()
            w = torch.softmax(torch.where(live, scale * q @ k.T, -torch.inf), 1)
            w = torch.where(live, w, 0.0)
            y, A = w @ v, w @ v.abs()
            X = abs(scale) * torch.where(live, q.abs() @ k.abs().T, 0.0).amax(1, keepdim=True)
            o[a:a + n, h] = y
            tol[a:a + n, h] = (y.abs() * 2.0 ** -11 + 2.0 ** -25 + m * 2.0 ** -25 * v.abs().amax() +
                               A * (2.0 ** -11 + 2 * (D + 8) * 2.0 ** -23 * X + (m / 8 + 64) * 2.0 ** -23))
        tol[a:a + max(0, n - m)] = 0.0                             # rows that see no key
        a, c = a + n, c + m
    return o, tol


def check(O, Q, K, V, nq, nk, scale):
    o, tol = definition(Q, K, V, nq, nk, scale)
    off = (O[:len(o)].double() - o).abs()
    assert bool((off <= tol).all()), f"{(~(off <= tol)).sum().item()} of {off.numel()} off, worst {off.max().item():.3e}"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 64, 127, 128, 129, 200, 255, 256, 257, 384, 500, 1000])
def test_one_prompt(n, D):
    Q, K, V = inputs(n, [n], [n], 2, 1, D)
    O = i8.int8_attention_prompt(Q, K, V, cum([n]))
    check(O, Q, K, V, [n], [n], D ** -0.5)
    assert device_status_clean()


@pytest.mark.parametrize("Hq,H,D", [(1, 1, 64), (3, 3, 128), (6, 2, 64), (10, 2, 128), (12, 1, 128)])
def test_packed_prompts(Hq, H, D):
    n = [5, 0, 300, 1, 128, 77, 513, 0, 256, 2]
    Q, K, V = inputs(Hq, n, n, Hq, H, D)
    O = i8.int8_attention_prompt(Q, K, V, cum(n))
    check(O, Q, K, V, n, n, D ** -0.5)
    assert device_status_clean()


@pytest.mark.parametrize("B,Hq,D", [(32, 5, 64), (33, 7, 128), (150, 3, 64), (300, 2, 128), (900, 1, 64)])
def test_many_prompts(B, Hq, D):
    """More sequences than a warp has lanes, and than four each; several pieces of work for every CTA."""
    n = [(37 * b) % 190 for b in range(B)]
    n[B // 2] = 600
    nk = [a + (b % 3) * 50 for b, a in enumerate(n)]
    Q, K, V = inputs(B, n, nk, Hq, 1, D)
    O = i8.int8_attention_prompt(Q, K, V, cum(n), cum(nk))
    check(O, Q, K, V, n, nk, D ** -0.5)
    assert device_status_clean()


@pytest.mark.parametrize("D", [64, 128])
def test_keys_from_before_the_queries_and_rows_that_see_none(D):
    nq = [1, 10, 200, 300, 7, 400, 129, 64, 0]
    nk = [900, 137, 200, 428, 0, 150, 1, 700, 30]
    Q, K, V = inputs(D, nq, nk, 4, 2, D)
    O = i8.int8_attention_prompt(Q, K, V, cum(nq), cum(nk))
    check(O, Q, K, V, nq, nk, D ** -0.5)
    none = i8.int8_attention_prompt(Q, K[:0], V[:0], cum(nq), cum([0] * 9))
    assert (none == 0).all()
    assert device_status_clean()


@pytest.mark.parametrize("nq,nk,Hq,H,D", [([3000], [3000], 2, 1, 128), ([2500, 40], [4000, 40], 3, 3, 64)])
def test_long_prompts(nq, nk, Hq, H, D):
    Q, K, V = inputs(7, nq, nk, Hq, H, D)
    O = i8.int8_attention_prompt(Q, K, V, cum(nq), cum(nk))
    check(O, Q, K, V, nq, nk, D ** -0.5)
    again = i8.int8_attention_prompt(Q, K, V, cum(nq), cum(nk))
    assert torch.equal(O, again)


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0, 1e-4])
def test_scales(scale):
    n = [300, 70]
    Q, K, V = inputs(8, n, n, 2, 2, 128)
    check(i8.int8_attention_prompt(Q, K, V, cum(n), scale=scale), Q, K, V, n, n, scale)


def test_maxima_that_rise_along_the_keys():
    """Each 128 keys score far above those before: the sums are rescaled at every step."""
    n = [1000]
    Q, K, V = inputs(9, n, n, 2, 2, 64)
    Q = Q.abs()
    K = K.abs() * (1 + torch.arange(1000, device="cuda") // 100)[:, None, None].half()
    check(i8.int8_attention_prompt(Q, K, V, cum(n), scale=1.0), Q, K, V, n, n, 1.0)
    K = K.flip(0).contiguous()
    check(i8.int8_attention_prompt(Q, K, V, cum(n), scale=1.0), Q, K, V, n, n, 1.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_infinities_and_nan_that_a_row_does_not_see(D, bad):
    """Bad keys and values of other sequences and of later tokens have no effect."""
    nq, nk = [200, 300, 100], [260, 300, 90]
    Q, K, V = inputs(10, nq, nk, 4, 2, D, more=50)
    o, tol = definition(Q, K, V, nq, nk, D ** -0.5)
    # key/value head 0 (query heads 0 and 1) of these keys gets a bad value in column 3
    at = [150, 260 + 10, 260 + 200, 260 + 299, 560 + 20, 650 + 20]
    see = torch.zeros(600, dtype=torch.bool, device="cuda")
    see[150 - 60:200] = True
    see[200 + 10:500] = True
    see[500 + 20 + 10:600] = True                                  # 100 rows on 90 keys
    for t in (V, K):
        kept = t.clone()
        t[at, 0, 3] = bad
        got = i8.int8_attention_prompt(Q, K, V, cum(nq), cum(nk))[:600]
        t.copy_(kept)
        fine = (got.double() - o).abs() <= tol
        assert fine[:, 2:].all() and fine[~see].all()
        if t is V:
            assert not torch.isfinite(got[see][:, :2, 3]).any()
            fine[:, :2, 3] = True
            assert fine.all()                                      # the other columns
        elif bad != bad:
            assert torch.isnan(got[see][:, :2]).all()
    assert device_status_clean()


@pytest.mark.parametrize("D", [64, 128])
def test_all_values_bad(D):
    n = [300, 129]
    Q, K, V = inputs(15, n, n, 2, 2, D)
    got = i8.int8_attention_prompt(Q, K, torch.full_like(V, float("nan")), cum(n))
    assert torch.isnan(got).all()
    assert device_status_clean()


def test_a_nan_query_stays_in_its_row():
    n = [200, 100]
    Q, K, V = inputs(11, n, n, 2, 1, 128)
    want = i8.int8_attention_prompt(Q, K, V, cum(n))
    Q[130, 1, 7] = float("nan")
    got = i8.int8_attention_prompt(Q, K, V, cum(n))
    assert torch.isnan(got[130, 1]).all()
    got[130, 1] = want[130, 1]
    assert torch.equal(got, want)


def test_strided_rows_and_rows_behind_are_left():
    n = [100, 150]
    qkv = torch.randn(260, 3, 4, 128, device="cuda").half()
    Q, K, V = qkv[:, 0], qkv[:, 1], qkv[:, 2]
    out = torch.full((260, 4 * 128 + 64), 7.0, dtype=torch.float16, device="cuda")
    O = out[:, :512].unflatten(1, (4, 128))
    i8.int8_attention_prompt(Q, K, V, cum(n), O=O)
    check(O, Q, K, V, n, n, 128 ** -0.5)
    assert (out[250:] == 7.0).all() and (out[:, 512:] == 7.0).all()


def test_a_replayed_graph_and_another_stream():
    n = [300, 20, 130]
    Q, K, V = inputs(12, n, n, 4, 2, 128)
    cu = cum(n)
    want = i8.int8_attention_prompt(Q, K, V, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = i8.int8_attention_prompt(Q, K, V, cu, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    O = torch.zeros_like(Q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        i8.int8_attention_prompt(Q, K, V, cu, O=O)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, want)
    other = [10, 400, 40]                                          # lengths are read at replay
    cu.copy_(cum(other))
    graph.replay()
    torch.cuda.synchronize()
    check(O, Q, K, V, other, other, 128 ** -0.5)


@pytest.mark.parametrize("cu_q,cu_k", [([0, 101, 101], [0, 50, 100]), ([0, 50, 100], [0, 50, 101]),
                                       ([0, 50, 40], [0, 50, 100]), ([-1, 50, 100], [0, 50, 100]),
                                       ([0, 50, 100], [60, 50, 100])])
def test_bad_ranges_are_reported(cu_q, cu_k):
    Q, K, V = inputs(13, [100], [100], 2, 2, 64)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    i8.int8_attention_prompt(Q, K, V, dev(cu_q), dev(cu_k))
    assert i8.int8_read_and_clear_device_status() == 3
    assert device_status_clean()


def test_binding_refusals():
    Q, K, V = inputs(14, [50], [50], 4, 2, 64)
    cu, f = cum([50]), i8.int8_attention_prompt
    with pytest.raises(ValueError):
        f(Q, K, V[:20], cu)
    with pytest.raises(ValueError):
        f(Q, K[:, :, :32], V[:, :, :32], cu)
    with pytest.raises(ValueError):
        f(Q, K, V, cu, cum([20, 30]))
    with pytest.raises(ValueError):
        f(Q, K, V, cu, O=torch.empty_like(K))
    with pytest.raises(TypeError):
        f(Q, K.bfloat16(), V, cu)
    with pytest.raises(TypeError):
        f(Q, K, V, cu.long())
    with pytest.raises(i8.I8RError):
        f(Q[:, :3], K, V, cu)
    with pytest.raises(i8.I8RError):
        f(Q, K, V, cu, scale=float("nan"))
    assert f(Q[:0], K, V, cum([0])).shape == (0, 4, 64)


def test_rows_far_apart():
    """Rows 2^25 elements apart: offsets past 32 bits in every tensor."""
    n, D = 130, 64
    Q, K, V = inputs(3, [n], [n], 1, 1, D)
    wide = torch.empty(n, 2 ** 25, dtype=torch.float16, device="cuda")          # 8.7 GB
    far = [wide[:, at:at + D].view(n, 1, D) for at in (0, 2 ** 23, 2 ** 24, 3 * 2 ** 23)]
    for t, x in zip(far, (Q, K, V)):
        t.copy_(x)
    i8.int8_attention_prompt(*far[:3], cum([n]), O=far[3])
    assert torch.equal(far[3], i8.int8_attention_prompt(Q, K, V, cum([n])))
    assert device_status_clean()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("below", [24.6, 25.5])
def test_one_high_score_over_many_low_ones(D, below):
    """131072 keys that each weigh 2^-below of the first: together a tail that fp16 shows.  Weights are
    rounded with 2^7 in front, so that a rounding among the subnormals is at most 2^-32 of the largest."""
    nq, n, H = 3, 131072, 2
    Q, K, V = (torch.zeros(r, H, D, dtype=torch.float16, device="cuda") for r in (nq, n, n))
    Q[:, :, 0] = 1.0
    K[0, :, 0] = 32.0
    V[1:] = 1.0
    scale = below * np.log(2.0) / 32
    O = i8.int8_attention_prompt(Q, K, V, cum([nq]), cum([n]), scale=scale).double()
    low = torch.arange(n - nq, n, device="cuda").double()[:, None, None]                   # a row's other keys
    o = low / (2.0 ** below + low)
    X = below * np.log(2.0)
    tol = (2.0 ** -11 * o + 2.0 ** -25 + n * 2.0 ** -32 +
           o * (2.0 ** -11 + 2 * 8 * 2.0 ** -23 * X + (n / 8 + 64) * 2.0 ** -23))
    off = (O - o).abs()
    assert bool((off <= tol).all()), f"{off.max().item():.3e} off {o.max().item():.3e}, tolerance {tol.max().item():.3e}"
    assert device_status_clean()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_infinite_keys_that_a_row_sees(D, bad):
    """A score of +inf makes its row NaN; a key whose score is -inf weighs nothing."""
    nq, nk, scale = [200, 300, 100], [260, 300, 90], D ** -0.5
    Q, K, V = inputs(10, nq, nk, 4, 2, D)
    at = [150, 260 + 10, 260 + 200, 260 + 299, 560 + 20]
    worse = K.clone()
    worse[at, 0, 3] = bad
    got = i8.int8_attention_prompt(Q, worse, V, cum(nq), cum(nk)).double()
    nan = never = 0
    a = c = 0
    for n, m in zip(nq, nk):
        live = torch.ones(n, m, device="cuda").tril(m - n).bool()
        for h in range(2):                                         # the query heads of key/value head 0
            q, k, v = Q[a:a + n, h].double(), K[c:c + m, 0].double(), V[c:c + m, 0].double()
            x = torch.where(live, scale * q @ k.T, -torch.inf)
            for key in at:
                if c <= key < c + m:
                    x[:, key - c] = torch.where(live[:, key - c], q[:, 3] * bad, -torch.inf)
            if m < n:
                assert (got[a:a + n - m, h] == 0).all()
            rows = slice(max(0, n - m), n)
            w = torch.softmax(x[rows], 1)                          # NaN in a row with +inf
            X = scale * torch.where(live[rows], q[rows].abs() @ k.abs().T, 0.0).amax(1, keepdim=True)
            y, A = w @ v, w @ v.abs()
            tol = (y.abs() * 2.0 ** -11 + 2.0 ** -25 + m * 2.0 ** -25 * v.abs().amax() +
                   A * (2.0 ** -11 + 2 * (D + 8) * 2.0 ** -23 * X + (m / 8 + 64) * 2.0 ** -23))
            z = got[a:a + n, h][rows]
            lost = torch.isnan(y)
            assert torch.equal(torch.isnan(z), lost)
            assert bool(((z - y).abs() <= tol)[~lost].all())
            nan, never = nan + lost.any(1).sum().item(), never + (~lost).any(1).sum().item()
        a, c = a + n, c + m
    assert nan > 50 and never > 50
    assert device_status_clean()


def test_a_long_prefix_beside_many_short_prompts():
    """The search for work passes over lengths that no sequence has: 2^20 cached keys of one row (4096
    lengths, in 256 keys) beside 4000 short prompts take little longer than the two apart."""
    B, far, D = 4000, 1 << 20, 64
    n = [1 + b % 5 for b in range(B)]
    Q, K, V = inputs(16, [1, *n], [far, *n], 1, 1, D)
    calls = {"long": (Q[:1], K[:far], V[:far], cum([1]), cum([far])),
             "short": (Q[1:], K[far:], V[far:], cum(n), cum(n)),
             "both": (Q, K, V, cum([1, *n]), cum([far, *n]))}
    ms, out = {}, {}
    for name, args in calls.items():
        O = torch.empty_like(args[0])
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            i8.int8_attention_prompt(*args, O=O)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        ms[name], out[name] = min(times[1:]), O
    assert torch.equal(out["both"], torch.cat([out["long"], out["short"]]))
    check(out["short"], *calls["short"][:3], n, n, D ** -0.5)
    check(out["long"], *calls["long"][:3], [1], [far], D ** -0.5)
    assert ms["both"] <= 3 * (ms["long"] + ms["short"]), ms
    assert device_status_clean()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [1.0, 100.0, -100.0])
def test_scores_whose_rounding_nears_the_weights_range(D, scale):
    """Scores up to 2^26 in units of log 2, which fp32 rounds to multiples of 4, first those below 2^22: the
    keys that are far ahead of those before them are the result, one after the other."""
    n = 700
    Q, K, V = (torch.zeros(n, 1, D, dtype=torch.float16, device="cuda") for _ in range(3))
    V.copy_(inputs(17, [n], [n], 1, 1, D)[2])
    Q[:, 0, :8] = torch.linspace(90, 100, n, device="cuda")[:, None].half()
    for key, x in ((3, 8.0), (200, 300.0), (450, 600.0)):          # 100 * 600 * 8 * 100 = 2^25.5
        K[key, 0, :8] = x if scale > 0 else -x
    O = i8.int8_attention_prompt(Q, K, V, cum([n]), scale=scale)
    for a, e, key in ((3, 200, 3), (200, 450, 200), (450, n, 450)):
        want = V[key].double()
        assert bool(((O[a:e].double() - want).abs() <= want.abs() * 2.0 ** -10 + 2.0 ** -24).all()), key
    assert device_status_clean()
