"""int8_attention_decode against softmax attention over the cache's values in 64 bits.

Tolerance, per value o = sum_t w_t v_t with A = sum_t w_t |v_t|, X = scale * max_t sum_d |q_d k_td|
and n tokens:
  * the result's rounding: 2^-11 |o| (2^-25 among the subnormals);
  * the softmax weights rounded to fp16 before the second product: 2^-11 A, and
    at most 2^-25 for each weight that is subnormal there (the largest is 1);
  * fp32 arithmetic, a whole step 2^-23 each: D + 8 of them on scores no larger
    than X, which the exponential turns into a relative error of the weights
    (numerator and sum), and n/16 + 64 in the sums over tokens and pieces.
"""
import numpy as np
import pytest
import torch

import int8_quantized_row_b200 as i8
from gpu_helpers import device_status_clean

pytestmark = pytest.mark.gpu
BLOCK = 64


class Cache:
    def __init__(self, seed, lens, H, D, spare=2, spread=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-n // BLOCK) for n in lens]
        self.lens, self.H, self.D, self.blocks = lens, H, D, sum(need) + spare
        order = torch.randperm(self.blocks, generator=g, device="cuda").cpu().numpy()
        table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.unused = torch.from_numpy(order[at:].copy()).cuda()
        self.table = torch.from_numpy(table).cuda()
        shape = (self.blocks, H, BLOCK, D)
        # rows past a sequence's end hold codes too: they have to have no effect
        self.codes = [torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
        self.scale = [torch.exp(spread * torch.randn(shape[:2], generator=g, device="cuda")) for _ in range(2)]
        self.lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def args(self):
        return (*self.codes, *self.scale, self.table, self.lengths)

    def values(self, b, h):
        n = self.lens[b]
        pages = self.table[b, :-(-n // BLOCK)].long()
        return [(c[pages, h].double() * (s[pages, h].double() / 127)[:, None, None]).flatten(0, 1)[:n]
                for c, s in zip(self.codes, self.scale)]


def queries(seed, B, Hq, D):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(B, Hq, D, generator=g, device="cuda").half()


def check(O, Q, cache, scale, rows=None):
    B, Hq, D = Q.shape
    G = Hq // cache.H
    for b in range(B) if rows is None else rows:
        n = cache.lens[b]
        if n == 0:
            assert (O[b] == 0).all()
            continue
        for h in range(cache.H):
            k, v = cache.values(b, h)
            q = Q[b, h * G:(h + 1) * G].double()
            w = torch.softmax(scale * q @ k.T, 1)
            o, A = w @ v, w @ v.abs()
            X = abs(scale) * (q.abs() @ k.abs().T).amax(1, keepdim=True)
            tol = (o.abs() * 2.0 ** -11 + 2.0 ** -25 + n * 2.0 ** -25 * v.abs().amax() +
                   A * (2.0 ** -11 + 2 * (D + 8) * 2.0 ** -23 * X + (n / 16 + 64) * 2.0 ** -23))
            off = (O[b, h * G:(h + 1) * G].double() - o).abs()
            assert bool((off <= tol).all()), f"sequence {b} of {n}, head {h}: {off.max().item():.3e}"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 2), (6, 2), (16, 16), (15, 3), (8, 1), (9, 1), (24, 2), (16, 1), (17, 1),
                                  (40, 1)])
def test_lengths_around_steps_and_blocks(Hq, H, D):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 200, 128, 129]
    cache = Cache(Hq * 100 + D, lens, H, D)
    Q = queries(1, len(lens), Hq, D)
    O = i8.int8_attention_decode(Q, *cache.args(), scale=0.03)
    check(O, Q, cache, 0.03)
    assert device_status_clean()


@pytest.mark.parametrize("lens,Hq,H,D", [
    ([5000], 8, 8, 128), ([9000], 5, 1, 128), ([20000], 12, 1, 64), ([1, 12000, 3, 0, 700], 16, 4, 128),
    ([3000] * 7, 6, 6, 64), ([1000], 1, 1, 64), ([16], 1, 1, 128), ([40000], 2, 2, 128)])
def test_long_sequences_split_over_the_grid(lens, Hq, H, D):
    cache = Cache(sum(lens), lens, H, D, spread=0.3)
    Q = queries(2, len(lens), Hq, D)
    O = i8.int8_attention_decode(Q, *cache.args())
    check(O, Q, cache, D ** -0.5)
    again = i8.int8_attention_decode(Q, *cache.args())
    assert torch.equal(O.view(torch.int16), again.view(torch.int16))
    assert device_status_clean()


def test_many_short_sequences():
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(0, 90, 500)]
    cache = Cache(4, lens, 2, 64)
    Q = queries(5, 500, 4, 64)
    check(i8.int8_attention_decode(Q, *cache.args(), scale=0.05), Q, cache, 0.05)


@pytest.mark.parametrize("Hq,H,D", [(4, 4, 128), (12, 1, 128), (6, 2, 64)])
def test_one_score_far_above_the_rest_and_equal_scores(Hq, H, D):
    lens = [700, 300]
    cache = Cache(6, lens, H, D)
    Q = queries(7, 2, Hq, D)
    check(i8.int8_attention_decode(Q, *cache.args(), scale=2.0), Q, cache, 2.0)
    check(i8.int8_attention_decode(Q, *cache.args(), scale=-0.5), Q, cache, -0.5)
    check(i8.int8_attention_decode(Q, *cache.args(), scale=0.0), Q, cache, 0.0)
    zero = torch.zeros_like(Q)
    check(i8.int8_attention_decode(zero, *cache.args()), zero, cache, D ** -0.5)


def test_scales_of_very_different_size():
    # blocks of one sequence whose scales differ by many powers of ten, a zero one among them
    cache = Cache(8, [640], 2, 128)
    pages = cache.table[0].long()
    for s, top in ((cache.scale[0], 1.0), (cache.scale[1], 300.0)):
        s[pages] = top * 10.0 ** -torch.arange(10, device="cuda").float()[:, None]
        s[pages[3]] = 0.0
    Q = queries(9, 1, 2, 128)
    check(i8.int8_attention_decode(Q, *cache.args()), Q, cache, 128 ** -0.5)


def test_what_the_lengths_leave_out_has_no_effect():
    lens = [70, 0, 16, 1]
    cache = Cache(10, lens, 2, 128)
    Q = queries(11, 4, 4, 128)
    want = i8.int8_attention_decode(Q, *cache.args())
    for s in cache.scale:
        s[cache.unused] = float("nan")
    for c in cache.codes:
        c[cache.table[0, 1].long(), :, 6:] = -128           # past token 70
        c[cache.table[2, 0].long(), :, 16:] = 127
    assert torch.equal(i8.int8_attention_decode(Q, *cache.args()), want)


def test_a_nan_stays_in_its_row():
    cache = Cache(12, [500, 500], 2, 128)
    Q = queries(13, 2, 4, 128)
    want = i8.int8_attention_decode(Q, *cache.args())
    Q[0, 1, 5] = float("nan")
    got = i8.int8_attention_decode(Q, *cache.args())
    assert torch.isnan(got[0, 1]).all()
    got[0, 1] = want[0, 1]
    assert torch.equal(got, want)


def test_blocks_shared_by_sequences():
    cache = Cache(14, [200, 130], 2, 64)
    cache.table[1, :2] = cache.table[0, :2]
    Q = queries(15, 2, 2, 64)
    check(i8.int8_attention_decode(Q, *cache.args()), Q, cache, 0.125)


def test_strided_queries_and_rows_behind_are_left():
    lens = [100, 3, 40]
    cache = Cache(16, lens, 2, 128)
    qkv = torch.randn(3, 3, 4, 128, device="cuda").half()
    Q = qkv[:, 0]
    out = torch.full((4, 5, 128 + 64), 7.0, dtype=torch.float16, device="cuda")
    wide = out.view(4, -1)[:3, :512].unflatten(1, (4, 128))
    i8.int8_attention_decode(Q, *cache.args(), O=wide)
    check(wide, Q.contiguous(), cache, 128 ** -0.5)
    assert (out.view(4, -1)[3] == 7.0).all() and (out.view(4, -1)[:, 512:] == 7.0).all()


def test_replayed_graphs_that_share_a_workspace():
    """Lengths and blocks are read at replay; two captured calls may use one workspace in turn."""
    cache = Cache(17, [900, 17, 300], 2, 128)
    other = Cache(18, [5, 2000], 4, 64)
    Q, R = queries(19, 3, 6, 128), queries(20, 2, 4, 64)
    size = max(i8.int8_attention_decode_workspace_size(6, 2, 128), i8.int8_attention_decode_workspace_size(4, 4, 64))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.zeros_like(Q), torch.zeros_like(R)], []
    side = torch.cuda.Stream()
    for q, c, o in ((Q, cache, outs[0]), (R, other, outs[1])):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            i8.int8_attention_decode(q, *c.args(), O=o, workspace_buf=ws)
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        check(outs[0], Q, cache, 128 ** -0.5)
        check(outs[1], R, other, 0.125)
        cache.lens = [400, 0, 257]
        cache.lengths.copy_(torch.tensor(cache.lens))
    assert device_status_clean()


def test_another_stream():
    cache = Cache(21, [3000, 5], 2, 128)
    Q = queries(22, 2, 2, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    O = i8.int8_attention_decode(Q, *cache.args(), stream=side)
    side.synchronize()
    check(O, Q, cache, 128 ** -0.5)


def test_offsets_past_32_bits():
    H, D, blocks = 8, 128, 40000                              # 2.6 GB of codes each
    codes = [torch.zeros(blocks, H, BLOCK, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.ones(blocks, H, device="cuda") for _ in range(2)]
    cache = Cache(23, [200], H, D)
    pages = torch.tensor([39999, 39990, 33000, 2], device="cuda")
    for big, small in zip(codes + scale, cache.codes + cache.scale):
        big[pages] = small[cache.table[0].long()]
    table = pages.int()[None]
    Q = queries(24, 1, H, D)
    O = i8.int8_attention_decode(Q, *codes, *scale, table, cache.lengths)
    assert torch.equal(O, i8.int8_attention_decode(Q, *cache.args()))
    x = [torch.randn(60, H, D, device="cuda").half() for _ in range(2)]
    one = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for t, c, s in ((table, codes, scale), (cache.table, cache.codes, cache.scale)):
        i8.int8_kv_append(*x, one(0, 40), one(200), t, *c, *s)
    assert torch.equal(codes[1][2], cache.codes[1][cache.table[0, 3].long()])
    got = i8.int8_kv_gather(*codes, *scale, one(0, 240), table, 240)
    want = i8.int8_kv_gather(*cache.codes, *cache.scale, one(0, 240), cache.table, 240)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert device_status_clean()


@pytest.mark.parametrize("what", ["block", "negative block", "length", "negative length"])
def test_bad_indexes_are_reported(what):
    cache = Cache(25, [100, 300], 2, 128)
    Q = queries(26, 2, 2, 128)
    if what == "block":
        cache.table[0, 1] = cache.blocks
    if what == "negative block":
        cache.table[0, 0] = -1
    if what == "length":
        cache.lengths[0] = 64 * cache.table.shape[1] + 1
    if what == "negative length":
        cache.lengths[0] = -3
    O = i8.int8_attention_decode(Q, *cache.args())
    assert i8.int8_read_and_clear_device_status() == 3
    check(O, Q, cache, 128 ** -0.5, rows=[1])
    assert device_status_clean()


def test_binding_refusals():
    cache = Cache(27, [100], 2, 128)
    Q = queries(28, 1, 4, 128)
    f = i8.int8_attention_decode
    with pytest.raises(ValueError):
        f(Q[:, :, :64], *cache.args())
    with pytest.raises(ValueError):
        f(Q.expand(2, 4, 128), *cache.args())
    with pytest.raises(ValueError):
        f(Q, *cache.args()[:5], cache.lengths.expand(2).contiguous())
    with pytest.raises(ValueError):
        f(Q, *cache.args(), O=torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        f(Q.float(), *cache.args())
    with pytest.raises(i8.I8RError):
        f(Q[:, :3], *cache.args())                          # 3 query heads on 2 key/value heads
    with pytest.raises(i8.I8RError):
        f(Q, *cache.args(), scale=float("inf"))
    with pytest.raises(i8.I8RError):
        f(Q, *cache.args(), workspace_buf=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("low", [256, 900])
@pytest.mark.parametrize("Hq,H,D", [(4, 4, 128), (24, 2, 128), (6, 2, 64), (16, 1, 64)])
def test_queries_of_nonzero_mean_and_a_channel_that_dominates(Hq, H, D, low):
    """Scores are sums over q * code, whatever their means: with q = i / 128, i a whole number up to 1000,
    no partial sum over i * code reaches 128 * 1000 * 127 < 2^24, so that fp32 holds every one exactly.
    Left are the roundings of the score's factors and of its distance from the maximum (at most 8
    steps of 2^-23 of the largest score, in numerator and sum), the weights' and the output's 2^-11,
    and the sums over tokens."""
    scale, lens = 0.25, [1000, 64, 300, 1]
    cache = Cache(40 + Hq + D, lens, H, D)
    g = torch.Generator(device="cuda").manual_seed(low + Hq)
    K, sK = cache.codes[0], cache.scale[0]
    K.copy_((6.35 * torch.randn(K.shape, generator=g, device="cuda")).round().clamp(-127, 127))
    K[..., 3] = torch.randint(115, 128, K.shape[:-1], generator=g, device="cuda")
    sK.fill_(20.0)
    Q = (torch.randint(low, 1001, (len(lens), Hq, D), generator=g, device="cuda") / 128).half()
    O = i8.int8_attention_decode(Q, *cache.args(), scale=scale)
    G = Hq // H
    for b, n in enumerate(lens):
        for h in range(H):
            k, v = cache.values(b, h)
            x = scale * Q[b, h * G:(h + 1) * G].double() @ k.T
            w = torch.softmax(x, 1)
            o, A = w @ v, w @ v.abs()
            tol = (o.abs() * 2.0 ** -11 + 2.0 ** -25 + n * 2.0 ** -25 * v.abs().amax() +
                   A * (2.0 ** -11 + 2 * 8 * 2.0 ** -23 * x.abs().amax(1, keepdim=True) + (n / 16 + 64) * 2.0 ** -23))
            off = (O[b, h * G:(h + 1) * G].double() - o).abs()
            assert bool((off <= tol).all()), f"sequence {b}, head {h}: {(off / tol).max().item():.2f} of the tolerance"
    assert device_status_clean()


@pytest.mark.parametrize("below", [24.6, 25.5, 28.0])
@pytest.mark.parametrize("G", [1, 12])
def test_one_high_score_over_many_low_ones(G, below):
    """131072 tokens that each weigh 2^-below of the first: together a tail that fp16 shows.  Weights are
    rounded with 2^14 in front, so the smallest normal one is 2^-28 of the largest and a rounding among
    the subnormals at most 2^-39 of it."""
    n, B, H, D = 131072, 24, 4, 64
    cache = Cache(50, [n], H, D, spare=0)
    first = cache.table[0, 0].long()
    K, V = cache.codes
    K.zero_()
    V.fill_(127)
    K[first, :, 0, 0] = 127
    V[first, :, 0] = 0
    for s in cache.scale:
        s.fill_(127.0)                                       # a code stands for itself
    table, lengths = cache.table.expand(B, -1).contiguous(), cache.lengths.expand(B).contiguous()
    Q = torch.zeros(B, H * G, D, dtype=torch.float16, device="cuda")
    Q[:, :, 0] = 1.0
    scale = below * np.log(2.0) / 127
    O = i8.int8_attention_decode(Q, *cache.codes, *cache.scale, table, lengths, scale=scale).double()
    o = 127 * (n - 1) / (2.0 ** below + n - 1)
    X = below * np.log(2.0)
    tol = (2.0 ** -11 * o + 2.0 ** -25 + 127 * n * 2.0 ** -39 +
           o * (2.0 ** -11 + 2 * 8 * 2.0 ** -23 * X + (n / 16 + 64) * 2.0 ** -23))
    assert (O - o).abs().max().item() <= tol, f"{(O - o).abs().max().item():.3e} off {o:.3e}, tolerance {tol:.3e}"
    assert device_status_clean()


@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("scale", [0.01, 1.0, 6.0, -6.0])
def test_scores_whose_rounding_exceeds_the_weights_range(G, scale):
    """Scores up to 2^28.4 in units of log 2, where fp32 rounds to multiples of 32: the key that is far ahead is
    the result, whichever way its distance from the maximum is rounded."""
    n, H, D = 300, 2, 64
    cache = Cache(60, [n], H, D)
    cache.scale[0].fill_(65504.0)
    cache.codes[0].zero_()
    pages = cache.table[0].long()
    for t, code in ((77, 127), (205, -127), (276, 100)):
        cache.codes[0][pages[t // BLOCK], :, t % BLOCK] = code
    Q = torch.linspace(8, 10, H * G, device="cuda")[None, :, None].expand(1, H * G, D).half().contiguous()
    O = i8.int8_attention_decode(Q, *cache.args(), scale=scale)
    for h in range(H):
        want = cache.values(0, h)[1][77 if scale > 0 else 205]
        got = O[0, h * G:(h + 1) * G].double()
        assert bool(((got - want).abs() <= want.abs() * 2.0 ** -10 + 2.0 ** -24).all())
    assert device_status_clean()


@pytest.mark.parametrize("G,D", [(1, 64), (2, 128), (12, 128)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("which", [0, 1])
def test_a_block_whose_scale_is_not_finite_shows(G, D, bad, which):
    """Its codes stand for infinities (of both signs) and, where they are 0, NaN: no row that sees them is finite,
    the others are as before."""
    lens, H = [300, 64, 30, 700], 4
    cache = Cache(61 + D, lens, H, D)
    Q = queries(62, len(lens), H * G, D)
    want = i8.int8_attention_decode(Q, *cache.args(), scale=0.05)
    for b, block in ((0, 2), (1, 0), (3, 5)):
        cache.scale[which][cache.table[b, block].long(), b] = bad              # of head b
        cache.codes[which][cache.table[b, block].long(), b, :, ::7] = 0
    got = i8.int8_attention_decode(Q, *cache.args(), scale=0.05)
    for b in (0, 1, 3):
        rows = got[b, b * G:(b + 1) * G]
        seen = rows if which == 0 else rows[:, ::7]                            # (a column of V's own)
        assert torch.isnan(seen).all()
        assert not torch.isfinite(rows).any()
        got[b, b * G:(b + 1) * G] = want[b, b * G:(b + 1) * G]
    assert torch.equal(got, want)
    assert device_status_clean()


@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("D", [64, 128])
def test_an_infinite_key_alone_in_its_block(G, D):
    """Token 128's key holds an infinity: its block's other codes are 0, which stand for NaN, whatever the sign of
    the query where the infinity is, and whether its warp has the blocks before it or not."""
    H, n, B = 2, 129, 1200
    cache = Cache(63, [n] * B, H, D)
    x = [torch.randn(B, H, D, device="cuda").half() for _ in range(2)]
    x[0][:, 0, 5] = float("inf")
    i8.int8_kv_append(*x, torch.arange(B + 1, dtype=torch.int32, device="cuda"), cache.lengths - 1, cache.table,
                      *cache.codes, *cache.scale)
    Q = queries(64, B, H * G, D)
    for sign in (1.0, -1.0):
        Q[:, :, 5] = sign
        O = i8.int8_attention_decode(Q, *cache.args())
        assert torch.isnan(O[:, :G]).all()
        assert torch.isfinite(O[:, G:]).all()
