"""The 8-bit key/value cache: int8_kv_append and int8_kv_gather against the codec in 64 bits.

Every step of the codec is one IEEE fp32 operation on exactly representable
operands (a product or quotient formed in double and rounded once to fp32 is
that operation), so codes and scales are compared bit for bit, and so are the
values read back (one fp32 product, one rounding to fp16).
"""
import numpy as np
import pytest
import torch

import int8_quantized_row_b200 as i8
from gpu_helpers import device_status_clean

pytestmark = pytest.mark.gpu
BLOCK = 64


def f32(v):
    return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def rhaz(v):
    v = f32(v)
    return np.clip(np.sign(v) * np.floor(np.abs(v) + 0.5), -127, 127)


class Plain:
    """A cache as the header defines it, a block and a head at a time (one of K and V)."""

    def __init__(self, codes, scale):
        self.codes, self.scale = codes.astype(np.float64), scale.astype(np.float64)

    def append(self, rows, table, past):
        at = 0
        while at < len(rows):
            page, o = table[(past + at) // BLOCK], (past + at) % BLOCK
            part = rows[at:at + BLOCK - o].astype(np.float64)
            for h in range(part.shape[1]):
                old = self.scale[page, h] if o else 0.0
                new = max(old, np.abs(part[:, h]).max())
                if new > old > 0:
                    self.codes[page, h, :o] = rhaz(self.codes[page, h, :o] * f32(old / new))
                inv = f32(127.0 / new) if new > 0 else 0.0
                self.codes[page, h, o:o + len(part)] = rhaz(part[:, h] * inv)
                self.scale[page, h] = new
            at += len(part)

    def gather(self, table, n):
        out = [self.codes[table[t // BLOCK], :, t % BLOCK] * f32(self.scale[table[t // BLOCK]] / 127.0)[:, None]
               for t in range(n)]
        return f32(np.array(out).reshape(n, *self.codes.shape[1::2])).astype(np.float16)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Setup:
    """Random sequences, a shuffled block table with blocks left over, and the cache on both sides."""

    def __init__(self, seed, past, new, H, D, spare=2):
        rng = np.random.default_rng(seed)
        self.past, self.new, self.H, self.D = past, new, H, D
        need = [-(-(p + n) // BLOCK) for p, n in zip(past, new)]
        self.blocks = sum(need) + spare
        order, wide = rng.permutation(self.blocks), max(1, max(need))
        self.table = np.full((len(past), wide), -1, np.int32)         # entries past a sequence's end name no block
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.blocks, H, BLOCK, D)
        self.codes = [rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2)]
        self.scale = [rng.uniform(0.5, 3, shape[:2]).astype(np.float32) for _ in range(2)]
        self.x = [(rng.standard_normal((sum(new), H, D)) * rng.uniform(0.2, 2, (sum(new), H, 1))).astype(np.float16)
                  for _ in range(2)]
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.all = np.concatenate([[0], np.cumsum(np.array(past) + np.array(new))]).astype(np.int32)

    def device(self):
        return ([dev(c) for c in self.codes], [dev(s) for s in self.scale])

    def want(self):
        plain = [Plain(c, s) for c, s in zip(self.codes, self.scale)]
        for p, x in zip(plain, self.x):
            for b, n in enumerate(self.past):
                p.append(x[self.cu[b]:self.cu[b + 1]], self.table[b], n)
        return plain

    def append(self, codes, scale, K=None, V=None, **kw):
        i8.int8_kv_append(dev(self.x[0]) if K is None else K, dev(self.x[1]) if V is None else V, dev(self.cu),
                          dev(np.array(self.past, np.int32)), dev(self.table), *codes, *scale, **kw)


CASES = [
    ([0], [1]), ([0], [64]), ([0], [65]), ([63], [1]), ([64], [1]), ([63], [2]), ([1], [63]), ([17], [300]),
    ([5, 0, 64, 127, 30], [1, 1, 1, 1, 1]),                     # a decode step
    ([5, 0, 64, 127, 30, 9], [0, 1, 0, 200, 34, 0]),            # ragged, some without new rows
    ([0, 0, 0], [9, 10, 11]), ([40, 3], [16, 17]),
]


@pytest.mark.parametrize("past,new", CASES)
@pytest.mark.parametrize("H,D", [(1, 64), (5, 64), (3, 128), (9, 128)])
def test_append_and_gather(past, new, H, D):
    s = Setup(sum(past) + 7 * sum(new) + H, past, new, H, D)
    codes, scale = s.device()
    s.append(codes, scale)
    want = s.want()
    for c, sc, w in zip(codes, scale, want):
        assert np.array_equal(sc.cpu().numpy().astype(np.float64), w.scale)
        assert np.array_equal(c.cpu().numpy().astype(np.float64), w.codes)   # the other blocks and rows untouched
    rows = int(s.all[-1]) + 3
    out = [torch.full((rows, H, D), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    i8.int8_kv_gather(*codes, *scale, dev(s.all), dev(s.table), rows, K=out[0], V=out[1])
    for o, w in zip(out, want):
        o = o.cpu().numpy()
        for b in range(len(past)):
            assert np.array_equal(o[s.all[b]:s.all[b + 1]], w.gather(s.table[b], past[b] + new[b]))
        assert (o[rows - 3:] == 7.0).all()
    assert device_status_clean()


def test_token_by_token_equals_the_definition():
    """Ninety single-token steps: the scale grows and the codes are rescaled again and again."""
    s = Setup(11, [0, 30], [90, 90], 2, 64)
    codes, scale = s.device()
    plain = [Plain(c, sc) for c, sc in zip(s.codes, s.scale)]
    cu = dev(np.array([0, 1, 2], np.int32))
    for step in range(90):
        x = [np.stack([v[step], v[90 + step]]) for v in s.x]
        past = [step, 30 + step]
        i8.int8_kv_append(dev(x[0]), dev(x[1]), cu, dev(np.array(past, np.int32)), dev(s.table), *codes, *scale)
        for p, v in zip(plain, x):
            for b in range(2):
                p.append(v[b:b + 1], s.table[b], past[b])
    for c, sc, p in zip(codes, scale, plain):
        assert np.array_equal(sc.cpu().numpy().astype(np.float64), p.scale)
        assert np.array_equal(c.cpu().numpy().astype(np.float64), p.codes)


@pytest.mark.parametrize("D", [64, 128])
def test_zero_rows_and_zero_scales(D):
    s = Setup(3, [0, 10], [20, 20], 2, D)
    for x in s.x:
        x[:20] = 0                                     # sequence 0: nothing but zeros
        x[20:40, 1] = 0
    for sc in s.scale:
        sc[s.table[1, 0]] = 0.0                        # sequence 1's kept codes stand for zeros
    for c in s.codes:
        c[s.table[1, 0]] = 0
    codes, scale = s.device()
    s.append(codes, scale)
    for c, sc, w in zip(codes, scale, s.want()):
        assert np.array_equal(sc.cpu().numpy().astype(np.float64), w.scale)
        assert np.array_equal(c.cpu().numpy().astype(np.float64), w.codes)


@pytest.mark.parametrize("D", [64, 128])
def test_halves_round_away_from_zero(D):
    s = Setup(4, [0], [64], 1, D)
    grid = np.arange(64 * D).reshape(64, 1, D) % 255 - 127
    for x in s.x:
        x[:] = grid / 2.0                              # absmax 63.5: the product is 2x the value, rounded
        x[0, 0, 0] = 127.0                             # absmax 127: value = code, halves are ties
    codes, scale = s.device()
    s.append(codes, scale)
    for c, w in zip(codes, s.want()):
        c = c.cpu().numpy().astype(np.float64)
        assert np.array_equal(c, w.codes)
        assert c[s.table[0, 0], 0, 0, 2] == -63.0      # -62.5 -> -63


def test_a_nan_or_infinity_shows_in_its_block_and_head_only():
    s = Setup(5, [10], [100], 2, 64)
    s.x[0][3, 1, 5] = np.nan
    s.x[1][80, 0, 9] = np.inf
    codes, scale = s.device()
    s.append(codes, scale)
    K, V = i8.int8_kv_gather(*codes, *scale, dev(s.all), dev(s.table), 110)
    bad = ~torch.isfinite(K).cpu()
    assert bad[:64, 1].all() and not bad[64:].any() and not bad[:, 0].any()
    bad = ~torch.isfinite(V).cpu()
    assert bad[64:, 0].all() and not bad[:64].any() and not bad[:, 1].any()


def test_strided_rows_another_stream_and_a_replayed_graph():
    s = Setup(6, [5, 70], [40, 3], 3, 128)
    qkv = torch.zeros(43, 3, 3, 128, dtype=torch.float16, device="cuda")
    qkv[:, 1], qkv[:, 2] = dev(s.x[0]), dev(s.x[1])
    want = s.want()
    side = torch.cuda.Stream()
    codes, scale = s.device()
    side.wait_stream(torch.cuda.current_stream())
    s.append(codes, scale, K=qkv[:, 1], V=qkv[:, 2], stream=side)
    side.synchronize()
    for c, w in zip(codes, want):
        assert np.array_equal(c.cpu().numpy().astype(np.float64), w.codes)
    # captured: lengths and blocks are read when the graph is replayed
    codes, scale = s.device()
    cu, past, table = dev(s.cu), dev(np.array([0, 0], np.int32)), dev(np.full_like(s.table, -1))
    K, V = qkv[:, 1], qkv[:, 2]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        i8.int8_kv_append(K, V, cu, past, table, *codes, *scale)
    past.copy_(torch.tensor(s.past))
    table.copy_(dev(s.table))
    graph.replay()
    torch.cuda.synchronize()
    for c, sc, w in zip(codes, scale, want):
        assert np.array_equal(c.cpu().numpy().astype(np.float64), w.codes)
        assert np.array_equal(sc.cpu().numpy().astype(np.float64), w.scale)
    assert device_status_clean()


def test_many_sequences():
    rng = np.random.default_rng(8)
    past = [int(v) for v in rng.integers(0, 200, 700)]
    new = [int(v) for v in rng.integers(0, 3, 700)]
    s = Setup(9, past, new, 1, 64)
    codes, scale = s.device()
    s.append(codes, scale)
    for c, sc, w in zip(codes, scale, s.want()):
        assert np.array_equal(sc.cpu().numpy().astype(np.float64), w.scale)
        assert np.array_equal(c.cpu().numpy().astype(np.float64), w.codes)


@pytest.mark.parametrize("B,longest", [(128, 3), (129, 3), (1024, 3), (1025, 3), (2500, 3), (1300, 40)])
def test_more_sequences_than_a_search_sees_at_once(B, longest):
    rng = np.random.default_rng(B)
    past = [int(v) for v in rng.integers(0, 70, B)]
    new = [int(v) for v in rng.integers(0, longest, B)]
    new[-1] = 1                                            # the last one of all has its row
    s = Setup(B, past, new, 3, 64)
    codes, scale = s.device()
    s.append(codes, scale)
    want = s.want()
    rows = int(s.all[-1])
    K, V = i8.int8_kv_gather(*codes, *scale, dev(s.all), dev(s.table), rows)
    for c, sc, o, w in zip(codes, scale, (K, V), want):
        assert np.array_equal(sc.cpu().numpy().astype(np.float64), w.scale)
        assert np.array_equal(c.cpu().numpy().astype(np.float64), w.codes)
        o = o.cpu().numpy()
        for b in range(0, B, 7):
            assert np.array_equal(o[s.all[b]:s.all[b + 1]], w.gather(s.table[b], past[b] + new[b]))
        assert np.array_equal(o[s.all[B - 1]:], w.gather(s.table[B - 1], past[B - 1] + new[B - 1]))
    assert device_status_clean()


@pytest.mark.parametrize("what", ["block", "negative block", "past", "past beyond the table", "rows", "order"])
def test_bad_indexes_are_reported_and_skipped(what):
    s = Setup(10, [5, 70], [40, 30], 2, 64)
    cu, past, table = s.cu.copy(), np.array(s.past, np.int32), s.table.copy()
    if what == "block":
        table[0, 0] = s.blocks
    if what == "negative block":
        table[0, 0] = -5
    if what == "past":
        past[0] = -1
    if what == "past beyond the table":
        past[0] = 64 * table.shape[1]
    if what == "rows":
        cu = np.array([0, 71, 71], np.int32)
    if what == "order":
        cu = np.array([40, 0, 70], np.int32)
    codes, scale = s.device()
    i8.int8_kv_append(dev(s.x[0]), dev(s.x[1]), dev(cu), dev(past), dev(table), *codes, *scale)
    assert i8.int8_read_and_clear_device_status() == 3
    if what in ("block", "negative block", "past", "past beyond the table"):     # sequence 1 is as it should be
        w = s.want()[0]
        pages = s.table[1, 1:2]
        assert np.array_equal(codes[0].cpu().numpy()[pages].astype(np.float64), w.codes[pages])
        pages = s.table[0, :1]                          # its one block (the other entry names none)
        assert np.array_equal(codes[0].cpu().numpy()[pages], s.codes[0][pages])
    if what in ("block", "negative block"):
        i8.int8_kv_gather(*codes, *scale, dev(s.all), dev(table), int(s.all[-1]))
        assert i8.int8_read_and_clear_device_status() == 3
    assert device_status_clean()


def test_binding_refusals():
    s = Setup(12, [5], [4], 2, 64)
    codes, scale = s.device()
    K, V, cu, past, table = dev(s.x[0]), dev(s.x[1]), dev(s.cu), dev(np.array([5], np.int32)), dev(s.table)

    def call(K=K, V=V, cu=cu, past=past, table=table, Kc=codes[0], sK=scale[0]):
        i8.int8_kv_append(K, V, cu, past, table, Kc, codes[1], sK, scale[1])

    for bad in (dict(K=K[:3]), dict(K=K[:, :1]), dict(cu=cu[:1]), dict(past=dev(np.array([5, 5], np.int32))),
                dict(Kc=codes[0][:, :, :32].contiguous()), dict(sK=scale[0][:, :1].contiguous()),
                dict(K=K.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(K=K.float()), dict(cu=cu.long()), dict(table=table.long()), dict(K=K.cpu())):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(i8.I8RError):
        wide = torch.zeros(4, 2 * 64 + 4, dtype=torch.float16, device="cuda")          # rows not 16-byte aligned
        call(K=wide[:, :128].unflatten(1, (2, 64)))
    call(K=K[:0], V=V[:0])                                                             # nothing to add
    assert device_status_clean()


def test_offsets_past_32_bits():
    """Blocks past 2^32 codes, and rows 2^25 elements apart."""
    H, D, rows = 1, 128, 130
    blocks = 2 ** 32 // (H * BLOCK * D) + 4
    s = Setup(21, [0], [rows], H, D, spare=0)
    codes, scale = s.device()
    s.append(codes, scale)
    near = i8.int8_kv_gather(*codes, *scale, dev(s.all), dev(s.table), rows)
    big = [torch.empty(blocks, H, BLOCK, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    big_scale = [torch.empty(blocks, H, device="cuda") for _ in range(2)]
    table = dev(np.array([[blocks - 1, 5, blocks - 3]], np.int32))
    wide = torch.empty(rows, 2 ** 25, dtype=torch.float16, device="cuda")       # 8.7 GB
    K, V = (wide[:, at:at + D].view(rows, H, D) for at in (0, 2 ** 24))
    K.copy_(dev(s.x[0]))
    V.copy_(dev(s.x[1]))
    i8.int8_kv_append(K, V, dev(s.cu), dev(np.array([0], np.int32)), table, *big, *big_scale)
    far = i8.int8_kv_gather(*big, *big_scale, dev(s.all), table, rows)
    for a, b in zip(near, far):
        assert torch.equal(a, b)
    assert device_status_clean()


def holds(s, codes, scale):
    """Codes and scales of the cache, bit for bit, after s was appended."""
    for c, sc, w in zip(codes, scale, s.want()):
        assert np.array_equal(sc.cpu().numpy().astype(np.float64), w.scale)
        assert np.array_equal(c.cpu().numpy(), w.codes.astype(np.int8))
    assert device_status_clean()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("offset,rows", [(5, 64), (0, 64), (63, 70), (1, 9), (40, 100)])
@pytest.mark.parametrize("grow", [0.2, 8.0])
def test_a_longer_row_range_among_single_tokens(D, offset, rows, grow):
    """At most 8 new rows a sequence on average: one warp a block and head, also where a block gets more rows
    than the warp holds (those are read twice), with scales that stay and scales that grow."""
    past = [(37 * b + 3) % 130 for b in range(16)]
    new = [b % 2 for b in range(16)]
    past[6], new[6] = 128 + offset, rows
    s = Setup(30 + rows, past, new, 3, D)
    for x in s.x:
        x *= np.float16(grow)
        x[s.cu[6] + rows - 1] *= np.float16(4)             # the largest in the last row
    codes, scale = s.device()
    s.append(codes, scale)
    holds(s, codes, scale)


@pytest.mark.parametrize("B,H,D", [(128, 96, 64), (120, 96, 128), (700, 9, 128), (700, 40, 64), (1100, 40, 64)])
def test_single_tokens_of_more_heads_than_a_pass_covers(B, H, D):
    """A block's CTA goes on to further heads, found by a warp (up to 128 sequences) or by the CTA."""
    s = Setup(31 + B, [(29 * b) % 64 for b in range(B)], [1] * B, H, D, spare=1)
    codes, scale = s.device()
    s.append(codes, scale)
    holds(s, codes, scale)
