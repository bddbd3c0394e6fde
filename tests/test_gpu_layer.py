"""A decoder layer run with the operators together, as a serving program would:
qkv with its bias, the 8-bit cache, attention, the output projection and the
two feed-forward products with bias, activation and residual.

Every stage is held against its 64-bit definition on the inputs that stage
really had, with the tolerances of the stage's own tests; then the same
layer is captured into a CUDA graph and replayed token after token, which has
to give the bits of the eager calls.
"""
import itertools

import numpy as np
import pytest
import torch

import int8_quantized_row_b200 as i8
import test_gpu_attention_decode as dec
import test_gpu_attention_prompt as pro
import test_gpu_fused_linear as lin
from gpu_helpers import device_status_clean

pytestmark = pytest.mark.gpu
BLOCK = 64
ALPHA = 6.0


class Layer:
    """d = Hq * D; weights by name; wq_only gives the Wq-only variant."""

    def __init__(self, Hq, H, D, seed, wq_only=False):
        self.Hq, self.H, self.D, self.d, self.wq_only = Hq, H, D, Hq * D, wq_only
        rng = np.random.default_rng(seed)
        self.w = {}
        for name, K, N in (("qkv", self.d, (Hq + 2 * H) * D), ("out", self.d, self.d), ("fc1", self.d, 4 * self.d),
                           ("fc2", 4 * self.d, self.d)):
            W = (rng.standard_normal((K, N)) * K ** -0.5).astype(np.float16)
            Wd = torch.from_numpy(W).cuda()
            Wq, sW = i8.int8_quantize_weight_colwise(Wd)
            b = (0.1 * rng.standard_normal(N)).astype(np.float16)
            self.w[name] = dict(W=W, W16=None if wq_only else Wd, Wq=Wq, sW=sW, b=b, bias=torch.from_numpy(b).cuda())
        self.gain = torch.ones(self.d, device="cuda", dtype=torch.float16)
        self.gain[torch.from_numpy(rng.choice(self.d, 3, replace=False)).cuda()] = 12.0      # outlier columns

    def norm(self, x):
        return torch.nn.functional.layer_norm(x, (self.d,), self.gain)

    def linear(self, name, x, act="none", residual=None, seen=None):
        w = self.w[name]
        y = i8.int8_mixed_linear_fused(x, w["Wq"], w["sW"], w["W16"], ALPHA, bias=w["bias"], act=act, residual=residual)
        if seen is not None:
            seen.append((name, x, act, residual, y))
        return y

    def split(self, qkv):
        q, k, v = qkv.view(-1, self.Hq + 2 * self.H, self.D).split([self.Hq, self.H, self.H], 1)
        return q, k, v

    def rest(self, x, o, seen=None):
        x = self.linear("out", o.reshape(-1, self.d), residual=x, seen=seen)
        h = self.linear("fc1", self.norm(x), act="relu", seen=seen)
        return self.linear("fc2", h, residual=x, seen=seen)

    def check_linears(self, seen):
        host = lambda t: None if t is None else t.cpu().numpy()
        for name, x, act, residual, y in seen:
            w = self.w[name]
            lin.check(y, *lin.definition(host(x), w["W"], self.wq_only, ALPHA, w["b"], act, host(residual)), name)


class Cache:
    def __init__(self, layer, B, tokens, seed):
        per = -(-tokens // BLOCK)
        order = np.random.default_rng(seed).permutation(B * per + 1)[:B * per]
        self.table = torch.from_numpy(order.reshape(B, per).astype(np.int32)).cuda()
        shape = (B * per + 1, layer.H, BLOCK, layer.D)
        self.codes = [torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2)]
        self.scale = [torch.zeros(shape[:2], device="cuda") for _ in range(2)]
        self.past = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.H, self.D = layer.H, layer.D

    def append(self, k, v, cu):
        i8.int8_kv_append(k, v, cu, self.past, self.table, *self.codes, *self.scale)
        self.past.add_(cu[1:] - cu[:-1])

    def gather(self, cu, rows):
        return i8.int8_kv_gather(*self.codes, *self.scale, cu, self.table, rows)

    def clone(self):
        c = object.__new__(Cache)
        c.__dict__.update(self.__dict__, codes=[t.clone() for t in self.codes], scale=[t.clone() for t in self.scale],
                          past=self.past.clone())
        return c


def cum(lens):
    return torch.tensor([0, *itertools.accumulate(lens)], dtype=torch.int32, device="cuda")


def prompt(layer, cache, x, lens, seen=None):
    """The layer over packed prompts whose first tokens may already be in the cache."""
    cu, before = cum(lens), cache.past.tolist()
    qkv = layer.linear("qkv", layer.norm(x), seen=seen)
    q, k, v = layer.split(qkv)
    cache.append(k, v, cu)
    if any(before):
        both = [a + b for a, b in zip(before, lens)]
        cu_k = cum(both)
        k, v = cache.gather(cu_k, sum(both))
    else:
        both, cu_k = lens, cu
    o = i8.int8_attention_prompt(q, k, v, cu, cu_k)
    if seen is not None:
        pro.check(o, q, k, v, lens, both, layer.D ** -0.5)
    return layer.rest(x, o, seen)


def token(layer, cache, x, cu, seen=None):
    """The layer over one new token per sequence."""
    q, k, v = layer.split(layer.linear("qkv", layer.norm(x), seen=seen))
    cache.append(k, v, cu)
    o = i8.int8_attention_decode(q, *cache.codes, *cache.scale, cache.table, cache.past)
    return q, o, layer.rest(x, o, seen)


def hidden(layer, rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, layer.d, generator=g, device="cuda").half()


class Lens:
    """The cache as the decode tests' check reads it."""

    def __init__(self, cache):
        self.lens, self.H, self.table, self.codes, self.scale = cache.past.tolist(), cache.H, cache.table, cache.codes, cache.scale

    values = dec.Cache.values


@pytest.mark.parametrize("Hq,H,D,wq_only", [(4, 4, 64, False), (6, 2, 128, True), (8, 1, 64, False)])
def test_prompts_then_tokens(Hq, H, D, wq_only):
    layer = Layer(Hq, H, D, seed=Hq, wq_only=wq_only)
    lens = [70, 1, 130, 64]
    cache = Cache(layer, len(lens), 200, seed=1)
    seen = []
    prompt(layer, cache, hidden(layer, sum(lens), 2), lens, seen)
    more = [30, 5, 1, 0]                                   # prompts that continue what is cached
    prompt(layer, cache, hidden(layer, sum(more), 3), more, seen)
    ones = cum([1] * len(lens))
    for step in range(3):
        q, o, _ = token(layer, cache, hidden(layer, len(lens), 4 + step), ones, seen)
        dec.check(o, q, Lens(cache), D ** -0.5)
    layer.check_linears(seen)
    assert cache.past.tolist() == [a + b + 3 for a, b in zip(lens, more)]
    assert device_status_clean()


@pytest.mark.parametrize("D", [64, 128])
def test_decode_attention_agrees_with_prompt_attention_on_the_same_cache(D):
    """One new token: both operators attend over the same codes.  The prompt form's keys and values
    went through fp16, half a step 2^-11 of each, which moves a score by at most 2^-11 X and a value
    by 2^-11 A; the rest is what either is allowed against 64 bits, once for each."""
    layer = Layer(6, 2, D, seed=9)
    lens = [100, 3, 64, 191]
    cache = Cache(layer, len(lens), 200, seed=3)
    prompt(layer, cache, hidden(layer, sum(lens), 1), lens)
    cu = cum([1] * len(lens))
    q, o, _ = token(layer, cache, hidden(layer, len(lens), 2), cu)
    both = cache.past.tolist()
    k, v = cache.gather(cum(both), sum(both))
    p = i8.int8_attention_prompt(q, k, v, cu, cum(both))
    want, tol = pro.definition(q, k, v, [1] * len(lens), both, D ** -0.5)
    at = 0
    for b, n in enumerate(both):
        for h in range(6):
            kk, vv, qq = k[at:at + n, h // 3].double(), v[at:at + n, h // 3].double(), q[b, h].double()
            w = torch.softmax(D ** -0.5 * kk @ qq, 0)
            X = D ** -0.5 * (kk.abs() @ qq.abs()).max()
            A = w @ vv.abs()
            off = (o[b, h].double() - p[b, h].double()).abs()
            assert bool((off <= 2 * tol[b, h] + A * 2.0 ** -11 * (1.01 + 2 * 1.01 * X) + 2.0 ** -25).all()), (b, h)
        at += n
    assert device_status_clean()


@pytest.mark.parametrize("Hq,H,D", [(4, 4, 128), (8, 2, 64)])
def test_a_captured_layer_replays_token_after_token(Hq, H, D):
    """The graph holds the whole layer, the cache's growth and its lengths included: each replay is
    the next token, across a block's end, and its output feeds the next one."""
    layer, B, steps = Layer(Hq, H, D, seed=5), 5, 8
    lens = [60, 1, 130, 64, 58]
    eager = Cache(layer, B, 200, seed=2)
    prompt(layer, eager, hidden(layer, sum(lens), 1), lens)
    ones = cum([1] * B)
    first = hidden(layer, B, 6)
    graphed = eager.clone()
    warm = eager.clone()
    x = first.clone()
    want = []
    for _ in range(steps):
        x = token(layer, eager, x, ones)[2]
        want.append(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(layer, warm, first, ones)
    torch.cuda.current_stream().wait_stream(side)
    x = first.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = token(layer, graphed, x, ones)[2]
        x.copy_(y)
    for t in range(steps):
        graph.replay()
        assert torch.equal(x, want[t]), f"token {t}"
    assert torch.equal(graphed.past, eager.past)
    for a, b in zip(graphed.codes + graphed.scale, eager.codes + eager.scale):
        assert torch.equal(a, b)
    assert device_status_clean()


def test_two_streams_at_once():
    """Prompts on one stream while tokens are made on another, each with its own cache: the same
    bits as one after the other."""
    layer = Layer(4, 2, 128, seed=8)
    lens, B, rounds = [300, 17, 129], 6, 6
    xs = [hidden(layer, sum(lens), 20 + r) for r in range(rounds)]
    start = hidden(layer, B, 40)
    ones = cum([1] * B)
    first = Cache(layer, B, 300, seed=4)
    prompt(layer, first, hidden(layer, 6 * 40, 41), [40] * 6)

    def prompts(out):
        for x in xs:
            out.append(prompt(layer, Cache(layer, len(lens), 300, seed=5), x, lens))

    def tokens(cache, out):
        x = start
        for _ in range(4 * rounds):
            x = token(layer, cache, x, ones)[2]
            out.append(x)
    want = [[], []]
    prompts(want[0])
    tokens(first.clone(), want[1])
    cache, got = first.clone(), [[], []]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        prompts(got[0])
    with torch.cuda.stream(streams[1]):
        tokens(cache, got[1])
    torch.cuda.synchronize()
    for a, b in zip(got[0] + got[1], want[0] + want[1]):
        assert torch.equal(a, b)
    assert device_status_clean()


def test_workspaces_that_are_no_buffer_are_refused():
    """A strided view counts bytes that are not its own; each call refuses it before any kernel runs."""
    T, K, N = 4, 256, 256
    x, w = torch.randn(T, K, device="cuda").half(), torch.randn(K, N, device="cuda").half()
    Wq, sW = i8.int8_quantize_weight_colwise(w)
    W4, S4 = i8.int4_quantize_weight_groupwise(w)
    codes = [torch.zeros(2, 1, 64, 64, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.ones(2, 1, device="cuda") for _ in range(2)]
    table, lengths = (torch.ones(n, dtype=torch.int32, device="cuda") for n in ((1, 1), (1,)))
    y = torch.empty(T, N, dtype=torch.float16, device="cuda")
    calls = [lambda ws: i8.int8_mixed_linear(x, Wq, sW, w, workspace_buf=ws),
             lambda ws: i8.int8_mixed_linear_wq(x, Wq, sW, workspace_buf=ws),
             lambda ws: i8.int8_mixed_linear_fused(x, Wq, sW, w, workspace_buf=ws),
             lambda ws: i8.int8_mixed_linear_fused(x, Wq, sW, workspace_buf=ws),
             lambda ws: i8.int8_mixed_linear_chain([(x, Wq, sW, w, 6.0, y)], workspace_buf=ws),
             lambda ws: i8.int4_linear(x, W4, S4, N, workspace_buf=ws),
             lambda ws: i8.int8_attention_decode(x[:1, :64].view(1, 1, 64), *codes, *scale, table, lengths,
                                                 workspace_buf=ws)]
    size = 64 << 20
    buf = torch.empty(2, size, dtype=torch.uint8, device="cuda")
    for call in calls:
        for strided in (buf.view(size, 2)[:, 0], buf[:1, ::2], buf[:, :size // 2]):
            with pytest.raises(ValueError):
                call(strided)
        for other in (torch.empty(size, dtype=torch.uint8), 4096):
            with pytest.raises(TypeError):
                call(other)
        call(buf)                                                  # any shape and type will do
        call(buf[1].view(torch.float32))
    assert device_status_clean()


def test_scales_of_a_layer_in_a_stacked_tensor():
    """Codes and scales of several layers in one tensor, with a layer's scales at an odd word."""
    layers, blocks, H, D = 3, 5, 3, 64
    codes = [torch.zeros(layers, blocks, H, 64, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.full((layers, blocks, H), 7.0, device="cuda") for _ in range(2)]
    x = [torch.randn(200, H, D, device="cuda").half() for _ in range(3)]
    table = torch.tensor([[4, 1, 3, 0]], dtype=torch.int32, device="cuda")
    one = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    outs = []
    for i in range(layers):
        assert scale[0][i].data_ptr() % 16 == 60 * i % 16
        cache = (codes[0][i], codes[1][i], scale[0][i], scale[1][i])
        i8.int8_kv_append(x[0], x[1], one(0, 200), one(0), table, *cache)
        outs.append((*i8.int8_kv_gather(*cache, one(0, 200), table, 200),
                     i8.int8_attention_decode(x[2][:1], *cache, table, one(200))))
    for out in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out, outs[0]))
    assert (scale[0][:, 2] == 7.0).all() and (scale[1][:, 2] == 7.0).all()      # the block that no sequence has
    assert device_status_clean()


def test_plain_numbers_of_any_kind_and_tables_that_are_no_tensors():
    """alpha and scale may be whatever float() takes, as in the older calls; a table that is no CUDA tensor is named."""
    x, w = torch.randn(4, 256, device="cuda").half(), torch.randn(256, 256, device="cuda").half()
    Wq, sW = i8.int8_quantize_weight_colwise(w)
    codes = [torch.randint(-127, 128, (2, 1, 64, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.ones(2, 1, device="cuda") for _ in range(2)]
    table, length = torch.ones(1, 1, dtype=torch.int32, device="cuda"), torch.full((1,), 50, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 64, device="cuda").half()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    calls = [lambda v: i8.int8_mixed_linear_fused(x, Wq, sW, w, alpha=v),
             lambda v: i8.int8_attention_decode(q, *codes, *scale, table, length, scale=v),
             lambda v: i8.int8_attention_prompt(q, q, q, cu, scale=v)]
    for call in calls:
        want = call(2.0)
        for number in (2, np.float32(2), np.float64(2), torch.tensor(2.0)):
            assert torch.equal(call(number), want)
    for bad in (None, [[1]], table.cpu(), table.cpu().numpy()):
        with pytest.raises(TypeError, match="block_table"):
            i8.int8_attention_decode(q, *codes, *scale, bad, length)
        with pytest.raises(TypeError, match="block_table"):
            i8.int8_kv_append(q, q, cu, length, bad, *codes, *scale)
    assert device_status_clean()
