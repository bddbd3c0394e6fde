"""int8_mixed_linear_fused against the layer's definition in 64 bits.

Y = fp16(act(XW + bias) + residual).  The int8 codes and int32 sums are exact on
both sides (each code is one fp32 product rounded half away from zero, formed
here from the double product), so what may differ is fp32 arithmetic and the
last rounding:
  * the last rounding is off by at most half a step: 2^-11 |y|, or 2^-25 among
    the subnormals;
  * every fp32 step is off by at most 2^-23 of its result (a whole step: the
    tensor cores may truncate); the outlier sum takes |O| of them, the rest of
    the path at most 16, on magnitudes no larger than
    M = |8-bit part| + sum |x w| over O + |bias| + |residual|;
  * gelu's slope is at most 1.13 and its own relative error is a few steps, so
    2 M (|O| + 16) 2^-23 covers all of it.
"""
import numpy as np
import pytest
import torch

import int8_quantized_row_b200 as i8
from gpu_helpers import device_status_clean, outlier_x

pytestmark = pytest.mark.gpu


def rhaz(v):
    v = v.astype(np.float32).astype(np.float64)            # the product, rounded to fp32
    return np.clip(np.sign(v) * np.floor(np.abs(v) + 0.5), -127, 127)


def recip(a):
    return np.where(a > 0, 127.0 / np.where(a > 0, a, 1.0), 0.0).astype(np.float32).astype(np.float64)


def weights(W):
    W = W.astype(np.float64)
    sW = np.abs(W).max(0)
    return rhaz(W * recip(sW)), sW


def definition(X, W, wq_only, alpha, bias, act, residual):
    """(y, M, |O|) in double: the value before the last rounding, and the magnitude its errors go by."""
    X = X.astype(np.float64)
    Wq, sW = weights(W)
    O = (np.abs(X) >= alpha).any(0)
    rest = np.where(O, 0.0, X)
    sX = np.abs(rest).max(1, keepdims=True)
    y8 = (rhaz(rest * recip(sX)) @ Wq) * sX * sW / 127.0 ** 2
    Wo = W[O].astype(np.float64)
    if wq_only:
        step = (sW / 127.0).astype(np.float32).astype(np.float64)
        Wo = (Wq[O] * step).astype(np.float32).astype(np.float16).astype(np.float64)
    y = y8 + X[:, O] @ Wo
    M = np.abs(y8) + np.abs(X[:, O]) @ np.abs(Wo)
    if bias is not None:
        y, M = y + bias.astype(np.float64), M + np.abs(bias.astype(np.float64))
    if act == "relu":
        y = np.where(y < 0, 0.0, y)
    if act == "gelu":
        t = torch.from_numpy(y)
        y = (0.5 * t * torch.special.erfc(-t / 2.0 ** 0.5)).numpy()
    if residual is not None:
        y, M = y + residual.astype(np.float64), M + np.abs(residual.astype(np.float64))
    return y, M, int(O.sum())


def check(got, y, M, n_out, what):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = np.abs(y) * 2.0 ** -11 + 2.0 ** -25 + 2 * M * (n_out + 16) * 2.0 ** -23
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - y)[bad].max():.3e}"


def inputs(T, K, N, seed, n_out=3):
    rng = np.random.default_rng(seed)
    X = outlier_x(rng, T, K, rng.choice(K, size=min(n_out, K), replace=False), row_prob=0.6)
    W = (rng.standard_normal((K, N)) * 0.03).astype(np.float16)
    bias = rng.standard_normal(N).astype(np.float16)
    res = (3 * rng.standard_normal((T, N))).astype(np.float16)
    return X, W, bias, res


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(X, W, wq_only, alpha, bias, act, res, **kw):
    Wd = dev(W)
    Wq, sW = i8.int8_quantize_weight_colwise(Wd)
    return i8.int8_mixed_linear_fused(dev(X), Wq, sW, None if wq_only else Wd, alpha, bias=dev(bias), act=act,
                                      residual=dev(res), **kw)


@pytest.mark.parametrize("T,K,N", [(1, 16, 16), (1, 1024, 528), (3, 272, 64), (16, 1024, 1024), (127, 528, 272),
                                   (128, 256, 512), (129, 272, 528), (300, 1024, 272), (513, 640, 784)])
@pytest.mark.parametrize("act,with_bias,with_res,wq_only", [
    ("relu", True, False, False), ("none", True, True, False), ("gelu", True, True, True), ("gelu", False, False, False),
    ("none", False, True, True), ("relu", False, True, False)])
def test_against_the_definition(T, K, N, act, with_bias, with_res, wq_only):
    X, W, bias, res = inputs(T, K, N, seed=T + K + N)
    bias, res = bias if with_bias else None, res if with_res else None
    Y = run(X, W, wq_only, 6.0, bias, act, res)
    check(Y, *definition(X, W, wq_only, 6.0, bias, act, res), f"T={T} K={K} N={N} {act}")
    assert device_status_clean()


@pytest.mark.parametrize("T", [2, 16, 200])
@pytest.mark.parametrize("alpha", [0.0, 2.0, float("inf")])
def test_every_share_of_outliers(T, alpha):
    # alpha 0: every column is an outlier; inf: none is; 2: most are, past the compacted rows
    X, W, bias, res = inputs(T, 640, 272, seed=T)
    for wq_only in (False, True):
        Y = run(X, W, wq_only, alpha, bias, "relu", res)
        check(Y, *definition(X, W, wq_only, alpha, bias, "relu", res), f"T={T} alpha={alpha} wq_only={wq_only}")
    assert device_status_clean()


@pytest.mark.parametrize("T", [1, 16, 300])
def test_without_epilogue_it_is_the_plain_layer_bit_for_bit(T):
    X, W, _, _ = inputs(T, 1024, 528, seed=T)
    Wd = dev(W)
    Wq, sW = i8.int8_quantize_weight_colwise(Wd)
    Xd = dev(X)
    assert torch.equal(i8.int8_mixed_linear_fused(Xd, Wq, sW, Wd, 6.0), i8.int8_mixed_linear(Xd, Wq, sW, Wd, 6.0))
    assert torch.equal(i8.int8_mixed_linear_fused(Xd, Wq, sW, None, 6.0), i8.int8_mixed_linear_wq(Xd, Wq, sW, 6.0))


@pytest.mark.parametrize("T", [1, 16, 129, 300])
def test_residual_in_place(T):
    X, W, bias, res = inputs(T, 272, 528, seed=T)
    Wd = dev(W)
    Wq, sW = i8.int8_quantize_weight_colwise(Wd)
    want = i8.int8_mixed_linear_fused(dev(X), Wq, sW, Wd, 6.0, bias=dev(bias), act="gelu", residual=dev(res))
    Y = dev(res)
    got = i8.int8_mixed_linear_fused(dev(X), Wq, sW, Wd, 6.0, bias=dev(bias), act="gelu", residual=Y, Y=Y)
    assert got is Y and torch.equal(got, want)


@pytest.mark.parametrize("T", [4, 200])
def test_nan_and_infinity_stay_in_their_places(T):
    X, W, bias, res = inputs(T, 64, 64, seed=1)
    res[2, 5], res[3, 7], bias[11] = np.nan, -np.inf, np.nan
    y = run(X, W, False, 6.0, bias, "relu", res).cpu().numpy()
    nan = np.zeros((T, 64), bool)
    nan[2, 5] = True
    nan[:, 11] = True                                   # relu keeps the bias's NaN
    assert np.array_equal(np.isnan(y), nan)
    assert y[3, 7] == -np.inf and np.isinf(y).sum() == 1


def test_no_rows():
    X, W, bias, _ = inputs(1, 64, 32, seed=2)
    Wd = dev(W)
    Wq, sW = i8.int8_quantize_weight_colwise(Wd)
    Y = i8.int8_mixed_linear_fused(dev(X)[:0], Wq, sW, Wd, 6.0, bias=dev(bias), act="relu")
    assert Y.shape == (0, 32)


@pytest.mark.parametrize("T", [16, 200])
def test_another_stream_and_a_replayed_graph(T):
    X, W, bias, res = inputs(T, 528, 272, seed=T)
    Wd = dev(W)
    Wq, sW = i8.int8_quantize_weight_colwise(Wd)
    Xd, bd, rd = dev(X), dev(bias), dev(res)
    want = i8.int8_mixed_linear_fused(Xd, Wq, sW, Wd, 6.0, bias=bd, act="relu", residual=rd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = i8.int8_mixed_linear_fused(Xd, Wq, sW, Wd, 6.0, bias=bd, act="relu", residual=rd, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(i8.int8_mixed_linear_workspace_size(T, 528, 272), dtype=torch.uint8, device="cuda")
    Y = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        i8.int8_mixed_linear_fused(Xd, Wq, sW, Wd, 6.0, bias=bd, act="relu", residual=rd, Y=Y, workspace_buf=ws)
    for k in range(2):
        rd.mul_(-1)
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, i8.int8_mixed_linear_fused(Xd, Wq, sW, Wd, 6.0, bias=bd, act="relu", residual=rd)), k
    assert device_status_clean()


def test_binding_refusals():
    X, W, bias, res = inputs(2, 64, 32, seed=3)
    Wd, Xd = dev(W), dev(X)
    Wq, sW = i8.int8_quantize_weight_colwise(Wd)
    f = i8.int8_mixed_linear_fused
    with pytest.raises(ValueError):
        f(Xd, Wq, sW, Wd, act="tanh")
    with pytest.raises(ValueError):
        f(Xd, Wq, sW, Wd, bias=dev(bias)[:16])
    with pytest.raises(ValueError):
        f(Xd, Wq, sW, Wd, residual=dev(res)[:1])
    with pytest.raises(ValueError):
        f(Xd, Wq, sW, Wd[:32])
    with pytest.raises(TypeError):
        f(Xd, Wq, sW, Wd, bias=dev(bias).float())
    with pytest.raises(ValueError):
        f(Xd, Wq, sW, Wd, residual=torch.zeros(32, 2, dtype=torch.float16, device="cuda").t())
    with pytest.raises(i8.I8RError):
        f(Xd, Wq, sW, Wd, float("nan"))
    with pytest.raises(i8.I8RError):
        f(Xd, Wq, sW, Wd, workspace_buf=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("T", [1, 4, 16, 128, 200])
def test_a_residual_that_the_call_before_has_just_written(T):
    X, W, bias, _ = inputs(T, 1024, 1024, seed=T)
    x, w, b = (torch.from_numpy(a).cuda() for a in (X, W, bias))
    Wq, sW = i8.int8_quantize_weight_colwise(w)
    residual, Y = (torch.zeros(T, 1024, dtype=torch.float16, device="cuda") for _ in range(2))

    def both(sync):
        for k in range(20):
            i8.int8_mixed_linear_fused(x, Wq, sW, w, 6.0, bias=b if k % 2 else None, act="relu", residual=Y, Y=residual)
            if sync:
                torch.cuda.synchronize()
            i8.int8_mixed_linear_fused(x, Wq, sW, w, 6.0, residual=residual, act="gelu", Y=Y)
            if sync:
                torch.cuda.synchronize()
            Y.mul_(0.25)
        return Y.clone()
    want = both(True)
    for _ in range(5):
        residual.zero_()
        Y.zero_()
        assert torch.equal(both(False), want)
    assert bool(torch.isfinite(want).all()) and device_status_clean()
