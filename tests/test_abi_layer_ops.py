"""Host-side checks of the decoder layer's operators through the C ABI (CPU only:
no call here gets as far as the device)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def so():
    from int8_quantized_row_b200 import build
    build.build()
    import int8_quantized_row_b200 as m
    return m.lib()


def p(addr=4096):
    return ctypes.c_void_p(addr)


NULL = ctypes.c_void_p(0)
OK, EINVAL, EALIGN, ERANGE, EWORKSPACE = 0, 1, 2, 3, 4


def test_fused_linear_refusals(so):
    f = so.int8_mixed_linear_fused
    size = so.int8_mixed_linear_workspace_size(16, 1024, 1024)
    size_wq = so.int8_mixed_linear_wq_workspace_size(16, 1024, 1024)

    def call(T=16, K=1024, N=1024, x=p(), w16=p(), alpha=6.0, bias=p(), act=1, res=p(), y=p(), ws=p(), wsb=size):
        return f(x, T, K, p(), p(), w16, N, alpha, bias, act, res, y, ws, wsb, NULL)

    assert call(K=1000) == EALIGN
    assert call(N=1000) == EALIGN
    assert call(K=133152) == ERANGE
    assert call(N=0) == ERANGE
    assert call(T=-1) == EINVAL
    assert call(alpha=float("nan")) == EINVAL
    assert call(act=3) == EINVAL
    assert call(act=-1) == EINVAL
    assert call(x=NULL) == EINVAL
    assert call(y=NULL) == EINVAL
    assert call(bias=p(4098)) == EALIGN
    assert call(res=p(4104)) == EALIGN
    assert call(wsb=size - 1) == EWORKSPACE
    assert call(ws=NULL) == EWORKSPACE
    assert call(ws=p(4096 + 16)) == EALIGN
    # the Wq-only variant needs its own, larger workspace
    assert call(w16=NULL, wsb=min(size, size_wq) - 1) == EWORKSPACE
    assert call(T=0, x=NULL, y=NULL, bias=p(1), res=p(1), ws=NULL, wsb=0) == OK


def test_cache_refusals(so):
    def append(k=p(), ldk=256, ldv=256, n=4, H=2, D=128, cu=p(), past=p(), B=2, kc=p(), sk=p(), blocks=9, table=p(),
               wide=3):
        return so.int8_kv_append(k, ldk, p(), ldv, n, H, D, cu, past, B, kc, p(), sk, p(), blocks, table, wide, NULL)

    def gather(kc=p(), sk=p(), blocks=9, H=2, D=128, table=p(), wide=3, cu=p(), B=2, rows=4, k=p()):
        return so.int8_kv_gather(kc, p(), sk, p(), blocks, H, D, table, wide, cu, B, rows, k, p(), NULL)

    for f in (append, gather):
        assert f(D=96) == ERANGE
        assert f(H=0) == ERANGE
        assert f(H=8193, **(dict(ldk=1 << 21, ldv=1 << 21) if f is append else {})) == ERANGE
        assert f(H=-1) == EINVAL
        assert f(B=-1) == EINVAL
        assert f(blocks=-1) == EINVAL
        assert f(blocks=0) == ERANGE
        assert f(wide=0) == ERANGE
        assert f(kc=NULL) == EINVAL
        assert f(kc=p(4104)) == EALIGN
        assert f(sk=NULL) == EINVAL
        assert f(table=NULL) == EINVAL
        assert f(table=p(4098)) == EALIGN
        assert f(cu=NULL) == EINVAL
        assert f(k=NULL) == EINVAL
        assert f(k=p(4098)) == EALIGN
        assert f(B=0, k=NULL) == OK
    assert append(n=-1) == EINVAL
    assert append(n=0, k=NULL) == OK
    assert append(ldk=255) == EINVAL
    assert append(ldv=260) == EALIGN
    assert append(past=NULL) == EINVAL
    assert gather(rows=-1) == EINVAL
    assert gather(rows=0, k=NULL) == OK


def test_decode_attention_refusals(so):
    size = so.int8_attention_decode_workspace_size
    f = so.int8_attention_decode

    def call(q=p(), ldq=512, B=2, Hq=4, H=2, D=128, kc=p(), blocks=9, table=p(), wide=3, lens=p(), scale=0.1, o=p(),
             ldo=512, ws=p(), wsb=None):
        wsb = size(Hq, H, D) if wsb is None else wsb
        return f(q, ldq, B, Hq, H, D, kc, p(), p(), p(), blocks, table, wide, lens, scale, o, ldo, ws, wsb, NULL)

    assert size(4, 2, 128) > 0 and size(4, 3, 128) == 0 and size(4, 2, 80) == 0 and size(-1, 2, 64) == 0
    assert call(D=32, wsb=1 << 30) == ERANGE
    assert call(Hq=5, wsb=1 << 30) == ERANGE
    assert call(Hq=1, wsb=1 << 30) == ERANGE
    assert call(Hq=-4, wsb=1 << 30) == EINVAL
    assert call(H=0, wsb=1 << 30) == ERANGE
    assert call(B=-1) == EINVAL
    assert call(scale=float("nan")) == EINVAL
    assert call(scale=float("inf")) == EINVAL
    assert call(ldq=511) == EINVAL
    assert call(ldo=516) == EALIGN
    assert call(q=NULL) == EINVAL
    assert call(o=p(4104)) == EALIGN
    assert call(lens=NULL) == EINVAL
    assert call(lens=p(4097)) == EALIGN
    assert call(kc=NULL) == EINVAL
    assert call(blocks=0) == ERANGE
    assert call(wide=0) == ERANGE
    assert call(table=NULL) == EINVAL
    assert call(wsb=size(4, 2, 128) - 1) == EWORKSPACE
    assert call(ws=NULL) == EWORKSPACE
    assert call(ws=p(4096 + 64)) == EALIGN
    assert call(B=0, q=NULL, ws=NULL, wsb=0) == OK


def test_prompt_attention_refusals(so):
    def call(q=p(), ldq=512, k=p(), ldk=256, v=p(), ldv=256, N=9, M=9, Hq=4, H=2, D=128, cq=p(), ck=p(), B=2, scale=0.1,
             o=p(), ldo=512):
        return so.int8_attention_prompt(q, ldq, k, ldk, v, ldv, N, M, Hq, H, D, cq, ck, B, scale, o, ldo, NULL)

    assert call(D=256, ldq=4096, ldk=4096, ldv=4096, ldo=4096) == ERANGE
    assert call(Hq=3) == ERANGE
    assert call(Hq=0) == ERANGE
    assert call(H=-2) == EINVAL
    assert call(N=-1) == EINVAL
    assert call(M=-1) == EINVAL
    assert call(B=-1) == EINVAL
    assert call(scale=float("nan")) == EINVAL
    assert call(scale=float("-inf")) == EINVAL
    for name, least in (("ldq", 512), ("ldk", 256), ("ldv", 256), ("ldo", 512)):
        assert call(**{name: least - 8}) == EINVAL
        assert call(**{name: least + 4}) == EALIGN
    for name in ("q", "k", "v", "o"):
        assert call(**{name: NULL}) == EINVAL
        assert call(**{name: p(4104)}) == EALIGN
    for name in ("cq", "ck"):
        assert call(**{name: NULL}) == EINVAL
        assert call(**{name: p(4097)}) == EALIGN
    assert call(N=1 << 30, B=1, Hq=8192, H=8192, ldq=1 << 20, ldk=1 << 20, ldv=1 << 20, ldo=1 << 20) == ERANGE
    assert call(N=0, q=NULL) == OK
    assert call(B=0, q=NULL) == OK


def test_scales_and_counts_need_word_alignment_only(so):
    """A layer's scales may begin anywhere in a stacked tensor.  (Without a GPU the calls end at the
    device's setup, after the checks.)"""
    size = so.int8_attention_decode_workspace_size(4, 2, 128)

    def calls(sk=p(), sv=p(), words=p()):
        yield so.int8_kv_append(p(), 256, p(), 256, 4, 2, 128, words, words, 2, p(), p(), sk, sv, 9, words, 3, NULL)
        yield so.int8_kv_gather(p(), p(), sk, sv, 9, 2, 128, words, 3, words, 2, 4, p(), p(), NULL)
        yield so.int8_attention_decode(p(), 512, 2, 4, 2, 128, p(), p(), sk, sv, 9, words, 3, words, 0.1, p(), 512, p(),
                                       size, NULL)

    import torch
    if not torch.cuda.is_available():                       # (no call may get as far as a launch)
        assert set(calls(p(4100), p(4108), p(4104))) <= {5, 7}
    for bad in (dict(sk=p(4098)), dict(sv=p(4097)), dict(words=p(4099))):
        assert set(calls(**bad)) == {EALIGN}


def test_decode_attention_counts_a_sequence_in_32_bits(so):
    """The blocks of one sequence, over all its heads and tiles of 16 query heads, are at most 2^32."""
    size = so.int8_attention_decode_workspace_size

    def call(Hq, H, blocks, wide, words=p()):
        return so.int8_attention_decode(p(), Hq * 64, 2, Hq, H, 64, p(), p(), p(), p(), blocks, words, wide, words, 0.1, p(),
                                        Hq * 64, p(), size(Hq, H, 64) - 1, NULL)

    assert call(8192, 1, 9, (1 << 23) + 1) == ERANGE               # 512 tiles of 2^23 blocks
    assert call(8192, 1, 9, 1 << 23) == EWORKSPACE                 # (the next check)
    assert call(129, 129, 9, 1 << 30) == ERANGE                    # a length has 2^25 blocks at most
    assert call(128, 128, 9, (1 << 31) - 1) == EWORKSPACE
    assert call(8, 8, 1 << 28, 9) == ERANGE
    assert call(8, 8, (1 << 28) - 1, 9) == EWORKSPACE


def test_scales_that_overflow_in_units_of_log_2_are_refused(so):
    """Scores are taken times log2(e): 3e38 times that is no fp32 number.  (B = 0: nothing to do after the checks.)"""
    def decode(scale):
        return so.int8_attention_decode(NULL, 512, 0, 4, 2, 128, NULL, NULL, NULL, NULL, 9, NULL, 3, NULL, scale, NULL,
                                        512, NULL, 0, NULL)

    def prompt(scale):
        return so.int8_attention_prompt(NULL, 512, NULL, 256, NULL, 256, 9, 9, 4, 2, 128, NULL, NULL, 0, scale, NULL, 512,
                                        NULL)

    for f in (decode, prompt):
        assert f(3e38) == EINVAL and f(-3e38) == EINVAL
        assert f(2e38) == OK and f(-2e38) == OK
