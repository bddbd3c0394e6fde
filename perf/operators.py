"""What is measured of a decoder layer's operators: the mixed int8 linear layer with bias,
activation and residual in its epilogue, the 8-bit key/value cache (append and read back),
attention of single tokens over that cache, and causal attention over packed prompts.

Sizes are those of this repository's workloads: 12288 = 96 heads of 128 (the 175B layer),
5120 = 40 heads of 128 (the 13B layer), 1024 = 16 heads of 64 (the small linear); grouped
variants share 8 key/value heads among 40 or 96 query heads (groups of 5 and 12).

The cache holds blocks of 64 tokens: codes int8 [blocks, kv heads, 64, D] and one absmax scale
per block and head; a value stands for code * scale / 127.
"""
import math
import random

import torch

own = False

BLOCK = 64
ALPHA = 6.0


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # One token through the 175B fc2: the weight's bytes are the whole cost.
        {"name": "linear fc2 1 token", "op": "linear", "T": 1, "K": 49152, "N": 12288, "outliers": 49, "hit": 1.0,
         "w16": True, "bias": True, "act": "none", "residual": True},
        # Sixteen decoding sequences through the 175B fc1 with its ReLU.
        {"name": "linear fc1 16 tokens", "op": "linear", "T": 16, "K": 12288, "N": 49152, "outliers": 7, "hit": 1.0,
         "w16": True, "bias": True, "act": "relu", "residual": False},
        # A prompt through the 13B fc1: bound by the tensor cores.
        {"name": "linear fc1 prompt", "op": "linear", "T": 2048, "K": 5120, "N": 20480, "outliers": 6, "hit": 0.25,
         "w16": False, "bias": True, "act": "gelu", "residual": True},
        # A small model's decode step: three sequences, one new token each.
        {"name": "cache 3 tokens", "op": "cache", "seed": 1, "B": 3, "Hkv": 16, "D": 64, "past": 90, "new": 1},
        # A 175B decode step: sixteen sequences, one new token each, read back for a later prompt chunk.
        {"name": "cache 16 tokens", "op": "cache", "seed": 2, "B": 16, "Hkv": 96, "D": 128, "past": 150, "new": 1},
        # The keys and values of packed prompts (about 4096 tokens, ragged), some continuing cached ones.
        {"name": "cache prompts", "op": "cache", "seed": 3, "B": 5, "Hkv": 96, "D": 128, "past": 100, "new": 1500},
        # One sequence of a 13B model: latency and a long axis to split.
        {"name": "decode 1 sequence", "op": "decode", "seed": 4, "B": 1, "Hq": 40, "Hkv": 40, "D": 128, "len": 1000},
        # Sixteen ragged sequences of the 175B layer (one key/value head per query head).
        {"name": "decode 16 sequences", "op": "decode", "seed": 5, "B": 16, "Hq": 96, "Hkv": 96, "D": 128, "len": 2048},
        # Many long sequences with grouped heads: the largest caches.
        {"name": "decode 64 long", "op": "decode", "seed": 6, "B": 64, "Hq": 96, "Hkv": 8, "D": 128, "len": 16384},
        # A short prompt of a small model: latency.
        {"name": "prompt 200 tokens", "op": "prompt", "seed": 7, "B": 1, "Hq": 16, "Hkv": 16, "D": 64, "len": 200,
         "prefix": 0},
        # Packed ragged prompts of the 175B layer, about 4096 tokens.
        {"name": "prompt packed", "op": "prompt", "seed": 8, "B": 5, "Hq": 96, "Hkv": 96, "D": 128, "len": 1500,
         "prefix": 0},
        # Two long prompts with grouped heads that continue cached prefixes.
        {"name": "prompt long", "op": "prompt", "seed": 9, "B": 2, "Hq": 40, "Hkv": 8, "D": 128, "len": 6000,
         "prefix": 700},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "cache", "decode", "prompt"])
    seed = rng.randrange(1, 1 << 30)
    if op == "linear":
        return {"op": op, "T": _log(rng, 1, 2048), "K": 16 * _log(rng, 16, 320), "N": 16 * _log(rng, 16, 1280),
                "outliers": rng.choice([0, 1, 3, 8, 70]), "hit": rng.choice([0.25, 1.0]), "w16": rng.random() < 0.5,
                "bias": rng.random() < 0.7, "act": rng.choice(["none", "relu", "gelu"]),
                "residual": rng.random() < 0.5, "seed": seed}
    Hkv = rng.choice([1, 2, 5, 8, 16, 40])
    D = rng.choice([64, 128])
    if op == "cache":
        B = _log(rng, 1, 48)
        return {"op": op, "seed": seed, "B": B, "Hkv": Hkv, "D": D, "past": rng.choice([0, 40, 300]),
                "new": rng.choice([1, 1, _log(rng, 2, 3000 // B + 2)])}
    group = rng.choice([1, 1, 2, 3, 5, 8, 12, 16])
    if op == "decode":
        B = _log(rng, 1, 64)
        Hkv = min(Hkv, 16) if group > 1 else Hkv
        return {"op": op, "seed": seed, "B": B, "Hq": Hkv * group, "Hkv": Hkv, "D": D,
                "len": _log(rng, 1, min(16384, 4000000 // (B * Hkv * group)))}
    Hkv = max(1, min(Hkv, 40 // group))
    B = _log(rng, 1, 12)
    return {"op": op, "seed": seed, "B": B, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "len": _log(rng, 1, 5000 // B),
            "prefix": rng.choice([0, 0, 130, 600])}


def _lens(case, key):
    """Ragged lengths around and up to `case[key]`: a longest one, short ones, an empty one where there are
    many; the same for every seed of the inputs (a length is part of the case)."""
    n, top = case["B"], case[key]
    r = random.Random(case["seed"] * 3 + len(key))
    out = [top] + [r.randint(max(0, top // 8), top) for _ in range(n - 1)]
    if n >= 4:
        out[r.randrange(1, n)] = min(top, 1)
    if n >= 8:
        out[r.randrange(1, n)] = 0
    r.shuffle(out)
    return out


def _news(case):
    return [1] * case["B"] if case["new"] == 1 else _lens(case, "new")


def _pasts(case):
    return _lens(case, "past") if case["past"] else [0] * case["B"]


def _prompt_lens(case):
    q = _lens(case, "len")
    r = random.Random(case["seed"] + 17)
    k = [n + (r.randint(0, case["prefix"]) if case["prefix"] else 0) for n in q]
    return q, k


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(v):
    out = [0]
    for n in v:
        out.append(out[-1] + n)
    return out


def _normal(g, *shape, sd=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float16) * sd


def _codes(v, inv):
    """Codes of v with the reciprocal scale inv: one 32-bit product, halves away from zero, +-127."""
    x = v * inv
    t = torch.trunc(x)
    t = t + torch.sign(x) * ((x - t).abs() >= 0.5)
    return t.clamp(-127, 127)


def _recip(absmax):
    # a division by a tensor: with a plain number on either side torch multiplies by a reciprocal instead
    return torch.where(absmax > 0, torch.full_like(absmax, 127.0) / absmax, torch.zeros_like(absmax))


def _step(absmax):
    return absmax / torch.full_like(absmax, 127.0)


def _cache(g, blocks, H, D):
    """A filled cache: normal values whose size varies by block and head, in codes and scales."""
    out = []
    for _ in range(2):
        s = torch.rand(blocks, H, generator=g, device="cuda") * 1.5 + 0.5
        c = torch.empty(blocks, H, BLOCK, D, dtype=torch.int8, device="cuda")
        for i in range(0, blocks, 512):
            v = torch.randn(min(512, blocks - i), H, BLOCK, D, generator=g, device="cuda")
            a = v.abs().amax((2, 3))
            c[i:i + 512] = _codes(v, _recip(a)[:, :, None, None]).to(torch.int8)
            s[i:i + 512] *= a
        out += [c, s]
    return out[0], out[2], out[1], out[3]


def _table(lens, seed, spare=3):
    """Block numbers for sequences of these lengths, in shuffled order, with some blocks left over."""
    need = [-(-n // BLOCK) for n in lens]
    total = sum(need) + spare
    order = list(range(total))
    random.Random(seed).shuffle(order)
    wide, at, rows = max(1, max(need)), 0, []
    for n in need:
        rows.append(order[at:at + n] + [0] * (wide - n))
        at += n
    return _i32(rows), total


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        X = _normal(g, T, K)
        n_out = min(case["outliers"], K)
        if n_out:
            cols = torch.randperm(K, generator=g, device="cuda")[:n_out]
            big = (torch.rand(T, n_out, generator=g, device="cuda") * 54 + 6).half()
            big = torch.where(torch.rand(T, n_out, generator=g, device="cuda") < 0.5, -big, big)
            hit = torch.rand(T, n_out, generator=g, device="cuda") < case["hit"]
            X[:, cols] = torch.where(hit, big, X[:, cols])
        W = _normal(g, K, N, sd=0.01)
        sW = W.abs().amax(0).float()
        Wq = torch.empty(K, N, dtype=torch.int8, device="cuda")
        for i in range(0, K, 4096):
            Wq[i:i + 4096] = _codes(W[i:i + 4096].float(), _recip(sW)).to(torch.int8)
        s.update(X=X, Wq=Wq, sW=sW, W16=W if case["w16"] else None,
                 b=_normal(g, N) if case["bias"] else None, R=_normal(g, T, N) if case["residual"] else None)
        return s
    H, D = case["Hkv"], case["D"]
    if case["op"] == "cache":
        past, new = _pasts(case), _news(case)
        both = [p + n for p, n in zip(past, new)]
        table, blocks = _table(both, case["seed"])
        s["Kc"], s["Vc"], s["sK"], s["sV"] = _cache(g, blocks, H, D)
        # the projection's output holds q, k and v of a token side by side
        qkv = _normal(g, sum(new), 3, H, D, sd=1.5)
        s.update(K=qkv[:, 1], V=qkv[:, 2], table=table, past=_i32(past), cu_new=_i32(_cum(new)),
                 cu_all=_i32(_cum(both)), rows=sum(both))
        return s
    Hq = case["Hq"]
    s["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "decode":
        lens = _lens(case, "len")
        table, blocks = _table(lens, case["seed"])
        s["Kc"], s["Vc"], s["sK"], s["sV"] = _cache(g, blocks, H, D)
        s.update(Q=_normal(g, case["B"], Hq, D), table=table, lens=_i32(lens))
        return s
    q, k = _prompt_lens(case)
    s.update(Q=_normal(g, sum(q), Hq, D), K=_normal(g, sum(k), H, D, sd=1.5), V=_normal(g, sum(k), H, D),
             cu_q=_i32(_cum(q)), cu_k=_i32(_cum(k)))
    return s


# ------------------------------------------------------------------------------- one pass

def run(s):
    return {"linear": _linear, "cache": _cache_pass, "decode": _decode, "prompt": _prompt}[s["op"]](s)


def _linear(s):
    if own:
        import int8_quantized_row_b200 as i8
        return i8.int8_mixed_linear_fused(s["X"], s["Wq"], s["sW"], s["W16"], ALPHA, bias=s["b"], act=s["act"],
                                          residual=s["R"])
    X, Wq, sW = s["X"].float(), s["Wq"], s["sW"]
    hit = (X.abs() >= ALPHA).any(0)
    rest = torch.where(hit, torch.zeros_like(X), X)
    sX = rest.abs().amax(1, keepdim=True)
    y = (_codes(rest, _recip(sX)) @ Wq.float()) * (sX / 16129.0 * sW)
    O = torch.nonzero(hit).squeeze(1)
    W = s["W16"][O].float() if s["W16"] is not None else (Wq[O].float() * _step(sW)).half().float()
    y = y + X[:, O] @ W
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["act"] == "relu":
        y = y.clamp_min(0)
    elif s["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.half()


def _append_plain(new, codes, scales, page, off, kept):
    """New rows [n, H, D] into codes and scales: a block's scale grows to the largest value it has to hold,
    and the codes it keeps (offsets below kept[block]) are rescaled then."""
    v = new.float()
    blocks, H = scales.shape
    top = torch.full_like(scales, -1.0).scatter_reduce(0, page[:, None].expand(-1, H), v.abs().amax(2), "amax")
    old = torch.where((kept > 0)[:, None], scales, torch.zeros_like(scales))
    grown = top > old
    written = torch.where(grown, top, torch.where(top >= 0, old, scales))
    ratio = torch.where(grown & (old > 0), old / written, torch.ones_like(old))
    was = torch.arange(BLOCK, device="cuda") < kept[:, None]
    q = codes.float()
    q = torch.where(was[:, None, :, None] & (top >= 0)[:, :, None, None], _codes(q, ratio[:, :, None, None]), q)
    q[page, :, off] = _codes(v, _recip(written)[page][:, :, None])
    codes.copy_(q)
    scales.copy_(written)


def _gather_plain(codes, scales, page, off):
    return (codes[page, :, off].float() * _step(scales)[page][:, :, None]).half()


def _places(table, cu, start):
    """Block and offset of each of the rows that cu counts: row i of sequence b is token start[b] + i."""
    n = (cu[1:] - cu[:-1]).long()
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    pos = torch.arange(len(b), device="cuda") - cu.long()[b] + start.long()[b]
    return table[b, pos // BLOCK].long(), pos % BLOCK


def _cache_pass(s):
    if own:
        import int8_quantized_row_b200 as i8
        i8.int8_kv_append(s["K"], s["V"], s["cu_new"], s["past"], s["table"], s["Kc"], s["Vc"], s["sK"], s["sV"])
        K, V = i8.int8_kv_gather(s["Kc"], s["Vc"], s["sK"], s["sV"], s["cu_all"], s["table"], s["rows"])
        return {"K": K, "V": V, "sK": s["sK"], "sV": s["sV"]}
    page, off = _places(s["table"], s["cu_new"], s["past"])
    some = s["cu_new"][1:] > s["cu_new"][:-1]
    first = s["table"].gather(1, (s["past"].long() // BLOCK).clamp_max(s["table"].shape[1] - 1)[:, None])[:, 0].long()
    kept = torch.zeros(s["sK"].shape[0], dtype=torch.long, device="cuda")
    kept.scatter_reduce_(0, first, torch.where(some, s["past"] % BLOCK, 0).long(), "amax")
    _append_plain(s["K"], s["Kc"], s["sK"], page, off, kept)
    _append_plain(s["V"], s["Vc"], s["sV"], page, off, kept)
    page, off = _places(s["table"], s["cu_all"], torch.zeros_like(s["past"]))
    return {"K": _gather_plain(s["Kc"], s["sK"], page, off), "V": _gather_plain(s["Vc"], s["sV"], page, off),
            "sK": s["sK"], "sV": s["sV"]}


def _decode(s):
    if own:
        import int8_quantized_row_b200 as i8
        return i8.int8_attention_decode(s["Q"], s["Kc"], s["Vc"], s["sK"], s["sV"], s["table"], s["lens"],
                                        scale=s["scale"])
    B, Hq, D = s["Q"].shape
    H = s["Hkv"]
    q = s["Q"].float().view(B, H, Hq // H, D)
    table = s["table"].long()
    k = s["Kc"][table].float() * _step(s["sK"])[table][..., None, None]      # [B, blocks, H, 64, D]
    x = torch.einsum("bhgd,bnhtd->bhgnt", q, k).flatten(3) * s["scale"]
    del k
    live = torch.arange(x.shape[3], device="cuda") < s["lens"][:, None]
    x = x.masked_fill(~live[:, None, None], -math.inf)
    top = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = p / p.sum(3, keepdim=True).clamp_min(1e-30)
    v = s["Vc"][table].float() * _step(s["sV"])[table][..., None, None]
    return torch.einsum("bhgnt,bnhtd->bhgd", p.unflatten(3, (-1, BLOCK)), v).reshape(B, Hq, D).half()


def _owners(cu, rows):
    """The sequence of each row, and its place in it."""
    i = torch.arange(rows, device="cuda")
    b = torch.searchsorted(cu.long(), i, right=True) - 1
    return b, i - cu.long()[b]


def _prompt(s):
    if own:
        import int8_quantized_row_b200 as i8
        return i8.int8_attention_prompt(s["Q"], s["K"], s["V"], s["cu_q"], s["cu_k"], scale=s["scale"])
    (n, Hq, D), (m, H, _) = s["Q"].shape, s["K"].shape
    bq, i = _owners(s["cu_q"], n)
    bk, j = _owners(s["cu_k"], m)
    nq, nk = s["cu_q"].diff().long(), s["cu_k"].diff().long()
    live = (bq[:, None] == bk) & (j <= (i + (nk - nq)[bq])[:, None])
    q = s["Q"].float().view(n, H, Hq // H, D).permute(1, 2, 0, 3).reshape(H, -1, D)
    x = (q @ s["K"].float().permute(1, 2, 0)).view(H, Hq // H, n, m).mul_(s["scale"])
    x.masked_fill_(~live, -math.inf)
    top = x.amax(3, keepdim=True)
    x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    x.div_(x.sum(3, keepdim=True).clamp_min(1e-30))
    o = x.view(H, -1, m) @ s["V"].float().permute(1, 0, 2)
    return o.view(H, Hq // H, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D).half()


# ------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "linear":
        T, K, N, o = case["T"], case["K"], case["N"], min(case["outliers"], case["K"])
        b = 2 * T * K + K * N + 4 * N + (2 * o * N if case["w16"] else 0) + 2 * T * N
        b += (2 * N if case["bias"] else 0) + (2 * T * N if case["residual"] else 0)
        return {"bytes": b, "flops": 2 * T * K * N + 2 * T * o * N}
    H, D = case["Hkv"], case["D"]
    if case["op"] == "cache":
        past, new = sum(_pasts(case)), sum(_news(case))
        # new rows read (16 bits) and written (8 bits); every row read back (8 bits) and written out (16 bits)
        return {"bytes": 2 * H * D * (3 * new + 3 * (past + new)), "flops": 4 * H * D * (2 * new + past)}
    Hq = case["Hq"]
    if case["op"] == "decode":
        lens = _lens(case, "len")
        b = 2 * H * D * sum(lens) + 8 * H * sum(-(-n // BLOCK) for n in lens) + 4 * case["B"] * Hq * D
        return {"bytes": b, "flops": 4 * Hq * D * sum(lens)}
    q, k = _prompt_lens(case)
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, k))
    return {"bytes": 2 * D * (2 * Hq * sum(q) + 2 * H * sum(k)), "flops": 4 * Hq * D * pairs}


# ------------------------------------------------------------------------------- in 64 bits

def _rhaz64(x):
    """Halves away from zero of the product rounded to 32 bits, as the codec is defined."""
    x = x.float().double()
    return (torch.floor(x.abs() + 0.5) * torch.sign(x)).clamp(-127, 127)


def _by(a, b):
    a, b = (x if torch.is_tensor(x) else torch.tensor(x, dtype=torch.float64, device="cuda").expand(1) for x in (a, b))
    return torch.div(a, b)


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _linear64, "cache": _cache64, "decode": _decode64, "prompt": _prompt64}[case["op"]](s)


def _linear64(s):
    X, sW = s["X"].double(), s["sW"].double()
    O = (s["X"].abs() >= ALPHA).sum(0) > 0
    X8, X16 = X * ~O, X * O
    sX = X8.abs().max(1).values
    inv = torch.where(sX > 0, _by(127.0, sX), 0.0 * sX).float().double()
    q = _rhaz64(X8 * inv[:, None])
    y = torch.empty(X.shape[0], sW.numel(), dtype=torch.float64, device="cuda")
    idx = O.nonzero()[:, 0]
    for n in range(0, sW.numel(), 2048):
        w = s["Wq"][:, n:n + 2048].double()
        c = sW[n:n + 2048]
        part = (q @ w) * sX[:, None] * c / 127.0 ** 2
        if s["W16"] is not None:
            w16 = s["W16"][idx, n:n + 2048].double()
        else:
            w16 = (w[idx] * _by(c, 127.0).float().double()).float().half().double()
        y[:, n:n + 2048] = part + X16[:, idx] @ w16
    if s["b"] is not None:
        y += s["b"].double()
    if s["act"] == "relu":
        y = torch.maximum(y, torch.zeros_like(y))
    if s["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    if s["R"] is not None:
        y += s["R"].double()
    return y


def _cache64(s):
    past, cu = s["past"].tolist(), s["cu_new"].tolist()
    out = {}
    for name in ("K", "V"):
        c, sc = s[name + "c"].double(), s["s" + name].double()
        for b, p in enumerate(past):
            rows = s[name][cu[b]:cu[b + 1]].double()
            at = 0
            while at < len(rows):
                blk, o = int(s["table"][b, (p + at) // BLOCK]), (p + at) % BLOCK
                r = rows[at:at + BLOCK - o].transpose(0, 1)                      # [H, rows, D]
                old = sc[blk] if o else torch.zeros_like(sc[blk])
                top = torch.maximum(old, r.abs().amax((1, 2)))
                f = torch.where((top > old) & (old > 0), old / top, torch.ones_like(old)).float().double()
                c[blk, :, :o] = _rhaz64(c[blk, :, :o] * f[:, None, None])
                inv = torch.where(top > 0, _by(127.0, top), torch.zeros_like(top)).float().double()
                c[blk, :, o:o + r.shape[1]] = _rhaz64(r * inv[:, None, None])
                sc[blk] = top
                at += r.shape[1]
        back = []
        for b, p in enumerate(past):
            n = p + cu[b + 1] - cu[b]
            pages = s["table"][b, :-(-n // BLOCK)].long()
            v = c[pages] * (sc[pages] / 127.0)[:, :, None, None]
            back.append(v.transpose(1, 2).flatten(0, 1)[:n])
        out[name], out["s" + name] = torch.cat(back), sc
    return out


def _decode64(s):
    B, Hq, D = s["Q"].shape
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // BLOCK)].long()
        for h in range(s["Hkv"]):
            k = (s["Kc"][pages, h].double() * (s["sK"][pages, h].double() / 127.0)[:, None, None]).flatten(0, 1)[:n]
            v = (s["Vc"][pages, h].double() * (s["sV"][pages, h].double() / 127.0)[:, None, None]).flatten(0, 1)[:n]
            g = slice(h * Hq // s["Hkv"], (h + 1) * Hq // s["Hkv"])
            out[b, g] = torch.softmax(s["Q"][b, g].double() @ k.T * s["scale"], 1) @ v
    return out


def _prompt64(s):
    n, Hq, D = s["Q"].shape
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device="cuda")
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cq) - 1):
        a, e, c, f = cq[b], cq[b + 1], ck[b], ck[b + 1]
        if a == e or c == f:
            continue
        live = torch.ones(e - a, f - c, device="cuda").tril((f - c) - (e - a)) > 0
        for h in range(Hq):
            kv = h * s["Hkv"] // Hq
            x = s["Q"][a:e, h].double() @ s["K"][c:f, kv].double().T * s["scale"]
            p = torch.softmax(torch.where(live, x, -math.inf), 1)
            out[a:e, h] = torch.nan_to_num(p, 0.0) @ s["V"][c:f, kv].double()
    return out
