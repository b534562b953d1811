"""The grouped-query attention operators as their users call them, case by case.

A layer of routed experts often stands behind grouped-query attention: n
query heads share n / G key and value heads of 64 or 128 values. Five uses:

  norm     RMS norm of every head's query and key with one weight of a head's
           size for each, and the rotation of their first values by position,
           in one pass (serving); with its gradients (training)
  append   serving: new keys and values into a paged cache of 8-bit codes
           (E4M3) with a power-of-two scale for every 16 tokens of a head
  decode   serving: attention of each request's newest token, or of its
           drafted tokens (a chain or a tree), over that cache
  prompt   attention over packed sequences, grouped heads
  train    the same with the gradients of queries, keys and values

`own` False computes them in plain torch operations in 32 bits, True calls
the package. Sizes are a layer of 64 query and 8 key heads at 4096 and 8192
tokens and its one-quarter share.

The cache, for page p, head h, block b of 16 tokens: keys k[p, h, b, d / 16,
t, d % 16], values v[p, h, b, d / 2, (t / 4) % 2, d % 2, t / 8, t % 4] of the
block's token t and value d, codes times 2^(scale - 127). The scale is the
smallest that brings the block's largest magnitude within 448; when a later
token raises it, the block's earlier codes are brought along.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 16


# ---------------------------------------------------------------- the cases
def _ints(text):
    return [int(v) for v in str(text).split(",")]


def _text(vals):
    return ",".join(str(int(v)) for v in vals)


def listed():
    ragged = [1 + (i * i * 7919 + 131 * i) % 6100 for i in range(64)]
    return [
        # one decode step of 64 requests on a quarter share (a call of a few
        # microseconds), and a training step's 8192 tokens with gradients
        {"name": "norm_decode64", "op": "norm", "tokens": 64, "heads": 16, "kv_heads": 2, "dim": 128, "rot": 128,
         "interleaved": False, "back": False},
        {"name": "norm_train8192", "op": "norm", "tokens": 8192, "heads": 64, "kv_heads": 8, "dim": 128, "rot": 64,
         "interleaved": False, "back": True},
        # one decode step of 64 requests; three prompts, one of them the
        # later piece of a longer one
        {"name": "append_decode64", "op": "append", "kv_heads": 8, "dim": 128, "page": 64,
         "new": _text([1] * 64), "lens": _text(ragged)},
        {"name": "append_prompt8192", "op": "append", "kv_heads": 8, "dim": 128, "page": 64,
         "new": "3111,700,4381", "lens": "3111,700,7005"},
        # one chat (latency); 64 ragged requests; few requests with long
        # documents on a quarter share; checking drafted trees
        {"name": "decode_one", "op": "decode", "heads": 64, "kv_heads": 8, "dim": 128, "nq": 1, "tree": False,
         "page": 64, "lens": "531"},
        {"name": "decode_64ragged", "op": "decode", "heads": 64, "kv_heads": 8, "dim": 128, "nq": 1, "tree": False,
         "page": 64, "lens": _text(ragged)},
        {"name": "decode_long", "op": "decode", "heads": 16, "kv_heads": 2, "dim": 128, "nq": 1, "tree": False,
         "page": 16, "lens": "65536,40001,1,57,131072,33333,9000,70"},
        {"name": "decode_tree8", "op": "decode", "heads": 64, "kv_heads": 8, "dim": 128, "nq": 8, "tree": True,
         "page": 32, "lens": "4100,33,1000,8192,2500,6001,350,1999"},
        # short prompts on a quarter share with narrow heads; three prompts
        # and a later piece of a fourth
        {"name": "prompt_short", "op": "prompt", "heads": 16, "kv_heads": 2, "dim": 64, "lens_q": "1,37,130",
         "lens_k": "1,37,130", "causal": True},
        {"name": "prompt_6144", "op": "prompt", "heads": 64, "kv_heads": 8, "dim": 128,
         "lens_q": "2300,511,1285,2048", "lens_k": "2300,511,1285,9216", "causal": True},
        # a training step's attention: short packed samples on a share with
        # narrow heads, and 4096 tokens of two samples
        {"name": "train_short", "op": "train", "heads": 16, "kv_heads": 2, "dim": 64, "lens_q": "17,129,385",
         "lens_k": "17,129,385", "causal": True},
        {"name": "train_4096", "op": "train", "heads": 64, "kv_heads": 8, "dim": 128, "lens_q": "2500,1596",
         "lens_k": "2500,1596", "causal": True},
    ]


def _cost(case):
    w = work(case)
    return w["bytes"] / 5e12 + w["flops"] / 1e15


def draw(rng):
    def span(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    while True:
        op = rng.choice(("norm", "append", "decode", "prompt", "train"))
        kv = rng.choice((1, 2, 3, 4, 8, 16))
        dim = rng.choice((64, 128, 128))
        heads = kv * rng.choice((1, 2, 4, 5, 6, 8, 8, 12, 16))
        if heads > 128:
            continue
        if op == "norm":
            case = {"op": op, "tokens": span(1, 8192), "heads": heads, "kv_heads": kv, "dim": dim,
                    "rot": rng.choice((dim // 4, dim // 2, dim, dim)), "interleaved": rng.random() < 0.4,
                    "back": rng.random() < 0.5}
        elif op == "append":
            one = rng.random() < 0.5
            new = [1 if one else span(1, 4096) for _ in range(span(1, 96 if one else 6))]
            case = {"op": op, "kv_heads": kv, "dim": dim, "page": rng.choice((16, 32, 48, 64, 128)),
                    "new": _text(new), "lens": _text([n + span(1, 5000) - 1 for n in new])}
        elif op == "decode":
            nq = rng.choice((1, 1, 1, 2, span(3, 32)))
            case = {"op": op, "heads": heads, "kv_heads": kv, "dim": dim, "nq": nq,
                    "tree": nq > 1 and rng.random() < 0.5, "page": rng.choice((16, 32, 48, 64, 128)),
                    "lens": _text([nq + span(1, 60000) - 1 for _ in range(span(1, 64))])}
        else:
            lq = [span(1, 4096) for _ in range(span(1, 6))]
            if op == "train" and max(lq) < 16:
                continue        # a lone key takes all the weight: the queries' gradient is zero, its digits are noise
            lk = lq if op == "train" or rng.random() < 0.5 else [n + span(1, 6000) - 1 for n in lq]
            case = {"op": op, "heads": heads, "kv_heads": kv, "dim": dim, "lens_q": _text(lq), "lens_k": _text(lk),
                    "causal": rng.random() < 0.8}
        if _cost(case) <= max(_cost(c) for c in listed() if c["op"] == op):
            return case


def _pairs(case):
    """Query-key pairs that the mask leaves, per head."""
    n = 0
    for lq, lk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
        n += lq * lk - (lq * (lq - 1) // 2 if case["causal"] else 0)
    return n


def work(case):
    kv, dim = case["kv_heads"], case["dim"]
    if case["op"] == "norm":
        n = case["tokens"] * (case["heads"] + kv) * dim
        # queries and keys read and written once; two rows of angles, the
        # position; the weights. Backward: inputs and gradients read,
        # gradients written
        return {"bytes": n * 4 + case["tokens"] * (case["rot"] * 4 + 4) + 4 * dim
                + (n * 6 + case["tokens"] * (case["rot"] * 4 + 4) + 12 * dim if case["back"] else 0),
                "flops": n * (7 + (13 if case["back"] else 0))}
    if case["op"] == "append":
        t = sum(_ints(case["new"]))
        # a value read in 16 bits and written in 8; scales of the touched blocks
        return {"bytes": t * kv * dim * 6 + 2 * kv * (t // BLOCK + 1), "flops": t * kv * dim * 4}
    h = case["heads"]
    if case["op"] == "decode":
        lens, nq = _ints(case["lens"]), case["nq"]
        t = nq * len(lens)
        pairs = sum(nq * n - nq * (nq - 1) // 2 for n in lens)
        return {"bytes": sum(lens) * kv * 2 * dim + sum(-(-n // BLOCK) for n in lens) * kv * 2 + t * h * dim * 4
                + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": 4 * pairs * h * dim}
    tq, tk = sum(_ints(case["lens_q"])), sum(_ints(case["lens_k"]))
    b_in = tq * h * dim * 2 + tk * kv * dim * 4
    b_out = tq * h * (dim * 2 + 4)
    pairs = _pairs(case)
    if case["op"] == "prompt":
        return {"bytes": b_in + b_out, "flops": 4 * pairs * h * dim}
    # with the backward: the inputs' gradients written, the output's gradient
    # read; four more products (dV, dP, dQ, dK)
    return {"bytes": 2 * b_in + b_out + tq * h * dim * 2, "flops": 12 * pairs * h * dim}


# ---------------------------------------------------------------- the inputs
def _randn(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _tree_masks(seed, n_seq, nq):
    """Bit j of token i's word: i may see drafted token j (itself and its
    ancestors). Each token's parent is one of the four before it, or the
    request's last accepted token."""
    import random
    rng = random.Random(seed)
    words = []
    for _ in range(n_seq):
        m = []
        for i in range(nq):
            p = rng.randrange(max(-1, i - 4), i) if i else -1
            m.append((m[p] if p >= 0 else 0) | (1 << i))
        words += m
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def _cached(gen, st, lens, page, kv, dim):
    """A cache whose pages hold the requests' tokens in random order."""
    pages = [-(-n // page) for n in lens]
    n_pages = sum(pages) + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(pages), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = perm[at:at + n]
        at += n
    blocks = page // BLOCK

    def codes(*tail):
        out = torch.empty(n_pages, kv, blocks, *tail, dtype=torch.uint8, device="cuda")
        flat = out.view(-1)
        for i in range(0, flat.numel(), 1 << 28):
            n = min(1 << 28, flat.numel() - i)
            x = torch.randn(n, generator=gen, device="cuda").mul_(112.0).clamp_(-448.0, 448.0)
            flat[i:i + n] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        return out

    st["k"], st["v"] = codes(dim // 16, BLOCK, 16), codes(dim // 2, 2, 2, 2, 4)
    for name in ("k_scales", "v_scales"):
        st[name] = torch.randint(119, 122, (n_pages, kv, blocks), generator=gen, device="cuda").to(torch.uint8)
    st["table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"op": case["op"], "case": dict(case)}
    kv, dim = case["kv_heads"], case["dim"]
    if case["op"] == "norm":
        t, h = case["tokens"], case["heads"]
        # queries, keys and values of a token lie together, as the projection writes them
        st["qkv"] = _randn(gen, t, (h + 2 * kv) * dim) * (0.5 + torch.rand(t, 1, generator=gen, device="cuda")).to(torch.bfloat16)
        st["q"] = st["qkv"][:, :h * dim].unflatten(1, (h, dim))
        st["kk"] = st["qkv"][:, h * dim:(h + kv) * dim].unflatten(1, (kv, dim))
        for name in ("w_q", "w_k"):
            st[name] = (1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(torch.bfloat16)
        max_pos = 16384
        freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        ang = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq[None]
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["pos"] = torch.randint(0, max_pos, (t,), generator=gen, device="cuda", dtype=torch.int32)
        if case["back"]:
            st["dq_out"], st["dk_out"] = _randn(gen, t, h, dim), _randn(gen, t, kv, dim)
        if own:
            import mixture_experts_layer_sigmoid_amd as moe
            st["plan"] = moe.QKNormRope(T=t, n_heads=h, n_kv_heads=kv, head_dim=dim, rotary=case["rot"],
                                        interleaved=case["interleaved"], eps=EPS, backward=case["back"])
        return st
    if case["op"] == "append":
        new, lens = _ints(case["new"]), _ints(case["lens"])
        _cached(gen, st, lens, case["page"], kv, dim)
        st["cu"] = _cu(new)
        t = sum(new)
        grow = torch.exp2(torch.randint(-1, 3, (t, 1, 1), generator=gen, device="cuda").float())
        st["k_new"] = (torch.randn(t, kv, dim, generator=gen, device="cuda") * grow).to(torch.bfloat16)
        st["v_new"] = (torch.randn(t, kv, dim, generator=gen, device="cuda") * grow).to(torch.bfloat16)
        if own:
            import mixture_experts_layer_sigmoid_amd as moe
            st["cache"] = moe.GroupedCache(st["k"], st["v"], st["k_scales"], st["v_scales"])
        return st
    h = case["heads"]
    if case["op"] == "decode":
        lens, nq = _ints(case["lens"]), case["nq"]
        _cached(gen, st, lens, case["page"], kv, dim)
        st["cu"] = _cu([nq] * len(lens))
        st["q"] = _randn(gen, nq * len(lens), h, dim)
        st["tree"] = _tree_masks(seed, len(lens), nq) if case["tree"] else None
        if own:
            import mixture_experts_layer_sigmoid_amd as moe
            st["cache"] = moe.GroupedCache(st["k"], st["v"], st["k_scales"], st["v_scales"])
            st["plan"] = moe.GroupedDecode(n_heads=h, n_kv_heads=kv, head_dim=dim, max_tokens=nq * len(lens),
                                           max_seqs=len(lens))
        return st
    lq, lk = _ints(case["lens_q"]), _ints(case["lens_k"])
    tq, tk = sum(lq), sum(lk)
    st["cu_q"], st["cu_k"] = _cu(lq), _cu(lk)
    st["q"] = _randn(gen, tq, h, dim)
    st["kk"], st["vv"] = _randn(gen, tk, kv, dim), _randn(gen, tk, kv, dim)
    if case["op"] == "train":
        st["dout"] = _randn(gen, tq, h, dim)
    if own:
        import mixture_experts_layer_sigmoid_amd as moe
        st["plan"] = moe.GroupedAttention(Tq=tq, Tk=tk, n_heads=h, n_kv_heads=kv, head_dim=dim, n_seqs=len(lq),
                                          causal=case["causal"], backward=case["op"] == "train")
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    return (_run_own if own else _run_plain)(st)


def _cache_values(st):
    """The cache as the numbers its bytes are: E4M3 codes and the scales' exponents."""
    f8 = torch.float8_e4m3fn
    return {"k": st["k"].view(f8), "v": st["v"].view(f8), "k_scales": st["k_scales"], "v_scales": st["v_scales"]}


def _run_own(st):
    import mixture_experts_layer_sigmoid_amd as moe
    if st["op"] == "norm":
        a = st["plan"]
        ins = (st["q"], st["kk"], st["w_q"], st["w_k"], st["cos"], st["sin"], st["pos"])
        q, k = a.forward(*ins)
        if not st["case"]["back"]:
            return {"q": q, "k": k}
        dq, dk, dw_q, dw_k = a.backward(st["dq_out"], st["dk_out"], *ins)
        return {"q": q, "k": k, "dq": dq, "dk": dk, "dw_q": dw_q, "dw_k": dw_k}
    if st["op"] == "append":
        moe.grouped_cache_append(st["k_new"], st["v_new"], st["cache"], st["table"], st["lens"], st["cu"])
        return _cache_values(st)
    if st["op"] == "decode":
        return {"out": st["plan"](st["q"], st["cache"], st["table"], st["lens"], st["cu"], st["tree"])}
    a = st["plan"]
    out, lse = a.forward(st["q"], st["kk"], st["vv"], st["cu_q"], st["cu_k"])
    if st["op"] == "prompt":
        return {"out": out, "lse": lse}
    dq, dk, dv = a.backward(st["dout"], st["q"], st["kk"], st["vv"], st["cu_q"], st["cu_k"])
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _run_plain(st):
    return {"norm": _plain_norm, "append": _plain_append, "decode": _plain_decode, "prompt": _plain_attention,
            "train": _plain_attention}[st["op"]](st)


def _turn(x, cos, sin, interleaved):
    """The first values of every head rotated; cos, sin [tokens, 1, pairs]."""
    r = 2 * cos.shape[-1]
    rot, rest = x[..., :r], x[..., r:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :r // 2], rot[..., r // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    rot = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((rot, rest), -1)


def _plain_norm(st):
    case, bf = st["case"], torch.bfloat16
    pos = st["pos"].long()
    cos, sin = st["cos"][pos][:, None], st["sin"][pos][:, None]
    res = {}
    for x, w, d, name in ((st["q"], st["w_q"], "dq_out", "q"), (st["kk"], st["w_k"], "dk_out", "k")):
        x, w = x.float(), w.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh = x * r
        res[name] = _turn(xh * w, cos, sin, case["interleaved"]).to(bf)
        if case["back"]:
            g = _turn(st[d].float(), cos, -sin, case["interleaved"])     # rotated back
            res["dw_" + name] = (g * xh).sum((0, 1))
            gw = g * w
            res["d" + name] = (r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(bf)
    return res


def _plain_append(st):
    dev, page = st["k_new"].device, st["case"]["page"]
    b = st["lens"].shape[0]
    t, kv, dim = st["k_new"].shape
    n_new = (st["cu"][1:] - st["cu"][:-1]).long()
    start = st["lens"].long() - n_new                                       # first new position
    req = torch.repeat_interleave(torch.arange(b, device=dev), n_new, output_size=t)
    pos = torch.arange(t, device=dev) - st["cu"].long()[req] + start[req]
    where = st["table"].long()[req, pos // page] * (page // BLOCK) + pos % page // BLOCK    # block of each token
    at = pos % BLOCK
    blocks = torch.unique(where)
    which = torch.searchsorted(blocks, where)
    first = torch.full((blocks.numel(),), BLOCK, device=dev).scatter_reduce(0, which, at, "amin")   # earlier tokens
    pg, bl = blocks // (page // BLOCK), blocks % (page // BLOCK)
    old = torch.arange(BLOCK, device=dev) < first[:, None]                  # [blocks, 16]
    for x, name in ((st["k_new"], "k"), (st["v_new"], "v")):
        codes, scales = st[name], st[name + "_scales"]
        x = x.float()
        amax = torch.zeros(blocks.numel(), kv, device=dev).index_reduce(0, which, x.abs().amax(-1), "amax")
        frac, e = torch.frexp(amax)                                         # amax = frac 2^e, frac in [1/2, 1)
        e = torch.where(amax == 0, torch.full_like(e, -127), (e - 9 + (frac > 0.875).int()).clamp(-127, 127))
        had = scales[pg, :, bl].int() - 127
        e = torch.where((first > 0)[:, None], torch.maximum(e, had), e)
        c = codes[pg, :, bl]                                                # [blocks, kv, the block's order]
        if name == "k":
            c = c.permute(0, 3, 1, 2, 4).reshape(-1, BLOCK, kv, dim)
        else:
            c = c.permute(0, 5, 3, 6, 1, 2, 4).reshape(-1, BLOCK, kv, dim)
        c = c.contiguous()
        moved = (c.view(torch.float8_e4m3fn).float() * torch.exp2((had - e).clamp(min=-60).float())[:, None, :, None])
        c = torch.where(old[:, :, None, None], moved.to(torch.float8_e4m3fn).view(torch.uint8), c)
        c[which, at] = (x * torch.exp2(-e[which].float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        if name == "k":
            c = c.view(-1, BLOCK, kv, dim // 16, 16).permute(0, 2, 3, 1, 4)
        else:
            c = c.view(-1, 2, 2, 4, kv, dim // 2, 2).permute(0, 4, 5, 2, 6, 1, 3)
        codes[pg, :, bl] = c
        scales[pg, :, bl] = (e + 127).to(torch.uint8)
    return _cache_values(st)


def _rows(st, table):
    """Keys and values [requests, kv_heads, tokens, dim] of the pages in table."""
    n, cols = table.shape
    out = []
    for name, order in (("k", (0, 2, 1, 3, 5, 4, 6)), ("v", (0, 2, 1, 3, 7, 5, 8, 4, 6))):
        c = st[name][table]                                    # [n, pages, kv, blocks, the block's order]
        x = c.view(torch.float8_e4m3fn).float()
        s = torch.exp2(st[name + "_scales"][table].float() - 127)
        x = (x * s.reshape(*s.shape, *([1] * (x.dim() - 4)))).permute(*order)
        out.append(x.reshape(n, x.shape[1], -1, st["case"]["dim"]))
    return out


def _plain_decode(st):
    case = st["case"]
    b, nq, h, kv, dim = st["lens"].shape[0], case["nq"], case["heads"], case["kv_heads"], case["dim"]
    dev, g = st["q"].device, case["heads"] // case["kv_heads"]
    q = st["q"].float().view(b, nq, kv, g, dim).permute(0, 2, 1, 3, 4).reshape(b, kv, nq * g, dim)
    span = st["table"].shape[1] * case["page"]
    out = torch.empty(b, kv, nq * g, dim, device=dev)
    step = max(1, (1 << 31) // (kv * span * (nq * g + 2 * dim)))
    pos = torch.arange(span, device=dev)
    tok = torch.arange(nq, device=dev)[None, :, None]
    for i in range(0, b, step):
        k, v = _rows(st, st["table"][i:i + step].long())
        off = pos - (st["lens"][i:i + step].long() - nq)[:, None, None]       # from the first new token
        if st["tree"] is None:
            see = off <= tok
        else:
            words = st["tree"].view(b, nq)[i:i + step, :, None]
            see = (off < 0) | (((words >> off.clamp(0, 63)) & 1).bool() & (off < nq))
        see = see.expand(-1, nq, -1).repeat_interleave(g, 1)[:, None]
        n = k.shape[0]
        s = torch.bmm(q[i:i + step].reshape(n * kv, nq * g, dim), k.view(n * kv, span, dim).transpose(1, 2).contiguous())
        s = torch.where(see, s.view(n, kv, nq * g, span) * dim ** -0.5, -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.bmm(p.view(n * kv, nq * g, span), v.view(n * kv, span, dim)).view(n, kv, nq * g, dim)
        out[i:i + step] = o / p.sum(-1, keepdim=True)
    out = out.view(b, kv, nq, g, dim).permute(0, 2, 1, 3, 4).reshape(b * nq, h, dim)
    return {"out": out.to(torch.bfloat16)}


def _plain_attention(st):
    case, dev, bf = st["case"], st["q"].device, torch.bfloat16
    tq, h, dim = st["q"].shape
    kv = case["kv_heads"]
    g, scale, train = h // kv, dim ** -0.5, case["op"] == "train"
    res = {"out": torch.empty_like(st["q"]), "lse": torch.empty(tq, h, device=dev)}
    if train:
        res.update(dq=torch.empty_like(st["q"]), dk=torch.empty_like(st["kk"]), dv=torch.empty_like(st["vv"]))
    a = c = 0
    for lq, lk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
        sq, sk = slice(a, a + lq), slice(c, c + lk)
        a, c = a + lq, c + lk
        i = torch.arange(lq, device=dev).repeat_interleave(g)[:, None]
        hide = (torch.arange(lk, device=dev)[None] - i > lk - lq) if case["causal"] else None
        step = max(1, (1 << 30) // max(1, lq * g * lk))

        def rows(x, hs):                                   # [kv heads, queries x heads of the group, dim]
            n = hs.stop - hs.start
            return x.view(tq, kv, g, dim)[sq, hs].permute(1, 0, 2, 3).float().reshape(n, lq * g, dim)

        def put(x, hs, y):
            x.view(tq, kv, g, -1)[sq, hs] = y.view(-1, lq, g, y.shape[-1]).permute(1, 0, 2, 3).to(x.dtype)

        for k0 in range(0, kv, step):
            hs = slice(k0, min(kv, k0 + step))
            q = rows(st["q"], hs)
            k, v = (st[n][sk, hs].transpose(0, 1).float().contiguous() for n in ("kk", "vv"))
            s = torch.bmm(q, k.transpose(1, 2).contiguous()) * scale
            if hide is not None:
                s.masked_fill_(hide, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            z = p.sum(-1, keepdim=True)
            p = p / z
            o = torch.bmm(p, v)
            put(res["out"], hs, o)
            put(res["lse"], hs, m + torch.log(z))
            if not train:
                continue
            do = rows(st["dout"], hs)
            res["dv"][sk, hs] = torch.bmm(p.transpose(1, 2).contiguous(), do).transpose(0, 1).to(bf)
            dp = torch.bmm(do, v.transpose(1, 2).contiguous())
            ds = p * (dp - (do * o).sum(-1, keepdim=True)) * scale
            put(res["dq"], hs, torch.bmm(ds, k))
            res["dk"][sk, hs] = torch.bmm(ds.transpose(1, 2).contiguous(), q).transpose(0, 1).to(bf)
    return res


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "decode": _exact_decode, "prompt": _exact_attention,
            "train": _exact_attention}[case["op"]](st, case)


def _exact_norm(st, case):
    """Pairs as complex numbers times e^{i angle}; the gradient by the
    chain rule through the norm's Jacobian, head by head."""
    turn = torch.complex(st["cos"].double(), st["sin"].double())[st["pos"].long()]
    r = case["rot"]

    def spin(x, t):
        y = x.clone()
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous()) * t
            y[..., :r] = torch.view_as_real(z).reshape(*x.shape[:-1], r)
        else:
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * t
            y[..., :r] = torch.cat((z.real, z.imag), -1)
        return y

    res = {}
    for name, src in (("q", "q"), ("k", "kk")):
        w = st["w_" + name].double()
        outs, grads, dw = [], [], torch.zeros_like(w)
        for head in range(st[src].shape[1]):
            x = st[src][:, head].double()
            norm = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
            outs.append(spin(x / norm * w, turn))
            if case["back"]:
                g = spin(st["d%s_out" % name][:, head].double(), turn.conj())
                dw += (g * x / norm).sum(0)
                along = (g * w * x).sum(-1, keepdim=True)
                grads.append(g * w / norm - x * along / (x.shape[-1] * norm.pow(3)))
        res[name] = torch.stack(outs, 1)
        if case["back"]:
            res["d" + name], res["dw_" + name] = torch.stack(grads, 1), dw
    return res


def _exact_append(st, case):
    """Token by block, request by request: the values over the block's scale, not rounded; the rest of the cache as it was."""
    page = case["page"]
    res, cu = {}, _ints(_text(st["cu"].tolist()))
    for name in ("k", "v"):
        codes = st[name].view(torch.float8_e4m3fn).double()
        scales = st[name + "_scales"].clone()
        flat = codes.flatten(3)
        dim = case["dim"]
        d, t = torch.arange(dim, device="cuda")[None], torch.arange(BLOCK, device="cuda")[:, None]
        if name == "k":
            at = (d // 16) * 256 + t * 16 + d % 16
        else:
            at = (d // 2) * 32 + (t // 4 % 2) * 16 + (d % 2) * 8 + (t // 8) * 4 + t % 4
        for b, (n, new) in enumerate(zip(_ints(case["lens"]), _ints(case["new"]))):
            x = st[name + "_new"][cu[b]:cu[b + 1]].double()
            start = n - new
            lo = start // BLOCK * BLOCK
            nb = -(-n // BLOCK) - start // BLOCK
            full = torch.zeros(nb * BLOCK, x.shape[1], dim, dtype=torch.float64, device="cuda")
            full[start - lo:start - lo + new] = x
            full = full.view(nb, BLOCK, -1, dim)
            amax = full.abs().amax((1, 3))                                       # [blocks, heads]
            e = torch.ceil(torch.log2(amax / 448)).clamp(-127, 127)
            e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
            e = torch.where(448 * torch.exp2(e - 1) >= amax, e - 1, e).clamp(-127, 127)
            blk = torch.arange(nb, device="cuda") + lo // BLOCK
            pg, bl = st["table"][b].long()[blk // (page // BLOCK)], blk % (page // BLOCK)
            was = scales[pg, :, bl].double() - 127
            if start > lo:
                e[0] = torch.maximum(e[0], was[0])
            val = full / torch.exp2(e)[:, None, :, None]
            pos = torch.arange(nb * BLOCK, device="cuda").view(nb, BLOCK) + lo
            had = flat[pg, :, bl][:, :, at].permute(0, 2, 1, 3)                  # [blocks, 16, heads, dim]
            had = torch.where((pos < start)[..., None, None], had * torch.exp2(was - e)[:, None, :, None], had)
            val = torch.where(((pos >= start) & (pos < n))[..., None, None], val, had).permute(0, 2, 1, 3)
            rows = flat[pg, :, bl]
            rows[:, :, at] = val
            flat[pg, :, bl] = rows
            scales[pg, :, bl] = (e + 127).to(torch.uint8)
        res[name], res[name + "_scales"] = flat.view(codes.shape), scales
    return res


def _exact_decode(st, case):
    """Request by request, head by head, over its own rows."""
    kv, dim, nq, page = case["kv_heads"], case["dim"], case["nq"], case["page"]
    g = case["heads"] // kv
    outs = []
    for b, n in enumerate(_ints(case["lens"])):
        k, v = _rows(st, st["table"][b:b + 1, :-(-n // page)].long())
        q = st["q"][b * nq:(b + 1) * nq].double()
        o = torch.empty_like(q)
        for head in range(kv):
            kh, vh = k[0, head, :n].double(), v[0, head, :n].double()
            s = torch.matmul(q[:, head * g:(head + 1) * g], kh.t()) / math.sqrt(dim)     # [nq, g, n]
            for i in range(nq):
                if st["tree"] is None:
                    s[i, :, n - nq + i + 1:] = -math.inf
                else:
                    word = int(st["tree"][b * nq + i])
                    s[i][:, [n - nq + j for j in range(nq) if not (word >> j) & 1]] = -math.inf
            o[:, head * g:(head + 1) * g] = torch.matmul(torch.softmax(s, -1), vh)
        outs.append(o)
    return {"out": torch.cat(outs)}


def _exact_attention(st, case):
    """Query head by query head; the backward from dP and the softmax's Jacobian."""
    h, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    train, g = case["op"] == "train", h // kv
    q, k, v = st["q"].double(), st["kk"].double(), st["vv"].double()
    res = {"out": torch.empty_like(q), "lse": torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")}
    if train:
        do = st["dout"].double()
        res.update(dq=torch.empty_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    a = c = 0
    for nq, nk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
        rq, rk = slice(a, a + nq), slice(c, c + nk)
        a, c = a + nq, c + nk
        for head in range(h):
            j = head // g
            s = (q[rq, head] @ k[rk, j].t()) / math.sqrt(dim)
            if case["causal"]:
                s += torch.full_like(s, -math.inf).triu(nk - nq + 1)
            l = torch.logsumexp(s, 1)
            p = (s - l[:, None]).exp()
            res["out"][rq, head], res["lse"][rq, head] = p @ v[rk, j], l
            if train:
                dp = do[rq, head] @ v[rk, j].t()
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(dim)
                res["dq"][rq, head] = ds @ k[rk, j]
                res["dk"][rk, j] += ds.t() @ q[rq, head]
                res["dv"][rk, j] += p.t() @ do[rq, head]
    return res
