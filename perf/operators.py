"""The operators on either side of the attention, as they are measured.

qkv_rope     norms of queries and keys for each head and the rotary positions (one or several axes) in one pass,
             from the projection's token-major output to the attention's head-major tensors; and its backward pass
kv4_append   tokens written into a key/value cache held in 4 bits (kv4_read gives back what was written)
kv4_decode   gated block-sparse decode over such a cache

A 4-bit cache row holds one token of one head: 32 channels share an fp16 scale s and an fp16 minimum m, and channel
value n in 0..15 stands for m + s n. Channel c sits in the 16-bit word (c % 32) // 4 * (d // 32) + c // 32 of the row, at
bits 4 (c % 4) of it.
"""
import math

import torch

own = False

BLOCK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _binding():
    from gated_block_sparse_gate_b200 import binding

    return binding


# ----------------------------------------------------------------------- cases


def _rope(name, **kw):
    case = dict(name=name, op="rope", B=1, N=1, Hq=32, Hkv=8, d=128, rot=128, axes=1, interleaved=False, norm=True,
                backward=False, dtype="bf16", max_pos=131072)
    case.update(kw)
    return case


def _append(name, **kw):
    case = dict(name=name, op="append", B=1, T=1, Hkv=8, d=128, L=8192, paged=True, ragged=False, dtype="bf16")
    case.update(kw)
    return case


def _decode(name, **kw):
    case = dict(name=name, op="decode", B=1, L=1000, Hq=32, Hkv=8, d=128, topk=32, tau=0.0, paged=False, varlen=False,
                shared=False, dtype="bf16")
    case.update(kw)
    return case


def listed():
    return [
        # one new token for each of 64 sequences, far into their contexts: the step before a decode
        _rope("rope_step_b64", B=64),
        # one training step of the 8192-token workload: forward and backward
        _rope("rope_train_n8192", N=8192, backward=True),
        # a long prompt of text and images: positions on three axes (time, height, width)
        _rope("rope_prefill_3axes_n65536", N=65536, axes=3),
        # exact fp32 training of a small model: odd length, neighbouring pairs, half of the channels left unrotated
        _rope("rope_train_f32_odd", B=3, N=1021, Hq=6, Hkv=2, d=64, rot=32, interleaved=True, backward=True,
              dtype="f32", max_pos=2048),
        # the decode step's one token of 64 sequences into their pages
        _append("append_step_b64", B=64),
        # a prompt of 32768 tokens into a contiguous cache
        _append("append_prompt_n32768", T=32768, L=32768, paged=False),
        # a batch of prompts of different lengths, fp32 keys and values, odd offsets
        _append("append_ragged_f32", B=7, T=509, Hkv=2, d=64, L=2000, ragged=True, dtype="f32"),
        # a single short conversation: the latency of one call
        _decode("decode_b1_l1000", L=1000, topk=4),
        # the decode workload: 64 sequences of 131072 tokens, 32 blocks for each query head
        _decode("decode_b64_l131072", B=64, L=131072),
        # the same with one selection for the query heads of a group, over pages
        _decode("decode_shared_paged_b64_l131072", B=64, L=131072, paged=True, shared=True),
        # a serving batch of uneven lengths (an idle slot among them), gates over a threshold, three query heads to one
        _decode("decode_varlen_tau_d64", B=17, L=20011, Hq=6, Hkv=2, d=64, topk=48, tau=0.002, paged=True, varlen=True),
        # exact fp32 queries over the cache
        _decode("decode_f32_varlen", B=4, L=4133, Hq=8, Hkv=2, topk=8, paged=True, varlen=True, shared=True,
                dtype="f32"),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("rope", "append", "decode", "decode"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 8, 12) if Hkv * g <= 32])
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "rope":
        backward = rng.random() < 0.5
        B = _span(rng, 1, 64)
        most = 60000 * 48 * 128 * 2 // (B * (Hq + 2 * Hkv) * d * (2 if dtype == "bf16" else 4) * (3 if backward else 1))
        c = _rope("", B=B, N=_span(rng, 1, max(1, min(60000, most))), Hq=Hq, Hkv=Hkv, d=d,
                  rot=rng.choice((d, d, d // 2, d // 4, 3 * d // 8)), axes=rng.choice((1, 1, 2, 3)),
                  interleaved=rng.random() < 0.4, norm=rng.random() < 0.75, backward=backward, dtype=dtype)
    elif op == "append":
        B, L = _span(rng, 1, 64), _span(rng, 70, 30000)
        most = 30000 * 8 * 128 // (B * Hkv * d)
        c = _append("", B=B, T=min(L, _span(rng, 1, max(1, most))), Hkv=Hkv, d=d, L=L, paged=rng.random() < 0.6,
                    ragged=rng.random() < 0.5, dtype=dtype)
    else:
        B, L = _span(rng, 1, 64), _span(rng, 1, 120000)
        if dtype == "f32":
            B, L = min(B, 16), min(L, 30000)
        c = _decode("", B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, topk=_span(rng, 1, 32), tau=rng.choice((0.0, 0.0, 0.003)),
                    paged=rng.random() < 0.5, varlen=rng.random() < 0.5, shared=rng.random() < 0.5, dtype=dtype)
    del c["name"]
    return c


# ----------------------------------------------------------------------- inputs


def _axis_of(case):
    """The axis of every rotated pair: equal sections, the last with what is left."""
    pairs, axes = case["rot"] // 2, case["axes"]
    return [min(i * axes // pairs, axes - 1) for i in range(pairs)]


def _positions(case, g):
    """int32 [B, N] or [B, N, axes]: consecutive tokens from a random offset; on several axes runs of text (all axes
    alike) and of image patches (one time, rows and columns of a 32-wide grid)."""
    B, N, A, P = case["B"], case["N"], case["axes"], case["max_pos"]
    off = torch.randint(0, max(1, P - N), (B, 1), generator=g, device="cuda")
    t = off + torch.arange(N, device="cuda")
    if A == 1:
        return t.to(torch.int32)
    i = torch.arange(N, device="cuda") % 1280
    patch = (i - 256).clamp(min=0)
    begin = t - patch
    pos = torch.stack([begin, begin + patch // 32, begin + patch % 32][:A], -1)
    pos = torch.where((i >= 256)[:, None], pos, t[..., None])
    return pos.clamp(0, P - 1).to(torch.int32).contiguous()


def _prepare_rope(case, g):
    B, N, Hq, Hkv, d = (case[k] for k in ("B", "N", "Hq", "Hkv", "d"))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    half = case["rot"] // 2
    angle = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] \
        * 500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    st = dict(case=case, qkv=normal(B, N, Hq + 2 * Hkv, d), pos=_positions(case, g), axes=_axis_of(case),
              cos=angle.cos().float().contiguous(), sin=angle.sin().float().contiguous(), wq=None, wk=None)
    if case["norm"]:
        st["wq"], st["wk"] = (1 + 0.2 * torch.randn(2, d, generator=g, device="cuda")).unbind()
    if case["backward"]:
        st.update(dQ=normal(B, Hq, N, d), dK=normal(B, Hkv, N, d), dV=normal(B, Hkv, N, d),
                  dqkv=torch.empty(B, N, Hq + 2 * Hkv, d, dtype=dt, device="cuda"))
    return st


def _cache(case, g, codes):
    """A 4-bit cache of the case's layout (contiguous or pages in a random order) and its block table."""
    B, Hkv, d, nb = case["B"], case["Hkv"], case["d"], -(-case["L"] // BLOCK)
    shape, table = (B, Hkv, nb * BLOCK), None
    if case["paged"]:
        pages = B * nb + 3
        shape = (pages, Hkv, BLOCK)
        table = torch.randperm(pages, generator=g, device="cuda")[:B * nb].view(B, nb).to(torch.int32)
    out = []
    for _ in range(2):
        if codes:
            c = torch.randint(0, 256, (*shape, d // 2), generator=g, device="cuda", dtype=torch.uint8)
            p = torch.rand(*shape, d // 32, 2, generator=g, device="cuda", dtype=torch.float16)
            p[..., 0].mul_(0.15).add_(0.2)    # a step of 0.2 to 0.35: groups of 32 standard normal values
            p[..., 1].sub_(2.6)               # a smallest value of -2.6 to -1.6
        else:
            c = torch.zeros(*shape, d // 2, device="cuda", dtype=torch.uint8)
            p = torch.zeros(*shape, d // 32, 2, device="cuda", dtype=torch.float16)
        out += [c, p]
    return out, table


def _prepare_append(case, g):
    B, T, Hkv, d, L = (case[k] for k in ("B", "T", "Hkv", "d", "L"))
    cache, table = _cache(case, g, False)
    count = None
    if case["ragged"]:
        count = torch.randint(0, T + 1, (B,), generator=g, device="cuda").to(torch.int32)
    start = torch.randint(0, L - T + 1, (B,), generator=g, device="cuda").to(torch.int32)
    spread = torch.exp(0.5 * torch.randn(Hkv, 1, d, generator=g, device="cuda"))  # channels of unlike sizes
    dt = DTYPES[case["dtype"]]
    K, V = ((torch.randn(B, Hkv, T, d, generator=g, device="cuda") * spread).to(dt) for _ in range(2))
    return dict(case=case, cache=cache, table=table, start=start, count=count, K=K, V=V)


def _prepare_decode(case, g):
    B, Hq, Hkv, d, L = (case[k] for k in ("B", "Hq", "Hkv", "d", "L"))
    cache, table = _cache(case, g, True)
    lens = None
    if case["varlen"]:
        lens = torch.randint(1, L + 1, (B,), generator=g, device="cuda").to(torch.int32)
        lens[0] = L
        if B > 2:
            lens[1] = 0
    q = torch.randn(B, Hq, d, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    S = math.sqrt(2) * torch.randn(B, Hkv if case["shared"] else Hq, -(-L // BLOCK), generator=g, device="cuda")
    return dict(case=case, cache=cache, table=table, lens=lens, q=q, S=S)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    case = dict(case)
    return {"rope": _prepare_rope, "append": _prepare_append, "decode": _prepare_decode}[case["op"]](case, g)


# ----------------------------------------------------------------------- plain forms


def _angles(st):
    """cos and sin [B, N, 1, rot / 2] of every rotated pair."""
    pos = st["pos"].long()
    pos = pos if pos.dim() == 3 else pos[..., None]
    at = pos[..., torch.tensor(st["axes"], device="cuda")]
    pair = torch.arange(at.shape[-1], device="cuda")
    return st["cos"][at, pair][:, :, None], st["sin"][at, pair][:, :, None]


def _rotate(y, c, s, interleaved):
    rot = 2 * c.shape[-1]
    z = y.clone()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z[..., 0:rot:2], z[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z[..., :rot // 2], z[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return z


EPS = 1e-6


def _plain_rope(st):
    case = st["case"]
    Hq, Hkv, dt = case["Hq"], case["Hkv"], st["qkv"].dtype
    q, k, v = st["qkv"].split((Hq, Hkv, Hkv), dim=2)
    c, s = _angles(st)
    out = {}
    for name, x, w in (("Q", q, st["wq"]), ("K", k, st["wk"])):
        y = x.float()
        if w is not None:
            y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * w
        out[name] = _rotate(y, c, s, case["interleaved"]).to(dt).transpose(1, 2).contiguous()
    out["V"] = v.transpose(1, 2).contiguous()
    if not case["backward"]:
        return out
    grads = []
    for name, x, w, dz in (("q", q, st["wq"], st["dQ"]), ("k", k, st["wk"], st["dK"])):
        g = _rotate(dz.float().transpose(1, 2), c, -s, case["interleaved"])
        if w is not None:
            x = x.float()
            r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            xh = x * r
            out["dw" + name] = (g * xh).sum((0, 1, 2))
            h = g * w
            g = r * (h - xh * (h * xh).mean(-1, keepdim=True))
        grads.append(g.to(dt))
    out["dqkv"] = torch.cat([*grads, st["dV"].transpose(1, 2)], dim=2)
    return out


def _values(codes, params):
    """The fp32 values [..., d] that 4-bit rows stand for."""
    d = 2 * codes.shape[-1]
    n = torch.stack((codes & 15, codes >> 4), -1).view(*codes.shape[:-1], 8, d // 32, 4).transpose(-3, -2)
    p = params.float()
    return (p[..., 1, None, None] + p[..., 0, None, None] * n).reshape(*codes.shape[:-1], d)


def _quantise(x):
    """(codes, params) of rows [..., d]; 64 bits, so that values next to a border go to the side they are on."""
    d = x.shape[-1]
    x = x.double().view(*x.shape[:-1], d // 32, 8, 4)
    lo, hi = x.amin((-1, -2)).clamp(-60000, 60000), x.amax((-1, -2)).clamp(-60000, 60000)
    m = lo.float().half()
    s = ((hi - m.double()) / 15).float().half()
    n = ((x - m.double()[..., None, None]) / s.double()[..., None, None]).round().clamp(0, 15)
    n = torch.where(s[..., None, None] > 0, n, 0).to(torch.uint8).transpose(-3, -2).reshape(*x.shape[:-3], d // 2, 2)
    return n[..., 0] | n[..., 1] << 4, torch.stack((s, m), -1)


def _rows(st, T):
    """The cache index (page or sequence, row in it) of every token [B, T], and which of them count."""
    case, t = st["case"], torch.arange(T, device="cuda")
    at = st["start"].long()[:, None] + t
    if st["table"] is None:
        first, row = torch.arange(case["B"], device="cuda")[:, None].expand_as(at), at
    else:
        first, row = st["table"].long().gather(1, at // BLOCK), at % BLOCK
    here = torch.ones_like(at, dtype=torch.bool) if st["count"] is None else t < st["count"][:, None]
    return first, row, here


def _plain_append(st):
    T = st["case"]["T"]
    first, row, here = _rows(st, T)
    heads = torch.arange(st["case"]["Hkv"], device="cuda")
    out = []
    for x, c, p in ((st["K"], *st["cache"][:2]), (st["V"], *st["cache"][2:])):
        codes, params = _quantise(x.transpose(1, 2))  # [B, T, Hkv, .]
        at = (first[:, :, None], heads, row[:, :, None])
        c[at] = torch.where(here[:, :, None, None], codes, c[at])
        p[at] = torch.where(here[:, :, None, None, None], params, p[at])
        back = torch.where(here[:, :, None, None], _values(c[at], p[at]), 0)
        out.append(back.transpose(1, 2).contiguous())
    return {"K": out[0], "V": out[1]}


def _plain_decode(st):
    case, S, q = st["case"], st["S"], st["q"].float()
    B, Hq, Hkv, d, L = (case[k] for k in ("B", "Hq", "Hkv", "d", "L"))
    R, nb = S.shape[1:]
    lens = torch.full((B,), L, device="cuda") if st["lens"] is None else st["lens"].long()
    cur = ((lens - 1) // BLOCK).clamp(min=0)
    # the kept blocks: the largest scores of the history, those of equal scores by index
    score = torch.where(torch.arange(nb, device="cuda") < cur[:, None, None], S, -math.inf)
    top, idx = score.sort(dim=-1, descending=True, stable=True)
    k = min(case["topk"], nb)
    keep = top[..., :k] > -math.inf
    if case["tau"]:
        keep &= top[..., :k] - score.logsumexp(-1, keepdim=True) >= math.log(case["tau"])
    top = torch.where(keep, top[..., :k], -math.inf)
    bias = torch.where(keep, top - top.logsumexp(-1, keepdim=True), -math.inf)
    blocks = torch.cat([torch.where(keep, idx[..., :k], 0), cur[:, None, None].expand(B, R, 1)], -1)
    bias = torch.cat([bias, torch.zeros(B, R, 1, device="cuda")], -1)[..., None]  # [B, R, n, 1]
    there = blocks[..., None] * BLOCK + torch.arange(BLOCK, device="cuda") < lens[:, None, None, None]
    b = torch.arange(B, device="cuda")[:, None, None]
    head = (torch.arange(R, device="cuda") * Hkv // R)[None, :, None]

    def take(codes, params):
        if st["table"] is not None:
            page = st["table"].long()[b, blocks]
            return _values(codes[page, head], params[page, head])
        codes, params = (t.view(B, Hkv, nb, BLOCK, *t.shape[3:]) for t in (codes, params))
        return _values(codes[b, head, blocks], params[b, head, blocks])

    n = blocks.shape[-1] * BLOCK
    z = q.view(B, R, -1, d) @ take(*st["cache"][:2]).view(B, R, n, d).transpose(-1, -2) / math.sqrt(d)
    z = z + torch.where(there, bias, -math.inf).view(B, R, 1, n)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (z - m).exp()
    l = p.sum(-1, keepdim=True)
    o = p @ take(*st["cache"][2:]).view(B, R, n, d) / torch.where(l > 0, l, 1)
    lse = torch.where(l > 0, m + l.log(), -math.inf)
    return {"O": o.view(B, Hq, d).to(st["q"].dtype), "LSE": lse.view(B, Hq)}


# ----------------------------------------------------------------------- the framework's calls


def _own_rope(st):
    gb, case = _binding(), st["case"]
    Hq, Hkv = case["Hq"], case["Hkv"]
    q, k, v = st["qkv"].split((Hq, Hkv, Hkv), dim=2)
    how = dict(wq=st["wq"], wk=st["wk"], eps=EPS, axes=st["axes"], interleaved=case["interleaved"])
    Q, K, V = gb.qkv_rope(q, k, v, st["cos"], st["sin"], st["pos"], **how)
    out = {"Q": Q, "K": K, "V": V}
    if case["backward"]:
        grads = st["dqkv"].split((Hq, Hkv, Hkv), dim=2)
        dwq, dwk = gb.qkv_rope_backward(q, k, st["cos"], st["sin"], st["pos"], st["dQ"], st["dK"], st["dV"],
                                        grads=grads, **how)[3:]
        out["dqkv"] = st["dqkv"]
        if dwq is not None:
            out.update(dwq=dwq, dwk=dwk)
    return out


def _own_append(st):
    gb = _binding()
    where = dict(block_table=st["table"], count=st["count"])
    gb.kv4_append(st["K"], st["V"], st["cache"], st["start"], **where)
    K, V = gb.kv4_read(st["cache"], st["start"], st["case"]["T"], dtype=torch.float32, **where)
    return {"K": K, "V": V}


def _own_decode(st):
    case = st["case"]
    O, LSE = _binding().kv4_decode(st["q"], st["cache"], st["S"], case["L"], topk=case["topk"], tau=case["tau"] or None,
                                   block_table=st["table"], seq_lens=st["lens"], group_shared=case["shared"])
    return {"O": O, "LSE": LSE}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "decode": _own_decode}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode}[op](state)


# ----------------------------------------------------------------------- work


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        tokens, row = case["B"] * case["N"], case["d"] * size
        heads, turned = case["Hq"] + 2 * case["Hkv"], case["Hq"] + case["Hkv"]
        tables = min(case["max_pos"], tokens) * case["rot"] * 4 + tokens * case["axes"] * 4
        n = 2 * heads * row * tokens + tables
        if case["backward"]:  # dQ, dK, dV read and the gradients written (the projection is read once for both)
            n += 2 * heads * row * tokens
        return {"bytes": n, "flops": tokens * turned * case["d"] * (24 if case["backward"] else 8)}
    row4 = case["d"] // 2 + case["d"] // 8
    if case["op"] == "append":  # keys and values in, 4-bit rows out; these in again and their values out
        rows = 2 * case["B"] * case["T"] * case["Hkv"] * (0.5 if case["ragged"] else 1)
        return {"bytes": rows * (case["d"] * size + 2 * row4 + 4 * case["d"]), "flops": rows * case["d"] * 6}
    B, Hq, Hkv, L = (case[k] for k in ("B", "Hq", "Hkv", "L"))
    nb, sel = -(-L // BLOCK), Hkv if case["shared"] else Hq
    k = min(case["topk"], nb - 1)
    G = sel // Hkv
    blocks = (nb - 1) * (1 - (1 - k / max(1, nb - 1)) ** G) + 1  # different blocks that a key/value head's rows keep
    full = 0.5 + 0.5 / B if case["varlen"] else 1.0  # lengths are even over the range, and one is the longest
    n = B * Hkv * min(blocks * BLOCK, L) * 2 * row4 * full + B * sel * nb * 4 * full + B * Hq * (2 * case["d"] * size + 4)
    return {"bytes": n, "flops": 4 * B * Hq * min((k + 1) * BLOCK, L) * case["d"] * full}


# ----------------------------------------------------------------------- in 64 bits


def _exact_rope(st):
    """The definition with complex numbers, and its gradients by differentiation."""
    case = st["case"]
    Hq, Hkv, half = case["Hq"], case["Hkv"], case["rot"] // 2
    qkv = st["qkv"].double().requires_grad_(case["backward"])
    ws = [None if w is None else w.double().requires_grad_(case["backward"]) for w in (st["wq"], st["wk"])]
    pos = st["pos"].long().view(case["B"], case["N"], -1)
    turn = torch.stack([torch.complex(st["cos"][:, i].double(), st["sin"][:, i].double())[pos[..., a]]
                        for i, a in enumerate(st["axes"])], -1)[:, None]  # [B, 1, N, half]

    def head_major(x, w):
        x = x.permute(0, 2, 1, 3)
        if w is not None:
            x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
        pairs = x[..., :2 * half].reshape(*x.shape[:-1], *((half, 2) if case["interleaved"] else (2, half)))
        if not case["interleaved"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.reshape(*x.shape[:-1], 2 * half), x[..., 2 * half:]], -1)

    Q, K = head_major(qkv[:, :, :Hq], ws[0]), head_major(qkv[:, :, Hq:Hq + Hkv], ws[1])
    V = qkv[:, :, Hq + Hkv:].permute(0, 2, 1, 3)
    out = {"Q": Q.detach(), "K": K.detach(), "V": V.detach()}
    if case["backward"]:
        loss = sum((a * b.double()).sum() for a, b in ((Q, st["dQ"]), (K, st["dK"]), (V, st["dV"])))
        grads = torch.autograd.grad(loss, [qkv] + [w for w in ws if w is not None])
        out["dqkv"] = grads[0]
        if ws[0] is not None:
            out["dwq"], out["dwk"] = grads[1:]
    return out


def _exact_append(st):
    case = st["case"]
    B, T, Hkv, d = (case[k] for k in ("B", "T", "Hkv", "d"))
    out = {}
    for name in ("K", "V"):
        x = st[name].double()
        back = torch.empty_like(x)
        for c in range(0, d, 32):
            g = x[..., c:c + 32]
            m = g.min(-1, keepdim=True).values.float().half().double()
            s = ((g.max(-1, keepdim=True).values - m) / 15).float().half().double()
            n = torch.where(s > 0, torch.round((g - m) / s).clamp(0, 15), 0)
            back[..., c:c + 32] = m + s * torch.nan_to_num(n)
        if st["count"] is not None:
            for b in range(B):
                back[b, :, int(st["count"][b]):] = 0
        out[name] = back
    return out


def _exact_decode(st):
    case = st["case"]
    B, Hq, Hkv, d, L = (case[k] for k in ("B", "Hq", "Hkv", "d", "L"))
    R, nb = st["S"].shape[1:]
    c = torch.arange(d, device="cuda")
    bit = 16 * (c % 32 // 4 * (d // 32) + c // 32) + 4 * (c % 4)
    O = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
    LSE = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = L if st["lens"] is None else int(st["lens"][b])
        if n < 1:
            continue
        cur = (n - 1) // BLOCK
        s = st["S"][b, :, :cur].double()
        before = torch.ones(cur, cur, dtype=torch.bool, device="cuda").tril(-1)  # equal scores of a lower index
        place = ((s[:, None, :] > s[:, :, None]) | (s[:, None, :] == s[:, :, None]) & before).sum(2)
        kept = place < case["topk"]
        if case["tau"]:
            kept &= torch.softmax(s, 1) >= case["tau"]
        for h in range(R):
            at = kept[h].nonzero().view(-1)
            gate = torch.log_softmax(s[h, at], 0) if len(at) else s[h, at]
            at = torch.cat([at, torch.tensor([cur], device="cuda")])
            bias = torch.cat([gate, torch.zeros(1, dtype=torch.float64, device="cuda")]).repeat_interleave(BLOCK)
            token = (at[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).view(-1)
            kv = h * Hkv // R
            rows = []
            for codes, params in (st["cache"][:2], st["cache"][2:]):
                if st["table"] is None:
                    x, p = codes[b, kv, token], params[b, kv, token]
                else:
                    page = st["table"][b].long()[at]
                    x, p = codes[page, kv].flatten(0, 1), params[page, kv].flatten(0, 1)
                value = (x[:, bit // 8] >> (bit % 8)).long() & 15
                p = p.double()[:, c // 32]
                rows.append(p[..., 1] + p[..., 0] * value)
            G = Hq // R
            z = st["q"][b, h * G:(h + 1) * G].double() @ rows[0].T / math.sqrt(d) + bias
            z = z[:, token < n]
            LSE[b, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
            O[b, h * G:(h + 1) * G] = torch.softmax(z, 1) @ rows[1][token < n]
    return {"O": O, "LSE": LSE}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode}[case["op"]](st)
