"""Cases and plain forms of the operators around the ternary linears of a batched or prompt step.

A BitNet layer run for more than one token of one sequence is: residual add, RMSNorm and int8
quantisation of every linear's input (`norm`), rotation of q and k and the append of k and v to a paged
4-bit cache (`append`), attention over that cache (`attn`), and, behind the last layer, the token head as
an 8-bit product with a scale per token and per channel (`gemm`). The plain forms below are elementary
torch operations; with `own` the same passes go through the framework's calls.

A page of the 4-bit cache holds `page` tokens of every kv head; the block of one head is
    K codes [page][D/2] | V codes [page][D/2] | fp16 [page][4] = k scale, k min, v scale, v min
with the code of dimension d in bits 4 (d mod 2) of byte d div 2, and stands for min + scale * code.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
EPS = 1e-5
THETA = 500000.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the input of q/k/v, one token of a decode step: latency
        dict(name="norm add, one token", op="norm", mode="add", m=1, k=2560, x="f32", r="f32"),
        # the input of down_proj for a prompt: squared ReLU of gate times up
        dict(name="norm relu2, prompt", op="norm", mode="relu2", m=2043, k=6912, x="bf16", r="bf16"),
        # the input of gate/up, a large batch of prompts: bf16 branch onto an fp32 residual stream
        dict(name="norm add, large", op="norm", mode="add", m=8192, k=4096, x="bf16", r="f32"),
        # one new token of each of 64 sequences
        dict(name="append, 64 sequences", op="append", h=20, kvh=5, d=128, page=64, seqs=64, qmax=1, kvmax=4096, ragged=True, x="f32"),
        # the prompts of five requests at once, of unequal lengths
        dict(name="append, prompts", op="append", h=32, kvh=8, d=128, page=64, seqs=5, qmax=2500, kvmax=2500, ragged=True, x="bf16"),
        # one sequence at the position that the decode step is benchmarked at
        dict(name="attn, one sequence", op="attn", h=20, kvh=5, d=128, page=64, seqs=1, qmax=1, kvmax=1024, ragged=False),
        # a serving batch of unequal lengths
        dict(name="attn, 64 sequences", op="attn", h=20, kvh=5, d=128, page=64, seqs=64, qmax=1, kvmax=8192, ragged=True),
        # one sequence with a very long history: the split along the keys
        dict(name="attn, long history", op="attn", h=32, kvh=8, d=128, page=128, seqs=1, qmax=1, kvmax=131072, ragged=False),
        # a prompt chunk behind its own earlier part, and shorter ones beside it
        dict(name="attn, prompt chunks", op="attn", h=32, kvh=8, d=128, page=64, seqs=3, qmax=2048, kvmax=8190, ragged=True),
        # the token head for one token: every weight once
        dict(name="gemm head, one token", op="gemm", m=1, n=65536, k=2560, y="f32"),
        # a projection for a serving batch
        dict(name="gemm, 61 tokens", op="gemm", m=61, n=2560, k=6912, y="bf16"),
        # a projection for a batch of prompts
        dict(name="gemm, prompts", op="gemm", m=4095, n=14336, k=4096, y="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "attn", "attn", "gemm"])
    if op == "norm":
        k = rng.choice([64 * rng.randint(4, 108), _log(rng, 100, 14336), 2560, 4096, 6912])
        m = _log(rng, 1, max(1, min(8192, (8192 * 4096) // k)))
        return dict(op=op, mode=rng.choice(["plain", "add", "relu2"]), m=m, k=k, x=rng.choice(["f32", "bf16"]),
                    r=rng.choice(["f32", "bf16"]))
    if op in ("append", "attn"):
        kvh = rng.choice([1, 2, 4, 5, 8])
        base = dict(op=op, h=kvh * rng.choice([1, 2, 3, 4] if kvh > 4 else [1, 2, 4, 5, 8]), kvh=kvh, d=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
        if op == "append":
            qmax = rng.choice([1, _log(rng, 1, 2048)])
            seqs = _log(rng, 1, max(1, min(64, 6000 // qmax)))
            return dict(base, seqs=seqs, qmax=qmax, kvmax=qmax + _log(rng, 1, 4096), x=rng.choice(["f32", "bf16"]))
        if rng.random() < 0.6:  # single tokens, or a few at a time
            qmax = rng.choice([1, 1, 1, rng.randint(2, 8)])
            kvmax = qmax + _log(rng, 1, 65536)
            seqs = _log(rng, 1, max(1, min(64, (32 * 8192) // kvmax)))
        else:  # prompts and chunks of prompts
            qmax = _log(rng, 16, 2048)
            kvmax = qmax + rng.choice([0, _log(rng, 1, 6000)])
            seqs = _log(rng, 1, max(1, min(8, (3 * 2048 * 8190) // (qmax * kvmax))))
        return dict(base, seqs=seqs, qmax=qmax, kvmax=kvmax)
    n, k = rng.choice([2560, 4096, 6912, _log(rng, 33, 14336)]), rng.choice([2560, 4096, 6912, 16 * _log(rng, 4, 432)])
    most = max(1, min(4096, (4095 * 14336 * 4096) // (n * k)))
    return dict(op=op, m=rng.choice([1, _log(rng, 1, min(64, most)), _log(rng, 1, most)]), n=n, k=k, y=rng.choice(["f32", "bf16"]))


# ----------------------------------------------------------------- inputs
def _lengths(c):
    """New tokens and cache lengths of every sequence (lengths include the new tokens), the case's own."""
    s = c["seqs"]
    if not c["ragged"]:
        return np.full(s, c["qmax"]), np.full(s, c["kvmax"])
    g = np.random.default_rng([s, c["qmax"], c["kvmax"], c["h"], c["d"]])
    old = c["kvmax"] - c["qmax"]
    q = g.integers(max(1, c["qmax"] // 4), c["qmax"] + 1, s)
    o = g.integers(old // 4, old + 1, s)
    i = int(g.integers(0, s))
    q[i], o[i] = c["qmax"], old
    return q, q + o


def _block(c):
    return c["page"] * (c["d"] + 8)


def _paged(c, g):
    """Page table, lengths and a cache filled with keys and values of unit variance."""
    q, kv = _lengths(c)
    need = -(-kv // c["page"])
    mp, total = int(need.max()), int(need.sum())
    order = torch.randperm(total, generator=g, device=DEV).int()
    table = torch.zeros((c["seqs"], mp), dtype=torch.int32, device=DEV)
    row = torch.from_numpy(np.repeat(np.arange(c["seqs"]), need)).to(DEV)
    col = torch.from_numpy(np.concatenate([np.arange(n) for n in need])).to(DEV)
    table[row, col] = order
    nb = total * c["kvh"]
    half, p = c["page"] * c["d"], c["page"]
    pages = torch.empty((nb, _block(c)), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // half)
    for i in range(0, nb, step):
        n = min(step, nb - i)
        code = torch.randn((n, 2 * half), generator=g, device=DEV).mul_(2.9).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        pages[i:i + n, :half] = code[:, ::2] | (code[:, 1::2] << 4)
        sc = torch.rand((n, p, 2), generator=g, device=DEV) * 0.2 + 0.25
        mn = -7.5 * sc + 0.3 * torch.randn((n, p, 2), generator=g, device=DEV)
        pages[i:i + n, half:] = torch.stack([sc, mn], 3).half().reshape(n, p * 4).view(torch.uint8)
    start = np.concatenate([[0], np.cumsum(q)])
    return dict(pages=pages.reshape(total, c["kvh"], _block(c)), table=table, q=q, kv=kv, qmax=int(q.max()), kvmax=int(kv.max()),
                tokens=int(start[-1]), start=torch.from_numpy(start).int().to(DEV), len=torch.from_numpy(kv).int().to(DEV))


def _rope_table(n, d):
    ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * THETA ** (-2.0 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
    return torch.stack([ang.cos(), ang.sin()], 2).float().contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        s = dict(x=rnd(m, k).to(DTYPES[c["x"]]), gain=(1 + 0.1 * rnd(k)).contiguous(), eps=EPS)
        s["r"] = rnd(m, k).mul_(2).to(DTYPES[c["r"]]) if c["mode"] != "plain" else None
        s["sum"] = torch.empty((m, k), dtype=DTYPES[c["r"]], device=DEV) if c["mode"] == "add" else None
        s["xq"] = torch.empty((m, k), dtype=torch.int8, device=DEV)
        s["xscale"] = torch.empty(m, dtype=torch.float32, device=DEV)
    elif c["op"] == "append":
        s = _paged(c, g)
        t, d = s["tokens"], c["d"]
        dt = DTYPES[c["x"]]
        s["xq"], s["xk"], s["xv"] = rnd(t, c["h"] * d).to(dt), rnd(t, c["kvh"] * d).mul_(2).to(dt), rnd(t, c["kvh"] * d).to(dt)
        s["rope"] = _rope_table(c["kvmax"], d)
        s["q_out"] = torch.empty((t, c["h"] * d), dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty((t, c["kvh"] * d), dtype=dt, device=DEV)
        s["v_out"] = torch.empty((t, c["kvh"] * d), dtype=dt, device=DEV)
    elif c["op"] == "attn":
        s = _paged(c, g)
        s["xq"] = rnd(s["tokens"], c["h"] * c["d"]).bfloat16()
        s["out"] = torch.empty_like(s["xq"])
        s["scale"] = 1.0 / math.sqrt(c["d"])
        s["ws"] = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    else:
        m, n, k = c["m"], c["n"], c["k"]
        code = lambda r: rnd(r, k).mul_(32).round_().clamp_(-127, 127).to(torch.int8)  # noqa: E731
        s = dict(x=code(m), w=code(n))
        s["sx"] = (torch.rand(m, generator=g, device=DEV) + 0.5) * 0.03
        s["sw"] = (torch.rand(n, generator=g, device=DEV) + 0.5) * 6e-4
        s["y"] = torch.empty((m, n), dtype=DTYPES[c["y"]], device=DEV)
    s["case"] = c
    return s


# ------------------------------------------------------------ plain forms
def _plain_norm(s):
    c = s["case"]
    v, out = s["x"].float(), []
    if c["mode"] == "add":
        out = [(v + s["r"].float()).to(s["r"].dtype)]
        v = out[0].float()
    elif c["mode"] == "relu2":
        v = v.clamp_min(0)
        v = v * v * s["r"].float()
    r = (1.0 / (v.double().square().mean(1, keepdim=True) + s["eps"]).sqrt()).float()
    y = v * r * s["gain"]
    a = y.abs().amax(1, keepdim=True)
    top = torch.full_like(a, 127.0)  # divisions are tensor by tensor: one by a number is a product with its reciprocal
    q = torch.where(a > 0, (y * (top / a)).round().clamp(-127, 127), torch.zeros_like(y))
    return out + [q.to(torch.int8), (a / top)[:, 0]]


def _token_places(s):
    """Sequence, position, page and slot of every new token."""
    c = s["case"]
    t = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(s["start"][1:].contiguous(), t.int(), right=True)
    pos = s["len"][seq] - s["start"][seq + 1] + t
    return seq, pos, s["table"][seq, pos // c["page"]].long(), pos % c["page"]


def _rotate(x, cs):
    h = x.shape[2] // 2
    a, b, co, si = x[..., :h], x[..., h:], cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat([a * co - b * si, b * co + a * si], 2)


def _codes(x):
    """4-bit codes of the last axis and their fp16 scale and minimum."""
    lo, hi = x.amin(2, keepdim=True), x.amax(2, keepdim=True)
    sc, mn = ((hi - lo) / torch.full_like(lo, 15.0)).half(), lo.half()
    inv = torch.where(sc > 0, 1.0 / sc.float(), torch.zeros_like(lo))
    return ((x - mn.float()) * inv).round().clamp(0, 15).to(torch.uint8), sc, mn


def _plain_append(s):
    c = s["case"]
    t, d, p = s["tokens"], c["d"], c["page"]
    _, pos, page, slot = _token_places(s)
    cs = s["rope"][pos]
    q = _rotate(s["xq"].float().view(t, c["h"], d), cs).bfloat16().view(t, -1)
    ck, sk, mk = _codes(_rotate(s["xk"].float().view(t, c["kvh"], d), cs))
    cv, sv, mv = _codes(s["xv"].float().view(t, c["kvh"], d))
    half = p * d // 2
    k_b = s["pages"][:, :, :half].view(-1, c["kvh"], p, d // 2)
    v_b = s["pages"][:, :, half:2 * half].view(-1, c["kvh"], p, d // 2)
    par = s["pages"][:, :, 2 * half:].view(-1, c["kvh"], p, 8)
    k_b[page, :, slot] = ck[..., ::2] | (ck[..., 1::2] << 4)
    v_b[page, :, slot] = cv[..., ::2] | (cv[..., 1::2] << 4)
    par[page, :, slot] = torch.cat([sk, mk, sv, mv], 2).view(torch.uint8)

    def read(b, o):
        code = b[page, :, slot]
        code = torch.stack([code & 15, code >> 4], 3).view(t, c["kvh"], d).float()
        f = par[page, :, slot].view(torch.float16)[..., o:o + 2].float()
        return (f[..., 1:] + f[..., :1] * code).view(t, -1).to(s["k_out"].dtype)

    return [q, read(k_b, 0), read(v_b, 2)]


def _plain_attn(s):
    c = s["case"]
    S, t, d, p, kvh = c["seqs"], s["tokens"], c["d"], c["page"], c["kvh"]
    g, half = c["h"] // kvh, p * d // 2
    b = s["pages"][s["table"].long()]  # [S][pages][kvh][block]: padded table entries name page 0 and are masked
    kv = b.shape[1] * p
    par = b[..., 2 * half:].reshape(S, -1, kvh, p, 8).view(torch.float16).float()

    def values(lo, o):
        code = b[..., lo:lo + half].reshape(S, -1, kvh, p, d // 2)
        code = torch.stack([code & 15, code >> 4], 5).view(S, -1, kvh, p, d).float()
        return (par[..., o + 1:o + 2] + par[..., o:o + 1] * code).transpose(1, 2).reshape(S, kvh, kv, d)

    seq, pos, _, _ = _token_places(s)
    row = torch.arange(t, device=DEV) - s["start"][seq]
    q = torch.zeros((S, s["qmax"], kvh, g, d), device=DEV)
    q[seq, row] = s["xq"].float().view(t, kvh, g, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(S, kvh, g * s["qmax"], d)
    limit = torch.zeros((S, s["qmax"]), dtype=torch.long, device=DEV)
    limit[seq, row] = pos
    sc = (q @ values(0, 0).transpose(2, 3)).mul_(s["scale"]).view(S, kvh, g, s["qmax"], kv)
    sc.masked_fill_(torch.arange(kv, device=DEV) > limit[:, None, None, :, None], -math.inf)
    sc = (sc - sc.amax(4, keepdim=True)).exp_()
    l = sc.sum(4, keepdim=True)
    o = (sc.view(S, kvh, -1, kv) @ values(half, 2)).view(S, kvh, g, s["qmax"], d) / l
    return [o.permute(0, 3, 1, 2, 4)[seq, row].reshape(t, -1).bfloat16()]


def _plain_gemm(s):
    y = s["x"].float() @ s["w"].float().t()
    return [(y * s["sw"] * s["sx"][:, None]).to(s["y"].dtype)]


# ------------------------------------------------------- the framework's
def _own(s):
    from packed_ternary_weight_b200 import tern
    c = s["case"]
    if c["op"] == "norm":
        mode = {"plain": tern.NORM_PLAIN, "add": tern.NORM_ADD, "relu2": tern.NORM_RELU2}[c["mode"]]
        tern.norm_quantize(mode, s["x"], s["r"], s["gain"], s["eps"], s["sum"], s["xq"], s["xscale"])
        return ([s["sum"]] if c["mode"] == "add" else []) + [s["xq"], s["xscale"]]
    if c["op"] == "gemm":
        tern.gemm_i8(s["x"], s["sx"], s["w"], s["sw"], s["y"])
        return [s["y"]]
    cache = tern.KV4Cache(s["pages"], c["kvh"], c["d"], c["page"])
    batch = tern.KV4Batch(s["start"], s["len"], s["table"], s["tokens"], s["qmax"], s["kvmax"])
    if c["op"] == "append":
        cache.append(batch, s["xq"], s["xk"], s["xv"], s["rope"], s["q_out"])
        cache.read(batch, s["k_out"], s["v_out"])
        return [s["q_out"], s["k_out"], s["v_out"]]
    cache.attention(batch, s["xq"], s["scale"], s["out"], s["ws"])
    return [s["out"]]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attn, "gemm": _plain_gemm}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"] == "norm":
        e = c["m"] * c["k"]
        b = e * (size[c["x"]] + 1) + 4 * c["k"] + 4 * c["m"]
        b += 0 if c["mode"] == "plain" else e * size[c["r"]] * (2 if c["mode"] == "add" else 1)
        return {"bytes": b, "flops": 8 * e}
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * size[c["y"]], "flops": 2 * m * n * k}
    q, kv = _lengths(c)
    d, t, tok = c["d"], int(q.sum()), c["kvh"] * (c["d"] + 8)
    if c["op"] == "append":  # q, k, v and the rotation read; q, the cache and the values read back written; the cache read
        x = size[c["x"]]
        b = t * (c["h"] * d * (x + 2) + 2 * c["kvh"] * d * 2 * x + 2 * tok + 4 * d)
        return {"bytes": b, "flops": t * (c["h"] + 2 * c["kvh"]) * d * 8}
    pairs = float((q * (kv - (q - 1) / 2)).sum())
    return {"bytes": int(kv.sum()) * tok + 4 * t * c["h"] * d, "flops": 4 * pairs * c["h"] * d}


# ------------------------------------------------------------------ exact
def _exact_norm(s):
    """The definition with its stated roundings to 32 bits, each taken from a value in 64 bits."""
    c = s["case"]
    r32 = lambda v: v.float().double()  # noqa: E731
    x, g = s["x"].double(), s["gain"].double()
    res = [] if c["mode"] != "add" else [None]
    if c["mode"] == "add":
        x = x + s["r"].double()
        res = [x]
        x = r32(x).to(s["r"].dtype).double()
    elif c["mode"] == "relu2":
        x = torch.relu(x)
        x = r32(r32(x * x) * s["r"].double())
    inv = r32(torch.rsqrt((x * x).sum(1) / c["k"] + s["eps"]))
    y = r32(r32(x * inv[:, None]) * g[None])
    a = y.abs().max(1).values
    up = torch.where(a > 0, r32(127.0 / a), torch.zeros_like(a))
    q = torch.round(r32(y * up[:, None])).clamp(-127, 127)
    return res + [q.to(torch.int8), a / 127.0]


def _exact_places(s, i):
    c = s["case"]
    q, kv = int(s["q"][i]), int(s["kv"][i])
    pos = np.arange(kv - q, kv)
    return q, kv, pos


def _exact_append(s):
    c = s["case"]
    d, qs, ks, vs = c["d"], [], [], []
    r32 = lambda v: v.float().double()  # noqa: E731
    at = 0
    for i in range(c["seqs"]):
        n, _, pos = _exact_places(s, i)
        ang = torch.from_numpy(pos).to(DEV).double()[:, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64, device=DEV), -torch.arange(0, d, 2, device=DEV).double() / d)[None]
        co, si = r32(ang.cos())[:, None], r32(ang.sin())[:, None]

        def turn(x, heads):
            x = x[at:at + n].double().reshape(n, heads, d)
            a, b = x.split(d // 2, 2)
            return torch.cat((r32(a * co) - r32(b * si), r32(b * co) + r32(a * si)), 2)

        def four(x):
            mx, mn = x.max(2).values, x.min(2).values
            scale, low = (r32(r32(mx - mn) / 15)).half().double(), mn.half().double()
            up = torch.where(scale > 0, r32(1 / scale), torch.zeros_like(scale))
            code = torch.round(r32(r32(x - low[..., None]) * up[..., None])).clamp(0, 15)
            return (low[..., None] + scale[..., None] * code).reshape(n, -1)

        qs.append(turn(s["xq"], c["h"]).reshape(n, -1))
        ks.append(four(r32(turn(s["xk"], c["kvh"]))))
        vs.append(four(s["xv"][at:at + n].double().reshape(n, c["kvh"], d)))
        at += n
    return [torch.cat(qs), torch.cat(ks), torch.cat(vs)]


def _exact_attn(s):
    c = s["case"]
    if 4 * c["seqs"] * c["qmax"] * c["kvmax"] * c["h"] * c["d"] > 2e13:
        return None
    d, p, g = c["d"], c["page"], c["h"] // c["kvh"]
    outs, at = [], 0
    for i in range(c["seqs"]):
        n, kv, pos = _exact_places(s, i)
        b = s["pages"][s["table"][i, :-(-kv // p)].long()]
        q = s["xq"][at:at + n].double().reshape(n, c["kvh"], g, d)
        at += n
        out = torch.empty((n, c["kvh"], g, d), dtype=torch.float64, device=DEV)
        for j in range(c["kvh"]):
            byte = b[:, j, :p * d].reshape(-1, 2, p, d // 2)
            par = b[:, j, p * d:].contiguous().view(torch.float16).reshape(-1, p, 2, 2).double()
            val = torch.empty((byte.shape[0], 2, p, d), dtype=torch.float64, device=DEV)
            val[..., 0::2], val[..., 1::2] = (byte % 16).double(), (byte // 16).double()
            val = par[..., 1].transpose(1, 2)[..., None] + par[..., 0].transpose(1, 2)[..., None] * val
            k, v = val[:, 0].reshape(-1, d)[:kv], val[:, 1].reshape(-1, d)[:kv]
            for e in range(0, n, 256):
                f = min(n, e + 256)
                sc = torch.einsum("ngd,kd->ngk", q[e:f, j], k) / math.sqrt(d)
                late = torch.arange(kv, device=DEV)[None] > torch.from_numpy(pos[e:f]).to(DEV)[:, None]
                sc = torch.where(late[:, None], torch.full_like(sc, -math.inf), sc)
                out[e:f, j] = torch.einsum("ngk,kd->ngd", torch.softmax(sc, 2), v)
        outs.append(out.reshape(n, -1))
    return [torch.cat(outs)]


def _exact_gemm(s):
    c = s["case"]
    if 2 * c["m"] * c["n"] * c["k"] > 2e13:
        return None
    acc = torch.einsum("mk,nk->mn", s["x"].double(), s["w"].double())
    return [acc * (s["sw"].double()[None] * s["sx"].double()[:, None])]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attn": _exact_attn, "gemm": _exact_gemm}[case["op"]](s)
