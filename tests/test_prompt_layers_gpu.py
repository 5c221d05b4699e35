"""The operators of a step of many tokens run together: a small BitNet stack over a batch of prompts, then over single
tokens, then handed to the persistent decode step. Every stage is compared with the oracle's on the device's inputs of
that stage: all of them exactly, but for the attention, which has a bound."""
import numpy as np
import pytest

import oracle
from oracle import decode, prompt
from packed_ternary_weight_b200 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D, F, H, KVH, HD, LAYERS, VOCAB = 256, 512, 4, 2, 128, 2, 300


@pytest.fixture(scope="module")
def tern():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from packed_ternary_weight_b200 import tern as t
    t.device_error()
    return t


class Stack:
    """The stack on the device: packed weights, gains, one cache per layer, an 8-bit token head."""

    def __init__(self, tern, seqs, max_len, page):
        self.t, self.page = tern, page
        m = self.m = synth.decode_model(D=D, F=F, H=H, KVH=KVH, n_layers=LAYERS, pos=0, max_pos=max_len, seed=31)
        self.lin = [[(tern.desc_of(lay), torch.from_numpy(tern.pack_layer(lay)[1]).cuda()) for lay in lw] for lw in m.layers]
        self.gains = [[torch.from_numpy(np.asarray(g, np.float32)).cuda() for g in gs] for gs in m.gains]
        self.rope = torch.from_numpy(tern.decode_rope_table(max_len)).cuda()
        pages = seqs * -(-max_len // page)
        n = tern.KV4Cache.size(KVH, HD, page, pages)
        self.pages = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(LAYERS)]
        self.cache = [tern.KV4Cache(p, KVH, HD, page) for p in self.pages]
        self.table = torch.from_numpy(np.random.default_rng(1).permutation(pages).astype(np.int32).reshape(seqs, -1)).cuda()
        g = torch.Generator().manual_seed(9)
        w = (torch.randn((VOCAB, D), generator=g) * 0.05).bfloat16().cuda()
        self.head, self.head_scale = torch.empty((VOCAB, D), dtype=torch.int8, device="cuda"), torch.empty(VOCAB, device="cuda")
        tern.quantize_act(w, self.head, self.head_scale)
        self.final = torch.ones(D, device="cuda")
        self.ws = torch.zeros(max(tern.workspace_size(d, 256) for lw in self.lin for d, _ in lw), dtype=torch.uint8, device="cuda")
        self.aws = torch.zeros(max(1, self.cache[0].attention_workspace_size(seqs, max_len, max_len, H)), dtype=torch.uint8, device="cuda")

    def linear(self, layer, i, xq, xs):
        d, w = self.lin[layer][i]
        y = torch.empty((xq.shape[0], d.n), device="cuda")
        self.t.gemm_batched(d, w, xq.shape[0], self.t.ACT_INT8, xq, xs, self.t.OUT_F32, y, self.ws)
        return y

    def norm(self, mode, x, r, gain):
        xq, xs = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(x.shape[0], device="cuda")
        s = torch.empty_like(r) if mode == self.t.NORM_ADD else None
        self.t.norm_quantize(mode, x, r, gain, 1e-5, s, xq, xs)
        return s, xq, xs

    def step(self, h, start, length):
        """One pass of the new tokens h [tokens][D]; returns the logits and what every stage gave."""
        n = h.shape[0]
        got = self.enqueue(h, self.t.KV4Batch(start, length, self.table, n, n, int(length.max())))
        torch.cuda.synchronize()
        assert self.t.device_error() == self.t.OK
        return got

    def enqueue(self, h, batch):
        t, n = self.t, h.shape[0]
        rec, down = [], None
        for li in range(LAYERS):
            r = {"h_in": h}
            if down is None:
                _, xq, xs = self.norm(t.NORM_PLAIN, h, None, self.gains[li][0])
            else:
                h, xq, xs = self.norm(t.NORM_ADD, down, h, self.gains[li][0])
            r.update(h=h, x1=(xq, xs))
            q, k, v = (self.linear(li, i, xq, xs) for i in range(3))
            qo, attn = (torch.empty((n, H * HD), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.cache[li].append(batch, q, k, v, self.rope, qo)
            self.cache[li].attention(batch, qo, HD ** -0.5, attn, self.aws)
            r.update(q=q, k=k, v=v, qo=qo, attn=attn)
            _, xq, xs = self.norm(t.NORM_PLAIN, attn, None, self.gains[li][1])
            r.update(x2=(xq, xs))
            o = self.linear(li, 3, xq, xs)
            h, xq, xs = self.norm(t.NORM_ADD, o, h, self.gains[li][2])
            r.update(o=o, h2=h, x3=(xq, xs))
            gate, up = self.linear(li, 4, xq, xs), self.linear(li, 5, xq, xs)
            _, xq, xs = self.norm(t.NORM_RELU2, gate, up, self.gains[li][3])
            r.update(gate=gate, up=up, x4=(xq, xs))
            down = self.linear(li, 6, xq, xs)
            r.update(down=down)
            rec.append(r)
        h, xq, xs = self.norm(t.NORM_ADD, down, h, self.final)
        logits = torch.empty((n, VOCAB), device="cuda")
        t.gemm_i8(xq, xs, self.head, self.head_scale, logits)
        return logits, (h, xq, xs), rec


def host(t):
    return t.float().cpu().numpy()


def same(got, want):
    assert np.array_equal(host(got[0]).astype(np.int8), want[1]) and np.array_equal(host(got[1]), want[2])


def check_stages(st, rec, last, logits, start, length):
    pos = np.concatenate([np.arange(length[s] - (start[s + 1] - start[s]), length[s]) for s in range(len(length))])
    seq = np.concatenate([np.full(start[s + 1] - start[s], s) for s in range(len(length))])
    cs = [decode.rope_cos_sin(int(p)) for p in pos]
    cos, sin = np.stack([c for c, _ in cs]), np.stack([s for _, s in cs])
    table = st.table.cpu().numpy()
    n = len(pos)

    def lin(li, i, x):
        lay = st.m.layers[li][i]
        return oracle.gemv_bitnet_int8(lay.trits, host(x[0]).astype(np.int8), host(x[1]), lay.tensor_scale)

    for li, r in enumerate(rec):
        g = [host(x) for x in st.gains[li]]
        if li == 0:
            same(r["x1"], prompt.norm_quantize("plain", host(r["h_in"]), None, g[0], 1e-5))
        else:
            want = prompt.norm_quantize("add", host(rec[li - 1]["down"]), host(r["h_in"]), g[0], 1e-5)
            assert np.array_equal(host(r["h"]), want[0])
            same(r["x1"], want)
        for i, name in enumerate("qkv"):
            assert np.array_equal(host(r[name]), lin(li, i, r["x1"])), (li, name)
        qr = prompt.rotate(host(r["q"]).reshape(n, H, HD), cos, sin)
        assert np.array_equal(host(r["qo"]).reshape(n, H, HD), prompt.bf16_value(qr))
        oc = prompt.Cache(st.pages[li].cpu().numpy(), KVH, HD, st.page)
        kr = prompt.rotate(host(r["k"]).reshape(n, KVH, HD), cos, sin)
        vr = host(r["v"]).reshape(n, KVH, HD)
        for t in range(n):
            for w, x in ((0, kr[t]), (1, vr[t])):
                c, s, m = prompt.quantize4(x)
                for h in range(KVH):
                    c1, s1, m1 = oc.get(int(table[seq[t], pos[t] // st.page]), int(pos[t]) % st.page, h, w)
                    assert np.array_equal(c1, c[h]) and s1 == s[h] and m1 == m[h]
        ref, tol = prompt.attention(oc, table, start, length, H, HD ** -0.5, host(r["qo"]).reshape(n, H, HD))
        assert (np.abs(host(r["attn"]).reshape(n, H, HD) - ref) <= tol).all()
        same(r["x2"], prompt.norm_quantize("plain", host(r["attn"]), None, g[1], 1e-5))
        assert np.array_equal(host(r["o"]), lin(li, 3, r["x2"]))
        want = prompt.norm_quantize("add", host(r["o"]), host(r["h"]), g[2], 1e-5)
        assert np.array_equal(host(r["h2"]), want[0])
        same(r["x3"], want)
        assert np.array_equal(host(r["gate"]), lin(li, 4, r["x3"])) and np.array_equal(host(r["up"]), lin(li, 5, r["x3"]))
        same(r["x4"], prompt.norm_quantize("relu2", host(r["gate"]), host(r["up"]), g[3], 1e-5))
        assert np.array_equal(host(r["down"]), lin(li, 6, r["x4"]))
    h, xq, xs = last
    want = prompt.norm_quantize("add", host(rec[-1]["down"]), host(rec[-1]["h2"]), host(st.final), 1e-5)
    assert np.array_equal(host(h), want[0])
    same((xq, xs), want)
    assert np.array_equal(host(logits), prompt.gemm_i8(want[1], want[2], host(st.head).astype(np.int8), host(st.head_scale)))


def dev32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def test_prompts_then_single_tokens(tern):
    st = Stack(tern, 3, 96, 16)
    g = torch.Generator().manual_seed(2)
    start, length = [0, 40, 41, 76], [40, 1, 35]
    h = torch.randn((76, D), generator=g).cuda()
    logits, last, rec = st.step(h, dev32(start), dev32(length))
    check_stages(st, rec, last, logits, start, length)
    for _ in range(2):
        length = [n + 1 for n in length]
        h = torch.randn((3, D), generator=g).cuda()
        logits, last, rec = st.step(h, dev32([0, 1, 2, 3]), dev32(length))
        check_stages(st, rec, last, logits, [0, 1, 2, 3], length)
    # a chunk of one sequence beside one token of another; the third has none
    length = [length[0] + 20, length[1], length[2] + 1]
    h = torch.randn((21, D), generator=g).cuda()
    logits, last, rec = st.step(h, dev32([0, 20, 20, 21]), dev32(length))
    check_stages(st, rec, last, logits, [0, 20, 20, 21], length)


def test_captured_token_steps(tern):
    st = Stack(tern, 2, 64, 16)
    g = torch.Generator().manual_seed(3)
    h = torch.randn((40, D), generator=g).cuda()
    st.step(h, dev32([0, 30, 40]), dev32([30, 10]))
    keep = [p.clone() for p in st.pages]
    start, length = dev32([0, 1, 2]), dev32([31, 11])
    h = torch.randn((2, D), generator=g).cuda()
    want = st.step(h, start, length)[0]
    for p, k in zip(st.pages, keep):
        p.copy_(k)
    batch = tern.KV4Batch(start, length, st.table, 2, 1, 64)   # bounds that later lengths stay within
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = st.enqueue(h, batch)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert tern.device_error() == tern.OK


def test_prompt_handed_to_the_decode_step(tern):
    # a prompt through the operators; its cache read back into the decode step's bf16 layout, which then takes a token
    n, max_pos = 37, 40
    st = Stack(tern, 1, max_pos, 16)
    h = torch.randn((n, D), generator=torch.Generator().manual_seed(4)).cuda()
    st.step(h, dev32([0, n]), dev32([n]))
    kc = torch.zeros((LAYERS, KVH, max_pos, HD), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    batch = tern.KV4Batch(dev32([0, n]), dev32([n]), st.table, n, n, n)
    for li in range(LAYERS):
        k, v = (torch.empty((n, KVH * HD), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        st.cache[li].read(batch, k, v)
        kc[li, :, :n] = k.view(n, KVH, HD).transpose(0, 1)
        vc[li, :, :n] = v.view(n, KVH, HD).transpose(0, 1)
    gains = torch.from_numpy(np.concatenate([np.concatenate(g) for g in st.m.gains]).astype(np.float32)).cuda()
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    ref_k, ref_v = (bits(t).cpu().numpy().view(np.uint16).copy() for t in (kc, vc))
    model = tern.DecodeModel([w for lw in st.lin for _, w in lw], gains, bits(kc), bits(vc), st.rope, D, F, H, KVH, max_pos)
    ws = torch.zeros(model.workspace_size(), dtype=torch.uint8, device="cuda")
    h0 = torch.randn(D, generator=torch.Generator().manual_seed(5)).cuda()
    out, trace = torch.empty(D, device="cuda"), torch.zeros((LAYERS, 2 * H * HD + 2 * KVH * HD), device="cuda")
    model.step(n, h0, out, ws, trace=trace)
    torch.cuda.synchronize()
    assert tern.device_error() == tern.OK
    # the keys it attended to: layer 0's attention against the oracle on the values read back
    lw = [(lay.trits, lay.tensor_scale) for lay in st.m.layers[0]]
    rec = {}
    decode.decode_layer(host(h0), lw, st.m.gains[0], ref_k[0], ref_v[0], n, decode.rope_cos_sin(n), first=1, last=2, rec=rec)
    got = host(trace[0])[H * HD + 2 * KVH * HD:]
    assert np.abs(got - rec["attn"]).max() <= 1e-4 * np.abs(rec["attn"]).max()


FIRST_CALLS = """
import sys, torch
sys.path.insert(0, {root!r})
from packed_ternary_weight_b200 import tern
z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
x, w, y = z(64, 512, dt=torch.int8) + 1, z(512, 512, dt=torch.int8) + 1, z(64, 512)
sx, sw = z(64) + 1, z(512) + 1
xf, xq, xs, gain = z(64, 512) + 1, z(64, 512, dt=torch.int8), z(64), z(512) + 1
cache = tern.KV4Cache(z(8 * 2 * 16 * 72, dt=torch.uint8), 2, 64, 16)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
batch = tern.KV4Batch(i32([0, 64]), i32([64]), i32([[0, 1, 2, 3]]), 64, 64, 64)
q, k, qo, rope = z(64, 128) + 1, z(64, 128) + 1, z(64, 128, dt=torch.bfloat16), z(64, 32, 2)
rope[..., 0] = 1
out, ws = torch.empty_like(qo), z(cache.attention_workspace_size(1, 64, 64, 2), dt=torch.uint8)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    tern.gemm_i8(x, sx, w, sw, y)
    tern.norm_quantize(tern.NORM_PLAIN, xf, None, gain, 1e-5, None, xq, xs)
    cache.append(batch, q, k, k, rope, qo)
    cache.attention(batch, qo, 0.125, out, ws)
g.replay()
torch.cuda.synchronize()
assert (y == 512).all() and (xq == 127).all() and (out == 1).all() and tern.device_error() == tern.OK
"""


def test_first_calls_of_a_process_in_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
