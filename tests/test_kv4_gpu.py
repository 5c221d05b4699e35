"""The paged 4-bit cache (append, read, attention) against the oracle. Append and read are exact; attention is held to
the bound that oracle.prompt.attention derives for every output."""
import numpy as np
import pytest

from oracle import decode, prompt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tern():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from packed_ternary_weight_b200 import tern as t
    t.device_error()
    return t


def util():
    from tests import prompt_util
    return prompt_util


def rope_rows(pos, d):
    cs = [decode.rope_cos_sin(p, d) for p in pos]
    return np.stack([c for c, _ in cs]), np.stack([s for _, s in cs])


# ------------------------------------------------------- append and read
def run_append(tern, b, heads, dt=torch.float32, max_pos=None, seed=0, ld_pad=0, with_q=True):
    """Appends random tokens; returns the device results and the oracle's."""
    u = util()
    g = np.random.default_rng(seed + 50)
    n, d, kvh = b.rows, b.d, b.kvh

    def buf(h):
        a = torch.from_numpy(g.standard_normal((n, h * d + ld_pad)).astype(np.float32) * 1.5).cuda().to(dt)
        return a[:, :h * d], a[:, :h * d].float().cpu().numpy().reshape(n, h, d)

    q, hq = buf(heads) if with_q else (None, None)
    k, hk = buf(kvh)
    v, hv = buf(kvh)
    top = int(b.len.max()) if max_pos is None else max_pos
    rope = torch.from_numpy(tern.decode_rope_table(max(1, top), d)).cuda()
    cache, batch = b.device()
    qo = torch.full((n, heads * d), 9.0, dtype=torch.bfloat16, device="cuda") if with_q else None
    cache.append(batch, q, k, v, rope, qo)
    ko = torch.full((n, kvh * d), 9.0, device="cuda")
    vo = torch.full((n, kvh * d), 9.0, device="cuda")
    cache.read(batch, ko, vo)
    torch.cuda.synchronize()
    raw = b.raw.copy()
    oc = b.oracle_cache(raw)
    eq = np.full((n, max(heads, 1), d), 9.0, np.float32)
    ek, ev = np.full((n, kvh, d), 9.0, np.float32), np.full((n, kvh, d), 9.0, np.float32)
    for t, (s, pos) in enumerate(b.positions()):
        if pos < 0:
            eq[t], ek[t], ev[t] = 0, 0, 0
            continue
        c, sn = rope_rows([pos], d)
        if with_q:
            eq[t] = prompt.bf16_value(prompt.rotate(hq[t:t + 1], c, sn)[0])
        for w, x, e in ((0, prompt.rotate(hk[t:t + 1], c, sn)[0], ek), (1, hv[t], ev)):
            codes, sc, m = prompt.quantize4(x)
            for h in range(kvh):
                oc.put(int(b.table[s, pos // b.page]), pos % b.page, h, w, codes[h], sc[h], m[h])
                e[t, h] = (m[h].astype(np.float64) + sc[h].astype(np.float64) * codes[h]).astype(np.float32)
    return (b.pages.cpu().numpy(), None if qo is None else qo.float().cpu().numpy().reshape(n, -1, d),
            ko.cpu().numpy().reshape(n, kvh, d), vo.cpu().numpy().reshape(n, kvh, d)), (raw, eq, ek, ev)


@pytest.mark.parametrize("d,page,kvh,heads", [(128, 64, 5, 20), (128, 16, 1, 1), (64, 32, 3, 9), (64, 256, 8, 8), (128, 128, 2, 14)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_append_and_read(tern, d, page, kvh, heads, dt):
    b = util().Batch([1, 17, 0, 3, 40], [100, 17, 33, page + 2, 2 * page + 41], kvh, d, page, seed=d + page, tail=5)
    got, want = run_append(tern, b, heads, dt)
    assert np.array_equal(got[0], want[0])               # every byte of the pages, the untouched ones among them
    for a, e in zip(got[1:], want[1:]):
        assert np.array_equal(a, e)                      # the rows behind the last sequence among them
    assert tern.device_error() == tern.OK


def test_append_strided_and_keys_only(tern):
    b = util().Batch([3, 5], [20, 5], 2, 128, 16, seed=3)
    got, want = run_append(tern, b, 4, torch.bfloat16, ld_pad=16)
    assert all(np.array_equal(a, e) for a, e in zip(got, want))
    got, want = run_append(tern, b, 4, with_q=False)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[2], want[2])
    assert tern.device_error() == tern.OK


def test_append_many_sequences(tern):
    # the search for a row's sequence: hundreds of them, runs of empty ones
    new = np.array([0, 0, 1, 2, 0] * 130 + [0, 0])
    b = util().Batch(new, new + 1, 1, 64, 16, seed=4)
    got, want = run_append(tern, b, 1)
    assert all(np.array_equal(a, e) for a, e in zip(got, want))


def test_positions_before_the_start(tern):
    # a length shorter than the new tokens: the first ones are at negative positions
    b = util().Batch([4, 3], [2, 0], 2, 64, 16, seed=5)
    got, want = run_append(tern, b, 2)
    assert all(np.array_equal(a, e) for a, e in zip(got, want))
    assert tern.device_error() == tern.OK


def test_extreme_values(tern):
    u = util()
    b = u.Batch([6], [6], 1, 64, 16, seed=6)
    k = torch.randn((6, 64), device="cuda")
    k[0] = 0
    k[1] = -3.5
    k[2] = 1e-7                                           # below half a step of fp16
    k[3] *= 2e4
    k[4] = torch.where(torch.arange(64, device="cuda") % 2 == 0, 60000.0, -60000.0)
    k[5] *= 1e-6
    v = k.flip(0).contiguous()
    rope = torch.from_numpy(tern.decode_rope_table(6, 64)).cuda()
    rope[..., 0], rope[..., 1] = 1, 0
    cache, batch = b.device()
    cache.append(batch, None, k, v, rope, None)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cache.read(batch, ko, vo)
    for x, y in ((k, ko), (v, vo)):
        c, s, m = prompt.quantize4(x.cpu().numpy())
        want = (m.astype(np.float64)[:, None] + s.astype(np.float64)[:, None] * c).astype(np.float32)
        assert np.array_equal(y.cpu().numpy(), want)


def bad_descriptions(u):
    """(batch, sequences left out) for each way in which the device data can be wrong."""
    def make(**k):
        return u.Batch([2, 3, 2], [20, 30, 40], 2, 64, 16, seed=7, **k)
    b = make()
    b.table[1, 1] = 10 ** 6
    yield "page", b, None
    b = make()
    b.table[1, 1] = -1
    yield "negative page", b, None
    b = make()
    b.len[1] = 5000
    yield "length", b, 1
    b = make()
    b.len[1] = -4
    yield "negative length", b, 1


@pytest.mark.parametrize("which", range(4))
def test_bad_descriptions_are_left_out_and_reported(tern, which):
    u = util()
    name, b, out = list(bad_descriptions(u))[which]
    good = u.Batch([2, 3, 2], [20, 30, 40], 2, 64, 16, seed=7)
    good.fill_values()
    b.raw = good.raw.copy()
    cache, batch = b.device(max_len=60)
    q = torch.randn((7, 128), device="cuda").bfloat16()
    o = torch.full_like(q, 9.0)
    ws = u.workspace(cache, 2, 3, 3, 60)
    cache.attention(batch, q, 0.1, o, ws)
    assert tern.device_error() == tern.EFORMAT, name
    assert tern.device_error() == tern.OK
    gc, gb = good.device(max_len=60)
    o2 = torch.full_like(q, 9.0)
    gc.attention(gb, q, 0.1, o2, ws)
    assert torch.equal(o[:2], o2[:2]) and torch.equal(o[5:], o2[5:])     # the other sequences are whole
    if out is None:
        # without the bad page: as if its sixteen positions were not there
        ref, tol = attention_without(good, q, 0.1, 1, range(16, 30 if which < 2 else 0))
        got = o[2:5].float().cpu().numpy().reshape(3, 2, 64)
        assert (np.abs(got - ref) <= tol).all()
    else:
        assert (o[2:5] == 9).all()
    k = torch.randn((7, 128), device="cuda")
    rope = torch.from_numpy(tern.decode_rope_table(60, 64)).cuda()
    cache.append(batch, None, k, k, rope, None)
    assert tern.device_error() == tern.EFORMAT
    ko = torch.full((7, 128), 9.0, device="cuda")
    cache.read(batch, ko, None)
    assert tern.device_error() == tern.EFORMAT
    assert (ko[2:5] == (0 if out is None else 9)).all() and (ko[:2] != 9).all()


def attention_without(b, q, scale, s, gone):
    """Oracle of sequence s with the positions `gone` left out (heads == kv heads)."""
    c = b.oracle_cache()
    n, ln = int(b.new[s]), int(b.len[s])
    out = np.zeros((n, b.kvh, b.d))
    tol = np.zeros_like(out)
    qh = q.float().cpu().numpy().reshape(-1, b.kvh, b.d)
    for h in range(b.kvh):
        kc, ks, km = c.parts(b.table[s], ln, h, 0)
        vc, vs, vm = c.parts(b.table[s], ln, h, 1)
        for i in range(n):
            at = [j for j in range(ln - n + i + 1) if j not in gone]
            sc = (km[at, None] + ks[at, None] * kc[at]) @ qh[b.start[s] + i, h].astype(np.float64) * scale
            p = np.exp(sc - sc.max())
            p /= p.sum()
            v = vm[at, None] + vs[at, None] * vc[at]
            out[i, h] = p @ v
            tol[i, h] = 2.0 ** -8 * np.abs(out[i, h]) + 2.0 ** -11 * (p @ (vs[at, None] * vc[at])) * 1.01 + 1e-4
    return out, tol


@pytest.mark.parametrize("what", ["rows beyond the buffer", "too many new", "position without a rotation", "rows out of order"])
def test_bad_rows_are_reported(tern, what):
    u = util()
    b = u.Batch([2, 3], [20, 30], 2, 64, 16, seed=8)
    b.fill_values()
    max_pos, max_new = 40, None
    if what == "rows beyond the buffer":
        b.start[2] = 50
    elif what == "too many new":
        max_new = 2
    elif what == "position without a rotation":
        max_pos = 29
    else:
        b.start[:] = [2, 0, 5]
    cache, batch = b.device(max_new=max_new)
    k = torch.randn((5, 128), device="cuda")
    rope = torch.from_numpy(tern.decode_rope_table(max_pos, 64)).cuda()
    cache.append(batch, None, k, k, rope, None)
    assert tern.device_error() == tern.EFORMAT
    if what != "position without a rotation":
        q = torch.zeros((5, 128), device="cuda").bfloat16()
        cache.attention(batch, q, 0.1, q.clone(), u.workspace(cache, 2, 2, 50, 100))
        assert tern.device_error() == tern.EFORMAT


# -------------------------------------------------------------- attention
def run_attention(tern, b, heads, scale=None, seed=0, spread=1.0, max_new=None, max_len=None, ws=None, q=None):
    u = util()
    g = np.random.default_rng(seed + 70)
    scale = 1 / np.sqrt(b.d) if scale is None else scale
    if q is None:
        q = u.bf16_dev(g.standard_normal((b.rows, heads * b.d)) * spread)
    cache, batch = b.device(max_new, max_len)
    out = torch.full_like(q, 9.0)
    if ws is None:
        ws = u.workspace(cache, heads, len(b.new), max(int(b.new.max()), max_new or 0), max(int(b.len.max()), max_len or 0))
    cache.attention(batch, q, scale, out, ws)
    torch.cuda.synchronize()
    assert tern.device_error() == tern.OK
    most = (max_new or int(b.new.max())) * (heads // b.kvh)    # one sequence whose bound is a prompt's runs as one
    ref, tol = prompt.attention(b.oracle_cache(), b.table, b.start, b.len, heads, scale, q.float().cpu().numpy().reshape(b.rows, heads, b.d),
                                len(b.new) == 1 and most > 16)
    got = out.float().cpu().numpy().reshape(b.rows, heads, b.d)
    n = b.tokens
    bad = ~(np.abs(got[:n] - ref[:n]) <= tol[:n])
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got[:n] - ref[:n])[bad])), np.argwhere(bad)[:4])
    assert (got[n:] == 9).all()
    return q, out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kvh,group", [(1, 1), (2, 3), (2, 4), (1, 8), (1, 11), (1, 16), (1, 24), (1, 40)])
def test_single_tokens(tern, d, kvh, group):
    b = util().Batch([1, 1, 1, 1, 0, 1], [1, 15, 64, 65, 9, 300], kvh, d, 32, seed=group, tail=2)
    b.fill_values()
    run_attention(tern, b, kvh * group)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(tern, page):
    b = util().Batch([1, 2, 1], [page - 1, page + 1, 3 * page], 2, 64, page, seed=page)
    b.fill_values()
    run_attention(tern, b, 4)


@pytest.mark.parametrize("new", [2, 5, 8, 9, 31, 32, 33, 70, 129])
@pytest.mark.parametrize("d", [64, 128])
def test_several_new_tokens(tern, new, d):
    b = util().Batch([new, 1, new - 1], [new, 200, new + 90], 1, d, 16, seed=new)
    b.fill_values()
    run_attention(tern, b, 3)


@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("length", [127, 128, 129, 255, 256, 257, 400])
def test_prompts(tern, length, group):
    b = util().Batch([length, 130], [length, 140], 1, 128, 64, seed=length)
    b.fill_values()
    run_attention(tern, b, group)


def test_rows_that_see_nothing(tern):
    b = util().Batch([5, 3, 200, 1], [2, 0, 150, 0], 2, 64, 16, seed=11)
    b.fill_values()
    _, out = run_attention(tern, b, 4)
    assert (out[:3] == 0).all() and (out[5:8] == 0).all() and (out[-1] == 0).all()


def test_split_and_joined(tern):
    b = util().Batch([1, 1], [3000, 700], 1, 128, 64, seed=12)
    b.fill_values()
    q, first = run_attention(tern, b, 4)
    cache, batch = b.device()
    ws = util().workspace(cache, 4, 2, 1, 3000)
    for _ in range(3):                                    # the workspace is left ready; the join's order is fixed
        out = torch.empty_like(q)
        cache.attention(batch, q, 1 / np.sqrt(128), out, ws)
        assert torch.equal(out, first)


def test_one_workspace_for_unequal_batches(tern):
    u = util()
    ws = None
    batches = [u.Batch([1], [2000], 1, 64, 64, seed=13), u.Batch([1] * 6, [900] * 6, 2, 64, 64, seed=14), u.Batch([7, 2], [600, 1100], 1, 64, 64, seed=15)]
    cache, _ = batches[0].device()
    for b in batches:
        b.fill_values()
    n = max(tern.KV4Cache(torch.empty(64 * 72 * 2, dtype=torch.uint8, device="cuda"), 2, 64, 64).attention_workspace_size(6, 7, 2000, 8), 1)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for b in batches + batches[::-1]:
        run_attention(tern, b, 4 * b.kvh, ws=ws)


def test_peaked_and_flat_scores(tern):
    b = util().Batch([1, 3], [500, 300], 2, 128, 32, seed=16)
    b.fill_values(spread=3.0)
    run_attention(tern, b, 8, spread=20.0)                # one key takes nearly everything
    run_attention(tern, b, 8, scale=0.0)                  # all alike
    run_attention(tern, b, 8, scale=-0.05)


def test_prompts_peaked_flat_and_negative(tern):
    b = util().Batch([40, 33], [300, 33], 1, 128, 32, seed=22)
    b.fill_values(spread=2.0)
    run_attention(tern, b, 4, spread=10.0)
    run_attention(tern, b, 4, scale=0.0)
    run_attention(tern, b, 4, scale=-0.05)
    run_attention(tern, b, 4, spread=1e-6, scale=3.0)
    run_attention(tern, b, 4, spread=1e9, scale=1e-9)


def test_prompt_rows_of_very_different_size(tern):
    # one huge query row must not cost the others their bits
    u = util()
    b = u.Batch([30], [200], 1, 64, 16, seed=23)
    b.fill_values()
    g = np.random.default_rng(5)
    q = g.standard_normal((30, 4 * 64))
    q[7, 64:128] *= 1e12
    q[9, :64] *= 1e-12
    run_attention(tern, b, 4, q=u.bf16_dev(q))
    b = u.Batch([3], [200], 1, 64, 16, seed=24)
    b.fill_values()
    run_attention(tern, b, 4, q=u.bf16_dev(q[6:9]))


def test_maxima_that_keep_growing(tern):
    # keys ordered so that every block passes the running maximum by more than any threshold: the accumulators are
    # rescaled again and again
    u = util()
    for new, heads in ((1, 4), (40, 4)):
        b = u.Batch([new], [700], 1, 64, 16, seed=25)
        c = b.oracle_cache()
        for j in range(700):
            x = np.full(64, 0.02 * j, np.float32)
            x[::2] += 0.01
            for w in range(2):
                q, s, m = prompt.quantize4((x if w == 0 else b.g.standard_normal(64).astype(np.float32))[None])
                c.put(int(b.table[0, j // 16]), j % 16, 0, w, q[0], s[0], m[0])
        run_attention(tern, b, heads, scale=1.0, q=u.bf16_dev(np.abs(b.g.standard_normal((new, heads * 64))) + 0.5))


@pytest.mark.parametrize("new,heads", [(5, 2), (60, 2)])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_values_that_are_not_numbers_stay_behind_the_mask(tern, new, heads, which, bad):
    # a position whose key or value scale is not finite: rows that do not see it are as without it; rows that do are
    # not numbers (its keys being infinite may also leave no finite score)
    u = util()
    b = u.Batch([new], [400], 1, 64, 16, seed=26)
    b.fill_values()
    q, want = run_attention(tern, b, heads)
    at = 400 - new + new // 2
    codes, s, m = b.oracle_cache().get(int(b.table[0, at // 16]), at % 16, 0, which)
    codes[:] = 3
    b.oracle_cache().put(int(b.table[0, at // 16]), at % 16, 0, which, codes, np.float16(bad), m)
    cache, batch = b.device()
    out = torch.empty_like(q)
    cache.attention(batch, q, 1 / 8, out, u.workspace(cache, heads, 1, new, 400))
    torch.cuda.synchronize()
    assert torch.equal(out[:new // 2], want[:new // 2])
    if which == 1 or bad == "nan":
        assert not out[new // 2:].isfinite().all(1).any()


def test_hundreds_of_sequences(tern):
    # more sequences than threads: the search for a CTA's share takes several turns
    new = np.array([1, 0, 2, 1, 1] * 200)
    length = new + np.arange(1000) % 7
    b = util().Batch(new, length, 1, 64, 16, seed=27)
    b.fill_values()
    run_attention(tern, b, 2)
    new = np.array([0, 1, 1, 1, 20] + [1] * 900)
    b = util().Batch(new, new + 3, 1, 64, 16, seed=28)
    b.fill_values()
    run_attention(tern, b, 2)                             # one prompt among nine hundred single tokens


def test_prompts_cut_between_ctas(tern):
    # long histories and few rows: one tile's blocks go to several CTAs; the join's order is fixed
    u = util()
    b = u.Batch([10, 6], [6000, 3000], 1, 64, 64, seed=29)
    b.fill_values()
    q, first = run_attention(tern, b, 4)
    cache, batch = b.device()
    ws = u.workspace(cache, 4, 2, 10, 6000)
    for _ in range(3):
        out = torch.empty_like(q)
        cache.attention(batch, q, 1 / 8, out, ws)
        assert torch.equal(out, first)


@pytest.mark.parametrize("page_entry", [10 ** 6, -1])
def test_bad_page_in_a_prompt(tern, page_entry):
    u = util()
    good = u.Batch([50, 40], [60, 90], 2, 64, 16, seed=30)
    good.fill_values()
    b = u.Batch([50, 40], [60, 90], 2, 64, 16, seed=30)
    b.raw = good.raw.copy()
    b.table[0, 2] = page_entry                            # positions 32 .. 47 of the first sequence
    q = torch.randn((90, 128), device="cuda").bfloat16()
    outs = []
    for x in (b, good):
        cache, batch = x.device()
        o = torch.full_like(q, 9.0)
        cache.attention(batch, q, 0.1, o, u.workspace(cache, 2, 2, 50, 90))
        assert tern.device_error() == (tern.EFORMAT if x is b else tern.OK)
        outs.append(o)
    assert torch.equal(outs[0][50:], outs[1][50:])
    ref, tol = attention_without(good, q, 0.1, 0, range(32, 48))
    got = outs[0][:50].float().cpu().numpy().reshape(50, 2, 64)
    # the expanded operands' own terms: scores off by 2^-11 sum |q| |k|, values and probabilities by 2^-11 each
    qn = np.abs(q[:50].float().cpu().numpy().reshape(50, 2, 64)).sum(2, keepdims=True)
    assert (np.abs(got - ref) <= tol + 2.0 ** -10 * 5 + 2 * 2.0 ** -11 * 0.1 * qn * 5 * 5).all()


def test_bounds_larger_than_the_batch(tern):
    b = util().Batch([1, 2], [70, 40], 1, 64, 16, seed=17)
    b.fill_values()
    b.table = np.concatenate([b.table, np.full((2, 200), -7, np.int32)], 1)
    run_attention(tern, b, 4, max_new=40, max_len=3000)
    run_attention(tern, b, 4, max_new=400, max_len=3000)


def test_in_place_and_other_stream(tern):
    u = util()
    b = u.Batch([1, 40], [1500, 40], 2, 64, 16, seed=18)
    b.fill_values()
    q, want = run_attention(tern, b, 6)
    cache, batch = b.device()
    ws = u.workspace(cache, 6, 2, 40, 1500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.attention(batch, q, 1 / 8, q, ws)
    torch.cuda.synchronize()
    assert torch.equal(q, want)


def test_not_a_number_in_one_row(tern):
    u = util()
    b = u.Batch([9], [700], 1, 128, 16, seed=19)
    b.fill_values()
    q, want = run_attention(tern, b, 4)
    q[3, 130] = float("nan")                              # head 1 of token 3
    cache, batch = b.device()
    out = torch.empty_like(q)
    cache.attention(batch, q, 1 / np.sqrt(128), out, u.workspace(cache, 4, 1, 9, 700))
    keep = torch.ones((9, 4, 128), dtype=torch.bool, device="cuda")
    keep[3, 1] = False
    assert torch.equal(out.view(9, 4, 128)[keep], want.view(9, 4, 128)[keep]) and out.view(9, 4, 128)[3, 1].isnan().all()


def test_replay_follows_the_lengths(tern):
    # one captured step per token: append and attention; lengths and rows change between replays
    u = util()
    d, kvh, heads, page = 64, 2, 4, 16
    b = u.Batch([1, 1], [600, 40], kvh, d, page, seed=20)
    b.fill_values()
    cache, batch = b.device(max_len=600)
    start, length, _ = batch._keep
    ws = u.workspace(cache, heads, 2, 1, 600)
    rope = torch.from_numpy(tern.decode_rope_table(600, d)).cuda()
    xq, xk, xv = (torch.zeros((2, h * d), device="cuda") for h in (heads, kvh, kvh))
    qo = torch.empty((2, heads * d), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(qo)

    def step():
        cache.append(batch, xq, xk, xv, rope, qo)
        cache.attention(batch, qo, 0.125, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(1)
    for lens in ([600, 40], [300, 33], [17, 1], [599, 20]):
        length.copy_(torch.tensor(lens, dtype=torch.int32))
        for x in (xq, xk, xv):
            x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        raw = b.pages.cpu().numpy()
        ref, tol = prompt.attention(b.oracle_cache(raw), b.table, b.start, lens, heads, 0.125, qo.float().cpu().numpy().reshape(2, heads, d))
        assert (np.abs(got.float().cpu().numpy().reshape(2, heads, d) - ref) <= tol).all()
    assert tern.device_error() == tern.OK


def test_offsets_beyond_32_bits(tern):
    # pages whose bytes start above 2^32
    kvh, d, page = 8, 128, 256
    size = kvh * page * (d + 8)
    total = (1 << 32) // size + 40
    pages = torch.empty(total * size, dtype=torch.uint8, device="cuda")
    cache = tern.KV4Cache(pages, kvh, d, page)
    table = torch.tensor([[total - 1, total - 9, 3]], dtype=torch.int32, device="cuda")
    n = 600
    batch = tern.KV4Batch(torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda"), table, n, n, n)
    small = torch.empty(3 * size, dtype=torch.uint8, device="cuda")
    cache2 = tern.KV4Cache(small, kvh, d, page)
    batch2 = tern.KV4Batch(batch._keep[0], batch._keep[1], torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"), n, n, n)
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn((n, kvh * d), generator=g, device="cuda") for _ in range(3))
    rope = torch.from_numpy(tern.decode_rope_table(n, d)).cuda()
    ws = util().workspace(cache, kvh, 1, n, n)
    outs = []
    for c, b in ((cache, batch), (cache2, batch2)):
        qo, ko = torch.empty((n, kvh * d), dtype=torch.bfloat16, device="cuda"), torch.empty((n, kvh * d), device="cuda")
        c.append(b, q, k, v, rope, qo)
        c.read(b, ko, None)
        o = torch.empty_like(qo)
        c.attention(b, qo, 0.09, o, ws)
        one = tern.KV4Batch(torch.tensor([0, 1], dtype=torch.int32, device="cuda"), b._keep[1], b._keep[2], 1, 1, n)
        o1 = torch.empty((1, kvh * d), dtype=torch.bfloat16, device="cuda")
        c.attention(one, qo[-1:].contiguous(), 0.09, o1, ws)
        outs.append((ko, o, o1))
    torch.cuda.synchronize()
    assert tern.device_error() == tern.OK
    for a, e in zip(*outs):
        assert torch.equal(a, e)


def test_binding_refuses(tern):
    u = util()
    b = u.Batch([2], [2], 2, 64, 16, seed=21)
    cache, batch = b.device()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros((2, 256), device="cuda"), torch.zeros((2, 128), device="cuda")
    rope, qo = torch.zeros((4, 32, 2), device="cuda"), torch.zeros((2, 256), **bf)
    ok = dict(q=q, k=k, v=k, rope=rope, q_out=qo)
    for bad in (dict(q=q[:1]), dict(k=q), dict(v=k.bfloat16()), dict(rope=rope[:, :16]), dict(q_out=None), dict(q_out=q), dict(k=k.cpu()),
                dict(q=torch.zeros((2, 100), device="cuda")), dict(rope=rope.double())):
        with pytest.raises(tern.TernError):
            cache.append(batch, **(ok | bad))
    for bad in (dict(k=None, v=None), dict(k=q), dict(k=k, v=k.bfloat16()), dict(k=k[:1], v=None)):
        with pytest.raises(tern.TernError):
            cache.read(batch, **(dict(k=k, v=k) | bad))
    o = torch.zeros((2, 256), **bf)
    for bad in (dict(q=q), dict(out=o[:1]), dict(q=o[:, :128]), dict(scale=float("inf")), dict(out=o.cpu())):
        with pytest.raises(tern.TernError):
            cache.attention(batch, **(dict(q=o, scale=0.1, out=o) | bad))
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(start=i.long()), dict(len=i), dict(table=i), dict(table=i.view(1, 3))):
        with pytest.raises(tern.TernError):
            tern.KV4Batch(**(dict(start=i, len=i[:2], table=torch.zeros((2, 3), dtype=torch.int32, device="cuda"), tokens=2, max_new=1, max_len=4) | bad))
    for bad in ((b.pages[1:], 2, 64, 16), (b.pages.int(), 2, 64, 16), (b.pages, 0, 64, 16)):
        with pytest.raises(tern.TernError):
            tern.KV4Cache(*bad)
