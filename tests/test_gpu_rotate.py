"""jf_rotate_append_kv and its packed form against 64-bit rotations: layouts, head shapes, partial and
interleaved rotation, norms, strided inputs, far positions, what must not be written, bad pages and
lengths, streams and graphs."""
import math

import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module")
def jf():
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf as mod
    return mod


def make(B, N, Hq, Hkv, D, sizes, lens, seed, R, norm, spread=100000):
    g = torch.Generator().manual_seed(seed)
    need = [-(-(p + n) // PAGE) for p, n in zip(lens, sizes)]
    cap = -(-(max(lens) + N) // PAGE)
    order = torch.randperm(sum(need) + 3, generator=g).to(torch.int32)
    table = torch.full((B, cap), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    return dict(qkv=bf(B, N, (Hq + 2 * Hkv) * D), pos=torch.randint(0, spread, (B, N), generator=g, dtype=torch.int32),
                freq=10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R) if R else None,
                wq=bf(D) + 1 if norm else None, wk=bf(D) + 1 if norm else None, table=table,
                lens=torch.tensor(lens, dtype=torch.int32), kc=bf(sum(need) + 3, PAGE, Hkv, D),
                vc=bf(sum(need) + 3, PAGE, Hkv, D), sizes=sizes, shape=(B, N, Hq, Hkv, D))


def cuda(t):
    return None if t is None else t.cuda()


def bits(t):
    return t.cpu().contiguous().view(torch.int16)


def call(jf, w, layout, inter, scale, out=None, norm_eps=1e-6, dev_err=None, k_cache=None, v_cache=None, stream=None):
    B, N, Hq, Hkv, D = w["shape"]
    kc, vc = cuda(w["kc"]) if k_cache is None else k_cache, cuda(w["vc"]) if v_cache is None else v_cache
    heads = w["qkv"].view(B, N, Hq + 2 * Hkv, D)
    pos, extra = w["pos"], {}
    if layout == "packed":
        heads = torch.cat([heads[b, :n] for b, n in enumerate(w["sizes"])])
        pos = torch.cat([pos[b, :n] for b, n in enumerate(w["sizes"])])
        cu = [0]
        for n in w["sizes"]:
            cu.append(cu[-1] + n)
        extra = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), N_max=N)
    elif layout == "ragged":
        extra = dict(tree_len=torch.tensor(w["sizes"], dtype=torch.int32).cuda())
    x = heads.cuda()
    q, k, v = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :]
    if out is None:
        out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    got = jf.rotate_append_kv(q, k, v, kc, vc, w["table"].cuda(), w["lens"].cuda(),
                              pos=pos.cuda() if w["freq"] is not None else None, freq=cuda(w["freq"]),
                              interleaved=inter, rotary_scale=scale, q_norm=cuda(w["wq"]), k_norm=cuda(w["wk"]),
                              norm_eps=norm_eps, out=out, dev_err=dev_err, stream=stream, **extra)
    return got, kc, vc


def check(w, layout, inter, scale, got, kc, vc, norm_eps=1e-6):
    B, N, Hq, Hkv, D = w["shape"]
    heads = w["qkv"].view(B, N, Hq + 2 * Hkv, D)
    kw, vw = w["kc"].clone(), w["vc"].clone()
    kc, vc, got = kc.cpu(), vc.cpu(), got.cpu()
    first = 0
    for b, n in enumerate(w["sizes"]):
        rows = got[first:first + n] if layout == "packed" else got[b, :n]
        want, tol = ref.rotate(heads[b, :n, :Hq], w["pos"][b, :n], w["freq"], inter, scale, w["wq"], norm_eps)
        assert ref.within(rows, want, tol), ("q", b)
        if layout == "ragged":
            assert (got[b, n:] == -7.0).all()
        first += n
        t = torch.arange(n) + int(w["lens"][b])
        at = w["table"][b][t // PAGE].long(), t % PAGE
        want, tol = ref.rotate(heads[b, :n, Hq:Hq + Hkv], w["pos"][b, :n], w["freq"], inter, scale, w["wk"], norm_eps)
        assert ref.within(kc[at], want, tol), ("k", b)
        kw[at] = kc[at]                                   # everything else stays as it was
        vw[at] = heads[b, :n, Hq + Hkv:]
    assert torch.equal(bits(kc), bits(kw)) and torch.equal(bits(vc), bits(vw))


SHAPES = [
    # B  N    Hq Hkv D    R    interleaved norm scale
    (1, 1, 4, 1, 64, 64, False, False, 1.0),
    (1, 1, 32, 8, 128, 128, True, True, 1.0),
    (3, 7, 4, 2, 128, 64, False, True, 1.0),
    (2, 33, 5, 5, 64, 16, True, False, 1.25),
    (2, 17, 6, 3, 64, 48, False, True, 0.5),
    (2, 20, 64, 4, 128, 96, True, True, 1.0),
    (1, 9, 1, 1, 128, 112, False, False, -1.0),
    (3, 5, 3, 1, 64, 0, False, True, 1.0),
    (2, 6, 8, 2, 128, 0, False, False, 1.0),
    (4, 200, 8, 2, 128, 128, False, True, 1.1386),
    (2, 700, 4, 1, 64, 32, True, True, 1.0),
    (40, 18, 2, 1, 64, 64, False, False, 1.0),
]


@pytest.mark.parametrize("layout", ["padded", "ragged", "packed"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rotation_and_append(jf, shape, layout):
    B, N, Hq, Hkv, D, R, inter, norm, scale = shape
    sizes = [N] * B if layout == "padded" else [1 + (N - 1) * (b + 1) // B for b in range(B)]
    w = make(B, N, Hq, Hkv, D, sizes, [(37 * b + 5) % 70 for b in range(B)], seed=B * N + D, R=R, norm=norm)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, kc, vc = call(jf, w, layout, inter, scale, dev_err=err)
    assert err.item() == 0
    check(w, layout, inter, scale, got, kc, vc)


@pytest.mark.parametrize("inter", [False, True])
def test_far_and_negative_positions(jf, inter):
    w = make(1, 8, 4, 1, 128, [8], [3], seed=1, R=128, norm=False)
    w["pos"] = torch.tensor([[0, 1, -1, 131071, 1000000, -123456, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    got, kc, vc = call(jf, w, "padded", inter, 1.0)
    check(w, "padded", inter, 1.0, got, kc, vc)


def test_fast_frequencies_and_quarter_turns(jf):
    """Frequencies of a whole turn and more, and exact quarters of a turn."""
    w = make(1, 6, 2, 1, 64, [6], [0], seed=2, R=16, norm=False)
    w["freq"] = torch.tensor([0.0, math.pi / 2, 2 * math.pi, 7.0, 100.0, -1.0, math.pi, 1e-12], dtype=torch.float64)
    w["pos"] = torch.arange(6, dtype=torch.int32)[None]
    got, kc, vc = call(jf, w, "padded", False, 1.0)
    check(w, "padded", False, 1.0, got, kc, vc)


def test_norm_of_zero_and_of_large_heads(jf):
    w = make(1, 4, 4, 2, 128, [4], [0], seed=3, R=128, norm=True)
    w["qkv"][0, 0] = 0.0
    w["qkv"][0, 1] *= 1e15
    w["qkv"][0, 2] *= 1e-12
    got, kc, vc = call(jf, w, "padded", False, 1.0, norm_eps=1e-5)
    check(w, "padded", False, 1.0, got, kc, vc, norm_eps=1e-5)


@pytest.mark.parametrize("alone", ["wq", "wk"])
def test_one_norm_alone(jf, alone):
    for R in (0, 64):
        w = make(2, 11, 6, 2, 128, [11, 4], [3, 20], seed=12, R=R, norm=True)
        w[alone] = None
        got, kc, vc = call(jf, w, "ragged", False, 1.0)
        check(w, "ragged", False, 1.0, got, kc, vc)


def test_packed_equals_padded(jf):
    w = make(5, 40, 8, 2, 128, [40, 1, 17, 39, 2], [0, 15, 16, 100, 31], seed=4, R=64, norm=True)
    a, ka, va = call(jf, w, "ragged", False, 1.0)
    p, kp, vp = call(jf, w, "packed", False, 1.0)
    assert torch.equal(bits(ka), bits(kp)) and torch.equal(bits(va), bits(vp))
    assert torch.equal(bits(p), bits(torch.cat([a[b, :n] for b, n in enumerate(w["sizes"])])))


def test_many_packed_sequences(jf):
    """1200 sequences of one to three tokens: three rounds of the search for a row's sequence."""
    B = 1200
    w = make(B, 3, 2, 1, 64, [1 + b % 3 for b in range(B)], [b % 40 for b in range(B)], seed=5, R=64, norm=False)
    got, kc, vc = call(jf, w, "packed", False, 1.0)
    check(w, "packed", False, 1.0, got, kc, vc)


@pytest.mark.parametrize("norm", [False, True])
def test_queries_in_place_and_keys_alone(jf, norm):
    w = make(2, 9, 4, 2, 128, [9, 9], [3, 20], seed=6, R=128, norm=norm)
    B, N, Hq, Hkv, D = w["shape"]
    got, kc, vc = call(jf, w, "padded", False, 1.0)
    x = w["qkv"].view(B, N, -1, D).cuda()
    q, k, v = (t.contiguous() for t in x.split([Hq, Hkv, Hkv], dim=2))
    args = (w["table"].cuda(), w["lens"].cuda())
    kw = dict(pos=w["pos"].cuda(), freq=w["freq"].cuda(), q_norm=cuda(w["wq"]), k_norm=cuda(w["wk"]))
    k2, v2 = w["kc"].cuda(), w["vc"].cuda()
    assert jf.rotate_append_kv(q, k, v, k2, v2, *args, out=q, **kw) is q
    assert torch.equal(bits(q), bits(got)) and torch.equal(bits(k2), bits(kc)) and torch.equal(bits(v2), bits(vc))
    k3, v3 = w["kc"].cuda(), w["vc"].cuda()
    assert jf.rotate_append_kv(None, k, v, k3, v3, *args, **kw) is None
    assert torch.equal(bits(k3), bits(kc)) and torch.equal(bits(v3), bits(vc))


@pytest.mark.parametrize("layout", ["padded", "packed"])
def test_bad_pages_and_lengths(jf, layout):
    """What is malformed is reported and not written; everything else is."""
    w = make(4, 20, 2, 1, 64, [20] * 4, [10, 10, 10, 10], seed=7, R=64, norm=False)
    pages = w["kc"].shape[0]
    clean, kc0, vc0 = call(jf, w, layout, False, 1.0)
    table, lens = w["table"].clone(), w["lens"].clone()
    w["table"][0, 1] = pages                       # tokens 6 .. of sequence 0
    w["table"][1, 0] = -5                          # tokens 0 .. 5 of sequence 1
    w["lens"][2] = -1
    w["lens"][3] = 16 * table.shape[1] - 19        # one token too far
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, kc, vc = call(jf, w, layout, False, 1.0, dev_err=err)
    assert err.item() == jf.DEVERR_BAD_PAGE | jf.DEVERR_BAD_PREFIX
    assert torch.equal(bits(got), bits(clean))     # queries need no page
    kw, vw = w["kc"].clone(), w["vc"].clone()
    for b, lo, hi in ((0, 0, 6), (1, 6, 20)):      # page 1 of sequence 0 holds its tokens 6 .. 19 (10 + 6 = 16)
        t = torch.arange(lo, hi) + 10
        at = table[b][t // PAGE].long(), t % PAGE
        kw[at], vw[at] = kc0.cpu()[at], vc0.cpu()[at]
    assert torch.equal(bits(kc), bits(kw)) and torch.equal(bits(vc), bits(vw))


def test_bad_spans_and_tree_lengths(jf):
    w = make(4, 8, 2, 1, 64, [8] * 4, [0] * 4, seed=8, R=64, norm=False)
    B, N, Hq, Hkv, D = w["shape"]
    x = w["qkv"].view(B * N, -1, D).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    for cu in ([0, 8, 8, 20, 32], [0, 8, 4, 16, 32], [0, 9, 17, 24, 40], [-3, 4, 12, 20, 32], [5, 5, 5, 5, 5]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
        kc, vc = w["kc"].cuda(), w["vc"].cuda()
        jf.rotate_append_kv(q, k, v, kc, vc, w["table"].cuda(), w["lens"].cuda(), pos=w["pos"].flatten().cuda(),
                            freq=w["freq"].cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), N_max=8,
                            out=out, dev_err=err)
        assert err.item() == jf.DEVERR_BAD_TREE_LEN, cu
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = w["qkv"].view(B, N, -1, D).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], dim=2)
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    jf.rotate_append_kv(q, k, v, w["kc"].cuda(), w["vc"].cuda(), w["table"].cuda(), w["lens"].cuda(),
                        pos=w["pos"].cuda(), freq=w["freq"].cuda(),
                        tree_len=torch.tensor([0, 9, 3, 8], dtype=torch.int32).cuda(), out=out, dev_err=err)
    assert err.item() == jf.DEVERR_BAD_TREE_LEN
    assert (out[0, 1:] == -7.0).all() and (out[2, 3:] == -7.0).all() and (out[1] != -7.0).any()


def test_packed_rows_behind_the_last_sequence(jf):
    w = make(3, 10, 4, 2, 64, [10, 4, 7], [3, 30, 0], seed=12, R=64, norm=True)
    want, kw, vw = call(jf, w, "packed", False, 1.0)
    B, N, Hq, Hkv, D = w["shape"]
    x = torch.cat([w["qkv"].view(B, N, -1, D)[b, :n] for b, n in enumerate(w["sizes"])] + [torch.full((9, Hq + 2 * Hkv, D), float("nan")).to(torch.bfloat16)]).cuda()
    pos = torch.cat([w["pos"][b, :n] for b, n in enumerate(w["sizes"])] + [torch.full((9,), 5, dtype=torch.int32)]).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    kc, vc = w["kc"].cuda(), w["vc"].cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    jf.rotate_append_kv(q, k, v, kc, vc, w["table"].cuda(), w["lens"].cuda(), pos=pos, freq=w["freq"].cuda(),
                        q_norm=w["wq"].cuda(), k_norm=w["wk"].cuda(),
                        cu_seqlens=torch.tensor([0, 10, 14, 21], dtype=torch.int32).cuda(), N_max=N, out=out, dev_err=err)
    assert err.item() == 0 and (out[21:] == -7.0).all()
    assert torch.equal(bits(out[:21]), bits(want)) and torch.equal(bits(kc), bits(kw)) and torch.equal(bits(vc), bits(vw))


def test_pool_past_32_bit_offsets(jf):
    """A pool of more than 2^31 elements: its last page is written, and read from a far offset."""
    Hkv, D = 8, 128
    pages = (1 << 31) // (PAGE * Hkv * D) + 5
    w = make(1, 5, 8, Hkv, D, [5], [14], seed=9, R=128, norm=False)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    kc = torch.zeros((pages, PAGE, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    w["table"] = table
    got, _, _ = call(jf, w, "padded", False, 1.0, k_cache=kc, v_cache=vc)
    t = torch.arange(5) + 14
    at = (pages - 1 - t // PAGE), t % PAGE
    want, tol = ref.rotate(w["qkv"].view(5, -1, D)[:, 8:16], w["pos"][0], w["freq"], False, 1.0, None, 0.0)
    assert ref.within(kc[at[0].cuda(), at[1].cuda()].cpu(), want, tol)
    assert torch.equal(vc[at[0].cuda(), at[1].cuda()].cpu(), w["qkv"].view(5, -1, D)[:, 16:])
    assert kc.view(-1)[:kc.numel() - 2 * PAGE * Hkv * D].count_nonzero() == 0


def test_streams_and_graphs(jf):
    w = make(2, 30, 4, 2, 128, [30, 30], [3, 20], seed=10, R=128, norm=True)
    want, kw, vw = call(jf, w, "padded", False, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    with torch.cuda.stream(side):
        kc, vc = w["kc"].cuda(), w["vc"].cuda()
    side.synchronize()
    got, _, _ = call(jf, w, "padded", False, 1.0, out=out, k_cache=kc, v_cache=vc, stream=side)
    side.synchronize()
    assert torch.equal(bits(got), bits(want)) and torch.equal(bits(kc), bits(kw)) and torch.equal(bits(vc), bits(vw))
    B, N, Hq, Hkv, D = w["shape"]
    x = torch.zeros((B, N, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([Hq, Hkv, Hkv], dim=2)
    kc, vc = w["kc"].cuda(), w["vc"].cuda()
    args = (q, k, v, kc, vc, w["table"].cuda(), w["lens"].cuda())
    kwargs = dict(pos=w["pos"].cuda(), freq=w["freq"].cuda(), q_norm=w["wq"].cuda(), k_norm=w["wk"].cuda(), out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jf.rotate_append_kv(*args, **kwargs)
    out.zero_()
    x.copy_(w["qkv"].view(x.shape).cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want)) and torch.equal(bits(kc), bits(kw))
