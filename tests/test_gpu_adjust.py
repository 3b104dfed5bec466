"""jf_adjust_logits, its packed form and jf_count_tokens against 64-bit rows and whole-number counts."""
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def jf():
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf as mod
    return mod


def new_err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def cuda(t):
    return None if t is None else t.cuda()


def make(B, N, V, dtype, seed, counts=True, bias=True, grammar=True, sizes=None):
    g = torch.Generator().manual_seed(seed)
    parent, sees = ref.random_trees(B, N, g)
    few = min(V, 12)                                # drafted tokens repeat along branches
    w = dict(shape=(B, N, V), sizes=sizes or [N] * B, sees=sees, mask=ref.pack_bits(sees), parent=parent,
             logits=(torch.randn((B, N, V), generator=g) * 3).to(dtype),
             draft=torch.randint(0, few, (B, N), generator=g, dtype=torch.int32) * (V // few),
             count=None, bias=None, allowed=None, allowed_row=None, rep=None, pres=None, freq=None)
    if counts:
        count = torch.randint(0, 4, (B, V), generator=g, dtype=torch.int32)
        count *= (torch.rand((B, V), generator=g) < 0.3).to(torch.int32)
        w["count"] = count | (torch.rand((B, V), generator=g) < 0.3).to(torch.int32) * ref.PROMPT
        w["rep"] = 0.7 + torch.rand(B, generator=g)
        w["pres"] = torch.rand(B, generator=g) - 0.2
        w["freq"] = torch.rand(B, generator=g) - 0.2
    if bias:
        w["bias"] = torch.randn((B, V), generator=g) * (torch.rand((B, V), generator=g) < 0.2)
    if grammar:
        words = torch.randint(-2 ** 31, 2 ** 31, (B * N, -(-V // 32)), generator=g).to(torch.int32)
        words[B * N // 2] = 0                       # a row whose grammar leaves nothing
        w["allowed"] = words
        row = torch.randperm(B * N, generator=g).to(torch.int32).view(B, N)
        row[torch.rand((B, N), generator=g) < 0.2] = -1
        w["allowed_row"] = row
    return w


def rows_of(w, x, layout):
    return torch.cat([x[b, :n] for b, n in enumerate(w["sizes"])]) if layout == "packed" and x is not None else x


def call(jf, w, layout, out_dtype=None, masked=-INF, out=None, logits=None, dev_err=None, stream=None):
    B, N, V = w["shape"]
    extra = {}
    if layout == "packed":
        cu = [0]
        for n in w["sizes"]:
            cu.append(cu[-1] + n)
        extra = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), N_max=N)
    elif layout == "ragged":
        extra = dict(tree_len=torch.tensor(w["sizes"], dtype=torch.int32).cuda())
    logits = rows_of(w, w["logits"], layout).cuda() if logits is None else logits
    if out is None:
        out = torch.full(logits.shape, -7.0, dtype=out_dtype or logits.dtype, device="cuda")
    with_draft = w["draft"] is not None
    return jf.adjust_logits(
        logits, count=cuda(w["count"]), draft=cuda(rows_of(w, w["draft"], layout)) if with_draft else None,
        mask=cuda(rows_of(w, w["mask"], layout)) if with_draft else None, bias=cuda(w["bias"]),
        allowed=cuda(w["allowed"]), allowed_row=cuda(rows_of(w, w["allowed_row"], layout)),
        repetition=cuda(w["rep"]), presence=cuda(w["pres"]), frequency=cuda(w["freq"]), masked=masked, out=out,
        dev_err=dev_err, stream=stream, **extra)


def expected(w, b, i, masked, dtype):
    B, N, V = w["shape"]
    had = torch.zeros(V, dtype=torch.int64)
    prompt = torch.zeros(V, dtype=torch.bool)
    if w["count"] is not None:
        had += w["count"][b].long() % ref.PROMPT
        prompt = w["count"][b] >= ref.PROMPT
    if w["draft"] is not None:
        for j in range(1, w["sizes"][b]):
            if w["sees"][b, i, j] and 0 <= int(w["draft"][b, j]) < V:
                had[int(w["draft"][b, j])] += 1
    one = lambda k, d: d if w[k] is None else float(w[k][b])  # noqa: E731
    ok = None
    if w["allowed"] is not None:
        row = b * N + i if w["allowed_row"] is None else int(w["allowed_row"][b, i])
        ok = ref.unpack(w["allowed"][row], V) if 0 <= row < w["allowed"].shape[0] else None
    return ref.adjust(w["logits"][b, i], had, prompt, one("rep", 1.0), one("pres", 0.0), one("freq", 0.0),
                      None if w["bias"] is None else w["bias"][b], ok, masked, dtype)


def check(w, layout, got, masked=-INF):
    first = 0
    got = got.cpu()
    for b, n in enumerate(w["sizes"]):
        for i in range(n):
            want, tol = expected(w, b, i, masked, got.dtype)
            assert ref.within(got[first + i] if layout == "packed" else got[b, i], want, tol), (b, i)
        first += n
        if layout == "ragged":
            assert (got[b, n:] == -7.0).all()


SHAPES = [
    # B  N   V      in              out
    (1, 1, 1, torch.float32, torch.float32),
    (2, 3, 7, torch.bfloat16, torch.bfloat16),
    (1, 5, 8, torch.bfloat16, torch.float32),
    (3, 9, 2048, torch.bfloat16, torch.bfloat16),
    (2, 17, 2049, torch.float32, torch.float32),
    (2, 40, 5000, torch.bfloat16, torch.bfloat16),
    (2, 33, 4104, torch.bfloat16, torch.float32),
    (1, 70, 1031, torch.bfloat16, torch.float32),
    (4, 18, 50257, torch.float32, torch.float32),
    (2, 16, 151936, torch.bfloat16, torch.bfloat16),
]


@pytest.mark.parametrize("layout", ["padded", "ragged", "packed"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows(jf, shape, layout):
    B, N, V, dt, odt = shape
    sizes = None if layout == "padded" else [1 + (N - 1) * (b + 1) // B for b in range(B)]
    w = make(B, N, V, dt, seed=N + V, sizes=sizes)
    err = new_err()
    got = call(jf, w, layout, odt, dev_err=err)
    assert err.item() == 0 and got.dtype == odt
    check(w, layout, got)


@pytest.mark.parametrize("counts,drafts,bias,grammar", [
    (True, True, False, False), (True, False, False, False), (False, True, False, False), (False, False, True, False),
    (False, False, False, True), (False, False, False, False), (True, True, True, True)])
@pytest.mark.parametrize("V", [4096, 999])
def test_each_part_alone(jf, counts, drafts, bias, grammar, V):
    w = make(2, 11, V, torch.bfloat16, seed=5, counts=counts, bias=bias, grammar=grammar)
    if not counts and drafts:                       # penalties on drafted tokens without any history
        w["rep"], w["freq"] = torch.tensor([1.5, 0.8]), torch.tensor([0.25, 0.5])
    if not drafts:
        w["draft"] = None
    if grammar:
        w["allowed_row"] = None                     # row b * N + i
    check(w, "padded", call(jf, w, "padded"))


@pytest.mark.parametrize("V,dt", [(2056, torch.bfloat16), (2051, torch.float32)])
def test_in_place(jf, V, dt):
    w = make(3, 21, V, dt, seed=6, sizes=[21, 4, 13])
    for layout in ("ragged", "packed"):
        want = call(jf, w, layout)
        logits = rows_of(w, w["logits"], layout).cuda()
        got = call(jf, w, layout, logits=logits, out=logits)
        assert got is logits
        if layout == "ragged":                      # padding rows keep their logits
            for b, n in enumerate(w["sizes"]):
                assert torch.equal(got[b, n:].cpu(), w["logits"][b, n:])
                assert torch.equal(got[b, :n], want[b, :n])
        else:
            assert torch.equal(got, want)


def test_rows_that_start_anywhere(jf):
    """V a multiple of 8 with arrays that are not 16-byte aligned: element by element, equal bit for bit."""
    w = make(2, 6, 4104, torch.bfloat16, seed=7)
    want = call(jf, w, "padded")
    flat = torch.empty(w["logits"].numel() + 1, dtype=torch.bfloat16, device="cuda")
    logits = flat[1:].view(w["logits"].shape)
    logits.copy_(w["logits"])
    assert torch.equal(call(jf, w, "padded", logits=logits), want)
    out = torch.empty_like(flat)[1:].view(w["logits"].shape)
    assert torch.equal(call(jf, w, "padded", out=out), want)


def test_one_token_along_a_chain(jf):
    """Node i of a chain of 300 equal tokens has seen it i times; the root's own draft entry does not count."""
    w = make(1, 300, 100, torch.float32, seed=8, bias=False, grammar=False)
    w["sees"] = torch.ones(300, 300, dtype=torch.bool).tril()[None]
    w["mask"] = ref.pack_bits(w["sees"])
    w["draft"].fill_(42)
    w["draft"][0, 0] = -1
    err = new_err()
    got = call(jf, w, "padded", dev_err=err)
    assert err.item() == 0
    check(w, "padded", got)


def test_infinities_and_nan(jf):
    """Forbidden tokens' logits may be anything; -inf stays -inf under every penalty; a finite mask value."""
    for V in (64, 67):
        w = make(1, 8, V, torch.bfloat16, seed=9)
        w["allowed_row"] = torch.arange(8, dtype=torch.int32)[None]
        for i in range(8):
            ok = ref.unpack(w["allowed"][i], V)
            w["logits"][0, i][~ok] = torch.tensor([float("nan"), INF, -INF, 1.0])[torch.arange(int((~ok).sum())) % 4].to(torch.bfloat16)
            w["logits"][0, i, int(ok.nonzero()[0]) if ok.any() else 0] = -INF
        w["pres"].abs_()
        lowest = torch.finfo(torch.bfloat16).min
        for masked in (-INF, lowest, -1.0e4):
            got = call(jf, w, "padded", masked=masked)
            check(w, "padded", got, masked)
            assert not torch.isnan(got).any()
            empty = [i for i in range(8) if not ref.unpack(w["allowed"][i], V).any()]
            assert empty and (got[0, empty].float() == torch.tensor(masked).to(torch.bfloat16).float().item()).all()


def test_malformed_inputs_are_reported(jf):
    w = make(2, 10, 500, torch.float32, seed=10)
    w["draft"][0, 3], w["draft"][1, 4] = 500, -2
    err = new_err()
    check(w, "padded", call(jf, w, "padded", dev_err=err))
    assert err.item() == jf.DEVERR_BAD_TOKEN
    w = make(2, 10, 500, torch.float32, seed=11)
    w["allowed_row"][0, 0], w["allowed_row"][1, 9] = 20, -2
    err = new_err()
    check(w, "padded", call(jf, w, "padded", dev_err=err))
    assert err.item() == jf.DEVERR_BAD_PATH
    w = make(2, 10, 500, torch.float32, seed=12)
    err, lens = new_err(), torch.tensor([0, 11], dtype=torch.int32).cuda()
    out = torch.full(w["logits"].shape, -7.0, device="cuda")
    jf.adjust_logits(w["logits"].cuda(), bias=w["bias"].cuda(), tree_len=lens, out=out, dev_err=err)
    assert err.item() == jf.DEVERR_BAD_TREE_LEN and (out[0, 1:] == -7.0).all() and (out[1] != -7.0).all()
    flat = w["logits"].view(20, 500).cuda()
    for cu in ([0, 10, 10], [0, 11, 20], [-1, 9, 19], [0, 10, 21], [12, 4, 14]):
        err = new_err()
        out = torch.full(flat.shape, -7.0, device="cuda")
        jf.adjust_logits(flat, bias=w["bias"].cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), N_max=10,
                         out=out, dev_err=err)
        assert err.item() == jf.DEVERR_BAD_TREE_LEN, cu


def test_packed_rows_behind_the_last_sequence(jf):
    w = make(2, 10, 600, torch.float32, seed=15, sizes=[10, 4])
    B, N, V = w["shape"]
    rows = lambda k: torch.cat([rows_of(w, w[k], "packed"), w[k].flatten(0, 1)[:6]]).cuda()  # noqa: E731
    out = torch.full((20, V), -7.0, device="cuda")
    jf.adjust_logits(rows("logits"), count=w["count"].cuda(), draft=rows("draft"), mask=rows("mask"), bias=w["bias"].cuda(),
                     allowed=w["allowed"].cuda(), allowed_row=rows("allowed_row"), repetition=w["rep"].cuda(),
                     presence=w["pres"].cuda(), frequency=w["freq"].cuda(),
                     cu_seqlens=torch.tensor([0, 10, 14], dtype=torch.int32).cuda(), N_max=N, out=out)
    assert (out[14:] == -7.0).all()
    check(w, "packed", out[:14])


def test_dense_bias_and_full_histories(jf):
    """Every token changed: no part of a slice is a plain copy."""
    for V, dt in ((4096, torch.bfloat16), (2500, torch.float32)):
        w = make(2, 7, V, dt, seed=16)
        w["bias"] = torch.randn(2, V, generator=torch.Generator().manual_seed(1)) + 3.0
        w["count"] = w["count"] | ref.PROMPT
        check(w, "padded", call(jf, w, "padded"))


def test_largest_tree(jf):
    """4096 nodes: all words of the ancestor masks; a few rows are looked at."""
    N = jf.MAX_NODES
    w = make(1, N, 40, torch.float32, seed=18)
    got = call(jf, w, "padded").cpu()
    for i in (0, 1, 63, 64, 2047, 2048, 3333, N - 1):
        want, tol = expected(w, 0, i, -INF, torch.float32)
        assert ref.within(got[0, i], want, tol), i


@pytest.mark.parametrize("V", [50000, 50001])
def test_rows_past_32_bit_offsets(jf, V):
    """More than 2^32 logits, in place: the last sequence's rows are adjusted, what has nothing to adjust stays."""
    N, B = 4096, -(-(1 << 32) // (4096 * V)) + 1
    few = 3                                         # rows of the last sequence that are looked at
    w = make(1, few, V, torch.bfloat16, seed=19)
    x = torch.zeros((B * N, V), dtype=torch.bfloat16, device="cuda")
    x[-few:] = w["logits"][0].cuda()
    cu = [N * b for b in range(B)] + [N * B - few, N * B]
    rows = torch.full((N * B,), -1, dtype=torch.int32, device="cuda")
    rows[-few:] = w["allowed_row"][0].cuda()
    last = lambda k, fill: torch.cat([torch.full((B,) + w[k].shape[1:], fill, dtype=w[k].dtype), w[k]]).cuda()  # noqa: E731
    draft = torch.zeros(N * B, dtype=torch.int32, device="cuda")
    draft[-few:] = w["draft"][0].cuda()
    mask = torch.zeros((N * B, N // 64), dtype=torch.int64, device="cuda")
    mask[-few:, :1] = w["mask"][0].cuda()
    err = new_err()
    jf.adjust_logits(x, count=last("count", 0), draft=draft, mask=mask, bias=last("bias", 0.0), allowed=w["allowed"].cuda(),
                     allowed_row=rows, repetition=last("rep", 1.0), presence=last("pres", 0.0), frequency=last("freq", 0.0),
                     cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), N_max=N, out=x, dev_err=err)
    assert err.item() == 0
    check(w, "padded", x[-few:].view(1, few, V))
    for at in range(0, B * N - few, N):             # (count_nonzero of it all would take an int64 copy)
        assert not x[at:min(at + N, B * N - few)].any()


def test_refused_tensors(jf):
    w = make(1, 4, 64, torch.float32, seed=13)
    x = w["logits"].cuda()
    with pytest.raises(TypeError):
        jf.adjust_logits(x.half())
    with pytest.raises(ValueError):
        jf.adjust_logits(x, bias=torch.zeros(2, 64, device="cuda"))
    with pytest.raises(ValueError):
        jf.adjust_logits(x, allowed=torch.zeros(3, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(jf.JFError):
        jf.adjust_logits(x, draft=torch.zeros(1, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        jf.adjust_logits(x.transpose(1, 2))
    with pytest.raises(jf.JFError):
        jf.adjust_logits(x.to(torch.float32), out=x.view(-1).view(torch.bfloat16)[:256].view(1, 4, 64))


def test_streams_and_graphs(jf):
    w = make(2, 12, 5000, torch.bfloat16, seed=14)
    want = call(jf, w, "padded")
    side = torch.cuda.Stream()
    x, out = w["logits"].cuda(), torch.zeros(w["logits"].shape, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    call(jf, w, "padded", logits=x, out=out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x = torch.zeros_like(want)
    held = {k: cuda(w[k]) for k in ("count", "draft", "mask", "bias", "allowed", "allowed_row")}
    held.update(repetition=w["rep"].cuda(), presence=w["pres"].cuda(), frequency=w["freq"].cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jf.adjust_logits(x, out=out, **held)
    x.copy_(w["logits"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ----------------------------------------------------------------------------- counts

def counted(count, token, path, length, extra, row, prompt, V):
    B, N = token.shape
    src = torch.zeros((B, V), dtype=torch.int32) if count is None else \
        torch.stack([count[int(row[b])] if row is not None else count[b] for b in range(B)])
    out = src.clone()
    for b in range(B):
        n = N if length is None else int(length[b])
        ids = [int(token[b, int(path[b, k])]) for k in range(1, n + 1)] if path is not None else token[b, :n].tolist()
        if extra is not None and int(extra[b]) >= 0:
            ids.append(int(extra[b]))
        for v in ids:
            out[b, v] = int(out[b, v]) | ref.PROMPT if prompt else int(out[b, v]) + 1
    return out


@pytest.mark.parametrize("B,N,V", [(1, 1, 1), (3, 7, 5), (2, 300, 4096), (4, 33, 4099), (2, 1000, 50257), (9, 2, 151936)])
@pytest.mark.parametrize("kind", ["tokens", "lengths", "path", "prompt", "rows", "zeros"])
def test_counts(jf, B, N, V, kind):
    g = torch.Generator().manual_seed(B + N + V)
    rows = B + 2
    count = torch.randint(0, 5, (rows, V), generator=g, dtype=torch.int32)
    count |= (torch.rand((rows, V), generator=g) < 0.1).to(torch.int32) * ref.PROMPT
    token = torch.randint(0, max(1, V // 50), (B, N), generator=g, dtype=torch.int32)
    path = length = extra = row = None
    if kind in ("lengths", "prompt", "zeros"):
        length = torch.randint(0, N + 1, (B,), generator=g, dtype=torch.int32)
        length[0] = 0 if kind == "lengths" else N
    if kind == "path":
        length = torch.randint(0, N, (B,), generator=g, dtype=torch.int32)
        path = torch.full((B, N), -1, dtype=torch.int32)
        for b in range(B):
            path[b, 0] = 0
            path[b, 1:int(length[b]) + 1] = (torch.randperm(N - 1, generator=g)[:int(length[b])] + 1).sort().values.to(torch.int32)
        extra = torch.randint(0, V, (B,), generator=g, dtype=torch.int32)
        extra[B // 2] = -1
    if kind == "rows":
        row = torch.randint(0, rows, (B,), generator=g, dtype=torch.int32)
    src = None if kind == "zeros" else count
    prompt = kind in ("prompt", "zeros")
    want = counted(src, token, path, length, extra, row, prompt, V)
    err = new_err()
    kw = dict(path=cuda(path), length=cuda(length), extra=cuda(extra), row=cuda(row), prompt=prompt, dev_err=err)
    got = jf.count_tokens(cuda(src), token.cuda(), V=V, **kw)
    assert torch.equal(got.cpu(), want) and err.item() == 0
    if kind not in ("rows", "zeros"):               # in place: the rows behind the sequences stay
        held = count.cuda()[:B].clone()
        assert jf.count_tokens(held, token.cuda(), out=held, **kw) is held
        assert torch.equal(held.cpu(), want) and err.item() == 0


def test_counts_past_32_bit_offsets(jf):
    """More than 2^32 entries: a new table from one row, and the last sequence's tokens in place."""
    V = 70001
    B = (1 << 32) // V + 2
    token = torch.full((B, 2), 5, dtype=torch.int32, device="cuda")
    token[-1] = torch.tensor([V - 1, 7], dtype=torch.int32)
    one = torch.zeros((1, V), dtype=torch.int32, device="cuda")
    one[0, 7] = 40
    count = jf.count_tokens(one, token, row=torch.zeros(B, dtype=torch.int32, device="cuda"))
    want = one[0].clone()
    want[5] += 2
    assert torch.equal(count[0], want) and torch.equal(count[-2], want)
    want = one[0].clone()
    want[7] += 1
    want[V - 1] += 1
    assert torch.equal(count[-1], want)
    jf.count_tokens(count, token, out=count)
    want[7] += 1
    want[V - 1] += 1
    assert torch.equal(count[-1], want) and int(count[-2, 5]) == 4


def test_count_reports(jf):
    V, B, N = 100, 4, 6
    token = torch.full((B, N), 3, dtype=torch.int32)
    token[0, 2], token[1, 5] = 100, -1
    for in_place in (False, True):
        count = torch.zeros((B, V), dtype=torch.int32, device="cuda")
        out = count if in_place else None
        err = new_err()
        got = jf.count_tokens(count, token.cuda(), out=out, dev_err=err)
        assert err.item() == jf.DEVERR_BAD_TOKEN and got[:, 3].tolist() == [5, 5, 6, 6]
        count.zero_()
        err = new_err()
        lens = torch.tensor([7, -1, 2, 6], dtype=torch.int32).cuda()
        got = jf.count_tokens(count, torch.full((B, N), 3, dtype=torch.int32).cuda(), length=lens, out=out, dev_err=err)
        assert err.item() == jf.DEVERR_BAD_TREE_LEN and got[:, 3].tolist() == [6, 0, 2, 6]
        count.zero_()
        err = new_err()
        path = torch.tensor([[0, 1, 6, -1, -1, -1], [0, 2, 3, -1, -1, -1], [0, -1, -1, -1, -1, -1], [0, 1, 2, 3, 4, 5]])
        got = jf.count_tokens(count, torch.full((B, N), 3, dtype=torch.int32).cuda(), path=path.to(torch.int32).cuda(),
                              length=torch.tensor([2, 2, -1, 9], dtype=torch.int32).cuda(), out=out, dev_err=err)
        assert err.item() == jf.DEVERR_BAD_PATH and got[:, 3].tolist() == [1, 2, 0, 5]
    err = new_err()
    got = jf.count_tokens(torch.ones((3, V), dtype=torch.int32, device="cuda"), token[2:, :1].cuda(),
                          row=torch.tensor([3, 1], dtype=torch.int32).cuda(), dev_err=err)
    assert err.item() == jf.DEVERR_BAD_PATH and got[0].sum().item() == 1 and got[1].sum().item() == V + 1


def test_counts_on_a_side_stream_and_in_a_graph(jf):
    g = torch.Generator().manual_seed(3)
    count = torch.randint(0, 5, (3, 5000), generator=g, dtype=torch.int32).cuda()
    token = torch.randint(0, 5000, (3, 40), generator=g, dtype=torch.int32).cuda()
    want = jf.count_tokens(count, token)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = jf.count_tokens(count, token, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    held = torch.zeros_like(count)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jf.count_tokens(held, token, out=held)
    held.copy_(count)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, want)
