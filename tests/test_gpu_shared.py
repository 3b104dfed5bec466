"""jf_tree_attention_shared and its packed form against attention in 64 bits over each sequence's whole
context, one sequence at a time: group and row-tile boundaries, shared prefixes from none to all of
the context, ragged and packed trees, hostile padding, malformed groups, streams and graphs."""
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


def new_err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def make(groups, N, Hq, Hkv, D, pages, own, seed, sizes=None, scale_q=1.0):
    """groups: sequences of each; pages: shared pages of each; own: cached tokens of each sequence's own
    behind the shared ones.  Slots and table entries that must not be read hold NaN and -9."""
    g = torch.Generator().manual_seed(seed)
    B = sum(groups)
    start = [0]
    for n in groups:
        start.append(start[-1] + n)
    sizes = sizes or [N] * B
    of = [u for u, n in enumerate(groups) for _ in range(n)]
    alone = [groups[of[b]] < 2 for b in range(B)]
    lens = [PAGE * pages[of[b]] + own[b] for b in range(B)]
    need = [-(-(lens[b] + sizes[b]) // PAGE) for b in range(B)]
    total = sum(pages[u] for u in range(len(groups))) + sum(need)
    order = torch.randperm(total, generator=g).to(torch.int32)
    cap = -(-(max(lens) + N) // PAGE)
    table = torch.full((B, cap), -9, dtype=torch.int32)
    kc = torch.full((total, PAGE, Hkv, D), float("nan"), dtype=torch.bfloat16)
    vc = torch.full((total, PAGE, Hkv, D), float("nan"), dtype=torch.bfloat16)
    real = torch.full((B, cap), -1, dtype=torch.int32)
    at = 0
    for u, n in enumerate(groups):
        mine = order[at:at + pages[u]]
        at += pages[u]
        for b in range(start[u], start[u + 1]):
            more = need[b] - pages[u]
            real[b, :pages[u]] = mine
            real[b, pages[u]:need[b]] = order[at:at + more]
            at += more
            table[b, pages[u]:need[b]] = real[b, pages[u]:need[b]]
            if b == start[u] or alone[b]:
                table[b, :pages[u]] = mine           # the shared pages: in the first row only
    for b in range(B):
        t = torch.arange(lens[b] + sizes[b])
        where = real[b][t // PAGE].long(), t % PAGE
        kc[where] = torch.randn((len(t), Hkv, D), generator=g).to(torch.bfloat16)
        vc[where] = torch.randn((len(t), Hkv, D), generator=g).to(torch.bfloat16)
    _, sees = ref.random_trees(B, N, g)
    q = (scale_q * torch.randn((B, N, Hq, D), generator=g)).to(torch.bfloat16)
    return dict(q=q, kc=kc, vc=vc, table=table, real=real, lens=lens, sizes=sizes, sees=sees, mask=ref.pack_bits(sees),
                start=start, pages=pages, shape=(B, N, Hq, Hkv, D))


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def call(jf, w, layout, err=None, workspace=None, stream=None, out=None, lse=None):
    B, N, Hq, Hkv, D = w["shape"]
    q, mask, extra = w["q"], w["mask"], {}
    if layout == "packed":
        q, mask = (torch.cat([x[b, :n] for b, n in enumerate(w["sizes"])]) for x in (q, mask))
        cu = [0]
        for n in w["sizes"]:
            cu.append(cu[-1] + n)
        extra = dict(cu_seqlens=ints(cu), N_max=N)
    elif layout == "ragged":
        extra = dict(tree_len=ints(w["sizes"]))
    if out is None:
        out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((Hq, q.shape[0]) if layout == "packed" else (B, Hq, N), -7.0, device="cuda")
    if workspace is None:                             # nothing may depend on what it held
        size = jf.jf_tree_attention_shared_workspace_size(B, N, len(w["pages"]), Hq, Hkv, D, w["table"].shape[1],
                                                          q.shape[0] if layout == "packed" else 0)
        workspace = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    jf.tree_attention_shared(q.cuda(), w["kc"].cuda(), w["vc"].cuda(), w["table"].cuda(), ints(w["lens"]), mask.cuda(),
                             ints(w["start"]), ints(w["pages"]), out=out, lse=lse, workspace=workspace, dev_err=err,
                             stream=stream, **extra)
    return out, lse


def check(w, layout, out, lse, only=None):
    """u = 2^-23 covers one fp32 operation (rounded or truncated).  A score is off by D u sum |q_d k_d| scale, its
    exponential relatively by that, 8 u and the merge's weights (8 u); probabilities reach the value product
    rounded to bf16 (half a step of the value), their sums add L u; the output is rounded to bf16 once."""
    B, N, Hq, Hkv, D = w["shape"]
    u, half, G = 2.0 ** -23, ref.half_step(torch.bfloat16), Hq // Hkv
    first = 0
    for b, n in enumerate(w["sizes"]):
        L = w["lens"][b] + n
        rows = out[first:first + n] if layout == "packed" else out[b, :n]
        ls = lse[:, first:first + n].t() if layout == "packed" else lse[b, :, :n].t()
        first += n
        if layout == "ragged":
            assert (out[b, n:] == -7.0).all() and (lse[b, :, n:] == -7.0).all()
        if only is not None and b not in only:
            continue
        pages = w["real"][b, :-(-L // PAGE)].long()
        k, v = (x[pages].flatten(0, 1)[:L].double().cuda() for x in (w["kc"], w["vc"]))
        q = w["q"][b, :n].double().cuda().view(n, Hkv, G, D)
        hidden = torch.cat([torch.zeros((n, w["lens"][b]), dtype=torch.bool), ~w["sees"][b, :n, :n]], 1).cuda()
        s = torch.einsum("ngqd,tgd->gqnt", q, k) * D ** -0.5
        size = torch.einsum("ngqd,tgd->gqnt", q.abs(), k.abs()).amax(-1, keepdim=True) * D ** -0.5
        s = s.masked_fill(hidden, -float("inf"))
        z = torch.logsumexp(s, -1, keepdim=True)
        p = torch.exp(s - z)
        want = torch.einsum("gqnt,tgd->ngqd", p, v).reshape(n, Hq, D)
        spread = torch.einsum("gqnt,tgd->ngqd", p, v.abs()).reshape(n, Hq, D)
        off = (D * u * size + (16 + L) * u).permute(2, 0, 1, 3).reshape(n, Hq, 1)
        assert ref.within(rows, want, spread * (half + 2 * off) + half * want.abs()), b
        z = z.permute(2, 0, 1, 3).reshape(n, Hq)
        assert ref.within(ls, z, off[..., 0] + 4 * u * (1 + z.abs())), b


CASES = [
    # groups, N, Hq, Hkv, D, shared pages, own tokens
    ([1], 1, 4, 1, 64, [3], [5]),
    ([2], 1, 1, 1, 64, [1], [0, 0]),                       # fewer than 128 keys, no token of their own
    ([4], 1, 32, 8, 128, [8], [0, 7, 15, 16]),             # P = S, P = S + 16
    ([3, 1, 2], 1, 8, 2, 128, [9, 4, 0], [3, 200, 17, 40, 0, 300]),
    ([5, 3], 1, 16, 16, 64, [40, 17], [1, 2, 3, 4, 5, 6, 7, 8]),
    ([2, 2], 1, 128, 1, 128, [20, 3], [100, 0, 31, 129]),  # 128 query heads of one kv-head
    ([33], 1, 8, 2, 128, [16], list(range(33))),           # 132 rows: one more row tile than 128
    ([65], 1, 16, 4, 64, [24], [b % 50 for b in range(65)]),   # 260 rows
    ([3], 17, 8, 2, 128, [12], [0, 130, 5]),
    ([2, 3], 40, 8, 1, 64, [7, 30], [9, 0, 500, 64, 128]),
    ([2], 70, 4, 4, 128, [5], [33, 0]),                    # two mask words
    ([1, 1, 1], 5, 8, 8, 64, [2, 0, 9], [0, 0, 3]),        # nothing to share
    ([4, 4], 3, 64, 4, 128, [70, 130], [10, 200, 0, 1, 600, 5, 90, 1000]),
]


@pytest.mark.parametrize("layout", ["padded", "ragged", "packed"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_parts_and_groups(jf, case, layout):
    groups, N, Hq, Hkv, D, pages, own = CASES[case]
    B = sum(groups)
    sizes = None if layout == "padded" else [1 + (N - 1) * ((3 * b + 1) % B + 1) // B for b in range(B)]
    w = make(groups, N, Hq, Hkv, D, pages, own, seed=case, sizes=sizes)
    err = new_err()
    out, lse = call(jf, w, layout, err)
    assert err.item() == 0
    check(w, layout, out, lse)
    again, lse2 = call(jf, w, layout, err)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


MORE = [
    # groups, N, Hq, Hkv, D, shared pages, own tokens: 24 and 48 rows a group, 80 with 8 of a sequence's own
    ([6], 1, 8, 2, 128, [21], [3, 0, 40, 17, 16, 100]),
    ([7, 5], 1, 16, 4, 64, [9, 33], list(range(0, 120, 10))),
    ([3, 3], 4, 8, 2, 128, [10, 3], [5, 0, 61, 200, 33, 2]),
    ([2, 4], 4, 16, 4, 64, [40, 20], [15, 16, 17, 31, 32, 33]),
    ([10], 2, 8, 2, 128, [15], [7 * b for b in range(10)]),
    ([11, 9], 2, 4, 1, 64, [50, 4], [9 * b for b in range(20)]),
    ([20], 1, 16, 2, 128, [37], [50 * b for b in range(20)]),
]


@pytest.mark.parametrize("layout", ["padded", "packed"])
@pytest.mark.parametrize("case", range(len(MORE)))
def test_rows_between(jf, case, layout):
    groups, N, Hq, Hkv, D, pages, own = MORE[case]
    w = make(groups, N, Hq, Hkv, D, pages, own, seed=100 + case)
    err = new_err()
    out, lse = call(jf, w, layout, err)
    assert err.item() == 0
    check(w, layout, out, lse)


@pytest.mark.parametrize("groups,N,pages", [([2, 1], 5, [0, 0]), ([2, 2], 40, [0, 0]), ([40], 1, [0])])
def test_rows_that_see_nothing(jf, groups, N, pages):
    """An empty context and a mask without bits: zeros and -inf; rows beside them are as always."""
    B = sum(groups)
    w = make(groups, N, 8, 2, 64, pages, [0] * B, seed=60)
    w["sees"][0, 0] = False
    w["sees"][B - 1, N // 2] = False
    w["mask"] = ref.pack_bits(w["sees"])
    out, lse = call(jf, w, "padded")
    for b, i in ((0, 0), (B - 1, N // 2)):
        assert (out[b, i] == 0).all() and (lse[b, :, i] == -float("inf")).all()
    keep = torch.ones((B, N), dtype=torch.bool)
    keep[0, 0] = keep[B - 1, N // 2] = False
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse.transpose(1, 2)[keep.cuda()]).all()
    check(w, "padded", out, lse, only={b for b in range(B) if keep[b].all()})


def test_packed_rows_behind_the_last_sequence(jf):
    w = make([3, 2], 6, 8, 2, 128, [9, 3], [4, 0, 70, 16, 8], seed=61)
    B, N, Hq, Hkv, D = w["shape"]
    q = torch.cat([w["q"].flatten(0, 1), torch.full((7, Hq, D), float("nan"), dtype=torch.bfloat16)]).cuda()
    mask = torch.cat([w["mask"].flatten(0, 1), torch.zeros((7, 1), dtype=torch.int64)]).cuda()
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, B * N + 7), -7.0, device="cuda")
    jf.tree_attention_shared(q, w["kc"].cuda(), w["vc"].cuda(), w["table"].cuda(), ints(w["lens"]), mask, ints(w["start"]),
                             ints(w["pages"]), cu_seqlens=ints(list(range(0, B * N + 1, N))), N_max=N, out=out, lse=lse)
    assert (out[B * N:] == -7.0).all() and (lse[:, B * N:] == -7.0).all()
    check(w, "packed", out[:B * N], lse[:, :B * N])


@pytest.mark.parametrize("scale_q", [1e-3, 12.0])
def test_flat_and_peaked_rows(jf, scale_q):
    """Parts whose log-sum-exps lie far apart, and the rescale of a risen maximum."""
    w = make([3, 2], 2, 8, 2, 128, [20, 9], [0, 300, 40, 700, 1], seed=50, scale_q=scale_q)
    out, lse = call(jf, w, "padded")
    check(w, "padded", out, lse)


def test_long_prefixes(jf):
    w = make([6, 2], 1, 8, 1, 128, [2048, 1500], [5, 900, 0, 16, 33, 64, 2000, 1], seed=51)
    out, lse = call(jf, w, "padded")
    check(w, "padded", out, lse)


def test_many_sequences(jf):
    groups = [1 + 7 * u % 13 for u in range(150)]
    B = sum(groups)
    w = make(groups, 1, 4, 1, 64, [u % 5 for u in range(150)], [b % 23 for b in range(B)], seed=52)
    for layout in ("padded", "packed"):
        out, lse = call(jf, w, layout)
        check(w, layout, out, lse, only=set(range(0, B, 7)))


@pytest.mark.parametrize("groups", [[1] * 4096, [4096], [4] * 1024])
def test_as_many_sequences_as_there_may_be(jf, groups):
    w = make(groups, 1, 2, 1, 64, [2] * len(groups), [b % 19 for b in range(4096)], seed=61)
    for layout in ("padded", "packed"):
        out, lse = call(jf, w, layout)
        check(w, layout, out, lse, only={0, 1, 2, 1023, 1024, 2047, 3000, 4094, 4095})


@pytest.mark.parametrize("N,groups", [(1030, [2]), (4096, [1, 2])])
def test_large_trees(jf, N, groups):
    B = sum(groups)
    w = make(groups, N, 2, 1, 64, [3] * len(groups), [5, 0, 40][:B], seed=62, sizes=[N, 1, N - 3][:B])
    for layout in ("ragged", "packed"):
        out, lse = call(jf, w, layout)
        check(w, layout, out, lse)


@pytest.mark.parametrize("groups,N", [([3, 2], 1), ([4], 20)])
def test_pool_past_32_bit_offsets(jf, groups, N):
    """The pages that are read lie at the end of a pool of more than 2^32 elements."""
    w = make(groups, N, 16, 8, 128, [6] * len(groups), [3 + 30 * b for b in range(sum(groups))], seed=63)
    out, lse = call(jf, w, "padded")
    few = w["kc"].shape[0]
    first = (1 << 32) // (PAGE * 8 * 128) + 3
    pools = []
    for x in (w["kc"], w["vc"]):
        pool = torch.zeros((first + few, PAGE, 8, 128), dtype=torch.bfloat16, device="cuda")
        pool[first:] = x.cuda()
        pools.append(pool)
    B, N, Hq, Hkv, D = w["shape"]
    table = torch.where(w["table"] >= 0, w["table"] + first, w["table"]).cuda()
    err = new_err()
    far, far_lse = jf.tree_attention_shared(w["q"].cuda(), *pools, table, ints(w["lens"]), w["mask"].cuda(), ints(w["start"]),
                                            ints(w["pages"]), with_lse=True, dev_err=err)
    assert torch.equal(far, out) and torch.equal(far_lse, lse) and err.item() == 0
    check(w, "padded", out, lse)


def test_agrees_with_the_unshared_call(jf):
    w = make([4, 3], 9, 8, 2, 128, [30, 11], [0, 5, 77, 16, 300, 2, 1], seed=53)
    out, lse = call(jf, w, "padded")
    table = w["real"].cuda()
    kc, vc = w["kc"].cuda(), w["vc"].cuda()
    want, wl = jf.tree_attention(w["q"].cuda(), kc, vc, table, ints(w["lens"]), w["mask"].cuda(), with_lse=True)
    # two bf16 roundings of values within the probabilities' rounding of each other
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()
    assert (lse - wl).abs().max() <= 1e-4


def test_malformed_groups_stay_in_bounds(jf):
    w = make([3, 2], 2, 4, 1, 64, [4, 2], [5, 6, 7, 8, 9], seed=54)
    for start in ([0, 3, 4], [1, 3, 5], [0, 4, 3], [0, 6, 5], [-2, 3, 5], [0, 3, 9]):
        bad = dict(w, start=start)
        err = new_err()
        out, lse = call(jf, bad, "padded", err)
        assert err.item() == jf.DEVERR_BAD_GROUP, start
        assert torch.isfinite(out.float()).all()
    for pages in ([-1, 2], [1000, 2], [2 ** 30, 2]):
        err = new_err()
        call(jf, dict(w, pages=pages), "padded", err)
        assert err.item() & jf.DEVERR_BAD_GROUP
    err = new_err()                                    # a sequence shorter than what it shares
    lens = list(w["lens"])
    lens[1] = 60
    out, lse = call(jf, dict(w, lens=lens), "padded", err)
    assert err.item() & jf.DEVERR_BAD_PREFIX
    keep = [0, 2, 3, 4]
    check(dict(w, lens=w["lens"]), "padded", out, lse, only=set(keep))


def test_bad_pages_and_lengths(jf):
    w = make([2, 2], 2, 4, 1, 64, [4, 2], [20, 6, 30, 8], seed=55)
    pool = w["kc"].shape[0]
    for where, value in (((0, 1), -1), ((0, 2), pool), ((2, 0), 2 ** 31 - 1), ((1, 4), -5), ((3, 2), pool + 7)):
        table = w["table"].clone()
        table[where] = value
        err = new_err()
        out, lse = call(jf, dict(w, table=table), "padded", err)
        assert err.item() == jf.DEVERR_BAD_PAGE, where
        others = {2, 3} if where[0] < 2 else {0, 1}
        check(w, "padded", out, lse, only=others)
    for b, P in ((0, -3), (3, 10 ** 6)):
        lens = list(w["lens"])
        lens[b] = P
        err = new_err()
        out, lse = call(jf, dict(w, lens=lens), "padded", err)
        assert err.item() & jf.DEVERR_BAD_PREFIX
        check(w, "padded", out, lse, only={0, 1, 2, 3} - {b})


def test_bad_spans(jf):
    w = make([2, 2], 4, 4, 1, 64, [4, 2], [20, 6, 30, 8], seed=56)
    B, N, Hq, Hkv, D = w["shape"]
    q, mask = w["q"].flatten(0, 1).cuda(), w["mask"].flatten(0, 1).cuda()
    for cu in ([0, 4, 4, 12, 16], [0, 9, 8, 12, 16], [0, 4, 8, 12, 17], [-1, 3, 8, 12, 16], [16, 12, 8, 4, 0]):
        err = new_err()
        out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
        jf.tree_attention_shared(q, w["kc"].nan_to_num().cuda(), w["vc"].nan_to_num().cuda(),
                                 w["real"].clamp(min=0).cuda(), ints(w["lens"]), mask, ints(w["start"]),
                                 ints(w["pages"]), cu_seqlens=ints(cu), N_max=N, out=out, dev_err=err)
        assert err.item() & jf.DEVERR_BAD_TREE_LEN, cu
    err = new_err()
    bad = dict(w, sizes=[0, 5, 3, 4])
    out = torch.full(w["q"].shape, -7.0, dtype=torch.bfloat16, device="cuda")
    jf.tree_attention_shared(w["q"].cuda(), w["kc"].cuda(), w["vc"].cuda(), w["real"].cuda(), ints(w["lens"]),
                             w["mask"].cuda(), ints(w["start"]), ints(w["pages"]), tree_len=ints(bad["sizes"]), out=out,
                             dev_err=err)
    assert err.item() == jf.DEVERR_BAD_TREE_LEN and (out[2, 3:] == -7.0).all() and (out[0, 1:] == -7.0).all()


def test_refused(jf):
    w = make([2], 1, 4, 1, 64, [2], [3, 4], seed=57)
    with pytest.raises(jf.JFError) as e:
        call(jf, w, "padded", workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(ValueError):
        call(jf, dict(w, start=[0, 1, 2]), "padded")
    with pytest.raises(jf.JFError):
        jf.jf_tree_attention_shared_workspace_size(5000, 1, 1, 4, 1, 64, 10)
    q = w["q"].cuda()
    with pytest.raises(jf.JFError):                    # q read by other tiles' CTAs: not in place
        call(jf, w, "padded", out=q, lse=torch.empty(2, 4, 1, device="cuda"))
        jf.tree_attention_shared(q, w["kc"].cuda(), w["vc"].cuda(), w["real"].cuda(), ints(w["lens"]), w["mask"].cuda(),
                                 ints(w["start"]), ints(w["pages"]), out=q)


@pytest.mark.parametrize("groups,N,own", [([3], 2, [3, 4, 500]), ([20], 1, [9 * b + 3 for b in range(20)]),
                                          ([2, 3], 20, [2, 30, 4, 90, 6])])
def test_streams_graphs_and_workspaces(jf, groups, N, own):
    """Calls of one kernel, of two side by side, and of the one for many rows."""
    Hq, pages = 16, [20] * len(groups)
    a = make(groups, N, Hq, 2, 128, pages, own, seed=58)
    b = make([2, 2], 1, 8, 2, 128, [9, 30], [0, 44, 10, 2], seed=59)
    want = [call(jf, w, "padded") for w in (a, b)]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for w, s in zip((a, b), sides):                    # two calls at once, a workspace each
        got.append(call(jf, w, "padded", stream=s, out=torch.empty_like(want[len(got)][0]),
                        lse=torch.empty_like(want[len(got)][1])))
    torch.cuda.synchronize()
    for (o, l), (x, y) in zip(want, got):
        assert torch.equal(o, x) and torch.equal(l, y)
    held = dict(k=a["kc"].cuda(), v=a["vc"].cuda(), t=a["table"].cuda(), n=ints(a["lens"]), m=a["mask"].cuda(),
                g=ints(a["start"]), p=ints(a["pages"]))
    q, out, lse = torch.zeros(a["q"].shape, dtype=torch.bfloat16, device="cuda"), torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    ws = torch.empty(jf.jf_tree_attention_shared_workspace_size(sum(groups), N, len(groups), Hq, 2, 128, a["table"].shape[1]),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jf.tree_attention_shared(q, held["k"], held["v"], held["t"], held["n"], held["m"], held["g"], held["p"], out=out,
                                 lse=lse, workspace=ws)
    q.copy_(a["q"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1])
    held["n"].copy_(ints([n - 2 for n in a["lens"]][:1] + a["lens"][1:]))    # lengths are data: the graph follows them
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out[0], want[0][0][0])
