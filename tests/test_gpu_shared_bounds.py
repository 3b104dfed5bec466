"""Shared pages right up to the block table's end: ragged and packed trees far smaller than N, tables that end
with the longest sequence, entries of the other rows that must not be read."""
import pytest
import torch

from test_gpu_shared import PAGE, call, check, ints, jf, make, new_err  # noqa: F401  (jf: a fixture)

pytestmark = pytest.mark.gpu


def tight(w):
    """The same sequences under a table that ends with the longest of them."""
    wide = max(-(-(p + n) // PAGE) for p, n in zip(w["lens"], w["sizes"]))
    return dict(w, table=w["table"][:, :wide].contiguous(), real=w["real"][:, :wide].contiguous())


# name, groups, N, Hq, Hkv, D, shared pages, own tokens, nodes.  "rows" runs in the kernel of few rows alone,
# "tiles" in that of many alone, "pair" has shared parts in the one and own parts in the other.
TIGHT = [
    ("rows", [2, 1], 32, 2, 2, 128, [10, 6], [0, 0, 4], [1, 1, 32]),
    ("rows", [4], 16, 4, 4, 64, [6], [4, 0, 3, 9], [4, 4, 4, 4]),
    ("rows", [3, 2], 12, 2, 2, 64, [9, 9], [0, 3, 15, 7, 1], [1, 2, 1, 12, 3]),
    ("tiles", [2, 1], 64, 8, 2, 128, [10, 6], [0, 0, 4], [1, 1, 64]),
    ("tiles", [3, 3], 40, 16, 2, 64, [20, 17], [0, 5, 15, 33, 0, 1], [1, 3, 2, 1, 40, 9]),
    ("pair", [12], 16, 8, 2, 128, [9], [b % 16 for b in range(12)], [1 + b % 4 for b in range(12)]),
    ("pair", [9, 8], 8, 16, 2, 64, [30, 30], [3 * b % 16 for b in range(17)], [1 + b % 3 for b in range(17)]),
]


@pytest.mark.parametrize("layout", ["ragged", "packed"])
@pytest.mark.parametrize("case", range(len(TIGHT)), ids=["%s%d" % (c[0], i) for i, c in enumerate(TIGHT)])
def test_tables_that_end_with_the_longest_sequence(jf, case, layout):  # noqa: F811
    _, groups, N, Hq, Hkv, D, pages, own, sizes = TIGHT[case]
    w = tight(make(groups, N, Hq, Hkv, D, pages, own, seed=200 + case, sizes=sizes))
    err = new_err()
    out, lse = call(jf, w, layout, err)
    assert err.item() == 0
    check(w, layout, out, lse)
    old = w["table"].clone()                       # pages of other sequences in their place: not read either
    w["table"] = torch.where(old < 0, torch.full_like(old, int(w["real"][-1, 0])), old)
    again, lse2 = call(jf, w, layout, err)
    assert err.item() == 0 and torch.equal(out, again) and torch.equal(lse, lse2)


def test_shared_pages_past_what_a_sequence_has(jf):  # noqa: F811
    """Shared pages up to the table's end leave no room for the trees: reported, in bounds, the other group right."""
    for N, Hq in ((2, 4), (40, 16)):
        w = make([3, 2], N, Hq, 2, 64, [4, 2], [5, 6, 7, 8, 9], seed=210)
        cap = w["table"].shape[1]
        for pages in (cap, cap + 1):
            err = new_err()
            out, lse = call(jf, dict(w, pages=[pages, 2]), "padded", err)
            want = jf.DEVERR_BAD_PREFIX | (jf.DEVERR_BAD_GROUP if pages > cap else 0)
            assert err.item() == want, pages
            check(w, "padded", out, lse, only={3, 4})


def test_descending_spans(jf):  # noqa: F811
    """Spans that go back and overlap: nothing is computed, whatever their sum (here several times 2^31 positions)."""
    w = make([2, 2], 4, 4, 1, 64, [4, 2], [20, 6, 30, 8], seed=211)
    B, N, Hq, Hkv, D = w["shape"]
    want, _ = call(jf, w, "packed")
    q, mask = w["q"].flatten(0, 1).cuda(), w["mask"].flatten(0, 1).cuda()
    rest = (w["kc"].cuda(), w["vc"].cuda(), w["table"].cuda(), ints(w["lens"]), mask, ints(w["start"]), ints(w["pages"]))
    for cu in ([0, 4, 8, 4, 8], [4, 0, 4, 8, 12], [0, 4, 8, 12, 11], [0, 16, 0, 16, 0]):
        err = new_err()
        jf.tree_attention_shared(q, *rest, cu_seqlens=ints(cu), N_max=N, dev_err=err)
        assert err.item() == jf.DEVERR_BAD_TREE_LEN, cu
    err = new_err()
    jf.tree_attention_shared(q, *rest[:5], ints([0, 3, 2]), rest[6], cu_seqlens=ints([0, 4, 8, 4, 8]), N_max=N, dev_err=err)
    assert err.item() == jf.DEVERR_BAD_TREE_LEN | jf.DEVERR_BAD_GROUP
    B, T, H, wide = 128, 4096, 128, 8192
    big = torch.zeros((T, H, 64), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((8, PAGE, H, 64), dtype=torch.bfloat16, device="cuda")
    err = new_err()
    jf.tree_attention_shared(big, pool, pool, torch.zeros((B, wide), dtype=torch.int32, device="cuda"),
                             ints([wide * PAGE - T] * B), torch.zeros((T, T // 64), dtype=torch.int64, device="cuda"),
                             ints(list(range(B + 1))), ints([0] * B), cu_seqlens=ints([T * (b % 2) for b in range(B + 1)]),
                             N_max=T, dev_err=err)
    assert err.item() & jf.DEVERR_BAD_TREE_LEN
    err = new_err()
    out = jf.tree_attention_shared(q, *rest, cu_seqlens=ints(list(range(0, 17, 4))), N_max=N, dev_err=err)
    assert err.item() == 0 and torch.equal(out, want)


def test_wide_tables(jf):  # noqa: F811
    """Tables of 2^20 pages: the positions that they could take fit in the schedule, and the results do not change."""
    w = make([40, 24], 16, 32, 8, 64, [9, 20], [b % 40 for b in range(64)], seed=212)
    out, lse = call(jf, w, "padded")
    table = torch.full((64, 1 << 20), -9, dtype=torch.int32)
    table[:, :w["table"].shape[1]] = w["table"]
    err = new_err()
    far, far_lse = call(jf, dict(w, table=table), "padded", err)
    assert err.item() == 0 and torch.equal(out, far) and torch.equal(lse, far_lse)
    check(w, "padded", out, lse, only={0, 39, 40, 63})


@pytest.mark.parametrize("groups,N,Hq,Hkv,D,pages,own,sizes", [
    ([6, 3], 1, 8, 2, 128, [2, 1], [3, 0, 15, 7, 1, 2, 4, 0, 9], [1] * 9),       # single tokens, three pages at most
    ([2, 2], 9, 8, 2, 64, [1, 0], [0, 1, 5, 0], [3, 9, 2, 1]),
    ([3, 1], 30, 4, 1, 64, [12, 3], [2, 9, 0, 1], [30, 4, 17, 22]),
    ([2, 3], 70, 16, 2, 128, [20, 9], [0, 5, 15, 33, 0], [70, 3, 2, 1, 40]),
])
def test_packed_rows_without_n_max(jf, groups, N, Hq, Hkv, D, pages, own, sizes):  # noqa: F811
    w = tight(make(groups, N, Hq, Hkv, D, pages, own, seed=213, sizes=sizes))
    q, mask = (torch.cat([x[b, :n] for b, n in enumerate(sizes)]).cuda() for x in (w["q"], w["mask"]))
    cu = [0]
    for n in sizes:
        cu.append(cu[-1] + n)
    err = new_err()
    out, lse = jf.tree_attention_shared(q, w["kc"].cuda(), w["vc"].cuda(), w["table"].cuda(), ints(w["lens"]), mask,
                                        ints(w["start"]), ints(pages), with_lse=True, cu_seqlens=ints(cu), dev_err=err)
    assert err.item() == 0
    check(w, "packed", out, lse)


@pytest.mark.parametrize("groups,N", [([3, 2], 2), ([200, 300], 3), ([3, 2], 40)])
def test_old_descriptors_in_the_workspace(jf, groups, N):  # noqa: F811
    """A call that computes nothing leaves the merge what the workspace held, here lists of a million pieces and more than
    the workspace has rows: no row is merged from them."""
    B = sum(groups)
    w = make(groups, N, 8, 1, 64, [4, 2], [5 + b % 9 for b in range(B)], seed=214)
    size = jf.jf_tree_attention_shared_workspace_size(B, N, 2, 8, 1, 64, w["table"].shape[1])
    rows = size // (65 * 4)
    for n in (rows // 2, 20000, 10 ** 6):
        ws = torch.zeros(size // 16 + 1, 4, dtype=torch.int32, device="cuda")
        ws[:, 0], ws[:, 1] = 3, n
        out = torch.full(w["q"].shape, -7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, 8, N), -7.0, device="cuda")
        err = new_err()
        call(jf, dict(w, start=[0, 3, 2]), "padded", err, workspace=ws.view(torch.uint8).flatten(), out=out, lse=lse)
        assert err.item() == jf.DEVERR_BAD_GROUP
        assert (out == -7.0).all() and (lse == -7.0).all()
