"""NaN and infinite scores in attention over shared prefixes: a row that sees one has NaN in its output and its
log-sum-exp, wherever the key lies and however the item is cut; every other row is as without it."""
import pytest
import torch

import step_reference as ref
from test_gpu_shared import PAGE, call, jf, make  # noqa: F401  (jf: a fixture)

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

# name, groups, N, Hq, Hkv, D, shared pages, own tokens.  "rows": the kernel of few rows alone, "tiles": that of many
# alone, "pair": both.  Few long items are cut into pieces, many short ones are mostly whole.
CASES = [
    ("rows_cut", [3, 2], 1, 8, 2, 128, [90, 40], [70, 33, 40, 90, 50]),
    ("rows_cut_two_warps", [6, 5], 1, 8, 2, 64, [70, 33], [40 + b for b in range(11)]),
    ("rows_whole", [3] * 500, 1, 4, 2, 64, [2] * 500, [20 + b % 9 for b in range(1500)]),
    ("tiles_cut", [2, 2], 40, 8, 2, 128, [60, 40], [200, 33, 140, 60]),
    ("tiles_cut_one_tile", [2], 36, 4, 2, 64, [50], [130, 40]),
    ("tiles_whole", [2] * 90, 36, 4, 2, 64, [2] * 90, [18 + b % 9 for b in range(180)]),
    ("pair_cut", [20], 2, 16, 2, 128, [60], [30 + 7 * b for b in range(20)]),
    ("pair_whole", [12] * 60, 3, 8, 2, 64, [3] * 60, [17 + b % 13 for b in range(720)]),
]
WHERE = ["shared", "own", "q"]


def hit_rows(w, b, k, v, q):
    """(expected out [n, Hq, D], lse [n, Hq], their tolerances, rows that must be NaN [n, Hq]) of sequence b, in 64 bits."""
    B, N, Hq, Hkv, D = w["shape"]
    G, n = Hq // Hkv, w["sizes"][b]
    L = w["lens"][b] + n
    pages = w["real"][b, :-(-L // PAGE)].long().cuda()
    k, v = (x[pages].flatten(0, 1)[:L].double() for x in (k, v))
    x = q[b, :n].double().view(n, Hkv, G, D)
    hidden = torch.cat([torch.zeros((n, w["lens"][b]), dtype=torch.bool), ~w["sees"][b, :n, :n]], 1).cuda()
    s = torch.einsum("ngqd,tgd->gqnt", x, k) * D ** -0.5
    s = s.masked_fill(hidden, -INF)
    bad = (torch.isnan(s) | (s == INF)).any(-1)                             # [Hkv, G, n]
    size = torch.einsum("ngqd,tgd->gqnt", x.nan_to_num(0, 0, 0).abs(), k.nan_to_num(0, 0, 0).abs()).amax(-1) * D ** -0.5
    s = s.masked_fill(bad[..., None], 0.0)
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[..., None])
    u, half = 2.0 ** -23, ref.half_step(torch.bfloat16)                     # as in test_gpu_shared.check
    off = (D * u * size + (16 + L) * u).permute(2, 0, 1).reshape(n, Hq)
    want = torch.einsum("gqnt,tgd->ngqd", p, v).reshape(n, Hq, D)
    spread = torch.einsum("gqnt,tgd->ngqd", p, v.abs()).reshape(n, Hq, D)
    z = z.permute(2, 0, 1).reshape(n, Hq)
    return (want, spread * (half + 2 * off[..., None]) + half * want.abs(), z, off + 4 * u * (1 + z.abs()),
            bad.permute(2, 0, 1).reshape(n, Hq))


@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("case", range(len(CASES)), ids=[c[0] for c in CASES])
def test_nonfinite_scores(jf, case, value, where):  # noqa: F811
    _, groups, N, Hq, Hkv, D, pages, own = CASES[case]
    w = make(groups, N, Hq, Hkv, D, pages, own, seed=300 + case)
    B = sum(groups)
    u = len(groups) // 2                              # the group, its last sequence, the kv-head, a row that it hits
    b = w["start"][u + 1] - 1
    if where == "q":
        w["q"][b, N // 2, Hq - 1, 3] = value
    else:
        t = 16 * (pages[u] // 2) + 5 if where == "shared" else 16 * pages[u] + own[b] // 2
        w["kc"][int(w["real"][b, t // PAGE]), t % PAGE, Hkv - 1, 3] = value
    out, lse = call(jf, w, "padded")
    k, v, q = w["kc"].cuda(), w["vc"].cuda(), w["q"].cuda()
    seen = 0
    first, last = w["start"][u], w["start"][u + 1]
    for c in sorted({0, B - 1, first, last - 1, max(first - 1, 0), min(last, B - 1)} | set(range(first, last, 3))):
        want, tol, z, ztol, bad = hit_rows(w, c, k, v, q)
        seen += int(bad.sum())
        rows, ls = out[c], lse[c].t()
        assert torch.isnan(rows[bad]).all() and torch.isnan(ls[bad]).all(), c
        assert ref.within(rows[~bad], want[~bad], tol[~bad]) and ref.within(ls[~bad], z[~bad], ztol[~bad]), c
    assert seen > 0
