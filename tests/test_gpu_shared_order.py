"""Attention over shared prefixes right behind the kernels that write its inputs, its kernels one behind the other: every
call of a captured chain sees what the call before it in the stream wrote, and nothing older."""
import pytest
import torch

from test_gpu_shared import call, ints, jf, make  # noqa: F401  (jf: a fixture)

pytestmark = pytest.mark.gpu

# groups, N, shared pages, own tokens: both kernels (the second one's inputs are older than the first one), then
# either alone.
CASES = [([20], 2, [30], [9 * b + 3 for b in range(20)]), ([9, 12], 4, [20, 40], [17 * b % 90 for b in range(21)]),
         ([2, 3], 1, [20, 30], [5, 60, 0, 100, 9]), ([2, 1], 40, [20, 0], [7, 50, 90])]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_inputs_written_just_before(jf, case, captured):  # noqa: F811
    groups, N, pages, own = CASES[case]
    ways = [make(groups, N, 16, 2, 128, pages, own, seed=400 + 10 * case + k) for k in range(3)]
    want = [call(jf, w, "padded") for w in ways]
    # The pools of all three side by side, so that a change of inputs is one of tables, queries and lengths.
    first, at = [], 0
    for w in ways:
        first.append(at)
        at += w["kc"].shape[0]
    kc, vc = (torch.cat([w[x] for w in ways]).cuda() for x in ("kc", "vc"))
    held = [dict(q=w["q"].cuda(), table=torch.where(w["table"] >= 0, w["table"] + f, w["table"]).cuda(), lens=ints(w["lens"]),
                 mask=w["mask"].cuda()) for w, f in zip(ways, first)]
    now = {x: torch.zeros_like(held[0][x]) for x in held[0]}
    start, shared = ints(ways[0]["start"]), ints(pages)
    B, N, Hq, Hkv, D = ways[0]["shape"]
    ws = torch.empty(jf.jf_tree_attention_shared_workspace_size(B, N, len(groups), Hq, Hkv, D, now["table"].shape[1]),
                     dtype=torch.uint8, device="cuda")
    got = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in want]

    def chain():
        for h, (out, lse) in zip(held, got):
            for x in now:
                now[x].copy_(h[x])
            jf.tree_attention_shared(now["q"], kc, vc, now["table"], now["lens"], now["mask"], start, shared, out=out,
                                     lse=lse, workspace=ws)
            for x in now:                              # and what is left behind is of no use to a late reader
                now[x].zero_()

    if captured:
        graph = torch.cuda.CUDAGraph()
        chain()
        with torch.cuda.graph(graph):
            chain()
    for _ in range(20):
        for out, lse in got:
            out.zero_(), lse.zero_()
        graph.replay() if captured else chain()
        torch.cuda.synchronize()
        for (o, l), (x, y) in zip(want, got):
            assert torch.equal(o, x) and torch.equal(l, y)
