"""The calls around a step as a decoding loop runs them: rotation and append, attention over a shared
prefix, adjusted logits, verification or beam selection, compaction or fork, counts; nothing returns
to the host between them.

Speculation: samples of two prompts, each prompt's pages shared, ragged trees.  One step is captured
into a graph and replayed with new inputs; after each replay the CPU redoes the step from the state the
GPU started it with (rotation, attention and logits in 64 bits within their bounds, walk, compaction
and counts exactly).

Beams: every beam's cache and counts go through the forks; the CPU keeps every beam's whole token history
and recounts it."""
import numpy as np
import pytest
import torch

import oracle
import step_reference as ref

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module")
def jf():
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf as mod
    return mod


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def attended(q, k, v, L, hidden, G, scale):
    """Rows q [n, Hq, D] over keys k, v [L, Hkv, D] in 64 bits, and the bound of test_gpu_shared.py."""
    u, half, D = 2.0 ** -23, ref.half_step(torch.bfloat16), q.shape[-1]
    k, v = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    s = torch.einsum("nhd,thd->hnt", q.double(), k) * scale
    size = torch.einsum("nhd,thd->hnt", q.double().abs(), k.abs()).amax(-1) * scale
    p = torch.softmax(s.masked_fill(hidden, -float("inf")), -1)
    want = torch.einsum("hnt,thd->nhd", p, v)
    off = (D * u * size + (16 + L) * u).t()[..., None]
    return want, torch.einsum("hnt,thd->nhd", p, v.abs()) * (half + 2 * off) + half * want.abs()


@pytest.mark.parametrize("inter,norm,D", [(False, True, 128), (True, False, 64)])
def test_speculation_over_shared_prompts(jf, inter, norm, D):
    B, N, Hkv, G, V, steps, R = 5, 20, 2, 4, 700, 5, 64
    Hq = Hkv * G
    gen = torch.Generator().manual_seed(D)
    start, pages = [0, 3, 5], [6, 2]                # three and two samples of two prompts
    P0 = [6 * PAGE] * 3 + [2 * PAGE] * 2
    more = -(-((steps + 1) * N) // PAGE) + 1        # pages of a sequence's own
    total = sum(pages) + B * more
    order = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.zeros((B, max(pages) + more), dtype=torch.int32)
    at = 0
    for u in range(2):
        table[start[u]:start[u + 1], :pages[u]] = order[at:at + pages[u]]
        at += pages[u]
        for b in range(start[u], start[u + 1]):
            table[b, pages[u]:pages[u] + more] = order[at:at + more]
            at += more
    freq, rs = jf.rotary_frequencies(R, base=10000.0, scaling=("yarn", 4.0, 2048))
    wq, wk = ((torch.randn(D, generator=gen) * 0.2 + 1).to(torch.bfloat16) if norm else None for _ in range(2))
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)  # noqa: E731
    kc, vc = bf(total, PAGE, Hkv, D).cuda(), bf(total, PAGE, Hkv, D).cuda()
    prompt = torch.randint(0, V, (B, 40), generator=gen, dtype=torch.int32)
    count = jf.count_tokens(None, prompt.cuda(), prompt=True, V=V)
    rep, pres, fr = torch.full((B,), 1.3), torch.full((B,), 0.4), torch.linspace(0.0, 0.3, B)
    held = dict(qkv=torch.zeros((B, N, Hq + 2 * Hkv, D), dtype=torch.bfloat16), logits=torch.zeros((B, N, V)),
                parent=torch.zeros((B, N), dtype=torch.int32), draft=torch.zeros((B, N), dtype=torch.int32),
                allowed=torch.zeros((B * N, -(-V // 32)), dtype=torch.int32), row=torch.zeros((B, N), dtype=torch.int32),
                tl=torch.ones(B, dtype=torch.int32), P=torch.tensor(P0, dtype=torch.int32))
    held = {k: t.cuda() for k, t in held.items()}
    out = torch.zeros((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
    qr = torch.zeros_like(out)
    adj = torch.zeros((B, N, V), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fixed = dict(gs=ints(start), sp=ints(pages), table=table.cuda(), rep=rep.cuda(), pres=pres.cuda(), fr=fr.cuda(),
                 wq=None if wq is None else wq.cuda(), wk=None if wk is None else wk.cuda())
    result = {}

    def step():
        h, f = held, fixed
        mask, _, pos = jf.build_tree_mask(h["parent"], h["P"], dev_err=err, tree_len=h["tl"])
        q, k, v = h["qkv"].split([Hq, Hkv, Hkv], dim=2)
        jf.rotate_append_kv(q, k, v, kc, vc, f["table"], h["P"], pos=pos, freq=freq, interleaved=inter, rotary_scale=rs,
                            q_norm=f["wq"], k_norm=f["wk"], tree_len=h["tl"], out=qr, dev_err=err)
        jf.tree_attention_shared(qr, kc, vc, f["table"], h["P"], mask, f["gs"], f["sp"], tree_len=h["tl"], out=out,
                                 dev_err=err)
        jf.adjust_logits(h["logits"], count=count, draft=h["draft"], mask=mask, allowed=h["allowed"],
                         allowed_row=h["row"], repetition=f["rep"], presence=f["pres"], frequency=f["fr"],
                         tree_len=h["tl"], out=adj, dev_err=err)
        am, acc, path, bonus = jf.tree_verify(adj, h["draft"], h["parent"], dev_err=err, tree_len=h["tl"])
        newp = jf.compact_accepted_kv(kc, vc, f["table"], h["P"], path, acc, dev_err=err)
        jf.count_tokens(count, h["draft"], path=path, length=acc, extra=bonus, out=count, dev_err=err)
        result.update(pos=pos, acc=acc, path=path, bonus=bonus, newp=newp)

    graph = torch.cuda.CUDAGraph()
    accepted = 0
    for s in range(steps):
        tl = torch.randint(1, N + 1, (B,), generator=gen, dtype=torch.int32)
        parent, sees = ref.random_trees(B, N, gen, back=3)
        draft = torch.randint(0, V, (B, N), generator=gen, dtype=torch.int32)
        logits = torch.randn((B, N, V), generator=gen)
        allowed = torch.randint(-2 ** 31, 2 ** 31, (B * N, -(-V // 32)), generator=gen).to(torch.int32)
        row = torch.arange(B * N, dtype=torch.int32).view(B, N)
        row[1::2] = -1
        for b in range(B):                          # most drafted tokens are what the target would say
            for c in range(1, int(tl[b])):
                v = int(draft[b, c])
                allowed[b * N + int(parent[b, c]), v // 32] |= torch.tensor(1 << (v % 32)).to(torch.int32)
                if torch.rand(1, generator=gen) < 0.7:
                    logits[b, int(parent[b, c]), v] = 12.0 + float(torch.rand(1, generator=gen))
        new = dict(qkv=bf(B, N, Hq + 2 * Hkv, D), logits=logits, parent=parent, draft=draft, allowed=allowed, row=row, tl=tl)
        before = dict(k=kc.cpu(), v=vc.cpu(), count=count.cpu(), P=held["P"].cpu())
        for k, t in new.items():
            held[k].copy_(t)
        if s == 0:
            step()                                  # kernels are set up before the capture
            torch.cuda.synchronize()
            kc.copy_(before["k"])
            vc.copy_(before["v"])
            count.copy_(before["count"])
            with torch.cuda.graph(graph):
                step()
        graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0
        # ---- the CPU's step, from the same state
        P, got = before["P"], {k: t.cpu() for k, t in result.items()}
        k_now, v_now = before["k"].clone(), before["v"].clone()
        for b in range(B):
            n, p = int(tl[b]), int(P[b])
            depth = sees[b, :n, :n].sum(-1) - 1
            assert (got["pos"][b, :n] == p + depth).all()
            x = new["qkv"][b, :n]
            want, tol = ref.rotate(x[:, :Hq], p + depth, freq.cpu(), inter, rs, wq, 1e-6)
            assert ref.within(qr[b, :n].cpu(), want, tol), (s, b)
            # the step's K as the GPU rounded it: nodes of the accepted path have moved, the others not
            want, tol = ref.rotate(x[:, Hq:Hq + Hkv], p + depth, freq.cpu(), inter, rs, wk, 1e-6)
            acc, path = int(got["acc"][b]), got["path"][b]
            lies = torch.arange(n)
            lies_at = {int(path[j]): j for j in range(acc + 1)}
            slot = lambda t: (int(table[b, (p + t) // PAGE]), (p + t) % PAGE)  # noqa: E731
            k_own, v_own = torch.empty((n, Hkv, D), dtype=torch.bfloat16), x[:, Hq + Hkv:]
            for i in range(n):
                t = lies_at.get(i, i if i > acc else None)
                k_own[i] = kc[slot(t)].cpu() if t is not None else want[i].to(torch.bfloat16)
                if t is not None:
                    assert ref.within(k_own[i], want[i], tol[i]) and torch.equal(vc[slot(t)].cpu(), v_own[i]), (s, b, i)
            for i in lies:                          # what the pool held before compaction
                k_now[slot(int(i))], v_now[slot(int(i))] = k_own[i], v_own[i]
            pages_b = table[b, :-(-(p + n) // PAGE)].long()
            known = torch.tensor([lies_at.get(i, i if i > acc else None) is not None for i in range(n)])
            rows = [i for i in range(n) if known[sees[b, i, :n]].all()]     # rows whose branch's K is known to the bit
            hidden = torch.cat([torch.zeros((n, p), dtype=torch.bool), ~sees[b, :n, :n]], 1)
            keys, vals = (c[pages_b].flatten(0, 1)[:p + n] for c in (k_now, v_now))
            want, tol = attended(qr[b, :n].cpu(), keys, vals, p + n, hidden, G, D ** -0.5)
            assert len(rows) > 0 and ref.within(out[b, rows].cpu(), want[rows], tol[rows]), (s, b)
            for i in range(n):
                had = before["count"][b].long() % ref.PROMPT
                for j in range(1, n):
                    if sees[b, i, j]:
                        had[int(draft[b, j])] += 1
                ok = ref.unpack(allowed[b * N + i], V) if b % 2 == 0 else None
                want, tol = ref.adjust(logits[b, i], had, before["count"][b] >= ref.PROMPT, 1.3, 0.4, float(fr[b]), None,
                                       ok, -float("inf"), torch.float32)
                assert ref.within(adj[b, i].cpu(), want, tol), (s, b, i)
            am = adj[b, :n].cpu().argmax(-1).numpy().astype(np.int32)[None]
            a, pth, bo = oracle.tree_walk(am, draft[b:b + 1, :n].numpy(), parent[b:b + 1, :n].numpy())
            assert a[0] == acc and (pth[0] == path[:n].numpy()).all() and bo[0] == int(got["bonus"][b])
            assert int(got["newp"][b]) == p + acc + 1
            again = before["count"][b].clone()
            for t in [int(draft[b, int(path[j])]) for j in range(1, acc + 1)] + [int(bo[0])]:
                again[t] += 1
            assert torch.equal(count[b].cpu(), again), (s, b)
            accepted += acc
        held["P"].copy_(result["newp"])
    assert accepted > steps


def test_beams_over_shared_prompts(jf):
    """Beams of two prompts: what they share (the prompt, and ancestors' full pages) is found from their
    block tables each step, the attention agrees with the unshared call, and after every fork each beam's
    counts are those of its whole history."""
    B, W, Hkv, G, D, V, steps = 2, 4, 2, 4, 64, 300, 40
    Hq, cap = G * Hkv, 8
    gen = torch.Generator().manual_seed(9)
    pages = 2 * B * cap + steps * B * W + 8
    kc = torch.zeros((pages, PAGE, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    free = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((B * W, cap), -1, dtype=torch.int32)
    lens = []
    for b, n in enumerate((37, 5)):
        full = [free.pop() for _ in range(n // PAGE)]
        for w in range(W):
            table[b * W + w, :len(full)] = torch.tensor(full, dtype=torch.int32)
            table[b * W + w, len(full)] = free.pop()
        lens += [n] * W
    for r in range(B * W):                          # the prompts' keys and values (equal in equal places)
        g2 = torch.Generator().manual_seed(r // W)
        t = torch.arange(lens[r])
        x = torch.randn((2, lens[r], Hkv, D), generator=g2).to(torch.bfloat16).cuda()
        at = table[r][t // PAGE].long().cuda(), (t % PAGE).cuda()
        kc[at], vc[at] = x[0], x[1]
    table, lens = table.cuda(), ints(lens)
    freq, rs = jf.rotary_frequencies(D)
    prompt = torch.randint(0, V, (B * W, 20), generator=gen, dtype=torch.int32)
    prompt = prompt.view(B, W, 20)[:, :1].expand(-1, W, -1).reshape(B * W, 20).contiguous()
    count = jf.count_tokens(None, prompt.cuda(), prompt=True, V=V)
    history = [[] for _ in range(B * W)]
    score = torch.zeros((B, W), device="cuda")
    score[:, 1:] = -float("inf")
    gs = ints([0, W, 2 * W])
    mask = torch.ones((B * W, 1, 1), dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pres, fr = torch.full((B * W,), 0.7).cuda(), torch.full((B * W,), 0.2).cuda()
    base = torch.arange(B, device="cuda")[:, None] * W
    saw_sharing = 0
    for s in range(steps):
        qkv = torch.randn((B * W, 1, (Hq + 2 * Hkv), D), generator=gen).to(torch.bfloat16).cuda()
        q, k, v = qkv.split([Hq, Hkv, Hkv], dim=2)
        qr = jf.rotate_append_kv(q, k, v, kc, vc, table, lens, pos=lens[:, None].contiguous(), freq=freq, rotary_scale=rs,
                                 dev_err=err)
        # entries that all beams of a prompt have in common, from the front, before the page they write
        same = (table.view(B, W, -1) == table.view(B, W, -1)[:, :1]).all(1) & (table.view(B, W, -1)[:, 0] >= 0)
        shared = torch.minimum(same.int().cumprod(1).sum(1), lens.view(B, W).amin(1) // PAGE).to(torch.int32)
        saw_sharing += int((shared > 0).sum())
        out, lse = jf.tree_attention_shared(qr, kc, vc, table, lens, mask, gs, shared, with_lse=True, dev_err=err)
        want, wl = jf.tree_attention(qr, kc, vc, table.clamp(min=0), lens, mask, with_lse=True, dev_err=err)
        assert err.item() == 0
        assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()
        assert (lse - wl).abs().max() <= 1e-4
        logits = torch.randn((B * W, 1, V), generator=gen).cuda()
        adj = jf.adjust_logits(logits, count=count, presence=pres, frequency=fr, dev_err=err)
        parent, token, score, _ = jf.beam_select(adj.view(B, W, V), score, K=W)
        fresh = torch.tensor([free.pop() for _ in range(B * W)], dtype=torch.int32).view(B, W).cuda()
        table, lens = jf.beam_fork_kv(kc, vc, table, lens + 1, parent, fresh, dev_err=err)
        rows = (parent + base).flatten().to(torch.int32)
        count = jf.count_tokens(count, token.view(B * W, 1), row=rows, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == 0, s
        history = [history[int(r)] + [int(t)] for r, t in zip(rows, token.flatten())]
        for r in range(B * W):
            want_count = torch.zeros(V, dtype=torch.int32)
            want_count[prompt[r].long()] = ref.PROMPT
            for t in history[r]:
                want_count[t] += 1
            assert torch.equal(count[r].cpu(), want_count), (s, r)
    assert saw_sharing > steps


def test_new_tensors_on_a_side_stream(jf):
    """Calls that make their outputs and workspaces, given a stream: the same bits as on the current one, and
    padding rows are zero."""
    g = torch.Generator().manual_seed(8)
    B, N, Hq, Hkv, D, V = 3, 5, 4, 2, 64, 1000
    q, k, v = (torch.randn((B, N, H, D), generator=g).to(torch.bfloat16).cuda() for H in (Hq, Hkv, Hkv))
    table = torch.arange(B * 4, dtype=torch.int32).view(B, 4)
    table[1:, :2] = table[0, :2]                     # two shared pages
    lens = torch.tensor([33, 40, 50], dtype=torch.int32).cuda()
    sizes = torch.tensor([5, 1, 3], dtype=torch.int32).cuda()
    kc, vc = (torch.randn((B * 4, 16, Hkv, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    _, sees = ref.random_trees(B, N, g)
    mask, table = ref.pack_bits(sees).cuda(), table.cuda()
    pos = torch.randint(0, 100, (B, N), generator=g, dtype=torch.int32).cuda()
    freq, scale = jf.rotary_frequencies(D)
    start, pages = torch.tensor([0, B], dtype=torch.int32).cuda(), torch.tensor([2], dtype=torch.int32).cuda()
    x = torch.randn((B, N, V), generator=g).cuda()
    draft = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32).cuda()
    rep = torch.full((B,), 1.5).cuda()

    def step(stream):
        count = jf.count_tokens(None, draft, length=sizes, prompt=True, V=V, stream=stream)
        k2, v2 = kc.clone(), vc.clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        turned = jf.rotate_append_kv(q, k, v, k2, v2, table, lens, pos=pos, freq=freq, rotary_scale=scale,
                                     tree_len=sizes, stream=stream)
        out, lse = jf.tree_attention_shared(turned, k2, v2, table, lens, mask, start, pages, with_lse=True,
                                            tree_len=sizes, stream=stream)
        y = jf.adjust_logits(x, count=count, draft=draft, mask=mask, repetition=rep, tree_len=sizes, stream=stream)
        torch.cuda.synchronize()
        return count, turned, out, lse, y, k2, v2

    want = step(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = step(stream if stream is side else torch.cuda.ExternalStream(stream))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    count, turned, out, lse, y = want[:5]
    for b, n in enumerate(sizes.tolist()):
        assert not turned[b, n:].any() and not out[b, n:].any() and not y[b, n:].any() and not lse[b, :, n:].any()
        assert turned[b, :n].any() and out[b, :n].any() and y[b, :n].any()
