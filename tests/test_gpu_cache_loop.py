"""The bounded-cache and beam calls as a decoding loop runs them, against the CPU doing the
same steps on its own state.

Speculation with a bounded cache: ragged draft trees, mask, attention, greedy verification,
compaction, then the accepted rows' attention weight, the choice of the kept keys and their
move, in place; the next step starts from the evicted cache.  Masks, paths, kept positions,
lengths and the whole K/V pool agree bit for bit after every step, weights within the bound
of their fp32 sums.  (Which keys stay is decided on the GPU's weights: two weights may be
closer than their rounding.)

Beams: attention of every beam over its own paged context, selection, fork; the CPU keeps
every beam's whole history apart.  Once the caches are full, the beams' shared pages are
evicted into new ones."""
import dataclasses

import numpy as np
import pytest
import torch

import cache_reference as ref
import oracle
from test_gpu_beam import check_beams
from test_gpu_cache import close, dev, new_err
from test_gpu_ragged import check_rows
from tree_speculative_decoding_jf_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module")
def jf():
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf as mod
    return mod


def bf16_bits(rng, shape):
    return wl.to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def from_bits(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).cuda()


def to_bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("G,D,budget", [(4, 64, 112), (8, 128, 48)])
def test_speculation_with_a_bounded_cache(jf, G, D, budget):
    B, N, Hkv, V, steps, sink, recent = 3, 24, 2, 256, 7, 2, 16
    Hq = G * Hkv
    P0 = np.array([100, 60, 0], np.int32)
    base = wl.make_workload("bounded", B, N, Hq, Hkv, D, V, np.full(B, max(budget, 100) + N), tree="chain",
                            permute_pages=True, seed=G + D, with_logits=False)
    rng = np.random.default_rng(G * 100 + D)
    k_np, v_np, bt = base.k_cache.copy(), base.v_cache.copy(), base.block_table
    k_gpu, v_gpu, bt_gpu = from_bits(k_np), from_bits(v_np), dev(bt)
    cap = bt.shape[1] * PAGE
    weight = torch.zeros((B, Hkv, cap), device="cuda")
    P, P_dev = P0.copy(), dev(P0)
    evicted = 0
    for step in range(steps):
        tree_len = rng.integers(1, N + 1, B)
        parent = np.full((B, N), -1, np.int32)
        for b in range(B):
            n = int(tree_len[b])
            parent[b, :n] = [-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)]
        draft = rng.integers(0, V, (B, N)).astype(np.int32)
        q = bf16_bits(rng, (B, N, Hq, D))
        k_new, v_new = bf16_bits(rng, (B, N, Hkv, D)), bf16_bits(rng, (B, N, Hkv, D))
        slots = np.array([[bt[b, (P[b] + i) // 16] * 16 + (P[b] + i) % 16 for i in range(N)] for b in range(B)])
        for np_pool, gpu_pool, new in ((k_np, k_gpu, k_new), (v_np, v_gpu, v_new)):
            np_pool.reshape(-1, Hkv, D)[slots.reshape(-1)] = new.reshape(-1, Hkv, D)
            gpu_pool.view(-1, Hkv, D)[dev(slots.reshape(-1))] = from_bits(new.reshape(-1, Hkv, D))
        logits = rng.standard_normal((B, N, V)).astype(np.float32)
        for b in range(B):
            for c in range(1, int(tree_len[b])):
                if rng.random() < 0.7:
                    logits[b, parent[b, c], draft[b, c]] = 10.0 + rng.random()
        w = dataclasses.replace(base, prefix_len=P.copy(), parent=parent, q=q, k_cache=k_np, v_cache=v_np,
                                logits=logits, logits_dtype="f32", draft=draft)
        # ---- GPU: one step, no host round trip
        err = new_err()
        tl, t_par, qg = dev(tree_len.astype(np.int32)), dev(parent), from_bits(q)
        mask, _, _ = jf.build_tree_mask(t_par, P_dev, dev_err=err, tree_len=tl)
        out, lse = jf.tree_attention(qg, k_gpu, v_gpu, bt_gpu, P_dev, mask, scale=w.scale, with_lse=True,
                                     dev_err=err, tree_len=tl)
        _, acc, path, _ = jf.tree_verify(dev(logits), dev(draft), t_par, dev_err=err, tree_len=tl)
        newp = jf.compact_accepted_kv(k_gpu, v_gpu, bt_gpu, P_dev, path, acc, dev_err=err)
        before = weight.clone()
        jf.accumulate_attention_weight(qg, k_gpu, bt_gpu, P_dev, lse, path=path, accept_len=acc, weight=weight,
                                       scale=w.scale, out=weight, dev_err=err)
        summed = weight.clone()
        keep, kept = jf.select_kept_keys(weight, newp, budget, sink=sink, recent=recent, dev_err=err)
        jf.evict_kv(k_gpu, v_gpu, bt_gpu, newp, keep, kept, weight=weight, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == 0, step
        # ---- CPU
        check_rows(w, [int(x) for x in tree_len], out.float().cpu().numpy(), lse.cpu().numpy(), rows_per_seq=64,
                   seed=step)
        am = oracle.argmax(logits, "f32")
        r_path, r_acc = np.full((B, N), -1, np.int32), np.zeros(B, np.int32)
        for b in range(B):
            n = int(tree_len[b])
            a, pth, _ = oracle.tree_walk(am[b:b + 1, :n], draft[b:b + 1, :n], parent[b:b + 1, :n])
            r_acc[b], r_path[b, :n] = a[0], pth[0]
        assert (acc.cpu().numpy() == r_acc).all() and (path.cpu().numpy() == r_path).all()
        k_np, v_np, r_newp, ok = oracle.compact_accepted_kv(k_np, v_np, bt, P, r_path, r_acc)
        assert ok and (newp.cpu().numpy() == r_newp).all()
        qd = wl.bf16_bits_to_f32(q).astype(np.float64)
        kd = wl.bf16_bits_to_f32(k_np).astype(np.float64)
        for b in range(B):
            want, tol = ref.attention_weight(qd[b], kd, bt[b], int(P[b]), r_path[b, :r_acc[b] + 1].astype(np.int64),
                                             lse[b].cpu().numpy(), before[b].cpu().numpy(), before[b].cpu().numpy(),
                                             w.scale)
            close(summed[b], want, tol)
        r_keep, r_kept = ref.select_kept(summed.cpu().numpy(), r_newp, sink, recent, budget)
        assert (keep.cpu().numpy() == r_keep).all() and (kept.cpu().numpy() == r_kept).all()
        k_np, v_np, r_w = ref.evict_kv(k_np, v_np, bt, bt, r_keep, r_kept, summed.cpu().numpy())
        assert (to_bits(k_gpu) == k_np).all() and (to_bits(v_gpu) == v_np).all(), step
        assert (weight.cpu().numpy() == r_w).all()
        evicted += int((r_newp - r_kept).sum())
        P, P_dev = r_kept.astype(np.int32), kept
    assert evicted > 0                         # the bound was reached


def test_beam_decoding(jf):
    B, W, Hkv, G, D, V, steps = 2, 4, 2, 4, 64, 500, 66     # 21 + 59 tokens fill the five pages
    Hq, R = G * Hkv, 2 * 4
    rng = np.random.default_rng(77)
    start, budget, cap_pages = np.array([21, 3]), 40, 5
    pages = B * cap_pages + steps * R + 2 * R * cap_pages
    k_gpu = torch.zeros((pages, PAGE, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v_gpu = torch.zeros_like(k_gpu)
    free = list(rng.permutation(pages).astype(np.int32))
    take = lambda n: np.array([free.pop() for _ in range(n)], np.int32)   # noqa: E731
    # Each prompt's context is shared by its beams, then forked once so that every beam owns its last page.
    table = np.full((B, cap_pages), -1, np.int32)
    hist = []                                  # per beam: (K, V) bits [tokens][Hkv][D], and per head its kept tokens
    for b in range(B):
        n = int(start[b])
        table[b, :-(-n // PAGE)] = take(-(-n // PAGE))
        kb, vb = bf16_bits(rng, (n, Hkv, D)), bf16_bits(rng, (n, Hkv, D))
        t = np.arange(n)
        idx = (dev(table[b, t // PAGE].astype(np.int64)), dev(t % PAGE))
        k_gpu[idx], v_gpu[idx] = from_bits(kb), from_bits(vb)
        hist += [(kb, vb)] * W
    err = new_err()
    bt, lens = jf.beam_fork_kv(k_gpu, v_gpu, dev(table), dev(start.astype(np.int32)),
                               torch.zeros((B, W), dtype=torch.int32, device="cuda"), dev(take(R).reshape(B, W)),
                               dev_err=err)
    weight = torch.zeros((R, Hkv, cap_pages * PAGE), device="cuda")
    score = torch.full((B, W), -np.inf, device="cuda")
    score[:, 0] = 0.0
    finished = torch.zeros((B, W), dtype=torch.int32, device="cuda")
    scale, evictions, one = D ** -0.5, 0, torch.full((R, 1), -1, dtype=torch.int32, device="cuda")
    for step in range(steps):
        # the token each beam decodes: its K/V at position lens, its query
        P = lens.cpu().numpy()
        tb = bt.cpu().numpy()
        q, kn, vn = bf16_bits(rng, (R, 1, Hq, D)), bf16_bits(rng, (R, Hkv, D)), bf16_bits(rng, (R, Hkv, D))
        idx = (dev(tb[np.arange(R), P // PAGE].astype(np.int64)), dev(P.astype(np.int64) % PAGE))
        k_gpu[idx], v_gpu[idx] = from_bits(kn), from_bits(vn)
        hist = [(np.concatenate([h[0], kn[r:r + 1]]), np.concatenate([h[1], vn[r:r + 1]])) for r, h in enumerate(hist)]
        mask, _, _ = jf.build_tree_mask(one, lens, dev_err=err)
        out, lse = jf.tree_attention(from_bits(q), k_gpu, v_gpu, bt, lens, mask, scale=scale, with_lse=True, dev_err=err)
        jf.accumulate_attention_weight(from_bits(q), k_gpu, bt, lens, lse, weight=weight, scale=scale, out=weight,
                                       dev_err=err)
        got = out.float().cpu().numpy()
        for r in range(R):                     # the oracle's attention is over the history
            kf, vf = (wl.bf16_bits_to_f32(x).astype(np.float64) for x in hist[r])
            qf = wl.bf16_bits_to_f32(q[r, 0]).astype(np.float64)
            for h in range(Hq):
                s = scale * kf[:, h // G] @ qf[h]
                e = np.exp(s - s.max())
                want = (e / e.sum()) @ vf[:, h // G]
                assert (np.abs(got[r, 0, h] - want) <= 2e-3 + 1e-2 * np.abs(want)).all(), (step, r, h)
        # the next beams
        logits = (3 * rng.standard_normal((B, W, V))).astype(np.float32)
        picked = jf.beam_select(dev(logits), score, W, finished=finished, eos_token=7)
        check_beams(logits, score.cpu().numpy(), finished.cpu().numpy(), 7, picked, W)
        parent, _, score, finished = picked
        lens = lens + 1
        if int(lens.max()) >= cap_pages * PAGE:
            # full: the beams share pages, so the kept rows move into pages of their own
            table2 = np.full((R, cap_pages), -1, np.int32)
            table2[:, :-(-budget // PAGE)] = take(R * -(-budget // PAGE)).reshape(R, -1)
            keep, kept = jf.select_kept_keys(weight, lens, budget, sink=1, recent=8, dev_err=err)
            moved = torch.zeros_like(weight)
            jf.evict_kv(k_gpu, v_gpu, bt, lens, keep, kept, new_block_table=dev(table2), weight=weight,
                        weight_out=moved, dev_err=err)
            want_keep, want_kept = ref.select_kept(weight.cpu().numpy(), lens.cpu().numpy(), 1, 8, budget)
            assert (keep.cpu().numpy() == want_keep).all() and (kept.cpu().numpy() == want_kept).all()
            hist = [tuple(np.stack([c[want_keep[r, g, :want_kept[r]], g] for g in range(Hkv)], 1) for c in hist[r])
                    for r in range(R)]
            bt, lens, weight = dev(table2), kept, moved
            evictions += 1
        bt, lens = jf.beam_fork_kv(k_gpu, v_gpu, bt, lens, parent, dev(take(R).reshape(B, W)), dev_err=err)
        rows = (parent.long() + torch.arange(B, device="cuda")[:, None] * W).flatten()
        weight = weight[rows].contiguous()
        hist = [hist[r] for r in rows.tolist()]
        torch.cuda.synchronize()
        assert err.item() == 0, step
        tb, P = bt.cpu().numpy(), lens.cpu().numpy()
        for r in range(R):                     # every beam's pages hold its own history
            t = np.arange(P[r])
            assert len(hist[r][0]) == P[r]
            for pool, h in ((k_gpu, hist[r][0]), (v_gpu, hist[r][1])):
                assert (to_bits(pool[dev(tb[r, t // PAGE].astype(np.int64)), dev(t % PAGE)]) == h).all(), (step, r)
    assert evictions >= 1
