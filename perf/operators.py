"""Cases for timing the cache operators that run between two decoding steps: the attention
weight every cached key has received, the choice of the keys a smaller cache keeps, the
move of their K/V, beam selection over beams and vocabulary, and the fork of the beams'
paged caches.

``listed`` names fixed cases and ``draw`` makes more of the same ranges; ``prepare`` builds
a case's inputs on the GPU from a seed; ``run`` is one pass, with the library's calls where
``own`` is true and with elementary torch operations otherwise; ``exact`` is the result in
64 bits; ``work`` counts the bytes and operations one pass cannot do without.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # One sequence after a verified budget-16 chain: 5 accepted rows over a 2K cache (latency).
        dict(name="weight_chain16_2k", op="weight", B=1, N=16, Hq=32, Hkv=8, D=128, P=2048, step=0, rows=5,
             path=True, packed=False),
        # Eight 32K contexts after a budget-256 tree: up to 7 accepted rows per sequence (reads all of K).
        dict(name="weight_tree256_32k", op="weight", B=8, N=256, Hq=32, Hkv=4, D=128, P=32768, step=129, rows=7,
             path=True, packed=False),
        # The last 512 prompt rows score a 16K prompt before its first eviction (matrix products and exponentials).
        dict(name="weight_window512_16k", op="weight", B=2, N=512, Hq=32, Hkv=8, D=128, P=16001, step=77, rows=512,
             path=False, packed=False),
        # One sequence a little over its budget: the steady state of a bounded cache (latency).
        dict(name="select_2k", op="select", B=1, Hkv=8, P=2304, step=0, sink=4, recent=64, budget=2048),
        # 32 long contexts cut to an eighth.
        dict(name="select_b32_32k", op="select", B=32, Hkv=8, P=32768, step=301, sink=4, recent=256, budget=4096),
        # The move that follows select_2k.
        dict(name="evict_2k", op="evict", B=1, Hkv=8, D=128, P=2304, step=0, budget=2048),
        # Eight 32K contexts halved.
        dict(name="evict_b8_32k", op="evict", B=8, Hkv=4, D=128, P=33024, step=129, budget=16384),
        # One prompt, four beams, twice as many continuations (latency).
        dict(name="beam_w4", op="beam", B=1, W=4, K=8, V=151936, dtype="bf16", done=0),
        # Five beams of six prompts in fp32 over an odd vocabulary, some beams finished.
        dict(name="beam_f32_odd", op="beam", B=6, W=5, K=5, V=50257, dtype="f32", done=3),
        # 32 prompts of eight beams: 256 rows of logits.
        dict(name="beam_b32_w8", op="beam", B=32, W=8, K=16, V=151936, dtype="bf16", done=0),
        # Four beams of one prompt.
        dict(name="fork_w4", op="fork", B=1, W=4, K=4, Hkv=8, D=128, P=2055, step=0),
        # 32 prompts of eight beams: 256 partial pages and 256 block-table rows.
        dict(name="fork_b32_w8", op="fork", B=32, W=8, K=8, Hkv=8, D=128, P=4111, step=37),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weight", "weight", "weight", "select", "evict", "beam", "beam", "fork"])
    heads, D = rng.choice([(32, 8), (32, 4), (4, 1), (12, 4), (16, 16)]), rng.choice([64, 128, 128])
    if op == "weight":
        Hq, Hkv = heads
        path = rng.random() < 0.7
        B = _log(rng, 1, 16)
        P = _log(rng, 17, 32768)
        N = _log(rng, 1, 256) if path else _log(rng, 1, 512)
        rows = min(N, _log(rng, 1, 24)) if path else N
        while B * Hq * rows * P > 2 * 32 * 512 * 16001:
            P = max(1, P // 2)
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, P=P, step=rng.randrange(0, 1 + P // (2 * B)), rows=rows,
                    path=path, packed=path and rng.random() < 0.4)
    if op == "select":
        B, P = _log(rng, 1, 32), _log(rng, 40, 32768)
        sink, recent = rng.randrange(0, 8), rng.randrange(0, min(256, P // 4) + 1)
        budget = max(sink + recent, 1) + rng.randrange(0, P)
        return dict(op=op, B=B, Hkv=heads[1], P=P, step=rng.randrange(0, 1 + P // (2 * B)), sink=sink, recent=recent,
                    budget=budget)
    if op == "evict":
        B, P = _log(rng, 1, 8), _log(rng, 40, 33024)
        return dict(op=op, B=B, Hkv=min(heads[1], 8), D=D, P=P, step=rng.randrange(0, 1 + P // (2 * B)),
                    budget=max(1, rng.randrange(P // 8, P) // (2 if heads[1] > 4 else 1)))
    if op == "beam":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        B, W, V = _log(rng, 1, 32 if dtype == "bf16" else 16), rng.randrange(1, 9), _log(rng, 1000, 151936)
        K = rng.choice([W, 2 * W, rng.randrange(1, 33)])
        return dict(op=op, B=B, W=W, K=K, V=V, dtype=dtype, done=rng.choice([0, 0, 2, 5]))
    B, W, K = _log(rng, 1, 32), rng.randrange(1, 9), rng.randrange(1, 9)
    return dict(op=op, B=B, W=W, K=K, Hkv=min(heads[1], 8), D=D, P=_log(rng, 1, 4111), step=rng.randrange(0, 40))


def _lengths(case):
    """Cached tokens of every sequence: P and shorter ones (the batch is ragged)."""
    return [max(1, case["P"] - b * case["step"]) for b in range(case["B"])]


def _rows(case):
    """Query rows of every sequence: all N of a window, 1 .. rows accepted nodes after a verify."""
    return [1 + (5 * b + case["rows"] - 1) % case["rows"] if case["path"] else case["N"] for b in range(case["B"])]


def _tree_sizes(case):
    """Nodes of every sequence's tree in the packed layout."""
    return [max(r, case["N"] - 3 * b) for b, r in enumerate(_rows(case))]


# ----------------------------------------------------------------------------- inputs

def _paged(case, lens, extra, g, spare=0):
    """A pool with every sequence's pages in random order, `spare` more pages per sequence
    in a second table, and the block tables (-1 past a sequence's pages)."""
    need = [(n + extra + PAGE - 1) // PAGE for n in lens]
    cap = max(need)
    pages = sum(need) + spare * len(lens)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), cap), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    second = torch.full((len(lens), cap), -1, dtype=torch.int32, device="cuda")
    if spare:
        second[:, :spare] = order[at:].view(len(lens), spare)
    shape = (pages, PAGE, case["Hkv"], case["D"])
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return k, v, table, second


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    made = {"weight": _prepare_weight, "select": _prepare_select, "evict": _prepare_evict, "beam": _prepare_beam,
            "fork": _prepare_fork}[case["op"]](case, g)
    return dict(made, case=case)


def _prepare_weight(case, g):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    lens, rows = _lengths(case), _rows(case)
    k, _, table, _ = _paged(case, lens, N, g)
    cap = table.shape[1] * PAGE
    scale = D ** -0.5
    path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    sizes = _tree_sizes(case) if case["packed"] else [N] * B
    for b, r in enumerate(rows):     # accepted nodes: the root, then rising node ids
        path[b, 0] = 0
        if r > 1:
            ids = torch.randperm(sizes[b] - 1, generator=g, device="cuda")[:r - 1] + 1
            path[b, 1:r] = ids.sort().values.to(torch.int32)
    q = torch.randn((B, N, Hq, D), generator=g, device="cuda", dtype=torch.bfloat16)
    # The log-sum-exp every row's attention left behind: over the prefix and the row's own branch.
    lse = torch.zeros((B, Hq, N), device="cuda")
    for b in range(B):
        L = lens[b] + rows[b]
        kb = k[table[b, :(L + PAGE - 1) // PAGE].long()].flatten(0, 1)[:L].float()
        ids = path[b, :rows[b]].long() if case["path"] else torch.arange(N, device="cuda")
        seen = torch.arange(L, device="cuda") <= lens[b] + torch.arange(rows[b], device="cuda")[:, None]
        for h in range(Hq):
            s = q[b, ids, h].float() @ kb[:, h // (Hq // Hkv)].t() * scale
            lse[b, h, ids] = s.masked_fill_(~seen, -math.inf).logsumexp(-1)
    # A few passes' worth of weight so far, so that neither part of the sum hides the other.
    weight = torch.rand((B, Hkv, cap), generator=g, device="cuda") * (4.0 * case["rows"] * Hq / (Hkv * case["P"]))
    state = dict(k_cache=k, block_table=table, prefix_len=_ints(lens), accept_len=_ints([r - 1 for r in rows]),
                 path=path if case["path"] else None, weight=weight, weight_out=torch.zeros_like(weight),
                 scale=scale, cu_seqlens=None)
    if case["packed"]:
        cu = [0]
        for n in sizes:
            cu.append(cu[-1] + n)
        at = torch.cat([torch.arange(n, device="cuda") + b * N for b, n in enumerate(sizes)])
        q = q.flatten(0, 1)[at].contiguous()
        lse = lse.transpose(0, 1).flatten(1)[:, at].contiguous()
        state["cu_seqlens"] = _ints(cu)
    return dict(state, q=q, lse=lse)


def _prepare_select(case, g):
    weight = torch.randn((case["B"], case["Hkv"], -(-case["P"] // PAGE) * PAGE), generator=g, device="cuda")
    return dict(weight=torch.exp(1.5 * weight - 4.0), seq_len=_ints(_lengths(case)))


def _prepare_evict(case, g):
    lens, n = _lengths(case), case["budget"]
    k, v, table, new_table = _paged(case, lens, 0, g, spare=-(-min(n, case["P"]) // PAGE))
    cap = table.shape[1] * PAGE
    keep = torch.full((case["B"], case["Hkv"], n), -1, dtype=torch.int32, device="cuda")
    for b, L in enumerate(lens):
        kept = torch.rand((case["Hkv"], L), generator=g, device="cuda").argsort(-1)[:, :n].sort(-1).values
        keep[b, :, :kept.shape[1]] = kept.to(torch.int32)
    weight = torch.rand((case["B"], case["Hkv"], cap), generator=g, device="cuda")
    return dict(k_cache=k, v_cache=v, block_table=table, new_block_table=new_table, seq_len=_ints(lens), keep=keep,
                kept_len=_ints([min(L, n) for L in lens]), weight=weight, weight_out=torch.zeros_like(weight))


def _prepare_beam(case, g):
    B, W, V = case["B"], case["W"], case["V"]
    logits = torch.randn((B, W, V), generator=g, device="cuda").mul_(2.5)
    logits = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
    score = -8.0 * torch.rand((B, W), generator=g, device="cuda") - 4.0
    finished = torch.zeros(B * W, dtype=torch.int32, device="cuda")
    finished[torch.randperm(B * W, generator=g, device="cuda")[:min(case["done"], B * W - 1)]] = 1
    return dict(logits=logits, score=score, finished=finished.view(B, W), eos=V - 1)


def _prepare_fork(case, g):
    B, W, K = case["B"], case["W"], case["K"]
    lens = _lengths(case)
    full, cap = [n // PAGE for n in lens], max(lens) // PAGE + 1
    shared = sum(full)
    pages = shared + B * W + B * K
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, W, cap), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(full):     # the beams of a prompt share its full pages; the last page is each beam's own
        table[b, :, :n] = order[at:at + n]
        table[b, :, n] = order[shared + b * W:shared + (b + 1) * W]
        at += n
    shape = (pages, PAGE, case["Hkv"], case["D"])
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    parent = torch.randint(0, W, (B, K), generator=g, device="cuda", dtype=torch.int32)
    return dict(k_cache=k, v_cache=v, block_table=table.view(B * W, cap), prefix_len=_ints(lens).repeat_interleave(W),
                parent=parent, fresh_page=order[shared + B * W:].view(B, K).contiguous())


# ----------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"weight": _own_weight, "select": _own_select, "evict": _own_evict, "beam": _own_beam,
                "fork": _own_fork}[op](state)
    return {"weight": _plain_weight, "select": _plain_select, "evict": _plain_evict, "beam": _plain_beam,
            "fork": _plain_fork}[op](state)


def _own_weight(s):
    from tree_speculative_decoding_jf_gb300 import jf
    return {"weight": jf.accumulate_attention_weight(
        s["q"], s["k_cache"], s["block_table"], s["prefix_len"], s["lse"], path=s["path"], accept_len=s["accept_len"],
        weight=s["weight"], scale=s["scale"], cu_seqlens=s["cu_seqlens"], out=s["weight_out"])}


def _own_select(s):
    from tree_speculative_decoding_jf_gb300 import jf
    c = s["case"]
    keep, kept_len = jf.select_kept_keys(s["weight"], s["seq_len"], c["budget"], sink=c["sink"], recent=c["recent"])
    return {"keep": keep, "kept_len": kept_len}


def _own_evict(s):
    from tree_speculative_decoding_jf_gb300 import jf
    jf.evict_kv(s["k_cache"], s["v_cache"], s["block_table"], s["seq_len"], s["keep"], s["kept_len"],
                new_block_table=s["new_block_table"], weight=s["weight"], weight_out=s["weight_out"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weight": s["weight_out"]}


def _own_beam(s):
    from tree_speculative_decoding_jf_gb300 import jf
    parent, token, score, finished = jf.beam_select(s["logits"], s["score"], s["case"]["K"], finished=s["finished"],
                                                    eos_token=s["eos"])
    return {"parent": parent, "token": token, "score": score, "finished": finished}


def _own_fork(s):
    from tree_speculative_decoding_jf_gb300 import jf
    table, lens = jf.beam_fork_kv(s["k_cache"], s["v_cache"], s["block_table"], s["prefix_len"], s["parent"],
                                  s["fresh_page"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "block_table": table, "prefix_len": lens}


def _plain_weight(s):
    """weight[b, g, t] + sum over rows r and the heads h of group g of exp(scale q.k - lse),
    rows seeing the keys t <= P_b + r; keys P_b .. P_b + rows - 1 start from zero."""
    c = s["case"]
    B, N, Hq, Hkv, D, R = (c[k] for k in ("B", "N", "Hq", "Hkv", "D", "rows"))
    P, count = s["prefix_len"].long(), s["accept_len"].long() + 1
    r = torch.arange(R, device="cuda")
    ids = s["path"][:, :R].long().clamp_(min=0) if c["path"] else r.expand(B, R)
    first = s["cu_seqlens"][:-1].long() if c["packed"] else torch.arange(B, device="cuda") * N
    at = (first[:, None] + ids).flatten()
    q = s["q"].view(-1, Hq, D)[at.clamp(max=s["q"].numel() // (Hq * D) - 1)].float()
    q = q.view(B, R, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    lse = s["lse"] if c["packed"] else s["lse"].transpose(0, 1).reshape(Hq, -1)
    lse = lse[:, at.clamp(max=lse.shape[1] - 1)].view(Hkv, Hq // Hkv, B, R).permute(2, 0, 3, 1).reshape(B, Hkv, -1, 1)
    k = s["k_cache"][s["block_table"].long().clamp_(min=0)].float().flatten(1, 2)            # [B, cap, Hkv, D]
    p = q @ k.permute(0, 2, 3, 1)                                                             # [B, Hkv, R * G, cap]
    p.mul_(s["scale"]).sub_(lse).exp_()
    t = torch.arange(k.shape[1], device="cuda")
    seen = (t <= P[:, None, None] + r[:, None]) & (r[:, None] < count[:, None, None])        # [B, R, cap]
    p.masked_fill_(~seen.repeat_interleave(Hq // Hkv, 1)[:, None], 0.0)
    old = s["weight"].masked_fill(t >= P[:, None, None], 0.0)
    live = t < (P + count)[:, None, None]
    return {"weight": torch.where(live, old + p.sum(2), s["weight_out"])}


def _plain_select(s):
    """Per kv-head: the first `sink` and last `recent` keys, then the greatest weights (ties:
    the lowest position), in rising position."""
    c = s["case"]
    w, K = s["weight"], c["budget"]
    L = s["seq_len"].long()[:, None, None]
    t = torch.arange(w.shape[2], device="cuda")
    rank = w.masked_fill((t < c["sink"]) | (t >= L - c["recent"]), math.inf).masked_fill(t >= L, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    order = torch.cat([order, order.new_full(order.shape[:2] + (max(0, K - order.shape[2]),), w.shape[2])], -1)
    order = order.masked_fill(torch.arange(K, device="cuda") >= L, w.shape[2]).sort(-1).values
    keep = order.masked_fill(order == w.shape[2], -1).to(torch.int32)
    return {"keep": keep, "kept_len": s["seq_len"].clamp(max=K)}


def _plain_evict(s):
    """Row j of every head's new cache = row keep[j] of its old one, and its weight."""
    k, v, keep = s["k_cache"], s["v_cache"], s["keep"].long()
    B, Hkv, n = keep.shape
    b, g, j = torch.nonzero(keep >= 0, as_tuple=True)
    t = keep[b, g, j]
    src, dst = s["block_table"][b, t // PAGE].long(), s["new_block_table"][b, j // PAGE].long()
    k[dst, j % PAGE, g] = k[src, t % PAGE, g]
    v[dst, j % PAGE, g] = v[src, t % PAGE, g]
    s["weight_out"][b, g, j] = s["weight"][b, g, t]
    return {"k_cache": k, "v_cache": v, "weight": s["weight_out"]}


def _plain_beam(s):
    """The K best (beam, token) pairs by score + log softmax (ties: the lowest pair); a
    finished beam goes on with its end token alone, at its own score.  In 64 bits: two
    pairs' scores may lie closer than fp32 tells apart."""
    B, W, V = s["logits"].shape
    x = s["logits"].double()
    x = x - x.amax(-1, keepdim=True)
    x = x - x.exp().sum(-1, keepdim=True).log() + s["score"].double()[..., None]
    over = s["finished"].bool()[..., None]
    end = torch.arange(V, device="cuda") == s["eos"]
    x = torch.where(over, torch.where(end, s["score"].double()[..., None], -math.inf), x).view(B, W * V)
    best = x.sort(dim=-1, descending=True, stable=True)
    pick = best.indices[:, :s["case"]["K"]]
    parent, token = pick // V, pick % V
    finished = s["finished"].gather(1, parent) | (token == s["eos"])
    return {"parent": parent.to(torch.int32), "token": token.to(torch.int32),
            "score": best.values[:, :s["case"]["K"]].float(), "finished": finished.to(torch.int32)}


def _plain_fork(s):
    """Beam j of prompt b takes its parent's full pages by id and its partial page by copy
    into a fresh page."""
    k, v, parent, fresh = s["k_cache"], s["v_cache"], s["parent"].long(), s["fresh_page"].long().flatten()
    B, K = parent.shape
    W, cap = s["block_table"].shape[0] // B, s["block_table"].shape[1]
    row = (parent + torch.arange(B, device="cuda")[:, None] * W).flatten()
    lens = s["prefix_len"][row].long()
    full, part = lens // PAGE, lens % PAGE
    old = s["block_table"][row].long()
    at = torch.arange(cap, device="cuda")
    table = torch.where(at < full[:, None], old, torch.where(at == full[:, None], fresh[:, None], -1))
    src = old.gather(1, full.clamp(max=cap - 1)[:, None])[:, 0]
    beam, slot = torch.nonzero(torch.arange(PAGE, device="cuda") < part[:, None], as_tuple=True)
    k[fresh[beam], slot] = k[src[beam], slot]
    v[fresh[beam], slot] = v[src[beam], slot]
    return {"k_cache": k, "v_cache": v, "block_table": table.to(torch.int32), "prefix_len": lens.to(torch.int32)}


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"weight": _exact_weight, "select": _exact_select, "evict": _exact_evict, "beam": _exact_beam,
            "fork": _exact_fork}[case["op"]](case, s)


def _exact_weight(case, s):
    lens, rows, G = _lengths(case), _rows(case), case["Hq"] // case["Hkv"]
    if 2.0 * case["D"] * case["Hq"] * sum(r * (n + r) for r, n in zip(rows, lens)) > 4e12:
        return None
    out = s["weight_out"].double()
    for b, (P, R) in enumerate(zip(lens, rows)):
        nodes = s["path"][b, :R].tolist() if case["path"] else list(range(R))
        if case["packed"]:
            at = [int(s["cu_seqlens"][b]) + i for i in nodes]
            q, lse = s["q"][at].double(), s["lse"][:, at].double().t()
        else:
            q, lse = s["q"][b, nodes].double(), s["lse"][b][:, nodes].double().t()           # [R, Hq, D], [R, Hq]
        L = P + R
        keys = s["k_cache"][s["block_table"][b, :-(-L // PAGE)].long()].reshape(-1, case["Hkv"], case["D"])[:L]
        hidden = torch.ones((R, L), dtype=torch.bool, device="cuda").triu(P + 1)
        for g in range(case["Hkv"]):
            total = torch.zeros(L, dtype=torch.float64, device="cuda")
            total[:P] = s["weight"][b, g, :P]
            kg = keys[:, g].double()
            for h in range(g * G, (g + 1) * G):
                e = torch.exp(torch.addmm(-lse[:, h, None], q[:, h], kg.t(), alpha=s["scale"]))
                total += e.masked_fill(hidden, 0.0).sum(0)
            out[b, g, :L] = total
    return {"weight": out}


def _exact_select(case, s):
    return None


def _exact_evict(case, s):
    k, v, w = s["k_cache"].double().cpu(), s["v_cache"].double().cpu(), s["weight_out"].double()
    old, new = s["block_table"].tolist(), s["new_block_table"].tolist()
    if k.numel() > 1 << 28:
        return None
    moved = [(k.clone(), k), (v.clone(), v)]
    for b, n in enumerate(s["kept_len"].tolist()):
        for g in range(case["Hkv"]):
            kept = s["keep"][b, g, :n].cpu().numpy()
            src = np.take(old[b], kept // PAGE) * PAGE + kept % PAGE
            dst = np.take(new[b], np.arange(n) // PAGE) * PAGE + np.arange(n) % PAGE
            for to, was in moved:
                to.view(-1, case["Hkv"], case["D"]).numpy()[dst, g] = was.view(-1, case["Hkv"], case["D"]).numpy()[src, g]
            w[b, g, :n] = s["weight"][b, g].double()[torch.from_numpy(kept).long().cuda()]
    return {"k_cache": moved[0][0], "v_cache": moved[1][0], "weight": w}


def _exact_beam(case, s):
    B, W, V, K = case["B"], case["W"], case["V"], case["K"]
    out = torch.empty((B, K), dtype=torch.float64)
    for b in range(B):
        every = []
        for w in range(W):
            start = float(s["score"][b, w])
            if int(s["finished"][b, w]):
                every.append(torch.tensor([start], dtype=torch.float64))
            else:
                x = s["logits"][b, w].double()
                every.append((start + (x - torch.logsumexp(x, 0))).topk(min(K, V)).values.cpu())
        best = torch.cat(every).sort(descending=True).values[:K]
        out[b] = -math.inf
        out[b, :best.numel()] = best
    return {"parent": None, "token": None, "score": out, "finished": None}


def _exact_fork(case, s):
    k, v = s["k_cache"].double().cpu(), s["v_cache"].double().cpu()
    parent, fresh, table = s["parent"].tolist(), s["fresh_page"].tolist(), s["block_table"].tolist()
    lens = _lengths(case)
    for b in range(case["B"]):
        for j in range(case["K"]):
            n = lens[b] % PAGE
            page = table[b * case["W"] + parent[b][j]][lens[b] // PAGE]
            k[fresh[b][j], :n] = k[page, :n].clone()
            v[fresh[b][j], :n] = v[page, :n].clone()
    return {"k_cache": k, "v_cache": v, "block_table": None, "prefix_len": None}


# ----------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "beam":
        rows = case["B"] * case["W"]
        live = rows - min(case["done"], rows - 1)
        return {"bytes": live * case["V"] * (2 if case["dtype"] == "bf16" else 4) + 8 * rows + 16 * case["B"] * case["K"],
                "flops": 3 * live * case["V"]}
    lens = _lengths(case)
    if op == "weight":
        rows, G = _rows(case), case["Hq"] // case["Hkv"]
        keys, every = sum(n + r for n, r in zip(lens, rows)), sum(rows)
        pairs = sum(r * n + r * (r + 1) // 2 for n, r in zip(lens, rows))
        return {"bytes": case["Hkv"] * (keys * (case["D"] * 2 + 4) + sum(lens) * 4)      # K, new weights, old weights
                + every * case["Hq"] * (case["D"] * 2 + 4),                               # query rows and their lse
                "flops": 2 * case["D"] * case["Hkv"] * G * pairs}
    if op == "select":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": 4 * case["Hkv"] * (sum(lens) + kept), "flops": 0}
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": case["Hkv"] * kept * (2 * 2 * 2 * case["D"] + 4 + 8), "flops": 0}
    part = sum(n % PAGE for n in lens) * case["K"]
    tables = sum(n // PAGE + 1 for n in lens) * case["K"]
    return {"bytes": part * case["Hkv"] * case["D"] * 2 * 2 * 2 + tables * 8, "flops": 0}
