"""Cases for timing the operators that stand before and after the attention and the verification of
a decoding step: the rotation of queries and keys with the append to the paged cache, attention for
sequences that share a long prefix, the penalties, biases and grammar masks on the logits, and the
token counts that the penalties read.

``listed`` names fixed cases and ``draw`` makes more of the same ranges; ``prepare`` builds a case's
inputs on the GPU from a seed; ``run`` is one pass, with the library's calls where ``own`` is true
and with elementary torch operations otherwise; ``exact`` is the result in 64 bits; ``work`` counts
the bytes and operations one pass cannot do without.
"""
import math

import torch

own = False

PAGE = 16
PROMPT = 1 << 30          # a token count's flag: the token is in the prompt


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # One sequence's budget-16 chain: heads normalised, rotated, appended after 2K tokens (latency).
        dict(name="rotate_chain16", op="rotate", B=1, N=16, Hq=32, Hkv=8, D=128, R=128, P=2048, seen=2048, layout="padded",
             pairs="half", norm=True, scaling=1.0),
        # Eight packed trees of up to 256 nodes, far positions with frequencies scaled by four.
        dict(name="rotate_tree256_b8", op="rotate", B=8, N=256, Hq=32, Hkv=4, D=128, R=128, P=4096, seen=120000,
             layout="packed", pairs="half", norm=True, scaling=4.0),
        # Prompt chunks of 4096 tokens of eight sequences, interleaved pairs in half of each head (bytes).
        dict(name="rotate_prompt4k_b8", op="rotate", B=8, N=4096, Hq=32, Hkv=8, D=128, R=64, P=777, seen=777,
             layout="ragged", pairs="interleaved", norm=False, scaling=1.0),
        # One prompt's four beams a few tokens after their fork (latency).
        dict(name="shared_beams4_2k", op="shared", B=4, groups=1, N=1, Hq=32, Hkv=8, D=128, pages=128, own=12,
             layout="padded"),
        # 32 prompts of eight beams: 256 sequences, each prompt's cache read once.
        dict(name="shared_beams256_4k", op="shared", B=256, groups=32, N=1, Hq=32, Hkv=8, D=128, pages=256, own=48,
             layout="padded"),
        # 64 requests behind one 32K system prompt, each with up to 1500 tokens of its own.
        dict(name="shared_prompt64_32k", op="shared", B=64, groups=1, N=1, Hq=32, Hkv=4, D=128, pages=2048, own=1500,
             layout="padded"),
        # Packed trees of 16 requests in three uneven groups (matrix products).
        dict(name="shared_tree16_8k", op="shared", B=16, groups=3, N=64, Hq=32, Hkv=8, D=128, pages=512, own=300,
             layout="packed"),
        # One sequence's budget-16 chain under penalties, some nodes under a grammar.
        dict(name="adjust_chain16", op="adjust", B=1, N=16, V=151936, dtype="bf16", penalties=True, bias=False,
             grammar=True, layout="padded"),
        # Eight budget-256 trees: 2048 rows of logits (bytes).
        dict(name="adjust_tree256_b8", op="adjust", B=8, N=256, V=151936, dtype="bf16", penalties=True, bias=False,
             grammar=True, layout="padded"),
        # Packed rows of fp32 logits over an odd vocabulary, with biases.
        dict(name="adjust_f32_odd", op="adjust", B=6, N=9, V=50257, dtype="f32", penalties=True, bias=True, grammar=True,
             layout="packed"),
        # 32 new prompts of up to 32K tokens enter their sequences' counts, in place.
        dict(name="count_prompt_32k", op="count", B=32, N=32768, V=151936, kind="prompt"),
        # 256 new beams take their parents' counts and one more token each.
        dict(name="count_beams_b32_w8", op="count", B=256, N=1, V=151936, kind="beams"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "shared", "shared", "shared", "adjust", "adjust", "count"])
    (Hq, Hkv), D = rng.choice([(32, 8), (32, 4), (4, 1), (16, 16), (64, 4)]), rng.choice([64, 128, 128])
    layout = rng.choice(["padded", "ragged", "packed"])
    if op == "rotate":
        N = _log(rng, 1, 4096)
        B = max(1, min(_log(rng, 1, 32), 8 * 4096 * 48 // (N * (Hq + 2 * Hkv))))
        P = _log(rng, 1, 4096)
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, 16, 48]), P=P,
                    seen=P + rng.choice([0, _log(rng, 1, 1000000)]), layout=layout,
                    pairs=rng.choice(["half", "half", "interleaved"]), norm=rng.random() < 0.5,
                    scaling=rng.choice([1.0, 1.0, 4.0]))
    if op == "shared":
        N = 1 if rng.random() < 0.6 else _log(rng, 2, 64)
        B, pages, own = _log(rng, 1, 256 if N == 1 else 16), _log(rng, 1, 2048), _log(rng, 1, 1500)
        while B * (16 * pages + own) > (1 << 21 if N == 1 else 1 << 17):
            pages = max(1, pages // 2)
            own = max(1, own // 2)
        return dict(op=op, B=B, groups=max(1, min(B, _log(rng, 1, 32))), N=N, Hq=min(Hq, 32), Hkv=min(Hkv, 8), D=D,
                    pages=0 if rng.random() < 0.08 else pages, own=own, layout=layout)
    if op == "adjust":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        N, V = _log(rng, 1, 256), _log(rng, 1000, 151936)
        if rng.random() < 0.5:
            V = -(-V // 8) * 8
        B = _log(rng, 1, max(1, min(32, 1024 // N)))
        penalties, bias, grammar = rng.choice([(True, False, True), (True, True, True), (True, False, False),
                                               (False, False, True), (False, True, False)])
        return dict(op=op, B=B, N=N, V=V, dtype=dtype, penalties=penalties, bias=bias, grammar=grammar, layout=layout)
    kind = rng.choice(["prompt", "accepted", "beams"])
    B, V = _log(rng, 1, 32 if kind != "beams" else 256), _log(rng, 1000, 151936)
    N = {"prompt": _log(rng, 1, 32768), "accepted": _log(rng, 1, 256), "beams": 1}[kind]
    return dict(op=op, B=B, N=N, V=V, kind=kind)


def _sizes(case):
    """Nodes of every sequence: all N, or ragged ones (packed and padded batches of trees)."""
    N = case["N"]
    if case["layout"] == "padded":
        return [N] * case["B"]
    return [max(1, N - (b * 5) % max(1, N // 2 + 1)) for b in range(case["B"])]


def _groups(case):
    """First sequence of every group, then the number of sequences (later groups are larger unless the count divides)."""
    B, n = case["B"], case["groups"]
    if B % n == 0:
        return [u * (B // n) for u in range(n + 1)]
    return [u + (B - n) * u * u // (n * n) for u in range(n + 1)]


def _shared_lengths(case):
    """(pages shared by each group, cached tokens of each sequence)."""
    start = _groups(case)
    pages = [max(0, case["pages"] - 5 * u % max(1, case["pages"])) for u in range(case["groups"])]
    lens = []
    for u in range(case["groups"]):
        for b in range(start[u], start[u + 1]):
            lens.append(16 * pages[u] + (11 + 37 * b) % (case["own"] + 1))
    return pages, lens


# ----------------------------------------------------------------------------- inputs

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bf16(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _trees(case, g):
    """Random trees: (parent [B, N], ancestor-or-self [B, N, N], depth [B, N])."""
    B, N = case["B"], case["N"]
    parent = torch.full((B, N), -1, dtype=torch.int64, device="cuda")
    sees = torch.eye(N, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    rows = torch.arange(B, device="cuda")
    back = torch.randint(1, 9, (B, N), generator=g, device="cuda")
    for i in range(1, N):
        parent[:, i] = (i - back[:, i]).clamp(min=0)
        sees[:, i] |= sees[rows, parent[:, i]]
    return parent, sees, sees.sum(-1) - 1


def _pack_bits(sees):
    """Bool [..., N, N] -> int64 [..., N, ceil(N / 64)], bit j of word w for node 64 w + j."""
    N = sees.shape[-1]
    words = torch.nn.functional.pad(sees, (0, -N % 64)).unflatten(-1, (-1, 64))
    return (words.long() << torch.arange(64, device="cuda")).sum(-1)


def _node_rows(case, x):
    """The per-node array of the layout: [B, N, ...], or its real rows only when packed."""
    if case["layout"] != "packed":
        return x
    return torch.cat([x[b, :n] for b, n in enumerate(_sizes(case))]).contiguous()


def _layout_args(case):
    sizes = _sizes(case)
    cu = [0]
    for n in sizes:
        cu.append(cu[-1] + n)
    return dict(tree_len=_ints(sizes) if case["layout"] == "ragged" else None,
                cu_seqlens=_ints(cu) if case["layout"] == "packed" else None)


def _tokens(shape, V, g):
    """Token ids as text has them: a few of them most of the time."""
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    return ((u ** 4) * V).long().clamp_(max=V - 1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    made = {"rotate": _prepare_rotate, "shared": _prepare_shared, "adjust": _prepare_adjust,
            "count": _prepare_count}[case["op"]](case, g)
    return dict(made, case=case)


def _prepare_rotate(case, g):
    B, N, Hq, Hkv, D, R, P = (case[k] for k in ("B", "N", "Hq", "Hkv", "D", "R", "P"))
    sizes = _sizes(case)
    lens = [max(0, P - 3 * b) for b in range(B)]
    need = [-(-(p + n) // PAGE) for p, n in zip(lens, sizes)]
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    # The table has room for N nodes behind every prefix, as a padded batch's has.
    table = torch.full((B, -(-(max(lens) + N) // PAGE)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pool = (sum(need), PAGE, Hkv, D)
    if N <= 256:
        depth = _trees(case, g)[2]
    else:                                     # a chunk of a prompt
        depth = torch.arange(N, device="cuda").expand(B, N)
    pos = (depth + _ints([p + case["seen"] - P for p in lens])[:, None]).to(torch.int32)
    real = torch.arange(N, device="cuda") < _ints(sizes)[:, None]
    pos = pos.masked_fill(~real, -1)
    base = 1000000.0 if case["scaling"] > 1 else 10000.0
    freq = base ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R) / case["scaling"]
    tokens = sum(sizes) if case["layout"] == "packed" else B * N
    # One projection's output: query heads, key heads, value heads of a token side by side.
    qkv = _bf16((tokens, (Hq + 2 * Hkv) * D), g)
    norm = [1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2)] if case["norm"] else [None, None]
    q_norm, k_norm = (None if w is None else w.to(torch.bfloat16) for w in norm)
    out = torch.zeros((tokens, Hq, D) if case["layout"] == "packed" else (B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
    return dict(qkv=qkv, pos=_node_rows(case, pos), freq=freq, rotary_scale=0.1 * math.log(case["scaling"]) + 1.0,
                q_norm=q_norm, k_norm=k_norm, block_table=table, prefix_len=_ints(lens), k_cache=_bf16(pool, g),
                v_cache=_bf16(pool, g), out=out, **_layout_args(case))


def _prepare_shared(case, g):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    start, sizes = _groups(case), _sizes(case)
    pages, lens = _shared_lengths(case)
    owned = []
    for u in range(case["groups"]):
        owned += [-(-(lens[b] + sizes[b]) // PAGE) - pages[u] for b in range(start[u], start[u + 1])]
    total = sum(pages) + sum(owned)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    cap = -(-(max(lens) + N) // PAGE)
    table = torch.full((B, cap), -1, dtype=torch.int32, device="cuda")
    at = 0
    for u in range(case["groups"]):
        table[start[u]:start[u + 1], :pages[u]] = order[at:at + pages[u]]
        at += pages[u]
        for b in range(start[u], start[u + 1]):
            table[b, pages[u]:pages[u] + owned[b]] = order[at:at + owned[b]]
            at += owned[b]
    sees = _trees(case, g)[1]
    q = _node_rows(case, _bf16((B, N, Hq, D), g))
    lse = torch.zeros((Hq, q.shape[0]) if case["layout"] == "packed" else (B, Hq, N), device="cuda")
    return dict(q=q, out=torch.zeros_like(q), lse=lse, k_cache=_bf16((total, PAGE, Hkv, D), g),
                v_cache=_bf16((total, PAGE, Hkv, D), g), block_table=table, prefix_len=_ints(lens), sees=sees,
                mask=_node_rows(case, _pack_bits(sees)), group_start=_ints(start), shared_pages=_ints(pages),
                scale=D ** -0.5, **_layout_args(case))


def _prepare_adjust(case, g):
    B, N, V = case["B"], case["N"], case["V"]
    _, sees, _ = _trees(case, g)
    logits = torch.randn((B, N, V), generator=g, device="cuda").mul_(2.5)
    logits = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
    s = dict(logits=_node_rows(case, logits), sees=sees, count=None, draft=None, mask=None, bias=None, allowed=None,
             allowed_row=None, repetition=None, presence=None, frequency=None, **_layout_args(case))
    s["out"] = torch.zeros_like(s["logits"])
    if case["penalties"]:
        count = torch.zeros((B, V), dtype=torch.int32, device="cuda")
        count.scatter_add_(1, _tokens((B, 300), V, g).long(), torch.ones((B, 300), dtype=torch.int32, device="cuda"))
        prompt = torch.zeros((B, V), dtype=torch.int32, device="cuda")
        prompt.scatter_(1, _tokens((B, 2000), V, g).long(), PROMPT)
        s.update(count=count | prompt, draft=_node_rows(case, _tokens((B, N), V, g)), mask=_node_rows(case, _pack_bits(sees)),
                 repetition=1.0 + 0.3 * torch.rand(B, generator=g, device="cuda"),
                 presence=0.5 * torch.rand(B, generator=g, device="cuda"),
                 frequency=0.2 * torch.rand(B, generator=g, device="cuda"))
    if case["bias"]:
        bias = 3.0 * torch.randn((B, V), generator=g, device="cuda")
        s["bias"] = bias * (torch.rand((B, V), generator=g, device="cuda") < 0.01)
    if case["grammar"]:
        # A grammar allows a sixteenth of the vocabulary, none in a row that it has closed; every third sequence has none.
        words = [torch.randint(-2 ** 31, 2 ** 31, (B, N, -(-V // 32)), generator=g, device="cuda") for _ in range(4)]
        allowed = (words[0] & words[1] & words[2] & words[3]).to(torch.int32)
        if B * N > 4:
            allowed[0, N // 2] = 0
        at = torch.arange(B * N, device="cuda", dtype=torch.int32).view(B, N)
        at[2::3] = -1
        s.update(allowed=allowed.view(B * N, -1), allowed_row=_node_rows(case, at))
    return s


def _prepare_count(case, g):
    B, N, V = case["B"], case["N"], case["V"]
    count = torch.zeros((B, V), dtype=torch.int32, device="cuda")
    count.scatter_add_(1, _tokens((B, 300), V, g).long(), torch.ones((B, 300), dtype=torch.int32, device="cuda"))
    count.scatter_(1, _tokens((B, 500), V, g).long(), PROMPT + 1)
    s = dict(count=count, token=_tokens((B, N), V, g), row=None, path=None, extra=None,
             length=_ints([max(1, N - 41 * b) for b in range(B)]))
    if case["kind"] == "beams":               # eight beams of a prompt, their parents among its old beams
        first = torch.arange(B, device="cuda") // 8 * 8
        pick = torch.randint(0, 8, (B,), generator=g, device="cuda")
        s["row"] = (first + pick).clamp(max=B - 1).to(torch.int32)
    if case["kind"] == "accepted":            # a verified path: the root, the accepted nodes, then the bonus token
        path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
        path[:, 0] = 0
        took = [(3 * b + 2) % min(N, 9) for b in range(B)]
        for b, n in enumerate(took):
            path[b, 1:n + 1] = (torch.randperm(N - 1, generator=g, device="cuda")[:n] + 1).sort().values.to(torch.int32)
        s.update(path=path, length=_ints(took), extra=_tokens((B,), V, g))
    s["out"] = count if case["kind"] == "prompt" else torch.empty_like(count)
    return s


# ----------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotate": _own_rotate, "shared": _own_shared, "adjust": _own_adjust, "count": _own_count}[op](state)
    return {"rotate": _plain_rotate, "shared": _plain_shared, "adjust": _plain_adjust, "count": _plain_count}[op](state)


def _split(s):
    """The projection's query, key and value heads, as views."""
    c = s["case"]
    x = s["qkv"].view(s["out"].shape[:-2] + (-1, c["D"]))
    return x.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=-2)


def _own_rotate(s):
    from tree_speculative_decoding_jf_gb300 import jf
    q, k, v = _split(s)
    out = jf.rotate_append_kv(
        q, k, v, s["k_cache"], s["v_cache"], s["block_table"], s["prefix_len"], pos=s["pos"], freq=s["freq"],
        interleaved=s["case"]["pairs"] == "interleaved", rotary_scale=s["rotary_scale"], q_norm=s["q_norm"],
        k_norm=s["k_norm"], norm_eps=1e-6, tree_len=s["tree_len"], cu_seqlens=s["cu_seqlens"], N_max=s["case"]["N"],
        out=s["out"])
    return {"q": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_shared(s):
    from tree_speculative_decoding_jf_gb300 import jf
    jf.tree_attention_shared(
        s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["prefix_len"], s["mask"], s["group_start"],
        s["shared_pages"], scale=s["scale"], tree_len=s["tree_len"], cu_seqlens=s["cu_seqlens"], N_max=s["case"]["N"],
        out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_adjust(s):
    from tree_speculative_decoding_jf_gb300 import jf
    return {"logits": jf.adjust_logits(
        s["logits"], count=s["count"], draft=s["draft"], mask=s["mask"], bias=s["bias"], allowed=s["allowed"],
        allowed_row=s["allowed_row"], repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
        tree_len=s["tree_len"], cu_seqlens=s["cu_seqlens"], N_max=s["case"]["N"], out=s["out"])}


def _own_count(s):
    from tree_speculative_decoding_jf_gb300 import jf
    return {"count": jf.count_tokens(s["count"], s["token"], path=s["path"], length=s["length"], extra=s["extra"],
                                     row=s["row"], prompt=s["case"]["kind"] == "prompt", out=s["out"])}


def _nodes(s):
    """Sequence and node of every real row, and its row in the per-node arrays."""
    c = s["case"]
    if c["layout"] == "packed":
        size = s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]
    else:
        size = s["tree_len"] if c["layout"] == "ragged" else torch.full((c["B"],), c["N"], device="cuda")
    b, i = torch.nonzero(torch.arange(c["N"], device="cuda") < size[:, None], as_tuple=True)
    row = s["cu_seqlens"][b].long() + i if c["layout"] == "packed" else b * c["N"] + i
    return b, i, row


def _plain_rotate(s):
    """x <- x / sqrt(mean(x^2) + eps) * w per head where there are weights; pair (x, y) of angle a = pos * freq ->
    scale * (x cos a - y sin a, y cos a + x sin a); then keys and values at slot P + node of their sequence."""
    c = s["case"]
    b, i, row = _nodes(s)
    q, k, v = (x.flatten(0, -3)[row] for x in _split(s))
    a = s["pos"].flatten()[row].double()[:, None] * s["freq"]
    cos, sin = ((f(a) * s["rotary_scale"]).float()[:, None] for f in (torch.cos, torch.sin))

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.float()
        x, rest = x[..., :c["R"]], x[..., c["R"]:]
        if c["pairs"] == "half":
            x0, x1 = x.chunk(2, -1)
            x = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
        else:
            x0, x1 = x[..., 0::2], x[..., 1::2]
            x = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
        return torch.cat([x, rest], -1).to(torch.bfloat16)

    s["out"].view(-1, c["Hq"], c["D"])[row] = turned(q, s["q_norm"])
    t = s["prefix_len"][b].long() + i
    page, slot = s["block_table"][b, t // PAGE].long(), t % PAGE
    s["k_cache"][page, slot] = turned(k, s["k_norm"])
    s["v_cache"][page, slot] = v
    return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_shared(s):
    """softmax(scale q.k) v over the cached tokens and the node's own branch, a few sequences at a time."""
    c = s["case"]
    B, N, Hq, Hkv, D = (c[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    cap = s["block_table"].shape[1] * PAGE
    at_b, at_i, row = _nodes(s)
    q = s["q"].new_zeros((B, N, Hq, D))
    q[at_b, at_i] = s["q"].view(-1, Hq, D)[row]
    out = torch.empty((B, N, Hq, D), device="cuda")
    lse = torch.empty((B, Hq, N), device="cuda")
    t = torch.arange(cap, device="cuda")
    step = max(1, (1 << 28) // (cap * max(Hkv * D, Hq * N)))
    for b0 in range(0, B, step):
        b1 = min(B, b0 + step)
        at = s["block_table"][b0:b1].long().clamp(min=0)
        k, v = (x[at].float().flatten(1, 2).permute(0, 2, 1, 3) for x in (s["k_cache"], s["v_cache"]))
        x = q[b0:b1].float().view(b1 - b0, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
        x = (x @ k.transpose(2, 3)).mul_(s["scale"])                           # [b, Hkv, N * G, cap]
        P = s["prefix_len"][b0:b1].long()[:, None]
        node = t - P
        mine = s["sees"][b0:b1].gather(2, node.clamp(0, N - 1)[:, None].expand(-1, N, -1))
        seen = (node < 0)[:, None] | (mine & (node < N)[:, None])
        x.masked_fill_(~seen[:, None].repeat_interleave(Hq // Hkv, 2), -math.inf)
        m = x.amax(-1, keepdim=True)
        x = x.sub_(m).exp_()
        z = x.sum(-1, keepdim=True)
        v = v.masked_fill((t >= P + N)[:, None, :, None], 0.0)
        o = (x @ v).div_(z).view(b1 - b0, Hkv, N, Hq // Hkv, D)
        out[b0:b1] = o.permute(0, 2, 1, 3, 4).flatten(2, 3)
        lse[b0:b1] = (m + z.log()).view(b1 - b0, Hkv, N, Hq // Hkv).permute(0, 1, 3, 2).flatten(1, 2)
    s["out"].view(-1, Hq, D)[row] = out[at_b, at_i].to(torch.bfloat16)
    if c["layout"] == "packed":
        s["lse"][:, row] = lse.transpose(0, 1)[:, at_b, at_i]
    else:
        s["lse"].transpose(1, 2)[at_b, at_i] = lse.transpose(1, 2)[at_b, at_i]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_adjust(s):
    """Per node: tokens of the prompt, the output or the node's branch lose x (x - 1/r or r), those of the output or the
    branch presence + frequency * times; then the bias; tokens that the grammar forbids become -inf."""
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    b, i, row = _nodes(s)
    x = s["logits"].view(-1, V)[row].float()
    if c["penalties"]:
        times = (s["count"] & (PROMPT - 1))[b]
        draft = torch.zeros((B, N), dtype=torch.int64, device="cuda")
        draft[b, i] = s["draft"].flatten()[row].long()
        branch = s["sees"][b, i].clone()
        branch[:, 0] = False
        r, j = torch.nonzero(branch, as_tuple=True)
        times.index_put_((r, draft[b[r], j]), torch.ones_like(r, dtype=torch.int32), accumulate=True)
        rep, pres, freq = (s[k][b][:, None] for k in ("repetition", "presence", "frequency"))
        x = torch.where((times > 0) | (s["count"] >= PROMPT)[b], torch.where(x > 0, x / rep, x * rep), x)
        x = x - torch.where(times > 0, pres + freq * times, 0.0)
    if c["bias"]:
        x = x + s["bias"][b]
    if c["grammar"]:
        at = s["allowed_row"].flatten()[row].long()
        bits = (s["allowed"][at.clamp(min=0)][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        ok = bits.flatten(1)[:, :V].bool() | (at < 0)[:, None]
        x = x.masked_fill(~ok, -math.inf)
    s["out"].view(-1, V)[row] = x.to(s["out"].dtype)
    return {"logits": s["out"]}


def _plain_count(s):
    """count_out[b] = count[row[b]] + 1 for every token (in the prompt: its flag)."""
    c = s["case"]
    B, V = c["B"], c["V"]
    out, n = s["out"], s["length"].long()[:, None]
    if c["kind"] != "prompt":
        out.copy_(s["count"] if s["row"] is None else s["count"][s["row"].long()])
    at = torch.arange(c["N"], device="cuda").expand(B, -1)
    if s["path"] is not None:
        token = s["token"].gather(1, s["path"].long().clamp(min=0))
        live = (at >= 1) & (at <= n)
        out.scatter_add_(1, s["extra"].long()[:, None], torch.ones((B, 1), dtype=torch.int32, device="cuda"))
    else:
        token, live = s["token"], at < n
    if c["kind"] == "prompt":
        flag = torch.zeros((B, V + 1), dtype=torch.bool, device="cuda")
        flag.scatter_(1, torch.where(live, token.long(), V), True)
        out |= flag[:, :V].to(torch.int32) * PROMPT
    else:
        out.scatter_add_(1, token.long(), live.to(torch.int32))
    return {"count": out}


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "count":
        return None                           # whole numbers: held to the plain form
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "shared": _exact_shared, "adjust": _exact_adjust}[case["op"]](case, s)


def _exact_rotate(case, s):
    Hq, Hkv, D, R = (case[k] for k in ("Hq", "Hkv", "D", "R"))
    out, kc, vc = s["out"].double(), s["k_cache"].double(), s["v_cache"].double()
    first = s["cu_seqlens"].tolist() if case["layout"] == "packed" else [b * case["N"] for b in range(case["B"])]
    half = torch.arange(R // 2, device="cuda")
    lo, hi = (half, half + R // 2) if case["pairs"] == "half" else (2 * half, 2 * half + 1)
    for b, n in enumerate(_sizes(case)):
        x = s["qkv"][first[b]:first[b] + n].double().view(n, Hq + 2 * Hkv, D)
        turn = torch.polar(torch.full((n, R // 2), s["rotary_scale"], dtype=torch.float64, device="cuda"),
                           torch.outer(s["pos"].view(-1)[first[b]:first[b] + n].double(), s["freq"]))
        for heads, w in ((slice(0, Hq), s["q_norm"]), (slice(Hq, Hq + Hkv), s["k_norm"])):
            y = x[:, heads]
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6) * w.double()
            z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None]
            y = y.clone()
            y[..., lo], y[..., hi] = z.real, z.imag
            x[:, heads] = y
        out.view(-1, Hq, D)[first[b]:first[b] + n] = x[:, :Hq]
        t = torch.arange(n, device="cuda") + int(s["prefix_len"][b])
        at = s["block_table"][b][t // PAGE].long() * PAGE + t % PAGE
        kc.view(-1, Hkv, D)[at] = x[:, Hq:Hq + Hkv]
        vc.view(-1, Hkv, D)[at] = x[:, Hq + Hkv:]
    return {"q": out, "k_cache": kc, "v_cache": vc}


def _exact_shared(case, s):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    G, sizes, lens = Hq // Hkv, _sizes(case), _shared_lengths(case)[1]
    if 4.0 * D * Hq * sum(n * (p + n) for n, p in zip(sizes, lens)) > 4e12:
        return None
    packed = case["layout"] == "packed"
    first = s["cu_seqlens"].tolist() if packed else [b * N for b in range(B)]
    rows = sum(sizes) if packed else B * N
    out = torch.zeros((rows, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, Hq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(sizes):
        L = lens[b] + n
        pages = s["block_table"][b, :-(-L // PAGE)].long()
        k, v = (x[pages].flatten(0, 1)[:L].double() for x in (s["k_cache"], s["v_cache"]))
        q = s["q"].reshape(-1, Hq, D)[first[b]:first[b] + n].double()
        hidden = torch.cat([torch.zeros((n, lens[b]), dtype=torch.bool, device="cuda"), ~s["sees"][b, :n, :n]], 1)
        for g in range(Hkv):
            e = torch.einsum("ihd,td->hit", q[:, g * G:(g + 1) * G], k[:, g]) * s["scale"]
            e = e.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(e, -1)
            lse[first[b]:first[b] + n, g * G:(g + 1) * G] = z.t()
            out[first[b]:first[b] + n, g * G:(g + 1) * G] = torch.einsum("hit,td->ihd", torch.exp(e - z[..., None]), v[:, g])
    if packed:
        return {"out": out, "lse": lse.t()}
    return {"out": out.view(B, N, Hq, D), "lse": lse.view(B, N, Hq).transpose(1, 2)}


def _exact_adjust(case, s):
    N, V = case["N"], case["V"]
    packed = case["layout"] == "packed"
    first = s["cu_seqlens"].tolist() if packed else [b * N for b in range(case["B"])]
    out = s["out"].double().view(-1, V)
    for b, n in enumerate(_sizes(case)):
        sees = s["sees"][b].tolist()
        for i in range(n):
            x = s["logits"].view(-1, V)[first[b] + i].double()
            if case["penalties"]:
                had = (s["count"][b] % PROMPT).double()
                branch = [j for j in range(1, i + 1) if sees[i][j]]
                if branch:
                    tokens = s["draft"].view(-1)[first[b]:first[b] + n][branch].long()
                    had += torch.bincount(tokens, minlength=V)
                rep = float(s["repetition"][b])
                scaled = torch.minimum(x / rep, x * rep) if rep >= 1 else torch.maximum(x / rep, x * rep)
                x = torch.where((had > 0) | (s["count"][b] >= PROMPT), scaled, x)
                x = x - had.clamp(max=1.0) * float(s["presence"][b]) - had * float(s["frequency"][b])
            if case["bias"]:
                x = x + s["bias"][b].double()
            if case["grammar"] and int(s["allowed_row"].view(-1)[first[b] + i]) >= 0:
                word = s["allowed"][int(s["allowed_row"].view(-1)[first[b] + i])].long()
                v = torch.arange(V, device="cuda")
                x[(word[v // 32] >> (v % 32)) % 2 == 0] = -math.inf
            out[first[b] + i] = x
    return {"logits": out.view(s["out"].shape)}


# ----------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "rotate":
        tokens, c = sum(_sizes(case)), case
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": tokens * (2 * heads * c["D"] * 2 + 4), "flops": tokens * (c["Hq"] + c["Hkv"]) * 3 * c["R"]}
    if op == "shared":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        sizes, start = _sizes(case), _groups(case)
        pages, lens = _shared_lengths(case)
        own_keys, pairs = 0, 0
        for u in range(case["groups"]):
            for b in range(start[u], start[u + 1]):
                own_keys += lens[b] - 16 * pages[u] + sizes[b]
                pairs += sizes[b] * (lens[b] + sizes[b])
        keys = 16 * sum(pages) + own_keys
        return {"bytes": keys * Hkv * D * 2 * 2 + sum(sizes) * Hq * (2 * D * 2 + 4), "flops": 4 * D * Hq * pairs}
    B, V = case["B"], case["V"]
    if op == "adjust":
        rows, size = sum(_sizes(case)), 2 if case["dtype"] == "bf16" else 4
        every = B * V * (4 * case["penalties"] + 4 * case["bias"])
        grammar = sum(n for b, n in enumerate(_sizes(case)) if b % 3 != 2) * (-(-V // 32)) * 4 if case["grammar"] else 0
        return {"bytes": rows * V * size * 2 + every + grammar, "flops": rows * V * 4}
    tokens = sum(max(1, case["N"] - 41 * b) for b in range(B)) if case["kind"] == "prompt" else B
    if case["kind"] == "prompt":
        return {"bytes": tokens * 4 * 3, "flops": 0}
    return {"bytes": 2 * B * V * 4 + tokens * 4, "flops": 0}
