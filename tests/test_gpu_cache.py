"""GPU parity of the bounded-cache calls (accumulated attention weight, kept positions,
eviction) with plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module")
def jf():
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf as mod
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def new_err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Pool:
    """A paged K (and V) pool: every sequence's pages in random order, NaN in every slot that
    no sequence's first `live` positions use, -1 in the table past a sequence's pages."""

    def __init__(self, rng, live, cap_pages, Hkv, D, spare=0):
        B = len(live)
        need = [-(-n // PAGE) for n in live]
        pages = sum(need) + spare + 3
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((B, cap_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.spare = order[at:at + spare]
        full = torch.full((pages, PAGE, Hkv, D), float("nan"), dtype=torch.bfloat16)
        self.k, self.v = full.clone(), full.clone()
        for b, n in enumerate(live):
            t = np.arange(n)
            for c in (self.k, self.v):
                c[self.table[b, t // PAGE], t % PAGE] = torch.from_numpy(
                    rng.standard_normal((n, Hkv, D)).astype(np.float32)).to(torch.bfloat16)


def weight_case(seed, prefix, rows, N, Hq, Hkv, D, path, cap_pages=None, dead_rows=()):
    """Inputs of one accumulate call and the expected output; rows[b] < 0 clears nothing but
    gives no rows.  The lse is the exact one of the rows' own keys, rounded to fp32."""
    rng = np.random.default_rng(seed)
    B, G, scale = len(prefix), Hq // Hkv, D ** -0.5
    cap_pages = cap_pages or max(1, max(-(-(p + max(r, 1)) // PAGE) for p, r in zip(prefix, rows)))
    pool = Pool(rng, [p + r for p, r in zip(prefix, rows)], cap_pages, Hkv, D)
    q = torch.from_numpy(rng.standard_normal((B, N, Hq, D)).astype(np.float32)).to(torch.bfloat16)
    qn, kn = q.double().numpy(), pool.k.double().numpy()
    cap = cap_pages * PAGE
    weight = rng.random((B, Hkv, cap)).astype(np.float32) * np.float32(0.01)
    before = np.full((B, Hkv, cap), -7.0, np.float32)
    lse = np.full((B, Hq, N), np.nan, np.float32)
    nodes, paths = [], np.full((B, N), -1, np.int32)
    for b in range(B):
        R = rows[b]
        ids = np.concatenate([[0], np.sort(rng.permutation(N - 1)[:R - 1]) + 1])[:R].astype(np.int64) \
            if path else np.arange(R)
        paths[b, :R] = ids
        nodes.append(ids)
        L = prefix[b] + R
        kk = ref.rows_of(kn, pool.table[b], np.arange(L)) if L else np.zeros((0, Hkv, D))
        for k, node in enumerate(ids):
            for h in range(Hq):
                s = scale * kk[:prefix[b] + k + 1, h // G] @ qn[b, node, h]
                m = s.max()
                lse[b, h, node] = m + np.log(np.exp(s - m).sum())
            if (b, k) in dead_rows:
                lse[b, :, node] = -np.inf
    want = np.empty((B, Hkv, cap))
    tol = np.empty((B, Hkv, cap))
    for b in range(B):
        want[b], tol[b] = ref.attention_weight(qn[b], kn, pool.table[b], prefix[b], nodes[b], lse[b], weight[b],
                                               before[b], scale)
    acc = np.array([r - 1 for r in rows], np.int32)
    return dict(pool=pool, q=q.cuda(), lse=dev(lse), weight=dev(weight), out=dev(before), want=want, tol=tol,
                path=dev(paths) if path else None, accept_len=dev(acc), prefix=dev(np.array(prefix, np.int32)),
                table=dev(pool.table), k=pool.k.cuda(), scale=scale, rows=rows, paths=paths)


def close(got, want, tol):
    g = got.cpu().numpy().astype(np.float64)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5].tolist(), g[bad][:5], want[bad][:5], tol[bad][:5])


CASES = [
    # prefix lengths, rows, N, Hq, Hkv, D, path
    ([2048], [5], 16, 32, 8, 128, True),
    ([0], [1], 1, 4, 1, 64, False),                        # a first token
    ([1], [1], 1, 4, 4, 128, False),                       # G = 1
    ([130, 0, 15, 16, 700], [3, 1, 0, 9, 17], 20, 8, 2, 64, True),
    ([127, 128, 129, 1000], [1, 2, 1, 40], 40, 12, 4, 128, True),     # G = 3
    ([300, 5], [64, 64], 64, 14, 2, 128, False),           # G = 7, 448 rows a kv-head
    ([37, 513], [200, 200], 200, 8, 1, 64, False),         # 1600 rows a kv-head, window from the start
    ([900], [33], 256, 40, 8, 128, True),                  # G = 5
    ([4000, 77], [129, 1], 256, 16, 1, 128, True),         # G = 16, 2064 rows
    ([31], [300], 300, 2, 2, 128, False),                  # G = 1, long window over a short prefix
    ([260] * 9, [4] * 9, 8, 4, 2, 64, True),
    ([20, 0, 3], [0, 0, 0], 4, 4, 2, 128, True),           # nothing accepted anywhere
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_weight_matches_reference(jf, case):
    prefix, rows, N, Hq, Hkv, D, path = CASES[case]
    c = weight_case(case, prefix, rows, N, Hq, Hkv, D, path)
    err = new_err()
    full = not path and all(r == N for r in rows)
    got = jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], c["lse"], path=c["path"],
                                         accept_len=None if full else c["accept_len"], weight=c["weight"],
                                         scale=c["scale"], out=c["out"], dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    close(got, c["want"], c["tol"])


@pytest.mark.parametrize("D,G", [(64, 4), (128, 8), (128, 3)])
def test_weight_long_cache(jf, D, G):
    """More key tiles than CTAs of one wave, ragged, with a capacity past the live keys."""
    prefix, rows = [20011, 1, 9000], [6, 2, 11]
    c = weight_case(50 + D + G, prefix, rows, 12, G * 2, 2, D, True, cap_pages=1300)
    err = new_err()
    jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], c["lse"], path=c["path"],
                                   accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"], out=c["out"],
                                   dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    close(c["out"], c["want"], c["tol"])


def test_weight_rows_that_attended_to_nothing(jf):
    c = weight_case(3, [100, 40], [5, 3], 8, 8, 2, 64, True, dead_rows={(0, 1), (1, 0), (1, 1), (1, 2)})
    got = jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], c["lse"], path=c["path"],
                                         accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"],
                                         out=c["out"])
    close(got, c["want"], c["tol"])


def test_weight_from_zero_in_place_and_repeatable(jf):
    c = weight_case(4, [333, 64], [7, 2], 9, 8, 2, 128, True)
    args = (c["q"], c["k"], c["table"], c["prefix"], c["lse"])
    kw = dict(path=c["path"], accept_len=c["accept_len"], scale=c["scale"])
    zero = jf.accumulate_attention_weight(*args, **kw)
    a = jf.accumulate_attention_weight(*args, weight=c["weight"], **kw)
    b = jf.accumulate_attention_weight(*args, weight=c["weight"], **kw)
    assert torch.equal(a, b)
    w = c["weight"].clone()
    jf.accumulate_attention_weight(*args, weight=w, out=w, **kw)
    for s, (P, R) in enumerate(zip([333, 64], [7, 2])):
        assert torch.equal(w[s, :, :P + R], a[s, :, :P + R])
        assert torch.equal(w[s, :, P + R:], c["weight"][s, :, P + R:])
        assert (zero[s, :, P + R:] == 0).all()
        close(zero[s, :, :P + R], c["want"][s, :, :P + R] - np.where(
            np.arange(P + R) < P, c["weight"][s, :, :P + R].cpu().numpy().astype(np.float64), 0.0),
            c["tol"][s, :, :P + R] + 2.0 ** -23)


@pytest.mark.parametrize("seed,D,G", [(0, 64, 4), (1, 128, 8), (2, 128, 6)])
def test_weight_packed_equals_padded(jf, seed, D, G):
    """Packed rows give the padded call's bits."""
    sizes, prefix, rows, N = [5, 40, 1, 17], [100, 3, 700, 0], [2, 30, 1, 0], 40
    c = weight_case(seed + 20, prefix, rows, N, G * 2, 2, D, True)
    for b, n in enumerate(sizes):                          # paths inside each tree's own nodes
        ids = np.arange(rows[b])
        c["paths"][b] = -1
        c["paths"][b, :rows[b]] = ids
    path = dev(c["paths"])
    lse = torch.nan_to_num(c["lse"], nan=3.0)
    kw = dict(path=path, accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"])
    pad = jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], lse, **kw)
    at = torch.cat([torch.arange(n) + b * N for b, n in enumerate(sizes)]).cuda()
    qp = c["q"].flatten(0, 1)[at].contiguous()
    lp = lse.transpose(0, 1).flatten(1)[:, at].contiguous()
    cu = dev(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32))
    err = new_err()
    got = jf.accumulate_attention_weight(qp, c["k"], c["table"], c["prefix"], lp, cu_seqlens=cu, dev_err=err, **kw)
    assert torch.equal(got, pad) and err.item() == 0
    # every node a row: spans are the row counts
    cu2 = dev(np.array([0, 5, 5, 6, 23], np.int32))        # the second span is empty: bad
    err = new_err()
    pool = c["pool"]
    got = jf.accumulate_attention_weight(qp, c["k"], c["table"], dev(np.zeros(4, np.int32)), lp, cu_seqlens=cu2,
                                         scale=c["scale"], path=None, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() & jf.DEVERR_BAD_TREE_LEN
    assert (got[1] == 0).all() and pool is c["pool"]


def test_weight_reports_bad_input_and_stays_in_bounds(jf):
    c = weight_case(8, [100, 50, 60, 30], [3, 3, 3, 3], 6, 4, 2, 64, True, cap_pages=7)
    for what, bit in (("prefix", jf.DEVERR_BAD_PREFIX), ("neg", jf.DEVERR_BAD_PREFIX), ("acc", jf.DEVERR_BAD_PATH),
                      ("path", jf.DEVERR_BAD_PATH), ("page", jf.DEVERR_BAD_PAGE), ("page2", jf.DEVERR_BAD_PAGE)):
        prefix, acc, path, table = (c[k].clone() for k in ("prefix", "accept_len", "path", "table"))
        if what == "prefix":
            prefix[1] = 7 * 16 - 1
        elif what == "neg":
            prefix[1] = -5
        elif what == "acc":
            acc[1] = 6
        elif what == "path":
            path[1, 1] = 6
        else:
            table[1, 1] = -1 if what == "page" else c["k"].shape[0]
        err, out = new_err(), c["out"].clone()
        jf.accumulate_attention_weight(c["q"], c["k"], table, prefix, c["lse"], path=path, accept_len=acc,
                                       weight=c["weight"], scale=c["scale"], out=out, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() & bit, what
        for b in (0, 2, 3):                                # the other sequences are as without it
            close(out[b], c["want"][b], c["tol"][b])


def test_weight_on_another_stream_and_in_a_graph(jf):
    c = weight_case(9, [1000, 1500], [4, 2], 8, 8, 2, 128, True)
    args = (c["q"], c["k"], c["table"], c["prefix"], c["lse"])
    kw = dict(path=c["path"], accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"])
    want = jf.accumulate_attention_weight(*args, out=c["out"].clone(), **kw)
    s = torch.cuda.Stream()
    out = c["out"].clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        jf.accumulate_attention_weight(*args, out=out, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want)
    out.fill_(-7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jf.accumulate_attention_weight(*args, out=out, **kw)
    for _ in range(2):
        out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_calls_on_a_given_stream(jf):
    """stream= instead of the current stream, for every call of the cache."""
    c = weight_case(11, [500, 300], [4, 2], 8, 8, 2, 64, True)
    kw = dict(path=c["path"], accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"])
    args = (c["q"], c["k"], c["table"], c["prefix"], c["lse"])
    want_w = jf.accumulate_attention_weight(*args, out=c["out"].clone(), **kw)
    lens = c["prefix"] + c["accept_len"] + 1
    want_keep, want_len = jf.select_kept_keys(want_w, lens, 100, sink=1, recent=5)
    k1, v1 = c["k"].clone(), c["k"].clone()
    jf.evict_kv(k1, v1, c["table"], lens, want_keep, want_len, weight=want_w.clone())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, k2, v2 = c["out"].clone(), c["k"].clone(), c["k"].clone()
    keep, kept = torch.empty_like(want_keep), torch.empty_like(want_len)
    torch.cuda.synchronize()
    jf.accumulate_attention_weight(*args, out=out, stream=s, **kw)
    jf.jf_select_kept(out, lens, keep, kept, 1, 5, stream=s)
    jf.evict_kv(k2, v2, c["table"], lens, keep, kept, stream=s)
    s.synchronize()
    assert torch.equal(out, want_w) and torch.equal(keep, want_keep) and torch.equal(kept, want_len)
    assert torch.equal(k1.view(torch.int16), k2.view(torch.int16)) and torch.equal(v1.view(torch.int16), v2.view(torch.int16))


def test_tensors_of_a_call_on_a_given_stream(jf):
    """What a call makes for itself is made on its stream: a busy current stream neither clears
    the result late nor loses the contents of memory that it still reads."""
    c = weight_case(12, [500, 300], [4, 2], 8, 8, 2, 64, True)
    kw = dict(path=c["path"], accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"])
    args = (c["q"], c["k"], c["table"], c["prefix"], c["lse"])
    want = jf.accumulate_attention_weight(*args, **kw)
    lens = c["prefix"] + c["accept_len"] + 1
    want_keep, want_len = jf.select_kept_keys(want, lens, 100, sink=1, recent=5)
    logits, score = torch.randn(2, 3, 4000, device="cuda"), torch.zeros(2, 3, device="cuda")
    want_beams = jf.beam_select(logits, score, 5)
    fresh = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    table = torch.arange(10, 28, dtype=torch.int32, device="cuda").view(6, 3)
    cache = [torch.randn(28, 16, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2)]
    plen = torch.full((6,), 20, dtype=torch.int32, device="cuda")
    want_fork = jf.beam_fork_kv(*(x.clone() for x in cache), table, plen, want_beams[0], fresh)
    s = torch.cuda.Stream()

    def check(call, wants):
        """call(), with the current stream asleep before it reads tensors like call's."""
        held = [torch.full_like(w, 3) for w in wants for _ in range(4)]
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        copies = [h.clone() for h in held]
        del held                               # its memory is free to the current stream
        got = call()
        s.synchronize()
        torch.cuda.synchronize()
        for g, w in zip(got, wants):
            assert torch.equal(g, w)
        for x in copies:
            assert (x == 3).all()

    check(lambda: [jf.accumulate_attention_weight(*args, stream=s, **kw)], [want])
    check(lambda: jf.select_kept_keys(want, lens, 100, sink=1, recent=5, stream=s), [want_keep, want_len])
    check(lambda: jf.beam_select(logits, score, 5, stream=s), list(want_beams))
    check(lambda: jf.beam_select(logits, score, 5, stream=s.cuda_stream), list(want_beams))
    check(lambda: jf.beam_fork_kv(*cache, table, plen, want_beams[0], fresh, stream=s), list(want_fork))
    got = jf.select_kept_keys(want, lens, 100, sink=1, recent=5, stream=0)   # the default stream
    torch.cuda.synchronize()
    assert torch.equal(got[0], want_keep) and torch.equal(got[1], want_len)


@pytest.mark.parametrize("prefix,rows,N,Hq,Hkv,D,path", [
    ([200, 70], [5, 3], 8, 12, 4, 64, True),               # G = 3: rows do not fill 32 columns
    ([300], [45], 64, 6, 2, 128, False),                   # 135 rows: a full block of 126 and a rest
    ([130, 9], [1, 1], 1, 8, 2, 128, False),               # one token
])
def test_weight_of_keys_with_infinities(jf, prefix, rows, N, Hq, Hkv, D, path):
    """A cached key whose scores are all -inf receives nothing: its weight and the others' stay
    what they are without it."""
    c = weight_case(31, prefix, rows, N, Hq, Hkv, D, path)
    c["q"][..., 5] = c["q"][..., 5].abs() + 0.25            # (the lse is an input like any other)
    lse = torch.full_like(c["lse"], 6.0)
    k = c["k"].clone()
    at = [(b, t) for b, P in enumerate(prefix) for t in (0, P // 2, P - 1)]
    for b, t in at:
        k[c["table"][b, t // PAGE].long(), t % PAGE, :, 5] = -float("inf")
    got = jf.accumulate_attention_weight(c["q"], k, c["table"], c["prefix"], lse, path=c["path"],
                                         accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"],
                                         out=c["out"].clone())
    plain = jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], lse, path=c["path"],
                                           accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"],
                                           out=c["out"].clone())
    want = plain.clone()
    for b, t in at:
        want[b, :, t] = c["weight"][b, :, t]
    assert torch.equal(got, want)
    # +inf with these lse is an infinite weight for the rows that see the key, and for no other key
    b, t = len(prefix) - 1, prefix[-1] // 2
    k = c["k"].clone()
    k[c["table"][b, t // PAGE].long(), t % PAGE, :, 5] = float("inf")
    got = jf.accumulate_attention_weight(c["q"], k, c["table"], c["prefix"], lse, path=c["path"],
                                         accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"],
                                         out=c["out"].clone())
    assert torch.isposinf(got[b, :, t]).all()
    plain[b, :, t] = float("inf")
    assert torch.equal(got, plain)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (12, 4, 128), (4, 4, 128)])
def test_weight_where_dead_rows_alone_see_nan(jf, Hq, Hkv, D):
    """Keys (NaN here) that only rows with an lse of -inf see keep their weight: a padded
    sequence whose rows attended to nothing, and the later rows of another."""
    prefix, rows = [90, 40, 0], [6, 4, 2]
    dead = {(0, 4), (0, 5)} | {(b, k) for b in (1, 2) for k in range(4)}
    c = weight_case(32, prefix, rows, 8, Hq, Hkv, D, True, dead_rows=dead)
    k = c["k"].clone()
    seen = [(0, 94), (0, 95)] + [(1, t) for t in range(44)] + [(2, 0), (2, 1)]
    for b, t in seen:
        k[c["table"][b, t // PAGE].long(), t % PAGE] = float("nan")
    c["q"][1, c["path"][1, 2].long()] = float("nan")       # a dead row's query may hold anything
    got = jf.accumulate_attention_weight(c["q"], k, c["table"], c["prefix"], c["lse"], path=c["path"],
                                         accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"],
                                         out=c["out"])
    close(got, c["want"], c["tol"])
    for b, t in seen:
        assert torch.equal(got[b, :, t], c["weight"][b, :, t] if t < prefix[b] else torch.zeros(Hkv, device="cuda"))


def test_weight_of_nan_keys_is_nan(jf):
    """A NaN key that a live row sees is a NaN weight, at its own position alone."""
    c = weight_case(33, [300], [5], 8, 12, 4, 128, True)
    k = c["k"].clone()
    k[c["table"][0, 130 // PAGE].long(), 130 % PAGE, 1, 7] = float("nan")
    got = jf.accumulate_attention_weight(c["q"], k, c["table"], c["prefix"], c["lse"], path=c["path"],
                                         accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"],
                                         out=c["out"])
    want, tol = c["want"].copy(), c["tol"]
    assert torch.isnan(got[0, 1, 130])
    got[0, 1, 130] = want[0, 1, 130] = 0.0
    close(got, want, tol)


# ------------------------------------------------------------------------------- kept positions

def run_select(jf, w, L, budget, sink, recent):
    err = new_err()
    keep, kept = jf.select_kept_keys(dev(w), dev(np.array(L, np.int32)), budget, sink=sink, recent=recent, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    want, want_len = ref.select_kept(w, np.array(L, np.int32), sink, recent, budget)
    assert (kept.cpu().numpy() == want_len).all()
    assert (keep.cpu().numpy() == want).all()


@pytest.mark.parametrize("L,budget,sink,recent", [
    ([2304], 2048, 4, 64), ([1, 0, 16, 500], 16, 0, 0), ([33, 100], 1, 0, 0), ([33, 100], 1, 1, 0),
    ([33, 100], 1, 0, 1), ([700, 701], 20, 10, 10), ([700, 300], 699, 3, 5), ([4097, 513, 512, 511], 500, 4, 32),
    ([9000, 8193, 20000], 3000, 2, 100),
])
@pytest.mark.parametrize("kind", ["weights", "ties"])
def test_select_matches_reference(jf, L, budget, sink, recent, kind):
    rng = np.random.default_rng(len(L) * 1000 + budget)
    w = np.exp(1.5 * rng.standard_normal((len(L), 3, -(-max(L) // PAGE) * PAGE + PAGE))).astype(np.float32)
    if kind == "ties":
        w = np.floor(w).astype(np.float32)
    run_select(jf, w, L, budget, sink, recent)


def test_select_special_values(jf):
    """NaN below -inf, -0 equal to +0, infinities, one value everywhere, ordered rows."""
    rng = np.random.default_rng(1)
    n = 1000
    rows = [np.zeros(n), np.where(rng.random(n) < 0.5, -0.0, 0.0), np.full(n, np.nan),
            rng.choice([np.nan, -np.inf, np.inf, 0.0, -1.0, 1.0, 1e-45, -1e-45], n), np.arange(n) * 1.0,
            -np.arange(n) * 1.0, np.full(n, -np.inf), rng.standard_normal(n) * 1e38]
    w = np.array(rows, np.float32)[None].repeat(2, 0)
    w = np.pad(w, ((0, 0), (0, 0), (0, 8)))
    for budget, sink, recent in ((400, 5, 7), (1, 0, 0), (999, 0, 0), (12, 5, 7)):
        run_select(jf, w, [n, n - 3], budget, sink, recent)


@pytest.mark.parametrize("cap", [1003, 4097, 333])
def test_select_rows_off_sixteen_bytes(jf, cap):
    """Rows that start at any 4-byte offset, and a tensor that does."""
    rng = np.random.default_rng(cap)
    w = rng.standard_normal((3, 5, cap)).astype(np.float32)
    run_select(jf, w, [cap, cap - 1, cap // 2], cap // 3, 3, 9)
    flat = torch.zeros(w.size + 1, device="cuda")
    view = flat[1:].view(w.shape)
    view.copy_(dev(w))
    L = np.array([cap, cap - 2, 7], np.int32)
    keep, kept = jf.select_kept_keys(view, dev(L), 40, sink=1, recent=2)
    want, want_len = ref.select_kept(w, L, 1, 2, 40)
    assert (keep.cpu().numpy() == want).all() and (kept.cpu().numpy() == want_len).all()


@pytest.mark.parametrize("rows", [80, 200])
def test_select_many_rows(jf, rows):
    """A row a CTA, short and longer than one CTA holds."""
    rng = np.random.default_rng(rows)
    w = np.exp(rng.standard_normal((rows // 4, 4, 3000 if rows == 80 else 40000))).astype(np.float32)
    n = w.shape[2]
    if rows == 200:                            # (the reference sorts every row: a few of them)
        w[1:] = w[:1]
        L = np.full(rows // 4, n, np.int32)
        keep, _ = jf.select_kept_keys(dev(w), dev(L), 7000, sink=2, recent=30)
        want, _ = ref.select_kept(w[:1], L[:1], 2, 30, 7000)
        assert (keep.cpu().numpy() == want).all()
    else:
        run_select(jf, w, [n - 100 * i for i in range(rows // 4)], 700, 2, 30)


@pytest.mark.parametrize("rows", [1, 40])
def test_select_long_rows(jf, rows):
    """Rows longer than a cluster holds at once, and clusters of every size."""
    rng = np.random.default_rng(rows)
    w = rng.random((rows, 1, 80000 if rows == 1 else 17008)).astype(np.float32)
    L = [79999] if rows == 1 else [17008 - 400 * i for i in range(rows)]
    run_select(jf, w, L, 30000 if rows == 1 else 5000, 4, 100)
    w[:] = np.floor(w * 3)
    run_select(jf, w, L, 30000 if rows == 1 else 5000, 4, 100)


@pytest.mark.parametrize("kind", ["weights", "few values", "one value"])
def test_select_rows_past_shared_memory(jf, kind):
    """Slices that a cluster of eight cannot hold on chip."""
    rng = np.random.default_rng(2)
    n = 450000
    w = rng.standard_normal((2, 1, n)).astype(np.float32)
    if kind != "weights":
        w = np.floor(w * 2) if kind == "few values" else np.zeros_like(w)
    err = new_err()
    L = np.array([n, 300], np.int32)
    keep, kept = jf.select_kept_keys(dev(w), dev(L), 100000, sink=3, recent=50, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and kept.tolist() == [100000, 300]
    mid = w[0, 0, 3:n - 50]
    order = np.lexsort((np.arange(len(mid)), -mid.astype(np.float64)))[:100000 - 53] + 3
    want = np.sort(np.concatenate([np.arange(3), order, np.arange(n - 50, n)]))
    assert (keep[0, 0].cpu().numpy() == want).all()
    assert (keep[1, 0, :300].cpu().numpy() == np.arange(300)).all() and (keep[1, 0, 300:] == -1).all()


@pytest.mark.parametrize("rows,n", [(1, 300000), (1, 393216), (80, 300000), (80, 400000)])
@pytest.mark.parametrize("kind", ["weights", "few values"])
def test_select_the_longest_slices(jf, rows, n, kind):
    """Slices at and past what fits on chip, for few rows and for many."""
    rng = np.random.default_rng(n + rows)
    w = rng.standard_normal(n).astype(np.float32)
    if kind == "few values":
        w = np.floor(w * 2)
    budget, sink, recent = 100000, 3, 50
    err = new_err()
    keep, kept = jf.select_kept_keys(dev(w).expand(rows, 1, n).contiguous(), dev(np.full(rows, n, np.int32)),
                                     budget, sink=sink, recent=recent, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and (kept == budget).all()
    mid = w[sink:n - recent].astype(np.float64)
    order = np.lexsort((np.arange(len(mid)), -mid))[:budget - sink - recent] + sink
    want = np.sort(np.concatenate([np.arange(sink), order, np.arange(n - recent, n)]))
    assert (keep.cpu().numpy() == want).all()


@pytest.mark.parametrize("n", [8192, 8193, 20480, 20481, 32768, 32769, 65536, 81921])
@pytest.mark.parametrize("rows", [1, 200])
def test_select_at_the_borders_of_the_forms(jf, rows, n):
    """The longest rows that each form takes, and one key more, for few rows and for many."""
    rng = np.random.default_rng(n)
    w = np.exp(2 * rng.standard_normal(n)).astype(np.float32)
    cap = (n + 15) // 16 * 16
    full = torch.zeros(rows, 1, cap, device="cuda")
    full[:, 0, :n] = dev(w)
    keep, kept = jf.select_kept_keys(full, dev(np.full(rows, n, np.int32)), n // 3, sink=4, recent=37)
    want, _ = ref.select_kept(w[None, None], np.array([n], np.int32), 4, 37, n // 3)
    assert (kept == n // 3).all() and (keep.cpu().numpy() == want).all()


@pytest.mark.parametrize("rows", [1, 80])
@pytest.mark.parametrize("equal", [1, 255, 256, 257, 2000])
def test_select_equal_keys_at_the_border(jf, rows, equal):
    """`equal` keys of one value, of which some stay, around the number that is listed."""
    rng = np.random.default_rng(equal)
    n = 20000
    w = rng.random(n) + 2.0
    w[rng.permutation(n)[:n // 2]] -= 2.0      # below 1
    at = rng.permutation(n)[:equal]
    w[at] = 1.5
    w = w.astype(np.float32)
    above = int((w > 1.5).sum())
    for b in {above + 1, above + (equal + 1) // 2, above + equal}:
        keep, _ = jf.select_kept_keys(dev(w).expand(rows, 1, n).contiguous(), dev(np.full(rows, n, np.int32)), b)
        want, _ = ref.select_kept(w[None, None], np.array([n], np.int32), 0, 0, b)
        assert (keep.cpu().numpy() == want).all()


def test_select_clamps_lengths(jf):
    w = np.random.default_rng(0).random((2, 2, 64)).astype(np.float32)
    err = new_err()
    keep, kept = jf.select_kept_keys(dev(w), dev(np.array([-3, 70], np.int32)), 8, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() & jf.DEVERR_BAD_PREFIX
    assert kept.tolist() == [0, 8] and (keep[0] == -1).all() and keep[1].max().item() < 64


# ------------------------------------------------------------------------------------ eviction

def evict_case(seed, lens, budget, Hkv, D, out_of_place, kind="random", weights=True):
    rng = np.random.default_rng(seed)
    B, cap_pages = len(lens), max(1, -(-max(max(lens), budget) // PAGE))
    per = -(-min(budget, max(lens)) // PAGE)
    pool = Pool(rng, lens, cap_pages, Hkv, D, spare=per * B if out_of_place else 0)
    new_table = pool.table
    if out_of_place:
        new_table = np.full((B, cap_pages), -1, np.int32)
        new_table[:, :per] = pool.spare.reshape(B, per)
    keep = np.full((B, Hkv, budget), -1, np.int32)
    kept = np.minimum(lens, budget).astype(np.int32)
    for b, L in enumerate(lens):
        for g in range(Hkv):
            n = int(kept[b])
            keep[b, g, :n] = {"random": np.sort(rng.permutation(L)[:n]), "last": np.arange(L - n, L),
                              "first": np.arange(n)}[kind]
    weight = rng.random((B, Hkv, cap_pages * PAGE)).astype(np.float32) if weights else None
    return pool, new_table, keep, kept, weight


@pytest.mark.parametrize("lens,budget,Hkv,D,kind", [
    ([2304], 2048, 8, 128, "random"), ([2304], 2048, 8, 128, "last"), ([100, 7, 0, 16], 20, 2, 64, "random"),
    ([500, 333], 120, 3, 128, "random"), ([3000, 2999], 2990, 1, 64, "last"), ([64, 65], 64, 2, 128, "first"),
    ([33], 1, 1, 64, "last"), ([5000, 1, 4096], 1000, 4, 128, "random"), ([40], 64, 2, 64, "random"),
])
@pytest.mark.parametrize("out_of_place", [False, True])
def test_evict_matches_reference(jf, lens, budget, Hkv, D, kind, out_of_place):
    pool, new_table, keep, kept, weight = evict_case(budget, lens, budget, Hkv, D, out_of_place, kind)
    bits = lambda t: t.view(torch.int16).numpy()   # noqa: E731
    rk, rv, rw = ref.evict_kv(bits(pool.k), bits(pool.v), pool.table, new_table, keep, kept, weight)
    k, v, w, err = pool.k.cuda(), pool.v.cuda(), dev(weight), new_err()
    got = jf.evict_kv(k, v, dev(pool.table), dev(np.array(lens, np.int32)), dev(keep), dev(kept),
                      new_block_table=dev(new_table) if out_of_place else None, weight=w, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and (got.cpu().numpy() == kept).all()
    assert (bits(k.cpu()) == rk).all() and (bits(v.cpu()) == rv).all()
    assert (w.cpu().numpy() == rw).all()


def test_evict_weights_to_another_array_or_none(jf):
    pool, table, keep, kept, weight = evict_case(2, [300, 200], 100, 2, 64, False)
    bits = lambda t: t.view(torch.int16).numpy()   # noqa: E731
    rk, _, rw = ref.evict_kv(bits(pool.k), bits(pool.v), table, table, keep, kept, weight)
    for with_weight in (True, False):
        k, v, out = pool.k.cuda(), pool.v.cuda(), torch.full(weight.shape, -3.0, device="cuda")
        jf.evict_kv(k, v, dev(table), dev(np.array([300, 200], np.int32)), dev(keep), dev(kept),
                    weight=dev(weight) if with_weight else None, weight_out=out if with_weight else None)
        torch.cuda.synchronize()
        assert (bits(k.cpu()) == rk).all()
        if with_weight:
            assert (out[..., :100].cpu().numpy() == rw[..., :100]).all() and (out[..., 100:] == -3.0).all()


def test_evict_reports_bad_input_and_stays_in_bounds(jf):
    pool, table, keep, kept, weight = evict_case(5, [300, 200], 100, 2, 64, False)
    L = np.array([300, 200], np.int32)
    bits = lambda t: t.view(torch.int16).numpy()   # noqa: E731
    rk, rv, rw = ref.evict_kv(bits(pool.k), bits(pool.v), table, table, keep, kept, weight)
    for what, bit in (("order", jf.DEVERR_BAD_PATH), ("past", jf.DEVERR_BAD_PATH), ("low", jf.DEVERR_BAD_PATH),
                      ("kept", jf.DEVERR_BAD_PATH), ("len", jf.DEVERR_BAD_PREFIX), ("page", jf.DEVERR_BAD_PAGE)):
        kp, kl, sl, tb = keep.copy(), kept.copy(), L.copy(), table.copy()
        if what == "order":
            kp[1, 0, 50] = kp[1, 0, 49]
        elif what == "past":
            kp[1, 0, 99] = 200
        elif what == "low":
            kp[1, 1, 0] = -1
        elif what == "kept":
            kl[1] = 101
        elif what == "len":
            sl[1] = -1
        else:
            tb[1, 12] = pool.k.shape[0] + 5
            kp[1, :, 99] = 199
        k, v, w, err = pool.k.cuda(), pool.v.cuda(), dev(weight), new_err()
        jf.evict_kv(k, v, dev(tb), dev(sl), dev(kp), dev(kl), weight=w, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() & bit, what
        own = table[0][table[0] >= 0]
        assert (bits(k.cpu())[own] == rk[own]).all() and (w[0].cpu().numpy() == rw[0]).all()
        other = np.setdiff1d(np.arange(pool.k.shape[0]), table[table >= 0])
        assert (bits(v.cpu())[other] == bits(pool.v)[other]).all()


def test_pages_past_four_gigabytes(jf):
    """Page ids whose byte offsets pass 32 bits, in every call that reads or moves pages."""
    Hkv, D, pages = 8, 128, 140000                          # 16 KB pages of one head set: 4.6 GB a pool
    k = torch.zeros((pages, PAGE, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    rng = np.random.default_rng(0)
    table = np.array([[139999, 3, 139990, 131072]], np.int32)
    P, R, N = 50, 2, 2
    t = np.arange(P + R)
    new = torch.from_numpy(rng.standard_normal((2, P + R, Hkv, D)).astype(np.float32)).to(torch.bfloat16)
    idx = dev(table[0][t // PAGE].astype(np.int64)), dev(t % PAGE)
    k[idx], v[idx] = new[0].cuda(), new[1].cuda()
    q = torch.from_numpy(rng.standard_normal((1, N, 16, D)).astype(np.float32)).to(torch.bfloat16)
    lse = rng.random((1, 16, N)).astype(np.float32) + 4
    small = np.zeros((4, PAGE, Hkv, D))
    small.reshape(-1, Hkv, D)[:P + R] = new[0].double().numpy()
    want, tol = ref.attention_weight(q[0].double().numpy(), small, np.arange(4), P, np.arange(R), lse[0], None,
                                     np.zeros((Hkv, 64)), D ** -0.5)
    err = new_err()
    got = jf.accumulate_attention_weight(q.cuda(), k, dev(table), dev(np.array([P], np.int32)), dev(lse), dev_err=err)
    close(got[0], want, tol)
    keep, kept = jf.select_kept_keys(got, dev(np.array([P + R], np.int32)), 20)
    jf.evict_kv(k, v, dev(table), dev(np.array([P + R], np.int32)), keep, kept, weight=got, dev_err=err)
    torch.cuda.synchronize()
    kp = keep[0].cpu().numpy()
    for g in range(Hkv):
        for j in range(20):
            assert torch.equal(k[table[0, j // PAGE], j % PAGE, g].cpu(), new[0][kp[g, j], g])
            assert torch.equal(v[table[0, j // PAGE], j % PAGE, g].cpu(), new[1][kp[g, j], g])
    fresh = torch.tensor([[139000, 138000]], dtype=torch.int32, device="cuda")
    nt, nl = jf.beam_fork_kv(k, v, dev(table), dev(np.array([20], np.int32)), torch.zeros((1, 2), dtype=torch.int32,
                             device="cuda"), fresh, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and nl.tolist() == [20, 20]
    assert nt.tolist() == [[139999, 139000, -1, -1], [139999, 138000, -1, -1]]
    assert torch.equal(k[139000, :4], k[3, :4]) and torch.equal(v[138000, :4], v[3, :4])


# ------------------------------------------------------------------- shapes and layouts of the weight

@pytest.mark.parametrize("Hq,Hkv,D,prefix,sizes", [
    (32, 8, 128, [200, 0, 77], [75, 3, 130]),              # 32 rows a block: two and four full ones and rests
    (12, 4, 64, [131, 40, 9], [100, 1, 87]),               # 42 rows a block
    (40, 8, 128, [16, 300], [51, 52]),                     # 25 rows a block
    (8, 8, 64, [5, 128], [300, 129]),                      # 128 rows a block
])
def test_weight_packed_rows_without_a_path(jf, Hq, Hkv, D, prefix, sizes):
    """Every packed row counts: full blocks of rows at offsets that are no multiple of a block."""
    c = weight_case(60 + Hq, prefix, sizes, max(sizes), Hq, Hkv, D, False)
    at = torch.cat([torch.arange(n) + b * max(sizes) for b, n in enumerate(sizes)]).cuda()
    q = c["q"].flatten(0, 1)[at].contiguous()
    lse = c["lse"].transpose(0, 1).flatten(1)[:, at].contiguous()
    cu, err = dev(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)), new_err()
    got = jf.accumulate_attention_weight(q, c["k"], c["table"], c["prefix"], lse, cu_seqlens=cu, weight=c["weight"],
                                         scale=c["scale"], out=c["out"], dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    close(got, c["want"], c["tol"])


@pytest.mark.parametrize("Hq,Hkv,D", [(12, 4, 64), (32, 8, 128)])
def test_weight_packed_scattered_paths(jf, Hq, Hkv, D):
    """Accepted nodes anywhere in each packed tree, against the 64-bit sums and the padded call's bits."""
    sizes, prefix, rows, N = [9, 41, 30], [100, 3, 700], [4, 37, 1], 41
    c = weight_case(70 + Hq, prefix, rows, N, Hq, Hkv, D, True)
    rng = np.random.default_rng(Hq)
    qn, kn = c["q"].double().cpu().numpy(), c["pool"].k.double().numpy()
    lse = torch.from_numpy((rng.random(c["lse"].shape) + 5).astype(np.float32)).cuda()
    paths, want, tol = np.full((3, N), -1, np.int32), np.empty_like(c["want"]), np.empty_like(c["tol"])
    before = c["out"].cpu().numpy()
    for b, (n, r) in enumerate(zip(sizes, rows)):
        paths[b, :r] = np.concatenate([[0], np.sort(rng.permutation(n - 1)[:r - 1]) + 1])
        want[b], tol[b] = ref.attention_weight(qn[b], kn, c["pool"].table[b], prefix[b], paths[b, :r].astype(np.int64),
                                               lse[b].cpu().numpy(), c["weight"][b].cpu().numpy(), before[b], c["scale"])
    kw = dict(path=dev(paths), accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"])
    pad = jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], lse, out=c["out"].clone(), **kw)
    at = torch.cat([torch.arange(n) + b * N for b, n in enumerate(sizes)]).cuda()
    cu, err = dev(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)), new_err()
    got = jf.accumulate_attention_weight(c["q"].flatten(0, 1)[at].contiguous(), c["k"], c["table"], c["prefix"],
                                         lse.transpose(0, 1).flatten(1)[:, at].contiguous(), cu_seqlens=cu,
                                         out=c["out"].clone(), dev_err=err, **kw)
    assert err.item() == 0 and torch.equal(got, pad)
    close(got, want, tol)


@pytest.mark.parametrize("Hq,Hkv,D,path", [
    (66, 2, 64, True), (66, 2, 128, False), (128, 2, 128, True), (71, 1, 64, False), (71, 1, 128, True),
    (128, 1, 64, False), (256, 2, 128, True),              # 33, 64, 71 and 128 heads a kv-head
])
def test_weight_of_wide_groups(jf, Hq, Hkv, D, path):
    prefix, rows, N = [140, 0, 33], [7, 2, 9], 9
    if not path:
        rows = [9, 9, 9]
    c = weight_case(80 + Hq, prefix, rows, N, Hq, Hkv, D, path)
    err = new_err()
    got = jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], c["lse"], path=c["path"],
                                         accept_len=c["accept_len"] if path else None, weight=c["weight"],
                                         scale=c["scale"], out=c["out"], dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    close(got, c["want"], c["tol"])


@pytest.mark.parametrize("heads", [40, 80, 160])
def test_weight_of_many_kv_heads(jf, heads):
    """Kv-heads that do not divide the SMs, and more of them than SMs."""
    c = weight_case(90 + heads, [300, 15], [5, 2], 6, heads, heads, 64, True)
    err = new_err()
    got = jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], c["lse"], path=c["path"],
                                         accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"],
                                         out=c["out"], dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    close(got, c["want"], c["tol"])


@pytest.mark.parametrize("B", [769, 1600])
def test_weight_of_many_sequences(jf, B):
    """More sequences than a block has threads: their costs are scanned in several passes."""
    rng = np.random.default_rng(B)
    prefix = [int(x) for x in rng.integers(0, 60, B)]
    prefix[-1] = 400                                       # the last one spans several tiles
    rows = [int(x) for x in rng.integers(0, 3, B)]
    rows[-1] = 2
    c = weight_case(B, prefix, rows, 2, 4, 2, 64, True)
    err = new_err()
    got = jf.accumulate_attention_weight(c["q"], c["k"], c["table"], c["prefix"], c["lse"], path=c["path"],
                                         accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"],
                                         out=c["out"], dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    close(got, c["want"], c["tol"])


# --------------------------------------------------------------------------- order of work

def on_its_stream(call, outs, wants):
    """call(stream) does its work on stream, behind what is queued there: while that stream
    sleeps, the outputs are what they were.  (A first call before: loading a kernel and growing
    the pool of memory wait for the device.)"""
    s = torch.cuda.Stream()
    was, seen = [o.clone() for o in outs], [o.clone() for o in outs]
    call(s)
    torch.cuda.synchronize()
    for o, w in zip(outs, was):
        o.copy_(w)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    call(s)
    for to, o in zip(seen, outs):                          # on the current stream
        to.copy_(o)
    torch.cuda.current_stream().synchronize()
    asleep = not s.query()
    s.synchronize()
    assert asleep, "the stream woke too early to tell"
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))   # noqa: E731
    assert all(same(a, b) for a, b in zip(seen, was))
    assert all(same(a, b) for a, b in zip(outs, wants))


def test_cache_calls_wait_for_their_stream(jf):
    c = weight_case(13, [500, 300], [4, 2], 8, 8, 2, 64, True)
    kw = dict(path=c["path"], accept_len=c["accept_len"], weight=c["weight"], scale=c["scale"])
    args = (c["q"], c["k"], c["table"], c["prefix"], c["lse"])
    want = jf.accumulate_attention_weight(*args, out=c["out"].clone(), **kw)
    out = c["out"].clone()
    on_its_stream(lambda s: jf.accumulate_attention_weight(*args, out=out, stream=s, **kw), [out], [want])
    lens = c["prefix"] + c["accept_len"] + 1
    keep, kept = jf.select_kept_keys(want, lens, 100, sink=1, recent=5)
    k2, l2 = torch.full_like(keep, -9), torch.full_like(kept, -9)
    on_its_stream(lambda s: jf.jf_select_kept(want, lens, k2, l2, 1, 5, stream=s), [k2, l2], [keep, kept])
    k_old, v_old = c["k"], torch.randn_like(c["k"])
    kv, w = [k_old.clone(), v_old.clone()], want.clone()
    jf.evict_kv(*kv, c["table"], lens, keep, kept, weight=w)
    torch.cuda.synchronize()
    mine = [k_old.clone(), v_old.clone(), want.clone()]
    on_its_stream(lambda s: jf.evict_kv(mine[0], mine[1], c["table"], lens, keep, kept, weight=mine[2], stream=s),
                  mine, [*kv, w])


def test_eviction_in_a_graph(jf):
    """Weight, choice and move of one step, captured once and replayed over restored caches."""
    c = weight_case(14, [900, 640, 7], [4, 2, 1], 8, 8, 2, 128, True)
    lens = c["prefix"] + c["accept_len"] + 1
    k, v, w = c["k"].clone(), c["k"].flip(0).contiguous(), c["weight"].clone()
    err = new_err()

    def step():
        jf.accumulate_attention_weight(c["q"], k, c["table"], c["prefix"], c["lse"], path=c["path"],
                                       accept_len=c["accept_len"], weight=w, scale=c["scale"], out=w, dev_err=err)
        keep, kept = jf.select_kept_keys(w, lens, 300, sink=2, recent=20, dev_err=err)
        jf.evict_kv(k, v, c["table"], lens, keep, kept, weight=w, dev_err=err)
        return keep, kept

    def restore():
        k.copy_(c["k"])
        v.copy_(c["k"].flip(0))
        w.copy_(c["weight"])

    want = [x.clone() for x in (*step(), k, v, w)]
    restore()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        restore()
        graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0
        for a, b in zip((*got, k, v, w), want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
