"""GPU parity of beam selection and the beams' cache fork with plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from test_gpu_cache import Pool, dev, new_err, on_its_stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jf():
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf as mod
    return mod


def check_beams(logits, score, finished, eos, got, K):
    """Every prompt's output against the definition.  Within a beam the order is exact (by
    logit, then token).  Across beams a pair may stand where the exact ranking has one whose
    s differs by less than the stated precision: with u = 2^-24, a sum of V exponentials is
    off by at most (40 + 2 span) u relative (under 40 roundings on any path of the sum; the
    exponent's product and the exponential by 2 span u), span the logits' finite range."""
    parent, token, new_score, new_fin = (x.cpu().numpy() for x in got)
    B, W, V = logits.shape
    for b in range(B):
        s = ref.beam_scores(logits[b], score[b], None if finished is None else finished[b], eos)
        flat = s.reshape(-1)
        order = np.lexsort((np.arange(flat.size), -flat))[:K]
        pick = parent[b].astype(np.int64) * V + token[b]
        assert ((parent[b] >= 0) & (parent[b] < W) & (token[b] >= 0) & (token[b] < V)).all()
        assert len(set(pick.tolist())) == K
        fin = logits[b][np.isfinite(logits[b])].astype(np.float64)
        span = fin.max() - fin.min() if fin.size else 0.0
        tol = (40 + 2 * span) * 2.0 ** -24
        a, e = flat[pick], flat[order]
        assert (np.isneginf(a) == np.isneginf(e)).all(), b
        live = ~np.isneginf(e)
        assert (np.abs(a[live] - e[live]) <= 2 * tol).all(), (b, a, e)
        if not live.all():                     # pairs at -inf: the lowest ones, in order
            assert (pick[~live] == order[~live]).all(), (b, pick, order)
        assert (np.isneginf(new_score[b]) == ~live).all()
        assert (np.abs(new_score[b][live] - a[live]) <= tol + 2.0 ** -24 * np.abs(a[live])).all()
        for w in range(W):
            mine = pick[(parent[b] == w) & live]
            row = np.lexsort((np.arange(V), -s[w]))[:len(mine)] + w * V
            assert (mine == row).all(), (b, w)
        for j in range(K):
            f = (finished is not None and finished[b, parent[b, j]] != 0) or token[b, j] == eos
            assert new_fin[b, j] == int(f)


def run_beams(jf, logits, score, K, finished=None, eos=-1, dtype=torch.bfloat16):
    t = torch.from_numpy(np.ascontiguousarray(logits, np.float32)).to(dtype)
    got = jf.beam_select(t.cuda(), dev(score.astype(np.float32)), K,
                         finished=None if finished is None else dev(finished.astype(np.int32)), eos_token=eos)
    torch.cuda.synchronize()
    check_beams(t.float().numpy(), score.astype(np.float32), finished, eos, got, K)
    return got


@pytest.mark.parametrize("B,W,V,K", [
    (1, 4, 151936, 8), (2, 1, 1000, 1), (3, 5, 50257, 5), (1, 3, 32003, 6), (4, 8, 4097, 16), (2, 2, 17, 8),
    (1, 1, 1, 1), (1, 64, 700, 64), (2, 6, 8, 40), (1, 2, 131072, 64), (5, 7, 2049, 33), (40, 3, 16387, 4),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beams_match_reference(jf, B, W, V, K, dtype):
    rng = np.random.default_rng(B * 100 + W * 10 + K)
    logits = 2.5 * rng.standard_normal((B, W, V))
    score = -8 * rng.random((B, W)) - 2
    run_beams(jf, logits, score, K, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_finished_and_unused_beams(jf, dtype):
    rng = np.random.default_rng(5)
    B, W, V, K = 6, 5, 5003, 10
    logits = 3 * rng.standard_normal((B, W, V))
    score = -3 * rng.random((B, W)) - 1
    finished = np.zeros((B, W), np.int32)
    finished[0, 2] = 1                         # one finished beam
    finished[1] = 1                            # all of them: W pairs, then -inf ones
    score[2, 1:] = -np.inf                     # the first step: one beam in use
    score[3] = -np.inf                         # none in use
    finished[4, :4] = 1
    score[4, 4] = -np.inf
    score[5, 0] = -np.inf
    finished[5, 0] = 1                         # finished at -inf
    for eos in (0, 4, V - 1):
        run_beams(jf, logits, score, K, finished, eos, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_tokens_and_ties(jf, dtype):
    rng = np.random.default_rng(6)
    V = 20011
    logits = rng.standard_normal((5, 3, V)) * 2
    allowed = rng.permutation(V)[:7]
    masked = np.full_like(logits[0], -np.inf)
    masked[:, allowed] = logits[0][:, allowed]
    logits[0] = masked                         # seven tokens allowed in each beam
    logits[1, 1] = -np.inf                     # a beam without any
    logits[2] = -np.inf                        # a prompt without any
    logits[3] = np.round(logits[3])            # many ties
    logits[4] = 1.5                            # one value everywhere
    score = np.tile(np.array([[-1.0, -2.5, -2.5]]), (5, 1))
    for K in (4, 16, 40):
        run_beams(jf, logits, score, K, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logits_of_beams_that_are_not_live_are_not_read(jf, dtype):
    rng = np.random.default_rng(15)
    B, W, V, K = 2, 4, 3001, 9
    logits = 2 * rng.standard_normal((B, W, V))
    score = -rng.random((B, W)) - 1
    finished = np.zeros((B, W), np.int32)
    finished[0, 1] = 1
    score[1, 2:] = -np.inf
    t = torch.from_numpy(logits.astype(np.float32)).to(dtype)
    clean = t.float().numpy().copy()
    t[0, 1], t[1, 2], t[1, 3] = float("nan"), float("inf"), float("nan")
    got = jf.beam_select(t.cuda(), dev(score.astype(np.float32)), K, finished=dev(finished), eos_token=5)
    torch.cuda.synchronize()
    check_beams(clean, score.astype(np.float32), finished, 5, got, K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_inf_logits_leave_no_stale_output(jf, dtype, bad):
    """A prompt with NaN or +inf gives pairs in range, whatever the outputs held, and the
    prompts beside it their own results."""
    rng = np.random.default_rng(21)
    B, W, V, K = 4, 2, 3001, 7
    logits = 2 * rng.standard_normal((B, W, V))
    score = (-rng.random((B, W)) - 1).astype(np.float32)
    t = torch.from_numpy(logits.astype(np.float32)).to(dtype)
    clean = t.float().numpy().copy()
    t[0] = bad                                 # everywhere
    t[1, 1, 5] = bad                           # in one logit
    t[2, :, 17] = bad                          # in one logit of every beam
    ws = torch.empty(jf.jf_beam_select_workspace_size(B, W, V, K, jf._logit_dtype(t)), dtype=torch.uint8, device="cuda")
    out = [torch.full((B, K), -(1 << 30), dtype=torch.int32, device="cuda") for _ in range(2)]
    new_score = torch.full((B, K), 1e30, device="cuda")
    new_fin = torch.full((B, K), 77, dtype=torch.int32, device="cuda")
    jf.jf_beam_select(t.cuda(), dev(score), *out, new_score, ws, new_finished=new_fin)
    torch.cuda.synchronize()
    parent, token = (x.cpu().numpy() for x in out)
    assert ((parent >= 0) & (parent < W)).all() and ((token >= 0) & (token < V)).all()
    assert (new_score.cpu().numpy() != np.float32(1e30)).all()
    assert np.isin(new_fin.cpu().numpy(), (0, 1)).all()
    good = slice(3, 4)
    check_beams(clean[good], score[good], None, -1, [x[good] for x in (*out, new_score, new_fin)], K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scores_of_every_size(jf, dtype):
    """Sharp and flat rows, logits and scores far from zero: the fp32 bound of the merge stays
    below the K-th pair."""
    rng = np.random.default_rng(16)
    B, W, V, K = 6, 3, 9001, 12
    logits = rng.standard_normal((B, W, V))
    logits[0] *= 30.0                          # almost all probability on one token
    logits[1] += 60.0
    logits[2] -= 60.0
    logits[3] *= 1e-3
    logits[4, :, 17] = 200.0
    score = -rng.random((B, W)) * 3
    score[1], score[5] = score[1] - 300.0, score[5] + 50.0
    run_beams(jf, logits, score, K, dtype=dtype)


def test_unaligned_logits(jf):
    """A logits tensor that starts two bytes past a 16-byte boundary."""
    rng = np.random.default_rng(7)
    B, W, V, K = 2, 3, 4096, 6
    logits = torch.from_numpy((2 * rng.standard_normal(B * W * V + 1)).astype(np.float32)).to(torch.bfloat16).cuda()
    view = logits[1:].view(B, W, V)
    score = (-rng.random((B, W))).astype(np.float32)
    got = jf.beam_select(view, dev(score), K)
    torch.cuda.synchronize()
    check_beams(view.float().cpu().numpy(), score, None, -1, got, K)


def test_beams_and_fork_on_a_given_stream(jf):
    rng = np.random.default_rng(18)
    logits = dev((2 * rng.standard_normal((3, 4, 20000))).astype(np.float32))
    score = dev((-rng.random((3, 4))).astype(np.float32))
    want = jf.beam_select(logits, score, 6)
    pool, _, fresh = fork_case(3, 3, 4, 6, 2, 64, rng.integers(1, 60, 12), 5)
    table, lens = dev(pool.table), dev(rng.integers(1, 60, 12).astype(np.int32))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = jf.beam_select(logits, score, 6, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ta, la = jf.beam_fork_kv(pool.k.cuda(), pool.v.cuda(), table, lens, want[0], dev(fresh))
    torch.cuda.synchronize()
    k, v = pool.k.cuda(), pool.v.cuda()
    torch.cuda.synchronize()
    tb, lb = jf.beam_fork_kv(k, v, table, lens, want[0], dev(fresh), stream=s)
    s.synchronize()
    assert torch.equal(ta, tb) and torch.equal(la, lb)


def test_beams_in_a_graph(jf):
    rng = np.random.default_rng(8)
    B, W, V, K = 3, 4, 30000, 8
    logits = dev((2 * rng.standard_normal((B, W, V))).astype(np.float32)).to(torch.bfloat16)
    score = dev((-rng.random((B, W))).astype(np.float32))
    want = jf.beam_select(logits, score, K)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = jf.beam_select(logits, score, K)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def fork_case(seed, B, W, K, Hkv, D, lens, cap_pages):
    rng = np.random.default_rng(seed)
    pool = Pool(rng, lens, cap_pages, Hkv, D, spare=B * K)
    parent = rng.integers(0, W, (B, K)).astype(np.int32)
    return pool, parent, pool.spare.reshape(B, K)


@pytest.mark.parametrize("B,W,K,Hkv,D,cap", [(1, 4, 4, 8, 128, 20), (3, 2, 5, 2, 64, 9), (2, 3, 1, 1, 128, 4),
                                             (8, 4, 8, 4, 128, 300)])
def test_fork_matches_reference(jf, B, W, K, Hkv, D, cap):
    rng = np.random.default_rng(cap)
    lens = rng.integers(0, cap * 16 + 1, B * W)
    lens[0], lens[-1] = 0, cap * 16            # an empty beam, and one that fills its table
    if B * W > 4:
        lens[1], lens[2] = 16, 17
    pool, parent, fresh = fork_case(cap, B, W, K, Hkv, D, lens, cap)
    parent.reshape(-1)[0] = 0
    parent[-1, -1] = W - 1
    k, v, err = pool.k.cuda(), pool.v.cuda(), new_err()
    table, new_len = jf.beam_fork_kv(k, v, dev(pool.table), dev(lens.astype(np.int32)), dev(parent), dev(fresh),
                                     dev_err=err)
    torch.cuda.synchronize()
    want_table, want_len, copies = ref.beam_fork(pool.table, lens, parent, fresh)
    assert err.item() == 0
    assert (table.cpu().numpy() == want_table).all() and (new_len.cpu().numpy() == want_len).all()
    for cache, got in ((pool.k, k), (pool.v, v)):
        bits = cache.view(torch.int16).clone()
        for to, frm, slots in copies:
            bits[to, :slots] = cache.view(torch.int16)[frm, :slots]
        assert torch.equal(got.view(torch.int16).cpu(), bits)


def test_fork_reports_bad_input_and_stays_in_bounds(jf):
    lens = np.array([20, 33, 5, 40], np.int32)
    pool, parent, fresh = fork_case(2, 2, 2, 2, 2, 64, lens, 4)
    parent[:] = [[0, 1], [0, 1]]
    for what, bit in (("parent", jf.DEVERR_BAD_PATH), ("len", jf.DEVERR_BAD_PREFIX), ("fresh", jf.DEVERR_BAD_PAGE),
                      ("page", jf.DEVERR_BAD_PAGE)):
        pr, ln, fr, tb = parent.copy(), lens.copy(), fresh.copy(), pool.table.copy()
        if what == "parent":
            pr[1, 0] = 2
        elif what == "len":
            ln[2] = 65
        elif what == "fresh":
            fr[1, 0] = pool.k.shape[0]
        else:
            tb[2, 0] = -1
        k, v, err = pool.k.cuda(), pool.v.cuda(), new_err()
        table, new_len = jf.beam_fork_kv(k, v, dev(tb), dev(ln), dev(pr), dev(fr), dev_err=err)
        torch.cuda.synchronize()
        assert err.item() & bit, what
        want_table, want_len, _ = ref.beam_fork(pool.table, lens, parent, fresh)
        for j in (0, 1, 3):                    # the other beams are as without it
            assert (table[j].cpu().numpy() == want_table[j]).all() and new_len[j].item() == want_len[j]
        if what in ("parent", "len"):
            assert new_len[2].item() == 0 and (table[2] == -1).all()


@pytest.mark.parametrize("low", ["lowest", -1e30, -1e12])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masks_of_the_lowest_value(jf, dtype, low):
    """Tokens masked with a finite value: a beam that has nothing else spreads its score evenly,
    score - log V each, and does not outrank one with tokens of its own.  Scores against
    (score - log sum exp(x - max)) + (x - max) in 64 bits, where nothing large cancels; the
    fp32 sum of the exponentials is within 2^-17 of it (with u = 2^-24: 29 u for a slice of
    one step and 6 u for each of up to five, 2.25 u times the unmasked logits' span, below 16;
    masked ones underflow), and new_score is rounded once more."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    rng = np.random.default_rng(41)
    B, W, V, K = 4, 3, 5003, 20
    logits = rng.standard_normal((B, W, V)) * 2
    allowed = rng.permutation(V)[:7]
    logits[0, 1] = low                         # all masked, beside two beams that are not
    logits[1] = low                            # a prompt with nothing else
    keep = logits[2, :, allowed].copy()
    logits[2] = low                            # seven tokens allowed in each beam
    logits[2, :, allowed] = keep
    logits[3, 0] = low
    logits[3, 1, ::2] = low
    score = np.array([[-1.0, -1.0, -2.5], [-1.0, -0.5, -3.0], [-2.0, -1.0, -4.0], [-0.25, -9.0, -1.0]], np.float32)
    t = torch.from_numpy(logits.astype(np.float32)).to(dtype)
    parent, token, new_score, _ = (x.cpu().numpy() for x in jf.beam_select(t.cuda(), dev(score), K))
    x = t.double().numpy()
    d = x - x.max(-1, keepdims=True)
    s = (score.astype(np.float64)[..., None] - np.log(np.exp(d).sum(-1, keepdims=True))) + d
    tol = 2.0 ** -17
    for b in range(B):
        flat = s[b].reshape(-1)
        order = np.lexsort((np.arange(flat.size), -flat))[:K]
        pick = parent[b].astype(np.int64) * V + token[b]
        assert len(set(pick.tolist())) == K
        assert (np.abs(flat[pick] - flat[order]) <= 2 * tol + 2.0 ** -50 * np.abs(flat[order])).all(), b
        assert (np.abs(new_score[b] - flat[pick]) <= tol + 2.0 ** -24 * np.abs(flat[pick])).all(), b
        for w in range(W):                     # in a beam: by logit, then by token
            mine = pick[parent[b] == w]
            assert (mine == np.lexsort((np.arange(V), -x[b, w]))[:len(mine)] + w * V).all(), (b, w)


@pytest.mark.parametrize("what", ["fresh past", "fresh below", "fresh unused slots", "partial", "full"])
def test_fork_of_bad_pages_leaves_no_tokens(jf, what):
    """A beam whose pages are not in the pool gets length 0 and no pages, like one with a bad
    parent: a caller that reads dev_err late does not attend over what it was not given."""
    lens = np.array([20, 33, 37, 48], np.int32)
    pool, parent, fresh = fork_case(4, 2, 2, 2, 2, 64, lens, 4)
    parent[:] = [[0, 1], [0, 1]]
    fr, tb, beam = fresh.copy(), pool.table.copy(), 2
    if what == "fresh past":
        fr[1, 0] = pool.k.shape[0]
    elif what == "fresh below":
        fr[1, 0] = -1
    elif what == "fresh unused slots":         # 48 tokens: the fresh page takes no copy, the next token does
        fr[1, 1], beam = -2, 3
    elif what == "partial":
        tb[2, 2] = -1
    else:
        tb[2, 1] = pool.k.shape[0] + 7
    k, v, err = pool.k.cuda(), pool.v.cuda(), new_err()
    table, new_len = jf.beam_fork_kv(k, v, dev(tb), dev(lens), dev(parent), dev(fr), dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == jf.DEVERR_BAD_PAGE
    want_table, want_len, copies = ref.beam_fork(pool.table, lens, parent, fresh)
    want_table[beam], want_len[beam] = -1, 0
    assert (table.cpu().numpy() == want_table).all() and (new_len.cpu().numpy() == want_len).all()
    for cache, got in ((pool.k, k), (pool.v, v)):          # the other beams' copies; nothing outside fresh pages
        bits = cache.view(torch.int16).clone()
        for to, frm, slots in copies:
            bits[to, :slots] = cache.view(torch.int16)[frm, :slots]
        out = got.view(torch.int16).cpu()
        own = int(fresh[1, beam - 2])
        rows = [i for i in range(len(bits)) if i != own]
        assert torch.equal(out[rows], bits[rows])


@pytest.mark.parametrize("B,W,V", [(1, 4, 151936), (16, 8, 50257), (3, 2, 1001), (1, 16, 262144)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scores_of_many_equal_logits(jf, dtype, B, W, V):
    """Rows of one value far below a few others, whose roundings all go the same way: scores
    within the stated error of logsumexp, (80 ceil(W V / 2^21) + 3 span) 2^-24, and the
    rounding of the fp32 score."""
    rng = np.random.default_rng(V + W)
    K = 4
    logits = np.empty((B, W, V), np.float32)
    logits[:] = -rng.uniform(9.0, 17.0, (B, W, 1))
    logits[..., V // 3] = 0.25
    logits[..., 2 * V // 3] = rng.uniform(-3.0, 0.0, (B, W))
    score = (-3 * rng.random((B, W)) - 1).astype(np.float32)
    t = torch.from_numpy(logits).to(dtype)
    parent, token, new_score, _ = (x.cpu().numpy() for x in jf.beam_select(t.cuda(), dev(score), K))
    x = t.double().numpy()
    worst = 0.0
    for b in range(B):
        d = x[b] - x[b].max(-1, keepdims=True)
        s = (score[b].astype(np.float64)[:, None] - np.log(np.exp(d).sum(-1, keepdims=True))) + d
        span = -d.min()
        tol = (80 * -(-W * V // 2 ** 21) + 3 * span) * 2.0 ** -24
        a = s[parent[b], token[b]]
        e = np.sort(s.reshape(-1))[::-1][:K]
        worst = max(worst, float(np.abs(new_score[b] - a).max()))
        assert (np.abs(a - e) <= 2 * tol).all(), b
        assert (np.abs(new_score[b] - a) <= tol + 2.0 ** -24 * np.abs(a)).all(), (b, worst)


def test_beam_calls_wait_for_their_stream(jf):
    rng = np.random.default_rng(19)
    B, W, V, K = 3, 4, 20000, 6
    logits = dev((2 * rng.standard_normal((B, W, V))).astype(np.float32))
    score = dev((-rng.random((B, W))).astype(np.float32))
    want = jf.beam_select(logits, score, K)
    ws = torch.empty(jf.jf_beam_select_workspace_size(B, W, V, K, jf._logit_dtype(logits)), dtype=torch.uint8,
                     device="cuda")
    out = [torch.full_like(x, -9) for x in want]
    on_its_stream(lambda s: jf.jf_beam_select(logits, score, out[0], out[1], out[2], ws, new_finished=out[3], stream=s),
                  out, list(want))


def test_fork_on_a_given_stream_copies_its_pages(jf):
    rng = np.random.default_rng(20)
    B, W, K, cap = 3, 4, 6, 5
    lens = rng.integers(1, cap * 16, B * W)
    pool, parent, fresh = fork_case(20, B, W, K, 2, 64, lens, cap)
    want_table, want_len, copies = ref.beam_fork(pool.table, lens, parent, fresh)
    want = [dev(want_table), dev(want_len)]
    for cache in (pool.k, pool.v):
        bits = cache.view(torch.int16).clone()
        for to, frm, slots in copies:
            bits[to, :slots] = cache.view(torch.int16)[frm, :slots]
        want.append(bits.cuda())
    err, outs = new_err(), [torch.full_like(want[0], -9), torch.full_like(want[1], -9), pool.k.cuda(), pool.v.cuda()]
    args = (dev(pool.table), dev(lens.astype(np.int32)), dev(parent), dev(fresh))
    on_its_stream(lambda s: jf.jf_beam_fork_kv(outs[2], outs[3], *args, outs[0], outs[1], dev_err=err, stream=s),
                  outs, want)
    assert err.item() == 0


def test_beams_that_share_a_context_in_a_graph(jf):
    """Selection and fork of one step, captured once and replayed."""
    rng = np.random.default_rng(22)
    B, W, cap = 2, 5, 6
    lens = rng.integers(1, cap * 16, B * W)
    pool, _, fresh = fork_case(22, B, W, W, 2, 128, lens, cap)
    logits = dev((2 * rng.standard_normal((B, W, 4001))).astype(np.float32)).to(torch.bfloat16)
    score = dev((-rng.random((B, W))).astype(np.float32))
    table, plen, fr, err = dev(pool.table), dev(lens.astype(np.int32)), dev(fresh), new_err()
    k, v = pool.k.cuda(), pool.v.cuda()

    def step():
        picked = jf.beam_select(logits, score, W)
        return (*picked, *jf.beam_fork_kv(k, v, table, plen, picked[0], fr, dev_err=err))

    want = [x.clone() for x in (*step(), k, v)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        k.copy_(pool.k)
        v.copy_(pool.v)
        for x in got:
            x.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0
        for a, b in zip((*got, k, v), want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
