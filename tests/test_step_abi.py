"""The calls around a step reject bad host arguments before any launch, and their Python wrappers bad
tensors; frequencies against their formulas.  CPU only (no kernel is launched)."""
import ctypes
import math

import pytest
import torch

P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


def at(n):
    return ctypes.c_void_p(n << 32)      # far apart, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_jf_gb300 import build
    return ctypes.CDLL(build.build())


def refused(fn, args, changes):
    for where, value, status in changes:
        bad = list(args)
        for k, v in zip(where, value) if isinstance(where, tuple) else ((where, value),):
            bad[k] = v
        assert fn(*bad) == status, (where, value)


ROTATE = [P, i64, P, i64, P, i64, P, P, i32, i32, f32, P, P, f32, P, P, P]


def test_rotate_refusals(lib):
    fn = lib.jf_rotate_append_kv
    fn.argtypes = ROTATE + [i32] * 8 + [P] * 5
    odd = ctypes.c_void_p((9 << 32) + 8)
    #       q      stride k      stride v      stride pos    freq   R    int scale qn    kn    eps   bt     pfx     tl
    args = [at(1), 4096, at(2), 1024, at(3), 1024, at(4), at(5), 128, 0, 1.0, None, None, 1e-6, at(6), at(7), None,
            # B N  Hq  Hkv D   pg  mp  np  q_out  kc      vc      err   stream
            2, 16, 32, 8, 128, 16, 10, 99, at(8), at(10), at(11), None, None]
    refused(fn, args, [
        (2, None, 1), (4, None, 1), (14, None, 1), (15, None, 1), (26, None, 1), (27, None, 1),
        (0, None, 1), (25, None, 1),                     # q without q_out, q_out without q
        (6, None, 1),                                    # frequencies without positions
        (17, 0, 1), (18, 0, 1), (19, 0, 1), (20, 0, 1), (23, 0, 1), (24, 0, 1),
        (10, float("nan"), 1), (10, float("inf"), 1), (13, -1.0, 1), (13, float("nan"), 1),
        (1, 4088, 1), (3, 1016, 1), (5, 1016, 1),        # tokens that overlap
        (21, 96, 3), (22, 32, 3), (8, 8, 3), (8, 144, 3), (8, 120, 3), (17, 1 << 27, 3), (24, 1 << 27, 3),
        (3, (1 << 31) + 8, 3), (23, 1 << 27, 3),
        (0, odd, 7), (2, odd, 7), (4, odd, 7), (25, odd, 7), (26, odd, 7), (27, odd, 7), (11, odd, 7), (12, odd, 7),
        (1, 4100, 7), (3, 1028, 7), (5, 1028, 7), (7, ctypes.c_void_p((9 << 32) + 4), 7)])
    near = lambda n, by: ctypes.c_void_p((n << 32) + by)  # noqa: E731
    refused(fn, args, [(25, at(2), 1), (25, at(3), 1),   # q_out over k, v
                       (25, near(1, 4096 * 2), 1),       # over a later token of q
                       ((1, 25), (4104, at(1)), 1),      # over q, whose rows lie further apart
                       (26, at(1), 1), (27, at(2), 1), (26, at(11), 1), (26, at(8), 1), (27, near(3, 2048), 1)])


def test_rotate_packed_refusals(lib):
    fn = lib.jf_rotate_append_kv_packed
    fn.argtypes = ROTATE + [i32] * 9 + [P] * 5
    args = [at(1), 4096, at(2), 1024, at(3), 1024, at(4), at(5), 128, 0, 1.0, None, None, 1e-6, at(6), at(7), at(9),
            2, 16, 30, 32, 8, 128, 16, 10, 99, at(8), at(10), at(11), None, None]
    refused(fn, args, [(16, None, 1), (19, 0, 1), (19, 0x7FFFFFF8, 3), (22, 96, 3)])


ADJUST = [P, i32, P, P, P, P, P, P, i32, P, P, P, f32, P]


def test_adjust_refusals(lib):
    fn = lib.jf_adjust_logits
    fn.argtypes = ADJUST + [i32] * 3 + [P, i32, P, P]
    #       logits dt cnt    draft  mask   bias   allow  arow   n   rep    pres   freq   masked         tl
    args = [at(1), 0, at(2), at(3), at(4), at(5), at(6), at(7), 32, at(8), at(9), at(10), -float("inf"), None,
            # B N  V   out     odt err   stream
            2, 16, 64, at(11), 0, None, None]
    refused(fn, args, [
        (0, None, 1), (17, None, 1), (1, 2, 1), (18, 2, 1), ((1, 18), (1, 0), 1), (14, 0, 1), (15, 0, 1), (16, 0, 1),
        (3, None, 1), (4, None, 1), (8, 0, 1), ((6, 7), (None, at(7)), 1), (12, float("nan"), 1),
        (15, 4097, 3), (16, 0x7FFFFFFF, 3), ((14, 15, 16), (1 << 20, 4096, 1 << 20), 3),
        (17, ctypes.c_void_p((1 << 32) + 128), 1),       # part of the logits
        ((17, 18), (at(1), 1), 1),                       # fp32 over bf16
        (17, at(2), 1), (17, at(5), 1), (17, at(6), 1),
        (0, ctypes.c_void_p((1 << 32) + 1), 7), (4, ctypes.c_void_p((4 << 32) + 4), 7)])
    fn = lib.jf_adjust_logits_packed
    fn.argtypes = ADJUST + [i32] * 4 + [P, i32, P, P]
    args = args[:13] + [at(12), 2, 16, 20, 64, at(11), 0, None, None]
    refused(fn, args, [(13, None, 1), (16, 0, 1), (16, 0x7FFFFFF8, 3)])


def test_count_refusals(lib):
    fn = lib.jf_count_tokens
    fn.argtypes = [P, P, i32, P, P, P, P, i32, i32, i32, i32, P, P, P]
    #       count  row  in token  path   len    extra  prompt B N V    out    err stream
    args = [at(1), None, 4, at(2), at(3), at(4), at(5), 0, 4, 16, 100, at(6), None, None]
    refused(fn, args, [(3, None, 1), (11, None, 1), (8, 0, 1), (9, 0, 1), (10, 0, 1), (5, None, 1), (2, 0, 1),
                       (2, 3, 1),                        # fewer rows than sequences, without a row index
                       ((0, 1), (None, at(7)), 1),       # rows of nothing
                       ((1, 11), (at(7), at(1)), 1),     # gathered in place
                       (11, ctypes.c_void_p((1 << 32) + 4), 1), (11, at(2), 1), (11, at(3), 1), (11, at(4), 1),
                       (11, at(5), 1), (8, 65536, 3), (10, 0x7FFFFFFF, 3),
                       (11, ctypes.c_void_p((6 << 32) + 2), 7)])


def test_shared_refusals(lib):
    fn = lib.jf_tree_attention_shared
    fn.argtypes = [P] * 9 + [i32] * 9 + [f32, P, P, P, sz, P, P]
    #       q      k      v      bt     pfx    tl    mask   gs     sp     ng B  N   Hq  Hkv D   pg  mp  np  scale
    args = [at(1), at(2), at(3), at(4), at(5), None, at(6), at(7), at(8), 2, 4, 16, 32, 8, 128, 16, 10, 99, 0.1,
            # out   lse   ws      bytes    err  stream
            at(9), None, at(10), 1 << 40, None, None]
    refused(fn, args, [(0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (4, None, 1), (6, None, 1), (7, None, 1),
                       (8, None, 1), (19, None, 1), (9, 0, 1), (9, 5, 1), (10, 0, 1), (11, 0, 1), (12, 0, 1), (13, 0, 1),
                       (16, 0, 1), (17, 0, 1), (18, 0.0, 1), (18, float("nan"), 1), (18, float("inf"), 1),
                       (17, 1 << 27, 3), ((10, 9), (4097, 1), 3), (11, 4097, 3), (12, 33, 3), (13, 5, 3), (14, 96, 3),
                       (15, 32, 3), ((11, 16), (17, 1), 3), ((12, 13), (256, 1), 3),
                       (0, ctypes.c_void_p((1 << 32) + 8), 7), (1, ctypes.c_void_p((2 << 32) + 8), 7),
                       (19, ctypes.c_void_p((9 << 32) + 8), 7), (6, ctypes.c_void_p((6 << 32) + 4), 7),
                       (19, at(1), 1), (19, at(2), 1), (19, ctypes.c_void_p((3 << 32) + 16), 1)])
    fn = lib.jf_tree_attention_shared_packed
    fn.argtypes = [P] * 9 + [i32] * 10 + [f32, P, P, P, sz, P, P]
    args = args[:5] + [at(11)] + args[6:12] + [40] + args[12:]
    refused(fn, args, [(5, None, 1), (12, 0, 1), (12, 0x7FFFFFF8, 3)])


@pytest.fixture(scope="module")
def jf():
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf as mod
    return mod


def test_frequencies(jf):
    freq, scale = jf.rotary_frequencies(64, device="cpu")
    assert freq.dtype == torch.float64 and scale == 1.0
    for f in range(32):
        assert math.isclose(float(freq[f]), 10000.0 ** (-2 * f / 64), rel_tol=1e-14)
    linear, scale = jf.rotary_frequencies(64, scaling=("linear", 8.0), device="cpu")
    assert torch.allclose(linear * 8, freq, rtol=1e-15, atol=0) and scale == 1.0
    base, length, factor, R = 1000000.0, 32768, 4.0, 128
    freq, _ = jf.rotary_frequencies(R, base=base, device="cpu")
    yarn, scale = jf.rotary_frequencies(R, base=base, scaling=("yarn", factor, length), device="cpu")
    assert math.isclose(scale, 0.1 * math.log(4.0) + 1.0)
    ratio = yarn / freq
    turns = length * freq / (2 * math.pi)
    assert torch.allclose(ratio[turns > 40], torch.ones(1, dtype=torch.float64))     # many turns: kept
    assert torch.allclose(ratio[turns < 0.8], torch.full((1,), 0.25, dtype=torch.float64))
    assert (ratio[1:] <= ratio[:-1] + 1e-12).all()
    between = ratio[(ratio < 0.999) & (ratio > 0.251)]
    assert between.numel() > 5
    step = between[1:] - between[:-1]
    assert torch.allclose(step, step[:1].expand_as(step), rtol=1e-6, atol=0)         # a linear ramp over the pairs
    with pytest.raises(ValueError):
        jf.rotary_frequencies(64, scaling=("other", 2.0), device="cpu")
    with pytest.raises(ValueError):
        jf.rotary_frequencies(64, scaling=("linear", 0.5), device="cpu")


def test_token_rows(jf):
    """Strides of the views that q, k and v may be."""
    qkv = torch.zeros(6, (8 + 2 + 2) * 64, dtype=torch.bfloat16)
    x = qkv.view(2, 3, 12, 64)
    assert jf._token_rows("k", x[:, :, 8:10], (2, 3)) == 12 * 64
    assert jf._token_rows("k", x[:, :1, 8:10], (2, 1)) == 3 * 12 * 64
    assert jf._token_rows("k", qkv.view(6, 12, 64)[:, 8:10], (6,)) == 12 * 64
    assert jf._token_rows("k", x[:1, :1, 8:10], (1, 1)) == 2 * 64
    for bad in (x[:, :2, 8:10], x.transpose(2, 3)):
        with pytest.raises(ValueError):
            jf._token_rows("k", bad, tuple(bad.shape[:2]))
