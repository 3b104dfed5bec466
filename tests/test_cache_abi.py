"""The bounded-cache and beam calls reject bad host arguments before any launch, and their
Python wrappers bad tensors.  CPU only (no kernel is launched)."""
import ctypes

import pytest
import torch

P, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: every call below fails early
OTHER = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_jf_gb300 import build
    return ctypes.CDLL(build.build())


def refused(fn, args, changes):
    for at, value, status in changes:
        bad = list(args)
        bad[at] = value
        assert fn(*bad) == status, (at, value)


def test_attention_weight_refusals(lib):
    fn = lib.jf_attention_weight
    fn.argtypes = [P] * 8 + [i32] * 8 + [f32, P, P, P]
    #       q     k     bt    pfx   path  acc   lse   w    B  N   Hq  Hkv D    pg  mp  np  scale out
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 1, 16, 32, 8, 128, 16, 10, 10, 0.1, FAKE, None, None]
    refused(fn, args, [(0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (6, None, 1), (17, None, 1),
                       (5, None, 1),                       # a path without lengths
                       (8, 0, 1), (9, 0, 1), (11, 0, 1), (14, 0, 1), (15, 0, 1), (16, 0.0, 1),
                       (16, float("inf"), 1), (16, float("nan"), 1),
                       (9, 4097, 3), (12, 96, 3), (13, 32, 3), (11, 5, 3), (10, 2000, 3), (0, ODD, 7), (1, ODD, 7)])
    fn = lib.jf_attention_weight_packed
    fn.argtypes = [P] * 9 + [i32] * 9 + [f32, P, P, P]
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 1, 16, 20, 32, 8, 128, 16, 10, 10, 0.1, FAKE, None,
            None]
    refused(fn, args, [(4, None, 1), (11, 0, 1), (11, 0x7FFFFFF8, 3), (14, 96, 3)])


def test_select_refusals(lib):
    fn = lib.jf_select_kept
    fn.argtypes = [P, P] + [i32] * 6 + [P, P, P, P]
    #       w     len   B  H  cap  sink rec budget keep kept
    args = [FAKE, FAKE, 1, 2, 100, 4, 10, 50, FAKE, FAKE, None, None]
    refused(fn, args, [(0, None, 1), (1, None, 1), (8, None, 1), (9, None, 1), (2, 0, 1), (3, 0, 1), (4, 0, 1),
                       (5, -1, 1), (6, -1, 1), (7, 13, 1), (7, 0, 1), (5, 0x7FFFFFFF, 1),
                       (4, (1 << 30) + 1, 3), (7, (1 << 30) + 1, 3), (2, 1 << 28, 3)])


def test_select_refuses_lengths_in_place(lib):
    """Other heads' blocks read the lengths while the first head's writes the kept ones."""
    fn = lib.jf_select_kept
    fn.argtypes = [P, P] + [i32] * 6 + [P, P, P, P]
    at = ctypes.c_void_p
    #       w     len          B  H  cap  sink rec budget keep kept
    args = [FAKE, at(0x20000), 4, 2, 100, 4, 10, 50, at(0x30000), at(0x40000), None, None]
    refused(fn, args, [(9, at(0x20000), 1),              # kept_len is seq_len
                       (9, at(0x2000C), 1), (9, at(0x1FFF4), 1),     # it shares one element
                       (8, at(0x20000), 1), (8, at(0x20000 - 4 * 4 * 2 * 50 + 4), 1)])   # so does keep


def test_evict_refusals(lib):
    fn = lib.jf_evict_kv
    fn.argtypes = [P] * 9 + [i32] * 7 + [P, P]
    #       k     v     bt    len    keep  kept  new   w     wo    B  H  D    bud pg  mp  np
    args = [FAKE, FAKE, FAKE, OTHER, FAKE, FAKE, None, None, None, 1, 2, 128, 20, 16, 10, 10, None, None]
    refused(fn, args, [(0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (4, None, 1), (5, None, 1),
                       (7, FAKE, 1), (8, FAKE, 1),         # weights need both arrays
                       (3, FAKE, 1),                       # the new lengths may not be the old ones
                       (9, 0, 1), (10, 0, 1), (12, 0, 1), (14, 0, 1), (15, 0, 1), (11, 96, 3), (13, 32, 3),
                       (0, ODD, 7), (1, ODD, 7)])


def test_evict_refuses_pools_whose_rows_pass_32_bits(lib):
    """Pool rows (page * 16 + slot) are 32-bit: a row past them would silently stay in place."""
    fn = lib.jf_evict_kv
    fn.argtypes = [P] * 9 + [i32] * 7 + [P, P]
    args = [FAKE, FAKE, FAKE, OTHER, FAKE, FAKE, None, None, None, 1, 2, 128, 20, 16, 10, 10, None, None]
    refused(fn, args, [(15, 1 << 27, 3), (15, 0x7FFFFFFF, 3)])


def test_beam_select_refusals(lib):
    size = lib.jf_beam_select_workspace_size
    size.argtypes, size.restype = [i32] * 5, sz
    none = ctypes.c_size_t(-1).value
    for bad in ((0, 4, 100, 8, 0), (1, 0, 100, 8, 0), (1, 65, 100, 8, 0), (1, 4, 100, 65, 0), (1, 4, 2, 9, 0),
                (1, 4, 100, 8, 7), (1, 4, 1 << 30, 8, 0), (1 << 20, 4, 100, 8, 0)):
        assert size(*bad) == none, bad
    fn = lib.jf_beam_select
    fn.argtypes = [P, i32, P, P, i32, i32, i32, i32, i32, P, P, P, P, P, sz, P]
    #       lg    dt sc    fin   eos B  W  V    K  par   tok   ns     nf     ws    bytes
    args = [FAKE, 0, FAKE, FAKE, 5, 1, 4, 100, 8, FAKE, FAKE, OTHER, OTHER, FAKE, 1 << 20, None]
    refused(fn, args, [(0, None, 1), (2, None, 1), (9, None, 1), (10, None, 1), (11, None, 1), (13, None, 1),
                       (1, 7, 1), (4, -1, 1), (4, 100, 1), (4, -2, 1), (11, FAKE, 1), (12, FAKE, 1), (5, 0, 1),
                       (6, 65, 3), (8, 65, 3), (0, ctypes.c_void_p(0x10001), 7), (13, ctypes.c_void_p(0x10004), 7)])


def test_beam_fork_refusals(lib):
    fn = lib.jf_beam_fork_kv
    fn.argtypes = [P] * 6 + [i32] * 8 + [P, P, P, P]
    #       k     v     bt    len   par   fresh B  W  K  H  D    pg  mp  np  nt     nl
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 4, 4, 2, 128, 16, 10, 10, OTHER, OTHER, None, None]
    refused(fn, args, [(at, None, 1) for at in (0, 1, 2, 3, 4, 5, 14, 15)] +
            [(14, FAKE, 1), (15, FAKE, 1), (6, 0, 1), (7, 0, 1), (8, 0, 1), (9, 0, 1), (12, 0, 1), (13, 0, 1),
             (10, 96, 3), (11, 8, 3), (0, ODD, 7), (1, ODD, 7)])


def test_arrays_that_overlap_in_part_are_refused(lib):
    """An output whose blocks write where others still read."""
    at = ctypes.c_void_p
    fn = lib.jf_attention_weight
    fn.argtypes = [P] * 8 + [i32] * 8 + [f32, P, P, P]
    w, n = 0x100000, 4 * 2 * 8 * 160           # weight [2][8][160]
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, at(w), 2, 16, 32, 8, 128, 16, 10, 10, 0.1, at(2 * w), None, None]
    refused(fn, args, [(17, at(w + 4), 1), (17, at(w + n - 4), 1), (17, at(w - n + 4), 1)])
    fn = lib.jf_attention_weight_packed
    fn.argtypes = [P] * 9 + [i32] * 9 + [f32, P, P, P]
    args = [FAKE] * 8 + [at(w), 2, 16, 20, 32, 8, 128, 16, 10, 10, 0.1, at(2 * w), None, None]
    refused(fn, args, [(19, at(w + n - 4), 1)])
    fn = lib.jf_evict_kv
    fn.argtypes = [P] * 9 + [i32] * 7 + [P, P]
    args = [FAKE, FAKE, FAKE, OTHER, FAKE, FAKE, None, at(w), at(2 * w), 2, 8, 128, 20, 16, 10, 10, None, None]
    refused(fn, args, [(8, at(w + 4), 1), (8, at(w + n - 4), 1), (8, at(w - n + 4), 1)])
    fn = lib.jf_beam_select
    fn.argtypes = [P, i32, P, P, i32, i32, i32, i32, i32, P, P, P, P, P, sz, P]
    s, f = 0x30000, 0x40000                    # score and finished [2][4], the outputs [2][8]
    args = [FAKE, 0, at(s), at(f), 5, 2, 4, 100, 8, FAKE, FAKE, at(0x50000), at(0x60000), at(0x70000), 1 << 20, None]
    refused(fn, args, [(11, at(s + 28), 1), (11, at(s - 60), 1), (12, at(f + 28), 1), (12, at(f - 60), 1)])
    fn = lib.jf_beam_fork_kv
    fn.argtypes = [P] * 6 + [i32] * 8 + [P, P, P, P]
    t, m = 0x30000, 0x40000                    # block_table [8][10], prefix_len [8]; the new ones [6][10], [6]
    args = [FAKE, FAKE, at(t), at(m), FAKE, FAKE, 2, 4, 3, 2, 128, 16, 10, 10, at(0x50000), at(0x60000), None, None]
    refused(fn, args, [(14, at(t + 4 * 79), 1), (14, at(t - 4 * 59), 1), (15, at(m + 28), 1), (15, at(m - 20), 1)])


@pytest.mark.gpu
def test_wrappers_refuse_bad_tensors():
    from tree_speculative_decoding_jf_gb300 import jf
    w = torch.zeros((2, 3, 64), device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        jf.select_kept_keys(w.cpu(), n, 8)
    with pytest.raises(ValueError):
        jf.select_kept_keys(w.transpose(1, 2), n, 8)
    with pytest.raises(TypeError):
        jf.select_kept_keys(w.half(), n, 8)
    with pytest.raises(ValueError):
        jf.select_kept_keys(w, n[:1], 8)
    with pytest.raises(jf.JFError):
        jf.select_kept_keys(w, n, 8, sink=5, recent=5)
    logits = torch.zeros((1, 2, 50), device="cuda")
    score = torch.zeros((1, 2), device="cuda")
    with pytest.raises(TypeError):
        jf.beam_select(logits.half(), score, 4)
    with pytest.raises(jf.JFError):
        jf.beam_select(logits, score, 65)
    with pytest.raises(jf.JFError):              # finished beams need an end token
        jf.beam_select(logits, score, 4, finished=torch.zeros((1, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(jf.JFError):              # a workspace of the wrong size
        i = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
        jf.jf_beam_select(logits, score, i, i.clone(), torch.zeros((1, 4), device="cuda"),
                          torch.zeros(16, dtype=torch.uint8, device="cuda"))
