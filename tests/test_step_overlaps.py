"""The calls around a step refuse outputs that share a byte with an input, with each other or with the workspace,
whatever the array.  CPU only, and not even run where there is a device: nothing is dereferenced, and a call that
were taken has no device to go on with."""
import ctypes

import pytest
import torch

P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
INVALID = 1
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would be launched")


@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_jf_gb300 import build
    return ctypes.CDLL(build.build())


def at(n, by=0):
    return ctypes.c_void_p((n << 32) + by)      # far apart, aligned, never dereferenced


def none_overlap(fn, args, outputs, sizes, pairs=()):
    """sizes: {argument: bytes} of every array.  An output's last 16 bytes over an array's first and its first over the
    array's last are refused; so is an array that begins where the output does."""
    for out in outputs:
        for other, size in sizes.items():
            if other == out or (out, other) in pairs:
                continue
            base = 40 << 32
            for out_at, other_at in ((base, base), (base, base + sizes[out] - 16), (base + (size - 1) // 16 * 16, base)):
                bad = list(args)
                bad[out], bad[other] = ctypes.c_void_p(out_at), ctypes.c_void_p(other_at)
                assert fn(*bad) == INVALID, (out, other, out_at - base, other_at - base)


ROTATE = [P, i64, P, i64, P, i64, P, P, i32, i32, f32, P, P, f32, P, P, P]


@pytest.mark.parametrize("packed", [False, True])
def test_rotate(lib, packed):
    B, N, T, Hq, Hkv, D, pages, wide = 2, 16, 30, 32, 8, 128, 99, 10
    rows = T if packed else B * N
    fn = lib.jf_rotate_append_kv_packed if packed else lib.jf_rotate_append_kv
    fn.argtypes = ROTATE + [i32] * (9 if packed else 8) + [P] * 5
    args = [at(1), Hq * D, at(2), Hkv * D, at(3), Hkv * D, at(4), at(5), D, 0, 1.0, at(6), at(7), 1e-6, at(8), at(9), at(10),
            B, N] + [T] * packed + [Hq, Hkv, D, 16, wide, pages, at(11), at(12), at(13), None, None]
    q_out = 26 if packed else 25
    sizes = {0: rows * Hq * D * 2, 2: rows * Hkv * D * 2, 4: rows * Hkv * D * 2, 6: rows * 4, 7: D // 2 * 8, 11: D * 2, 12: D * 2,
             14: B * wide * 4, 15: B * 4, 16: (B + packed) * 4, q_out: rows * Hq * D * 2, q_out + 1: pages * 16 * Hkv * D * 2,
             q_out + 2: pages * 16 * Hkv * D * 2}
    none_overlap(fn, args, [q_out + 1, q_out + 2], sizes)
    none_overlap(fn, args, [q_out], {k: v for k, v in sizes.items() if k != 0})     # over q: in place


ADJUST = [P, i32, P, P, P, P, P, P, i32, P, P, P, f32, P]


@pytest.mark.parametrize("packed", [False, True])
def test_adjust(lib, packed):
    B, N, T, V, allowed = 6, 70, 300, 1000, 9
    rows = T if packed else B * N
    fn = lib.jf_adjust_logits_packed if packed else lib.jf_adjust_logits
    fn.argtypes = ADJUST + [i32] * (4 if packed else 3) + [P, i32, P, P]
    args = [at(1), 0, at(2), at(3), at(4), at(5), at(6), at(7), allowed, at(8), at(9), at(10), -float("inf"), at(11),
            B, N] + [T] * packed + [V, at(12), 0, None, None]
    out = 18 if packed else 17
    sizes = {2: B * V * 4, 3: rows * 4, 4: rows * 2 * 8, 5: B * V * 4, 6: allowed * 32 * 4, 7: rows * 4, 9: B * 4, 10: B * 4,
             11: B * 4, 13: (B + packed) * 4, out: rows * V * 2}
    none_overlap(fn, args, [out], sizes)


@pytest.mark.parametrize("packed", [False, True])
def test_shared(lib, packed):
    B, N, T, Hq, Hkv, D, pages, wide, groups = 6, 70, 300, 16, 4, 64, 99, 11, 3
    rows = T if packed else B * N
    fn = lib.jf_tree_attention_shared_packed if packed else lib.jf_tree_attention_shared
    fn.argtypes = [P] * 9 + [i32] * (10 if packed else 9) + [f32, P, P, P, sz, P, P]
    args = [at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9), groups, B, N] + [T] * packed + [
        Hq, Hkv, D, 16, wide, pages, 0.1, at(10), at(11), at(12), 1 << 40, None, None]
    out = 20 if packed else 19
    pool = pages * 16 * Hkv * D * 2
    sizes = {0: rows * Hq * D * 2, 1: pool, 2: pool, 3: B * wide * 4, 4: B * 4, 5: (B + packed) * 4, 6: rows * 2 * 8,
             7: (groups + 1) * 4, 8: groups * 4, out: rows * Hq * D * 2, out + 1: rows * Hq * 4,
             out + 2: 2 * rows * Hq * (D + 1) * 4}       # the workspace holds that much at least
    if not packed:
        args[5] = None                                   # then with lengths: another array to stay clear of
        none_overlap(fn, args, [out, out + 1, out + 2], {k: v for k, v in sizes.items() if k != 5})
        args[5] = at(6)
    none_overlap(fn, args, [out, out + 1, out + 2], sizes)
