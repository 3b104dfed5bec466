"""Sizes that attention over shared prefixes takes and refuses: what its schedule's 32-bit positions allow, on either
side.  CPU only: what is taken is refused for its missing workspace (without a device: for that), before any launch."""
import ctypes

import pytest

P, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
UNSUPPORTED, TOO_SMALL, CUDA = 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_jf_gb300 import build
    return ctypes.CDLL(build.build())


def at(n):
    return ctypes.c_void_p(n << 48)      # far apart, aligned, never dereferenced


def status(lib, B, N, Hq, Hkv, D, max_pages, n_groups, T=0):
    head = [at(1), at(2), at(3), at(4), at(5)]
    mid = [at(7), at(8), at(9), n_groups, B, N]
    rest = [Hq, Hkv, D, 16, max_pages, 99, 0.1, at(10), None, None, 0, None, None]
    if T:
        fn = lib.jf_tree_attention_shared_packed
        fn.argtypes = [P] * 9 + [i32] * 10 + [f32, P, P, P, sz, P, P]
        return fn(*head, at(6), *mid, T, *rest)
    fn = lib.jf_tree_attention_shared
    fn.argtypes = [P] * 9 + [i32] * 9 + [f32, P, P, P, sz, P, P]
    return fn(*head, None, *mid, *rest)


def taken(s):
    assert s in (UNSUPPORTED, TOO_SMALL, CUDA), s
    return s != UNSUPPORTED


def stated(B, N, Hq, Hkv, max_pages, n_groups, T=0):
    """The limit as include/jf.h words it."""
    M, G = T or B * N, Hq // Hkv
    r = M * G / n_groups
    few = lambda rows: 16 if rows <= 16 else 32 if rows <= 32 else 64  # noqa: E731
    if 2 * M * Hq >= 2 ** 31 - 2 ** 20:
        return False
    if r <= 64:
        return Hkv * (2 * M * G / few(r) + B + n_groups) * (max_pages + 4) < 2 ** 31
    ok = Hkv * (2 * M * G / (128 if r <= 128 else 256) + B + n_groups) * (max_pages / 8 + 7) < 2 ** 31
    return ok and (N * G > 64 or Hkv * (M * G / few(N * G) + B) * (max_pages + 4) < 2 ** 31)


@pytest.mark.parametrize("B,N,Hq,Hkv,max_pages", [(256, 256, 32, 8, 8192), (128, 256, 64, 8, 8192), (64, 1024, 32, 8, 8192),
                                                  (64, 16, 32, 8, 1 << 20), (4096, 1, 32, 8, 8192)])
def test_ordinary_sizes(lib, B, N, Hq, Hkv, max_pages):
    for groups in (1, B // 8):
        for D in (64, 128):
            assert taken(status(lib, B, N, Hq, Hkv, D, max_pages, groups))
            assert taken(status(lib, B, N, Hq, Hkv, D, max_pages, groups, T=B * N - 5))


# B, N, Hq, Hkv, D, groups: 16, 32 and 64 rows a group, one and two row tiles, own parts in either kernel
SIZES = [(4096, 1, 128, 16, 128, 2048), (4000, 1, 64, 16, 64, 500), (4096, 4, 64, 16, 128, 1024), (4096, 1, 64, 64, 128, 1),
         (1024, 4, 256, 8, 64, 1024), (300, 500, 16, 16, 64, 300), (4096, 100, 128, 64, 128, 8), (4096, 16, 64, 16, 64, 4096)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_either_side_of_the_limit(lib, case, packed):
    B, N, Hq, Hkv, D, groups = SIZES[case]
    T = B * N - 3 if packed else 0
    lo, hi = -(-N // 16), 1 << 26                        # refused for its own sake beyond
    assert taken(status(lib, B, N, Hq, Hkv, D, lo, groups, T))
    if taken(status(lib, B, N, Hq, Hkv, D, hi, groups, T)):
        assert stated(B, N, Hq, Hkv, hi, groups, T)      # none of these is that small
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if taken(status(lib, B, N, Hq, Hkv, D, mid, groups, T)):
            lo = mid
        else:
            hi = mid
    # Everything that the header promises is taken, and little beyond it.
    assert not stated(B, N, Hq, Hkv, hi, groups, T)
    assert stated(B, N, Hq, Hkv, int(lo * 0.99) - 64, groups, T)


def test_rows_of_the_workspace(lib):
    assert taken(status(lib, 1, 4096, 128, 128, 64, 256, 1))
    T = (2 ** 31 - 2 ** 20) // (2 * 128)
    assert not taken(status(lib, 4096, 4096, 128, 128, 64, 256, 4096, T=T))
    assert taken(status(lib, 4096, 4096, 128, 128, 64, 256, 4096, T=T - 1))


def test_largest_tree_of_packed_rows():
    """What the packed form takes for its largest tree where it is not told."""
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf
    #   T    B  pages words  nodes
    for T, B, pages, words, want in [(7, 7, 1, 1, 1), (1, 1, 1, 1, 1), (20, 3, 100, 1, 18), (500, 3, 100, 1, 64),
                                     (500, 3, 2, 1, 32), (500, 3, 100, 2, 128), (70, 3, 100, 2, 68),
                                     (66, 3, 100, 2, 65), (5, 3, 100, 2, 65), (9000, 2, 1000, 64, 4096)]:
        got = jf._largest_tree(T, B, pages, words)
        assert got == want and (got + 63) // 64 == words, (T, B, pages, words)
