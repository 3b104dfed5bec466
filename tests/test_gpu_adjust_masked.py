"""What forbidden tokens get in adjusted logits: a finite value is finite in the output's type too."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def jf():
    from tree_speculative_decoding_jf_gb300 import build
    build.build()
    from tree_speculative_decoding_jf_gb300 import jf as mod
    return mod


@pytest.mark.parametrize("V", [2048, 501])
@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("masked", [torch.finfo(F32).min, torch.finfo(F32).max, torch.finfo(BF16).min, -3.39e38, 3.3962e38, -1e30,
                                    -65504.0, 0.0, -float("inf"), float("inf")])
def test_masked_value(jf, types, V, masked):
    g = torch.Generator().manual_seed(V)
    logits = torch.randn((1, 3, V), generator=g).to(types[0]).cuda()
    allowed = torch.randint(-2 ** 31, 2 ** 31, (3, -(-V // 32)), generator=g).to(torch.int32)
    allowed[1] = 0
    ok = ((allowed.long()[:, torch.arange(V) // 32] >> (torch.arange(V) % 32)) & 1).bool().cuda()
    out = torch.full(logits.shape, -7.0, dtype=types[1], device="cuda")
    jf.adjust_logits(logits, allowed=allowed.cuda(), masked=masked, out=out)
    # Rounded to nearest even on the way; only a finite value that would round past the range does not.
    want = torch.tensor(masked, dtype=F32).to(types[1])
    if abs(masked) < float("inf") and not torch.isfinite(want):
        want = torch.tensor(torch.finfo(types[1]).max if masked > 0 else torch.finfo(types[1]).min, dtype=types[1])
    assert (out[0][~ok] == want.item()).all() and torch.equal(out[0][ok], logits[0][ok].to(types[1]))
