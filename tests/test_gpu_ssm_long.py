"""The scan over many chunks in one workgroup: sets of tiles and rings of decays are used again and again
(three sets and three decays in the form for p = 128 in bf16, p / 8 decays in the others and in the pass that
forms a split's states).  Definitions, tolerances and checks are those of the short cases.
"""
import pytest
import torch

from tests import mixers_reference as ref
from tests.test_gpu_ssm import DT, _check, _cuda, _inputs, _kda

pytestmark = pytest.mark.gpu

# B, T, H, G, n, p, dtype, strong, lens, seg_len
LONG = [
    (2, 1400, 2, 1, 128, 128, "bf16", False, [1400, 777], 1408),
    (2, 1400, 2, 2, 64, 128, "bf16", True, [1301, 1400], 1408),
    (1, 1473, 2, 1, 128, 64, "bf16", False, None, 1536),
    (2, 1350, 2, 1, 64, 64, "bf16", False, [1350, 641], 1408),
    (1, 1290, 2, 1, 128, 128, "f32", False, None, 1344),
    (2, 1290, 2, 2, 64, 64, "f32", True, [1290, 100], 1344),
    (1, 1290, 2, 1, 128, 64, "f32", False, [1289], 1344),
    (1, 1290, 2, 1, 64, 128, "f32", False, None, 1344),
    # split: 18 chunks a segment, whose states and outputs both wrap
    (2, 2300, 2, 1, 128, 128, "bf16", False, [2300, 1200], 1152),
    (1, 3500, 1, 1, 128, 64, "bf16", False, None, 1152),
    (1, 2400, 1, 1, 64, 128, "bf16", False, [2395], 1152),
    (1, 2310, 1, 1, 128, 128, "f32", False, None, 1152),
    (1, 2310, 1, 1, 64, 64, "f32", False, None, 640),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c[:7])) + f"-seg{c[-1]}")
def test_ssm_prefill_over_many_chunks_matches_definition(case):
    kda = _kda()
    B, T, H, G, n, p, dtype, strong, lens, seg = case
    print("ssm_prefill", case, flush=True)
    i = _inputs(B, T, H, G, n, p, dtype, 21, strong=strong)
    if not strong:
        i["A"] = i["A"] / 100        # states that remember hundreds of tokens
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    y = torch.full((B, T, H, p), 5.0, dtype=DT[dtype], device="cuda")
    S = torch.full((B, H, n, p), float("nan"), device="cuda")
    kda.ssm_prefill(**_cuda(i), lens=None if ln is None else ln.cuda(), seg_len=seg, y=y, S_T=S)
    torch.cuda.synchronize()
    _check(i, y, S, ln, dtype)
    for b, m in enumerate(ref.lens_of(ln, B, T)):
        assert bool((y[b, m:] == 5.0).all())
