"""How near the bf16 chunked prefill of the grouped gated delta rule comes to the
float64 form: the outputs' rounding to bf16 is all that shows of them."""
import numpy as np
import pytest
import torch

import gdn_reference as ref
from gdn_reference import f64, rel
from linear_attention_serving_k1_gb300 import kda

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
# Before the outputs are rounded, their relative error (2-norm): S, P and U in the
# output's products and T, X in those that make U, each carried as two bf16 terms (2^-16
# at most, dropped products of two small terms among them), and the carried state's
# own error of the same size.  Eight such terms.
EPS_OUT = 8 * 2.0 ** -16
# Rounding turns an error e of a value into a whole step with probability e / step, so the
# mean square against the correctly rounded values is e times the step, which is 2^-7
# of a value at most.
TOL_ROUNDED = float(np.sqrt(2.0 ** -7 * EPS_OUT))


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def _rounded(x):
    return f64(torch.tensor(x).to(BF16))


@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(2, 4, 128, 128), (1, 3, 128, 192), (2, 2, 64, 64)])
@pytest.mark.parametrize("lens,decay", [([300, 65], "layer"), ([1, 64, 127, 500], -0.01), ([400], 0.0), ([200, 200], -3.0)])
def test_outputs_are_the_rounded_values(Hk, Hv, Dk, Dv, lens, decay):
    x = ref.inputs(sum(lens), Hk, Hv, Dk, Dv, BF16, seed=41, decay=decay)
    s0 = 0.3 * torch.randn(len(lens), Hv, Dk, Dv, generator=torch.Generator().manual_seed(7))
    out, _, _ = kda.gdn_prefill(*[y.cuda() for y in x], s0.cuda(), _cu(lens), max_seq_len=max(lens))
    assert rel(f64(out), _rounded(ref.prefill(*x, s0.numpy(), lens)[0])) <= TOL_ROUNDED


def test_outputs_of_segments_are_the_rounded_values():
    """Few long chains, in segments whose starts come from a join."""
    lens = [1600, 300]
    x = ref.inputs(sum(lens), 1, 2, 128, 128, BF16, seed=42, decay=-0.02)
    out, _, _ = kda.gdn_prefill(*[y.cuda() for y in x], None, _cu(lens))
    assert rel(f64(out), _rounded(ref.prefill(*x, None, lens)[0])) <= TOL_ROUNDED
