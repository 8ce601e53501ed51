"""How near the prefill of the grouped gated delta rule comes to the float64 form: of
bf16 outputs only their rounding shows, and states keep their precision over long
sequences, in segments, and with weak decays and none."""
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


# States of the chunked form: of the four operands on their way (S, X, U, T), each the
# sum of two bf16 terms, the second's rounding is 2^-18 of the value in the mean square;
# together 2^-17, and as much again for what the state still holds of earlier chunks.
TOL_STATE = 2.0 ** -16


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 192)])
@pytest.mark.parametrize("decay", [0.0, -1e-3, -0.02, "layer"])
@pytest.mark.parametrize("lens,hint", [([1500, 64, 640], 64), ([2000, 300], 2000)])
def test_states_of_long_sequences(Dk, Dv, decay, lens, hint):
    """Without decay, with a weak one and a layer's, in one pass (a hint of short sequences) and in segments."""
    x = ref.inputs(sum(lens), 1, 1, Dk, Dv, BF16, seed=43, decay=decay)
    s0 = 0.3 * torch.randn(len(lens), 1, Dk, Dv, generator=torch.Generator().manual_seed(3))
    _, final, ck = kda.gdn_prefill(*[y.cuda() for y in x], s0.cuda(), _cu(lens), ckpt_stride=64, max_seq_len=hint)
    _, want, wck = ref.prefill(*x, s0.numpy(), lens, 64)
    for got, w in [*zip(final, want), *zip(ck, wck)]:
        assert rel(f64(got), w) <= TOL_STATE


@pytest.mark.parametrize("Dk,Dv", [(128, 64), (64, 192)])
@pytest.mark.parametrize("decay", [0.0, -1e-3, -0.02, "layer"])
def test_fp32_states_of_long_sequences(Dk, Dv, decay):
    """A few roundings of the state's own size, whatever the length; the same decay at every token adds its own rounding (at
    most a half step, 2^-25 below 1) up over the state's memory of 1 / |g| tokens."""
    lens = [1500, 64]
    x = ref.inputs(sum(lens), 1, 1, Dk, Dv, torch.float32, seed=44, decay=decay)
    _, final, ck = kda.gdn_prefill(*[y.cuda() for y in x], None, _cu(lens), ckpt_stride=64)
    _, want, wck = ref.prefill(*x, None, lens, 64)
    memory = 1 / abs(decay) if decay not in ("layer", 0.0) else 0.0
    tol = 16 * 2.0 ** -24 + memory * 2.0 ** -25
    for got, w in [*zip(final, want), *zip(ck, wck)]:
        assert rel(f64(got), w) <= tol


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64)])
@pytest.mark.parametrize("decay", [-1e-4, -1e-3, -4e-3, -0.03])
def test_fp32_states_under_the_same_weak_decay_throughout(Dk, Dv, decay):
    """The rounding of the decays does not add up from token to token: at most half a step (2^-25 below 1) for every 64
    tokens that the state remembers, beside a few roundings of the state's own size."""
    lens = [2000]
    x = ref.inputs(sum(lens), 1, 2, Dk, Dv, torch.float32, seed=45, decay=decay)
    _, final, ck = kda.gdn_prefill(*[y.cuda() for y in x], None, _cu(lens), ckpt_stride=320)
    _, want, wck = ref.prefill(*x, None, lens, 320)
    tol = 16 * 2.0 ** -24 + min(2000, 1 / abs(decay)) / 64 * 2.0 ** -25
    for got, w in [*zip(final, want), *zip(ck, wck)]:
        assert rel(f64(got), w) <= tol
