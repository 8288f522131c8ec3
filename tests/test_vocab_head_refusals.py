"""What Fp8VocabHead copies by itself (the generator's state, the log sum exp of a training forward) is checked as what the
library is given is: nothing is spread over the rows or changed in type silently.  On the CPU, as test_vocab_head_state.py."""

import pytest
import torch

import fp8_precision_numerics_amd as fm
from test_vocab_head_state import H, T, V, forward, head, host, inputs  # noqa: F401 (host: the entry points' stand-ins)


def train(hd, d, **kw):
    args = dict(rng=d["rng"], lse=torch.zeros(T))
    args.update(kw)
    hd.forward(d["x"], d["residual"], d["norm_weight"], d["norm_bias"], d["targets"], torch.zeros(T), **args)


@pytest.mark.parametrize("rng", [torch.tensor([7]), torch.tensor(7), torch.tensor([[7, 5]]), torch.tensor([7, 5, 3])])
def test_the_generator_has_a_seed_and_an_offset(rng):
    hd, d = head(), inputs()
    hd.quantize_weights(d["weight"])
    with pytest.raises(ValueError, match="rng must be"):
        train(hd, d, rng=rng)


@pytest.mark.parametrize("dtype", [torch.int32, torch.float32, torch.float64])
def test_the_generators_state_is_whole_numbers_of_64_bits(dtype):
    hd, d = head(), inputs()
    hd.quantize_weights(d["weight"])
    with pytest.raises(TypeError, match="rng must be"):
        train(hd, d, rng=d["rng"].to(dtype))


@pytest.mark.parametrize("lse,error", [(torch.zeros(T, T), ValueError), (torch.zeros(2, T), ValueError), (torch.zeros(T + 1), ValueError), (torch.zeros(T, dtype=torch.bfloat16), TypeError),
                                       (torch.zeros(T, dtype=torch.float64), TypeError)])
def test_the_log_sum_exp_is_one_fp32_value_a_row(lse, error):
    hd, d = head(), inputs()
    hd.quantize_weights(d["weight"])
    for on in (True, False):
        with pytest.raises(error, match="lse must be"):
            train(hd, d, lse=lse, train=on)


def test_a_refused_forward_leaves_the_kept_one():
    """A training forward that is refused for its arguments changes nothing that a backward of the one before it sees."""
    hd, d = head(), inputs()
    hd.quantize_weights(d["weight"])
    forward(hd, d)
    with pytest.raises(ValueError):
        train(hd, d, rng=None)
    with pytest.raises(TypeError):
        train(hd, d, lse=torch.zeros(T, dtype=torch.float64))
    assert hd._kept and torch.equal(hd.rng, d["rng"])


@pytest.mark.parametrize("dropout", [0.999995, 1.0, -0.1, float("nan")])
def test_a_dropout_that_drops_everything_is_refused_at_once(dropout):
    with pytest.raises(ValueError, match="dropout"):
        fm.Fp8VocabHead(T, H, V, dropout=dropout, device="cpu")
