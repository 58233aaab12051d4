"""The linear module with an epilogue, and the autograd forms of the operators, on the host."""
import pytest
import torch

pytest.importorskip("int8_mixed_precision_rowwise_amd")
from int8_mixed_precision_rowwise_amd import training as T  # noqa: E402

bf = torch.bfloat16


@pytest.mark.parametrize("bias", [True, False])
def test_from_linear_keeps_the_parameters(bias):
    lin = torch.nn.Linear(24, 16, bias=bias, dtype=bf)
    cfg = T.Int8MixedPrecisionConfig(stochastic_rounding=True)
    m = T.Int8MixedPrecisionActLinear.from_linear(lin, cfg, 7, activation="silu")
    assert type(m) is T.Int8MixedPrecisionActLinear and m.weight is lin.weight and m.bias is lin.bias
    assert (m.in_features, m.out_features, m.config, m.seed, m.step, m.activation) == (24, 16, cfg, 7, 0, "silu")
    assert "activation=silu" in repr(m) and f"bias={bias}" in repr(m)
    assert T.Int8MixedPrecisionActLinear.from_linear(lin, cfg, 7).activation == "none"
    again = T.Int8MixedPrecisionActLinear(24, 16, bias=bias, activation="silu", config=cfg)
    again.load_state_dict(m.state_dict())
    assert again.seed == 7 and torch.equal(again.weight, lin.weight)
    # what the forward hands on is all there: the call is refused for its device only
    with pytest.raises(ValueError, match="device tensors"):
        m(torch.zeros(3, 24, dtype=bf))


def test_from_linear_refuses_what_the_constructor_refuses():
    lin = torch.nn.Linear(24, 16, dtype=bf)
    for bad in (dict(fp8=True), dict(output=False), dict(grad_input=False), dict(grad_weight=False)):
        with pytest.raises(ValueError, match="all three GEMMs in INT8"):
            T.Int8MixedPrecisionActLinear.from_linear(lin, T.Int8MixedPrecisionConfig(**bad), 0)
    with pytest.raises(ValueError, match="activation must be one of"):
        T.Int8MixedPrecisionActLinear.from_linear(lin, T.Int8MixedPrecisionConfig(), 0, activation="tanh")
