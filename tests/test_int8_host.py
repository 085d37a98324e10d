"""Refusals and host logic of the 8-bit layer and of the optimizer (no GPU)."""

import pytest
import torch


def test_int8_buffers_are_checked(metis_lib):
    with pytest.raises(ValueError):
        metis_lib.Int8(0, 16)
    with pytest.raises(ValueError):
        metis_lib.Int8(4, 16, codes=torch.zeros(4, 16, dtype=torch.int8), scales=torch.zeros(4))      # not CUDA
    with pytest.raises(ValueError):
        metis_lib.Int8(4, 16, codes=torch.zeros(4, 16), scales=torch.zeros(4))
    with pytest.raises(ValueError):
        metis_lib.Int8(4, 16, codes=torch.zeros(16, 4, dtype=torch.int8).t(), scales=torch.zeros(4))
    with pytest.raises(ValueError):
        metis_lib.Int8(4, 16, codes=torch.zeros(4, 16, dtype=torch.int8), scales=torch.zeros(8)[::2])


def test_dense_matrix_check(metis_lib):
    with pytest.raises(ValueError):
        metis_lib._dense(torch.zeros(4, 4), "M")
    with pytest.raises(ValueError):
        metis_lib._dense(torch.zeros(4, 4, dtype=torch.float16), "M")


def test_int8_linear_refusals(metis_lib):
    from spectral_quantized_gemm_b200.int8_linear import Int8Linear
    for sizes in ((0, 4), (4, 0), (131072, 4), (4, 131072)):
        with pytest.raises(ValueError):
            Int8Linear(*sizes)
    layer = Int8Linear(5, 7)
    assert layer.weight.shape == (5, 7) and layer.weight.abs().max() <= 5 ** -0.5
    with pytest.raises(ValueError):
        layer(torch.zeros(2, 6))
    with pytest.raises(ValueError):
        layer(torch.zeros(131072, 5))


def test_null_context_is_an_argument_error(metis_lib):
    assert metis_lib._quant_i8(None, None, 1, 1, 1, 0, None, None) == 1
    assert metis_lib._gemm_i8(None, None, None, None, 0, 0) == 1
    assert metis_lib._linear_i8(None, None, 1, 0, None, None, None, 0, 0) == 1
    assert metis_lib._adamw(None, None, 0, None) == 1


@pytest.mark.parametrize("bad", [dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(state_bits=16), dict(rounding="up"),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(weight_decay=-0.1), dict(lr=-1.0),
                                 dict(lr=float("nan")), dict(lr=torch.tensor(1e-3)),
                                 dict(lr=torch.tensor(1e-3), capturable=True)])
def test_adamw_refuses_bad_options(metis_lib, bad):
    from spectral_quantized_gemm_b200.optim import AdamW
    with pytest.raises(ValueError):
        AdamW([torch.nn.Parameter(torch.zeros(3))], **bad)


def test_adamw_refuses_bad_parameters(metis_lib):
    from spectral_quantized_gemm_b200.optim import AdamW
    with pytest.raises(ValueError):
        AdamW([torch.nn.Parameter(torch.zeros(3, dtype=torch.float64))])
    with pytest.raises(ValueError):
        AdamW([torch.nn.Parameter(torch.zeros(3, 8)[:, ::2])])
    p = torch.nn.Parameter(torch.zeros(3))
    with pytest.raises(ValueError):
        AdamW([p, p])
    opt = AdamW([p])
    with pytest.raises(ValueError):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.zeros(2))], "state_bits": 4})
    assert len(opt.param_groups) == 1
    p.grad = torch.ones(3)
    with pytest.raises(ValueError):
        opt.step()                       # a CPU parameter


def test_adamw_without_gradients_does_nothing(metis_lib):
    from spectral_quantized_gemm_b200.optim import AdamW
    p = torch.nn.Parameter(torch.ones(3))
    opt = AdamW([p])
    assert opt.step() is None and opt.step(lambda: 5) == 5
    assert not opt.state and torch.equal(p, torch.ones(3))


def test_entry_layout_matches_the_struct(metis_lib):
    """The optimizer fills the entries as eight 64-bit words each."""
    from spectral_quantized_gemm_b200 import optim
    T = metis_lib.AdamWTensor
    assert metis_lib.ctypes.sizeof(T) == 8 * optim.ENTRY_WORDS
    assert [getattr(T, f).offset for f, _ in T._fields_] == [0, 8, 16, 24, 32, 40, 48, 56, 60]


@pytest.mark.parametrize("dtype,ld", [(torch.bfloat16, 80), (torch.float32, 80)])
def test_layer_outputs_are_padded_and_no_views(metis_lib, dtype, ld):
    from spectral_quantized_gemm_b200.int8_linear import _output
    for rows, cols in ((3, 77), (1, 77), (3, ld), (0, 77)):
        y = _output(rows, cols, dtype, "cpu")
        assert y.shape == (rows, cols) and y.stride() == (ld, 1) and not y._is_view()
