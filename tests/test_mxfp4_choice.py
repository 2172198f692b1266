"""The choice between the MXFP4 products' kernels, replayed on the host: every kernel is taken by a size that the GPU tests run, with
every format of its result; and the check of a result's error as a whole finds what it is there to find."""
import pytest
import torch

import mxfp4_choice
from test_gpu_mxfp4_shapes import GRADIENTS, PRODUCTS, SWIGLU, check_rms, drawn, rms


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    return mxfp4_choice.load(tmp_path_factory.mktemp("choice"))


@pytest.mark.parametrize("kind", PRODUCTS)
def test_products_take_every_kernel(choice, kind):
    x4 = kind == "mxfp4"
    taken = [choice.gemm_shape(x4, 0, 0, rows, E, N, K) for E, rows, N, K in PRODUCTS[kind]]
    assert taken == list(range(choice.gemm_shapes(x4, 0)))


@pytest.mark.parametrize("kind, h_kind", SWIGLU)
def test_gate_and_up_take_every_kernel(choice, kind, h_kind):
    x4, codes = kind == "mxfp4", h_kind == "mxfp4"
    taken = [choice.gemm_shape(x4, 1, codes, rows, E, f, d) for E, rows, f, d in SWIGLU[kind, h_kind]]
    assert taken == [i for i in range(choice.gemm_shapes(x4, 1)) if not codes or choice.holds_groups(x4, i)]


@pytest.mark.parametrize("pairs", GRADIENTS)
def test_gradients_take_every_kernel(choice, pairs):
    taken = [choice.dgrad_shape(pairs - 1, rows, E, N, K) for E, rows, N, K in GRADIENTS[pairs]]
    assert taken == list(range(choice.dgrad_shapes()))


def test_drawn_cases_are_of_every_kind():
    cases = drawn(2)
    assert len(cases) == 12 and len({c["name"] for c in cases}) == 12


@pytest.mark.parametrize("K", [544, 7168])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_check_of_the_whole_error(K, out):
    """Sums in fp32 pass; with blocks of 256 rounded to bf16, or with one product left out, they do not."""
    g = torch.Generator().manual_seed(K)
    x, w = (torch.randn(n, K, generator=g, dtype=torch.float64) for n in (64, 48))
    want = x @ w.t()
    bound = K * 2.0 ** -23 * rms(want)
    check_rms((x.float() @ w.float().t()).to(out), want, bound)
    low = torch.zeros_like(want)
    for k in range(0, K, 256):
        low = (low + x[:, k:k + 256] @ w[:, k:k + 256].t()).to(torch.bfloat16).double()
    for wrong in ([low] if out is torch.float32 or K > 544 else []) + [x[:, 1:] @ w[:, 1:].t()]:
        with pytest.raises(AssertionError):
            check_rms(wrong.to(out), want, bound)
