"""fp32 products keep their sums in two levels: runs of 8 steps (256 products of a wave's own), then those. Shown with
sums that one chain of additions gets wrong: a 1 and then products of 2^-27, which each change nothing beside the
1 (four of them together neither: 2^-25 is half of half its last place), though thousands do. In two levels only the
run that holds the 1 loses them; the other runs are whole numbers of 2^-27 below 2^-18, exact, and so is adding a run
of 2^-19 to the 1."""
import numpy as np
import pytest
import torch

import token_dispatch_expert_amd as moe

import gpu_harness as H
import training_ref as ref

pytestmark = pytest.mark.gpu

F32 = torch.float32
TINY = 2.0 ** -27
RUN = 256
SPLIT = 4          # the most groups of waves that share a contraction, each with sums of its own
N_SUM = 8192       # whole runs, also of a split contraction


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


# what the run with the 1 may lose; the outer sums and the join of the groups are exact
BOUND = RUN * TINY


def test_one_chain_would_fail():
    """The bound tells the two apart: a chain over a quarter of the contraction loses more than it."""
    acc = np.float32(1)
    for _ in range(N_SUM // SPLIT // 4):
        acc = np.float32(acc + np.float32(4 * TINY))  # (four products of an instruction at best summed first)
    assert (N_SUM // SPLIT - 1) * TINY - float(acc - 1) > 2 * BOUND


def one_and_tiny(shape, along, dev):
    """TINY everywhere but a 1 at the start of axis `along`."""
    t = torch.full(shape, TINY, device=dev)
    t.select(along, 0).fill_(1.0)
    return t


# rows, experts, width: tiles of 16 x 64 with the contraction split in four and whole, 64 x 64 split in two and whole
@pytest.mark.parametrize("rows,E,width", [(20, 1, 72), (800, 20, 648), (1024, 1, 648), (2048, 1, 1032)],
                         ids=["16-rows-split", "16-rows", "64-rows-split", "64-rows"])
def test_rows_products(dev, rows, E, width):
    off = ref.offsets_of([rows // E] * E, dev)
    true = 1.0 + (N_SUM - 1) * TINY
    x, w = one_and_tiny((rows, N_SUM), 1, dev), torch.ones((E, width, N_SUM), device=dev)
    y = torch.empty((rows, width), device=dev)
    moe.moe_grouped_gemm(x, off, w, y)
    assert (y.double() - true).abs().max() <= BOUND
    w = w.reshape(E, N_SUM, width)
    dx = torch.empty((rows, width), device=dev)
    moe.moe_grouped_gemm_dgrad(x, off, w, dx)
    assert (dx.double() - true).abs().max() <= BOUND
    dy2 = torch.full((rows, N_SUM), TINY, device=dev)  # a second pair without a 1: nothing of it is lost
    moe.moe_grouped_gemm_dgrad(x, off, w, dx, dy2=dy2, w2=w)
    assert (dx.double() - true - N_SUM * TINY).abs().max() <= BOUND


@pytest.mark.parametrize("N,K", [(72, 136), (1032, 1160)], ids=["split", "whole"])
def test_weight_gradient(dev, N, K):
    dy, x = one_and_tiny((N_SUM, N), 0, dev), torch.ones((N_SUM, K), device=dev)
    dw = torch.empty((1, N, K), device=dev)
    moe.moe_grouped_gemm_wgrad(dy, x, ref.offsets_of([N_SUM], dev), dw)
    assert (dw.double() - 1.0 - (N_SUM - 1) * TINY).abs().max() <= BOUND
