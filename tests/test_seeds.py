"""Inputs drawn from torch's own generators are the same in every run, whatever ran before."""
import pytest
import torch


@pytest.mark.parametrize("n", [3, 5, 3])
def test_every_test_starts_from_the_same_seed(n):
    assert torch.equal(torch.rand(n), torch.rand(n, generator=torch.Generator().manual_seed(0)))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 5, 3])
def test_and_on_the_gpu(n):
    assert torch.equal(torch.rand(n, device="cuda"), torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)))
