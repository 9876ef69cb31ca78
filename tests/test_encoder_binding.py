"""The binding of the embedding head's operators on a host without a GPU: which way a call takes, and what it refuses
before any device work."""
import pytest
import torch

from late_interaction_retrieval_amd import binding as bd


@pytest.fixture
def step(monkeypatch):
    """A table of host tensors, and the C entry point replaced by one that counts its calls."""
    calls = []
    tab = bd.AdamWTensors.zeros([torch.zeros(5)])

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

        def maxsim_adamw(self, *args):
            calls.append(args)
            return bd.MAXSIM_OK

    real = bd._lib
    monkeypatch.setattr(bd, "_lib", Lib())
    return tab, calls


@pytest.mark.parametrize("status", range(1, 8))
def test_a_step_that_failed_is_not_made_again(step, monkeypatch, status):
    """The extension's call may have launched a part of the step: its status is raised, and no second call follows."""
    tab, calls = step
    monkeypatch.setattr(bd._fast, "adamw", lambda *a: status)
    with pytest.raises(bd.MaxSimError) as e:
        bd.maxsim_adamw(tab, [torch.zeros(5)], 1)
    assert e.value.status == status and not calls


def test_a_step_that_was_made_is_not_made_again(step, monkeypatch):
    tab, calls = step
    monkeypatch.setattr(bd._fast, "adamw", lambda *a: bd.MAXSIM_OK)
    assert bd.maxsim_adamw(tab, [torch.zeros(5)], 1) is None and not calls


def test_a_step_that_the_extension_leaves_alone_goes_the_general_way(step, monkeypatch):
    tab, calls = step
    monkeypatch.setattr(bd._fast, "adamw", lambda *a: None)
    with pytest.raises(ValueError, match="must be on the device"):  # host tensors
        bd.maxsim_adamw(tab, [torch.zeros(5)], 1)
