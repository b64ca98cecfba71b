"""What H3BlockTrain refuses before it launches anything: its calls see only
pointers, so tensors of other sizes would be read past their ends."""
import pytest
import torch

from omni_modal_diffusion_b200 import build as B
from omni_modal_diffusion_b200 import h3
from omni_modal_diffusion_b200.pipeline import H3BlockTrain

BF16 = torch.bfloat16
D, H, F, I = 64, 1, 128, 128


@pytest.fixture(scope="module")
def block():
    B.build()
    return H3BlockTrain(h3.make_dims(D, H, F), h3.h3_make_ranges(10, 0, 20), device="cpu")


def arguments():
    W = {"Wqkv": (3 * I, D), "qn_w": (128,), "kn_w": (128,), "Wo": (D, I), "Wgu": (2 * F, D), "Wd": (D, F)}
    return {"x": torch.zeros(128, D), "mod": torch.zeros(3, 6, D), "pos": torch.zeros(128, 3),
            "W": {n: torch.zeros(*s, dtype=BF16) for n, s in W.items()}}


WRONG = {"x": [(D,), (1, D), (30, D), (256, D)], "mod": [(3, 3, D), (6, D), (3, 6, 2 * D)], "pos": [(30, 3), (128, 2)],
         "Wqkv": [(I, D), (3 * I, 2 * D)], "qn_w": [(64,)], "kn_w": [(256,)], "Wo": [(D, D)], "Wgu": [(F, D)], "Wd": [(F,)]}


@pytest.mark.parametrize("name,shape", [(n, s) for n, shapes in WRONG.items() for s in shapes], ids=str)
@pytest.mark.parametrize("call", ("forward", "backward"))
def test_tensors_of_other_sizes(block, call, name, shape):
    a = arguments()
    if name in a:
        a[name] = torch.zeros(*shape)
    else:
        a["W"][name] = torch.zeros(*shape, dtype=BF16)
    with pytest.raises(ValueError, match="elements"):
        getattr(block, call)(a["x"], a["mod"], a["pos"], a["W"])


@pytest.mark.parametrize("call", ("forward", "backward"))
def test_missing_weights(block, call):
    a = arguments()
    del a["W"]["Wo"]
    with pytest.raises(ValueError, match="Wo"):
        getattr(block, call)(a["x"], a["mod"], a["pos"], a["W"])


@pytest.mark.parametrize("name", ("x", "mod", "pos", "Wd"))
@pytest.mark.parametrize("call", ("forward", "backward"))
def test_tensors_on_another_device(block, call, name):
    a = arguments()
    where = a if name in a else a["W"]
    where[name] = where[name].to("meta")
    with pytest.raises(ValueError, match=f"{'dx' if (name, call) == ('x', 'backward') else name} is on meta"):
        getattr(block, call)(a["x"], a["mod"], a["pos"], a["W"])


def test_backward_comes_after_forward(block):
    """Until a forward call has run, what backward reads of it is not there."""
    a = arguments()
    with pytest.raises(RuntimeError, match="forward"):
        block.backward(a["x"], a["mod"], a["pos"], a["W"])
