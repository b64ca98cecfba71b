"""H3BlockTrain's arguments where a call runs."""
import pytest
import torch

from omni_modal_diffusion_b200 import h3
from omni_modal_diffusion_b200.pipeline import H3BlockTrain

pytestmark = pytest.mark.gpu
D, H, F, I = 64, 1, 128, 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    from omni_modal_diffusion_b200 import build
    build.build()
    assert torch.cuda.is_available()


def test_frozen_names_from_a_generator():
    shapes = {"Wqkv": (3 * I, D), "qn_w": (128,), "kn_w": (128,), "Wo": (D, I), "Wgu": (2 * F, D), "Wd": (D, F)}
    W = {n: torch.ones(*s, dtype=torch.bfloat16, device="cuda") for n, s in shapes.items()}
    tr = H3BlockTrain(h3.make_dims(D, H, F), h3.h3_make_ranges(10, 0, 20))
    x, mod, pos = (torch.zeros(*s, device="cuda") for s in ((128, D), (3, 6, D), (128, 3)))
    tr.forward(x, mod, pos, W)
    g = tr.backward(torch.zeros_like(x), mod, pos, W, frozen=(n for n in ("Wo", "Wgu", "mod")))
    torch.cuda.synchronize()
    assert h3.h3_device_status() == 0
    assert sorted(g) == ["Wd", "Wqkv", "kn_w", "qn_w"]
