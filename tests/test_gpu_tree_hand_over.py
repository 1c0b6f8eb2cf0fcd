"""A captured serving step plans one step ahead: its layers say so when their pages are to go to the device."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


@pytest.mark.parametrize("graphs", [True, False], ids=["graphs", "direct"])
@pytest.mark.parametrize("kind", ["LayerCache", "F16LayerCache"])
def test_layers_of_a_serving_step(kind, graphs):
    import torch
    from mixed_precision_bit_gb300 import cache, kitty
    cfg = kitty.Config(num_kv_heads=2, num_q_heads=8, in_dtype=kitty.BF16)
    layers = [getattr(cache, kind)(cfg, 3, 4, 12) for _ in range(2)]
    q = torch.zeros((3, 8, 128), dtype=torch.int16, device="cuda")
    layers[0].attend(q, torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda"))  # outside any capture
    torch.cuda.synchronize()
    step = cache.ServingStep(layers, graphs=graphs)
    for x in (*step.q, *step.k_new, *step.v_new):
        x.zero_()
    step.run()
    if graphs:
        with pytest.raises(ValueError, match="has not been made.*one step ahead"):
            layers[0].pages_to_device()
        layers[0].clear()  # (which drops the plan)
    layers[0].pages_to_device()
    layers[0].pages_to_host()
