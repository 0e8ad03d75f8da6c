"""Further refusals of the operators around the gather, on the host, before any CUDA call."""
import pytest

from test_mla_host import plan

# addresses of a call without overlap: 2 requests, a table of 2 x 4, 4 free ids, 10 tokens
PLACES = dict(ctx=4096, new=4104, bt=4112, free=4144, lens=4160, cu=4168, cuseq=4180, taken=4192, err=4196, slots=4200,
              pos=4280, t2s=4320)


@pytest.mark.parametrize("name,at", [
    ("lens", 4096), ("lens", 4104), ("lens", 4100), ("lens", 4156), ("cu", 4088), ("cu", 4096), ("cuseq", 4096),
    ("cuseq", 4152), ("taken", 4108), ("taken", 4144), ("err", 4096), ("slots", 4096), ("slots", 4024), ("slots", 4152),
    ("pos", 4096), ("pos", 4060), ("t2s", 4104), ("t2s", 4156), ("bt", 4096), ("bt", 4068), ("bt", 4132), ("ctx", 4160),
    ("new", 4160), ("ctx", 4140), ("free", 4112), ("free", 4316)])
def test_plan_refuses_results_in_place_of_its_inputs(cuda_lib, name, at):
    """Lengths and free ids are read by every part of the call while others write results."""
    assert plan(cuda_lib, **{**PLACES, name: at}) == 2
