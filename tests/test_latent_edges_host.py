"""CPU checks of the latent operators at their edges: what the sources may not hold, and refusals."""
import pathlib
import re

from gated_deltanet_linear_mixer_gb300 import _build


def test_no_load_is_multicast():
    """One library serves single processes and replicas of several GPUs: no thread block's bulk load
    writes into another's shared memory."""
    files = [p for p in pathlib.Path(_build.CSRC).iterdir() if p.suffix in (".cu", ".cuh", ".h", ".cpp")]
    assert len(files) > 20
    for p in files:
        text = re.sub(r'"\s*"', "", p.read_text())  # literals side by side are one
        assert not re.search(r"cp\.async\.bulk[\w.:]*multicast", text), p.name
