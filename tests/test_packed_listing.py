"""The compiler's listing of the prompt kernels over a 4-bit cache, which load to
LDS with inline assembly as the 16-bit ones do, held to the same checks."""
import concurrent.futures
import os
import subprocess

import pytest

from test_activation_aware_amd import build
from test_attention_listing import unwaited_reads, wait_state_faults

PROMPTS = ["packed_prompts_d%d" % d for d in (64, 128, 256)]


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    folder = tmp_path_factory.mktemp("listing")

    def one(unit):
        out = folder / (unit + ".s")
        cmd = [build.hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-I", os.path.join(build.ROOT, "include"),
               "-o", str(out), os.path.join(build.CSRC, unit + ".hip")]
        done = subprocess.run(cmd, capture_output=True, text=True)
        assert done.returncode == 0, done.stderr
        return out.read_text()

    with concurrent.futures.ThreadPoolExecutor(min(6, os.cpu_count() or 1)) as ex:
        return dict(zip(PROMPTS, ex.map(one, PROMPTS)))


@pytest.mark.parametrize("unit", PROMPTS)
def test_loads_to_lds_wait_for_their_resource(listings, unit):
    loads, bad = wait_state_faults(listings[unit])
    assert loads > 0
    assert not bad, (len(bad), bad[:5])


@pytest.mark.parametrize("unit", PROMPTS)
def test_a_stage_is_loaded_after_its_reads(listings, unit):
    places, bad = unwaited_reads(listings[unit])
    assert places > 0
    assert not bad, (len(bad), places, bad[:8])
