"""The compiler's listing of the attention kernels: what the direct-to-LDS
loads, which are inline assembly that the compiler's own checks do not look
into, have to keep to.  Compiles the units for the GPU; runs nothing there."""
import concurrent.futures
import glob
import os
import re
import subprocess

import pytest

from test_activation_aware_amd import build

UNITS = sorted(os.path.basename(p)[:-4] for p in glob.glob(os.path.join(build.CSRC, "paged_attention_*.hip")))


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
        return dict(zip(UNITS, ex.map(one, UNITS)))


def instructions(text):
    """(mnemonic, operands) of each line; a label as ("label", name)."""
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if not line or line.startswith((".p2align", ".set", ".long", ".short")):
            continue
        if line.endswith(":"):
            yield "label", line[:-1]
        elif not line.startswith("."):
            name, _, rest = line.partition(" ")
            name, _, more = name.partition("\t")
            yield name.strip(), (more + " " + rest).strip()


def scalar_registers(operand):
    """The numbers of s5 or s[4:7]; none for anything else."""
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", operand.strip())
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def wait_state_faults(text):
    """Loads to LDS that read a scalar register less than five wait states after
    a vector instruction wrote it (a vector memory instruction does not wait for
    that by itself), or for which a jump leaves that open."""
    code, bad, loads = list(instructions(text)), [], 0
    for i, (name, args) in enumerate(code):
        if not (name.startswith("buffer_load") and args.endswith("lds")):
            continue
        loads += 1
        reads = scalar_registers(args.split(",")[1].strip())
        assert len(reads) == 4, args
        states, j = 0, i - 1
        while states < 5:
            n, a = code[j]
            if n == "label":
                bad.append((i, "a jump"))
                break
            written = a.split(",")[:2 if "_co_" in n else 1]  # a carry is the second operand
            if n.startswith("v_") and any(scalar_registers(o) & reads for o in written):
                bad.append((i, f"{n} {a}: {states} wait states"))
                break
            states += int(a, 0) + 1 if n == "s_nop" else 1
            j -= 1
    return loads, bad


def test_the_check_finds_a_missing_wait():
    """On a listing written here: four wait states are too few, five are enough."""
    head = "kernel:\n\tv_readfirstlane_b32 s6, v5\n\ts_and_b32 s5, s5, 0xffff\n\ts_mov_b32 s7, 0x20000\n"
    load = "\ts_mov_b32 m0, s43\n\ts_nop {}\n\tbuffer_load_dwordx4 v75, s[4:7], 0 offen lds\n"
    assert wait_state_faults(head + load.format(0)) == (1, [(6, "v_readfirstlane_b32 s6, v5: 4 wait states")])
    assert wait_state_faults(head + load.format(1)) == (1, [])
    assert wait_state_faults("\ts_nop 7\n.LBB0_1:\n" + load.format(0))[1] != []


@pytest.mark.parametrize("unit", UNITS)
def test_loads_to_lds_wait_for_their_resource(listings, unit):
    loads, bad = wait_state_faults(listings[unit])
    assert loads > 0
    assert not bad, (len(bad), bad[:5])


def unwaited_reads(text):
    """Barriers, and first loads of a stage in the key form, before which the
    straight code has no wait for the wave's own LDS reads (of the stage that is
    loaded next).  Returns (places looked at, those without a wait)."""
    code, kernel, places, bad = list(instructions(text)), "", 0, []
    for i, (name, args) in enumerate(code):
        if name == "label" and args.startswith("_Z"):
            kernel = args
        first_load = "attn_keys_kernel" in kernel and name.startswith("buffer_load") and args.endswith("lds") and not any(
            n.startswith("buffer_load") for n, _ in code[max(0, i - 12):i])
        if name != "s_barrier" and not first_load:
            continue
        places += 1
        j = i - 1
        while not (code[j][0] == "s_waitcnt" and "lgkmcnt(0)" in code[j][1]):
            if code[j][0].startswith("ds_") or code[j][0] == "label":
                bad.append((kernel, name, code[j]))
                break
            j -= 1
    return places, bad


def test_the_check_finds_an_unwaited_read():
    head = "_Z4attn:\n\tds_read_b128 v[0:3], v5\n"
    assert unwaited_reads(head + "\ts_barrier\n")[1] != []
    assert unwaited_reads(head + "\ts_waitcnt lgkmcnt(0)\n\tv_mov_b32 v1, 0\n\ts_barrier\n") == (1, [])
    assert unwaited_reads(head + "\ts_waitcnt lgkmcnt(0)\n.LBB0_3:\n\ts_barrier\n")[1] != []


@pytest.mark.parametrize("unit", UNITS)
def test_a_stage_is_loaded_after_its_reads(listings, unit):
    places, bad = unwaited_reads(listings[unit])
    assert places > 0
    assert not bad, (len(bad), places, bad[:8])
