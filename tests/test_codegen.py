"""Properties of the gfx950 code the build emits (device assembly of each
kernel source, compiled with the build's own flags): no packed-fp32 vector
arithmetic (the flags switch its selection off, and every fp32 operation
must round on its own), and no writes through the scalar data cache (all
stores are vector stores).  Runs on the host; needs hipcc."""

import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

from momentum_compression_amd import build as B

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists(
    "/opt/rocm/bin/hipcc"), reason="hipcc not available")

KERNEL_SOURCES = [s for s in B.SOURCES if s != "api.hip"] + [B.PROBE_SRC]
PACKED_FP32 = re.compile(r"^\s+v_pk_(add|mul|fma)_f32\b", re.M)
SCALAR_WRITE = re.compile(r"^\s+s_(store|buffer_store|scratch_store|atomic|buffer_atomic|dcache_wb)", re.M)
KERNEL = re.compile(r"^\s+\.amdhsa_kernel\s+(\S+)", re.M)


@pytest.fixture(scope="module")
def device_asm(tmp_path_factory):
    out = tmp_path_factory.mktemp("asm")

    def one(src):
        dst = out / (src + ".s")
        cmd = [B.hipcc(), *B.FLAGS, "--cuda-device-only", "-S",
               os.path.join(B.CSRC, src), "-o", str(dst)]
        subprocess.run(cmd, check=True, capture_output=True)
        return src, dst.read_text()

    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        return dict(ex.map(one, KERNEL_SOURCES))


def test_every_source_emits_kernels(device_asm):
    for src, text in device_asm.items():
        assert KERNEL.search(text), f"{src}: no kernel in the device assembly"


def test_no_packed_fp32_arithmetic(device_asm):
    for src, text in device_asm.items():
        m = PACKED_FP32.search(text)
        assert m is None, f"{src}: {m.group(0).strip()}"


def test_no_scalar_cache_writes(device_asm):
    for src, text in device_asm.items():
        m = SCALAR_WRITE.search(text)
        assert m is None, f"{src}: {m.group(0).strip()}"


LABEL = re.compile(r"^([.\w$]+):")
BRANCH = re.compile(r"^\s+s_(c?)branch\w*\s+([.\w$]+)")
TILE_LOAD = re.compile(r"^\s+buffer_load_\w+\s.*\blds\b")
DRAIN = re.compile(r"^\s+s_waitcnt\b.*\bvmcnt\(0\)")


def open_barriers(text):
    """(barriers, those that some path reaches with a load into LDS of its own
    wave on its way): other waves read past such a barrier what that load has
    not brought yet."""
    lines = [ln.split(";")[0].rstrip() for ln in text.splitlines()]
    at = {m.group(1): n for n, ln in enumerate(lines) if (m := LABEL.match(ln))}
    barriers = sum(bool(re.match(r"^\s+s_barrier\b", ln)) for ln in lines)
    seen, bad = set(), set()
    todo = [n + 1 for n, ln in enumerate(lines) if TILE_LOAD.match(ln)]
    while todo:  # lines reached with a load under way
        n = todo.pop()
        while n < len(lines) and n not in seen:
            seen.add(n)
            ln = lines[n]
            if DRAIN.match(ln) or re.match(r"^\s+s_endpgm", ln):
                break
            if re.match(r"^\s+s_barrier\b", ln):
                bad.add(n + 1)
            if m := BRANCH.match(ln):
                todo.append(at[m.group(2)])
                if not m.group(1):
                    break
            n += 1
    return barriers, sorted(bad)


def test_open_barriers_are_found():
    """The search itself, on a loop whose short cut passes the wait."""
    loop = """
k:
	buffer_load_dwordx4 v1, s[0:3], 0 offen lds
.LBB0_1:
	s_waitcnt vmcnt(0) lgkmcnt(0)
	s_barrier
	buffer_load_dwordx4 v1, s[0:3], 0 offen lds
	s_cbranch_vccnz {}
	s_waitcnt vmcnt(0)
.LBB0_2:
	s_barrier
	s_cbranch_scc1 .LBB0_1
	s_endpgm
"""
    assert open_barriers(loop.format(".LBB0_1")) == (2, [])
    assert open_barriers(loop.format(".LBB0_2")) == (2, [11])


@pytest.mark.parametrize("src", ["attn_fwd.hip", "attn_bwd.hip"])
def test_barriers_wait_for_tile_loads(device_asm, src):
    """A barrier orders the LDS accesses of the waves that meet at it, not the
    loads into LDS that they have issued: each wave has to have waited for its
    own on every path."""
    text = device_asm[src]
    assert any(TILE_LOAD.match(ln) for ln in text.splitlines())
    barriers, bad = open_barriers(text)
    assert barriers > 0 and not bad, f"{src}: {len(bad)} of {barriers} barriers, lines {bad[:8]}"
