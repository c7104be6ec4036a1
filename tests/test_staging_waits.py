"""Requests straight into LDS (fp32 B and C rows of full blocks) are waited for
before the barrier behind which other waves read them: in the code that the
compiler made of the scan kernels, every barrier that is followed by such
requests (one phase asks for the next one's tile) has a wait for all vector
memory in front of it, since the requests before it may not have landed.
Without a GPU; reads the gfx950 code of the object file that build() leaves.
"""
import os
import re
import subprocess

import pytest

import selective_state_space_30_amd as ssm
from selective_state_space_30_amd import _build

OBJECT = os.path.join(_build.BUILD_DIR, "ssm_kernels.o")
LLVM = os.path.join(_build.ROCM, "llvm", "bin")


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    if not os.path.exists(OBJECT) or os.path.getmtime(OBJECT) > os.path.getmtime(ssm.LIB_PATH):
        pytest.skip("no object file of the built library")
    d = str(tmp_path_factory.mktemp("code"))
    bundle, code = os.path.join(d, "bundle"), os.path.join(d, "code")
    run = lambda *a: subprocess.run(a, check=True, stdout=subprocess.PIPE, text=True).stdout  # noqa: E731
    run(os.path.join(LLVM, "llvm-objcopy"), "--dump-section", ".hip_fatbin=" + bundle, OBJECT,
        os.path.join(d, "rest.o"))
    run(os.path.join(LLVM, "clang-offload-bundler"), "--unbundle", "--type=o", "--input=" + bundle,
        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", "--output=" + code)
    return run(os.path.join(LLVM, "llvm-objdump"), "-d", "--no-show-raw-insn", code)


def test_requests_into_lds_are_waited_for(listing):
    found, bad = 0, []
    for name, body in re.findall(r"^[0-9a-f]+ <(\S*scan_kernel\S*)>:\n(.*?)(?=^[0-9a-f]+ <|\Z)",
                                 listing, flags=re.S | re.M):
        lines = [l.split("//")[0].strip() for l in body.splitlines() if l.startswith("\t")]
        for i, l in enumerate(lines):
            if l != "s_barrier":
                continue
            ahead = []
            for m in lines[i + 1:i + 80]:
                if m == "s_barrier":
                    break
                ahead.append(m)
            if not any(m.startswith("buffer_load") and m.endswith(" lds") for m in ahead):
                continue
            found += 1
            if not any(re.search(r"s_waitcnt.*vmcnt\(0\)", m) for m in lines[max(0, i - 6):i]):
                bad.append(name)
    assert found > 50, "the kernels' barriers were not found"
    assert not bad, "%d barriers of %s" % (len(bad), sorted(set(bad)))
