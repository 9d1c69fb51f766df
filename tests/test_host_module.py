"""The binding with and without qmv_host.so, the C++ form of its usual calls: it holds to
one torch and Python, the library's calls do not."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

PKG = "bit_weight_only_packed_gb300"


@pytest.fixture(scope="module")
def build():
    from bit_weight_only_packed_gb300 import build
    build.build()
    return build


USE = """
import sys, warnings; sys.path.insert(0, {root!r})
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter('always')
    from bit_weight_only_packed_gb300 import qmv as q
import torch
print('warned', sum('qmv_host.so is not used' in str(x.message) for x in w))
p = q.Pack(64, 256, 2, 32)
assert q.qmv_pack_info(p) == (64, 256, 2, 32)
assert q.W4Pack(64, 256, 128).info()[:3] == (64, 256, 128)
for call in (lambda: q.qmv_softmax(torch.zeros(2, 8)),
             lambda: q.qmv_block_norm(*[torch.zeros(2, 8, dtype=torch.float16)] * 2, torch.zeros(8, dtype=torch.float16)),
             lambda: q.qmv_verify_draft(torch.zeros(1, 2, 8), None, torch.zeros(1, 1, dtype=torch.int32),
                                        torch.zeros(1, 1), torch.zeros(1)),
             lambda: q.qmv_w4_gemv(q.W4Pack(64, 256, 128), torch.zeros(1, 256, dtype=torch.float16))):
    try:
        call()
        raise SystemExit('not refused')
    except ValueError:
        pass
print('usable')
"""


@pytest.mark.parametrize("what", ["as built", "missing", "for another torch", "no note", "not a module"])
def test_the_library_is_usable_whatever_the_module_is(build, tmp_path, what):
    pkg = tmp_path / PKG
    (pkg / "_lib").mkdir(parents=True)
    for n in os.listdir(os.path.join(ROOT, PKG)):
        if n.endswith(".py"):
            shutil.copy(os.path.join(ROOT, PKG, n), pkg / n)
    shutil.copy(build.LIB, pkg / "_lib" / "libqmv.so")
    host, note = pkg / "_lib" / "qmv_host.so", pkg / "_lib" / "qmv_host.so.for"
    if what != "missing":
        shutil.copy(build.HOST_LIB, host)
        note.write_text(build.host_abi())
    if what == "for another torch":
        note.write_text("torch 1.0, cpython-312")
    if what == "no note":
        note.unlink()
    if what == "not a module":
        host.write_bytes(b"no module")
    r = subprocess.run([sys.executable, "-c", USE.format(root=str(tmp_path))], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert f"warned {int(what != 'as built')}" in r.stdout and "usable" in r.stdout


def test_it_is_built_again_for_another_torch(build, tmp_path, monkeypatch):
    lib = tmp_path / "qmv_host.so"
    monkeypatch.setattr(build, "HOST_LIB", str(lib))
    ran = []

    def compiler(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", compiler)
    build.build_host()
    build.build_host()
    assert len(ran) == 1
    monkeypatch.setattr(build, "host_abi", lambda: "torch 99")
    build.build_host()
    build.build_host()
    assert len(ran) == 2


def test_a_module_that_cannot_be_built_does_not_cost_the_library(build, tmp_path, monkeypatch):
    monkeypatch.setattr(build, "HOST_LIB", str(tmp_path / "qmv_host.so"))
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "no headers"))
    with pytest.warns(UserWarning, match="could not be built"):
        assert build.build() == build.LIB


@pytest.mark.gpu
def test_the_python_form_gives_the_same(monkeypatch):
    from bit_weight_only_packed_gb300 import qmv as q
    from test_gpu_step_edges import case, same
    assert not isinstance(q._host, q._NoHost)
    run = case()
    ref = run()
    monkeypatch.setattr(q, "_host", q._NoHost())
    assert same(run(), ref)
