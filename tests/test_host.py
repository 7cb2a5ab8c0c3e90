"""Host-side logic that needs no GPU: the seeded input generators, the bench's traffic
lookup and its reference arm (the oracle timed on host cores)."""
import importlib.util
import json
import os
import subprocess
import sys

import pytest
import torch

from gated_delta_rule_155_b200 import inputs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bench_module():
    spec = importlib.util.spec_from_file_location("bench_under_test", os.path.join(ROOT, "bench.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_packed_lengths_follow_their_law():
    lens = inputs.packed_lengths(32768, 4096, 5)
    assert sum(lens) == 32768 and all(1 <= n <= 4096 for n in lens)
    assert lens == inputs.packed_lengths(32768, 4096, 5)          # seeded
    assert lens != inputs.packed_lengths(32768, 4096, 6)
    assert inputs.packed_lengths(10, 4096, 5) == [10]              # the last draw is trimmed


def test_varlen_inputs_layout():
    lens = [3, 0, 5]
    d = inputs.varlen_inputs(lens, 2, 64, 64, io="f32", seed=1, s0_std=0.1)
    assert d["q"].shape == (8, 2, 64) and d["v"].shape == (8, 2, 64) and d["beta"].shape == (8, 2)
    assert d["cu_seqlens"].dtype == torch.int32 and d["cu_seqlens"].tolist() == [0, 3, 3, 8]
    assert d["s0"].shape == (3, 2, 64, 64)
    assert inputs.varlen_inputs(lens, 2, 64, 64, io="f32", seed=1)["s0"] is None


def test_prefill_inputs_are_seeded_and_follow_the_laws():
    a = inputs.prefill_inputs(2, 33, 3, 64, 64, io="f32", seed=7, s0_std=0.02)
    b = inputs.prefill_inputs(2, 33, 3, 64, 64, io="f32", seed=7, s0_std=0.02)
    for n in ("q", "k", "v", "g", "beta", "s0"):
        assert torch.equal(a[n], b[n]), n
    qn = a["q"].double().norm(dim=-1)
    assert torch.allclose(qn, torch.ones_like(qn), atol=1e-6)      # unit rows
    assert bool((a["g"] <= 0).all()) and bool(((a["beta"] > 0) & (a["beta"] < 1)).all())
    c = inputs.prefill_inputs(2, 33, 3, 64, 64, io="bf16", seed=7)
    assert c["q"].dtype == torch.bfloat16
    # bf16 inputs are the fp32 draws rounded once
    assert torch.equal(c["v"], a["v"].to(torch.bfloat16))


def test_traffic_lookup_requires_the_captured_sources(monkeypatch, tmp_path):
    bench = _bench_module()
    sha = bench.kernel_source_sha()
    assert sha == bench.kernel_source_sha() and len(sha) == 16
    prof = tmp_path / "profiles"
    prof.mkdir()
    (prof / "traffic.json").write_text(json.dumps({
        "k_same": {"source_sha": sha, "dram_bytes_per_launch": 123},
        "k_old": {"source_sha": "0" * 16, "dram_bytes_per_launch": 456}}))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setattr(bench, "kernel_source_sha", lambda kernel=None: sha)
    assert bench.traffic_for("k_same") == 123
    assert bench.traffic_for("k_old") is None        # kernel changed since the capture
    assert bench.traffic_for("missing") is None


def test_each_profiled_kernel_hashes_its_own_sources():
    bench = _bench_module()
    for k, files in bench.KERNEL_SOURCES.items():
        for f in files:
            assert os.path.exists(os.path.join(ROOT, "gated_delta_rule_155_b200", "csrc", f)), (k, f)
    # the prefill and the backward are compiled from different files, so their hashes differ
    assert bench.kernel_source_sha("kda_chunk_tc") != bench.kernel_source_sha("kda_backward")
    assert bench.kernel_source_sha("kda_chunk_tc") == bench.kernel_source_sha("kda_chunk_tc_packed")


def test_reference_arm_prints_one_json_line():
    """`bench.py --impl reference` times the oracle on the host and prints the contract's line."""
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--impl", "reference", "--steps", "1",
                        "--warmup", "0"], capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [ln for ln in r.stdout.strip().splitlines() if ln.startswith("{")]
    assert len(lines) == 1
    d = json.loads(lines[0])
    assert d["impl"] == "reference" and d["unit"] == "tokens/s" and d["value"] > 0
    assert d["higher_is_better"] is True and d["dtype"] == "f64"
    assert d["cpu_baseline"]["kind"] == "oracle" and d["cpu_baseline"]["cores"] >= 1
    assert d["e2e"]["h2d_bytes_per_step"] == 0 and d["e2e"]["value"] == d["value"]


def _package_without_short_calls(path):
    """A copy of the binding beside the built library, without the extension module."""
    from gated_delta_rule_155_b200 import build

    build.build()
    pkg = path / "gated_delta_rule_155_b200"
    pkg.mkdir()
    for name in ("__init__.py", "kda.py", "build.py"):
        (pkg / name).write_bytes(open(os.path.join(build.PKG, name), "rb").read())
    os.symlink(build.LIB, pkg / "libkda.so")
    return path


def test_the_binding_loads_without_the_short_calls(tmp_path):
    """The library and every entry point are there; what is missing is named in a warning."""
    code = ("import warnings, torch\n"
            "with warnings.catch_warnings(record=True) as w:\n"
            "    warnings.simplefilter('always')\n"
            "    from gated_delta_rule_155_b200 import kda\n"
            "assert any('_calls' in str(x.message) for x in w), [str(x.message) for x in w]\n"
            "assert all(hasattr(kda.library(), n) for n in kda.EXPORTED_SYMBOLS)\n"
            "q, g, s = torch.zeros(1, 2, 64), torch.zeros(1, 2), torch.zeros(1, 2, 64, 64)\n"
            "for f, a in ((kda.kda_gdr_decode, (q, q, q, g, g, s)), (kda.kda_gdr_forward, (q, q, q, g, g, g[0].int())),\n"
            "             (kda.kda_pages_free, (g[0].int(), g[0].int()))):\n"
            "    try:\n"
            "        f(*a)\n"
            "    except (ValueError, RuntimeError):\n"
            "        continue\n"
            "    raise SystemExit('host tensors were taken')\n")
    subprocess.run([sys.executable, "-c", code], cwd=_package_without_short_calls(tmp_path), check=True)


def test_the_library_is_built_without_a_host_compiler(monkeypatch, tmp_path):
    from gated_delta_rule_155_b200 import build

    build.build()
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="_calls"):
        assert build.build() == build.LIB
    old = build.calls_path()                                       # one of older sources is not left to be loaded
    open(old, "w").close()
    os.utime(old, (0, 0))
    with pytest.warns(RuntimeWarning, match="_calls"):
        assert build.build() == build.LIB
    assert not os.path.exists(old)


def test_short_calls_built_for_another_torch_are_not_loaded(monkeypatch, tmp_path):
    """Neither current nor loaded, however new the file is: it reads tensors as the other torch lays them out."""
    from gated_delta_rule_155_b200 import build

    here = build.build_calls()
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    assert build.build_calls() == here                             # nothing to do
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(OSError):
        build.build_calls()                                        # to be built again
    monkeypatch.undo()
    root = _package_without_short_calls(tmp_path)
    for name in ("_calls.so", os.path.basename(here).replace(torch.__version__, "0.0.1")):
        (root / "gated_delta_rule_155_b200" / name).write_bytes(open(here, "rb").read())
    code = ("import warnings\nwarnings.simplefilter('ignore')\nfrom gated_delta_rule_155_b200 import kda\n"
            "assert isinstance(kda._calls, kda._NoCalls)\n")
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True)
