"""Which sources the recorded profiles' digests stand for (CPU only)."""
import importlib.util
import os
import shutil

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_digest_changes_with_every_source_its_kernels_are_compiled_from(tmp_path):
    package = tmp_path / "package"
    for folder in ("csrc", "layers", "blocks"):
        shutil.copytree(os.path.join(ROOT, "precision_gemm_02_amd", folder), package / folder)
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    shutil.copy(os.path.join(ROOT, "precision_gemm_02_amd", "build.py"), package)
    spec = importlib.util.spec_from_file_location("build_copy", package / "build.py")
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)

    def digests():
        return [build.source_digest(), build.layer_digest(), build.block_digest()]

    before = digests()
    assert len(set(before)) == 3 and digests() == before
    for path, changed in ((package / "csrc" / "gemm_tile.hpp", (True, False, False)),
                          (tmp_path / "include" / "pgemm.h", (True, False, False)),
                          (package / "blocks" / "norm.hpp", (False, False, True)),
                          (tmp_path / "include" / "pgemm_blocks.h", (False, False, True)),
                          (package / "layers" / "prod.hpp", (False, True, True)),
                          (package / "layers" / "plan.hpp", (False, True, True)),
                          (tmp_path / "include" / "pgemm_layers.h", (False, True, True))):
        path.write_text(path.read_text() + "\n")
        now = digests()
        assert tuple(a != b for a, b in zip(now, before)) == changed, path
        before = now
