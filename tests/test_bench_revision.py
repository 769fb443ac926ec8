"""The revision that the benchmark compares its traffic record with: of the path's own sources, no others."""
import os
import shutil

import bench


def test_kernel_revision_covers_the_benchmark_path_alone(tmp_path):
    src = os.path.join(bench.ROOT, "sparse_attention_decode_csa2_gb300", "csrc")
    d = tmp_path / "csrc"
    shutil.copytree(src, d)
    rev = bench.kernel_revision(str(d))
    assert rev == bench.kernel_revision()
    beside = [n for n in os.listdir(d) if n.startswith("kv8")]
    for n in beside:  # nothing of the path includes them
        with open(d / n, "a") as f:
            f.write("// changed\n")
    assert beside and bench.kernel_revision(str(d)) == rev
    for n in set(os.listdir(d)) - set(beside):
        with open(d / n) as f:
            assert '#include "kv8' not in f.read()
        with open(d / n, "a") as f:
            f.write("// changed\n")
        now = bench.kernel_revision(str(d))
        assert now != rev
        rev = now
