"""The bench reports the recorded per-launch DRAM traffic as long as the kernels' code is the code that
was captured: comments may change, code may not."""
import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_recorded_traffic_is_reported():
    recorded = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))
    for name, entry in recorded.items():
        assert bench.recorded_traffic(name) == entry["dram_bytes_per_launch"] > 0


def test_source_hash_sees_code_and_not_comments(tmp_path, monkeypatch):
    def h(text):
        (tmp_path / "k.cuh").write_text(text)
        return bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setattr(bench, "KERNEL_SOURCES", ["k.cuh"])
    base = h('int a = 1;\nasm("x // y;");\n')
    assert h('// one\nint a = 1;   /* two\nlines */\n\nasm("x // y;");  // three "q\n') == base
    for other in ('int a = 2;\nasm("x // y;");\n', 'int a = 1;\nasm("x // z;");\n', 'int a = 1;\nasm("x");\n',
                  '#define a\nint a = 1;\nasm("x // y;");\n', 'inta = 1;\nasm("x // y;");\n'):
        assert h(other) != base
