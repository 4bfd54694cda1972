"""The dense workloads' DRAM-traffic record goes stale with the sources of what they run, not with those of the 4-bit cache."""

import bench


def test_the_4_bit_cache_s_files_leave_the_hash(tmp_path, monkeypatch):
    csrc = tmp_path / "exact_io_aware_84_b200" / "csrc"
    csrc.mkdir(parents=True)
    (csrc / "fa_fwd_sm100.cu").write_text("__global__ void k() {}\n")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    h = bench.kernel_sources_hash()
    for name in ("fa_kv4.cu", "fa_kv4.cuh", "fa_kv4_attn.cu"):
        (csrc / name).write_text("__global__ void other() {}\n")
        assert bench.kernel_sources_hash() == h
    (csrc / "fa_kernels.h").write_text("constexpr int kBlockM = 64;\n")
    assert bench.kernel_sources_hash() != h
