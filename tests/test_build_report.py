"""The build's reading of the compiler's resource report: kernels with accumulation registers must not spill vector registers."""
import pytest

from fourier_domain_linear_amd import build


def _kernel(name, vgprs, agprs, sgpr_spill, vgpr_spill):
    at = "a.hip:41:1: remark: "
    return "\n".join(at + t + f" [{build.REPORT}]" for t in (
        f"Function Name: {name}", "    TotalSGPRs: 60", f"    VGPRs: {vgprs}", f"    AGPRs: {agprs}", "    ScratchSize [bytes/lane]: 0",
        "    Occupancy [waves/SIMD]: 1", f"    SGPRs Spill: {sgpr_spill}", f"    VGPRs Spill: {vgpr_spill}", "    LDS Size [bytes/block]: 0"))


def test_which_kernels_spill():
    fine = [_kernel("plain", 128, 0, 0, 0), _kernel("scalars", 256, 127, 8, 0), _kernel("no_accumulators", 256, 0, 0, 7)]
    assert build.spilling_kernels("\n".join(fine)) == []
    said = build.spilling_kernels("\n".join([fine[1], _kernel("bad", 256, 127, 0, 3), fine[2], _kernel("worse", 256, 1, 2, 40)]))
    assert [s.split()[0] for s in said] == ["bad", "worse"]


@pytest.mark.parametrize("src", build.NO_SPILLS)
def test_the_attention_sources_are_looked_over(src):
    assert src in build.SOURCES


def test_a_spilling_kernel_ends_the_build(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BUILD", str(tmp_path))

    class Done:
        returncode, stdout = 0, ""
        stderr = _kernel("bad", 256, 127, 0, 3)

    def run(cmd, **kw):
        assert build.REPORT in cmd
        (tmp_path / "attn_bwd.o").write_bytes(b"")
        return Done

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="bad"):
        build._compile("attn_bwd.hip")
    assert not (tmp_path / "attn_bwd.o").exists()
    Done.stderr = ""
    with pytest.raises(RuntimeError, match="no resource report"):
        build._compile("attn_bwd.hip")
    Done.stderr = _kernel("fine", 256, 127, 3, 0)
    assert build._compile("attn_bwd.hip") == str(tmp_path / "attn_bwd.o")
