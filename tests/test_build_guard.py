"""Sources whose kernels count vector-memory waits by hand are built under the
guard against register spills to scratch (CPU only)."""
import os

from fp8_grouped_gemm_amd import build


def test_hand_counted_waits_are_guarded():
    counted = []
    for src in build.SOURCES:
        with open(os.path.join(build.CSRC, src)) as f:
            text = f.read()
        if "MOE_WAIT_VMCNT(" in text or "wait_vmcnt(" in text:
            counted.append(src)
    # (gemm_sa.hip spills by choice)
    assert len(counted) > 1 and set(counted) - {"gemm_sa.hip"} <= set(build.NO_SCRATCH), counted


def test_a_spill_is_found_in_the_report():
    report = "".join(f"x.hip:1:0: remark: Function Name: {n} [-Rpass-analysis=kernel-resource-usage]\n"
                     f"x.hip:1:0: remark:     ScratchSize [bytes/lane]: {b} [-Rpass-analysis=kernel-resource-usage]\n"
                     for n, b in (("clean", 0), ("spills", 24)))
    assert build._scratch_users(report) == [("spills", 24)]
