"""What the compiler reports of the kernels that it built (no GPU)."""
import os

import pytest


@pytest.fixture(scope="module")
def resources(kvc):
    from entropy_coding_amd import build
    if not all(os.path.exists(build.resource_file(s)) for s in build.KERNELS):
        build.build()
    return build.resources


@pytest.mark.parametrize("src,name,least", [("kvc_attention.hip", "k_attend", 28), ("kvc_attention_wide.hip", "k_attend", 42)])
def test_attention_keeps_its_sums_in_registers(resources, src, name, least):
    """No variant of the attention kernels, for any channel count, type, page
    size or number of rows, puts registers into scratch memory."""
    kernels = {k: r for k, r in resources(src).items() if name in k}
    assert len(kernels) >= least
    spilled = {k: r["ScratchSize [bytes/lane]"] for k, r in kernels.items() if r["ScratchSize [bytes/lane]"]}
    assert not spilled
    assert all(r["Dynamic Stack"] == "False" for r in kernels.values())


def test_a_workgroup_of_attention_fits_the_cu(resources):
    """LDS of 160 KB a CU, 512 vector registers a SIMD lane."""
    for src in ("kvc_attention.hip", "kvc_attention_wide.hip"):
        for k, r in resources(src).items():
            assert r["LDS Size [bytes/block]"] <= 160 * 1024 and r["VGPRs"] + r["AGPRs"] <= 512, k
