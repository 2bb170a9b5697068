"""What the compiler reports of the speculative step's kernels (no GPU): none
puts registers into scratch memory or calls a function that is not inlined (a
helper that calls itself by mistake shows here first)."""
import pytest

from test_kernel_resources import resources  # noqa: F401  (a fixture)


@pytest.mark.parametrize("src,least", [("kvc_qkv.hip", 32), ("kvc_verify.hip", 2), ("kvc_pages.hip", 3)])
def test_no_scratch_memory(resources, src, least):  # noqa: F811
    kernels = resources(src)
    assert len(kernels) >= least
    for name, r in kernels.items():
        assert r["ScratchSize [bytes/lane]"] == 0 and r["Dynamic Stack"] == "False", name
        assert r["LDS Size [bytes/block]"] <= 64 * 1024, name
