"""Words that one CTA of a pair writes into the other one's shared memory are in place before the barrier that the other one
reads them behind: the pairs' kernels write them by dsmem_publish_u32 alone, which has the fence."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_sampling_gb300", "csrc")


def test_pairs_publish_what_they_write():
    for name in ("vsamp_block_matmul.cuh", "vsamp_tensor.cuh"):
        code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        helper = re.search(r"void dsmem_publish_u32\([^{]*\{(.*?)\n\}", code, re.S)
        if helper:
            assert re.search(r"dsmem_store_u32\(addr, v\);\s*fence_cluster\(\);", helper.group(1))
            assert re.search(r'void fence_cluster\(\) \{ asm volatile\("fence\.acq_rel\.cluster;"', code)
            code = code.replace(helper.group(0), "")
        assert not re.findall(r"dsmem_store\w*\(|st\.shared::cluster|st\.async", code), name


def test_arrivals_on_the_other_cta_are_followed_by_a_fence():
    """The warps that arrive on the other CTA's barriers wait for these arrivals at their end."""
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "vsamp_block_matmul.cuh")).read())
    kernel = code[code.index("block_matmul_kernel("):]
    last = kernel.rindex("mbar_arrive_pair(")
    assert last < kernel.index("fence_cluster();") < kernel.index("bool gave_up")
