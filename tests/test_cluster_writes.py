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
            assert re.search(r'dsmem_store_u32\(addr, v\);\s*asm volatile\("fence\.acq_rel\.cluster;"', helper.group(1))
            code = code.replace(helper.group(0), "")
        assert not re.findall(r"dsmem_store\w*\(|st\.shared::cluster|st\.async", code), name
