"""Dynamic shared memory of the kernels, read from their sources: an array that is used as
another type must be declared with that type's alignment, since static shared memory may
end anywhere in front of it."""
import glob
import os
import re

from llama2_decoder_forward_gb300 import build

SIZE = {"char": 1, "uint8_t": 1, "bf16": 2, "int": 4, "int32_t": 4, "uint32_t": 4, "unsigned": 4, "float": 4, "int2": 8,
        "uint2": 8, "float2": 8, "uint64_t": 8, "double": 8, "int4": 16, "uint4": 16, "float4": 16}


def test_dynamic_shared_memory_is_aligned_for_its_uses():
    declared = 0
    for fn in sorted(glob.glob(os.path.join(build.CSRC, "*.cu")) + glob.glob(os.path.join(build.CSRC, "*.cuh"))):
        src = re.sub(r"//[^\n]*", "", open(fn).read())
        for m in re.finditer(r"extern __shared__ (?:__align__\((\d+)\) )?(\w+) (\w+)\[\];", src):
            declared += 1
            align = int(m[1]) if m[1] else SIZE.get(m[2], 4)
            body = src[m.end():]  # up to the next kernel
            body = body[:body.find("__global__")] if "__global__" in body else body
            for t in re.findall(r"reinterpret_cast<(?:volatile |const )*(\w+) ?\*>\(\s*%s\b" % m[3], body):
                assert SIZE[t] <= align, "%s: %s of %s used as %s" % (os.path.basename(fn), m[3], m[2], t)
    assert declared >= 12
