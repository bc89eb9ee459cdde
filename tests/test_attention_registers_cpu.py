"""The attention kernels of 16 warps divide the registers that their block is
launched with among the warps' roles: 128 a thread, all that 512 threads can
have.  With fewer a call is refused on the GPU; the compiler's report shows it here."""
import os
import re

from gated_delta_rule_gateddeltanet_gb300 import build


def test_attention_kernels_have_the_registers_that_their_roles_divide():
    build.build()
    log = open(os.path.join(build.BUILD, "ptxas.log")).read()
    used = re.findall(r"entry function '(\w*paged_attention_kernel\w*)'.*?Used (\d+) registers", log, re.S)
    assert len(used) >= 40
    # (those of 8 warps, whose roles share alike, hold outputs of more than 64 registers and use more)
    assert {name: int(n) for name, n in used if int(n) < 128} == {}
    assert sum(int(n) == 128 for _, n in used) >= 30
