"""The inline loads from memory to LDS in csrc/expert_gemm.hpp, as the compiler puts them. It keeps
the wait states that gfx950 asks for between its own instructions, and sees none of those inside
inline assembly: a scalar register that the vector unit has written (v_readfirstlane) may be read by
a memory instruction five wait states later at the earliest."""
import os
import re
import subprocess

import pytest

from combine_ep_get_03_amd import build

SOURCE = """
#include "expert_gemm.hpp"
using namespace ep;
__global__ void loads(const uint64_t* base, const uint32_t* word, float* out) {
    __shared__ float lds[512];
    const int l = threadIdx.x;
    // everything that the load reads in scalar registers comes out of a vector register
    const i32x4 buf = scalar_buffer(reinterpret_cast<const void*>(base[l]), word[l]);
    %s(buf, word[64 + l], word[128 + l], word[192 + l]);
    wait_loads<0>();
    lds_barrier();
    out[l] = lds[l];
}
"""
WAIT_STATES = 5


def assembly(tmp_path, source):
    src = tmp_path / "loads.hip"
    src.write_text(source)
    out = tmp_path / "loads.s"
    subprocess.run([build.HIPCC, *build.CFLAGS, "-w", "--cuda-device-only", "-S", str(src), "-o",
                    str(out)], check=True, capture_output=True)
    return out.read_text()


def scalars(text):
    regs = {int(r) for r in re.findall(r"\bs(\d+)\b", text)}
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        regs |= set(range(int(a), int(b) + 1))
    return regs


def waits(text):
    """Of every load to LDS: the wait states since the vector unit wrote a scalar that it reads."""
    written, now, found = {}, 0, []
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        op, _, args = line.partition(" ")
        if op.startswith("buffer_load") and args.endswith("lds"):
            found.append(min((now - written[r] for r in scalars(args) if r in written),
                             default=WAIT_STATES))
        target = args.split(",")[0]
        for r in scalars(target):
            written.pop(r, None)  # the scalar unit's own writes are waited for
            if op.startswith("v_"):
                written[r] = now + 1
        now += int(args, 0) + 1 if op == "s_nop" else 1
    return found


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="needs hipcc")
@pytest.mark.parametrize("load", ["load_lds16", "load_lds4"])
def test_inline_loads_wait_for_their_scalars(tmp_path, load):
    text = assembly(tmp_path, SOURCE % load)
    found = waits(text)
    assert len(found) == 1 and "v_readfirstlane" in text
    assert found[0] >= WAIT_STATES


def test_the_count_of_wait_states():
    """Of the count itself: registers written by either unit, single and in ranges."""
    load = "buffer_load_dwordx4 v1, s[4:7], s8 offen lds"
    assert waits(f"v_readfirstlane_b32 s4, v0\n{load}") == [0]
    assert waits(f"v_readfirstlane_b32 s8, v0\ns_nop 0\n{load}") == [1]
    assert waits(f"v_readlane_b32 s7, v0, 3\ns_mov_b32 m0, s9\ns_nop 3\n{load}") == [5]
    assert waits(f"v_cmp_eq_u32_e64 s[6:7], v0, v1\ns_nop 4\n{load}") == [5]
    assert waits(f"v_readfirstlane_b32 s4, v0\ns_mov_b32 s4, 0\n{load}") == [5]
    assert waits(f"v_readfirstlane_b32 s9, v0\n{load}") == [5]
