"""The compiled kernels behind the layer hold no select that reads an addition's carry.

hipcc has turned `buffer range = row < T ? bytes : 0` into the two halves of a 64-bit address addition followed at once by
s_cselect, which then chooses by the carry and not by the comparison: a load past the end of a tensor. What the source says
cannot show it, so the listing is searched: an s_cselect_b32 or a branch whose condition the last scalar instruction to write one was s_addc or
s_subb. (A carry that is kept, for a division in 64 bits, is s_add and s_cselect_b64 with -1.)"""
import re
import subprocess
from pathlib import Path

import pytest

from combine_moe_dispatch_02_amd import build

CSRC = Path(build.__file__).parent / "csrc"
WRITES = re.compile(r"\s+(s_(?:add|sub|addc|subb|min|max|and|or|xor|andn2|orn2|nand|nor|xnor|not|lshl|lshr|ashr|bfe|bcnt0|bcnt1|abs"
                    r"|absdiff|cmp|bitcmp0|bitcmp1|wqm)\w*)")
READS = re.compile(r"\s+(s_cselect_b32|s_cbranch_scc\d)\b")


def selects_by_carry(listing: str):
    kernel = last = None
    for line in listing.splitlines():
        if m := re.match(r"(_Z\w+):", line):
            kernel, last = m.group(1), None
        elif line.startswith(".L"):
            last = None
        elif READS.match(line) and last and last.startswith(("s_addc", "s_subb")):
            yield kernel, last, line.strip()
        if m := WRITES.match(line):
            last = m.group(1)


def test_the_search_finds_one():
    bad = "_Z1kv:\n\ts_cmp_lt_i32 s0, s1\n\ts_add_u32 s2, s3, s4\n\ts_addc_u32 s5, s6, s7\n\ts_cselect_b32 s8, 0, s9\n"
    assert list(selects_by_carry(bad)) == [("_Z1kv", "s_addc_u32", "s_cselect_b32 s8, 0, s9")]
    good = "_Z1kv:\n\ts_add_u32 s2, s3, s4\n\ts_addc_u32 s5, s6, s7\n\ts_cmp_lt_i32 s0, s1\n\ts_cselect_b32 s8, 0, s9\n"
    assert not list(selects_by_carry(good))


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    out = tmp_path_factory.mktemp("listing")
    runs = {n: subprocess.Popen([build.HIPCC, *build.CFLAGS, "--cuda-device-only", "-S", str(CSRC / f"{n}.hip"), "-o", str(out / f"{n}.s")],
                                stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True) for n in ("sandwich", "adapter", "norm")}
    for n, p in runs.items():
        err = p.communicate(timeout=600)[1]
        assert p.returncode == 0, (n, err[-2000:])
    return {n: (out / f"{n}.s").read_text() for n in runs}


@pytest.mark.parametrize("name", ["sandwich", "adapter", "norm"])
def test_no_select_reads_a_carry(listings, name):
    assert "s_cselect_b32" in listings[name] or "s_cbranch_scc" in listings[name]
    assert not list(selects_by_carry(listings[name]))
