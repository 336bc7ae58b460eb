"""Which sources the bounds-checked library compiles anew: those with a check in themselves or in a header that they include."""
import os
import re

import __graft_entry__


def test_sources_with_checks():
    b = __graft_entry__._build_module()
    checked = {os.path.basename(s) for s in b.sources() if b._has_checks(s)}
    for s in b.sources():
        if re.search("MT_CHECK", open(s).read()):
            assert os.path.basename(s) in checked
    assert {"mt_rows.cu", "mt_scan1d_ext.cu", "mt_select.cu", "mt_abi.cu"} <= checked  # the first two by headers of headers
    assert not any(n.startswith(("mt_gated", "mt_beam", "mt_copy", "mt_ssm", "mt_conv", "mt_embed", "mt_seq")) for n in checked)


def test_the_definitions_make_no_check():
    """mt_tile.cuh, which every kernel includes, names the checks only where it defines them."""
    b = __graft_entry__._build_module()
    text = open(os.path.join(b.CSRC, "mt_tile.cuh")).read()
    code = "\n".join(line.split("//")[0] for line in text.splitlines())
    assert not [line for line in code.splitlines() if "MT_CHECK" in line and not re.match(r"\s*#\s*(if|ifndef|define)", line)]
