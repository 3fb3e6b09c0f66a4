"""The packed form of the calls next to the verify step: argument counts, ranges and types, and
that the binding packs what the header declares.  No GPU."""
import os
import re
import struct

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kd():
    from tree_speculative_decoding_kd_b200 import build
    build.build()
    from tree_speculative_decoding_kd_b200 import kd as _kd
    return _kd


def test_op_codes_are_the_headers(kd):
    src = open(os.path.join(ROOT, "include", "kd_verify.h")).read()
    codes = {n.lower(): int(v) for n, v in re.findall(r"#define KD_OP_(\w+)\s+(\d+)", src)}
    assert codes == {name[3:]: i for i, name in enumerate(kd._PACKED)}


def test_signatures_match_the_headers(kd):
    """Kinds of the parameters (pointer, int, int64, float), in order."""
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kd_verify.h")).read(), flags=re.S)
    for name in kd._PACKED:
        params = re.search(r"\bint " + name + r"\s*\(([^)]*)\)", src).group(1).split(",")
        kinds = [kd._p if "*" in p or "cudaStream_t" in p else kd._i64 if "int64_t" in p else kd._f if "float" in p else kd._i
                 for p in params]
        assert kinds == kd._SIGS[name][1], name


def test_packed_calls_refuse(kd):
    lib = kd.lib
    args = [16, 512, 128, 16, 512, 128, 16, 16, 1e-6, 16, 100, 16, 0, 4, 4, 128, 128, 0, 0, 16, 512, 128, 16, 512, 128, 0, 0]
    pack = lambda a: struct.pack("8qd18q", *a)  # noqa: E731
    assert lib.kd_call_packed(0, pack(args), 27) == 0                   # T = 0: nothing to do
    assert lib.kd_call_packed(0, pack(args), 26) == -1
    assert lib.kd_call_packed(0, None, 27) == -1
    assert lib.kd_call_packed(8, pack(args), 27) == -1 and lib.kd_call_packed(-1, pack(args), 27) == -1
    for i, v in ((12, 1 << 32), (13, (1 << 32) + 4), (15, -(1 << 40)), (8, -1.0), (8, float("nan"))):
        bad = list(args)
        bad[i] = v
        assert lib.kd_call_packed(0, pack(bad), 27) == -1, i
    with pytest.raises(kd.KdError):
        kd._call_qk_norm_rope(*[12 if i == 15 else a for i, a in enumerate(args)])
