"""What the sources of the attention with modified scores keep to."""
import os
import re

from paged_kv_attention_25_gb300 import pkv

CSRC = os.path.join(os.path.dirname(pkv.__file__), "csrc")


def test_only_metadata_is_read_through_the_non_coherent_path():
    """The plan, exponents, rows and partial results may be what the kernel ahead wrote after it let this one start."""
    allowed = {
        "score.cuh": {"a.first_keys", "a.t.positions", "a.t.cu_q_lens", "a.t.ctx_lens", "a.t.prefix_lens"},
        "score.cu": {"bt_row", "t.positions"},
        "score_tc.cuh": {"a.t.positions", "a.first_keys", "a.positions", "sa.first_keys", "bt", "bt_row"},
    }
    for name, names in allowed.items():
        with open(os.path.join(CSRC, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        read = {m.group(1) for m in re.finditer(r"__ldg\(\s*&?([A-Za-z_.]+)", code)}
        assert read <= names, (name, read - names)


def test_register_splits_fit_the_launch():
    """setmaxnreg.inc waits for registers that others of the CTA gave back: the shares never exceed the launch's."""
    with open(os.path.join(CSRC, "score_tc.cuh")) as f:
        text = f.read()
    widen, codes, soft = (int(re.search(rf"{n} = (\d+)", text).group(1)) for n in ("kRegsWiden", "kRegsCodes", "kRegsSoft"))
    assert 128 * (2 * soft + widen + codes) <= 512 * 128 and max(widen, codes) <= 128 <= soft
    down, up = (int(x) for x in (re.search(r"else asm volatile\(\"setmaxnreg.dec.sync.aligned.u32 (\d+);", text).group(1),
                                 re.search(r"else asm volatile\(\"setmaxnreg.inc.sync.aligned.u32 (\d+);", text).group(1)))
    assert 128 * (2 * up + down) <= 384 * 168 and down <= 168 <= up
