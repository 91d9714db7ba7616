"""The native binding's library calls are made without the interpreter's lock, as ctypes makes those of the other calls: one
that waits for another thread's plan does not stop every Python thread."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_attention_25_gb300", "csrc")


def test_calls_that_launch_let_go_of_the_interpreter():
    with open(os.path.join(CSRC, "binding.cpp")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    names = {"tree_mask", "tree_attn", "summarize", "select_blocks", "sparse_attn", "fork", "copy_blocks", "compact"}
    assert set(re.findall(r"run\(pkv_(\w+), p->handle", text)) == names
    assert not names & set(re.findall(r"pkv_(\w+)\(", text))
