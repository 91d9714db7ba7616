"""Kernels of the calls that read their metadata on the device may be scheduled before the kernel ahead of them ends.
Arrays that a kernel ahead may write while it has let them start are not read through the non-coherent path (__ldg)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_attention_25_gb300", "csrc")

# Tables, lengths, positions and ids: no kernel that releases the next one early writes them.
READ_ONLY = {
    "tree.cu": {"bt_row", "a.cu_q_lens", "a.positions", "cu", "parents"},
    "tree_tc.cu": {"bt", "bt_row"},
    "sched.cuh": {"cu", "a.cu_q_lens", "a.ctx_lens", "a.prefix_lens"},
    "rows.cuh": set(),
    "sparse.cu": {"cu", "a.cu_q_lens", "a.positions", "a.ctx_lens", "a.block_tables", "bt_row"},
    "pages.cu": {"a.lens", "a.caps", "a.parents", "a.new_caps", "a.tables", "old", "src", "dst", "cu", "row"},
}


def test_only_metadata_is_read_through_the_non_coherent_path():
    for name, allowed in READ_ONLY.items():
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        if name == "sparse.cu":     # summarize_kernel reads keys (row): it is launched behind the end of the kernel ahead
            text = re.sub(r"__ldg\(reinterpret_cast<const uint(32_t|16_t|2)\*>\(row\)\)", "", text)
            assert "summarize_kernel<D, F8, 1><<<" in text and "launch_dependent(summarize_kernel" not in text
        code = re.sub(r"//[^\n]*", "", text)
        read = {m.group(1) for m in re.finditer(r"__ldg\(\s*([A-Za-z_.]+|reinterpret_cast)", code)}
        assert read <= allowed, (name, read - allowed)
