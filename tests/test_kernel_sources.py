"""Rules of the kernel sources that no run on a GPU can show to be broken."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_38_b200", "csrc")


def _kernels():
    """(file, name, body) of every kernel."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^\n]*?\)\s+)?(\w+)\s*\(", text):
            start = at = text.index("{", m.end())
            depth = 0
            while True:
                depth += (text[at] == "{") - (text[at] == "}")
                at += 1
                if depth == 0:
                    break
            yield name, m.group(1), text[start:at]


def test_kernels_that_overlap_the_one_before_read_its_results_coherently():
    """A kernel that waits for the one before it (griddepcontrol.wait) runs while that one writes the workspace: __ldg
    is for data that nothing writes during the kernel, so it may not name the workspace."""
    seen = {}
    for file, name, body in _kernels():
        if "wait_previous()" in body:
            seen[name] = [c for c in re.findall(r"__ldg\(([^;]*);", body) if re.search(r"\bpartial\b|\bwork\.", c)]
    assert {"conv1d_window_kernel", "conv1d_reduce_kernel", "norm_reduce_kernel", "ssd_varlen_kernel",
            "ssd_varlen_combine_kernel"} <= set(seen), sorted(seen)
    assert not any(seen.values()), seen
